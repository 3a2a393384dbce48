"""Build libtt.so (HIP for gfx950) and _bind.so (the binding of the serving calls) in-tree.

    python -m exact_byte_level_amd.build

Steps: generate the Unicode class table from the ``regex`` module's tables
(csrc/gen_unicode_table.py -> csrc/_gen/unicode_table.inc), then compile the
kernels and the C-ABI host code with hipcc into exact_byte_level_amd/libtt.so,
then csrc/tt_bind.cpp with g++ against PyTorch's headers into
exact_byte_level_amd/_bind.so.
"""
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
GEN = os.path.join(CSRC, "_gen")
LIB = os.path.join(HERE, "libtt.so")
BIND = os.path.join(HERE, "_bind.so")
ARCH = os.environ.get("TT_OFFLOAD_ARCH", "gfx950")

HIPCC_FLAGS = [
    "-O3", "--offload-arch=" + ARCH, "-std=c++17", "-fPIC", "-shared",
    # packed-FP32 instructions off for all device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function",
]


def build(verbose=False):
    os.makedirs(GEN, exist_ok=True)
    inc = os.path.join(GEN, "unicode_table.inc")
    subprocess.check_call([sys.executable, os.path.join(CSRC, "gen_unicode_table.py"), inc])
    _compile(["hipcc"] + HIPCC_FLAGS + [
        "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-I", GEN,
        os.path.join(CSRC, "tt_kernels.hip"), os.path.join(CSRC, "tt_api.cpp"),
        os.path.join(CSRC, "tt_serve_kernels.hip"), os.path.join(CSRC, "tt_serve_api.cpp")], LIB, verbose)
    _compile(_bind_command(), BIND, verbose)
    return LIB


def _bind_command():
    import sysconfig

    import torch
    from torch.utils.cpp_extension import include_paths, library_paths
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-D__HIP_PLATFORM_AMD__",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI, "-I", os.path.join(ROOT, "include")]
    for d in include_paths() + [sysconfig.get_paths()["include"], os.path.join(rocm, "include")]:
        cmd += ["-isystem", d]
    cmd.append(os.path.join(CSRC, "tt_bind.cpp"))
    # found again by their names at run time: PyTorch has loaded them by then
    for d in library_paths() + [os.path.join(rocm, "lib")]:
        cmd += ["-L", d]
    return cmd + ["-ltorch_python", "-ltorch_cpu", "-lc10", "-lamdhip64"]


def _compile(cmd, out, verbose):
    """Run a compiler, its output put in place at once if it ends well."""
    tmp = out + ".tmp"
    cmd = cmd + ["-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    text = "\n".join(l for l in res.stdout.splitlines() if "packed-fp32-ops" not in l)
    if res.returncode != 0:
        raise RuntimeError("%s failed:\n%s" % (cmd[0], text))
    if verbose and text.strip():
        print(text)
    os.replace(tmp, out)


if __name__ == "__main__":
    print(build(verbose=True))
