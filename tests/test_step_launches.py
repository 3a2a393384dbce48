"""Launch shapes of the operators around the model at the ends of their documented ranges, and how their calls are cut up (no GPU needed): the
calls run against a stand-in for the runtime's launch, which writes down what it is asked for and starts nothing."""
import json
import os
import struct
import subprocess
import sys

import pytest

import exact_byte_level_amd as tt
from tests.test_serve_launches import STAND_IN

# Reads a JSON list of calls, [name, arguments as hex of a struct]; prints [return code, launches] of each.
CALLS = r"""
import ctypes, json, sys
stand_in = ctypes.CDLL(sys.argv[1], ctypes.RTLD_GLOBAL)  # found before the runtime's own
lib = ctypes.CDLL(sys.argv[2])
count = ctypes.c_int64.in_dll(stand_in, "launches")
shapes = ((ctypes.c_uint64 * 7) * 65536).in_dll(stand_in, "shapes")
out = []
for name, args in json.load(sys.stdin):
    count.value = 0
    code = getattr(lib, name)(bytes.fromhex(args), None)
    out.append([code, [list(s) for s in shapes[:count.value]]])
print(json.dumps(out))
"""

P = 1 << 20  # an address that nothing reads
ROOM = 1 << 50


def pack(*values):
    return struct.pack("=" + "".join("d" if isinstance(v, float) else "q" for v in values), *values).hex()


def cache(blocks=100, size=16, heads=8, dim=128, kind=2):
    return [P, size * heads * dim, heads * dim, dim, P, size * heads * dim, heads * dim, dim, 0, 0, blocks, size, heads, dim, kind]


def write(tokens, heads=8, dim=128, kind=2, src=2):
    return ["tt_write_cache", pack(P, heads * dim, dim, P, heads * dim, dim, P, tokens, src, *cache(heads=heads, dim=dim, kind=kind))]


def attend(queries, heads, kv, dim=128, kind=2, rows=False, table_rows=None, size=16):
    return ["tt_attend_cache", pack(P, heads * dim, dim, P, heads * dim, dim, 0, 0, queries, heads, 2, *cache(heads=kv, dim=dim, kind=kind, size=size), P, 8,
                                    queries if table_rows is None else table_rows, 8, P, P if rows else 0, 1.0, 0.0, 0, P, ROOM)]


def sample(rows, vocab, kind=0, limits=True):
    p = P if limits else 0
    return ["tt_sample_tokens", pack(P, vocab, rows, vocab, kind, P, P, p, p, p, P, 0, P, ROOM)]


CASES = [
    write(1), write(1 << 24), write((1 << 31) - 1, 1, 8), write(100_000, 4096, 256, 3, 0), write(5, 3, 24, 1, 1),
    attend(1, 1, 1), attend(1, 4096, 4096), attend(1, 4096, 1, 256), attend(512, 64, 8), attend(513, 64, 8), attend(511, 8, 1, 64), attend((1 << 31) - 1, 1, 1, 8),
    attend((1 << 19) - 1, 4096, 4096, 64), attend(1 << 19, 4095, 1, 256, 3), attend(301, 12, 12, 64, 1 + 1, True, 40), attend(512, 8, 1, 128, 3, True, 1),
    attend(512, 17, 1, 128, 2, True, 1), attend(256, 32, 8), attend(257, 32, 8), attend(513, 1, 1), attend(300, 4096, 4096, 64, 2, True, 4), attend(3, 8, 8, 8, 3, False, None, 1 << 20),
    sample(1, 1), sample(1 << 24, 1), sample(1 << 24, 2048), sample(1 << 11, 1 << 24), sample(1, 1 << 24, 2), sample(256, 262_144, 0), sample(256, 262_144, 1, False),
    sample(65_537, 512), sample(3, 524_289), sample(4096, 524_288), sample(5, 0)]


@pytest.fixture(scope="module")
def results(tmp_path_factory):
    at = tmp_path_factory.mktemp("stand_in")
    source, made = at / "launch.cpp", at / "launch.so"
    source.write_text(STAND_IN)
    subprocess.check_call(["g++", "-O1", "-shared", "-fPIC", "-o", str(made), str(source)])
    run = subprocess.run([sys.executable, "-c", CALLS, str(made), tt.LIB_PATH], input=json.dumps(CASES), stdout=subprocess.PIPE,
                         text=True, timeout=120, env=dict(os.environ), check=True)
    return json.loads(run.stdout)


@pytest.mark.parametrize("at", range(len(CASES)), ids=lambda i: "%s-%d" % (CASES[i][0], i))
def test_launches_fit(results, at):
    code, launches = results[at]
    assert code == tt.TT_OK and 1 <= len(launches) <= 50_000
    for gx, gy, gz, bx, by, bz, lds in launches:
        assert bx * by * bz <= 1024 and lds <= 160 * 1024
        for grid, block in ((gx, bx), (gy, by), (gz, bz)):
            assert grid >= 1 and grid * block < 1 << 32, (grid, block)


def groups(results, case):
    return [s[0] for s in results[CASES.index(case)][1]]


def test_how_calls_are_cut_up(results):
    """A few workgroups more than the card holds at a time where tokens are dealt out, a workgroup for each query and head of keys otherwise; the
    joining launch only in the first case."""
    assert groups(results, attend(1, 1, 1)) == [512, 4]
    assert groups(results, attend(512, 64, 8)) == [512 * 8]
    assert groups(results, attend(513, 64, 8)) == [513 * 8]
    assert groups(results, attend(511, 8, 1, 64))[0] == 768
    assert groups(results, attend(256, 32, 8)) == [512, 256 * 32 // 4] and groups(results, attend(257, 32, 8)) == [257 * 8]
    assert groups(results, attend(513, 1, 1)) == [513]
    assert groups(results, attend(301, 12, 12, 64, 2, True, 40)) == [1, 768, 301 * 12 // 4]
    assert len(groups(results, attend(512, 17, 1, 128, 2, True, 1))) == 2  # too many heads for two queries of a row in a product
    # without limits two launches, with them three, and two more where there is much to go over again
    assert len(groups(results, sample(256, 262_144, 1, False))) == 2
    assert len(groups(results, sample(1, 1))) == 3 and len(groups(results, sample(256, 262_144, 0))) == 5
