"""Launch shapes of the serving calls at the ends of their documented ranges (no GPU needed): the calls run against a stand-in for
the runtime's launch, which writes down what it is asked for and starts nothing."""
import json
import os
import subprocess
import sys

import pytest

import exact_byte_level_amd as tt

STAND_IN = r"""
#include <cstddef>
#include <cstdint>
struct Dim { uint32_t x, y, z; };
extern "C" {
int64_t launches = 0;
uint64_t shapes[65536][7];
int __hipPushCallConfiguration(Dim g, Dim b, size_t lds, void*) {
  const uint64_t v[7] = {g.x, g.y, g.z, b.x, b.y, b.z, lds};
  for (int i = 0; launches < 65536 && i < 7; ++i) shapes[launches][i] = v[i];
  ++launches;
  return 0;
}
int __hipPopCallConfiguration(Dim*, Dim*, size_t*, void**) { return 0; }
int hipLaunchKernel(const void*, Dim, Dim, void**, size_t, void*) { return 0; }
int hipGetLastError() { return 0; }
}
"""

# Reads a JSON list of calls, [name, arguments] with the fields of a struct as a list; prints [return code, launches] of each.
CALLS = r"""
import ctypes, json, struct, sys
stand_in = ctypes.CDLL(sys.argv[1], ctypes.RTLD_GLOBAL)  # found before the runtime's own
lib = ctypes.CDLL(sys.argv[2])
count = ctypes.c_int64.in_dll(stand_in, "launches")
shapes = ((ctypes.c_uint64 * 7) * 65536).in_dll(stand_in, "shapes")
out = []
for name, args in json.load(sys.stdin):
    count.value = 0
    keep = [struct.pack("=%dq" % len(a), *a) if isinstance(a, list) else ctypes.c_int64(a) for a in args]
    code = getattr(lib, name)(*keep)
    out.append([code, [list(s) for s in shapes[:count.value]]])
print(json.dumps(out))
"""

P = 1 << 20  # an address that nothing reads
MOST = 1 << 24


def grammar(states, classes, tokens):
    return [P, P, P, states, classes, -1, P, 1 << 20, P, tokens]


def bits(states, classes, rows, vocab):
    return ["tt_grammar_bits", [grammar(states, classes, vocab), P, rows, P, (vocab + 31) // 32, vocab, 0]]


def plan(rows, places, offsets, in_place):
    return ["tt_plan_blocks", [[P, P if offsets else 0, rows, places, 16, P, 8, 8, P, 1 << 30, P, P, P, P, P if in_place else 2 * P,
                                P if in_place else 2 * P, P], 0]]


def shape(rows, vocab, types=(0, 0)):
    return ["tt_shape_logits", [[P, vocab, 2 * P, vocab, rows, vocab, *types, P, (vocab + 31) // 32, P, 5, 5, P, P, P, P, P, P, P, 6, P,
                                 (vocab + 31) // 32, 3, P, P], 0]]


def token_bits(n, rows, vocab, offsets=True):
    return ["tt_token_bits", [P, n, P if offsets else 0, rows, vocab, P, (vocab + 31) // 32, 0, 0]]


CASES = [
    # sets of every state of a large automaton, over vocabularies of 2^17 and 2^18 tokens
    bits(16_384, 3, 16_384, 262_144), bits(16_400, 64, 16_400, 262_144), bits(32_767, 3, 32_767, 131_073), bits(32_767, 200, 32_767, 262_144),
    bits(9_000, 64, 9_000, 262_144), bits(100, 3, MOST, 64), bits(32_767, 64, MOST, 1), bits(32_767, 256, 63, MOST), bits(32_767, 64, 64, MOST),
    token_bits(10, (1 << 22) - 1, 32), token_bits(10, 1 << 22, 32), token_bits(10, MOST, 64), token_bits(1 << 31, 60, MOST),
    token_bits((1 << 35) - 1, 1, 1000, offsets=False), token_bits((1 << 35) + 8193, 1, 1000, offsets=False), token_bits(1 << 36, 1000, 1 << 20),
    shape(MOST - 1, 1), shape(MOST, 1), shape(MOST, 2048, (2, 2)), shape(64, MOST, (1, 0)), shape(1, MOST),
    plan(MOST, (1 << 31) - 1, True, True), plan(MOST, MOST, False, False), plan(1, 1, False, True),
    ["tt_release_blocks", [P, P, MOST, 1, P, 0x7FFFFFFF, 0x7FFFFFFF, P, 1 << 30, P, P, P, P, 0]],
    ["tt_grammar_advance", [grammar(5, 5, 5), P, P, MOST, P, 0]],
]


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
    assert code == tt.TT_OK and 1 <= len(launches) <= 64
    for gx, gy, gz, bx, by, bz, lds in launches:
        assert bx * by * bz <= 1024 and lds <= 160 * 1024
        for grid, block in ((gx, bx), (gy, by), (gz, bz)):
            assert grid >= 1 and grid * block < 1 << 32, (grid, block)
