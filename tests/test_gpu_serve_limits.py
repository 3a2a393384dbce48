"""Serving calls at the ends of their documented ranges."""
import ctypes
import struct

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import exact_byte_level_amd as tt  # noqa: E402
from tests import serve_oracle as so  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


@pytest.mark.parametrize("rows", [3, 64, 70])
def test_strings_up_to_the_end_of_their_range(rows):
    """2^31 - 1 bytes of strings; tokens that begin in the last 16 bytes, where no whole load of 16 fits any more."""
    size = 2**31 - 1
    strings = torch.zeros(size, dtype=torch.uint8, device="cuda")
    tail = np.frombuffer(b"abcabaacbbcaabcabcaabbccabcabcbacbacbacbaaaabcab", np.uint8).copy()
    strings[-len(tail):] = dev(tail)
    cuts = np.array([0, 2, 3, 20, 32, 33, 34, 36, 39, 44, 47, 48])
    words = [bytes(tail[a:b]) for a, b in zip(cuts, cuts[1:])]
    offsets = dev((size - len(tail) + cuts).astype(np.int32))
    rng = np.random.default_rng(rows)
    nxt = np.full((70, 256), -1)
    nxt[:, 97:100] = rng.integers(0, 70, (70, 3))
    nxt[:, 97:100][rng.random((70, 3)) < 0.1] = -1
    g = tt.Grammar(nxt, accept=np.zeros(70))
    fields = g._fields + struct.pack("=4q", strings.data_ptr(), size, offsets.data_ptr(), len(words))
    q = rng.integers(0, 70, rows).astype(np.int32)
    states, bits = dev(q), torch.zeros((rows, 1), dtype=torch.int32, device="cuda")
    call = ctypes.CDLL(tt.LIB_PATH).tt_grammar_bits
    call.argtypes = [ctypes.c_char_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                     ctypes.c_void_p]
    assert call(fields, states.data_ptr(), rows, bits.data_ptr(), 1, len(words), torch.cuda.current_stream().cuda_stream) == tt.TT_OK
    torch.cuda.synchronize()
    assert np.array_equal(bits.cpu().numpy(), so.grammar_bits(nxt, np.zeros(70), -1, words, q, len(words)))
