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


def random_grammar(rng, states, classes):
    cls = rng.integers(0, classes, 256)
    table = rng.integers(0, states, (states, classes))
    table[rng.random(table.shape) < 0.2] = -1
    return table[:, cls], rng.random(states) < 0.5


def random_strings(rng, n, longest):
    strings = [bytes(rng.integers(0, 256, int(rng.integers(0, longest + 1))).astype(np.uint8)) for _ in range(n)]
    return strings, np.frombuffer(b"".join(strings), np.uint8), np.concatenate([[0], np.cumsum([len(s) for s in strings])])


@pytest.mark.parametrize("states, classes, rows", [
    (8960, 3, 70), (8960, 64, 64), (8961, 3, 70), (8961, 3, 130), (8961, 64, 128), (20_000, 3, 200), (20_000, 40, 200), (32_767, 4, 300),
    (9000, 90, 127), (9000, 90, 128), (32_767, 256, 200)])
def test_grammar_bits_of_large_automata(states, classes, rows):
    """Around the number of states whose sets of classes LDS holds, with and without the automaton beside them."""
    rng = np.random.default_rng(states + classes + rows)
    nxt, accept = random_grammar(rng, states, classes)
    strings, data, offsets = random_strings(rng, 600, 19)
    g, t = tt.Grammar(nxt, accept, end_id=600), tt.TokenStrings(data, offsets)
    q = rng.integers(-2, states, rows).astype(np.int32)
    got = tt.grammar_bits(g, t, dev(q), 602)
    assert np.array_equal(got.cpu().numpy(), so.grammar_bits(nxt, accept, 600, strings, q, 602))


def test_every_state_of_a_large_automaton_over_a_large_vocabulary():
    """16,400 states and 262,144 tokens: a thread for each pair would be more than a launch may have."""
    rng = np.random.default_rng(9)
    nxt, accept = random_grammar(rng, 16_400, 12)
    strings, data, offsets = random_strings(rng, 262_143, 4)
    g, t = tt.Grammar(nxt, accept, end_id=262_143), tt.TokenStrings(data, offsets)
    every = tt.grammar_bits(g, t, vocab=262_144)
    some = np.sort(rng.choice(16_400, 40, replace=False)).astype(np.int32)  # few enough to be walked one by one
    assert torch.equal(every[dev(some).long()], tt.grammar_bits(g, t, dev(some), 262_144))
    two = some[[0, -1]]
    assert np.array_equal(every[dev(two).long()].cpu().numpy(), so.grammar_bits(nxt, accept, 262_143, strings, two, 262_144))
