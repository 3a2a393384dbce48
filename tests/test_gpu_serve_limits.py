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


@pytest.mark.parametrize("add", [False, True])
def test_token_bits_of_four_million_texts(add):
    """More texts than workgroups of 1,024 threads fit one launch."""
    rows, vocab = 2**22 + 5, 40
    g = torch.Generator("cuda").manual_seed(3)
    new = torch.randint(0, 4, (rows,), device="cuda", generator=g)
    offsets = torch.zeros(rows + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = torch.cumsum(new, 0)
    n = int(offsets[-1])
    ids = torch.randint(-1, vocab + 2, (n,), device="cuda", generator=g)
    member = torch.zeros((rows, 64), dtype=torch.bool, device="cuda")
    fine = (ids >= 0) & (ids < vocab)
    member[torch.repeat_interleave(torch.arange(rows, device="cuda"), new)[fine], ids[fine]] = True
    place = torch.ones(32, dtype=torch.int64, device="cuda") << torch.arange(32, device="cuda")
    want = torch.stack([(member[:, k:k + 32] * place).sum(1).to(torch.int32) for k in (0, 32)], 1)
    del member
    bits = torch.full((rows, 2), 0x50, dtype=torch.int32, device="cuda")
    tt.token_bits_into(ids.int(), bits, vocab, offsets=offsets, add=add)
    assert torch.equal(bits, want | 0x50 if add else want)


def test_token_bits_of_a_text_of_more_than_2_to_35_ids():
    """A text whose parts are more than one launch holds: ids at its ends and around the place where the second begins."""
    n = 2**35 + 9000
    if torch.cuda.mem_get_info()[0] < 4 * n + 2**34:
        pytest.skip("needs 145 GB of free memory")
    ids = torch.empty(n, dtype=torch.int32, device="cuda")
    ids.fill_(-1)
    second = (2**32 - 1) // 1024 * 8192
    marks = [0, 8191, 8192, 2**33, second - 1, second, second + 8191, second + 8192, n - 5, n - 1]
    for k, at in enumerate(marks):
        ids[at] = 37 * k
    got = tt.token_bits(ids, 1000).cpu().numpy()
    assert np.flatnonzero(so.unpack(got, 1000)[0]).tolist() == [37 * k for k in range(len(marks))]


def test_logits_of_sixteen_million_rows():
    """As many rows as are allowed, one workgroup more than a launch holds; in place, row r by set r."""
    rows = 2**24
    g = torch.Generator("cuda").manual_seed(4)
    x = torch.randn((rows, 3), device="cuda", generator=g)
    allowed = torch.randint(0, 8, (rows, 1), device="cuda", generator=g).int()
    seen = torch.randint(0, 8, (rows, 1), device="cuda", generator=g).int()
    half = torch.full((rows,), 0.5, device="cuda")
    place = torch.arange(3, device="cuda", dtype=torch.int32)
    want = torch.where((seen >> place) & 1 == 1, torch.where(x > 0, x * 2, x / 2), x) * 2  # by powers of two: exact
    want[(allowed >> place) & 1 == 0] = -float("inf")
    tt.shape_logits_into(x, x, seen=seen, repetition=half, allowed=allowed, temperature=half)
    assert torch.equal(x, want)


def test_token_bits_of_an_add_that_is_no_truth_value():
    """Its error is raised, and nothing is written."""
    bits = torch.full((1, 2), 5, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="ambiguous"):
        tt.token_bits_into(torch.arange(4, dtype=torch.int32, device="cuda"), bits, 64, add=np.array([1, 2]))
    assert bits.tolist() == [[5, 5]]


def test_refusals_of_offsets():
    """Before anything of their size is made."""
    cache = tt.BlockTable(2, 4, 8, 16)
    for n in (2**31, 2**40, 2**62):
        with pytest.raises(tt.TTError) as e:
            cache.plan(torch.tensor([0, 1, n], device="cuda"))
        assert e.value.code == tt.TT_ETOOBIG
    for shape in ((0,), (2,), (4,), (1, 3)):
        with pytest.raises(ValueError, match="offsets"):
            cache.plan(torch.zeros(shape, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError, match="offsets"):
        cache.plan(torch.zeros(3, dtype=torch.int64))
    assert cache.lengths.tolist() == [-1, -1] and int(cache.n_free) == 8
    with pytest.raises(tt.TTError) as e:
        tt.token_bits(torch.zeros(3, dtype=torch.int32, device="cuda"), 40, offsets=torch.zeros(0, dtype=torch.int64, device="cuda"))
    assert e.value.code == tt.TT_EINVAL
