"""Token sets and grammar masks on the GPU against the sequential definition."""
import os

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import exact_byte_level_amd as tt  # noqa: E402
from oracle.bpe import Vocab  # noqa: E402
from tests import serve_oracle as so  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def room(rows, words, pad, fill=0x5A5A5A5A):
    """[rows, words] of a wider buffer, and the buffer."""
    wide = torch.full((rows, words + pad), fill, dtype=torch.int32, device="cuda")
    return wide[:, :words], wide


# --------------------------------------------------------------- token sets

@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("rows, n, vocab, pad", [
    (1, 0, 40, 0), (1, 1, 1, 0), (1, 5000, 33, 2), (3, 100, 31, 1), (7, 3000, 32, 0), (64, 20000, 1000, 0),
    (5, 400, 100_257, 3), (2, 300_000, 50_256, 0), (300, 9000, 5000, 0), (1, 700_000, 600_001, 0), (2, 5000, 1_200_000, 1),
    (1, 65_536, 5000, 0), (1500, 100_000, 20_000, 0), (3, 90_001, 1_200_000, 0), (12, 150_000, 60_000, 0), (5, 200_000, 33, 1), (2500, 70_000, 3000, 2)])
def test_token_bits(rows, n, vocab, pad, add):
    rng = np.random.default_rng(rows * 7 + n)
    ids = np.minimum((rng.random(n) ** 3 * vocab).astype(np.int32), vocab - 1)
    wild = rng.random(n) < 0.02
    ids[wild] = rng.choice(np.array([-1, vocab, vocab + 31, 2**31 - 1, -2**31], np.int32), int(wild.sum()))
    offsets = np.sort(np.concatenate([[0, n], rng.integers(0, n + 1, rows - 1)])).astype(np.int64)
    bits, wide = room(rows, so.words(vocab), pad)
    before = bits.cpu().numpy()
    tt.token_bits_into(dev(ids), bits, vocab, offsets=dev(offsets), add=add)
    want = so.token_bits(ids, offsets, vocab)
    assert np.array_equal(bits.cpu().numpy(), want | before if add else want)
    assert (wide[:, so.words(vocab):] == 0x5A5A5A5A).all()


def test_token_bits_of_many_long_texts():
    """More texts than a workgroup looks at in one go, long enough to be dealt out."""
    rng = np.random.default_rng(1)
    rows, n, vocab = 1030, 12_700_000, 70
    ids = rng.integers(-1, vocab + 1, n).astype(np.int32)
    cuts = np.sort(rng.integers(0, n, rows - 1))
    cuts[5:300] = cuts[5]  # empty texts, and after them one of many ids
    offsets = np.concatenate([[0], cuts, [n]]).astype(np.int64)
    offsets[400] = offsets[399] + 1
    member = np.zeros((rows, vocab), bool)
    fine = (ids >= 0) & (ids < vocab)
    member[(np.searchsorted(offsets, np.arange(n), side="right") - 1)[fine], ids[fine]] = True
    assert np.array_equal(tt.token_bits(dev(ids), vocab, offsets=dev(offsets)).cpu().numpy(), so.pack(member))


def test_token_bits_of_one_text_without_offsets():
    ids = np.arange(0, 900, 7, dtype=np.int32)
    got = tt.token_bits(dev(ids), 900)
    assert np.array_equal(got.cpu().numpy(), so.token_bits(ids, [0, len(ids)], 900))


def test_token_bits_bounds_are_kept():
    """Offsets that leave the ids, fall or are wild read nothing outside."""
    ids = np.arange(64, dtype=np.int32)
    offsets = np.array([-5, 10, 4, 70, 2**62, -2**62, 64], np.int64)
    got = tt.token_bits(dev(ids), 64, offsets=dev(offsets))
    assert np.array_equal(got.cpu().numpy(), so.token_bits(ids, offsets, 64))
    ids = np.arange(70_000, dtype=np.int32)
    offsets = np.array([-5, 10_000, 4000, 71_000, 2**62, -2**62, 64], np.int64)
    got = tt.token_bits(dev(ids), 65_000, offsets=dev(offsets))
    assert np.array_equal(got.cpu().numpy(), so.token_bits(ids, offsets, 65_000))


def test_token_bits_of_a_batch_call():
    """Straight from encode_batch, on another stream, and replayed in a graph on new ids."""
    merges = np.load(os.path.join(ROOT, "data", "vocab_c1.npy"))
    tt.load(merges)
    text = b"def f(x):\n    return x + 1\n" * 40
    cut = np.array([0, 100, 100, 431, len(text)], np.int64)
    ids, off = tt.encode_batch(torch.frombuffer(bytearray(text), dtype=torch.uint8).cuda(), dev(cut))
    vocab = 256 + len(merges)
    want = so.token_bits(ids.cpu().numpy(), off.numpy(), vocab)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    got = tt.token_bits(ids, vocab, offsets=off.cuda(), stream=stream)
    stream.synchronize()
    assert np.array_equal(got.cpu().numpy(), want)
    rng = np.random.default_rng(0)
    some, offsets, bits = ids.clone(), off.cuda(), torch.empty_like(got)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tt.token_bits_into(some, bits, vocab, offsets=offsets)
    for _ in range(4):
        new = rng.integers(0, vocab, len(some)).astype(np.int32)
        some.copy_(dev(new))
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(bits.cpu().numpy(), so.token_bits(new, off.numpy(), vocab))
        tt.token_bits(some, vocab)


# ----------------------------------------------------------------- grammars

def random_grammar(rng, states, classes, density):
    """A random automaton over bytes that fall into `classes` classes."""
    cls = rng.integers(0, classes, 256)
    table = rng.integers(0, states, (states, classes))
    table[rng.random(table.shape) > density] = -1
    return table[:, cls], rng.random(states) < 0.5


def random_strings(rng, n, longest):
    strings = [bytes(rng.integers(0, 256, int(rng.integers(0, longest + 1))).astype(np.uint8)) for _ in range(n)]
    return strings, np.frombuffer(b"".join(strings), np.uint8), np.concatenate([[0], np.cumsum([len(s) for s in strings])])


@pytest.mark.parametrize("states, classes, density, tokens, longest, vocab, rows, pad", [
    (1, 1, 1.0, 1, 3, 1, 1, 0), (2, 3, 0.8, 40, 6, 45, 4, 1), (300, 40, 0.9, 500, 20, 500, 33, 0),
    (30, 256, 0.7, 1000, 9, 1025, 7, 0), (5, 4, 0.5, 70, 0, 70, 3, 0), (4, 5, 0.97, 300, 300, 300, 5, 2),
    (2000, 200, 0.95, 200, 40, 64, 64, 0), (700, 90, 0.9, 3000, 12, 3001, 100, 0), (32767, 3, 0.9, 100, 9, 100, 50, 0), (32767, 3, 0.9, 100, 9, 100, 70, 0), (300, 40, 0.9, 500, 20, 500, 130, 0),
    (12, 20, 1.0, 0, 0, 40, 3, 0), (12, 20, 1.0, 0, 0, 40, 64, 0), (3000, 50, 0.9, 700, 20, 700, 70, 0),
    (60, 20, 0.97, 5000, 24, 5001, 65, 1), (64, 64, 0.9, 5000, 6, 4097, 64, 0), (65, 65, 0.9, 300, 6, 290, 65, 0)])
def test_grammar_bits_and_advance(states, classes, density, tokens, longest, vocab, rows, pad):
    rng = np.random.default_rng(states + tokens)
    nxt, accept = random_grammar(rng, states, classes, density)
    strings, data, offsets = random_strings(rng, tokens, longest)
    for end in (-1, vocab - 1, min(3, vocab - 1)):
        g, t = tt.Grammar(nxt, accept, end_id=end), tt.TokenStrings(data, offsets)
        q = rng.integers(0, states, rows).astype(np.int32)
        wild = rng.random(rows) < 0.2
        q[wild] = rng.choice(np.array([-1, -2, states, -3, 2**31 - 1, -2**31], np.int32), int(wild.sum()))
        bits, wide = room(rows, so.words(vocab), pad)
        tt.grammar_bits_into(g, t, dev(q), bits, vocab)
        want = so.grammar_bits(nxt, accept, end, strings, q, vocab)
        got = bits.cpu().numpy()
        assert np.array_equal(got, want)
        assert (wide[:, so.words(vocab):] == 0x5A5A5A5A).all()
        chosen = rng.integers(-1, vocab + 2, rows).astype(np.int32)
        states_d = dev(q)
        out = torch.empty_like(states_d)
        tt.grammar_advance_into(g, t, states_d, dev(chosen), out)
        after = [so.advance(nxt, accept, end, strings, int(a), int(b)) for a, b in zip(q, chosen)]
        assert out.tolist() == after
        tt.grammar_advance_into(g, t, states_d, dev(chosen))
        assert states_d.tolist() == after


@pytest.mark.parametrize("states, classes, rows", [(300, 40, 5000), (700, 60, 3000), (40, 100, 2000)])
def test_grammar_bits_of_many_rows(states, classes, rows):
    """More sets than LDS holds at a time, some rows free or dead: each row is its state's of the call for all states."""
    rng = np.random.default_rng(states)
    nxt, accept = random_grammar(rng, states, classes, 0.8)
    strings, data, offsets = random_strings(rng, 60_000, 9)
    g, t = tt.Grammar(nxt, accept, end_id=60_000), tt.TokenStrings(data, offsets)
    every = tt.grammar_bits(g, t, vocab=60_003)
    some = rng.integers(0, states, 3)
    assert np.array_equal(every.cpu().numpy()[some], so.grammar_bits(nxt, accept, 60_000, strings, some, 60_003))
    q = rng.integers(-2, states, rows).astype(np.int32)
    got = tt.grammar_bits(g, t, dev(q), 60_003).cpu().numpy()
    want = every.cpu().numpy()[np.maximum(q, 0)]
    want[q == -1] = 0
    want[q == -2] = so.pack(np.ones((1, 60_003), bool))
    assert np.array_equal(got, want)


def test_grammar_over_the_tokenizer():
    """The loaded tokenizer's own strings; the sets of every state; a token is in a state's set exactly if the step
    over it does not end in the dead state."""
    merges = np.load(os.path.join(ROOT, "data", "vocab_c1.npy"))
    tt.load(merges)
    vocab = Vocab(merges)
    tokens = tt.TokenStrings.of_tokenizer()
    strings = [bytes([b]) for b in range(256)]
    for x, y in merges.tolist():
        strings.append(strings[x] + strings[y])
    n = len(strings)
    assert tokens.n_tokens == n and vocab is not None
    data, off = tokens.strings.cpu().numpy().tobytes(), tokens.offsets.tolist()
    assert [data[off[v]:off[v + 1]] for v in range(n)] == strings
    nxt = np.full((4, 256), -1)  # words of small letters, single spaces between, a full stop at the end
    nxt[0, 97:123] = 1
    nxt[1, 97:123] = 1
    nxt[1, 32] = 2
    nxt[2, 97:123] = 1
    nxt[1, 46] = 3
    g = tt.Grammar(nxt, [0, 0, 0, 1], end_id=n)
    bits = tt.grammar_bits(g, tokens, vocab=n + 1)
    assert np.array_equal(bits.cpu().numpy(), so.grammar_bits(nxt, [0, 0, 0, 1], n, strings, range(4), n + 1))
    member = so.unpack(bits.cpu().numpy(), n + 1)
    assert member[3].sum() == 1 and member[3, n]
    every = torch.arange(n, dtype=torch.int32, device="cuda")
    for q in range(4):
        out = torch.empty_like(every)
        tt.grammar_advance_into(g, tokens, torch.full_like(every, q), every, out)
        assert np.array_equal(out.cpu().numpy() >= 0, member[q, :n])


def test_grammar_table_that_names_no_state_is_dead():
    """Entries outside the states and classes outside the table, which the C ABI may be given, read nothing outside."""
    nxt = np.full((3, 256), -1)
    nxt[:, 97] = 1
    g, t = tt.Grammar(nxt), tt.TokenStrings(np.frombuffer(b"abaa", np.uint8), [0, 1, 2, 4])
    a = int(g.classes[97])
    g.next[1, a] = 3  # as if there were a fourth state
    bits = tt.grammar_bits(g, t)
    assert bits.tolist() == [[1], [0], [1]]  # from 1 every "a" is dead; "aa" is dead everywhere
    g.classes.fill_(255)  # no such class: taken as the last one
    assert tt.grammar_bits(g, t).shape == (3, 1)
    g2 = tt.Grammar(nxt)
    t.offsets.copy_(torch.tensor([0, 900, -5, 4], dtype=torch.int32))
    assert tt.grammar_bits(g2, t).shape == (3, 1)


def test_grammar_in_a_graph():
    rng = np.random.default_rng(1)
    nxt, accept = random_grammar(rng, 20, 10, 0.9)
    strings, data, offsets = random_strings(rng, 400, 8)
    g, t = tt.Grammar(nxt, accept), tt.TokenStrings(data, offsets)
    q = rng.integers(0, 20, 6).astype(np.int32)
    states, chosen = dev(q), torch.zeros(6, dtype=torch.int32, device="cuda")
    bits = torch.empty((6, so.words(400)), dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tt.grammar_advance_into(g, t, states, chosen)
        tt.grammar_bits_into(g, t, states, bits)
    for _ in range(5):
        pick = rng.integers(0, 400, 6).astype(np.int32)
        q = rng.integers(0, 20, 6).astype(np.int32)
        chosen.copy_(dev(pick))
        states.copy_(dev(q))
        graph.replay()
        torch.cuda.synchronize()
        q = np.array([so.advance(nxt, accept, -1, strings, int(a), int(b)) for a, b in zip(q, pick)])
        assert states.tolist() == q.tolist()
        assert np.array_equal(bits.cpu().numpy(), so.grammar_bits(nxt, accept, -1, strings, q, 400))
        tt.grammar_bits(g, t)
