"""Grammar calls on tables, classes and string offsets that the C ABI may be given and Python's constructors refuse: entries that name
no state are dead, classes outside the table are its last one, spans are kept inside the strings.  For few states and for many."""
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


def defined(g, t):
    """The automaton and the strings that the device arrays stand for."""
    cls = np.minimum(g.classes.cpu().numpy().astype(int), g.n_classes - 1)
    nxt = g.next.cpu().numpy().astype(int)[:, cls]
    nxt[(nxt < 0) | (nxt >= g.n_states)] = -1
    data = t.strings.cpu().numpy().tobytes()
    off = np.clip(t.offsets.cpu().numpy().astype(np.int64), 0, len(data))
    return nxt, [data[a:b] for a, b in zip(off, off[1:])]


def check(g, t, accept, end, rows, rng, vocab):
    nxt, strings = defined(g, t)
    q = rng.integers(-2, g.n_states + 1, rows).astype(np.int32)
    states = torch.from_numpy(q).cuda()
    want = so.grammar_bits(nxt, accept, end, strings, q, vocab)
    assert np.array_equal(tt.grammar_bits(g, t, states, vocab).cpu().numpy(), want)
    chosen = rng.integers(-1, vocab + 1, rows).astype(np.int32)
    tt.grammar_advance_into(g, t, states, torch.from_numpy(chosen).cuda())
    assert states.tolist() == [so.advance(nxt, accept, end, strings, int(a), int(b)) for a, b in zip(q, chosen)]
    return want


@pytest.mark.parametrize("rows", [3, 63, 64, 200])
@pytest.mark.parametrize("states, classes", [(3, 2), (40, 30), (300, 64), (50, 120)])
@pytest.mark.parametrize("what", ["next", "classes", "one class", "offsets", "all"])
def test_wild_tables(what, states, classes, rows):
    rng = np.random.default_rng(states + rows)
    cls = np.concatenate([np.arange(classes), rng.integers(0, classes, 256 - classes)])
    table = rng.integers(0, states, (states, classes))
    table[rng.random(table.shape) < 0.1] = -1
    accept = rng.random(states) < 0.5
    strings = [bytes(rng.integers(0, 256, int(rng.integers(0, 22))).astype(np.uint8)) for _ in range(700)]
    data = np.frombuffer(b"".join(strings), np.uint8)
    g = tt.Grammar(table[:, cls], accept, end_id=700)
    t = tt.TokenStrings(data, np.concatenate([[0], np.cumsum([len(s) for s in strings])]))
    if what in ("next", "all"):
        wild = torch.from_numpy(rng.random(tuple(g.next.shape)) < 0.1).cuda()
        some = rng.choice(np.array([states, states + 1, 32767, -2, -32768], np.int16), tuple(g.next.shape))
        g.next.copy_(torch.where(wild, torch.from_numpy(some).cuda(), g.next))
    if what in ("classes", "all"):
        g.classes[97:140] = torch.from_numpy(rng.choice(np.array([g.n_classes - 1, min(g.n_classes, 255), 255], np.uint8), 43)).cuda()
    if what == "one class":
        g.classes.fill_(255)
    if what in ("offsets", "all"):
        off = t.offsets.cpu().numpy()
        at = rng.random(len(off)) < 0.1
        off[at] = rng.choice(np.array([-1, -5, -2**31, len(data), len(data) - 1, len(data) - 15, len(data) + 1, 2**31 - 1], np.int32), int(at.sum()))
        long = np.clip(off[1:].astype(int), 0, len(data)) - np.clip(off[:-1].astype(int), 0, len(data)) > 60
        off[:-1][long] = np.clip(off[1:], 0, len(data))[long] - 30  # spans over half of the strings only cost the reference time
        t.offsets.copy_(torch.from_numpy(off))
    want = check(g, t, accept, 700, rows, rng, 702)
    assert what == "one class" or want.any()


def test_a_state_past_the_last_by_hand():
    nxt = np.full((3, 256), -1)
    nxt[:, 97] = 1
    for rows in (3, 66):
        g, t = tt.Grammar(nxt), tt.TokenStrings(np.frombuffer(b"abaa", np.uint8), [0, 1, 2, 4])
        states = torch.arange(rows, dtype=torch.int32, device="cuda") % 3
        g.classes.fill_(255)  # every byte is of the last class, "a"'s or the others'
        dead = int(g.next[0, -1]) < 0
        assert tt.grammar_bits(g, t, states).tolist() == [[0 if dead else 7]] * rows
        g = tt.Grammar(nxt)
        t.offsets.copy_(torch.tensor([0, 900, -5, 4], dtype=torch.int32))  # "abaa", nothing (from 900 to -5), all four again
        assert tt.grammar_bits(g, t, states).tolist() == [[0]] * rows
        t.offsets.copy_(torch.tensor([2, 900, 3, 4], dtype=torch.int32))  # "aa", nothing, "a"
        assert tt.grammar_bits(g, t, states).tolist() == [[5]] * rows
