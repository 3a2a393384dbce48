"""Host-side checks of the serving calls (no GPU needed): exports, refusals before any device work, argument checks of
the binding, and the oracle's own pins."""
import ctypes
import os
import re
import struct

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import exact_byte_level_amd as tt  # noqa: E402
from tests import serve_oracle as so  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 20  # an address that no refused call touches


@pytest.fixture(scope="module")
def lib():
    """The C calls with their argument types."""
    L = ctypes.CDLL(tt.LIB_PATH)
    vp, i64 = ctypes.c_void_p, ctypes.c_int64
    L.tt_plan_blocks.argtypes = L.tt_shape_logits.argtypes = L.tt_vocab_size.argtypes = L.tt_vocab_strings.argtypes = [vp, vp]
    L.tt_release_blocks.argtypes = [vp, vp, i64, i64, vp, i64, i64, vp, i64, vp, vp, vp, vp, vp]
    L.tt_token_bits.argtypes = [vp, i64, vp, i64, i64, vp, i64, ctypes.c_int, vp]
    L.tt_grammar_bits.argtypes = [vp, vp, i64, vp, i64, i64, vp]
    L.tt_grammar_advance.argtypes = [vp, vp, vp, i64, vp, vp]
    return L


def test_exports_every_declared_symbol(lib):
    with open(os.path.join(ROOT, "include", "tt_serve.h")) as f:
        names = re.findall(r"^int (tt_\w+)\(", f.read(), re.M)
    assert sorted(names) == ["tt_grammar_advance", "tt_grammar_bits", "tt_plan_blocks", "tt_release_blocks",
                             "tt_shape_logits", "tt_token_bits", "tt_vocab_size", "tt_vocab_strings"]
    raw = ctypes.CDLL(tt.LIB_PATH)
    assert all(hasattr(raw, n) for n in names)
    assert tt.strerror(tt.TT_ENOBLOCKS) == "not enough free blocks"


PLAN = dict(lengths=P, offsets=P, rows=4, places=8, block_size=16, table=P, table_stride=8, width=8, free_blocks=P,
            free_cap=8, n_free=P, slots=P, positions=0, row_of=0, out_lengths=P, out_n_free=P, out_n=P)


@pytest.mark.parametrize("change, code", [
    (dict(rows=-1), tt.TT_EINVAL), (dict(lengths=0), tt.TT_EINVAL), (dict(block_size=0), tt.TT_EINVAL),
    (dict(table=0), tt.TT_EINVAL), (dict(table_stride=7), tt.TT_EINVAL), (dict(free_blocks=0), tt.TT_EINVAL),
    (dict(n_free=0), tt.TT_EINVAL), (dict(slots=0), tt.TT_EINVAL), (dict(places=-1), tt.TT_EINVAL),
    (dict(out_lengths=0), tt.TT_EINVAL), (dict(out_n_free=0), tt.TT_EINVAL), (dict(out_n=0), tt.TT_EINVAL),
    (dict(offsets=0, places=3), tt.TT_EINVAL), (dict(width=-1), tt.TT_EINVAL), (dict(free_cap=-1), tt.TT_EINVAL),
    (dict(places=1 << 31), tt.TT_ETOOBIG), (dict(rows=(1 << 24) + 1), tt.TT_ETOOBIG),
    (dict(block_size=(1 << 20) + 1), tt.TT_ETOOBIG), (dict(free_cap=1 << 31), tt.TT_ETOOBIG),
    (dict(width=1 << 27, table_stride=1 << 27), tt.TT_ETOOBIG)])
def test_plan_refuses(lib, change, code):
    args = dict(PLAN, **change)
    assert list(args) == list(PLAN)
    assert lib.tt_plan_blocks(struct.pack("=17q", *args.values()), None) == code
    assert lib.tt_plan_blocks(None, None) == tt.TT_EINVAL


@pytest.mark.parametrize("at, value, code", [
    (0, 0, tt.TT_EINVAL), (1, 0, tt.TT_EINVAL), (2, -1, tt.TT_EINVAL), (3, 0, tt.TT_EINVAL), (4, 0, tt.TT_EINVAL),
    (5, 7, tt.TT_EINVAL), (7, 0, tt.TT_EINVAL), (9, 0, tt.TT_EINVAL), (10, 0, tt.TT_EINVAL), (11, 0, tt.TT_EINVAL),
    (12, 0, tt.TT_EINVAL), (2, 1 << 25, tt.TT_ETOOBIG), (8, 1 << 31, tt.TT_ETOOBIG)])
def test_release_refuses(lib, at, value, code):
    args = [P, P, 4, 16, P, 8, 8, P, 8, P, P, P, P]
    args[at] = value
    assert lib.tt_release_blocks(*args, None) == code


@pytest.mark.parametrize("args, code", [
    ((P, -1, P, 1, 100, P, 4, 0), tt.TT_EINVAL), ((0, 5, P, 1, 100, P, 4, 0), tt.TT_EINVAL),
    ((P, 5, 0, 2, 100, P, 4, 0), tt.TT_EINVAL), ((P, 5, P, -1, 100, P, 4, 0), tt.TT_EINVAL),
    ((P, 5, P, 2, -1, P, 4, 0), tt.TT_EINVAL), ((P, 5, P, 2, 100, 0, 4, 0), tt.TT_EINVAL),
    ((P, 5, P, 2, 100, P, 3, 0), tt.TT_EINVAL), ((P, 5, P, 1, (1 << 24) + 1, P, 1 << 20, 0), tt.TT_ETOOBIG),
    ((P, 5, P, 1 << 20, 1 << 20, P, 1 << 20, 0), tt.TT_ETOOBIG),
    ((P, 5, P, 0, 100, 0, 0, 0), tt.TT_OK), ((P, 5, P, 3, 0, 0, 0, 0), tt.TT_OK)])
def test_token_bits_refuses(lib, args, code):
    assert lib.tt_token_bits(*args, None) == code


GRAMMAR = dict(classes=P, next=P, accept=P, n_states=5, n_classes=7, end_id=-1, strings=P, n_bytes=10,
               string_offsets=P, n_tokens=4)


@pytest.mark.parametrize("change, code", [
    (dict(classes=0), tt.TT_EINVAL), (dict(next=0), tt.TT_EINVAL), (dict(accept=0), tt.TT_EINVAL),
    (dict(n_states=0), tt.TT_EINVAL), (dict(n_classes=0), tt.TT_EINVAL), (dict(n_classes=257), tt.TT_EINVAL),
    (dict(end_id=-2), tt.TT_EINVAL), (dict(strings=0), tt.TT_EINVAL), (dict(string_offsets=0), tt.TT_EINVAL),
    (dict(n_bytes=-1), tt.TT_EINVAL), (dict(n_states=32768), tt.TT_ETOOBIG), (dict(n_tokens=(1 << 24) + 1), tt.TT_ETOOBIG)])
def test_grammar_refuses(lib, change, code):
    args = struct.pack("=10q", *dict(GRAMMAR, **change).values())
    assert lib.tt_grammar_bits(args, P, 3, P, 1, 20, None) == code
    assert lib.tt_grammar_advance(args, P, P, 3, P, None) == code


def test_grammar_refuses_rows(lib):
    g = struct.pack("=10q", *GRAMMAR.values())
    assert lib.tt_grammar_bits(None, P, 3, P, 1, 20, None) == tt.TT_EINVAL
    assert lib.tt_grammar_bits(g, 0, 3, P, 1, 20, None) == tt.TT_EINVAL
    assert lib.tt_grammar_bits(g, P, 3, 0, 1, 20, None) == tt.TT_EINVAL
    assert lib.tt_grammar_bits(g, P, 3, P, 1, 33, None) == tt.TT_EINVAL
    assert lib.tt_grammar_bits(g, P, 3, P, 1, -1, None) == tt.TT_EINVAL
    assert lib.tt_grammar_bits(g, P, 0, 0, 0, 33, None) == tt.TT_OK
    assert lib.tt_grammar_advance(g, P, 0, 3, P, None) == tt.TT_EINVAL
    assert lib.tt_grammar_advance(g, P, P, 3, 0, None) == tt.TT_EINVAL


SHAPE = dict(logits=P, logits_stride=100, out=2 * P, out_stride=100, rows=3, vocab=100, in_type=1, out_type=1, seen=P,
             seen_stride=4, generated=P, generated_stride=5, generated_cap=5, n_generated=P, repetition=P, frequency=P,
             presence=P, bias_offsets=P, bias_ids=P, bias_values=P, n_bias=6, allowed=P, allowed_stride=4,
             allowed_count=3, allowed_rows=P, temperature=P)


@pytest.mark.parametrize("change, code", [
    (dict(rows=-1), tt.TT_EINVAL), (dict(vocab=-1), tt.TT_EINVAL), (dict(in_type=3), tt.TT_EINVAL),
    (dict(out_type=2), tt.TT_EINVAL), (dict(in_type=0), tt.TT_EINVAL), (dict(logits=0), tt.TT_EINVAL),
    (dict(out=0), tt.TT_EINVAL), (dict(out_stride=99), tt.TT_EINVAL), (dict(logits_stride=-1), tt.TT_EINVAL),
    (dict(out=P, out_type=0), tt.TT_EINVAL), (dict(out=P, out_stride=104), tt.TT_EINVAL),
    (dict(generated_cap=-1), tt.TT_EINVAL), (dict(n_bias=-1), tt.TT_EINVAL), (dict(bias_ids=0), tt.TT_EINVAL),
    (dict(bias_values=0), tt.TT_EINVAL), (dict(allowed_count=-1), tt.TT_EINVAL), (dict(seen_stride=-1), tt.TT_EINVAL),
    (dict(vocab=(1 << 24) + 1), tt.TT_ETOOBIG), (dict(rows=(1 << 24) + 1), tt.TT_ETOOBIG),
    (dict(n_bias=(1 << 30) + 1), tt.TT_ETOOBIG), (dict(generated_cap=(1 << 30) + 1), tt.TT_ETOOBIG), (dict(rows=0), tt.TT_OK), (dict(vocab=0), tt.TT_OK)])
def test_shape_refuses(lib, change, code):
    args = dict(SHAPE, **change)
    assert list(args) == list(SHAPE)
    assert lib.tt_shape_logits(struct.pack("=26q", *args.values()), None) == code
    assert lib.tt_shape_logits(None, None) == tt.TT_EINVAL


def test_vocab_refuses(lib):
    n = ctypes.c_int64()
    assert lib.tt_vocab_size(None, ctypes.byref(n)) == tt.TT_EINVAL
    assert lib.tt_vocab_strings(None, None) == tt.TT_EINVAL


def test_binding_refuses_host_tensors():
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    i64 = lambda *s: torch.zeros(s, dtype=torch.int64)  # noqa: E731
    with pytest.raises(ValueError, match="lengths is not on a GPU"):
        tt.plan_blocks_into(i32(2), i32(2, 3), i32(4), i32(1), 16, i64(2), i64(1))
    with pytest.raises(ValueError, match="lengths is not on a GPU"):
        tt.release_blocks_into(i32(2), i32(2), i32(2, 3), i32(4), i32(1), 16, i64(1))
    with pytest.raises(ValueError, match="bits is not on a GPU"):
        tt.token_bits_into(i32(3), i32(1, 1), 32)
    with pytest.raises(ValueError, match="logits is not on a GPU"):
        tt.shape_logits_into(torch.zeros(1, 8), torch.zeros(1, 8))


def test_binding_refuses_what_is_no_tensor():
    with pytest.raises(ValueError, match="logits: a tensor is needed"):
        tt.shape_logits_into([1.0], torch.zeros(1, 1))
    with pytest.raises(ValueError, match="bits: a tensor is needed"):
        tt.token_bits_into(torch.zeros(1, dtype=torch.int32), None, 32)


def test_grammar_checks_its_table():
    ok = np.full((3, 256), -1)
    for bad in (ok[:, :255], np.zeros((0, 256), int), ok.astype(float), np.full((3, 256), 3), np.full((3, 256), -2)):
        with pytest.raises(ValueError):
            tt.Grammar(bad, device="cpu")
    with pytest.raises(ValueError):
        tt.Grammar(ok, accept=np.zeros(2), device="cpu")
    nxt = ok.copy()
    nxt[0, 97:123] = 1
    nxt[1, 48:58] = 2
    g = tt.Grammar(nxt, device="cpu")
    assert g.n_classes == 3  # letters, digits, the rest
    assert np.array_equal(g.next.numpy()[:, g.classes.numpy()], nxt)


def test_token_strings_check_their_offsets():
    for offsets in ([], [-1, 2], [0, 3, 2], [0, 5]):
        with pytest.raises(ValueError):
            tt.TokenStrings(np.arange(4), np.asarray(offsets, np.int64), device="cpu")
    assert tt.TokenStrings(np.arange(4), [0, 1, 1, 4], device="cpu").n_tokens == 3


def test_oracle_by_hand():
    table = np.full((2, 3), -1, np.int32)
    table[0, 0] = 9
    got = so.plan(np.array([3, -1], np.int32), table, np.array([5, 6, 7], np.int32), 3, 4, 6, np.array([0, 2, 3]))
    assert got["n"] == 3 and got["n_free"] == 1 and got["lengths"].tolist() == [5, 1]
    assert got["slots"].tolist() == [39, 28, 24, -1, -1, -1] and got["table"].tolist() == [[9, 7, -1], [6, -1, -1]]
    back = so.release(got["lengths"], np.array([1, 0]), got["table"], np.array([5, 0, 0], np.int32), 1, 4)
    assert back["free"].tolist() == [5, 9, 7] and back["lengths"].tolist() == [-1, 1] and back["n"] == 2
    assert so.token_bits(np.array([0, 33, -1, 40]), [0, 2, 4], 34).tolist() == [[1, 2], [0, 0]]
    nxt = np.full((2, 256), -1)
    nxt[0, 97] = 1
    assert so.grammar_bits(nxt, [0, 1], 3, [b"a", b"aa", b""], [0, 1, -1, -2], 4).tolist() == [[1], [8], [0], [15]]
    x, _ = so.shape_logits(np.array([[2.0, -2.0, 1.0, 0.5]]), generated=np.array([[0, 1, 0]]), repetition=[2.0],
                           frequency=[0.25], presence=[1.0], bias_offsets=[0, 2], bias_ids=np.array([2, 2]),
                           bias_values=np.array([9.0, 3.0]), allowed=np.array([[7]], np.int32), temperature=[0.5])
    assert x.tolist() == [[-1.0, -10.5, 8.0, -np.inf]]
