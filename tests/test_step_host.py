"""Host-side checks of the operators around the model (no GPU needed): exports, refusals before any device work, argument
checks of the binding, the oracle's own pins."""
import ctypes
import os
import re
import struct

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import exact_byte_level_amd as tt  # noqa: E402
from tests import step_oracle as so  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 20  # an address that no refused call touches


@pytest.fixture(scope="module")
def lib():
    L = ctypes.CDLL(tt.LIB_PATH)
    vp, i64 = ctypes.c_void_p, ctypes.c_int64
    L.tt_write_cache.argtypes = L.tt_attend_cache.argtypes = L.tt_sample_tokens.argtypes = [vp, vp]
    L.tt_attend_workspace.argtypes, L.tt_attend_workspace.restype = [i64] * 4, i64
    L.tt_sample_workspace.argtypes, L.tt_sample_workspace.restype = [i64] * 2, i64
    return L


def test_exports_every_declared_symbol(lib):
    with open(os.path.join(ROOT, "include", "tt_step.h")) as f:
        names = re.findall(r"^(?:int|int64_t) (tt_\w+)\(", f.read(), re.M)
    assert sorted(names) == ["tt_attend_cache", "tt_attend_workspace", "tt_sample_tokens", "tt_sample_workspace", "tt_write_cache"]
    assert all(hasattr(lib, n) for n in names)


CACHE = dict(ck=P, ck_block=4096, ck_place=256, ck_head=128, cv=P, cv_block=4096, cv_place=256, cv_head=128, key_scale=0, value_scale=0,
             blocks=9, block_size=16, cache_heads=2, dim=128, cache_type=2)
BAD_CACHES = [
    (dict(blocks=-1), tt.TT_EINVAL), (dict(block_size=0), tt.TT_EINVAL), (dict(cache_heads=0), tt.TT_EINVAL), (dict(dim=0), tt.TT_EINVAL),
    (dict(dim=12), tt.TT_EINVAL), (dict(cache_type=0), tt.TT_EINVAL), (dict(cache_type=4), tt.TT_EINVAL), (dict(ck=0), tt.TT_EINVAL),
    (dict(cv=0), tt.TT_EINVAL), (dict(cache_type=1), tt.TT_EINVAL), (dict(blocks=1 << 31), tt.TT_ETOOBIG),
    (dict(block_size=(1 << 20) + 1), tt.TT_ETOOBIG), (dict(cache_heads=4098), tt.TT_ETOOBIG), (dict(dim=264), tt.TT_ETOOBIG)]

WRITE = dict(keys=P, key_stride=256, key_head_stride=128, values=P, value_stride=256, value_head_stride=128, slots=P, tokens=3, in_type=2, **CACHE)


@pytest.mark.parametrize("change, code", BAD_CACHES + [
    (dict(tokens=-1), tt.TT_EINVAL), (dict(in_type=3), tt.TT_EINVAL), (dict(in_type=-1), tt.TT_EINVAL), (dict(in_type=1), tt.TT_EINVAL),
    (dict(keys=0), tt.TT_EINVAL), (dict(values=0), tt.TT_EINVAL), (dict(slots=0), tt.TT_EINVAL), (dict(tokens=1 << 31), tt.TT_ETOOBIG),
    (dict(tokens=0, keys=0, values=0, slots=0), tt.TT_OK), (dict(blocks=0, ck=0, cv=0), tt.TT_OK)])
def test_write_refuses(lib, change, code):
    args = dict(WRITE, **change)
    assert list(args) == list(WRITE)
    assert lib.tt_write_cache(struct.pack("=24q", *args.values()), None) == code
    assert lib.tt_write_cache(None, None) == tt.TT_EINVAL


ATTEND = dict(query=P, query_stride=1024, query_head_stride=128, out=2 * P, out_stride=1024, out_head_stride=128, lse=0, lse_stride=0, queries=3,
              heads=8, type=2, **CACHE, table=P, table_stride=5, table_rows=3, width=5, lengths=P, rows=0, scale=1.0, softcap=0.0, window=0,
              workspace=P, workspace_bytes=1 << 40)


@pytest.mark.parametrize("change, code", BAD_CACHES + [
    (dict(queries=-1), tt.TT_EINVAL), (dict(heads=1), tt.TT_EINVAL), (dict(heads=7), tt.TT_EINVAL), (dict(heads=0), tt.TT_EINVAL),
    (dict(type=0), tt.TT_EINVAL), (dict(type=3), tt.TT_EINVAL), (dict(type=1), tt.TT_EINVAL), (dict(query=0), tt.TT_EINVAL),
    (dict(out=0), tt.TT_EINVAL), (dict(lengths=0), tt.TT_EINVAL), (dict(table=0), tt.TT_EINVAL), (dict(table_rows=-1), tt.TT_EINVAL),
    (dict(width=-1), tt.TT_EINVAL), (dict(window=-1), tt.TT_EINVAL), (dict(softcap=-1.0), tt.TT_EINVAL), (dict(softcap=float("nan")), tt.TT_EINVAL), (dict(softcap=1e-7), tt.TT_EINVAL), (dict(softcap=1e21), tt.TT_EINVAL),
    (dict(workspace=0), tt.TT_EINVAL), (dict(workspace=P + 8), tt.TT_EINVAL), (dict(workspace_bytes=1000), tt.TT_EINVAL),
    (dict(heads=4098), tt.TT_ETOOBIG), (dict(queries=1 << 31), tt.TT_ETOOBIG), (dict(queries=1 << 28), tt.TT_ETOOBIG),
    (dict(table_rows=1 << 31), tt.TT_ETOOBIG), (dict(width=1 << 27), tt.TT_ETOOBIG),
    (dict(queries=0, query=0, out=0, lengths=0, table=0, workspace=0, workspace_bytes=0), tt.TT_OK)])
def test_attend_refuses(lib, change, code):
    args = dict(ATTEND, **change)
    assert list(args) == list(ATTEND)
    kinds = "".join("d" if isinstance(v, float) else "q" for v in args.values())
    assert lib.tt_attend_cache(struct.pack("=" + kinds, *args.values()), None) == code
    assert lib.tt_attend_cache(None, None) == tt.TT_EINVAL


@pytest.mark.parametrize("args, code", [
    ((-1, 8, 2, 64), tt.TT_EINVAL), ((1, 8, 0, 64), tt.TT_EINVAL), ((1, 7, 2, 64), tt.TT_EINVAL), ((1, 8, 2, 60), tt.TT_EINVAL),
    ((1, 0, 2, 64), tt.TT_EINVAL), ((1, 8200, 2, 64), tt.TT_ETOOBIG), ((1, 8, 2, 512), tt.TT_ETOOBIG), ((1 << 30, 8, 2, 64), tt.TT_ETOOBIG)])
def test_attend_workspace_refuses(lib, args, code):
    assert lib.tt_attend_workspace(*args) == code


def test_attend_workspace_stays_small(lib):
    for queries in (0, 1, 7, 300, 1024, 1025, 100_000):
        for heads, kv in ((1, 1), (64, 8), (64, 64), (96, 1), (4096, 4096), (4096, 1)):
            for dim in (8, 64, 200, 256):
                assert 0 <= lib.tt_attend_workspace(queries, heads, kv, dim) < 64 << 20


SAMPLE = dict(logits=P, logits_stride=100, rows=3, vocab=100, type=0, uniform=P, temperature=0, top_k=0, top_p=0, min_p=0, tokens=P, logprobs=0,
              workspace=P, workspace_bytes=1 << 40)


@pytest.mark.parametrize("change, code", [
    (dict(rows=-1), tt.TT_EINVAL), (dict(vocab=-1), tt.TT_EINVAL), (dict(type=3), tt.TT_EINVAL), (dict(type=-1), tt.TT_EINVAL),
    (dict(logits=0), tt.TT_EINVAL), (dict(uniform=0), tt.TT_EINVAL), (dict(tokens=0), tt.TT_EINVAL), (dict(logits_stride=-1), tt.TT_EINVAL),
    (dict(rows=(1 << 24) + 1), tt.TT_ETOOBIG), (dict(vocab=(1 << 24) + 1), tt.TT_ETOOBIG), (dict(rows=1 << 20, vocab=1 << 16), tt.TT_ETOOBIG),
    (dict(rows=0, logits=0, uniform=0, tokens=0, workspace=0, workspace_bytes=0), tt.TT_OK)])
def test_sample_refuses(lib, change, code):
    args = dict(SAMPLE, **change)
    assert list(args) == list(SAMPLE)
    assert lib.tt_sample_tokens(struct.pack("=14q", *args.values()), None) == code
    assert lib.tt_sample_tokens(None, None) == tt.TT_EINVAL


def test_sample_workspace_refuses(lib):
    assert lib.tt_sample_workspace(-1, 5) == lib.tt_sample_workspace(5, -1) == tt.TT_EINVAL
    assert lib.tt_sample_workspace(1 << 25, 1) == lib.tt_sample_workspace(1 << 24, 1 << 24) == tt.TT_ETOOBIG
    assert lib.tt_sample_workspace(0, 0) >= 0


def test_binding_refuses_host_tensors():
    x, cache = torch.zeros(2, 2, 64, dtype=torch.bfloat16), torch.zeros(3, 16, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="keys is not on a GPU"):
        tt.write_cache_into(x, x, torch.zeros(2, dtype=torch.int64), cache, cache)
    with pytest.raises(ValueError, match="query is not on a GPU"):
        tt.attend_cache_into(x, cache, cache, torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), x)
    with pytest.raises(ValueError, match="logits is not on a GPU"):
        tt.sample_tokens_into(torch.zeros(2, 9), torch.zeros(2), torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="a tensor is needed"):
        tt.sample_tokens_into([1.0], torch.zeros(2), torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="a tensor is needed"):
        tt.attend_cache_into(None, cache, cache, None, None, x)


def test_oracle_by_hand():
    v = so.e4m3_values()
    assert v[0] == 0 and v[1] == 2.0**-9 and v[0x38] == 1 and v[0x7E] == 448 and np.isnan(v[0xFF]) and v[0xB8] == -1
    fine = np.delete(np.arange(256, dtype=np.uint8), [127, 255])
    assert np.array_equal(so.e4m3(v[fine]), fine)
    assert so.e4m3(np.array([1.0625, 1.1875, 500.0, -np.inf, 2.0**-10, -2.0**-10, 2.0**-10 * 1.01, 460.0])).tolist() == [
        0x38, 0x3A, 0x7E, 0xFE, 0, 0x80, 1, 0x7E]
    keys = np.zeros((2, 2, 1, 8))
    values = np.arange(32.0).reshape(2, 2, 1, 8)
    keys[1, 0, 0, 0] = 3.0
    query = np.zeros((2, 1, 8))
    query[0, 0, 0] = 1.0
    out, lse, _, _ = so.attend(query, keys, values, np.array([[1, 0], [-1, 5]]), [3, 2], scale=np.log(2) / 3)
    # weights 2, 1, 1 of block 1's two places and block 0's first
    assert np.allclose(out[0, 0], (2 * values[1, 0, 0] + values[1, 1, 0] + values[0, 0, 0]) / 4) and np.isclose(lse[0, 0], np.log(4))
    assert (out[1] == 0).all() and lse[1, 0] == -np.inf
    x = np.log(np.array([[4.0, 2.0, 1.0, 1.0]]))
    draw = lambda u, **o: so.sample(x, [u], **{k: [w] for k, w in o.items()})[0][0]  # noqa: E731
    assert [draw(u) for u in (0, 0.49, 0.5, 0.74, 0.75, 0.875, 0.99)] == [0, 0, 1, 1, 2, 3, 3]
    assert [draw(u, top_k=2) for u in (0.6, 0.7)] == [0, 1] and [draw(u, top_p=0.8) for u in (0.57, 0.58, 0.9)] == [0, 1, 2]
    assert draw(0.99, min_p=0.5) == 1 and draw(0.99, min_p=0.51) == 0 and draw(0.99, temperature=0) == 0
    assert so.sample(np.full((1, 3), -np.inf), [0.5])[0][0] == -1
