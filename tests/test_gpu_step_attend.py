"""Attention over a paged cache on the GPU against the definition in 64 bits.

Tolerances: the oracle gives how far a computation in 32 bits may be off, with 2 percent for products of such errors; on top
comes the one rounding to the output's type, half a step of the value.
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import exact_byte_level_amd as tt  # noqa: E402
from tests import step_oracle as so  # noqa: E402

F8 = torch.float8_e4m3fn
TYPES = [(torch.bfloat16, torch.bfloat16), (torch.float16, torch.float16), (torch.bfloat16, F8), (torch.float16, F8)]
TINY = {torch.float16: 2.0**-24, torch.bfloat16: 2.0**-133}


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()


def host(t):
    return t.double().cpu().numpy()


def near(got, want, slack):
    g = host(got)
    assert g.shape == want.shape and np.isfinite(g).all()
    room = 1.02 * slack + torch.finfo(got.dtype).eps / 2 * (np.abs(want) + slack) + TINY[got.dtype] / 2
    bad = np.abs(g - want) > room
    assert not bad.any(), (np.argwhere(bad)[:4], g[bad][:4], want[bad][:4], room[bad][:4])


def near_sums(got, want, slack):
    g = host(got)
    fine = np.isfinite(want)
    assert np.array_equal(g[~fine], want[~fine])
    assert (np.abs(g - np.where(fine, want, 0))[fine] <= 1.02 * slack[fine] + 2.0**-24 * np.abs(want[fine])).all()


def make(lengths, heads, kv, dim, bs, src=torch.bfloat16, dst=torch.bfloat16, rows=None, by_head=False, seed=0, strength=1.5, garbage=float("nan")):
    """Inputs as a serving program has them; what no request holds is `garbage`."""
    rng, g = np.random.default_rng(seed), torch.Generator("cuda").manual_seed(seed)
    lengths = np.asarray(lengths)
    n = len(lengths)
    row_of = np.arange(n) if rows is None else np.asarray(rows)
    n_rows = int(row_of.max()) + 1
    held = np.zeros(n_rows, np.int64)
    np.maximum.at(held, row_of[row_of >= 0], -(-np.maximum(lengths, 0) // bs)[row_of >= 0])
    blocks, width = int(held.sum()) + 2, max(1, int(held.max())) + 1
    order = rng.permutation(blocks)
    table = np.full((n_rows, width), -1, np.int32)
    at = 0
    for r in range(n_rows):
        table[r, :held[r]] = order[at:at + held[r]]
        at += held[r]
    shape = (blocks, kv, bs, dim) if by_head else (blocks, bs, kv, dim)
    caches = [torch.randn(shape, device="cuda", generator=g) for _ in range(2)]
    if by_head:
        caches = [c.transpose(1, 2) for c in caches]
    live = torch.zeros(blocks, bs, dtype=torch.bool)
    for i in range(n):
        for p in range(max(0, int(lengths[i]))):
            if row_of[i] >= 0:
                live[table[row_of[i], p // bs], p % bs] = True
    for c in caches:
        c.masked_fill_(~live.cuda()[:, :, None, None], garbage)
    caches = [c.to(dst) for c in caches]
    query = torch.randn((n, heads, dim), device="cuda", generator=g).mul_(strength).to(src)
    o = dict(query=query, key_cache=caches[0], value_cache=caches[1], table=torch.from_numpy(table).cuda(), lengths=torch.from_numpy(lengths.astype(np.int32)).cuda())
    if rows is not None:
        o["rows"] = torch.from_numpy(row_of.astype(np.int32)).cuda()
    if dst == F8:
        o["key_scale"], o["value_scale"] = (torch.from_numpy(rng.uniform(0.3, 2, kv).astype(np.float32)).cuda() for _ in range(2))
    return o


def check(o, **options):
    options.setdefault("scale", 1 / math.sqrt(o["query"].shape[-1]))
    plain = {k: (v.cpu().numpy() if isinstance(v, torch.Tensor) else v) for k, v in dict(o, **options).items() if k not in ("query", "key_cache", "value_cache")}
    want, lse, slack, lse_slack = so.attend(host(o["query"]), host(o["key_cache"]), host(o["value_cache"]), **plain)
    out, sums = tt.attend_cache(**o, lse=True, **options)
    near(out, want, slack)
    near_sums(sums, lse, lse_slack)
    return out, sums


@pytest.mark.parametrize("src, dst", TYPES)
@pytest.mark.parametrize("dim", [8, 24, 64, 72, 96, 128, 136, 200, 256])
def test_types_and_dims(src, dst, dim):
    check(make([130, 1, 37, 0, 300, -1], 6, 2, dim, 16, src, dst, seed=dim))


@pytest.mark.parametrize("heads, kv", [(1, 1), (7, 7), (8, 1), (15, 1), (16, 1), (17, 1), (40, 2), (96, 3), (64, 1)])
def test_heads(heads, kv):
    check(make([200, 33], heads, kv, 64, 16, seed=heads))
    check(make([130], heads, kv, 128, 16, torch.float16, F8, seed=heads))


@pytest.mark.parametrize("bs", [1, 3, 8, 16, 24, 31, 32, 64, 100, 128, 300, 1000])
@pytest.mark.parametrize("by_head", [False, True])
def test_block_sizes(bs, by_head):
    check(make([257, 31, 1000, 5], 4, 2, 64, bs, by_head=by_head, seed=bs))


@pytest.mark.parametrize("length", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 513, 4097])
def test_lengths(length):
    check(make([length], 4, 1, 128, 16, seed=length))
    check(make([length, length], 4, 2, 64, 24, torch.float16, F8, seed=length))


def test_many_requests_of_all_lengths():
    """Cuts through long requests, many short ones to a workgroup."""
    rng = np.random.default_rng(3)
    lengths = np.floor(np.exp(rng.uniform(0, 8, 70))).astype(int)
    lengths[rng.random(70) < 0.15] = -1
    check(make(lengths, 2, 1, 64, 16, seed=5))
    check(make(lengths[:20], 10, 5, 128, 32, torch.float16, torch.float16, seed=6))


def test_more_queries_than_are_dealt_out():
    rng = np.random.default_rng(4)
    lengths, rows = rng.integers(-1, 200, 1500), rng.integers(0, 30, 1500)
    check(make(lengths, 1, 1, 64, 16, rows=rows, seed=7))
    check(make(lengths[:700], 14, 7, 8, 16, rows=rows[:700], seed=8))


def test_several_tokens_of_a_row():
    """As a plan of several new tokens gives them: each sees what stands up to itself; places without a token give zeros."""
    positions, rows = [95, 96, 97, 98, 0, 1, 2, 700, -1, -1], [2, 2, 2, 2, 0, 0, 0, 1, -1, -1]
    o = make([max(0, p + 1) for p in positions], 6, 3, 64, 16, rows=rows, seed=9)
    o["lengths"][-2:] = 40  # a row that is none: nothing is seen
    out, lse = check(o)
    assert (out[-2:] == 0).all() and (lse[-2:] == -math.inf).all()
    o["rows"][-2:] = 3  # as many rows as there are
    check(o)


@pytest.mark.parametrize("window", [1, 5, 16, 33, 128, 129, 1000, 5000, 2**40])
def test_windows(window):
    check(make([1, 20, 129, 1500, 0], 4, 2, 64, 16, seed=3), window=window)
    check(make([1500, 300], 4, 1, 128, 24, torch.float16, F8, seed=4), window=window)


@pytest.mark.parametrize("softcap", [1e-6, 0.5, 30.0, 50.0, 1e4, 1e20])
def test_softcaps(softcap):
    check(make([1, 20, 600], 4, 2, 128, 16, seed=3, strength=8.0), softcap=softcap)
    check(make([600], 4, 2, 64, 16, torch.float16, F8, seed=3, strength=8.0), softcap=softcap, window=100)


def test_scales():
    for scale in (1.0, -0.3, 0.0, 1e-6):
        check(make([100, 700], 4, 2, 64, 16, seed=11), scale=scale)
    o = make([90], 2, 1, 64, 16, seed=12)
    want = tt.attend_cache(**o, scale=0.125)
    assert torch.equal(tt.attend_cache(**o), want)


def test_strong_scores():
    """One token outweighs the others, early and late; scores in the hundreds."""
    for place in (0, 5, 127, 128, 700, 1199):
        o = make([1200], 2, 1, 64, 16, seed=place)
        row = o["table"][0]
        o["key_cache"][row[place // 16], place % 16, 0] = 4 * o["query"][0, 0]
        check(o, scale=1.0)


def test_blocks_that_are_not_there():
    """Tokens in blocks outside the cache are not seen, as if they were not there."""
    o = make([100, 400, 64], 4, 2, 64, 16, seed=1)
    o["table"][0, 2] = -1
    o["table"][1, 0:9] = 2**31 - 1
    o["table"][1, 20] = o["key_cache"].shape[0]
    o["table"][2] = -1
    out, lse = check(o)
    assert (out[2] == 0).all() and (lse[2] == -math.inf).all()


def test_lengths_past_the_table():
    o = make([50, 64], 2, 1, 64, 16, seed=2, garbage=0.5)
    o["lengths"][:] = 2**31 - 1  # taken as width * block_size
    check(o)


def test_masked_places_hold_anything():
    for garbage in (float("nan"), float("inf"), float("-inf")):
        for dst in (torch.bfloat16, torch.float16):
            check(make([1, 18, 129], 4, 2, 64, 16, dst, dst, seed=6, garbage=garbage))
            check(make([18, 300], 4, 2, 64, 16, dst, dst, seed=6, garbage=garbage), window=17)
    low = torch.finfo(torch.bfloat16).min
    check(make([18, 300], 4, 2, 64, 16, seed=6, garbage=low))


def test_scores_of_minus_infinity():
    """A key that drives a score to -infinity weighs nothing; a query all of whose scores are that gets zeros."""
    o = make([40, 300], 2, 1, 64, 16, seed=8)
    o["query"][:, :, 0] = 1.0
    t = o["table"]
    o["key_cache"][t[1, 3], 4, 0, 0] = -math.inf
    for b in t[0, :3].tolist():
        o["key_cache"][b, :, 0, 0] = -math.inf
    out, lse = tt.attend_cache(**o, lse=True)
    assert (out[0] == 0).all() and (lse[0] == -math.inf).all()
    q, k, v = host(o["query"])[1], host(o["key_cache"]), host(o["value_cache"])
    at = [(int(t[1, p // 16]), p % 16) for p in range(300) if p != 52]
    b, p = np.array(at).T
    x = q @ k[b, p, 0].T / 8
    w = np.exp(x - x.max(1, keepdims=True))
    want = w @ v[b, p, 0] / w.sum(1, keepdims=True)
    assert np.abs(host(out)[1] - want).max() < 2.0**-8 * np.abs(want).max()


def test_nan_that_is_seen_comes_out():
    o = make([40, 300], 2, 1, 64, 16, seed=8)
    o["key_cache"][o["table"][1, 3], 4, 0, 5] = math.nan
    out = tt.attend_cache(**o)
    assert torch.isnan(out[1]).all() and torch.isfinite(out[0]).all()


@pytest.mark.parametrize("src, dst", TYPES)
@pytest.mark.parametrize("heads, kv, dim", [(2, 2, 64), (4, 2, 40), (8, 1, 128), (3, 1, 136), (2, 1, 256)])
@pytest.mark.parametrize("window", [0, 20])
def test_values_that_are_not_finite_reach_only_who_sees_them(src, dst, heads, kv, dim, window):
    """Queries of one row that see more and more of it: an infinity or NaN among its values goes into the outputs of those that
    see it, at its elements, and into no other."""
    lengths = [300, 60, 90, 91, 89, 130, 61, 92, 10, 299, 93, 40]
    o = make(lengths, heads, kv, dim, 16, src, dst, rows=[0] * 9 + [1] * 3, seed=dim, garbage=0.5)
    infinity = math.nan if dst == F8 else math.inf
    for row, place, head, d, bad in ((0, 90, 0, 7, math.nan), (0, 60, kv - 1, dim - 1, infinity), (0, 9, 0, 0, -infinity), (1, 39, 0, 1, math.nan), (1, 92, 0, 2, infinity), (0, 299, 0, 3, math.nan)):
        o["value_cache"].view(torch.uint8 if dst == F8 else torch.int16)[o["table"][row, place // 16], place % 16, head, d] = \
            torch.tensor([bad], device="cuda").to(dst).view(torch.uint8 if dst == F8 else torch.int16)[0]
    plain = {k: (v.cpu().numpy() if isinstance(v, torch.Tensor) else v) for k, v in o.items() if k not in ("query", "key_cache", "value_cache")}
    with np.errstate(invalid="ignore"):
        want, sums, slack, sums_slack = so.attend(host(o["query"]), host(o["key_cache"]), host(o["value_cache"]), scale=1 / math.sqrt(dim), window=window, **plain)
    fine = np.isfinite(want)
    assert not fine.all() and fine.mean() > 0.9
    got, lse = tt.attend_cache(**o, lse=True, window=window)
    near_sums(lse, sums, sums_slack)
    g = host(got)
    assert np.array_equal(np.isfinite(g), fine)
    room = 1.02 * slack + torch.finfo(src).eps / 2 * (np.abs(want) + slack) + TINY[src] / 2
    assert (np.abs(g[fine] - want[fine]) <= room[fine]).all()


def test_strides_and_alignment():
    """Queries out of a wider projection, an output with gaps, caches that are parts of one tensor, at odd addresses."""
    for src, dst in TYPES:
        o = make([70, 300], 4, 2, 40, 16, src, dst, seed=10)
        want, sums = check(o)
        wide = torch.zeros(2, 4 * 48 + 5, dtype=src, device="cuda")
        query = wide[:, 3:3 + 4 * 48].view(2, 4, 48)[..., 1:41]
        query.copy_(o["query"])
        k, v = o["key_cache"], o["value_cache"]
        pool = torch.zeros(3 + k.shape[0] * 16 * 2 * 91, device="cuda").to(dst)
        both = pool[3:].view(k.shape[0], 16, 2, 91)
        both.view(torch.uint8 if dst == F8 else torch.int16)[..., 1:41] = k.view(torch.uint8 if dst == F8 else torch.int16)
        both.view(torch.uint8 if dst == F8 else torch.int16)[..., 46:86] = v.view(torch.uint8 if dst == F8 else torch.int16)
        out = torch.full((2, 4, 47), 7.0, dtype=src, device="cuda")
        lse = torch.full((2, 9), 7.0, device="cuda")
        table = torch.full((2, o["table"].shape[1] + 3), -5, dtype=torch.int32, device="cuda")
        table[:, :-3] = o["table"]
        tt.attend_cache_into(**dict(o, query=query, key_cache=both[..., 1:41], value_cache=both[..., 46:86], table=table[:, :-3]), out=out[..., 2:42], lse=lse[:, 1:5])
        assert torch.equal(out[..., 2:42], want) and torch.equal(lse[:, 1:5], sums)
        assert (out[..., :2] == 7).all() and (out[..., 42:] == 7).all() and (lse[:, 0] == 7).all() and (lse[:, 5:] == 7).all()


def test_the_same_twice():
    """Nothing depends on the order in which workgroups run."""
    o = make([5000, 37, 2000], 8, 2, 128, 16, seed=14)
    first = tt.attend_cache(**o, lse=True)
    for _ in range(5):
        again = tt.attend_cache(**o, lse=True)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_no_queries_and_no_cache():
    o = make([3], 2, 1, 64, 16)
    none = dict(o, query=o["query"][:0], lengths=o["lengths"][:0], table=o["table"][:0])
    assert tt.attend_cache(**none).shape == (0, 2, 64)
    empty = dict(o, key_cache=o["key_cache"][:0], value_cache=o["value_cache"][:0])
    out, lse = tt.attend_cache(**empty, lse=True)
    assert (out == 0).all() and (lse == -math.inf).all()
    out = tt.attend_cache(**dict(o, table=o["table"][:, :0]))
    assert (out == 0).all()
    out = tt.attend_cache(**dict(o, table=o["table"][:0], rows=torch.zeros(1, dtype=torch.int32, device="cuda")))
    assert (out == 0).all()


def test_a_cache_past_32_bits():
    """Blocks whose offsets pass 2^32 bytes and elements; a request that lies at both ends."""
    cache = torch.zeros(1_050_000, 16, 1, 256, dtype=F8, device="cuda")
    table = torch.tensor([[1_049_999, 3, 1_049_000]], dtype=torch.int32, device="cuda")
    g = torch.Generator("cuda").manual_seed(0)
    for b in table[0].tolist():
        cache[b] = torch.randn(16, 1, 256, device="cuda", generator=g).to(F8)
    small = torch.cat([cache[b][None].view(torch.uint8) for b in table[0].tolist()]).view(F8)
    query = torch.randn(1, 2, 256, device="cuda", generator=g).bfloat16()
    lengths = torch.tensor([45], dtype=torch.int32, device="cuda")
    got = tt.attend_cache(query, cache, cache, table, lengths)
    want = tt.attend_cache(query, small, small, torch.arange(3, dtype=torch.int32, device="cuda")[None], lengths)
    assert torch.equal(got, want) and float(want.abs().sum()) > 0
    check(dict(query=query, key_cache=small, value_cache=small, table=torch.arange(3, dtype=torch.int32, device="cuda")[None], lengths=lengths))


def test_refuses():
    o = make([30, 20], 4, 2, 64, 16)
    out = torch.empty_like(o["query"])
    i32 = dict(dtype=torch.int32, device="cuda")
    bad = [dict(query=o["query"].float()), dict(query=o["query"].half()), dict(query=o["query"][:, :3]), dict(query=o["query"][..., :32]), dict(out=out[:1]),
           dict(out=out.half()), dict(table=o["table"].long()), dict(table=o["table"][:1]), dict(lengths=o["lengths"][:1]), dict(lengths=o["lengths"].long()),
           dict(rows=torch.zeros(3, **i32)), dict(rows=torch.zeros(2, dtype=torch.int64, device="cuda")), dict(window=-1), dict(softcap=-0.5),
           dict(softcap=math.nan), dict(softcap=math.inf), dict(softcap=1e-7), dict(softcap=1e21), dict(key_scale=torch.ones(4, device="cuda")), dict(lse=torch.zeros(2, 3, device="cuda")),
           dict(lse=torch.zeros(2, 4, dtype=torch.float16, device="cuda")), dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda")),
           dict(workspace=torch.empty(1 << 24, dtype=torch.uint8, device="cuda")[1:]), dict(workspace=torch.empty(1 << 24, dtype=torch.int8, device="cuda")),
           dict(key_cache=o["key_cache"][:1]), dict(value_cache=o["value_cache"].half()), dict(table=None), dict(lengths=None), dict(table=o["table"].cpu())]
    for change in bad:
        with pytest.raises(ValueError):
            tt.attend_cache_into(**dict(dict(o, out=out), **change))
    with pytest.raises(TypeError):
        tt.attend_cache_into(**o, out=out, window=1.5)
