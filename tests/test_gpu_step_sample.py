"""Drawing tokens on the GPU against the definition in 64 bits: the tokens have to be the same.

Both sides hold weights and sums in 64 bits, off by at most 2^-40 of the sum, so a random number would have to come that near to
a border to tell them apart; the inputs' random numbers are fixed.  Logarithms of shares are rounded to 32 bits: half a
step, 2^-24 of the value, and 2^-40.
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import exact_byte_level_amd as tt  # noqa: E402
from tests import step_oracle as so  # noqa: E402

TYPES = [torch.float32, torch.float16, torch.bfloat16]


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()


def check(logits, uniform, **o):
    """logits: a tensor on the GPU; the others host arrays."""
    uniform = np.asarray(uniform, np.float32)
    tokens, logprobs, kept = so.sample(logits.double().cpu().numpy(), uniform, **o)
    kinds = dict(temperature=np.float32, top_k=np.int32, top_p=np.float32, min_p=np.float32)
    o = {k: torch.from_numpy(np.asarray(v).astype(kinds[k])).cuda() for k, v in o.items()}
    got, shares = tt.sample_tokens(logits, torch.from_numpy(uniform).cuda(), logprobs=True, **o)
    got, shares = got.cpu().numpy(), shares.double().cpu().numpy()
    bad = np.flatnonzero(got != tokens)
    assert not len(bad), (bad[:5], got[bad][:5], tokens[bad][:5], kept[bad][:5])
    fine = np.isfinite(logprobs)
    assert np.array_equal(shares[~fine], logprobs[~fine])
    assert (np.abs(shares - np.where(fine, logprobs, 0))[fine] <= 2.0**-24 * np.abs(logprobs[fine]) + 2.0**-40).all()
    return got, kept


def options(rng, rows, mode):
    """As float32 and int32 values, so that both sides take the same."""
    f = lambda lo, hi: rng.uniform(lo, hi, rows).astype(np.float32)  # noqa: E731
    some = rng.random((3, rows)) < 0.7
    o = {}
    if mode != "none":
        o["temperature"] = f(0.3, 1.5)
    if mode in ("top_k", "all"):
        o["top_k"] = np.where(some[0], np.exp(rng.uniform(0, 7, rows)), rng.integers(-1, 1, rows)).astype(np.int32)
    if mode in ("top_p", "all"):
        o["top_p"] = np.where(some[1], f(0.1, 0.999), np.float32(1)).astype(np.float32)
    if mode in ("min_p", "all"):
        o["min_p"] = np.where(some[2], f(0.001, 0.3), np.float32(0)).astype(np.float32)
    return o


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("mode", ["none", "temperature", "top_k", "top_p", "min_p", "all"])
@pytest.mark.parametrize("rows, vocab, spread", [(5, 1, 1.0), (7, 2, 1.0), (9, 7, 2.0), (3, 64, 4.0), (8, 511, 2.0), (4, 4096, 0.5), (6, 4097, 4.0), (3, 8193, 8.0),
                                                 (12, 20_003, 1.0), (5, 50_257, 4.0), (3, 100_257, 2.0), (2, 262_144, 4.0), (2, 262_147, 0.3)])
def test_draws(dtype, mode, rows, vocab, spread):
    rng = np.random.default_rng(rows * vocab)
    wide = torch.from_numpy(rng.normal(0, spread, (rows, vocab + 3)).astype(np.float32)).cuda().to(dtype)
    check(wide[:, :vocab], rng.random(rows), **options(rng, rows, mode))


@pytest.mark.parametrize("dtype", TYPES)
def test_many_draws_of_one_row(dtype):
    """Random numbers over the whole range, the same logits for all rows (stride 0): every kept token is drawn."""
    rng = np.random.default_rng(1)
    row = torch.from_numpy(rng.normal(0, 1.5, 300).astype(np.float32)).cuda().to(dtype)
    rows = 2000
    logits, u = row.expand(rows, 300), (np.arange(rows) + 0.5) / rows
    assert logits.stride(0) == 0
    for o in (dict(), dict(top_k=np.full(rows, 13)), dict(top_p=np.full(rows, np.float32(0.7))), dict(min_p=np.full(rows, np.float32(0.2)))):
        got, kept = check(logits, u, **o)
        if o:
            assert len(set(got.tolist())) == kept[0]


def test_rows_that_leave_little():
    rng = np.random.default_rng(2)
    rows, vocab = 40, 30_000
    x = rng.normal(0, 3, (rows, vocab)).astype(np.float32)
    x[rng.random((rows, vocab)) < 0.9] = -np.inf
    x[3] = -np.inf
    x[4] = -np.inf
    x[4, 29_999] = -5.0
    x[5] = np.nan
    x[6, 0:15_000] = np.nan
    x[7] = np.finfo(np.float32).min
    x[8, 11] = np.finfo(np.float32).max
    x[9] = np.where(x[9] == -np.inf, np.finfo(np.float32).min, x[9])
    x[10] = -np.inf
    x[10, [5, 20_000, 25_000]] = -1e30, -1e30, -2e30
    for mode in ("none", "temperature", "top_k", "top_p", "min_p", "all"):
        got, _ = check(torch.from_numpy(x).cuda(), rng.random(rows), **options(rng, rows, mode))
        assert got[3] == got[5] == -1 and got[4] == 29_999


def test_infinite_logits():
    x = torch.zeros(3, 500, device="cuda")
    x[0, [7, 300, 499]] = math.inf
    x[1] = math.inf
    x[2, 3] = math.inf
    x[2, 4:] = -math.inf
    for u in (0.0, 0.3, 0.5, 0.99):
        check(x, [u] * 3)
        check(x, [u] * 3, top_k=[2] * 3, temperature=np.float32([0.5, 2, 1e-3]))
        check(x, [u] * 3, top_p=np.float32([0.5, 0.25, 0.9]))
        check(x, [u] * 3, min_p=np.float32([0.5, 0.25, 0.9]))


@pytest.mark.parametrize("vocab", [10, 1000, 70_000])
def test_ties(vocab):
    """Equal logits go by their ids, also where a limit cuts through them."""
    rows = 60
    rng = np.random.default_rng(vocab)
    u = rng.random(rows)
    flat = torch.zeros(1, vocab, device="cuda").expand(rows, vocab)
    check(flat, u)
    check(flat, u, top_k=rng.integers(1, vocab + 2, rows))
    check(flat, u, top_p=np.float32(rng.integers(1, 8, rows) / 8))
    check(flat, u, top_k=rng.integers(1, vocab + 2, rows), top_p=np.float32(rng.integers(1, 8, rows) / 8))
    check(flat, u, min_p=np.full(rows, np.float32(1)))
    steps = torch.from_numpy(rng.integers(-2, 3, (rows, vocab)).astype(np.float32)).cuda().half()
    check(steps, u, top_k=rng.integers(1, vocab + 2, rows))
    check(steps, u, top_p=np.float32(rng.uniform(0.05, 1, rows)))
    check(steps, u, top_k=rng.integers(1, vocab + 2, rows), top_p=np.float32(rng.uniform(0.05, 1, rows)), min_p=np.float32(rng.uniform(0, 0.2, rows)))
    zeros = torch.zeros(rows, vocab, device="cuda")
    zeros[:, ::2] = -0.0  # equal to 0
    check(zeros, u, top_k=rng.integers(1, vocab + 2, rows))


def test_the_likeliest():
    rng = np.random.default_rng(5)
    x = torch.from_numpy(rng.integers(-5, 6, (50, 9000)).astype(np.float32)).cuda()
    first = [int(np.argmax(r)) for r in x.cpu().numpy()]
    u = rng.random(50)
    for o in (dict(temperature=np.zeros(50)), dict(temperature=np.full(50, -1.0)), dict(top_k=np.ones(50)), dict(top_p=np.zeros(50)), dict(min_p=np.full(50, 2.0)),
              dict(temperature=np.full(50, np.nan))):
        kinds = dict(top_k=np.int32)
        got, shares = tt.sample_tokens(x, torch.from_numpy(u.astype(np.float32)).cuda(), logprobs=True,
                                       **{k: torch.from_numpy(v.astype(kinds.get(k, np.float32))).cuda() for k, v in o.items()})
        assert got.tolist() == first and (shares == 0).all()


def test_temperatures_of_all_sizes():
    rng = np.random.default_rng(6)
    t = np.float32([1e-45, 1e-38, 1e-6, 0.01, 0.1, 10, 1e6, 1e30, np.inf])
    x = rng.normal(0, 4, (len(t), 5000)).astype(np.float32)
    x[:, 70] = -np.inf
    for o in (dict(), dict(top_k=np.full(len(t), 100)), dict(top_p=np.full(len(t), np.float32(0.9))), dict(min_p=np.full(len(t), np.float32(0.01)))):
        check(torch.from_numpy(x).cuda(), rng.random(len(t)), temperature=t, **o)


def test_random_numbers_at_the_ends():
    x = torch.from_numpy(np.random.default_rng(7).normal(0, 4, (1, 3000)).astype(np.float32)).cuda()
    u = np.float32([0, 2.0**-24, 1 - 2.0**-24, 1, 5, -1, np.nan, np.inf, -np.inf, 1e-45])
    check(x.expand(len(u), 3000), u)
    check(x.expand(len(u), 3000), u, top_k=np.full(len(u), 20))
    deep = torch.full((len(u), 3000), -700.0, device="cuda")  # the first tokens weigh next to nothing
    deep[:, 1000:] = 0
    check(deep, u)


def test_limits_that_limit_nothing():
    rng = np.random.default_rng(8)
    x = torch.from_numpy(rng.normal(0, 4, (6, 3000)).astype(np.float32)).cuda()
    u = rng.random(6)
    want = check(x, u)[0]
    nan = np.full(6, np.nan)
    for o in (dict(top_k=np.int32([0, -1, -2**31, 3000, 3001, 2**31 - 1])), dict(top_p=np.float32([1, 1.5, np.inf, 1, 1, 1])), dict(min_p=np.float32([0, -1, -np.inf, 0, 0, 0])),
              dict(top_p=nan), dict(min_p=nan)):
        assert check(x, u, **o)[0].tolist() == want.tolist()


def test_alignment_and_what_lies_beside():
    rng = np.random.default_rng(9)
    for dtype in TYPES:
        pool = torch.from_numpy(rng.normal(0, 4, 1 + 5 * 4099).astype(np.float32)).cuda().to(dtype)
        logits = pool[1:].view(5, 4099)[:, 3:4000]
        u = torch.from_numpy(rng.random(5).astype(np.float32)).cuda()
        tokens, shares = torch.full((9,), -7, dtype=torch.int32, device="cuda"), torch.full((9,), 7.0, device="cuda")
        tt.sample_tokens_into(logits, u, tokens[2:7], logprobs=shares[2:7])
        want = so.sample(logits.double().cpu().numpy(), u.cpu().numpy())[0]
        assert tokens.tolist() == [-7, -7] + want.tolist() + [-7, -7]
        assert shares[[0, 1, 7, 8]].tolist() == [7.0] * 4


def test_large_vocabularies():
    """2^24 ids, flat and steep."""
    g = torch.Generator("cuda").manual_seed(3)
    x = torch.randn(1, 1 << 24, device="cuda", generator=g)
    for spread, o in ((1.0, dict()), (4.0, dict(top_p=np.float32([0.95]))), (0.1, dict(top_k=np.int32([5_000_000]))), (2.0, dict(top_p=np.float32([0.5]), min_p=np.float32([0.01])))):
        check(x * spread, [0.37], **o)


def test_no_rows_and_no_tokens():
    none = tt.sample_tokens(torch.empty(0, 50, device="cuda"), torch.empty(0, device="cuda"))
    assert none.shape == (0,)
    got, shares = tt.sample_tokens(torch.empty(3, 0, device="cuda"), torch.rand(3, device="cuda"), logprobs=True)
    assert got.tolist() == [-1] * 3 and (shares == -math.inf).all()


def test_the_same_twice():
    g = torch.Generator("cuda").manual_seed(4)
    x, u = torch.randn(30, 60_000, device="cuda", generator=g), torch.rand(30, device="cuda", generator=g)
    o = dict(top_p=torch.full((30,), 0.97, device="cuda"), top_k=torch.full((30,), 30_000, dtype=torch.int32, device="cuda"))
    first = tt.sample_tokens(x, u, logprobs=True, **o)
    for _ in range(5):
        again = tt.sample_tokens(x, u, logprobs=True, **o)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("step", [0.0, 0.03125, 0.5])
def test_lists_that_top_k_cuts_down(dtype, step):
    """Limits of some hundred tokens in rows of which more are listed; many equal logits at the limit, fewer and more than a workgroup sorts; rows that
    are listed whole, with NaN and -infinity among what top_k takes."""
    rng, g = np.random.default_rng(11), torch.Generator("cuda").manual_seed(12)
    for vocab in (3000, 70_000):
        logits = torch.randn(12, vocab, device="cuda", generator=g).mul_(2)
        if step:
            logits = (logits / step).round_() * step
        if vocab == 3000:
            logits[3:6, 200:] = -float("inf")
            logits[6:9, 500:] = float("nan")
        k = rng.integers(257, 1100, 12)
        for o in (dict(), dict(top_p=rng.uniform(0.8, 0.999, 12).astype(np.float32)), dict(min_p=np.full(12, 1e-3, np.float32)),
                  dict(top_p=rng.uniform(0.8, 0.999, 12).astype(np.float32), min_p=np.full(12, 1e-4, np.float32), temperature=rng.uniform(0.5, 2, 12).astype(np.float32))):
            check(logits.to(dtype), rng.random(12, dtype=np.float32), top_k=k, **o)


def test_more_rows_gone_over_again_than_slots():
    """Flat rows, whose nuclei are far below the lists: which of them find a slot depends on the order of workgroups, the answers do not."""
    g = torch.Generator("cuda").manual_seed(9)
    logits = torch.randn(700, 6000, device="cuda", generator=g).mul_(0.3)
    u = torch.rand(700, device="cuda", generator=g)
    o = dict(top_p=torch.full((700,), 0.9, device="cuda"))
    check(logits[:40], u[:40].cpu().numpy(), top_p=np.full(40, 0.9, np.float32))
    first = tt.sample_tokens(logits, u, logprobs=True, **o)
    single = [tt.sample_tokens(logits[i:i + 100], u[i:i + 100], logprobs=True, top_p=o["top_p"][:100]) for i in range(0, 700, 100)]
    shares = torch.cat([s[1] for s in single])
    assert torch.equal(first[0], torch.cat([s[0] for s in single])) and ((first[1] - shares).abs() <= 2.0**-23 * shares.abs()).all()
    for _ in range(5):
        again = tt.sample_tokens(logits, u, logprobs=True, **o)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_refuses():
    x, u, tokens = torch.zeros(3, 50, device="cuda"), torch.zeros(3, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    bad = [dict(logits=x.double()), dict(logits=x.int()), dict(logits=x[0]), dict(logits=x.t()), dict(uniform=u[:2]), dict(uniform=u.double()), dict(uniform=u.cpu()),
           dict(tokens=tokens[:2]), dict(tokens=tokens.long()), dict(tokens=None), dict(uniform=None), dict(temperature=u[:1]), dict(temperature=u.half()),
           dict(top_k=u), dict(top_k=tokens.long()), dict(top_p=tokens), dict(min_p=u[:2]), dict(logprobs=u.double()), dict(logprobs=u[:1])]
    for change in bad:
        with pytest.raises(ValueError):
            tt.sample_tokens_into(**dict(dict(logits=x, uniform=u, tokens=tokens), **change))
