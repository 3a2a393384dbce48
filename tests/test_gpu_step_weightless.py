"""What is not kept weighs nothing and is never drawn, also where the random number falls right between two kept tokens.

Rows hold the same logits twice, with tokens of no weight between, and are drawn at a half: half the sum of all is the sum of
the first ones, up to the last bits of the two, which depend on how they are added up.  So the token has to be one that is kept by the
definition, whose share of the running sum takes in a half.  A sum of up to 2^21 terms in 64 bits is off by 2^21 2^-53 = 2^-32 of it at the worst, and
each side has one; weights are off by less than 2^-44: together below 2^-30.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import exact_byte_level_amd as tt  # noqa: E402

INFINITY = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()


def doubled(rng, rows, n, between):
    """[rows, n + between + n]: logits, tokens that are never drawn, the same logits in another order."""
    x = torch.full((rows, 2 * n + between), -INFINITY)
    x[:, :n] = torch.from_numpy(rng.normal(0, 3, (rows, n)).astype(np.float32))
    x[:, n + between:] = x[:, :n][:, torch.from_numpy(rng.permutation(n))]
    return x.cuda()


def check(x, **o):
    rows = x.shape[0]
    tokens, shares = tt.sample_tokens(x, torch.full((rows,), 0.5, device="cuda"), logprobs=True, **{k: torch.full((rows,), v, device="cuda") for k, v in o.items()})
    value = {k: float(np.float32(v)) for k, v in o.items()}
    for r in range(0, rows, 500):
        y = x[r:r + 500].double()
        w = torch.exp((y - y.amax(1, keepdim=True)) / value.get("temperature", 1.0))
        falling, order = torch.sort(w, dim=1, descending=True, stable=True)
        sums = torch.cumsum(falling, 1)
        kept = torch.ones_like(falling, dtype=torch.bool)
        if "top_p" in o:
            kept = sums - falling < value["top_p"] * sums[:, -1:]
        if "min_p" in o:
            kept &= falling >= value["min_p"]
        w = torch.zeros_like(w).scatter_(1, order, torch.where(kept, falling, 0.0))
        sums, at = torch.cumsum(w, 1), tokens[r:r + 500, None].long()
        all_of, upto, own = sums[:, -1], sums.gather(1, at)[:, 0], w.gather(1, at)[:, 0]
        bad = (own == 0) | (upto < all_of * (0.5 - 2.0**-30)) | (upto - own > all_of * (0.5 + 2.0**-30))
        assert not bad.any(), (int(bad.sum()), tokens[r:r + 500][bad][:5].tolist(), shares[r:r + 500][bad][:5].tolist())
        assert ((shares[r:r + 500] - torch.log(own / all_of)).abs() <= 2.0**-23 * shares[r:r + 500].abs()).all()


@pytest.mark.parametrize("n, between", [(3, 1), (40, 30), (100, 200), (150, 70), (250, 11)])
def test_rows_that_are_sorted_whole(n, between):
    rng = np.random.default_rng(n)
    x = doubled(rng, 4000, n, between)
    for o in (dict(min_p=1e-30), dict(top_p=1 - 2.0**-24), dict(min_p=1e-30, temperature=0.7)):
        check(x, **o)


@pytest.mark.parametrize("n, between", [(400, 300), (700, 1600)])
def test_rows_that_are_listed_whole(n, between):
    check(doubled(np.random.default_rng(n), 2000, n, between), min_p=1e-30)


@pytest.mark.parametrize("n, between", [(1000, 2000), (5120, 5000), (20_000, 6000), (12_345, 9999)])
def test_parts_without_limits(n, between):
    check(doubled(np.random.default_rng(n), 1000, n, between))


def test_several_parts_a_thread():
    """Rows of more than 512 parts: a thread's own parts have some without weight among them."""
    n, rng = 2048 * 260 + 77, np.random.default_rng(1)
    for between in (2048 * 3, 2048 * 4 + 5, 2048 * 30 + 1):
        check(doubled(rng, 40, n, between))


@pytest.mark.parametrize("n, between", [(5000, 4000), (40_000, 20_000)])
def test_rows_that_are_gone_over_again(n, between):
    rng = np.random.default_rng(n)
    x = doubled(rng, 300, n, between) * 0.1
    for o in (dict(min_p=1e-30), dict(top_p=1 - 2.0**-24)):
        check(x, **o)
