"""What is not kept weighs nothing and is never drawn, also where the random number falls right between two kept tokens.

Rows hold the same logits twice, with tokens of no weight between, and are drawn at a half: half the sum of all is the sum of
the first ones, up to the last bits of the two, which depend on how they are added up.  So one of two tokens has to come: the last kept one
of the first half or the first kept one of the second.
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


def check(x, n, between, **o):
    rows = x.shape[0]
    tokens, shares = tt.sample_tokens(x, torch.full((rows,), 0.5, device="cuda"), logprobs=True, **{k: torch.full((rows,), v, device="cuda") for k, v in o.items()})
    bad = (tokens != n - 1) & (tokens != n + between)
    assert not bad.any(), (int(bad.sum()), tokens[bad][:5].tolist(), shares[bad][:5].tolist())
    assert torch.isfinite(shares).all()


@pytest.mark.parametrize("n, between", [(3, 1), (40, 30), (100, 200), (150, 70), (250, 11)])
def test_rows_that_are_sorted_whole(n, between):
    rng = np.random.default_rng(n)
    x = doubled(rng, 4000, n, between)
    for o in (dict(min_p=1e-30), dict(top_p=1 - 2.0**-24), dict(min_p=1e-30, temperature=0.7)):
        check(x, n, between, **o)


@pytest.mark.parametrize("n, between", [(400, 300), (700, 1600)])
def test_rows_that_are_listed_whole(n, between):
    check(doubled(np.random.default_rng(n), 2000, n, between), n, between, min_p=1e-30)


@pytest.mark.parametrize("n, between", [(1000, 2000), (5120, 5000), (20_000, 6000), (12_345, 9999)])
def test_parts_without_limits(n, between):
    check(doubled(np.random.default_rng(n), 1000, n, between), n, between)


def test_several_parts_a_thread():
    """Rows of more than 512 parts: a thread's own parts have some without weight among them."""
    n, rng = 2048 * 260 + 77, np.random.default_rng(1)
    for between in (2048 * 3, 2048 * 4 + 5, 2048 * 30 + 1):
        check(doubled(rng, 40, n, between), n, between)


@pytest.mark.parametrize("n, between", [(5000, 4000), (40_000, 20_000)])
def test_rows_that_are_gone_over_again(n, between):
    rng = np.random.default_rng(n)
    x = doubled(rng, 300, n, between) * 0.1
    for o in (dict(min_p=1e-30), dict(top_p=1 - 2.0**-24)):
        check(x, n, between, **o)
