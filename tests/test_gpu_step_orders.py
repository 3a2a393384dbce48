"""Draws from rows whose likely tokens lie beside each other, as in vocabularies that are ordered by frequency and under grammars that allow a range of ids,
and from more rows than one launch takes."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import exact_byte_level_amd as tt  # noqa: E402
from tests.test_gpu_step_sample import TYPES, check  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()


def limits(rng, rows):
    f = lambda lo, hi: rng.uniform(lo, hi, rows).astype(np.float32)  # noqa: E731
    return (dict(), dict(top_k=np.full(rows, 50)), dict(top_k=rng.integers(1, 3000, rows)), dict(top_p=f(0.3, 0.999)), dict(min_p=f(1e-4, 0.1)),
            dict(top_k=np.full(rows, 50), top_p=f(0.3, 0.999)), dict(top_k=rng.integers(1, 3000, rows), top_p=f(0.3, 0.999), min_p=f(1e-5, 0.05), temperature=f(0.5, 1.5)))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("fall, spread", [(0.5, 2.5), (1.0, 2.0), (2.0, 0.5)])
@pytest.mark.parametrize("vocab, rows", [(3000, 9), (50_257, 5), (128_256, 3)])
def test_logits_that_fall_with_the_id(dtype, fall, spread, vocab, rows):
    rng = np.random.default_rng(vocab)
    x = rng.normal(0, spread, (rows, vocab)) - fall * np.log(np.arange(vocab) + 10)
    for o in limits(rng, rows):
        check(torch.from_numpy(x.astype(np.float32)).cuda().to(dtype), rng.random(rows), **o)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab, first, n", [(50_257, 512, 512), (50_257, 49_900, 357), (100_257, 0, 300), (128_256, 70_000, 1500), (262_144, 2047, 2), (4000, 100, 700)])
def test_all_likely_tokens_in_one_run_of_ids(dtype, vocab, first, n):
    rng = np.random.default_rng(vocab + first)
    rows = 4
    x = rng.normal(0, 1, (rows, vocab)) - 12
    x[:, first:first + n] = rng.normal(0, 2, (rows, n))
    x[1, np.r_[:first, first + n:vocab]] = -np.inf
    for o in limits(rng, rows):
        check(torch.from_numpy(x.astype(np.float32)).cuda().to(dtype), rng.random(rows), **o)


@pytest.mark.parametrize("rows, vocab", [(70_000, 60), (23_000, 6000)])
def test_more_rows_than_a_launch_takes(rows, vocab):
    """Each launch takes up where the last one ended, with a workspace that it left."""
    rng, g = np.random.default_rng(rows), torch.Generator("cuda").manual_seed(rows)
    x = torch.randn(rows, vocab, device="cuda", generator=g, dtype=torch.float16).mul_(2)
    u = rng.random(rows).astype(np.float32)
    o = dict(top_k=rng.integers(0, 900, rows).astype(np.int32), top_p=rng.uniform(0.3, 1.1, rows).astype(np.float32), min_p=rng.uniform(-0.01, 0.02, rows).astype(np.float32))
    on = {k: torch.from_numpy(v).cuda() for k, v in o.items()}
    tokens, shares = tt.sample_tokens(x, torch.from_numpy(u).cuda(), logprobs=True, **on)
    for some in (slice(0, 30), slice(rows // 2, rows // 2 + 30), slice(rows - 30, rows)):
        assert check(x[some], u[some], **{k: v[some] for k, v in o.items()})[0].tolist() == tokens[some].tolist()
    for r in range(0, rows, 5000):
        some = slice(r, r + 5000)
        got, logprobs = tt.sample_tokens(x[some], torch.from_numpy(u[some]).cuda(), logprobs=True, **{k: v[some] for k, v in on.items()})
        # sums over parts of other sizes: their last bits of 64, so at most the rounding to 32 bits differs
        assert got.equal(tokens[some]) and ((logprobs - shares[some]).abs() <= 2.0**-22 * shares[some].abs()).all()
