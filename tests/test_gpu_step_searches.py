"""Draws that search a row several times, one search right behind the other: the limit among equal logits, the part of the row, the token in
it.  All logits are alike, so the answer is known: of k kept tokens the one whose number is the whole part of u k."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import exact_byte_level_amd as tt  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("vocab", [600, 4096, 4097, 50_257, 262_144, 600_001])
def test_searches_one_behind_the_other(vocab):
    """Rows whose last tile, or last part, is short: some wavefronts are through with a search long before others."""
    rows, rng = 300, np.random.default_rng(vocab)
    x = torch.zeros(1, vocab, device="cuda").expand(rows, vocab)
    u = rng.random(rows).astype(np.float32)
    k = rng.integers(2, vocab, rows).astype(np.int32)
    k[:20] = vocab - 1 - np.arange(20)
    p = rng.integers(1, 16, rows).astype(np.float32) / 16
    by_mass = np.ceil(p.astype(np.float64) * vocab).astype(np.int64)
    both = np.ceil(p.astype(np.float64) * k).astype(np.int64)
    on = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    for kept, o in ((k, dict(top_k=on(k))), (by_mass, dict(top_p=on(p))), (both, dict(top_k=on(k), top_p=on(p))), (np.full(rows, vocab), dict(min_p=on(np.ones(rows, np.float32))))):
        want = np.floor(u.astype(np.float64) * kept).astype(np.int64).tolist()
        shares = on((-np.log(kept.astype(np.float64))).astype(np.float32))
        for _ in range(4):
            got, logprobs = tt.sample_tokens(x, on(u), logprobs=True, **o)
            assert got.tolist() == want
            assert ((logprobs - shares).abs() <= 2.0**-23 * shares.abs() + 2.0**-149).all()
    assert math.isclose(float(logprobs[0]), -math.log(vocab), rel_tol=1e-6)
