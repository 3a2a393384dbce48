"""Draws at temperatures so low that a step of float32 at the largest logit is a good part of what tells weights from zero, against the
definition in 64 bits: the same tokens, and the logarithms of their shares within half a step of 32 bits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from tests.test_gpu_step_sample import TYPES, check  # noqa: E402

TEMPERATURES = np.float32([1e-9, 3e-9, 1e-8, 1e-7, 3e-7, 1e-6, 1e-5, 1e-3])
TOPS = [14.0, 20.5, 25.0, 31.0, 40.0, 150.0, 1500.0, 5000.0, -25.0]


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab", [300, 5000, 70_000])
def test_the_likeliest_is_drawn(dtype, vocab):
    """The largest logit behind the first part, those one, two and so on steps of its type below it before and behind: at these temperatures they
    weigh anything from next to all of it to nothing."""
    rng = np.random.default_rng(vocab)
    rows = len(TEMPERATURES) * len(TOPS)
    temperature, top = np.repeat(TEMPERATURES, len(TOPS)), np.tile(np.float32(TOPS), len(TEMPERATURES))
    x = torch.from_numpy(top[:, None] - 1 - np.abs(rng.normal(0, 4, (rows, vocab))).astype(np.float32)).to(dtype)
    at = vocab * 3 // 4
    x[:, at] = torch.from_numpy(top).to(dtype)
    step = x[:, at]
    for k in range(1, 6):
        step = torch.nextafter(step, torch.full_like(step, -torch.inf)) if dtype == torch.float32 else below(step)
        x[:, (at + 7 * k * (-1)**k) % vocab] = step
    x[:, 5] = -torch.inf
    x = x.cuda()
    u = rng.random(rows).astype(np.float32)
    for o in (dict(), dict(top_p=np.full(rows, np.float32(0.9))), dict(min_p=np.full(rows, np.float32(0.01))), dict(top_k=np.full(rows, 3)),
              dict(top_k=np.full(rows, 40), top_p=np.full(rows, np.float32(0.999)), min_p=np.full(rows, np.float32(1e-6)))):
        check(x, u, temperature=temperature, **o)
        check(x, np.zeros(rows), temperature=temperature, **o)  # the first token that weighs anything


def below(x):
    """The next smaller number of 16 bits."""
    bits = x.view(torch.int16)
    return torch.where(bits < 0, bits + 1, bits - 1).view(x.dtype)
