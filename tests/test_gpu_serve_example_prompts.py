"""The serving example on prompts of any length."""
import re

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from examples.serve_step import answer  # noqa: E402

LIST = rb"\[?(\d{1,3}(, \d{1,3})*(,( )?)?)?\]?"


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()


def test_long_prompts():
    answers, _ = answer([b"short", b"one two three four five six seven eight nine ten " * 400])
    assert all(re.fullmatch(LIST, a) for a in answers)


def test_empty_prompts():
    """Beside others, whose texts do not change their answers, and by themselves."""
    got = [answer([before, b"", b"after"])[0][1] for before in (b"x", b"def f(n):", b"")]
    assert got[0] == got[1] == got[2] and all(re.fullmatch(LIST, a) for a in got)
    assert answer([b"", b""])[0][1] == answer([b"x", b""])[0][1]
