"""The serving example end to end: every answer follows its grammar."""
import re

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from examples.serve_step import answer  # noqa: E402


def test_answers_follow_the_grammar():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    prompts = [b"one", b"two words", b"x", b"a longer prompt, of a few more tokens than the others have"] * 5
    for seed in range(3):
        answers, ended = answer(prompts, seed=seed)
        assert any(ended.tolist())
        for text, done in zip(answers, ended.tolist()):
            if done:
                assert re.fullmatch(rb"\[\d{1,3}(, \d{1,3})*\]", text), text
            else:  # cut off: the beginning of such a list
                assert re.fullmatch(rb"\[?(\d{1,3}(, \d{1,3})*(,( )?)?)?\]?", text), text
