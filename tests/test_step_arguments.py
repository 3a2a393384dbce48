"""Calls of a step that make their results or workspaces refuse what is no tensor, or one of other dimensions, as the *_into calls do (no GPU needed)."""
import pytest

torch = pytest.importorskip("torch")

import exact_byte_level_amd as tt  # noqa: E402

X = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
CACHE = torch.zeros(3, 16, 2, 64, dtype=torch.bfloat16)


@pytest.mark.parametrize("query, key_cache", [(None, CACHE), ([1.0], CACHE), (X[0], CACHE), (X[0, 0, 0], CACHE), (X, None), (X, CACHE[0]), (X, "cache")])
def test_attend_refuses(query, key_cache):
    with pytest.raises(ValueError, match="is needed"):
        tt.attend_workspace(query, key_cache)
    table, lengths = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for lse in (False, True):
        with pytest.raises(ValueError):
            tt.attend_cache(query, key_cache, CACHE, table, lengths, lse=lse)


@pytest.mark.parametrize("logits", [None, [[1.0, 2.0]], X, X[0, 0], X[0, 0, 0], 3])
def test_sample_refuses(logits):
    with pytest.raises(ValueError, match="is needed"):
        tt.sample_workspace(logits)
    for logprobs in (False, True):
        with pytest.raises(ValueError, match="is needed"):
            tt.sample_tokens(logits, torch.zeros(2), logprobs=logprobs)


def test_host_tensors():
    with pytest.raises(ValueError, match="query is not on a GPU"):
        tt.attend_cache(X, CACHE, CACHE, torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="logits is not on a GPU"):
        tt.sample_tokens(torch.zeros(2, 9), torch.zeros(2))
