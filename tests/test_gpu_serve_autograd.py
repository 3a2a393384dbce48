"""Serving calls and autograd: results carry no gradient, and a tensor that a call wrote counts as modified."""
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


def test_a_gradient_that_needs_the_logits_from_before_raises():
    w = torch.randn(3, 40, device="cuda", requires_grad=True)
    logits = w.exp()  # its gradient is made from the result
    tt.shape_logits_into(logits, logits, temperature=torch.full((3,), 0.5, device="cuda"))
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        logits.sum().backward()
    logits = w.exp()
    out = tt.shape_logits(logits, temperature=torch.full((3,), 0.5, device="cuda"))
    assert not out.requires_grad
    logits.sum().backward()
    assert torch.equal(w.grad, logits.detach())


def test_what_is_written_counts_as_modified():
    i32 = dict(dtype=torch.int32, device="cuda")
    cache = tt.BlockTable(3, 4, 12, 16)
    slots, out_n = torch.empty(3, dtype=torch.int64, device="cuda"), torch.empty(1, dtype=torch.int64, device="cuda")
    positions, rows = torch.empty(3, **i32), torch.empty(3, **i32)
    written = [cache.table, cache.lengths, cache.n_free, slots, out_n, positions, rows]

    def versions(*tensors):
        return [t._version for t in tensors]

    before = versions(*written, cache.free_blocks)
    cache.plan_into(slots, out_n, positions=positions, rows=rows)
    assert versions(*written, cache.free_blocks) == [v + 1 for v in before[:-1]] + before[-1:]
    lengths, n_free = torch.empty_like(cache.lengths), torch.empty_like(cache.n_free)
    before = versions(cache.lengths, cache.n_free, lengths, n_free)
    tt.plan_blocks_into(cache.lengths, cache.table, cache.free_blocks, cache.n_free, 16, slots, out_n, out_lengths=lengths,
                        out_n_free=n_free)
    assert versions(cache.lengths, cache.n_free, lengths, n_free) == [before[0], before[1], before[2] + 1, before[3] + 1]
    done = torch.ones(3, dtype=torch.bool, device="cuda")
    written = [cache.lengths, cache.n_free, cache.free_blocks, out_n]
    before = versions(*written, cache.table, done)
    cache.release_into(done, out_n)
    assert versions(*written, cache.table, done) == [v + 1 for v in before[:4]] + before[4:]
    ids, bits = torch.arange(5, **i32), torch.empty((1, 2), **i32)
    tt.token_bits_into(ids, bits, 64)
    assert versions(ids, bits) == [0, 1]
    g, t = tt.Grammar(np.full((2, 256), 1)), tt.TokenStrings(np.arange(4), [0, 1, 4])
    states, out, bits = torch.zeros(2, **i32), torch.empty(2, **i32), torch.empty((2, 1), **i32)
    tt.grammar_bits_into(g, t, states, bits)
    tt.grammar_advance_into(g, t, states, states, out)
    assert versions(states, bits, out) == [0, 1, 1]
    tt.grammar_advance_into(g, t, states, out)
    assert versions(states, out) == [1, 1]


def test_tensors_of_inference_mode():
    """They have no versions."""
    with torch.inference_mode():
        x = torch.randn(2, 50, device="cuda")
        want = x * 2
        tt.shape_logits_into(x, x, temperature=torch.full((2,), 0.5, device="cuda"))
        assert torch.equal(x, want)
        cache = tt.BlockTable(2, 4, 8, 16)
        cache.plan(torch.tensor([0, 3, 20], device="cuda"))
        assert cache.lengths.tolist() == [3, 17]
    y = torch.randn(2, 50, device="cuda")
    with torch.inference_mode():
        tt.shape_logits_into(y, y, temperature=torch.full((2,), 0.5, device="cuda"))
    assert y._version == 1
