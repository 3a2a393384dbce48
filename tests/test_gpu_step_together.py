"""The operators around the model as a serving program runs them together: captured into graphs, on other streams, two calls at once, what autograd
sees, and a whole step from the plan to the drawn token, prompts first, against the definitions in 64 bits."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import exact_byte_level_amd as tt  # noqa: E402
from tests import step_oracle as so  # noqa: E402
from tests import serve_oracle  # noqa: E402
from tests.test_gpu_step_attend import host, make, near, near_sums  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()


def generator(seed):
    return torch.Generator("cuda").manual_seed(seed)


def test_a_step_from_plan_to_token():
    rows, kv, heads, dim, vocab, bs = 5, 2, 6, 64, 3001, 16
    g, rng = generator(1), np.random.default_rng(1)
    for dtype, scaled in ((torch.bfloat16, False), (torch.float8_e4m3fn, True)):
        table = tt.BlockTable(rows, width=20, blocks=rows * 20, block_size=bs)
        scale = [torch.tensor([0.5, 0.25], device="cuda") if scaled else None for _ in range(2)]
        layer = tt.KeyValueCache(table, kv, dim, dtype, key_scale=scale[0], value_scale=scale[1])
        kept = [[] for _ in range(rows)]  # keys and values of each row, as written
        new = np.array([30, 1, 0, 130, 17])
        offsets = torch.from_numpy(np.concatenate([[0], np.cumsum(new)])).cuda()
        slots, positions, row_of = table.plan(offsets)
        for step in range(4):
            n = slots.numel()
            k, v = (torch.randn(n, kv, dim, device="cuda", generator=g).bfloat16() for _ in range(2))
            q = torch.randn(n, heads, dim, device="cuda", generator=g).bfloat16()
            layer.write(k, v, slots)
            for i, r in enumerate(row_of.tolist()):
                if r >= 0:
                    kept[r].append((k[i].float(), v[i].float()))
            if step == 0:  # the prompts: every token sees those before it, and a plain attention says the same
                out, sums = layer.attend(q, positions + 1, row_of, lse=True)
                seen = (positions + 1).tolist()
            else:
                out, sums = layer.attend(q, lse=True)
                seen = table.lengths.tolist()
                assert layer.attend(q).equal(out)
            # by definition, over what was written, rounded as the cache rounds it
            back = torch.stack([layer.keys, layer.values]).float()
            for s, c in zip(scale, back):
                if s is not None:
                    c *= s[:, None]
            o = dict(table=table.table.cpu().numpy(), lengths=np.array(seen), rows=row_of.cpu().numpy(), scale=1 / 8)
            want, lse, slack, lse_slack = so.attend(host(q), host(back[0]), host(back[1]), **o)
            near(out, want, 1.02 * slack)
            near_sums(sums, lse, 1.02 * lse_slack)
            for r in range(rows):
                for p, (kk, vv) in enumerate(kept[r]):
                    b, at = int(table.table[r, p // bs]), p % bs
                    eps = 2.0**-4 if scaled else 0.0
                    for x, c in ((kk, back[0]), (vv, back[1])):
                        assert ((c[b, at] - x).abs() <= eps * x.abs() + (2.0**-10 * 0.5 if scaled else 0)).all()
            # the model's logits of the last tokens, shaped and drawn from
            logits = torch.randn(rows, vocab, device="cuda", generator=g).mul_(3).bfloat16()
            t, p = (torch.from_numpy(rng.uniform(0.4, 1, rows).astype(np.float32)).cuda() for _ in range(2))
            made = torch.randint(0, vocab, (rows, 9), device="cuda", generator=g).int()
            shaped = tt.shape_logits(logits, generated=made, repetition=torch.full((rows,), 1.3, device="cuda"), temperature=t)
            u = torch.rand(rows, device="cuda", generator=g)
            tokens, shares = tt.sample_tokens(shaped, u, logprobs=True, top_p=p)
            want, logprobs, _ = so.sample(host(shaped), u.cpu().numpy(), top_p=p.cpu().numpy())
            assert tokens.tolist() == want.tolist() and np.allclose(host(shares), logprobs, rtol=2.0**-23, atol=2.0**-40)
            plain, _ = serve_oracle.shape_logits(host(logits), generated=made.cpu().numpy(), repetition=np.full(rows, np.float32(1.3)), temperature=host(t))
            assert np.allclose(host(shaped), plain, rtol=1e-6)
            if step == 2:
                table.release(torch.arange(rows, device="cuda") == 3)
                kept[3] = []
            slots, positions, row_of = table.plan()
            assert table.lengths.tolist() == [-1 if step >= 2 and r == 3 else len(x) + 1 if len(x) else table.lengths[r].item() for r, x in enumerate(kept)]


def capture(f):
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        f()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f()
    return graph


@pytest.mark.parametrize("shared", [False, True])
def test_captured_and_replayed(shared):
    """One graph of all three calls (shared: several queries of a row), replayed on new inputs with eager work between."""
    rows = [2, 0, 2, 1, 2, 0] if shared else [2, 0, 1]
    lengths = [700, 12, 689, 129, 1, 300] if shared else [700, 12, 129]
    o = make(lengths, 6, 3, 64, 16, rows=rows, seed=3, garbage=0.25)
    n = len(rows)
    out, lse = torch.empty_like(o["query"]), torch.empty(n, 6, device="cuda")
    g = generator(5)
    k, v = (torch.empty(n, 3, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    slots = torch.zeros(n, dtype=torch.int64, device="cuda")
    logits, u = torch.empty(n, 70_001, device="cuda"), torch.empty(n, device="cuda")
    tokens, shares = torch.empty(n, dtype=torch.int32, device="cuda"), torch.empty(n, device="cuda")
    limits = dict(top_p=torch.full((n,), 0.9, device="cuda"), top_k=torch.zeros(n, dtype=torch.int32, device="cuda"), temperature=torch.ones(n, device="cuda"))
    spaces = tt.attend_workspace(o["query"], o["key_cache"]), tt.sample_workspace(logits)

    def step(out, lse, tokens, shares, spaces):
        tt.write_cache_into(k, v, slots, o["key_cache"], o["value_cache"])
        tt.attend_cache_into(**o, out=out, lse=lse, workspace=spaces[0])
        tt.sample_tokens_into(logits, u, tokens, logprobs=shares, workspace=spaces[1], **limits)

    def fill(i):
        for x in (k, v, o["query"]):
            x.copy_(torch.randn(x.shape, device="cuda", generator=g))
        logits.copy_(torch.randn(logits.shape, device="cuda", generator=g)).mul_((1.0, 4.0, 0.3, 2.0)[i])
        u.copy_(torch.rand(n, device="cuda", generator=g))
        held = o["table"][o["rows"].long()] if i else o["table"][:1].expand(n, -1)
        slots.copy_(held[:, 0].long() * 16 + torch.arange(n, device="cuda"))
        limits["top_k"].fill_((0, 30, 0, 5000)[i])

    fill(0)
    graph = capture(lambda: step(out, lse, tokens, shares, spaces))
    other = capture(lambda: step(out, lse, tokens, shares, spaces))  # shares the workspaces: replayed one after the other
    for i in range(4):
        fill(i)
        (graph if i % 2 else other).replay()
        got = [x.clone() for x in (out, lse, tokens, shares)]
        want = [torch.empty_like(x) for x in got]
        step(*want, (None, None))
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x, y), i
        graph.replay()
        other.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip((out, lse, tokens, shares), want))


def test_two_calls_at_once():
    """On two streams, with a workspace each."""
    streams = [torch.cuda.Stream() for _ in range(2)]
    o = [make([3000, 40, 900], 8, 2, 128, 16, seed=k, garbage=0.5) for k in range(2)]
    x = [torch.randn(40, 120_000, device="cuda", generator=generator(k)) for k in range(2)]
    u = torch.rand(40, device="cuda", generator=generator(9))
    p = torch.full((40,), 0.95, device="cuda")
    want = [(tt.attend_cache(**a), tt.sample_tokens(b, u, top_p=p)) for a, b in zip(o, x)]
    torch.cuda.synchronize()
    got = []
    for k in range(2):
        for _ in range(10):
            got.append((k, tt.attend_cache(**o[k], stream=streams[k]), tt.sample_tokens(x[k], u, top_p=p, stream=streams[k])))
            k = 1 - k
    torch.cuda.synchronize()
    for k, a, b in got:
        assert torch.equal(a, want[k][0]) and torch.equal(b, want[k][1])


def test_on_another_stream():
    """A call on a stream that is not the current one waits for what that stream was given before."""
    s = torch.cuda.Stream()
    cache = torch.zeros(40, 16, 1, 64, dtype=torch.bfloat16, device="cuda")
    x = torch.full((600, 1, 64), 2.0, dtype=torch.bfloat16, device="cuda")
    slots = torch.arange(600, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        big = torch.randn(3000, 3000, device="cuda")
        for _ in range(20):
            big = big @ big * 1e-2
        x.fill_(3.0)
    tt.write_cache_into(x, x, slots, cache, cache.clone(), stream=s)
    s.synchronize()
    assert (cache.view(-1, 64)[:600] == 3).all()


def test_what_is_written_counts_as_modified():
    o = make([20, 30], 2, 1, 64, 16, garbage=0.5)
    out, lse = torch.empty_like(o["query"]), torch.empty(2, 2, device="cuda")

    def versions(*tensors):
        return [t._version for t in tensors]

    before = versions(*o.values())
    tt.attend_cache_into(**o, out=out, lse=lse)
    assert versions(*o.values()) == before and versions(out, lse) == [1, 1]
    x = torch.ones(2, 1, 64, dtype=torch.bfloat16, device="cuda")
    slots = torch.zeros(2, dtype=torch.int64, device="cuda")
    slots[1] = 1
    before = versions(x, slots, o["key_cache"], o["value_cache"])
    tt.write_cache_into(x, x, slots, o["key_cache"], o["value_cache"])
    assert versions(x, slots, o["key_cache"], o["value_cache"]) == before[:2] + [before[2] + 1, before[3] + 1]
    logits, u = torch.randn(3, 50, device="cuda"), torch.rand(3, device="cuda")
    tokens, shares = torch.empty(3, dtype=torch.int32, device="cuda"), torch.empty(3, device="cuda")
    tt.sample_tokens_into(logits, u, tokens, logprobs=shares)
    assert versions(logits, u, tokens, shares) == [0, 0, 1, 1]
    w = torch.randn(2, 2, 64, device="cuda", requires_grad=True)
    assert not tt.attend_cache(**dict(o, query=w.bfloat16())).requires_grad
    with torch.inference_mode():
        y = tt.attend_cache(**o)
    assert y.shape == out.shape


def test_queries_of_a_row_with_windows_far_apart():
    """Bundles do not join queries that see no token in common; each sees its own window alone, in any order."""
    lengths = [3000, 10, 11, 12, 2990, 1500, 1490, 40, 41, 3001, 0, -1, 700, 17]
    rows = [0, 0, 0, 1, 0, 0, 0, 1, 1, 0, 1, 0, 1, 0]
    for heads, kv in ((2, 2), (8, 1), (6, 2), (9, 1)):
        o = make(lengths, heads, kv, 64, 24, rows=rows, seed=heads, garbage=0.5)
        plain = {k: v.cpu().numpy() for k, v in o.items() if k not in ("query", "key_cache", "value_cache")}
        for window in (0, 1, 16, 100, 2000):
            want, lse, slack, lse_slack = so.attend(host(o["query"]), host(o["key_cache"]), host(o["value_cache"]), **plain, scale=0.125, window=window)
            out, sums = tt.attend_cache(**o, scale=0.125, window=window, lse=True)
            near(out, want, slack)
            near_sums(sums, lse, lse_slack)


def test_many_queries_of_few_rows():
    rng = np.random.default_rng(8)
    for n, n_rows in ((512, 1), (512, 511), (100, 3), (17, 16)):
        rows = rng.integers(0, n_rows, n)
        rows[:2] = n_rows - 1, 0
        o = make(rng.integers(0, 150, n), 2, 1, 8, 16, rows=rows, seed=n_rows, garbage=0.5)
        plain = {k: v.cpu().numpy() for k, v in o.items() if k not in ("query", "key_cache", "value_cache")}
        want, lse, slack, lse_slack = so.attend(host(o["query"]), host(o["key_cache"]), host(o["value_cache"]), **plain, scale=0.3)
        out, sums = tt.attend_cache(**o, scale=0.3, lse=True)
        near(out, want, slack)
        near_sums(sums, lse, lse_slack)


def test_sampled_shares():
    """Many draws by evenly spread numbers come out as the shares say: every token as often as its weight, to one draw."""
    n = 4000
    x = torch.tensor([math.log(w) for w in (5, 1, 3, 0.5, 0.5)], device="cuda").expand(n, 5)
    u = (torch.arange(n, device="cuda") + 0.5) / n
    tokens, shares = tt.sample_tokens(x, u, logprobs=True)
    count = torch.bincount(tokens, minlength=5).tolist()
    assert all(abs(c - n * w / 10) <= 1 for c, w in zip(count, (5, 1, 3, 0.5, 0.5)))
    assert torch.allclose(shares.exp(), torch.tensor([0.5, 0.1, 0.3, 0.05, 0.05], device="cuda")[tokens.long()], rtol=1e-6)
