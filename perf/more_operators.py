"""What the operators around the model in a serving step are measured on: keys and values written to a paged cache, the
attention of new tokens over it, and the choice of the next token.

Cases, their inputs, one pass through an operator (in plain torch operations, or through the package's
entry points where ``own`` is true), its least bytes and operations, and its values by definition in 64 bits.

A cache is [blocks, block_size, heads, dim]; token p of a request whose row of the table is r lives in block
``table[r, p // block_size]`` at place ``p % block_size``, and slot s is place s % block_size of block s // block_size.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
SIZES = {"f32": 4, "f16": 2, "bf16": 2, "e4m3": 1}
MOST = 448.0  # the largest e4m3 value


# ---------------------------------------------------------------- cases

def listed():
    return [
        # the new tokens of a few requests, one each, some rows idle
        dict(name="write_step", op="write", tokens=8, heads=8, dim=128, block=16, src="bf16", dst="bf16", by_head=False, idle=0.25),
        # the next parts of many prompts into a cache of 8 bits; the launch's last places hold no token
        dict(name="write_prompts", op="write", tokens=48_000, heads=8, dim=128, block=16, src="bf16", dst="e4m3", by_head=False, idle=0.01),
        # one request's step, where the latency counts
        dict(name="attend_one", op="attend", queries=1, rows=1, context=4000, heads=32, kv=8, dim=128, block=16, src="bf16", dst="bf16",
             by_head=False, window=0, softcap=0.0, spread=0.0),
        # a small serving batch of long and short requests, blocks laid out by heads
        dict(name="attend_step", op="attend", queries=9, rows=9, context=9000, heads=28, kv=4, dim=128, block=64, src="f16", dst="f16",
             by_head=True, window=0, softcap=0.0, spread=0.7),
        # a full serving batch
        dict(name="attend_batch", op="attend", queries=64, rows=64, context=32_000, heads=64, kv=8, dim=128, block=16, src="bf16", dst="bf16",
             by_head=False, window=0, softcap=0.0, spread=0.7),
        # two very long texts over a cache of 8 bits, every query head on one head of keys
        dict(name="attend_long", op="attend", queries=2, rows=2, context=400_001, heads=16, kv=1, dim=128, block=128, src="bf16", dst="e4m3",
             by_head=False, window=0, softcap=0.0, spread=0.0),
        # a step that mixes prompts' last parts and single tokens: several tokens of a row, a window, capped scores, odd blocks
        dict(name="attend_mixed", op="attend", queries=301, rows=40, context=6001, heads=12, kv=12, dim=64, block=24, src="f16", dst="f16",
             by_head=False, window=1024, softcap=30.0, spread=0.7),
        # wide heads
        dict(name="attend_wide", op="attend", queries=33, rows=33, context=8000, heads=16, kv=4, dim=256, block=32, src="bf16", dst="bf16",
             by_head=False, window=0, softcap=50.0, spread=0.7),
        # the next token of one request, by its nucleus
        dict(name="sample_one", op="sample", rows=1, vocab=50_256, pad=0, src="f32", spread=4.0, mode="top_p", masked=0.0),
        # a serving batch with everything in use, some rows under a grammar
        dict(name="sample_batch", op="sample", rows=61, vocab=100_257, pad=7, src="f16", spread=4.0, mode="all", masked=0.3),
        # a large batch by temperature alone, and one with everything in 32 bits
        dict(name="sample_warm", op="sample", rows=192, vocab=100_256, pad=0, src="bf16", spread=2.0, mode="none", masked=0.0),
        dict(name="sample_large", op="sample", rows=256, vocab=262_144, pad=0, src="f32", spread=4.0, mode="all", masked=0.1),
    ]


def draw(rng):
    def near(lo, hi):  # whole numbers spread over their logarithm, odd ones among them
        return int(round(lo * (hi / lo) ** rng.random()))

    op = rng.choice(["write", "attend", "attend", "attend", "sample", "sample"])
    block = rng.choice([16, 32, 64, 128, near(8, 300)])
    if op == "write":
        src = rng.choice(["f32", "f16", "bf16"])
        return dict(op=op, tokens=near(1, 20_000), heads=rng.choice([1, 2, 4, 8, near(1, 16)]), dim=rng.choice([64, 128, 256, 8 * near(2, 32)]), block=block,
                    src=src, dst=rng.choice(["e4m3", "bf16" if src == "f32" else src]), by_head=rng.random() < 0.3, idle=round(0.3 * rng.random(), 2))
    if op == "attend":
        src = rng.choice(["f16", "bf16"])
        kv, dim = rng.choice([1, 2, 4, 8, near(1, 16)]), rng.choice([64, 128, 256, 8 * near(2, 32)])
        heads = kv * rng.choice([1, 2, 4, 8, near(1, 24)])
        context = near(1, 100_000)
        # as many queries as keep to the largest listed case's keys and values
        rows = near(1, max(1, min(300, 64 * 16_000 * 8 * 128 // (context * kv * dim), 32 * 16_000 * 64 // (context * heads))))
        return dict(op=op, queries=rows if rng.random() < 0.7 else rows + near(1, rows), rows=rows, context=context, heads=heads, kv=kv, dim=dim, block=block, src=src,
                    dst=rng.choice([src, src, "e4m3"]), by_head=rng.random() < 0.3, window=rng.choice([0, 0, near(1, 8000)]),
                    softcap=rng.choice([0.0, 0.0, 30.0]), spread=rng.choice([0.0, 0.7]))
    return dict(op=op, rows=near(1, 250), vocab=near(300, 260_000), pad=rng.choice([0, near(1, 64)]), src=rng.choice(["f32", "f16", "bf16"]),
                spread=rng.choice([1.0, 2.0, 4.0, 8.0]), mode=rng.choice(["none", "top_k", "top_p", "min_p", "all", "all"]), masked=rng.choice([0.0, 0.3]))


# ---------------------------------------------------------------- inputs

def generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def normal(shape, g, dtype, by=1.0):
    """Normal numbers of 16 bits, or e4m3 by way of them."""
    x = torch.randn(shape, device="cuda", generator=g, dtype=torch.float32 if dtype == torch.float32 else torch.bfloat16 if dtype == torch.bfloat16 else torch.float16)
    return x.mul_(by).to(dtype)


def new_cache(case, blocks, g):
    """Keys and values, each [blocks, block, heads, dim]; by_head: with all places of a head of a block one behind the other."""
    heads = case.get("kv", case["heads"])
    shape = (blocks, heads, case["block"], case["dim"]) if case["by_head"] else (blocks, case["block"], heads, case["dim"])
    both = [normal(shape, g, DTYPES[case["dst"]]) for _ in range(2)]
    return [c.transpose(1, 2) for c in both] if case["by_head"] else both


def scales(case, heads, rng):
    """What a cache of 8 bits is scaled by, a factor for each head."""
    if case["dst"] != "e4m3":
        return None, None
    return dev(rng.uniform(0.02, 0.06, heads).astype(np.float32)), dev(rng.uniform(0.02, 0.06, heads).astype(np.float32))


def lengths_of(case):
    """Sorted lengths: log-normal with `spread`, capped at the context, their sum the case's own; with spread a tenth of the rows is not in use."""
    rows, context = case["rows"], case["context"]
    if not case["spread"]:
        return np.full(rows, context, np.int64)
    at = (np.arange(rows) + 0.5) / rows
    # the normal distribution's quantiles, by its logistic approximation
    length = np.maximum(1, np.minimum(context, np.floor(context * np.exp(case["spread"] * np.log(at / (1 - at)) / 1.702 - 0.5)))).astype(np.int64)
    length[:rows // 10] = -1
    return length


def queries_of(case):
    """The sorted lengths' rows and how many places before its row's end each query stands."""
    extra = case["queries"] - case["rows"]
    row = np.concatenate([np.arange(case["rows"]), case["rows"] - 1 - np.arange(extra) // 32 % case["rows"]])  # up to 32 more tokens of the longest rows
    back = np.concatenate([np.zeros(case["rows"], np.int64), 1 + np.arange(extra) % 32 + 32 * (np.arange(extra) // (32 * case["rows"]))])
    return row, back


def seen_of(case):
    """How many tokens each query sees, by the sorted rows."""
    row, back = queries_of(case)
    length = lengths_of(case)[row]
    return np.where(length < 0, -1, np.maximum(length - back, 0))


def prepare(case, seed):
    rng, g = np.random.default_rng(seed), generator(seed)
    return {"write": prepare_write, "attend": prepare_attend, "sample": prepare_sample}[case["op"]](case, rng, g)


def prepare_write(case, rng, g):
    n, heads, dim, bs = case["tokens"], case["heads"], case["dim"], case["block"]
    blocks = -(-n // bs) + max(8, n // bs // 4)
    keys, values = new_cache(case, blocks, g)
    ks, vs = scales(case, heads, rng)
    # keys and values as a projection leaves them: beside each other
    made = normal((n, 2, heads, dim), g, DTYPES[case["src"]], 3.0)
    slots = torch.randperm(blocks * bs, device="cuda", generator=g)[:n] if n < bs else (
        torch.randperm(blocks, device="cuda", generator=g)[:-(-n // bs), None] * bs + torch.arange(bs, device="cuda")).reshape(-1)[:n].contiguous()
    slots[torch.rand(n, device="cuda", generator=g) < case["idle"]] = -1
    return dict(op="write", keys=made[:, 0], values=made[:, 1], slots=slots, key_cache=keys, value_cache=values, key_scale=ks, value_scale=vs)


def prepare_attend(case, rng, g):
    rows, bs, kv, dim = case["rows"], case["block"], case["kv"], case["dim"]
    order = rng.permutation(rows)  # row r has the order[r]-th length
    place = np.argsort(order)
    row, _ = queries_of(case)
    mix = rng.permutation(case["queries"])
    length, seen = lengths_of(case)[order], seen_of(case)[mix]
    held = -(-np.maximum(length, 0) // bs)
    blocks = int(held.sum()) + 4
    keys, values = new_cache(case, blocks, g)
    ks, vs = scales(case, kv, rng)
    ids = torch.randperm(blocks, device="cuda", generator=g).to(torch.int32)
    width = -(-case["context"] // bs) + 1
    at = torch.arange(width, device="cuda")
    first = dev(np.concatenate([[0], np.cumsum(held)[:-1]]))
    taken = at < dev(held)[:, None]
    table = torch.where(taken, ids[torch.where(taken, first[:, None] + at, 0)], -1)
    # a new block holds anything behind the row's last token
    ends = np.flatnonzero((length > 0) & (length % bs != 0))
    if len(ends):
        last, inside = table[dev(ends), dev(length[ends] // bs)].long(), dev(length[ends] % bs)
        keys[last, inside], values[last, inside] = float("nan"), float("nan")
    # queries as they are after their norm: as long as the scores of a trained model need
    query = normal((case["queries"], case["heads"], dim), g, DTYPES[case["src"]], 1.5)
    s = dict(op="attend", query=query, key_cache=keys, value_cache=values, table=table, lengths=dev(seen.astype(np.int32)), rows=None,
             scale=1 / math.sqrt(dim) / (0.04 if ks is not None else 1.0), window=case["window"], softcap=case["softcap"], key_scale=ks, value_scale=vs,
             out=torch.empty_like(query), lse=torch.empty((case["queries"], case["heads"]), device="cuda"))
    s["rows"] = dev(place[row[mix]].astype(np.int32))
    if own:
        import exact_byte_level_amd as tt
        s["workspace"] = tt.attend_workspace(query, keys)
    return s


def prepare_sample(case, rng, g):
    rows, vocab = case["rows"], case["vocab"]
    wide = torch.randn((rows, vocab + case["pad"]), device="cuda", generator=g).mul_(case["spread"])
    under = dev(rng.random(rows) < case["masked"])  # rows under a grammar: most tokens are not allowed
    if case["masked"]:
        allowed = torch.rand((rows, 1), device="cuda", generator=g) ** 4
        wide.masked_fill_(under[:, None] & (torch.rand(wide.shape, device="cuda", generator=g) > allowed), float("-inf"))
    mode = case["mode"]
    some = lambda lo, hi: rng.uniform(lo, hi, rows).astype(np.float32)  # noqa: E731
    off = lambda: rng.random(rows) < (0.4 if mode == "all" else 0.0)  # noqa: E731
    s = dict(op="sample", logits=wide.to(DTYPES[case["src"]])[:, :vocab], uniform=torch.rand(rows, device="cuda", generator=g),
             temperature=dev(some(0.3, 1.5)), top_k=None, top_p=None, min_p=None,
             tokens=torch.empty(rows, dtype=torch.int32, device="cuda"), logprobs=torch.empty(rows, device="cuda"))
    if mode in ("top_k", "all"):
        k = np.exp(rng.uniform(0, np.log(400), rows)).astype(np.int32)
        s["top_k"] = dev(np.where(off(), 0, k))
    if mode in ("top_p", "all"):
        s["top_p"] = dev(np.where(off(), np.float32(1), some(0.5, 0.99)))
    if mode in ("min_p", "all"):
        s["min_p"] = dev(np.where(off(), np.float32(0), some(0.01, 0.2)))
    if own:
        import exact_byte_level_amd as tt
        s["workspace"] = tt.sample_workspace(s["logits"])
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    return (run_own if own else {"write": plain_write, "attend": plain_attend, "sample": plain_sample}[state["op"]])(state)


def run_own(s):
    import exact_byte_level_amd as tt
    if s["op"] == "write":
        tt.write_cache_into(s["keys"], s["values"], s["slots"], s["key_cache"], s["value_cache"], key_scale=s["key_scale"], value_scale=s["value_scale"])
        return dict(keys=s["key_cache"], values=s["value_cache"])
    if s["op"] == "attend":
        tt.attend_cache_into(s["query"], s["key_cache"], s["value_cache"], s["table"], s["lengths"], s["out"], rows=s["rows"], scale=s["scale"],
                             window=s["window"], softcap=s["softcap"], key_scale=s["key_scale"], value_scale=s["value_scale"], lse=s["lse"],
                             workspace=s["workspace"])
        return dict(out=s["out"], lse=s["lse"])
    tt.sample_tokens_into(s["logits"], s["uniform"], s["tokens"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"],
                          logprobs=s["logprobs"], workspace=s["workspace"])
    return dict(tokens=s["tokens"], logprobs=s["logprobs"])


def plain_write(s):
    live = s["slots"] >= 0
    slots, bs = s["slots"][live], s["key_cache"].shape[1]
    at = torch.div(slots, bs, rounding_mode="floor"), slots % bs
    for x, cache, scale in ((s["keys"], s["key_cache"], s["key_scale"]), (s["values"], s["value_cache"], s["value_scale"])):
        x = x[live].float()
        if scale is not None:
            x = (x / scale[:, None]).clamp(-MOST, MOST)
        if cache.dtype == torch.float8_e4m3fn:
            cache.view(torch.uint8)[at] = x.to(cache.dtype).view(torch.uint8)
        else:
            cache[at] = x.to(cache.dtype)
    return dict(keys=s["key_cache"], values=s["value_cache"])


def plain_attend(s):
    """The tokens of every row taken out of the cache once, scores and weights of all its places, those that a query does not see put out.
    The softmax goes by all places of the longest row."""
    bs, (queries, heads, dim), kv = s["key_cache"].shape[1], s["query"].shape, s["key_cache"].shape[2]
    lengths = s["lengths"].long().clamp(min=0)
    longest = int(lengths.max())
    at = torch.arange(max(longest, 1), device="cuda")
    block = s["table"][:, torch.div(at, bs, rounding_mode="floor")].long().clamp(min=0)
    held = torch.zeros(s["table"].shape[0], dtype=torch.int64, device="cuda").scatter_reduce_(0, s["rows"].long(), lengths, "amax")
    place = at % bs
    pad = held[:, None] <= at
    q = s["query"].float().reshape(queries, kv, heads // kv, dim)
    per_row = torch.bincount(s["rows"], minlength=held.numel())
    most = int(per_row.max())  # queries of a row, one behind the other
    nth = torch.argsort(torch.argsort(s["rows"], stable=True)) - (torch.cumsum(per_row, 0) - per_row)[s["rows"].long()]
    spot = s["rows"].long() * most + nth
    slotted = q.new_zeros((held.numel() * most, *q.shape[1:]))
    slotted[spot] = q
    slotted = slotted.reshape(held.numel(), most, kv, heads // kv, dim).permute(0, 2, 1, 3, 4).reshape(held.numel(), kv, -1, dim)
    keys = s["key_cache"][block, place].float() if s["key_cache"].dtype != torch.float8_e4m3fn else s["key_cache"].view(torch.uint8)[block, place].view(torch.float8_e4m3fn).float()
    x = torch.matmul(slotted, keys.permute(0, 2, 3, 1)) * s["scale"]
    del keys
    if s["key_scale"] is not None:
        x = x * s["key_scale"][:, None, None]
    if s["softcap"]:
        x = torch.tanh(x / s["softcap"]) * s["softcap"]
    until = torch.zeros(held.numel() * most, dtype=torch.int64, device="cuda")
    until[spot] = lengths
    until = until.reshape(held.numel(), 1, most, 1, 1)
    unseen = at >= until
    if s["window"]:
        unseen |= at < until - s["window"]
    x = x.reshape(held.numel(), kv, most, heads // kv, -1).masked_fill_(unseen, float("-inf"))
    top = x.amax(-1, keepdim=True).clamp(min=-3e38)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    values = s["value_cache"][block, place].float() if s["value_cache"].dtype != torch.float8_e4m3fn else s["value_cache"].view(torch.uint8)[block, place].view(torch.float8_e4m3fn).float()
    values = values.masked_fill_(pad[:, :, None, None], 0.0)
    out = torch.matmul(x.reshape(held.numel(), kv, -1, x.shape[-1]), values.permute(0, 2, 1, 3)).reshape(*x.shape[:-1], dim)
    out = torch.where(total > 0, out / total.clamp(min=1e-30), 0.0)
    if s["value_scale"] is not None:
        out = out * s["value_scale"][:, None, None, None]
    lse = torch.where(total > 0, top + torch.log(total.clamp(min=1e-30)), float("-inf"))
    back = lambda y: y.transpose(1, 2).reshape(held.numel() * most, heads, -1)[spot]  # noqa: E731
    return dict(out=back(out).to(s["query"].dtype), lse=back(lse)[..., 0])


def plain_sample(s):
    x = s["logits"].double()
    rows, vocab = x.shape
    best = x.amax(1, keepdim=True)
    some = best > float("-inf")
    weight = torch.exp(torch.where(some, x - best, x) / s["temperature"].double()[:, None])
    order = torch.sort(s["logits"], dim=1, descending=True, stable=True).indices  # ties: lowest id first
    falling = weight.gather(1, order)
    total = torch.cumsum(falling, 1)
    at = torch.arange(vocab, device="cuda")
    kept = torch.ones_like(order, dtype=torch.bool)
    if s["top_k"] is not None:
        kept &= at < torch.where(s["top_k"] > 0, s["top_k"], vocab)[:, None]
    if s["top_p"] is not None:  # of those the fewest that reach p
        all_of = total.gather(1, kept.sum(1, keepdim=True) - 1)
        p = s["top_p"].double()[:, None]
        kept &= (p >= 1) | (at == 0) | (total - falling < p * all_of)
    if s["min_p"] is not None:
        kept &= (at == 0) | (falling >= s["min_p"].double()[:, None])
    weight = torch.zeros_like(weight).scatter_(1, order, torch.where(kept, falling, 0.0))
    running = torch.cumsum(weight, 1)
    reached = running > s["uniform"].double()[:, None] * running[:, -1:]
    token = reached.int().argmax(1)
    logprob = torch.log(weight.gather(1, token[:, None])[:, 0] / running[:, -1])
    return dict(tokens=torch.where(some[:, 0], token, -1).int(), logprobs=torch.where(some[:, 0], logprob, float("-inf")).float())


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    if case["op"] == "write":
        cells = 2 * case["tokens"] * (1 - case["idle"]) * case["heads"] * case["dim"]
        return dict(bytes=8 * case["tokens"] + cells * (SIZES[case["src"]] + SIZES[case["dst"]]), flops=0)
    if case["op"] == "attend":
        # the places of each row that some of its queries see, read once; every query's products
        row, _ = queries_of(case)
        seen, window = np.maximum(seen_of(case), 0), case["window"] or case["context"]
        upto, since = np.zeros(case["rows"], np.int64), np.full(case["rows"], 1 << 40)
        np.maximum.at(upto, row, seen)
        np.minimum.at(since, row, np.maximum(seen - window, 0))
        places = np.maximum(upto - since, 0).sum()
        cells = case["queries"] * case["heads"] * case["dim"]
        return dict(bytes=float(places) * (2 * case["kv"] * case["dim"] * SIZES[case["dst"]] + 4 / case["block"]) + 4 * cells + 4 * case["queries"] * (2 + case["heads"]),
                    flops=4.0 * np.minimum(seen, window).sum() * case["heads"] * case["dim"])
    return dict(bytes=case["rows"] * (case["vocab"] * SIZES[case["src"]] + 28), flops=10.0 * case["rows"] * case["vocab"])


# ---------------------------------------------------------------- by definition

def exact(case, seed):
    """run()'s outputs by definition, one request after the other in 64 bits."""
    s = prepare(case, seed)
    return {"write": exact_write, "attend": exact_attend, "sample": exact_sample}[case["op"]](s)


def exact_write(s):
    bs, got = s["key_cache"].shape[1], {}
    slots = s["slots"].tolist()
    keep = [i for i, slot in enumerate(slots) if slot >= 0]
    to = torch.tensor([slots[i] for i in keep], dtype=torch.int64, device="cuda")
    for name, x, cache, scale in (("keys", s["keys"], s["key_cache"], s["key_scale"]), ("values", s["values"], s["value_cache"], s["value_scale"])):
        new = cache.double()
        x = x[torch.tensor(keep, dtype=torch.int64, device="cuda")].double()
        if scale is not None:
            x = torch.minimum(torch.maximum(x / scale.double()[None, :, None], x.new_tensor(-MOST)), x.new_tensor(MOST))
        new[to // bs, to % bs] = x  # unrounded
        got[name] = new.cpu().numpy()
    return got


def exact_attend(s):
    query, bs = s["query"].double(), s["key_cache"].shape[1]
    (queries, heads, dim), kv = query.shape, s["key_cache"].shape[2]
    if float(s["lengths"].double().sum()) * kv * dim > 3e9:
        return None
    out, lse = torch.zeros_like(query), torch.full((queries, heads), -math.inf, dtype=torch.float64, device="cuda")
    unit = torch.ones(kv, device="cuda")
    key_scale, value_scale = ((unit if t is None else t).double() for t in (s["key_scale"], s["value_scale"]))
    for i, (n, r) in enumerate(zip(s["lengths"].tolist(), s["rows"].tolist())):
        since = max(0, n - s["window"]) if s["window"] else 0
        if n <= since:
            continue
        blocks = s["table"][r, since // bs:-(-n // bs)].long()
        k, v = (c[blocks].double().reshape(-1, kv, dim)[since % bs:][:n - since].transpose(0, 1) for c in (s["key_cache"], s["value_cache"]))
        score = torch.matmul(query[i].reshape(kv, -1, dim), k.transpose(1, 2).contiguous()) * (s["scale"] * key_scale)[:, None, None]
        if s["softcap"]:
            score = s["softcap"] * torch.tanh(score / s["softcap"])
        lse[i] = torch.logsumexp(score, 2).reshape(-1)
        out[i] = (torch.matmul(torch.softmax(score, 2), v.contiguous()) * value_scale[:, None, None]).reshape(heads, dim)
    return dict(out=out.cpu().numpy(), lse=lse.cpu().numpy())


def exact_sample(s):
    tokens, logprobs = [], []
    for r in range(s["logits"].shape[0]):
        x = s["logits"][r].double()
        best = float(x.max())
        if best == -math.inf:
            tokens.append(-1)
            logprobs.append(-math.inf)
            continue
        temperature = float(s["temperature"][r])
        ids = torch.argsort(-x, stable=True)
        w = torch.exp((x[ids] - best) / temperature)
        n = w.numel()
        if s["top_k"] is not None and int(s["top_k"][r]) > 0:
            n = min(n, int(s["top_k"][r]))
        if s["top_p"] is not None and float(s["top_p"][r]) < 1:
            sums = torch.cumsum(w[:n], 0)
            n = min(n, 1 + int((sums < float(s["top_p"][r]) * sums[-1]).sum()))
        if s["min_p"] is not None:
            n = max(1, min(n, int((w >= float(s["min_p"][r])).sum())))
        ids, by_id = torch.sort(ids[:n])
        sums = torch.cumsum(w[:n][by_id], 0)
        at = int(torch.searchsorted(sums, float(s["uniform"][r]) * sums[-1], right=True))
        tokens.append(int(ids[at]))
        logprobs.append(float(torch.log(w[by_id[at]] / sums[-1])))
    return dict(tokens=np.array(tokens, np.int32), logprobs=np.array(logprobs))
