"""What the serving operators are measured on: block tables, token sets, grammar masks and the shaping of logits.

Cases, their inputs, one pass through an operator (in plain torch operations, or through the package's
entry points where ``own`` is true), its least bytes and operations, and its values by definition in numpy.

A token set is a row of 32-bit words, token id v being bit v & 31 of word v >> 5.
"""
import functools
import os

import numpy as np
import torch

own = False

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
DEAD, FREE = -1, -2  # grammar states: nothing may follow; no grammar


# ---------------------------------------------------------------- cases

def listed():
    return [
        # a decode step of a few requests: one token each, some rows of the table idle
        dict(name="plan_step", op="plan", rows=8, tokens=0, block=16, context=4000),
        # a batch of prompts as one encode_batch call gives it: 64 texts, two million tokens, all new
        dict(name="plan_prompts", op="plan", rows=64, tokens=2_000_000, block=16, context=0),
        # a step that mixes prompts' next parts and single tokens over many requests, blocks of an odd size
        dict(name="plan_mixed", op="plan", rows=1500, tokens=48_000, block=24, context=9000),
        # requests that end: one in a small batch, and half of a large table's long rows
        dict(name="release_few", op="release", rows=16, block=16, context=3000, share=0.1),
        dict(name="release_many", op="release", rows=1024, block=16, context=32_000, share=0.5),
        # the set of one prompt's tokens, and of a batch of prompts
        dict(name="bits_one", op="bits", rows=1, tokens=2500, vocab=50_256, add=False),
        dict(name="bits_prompts", op="bits", rows=64, tokens=2_000_000, vocab=100_256, add=False),
        # the mask of one request's state, and of every state of a schema at once (done when the schema is loaded)
        dict(name="grammar_step", op="grammar", rows=1, states=300, table=3),
        dict(name="grammar_all", op="grammar", rows=1024, states=1024, table=3),
        # logits of one request, of a serving batch with everything on, and of a large batch in 32 bits
        dict(name="shape_one", op="shape", rows=1, vocab=50_256, pad=0, src="bf16", dst="f32", generated=400, biases=4, states=300),
        dict(name="shape_batch", op="shape", rows=61, vocab=100_257, pad=7, src="f16", dst="f16", generated=6000, biases=40, states=500),
        dict(name="shape_large", op="shape", rows=256, vocab=262_144, pad=0, src="f32", dst="f32", generated=2000, biases=16, states=64),
    ]


def draw(rng):
    def near(lo, hi):  # whole numbers spread over their logarithm, odd ones among them
        return int(round(lo * (hi / lo) ** rng.random()))

    op = rng.choice(["plan", "plan", "release", "bits", "grammar", "shape", "shape"])
    if op == "plan":
        rows = near(1, 4000)
        return dict(op=op, rows=rows, tokens=rng.choice([0, max(rows // 2, near(1, 2_000_000))]), block=rng.choice([16, 32, 64, 128, near(8, 300)]),
                    context=rng.choice([0, near(1, 30_000)]))
    if op == "release":
        return dict(op=op, rows=near(1, 1000), block=rng.choice([16, 32, 64, near(16, 300)]), context=near(1, 32_000), share=round(rng.random(), 2))
    if op == "bits":
        return dict(op=op, rows=near(1, 250), tokens=near(1, 2_000_000), vocab=near(300, 250_000), add=rng.random() < 0.3)
    if op == "grammar":
        return dict(op=op, rows=near(1, 1000), states=near(40, 1000), table=rng.choice([1, 2, 3]))
    rows = near(1, 250)
    src = rng.choice(list(DTYPES))
    return dict(op=op, rows=rows, vocab=near(300, 260_000), pad=rng.choice([0, near(1, 64)]), src=src, dst=rng.choice(["f32", src]),
                generated=near(1, 16_000), biases=near(1, 300), states=near(40, 600))


# ---------------------------------------------------------------- inputs

def generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def words(vocab):
    return (vocab + 31) // 32


@functools.lru_cache(maxsize=None)
def token_strings(table):
    """Bytes and offsets of the tokens of one of the repository's merge tables."""
    tok = [bytes([b]) for b in range(256)]
    for x, y in np.load(os.path.join(ROOT, "data", "vocab_c%d.npy" % table)).tolist():
        tok.append(tok[x] + tok[y])
    offsets = np.zeros(len(tok) + 1, np.int32)
    offsets[1:] = np.cumsum([len(t) for t in tok])
    return np.frombuffer(b"".join(tok), np.uint8).copy(), offsets


def schema(states, rng):
    """A byte automaton as a structured answer needs it: records of quoted names and of values (texts, whole
    numbers, one of two words), until the states are used up; the last state takes nothing and accepts."""
    nxt = np.full((states, 256), DEAD, np.int32)
    last, at = states - 1, 0

    def literal(at, text):
        for b in text:
            nxt[at, b] = at + 1
            at += 1
        return at

    while at + 24 < last:
        name = bytes(rng.integers(97, 123, int(rng.integers(3, 10))).astype(np.uint8))
        nxt[at, [32, 10]] = at
        at = literal(at, b'"' + name + b'": ')
        kind = int(rng.integers(0, 3))
        if kind == 0:  # a text: any bytes but a quote, a backslash and control characters, then a quote
            at = literal(at, b'"')
            nxt[at, 32:] = at
            nxt[at, 92] = DEAD
            nxt[at, 34] = at + 1
            at += 1
        elif kind == 1:  # a whole number of one digit or more
            nxt[at, 48:58] = at + 1
            at += 1
            nxt[at, 48:58] = at
        else:  # yes or no
            nxt[at, ord("y")], nxt[at, ord("n")] = at + 1, at + 3
            nxt[at + 1, ord("e")], nxt[at + 2, ord("s")] = at + 2, at + 4
            nxt[at + 3, ord("o")] = at + 4
            at += 4
        nxt[at, ord(",")] = at + 1
        nxt[at, ord("}")] = last
        at += 1
    nxt[at, ord("}")] = last
    accept = np.zeros(states, np.uint8)
    accept[last] = 1
    return nxt, accept


def split_of(total, rows, rng):
    """offsets of `rows` log-normal parts of `total` tokens; some are empty where there are several."""
    weight = np.minimum(rng.lognormal(0.0, 1.0, rows), 8.0)
    if rows > 3:
        weight[rng.random(rows) < 0.05] = 0.0
        weight[int(rng.integers(rows))] = 1.0
    ends = np.floor(np.cumsum(weight) / weight.sum() * total + 0.5).astype(np.int64)
    ends[-1] = total
    return np.concatenate([[0], np.minimum(ends, total)]).astype(np.int64)


def some_ids(shape, vocab, g):
    """Token ids as texts have them: low ids often, high ones seldom."""
    u = torch.rand(shape, device="cuda", generator=g)
    return (u * u * u * vocab).to(torch.int32).clamp_(max=vocab - 1)


def prepare(case, seed):
    rng, g = np.random.default_rng(seed), generator(seed)
    return {"plan": prepare_blocks, "release": prepare_blocks, "bits": prepare_bits, "grammar": prepare_grammar, "shape": prepare_shape}[case["op"]](case, rng, g)


def prepare_blocks(case, rng, g):
    rows, bs = case["rows"], case["block"]
    context = np.minimum(np.floor(case["context"] * np.exp(rng.normal(-0.5, 0.7, rows))), case["context"]).astype(np.int64)
    new = np.ones(rows, np.int64)
    s = dict(op=case["op"], block=bs)
    if case["op"] == "plan":
        if case["tokens"]:
            offsets = split_of(case["tokens"], rows, rng)
            new = np.diff(offsets)
            s["offsets"] = dev(offsets)
            places = (case["tokens"] + 255) // 256 * 256  # a launch's bucket: the places past the last token hold -1
        else:
            s["offsets"] = None
            places = rows
        if rows > 3:
            context[rng.random(rows) < 0.1] = -1  # not in use
    held = -(-np.maximum(context, 0) // bs)
    want = -(-(np.maximum(context, 0) + new) // bs)
    longest = min(case.get("tokens", 0), 16 * -(-case.get("tokens", 0) // rows)) or 1  # of a row's new tokens, 8 weights of about 1.5 on average
    width = max(-(-(case["context"] + longest) // bs), int(want.max())) + 2
    pool = rows * (-(-case["context"] // bs) + 2) + case.get("tokens", 0) // bs + 64
    order = torch.randperm(pool, device="cuda", generator=g).to(torch.int32)
    lengths, at = dev(context.astype(np.int32)), torch.arange(width, device="cuda")
    first = dev(np.concatenate([[0], np.cumsum(held)[:-1]]))
    taken = at < dev(held)[:, None]
    s["table"] = torch.where(taken, order[torch.where(taken, first[:, None] + at, 0)], -1)
    s["lengths"] = lengths
    s["free"] = torch.full((pool,), -1, dtype=torch.int32, device="cuda")
    n_free = pool - int(held.sum())
    s["free"][:n_free] = order[pool - n_free:]
    s["n_free"] = torch.tensor([n_free], dtype=torch.int32, device="cuda")
    if case["op"] == "release":
        s["done"] = dev(rng.random(rows) < case["share"])
    # what the step writes: a caller's program keeps these buffers
    s["out_lengths"], s["out_n_free"] = torch.empty_like(lengths), torch.empty_like(s["n_free"])
    s["n"] = torch.empty(1, dtype=torch.int64, device="cuda")
    if case["op"] == "plan":
        s["slots"] = torch.empty(places, dtype=torch.int64, device="cuda")
        s["positions"], s["rows"] = (torch.empty(places, dtype=torch.int32, device="cuda") for _ in range(2))
    return s


def prepare_bits(case, rng, g):
    rows, vocab = case["rows"], case["vocab"]
    ids = some_ids((case["tokens"],), vocab, g)
    ids[torch.rand(case["tokens"], device="cuda", generator=g) < 0.001] = -1  # padding
    bits = torch.randint(-2**31, 2**31, (rows, words(vocab)), device="cuda", generator=g).to(torch.int32)
    if vocab % 32:
        bits[:, -1] &= (1 << vocab % 32) - 1
    return dict(op="bits", vocab=vocab, add=case["add"], ids=ids, offsets=dev(split_of(case["tokens"], rows, rng)), bits=bits)


def prepare_grammar(case, rng, g):
    strings, offsets = token_strings(case["table"])
    nxt, accept = schema(case["states"], rng)
    rows, tokens = case["rows"], len(offsets) - 1
    states = np.arange(rows) if rows == case["states"] else rng.integers(0, case["states"], rows)
    vocab = tokens + 1  # the model's vocabulary has an end token behind the tokenizer's
    s = dict(op="grammar", next=dev(nxt), accept=dev(accept), strings=dev(strings), offsets=dev(offsets), longest=int(np.diff(offsets).max()),
             vocab=vocab, end=tokens, states=dev(states.astype(np.int32)), bits=torch.empty((rows, words(vocab)), dtype=torch.int32, device="cuda"))
    if own:
        import exact_byte_level_amd as tt
        s["grammar"], s["tokens"] = tt.Grammar(nxt, accept, end_id=tokens), tt.TokenStrings(strings, offsets)
    return s


def prepare_shape(case, rng, g):
    rows, vocab, gen = case["rows"], case["vocab"], case["generated"]
    wide = torch.randn((rows, vocab + case["pad"]), device="cuda", generator=g).mul_(4).to(DTYPES[case["src"]])
    n = np.maximum(1, gen * np.exp(-3 * rng.random(rows))).astype(np.int32)
    count = rng.integers(0, 2 * case["biases"] + 1, rows)
    bias_offsets = np.concatenate([[0], np.cumsum(count)]).astype(np.int64)
    some = lambda lo, hi: dev(rng.uniform(lo, hi, rows).astype(np.float32))  # noqa: E731
    rows_of = rng.integers(0, case["states"], rows)
    rows_of[rng.random(rows) < 0.3] = FREE  # requests without a grammar
    dense = torch.randint(-2**31, 2**31, (case["states"], words(vocab)), device="cuda", generator=g).to(torch.int32)
    sparse = torch.randint(-2**31, 2**31, dense.shape, device="cuda", generator=g).to(torch.int32) & dense
    seen = [torch.randint(-2**31, 2**31, (rows, words(vocab)), device="cuda", generator=g).to(torch.int32) for _ in range(4)]
    return dict(op="shape", logits=wide[:, :vocab], out=torch.empty((rows, vocab), dtype=DTYPES[case["dst"]], device="cuda"),
                seen=seen[0] & seen[1] & seen[2] & seen[3], generated=some_ids((rows, gen), vocab, g), n_generated=dev(n),
                repetition=some(1.0, 1.5), frequency=some(0.0, 0.8), presence=some(0.0, 0.8),
                bias_offsets=dev(bias_offsets), bias_ids=some_ids((int(bias_offsets[-1]),), vocab, g),
                bias_values=torch.randn(int(bias_offsets[-1]), device="cuda", generator=g).mul_(5),
                allowed=torch.where(torch.arange(case["states"], device="cuda")[:, None] % 2 == 0, dense, sparse), allowed_rows=dev(rows_of.astype(np.int32)),
                temperature=some(0.3, 1.5))


# ---------------------------------------------------------------- one pass

def run(state):
    return (run_own if own else {"plan": plain_plan, "release": plain_release, "bits": plain_bits, "grammar": plain_grammar, "shape": plain_shape}[state["op"]])(state)


def run_own(s):
    import exact_byte_level_amd as tt
    if s["op"] == "plan":
        tt.plan_blocks_into(s["lengths"], s["table"], s["free"], s["n_free"], s["block"], s["slots"], s["n"], offsets=s["offsets"],
                            positions=s["positions"], rows=s["rows"], out_lengths=s["out_lengths"], out_n_free=s["out_n_free"])
        return {k: s[k] for k in ("table", "slots", "positions", "rows", "out_lengths", "out_n_free", "n")}
    if s["op"] == "release":
        tt.release_blocks_into(s["lengths"], s["done"], s["table"], s["free"], s["n_free"], s["block"], s["n"],
                               out_lengths=s["out_lengths"], out_n_free=s["out_n_free"])
        return {k: s[k] for k in ("free", "out_lengths", "out_n_free", "n")}
    if s["op"] == "bits":
        tt.token_bits_into(s["ids"], s["bits"], s["vocab"], offsets=s["offsets"], add=s["add"])
        return s["bits"]
    if s["op"] == "grammar":
        tt.grammar_bits_into(s["grammar"], s["tokens"], s["states"], s["bits"], s["vocab"])
        return s["bits"]
    tt.shape_logits_into(s["logits"], s["out"], **{k: s[k] for k in (
        "seen", "generated", "n_generated", "repetition", "frequency", "presence", "bias_offsets", "bias_ids", "bias_values",
        "allowed", "allowed_rows", "temperature")})
    return s["out"]


def up(a, b):
    return torch.div(a + (b - 1), b, rounding_mode="floor")


def plain_plan(s):
    lengths, bs, table = s["lengths"].long(), s["block"], s["table"]
    rows, places = lengths.numel(), s["slots"].numel()
    start = lengths.clamp(min=0)
    if s["offsets"] is None:
        new = (lengths >= 0).long()
        end = torch.where(lengths >= 0, start + new, lengths)
        row = torch.arange(rows, device="cuda")  # a place for each row
        live, place = lengths >= 0, start
        total = new.sum()
    else:
        offsets = s["offsets"]
        new = offsets[1:] - offsets[:-1]
        end = torch.where((lengths < 0) & (new == 0), lengths, start + new)
        at = torch.arange(places, device="cuda")
        row = torch.searchsorted(offsets, at, right=True) - 1
        live = row < rows
        row = row.clamp(max=rows - 1)
        place = start[row] + at - offsets[row]
        total = offsets[-1]
    held = up(start, bs)
    need = up(start + new, bs) - held
    base = torch.cumsum(need, 0) - need
    block = torch.div(place, bs, rounding_mode="floor")
    nth = block - held[row]  # the how-manieth new block of its row; negative: a block that the row has
    fresh = s["free"][(s["n_free"].long() - 1 - base[row] - nth).clamp(0, s["free"].numel() - 1)]
    within = block.clamp(max=table.shape[1] - 1)
    have = torch.where(nth >= 0, fresh, table[row, within])
    opens = live & (nth >= 0) & (place == block * bs)
    flat = torch.cat([table.reshape(-1), table.new_zeros(1)])
    flat[torch.where(opens, row * table.shape[1] + within, flat.numel() - 1)] = have
    return dict(table=flat[:-1].reshape(table.shape), slots=torch.where(live, have.long() * bs + place - block * bs, -1),
                positions=torch.where(live, place, -1).int(), rows=torch.where(live, row, -1).int(),
                out_lengths=end.int(), out_n_free=(s["n_free"].long() - need.sum()).int(), n=total.reshape(1))


def plain_release(s):
    lengths, bs, table, free = s["lengths"].long(), s["block"], s["table"], s["free"]
    done = s["done"] & (lengths >= 0)
    many = torch.where(done, up(lengths.clamp(min=0), bs), 0)
    base = s["n_free"].long() + torch.cumsum(many, 0) - many
    at = torch.arange(table.shape[1], device="cuda")
    to = torch.where(at < many[:, None], base[:, None] + at, free.numel())
    flat = torch.cat([free, free.new_zeros(1)])
    flat[to.reshape(-1)] = table.reshape(-1)
    return dict(free=flat[:-1], out_lengths=torch.where(done, -1, lengths).int(), out_n_free=(s["n_free"].long() + many.sum()).int(), n=many.sum().reshape(1))


def pack(member):
    """[rows, 32 * words] truth values as words."""
    bit = torch.ones(32, dtype=torch.int64, device="cuda") << torch.arange(32, device="cuda")
    return (member.reshape(member.shape[0], -1, 32) * bit).sum(2).to(torch.int32)


def unpack(bits, vocab):
    member = (bits[:, :, None] >> torch.arange(32, device="cuda", dtype=torch.int32)) & 1
    return member.reshape(bits.shape[0], -1)[:, :vocab].bool()


def plain_bits(s):
    ids, offsets, vocab = s["ids"].long(), s["offsets"], s["vocab"]
    rows, wide = offsets.numel() - 1, 32 * words(vocab)
    row = torch.searchsorted(offsets, torch.arange(ids.numel(), device="cuda"), right=True) - 1
    member = torch.zeros(rows * wide + 1, dtype=torch.bool, device="cuda")
    member[torch.where((ids >= 0) & (ids < vocab), row * wide + ids, rows * wide)] = True
    got = pack(member[:-1].reshape(rows, wide))
    return got | s["bits"] if s["add"] else got


def plain_grammar(s):
    offsets, strings = s["offsets"].long(), s["strings"].long()
    start, length = offsets[:-1], offsets[1:] - offsets[:-1]
    n = s["next"].shape[0]
    step = torch.cat([torch.where(s["next"] < 0, n, s["next"]), torch.full((1, 256), n, device="cuda", dtype=torch.int32)]).reshape(-1)  # state n: dead
    now = s["states"][:, None].expand(-1, start.numel())
    for k in range(s["longest"]):  # one byte of every token
        byte = strings[(start + k).clamp(max=strings.numel() - 1)].int()
        now = torch.where(k < length, step[now * 256 + byte], now)
    member = torch.zeros((now.shape[0], 32 * words(s["vocab"])), dtype=torch.bool, device="cuda")
    member[:, :start.numel()] = (now < n) & (length > 0)
    member[:, s["end"]] = s["accept"][s["states"].long()].bool()
    return pack(member)


def plain_shape(s):
    x = s["logits"].float()
    rows, vocab = x.shape
    gen = s["generated"].long()
    live = torch.arange(gen.shape[1], device="cuda") < s["n_generated"][:, None]
    count = torch.zeros((rows, vocab), dtype=torch.int32, device="cuda").scatter_add_(1, gen, live.int())
    seen = unpack(s["seen"], vocab) | (count > 0)
    rho = s["repetition"][:, None]
    x = torch.where(seen, torch.where(x > 0, x / rho, x * rho), x)
    x = x - s["frequency"][:, None] * count - s["presence"][:, None] * (count > 0)
    entries = s["bias_ids"].numel()
    if entries:  # of an id named twice in a row, the later entry counts
        row = torch.searchsorted(s["bias_offsets"], torch.arange(entries, device="cuda"), right=True) - 1
        which = torch.full((rows * vocab,), -1, dtype=torch.int64, device="cuda").scatter_reduce_(
            0, row * vocab + s["bias_ids"].long(), torch.arange(entries, device="cuda"), "amax").reshape(rows, vocab)
        x = x + torch.where(which >= 0, s["bias_values"][which.clamp(min=0)], 0.0)
    at = s["allowed_rows"].long()
    allowed = unpack(s["allowed"][at.clamp(min=0)], vocab) | (at == FREE)[:, None]
    x = torch.where(allowed, x, float("-inf")) / s["temperature"][:, None]
    return x.to(s["out"].dtype)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    rows, op = case["rows"], case["op"]
    if op == "plan":
        new = case["tokens"] or rows
        return dict(bytes=12 * rows + 16 * new + 8 * (new // case["block"]) + (8 * rows if case["tokens"] else 0), flops=0)
    if op == "release":
        blocks = case["share"] * rows * 0.7 * case["context"] / case["block"]
        return dict(bytes=9 * rows + 8 * blocks, flops=0)
    if op == "bits":
        return dict(bytes=4 * case["tokens"] + 8 * rows + 4 * rows * words(case["vocab"]) * (2 if case["add"] else 1), flops=0)
    if op == "grammar":
        strings, offsets = token_strings(case["table"])
        return dict(bytes=strings.size + offsets.size * 4 + 512 * case["states"] + 4 * rows * words(offsets.size), flops=rows * offsets.size)
    size = {"f32": 4, "f16": 2, "bf16": 2}
    cells = rows * case["vocab"]
    return dict(bytes=cells * (size[case["src"]] + size[case["dst"]]) + cells // 4 + rows * (4 * case["generated"] // 3 + 12 * case["biases"]), flops=4 * cells)


# ---------------------------------------------------------------- by definition

def exact(case, seed):
    """run()'s outputs row by row in numpy, computed numbers in 64 bits."""
    s = {k: v.cpu() if isinstance(v, torch.Tensor) else v for k, v in prepare(case, seed).items()}
    a = {k: (v.float() if v.dtype in (torch.float16, torch.bfloat16) else v).numpy() for k, v in s.items() if isinstance(v, torch.Tensor)}
    if case["op"] in ("plan", "release"):
        return exact_blocks(case, s, a)
    if case["op"] == "bits":
        member = np.zeros((case["rows"], 32 * words(case["vocab"])), bool)
        for r in range(case["rows"]):
            ids = a["ids"][a["offsets"][r]:a["offsets"][r + 1]]
            member[r, ids[(ids >= 0) & (ids < case["vocab"])]] = True
        got = np.packbits(member, axis=1, bitorder="little").view(np.int32)
        return got | a["bits"] if case["add"] else got
    if case["op"] == "grammar":
        return exact_grammar(s, a)
    out = np.empty(a["out"].shape)
    for b in range(case["rows"]):
        x = a["logits"][b].astype(np.float64)
        count = np.bincount(a["generated"][b, :a["n_generated"][b]], minlength=x.size)
        seen = np.unpackbits(a["seen"][b].view(np.uint8), bitorder="little")[:x.size].astype(bool) | (count > 0)
        rho = float(a["repetition"][b])
        x[seen] *= np.where(x[seen] > 0, 1 / rho, rho)
        x -= float(a["frequency"][b]) * count + float(a["presence"][b]) * (count > 0)
        lo, hi = a["bias_offsets"][b], a["bias_offsets"][b + 1]
        named = dict(zip(a["bias_ids"][lo:hi].tolist(), a["bias_values"][lo:hi].tolist()))
        x[list(named)] += np.fromiter(named.values(), np.float64, len(named))
        if a["allowed_rows"][b] != FREE:
            x[np.unpackbits(a["allowed"][a["allowed_rows"][b]].view(np.uint8), bitorder="little")[:x.size] == 0] = -np.inf
        out[b] = x / float(a["temperature"][b])
    return out


def exact_blocks(case, s, a):
    bs, free, n_free, lengths = case["block"], a["free"].copy(), int(a["n_free"][0]), a["lengths"].copy()
    table = a["table"].copy()
    n = 0
    if case["op"] == "release":
        for r in np.flatnonzero(a["done"] & (lengths >= 0)):
            m = -(-int(lengths[r]) // bs)
            free[n_free + n:n_free + n + m] = table[r, :m]
            n, lengths[r] = n + m, -1
        return dict(free=free, out_lengths=lengths, out_n_free=np.array([n_free + n], np.int32), n=np.array([n]))
    places = a["slots"].size
    slots, positions, rows = np.full(places, -1, np.int64), np.full(places, -1, np.int32), np.full(places, -1, np.int32)
    for r in range(case["rows"]):
        single = s["offsets"] is None
        lo, hi = (r, r + int(lengths[r] >= 0)) if single else (int(a["offsets"][r]), int(a["offsets"][r + 1]))
        if lo == hi:
            continue
        start = max(int(lengths[r]), 0)
        for k in range(-(-start // bs), -(-(start + hi - lo) // bs)):
            n_free -= 1
            table[r, k] = free[n_free]
        at = start + np.arange(hi - lo)
        slots[lo:hi], positions[lo:hi], rows[lo:hi] = table[r, at // bs].astype(np.int64) * bs + at % bs, at, r
        lengths[r], n = start + hi - lo, n + hi - lo
    return dict(table=table, slots=slots, positions=positions, rows=rows, out_lengths=lengths, out_n_free=np.array([n_free], np.int32), n=np.array([n]))


def exact_grammar(s, a):
    """Every state at once along a tree of the tokens' prefixes; None where that takes long."""
    if a["states"].size * s["vocab"] > 5_000_000:
        return None
    data, off, n = a["strings"].tobytes(), a["offsets"], a["next"].shape[0]
    nxt = np.where(a["next"] < 0, n, a["next"])
    nxt = np.concatenate([nxt, np.full((1, 256), n)])
    member = np.zeros((a["states"].size, 32 * words(s["vocab"])), bool)
    after = {b"": a["states"].astype(np.int64)}
    for v in sorted(range(off.size - 1), key=lambda v: data[off[v]:off[v + 1]]):
        text = data[off[v]:off[v + 1]]
        for k in range(1, len(text) + 1):
            if text[:k] not in after:
                after[text[:k]] = nxt[after[text[:k - 1]], text[k - 1]]
        if text:
            member[:, v] = after[text] < n
    member[:, s["end"]] = a["accept"][a["states"]] != 0
    return np.packbits(member, axis=1, bitorder="little").view(np.int32)
