"""Plain definitions of the serving operators (include/tt_serve.h): sequential Python and numpy in 64 bits,
sharing no code with the package."""
import numpy as np

DEAD, FREE = -1, -2


def plan(lengths, table, free, n_free, block, places, offsets=None):
    """A dict of everything tt_plan_blocks writes; ``n`` is the count or a negative error code."""
    rows, width = table.shape
    out = dict(table=table.copy(), lengths=lengths.copy(), n_free=n_free, slots=np.full(places, -1, np.int64),
               positions=np.full(places, -1, np.int32), rows=np.full(places, -1, np.int32))
    error = plan_error(lengths, width, len(free), n_free, block, places, offsets)
    if error:
        return dict(out, n=error)
    n = 0
    for r in range(rows):
        start = max(int(lengths[r]), 0)
        if offsets is None:
            first, count = r, int(lengths[r] >= 0)
        else:
            first, count = int(offsets[r]), int(offsets[r + 1] - offsets[r])
        for i in range(count):
            p = start + i
            if p % block == 0:
                out["n_free"] -= 1
                out["table"][r, p // block] = free[out["n_free"]]
            b = int(out["table"][r, p // block])
            out["slots"][first + i] = b * block + p % block if b >= 0 else -1
            out["positions"][first + i] = p
            out["rows"][first + i] = r
        if count:
            out["lengths"][r] = start + count
        n += count
    return dict(out, n=n)


def plan_error(lengths, width, free_cap, n_free, block, places, offsets):
    start = np.maximum(lengths.astype(np.int64), 0)
    if offsets is None:
        count = (lengths >= 0).astype(np.int64)
    else:
        count = np.diff(offsets)
        if offsets[0] != 0 or (count < 0).any():
            return -7
    if not 0 <= n_free <= free_cap:
        return -1
    if (offsets is not None and offsets[-1] > places) or (start + count > width * block).any():
        return -8
    if (-(-(start + count) // block) - -(-start // block)).sum() > n_free:
        return -11
    return 0


def release(lengths, done, table, free, n_free, block):
    held = np.where((done != 0) & (lengths >= 0), -(-lengths.astype(np.int64) // block), 0)
    out = dict(lengths=lengths.copy(), free=free.copy(), n_free=n_free)
    if not 0 <= n_free <= len(free):
        return dict(out, n=-1)
    if (held > table.shape[1]).any() or n_free + held.sum() > len(free):
        return dict(out, n=-8)
    for r in range(len(lengths)):
        if done[r] and lengths[r] >= 0:
            for b in table[r, :held[r]]:
                out["free"][out["n_free"]] = b
                out["n_free"] += 1
            out["lengths"][r] = -1
    return dict(out, n=int(held.sum()))


def words(vocab):
    return (vocab + 31) // 32


def pack(member):
    """[rows, vocab] truth values as int32 words."""
    rows, vocab = member.shape
    wide = np.zeros((rows, 32 * words(vocab)), bool)
    wide[:, :vocab] = member
    return np.packbits(wide, axis=1, bitorder="little").view(np.int32).reshape(rows, words(vocab))


def unpack(bits, vocab):
    return np.unpackbits(np.ascontiguousarray(bits).view(np.uint8), axis=1, bitorder="little")[:, :vocab].astype(bool)


def token_bits(ids, offsets, vocab):
    member = np.zeros((len(offsets) - 1, vocab), bool)
    for r in range(len(offsets) - 1):
        lo, hi = (min(max(int(o), 0), len(ids)) for o in offsets[r:r + 2])
        for t in ids[lo:hi]:
            if 0 <= t < vocab:
                member[r, t] = True
    return pack(member)


def advance(nxt, accept, end_id, strings, q, t):
    """State after token t."""
    if q == FREE or t < 0:
        return q
    if not 0 <= q < len(nxt) or t == end_id or t >= len(strings) or not strings[t]:
        return DEAD
    for b in strings[t]:
        q = int(nxt[q, b])
        if q < 0:
            return DEAD
    return q


def grammar_bits(nxt, accept, end_id, strings, states, vocab):
    member = np.zeros((len(states), vocab), bool)
    for r, q in enumerate(states):
        if q == FREE:
            member[r] = True
            continue
        if not 0 <= q < len(nxt):
            continue
        for t in range(min(vocab, len(strings))):
            member[r, t] = advance(nxt, accept, end_id, strings, int(q), t) >= 0
        if 0 <= end_id < vocab:
            member[r, end_id] = bool(accept[q])
    return pack(member)


def shape_logits(logits, seen=None, generated=None, n_generated=None, repetition=None, frequency=None, presence=None,
                 bias_offsets=None, bias_ids=None, bias_values=None, allowed=None, allowed_rows=None, temperature=None):
    """(values in 64 bits, how far a computation in 32 bits may be off before the last rounding)."""
    rows, vocab = logits.shape
    out, slack = np.empty((rows, vocab)), np.zeros((rows, vocab))
    u = 2.0 ** -24
    for r in range(rows):
        x = logits[r].astype(np.float64)
        e = np.zeros(vocab)
        count = np.zeros(vocab, np.int64)
        if generated is not None:
            n = generated.shape[1] if n_generated is None else min(max(int(n_generated[r]), 0), generated.shape[1])
            for t in generated[r, :n]:
                if 0 <= t < vocab:
                    count[t] += 1
        was = count > 0
        if seen is not None:
            was |= unpack(seen[r:r + 1], vocab)[0]
        rho = 1.0 if repetition is None else float(repetition[r])
        with np.errstate(invalid="ignore", over="ignore"):
            x = np.where(was, np.where(x > 0, x / rho, x * rho), x)
            e += np.where(was, u * np.abs(x), 0)
            fee = (0.0 if frequency is None else float(frequency[r])) * count
            flat = 0.0 if presence is None else float(presence[r])
            x = np.where(count > 0, x - fee, x)  # the product, the difference, the second difference
            e += np.where(count > 0, u * (np.abs(fee) + np.abs(x)), 0)
            x = np.where(count > 0, x - flat, x)
            e += np.where(count > 0, u * np.abs(x), 0)
            if bias_offsets is not None:
                lo, hi = (min(max(int(o), 0), len(bias_ids)) for o in bias_offsets[r:r + 2])
                for t, b in dict(zip(bias_ids[lo:hi].tolist(), bias_values[lo:hi].tolist())).items():
                    if 0 <= t < vocab:
                        x[t] += b
                        e[t] += u * abs(x[t])
            if allowed is not None:
                q = r if allowed_rows is None else int(allowed_rows[r])
                if q != FREE:
                    ok = unpack(allowed[q:q + 1], vocab)[0] if 0 <= q < len(allowed) else np.zeros(vocab, bool)
                    x = np.where(ok, x, -np.inf)
            if temperature is not None and temperature[r] > 0:
                x, e = x / float(temperature[r]), e / float(temperature[r])
                e += u * np.abs(x)
        out[r], slack[r] = x, e
    return out, slack
