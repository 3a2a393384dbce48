"""Plain definitions of the operators around the model (include/tt_step.h): numpy in 64 bits, one token, query or row after
the other, sharing no code with the package."""
import math

import numpy as np

E4M3_MOST = 448.0


def e4m3_values():
    """The value of each byte: a sign, four bits of exponent (bias 7), three of mantissa; 127 and 255 are NaN."""
    out = np.empty(256)
    for b in range(256):
        e, m = b >> 3 & 15, b & 7
        v = (1 + m / 8) * 2.0**(e - 7) if e else m / 8 * 2.0**-6
        out[b] = math.nan if b & 127 == 127 else -v if b & 128 else v
    return out


def e4m3(x):
    """The nearest e4m3 value of each of x (as bytes), ties to even; beyond the largest it is the largest."""
    values = e4m3_values()[:127]
    out = np.empty(x.shape, np.uint8)
    for at in np.ndindex(x.shape):
        v = float(x[at])
        if math.isnan(v):
            out[at] = 127
            continue
        a = min(abs(v), E4M3_MOST)
        hi = int(np.searchsorted(values, a))
        if hi and (hi == 127 or a - values[hi - 1] < values[hi] - a or (a - values[hi - 1] == values[hi] - a and (hi - 1) % 2 == 0)):
            hi -= 1
        out[at] = hi | (128 if math.copysign(1, v) < 0 else 0)
    return out


def attend(query, keys, values, table, lengths, rows=None, scale=1.0, window=0, softcap=0.0, key_scale=None, value_scale=None):
    """(out, lse, how far out may be off before its rounding, how far lse may be off).

    query [N, H, D]; keys, values [blocks, block_size, heads, D] (64 bits).  The bounds are those of a computation in 32 bits:
    a sum of n terms is off by n half steps and as many again where a matrix instruction cuts off instead of rounding, n * 2^-23 of
    the sum of their magnitudes; an exponential, a logarithm or a tanh by 2^-22, and by as much as its argument is off.
    Weights go in two terms of 16 bits, off by 2^-16 (with float16, whose smallest step is 2^-24, by 2^-24 of the largest weight)."""
    n, heads, dim = query.shape
    blocks, bs, kv, _ = keys.shape
    out, lse = np.zeros(query.shape), np.full((n, heads), -np.inf)
    slack, lse_slack = np.zeros(query.shape), np.zeros((n, heads))
    for i in range(n):
        row = i if rows is None else int(rows[i])
        if not 0 <= row < len(table):
            continue
        length = min(int(lengths[i]), table.shape[1] * bs)
        places = range(max(0, length - window) if window else 0, max(0, length))
        at = [(int(table[row, p // bs]), p % bs) for p in places]
        at = [(b, p) for b, p in at if 0 <= b < blocks]
        if not at:
            continue
        b, p = np.array(at).T
        for h in range(heads):
            g = h // (heads // kv)
            k, v = keys[b, p, g], values[b, p, g]
            by = scale * (1.0 if key_scale is None else float(key_scale[g]))
            x = k @ query[i, h] * by
            off = np.max(np.abs(k) @ np.abs(query[i, h])) * abs(by) * (dim + 8) * 2.0**-23
            if softcap:
                x = softcap * np.tanh(x / softcap)
                off += 2.0**-20 * np.abs(x).max()  # of a tanh from 1/4 up; below that less
            top = x.max()
            if top == -np.inf:
                continue
            w = np.exp(x - top)
            total = w.sum()
            lse[i, h] = top + math.log(total)
            # the argument of the power of two: its own rounding beside the score's
            off += 2.0**-22 * (1 + 2 * np.abs(x).max())
            few = (len(at) + 64) * 2.0**-23
            lse_slack[i, h] = off + few + 2.0**-21 * (1 + abs(lse[i, h]))
            s = 1.0 if value_scale is None else float(value_scale[g])
            out[i, h] = w @ v / total * s
            slack[i, h] = (w @ np.abs(v) / total * (2 * off + 2 * few + 2.0**-16) + 2.0**-24 * np.abs(v).sum(0) / total) * abs(s)
    return out, lse, slack, lse_slack


def sample(logits, uniform, temperature=None, top_k=None, top_p=None, min_p=None):
    """(tokens, logprobs, how many tokens each row keeps)."""
    tokens, logprobs, kept = [], [], []
    for r, x in enumerate(logits.astype(np.float64)):
        x = np.where(np.isnan(x), -np.inf, x)
        if not len(x) or x.max() == -np.inf:
            tokens.append(-1)
            logprobs.append(-np.inf)
            kept.append(0)
            continue
        t = 1.0 if temperature is None else float(temperature[r])
        order = np.argsort(-x, kind="stable")
        top = x[order[0]]
        if not t > 0:
            order, w = order[:1], np.ones(1)
        elif top == np.inf:
            w = (x[order] == np.inf).astype(np.float64)
        else:
            with np.errstate(invalid="ignore"):
                w = np.exp((x[order] - top) / t)
            w[(x[order] == -np.inf) | (w < 2.0**-1000)] = 0
        n = len(order)
        if top_k is not None and top_k[r] > 0:
            n = min(n, int(top_k[r]))
        if top_p is not None and top_p[r] < 1:
            sums = np.cumsum(w[:n])
            n = min(n, 1 + int((sums < float(top_p[r]) * sums[-1]).sum()))
        if min_p is not None and min_p[r] > 0:
            n = max(1, min(n, int((w >= float(min_p[r])).sum())))
        ids = np.sort(order[:n])
        weight = np.zeros(len(x))
        weight[order[:n]] = w[:n]
        sums = np.cumsum(weight[ids])
        u = float(uniform[r])
        u = 0.0 if math.isnan(u) else min(max(u, 0.0), 1 - 2.0**-24)
        at = int(np.searchsorted(sums, u * sums[-1], side="right"))
        tokens.append(int(ids[at]))
        logprobs.append(math.log(weight[ids[at]] / sums[-1]))
        kept.append(n)
    return np.array(tokens, np.int32), np.array(logprobs), np.array(kept)
