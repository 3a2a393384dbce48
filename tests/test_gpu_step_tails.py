"""Attention where most of the output comes from tokens that weigh next to nothing each: a strong token without a value before, among or behind very many
weak ones, and scores that fall over a wide range, against the definition in 64 bits over the same inputs.

Tolerance, all relative to the output (the values that count share a sign), whatever the number of tokens:
* its one rounding, half a step;
* scores of d products in 32 bits: (d + 8) 2^-23 of the sum of their magnitudes, and 2^-22 (1 + 2 |x|) for the argument of the exponential;
  twice, for the weights above and below the line;
* weights in two terms of 16 bits: 2^-16 of each, and with float16 2^-21 of the largest in its 32 tokens, which here is at most 2^5 times
  the others: 2^-15 together.  Beside a strong token the others of its 32 are off by 2^-32 of it each, half the smallest step of float16 where the strong
  one is 2^7: together below 2^-27 of all, which is not relative to the output but times the largest value (of 20 tokens, 19 weak ones of
  e^-18 each are 2^-22 of all, and so off by 2^-5);
* sums: 2^-23 for each of the additions that one term goes through, 64 a tile of 128 tokens that a workgroup takes, and 600 to join them; twice.
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import exact_byte_level_amd as tt  # noqa: E402
from tests.test_gpu_step_attend import F8, TINY, TYPES  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()


def random(shape, seed):
    return torch.randn(shape, device="cuda", generator=torch.Generator("cuda").manual_seed(seed))


def check(query, keys, values, lengths, rows=None, scale=1.0, workers=256, **o):
    """query [N, H, D]; keys, values [n, heads, D] of one row, in blocks of 16."""
    n, kv, dim = keys.shape
    blocks = -(-n // 16)
    caches = [torch.cat([c, c.new_zeros(blocks * 16 - n, kv, dim, dtype=torch.float32).to(c.dtype)]).view(blocks, 16, kv, dim) if c.dtype != F8 else
              torch.cat([c.view(torch.uint8), torch.zeros(blocks * 16 - n, kv, dim, dtype=torch.uint8, device="cuda")]).view(F8).view(blocks, 16, kv, dim) for c in (keys, values)]
    table = torch.arange(blocks, dtype=torch.int32, device="cuda")[None]
    out, lse = tt.attend_cache(query, *caches, table, torch.tensor(lengths, dtype=torch.int32, device="cuda"), rows=torch.zeros(len(lengths), dtype=torch.int32, device="cuda"),
                               lse=True, scale=scale, **o)
    group = query.shape[1] // kv
    additions = 64 * (-(-(-(-n // 128)) // workers) + 1) + 600
    for i, length in enumerate(lengths):
        since = max(0, length - o["window"]) if o.get("window") else 0
        for h in range(query.shape[1]):
            k, v, q = keys[since:length, h // group].double(), values[since:length, h // group].double(), query[i, h].double()
            x = (k * q).sum(1) * scale
            products = float((k.abs() * q.abs()).sum(1).max()) * abs(scale)
            off = products * (dim + 8) * 2.0**-23 + 2.0**-22 * (1 + 2 * float(x.abs().max()))
            want = torch.softmax(x, 0)[None] @ v
            sums = float(torch.logsumexp(x, 0))
            room = want[0].abs() * (torch.finfo(query.dtype).eps / 2 + 2 * off + 2 * additions * 2.0**-23 + 2.0**-15) + TINY[query.dtype] / 2
            if query.dtype == torch.float16:
                room += 2.0**-27 * float(v.abs().max())
            error = (out[i, h].double() - want[0]).abs()
            assert (error <= room).all(), (i, h, float((error / want[0].abs()).max()), float((room / want[0].abs()).max()))
            assert abs(float(lse[i, h]) - sums) <= off + additions * 2.0**-23 + 2.0**-21 * (1 + abs(sums))


def weak(n, kv, dim, dst, seed):
    """Keys whose scores with a query near the first axis are small, and values of one sign."""
    keys = random((n, kv, dim), seed).mul_(0.25)
    keys[:, :, 0] = 0
    values = random((n, kv, dim), seed + 1).abs_().add_(0.5)
    return keys.to(dst), values.to(dst)


def axis(n, heads, dim, src, seed):
    query = random((n, heads, dim), seed).mul_(0.03)
    query[:, :, 0] = 1
    return query.to(src)


def put(cache, at, value):
    raw = cache.view(torch.uint8 if cache.dtype == F8 else torch.int16)
    raw[at] = torch.as_tensor(value, device="cuda", dtype=torch.float32).to(cache.dtype).view(raw.dtype)


@pytest.mark.parametrize("src, dst", TYPES)
@pytest.mark.parametrize("strength", [8.0, 14.0, 16.0, 18.0])
@pytest.mark.parametrize("n, heads, kv, dim", [(32_000, 2, 1, 64), (130_001, 4, 2, 128), (33_000, 1, 1, 256)])
def test_a_strong_token_without_a_value(src, dst, strength, n, heads, kv, dim):
    keys, values = weak(n, kv, dim, dst, n)
    for place in (0, n // 2, n - 1):
        k, v = keys.clone(), values.clone()
        put(k, (place, slice(None), 0), strength)
        put(v, (place,), torch.zeros(kv, dim))
        check(axis(1, heads, dim, src, place), k, v, [n], workers=512 // kv if dim < 256 else 256)


@pytest.mark.parametrize("src, dst", TYPES)
def test_strong_tokens_for_some_of_a_bundle(src, dst):
    """Queries of one row, some of which see the strong token, one by a window not."""
    n = 33_000
    keys, values = weak(n, 1, 64, dst, 5)
    put(keys, (40, slice(None), 0), 16.0)
    put(values, (40,), torch.zeros(1, 64))
    query = axis(6, 2, 64, src, 6)
    query[1, :, 0], query[2, :, 0], query[3, :, 0] = 1.125, 0.5, 0.0
    check(query, keys, values, [n, n - 5, n - 31, n - 32, 100, n - 200])
    check(query, keys, values, [n, n - 5, n - 31, n - 32, n - 65, n - 200], window=n - 60)


@pytest.mark.parametrize("src, dst", TYPES)
@pytest.mark.parametrize("falling", [True, False])
def test_scores_over_a_wide_range(src, dst, falling):
    """Scores between 0 and -20 in steps over the length, values only where they are below -8."""
    n, dim = 40_000, 64
    keys, values = weak(n, 1, dim, dst, 9)
    at = torch.arange(n, device="cuda")
    at = at if falling else n - 1 - at
    level = -torch.div(at * 41, n, rounding_mode="floor").float() / 2
    put(keys, (slice(None), 0, 0), level)
    raw = values.view(torch.uint8 if dst == F8 else torch.int16)
    raw[level > -8] = 0
    check(axis(2, 1, dim, src, 10), keys, values, [n, n - 77])


@pytest.mark.parametrize("src, dst", TYPES)
@pytest.mark.parametrize("strength", [10.0, 14.0, 16.0, 17.0, 18.0, 24.0])
@pytest.mark.parametrize("dim", [64, 128, 200])
def test_calls_with_a_workgroup_for_each_query(src, dst, strength, dim):
    """Many queries, so that each is one workgroup's: every wavefront of it meets a strong token first and has the weak ones to itself."""
    n, queries = 8000, 600
    keys, values = weak(n, 1, dim, dst, dim)
    for place in (0, 32, 64, 96):
        put(keys, (place, slice(None), 0), strength)
        put(values, (place,), torch.zeros(1, dim))
    query = axis(2, 1, dim, src, 3)
    check(torch.cat([query, query[:1].expand(queries - 2, 1, dim)]), keys, values, [n, n - 9] + [20] * (queries - 2), workers=1)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_weights_that_rise_and_fall_again_and_again(dtype):
    """Strong tokens without values and runs of weak ones in turn, by one workgroup: what is summed up keeps its scale."""
    n, queries, dim = 8000, 600, 64
    keys, values = weak(n, 1, dim, dtype, 21)
    at = torch.arange(n, device="cuda")
    level = torch.where(at // 128 % 3 == 0, torch.where(at // 128 % 2 == 0, 18.0, 30.0), 0.0)
    level[n // 2:] += 3.0
    put(keys, (slice(None), 0, 0), level)
    values.view(torch.int16)[level > 10] = 0
    query = axis(2, 1, dim, dtype, 22)
    check(torch.cat([query, query[:1].expand(queries - 2, 1, dim)]), keys, values, [n, n - 100] + [20] * (queries - 2), workers=1)
