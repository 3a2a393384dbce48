"""Quotients of shape_logits over the whole range of 32 bits: values from the smallest subnormal to infinity, zeros of either sign,
penalties and temperatures far from 1.

A result has to lie between the roundings of (exact value - e) and (exact value + e) to the output's type.  With
32-bit outputs e stands for no more than the reference's own 64 bits and a division's ties: 2^-40 of the value.  With 16-bit outputs
a quotient is two 32-bit roundings, 2^-24 of the value each, and half a 32-bit subnormal step.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import exact_byte_level_amd as tt  # noqa: E402

TYPES = [(torch.float32, torch.float32), (torch.float16, torch.float16), (torch.float16, torch.float32),
         (torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32)]
SHAPES = [(3, 301), (1100, 37)]  # tiles of both sizes


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()


def logits(rng, rows, vocab, kind, dtype):
    x = np.exp2(rng.uniform(-149, 128, (rows, vocab)) if kind != "common" else rng.uniform(-12, 6, (rows, vocab)))
    if kind == "largest":
        x = np.exp2(rng.uniform(125, 128, (rows, vocab)))
    x *= rng.choice([-1.0, 1.0], x.shape)
    if kind == "mixed":
        for v in (0.0, -0.0, np.inf, -np.inf, np.nan, float(torch.finfo(dtype).max), float(torch.finfo(dtype).min)):
            x[rng.random(x.shape) < 0.05] = v
    with np.errstate(over="ignore"):
        return torch.from_numpy(x.astype(np.float32)).to(dtype).cuda()


def check(got, want):
    """`want` in 64 bits."""
    dtype = got.dtype
    g = got.double().cpu().numpy()
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(g), nan)
    e = np.where(np.isfinite(want), np.abs(want), 0) * 2.0**-40
    if dtype != torch.float32:
        e = e * 2.0**17 * 1.001 + 2.0**-150
    with np.errstate(invalid="ignore", over="ignore"):
        lo, hi = (torch.from_numpy((want + s * e).astype(np.float32)).to(dtype).double().numpy() for s in (-1, 1))
    bad = ~nan & ~((lo <= g) & (g <= hi))
    assert not bad.any(), (g[bad][:4], want[bad][:4])
    assert np.array_equal(np.signbit(g[~nan]), np.signbit(want[~nan]))


def steps_of(values, rows, rng):
    return torch.from_numpy(rng.choice(np.array(values, np.float32), rows)).cuda()


DIVISORS = [0.7, 1.0, 3.0, 1e-35, 1e35, 1e-40, 2.0**-20, 2.0**-21, 2.0**100, 2.0**101, float(np.nextafter(np.float32(1), np.float32(0))),
            float(torch.finfo(torch.float32).max), float("inf")]


@pytest.mark.parametrize("kind", ["common", "wide", "mixed", "largest"])
@pytest.mark.parametrize("rows, vocab", SHAPES)
@pytest.mark.parametrize("src, dst", TYPES)
def test_temperature(src, dst, rows, vocab, kind):
    rng = np.random.default_rng(rows + vocab)
    x = logits(rng, rows, vocab, kind, src)
    t = steps_of(DIVISORS + [0.0, -1.0, -np.inf, np.nan], rows, rng) if rows > 10 else None
    for value in [None] if t is not None else DIVISORS + [0.0, -1.0, float("nan")]:
        temperature = t if value is None else torch.full((rows,), value, device="cuda")
        got = tt.shape_logits(x, dtype=dst, temperature=temperature)
        d = temperature.double().cpu().numpy()[:, None]
        with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
            check(got, x.double().cpu().numpy() / np.where(d > 0, d, 1.0))


@pytest.mark.parametrize("kind", ["common", "wide", "mixed", "largest"])
@pytest.mark.parametrize("rows, vocab", SHAPES)
@pytest.mark.parametrize("src, dst", TYPES)
def test_repetition(src, dst, rows, vocab, kind):
    rng = np.random.default_rng(rows + vocab + 1)
    x = logits(rng, rows, vocab, kind, src)
    seen = torch.full((rows, (vocab + 31) // 32), -1, dtype=torch.int32, device="cuda")
    r = steps_of(DIVISORS + [0.0, -2.0, -1e35, -np.inf], rows, rng) if rows > 10 else None
    for value in [None] if r is not None else DIVISORS + [0.0, -2.0, -1e35]:
        rho = r if value is None else torch.full((rows,), value, device="cuda")
        got = tt.shape_logits(x, dtype=dst, repetition=rho, seen=seen)
        d, x64 = rho.double().cpu().numpy()[:, None], x.double().cpu().numpy()
        with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
            check(got, np.where(x64 > 0, x64 / d, x64 * d))


@pytest.mark.parametrize("rows, vocab", SHAPES)
@pytest.mark.parametrize("src, dst", TYPES)
def test_nothing_to_do_keeps_every_bit(src, dst, rows, vocab):
    rng = np.random.default_rng(5)
    x = logits(rng, rows, vocab, "mixed", src)
    got, want = tt.shape_logits(x, dtype=dst), x.to(dst)
    whole = torch.int32 if dst == torch.float32 else torch.int16
    number = ~torch.isnan(want)
    assert torch.equal(torch.isnan(got), ~number)
    assert torch.equal(got.view(whole)[number], want.view(whole)[number])


def test_quotients_at_the_largest_value():
    """x / d rounds to the largest value where x times the reciprocal is infinite."""
    rng = np.random.default_rng(6)
    d = rng.uniform(0.25, 1.0, 2000).astype(np.float32)
    x = (float(torch.finfo(torch.float32).max) * d.astype(np.float64)).astype(np.float32)
    x = np.where(rng.random(2000) < 0.5, np.nextafter(x, np.float32(0)), x)
    want = x.astype(np.float64) / d
    reciprocal = np.float32(1) / d
    with np.errstate(over="ignore"):
        assert (np.isinf(x * reciprocal) & np.isfinite(want.astype(np.float32))).any()
    rows = np.repeat(x[:, None], 16, 1)
    check(tt.shape_logits(torch.from_numpy(rows).cuda(), temperature=torch.from_numpy(d).cuda()), np.repeat(want[:, None], 16, 1))
