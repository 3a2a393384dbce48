"""Shaping of logits on the GPU against the definition in 64 bits.

Tolerances: the definition says how far a computation in 32 bits may be off (half a step, 2^-24, of every
intermediate value, carried to the end), here with 2 percent for products of such errors; on top comes the one
rounding to the output's type, half a step of the value (and half the smallest subnormal step).
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import exact_byte_level_amd as tt  # noqa: E402
from tests import serve_oracle as so  # noqa: E402

TYPES = [(torch.float32, torch.float32), (torch.float16, torch.float16), (torch.float16, torch.float32),
         (torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32)]


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def near(got, want, slack):
    info = torch.finfo(got.dtype)
    tiny = {torch.float32: 2.0**-149, torch.float16: 2.0**-24, torch.bfloat16: 2.0**-133}[got.dtype]
    g = got.double().cpu().numpy()
    assert g.shape == want.shape
    assert np.array_equal(np.isnan(g), np.isnan(want))
    fine = np.isfinite(want)
    assert np.array_equal(g[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)])
    room = 1.02 * slack + info.eps / 2 * (np.abs(want) + slack) + tiny / 2
    bad = np.abs(g - np.where(fine, want, 0))[fine] > room[fine]
    assert not bad.any(), (g[fine][bad][:4], want[fine][bad][:4])


def options(rng, rows, vocab, cap, biases, sets):
    """Everything that shape_logits takes, as host arrays."""
    gen = np.minimum((rng.random((rows, cap)) ** 2 * vocab).astype(np.int32), vocab - 1)
    wild = rng.random(gen.shape) < 0.02
    gen[wild] = rng.choice(np.array([-1, vocab, 2**31 - 1, -2**31], np.int32), int(wild.sum()))
    count = rng.integers(0, 2 * biases + 1, rows)
    offsets = np.concatenate([[0], np.cumsum(count)]).astype(np.int64)
    n = int(offsets[-1])
    ids = rng.integers(-1, vocab + 1, n).astype(np.int32)
    word = lambda k: so.pack(rng.random((k, vocab)) < 0.5)  # noqa: E731
    f = lambda lo, hi: rng.uniform(lo, hi, rows).astype(np.float32)  # noqa: E731
    at = rng.integers(-3, sets + 1, rows).astype(np.int32)
    temperature = f(0.2, 2.0)
    temperature[rng.random(rows) < 0.2] = 0.0
    return dict(seen=word(rows), generated=gen, n_generated=rng.integers(-1, cap + 3, rows).astype(np.int32),
                repetition=f(0.8, 1.8), frequency=f(-0.5, 1.0), presence=f(-0.5, 1.0), bias_offsets=offsets, bias_ids=ids,
                bias_values=rng.normal(0, 5, n).astype(np.float32), allowed=word(sets), allowed_rows=at,
                temperature=temperature)


def host(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("src, dst", TYPES)
@pytest.mark.parametrize("rows, vocab, pad, cap, biases, sets", [
    (1, 1, 0, 1, 1, 1), (2, 7, 1, 3, 2, 1), (1, 31, 0, 40, 3, 2), (3, 32, 5, 9, 1, 3), (5, 4095, 2, 100, 9, 4),
    (2, 4096, 0, 50, 0, 2), (4, 4097, 3, 5000, 30, 3), (3, 20_003, 1, 700, 100, 5), (40, 1000, 0, 64, 4, 8),
    (2, 100_257, 7, 9000, 300, 2),
    # from here on enough tiles for the large ones
    (1100, 37, 0, 20, 3, 4), (1030, 300, 1, 64, 9, 7), (60, 70_003, 3, 3000, 300, 5), (350, 9000, 0, 500, 40, 5)])
def test_everything_at_once(src, dst, rows, vocab, pad, cap, biases, sets):
    rng = np.random.default_rng(rows * 31 + vocab)
    wide = torch.from_numpy(rng.normal(0, 4, (rows, vocab + pad)).astype(np.float32)).cuda().to(src)
    logits = wide[:, :vocab]
    o = options(rng, rows, vocab, cap, biases, sets)
    want, slack = so.shape_logits(host(logits), **o)
    keep = torch.full((rows, vocab + 3), 7.0, dtype=dst, device="cuda")
    tt.shape_logits_into(logits, keep[:, :vocab], **{k: dev(v) for k, v in o.items()})
    near(keep[:, :vocab], want, slack)
    assert (keep[:, vocab:] == 7).all()
    if src == dst:  # in place, and nothing beside the rows
        before = wide[:, vocab:].clone()
        tt.shape_logits_into(logits, logits, **{k: dev(v) for k, v in o.items()})
        assert torch.equal(logits.view(torch.int16 if src != torch.float32 else torch.int32),
                           keep[:, :vocab].view(torch.int16 if src != torch.float32 else torch.int32))
        assert torch.equal(wide[:, vocab:], before)


@pytest.mark.parametrize("only", [("seen", "repetition"), ("generated", "repetition"), ("generated", "n_generated", "frequency"),
                                  ("generated", "n_generated", "presence"), ("bias_offsets", "bias_ids", "bias_values"),
                                  ("allowed", "allowed_rows"), ("temperature",), ()])
def test_each_by_itself(only):
    rng = np.random.default_rng(len(only))
    rows, vocab = 4, 5001
    logits = torch.from_numpy(rng.normal(0, 4, (rows, vocab)).astype(np.float32)).cuda()
    o = {k: v for k, v in options(rng, rows, vocab, 300, 20, 3).items() if k in only}
    want, slack = so.shape_logits(host(logits), **o)
    got = tt.shape_logits(logits, **{k: dev(v) for k, v in o.items()})
    near(got, want, slack)
    if not only:
        assert torch.equal(got, logits)
    half = tt.shape_logits(logits.bfloat16(), dtype=torch.bfloat16, **{k: dev(v) for k, v in o.items()})
    near(half, *so.shape_logits(host(logits.bfloat16()), **o))


@pytest.mark.parametrize("src, dst", TYPES)
def test_infinities_and_nan(src, dst):
    """A token that is not allowed is -inf whatever its logit; what is allowed keeps its infinity or NaN; masks of the
    type's lowest value stay finite."""
    rng = np.random.default_rng(2)
    rows, vocab = 5, 300
    x = rng.normal(0, 2, (rows, vocab)).astype(np.float32)
    low = float(torch.finfo(src).min)
    for value in (np.inf, -np.inf, np.nan, low, 0.0, -0.0):
        x[rng.random(x.shape) < 0.1] = value
    logits = torch.from_numpy(x).cuda().to(src)
    o = options(rng, rows, vocab, 50, 10, 3)
    o["allowed_rows"] = np.array([0, 1, -1, -2, 3], np.int32)  # rows 2 and 4 have nothing left, row 3 everything
    o["repetition"][:] = 1.0  # the lowest value times a penalty is past the type's range
    o["temperature"][:] = 1.0
    o["frequency"][:] = 0.5
    o["bias_values"] = np.clip(o["bias_values"], -1, 1)  # stays short of the next step past float16's lowest
    want, slack = so.shape_logits(host(logits), **o)
    got = tt.shape_logits(logits, dtype=dst, **{k: dev(v) for k, v in o.items()})
    near(got, want, slack)
    assert (got[[2, 4]] == -float("inf")).all() and torch.isnan(got[3]).any()


def test_an_empty_set_and_a_set_of_one():
    rows, vocab = 3, 70
    logits = torch.randn(rows, vocab, device="cuda")
    member = np.zeros((rows, vocab), bool)
    member[1, 69] = True
    out = tt.shape_logits(logits, allowed=dev(so.pack(member)))
    assert (out[[0, 2]] == -float("inf")).all()
    assert torch.isfinite(out[1]).sum() == 1 and out[1, 69] == logits[1, 69]
    none = torch.empty((0, so.words(vocab)), dtype=torch.int32, device="cuda")  # no sets at all: none is there to go by
    rows_of = torch.tensor([-2, 0, -1], dtype=torch.int32, device="cuda")
    out = tt.shape_logits(logits, allowed=none, allowed_rows=rows_of)
    assert torch.equal(out[0], logits[0]) and (out[1:] == -float("inf")).all()


def test_counts_of_one_token_many_times():
    """One token 70,000 times (past 16 bits), another once; the same bias entry twice: the last counts."""
    vocab, cap = 9000, 70_001
    gen = np.full((1, cap), 8191, np.int32)
    gen[0, 5] = 0
    logits = torch.zeros(1, vocab, device="cuda")
    o = dict(generated=gen, frequency=np.array([1.0], np.float32), presence=np.array([0.5], np.float32),
             bias_offsets=np.array([0, 4], np.int64), bias_ids=np.array([4, 4, 4, 5], np.int32),
             bias_values=np.array([1, 2, 3, 4], np.float32))
    got = tt.shape_logits(logits, **{k: dev(v) for k, v in o.items()})
    assert got[0, 8191] == -70_000.5 and got[0, 0] == -1.5 and got[0, 4] == 3 and got[0, 5] == 4
    assert int((got != 0).sum()) == 4


def test_bias_bounds_are_kept():
    logits = torch.zeros(4, 40, device="cuda")
    o = dict(bias_offsets=dev(np.array([-9, 2, 1, 2**62, -1], np.int64)), bias_ids=dev(np.array([1, 2, 3], np.int32)),
             bias_values=dev(np.array([1, 2, 3], np.float32)))
    got = tt.shape_logits(logits, **o)
    want = torch.zeros(4, 40, device="cuda")
    want[0, 1], want[0, 2], want[2, 2], want[2, 3] = 1, 2, 2, 3
    assert torch.equal(got, want)


def test_rows_that_share_memory_and_single_positions():
    """A slice of the last position of [R, T, V], one row for all, and rows far apart."""
    rng = np.random.default_rng(4)
    full = torch.from_numpy(rng.normal(0, 3, (3, 5, 1001)).astype(np.float32)).cuda().half()
    o = options(rng, 3, 1001, 30, 4, 3)
    want, slack = so.shape_logits(host(full[:, -1]), **o)
    near(tt.shape_logits(full[:, -1], **{k: dev(v) for k, v in o.items()}), want, slack)
    one = full[:1, 0].expand(3, 1001)
    want, slack = so.shape_logits(host(one), **o)
    near(tt.shape_logits(one, **{k: dev(v) for k, v in o.items()}), want, slack)
    with pytest.raises(tt.TTError):  # what is written may not be shared
        tt.shape_logits_into(full[:, 0].float(), torch.empty(1, 1001, device="cuda").expand(3, 1001))


def test_refusals():
    x = torch.zeros(2, 64, device="cuda")
    bad = [dict(seen=torch.zeros(2, 1, dtype=torch.int32, device="cuda")), dict(seen=torch.zeros(2, 2, device="cuda")),
           dict(generated=torch.zeros(3, 4, dtype=torch.int32, device="cuda")), dict(repetition=torch.ones(3, device="cuda")),
           dict(repetition=torch.ones(2)), dict(bias_offsets=torch.zeros(3, dtype=torch.int64, device="cuda")),
           dict(bias_ids=torch.zeros(3, dtype=torch.int32, device="cuda")), dict(allowed=torch.zeros(1, 2, dtype=torch.int32, device="cuda")),
           dict(allowed_rows=torch.zeros(2, dtype=torch.int32, device="cuda")), dict(temperature=torch.ones(2, dtype=torch.float64, device="cuda")),
           dict(temperature=torch.ones(4, device="cuda")[::2])]
    for o in bad:
        with pytest.raises(ValueError):
            tt.shape_logits(x, **o)
    for y in (torch.zeros(2, 63, device="cuda"), torch.zeros(3, 64, device="cuda"), torch.zeros(2, 64, device="cuda").half(),
              torch.zeros(2, 128, device="cuda")[:, ::2], torch.zeros(2, 64)):
        with pytest.raises(ValueError):
            tt.shape_logits_into(x, y)
    assert tt.shape_logits(torch.zeros(0, 64, device="cuda")).shape == (0, 64)
    assert tt.shape_logits(torch.zeros(3, 0, device="cuda")).shape == (3, 0)


def test_on_another_stream_and_in_a_graph():
    rng = np.random.default_rng(6)
    rows, vocab = 3, 9001
    o = options(rng, rows, vocab, 100, 10, 4)
    d = {k: dev(v) for k, v in o.items()}
    x = torch.from_numpy(rng.normal(0, 4, (rows, vocab)).astype(np.float32)).cuda()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    got = tt.shape_logits(x, stream=stream, **d)
    stream.synchronize()
    near(got, *so.shape_logits(host(x), **o))
    out = torch.empty_like(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tt.shape_logits_into(x, out, **d)
    for turn in range(4):
        x.copy_(torch.from_numpy(rng.normal(0, 4, (rows, vocab)).astype(np.float32)))
        o["generated"] = rng.integers(0, vocab, o["generated"].shape).astype(np.int32)
        d["generated"].copy_(dev(o["generated"]))
        graph.replay()
        torch.cuda.synchronize()
        near(out, *so.shape_logits(host(x), **o))
        tt.shape_logits(x, **d)
