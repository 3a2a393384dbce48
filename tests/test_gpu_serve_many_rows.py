"""Block tables of more rows than a workgroup takes at a time, in place and with outputs of their own: blocks given back over
several chunks of 1,024 rows, and data errors of plans and releases."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import exact_byte_level_amd as tt  # noqa: E402,F401
from tests import serve_oracle as so  # noqa: E402
from tests.test_gpu_serve_blocks import check_release, random_state, run_plan, same  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()


def done_rows(rng, rows, which):
    """Truth values of the rows that end."""
    at = np.arange(rows)
    if which == "all":
        return np.ones(rows, bool)
    if which == "some":
        return rng.random(rows) < 0.4
    if which == "none":
        return np.zeros(rows, bool)
    if which == "last":
        return at == rows - 1
    return (at // 1024 % 2 == 1) & (rng.random(rows) < 0.7)  # chunks without a single one between others


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("which", ["all", "some", "none", "last", "odd chunks"])
@pytest.mark.parametrize("rows, block, context", [
    (1024, 16, 300), (1025, 16, 40), (1025, 3, 700), (2048, 16, 900), (2049, 5, 300), (5000, 7, 200), (3100, 1, 60)])
def test_release(rows, block, context, which, in_place):
    rng = np.random.default_rng(rows + context)
    lengths, table, free, n_free, _ = random_state(rng, rows, block, context, 0)
    done = done_rows(rng, rows, which)
    want = so.release(lengths, done, table, free, n_free, block)
    assert want["n"] >= 0 and (want["n"] > 0 or which in ("none", "last", "odd chunks"))
    check_release(lengths, done, table, free, n_free, block, in_place, want)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("rows", [1025, 3000])
def test_release_data_errors(rows, in_place):
    rng = np.random.default_rng(rows)
    lengths, table, free, n_free, _ = random_state(rng, rows, 16, 400, 0, idle=0.0, spare=0)
    done = np.ones(rows, np.uint8)
    cases = [(lengths, n_free + 1, -8), (lengths, -3, -1), (lengths, len(free) + 1, -1)]
    for at in (0, 1023, 1024, rows - 1):
        long = lengths.copy()
        long[at] = table.shape[1] * 16 + 1
        cases.append((long, n_free, -8))
    for lens, count, code in cases:
        want = so.release(lens, done, table, free, count, 16)
        assert want["n"] == code
        check_release(lens, done, table, free, count, 16, in_place, want)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("rows", [257, 1025, 2300])
def test_plan_data_errors(rows, in_place):
    rng = np.random.default_rng(rows)
    lengths, table, free, n_free, offsets = random_state(rng, rows, 16, 100, 12, idle=0.0, spare=0)
    places = int(offsets[-1]) + 1500
    used = -(-(lengths + np.diff(offsets)) // 16) - -(-lengths // 16)
    cases = [(lengths, -1, offsets, -1), (lengths, len(free) + 1, offsets, -1), (lengths, int(used.sum()) - 1, offsets, -11),
             (lengths, n_free, np.concatenate([offsets[:-1], [places + 1]]), -8)]
    for at in (0, 255, 256, rows - 1):
        long, falling = lengths.copy(), offsets.copy()
        long[at] = table.shape[1] * 16 + 1
        falling[at + 1:] -= falling[at + 1] + 1 if at == 0 else falling[at + 1] - falling[at] + 1
        cases += [(long, n_free, offsets, -8), (lengths, n_free, falling, -7)]
    for lens, free_count, off, code in cases:
        want = so.plan(lens, table, free, free_count, 16, places, off)
        assert want["n"] == code
        same(run_plan(lens, table, free, free_count, 16, places, off, in_place), want)
    want = so.plan(lengths, table, free, int(used.sum()), 16, places, offsets)  # just enough blocks
    assert want["n"] >= 0 and want["n_free"] == 0
    same(run_plan(lengths, table, free, int(used.sum()), 16, places, offsets, in_place), want)
    # a token each: rows at the end of their last block need one, and there is one too few
    short = int((lengths % 16 == 0).sum()) - 1
    want = so.plan(lengths, table, free, short, 16, rows)
    assert want["n"] == -11
    same(run_plan(lengths, table, free, short, 16, rows, None, in_place), want)
