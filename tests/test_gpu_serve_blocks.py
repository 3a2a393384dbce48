"""Block tables on the GPU against the sequential definition: prompts, single tokens, empty and idle rows, odd block
sizes, row counts around a workgroup's, data errors, strides, in-place updates, other streams, graph replays."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import exact_byte_level_amd as tt  # noqa: E402
from tests import serve_oracle as so  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def random_state(rng, rows, block, context, most_new, idle=0.2, spare=5, extra_width=1):
    """lengths, table, free list and offsets of a cache in use."""
    lengths = rng.integers(0, context + 1, rows).astype(np.int32)
    lengths[rng.random(rows) < idle] = -1
    new = rng.integers(0, most_new + 1, rows)
    new[rng.random(rows) < 0.3] = 0
    offsets = np.concatenate([[0], np.cumsum(new)]).astype(np.int64)
    start = np.maximum(lengths, 0).astype(np.int64)
    held = -(-start // block)
    want = -(-(start + np.maximum(new, 1)) // block)
    width = int(want.max(initial=0)) + extra_width
    pool = int(want.sum()) + spare
    order = rng.permutation(pool).astype(np.int32)
    table = np.full((rows, width), -1, np.int32)
    at = 0
    for r in range(rows):
        table[r, :held[r]] = order[at:at + held[r]]
        at += held[r]
    free = np.full(pool, -7, np.int32)
    free[:pool - at] = order[at:]
    return lengths, table, free, pool - at, offsets


def run_plan(lengths, table, free, n_free, block, places, offsets, in_place=False, pad=0, stream=None):
    wide = np.full((table.shape[0], table.shape[1] + pad), 77, np.int32)
    wide[:, :table.shape[1]] = table
    t = dev(wide)
    d = dict(lengths=dev(lengths), n_free=dev(np.array([n_free], np.int32)))
    slots = torch.full((places,), 99, dtype=torch.int64, device="cuda")
    pos, rows = (torch.full((places,), 99, dtype=torch.int32, device="cuda") for _ in range(2))
    out_n = torch.full((1,), 99, dtype=torch.int64, device="cuda")
    more = {} if in_place else dict(out_lengths=torch.empty_like(d["lengths"]), out_n_free=torch.empty_like(d["n_free"]))
    free_d = dev(free)
    off_d = None if offsets is None else dev(offsets)
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    tt.plan_blocks_into(d["lengths"], t[:, :table.shape[1]], free_d, d["n_free"], block, slots, out_n, offsets=off_d,
                        positions=pos, rows=rows, stream=stream, **more)
    torch.cuda.synchronize()
    assert np.array_equal(free_d.cpu().numpy(), free)
    if pad:
        assert (t[:, table.shape[1]:] == 77).all()
    if not in_place:
        assert np.array_equal(d["lengths"].cpu().numpy(), lengths)
    return dict(table=t[:, :table.shape[1]].cpu().numpy(), lengths=more.get("out_lengths", d["lengths"]).cpu().numpy(),
                n_free=int(more.get("out_n_free", d["n_free"])), slots=slots.cpu().numpy(), positions=pos.cpu().numpy(),
                rows=rows.cpu().numpy(), n=int(out_n))


def same(got, want):
    assert sorted(got) == sorted(want)
    for k in want:
        assert np.array_equal(got[k], want[k]), k


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("rows, block, context, most_new, pad", [
    (1, 16, 0, 1, 0), (1, 16, 40, 100, 3), (1, 1, 5, 9000, 0), (3, 7, 30, 40, 1), (64, 16, 500, 300, 0),
    (255, 24, 100, 40, 0), (256, 32, 64, 64, 5), (257, 17, 90, 33, 0), (700, 128, 2000, 5, 0), (1300, 3, 20, 12, 0),
    (5, 1 << 20, 100, 5000, 0)])
def test_prompts(rows, block, context, most_new, pad, in_place):
    rng = np.random.default_rng(rows * 1000 + block)
    lengths, table, free, n_free, offsets = random_state(rng, rows, block, context, most_new)
    for places in (int(offsets[-1]), int(offsets[-1]) + 300):
        want = so.plan(lengths, table, free, n_free, block, places, offsets)
        assert want["n"] >= 0
        same(run_plan(lengths, table, free, n_free, block, places, offsets, in_place, pad), want)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("rows, block, context", [(1, 16, 0), (1, 16, 16), (8, 16, 100), (256, 16, 64), (257, 5, 50),
                                                  (3001, 16, 40)])
def test_single_tokens(rows, block, context, in_place):
    rng = np.random.default_rng(rows + block)
    lengths, table, free, n_free, _ = random_state(rng, rows, block, context, 0)
    for places in (rows, rows + 9):
        want = so.plan(lengths, table, free, n_free, block, places)
        assert want["n"] >= 0
        same(run_plan(lengths, table, free, n_free, block, places, None, in_place), want)


def test_no_rows_no_places():
    empty = np.zeros(0, np.int32)
    got = run_plan(empty, np.zeros((0, 4), np.int32), np.arange(3, dtype=np.int32), 2, 16, 0, np.zeros(1, np.int64))
    assert got["n"] == 0 and got["n_free"] == 2
    got = run_plan(empty, np.zeros((0, 4), np.int32), empty, 0, 16, 5, None)
    assert got["n"] == 0 and (got["slots"] == -1).all()
    # rows without a single new token, and a table without room
    same(run_plan(np.array([-1, 0], np.int32), np.zeros((2, 0), np.int32), empty, 0, 16, 3, np.zeros(3, np.int64)),
         so.plan(np.array([-1, 0], np.int32), np.zeros((2, 0), np.int32), empty, 0, 16, 3, np.zeros(3, np.int64)))


def test_long_cache_passes_32_bits():
    """Slots beyond 2^32: block ids near 2^31 with blocks of 4,096 tokens."""
    lengths = np.array([4095, 5000], np.int32)
    table = np.array([[2**31 - 5, -1, -1], [2**31 - 9, 2**31 - 8, -1]], np.int32)
    free = np.array([2**31 - 1, 2**31 - 2], np.int32)
    offsets = np.array([0, 3, 4], np.int64)
    want = so.plan(lengths, table, free, 2, 4096, 4, offsets)
    assert want["slots"].max() > 2**42
    same(run_plan(lengths, table, free, 2, 4096, 4, offsets), want)


def test_block_that_is_missing_gives_no_slot():
    lengths = np.array([20, 4], np.int32)
    table = np.array([[3, -1], [4, -1]], np.int32)  # the block of tokens 16.. of row 0 is missing
    want = so.plan(lengths, table, np.array([8, 9], np.int32), 2, 16, 2)
    assert want["slots"].tolist() == [-1, 68]
    same(run_plan(lengths, table, np.array([8, 9], np.int32), 2, 16, 2, None), want)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("many", [False, True])
def test_data_errors_change_nothing(many, in_place):
    rng = np.random.default_rng(5)
    lengths, table, free, n_free, offsets = random_state(rng, 40, 16, 100, 200 if many else 4, idle=0.0, spare=0)
    places = int(offsets[-1]) + (3000 if many else 0)
    n = len(free)
    falling = offsets.copy()
    falling[7] = falling[9] + 1
    late = offsets + 1
    long = lengths.copy()
    long[3] = table.shape[1] * 16 + 1
    used = -(-(lengths + np.diff(offsets)) // 16) - -(-lengths // 16)
    cases = [(lengths, n_free, falling, -7), (lengths, n_free, late, -7), (lengths, -1, offsets, -1),
             (lengths, n + 1, offsets, -1), (long, n_free, offsets, -8), (lengths, int(used.sum()) - 1, offsets, -11),
             (lengths, n_free, np.concatenate([offsets[:-1], [places + 1]]), -8)]
    huge = offsets.copy()
    huge[1:] += 2**62
    cases.append((lengths, n_free, huge, -8))
    for lens, free_count, off, code in cases:
        want = so.plan(lens, table, free, free_count, 16, places, off)
        assert want["n"] == code
        same(run_plan(lens, table, free, free_count, 16, places, off, in_place), want)
    want = so.plan(lengths, table, free, int(used.sum()), 16, places, offsets)  # just enough blocks
    assert want["n"] >= 0 and want["n_free"] == 0
    same(run_plan(lengths, table, free, int(used.sum()), 16, places, offsets, in_place), want)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("rows, block, context, share", [(1, 16, 0, 1.0), (1, 16, 33, 1.0), (16, 16, 300, 0.2),
                                                         (256, 3, 200, 0.5), (257, 24, 900, 0.9), (1000, 5, 700, 0.4),
                                                         (600, 16, 9000, 1.0), (300, 16, 50, 0.0)])
def test_release(rows, block, context, share, in_place):
    rng = np.random.default_rng(rows + context)
    lengths, table, free, n_free, _ = random_state(rng, rows, block, context, 0)
    done = (rng.random(rows) < share)
    full = len(free) - n_free  # room in the list
    for kind in (np.uint8, bool):
        want = so.release(lengths, done, table, free, n_free, block)
        assert want["n"] >= 0 and want["n"] <= full
        check_release(lengths, done.astype(kind), table, free, n_free, block, in_place, want)


def check_release(lengths, done, table, free, n_free, block, in_place, want):
    d_len, d_n, d_free, d_table = dev(lengths), dev(np.array([n_free], np.int32)), dev(free), dev(table)
    out_n = torch.full((1,), 99, dtype=torch.int64, device="cuda")
    more = {} if in_place else dict(out_lengths=torch.empty_like(d_len), out_n_free=torch.empty_like(d_n))
    tt.release_blocks_into(d_len, dev(done), d_table, d_free, d_n, block, out_n, **more)
    got = dict(lengths=more.get("out_lengths", d_len).cpu().numpy(), n_free=int(more.get("out_n_free", d_n)),
               free=d_free.cpu().numpy(), n=int(out_n))
    same(got, want)
    assert np.array_equal(d_table.cpu().numpy(), table)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("rows", [9, 900])
def test_release_data_errors(rows, in_place):
    rng = np.random.default_rng(8)
    lengths, table, free, n_free, _ = random_state(rng, rows, 16, 400, 0, idle=0.0, spare=0)
    done = np.ones(rows, np.uint8)
    long = lengths.copy()
    long[rows // 2] = table.shape[1] * 16 + 1
    for lens, count, code in ((long, n_free, -8), (lengths, n_free + 1, -8), (lengths, -3, -1), (lengths, len(free) + 1, -1)):
        want = so.release(lens, done, table, free, count, 16)
        assert want["n"] == code
        check_release(lens, done, table, free, count, 16, in_place, want)


def test_a_cache_through_its_life():
    """Admission, steps, ends and re-admission through BlockTable, on a stream of its own; no block is held twice."""
    rng = np.random.default_rng(3)
    rows, width, blocks, block = 50, 20, 700, 8
    cache = tt.BlockTable(rows, width, blocks, block)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    lengths, table = np.full(rows, -1, np.int32), np.full((rows, width), -1, np.int32)
    free, n_free = np.arange(blocks - 1, -1, -1, dtype=np.int32), blocks
    for turn in range(12):
        new = np.where((lengths < 0) & (rng.random(rows) < 0.6), rng.integers(1, 60, rows), 0)
        offsets = np.concatenate([[0], np.cumsum(new)]).astype(np.int64)
        for off in (offsets, None, None):
            want = so.plan(lengths, table, free, n_free, block, rows if off is None else int(off[-1]), off)
            if off is None:
                slots, positions, where = cache.plan(stream=stream)
            else:
                with torch.cuda.stream(stream):
                    off = dev(off)
                slots, positions, where = cache.plan(off, stream=stream)
            torch.cuda.synchronize()
            assert np.array_equal(slots.cpu().numpy(), want["slots"])
            assert np.array_equal(positions.cpu().numpy(), want["positions"])
            assert np.array_equal(where.cpu().numpy(), want["rows"])
            lengths, table, n_free = want["lengths"], want["table"], want["n_free"]
            live = slots[slots >= 0]
            assert live.unique().numel() == live.numel()
        done = (rng.random(rows) < 0.5) | (lengths > 100)
        back = so.release(lengths, done, table, free, n_free, block)
        with torch.cuda.stream(stream):
            done = dev(done)
        assert cache.release(done, stream=stream) == back["n"]
        lengths, free, n_free = back["lengths"], back["free"], back["n_free"]
        assert np.array_equal(cache.lengths.cpu().numpy(), lengths) and int(cache.n_free) == n_free
        assert np.array_equal(cache.free_blocks[:n_free].cpu().numpy(), free[:n_free])
        assert np.array_equal(cache.table.cpu().numpy(), table)
        held = [b for r in range(rows) for b in table[r, :-(-max(int(lengths[r]), 0) // block)]]
        assert sorted(held + free[:n_free].tolist()) == list(range(blocks))


def test_errors_are_raised():
    cache = tt.BlockTable(2, 4, 3, 16)
    with pytest.raises(tt.TTError) as e:
        cache.plan(dev(np.array([0, 40, 70], np.int64)))
    assert e.value.code == tt.TT_ENOBLOCKS
    assert cache.lengths.tolist() == [-1, -1] and int(cache.n_free) == 3
    with pytest.raises(ValueError, match="table has 2 rows, not 3"):
        tt.plan_blocks_into(dev(np.zeros(3, np.int32)), cache.table, cache.free_blocks, cache.n_free, 16,
                            torch.empty(3, dtype=torch.int64, device="cuda"), torch.empty(1, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError, match="slots"):
        tt.plan_blocks_into(cache.lengths, cache.table, cache.free_blocks, cache.n_free, 16,
                            torch.empty(3, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int64, device="cuda"))


@pytest.mark.parametrize("rows", [8, 2500])
def test_steps_in_a_graph(rows):
    """A captured step in place, replayed with eager steps between: every replay against the definition."""
    rng = np.random.default_rng(rows)
    lengths, table, free, n_free, _ = random_state(rng, rows, 4, 30, 0, spare=20 * rows, extra_width=9)
    cache = tt.BlockTable(rows, table.shape[1], len(free), 4)
    cache.lengths.copy_(dev(lengths))
    cache.table.copy_(dev(table))
    cache.free_blocks.copy_(dev(free))
    cache.n_free.fill_(n_free)
    slots = torch.empty(rows, dtype=torch.int64, device="cuda")
    out_n = torch.empty(1, dtype=torch.int64, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.plan_into(slots, out_n)
    for turn in range(7):
        want = so.plan(lengths, table, free, n_free, 4, rows)
        if turn % 3 == 2:
            cache.plan_into(slots, out_n)
        else:
            graph.replay()
        torch.cuda.synchronize()
        assert int(out_n) == want["n"] >= 0 and int(cache.n_free) == want["n_free"]
        assert np.array_equal(slots.cpu().numpy(), want["slots"])
        lengths, table, n_free = want["lengths"], want["table"], want["n_free"]
        assert np.array_equal(cache.lengths.cpu().numpy(), lengths)
        assert np.array_equal(cache.table.cpu().numpy(), table)
