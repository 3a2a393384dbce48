"""Writing to a paged cache on the GPU, element by element against the definition: exact, since every element is divided and
rounded once."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import exact_byte_level_amd as tt  # noqa: E402
from tests import step_oracle as so  # noqa: E402

F8 = torch.float8_e4m3fn
TYPES = [(torch.bfloat16, torch.bfloat16), (torch.float16, torch.float16), (torch.float32, torch.bfloat16), (torch.float32, torch.float16),
         (torch.float32, F8), (torch.float16, F8), (torch.bfloat16, F8)]


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()


def raw(t):
    """The elements' bits on the host; bytes and words are one entry each."""
    return t.contiguous().view(torch.uint8 if t.element_size() == 1 else torch.int16).cpu().numpy()


def expected(x, scale, dtype):
    """Bits of x [N, heads, dim] / scale in a type: the quotient in 32 bits, then the one rounding."""
    q = x.float().cpu().numpy()
    if scale is not None:
        q = (q / scale.cpu().numpy()[None, :, None]).astype(np.float32)
    return so.e4m3(q) if dtype == F8 else raw(torch.from_numpy(q).to(dtype))


def check(n, heads, dim, blocks, bs, src, dst, scaled, by_head=False, seed=0, wild=True):
    rng, g = np.random.default_rng(seed), torch.Generator("cuda").manual_seed(seed)
    shape = (blocks, heads, bs, dim) if by_head else (blocks, bs, heads, dim)
    caches = [torch.randn(shape, device="cuda", generator=g).to(dst) for _ in range(2)]
    if by_head:
        caches = [c.transpose(1, 2) for c in caches]
    made = torch.randn((n, 2, heads, dim), device="cuda", generator=g).mul_(4).to(src)
    if wild and n and src != torch.float16:
        made.view(-1)[:: 37] *= 1000
    slots = rng.permutation(blocks * bs)[:n].astype(np.int64)
    if wild and n > 3:
        slots[rng.random(n) < 0.2] = rng.choice(np.array([-1, -2**63, blocks * bs, 2**40, 2**63 - 1], np.int64), 1)
    scale = [torch.from_numpy(rng.uniform(0.01, 3, heads).astype(np.float32)).cuda() if scaled else None for _ in range(2)]
    want = [raw(c).copy() for c in caches]
    live = (slots >= 0) & (slots < blocks * bs)
    for k in range(2):
        got = expected(made[:, k], scale[k], dst)
        want[k][slots[live] // bs, slots[live] % bs] = got[live]
    tt.write_cache_into(made[:, 0], made[:, 1], torch.from_numpy(slots).cuda(), *caches, key_scale=scale[0], value_scale=scale[1])
    for k in range(2):
        assert np.array_equal(raw(caches[k]), want[k])


@pytest.mark.parametrize("src, dst", TYPES)
@pytest.mark.parametrize("n, heads, dim, blocks, bs", [(1, 1, 8, 1, 1), (5, 3, 24, 4, 7), (33, 2, 128, 5, 16), (300, 5, 72, 40, 24), (64, 1, 256, 3, 300)])
def test_types_and_sizes(src, dst, n, heads, dim, blocks, bs):
    for scaled in (False, True):
        for by_head in (False, True):
            check(n, heads, dim, blocks, bs, src, dst, scaled, by_head, seed=n + dim)


def test_nothing_to_write():
    check(0, 2, 64, 3, 16, torch.bfloat16, torch.bfloat16, False)
    x = torch.ones(2, 1, 64, dtype=torch.bfloat16, device="cuda")
    empty = torch.empty(0, 16, 1, 64, dtype=torch.bfloat16, device="cuda")
    tt.write_cache_into(x, x, torch.zeros(2, dtype=torch.int64, device="cuda"), empty, empty)


def test_infinities_and_nan():
    x = torch.tensor([float("inf"), float("-inf"), float("nan"), 0.0, -0.0, 448.0, 449.0, -1e30], device="cuda").reshape(1, 1, 8)
    slot = torch.zeros(1, dtype=torch.int64, device="cuda")
    for dst in (torch.float16, torch.bfloat16, F8):
        caches = [torch.ones(1, 1, 1, 8, device="cuda").to(dst) for _ in range(2)]
        tt.write_cache_into(x, -x, slot, *caches)
        for cache, y in zip(caches, (x, -x)):
            got, want = cache.float().reshape(-1), y.reshape(-1)
            if dst == F8:
                want = want.clamp(-448, 448)
            want = want.to(dst).float()
            assert torch.equal(torch.isnan(got), torch.isnan(want))
            assert torch.equal(got.nan_to_num(7.0), want.nan_to_num(7.0))
            assert torch.equal(torch.signbit(got[3:5]), torch.signbit(want[3:5]))


def test_any_alignment_and_strides():
    """Rows that start at odd elements, caches that are parts of others; what lies beside them stays."""
    for dst in (torch.bfloat16, F8):
        pool = torch.zeros(2 + 6 * 5 * 2 * 50, device="cuda").to(dst)
        both = pool[1:-1].view(6, 5, 2, 50)
        k, v = both[..., 3:19], both[..., 27:43]
        base = torch.randn(1 + 7 * 2 * 40, device="cuda").bfloat16()
        keys, values = base[1:].view(7, 2, 40)[..., 1:17], base[1:].view(7, 2, 40)[..., 19:35]
        slots = torch.tensor([0, 29, 5, 11, -1, 17, 8], device="cuda")
        before = pool.float().clone()
        tt.write_cache_into(keys, values, slots, k, v)
        want = before[1:-1].view(6, 5, 2, 50).clone()
        for i, s in enumerate(slots.tolist()):
            if s >= 0:
                want[s // 5, s % 5, :, 3:19] = keys[i].to(dst).float()
                want[s // 5, s % 5, :, 27:43] = values[i].to(dst).float()
        assert torch.equal(pool.float()[1:-1].view(6, 5, 2, 50), want)
        assert (pool.float()[[0, -1]] == 0).all()


def test_offsets_past_32_bits():
    """The last places of a cache of more than 2^32 elements."""
    cache = torch.zeros(1_050_000, 16, 1, 256, dtype=F8, device="cuda")  # 4.3e9
    x = torch.full((2, 1, 256), 3.0, dtype=torch.bfloat16, device="cuda")
    last = cache.shape[0] * 16 - 1
    tt.write_cache_into(x, x, torch.tensor([last, 17], device="cuda"), cache, cache)
    assert (cache[-1, -1].float() == 3).all() and (cache[1, 1].float() == 3).all()
    assert (cache[-1, -2].float() == 0).all() and int((cache.view(torch.uint8)[-4096:] != 0).sum()) == 256


def test_refuses():
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    cache = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16, device="cuda")
    slots = torch.zeros(3, dtype=torch.int64, device="cuda")
    bad = [dict(keys=x[:, :1]), dict(values=x[:2]), dict(values=x.half()), dict(slots=slots[:2]), dict(slots=slots.int()), dict(keys=x.half(), values=x.half()),
           dict(key_cache=cache[..., :32]), dict(value_cache=cache[:3]), dict(key_cache=cache.half()), dict(key_cache=cache.transpose(2, 3)),
           dict(keys=x.int()), dict(key_cache=cache.float(), value_cache=cache.float()), dict(key_scale=torch.ones(3, device="cuda")),
           dict(value_scale=torch.ones(2, dtype=torch.float16, device="cuda")), dict(key_scale=torch.ones(2)), dict(slots=None), dict(slots=slots.cpu())]
    for change in bad:
        with pytest.raises(ValueError):
            tt.write_cache_into(**dict(dict(keys=x, values=x, slots=slots, key_cache=cache, value_cache=cache), **change))
    with pytest.raises(ValueError):
        tt.write_cache_into(x[..., :12], x[..., :12], slots, cache[..., :12], cache[..., :12])
