"""fh_kv_cache_write and fh_kv_cache_read: codes, scales and clip counts
bit-exact with the oracle's quantization of the same rows, values read back
exact, and nothing else touched."""
import numpy as np
import pytest
import torch

import oracle
import synthetic as S
from _gpu_util import bits_of, fh, to_dev
from _kv_ref import dequantize

pytestmark = pytest.mark.gpu


def rows(T, H, d, seed, loud=1.0):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((T, H, d)) * np.exp(rng.standard_normal((1, H, d))) * loud
    x[rng.random(x.shape) < 0.01] *= 30
    return S.to_bf16_bits(x)


def check(T, H, d, page, seed, k=None, v=None, skip=0, gscales=None, dev=None):
    m = fh()
    kb = rows(T, H, d, seed) if k is None else k
    vb = rows(T, H, d, seed + 1, 0.1) if v is None else v
    if gscales is None:  # a little small: some elements clip
        gscales = [oracle.scale_from_amax(float(np.abs(S.bf16_to_f32(x)).max()) * 0.8 or 1.0) for x in (kb, vb)]
    pages = -(-T // page) + 3
    cache = m.empty_kv_cache(pages, page, H, d, *gscales)
    for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales):
        t.fill_(0xA5)
    rng = np.random.default_rng(seed + 2)
    slots = rng.permutation(pages * page)[:T].astype(np.int64)
    if skip:
        slots[rng.permutation(T)[:skip]] = -1 - rng.integers(0, 5, skip)
        slots[int(rng.integers(0, T))] = pages * page  # beyond the cache
    clip = torch.full((1,), 5, dtype=torch.int64, device="cuda")
    kd, vd = (to_dev(x.reshape(T, -1)).view(T, H, d) for x in (kb, vb)) if dev is None else dev(kb, vb)
    sd = torch.from_numpy(slots).cuda()
    m.fh_kv_cache_write(cache, kd, vd, sd, clip)
    ko, vo = (torch.full((T, H, d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    m.fh_kv_cache_read(cache, sd, ko, vo)
    torch.cuda.synchronize()
    keep = (slots >= 0) & (slots < pages * page)
    clips = 5
    for xb, codes, scales, sg, back in ((kb, cache.k_codes, cache.k_scales, gscales[0], ko),
                                        (vb, cache.v_codes, cache.v_scales, gscales[1], vo)):
        oc, osc, ocl = oracle.quantize(np.ascontiguousarray(xb[keep]).reshape(-1, d), sg)
        clips += ocl
        gc = codes.cpu().numpy().transpose(0, 2, 1, 3).reshape(pages * page, H, d // 2)
        gs = scales.cpu().numpy().transpose(0, 2, 1, 3).reshape(pages * page, H, d // 16)
        np.testing.assert_array_equal(gc[slots[keep]].reshape(-1, d // 2), oc)
        np.testing.assert_array_equal(gs[slots[keep]].reshape(-1, d // 16), osc)
        rest = np.ones(pages * page, bool)
        rest[slots[keep]] = False
        assert (gc[rest] == 0xA5).all() and (gs[rest] == 0xA5).all(), "slots of no token were written"
        # Read back: one FP32 product of exact code * scale, then BF16.
        exact = dequantize(oc, osc, 1.0).astype(np.float32) * np.float32(sg)
        want = np.full((T, H * d), 7.0, np.float32)
        want[keep] = exact.reshape(-1, H * d)
        np.testing.assert_array_equal(bits_of(back).reshape(T, -1), S.to_bf16_bits(want))
    assert int(clip) == clips


@pytest.mark.parametrize("T,H,d,page,skip", [(1, 1, 64, 16, 0), (1, 8, 128, 16, 0), (5, 3, 128, 32, 0),
                                             (64, 8, 128, 16, 9), (77, 21, 128, 64, 3), (300, 2, 64, 128, 50),
                                             (33, 1, 128, 1024, 0), (9, 40, 64, 16, 2), (2, 130, 128, 16, 0),
                                             (1500, 4, 64, 32, 0)])
def test_write_and_read_bit_exact(T, H, d, page, skip):
    check(T, H, d, page, T + H, skip=skip)


def test_slices_of_the_fused_qkv_rows():
    """Keys and values as strided slices of [q | k | v] rows of 8064 (21 heads of 128)."""
    def dev(kb, vb):
        T = kb.shape[0]
        wide = torch.full((T, 8064), float("nan"), dtype=torch.bfloat16, device="cuda")
        wide[:, 2688:5376] = to_dev(kb.reshape(T, -1))
        wide[:, 5376:] = to_dev(vb.reshape(T, -1))
        return wide[:, 2688:5376].unflatten(1, (21, 128)), wide[:, 5376:].unflatten(1, (21, 128))
    check(301, 21, 128, 64, 9, dev=dev)


@pytest.mark.parametrize("off,ld", [(8, 528), (0, 520), (16, 544), (8, 1000)])
def test_rows_of_sixteen_byte_alignment(off, ld):
    """Rows that are 16-byte but not 32-byte aligned, and such that are, inside wider ones; read back likewise."""
    m = fh()
    T, H, d = 45, 4, 128
    kb, vb = rows(T, H, d, off), rows(T, H, d, ld)
    wide = [torch.full((T * ld + 64,), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    k, v, ko, vo = (w[off:off + T * ld].view(T, ld)[:, :H * d].unflatten(1, (H, d)) for w in wide)
    k.copy_(to_dev(kb.reshape(T, -1)).view(T, H, d))
    v.copy_(to_dev(vb.reshape(T, -1)).view(T, H, d))
    cache = m.empty_kv_cache(4, 16, H, d, 0.003, 0.005)
    slots = torch.randperm(64, device="cuda")[:T]
    slots[7] = -1
    m.fh_kv_cache_write(cache, k, v, slots)
    m.fh_kv_cache_read(cache, slots, ko, vo)
    keep = (slots >= 0).cpu().numpy()
    for xb, back, w, sg in ((kb, ko, wide[2], 0.003), (vb, vo, wide[3], 0.005)):
        oc, osc, _ = oracle.quantize(xb.reshape(-1, d), float(np.float32(sg)))
        want = dequantize(oc, osc, 1.0).astype(np.float32) * np.float32(sg)
        want = np.where(keep[:, None], S.to_bf16_bits(want).reshape(T, H * d), 0x4040)
        np.testing.assert_array_equal(bits_of(back.contiguous()).reshape(T, -1), want)
        back.fill_(3.0)
        assert (w == 3.0).all(), "something beside the rows was written"


def test_edge_values():
    """Zero blocks and negative zeros, a block that underflows the scale format, ties, clipped blocks, huge values."""
    x = np.zeros((8, 2, 64))
    x[1] = -0.0
    x[2] = 1e-6 * np.linspace(-1, 1, 64)
    x[3, 0] = np.tile([6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -6, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5], 4)
    x[4] = 3e38
    x[5, 1, 17] = -1e5
    x[6] = np.linspace(-4000, 4000, 64)
    check(8, 2, 64, 16, 3, k=S.to_bf16_bits(x), v=S.to_bf16_bits(-x), gscales=(1.0, 0.37))


@pytest.mark.parametrize("sg", [1.0, 0.0078125, 1.5, 1.25, 3.0, 0.1])
def test_borders_at_every_block_scale(sg):
    """Elements on the borders between two codes and next to them, at each of the 126 block scales: where s_g has few
    significant bits the borders are BF16 values, and ties."""
    s = np.arange(1, 127)
    s = np.where(s < 8, s * 2.0 ** -9, (8 + s % 8) * 2.0 ** (s // 8 - 10.0))
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    at = S.to_bf16_bits((s[:, None] * sg * mids).astype(np.float32)).astype(np.int64)  # [126, 7]
    near = np.concatenate([at, at - 1, at + 1], 1)
    near = np.concatenate([near, near | 0x8000, near[:, :18]], 1).reshape(126, 4, 15)
    top = np.broadcast_to(S.to_bf16_bits((6 * s * sg).astype(np.float32)).astype(np.int64)[:, None, None], (126, 4, 1))
    x = np.concatenate([top, near], 2).reshape(126, 1, 64).astype(np.uint16)
    check(126, 1, 64, 32, 9, k=x, v=x ^ 0x8000, gscales=(sg, sg))


def test_many_scales_take_turns():
    """More global scales than a table cache holds in one place, in turns: each call uses its own."""
    kb = rows(3, 1, 64, 5)
    for i in range(700):
        sg = float(np.float32(0.001 + 0.00001 * i))
        if i % 50 < 2:
            check(3, 1, 64, 16, i, k=kb, v=kb, gscales=(sg, float(np.float32(sg * 1.7))))


def test_slots_past_32_bit_offsets():
    """A cache whose codes take 4.9 GB each: tokens in its first and last pages."""
    m = fh()
    H, d, page, pages = 8, 128, 16, 600_000
    cache = m.empty_kv_cache(pages, page, H, d, 0.01, 0.02)
    n = pages * page
    slots = np.array([0, 17, n - 1, n - 16, n // 2, (1 << 32) // (H * 64) + 3, (1 << 31) // (H * 64)], np.int64)
    kb, vb = rows(len(slots), H, d, 1), rows(len(slots), H, d, 2)
    sd = torch.from_numpy(slots).cuda()
    m.fh_kv_cache_write(cache, to_dev(kb.reshape(7, -1)).view(7, H, d), to_dev(vb.reshape(7, -1)).view(7, H, d), sd)
    ko, vo = (torch.zeros((7, H, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    m.fh_kv_cache_read(cache, sd, ko, vo)
    at, off = slots // page, slots % page
    for xb, codes, back, sg in ((kb, cache.k_codes, ko, 0.01), (vb, cache.v_codes, vo, 0.02)):
        oc, osc, _ = oracle.quantize(xb.reshape(-1, d), float(np.float32(sg)))
        got = torch.stack([codes[int(a), :, int(o)] for a, o in zip(at, off)]).cpu().numpy()
        np.testing.assert_array_equal(got.reshape(-1, d // 2), oc)
        want = dequantize(oc, osc, 1.0).astype(np.float32) * np.float32(sg)
        np.testing.assert_array_equal(bits_of(back).reshape(-1, d), S.to_bf16_bits(want))


def test_empty_calls_and_other_stream():
    m = fh()
    cache = m.empty_kv_cache(2, 16, 2, 64, 1.0, 1.0)
    none = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    slots = torch.empty(0, dtype=torch.int64, device="cuda")
    m.fh_kv_cache_write(cache, none, none, slots)
    m.fh_kv_cache_read(cache, slots, none, none)
    zero = m.empty_kv_cache(0, 16, 2, 64, 1.0, 1.0)
    one = torch.ones((1, 2, 64), dtype=torch.bfloat16, device="cuda")
    m.fh_kv_cache_write(zero, one, one, torch.zeros(1, dtype=torch.int64, device="cuda"))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    slots = torch.tensor([20], device="cuda")
    torch.cuda.synchronize()
    m.fh_kv_cache_write(cache, one, one, slots, stream=side)
    back = torch.zeros_like(one)
    m.fh_kv_cache_read(cache, slots, back, back.clone(), stream=side)
    torch.cuda.synchronize()
    oc, osc, _ = oracle.quantize(np.full((1, 64), 0x3F80, np.uint16), 1.0)
    want = S.to_bf16_bits(dequantize(oc, osc, 1.0))
    np.testing.assert_array_equal(bits_of(back).reshape(2, 64), np.repeat(want, 2, 0))


def test_a_cache_keeps_what_it_was_made_of():
    """Calls read the C struct that was filled from the attributes, so none of them can be set afterwards."""
    cache = fh().empty_kv_cache(2, 16, 2, 64, 1.0, 1.0)
    for name, value in (("k_gscale", 2.0), ("v_codes", cache.v_codes.clone()), ("page_size", 32)):
        with pytest.raises(AttributeError):
            setattr(cache, name, value)
    assert cache.k_gscale == 1.0 and cache.page_size == 16
