"""Refusals of the key/value cache's entry points, through the C ABI and the
binding, without a GPU: malformed calls are rejected before any device work."""
import ctypes

import pytest
import torch

import nvfp4_quantized_linear_fh_b200 as fh

P = ctypes.c_void_p
FAKE = 1 << 20
INF = float("inf")


def cache(**kw):
    c = dict(k_codes=FAKE, k_scales=FAKE, v_codes=FAKE, v_scales=FAKE, num_pages=4, page_size=16, kv_heads=2,
             head_dim=128, k_gscale=1.0, v_gscale=1.0)
    c.update(kw)
    return fh._CKVCache(*c.values())


BAD_CACHES = [
    (1, dict(k_gscale=0.0)), (1, dict(v_gscale=float("nan"))), (1, dict(v_gscale=INF)), (1, dict(k_gscale=-1.0)),
    (1, dict(k_codes=None)), (1, dict(v_scales=None)), (2, dict(page_size=24)), (2, dict(page_size=8)),
    (2, dict(page_size=2048)), (2, dict(page_size=0)), (2, dict(page_size=-16)), (2, dict(head_dim=96)),
    (2, dict(head_dim=256)), (2, dict(kv_heads=0)), (2, dict(kv_heads=5000)), (2, dict(num_pages=-1)),
    (2, dict(num_pages=1 << 31)), (2, dict(page_size=1024, num_pages=1 << 30)), (2, dict(k_codes=FAKE + 8)),
    (2, dict(v_scales=FAKE + 4)),
]


def write(c, k=FAKE, v=FAKE, n=4, ldk=256, ldv=256, slots=FAKE, clip=None):
    return fh.lib().fh_kv_cache_write(ctypes.byref(c) if c is not None else None, k, v, n, ldk, ldv, slots, clip, None)


def read(c, k=FAKE, v=FAKE, n=4, ldk=256, ldv=256, slots=FAKE):
    return fh.lib().fh_kv_cache_read(ctypes.byref(c) if c is not None else None, slots, n, k, v, ldk, ldv, None)


def attend(c, q=FAKE, total_q=4, heads=4, ldq=512, table=FAKE, max_pages=4, lens=FAKE, starts=FAKE, batch=2, scale=1.0,
           causal=1, window=0, max_q=4, max_kv=64, out=2 * FAKE, ldo=512, lse=None, ws=FAKE, nbytes=1 << 40):
    return fh.lib().fh_kv_attention(ctypes.byref(c) if c is not None else None, q, total_q, heads, ldq, table, max_pages,
                                    lens, starts, batch, scale, causal, window, max_q, max_kv, out, ldo, lse, ws, nbytes,
                                    None)


@pytest.mark.parametrize("status,bad", BAD_CACHES, ids=lambda x: str(x))
def test_malformed_caches(status, bad):
    for call in (write, read, attend):
        assert call(cache(**bad)) == status
        assert fh.fh_last_error().startswith("fh_kv_")


def test_null_cache():
    assert write(None) == read(None) == attend(None) == 1


@pytest.mark.parametrize("call", [write, read])
def test_rows(call):
    c = cache()
    assert call(c, ldk=248) == call(c, ldv=248) == call(c, ldk=260) == call(c, n=-1) == 2
    assert call(c, k=None) == call(c, v=None) == call(c, slots=None) == 1
    assert call(c, k=FAKE + 8) == call(c, v=FAKE + 2) == call(c, slots=FAKE + 4) == 2
    assert call(c, n=0, k=None, v=None, slots=None) == 0
    assert call(cache(num_pages=0, k_codes=None, k_scales=None, v_codes=None, v_scales=None)) == 0
    assert write(c, clip=FAKE + 4) == 2


def test_attention_arguments():
    c = cache()
    assert attend(c, scale=INF) == attend(c, scale=float("nan")) == 1
    assert attend(c, heads=3) == attend(c, heads=0) == attend(c, heads=1) == attend(c, total_q=-1) == 2
    assert attend(c, batch=-1) == attend(c, total_q=1 << 30) == 2
    assert attend(c, ldq=504) == attend(c, ldo=508) == attend(c, ldo=500) == 2
    assert attend(c, max_pages=0) == attend(c, max_pages=(1 << 26) + 1) == attend(c, window=-1) == 2
    assert attend(c, window=1 << 31) == attend(c, max_q=-1) == attend(c, max_kv=-1) == 2
    for name in ("q", "table", "lens", "starts", "out", "ws"):
        assert attend(c, **{name: None}) == 1, name
    assert attend(c, q=FAKE + 8) == attend(c, out=FAKE + 8) == attend(c, ws=FAKE + 8) == attend(c, lse=FAKE + 2) == 2
    assert attend(c, table=FAKE + 2) == attend(c, lens=FAKE + 1) == attend(c, starts=FAKE + 3) == 2
    need = fh.fh_kv_attention_workspace_bytes(4, 2, 4, 2, 128)
    assert need > 0 and attend(c, nbytes=need - 1) == 1
    assert attend(c, out=FAKE) == 1  # q itself
    assert attend(cache(num_pages=0)) == 2
    assert attend(c, total_q=0, q=None, out=None) == attend(c, batch=0, lens=None) == 0
    assert fh.fh_kv_attention_workspace_bytes(4, 2, 3, 2, 128) == 0
    assert fh.fh_kv_attention_workspace_bytes(4, 2, 4, 2, 80) == 0
    with pytest.raises(ValueError):
        fh.empty_kv_attention_workspace(4, 2, 3, 2, 128)


def test_pages_arguments():
    def call(held=FAKE, target=FAKE, batch=2, page=16, table=FAKE, max_pages=4, free=FAKE, cap=8, count=FAKE,
             count_out=FAKE, lens=FAKE, starts=FAKE, slots=FAKE, slot_cap=8, status=FAKE):
        return fh.lib().fh_kv_pages_update(held, target, batch, page, table, max_pages, free, cap, count, count_out, lens,
                                           starts, slots, slot_cap, status, None)
    assert call(batch=-1) == call(batch=8193) == call(page=0) == call(page=24) == call(page=1 << 21) == 2
    assert call(max_pages=0) == call(max_pages=1 << 27) == call(cap=0) == call(cap=1 << 31) == 2
    assert call(slot_cap=-1) == call(slot_cap=1 << 31) == 2
    for name in ("held", "target", "table", "free", "count", "count_out", "lens", "starts", "slots", "status"):
        assert call(**{name: None}) == 1, name
        assert call(**{name: FAKE + 2}) == 2, name
    assert call(batch=0, held=None) == 0


def test_binding_refuses_what_is_no_cuda_tensor():
    u8 = torch.zeros((2, 2, 16, 64), dtype=torch.uint8)
    with pytest.raises(TypeError):
        fh.KVCache(u8, u8[..., :8], u8, u8[..., :8], 1.0, 1.0)
    with pytest.raises(TypeError):
        fh.fh_kv_pages_update(*[torch.zeros(1, dtype=torch.int32)] * 10, 16)
    with pytest.raises(TypeError):
        fh.fh_kv_pages_update(*[None] * 10, 16)
