"""An attention layer of the library's own calls, launched one behind the other: quantize, QKV projection, page
bookkeeping, cache write, attention, quantize, output projection, read-back over the projection's rows.  Kernels that
come up while the one before ends must find all that it and those before it wrote."""
import pytest
import torch

from _gpu_util import fh

pytestmark = pytest.mark.gpu


class Layer:
    def __init__(self, d, hq, hk, batch, seed):
        self.m, self.d, self.hq, self.hk, self.batch = fh(), d, hq, hk, batch
        m, g = self.m, torch.Generator(device="cuda").manual_seed(seed)
        self.page, self.width, self.cap = 16, 24, 640
        i32 = lambda *shape: torch.zeros(shape, dtype=torch.int32, device="cuda")
        self.x = torch.zeros((self.cap, 256), dtype=torch.bfloat16, device="cuda")
        n = (hq + 2 * hk) * d
        self.w = self.quantized((torch.randn((n, 256), device="cuda", generator=g) * 0.06).bfloat16(), 4e-4)
        self.wo = self.quantized((torch.randn((256, hq * d), device="cuda", generator=g) * 0.05).bfloat16(), 4e-4)
        self.xq, self.oq = m.empty_quantized(self.cap, 256), m.empty_quantized(self.cap, hq * d)
        self.qkv = torch.zeros((self.cap, n), dtype=torch.bfloat16, device="cuda")
        self.q, self.k, self.v = (t.unflatten(1, (-1, d)) for t in self.qkv.split([hq * d, hk * d, hk * d], 1))
        self.out = torch.zeros((self.cap, hq, d), dtype=torch.bfloat16, device="cuda")
        self.lse = torch.zeros((self.cap, hq), device="cuda")
        self.y = torch.zeros((self.cap, 256), dtype=torch.bfloat16, device="cuda")
        self.pages = batch * self.width
        self.lens, self.target, self.count, self.status = i32(batch), i32(batch), i32(1), i32(1)
        self.table, self.free = i32(batch, self.width), i32(self.pages)
        self.starts, self.slots = i32(batch + 1), torch.zeros(self.cap, dtype=torch.int64, device="cuda")
        self.cache = m.empty_kv_cache(self.pages, self.page, hk, d, 0.001, 0.001)
        self.ws = m.empty_kv_attention_workspace(self.cap, batch, hq, hk, d)
        self.reset()

    def quantized(self, w, sg):
        codes, scales = self.m.empty_quantized(*w.shape)
        self.m.fh_quantize_act(w, sg, codes, scales)
        return codes, scales, sg

    def reset(self):
        self.free.copy_(torch.arange(self.pages, dtype=torch.int32, device="cuda").flip(0))
        self.count.fill_(self.pages)
        for t in (self.lens, self.target, self.table):
            t.zero_()
        for t in (self.cache.k_codes, self.cache.k_scales, self.cache.v_codes, self.cache.v_scales):
            t.zero_()

    def step(self, wait=lambda: None):
        m = self.m
        m.fh_quantize_act(self.x, 2e-3, *self.xq)
        wait()
        m.fh_nvfp4_linear(*self.xq, 2e-3, *self.w, None, self.qkv)
        wait()
        m.fh_kv_pages_update(self.lens, self.target, self.table, self.free, self.count, self.count, self.lens, self.starts,
                             self.slots, self.status, self.page)
        wait()
        m.fh_kv_cache_write(self.cache, self.k, self.v, self.slots)
        wait()
        m.fh_kv_attention(self.q, self.cache, self.table, self.lens, self.starts, self.d ** -0.5, self.out, self.ws,
                          lse=self.lse)
        wait()
        m.fh_quantize_act(self.out.flatten(1), 1e-3, *self.oq)
        wait()
        m.fh_nvfp4_linear(*self.oq, 1e-3, *self.wo, None, self.y)
        wait()
        m.fh_kv_cache_read(self.cache, self.slots, self.k, self.v)
        wait()


@pytest.mark.parametrize("kernel", ["few", "tiles"])
@pytest.mark.parametrize("d,hq,hk", [(64, 8, 2), (128, 4, 4)])
def test_steps_without_and_with_waits_between(d, hq, hk, kernel, monkeypatch):
    monkeypatch.setenv("FH_KV_KERNEL", kernel)
    batch, steps = 6, 12
    layer = Layer(d, hq, hk, batch, 1)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.step()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        layer.step()

    def run(step):
        layer.reset()
        for t in (layer.out, layer.lse, layer.y, layer.qkv):
            t.zero_()
        torch.cuda.synchronize()
        gen, results = torch.Generator(device="cuda").manual_seed(7), []
        for i in range(steps):
            grow = torch.tensor([(i * 7 + b * 11) % 40 if (i + b) % 3 else 1 for b in range(batch)], device="cuda")
            layer.target.copy_(torch.where((layer.lens > 300) | (grow == 13), 0, layer.lens + grow))
            layer.x.copy_(torch.randn(layer.x.shape, device="cuda", generator=gen))
            step()
            results.append([t.clone() for t in (layer.qkv, layer.table, layer.free, layer.count, layer.lens, layer.starts,
                                                layer.slots, layer.status, layer.cache.k_codes, layer.cache.v_scales,
                                                layer.out, layer.lse, *layer.oq, layer.y)])
        layer.m.fh_device_status()
        return results
    want = run(lambda: layer.step(torch.cuda.synchronize))
    assert all(int(r[7]) == 0 for r in want) and all(int(r[4].max()) > 0 for r in want)
    assert any(bool(r[10].abs().sum() > 0) for r in want) and bool(want[-1][-1].isfinite().all())
    for form in (layer.step, graph.replay) * 3:
        for i, (a, b) in enumerate(zip(run(form), want)):
            for j, (s, t) in enumerate(zip(a, b)):
                assert torch.equal(s, t), (form, i, j)
