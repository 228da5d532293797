"""fh_kv_attention against attention in 64 bits over the dequantized cache, with
the bound of the kernels' roundings (tests/_kv_ref.py), over head layouts,
lengths, pages, masks and strides; then the whole run of a cache's calls."""
import contextlib
import math
import os

import numpy as np
import pytest
import torch

import synthetic as S
from _gpu_util import bits_of, fh, to_dev
from _kv_ref import attention, dequantize

pytestmark = pytest.mark.gpu


@contextlib.contextmanager
def selected(kernel):
    """FH_KV_KERNEL: which kernel takes the calls."""
    old = os.environ.get("FH_KV_KERNEL")
    os.environ["FH_KV_KERNEL"] = kernel
    try:
        yield
    finally:
        os.environ.pop("FH_KV_KERNEL")
        if old is not None:
            os.environ["FH_KV_KERNEL"] = old


@pytest.fixture(params=["few", "tiles"])
def kernel(request):
    with selected(request.param):
        yield request.param


class Case:
    """A cache of random codes and scales, and requests over it."""

    def __init__(self, lens, n_q, Hq, Hk, d, page, seed=0, q_scale=1.0, gap=0, extra_pages=1):
        self.m = fh()
        rng = self.rng = np.random.default_rng(seed)
        self.lens, self.n_q = np.array(lens), np.array(n_q)
        self.Hq, self.Hk, self.d, self.page = Hq, Hk, d, page
        B = len(lens)
        need = -(-self.lens // page)
        self.pages = int(need.sum()) + 2
        self.width = int(max(need.max(), 1)) + extra_pages
        order = rng.permutation(self.pages)
        self.table = np.full((B, self.width), -1, np.int64)
        at = 0
        for b in range(B):
            self.table[b, :need[b]] = order[at:at + need[b]]
            at += need[b]
        self.starts = np.concatenate(([0], np.cumsum(self.n_q)))
        self.T = int(self.starts[-1]) + gap
        self.q = S.to_bf16_bits(rng.standard_normal((self.T, Hq, d)) * q_scale)
        shape = (self.pages, Hk, page, d)
        self.arrays = []
        for _ in range(2):
            codes = rng.integers(0, 256, (*shape[:3], d // 2), dtype=np.uint8)
            # Scales of 0 and over the whole format's range among ordinary ones.
            s = rng.integers(0x38, 0x68, (*shape[:3], d // 16), dtype=np.uint8)
            s[rng.random(s.shape) < 0.02] = 0
            wild = rng.random(s.shape) < 0.02
            s[wild] = rng.integers(0, 0x70, wild.sum())
            self.arrays += [codes, s]
        self.gs = (float(np.float32(0.011)), float(np.float32(0.017)))

    def poison_tails(self):
        """NaN scales and any codes behind every request's last token, and in pages nobody has."""
        used = np.zeros((self.pages, self.page), bool)
        for b, L in enumerate(self.lens):
            for j in range(L):
                used[self.table[b, j // self.page], j % self.page] = True
        for i in (1, 3):
            a = self.arrays[i].transpose(0, 2, 1, 3)
            a[~used] = 0x7F
        return self

    def device(self):
        self.cache = self.m.KVCache(*(torch.from_numpy(a.copy()).cuda() for a in self.arrays), *self.gs)
        t = lambda a: torch.tensor(np.asarray(a, np.int32), device="cuda")
        self.t_table, self.t_lens, self.t_starts = t(self.table), t(self.lens), t(self.starts)
        self.t_q = to_dev(self.q.reshape(self.T, -1)).view(self.T, self.Hq, self.d)
        self.ws = self.m.empty_kv_attention_workspace(self.T, len(self.lens), self.Hq, self.Hk, self.d)
        return self

    def run(self, sm_scale, q=None, out=None, **kw):
        m = self.m
        if out is None:
            out = torch.full((self.T, self.Hq, self.d), 9.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((self.T, self.Hq), 9.0, dtype=torch.float32, device="cuda")
        m.fh_kv_attention(self.t_q if q is None else q, self.cache, self.t_table, self.t_lens, self.t_starts, sm_scale,
                          out, self.ws, lse=lse, **kw)
        m.fh_device_status()
        return S.bf16_to_f32(bits_of(out.contiguous())).astype(np.float64), lse.cpu().numpy().astype(np.float64)

    def reference(self, sm_scale, causal, window, lens=None, starts=None):
        kv = [dequantize(self.arrays[2 * i], self.arrays[2 * i + 1], self.gs[i]) for i in range(2)]  # [P, H, page, d]
        lens = self.lens if lens is None else lens
        starts = self.starts if starts is None else starts

        def there(b):
            t = self.table[b, np.arange(lens[b]) // self.page]
            return (t >= 0) & (t < self.pages)

        def of(x, b):
            j = np.arange(lens[b])
            page = self.table[b, j // self.page]
            page = np.where((page >= 0) & (page < self.pages), page, 0)
            return x[page, :, j % self.page]
        q = S.bf16_to_f32(self.q).astype(np.float64)
        return attention(q, lambda b: of(kv[0], b), lambda b: of(kv[1], b), lens, starts, sm_scale, causal, window, there)

    def check(self, sm_scale=None, causal=True, window=0, lens=None, starts=None, **kw):
        """The call as it chooses its kernel, and with either of the two selected."""
        sm_scale = float(np.float32(self.d ** -0.5)) if sm_scale is None else sm_scale
        ref = self.reference(sm_scale, causal, window, lens, starts)
        for kernel in ("", "few", "tiles"):
            with selected(kernel):
                out, lse = self.run(sm_scale, causal=causal, window=window, **kw)
            compare(out, lse, *ref)
        # Every call leaves the workspace's counters zero.
        assert int(self.ws[:4096].view(torch.int32).abs().sum()) == 0


def compare(out, lse, r_out, r_lse, t_out, t_lse):
    rest = np.isnan(r_lse)
    assert (out[rest] == 9.0).all() and (lse[rest] == 9.0).all(), "rows of no request were written"
    empty = np.isneginf(r_lse)
    assert (out[empty] == 0).all() and np.isneginf(lse[empty]).all()
    some = ~rest & ~empty
    err, tol = np.abs(out[some] - r_out[some]), t_out[some]
    assert (err <= tol).all(), f"out: {np.nanmax(err / tol)} of the bound, {(~(err <= tol)).sum()} of {err.size}"
    err, tol = np.abs(lse[some] - r_lse[some]), t_lse[some]
    assert (err <= tol).all(), f"lse: {np.nanmax(err / tol)} of the bound"


SHAPES = [  # lens, queries, q_heads, kv_heads, d, page
    ([1], [1], 1, 1, 128, 16),
    ([1], [1], 1, 1, 64, 16),
    ([2, 17, 16, 31], [1, 1, 1, 1], 8, 2, 128, 16),
    ([33, 127, 128, 129, 640], [1, 1, 1, 1, 1], 32, 8, 128, 16),
    ([33, 127, 128, 129, 640], [1, 1, 1, 1, 1], 8, 1, 64, 32),
    ([300, 5, 70], [1, 1, 1], 21, 21, 128, 64),
    ([300, 5, 70], [3, 5, 4], 5, 1, 128, 16),
    ([200, 90], [5, 2], 16, 1, 64, 128),
    ([257, 700], [1, 1], 24, 1, 128, 16),
    ([150], [150], 2, 1, 128, 16),
    ([400, 130, 60], [129, 7, 60], 4, 2, 128, 32),
    ([200, 300], [65, 130], 6, 2, 64, 64),
    ([1100], [1, ], 3, 1, 128, 1024),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [0, 1, 40])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "L%s_q%s_%dx%d_d%d_p%d" % (s[0][-1], s[1][0], *s[2:]))
def test_shapes_and_masks(shape, window, causal):
    Case(*shape, seed=len(shape[0]) + shape[0][0]).poison_tails().device().check(causal=causal, window=window)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n_q", [1, 3, 40, 200])
def test_rows_that_see_nothing(d, n_q):
    """No cached tokens at all, fewer than queries, requests without queries, rows behind the last request."""
    c = Case([0, n_q // 2, 100 + n_q, 0, 64], [n_q, n_q, n_q, 0, 0], 4, 2, d, 16, seed=n_q, gap=3).poison_tails().device()
    for causal in (True, False):
        c.check(causal=causal)
        c.check(causal=causal, window=5)


@pytest.mark.parametrize("n_q", [1, 50])
def test_entries_that_name_no_page_are_left_out(n_q):
    c = Case([200, 90, 64], [n_q, n_q, 1], 4, 1, 128, 16, seed=8)
    c.table[0, 3] = -1
    c.table[0, 12] = c.pages          # the last, ragged one
    c.table[1, 0] = -2 ** 31
    c.table[2, :] = 2 ** 31 - 1       # nothing left to see
    c.poison_tails = None
    c.device()
    for causal, window in ((True, 0), (False, 0), (True, 33)):
        c.check(causal=causal, window=window)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n_q,window", [(1, 37), (1, 150), (5, 90), (300, 41)])
def test_what_lies_before_the_window_does_not_count(n_q, window, d):
    """NaN scales in every token that no query sees, and in the pages that hold only such tokens entries of other
    pages, or none."""
    c = Case([700, 333, 450], [n_q, 1, n_q], 4, 2, d, 32, seed=window, extra_pages=0).poison_tails()
    for b, L in enumerate(c.lens):
        unseen = max(0, L - c.n_q[b] - window + 1)
        for j in range(unseen):
            for i in (1, 3):
                c.arrays[i][c.table[b, j // 32], :, j % 32] = 0x7F
        c.table[b, :unseen // 32] = np.resize([-1, c.table[0, -1], c.pages + 5], unseen // 32)
    c.device()
    for causal in (True, False):
        c.check(causal=causal, window=window)


def test_starts_that_decrease_stay_inside_the_buffers(kernel):
    """Their rows are unspecified; the rows behind them, and the workspace, are as after any call."""
    c = Case([600, 300, 400], [40, 1, 40], 4, 2, 64, 16, seed=13, gap=2).device()
    c.t_starts.copy_(torch.tensor([0, 40, 10, 50]))
    out, lse = c.run(0.1)
    assert (out[50:] == 9.0).all() and (lse[50:] == 9.0).all() and np.isfinite(out).all()
    assert int(c.ws[:4096].view(torch.int32).abs().sum()) == 0


def test_lengths_and_starts_out_of_range_are_cut():
    c = Case([48, 30], [2, 2], 4, 2, 128, 16, seed=4, extra_pages=0).device()
    width = c.width * 16
    c.t_lens.copy_(torch.tensor([10 ** 9, -5]))
    c.t_starts.copy_(torch.tensor([-3, 2, 10 ** 6]))
    c.check(causal=False, lens=np.array([width, 0]), starts=np.array([0, 2, c.T]))


@pytest.mark.parametrize("Hq,Hk,n_q", [(8, 2, 1), (21, 21, 1), (16, 1, 3), (2, 2, 70)])
def test_long_lines_split_over_many_ctas(Hq, Hk, n_q):
    """Ragged lengths whose tiles span several CTAs' pieces, and short ones between them."""
    c = Case([5000, 3, 2049, 130, 0], [n_q, 1, n_q, 1, 1], Hq, Hk, 128, 32, seed=12, q_scale=2.0).poison_tails().device()
    c.check()
    c.check(causal=False)
    c.check(window=1500)


@pytest.mark.parametrize("lens,n_q,Hq,Hk,d", [([3000], [20], 8, 8, 128), ([9000, 200], [40, 3], 4, 1, 64),
                                              ([130, 1500, 0, 700], [17, 300, 2, 9], 8, 4, 128)])
def test_few_rows_over_many_keys(lens, n_q, Hq, Hk, d):
    """Too few row tiles for the GPU: their keys are cut into pieces, some of which see nothing of some rows."""
    c = Case(lens, n_q, Hq, Hk, d, 32, seed=d, q_scale=2.0).poison_tails().device()
    for causal, window in ((True, 0), (False, 0), (True, 257), (False, 64)):
        c.check(causal=causal, window=window)


@pytest.mark.parametrize("n,Hq,Hk,d", [(700, 3, 1, 64), (1100, 2, 2, 128)])
def test_many_requests(n, Hq, Hk, d):
    """More requests than a CTA has threads, some without queries or tokens, one among them of many rows."""
    i = np.arange(n)
    lens, n_q = i * 7 % 41, np.where(i % 5 == 3, 0, i % 4)
    lens[n // 2], n_q[n // 2] = 400, 130
    c = Case(lens, n_q, Hq, Hk, d, 16, seed=n, gap=1).poison_tails().device()
    c.check()
    c.check(causal=False, window=9)


@pytest.mark.parametrize("n", [63, 64, 65])
def test_requests_of_equal_and_of_mixed_lengths(n):
    """Many rows: the requests' tiles are put in order of their keys, up to 64 requests; lengths come in pairs."""
    i = np.arange(n)
    lens, n_q = 20 + 30 * (i // 2 * 7 % 11), np.where(i % 9 == 4, 0, 1 + i * 5 % 90)
    c = Case(lens, n_q, 6, 2, 64, 16, seed=n, gap=2).poison_tails().device()
    c.check()
    c.check(window=33)


@pytest.mark.parametrize("lens,n_q,Hq,Hk,d", [([70, 9], [1, 2], 72, 1, 64), ([45, 200], [3, 1], 130, 2, 128),
                                              ([5], [1], 4096, 4096, 64), ([40], [1], 1000, 1000, 128)])
def test_many_heads(lens, n_q, Hq, Hk, d):
    """Groups that are no power of two and larger than a tile's rows, and as many heads as a cache may have."""
    c = Case(lens, n_q, Hq, Hk, d, 16, seed=Hq).poison_tails().device()
    c.check()
    c.check(causal=False, window=7)


def test_both_kernels_take_turns_on_one_workspace():
    """Calls of few and of many rows, split over CTAs in either way, one after another with one workspace."""
    c = Case([4000, 300], [30, 5], 8, 4, 128, 16, seed=21).device()
    few = Case([4000, 300, 2000], [1, 1, 1], 8, 4, 128, 16, seed=22).device()
    few.ws = c.ws = c.ws if c.ws.numel() > few.ws.numel() else few.ws

    def both():
        with selected("tiles"):
            a = c.run(0.09)
        with selected("few"):
            return a, few.run(0.09)
    first = both()
    for _ in range(3):
        c.check()
        few.check()
        for old, new in zip(first, both()):
            np.testing.assert_array_equal(old[0], new[0])
            np.testing.assert_array_equal(old[1], new[1])


@pytest.mark.parametrize("max_q,max_kv", [(1, 1), (1000, 10 ** 9), (0, 0), (7, 3000)])
@pytest.mark.parametrize("n_q", [1, 90])
def test_hints_do_not_change_the_result(max_q, max_kv, n_q):
    c = Case([900, 400], [n_q, 2], 4, 2, 128, 16, seed=3).device()
    c.check(max_q=max_q, max_kv=max_kv)


@pytest.mark.parametrize("n_q", [1, 64])
def test_strided_queries_and_outputs(n_q, kernel):
    """q as the first third of fused QKV rows, out inside a wider buffer whose rest stays as it was."""
    c = Case([100, 260], [n_q, n_q], 6, 3, 64, 16, seed=5).device()
    wide = torch.full((c.T, 6 * 64 + 2 * 3 * 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, :384] = c.t_q.reshape(c.T, -1)
    buf = torch.full((c.T, 512), 9.0, dtype=torch.bfloat16, device="cuda")
    sm = float(np.float32(0.125))
    out, lse = c.run(sm, q=wide[:, :384].unflatten(1, (6, 64)), out=buf[:, 64:448].unflatten(1, (6, 64)), causal=True)
    compare(out, lse, *c.reference(sm, True, 0))
    assert (buf[:, :64] == 9.0).all() and (buf[:, 448:] == 9.0).all()


@pytest.mark.parametrize("n_q", [1, 33])
@pytest.mark.parametrize("sm_scale,q_scale", [(0.0, 1.0), (-0.3, 1.0), (1.0, 8.0), (1e-3, 1e4), (0.1, 1e-30), (1e-37, 1e36)])
def test_scales_of_scores(n_q, sm_scale, q_scale):
    """Flat, reversed and very peaked softmaxes, and query rows far outside FP16's range."""
    c = Case([333, 64], [n_q, n_q], 4, 1, 128, 16, seed=6, q_scale=q_scale).device()
    c.check(sm_scale=float(np.float32(sm_scale)))


@pytest.mark.parametrize("n_q", [1, 33])
def test_scores_that_climb_slowly(n_q):
    """Keys whose scores rise along the sequence, so that the running maximum is passed again and again by less and by
    more than it has to be raised."""
    c = Case([1024], [n_q], 2, 1, 64, 16, seed=7)
    c.q[:] = S.to_bf16_bits(np.ones((c.T, 2, 64)))
    for j in range(1024):
        page, at = c.table[0, j // 16], j % 16
        c.arrays[0][page, 0, at] = 0x22                       # code 2: every element 1.0
        c.arrays[1][page, 0, at] = min(0x20 + j // 18, 0x70)  # growing scales
    c.device()
    for sm in (0.01, 0.5, 3.0):
        c.check(sm_scale=float(np.float32(sm)))


@pytest.mark.parametrize("n_q", [1, 40])
def test_a_query_row_without_a_value_stays_alone(n_q, kernel):
    """Rows with infinities or NaN come out NaN; all others are as without them."""
    c = Case([150, 80], [n_q, n_q], 4, 2, 128, 16, seed=9).device()
    sm = float(np.float32(0.09))
    plain, _ = c.run(sm, causal=True)
    q = c.t_q.clone()
    q[0, 1, 5] = float("nan")
    q[-1, 2, 0] = float("inf")
    out, _ = c.run(sm, q=q, causal=True)
    bad = np.zeros(out.shape[:2], bool)
    bad[0, 1] = bad[-1, 2] = True
    assert np.isnan(out[bad]).all()
    np.testing.assert_array_equal(out[~bad], plain[~bad])


def test_repeats_are_bit_identical_and_streams_keep_order(kernel):
    c = Case([3000, 17, 800], [1, 1, 1], 16, 4, 128, 16, seed=10).device()
    first = c.run(0.09)
    for _ in range(5):
        again = c.run(0.09)
        np.testing.assert_array_equal(first[0], again[0])
        np.testing.assert_array_equal(first[1], again[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(c.t_q)
    c.m.fh_kv_attention(c.t_q, c.cache, c.t_table, c.t_lens, c.t_starts, 0.09, out, c.ws, stream=side)
    side.synchronize()
    np.testing.assert_array_equal(S.bf16_to_f32(bits_of(out)), first[0])


def test_pages_past_32_bit_offsets(kernel):
    """Tokens in pages whose codes lie past 4 GB."""
    m = fh()
    H, d, page, pages = 8, 128, 16, 600_000
    cache = m.empty_kv_cache(pages, page, H, d, 0.01, 0.02)
    rng = np.random.default_rng(0)
    use = np.array([0, pages - 1, pages // 2, (1 << 32) // (H * 64 * page) + 1])
    small = []
    for t, hi in ((cache.k_codes, 256), (cache.k_scales, 0x60), (cache.v_codes, 256), (cache.v_scales, 0x60)):
        a = rng.integers(0, hi, (4, *t.shape[1:]), dtype=np.uint8)
        t[torch.from_numpy(use).cuda()] = torch.from_numpy(a).cuda()
        small.append(torch.from_numpy(a).cuda())
    near = m.KVCache(*small, 0.01, 0.02)
    for n_q in (1, 60):
        q = torch.randn((n_q, 16, d), device="cuda").bfloat16()
        ws = m.empty_kv_attention_workspace(n_q, 1, 16, H, d)
        lens, starts = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([63], [0, n_q]))
        outs = []
        for c, t in ((cache, use), (near, np.arange(4))):
            out = torch.empty_like(q)
            m.fh_kv_attention(q, c, torch.tensor(t[None], dtype=torch.int32, device="cuda"), lens, starts, 0.1, out, ws)
            outs.append(out)
        assert torch.equal(*outs) and outs[0].isfinite().all()


def _serve(graph):
    """A few serving steps of ragged requests, from lengths to attention: prompts, single tokens, a request that
    finishes and one that takes its place.  Every step's attention against the same over the cache read back."""
    m = fh()
    B, Hq, Hk, d, page, cap, pages = 4, 8, 2, 128, 16, 96, 24
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    lens, target, status = i32([0] * B), i32([0] * B), i32([0])
    free, count, starts = torch.arange(pages, dtype=torch.int32, device="cuda").flip(0).contiguous(), i32([pages]), i32([0] * (B + 1))
    table, slots = torch.full((B, 12), -1, dtype=torch.int32, device="cuda"), torch.zeros(cap, dtype=torch.int64, device="cuda")
    cache = m.empty_kv_cache(pages, page, Hk, d, 0.004, 0.003)
    for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales):
        t.fill_(0x7F)
    qkv = torch.zeros((cap, (Hq + 2 * Hk) * d), dtype=torch.bfloat16, device="cuda")
    q, k, v = (x.unflatten(1, (-1, d)) for x in qkv.split([Hq * d, Hk * d, Hk * d], 1))
    out = torch.full((cap, Hq, d), 9.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((cap, Hq), 9.0, device="cuda")
    ws = m.empty_kv_attention_workspace(cap, B, Hq, Hk, d)

    def step():
        m.fh_kv_pages_update(lens, target, table, free, count, count, lens, starts, slots, status, page)
        m.fh_kv_cache_write(cache, k, v, slots)
        m.fh_kv_attention(q, cache, table, lens, starts, 0.09, out, ws, causal=True, max_q=40, lse=lse)

    captured = None
    if graph:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()  # targets are the lengths: nothing moves
        torch.cuda.current_stream().wait_stream(side)
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            step()
        out.fill_(9.0)
        lse.fill_(9.0)
    gen = torch.Generator(device="cuda").manual_seed(3)
    plan = [[37, 5, 0, 18], [38, 6, 20, 19], [39, 7, 21, 20], [40, 0, 22, 17], [41, 30, 23, 18], [41, 31, 0, 19]]
    history = [[None] * 0 for _ in range(B)]
    for want in plan:
        old = lens.tolist()
        target.copy_(i32(want))
        qkv.copy_(torch.randn(qkv.shape, device="cuda", generator=gen))
        out.fill_(9.0)
        lse.fill_(9.0)
        captured.replay() if graph else step()
        m.fh_device_status()
        assert int(status) == 0 and lens.tolist() == want
        used = table[torch.arange(12, device="cuda")[None] < ((lens + page - 1) // page)[:, None]].tolist()
        assert len(used) == len(set(used)) and int(count) == pages - len(used)
        new = [max(0, w - o) for w, o in zip(want, old)]
        assert starts.tolist() == [0, *np.cumsum(new).tolist()]
        # What the cache should hold: the old tokens' values and the new ones', by their own quantization.
        total = sum(want)
        where = torch.cat([torch.tensor([int(table[b, j // page]) * page + j % page for j in range(want[b])],
                                        dtype=torch.int64) for b in range(B)]).cuda()
        kk, vv = (torch.empty((total, Hk, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        m.fh_kv_cache_read(cache, where, kk, vv)
        once = m.empty_kv_cache(6, page, Hk, d, 0.004, 0.003)
        n = sum(new)
        kn, vn = (torch.empty((n, Hk, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        at = torch.arange(n, device="cuda")
        m.fh_kv_cache_write(once, k[:n], v[:n], at)
        m.fh_kv_cache_read(once, at, kn, vn)
        e = 0
        for b in range(B):
            history[b] = history[b][:want[b]] + [(kn[starts[b] + i], vn[starts[b] + i]) for i in range(new[b])]
            for j in range(want[b]):
                assert torch.equal(kk[e + j], history[b][j][0]) and torch.equal(vv[e + j], history[b][j][1])
            e += want[b]
        arrays = [x.cpu().numpy() for x in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales)]
        kv = [dequantize(arrays[2 * i], arrays[2 * i + 1], g) for i, g in enumerate((0.004, 0.003))]
        tb = table.cpu().numpy()

        def of(x, b):
            j = np.arange(want[b])
            return x[tb[b, j // page], :, j % page]
        q64 = S.bf16_to_f32(bits_of(q.contiguous())).astype(np.float64)
        ref = attention(q64, lambda b: of(kv[0], b), lambda b: of(kv[1], b), want, starts.tolist(), 0.09, True, 0)
        compare(S.bf16_to_f32(bits_of(out)).astype(np.float64), lse.cpu().numpy().astype(np.float64), *ref)


@pytest.mark.parametrize("graph", [False, True], ids=["eager", "graph"])
def test_serving_steps(graph, kernel):
    _serve(graph)


@pytest.mark.parametrize("L,n_q,heads", [(6000, 60, 2), (600, 600, 64)], ids=["cut", "whole"])
def test_stall_times_out_and_the_context_survives(L, n_q, heads, monkeypatch):
    """With the test hook FH_KV_TEST_STALL=1 the first CTA's products stop after two key tiles; its other warps run into
    their bounded waits, meet, and free TMEM, with its keys cut into pieces (few row tiles) and not; the host reads
    FH_ERR_TIMEOUT.  Without the hook the same call on the same workspace is right again."""
    m = fh()
    m.fh_device_status()
    c = Case([L], [n_q], heads, heads, 128, 64, seed=2).device()
    with selected("tiles"):
        want = c.run(0.09)
        monkeypatch.setenv("FH_KV_TEST_STALL", "1")
        with pytest.raises(m.FHError) as e:
            c.run(0.09)
        assert e.value.status == m.FH_ERR_TIMEOUT
        monkeypatch.delenv("FH_KV_TEST_STALL")
        m.fh_device_status()  # the word was cleared
        again = c.run(0.09)
    np.testing.assert_array_equal(want[0], again[0])
    np.testing.assert_array_equal(want[1], again[1])
    assert int(c.ws[:4096].view(torch.int32).abs().sum()) == 0


def test_two_streams_with_workspaces_of_their_own():
    """Calls that overlap on the GPU, split over CTAs in both ways, each with its own workspace."""
    cases = [Case([20000, 900], [1, 1], 8, 2, 128, 16, seed=31).device(), Case([9000], [70], 8, 8, 128, 16, seed=32).device()]
    forms = ("few", "tiles")
    want = []
    for c, form in zip(cases, forms):
        with selected(form):
            want.append(c.run(0.09))
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [[torch.empty_like(c.t_q) for _ in range(20)] for c in cases]
    torch.cuda.synchronize()
    for i in range(20):
        for c, s, o, form in zip(cases, streams, outs, forms):
            with selected(form):
                c.m.fh_kv_attention(c.t_q, c.cache, c.t_table, c.t_lens, c.t_starts, 0.09, o[i], c.ws, stream=s)
    torch.cuda.synchronize()
    cases[0].m.fh_device_status()
    for w, o in zip(want, outs):
        for x in o:
            np.testing.assert_array_equal(S.bf16_to_f32(bits_of(x)), w[0])


def test_two_graphs_share_a_workspace_in_turns():
    c = Case([20000, 900], [1, 1], 8, 2, 128, 16, seed=33).device()
    d = Case([9000], [70], 8, 2, 128, 16, seed=34).device()
    d.ws = c.ws = d.ws if d.ws.numel() > c.ws.numel() else c.ws
    want, graphs, outs = [], [], []
    for x, form in ((c, "few"), (d, "tiles")):
        with selected(form):
            want.append(x.run(0.09)[0])
        out = torch.zeros_like(x.t_q)
        g = torch.cuda.CUDAGraph()
        with selected(form), torch.cuda.graph(g):
            x.m.fh_kv_attention(x.t_q, x.cache, x.t_table, x.t_lens, x.t_starts, 0.09, out, x.ws)
        graphs.append(g)
        outs.append(out)
    for _ in range(4):
        for g, o, w in zip(graphs, outs, want):
            o.zero_()
            g.replay()
            torch.cuda.synchronize()
            np.testing.assert_array_equal(S.bf16_to_f32(bits_of(o)), w)


@pytest.mark.parametrize("graph", [False, True], ids=["eager", "graph"])
def test_a_call_waits_for_its_own_and_for_other_streams(graph, kernel):
    """Calls launched while the one before still runs: the second one's query is copied in between, the third one's
    comes from another stream late, and the cache that both read is rewritten behind the second."""
    c = Case([900, 70], [3, 1], 8, 2, 128, 16, seed=31).device()
    q2, q3 = c.t_q.flip(0).contiguous(), (c.t_q * 0.5).contiguous()
    gen = torch.Generator(device="cuda").manual_seed(3)
    k, v = (torch.randn(32, 2, 128, generator=gen, device="cuda").bfloat16() * 0.1 for _ in range(2))
    at = torch.from_numpy(c.table[0, :2].copy()).cuda()
    slots = (at[:, None] * 16 + torch.arange(16, device="cuda")).flatten()
    before = [t.clone() for t in (c.cache.k_codes, c.cache.k_scales, c.cache.v_codes, c.cache.v_scales)]

    def restore():
        for t, b in zip((c.cache.k_codes, c.cache.k_scales, c.cache.v_codes, c.cache.v_scales), before):
            t.copy_(b)

    def call(q, out):
        c.m.fh_kv_attention(q, c.cache, c.t_table, c.t_lens, c.t_starts, 0.1, out, c.ws)
    outs = [torch.zeros_like(c.t_q) for _ in range(3)]
    want = [torch.zeros_like(c.t_q) for _ in range(3)]
    torch.cuda.synchronize()
    for q, o in ((c.t_q, want[0]), (q2, want[1])):
        call(q, o)
        torch.cuda.synchronize()
    c.m.fh_kv_cache_write(c.cache, k, v, slots)
    torch.cuda.synchronize()
    call(q3, want[2])
    torch.cuda.synchronize()
    assert not torch.equal(want[2], want[0])
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    q_in, q_late = c.t_q.clone(), torch.zeros_like(c.t_q)

    def run():
        side.wait_stream(main)
        with torch.cuda.stream(side):
            torch.cuda._sleep(400000)
            q_late.copy_(q3)
        call(q_in, outs[0])
        q_in.copy_(q2)
        call(q_in, outs[1])
        c.m.fh_kv_cache_write(c.cache, k, v, slots)
        main.wait_stream(side)
        call(q_late, outs[2])
    g = torch.cuda.CUDAGraph()
    if graph:
        with torch.cuda.graph(g, stream=main):
            run()
    for _ in range(3):
        restore()
        q_in.copy_(c.t_q)
        for t in (q_late, *outs):
            t.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(main):
            g.replay() if graph else run()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)


def test_as_many_requests_as_a_call_may_have(kernel):
    """2^31 - 2 requests, all but the eighth and the last without a query: threads' shares of them end near 2^31."""
    m = fh()
    c = Case([5, 20], [1, 2], 4, 2, 128, 32, seed=2, extra_pages=0, gap=1).device()
    n = 2 ** 31 - 2
    lens, table = (torch.zeros(n, dtype=torch.int32, device="cuda") for _ in range(2))
    starts = torch.ones(n + 1, dtype=torch.int32, device="cuda")
    starts[:8], starts[n] = 0, 3
    for at, b in ((7, 0), (n - 1, 1)):
        lens[at], table[at] = int(c.lens[b]), int(c.table[b, 0])
    c.t_lens, c.t_starts, c.t_table = lens, starts, table.view(n, 1)
    c.ws = m.empty_kv_attention_workspace(c.T, n, c.Hq, c.Hk, c.d)
    sm = float(np.float32(0.09))
    compare(*c.run(sm, causal=True), *c.reference(sm, True, 0))


@pytest.mark.parametrize("n_q", [1, 33])
@pytest.mark.parametrize("sm_scale,k_gscale,q_scale", [(1e19, 1e20, 3e-40), (-1e25, 1e13, 3e-39), (1e-20, 3e-21, 1e37),
                                                       (1e-30, 1e-20, 1e36)])
def test_products_of_scales_outside_fp32(n_q, sm_scale, k_gscale, q_scale):
    """sm_scale times the keys' scale is beyond FP32, or has few bits there, while the scores are ordinary."""
    c = Case([333, 64], [n_q, n_q], 4, 1, 128, 16, seed=6, q_scale=q_scale)
    c.gs = (float(np.float32(k_gscale)), c.gs[1])
    c.device().check(sm_scale=float(np.float32(sm_scale)))


@pytest.mark.parametrize("n_q", [1, 33])
@pytest.mark.parametrize("d", [64, 128])
def test_the_least_scales_of_values(d, n_q):
    """A scale of the values of which FP32 keeps few bits once it is divided by the softmax's denominator: 4000 equal
    keys, and values of 2688 times the scale."""
    c = Case([4000, 90], [n_q, n_q], 2, 1, d, 64, seed=4)
    c.arrays[0][:] = 0x22
    c.arrays[1][:] = 0x38
    c.arrays[2][:] = 0x77
    c.arrays[3][:] = 0x7E
    c.gs = (c.gs[0], float(np.float32(1e-39)))
    c.device().check(causal=False)


def test_numbers_of_numpy():
    """Scalars as numpy has them, where the other calls take them too."""
    c = Case([90, 40], [2, 1], 4, 2, 64, 16, seed=3).device()
    sm = np.float32(0.125)
    ref = c.reference(float(sm), True, 33)
    compare(*c.run(sm, causal=np.bool_(True), window=np.int32(33), max_q=np.int64(2), max_kv=np.int64(90)), *ref)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    one, status, slots = i32([0]), i32([9]), torch.zeros(4, dtype=torch.int64, device="cuda")
    c.m.fh_kv_pages_update(one, i32([3]), i32([[-1, -1]]), i32([5]), i32([1]), i32([0]), i32([0]), i32([0, 0]), slots,
                           status, np.int64(16))
    assert int(status) == 0 and slots.tolist() == [80, 81, 82, -1]


@pytest.mark.parametrize("d,L,n_q,log2w", [(64, 60000, 33, -23.86), (128, 60000, 33, -23.86), (64, 30000, 300, -24.6),
                                           (128, 200000, 2, -23.7)])
def test_many_small_weights_beside_a_large_one(d, L, n_q, log2w):
    """A token that all queries look at, and tens of thousands whose weights are each about one unit in the last place
    of its: they count by what they are together.

    The bound: a sum of one addition a 64 keys and 64 within them, 2^-24 each; the scores, 0 and -log2w, are exact but
    for three roundings and ex2's argument and result."""
    c = Case([L], [n_q], 1, 1, d, 128, seed=5)
    c.q[:] = S.to_bf16_bits(np.ones((c.T, 1, d)))
    c.arrays[0][:] = 0x22       # ones
    c.arrays[1][:] = 0          # times 0 ...
    c.arrays[1][c.table[0, 3], 0, 7] = 0x38  # ... but for one token
    c.arrays[2][:] = 0x22
    c.arrays[3][:] = 0x38
    c.gs = (1.0, c.gs[1])
    c.device()
    sm = float(np.float32(-log2w * math.log(2) / d))
    s = sm * d
    want = s + math.log1p((L - 1) * math.exp(-s))
    tol = (L / 64 + 64) * 2.0 ** -24 + 2.0 ** -21 * (1 + want) + 4 * 2.0 ** -24 * s
    for kernel in ("few", "tiles"):
        with selected(kernel):
            _, lse = c.run(sm, causal=False)
        assert np.abs(lse - want).max() <= tol, (kernel, np.abs(lse - want).max(), tol)
