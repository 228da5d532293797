"""Measured cases of the NVFP4 key/value cache: its page bookkeeping, its write and read-back, and the attention
that reads it.

An attention layer's keys and values are kept in pages of tokens, in the library's own format: E2M1 codes, one E4M3
scale per 16 elements of a head, and one FP32 scale per tensor.  The operators are

- ``pages``: requests grow, shrink or finish; pages move between their block tables and the free stack, and the new
  tokens get their places ("slots"), all from request lengths on the device;
- ``cache``: new keys and values are quantized into their slots, and read back as the BF16 values that they stand for;
- ``attention``: queries of ragged requests attend to their cached tokens, for single tokens, drafts, prompts and
  whole clips (heads shared or not, causal or not, with a window or without).

Head counts, the head size and the token counts of the fused-QKV and clip cases are those of the repository's
configurations and its attention benchmark (21 heads of 128, rows of 8064, 32768 rows, 4096 x 4096 tokens); the others
are ordinary sizes of serving.  Lengths are a fixed function of the case, so that the work is known; values, page
order and the order of the free stack come from the seed.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"


def listed():
    return [
        # A serving step: every running request gets one token, a few have finished, a few drop rejected draft tokens.
        dict(name="pages_decode", op="pages", batch=48, page=16, held=8192, new=1),
        # A wave of prompts arrives together with running requests: long slot maps.
        dict(name="pages_prompts", op="pages", batch=1500, page=32, held=4096, new=400),
        # One token of each of 64 requests into the cache of a layer with 8 heads (graph-padded rows among them).
        dict(name="cache_decode", op="cache", tokens=64, heads=8, dim=128, page=16, fused=False, pad=9),
        # A mid-sized chunk of prompt tokens, small heads, an odd count.
        dict(name="cache_chunk", op="cache", tokens=1531, heads=4, dim=64, page=32, fused=False, pad=0),
        # Keys and values as they stand in the rows of the fused QKV projection's output: 32768 x 8064, 21 heads of 128.
        dict(name="cache_qkv", op="cache", tokens=32768, heads=21, dim=128, page=64, fused=True, pad=0),
        # One request, one token: latency counts.
        dict(name="decode_one", op="attention", batch=1, q=1, kv=700, heads=32, kv_heads=8, dim=128, page=16, causal=True,
             window=0, lse=False),
        # A running batch of ragged requests, heads shared by four.
        dict(name="decode_batch", op="attention", batch=64, q=1, kv=8192, heads=32, kv_heads=8, dim=128, page=16,
             causal=True, window=0, lse=False),
        # Few requests with a long history: the long axis has to be split.
        dict(name="decode_long", op="attention", batch=6, q=1, kv=131072, heads=32, kv_heads=4, dim=128, page=64,
             causal=True, window=0, lse=False),
        # Drafts of five tokens to check at once, unshared heads as in the 21-head configuration.
        dict(name="draft_check", op="attention", batch=20, q=5, kv=3000, heads=21, kv_heads=21, dim=128, page=32,
             causal=True, window=0, lse=True),
        # A clip's 4096 latent tokens over 4096 cached tokens, 21 heads of 128: the attention benchmark's size.
        dict(name="clip_4096", op="attention", batch=1, q=4096, kv=4096, heads=21, kv_heads=21, dim=128, page=128,
             causal=False, window=0, lse=False),
        # Prompts of several requests, each behind what is cached of it already.
        dict(name="prompts_causal", op="attention", batch=4, q=1900, kv=5000, heads=32, kv_heads=8, dim=128, page=16,
             causal=True, window=0, lse=False),
        # Chunks of long prompts in a layer with a sliding window and small heads.
        dict(name="chunks_window", op="attention", batch=3, q=600, kv=16000, heads=16, kv_heads=2, dim=64, page=64,
             causal=True, window=4096, lse=True),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    page = rng.choice((16, 32, 64, 128))
    kind = rng.choice(("pages", "cache", "attention", "attention", "attention"))
    if kind == "pages":
        batch, new = spread(1, 2048), spread(1, 600)
        return dict(op="pages", batch=batch, page=page, held=spread(16, 8192), new=max(1, min(new, 600000 // batch)))
    if kind == "cache":
        heads, dim = rng.choice((1, 2, 4, 8, 16, 21)), rng.choice((64, 128))
        tokens = spread(1, min(32768, 88_000_000 // (heads * dim)))
        return dict(op="cache", tokens=tokens, heads=heads, dim=dim, page=page, fused=rng.random() < 0.5,
                    pad=rng.choice((0, 0, min(7, tokens - 1))))
    kv_heads = rng.choice((1, 2, 4, 8, 21))
    heads = kv_heads * rng.choice((1, 2, 4, 5, 8)) if kv_heads < 21 else 21
    dim = rng.choice((64, 128))
    window = rng.choice((0, 0, 0, spread(16, 8192)))
    causal = rng.random() < 0.75
    lse = rng.random() < 0.5
    if rng.random() < 0.6:  # single tokens and drafts
        q, kv = rng.choice((1, 1, 1, 2, 3, 5)), spread(1, 131072)
        room = 6 * 131072 * 4 * 128 // (kv * kv_heads * dim)
        batch = max(1, min(spread(1, 200), room))
        return dict(op="attention", batch=batch, q=q, kv=max(kv, q), heads=heads, kv_heads=kv_heads, dim=dim, page=page,
                    causal=causal, window=window, lse=lse)
    q = spread(6, 4096)
    kv = max(q, spread(64, 16384))
    batch = max(1, min(rng.randint(1, 6), 350_000_000 // (q * heads * kv)))
    while q * heads * kv > 350_000_000:
        q, kv = max(6, int(q * 0.8)), max(64, int(kv * 0.8))
    return dict(op="attention", batch=batch, q=q, kv=max(kv, q), heads=heads, kv_heads=kv_heads, dim=dim, page=page,
                causal=causal, window=window, lse=lse)


# --- lengths, a fixed function of the case ----------------------------------------------------------------------

def _ragged(n, lo, hi, phase=0.0):
    """n lengths spread over [lo, hi], in no order; the first is hi."""
    f = np.mod(phase + np.arange(n) * 0.6180339887498949, 1.0)
    f[0] = 1.0
    return (lo + np.floor(f * (hi - lo + 0.999))).astype(np.int64).clip(lo, hi)


def _page_lengths(case):
    """(held, target) token counts: most requests grow, some finish, some shrink, some have just come."""
    n = case["batch"]
    held = _ragged(n, 1, case["held"], 0.3)
    target = held + _ragged(n, 1, case["new"], 0.7)
    i = np.arange(n)
    target[i % 23 == 5] = 0
    target = np.where(i % 29 == 7, np.maximum(held - 3, 0), target)
    held = np.where(i % 31 == 11, 0, held)
    target = np.where(held == 0, np.maximum(target, 1), target)
    return held, target


def _attention_lengths(case):
    """(queries, cached tokens) of each request; a request has at least as many cached tokens as queries."""
    n = case["batch"]
    nq = np.full(n, case["q"]) if case["q"] <= 8 else _ragged(n, max(1, case["q"] // 3), case["q"], 0.1)
    kv = np.maximum(_ragged(n, max(1, case["kv"] // 8), case["kv"], 0.45), nq)
    return nq, kv


# --- inputs -----------------------------------------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    state = {"case": case, **{"pages": _prepare_pages, "cache": _prepare_cache, "attention": _prepare_attention}[case["op"]](case, g)}
    if own:
        import nvfp4_quantized_linear_fh_b200 as fh
        state["fh"] = fh
        if case["op"] != "pages":
            state["cache"] = fh.KVCache(*state["store"], *state["gscales"])
        if case["op"] == "attention":
            state["workspace"] = fh.empty_kv_attention_workspace(state["q"].shape[0], case["batch"], case["heads"],
                                                                 case["kv_heads"], case["dim"])
    return state


def _int32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)


def _prepare_pages(case, g):
    held, target = _page_lengths(case)
    page = case["page"]
    hp, tp = -(-held // page), -(-target // page)
    width = int(max(hp.max(), tp.max())) + 3
    total = int(hp.sum() + np.maximum(tp - hp, 0).sum()) + 17
    order = torch.randperm(total, device=DEV, generator=g).to(torch.int32)
    table = torch.full((case["batch"], width), -1, dtype=torch.int32, device=DEV)
    used = int(hp.sum())
    mask = torch.arange(width, device=DEV)[None] < torch.tensor(hp, device=DEV)[:, None]
    table[mask] = order[:used]
    free = torch.full((total,), -1, dtype=torch.int32, device=DEV)
    free[:total - used] = order[used:]
    rows = int(np.maximum(target - held, 0).sum())
    capacity = -(-(rows + 1) // 64) * 64  # as a captured step pads its rows
    state = dict(held=_int32(held), target=_int32(target), table=table, free=free, free_count=_int32([total - used]))
    state |= dict(free_count_out=_int32([0]), lens=_int32(np.zeros(len(held))), q_starts=_int32(np.zeros(len(held) + 1)),
                  slots=torch.zeros(capacity, dtype=torch.int64, device=DEV), status=_int32([0]))
    return state


def _scale_for(amax):
    """The smallest FP32 scale s with 2688 s >= amax."""
    s = np.float32(amax / 2688.0)
    while float(s) * 2688.0 < amax:
        s = np.nextafter(s, np.float32(np.inf))
    return float(s)


def _prepare_cache(case, g):
    t, h, d, page = case["tokens"], case["heads"], case["dim"], case["page"]
    if case["fused"]:  # rows of [q | k | v]
        rows = torch.empty((t, 3 * h * d), dtype=torch.bfloat16, device=DEV)
        q, k, v = (rows[:, i * h * d:(i + 1) * h * d].unflatten(1, (h, d)) for i in range(3))
        q.zero_()
    else:
        k, v = (torch.empty((t, h, d), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    spread = torch.exp(0.5 * torch.randn((1, h, d), device=DEV, generator=g))  # keys have loud channels
    k.copy_(torch.randn((t, h, d), device=DEV, generator=g) * spread)
    v.copy_(torch.randn((t, h, d), device=DEV, generator=g))
    n_pages = -(-t // page) + 5
    slots = torch.randperm(n_pages, device=DEV, generator=g)[:, None] * page + torch.arange(page, device=DEV)
    slots = slots.reshape(-1)[:t].clone()
    if case["pad"]:
        slots[-case["pad"]:] = -1
    # Scales calibrated a little under the largest value of this batch: a few elements clip, as outliers do.
    big = torch.stack((k.abs().max(), v.abs().max())).tolist()
    state = dict(k=k, v=v, slots=slots, gscales=(_scale_for(0.9 * big[0]), _scale_for(0.95 * big[1])))
    state["store"] = [torch.zeros((n_pages, h, page, d // m), dtype=torch.uint8, device=DEV) for m in (2, 16, 2, 16)]
    state["clips"] = torch.zeros(1, dtype=torch.int64, device=DEV)
    state["k_out"], state["v_out"] = (torch.zeros((t, h, d), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    return state


#: How often each magnitude code comes up among 256 elements of blocks that are scaled to their largest element.
_SHARES = (30, 52, 47, 37, 41, 26, 14, 9)


def _random_store(pages, heads, page, dim, loud, g):
    """Codes and scales as quantized keys or values have them."""
    lut = torch.repeat_interleave(torch.arange(8, dtype=torch.uint8, device=DEV), torch.tensor(_SHARES, device=DEV))
    codes = torch.empty((pages, heads, page, dim // 2), dtype=torch.uint8, device=DEV)
    scales = torch.empty((pages, heads, page, dim // 16), dtype=torch.uint8, device=DEV)
    step = max(1, 64_000_000 // (heads * page * dim // 2))
    for p in range(0, pages, step):  # in parts: the indexes are 64-bit
        c = codes[p:p + step]
        r = torch.randint(0, 1 << 20, c.shape, dtype=torch.int32, device=DEV, generator=g)
        c.copy_((lut[r & 255] | ((r >> 8) & 8)) | ((lut[(r >> 12) & 255] << 4) | ((r >> 4) & 128)))
        s = scales[p:p + step]
        size = loud * (1 + 0.22 * torch.randn(s.shape, device=DEV, generator=g)).clamp(0.3, 2.4)
        s.copy_(size.clamp(max=448.0).to(torch.float8_e4m3fn).view(torch.uint8))
    return codes, scales


def _prepare_attention(case, g):
    nq, kv = _attention_lengths(case)
    page, hk, d = case["page"], case["kv_heads"], case["dim"]
    need = -(-kv // page)
    total, width = int(need.sum()) + 3, int(need.max()) + 1
    order = torch.randperm(total, device=DEV, generator=g).to(torch.int32)
    table = torch.full((case["batch"], width), -1, dtype=torch.int32, device=DEV)
    mask = torch.arange(width, device=DEV)[None] < torch.tensor(need, device=DEV)[:, None]
    table[mask] = order[:int(need.sum())]
    loud = 150 * torch.exp(0.3 * torch.randn((1, hk, 1, d // 16), device=DEV, generator=g)).clamp(0.5, 1.6)
    kc, ks = _random_store(total, hk, page, d, loud, g)
    vc, vs = _random_store(total, hk, page, d, 150.0, g)
    q = (2.0 * torch.randn((int(nq.sum()), case["heads"], d), device=DEV, generator=g)).to(torch.bfloat16)
    starts = np.concatenate(([0], np.cumsum(nq)))
    row_b = np.repeat(np.arange(case["batch"]), nq)
    state = dict(q=q, store=[kc, ks, vc, vs], gscales=(float(np.float32(0.0019)), float(np.float32(0.0018))), table=table, lens=_int32(kv), q_starts=_int32(starts),
                 sm_scale=float(np.float32(d ** -0.5)), out=torch.zeros_like(q))
    state["lse"] = torch.zeros(q.shape[:2], dtype=torch.float32, device=DEV) if case["lse"] else None
    # What a host that plans the step knows: the places of the rows in a padded batch, and the longest of each.
    state |= dict(row_b=torch.tensor(row_b, device=DEV), row_i=torch.tensor(np.arange(len(row_b)) - starts[row_b], device=DEV),
                  max_q=int(nq.max()), max_kv=int(kv.max()))
    return state


# --- one pass ---------------------------------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return {"pages": _own_pages, "cache": _own_cache, "attention": _own_attention}[op](state)
    return {"pages": _plain_pages, "cache": _plain_cache, "attention": _plain_attention}[op](state)


def _own_pages(s):
    s["fh"].fh_kv_pages_update(s["held"], s["target"], s["table"], s["free"], s["free_count"], s["free_count_out"],
                               s["lens"], s["q_starts"], s["slots"], s["status"], s["case"]["page"])
    return {k: s[k] for k in ("table", "free", "free_count_out", "lens", "q_starts", "slots", "status")}


def _own_cache(s):
    s["clips"].zero_()
    s["fh"].fh_kv_cache_write(s["cache"], s["k"], s["v"], s["slots"], s["clips"])
    s["fh"].fh_kv_cache_read(s["cache"], s["slots"], s["k_out"], s["v_out"])
    return {"k": s["k_out"], "v": s["v_out"], "clips": s["clips"]}


def _own_attention(s):
    c = s["case"]
    s["fh"].fh_kv_attention(s["q"], s["cache"], s["table"], s["lens"], s["q_starts"], s["sm_scale"], s["out"], s["workspace"],
                            causal=c["causal"], window=c["window"], max_q=s["max_q"], max_kv=s["max_kv"], lse=s["lse"])
    return {"out": s["out"]} | ({"lse": s["lse"]} if c["lse"] else {})


def _plain_pages(s):
    page, table, free, count = s["case"]["page"], s["table"].long(), s["free"].long(), s["free_count"].long()
    held, target = s["held"].long(), s["target"].long()
    n, width = table.shape
    hp, tp = (held + page - 1) // page, (target + page - 1) // page
    grow, drop, new = (tp - hp).clamp(min=0), (hp - tp).clamp(min=0), (target - held).clamp(min=0)
    grown, dropped, starts = grow.cumsum(0), drop.cumsum(0), torch.nn.functional.pad(new.cumsum(0), (1, 0))
    i = torch.arange(free.numel(), device=table.device)
    # The pages given back, in the order of the requests and of their tables; they go onto the stack first.
    b = torch.searchsorted(dropped, i, right=True).clamp(max=n - 1)
    back = table[b, (tp[b] + i - (dropped - drop)[b]).clamp(0, width - 1)]
    pushed = (i >= count) & (i < count + dropped[-1])
    stack = torch.where(pushed, back[(i - count).clamp(min=0)], free)
    # Growing requests take pages from its top, in the order of the requests and of their tables.
    j = torch.arange(width, device=table.device)[None]
    taken = (grown - grow)[:, None] + j - hp[:, None]
    top = count + dropped[-1] - 1 - taken
    table = torch.where((j >= hp[:, None]) & (j < tp[:, None]), stack[top.clamp(0, free.numel() - 1)], table)
    r = torch.arange(s["slots"].numel(), device=table.device)
    b = torch.searchsorted(starts[1:], r, right=True).clamp(max=n - 1)
    token = held[b] + r - starts[b]
    slots = torch.where(r < starts[-1], table[b, (token // page).clamp(0, width - 1)] * page + token % page, -1)
    left = count + dropped[-1] - grown[-1]
    status = torch.zeros_like(s["status"])  # every input here can be served
    return {"table": table.int(), "free": stack.int(), "free_count_out": left.int(), "lens": target.int(),
            "q_starts": starts.int(), "slots": slots, "status": status}


def _quantized(x, gscale):
    """The values, in 32 bits, that NVFP4 keeps of x with this scale; and how many elements are out of its range.  The
    quotients are formed in 64 bits, where no value that is not on a border comes to lie on one."""
    x = x.double().unflatten(-1, (-1, 16))
    s = x.abs().amax(-1, keepdim=True) / (6.0 * gscale)
    unit = torch.exp2(torch.floor(torch.log2(s.clamp(min=2.0 ** -6))) - 3)
    s = (torch.round(s / unit) * unit).clamp(max=448.0)
    a = torch.where(s > 0, (x / (s * gscale)).abs(), 0.0)
    unit = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    a = (torch.round(a / unit) * unit).clamp(max=6.0)
    kept = (torch.copysign(a, x) * s).float() * torch.tensor(gscale, dtype=torch.float32, device=x.device)
    return kept.flatten(-2), (x.abs() > 2688.0 * gscale).flatten(-2)


def _plain_cache(s):
    kept = (s["slots"] >= 0)[:, None, None]
    (k, ck), (v, cv) = _quantized(s["k"], s["gscales"][0]), _quantized(s["v"], s["gscales"][1])
    clips = (ck & kept).sum() + (cv & kept).sum()
    return {"k": torch.where(kept, k, 0).bfloat16(), "v": torch.where(kept, v, 0).bfloat16(), "clips": clips.reshape(1)}


def _values(codes, scales, gscale):
    """FP32 values [batch, heads, tokens, dim] of gathered pages [batch, pages, heads, page, dim / 2]."""
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
    grid = torch.cat((grid, -grid))
    pairs = torch.stack((grid.repeat(16), grid.repeat_interleave(16)), -1)  # of a byte: the low nibble first
    x = pairs[codes.int()].flatten(-2).unflatten(-1, (-1, 16))
    x = (x * scales.view(torch.float8_e4m3fn).float()[..., None]).flatten(-2) * gscale
    return x.transpose(1, 2).flatten(2, 3)


def _plain_attention(s):
    c, kc, ks, vc, vs = s["case"], *s["store"]
    hk, group = c["kv_heads"], c["heads"] // c["kv_heads"]
    table = s["table"].long().clamp(min=0)[:, :-1]
    k, v = _values(kc[table], ks[table], s["gscales"][0]), _values(vc[table], vs[table], s["gscales"][1])
    n, rows = c["batch"], s["max_q"]
    lens, starts = s["lens"].long(), s["q_starts"].long()
    q = torch.zeros((n, rows, *s["q"].shape[1:]), device=k.device)
    q[s["row_b"], s["row_i"]] = s["q"].float()
    q = q.view(n, rows, hk, group, -1).permute(0, 2, 3, 1, 4).flatten(2, 3)  # [n, hk, group * rows, d]
    scores = (q @ k.transpose(-1, -2) * s["sm_scale"]).unflatten(2, (group, rows))
    at = torch.arange(k.shape[2], device=k.device)
    place = (lens - (starts[1:] - starts[:-1]))[:, None] + torch.arange(rows, device=k.device)  # of each query
    seen = (at < lens[:, None, None]).expand(n, rows, at.numel())
    if c["causal"]:
        seen = seen & (at <= place[..., None])
    if c["window"]:
        seen = seen & (at > place[..., None] - c["window"])
    scores = scores.masked_fill(~seen[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    weights = torch.exp(scores.sub_(torch.where(top == -math.inf, 0, top)))
    total = weights.sum(-1, keepdim=True)
    out = (weights.flatten(2, 3) @ v).unflatten(2, (group, rows)) / torch.where(total == 0, 1, total)
    out = out.permute(0, 3, 1, 2, 4).flatten(2, 3)[s["row_b"], s["row_i"]].bfloat16()
    if not c["lse"]:
        return {"out": out}
    lse = (top + torch.log(total)).squeeze(-1).permute(0, 3, 1, 2).flatten(2, 3)[s["row_b"], s["row_i"]]
    return {"out": out, "lse": lse}


# --- what a pass cannot do without ------------------------------------------------------------------------------

def work(case):
    if case["op"] == "pages":
        held, target = _page_lengths(case)
        page = case["page"]
        moved = np.abs(-(-held // page) - -(-target // page)).sum()
        rows = np.maximum(target - held, 0).sum()
        return {"bytes": float(16 * case["batch"] + 8 * moved + 8 * rows), "flops": 0.0}
    if case["op"] == "cache":
        values = 2 * (case["tokens"] - case["pad"]) * case["heads"] * case["dim"]
        return {"bytes": values * (2 + 0.5625 + 2) + 8.0 * case["tokens"], "flops": 0.0}
    nq, kv = _attention_lengths(case)
    pairs = bytes_ = 0.0
    for n, length in zip(nq.tolist(), kv.tolist()):
        place = length - n + np.arange(n)
        hi = np.minimum(place + 1, length) if case["causal"] else np.full(n, length)
        lo = np.maximum(place - case["window"] + 1, 0) if case["window"] else np.zeros(n)
        pairs += float(np.maximum(hi - lo, 0).sum())
        bytes_ += float(hi.max() - lo.min()) * case["kv_heads"] * case["dim"] * 2 * 0.5625
        bytes_ += n * case["heads"] * (case["dim"] * 4 + (4 if case["lse"] else 0))
    return {"bytes": bytes_, "flops": 4.0 * pairs * case["heads"] * case["dim"]}


# --- the definitions in 64 bits ---------------------------------------------------------------------------------

def exact(case, seed):
    if case["op"] == "pages":
        return None  # whole numbers only
    s = prepare(case, seed)
    return _exact_cache(s) if case["op"] == "cache" else _exact_attention(s)


def _nearest(a, grid):
    """The element of the sorted grid nearest to each a >= 0; of two equally near, the one with the even index."""
    hi = torch.searchsorted(grid, a).clamp(1, grid.numel() - 1)
    lo = hi - 1
    below, above = a - grid[lo], grid[hi] - a
    return grid[torch.where((above < below) | ((above == below) & (hi % 2 == 0)), hi, lo)]


def _exact_cache(s):
    e2m1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=DEV)
    byte = torch.arange(127, device=DEV)
    e4m3 = torch.where(byte < 8, byte * 2.0 ** -9, (8 + byte % 8) * torch.exp2((byte // 8 - 10).double()))
    result, clips = {}, 0
    for name, sg in zip(("k", "v"), s["gscales"]):
        y = torch.zeros(s[name].shape, dtype=torch.float64, device=DEV)
        step = max(1, 30_000_000 // y[0].numel())
        for t in range(0, y.shape[0], step):
            x = s[name][t:t + step].double()
            blocks = x.reshape(*x.shape[:2], -1, 16)
            scale = _nearest(blocks.abs().max(-1).values / (6 * sg), e4m3)[..., None]
            code = torch.where(scale > 0, _nearest((blocks.abs() / (scale * sg)).nan_to_num(0.0), e2m1), 0.0)
            kept = (s["slots"][t:t + step] >= 0)[:, None, None]
            y[t:t + step] = torch.where(kept, (torch.sign(blocks) * code * scale * sg).reshape(x.shape), 0.0)
            clips += int(((x.abs() > 2688 * sg) & kept).sum())
        result[name] = y
    return {**result, "clips": torch.tensor([clips], device=DEV)}


def _exact_store(codes, scales, gscale):
    """64-bit values of one head's tokens, from the bits of their codes and scales."""
    n = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).double()
    sign, m = torch.where(n >= 8, -1.0, 1.0), torch.where(n >= 8, n - 8, n)
    mag = torch.where(m < 4, m / 2, torch.where(m < 6, m - 2, 2 * m - 8))
    b = scales.double()
    e, f = torch.floor(b / 8), b % 8
    scale = torch.where(e == 0, f * 2.0 ** -9, (8 + f) * torch.exp2(e - 10))
    return sign * mag * scale.repeat_interleave(16, -1) * gscale


def _exact_attention(s):
    c, kc, ks, vc, vs = s["case"], *s["store"]
    nq, kv = _attention_lengths(c)
    group = c["heads"] // c["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device=DEV)
    start = 0
    for b, (n, length) in enumerate(zip(nq.tolist(), kv.tolist())):
        pages = s["table"][b, :-(-length // c["page"])].long()
        for h in range(c["kv_heads"]):
            k, v = (_exact_store(x[pages, h].flatten(0, 1)[:length], y[pages, h].flatten(0, 1)[:length], sg)
                    for x, y, sg in ((kc, ks, s["gscales"][0]), (vc, vs, s["gscales"][1])))
            step = max(1, 200_000_000 // (length * group))
            for i in range(0, n, step):
                m = min(step, n - i)
                rows, heads = slice(start + i, start + i + m), slice(h * group, (h + 1) * group)
                z = torch.einsum("ngd,kd->ngk", s["q"][rows, heads].double(), k) * s["sm_scale"]
                key = torch.arange(length, device=DEV)
                place = (length - n + i + torch.arange(m, device=DEV))[:, None]
                hidden = torch.zeros((m, length), dtype=torch.bool, device=DEV)
                if c["causal"]:
                    hidden |= key > place
                if c["window"]:
                    hidden |= key <= place - c["window"]
                z = z.masked_fill(hidden[:, None], -math.inf)
                lse[rows, heads] = torch.logsumexp(z, -1)
                out[rows, heads] = torch.einsum("ngk,kd->ngd", torch.exp(z - lse[rows, heads][..., None]).nan_to_num(0.0), v)
        start += n
    return {"out": out, "lse": lse} if c["lse"] else {"out": out}
