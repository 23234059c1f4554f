"""Work of the rotated appends and of attention over the per-head 8-bit cache: cases, inputs, plain forms.

Three operators of a serving step:

- ``latent_append``: the MLA step's append. Row t of the latent cache is [c_kv(t) | R(pos) k_pe(t)], quantized into an
  FP8 or per-token-scaled FP8 pool; the query's rope part q_pe is rotated into the last 64 dims of the decode's q.
- ``heads_append``: the append of a model with K and V heads. K is rotated, V is not; both go into a paged pool of 8-bit
  codes with one FP32 scale for each (64-token page, K or V, head). The query heads are rotated in the same call.
- ``decode``: one query token per request against that pool, over all its tokens, or over a sliding window and a few
  first tokens.

``run`` computes them with elementary torch operations where ``own`` is false, and calls the library where it is true.
"""
from __future__ import annotations

import math

import torch

own = False

PAGE = 64
LATENT, ROPE = 576, 64
MAX_POS = 131072            # rows of the cos / sin table of the append cases
QMAX = {"e4m3": 448.0, "int8": 127.0}


# ------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one token of a single stream, 16 query heads: the smallest MLA step, all launch latency
        dict(name="latent_append_1", op="latent_append", n=1, heads=16, pool="fp8", style="pairs"),
        # the decode step of a 44-request batch at 128 heads: q_pe is most of the traffic
        dict(name="latent_append_44", op="latent_append", n=44, heads=128, pool="fp8", style="pairs"),
        # a prefill chunk of odd length into the per-token-scaled pool
        dict(name="latent_append_20011", op="latent_append", n=20011, heads=16, pool="fp8_token", style="pairs"),
        # the decode step of 64 requests, 64 query heads over 8: one token each, mostly into started pages
        dict(name="heads_append_64", op="heads_append", batch=64, lo=1, hi=1, before=4096, heads=64, kv_heads=8, dim=128,
             rot=128, cache="e4m3", style="halves"),
        # verification of a few drafted tokens per request, small heads, half of each head rotated, INT8
        dict(name="heads_append_33x5", op="heads_append", batch=33, lo=1, hi=5, before=2000, heads=28, kv_heads=4, dim=64,
             rot=32, cache="int8", style="pairs"),
        # chunked prefill: ragged chunks of eight requests that continue cached prefixes
        dict(name="heads_append_8x8k", op="heads_append", batch=8, lo=129, hi=8190, before=4096, heads=32, kv_heads=8, dim=128,
             rot=128, cache="e4m3", style="halves"),
        # the tiny decode: one request of 256 tokens, latency of the call
        dict(name="decode_1x256", op="decode", batch=1, lo=256, hi=256, heads=32, kv_heads=8, dim=128, cache="e4m3", window=0, sinks=0),
        # a full batch at 32,768 tokens each: the largest read
        dict(name="decode_44x32k", op="decode", batch=44, lo=32768, hi=32768, heads=64, kv_heads=8, dim=128, cache="e4m3", window=0, sinks=0),
        # mixed serving batch, log-uniform lengths, 16 query heads per KV head, INT8
        dict(name="decode_mixed_64", op="decode", batch=64, lo=512, hi=32768, heads=64, kv_heads=4, dim=128, cache="int8", window=0, sinks=0),
        # one long context: the split over the card and the join of its parts
        dict(name="decode_1x1m", op="decode", batch=1, lo=1048576, hi=1048576, heads=32, kv_heads=4, dim=128, cache="e4m3", window=0, sinks=0),
        # sliding-window layer of small heads: 128 requests, 1,024 tokens and 4 first ones, ragged, both edges inside pages
        dict(name="window_128x1k", op="decode", batch=128, lo=100, hi=16384, heads=64, kv_heads=8, dim=64, cache="e4m3", window=1024, sinks=4),
        # streaming over long contexts: wide heads, 4,095 tokens and a 70-token prompt that stays visible
        dict(name="window_16x4k", op="decode", batch=16, lo=30000, hi=65536, heads=16, kv_heads=2, dim=256, cache="int8", window=4095, sinks=70),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["latent_append", "heads_append", "decode", "decode", "window"])
    if op == "latent_append":
        return dict(op=op, n=_log_int(rng, 1, 16384), heads=rng.choice([16, 32, 64, 80, 128]), pool=rng.choice(["fp8", "fp8_token"]),
                    style=rng.choice(["pairs", "halves"]))
    heads = dict(kv_heads=rng.choice([1, 2, 4, 5, 8]), dim=rng.choice([64, 128, 128, 256]), cache=rng.choice(["e4m3", "int8"]))
    heads["heads"] = heads["kv_heads"] * rng.choice([1, 2, 4, 5, 7, 8, 10, 16])
    if op == "heads_append":
        lo, hi = rng.choice([(1, 1), (1, 5), (3, 300), (100, 4000)])
        batch = _log_int(rng, 1, 16 if hi > 300 else 128)
        return dict(op=op, batch=batch, lo=lo, hi=hi, before=_log_int(rng, 1, 4096), rot=rng.choice([32, 64, heads["dim"]]),
                    style=rng.choice(["pairs", "halves"]), **heads)
    top = int(1.0e9) // (2 * heads["kv_heads"] * heads["dim"])          # tokens of at most 1 GB of cache
    batch = _log_int(rng, 1, 128)
    hi = _log_int(rng, 1, min(300000, max(1, top // batch)))
    lo = rng.choice([hi, max(1, hi // 20), 1])
    if op == "decode":
        return dict(op="decode", batch=batch, lo=lo, hi=hi, window=0, sinks=0, **heads)
    return dict(op="decode", batch=batch, lo=lo, hi=hi, window=_log_int(rng, 1, 8192), sinks=rng.choice([0, 1, 4, 63, 130]), **heads)


# ------------------------------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)


def _host_gen(seed):
    return torch.Generator().manual_seed(int(seed) * 104729 + 5)


def _lengths(case, seed):
    """The requests' lengths, log-uniform whole numbers in [lo, hi], and what an append finds cached before, uniform up to
    ``before``: the same requests for every seed, so that outputs keep their shapes, in an order of the seed's own."""
    lo, hi, same = case["lo"], case["hi"], _host_gen(0)
    u = torch.rand(case["batch"], generator=same, dtype=torch.float64)
    x = torch.exp(math.log(lo) + u * (math.log(hi) - math.log(lo))).round().to(torch.int64).clamp(lo, hi)
    before = torch.randint(0, case.get("before", 0) + 1, (case["batch"],), generator=same)
    order = torch.randperm(case["batch"], generator=_host_gen(seed))
    return x[order].tolist(), before[order].tolist()


def _table(rot):
    """cos | sin of every position, angles in 64 bits, held in FP32."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    ang = torch.arange(MAX_POS, dtype=torch.float64, device="cuda")[:, None] * inv
    return torch.cat([ang.cos(), ang.sin()], 1).float()


def _page_table(npages, seed):
    """CSR page table over a pool of shuffled pages, a few of them spare: (indptr list, page ids, pool pages)."""
    indptr = [0]
    for n in npages:
        indptr.append(indptr[-1] + n)
    pool = indptr[-1] + 3
    ids = torch.randperm(pool, generator=_host_gen(seed + 1))[:indptr[-1]].to(torch.int32)
    return indptr, ids, pool


def _pool(case, pages, gen):
    """A pool of quantized N(0, 1) heads with a few strong channels: codes [pages][2][heads][64][D], scales [pages][2][heads]."""
    h, d, qmax = case["kv_heads"], case["dim"], QMAX[case["cache"]]
    codes = torch.empty((pages, 2, h, PAGE, d), dtype=torch.uint8, device="cuda")
    scale = torch.empty((pages, 2, h), dtype=torch.float32, device="cuda")
    gain = torch.ones(2, h, 1, d, device="cuda")
    gain[0, :, :, ::37] = 6.0
    step = max(1, (64 << 20) // (2 * h * PAGE * d))
    for a in range(0, pages, step):
        b = min(pages, a + step)
        x = torch.randn((b - a, 2, h, PAGE, d), generator=gen, device="cuda") * gain
        s = x.abs().amax((3, 4)) / qmax
        codes[a:b] = _codes(x / s[..., None, None], case["cache"]).view(torch.uint8)
        scale[a:b] = s
    return codes, scale


def prepare(case, seed):
    g = _gen(seed)
    dev = "cuda"
    s = {"case": dict(case)}
    if case["op"] == "latent_append":
        n, heads = case["n"], case["heads"]
        pages = (2 * n + PAGE - 1) // PAGE + 1
        # prefill fills pages in order, a decode step touches one place in each of many pages
        slots = torch.randperm(pages * PAGE, generator=_host_gen(seed))[:n]
        if n > 1024:
            order = torch.randperm(pages, generator=_host_gen(seed))
            slots = (order[:, None] * PAGE + torch.arange(PAGE)).reshape(-1)[:n]
        s["c_kv"] = torch.randn((n, 512), generator=g, device=dev).bfloat16()
        s["k_pe"] = torch.randn((n, LATENT), generator=g, device=dev).bfloat16()[:, 512:]      # a view of the projection
        s["q_pe"] = torch.randn((n, heads, 2 * ROPE), generator=g, device=dev).bfloat16()[:, :, ROPE:]
        s["q"] = torch.randn((n, heads, LATENT), generator=g, device=dev).bfloat16()
        s["slots"] = slots.to(dev)
        s["positions"] = torch.randint(0, MAX_POS, (n,), generator=g, device=dev)
        s["table"] = _table(ROPE)
        width = PAGE * LATENT if case["pool"] == "fp8" else PAGE * (LATENT + 4)
        s["pool"] = torch.zeros((pages, width), dtype=torch.uint8, device=dev)
        return s
    h, d, heads, batch = case["kv_heads"], case["dim"], case["heads"], case["batch"]
    if case["op"] == "heads_append":
        new, before = _lengths(case, seed)
        indptr, ids, pages = _page_table([(a + b + PAGE - 1) // PAGE for a, b in zip(before, new)], seed)
        n = sum(new)
        qkv = torch.randn((n, (heads + 2 * h) * d), generator=g, device=dev)
        # one token in nine is up to eight times stronger: blocks whose scale has to grow
        qkv = (qkv * torch.exp2(3 * torch.rand((n, 1), generator=g, device=dev) * (torch.rand((n, 1), generator=g, device=dev) < 0.11))).bfloat16()
        s["q"] = qkv[:, :heads * d].view(n, heads, d)                   # views of one projection
        s["k"] = qkv[:, heads * d:(heads + h) * d].view(n, h, d)
        s["v"] = qkv[:, (heads + h) * d:].view(n, h, d)
        tok = [0]
        for x in new:
            tok.append(tok[-1] + x)
        s["tok_indptr"] = torch.tensor(tok, dtype=torch.int32, device=dev)
        s["kv_len"] = torch.tensor(before, dtype=torch.int32, device=dev)
        s["kv_indptr"] = torch.tensor(indptr, dtype=torch.int32, device=dev)
        s["kv_indices"] = ids.to(dev)
        s["codes"], s["scale"] = _pool(case, pages, g)
        s["table"] = _table(case["rot"])
        s["q_out"] = torch.empty((n, heads, d), dtype=torch.bfloat16, device=dev)
        return s
    lens, _ = _lengths(case, seed)
    indptr, ids, pages = _page_table([(x + PAGE - 1) // PAGE for x in lens], seed)
    s["kv_indices"] = ids.to(dev)
    s["codes"], s["scale"] = _pool(case, pages, g)
    s["q"] = torch.randn((batch, heads, d), generator=g, device=dev).bfloat16()
    s["sm_scale"] = d ** -0.5
    # the pages that each request sees: (request, first token of the page, entry of the page table)
    req, first, entry = [], [], []
    for r, n in enumerate(lens):
        for p in range((n + PAGE - 1) // PAGE):
            if not case["window"] or p * PAGE < case["sinks"] or (p + 1) * PAGE > n - case["window"]:
                req.append(r)
                first.append(p * PAGE)
                entry.append(indptr[r] + p)
    s["lens"], s["indptr"] = lens, indptr
    s["page_req"] = torch.tensor(req, dtype=torch.int64, device=dev)
    s["page_first"] = torch.tensor(first, dtype=torch.int64, device=dev)
    s["page_entry"] = torch.tensor(entry, dtype=torch.int64, device=dev)
    s["kv_len"] = torch.tensor(lens, dtype=torch.int64, device=dev)
    s["out"] = torch.empty((batch, heads, d), dtype=torch.bfloat16, device=dev)
    s["lse"] = torch.empty((batch, heads), dtype=torch.float32, device=dev)
    if own:
        # a serving step plans once on the host and runs every layer on that plan
        import quantized_kv_paged_gb300 as q
        args = (indptr, lens, heads, h, d, _CACHE(q)[case["cache"]])
        kw = dict(window=case["window"], sinks=case["sinks"])
        s["workspace"] = torch.empty(max(256, q.gqa_decode_plan(*args, **kw).workspace_bytes), dtype=torch.uint8, device=dev)
        s["plan"] = q.gqa_decode_plan(*args, workspace=s["workspace"], **kw)
    return s


def _CACHE(q):
    return {"e4m3": q.CACHE_E4M3, "int8": q.CACHE_INT8}


# ------------------------------------------------------------------------------------------------- plain forms
def _codes(x, cache):
    """x (in units of the block's scale) rounded to the cache's 8-bit type."""
    if cache == "int8":
        return x.round().clamp(-127, 127).to(torch.int8)
    return x.clamp(-448, 448).to(torch.float8_e4m3fn)


def _quotient(x, by):
    """x / by, one FP32 rounding (a division by a Python number is a product with its rounded reciprocal)."""
    return x / torch.full_like(x, by)


def _values(codes, cache):
    return codes.view(torch.int8 if cache == "int8" else torch.float8_e4m3fn)


def _rotate(x, cs, style):
    """x [n][heads][D]: the first r = table width dims rotated by the rows cs [n][r] (cos | sin), the rest as they are."""
    r = cs.shape[1]
    c, s = cs[:, None, :r // 2], cs[:, None, r // 2:]
    out = x.clone()
    if style == "halves":
        a, b = x[..., :r // 2], x[..., r // 2:r]
        out[..., :r // 2], out[..., r // 2:r] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        out[..., 0:r:2], out[..., 1:r:2] = a * c - b * s, b * c + a * s
    return out


def _latent_outputs(s):
    """The pool as the values its bytes stand for, and the decode's q."""
    if s["case"]["pool"] == "fp8":
        return {"codes": s["pool"].view(torch.float8_e4m3fn), "q": s["q"]}
    return {"codes": s["pool"][:, :PAGE * LATENT].view(torch.float8_e4m3fn), "scale": s["pool"][:, PAGE * LATENT:].view(torch.float32), "q": s["q"]}


def _plain_latent(s):
    cs = s["table"][s["positions"]]
    style = s["case"]["style"]
    row = torch.cat([s["c_kv"].float(), _rotate(s["k_pe"].float()[:, None], cs, style)[:, 0]], 1)
    page, off = s["slots"] // PAGE, s["slots"] % PAGE
    pages = s["pool"].shape[0]
    codes = s["pool"][:, :PAGE * LATENT].view(pages, PAGE, LATENT)
    if s["case"]["pool"] == "fp8_token":
        scale = _quotient(row.abs().amax(1), 448.0)
        s["pool"][:, PAGE * LATENT:].view(torch.float32)[page, off] = scale
        row = torch.where(scale[:, None] > 0, row / scale[:, None], row)
    codes[page, off] = _codes(row, "e4m3").view(torch.uint8)
    s["q"][..., 512:] = _rotate(s["q_pe"].float(), cs, style).bfloat16()
    return _latent_outputs(s)


def _placed(s):
    """Request, position and (page, offset) of every new token."""
    n = s["k"].shape[0]
    i = torch.arange(n, device="cuda", dtype=torch.int32)
    r = torch.searchsorted(s["tok_indptr"], i, right=True) - 1
    pos = (s["kv_len"][r] + i - s["tok_indptr"][r]).long()
    page = s["kv_indices"][s["kv_indptr"][r].long() + pos // PAGE].long()
    return pos, page, pos % PAGE


def _plain_heads(s):
    case = s["case"]
    cache, qmax = case["cache"], QMAX[case["cache"]]
    pos, page, off = _placed(s)
    cs = s["table"][pos]
    x = torch.stack([_rotate(s["k"].float(), cs, case["style"]), s["v"].float()], 1)        # [n][2][heads][D]
    pages = s["scale"].shape[0]
    first = torch.full((pages,), PAGE, device="cuda").scatter_reduce(0, page, off, "amin")
    need = _quotient(torch.zeros_like(s["scale"]).index_reduce(0, page, x.abs().amax(3), "amax"), qmax)
    touched = (first < PAGE).nonzero()[:, 0]
    old, need, first = s["scale"][touched], need[touched], first[touched]
    # the scale of a started block grows by the smallest power of two that holds the new tokens
    m_need, e_need = torch.frexp(need)
    m_old, e_old = torch.frexp(old)
    j = (e_need - e_old + (m_need > m_old).int()).clamp(min=0)
    fresh = (first == 0)[:, None, None] | (old == 0)
    j = torch.where(fresh, torch.zeros_like(j), j)
    scale = torch.where(fresh, need, torch.ldexp(old, j))
    block = s["codes"][touched]
    older = torch.arange(PAGE, device="cuda") < first[:, None]                               # [pages][64]
    shrunk = _codes(torch.ldexp(_values(block, cache).float(), -j[..., None, None]), cache).view(torch.uint8)
    s["codes"][touched] = torch.where(older[:, None, None, :, None], shrunk, block)
    s["scale"][touched] = scale
    sx = s["scale"][page][..., None]
    s["codes"][page, :, :, off] = _codes(torch.where(sx > 0, x / sx, x), cache).view(torch.uint8)
    return {"codes": _values(s["codes"], cache), "scale": s["scale"], "q": _rotate(s["q"].float(), cs, case["style"]).bfloat16()}


def _visible(s):
    """[pages][64]: the tokens that their request's query sees."""
    case = s["case"]
    t = s["page_first"][:, None] + torch.arange(PAGE, device="cuda")
    n = s["kv_len"][s["page_req"]][:, None]
    seen = t < n
    if case["window"]:
        seen &= (t >= n - case["window"]) | (t < case["sinks"])
    return seen


def _plain_decode(s):
    case = s["case"]
    h, d, batch = case["kv_heads"], case["dim"], case["batch"]
    group = case["heads"] // h
    page, req = s["kv_indices"][s["page_entry"]].long(), s["page_req"]
    q = s["q"].float().view(batch, h, group, d)
    k = _values(s["codes"][page, 0], case["cache"]).float() * s["scale"][page, 0][..., None, None]
    z = torch.matmul(q[req], k.transpose(2, 3)) * s["sm_scale"]                              # [pages][h][group][64]
    del k
    z = torch.where(_visible(s)[:, None, None], z, -torch.inf)
    m = torch.full((batch, h, group), -torch.inf, device="cuda").index_reduce(0, req, z.amax(3), "amax")
    p = torch.exp(z - m[req][..., None])
    total = torch.zeros((batch, h, group), device="cuda").index_add(0, req, p.sum(3))
    v = _values(s["codes"][page, 1], case["cache"]).float() * s["scale"][page, 1][..., None, None]
    out = torch.zeros((batch, h, group, d), device="cuda").index_add(0, req, torch.matmul(p, v)) / total[..., None]
    return {"out": out.view(batch, h * group, d).bfloat16(), "lse": (m + total.log()).view(batch, h * group)}


# ------------------------------------------------------------------------------------------------- one pass
def run(s):
    case = s["case"]
    if not own:
        return {"latent_append": _plain_latent, "heads_append": _plain_heads, "decode": _plain_decode}[case["op"]](s)
    import quantized_kv_paged_gb300 as q
    if case["op"] == "latent_append":
        kv = q.KV_FP8_E4M3 if case["pool"] == "fp8" else q.KV_FP8_PER_TOKEN
        style = q.ROPE_PAIRS if case["style"] == "pairs" else q.ROPE_HALVES
        q.mla_append_rope(s["c_kv"], s["k_pe"], s["slots"], s["positions"], s["table"], style, s["pool"], None, kv, q_pe=s["q_pe"], q=s["q"])
        return _latent_outputs(s)
    cache = _CACHE(q)[case["cache"]]
    if case["op"] == "heads_append":
        style = q.ROPE_PAIRS if case["style"] == "pairs" else q.ROPE_HALVES
        q.gqa_append_rope(s["k"], s["v"], s["tok_indptr"], s["kv_len"], s["kv_indptr"], s["kv_indices"], s["table"], style, s["codes"],
                          s["scale"], cache, q=s["q"], q_out=s["q_out"])
        return {"codes": _values(s["codes"], case["cache"]), "scale": s["scale"], "q": s["q_out"]}
    q.gqa_decode_run(s["plan"], s["q"], s["codes"], s["scale"], s["kv_indices"], s["sm_scale"], s["out"], s["lse"], s["workspace"])
    return {"out": s["out"], "lse": s["lse"]}


def work(case):
    if case["op"] == "latent_append":
        n, heads = case["n"], case["heads"]
        row = 2 * LATENT + LATENT + (4 if case["pool"] == "fp8_token" else 0) + 4 * ROPE + 16
        return {"bytes": n * (row + heads * 2 * 2 * ROPE), "flops": n * (heads + 1) * 3 * ROPE}
    h, d, heads = case["kv_heads"], case["dim"], case["heads"]
    mean = lambda lo, hi: float(lo) if lo == hi else (hi - lo) / math.log(hi / lo)  # noqa: E731
    if case["op"] == "heads_append":
        n = case["batch"] * mean(case["lo"], case["hi"])
        return {"bytes": n * (2 * h * d * 3 + 4 * heads * d + 4 * case["rot"]), "flops": n * (heads + h) * 3 * case["rot"]}
    # tokens seen by a request, averaged over its log-uniform length
    lo, hi = case["lo"], case["hi"]
    grid = [math.exp(math.log(lo) + (i + 0.5) / 200 * (math.log(hi) - math.log(lo))) for i in range(200)]
    seen = [x if not case["window"] else min(x, case["window"] + min(case["sinks"], max(0.0, x - case["window"]))) for x in grid]
    tokens = case["batch"] * sum(seen) / len(seen)
    return {"bytes": tokens * (2 * h * d + 8 * h / PAGE) + case["batch"] * heads * (4 * d + 4), "flops": tokens * heads * 4 * d}


# ------------------------------------------------------------------------------------------------- the definitions in 64 bits
def _turn64(x, cs, style):
    """Rotation as a product of complex numbers, in 64 bits."""
    r = cs.shape[1]
    w = torch.complex(cs[:, :r // 2].double(), cs[:, r // 2:].double())[:, None]
    x = x.double()
    head = x[..., :r].unflatten(-1, (2, r // 2)).transpose(-1, -2) if style == "halves" else x[..., :r].unflatten(-1, (r // 2, 2))
    y = torch.view_as_real(torch.view_as_complex(head.contiguous()) * w)
    y = y.transpose(-1, -2).flatten(-2) if style == "halves" else y.flatten(-2)
    return torch.cat([y, x[..., r:]], -1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "latent_append":
        cs = s["table"][s["positions"]]
        row = torch.cat([s["c_kv"].double(), _turn64(s["k_pe"][:, None], cs, case["style"])[:, 0]], 1)
        pages = s["pool"].shape[0]
        codes = torch.zeros((pages * PAGE, LATENT), dtype=torch.float64, device="cuda")
        q = torch.cat([s["q"][..., :512].double(), _turn64(s["q_pe"], cs, case["style"])], 2)
        if case["pool"] == "fp8":
            codes[s["slots"]] = row.clamp(-448, 448)
            return {"codes": codes.view(pages, PAGE * LATENT), "q": q}
        scale = torch.zeros(pages * PAGE, dtype=torch.float64, device="cuda")
        scale[s["slots"]] = row.abs().amax(1) / 448
        codes[s["slots"]] = row / scale[s["slots"]][:, None]
        return {"codes": codes.view(pages, PAGE * LATENT), "scale": scale.view(pages, PAGE), "q": q}
    if case["op"] == "heads_append":
        qmax = QMAX[case["cache"]]
        table, style = s["table"], case["style"]
        codes, scale = _values(s["codes"], case["cache"]).double(), s["scale"].double()
        q = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
        tok, before = s["tok_indptr"].tolist(), s["kv_len"].tolist()
        indptr, ids = s["kv_indptr"].tolist(), s["kv_indices"].tolist()
        for r in range(case["batch"]):
            t0, t1, at = tok[r], tok[r + 1], before[r]
            cs = table[at:at + t1 - t0]
            q[t0:t1] = _turn64(s["q"][t0:t1], cs, style)
            x = torch.stack([_turn64(s["k"][t0:t1], cs, style), s["v"][t0:t1].double()], 0).transpose(1, 2)      # [2][heads][n][D]
            i = 0
            while i < t1 - t0:
                page, o = ids[indptr[r] + (at + i) // PAGE], (at + i) % PAGE
                n = min(PAGE - o, t1 - t0 - i)
                new = x[:, :, i:i + n]
                need = new.abs().amax((2, 3)) / qmax
                if o == 0:
                    grown = need
                else:
                    grown = scale[page] * torch.exp2(torch.ceil(torch.log2(need / scale[page])).clamp(min=0))
                    codes[page, :, :, :o] *= (scale[page] / grown)[..., None, None]
                scale[page] = grown
                codes[page, :, :, o:o + n] = new / grown[..., None, None]
                i += n
        return {"codes": codes if case["cache"] == "e4m3" else None, "scale": scale, "q": q}
    h, d, batch, heads = case["kv_heads"], case["dim"], case["batch"], case["heads"]
    out = torch.empty((batch, heads, d), dtype=torch.float64, device="cuda")
    lse = torch.empty((batch, heads), dtype=torch.float64, device="cuda")
    ids = s["kv_indices"].long()
    for r, n in enumerate(s["lens"]):
        pages = ids[s["indptr"][r]:s["indptr"][r + 1]]
        t = torch.arange(n, device="cuda")
        if case["window"]:
            t = t[(t >= n - case["window"]) | (t < case["sinks"])]
        page, off = pages[t // PAGE], t % PAGE
        for j in range(h):
            k, v = (_values(s["codes"][page, i, j, off], case["cache"]).double() * s["scale"][page, i, j].double()[:, None] for i in (0, 1))
            group = slice(j * (heads // h), (j + 1) * (heads // h))
            z = s["q"][r, group].double() @ k.T * s["sm_scale"]
            lse[r, group] = torch.logsumexp(z, 1)
            out[r, group] = torch.softmax(z, 1) @ v
    return {"out": out, "lse": lse}
