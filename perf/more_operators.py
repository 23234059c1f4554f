"""Work of speculative decoding over the paged caches: cases, inputs, plain forms.

Three operators of a serving loop that drafts tokens:

- ``tree``: attention of drafted tokens over the per-head 8-bit cache. The drafted tokens of a request lie behind its cached
  ones; each sees the cached tokens (all, or a sliding window and a few first ones) and the drafted tokens of its own path,
  given as a bit mask, or all the drafted tokens before it (a chain).
- ``commit``: the accepted path's tokens move to the slots right behind the cached ones, in every layer. A block (page, K or V,
  head) has one scale, so a token that leaves its page is requantized, and the block that takes it may have to grow its scale.
- ``pages``: page tables, reference counts and a free list on the device: copying pages, forking requests (full pages are
  shared, the started one is copied), freeing, compacting and growing them, over the pools of all layers.

``run`` computes them with elementary torch operations where ``own`` is false, and calls the library where it is true.
"""
from __future__ import annotations

import math
import random

import torch

own = False

PAGE = 64
QMAX = {"e4m3": 448.0, "int8": 127.0}
# bytes that a page takes in each buffer of one layer's pool
POOLS = {"fp8": (PAGE * 576,), "fp8_token": (PAGE * 580,), "nvfp4": (PAGE * 288, PAGE * 36),
         "heads": (2 * 8 * PAGE * 128, 2 * 8 * 4), "heads64": (2 * 4 * PAGE * 64, 2 * 4 * 4)}


# ------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # a single stream that drafts a tree of 8: all latency
        dict(name="tree_1x300_8", op="tree", batch=1, lo=300, hi=300, tlo=8, thi=8, heads=32, kv_heads=8, dim=128, cache="e4m3", window=0, sinks=0,
             mask="tree"),
        # a full batch at 32,768 tokens that verifies a chain of 4 (a multi-token-prediction head): the largest read
        dict(name="tree_44x32k_4", op="tree", batch=44, lo=32768, hi=32768, tlo=4, thi=4, heads=64, kv_heads=8, dim=128, cache="e4m3", window=0,
             sinks=0, mask="chain"),
        # mixed serving batch, trees of 64 drafted tokens: 512 rows on every KV head, the matrix products count
        dict(name="tree_mixed16_64", op="tree", batch=16, lo=1000, hi=32768, tlo=64, thi=64, heads=64, kv_heads=8, dim=128, cache="e4m3", window=0,
             sinks=0, mask="tree"),
        # one long context, 33 drafted tokens, seven query heads on a KV head, INT8: the split over the card and its join
        dict(name="tree_1x200k_33", op="tree", batch=1, lo=200001, hi=200001, tlo=33, thi=33, heads=28, kv_heads=4, dim=128, cache="int8", window=0,
             sinks=0, mask="tree"),
        # sliding-window layer of small heads: ragged trees of 1 to 60, a window of 1,024 and 4 first tokens
        dict(name="tree_window64", op="tree", batch=64, lo=100, hi=16384, tlo=1, thi=60, heads=64, kv_heads=8, dim=64, cache="int8", window=1024,
             sinks=4, mask="tree"),
        # wide heads, trees of 20
        dict(name="tree_12x8k_20", op="tree", batch=12, lo=2000, hi=8191, tlo=20, thi=20, heads=16, kv_heads=2, dim=256, cache="e4m3", window=0, sinks=0,
             mask="tree"),
        # the end of a step for a single stream: up to 5 accepted tokens in 28 layers
        dict(name="commit_1", op="commit", batch=1, layers=28, tree=16, accept=5, kv_heads=8, dim=128, cache="e4m3"),
        # the end of a step of 64 requests, 48 layers, trees of 40: paths that cross pages
        dict(name="commit_64", op="commit", batch=64, layers=48, tree=40, accept=9, kv_heads=4, dim=128, cache="int8"),
        # a single prompt's started pages copied in a small model: all latency
        dict(name="pages_copy_3", op="pages", kind="copy", n=3, layers=4, pool="heads64", rows=0, held=0),
        # a prefix of 8,192 tokens duplicated in a 27-layer latent pool: bandwidth
        dict(name="pages_copy_128", op="pages", kind="copy", n=128, layers=27, pool="fp8_token", rows=0, held=0),
        # sampling of several continuations: 6 prompts forked into 48 requests, which grow and are then freed
        dict(name="pages_fork_48", op="pages", kind="fork", n=48, layers=48, pool="heads", rows=60, held=40),
        # requests come and go: half of them are freed, the pool is compacted, new ones take their place
        dict(name="pages_compact_80", op="pages", kind="compact", n=40, layers=27, pool="nvfp4", rows=80, held=60),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "window", "commit", "pages"])
    if op == "commit":
        tree = _log_int(rng, 2, 64)
        return dict(op=op, batch=_log_int(rng, 1, 64), layers=_log_int(rng, 2, 48), tree=tree, accept=rng.randint(1, min(tree, 12)),
                    kv_heads=rng.choice([1, 2, 4, 5]), dim=rng.choice([64, 128, 256]),
                    cache=rng.choice(["e4m3", "int8"]))
    if op == "pages":
        kind, pool = rng.choice(["copy", "fork", "compact"]), rng.choice(sorted(POOLS))
        layers = _log_int(rng, 2, 27)
        if kind == "copy":
            return dict(op=op, kind=kind, n=_log_int(rng, 1, 128), layers=layers, pool=pool, rows=0, held=0)
        if kind == "fork":
            n = _log_int(rng, 1, 48)
            return dict(op=op, kind=kind, n=n, layers=layers, pool=pool, rows=n + rng.randint(1, 12), held=_log_int(rng, 1, 40))
        n, held = _log_int(rng, 2, 32), _log_int(rng, 1, 40)
        layers = min(layers, max(1, int(2e9) // (2 * n * (held + 1) * sum(POOLS[pool]))))
        return dict(op=op, kind=kind, n=n, layers=layers, pool=pool, rows=2 * n, held=held)
    kv_heads, dim = rng.choice([1, 2, 4, 5, 8]), rng.choice([64, 128, 128, 256])
    heads = kv_heads * rng.choice([1, 2, 4, 5, 7, 8, 10, 16])
    thi = _log_int(rng, 1, 96)
    batch = _log_int(rng, 1, 64)
    # at most 0.5 GB of cache and 0.2 Tflop of products
    top = min(int(0.5e9) // (2 * kv_heads * dim), int(2e11) // (4 * dim * heads * thi))
    hi = _log_int(rng, 1, min(200000, max(1, top // batch)))
    case = dict(op="tree", batch=batch, lo=rng.choice([hi, max(1, hi // 20), 1]), hi=hi, tlo=rng.choice([thi, max(1, thi // 3), 1]), thi=thi, heads=heads,
                kv_heads=kv_heads, dim=dim, cache=rng.choice(["e4m3", "int8"]), window=0, sinks=0, mask=rng.choice(["tree", "tree", "chain"]))
    if op == "window":
        case.update(window=_log_int(rng, 96, 8192), sinks=rng.choice([0, 1, 4, 63, 130]))
    return case


# ------------------------------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 29)


def _host_gen(seed):
    return torch.Generator().manual_seed(int(seed) * 104729 + 11)


def _spread(lo, hi, n, gen):
    """n log-uniform whole numbers in [lo, hi]."""
    u = torch.rand(n, generator=gen, dtype=torch.float64)
    return torch.exp(math.log(lo) + u * (math.log(hi) - math.log(lo))).round().to(torch.int64).clamp(lo, hi)


def _page_table(npages, seed):
    """CSR page table over a pool of shuffled pages, a few of them spare: (indptr list, page ids, pool pages)."""
    indptr = [0]
    for n in npages:
        indptr.append(indptr[-1] + n)
    pool = indptr[-1] + 3
    ids = torch.randperm(pool, generator=_host_gen(seed + 1))[:indptr[-1]].to(torch.int32)
    return indptr, ids, pool


def _head_pool(case, pages, gen):
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


def _tree_parents(n, host):
    """A random tree: parent of every drafted token but the roots (-1), parents before their children."""
    return [-1 if i == 0 or host.random() < 0.1 else host.randrange(max(0, i - 8), i) for i in range(n)]


def prepare(case, seed):
    return {"tree": _prepare_tree, "commit": _prepare_commit, "pages": _prepare_pages}[case["op"]](case, seed)


def _prepare_tree(case, seed):
    g, dev = _gen(seed), "cuda"
    h, d, heads, batch = case["kv_heads"], case["dim"], case["heads"], case["batch"]
    # the same requests for every seed, so that outputs keep their shapes, in an order of the seed's own
    same, order = _host_gen(0), torch.randperm(batch, generator=_host_gen(seed))
    cached = _spread(case["lo"], case["hi"], batch, same)[order].tolist()
    drafted = _spread(case["tlo"], case["thi"], batch, same)[order].tolist()
    lens = [a + b for a, b in zip(cached, drafted)]
    indptr, ids, pages = _page_table([(x + PAGE - 1) // PAGE for x in lens], seed)
    tok = [0]
    for x in drafted:
        tok.append(tok[-1] + x)
    s = {"case": dict(case), "cached": cached, "lens": lens, "indptr": indptr, "tok": tok, "kv_indices": ids.to(dev)}
    s["codes"], s["scale"] = _head_pool(case, pages, g)
    s["q"] = torch.randn((tok[-1], heads, d), generator=g, device=dev).bfloat16()
    s["sm_scale"] = d ** -0.5
    s["mask"] = None
    if case["mask"] == "tree":
        host, words = random.Random(seed * 31 + 7), (max(drafted) + 31) // 32
        rows = []
        for n in drafted:
            seen = []
            for i, p in enumerate(_tree_parents(n, host)):
                seen.append((seen[p] if p >= 0 else 0) | 1 << i)
            rows += [[(m >> 32 * w) & 0xffffffff for w in range(words)] for m in seen]
        s["mask"] = torch.tensor(rows, dtype=torch.int64).to(torch.uint32).view(torch.int32).to(dev)
    s["out"] = torch.empty((tok[-1], heads, d), dtype=torch.bfloat16, device=dev)
    s["lse"] = torch.empty((tok[-1], heads), dtype=torch.float32, device=dev)
    if own:
        # a serving step plans once on the host and runs every layer on that plan
        import quantized_kv_paged_gb300 as q
        args = (indptr, lens, tok, heads, h, d, _CACHE(q)[case["cache"]])
        kw = dict(window=case["window"], sinks=case["sinks"])
        s["workspace"] = torch.empty(max(256, q.gqa_tree_plan(*args, **kw).workspace_bytes), dtype=torch.uint8, device=dev)
        s["plan"] = q.gqa_tree_plan(*args, workspace=s["workspace"], **kw)
    return s


def _prepare_commit(case, seed):
    g, host, dev = _gen(seed), random.Random(seed * 17 + 3), "cuda"
    batch, layers, tree = case["batch"], case["layers"], case["tree"]
    cached = [host.randint(0, 150) for _ in range(batch)]
    indptr, ids, pages = _page_table([(150 + tree + PAGE - 1) // PAGE] * batch, seed)
    path = [sorted(host.sample(range(tree), host.randint(1, case["accept"]))) for _ in range(batch)]
    s = {"case": dict(case)}
    # one buffer of all layers' pages; the call takes the layers' pools
    codes, scale = _head_pool(case, layers * pages, g)
    # tokens of some pages are up to eight times stronger than their neighbours': blocks that have to grow
    scale *= torch.exp2(3 * torch.rand((layers * pages, 1, 1), generator=g, device=dev))
    s["all_codes"], s["all_scale"] = codes.unflatten(0, (layers, pages)), scale.unflatten(0, (layers, pages))
    s["codes"], s["scale"] = list(s["all_codes"]), list(s["all_scale"])
    s["kv_len"] = torch.tensor(cached, dtype=torch.int32, device=dev)
    s["kv_indptr"] = torch.tensor(indptr, dtype=torch.int32, device=dev)
    s["kv_indices"] = ids.to(dev)
    s["path"] = torch.tensor([p + [0] * (case["accept"] - len(p)) for p in path], dtype=torch.int32, device=dev)
    s["path_len"] = torch.tensor([len(p) for p in path], dtype=torch.int32, device=dev)
    return s


def _prepare_pages(case, seed):
    # the same requests for every seed, so that outputs keep their shapes; the pages they hold and the contents are the seed's
    g, host, dev = _gen(seed), random.Random(case["n"] * 13 + 1), "cuda"
    n, rows, kind = case["n"], case["rows"], case["kind"]
    s = {"case": dict(case)}
    if kind == "copy":
        pages = 2 * n + 3
        order = torch.randperm(pages, generator=_host_gen(seed))
        s["src"], s["dst"] = order[:n].to(torch.int32).to(dev), order[n:2 * n].to(torch.int32).to(dev)
    else:
        limit = case["held"] + 4
        held = [host.randint(1, case["held"]) for _ in range(rows)]
        if kind == "fork":
            # the first rows hold prompts, the others are empty and take the forks
            prompts = rows - n
            lens = [h * PAGE - host.randint(0, PAGE - 1) if r < prompts else 0 for r, h in enumerate(held)]
            held = [(x + PAGE - 1) // PAGE for x in lens]
            pages = sum(held) + 4 * n + 2
            ids = torch.randperm(pages, generator=_host_gen(seed)).tolist()
            pick = [random.Random(seed * 13 + i).randrange(prompts) for i in range(n)]
            s["parents"] = torch.tensor(pick, dtype=torch.int32, device=dev)
            s["children"] = torch.arange(prompts, rows, dtype=torch.int32, device=dev)
            # each fork writes on for up to two pages
            s["tokens"] = torch.tensor([lens[p] + host.randint(1, 2 * PAGE) for p in pick], dtype=torch.int32, device=dev)
        else:
            # two halves of the requests: the first one's pages lie below the second one's, each in any order
            lens = [h * PAGE - host.randint(0, PAGE - 1) for h in held]
            live, low = sum(held), sum(held[:n])
            pages = live + max(2, live // 8)
            ids = torch.randperm(low, generator=_host_gen(seed)).tolist() + (low + torch.randperm(live - low, generator=_host_gen(seed + 1))).tolist()
            ids += list(range(live, pages))
            s["halves"] = [torch.arange(n, dtype=torch.int32, device=dev), torch.arange(n, rows, dtype=torch.int32, device=dev)]
            s["wants"] = [torch.tensor(lens[:n], dtype=torch.int32, device=dev), torch.tensor(lens[n:], dtype=torch.int32, device=dev)]
        table, at = [], 0
        for h in held:
            table.append(ids[at:at + h] + [-1] * (limit - h))
            at += h
        s["table"] = torch.tensor(table, dtype=torch.int32, device=dev)
        s["held"] = torch.tensor(held, dtype=torch.int32, device=dev)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
        s["refs"] = torch.zeros(pages, dtype=torch.int32, device=dev)
        s["refs"][torch.tensor(ids[:at], device=dev)] = 1
        free = sorted(ids[at:], reverse=True)
        s["free_list"] = torch.tensor(free + [0] * (pages - len(free)), dtype=torch.int32, device=dev)
        s["free_count"] = torch.tensor([len(free)], dtype=torch.int32, device=dev)
        s["status"] = torch.zeros(n, dtype=torch.int32, device=dev)
        s["status2"] = torch.zeros(n, dtype=torch.int32, device=dev)
        if own:
            import quantized_kv_paged_gb300 as q
            s["workspace"] = torch.zeros(q.kv_pages_workspace(pages, rows, n), dtype=torch.uint8, device=dev)
    # a buffer of all layers for each part of a pool; the calls take the layers' pools
    s["buffers"] = [torch.randint(0, 256, (case["layers"], pages, b), generator=g, dtype=torch.uint8, device=dev) for b in POOLS[case["pool"]]]
    s["pools"] = [layer for buffer in s["buffers"] for layer in buffer]
    return s


def _CACHE(q):
    return {"e4m3": q.CACHE_E4M3, "int8": q.CACHE_INT8}


# ------------------------------------------------------------------------------------------------- plain forms
def _codes(x, cache):
    """x (in units of the block's scale) rounded to the cache's 8-bit type."""
    if cache == "int8":
        return x.round().clamp(-127, 127).to(torch.int8)
    return x.clamp(-448, 448).to(torch.float8_e4m3fn)


def _values(codes, cache):
    return codes.view(torch.int8 if cache == "int8" else torch.float8_e4m3fn)


def _plain_tree(s):
    case = s["case"]
    h, d, cache = case["kv_heads"], case["dim"], case["cache"]
    group = case["heads"] // h
    for r, n in enumerate(s["lens"]):
        t0, t1, cached = s["tok"][r], s["tok"][r + 1], s["cached"][r]
        drafted = t1 - t0
        j = torch.arange(drafted, device="cuda")
        if s["mask"] is None:
            path = j[None, :] <= j[:, None]
        else:
            path = ((s["mask"][t0:t1].long()[:, j // 32] >> (j % 32)) & 1).bool()
        t = torch.arange(n, device="cuda")
        first = 0
        seen = torch.ones((drafted, n), dtype=torch.bool, device="cuda")
        if case["window"]:
            begin = cached + path.sum(1) - case["window"]
            seen = (t[None, :] >= begin[:, None]) | (t[None, :] < case["sinks"])
            first = max(0, cached - case["window"])
        seen[:, cached:] = path
        # without its invisible middle where there is a window
        if first > case["sinks"]:
            keep = torch.cat([t[:case["sinks"]], t[first:]])
            t, seen = keep, seen[:, keep]
        page, off = s["kv_indices"][s["indptr"][r] + t // PAGE].long(), t % PAGE
        k, v = (_values(s["codes"][page, i, :, off], cache).float() * s["scale"][page, i][..., None] for i in (0, 1))   # [n][h][d]
        q = s["q"][t0:t1].float().view(drafted, h, group, d).permute(1, 0, 2, 3).reshape(h, drafted * group, d)
        z = torch.matmul(q, k.permute(1, 2, 0)) * s["sm_scale"]
        z = torch.where(seen.repeat_interleave(group, 0), z, -torch.inf)
        m = z.amax(2, keepdim=True)
        p = torch.exp(z - m)
        total = p.sum(2, keepdim=True)
        out = torch.matmul(p, v.permute(1, 0, 2)) / total
        s["out"][t0:t1] = out.view(h, drafted, group, d).permute(1, 0, 2, 3).reshape(drafted, h * group, d).bfloat16()
        s["lse"][t0:t1] = (m + total.log()).view(h, drafted, group).permute(1, 0, 2).reshape(drafted, h * group)
    return {"out": s["out"], "lse": s["lse"]}


def _plain_commit(s):
    case = s["case"]
    cache, batch = case["cache"], case["batch"]
    k = torch.arange(case["accept"], device="cuda", dtype=torch.int32)
    live = k[None, :] < s["path_len"][:, None]
    to, frm = s["kv_len"][:, None] + k, s["kv_len"][:, None] + s["path"]
    row = s["kv_indptr"][:batch, None]
    page_of = lambda pos: s["kv_indices"][(row + pos // PAGE).long()].long()  # noqa: E731
    to_page, to_off, from_page, from_off = (x[live] for x in (page_of(to), (to % PAGE).long(), page_of(frm), (frm % PAGE).long()))
    for codes, scale in zip(s["codes"], s["scale"]):
        pages = scale.shape[0]
        rows = codes[from_page, :, :, from_off]                                          # [tokens][2][h][d]
        x = _values(rows, cache).float() * scale[from_page][..., None]
        moved = (from_page != to_page)[:, None, None]
        amax = torch.where(moved, x.abs().amax(3), 0.0)
        need = torch.zeros_like(scale).index_reduce(0, to_page, amax, "amax")
        need = need / torch.full_like(need, QMAX[cache])
        # a block's scale grows by the smallest power of two that holds the tokens from other pages
        m_need, e_need = torch.frexp(need)
        m_old, e_old = torch.frexp(scale)
        j = (e_need - e_old + (m_need > m_old).int()).clamp(min=0)
        j = torch.where((scale == 0) | (need == 0), torch.zeros_like(j), j)
        grown = torch.where(scale == 0, need, torch.ldexp(scale, j))
        first = torch.full((pages,), PAGE, device="cuda").scatter_reduce(0, to_page, to_off, "amin")
        touched = (first < PAGE).nonzero()[:, 0]
        older = torch.arange(PAGE, device="cuda") < first[touched][:, None]
        block = codes[touched]
        shrunk = _codes(torch.ldexp(_values(block, cache).float(), -j[touched][..., None, None]), cache).view(torch.uint8)
        codes[touched] = torch.where(older[:, None, None, :, None], shrunk, block)
        to_scale = grown[to_page][..., None]
        within = _codes(torch.ldexp(_values(rows, cache).float(), -j[to_page][..., None]), cache)
        across = _codes(torch.where(to_scale > 0, x / to_scale, x), cache)
        codes[to_page, :, :, to_off] = torch.where(moved[..., None], across.view(torch.uint8), within.view(torch.uint8))
        scale.copy_(grown)
    return {"codes": _values(s["all_codes"], cache), "scale": s["all_scale"]}


def _plain_copy(s, src, dst):
    for pool in s["pools"]:
        pool[dst.long()] = pool[src.long()]


def _plain_fork(s, parents, children):
    length = s["lens"][parents.long()]
    held = (length + PAGE - 1) // PAGE
    started = length % PAGE != 0
    # the k-th started page takes the k-th page from the free list's end
    rank = torch.cumsum(started.int(), 0)
    page = s["free_list"][(s["free_count"] - rank).clamp(min=0).long()]
    fits = ~started | (rank <= s["free_count"])
    s["status"].copy_(fits.int())
    slot = torch.arange(s["table"].shape[1], device="cuda")
    mine = fits[:, None] & (slot < held[:, None])
    rows = s["table"][parents.long()]
    last = started[:, None] & (slot == held[:, None] - 1)
    source = rows[last & mine]
    rows = torch.where(last, page[:, None], rows)
    s["table"][children.long()] = torch.where(mine, rows, s["table"][children.long()])
    s["held"][children.long()] = torch.where(fits, held, s["held"][children.long()])
    s["lens"][children.long()] = torch.where(fits, length, s["lens"][children.long()])
    s["refs"].index_add_(0, rows[mine].long(), torch.ones_like(rows[mine]))
    s["free_count"] -= (fits & started).sum().int()
    _plain_copy(s, source, page[fits & started])


def _plain_grow(s, rows, tokens, status):
    need = ((tokens + PAGE - 1) // PAGE - s["held"][rows.long()]).clamp(min=0)
    total = torch.cumsum(need, 0)
    fits = (need == 0) | (total <= s["free_count"])
    status.copy_(fits.int())
    need = torch.where(fits, need, 0)
    slot = torch.arange(s["table"].shape[1], device="cuda")
    have = s["held"][rows.long()]
    taken = (slot >= have[:, None]) & (slot < (have + need)[:, None])
    order = (total - need)[:, None] + slot - have[:, None]
    page = s["free_list"][(s["free_count"] - 1 - order).clamp(0, s["refs"].shape[0] - 1).long()]
    s["table"][rows.long()] = torch.where(taken, page, s["table"][rows.long()])
    s["refs"][page[taken].long()] = 1
    s["held"][rows.long()] = have + need
    s["free_count"] -= need.sum().int()


def _plain_free(s, rows):
    slot = torch.arange(s["table"].shape[1], device="cuda")
    pages = s["table"][rows.long()][slot < s["held"][rows.long()][:, None]].long()
    before = s["refs"].clone()
    s["refs"].index_add_(0, pages, torch.full_like(pages, -1, dtype=torch.int32))
    # the highest page first, so that the lowest one is taken next
    gone = ((before > 0) & (s["refs"] == 0)).nonzero()[:, 0].flip(0).int()
    s["free_list"][s["free_count"].long() + torch.arange(gone.shape[0], device="cuda")] = gone
    s["free_count"] += gone.shape[0]
    s["held"][rows.long()] = 0
    s["lens"][rows.long()] = 0


def _plain_compact(s):
    pages = s["refs"].shape[0]
    used = s["refs"] > 0
    live = int(used.sum())
    source = live + used[live:].nonzero()[:, 0]
    target = (~used[:live]).nonzero()[:, 0]
    _plain_copy(s, source, target)
    name = torch.arange(pages, dtype=torch.int32, device="cuda")
    name[source] = target.int()
    slot = torch.arange(s["table"].shape[1], device="cuda")
    s["table"].copy_(torch.where(slot < s["held"][:, None], name[s["table"].clamp(min=0).long()], s["table"]))
    s["refs"][target] = s["refs"][source]
    s["refs"][live:] = 0
    s["free_list"][:pages - live] = torch.arange(pages - 1, live - 1, -1, dtype=torch.int32, device="cuda")
    s["free_count"].fill_(pages - live)


def _plain_pages(s):
    kind = s["case"]["kind"]
    if kind == "copy":
        _plain_copy(s, s["src"], s["dst"])
    elif kind == "fork":
        _plain_fork(s, s["parents"], s["children"])
        _plain_grow(s, s["children"], s["tokens"], s["status2"])
        _plain_free(s, s["children"])
    else:
        for rows, want in zip(s["halves"], s["wants"]):
            _plain_free(s, rows)
            _plain_compact(s)
            _plain_grow(s, rows, want, s["status"])
    return _pages_outputs(s)


def _pages_outputs(s):
    names = () if s["case"]["kind"] == "copy" else ("table", "held", "lens", "refs", "free_count", "status", "status2")
    out = {name: s[name] for name in names}
    out["pools"] = s["buffers"]
    return out


# ------------------------------------------------------------------------------------------------- one pass
def run(s):
    case = s["case"]
    if not own:
        return {"tree": _plain_tree, "commit": _plain_commit, "pages": _plain_pages}[case["op"]](s)
    import quantized_kv_paged_gb300 as q
    if case["op"] == "tree":
        q.gqa_tree_run(s["plan"], s["q"], s["codes"], s["scale"], s["kv_indices"], s["mask"], s["sm_scale"], s["out"], s["lse"], s["workspace"])
        return {"out": s["out"], "lse": s["lse"]}
    if case["op"] == "commit":
        q.gqa_tree_commit(s["codes"], s["scale"], _CACHE(q)[case["cache"]], s["kv_len"], s["kv_indptr"], s["kv_indices"], s["path"], s["path_len"])
        return {"codes": _values(s["all_codes"], case["cache"]), "scale": s["all_scale"]}
    if case["kind"] == "copy":
        q.kv_pages_copy(s["pools"], s["src"], s["dst"])
        return _pages_outputs(s)
    tables = (s["table"], s["held"], s["lens"], s["refs"], s["free_list"], s["free_count"])
    if case["kind"] == "fork":
        q.kv_pages_fork(s["pools"], *tables, s["parents"], s["children"], s["status"], s["workspace"])
        q.kv_pages_grow(*tables, s["children"], s["tokens"], s["status2"], s["workspace"])
        q.kv_pages_free(*tables, s["children"], s["workspace"])
    else:
        for rows, want in zip(s["halves"], s["wants"]):
            q.kv_pages_free(*tables, rows, s["workspace"])
            q.kv_pages_compact(s["pools"], *tables, s["workspace"])
            q.kv_pages_grow(*tables, rows, want, s["status"], s["workspace"])
    return _pages_outputs(s)


def work(case):
    if case["op"] == "tree":
        h, d, heads = case["kv_heads"], case["dim"], case["heads"]
        same = _host_gen(0)
        cached = _spread(case["lo"], case["hi"], case["batch"], same).tolist()
        drafted = _spread(case["tlo"], case["thi"], case["batch"], same).tolist()
        if case["window"]:
            cached = [min(n, case["window"] + min(case["sinks"], max(0, n - case["window"]))) for n in cached]
        tokens = sum(a + b for a, b in zip(cached, drafted))
        # a drafted token sees the cached ones and at least itself
        rows = sum(b * (a + 1) for a, b in zip(cached, drafted))
        return {"bytes": tokens * (2 * h * d + 8 * h / PAGE) + sum(drafted) * heads * (4 * d + 4), "flops": rows * heads * 4 * d}
    if case["op"] == "commit":
        # of a path's mean length; what stays in its place need not be moved, but that is rare
        tokens = case["batch"] * (1 + case["accept"]) / 2 * case["layers"]
        return {"bytes": tokens * 2 * case["kv_heads"] * case["dim"] * 2, "flops": tokens * 2 * case["kv_heads"] * case["dim"] * 2}
    page = sum(POOLS[case["pool"]]) * case["layers"]
    if case["kind"] == "copy":
        moved, entries = case["n"], case["n"]
    elif case["kind"] == "fork":
        moved, entries = case["n"], 3 * case["n"] * case["held"] / 2
    else:
        # both halves move once, from above the other one to below it
        moved, entries = case["rows"] * (1 + case["held"]) / 2, 4 * case["rows"] * case["held"]
    return {"bytes": 2 * moved * page + 8 * entries, "flops": entries}


# ------------------------------------------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    return {"tree": _exact_tree, "commit": _exact_commit, "pages": _exact_pages}[case["op"]](case, prepare(case, seed))


def _exact_tree(case, s):
    h, d, heads = case["kv_heads"], case["dim"], case["heads"]
    group = heads // h
    out = torch.empty(s["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(s["lse"].shape, dtype=torch.float64, device="cuda")
    ids = s["kv_indices"].tolist()
    mask = None if s["mask"] is None else s["mask"].tolist()
    for r, n in enumerate(s["lens"]):
        t0, t1, cached = s["tok"][r], s["tok"][r + 1], s["cached"][r]
        pages = ids[s["indptr"][r]:s["indptr"][r + 1]]
        # drafted tokens that each one sees, from the mask's bits
        paths = []
        for i in range(t1 - t0):
            bits = (1 << (i + 1)) - 1 if mask is None else sum((w & 0xffffffff) << 32 * j for j, w in enumerate(mask[t0 + i]))
            paths.append([j for j in range(t1 - t0) if bits >> j & 1])
        used = torch.tensor(pages, device="cuda")
        for j in range(h):
            rows = slice(j * group, (j + 1) * group)
            if case["window"]:
                low = max(0, cached + 1 - case["window"])
                part = sorted(set(range(min(case["sinks"], cached) // PAGE + 1)) | set(range(low // PAGE, len(pages))))
                part = [p for p in part if p < len(pages)]
            else:
                part = list(range(len(pages)))
            at = torch.tensor(part, device="cuda")
            pos = (at[:, None] * PAGE + torch.arange(PAGE, device="cuda")).reshape(-1)
            block = s["codes"][used[at], :, j]
            k, v = (_values(block[:, i].contiguous(), case["cache"]).double() * s["scale"][used[at], i, j].double()[:, None, None] for i in (0, 1))
            k, v = k.reshape(-1, d), v.reshape(-1, d)
            for c0 in range(0, t1 - t0, 16):
                c1 = min(c0 + 16, t1 - t0)
                seen = torch.zeros((c1 - c0, pos.shape[0]), dtype=torch.bool, device="cuda")
                for i in range(c0, c1):
                    old = pos < cached
                    if case["window"]:
                        old &= (pos < case["sinks"]) | (pos > cached + len(paths[i]) - 1 - case["window"])
                    seen[i - c0] = old | torch.isin(pos, torch.tensor([cached + x for x in paths[i]], device="cuda"))
                z = torch.einsum("tgd,nd->tgn", s["q"][t0 + c0:t0 + c1, rows].double(), k) * s["sm_scale"]
                z = z.masked_fill(~seen[:, None], -math.inf)
                lse[t0 + c0:t0 + c1, rows] = torch.logsumexp(z, 2)
                out[t0 + c0:t0 + c1, rows] = torch.softmax(z, 2) @ v
    return {"out": out, "lse": lse}


def _exact_commit(case, s):
    cache = case["cache"]
    qmax = QMAX[cache]
    cached, indptr, ids = s["kv_len"].tolist(), s["kv_indptr"].tolist(), s["kv_indices"].tolist()
    paths = [p[:n] for p, n in zip(s["path"].tolist(), s["path_len"].tolist())]
    all_codes, all_scale = _values(s["all_codes"], cache).double(), s["all_scale"].double()
    for codes, scale in zip(all_codes, all_scale):
        for r, path in enumerate(paths):
            where = lambda pos: (ids[indptr[r] + pos // PAGE], pos % PAGE)  # noqa: E731,B023
            moves = [(where(cached[r] + i), where(cached[r] + p)) for i, p in enumerate(path)]
            values = [codes[f[0], :, :, f[1]] * scale[f[0]][..., None] for _, f in moves]
            for page in sorted({to[0] for to, _ in moves}):
                mine = [(to[1], f[0] != page, x) for (to, f), x in zip(moves, values) if to[0] == page]
                new = [x.abs().amax(2) / qmax for _, away, x in mine if away]
                if new:
                    need, old = torch.stack(new).amax(0), scale[page].clone()
                    grown = torch.where(need > 0, old * torch.exp2(torch.ceil(torch.log2(need / old)).clamp(min=0)), old)
                    first = min(o for o, _, _ in mine)
                    codes[page, :, :, :first] *= (old / grown)[..., None, None]
                    scale[page] = grown
                for o, _, x in mine:
                    codes[page, :, :, o] = x / scale[page][..., None]
    # INT8 codes are whole numbers of the FP32 arithmetic, which the quotients above only come near
    return {"codes": all_codes if cache == "e4m3" else None, "scale": all_scale}


def _exact_pages(case, s):
    """The bookkeeping with lists and sets, one request after the other."""
    buffers = [b.clone() for b in s["buffers"]]
    pools = [layer for b in buffers for layer in b]

    def copy(pairs):
        if pairs:
            src, dst = (torch.tensor(x, device="cuda") for x in zip(*pairs))
            for p in pools:
                p[dst] = p[src]

    if case["kind"] == "copy":
        copy(list(zip(s["src"].tolist(), s["dst"].tolist())))
        return {"pools": buffers}
    table, held, lens, refs = (s[x].tolist() for x in ("table", "held", "lens", "refs"))
    free = s["free_list"].tolist()[:int(s["free_count"])]
    status, status2 = s["status"].tolist(), s["status2"].tolist()

    def release(rows):
        gone = []
        for r in rows:
            for page in table[r][:held[r]]:
                refs[page] -= 1
                if refs[page] == 0:
                    gone.append(page)
            held[r] = lens[r] = 0
        free.extend(sorted(gone, reverse=True))

    def grow(rows, tokens, state):
        for i, (r, n) in enumerate(zip(rows, tokens)):
            state[i] = 1                      # the cases' pools are large enough
            while held[r] * PAGE < n:
                page = free.pop()
                table[r][held[r]] = page
                refs[page] = 1
                held[r] += 1

    if case["kind"] == "fork":
        pairs = []
        for i, (p, c) in enumerate(zip(s["parents"].tolist(), s["children"].tolist())):
            lens[c], status[i] = lens[p], 1
            held[c] = -(-lens[p] // PAGE)
            for j in range(held[c]):
                page = table[p][j]
                if (j + 1) * PAGE > lens[p]:
                    pairs.append((page, free[-1]))
                    page = free.pop()
                table[c][j] = page
                refs[page] += 1
        copy(pairs)
        grow(s["children"].tolist(), s["tokens"].tolist(), status2)
        release(s["children"].tolist())
    else:
        for half, want in zip(s["halves"], s["wants"]):
            release(half.tolist())
            used = [p for p, x in enumerate(refs) if x > 0]
            holes = [p for p in range(len(used)) if refs[p] == 0]
            names = dict(zip([p for p in used if p >= len(used)], holes))
            copy(list(names.items()))
            table = [[names.get(p, p) if j < held[r] else p for j, p in enumerate(row)] for r, row in enumerate(table)]
            for old, new in names.items():
                refs[new], refs[old] = refs[old], 0
            free[:] = range(len(refs) - 1, len(used) - 1, -1)
            grow(half.tolist(), want.tolist(), status)
    back = lambda x: torch.tensor(x, dtype=torch.int64, device="cuda")  # noqa: E731
    return {"table": back(table), "held": back(held), "lens": back(lens), "refs": back(refs), "free_count": back([len(free)]), "status": back(status),
            "status2": back(status2), "pools": buffers}
