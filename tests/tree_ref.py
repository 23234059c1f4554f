"""Plain restatements of the tree attention and of committing an accepted path, for the tests: numpy loops over requests,
heads and tokens. The attention is in 64 bits; the commit follows the header's FP32 arithmetic, so its bytes are compared
exactly."""
from __future__ import annotations

import numpy as np
import torch

from tests import heads_ref as R

PAGE = 64


def masks_of(paths, words):
    """uint32 [n][words] from each drafted token's list of visible drafted tokens."""
    out = np.zeros((len(paths), words), np.uint32)
    for i, p in enumerate(paths):
        for j in p:
            out[i, j // 32] |= np.uint32(1 << (j % 32))
    return out


def random_paths(rng, drafted, chain=False, empty=0.0):
    """Per request, each drafted token's visible drafted tokens: its ancestors and itself in a random tree."""
    paths = []
    for n in drafted:
        mine = []
        for i in range(n):
            parent = i - 1 if chain else (-1 if i == 0 or rng.random() < 0.15 else int(rng.integers(max(0, i - 6), i)))
            mine.append((mine[parent] if parent >= 0 else []) + [i])
        if empty:
            mine = [[] if rng.random() < empty else m for m in mine]
        paths += mine
    return paths


def attend(q, codes, scale, cache, kv_indptr, kv_indices, kv_len, tok, paths, sm_scale, window=0, sinks=0):
    """q float32 [n, H, D], paths one list of visible drafted tokens for each. Returns what heads_ref.attend returns, a row
    for each drafted token."""
    n, heads, dim = q.shape
    pages, kv_heads = codes.shape[0], codes.shape[2]
    group = heads // kv_heads
    out, absout = np.zeros((n, heads, dim)), np.zeros((n, heads, dim))
    lse, dot, vmax = np.full((n, heads), -np.inf), np.zeros((n, heads)), np.zeros((n, heads))
    ids = np.asarray(kv_indices)
    for r in range(len(kv_len)):
        drafted = int(tok[r + 1]) - int(tok[r])
        cached = int(kv_len[r]) - drafted
        for j in range(drafted):
            i = int(tok[r]) + j
            t = np.arange(cached)
            if window:
                t = t[(t >= cached + len(paths[i]) - window) | (t < sinks)]
            t = np.concatenate([t, cached + np.asarray(paths[i], np.int64)])
            page = ids[int(kv_indptr[r]) + t // PAGE].astype(np.int64) if t.size else t
            ok = (page >= 0) & (page < pages)
            t, page = t[ok], page[ok]
            if not t.size:
                continue
            for h in range(kv_heads):
                k, v = (R.decode(codes[page, x, h, t % PAGE], cache) * scale[page, x, h].astype(np.float64)[:, None] for x in (0, 1))
                sl = slice(h * group, (h + 1) * group)
                qq = q[i, sl].astype(np.float64)
                z = qq @ k.T * sm_scale
                m = z.max(1, keepdims=True)
                p = np.exp(z - m)
                total = p.sum(1, keepdims=True)
                out[i, sl], absout[i, sl] = p @ v / total, p @ np.abs(v) / total
                lse[i, sl] = (m + np.log(total))[:, 0]
                dot[i, sl] = (np.abs(qq) @ np.abs(k).T).max(1) * abs(sm_scale)
                vmax[i, sl] = np.abs(v).max()
    return out, lse, absout, dot, vmax


class Batch:
    """A batch of drafted tokens over a shuffled head pool, on the host and on the GPU."""

    def __init__(self, seed, cached, drafted, heads, kv_heads, dim, cache, chain=False, empty=0.0, extra_words=0, spare=2):
        rng = np.random.default_rng(seed)
        self.cached, self.drafted = list(cached), list(drafted)
        self.lens = np.array([a + b for a, b in zip(cached, drafted)], np.int32)
        self.tok = np.concatenate([[0], np.cumsum(drafted)]).astype(np.int32)
        held = [(int(x) + PAGE - 1) // PAGE + int(rng.integers(0, 2)) for x in self.lens]
        self.indptr = np.concatenate([[0], np.cumsum(held)]).astype(np.int32)
        self.pages = int(self.indptr[-1]) + spare
        self.ids = rng.permutation(self.pages)[:int(self.indptr[-1])].astype(np.int32)
        self.paths = random_paths(rng, drafted, chain, empty)
        self.words = (max(list(drafted) + [1]) + 31) // 32 + extra_words
        self.mask = masks_of(self.paths, self.words)
        self.dims, self.cache = (heads, kv_heads, dim), cache
        x = rng.standard_normal((self.pages, 2, kv_heads, PAGE, dim)).astype(np.float32)
        x[:, 0, :, :, ::29] *= 5
        self.scale = (np.abs(x).max((3, 4)) / R.QMAX[cache]).astype(np.float32)
        self.codes = R.encode(x / self.scale[..., None, None], cache).reshape(x.shape)
        self.q = torch.from_numpy(rng.standard_normal((int(self.tok[-1]), heads, dim)).astype(np.float32)).bfloat16()

    def plan(self, q, window=0, sinks=0, **kw):
        args = (self.indptr, self.lens, self.tok, *self.dims, self.cache)
        size = q.gqa_tree_plan(*args, window=window, sinks=sinks, **kw).workspace_bytes
        ws = torch.full((max(size, 256),), 0x7F, dtype=torch.uint8, device="cuda")
        return q.gqa_tree_plan(*args, window=window, sinks=sinks, workspace=ws, **kw), ws

    def run(self, q, sm_scale, window=0, sinks=0, chain=False, lse=True, **kw):
        plan, ws = self.plan(q, window, sinks, **kw)
        n, (heads, _, dim) = int(self.tok[-1]), self.dims
        out = torch.full((n, heads, dim), float("nan"), dtype=torch.bfloat16, device="cuda")
        le = torch.full((n, heads), float("nan"), device="cuda") if lse else None
        mask = None if chain else torch.from_numpy(self.mask.view(np.int32)).cuda()
        q.gqa_tree_run(plan, self.q.cuda(), torch.from_numpy(self.codes).cuda(), torch.from_numpy(self.scale).cuda(),
                       torch.from_numpy(self.ids).cuda(), mask, sm_scale, out, le, ws)
        torch.cuda.synchronize()
        assert int(ws[plan.status_offset:plan.status_offset + 4].view(torch.int32)[0]) == 0
        return out, le, plan

    def reference(self, sm_scale, window=0, sinks=0):
        return attend(R.bf16_to_f32(self.q), self.codes, self.scale, self.cache, self.indptr, self.ids, self.lens, self.tok, self.paths, sm_scale,
                      window, sinks)


def commit(codes, scale, cache, kv_len, kv_indptr, kv_indices, path, path_len):
    """codes [pages, 2, Hkv, 64, D] uint8 and scale [pages, 2, Hkv] float32 are changed in place."""
    pages, heads = codes.shape[0], codes.shape[2]
    for r in range(len(kv_len)):
        n, held = int(path_len[r]), int(kv_len[r])
        if not 0 < n <= path.shape[1]:
            continue
        p = path[r, :n].astype(np.int64)
        pos = np.stack([held + np.arange(n), held + p])
        entry = int(kv_indptr[r]) + pos // PAGE
        if p[0] < 0 or (np.diff(p) <= 0).any() or held < 0 or entry.max() >= min(int(kv_indptr[r + 1]), len(kv_indices)):
            continue
        page = np.asarray(kv_indices)[entry].astype(np.int64)
        if ((page < 0) | (page >= pages)).any():
            continue
        rows, from_scale = codes[page[1], :, :, pos[1] % PAGE].copy(), scale[page[1]].copy()
        away = page[0] != page[1]
        for to in dict.fromkeys(page[0].tolist()):
            mine = np.nonzero(page[0] == to)[0]
            first = int(pos[0, mine[0]] % PAGE)
            for kind in range(2):
                for h in range(heads):
                    with np.errstate(all="ignore"):
                        x = R.decode(rows[mine, kind, h], cache).astype(np.float32) * from_scale[mine, kind, h][:, None]
                    fin = np.abs(x[away[mine]])
                    fin = fin[np.isfinite(fin)]
                    need = np.float32(fin.max() if fin.size else 0.0) / R.QMAX[cache]
                    old, block = scale[to, kind, h], codes[to, kind, h]
                    new, shrink = old, np.float32(1)
                    if old == 0:
                        new = need
                    while new < need:
                        new, shrink = new * np.float32(2), shrink * np.float32(0.5)
                    scale[to, kind, h] = new
                    if shrink != 1:
                        block[:first] = R.encode(R.decode(block[:first], cache).astype(np.float32) * shrink, cache)
                    for i, k in enumerate(mine):
                        if away[k]:
                            with np.errstate(all="ignore"):
                                code = R.encode(x[i] / new if new > 0 else x[i], cache)
                        else:
                            code = rows[k, kind, h]
                            if shrink != 1:
                                code = R.encode(R.decode(code, cache).astype(np.float32) * shrink, cache)
                        block[int(pos[0, k] % PAGE)] = code


class Pages:
    """Page tables, counts and a free list on the host, with the calls' semantics one entry after the other."""

    def __init__(self, rng, rows, row_pages, pages, held, pools):
        ids = rng.permutation(pages)
        self.table = rng.integers(-5, pages + 5, (rows, row_pages)).astype(np.int32)
        self.held, self.lens = np.zeros(rows, np.int32), np.zeros(rows, np.int32)
        self.refs = np.zeros(pages, np.int32)
        at = 0
        for r, n in enumerate(held):
            self.table[r, :n] = ids[at:at + n]
            self.refs[ids[at:at + n]] = 1
            self.held[r] = n
            self.lens[r] = int(rng.integers(max(0, 64 * (n - 2) + 1), 64 * n + 1)) if n else 0
            at += n
        self.free = ids[at:].astype(np.int32).tolist()
        self.pools = pools

    def state(self):
        free = np.full(len(self.refs), -7, np.int32)
        free[:len(self.free)] = self.free
        return [torch.from_numpy(x.copy()).cuda() for x in (self.table, self.held, self.lens, self.refs, free, np.array([len(self.free)], np.int32))]

    def same(self, state, pools):
        table, held, lens, refs, free, count = (x.cpu().numpy() for x in state)
        assert held.tolist() == self.held.tolist() and lens.tolist() == self.lens.tolist() and refs.tolist() == self.refs.tolist()
        assert int(count[0]) == len(self.free) and free[:len(self.free)].tolist() == [int(x) for x in self.free]
        assert np.array_equal(table, self.table)
        for a, b in zip(pools, self.pools):
            assert np.array_equal(a.cpu().numpy(), b)

    def copy(self, pairs):
        n = len(self.refs)
        for p in self.pools:
            old = p.copy()
            for s, d in pairs:
                if 0 <= s < n and 0 <= d < n:
                    p[d] = old[s]

    def fork(self, parents, children):
        rows, row_pages = self.table.shape
        held, lens, table, named, status, pairs, short, wanted = self.held.copy(), self.lens.copy(), self.table.copy(), set(), [], [], len(self.free), 0
        for p, c in zip(parents, children):
            ok = 0 <= p < rows and 0 <= c < rows and p != c and c not in named and held[c] == 0
            named.add(c)
            n = -(-int(lens[p]) // 64) if ok else 0
            ok = ok and lens[p] >= 0 and n <= min(held[p], row_pages)
            need = int(ok and lens[p] % 64 != 0)
            wanted += need
            ok = ok and (wanted <= short)
            status.append(int(ok))
            if not ok:
                continue
            for j in range(n):
                page = int(table[p, j])
                if need and j == n - 1:
                    pairs.append((page, self.free[-1]))
                    page = int(self.free.pop())
                    self.refs[page] = 1
                else:
                    self.refs[page] += 1
                self.table[c, j] = page
            self.held[c], self.lens[c] = n, lens[p]
        self.copy(pairs)
        return status

    def grow(self, rows, tokens):
        named, status, short, wanted = set(), [], len(self.free), 0
        for r, t in zip(rows, tokens):
            ok = 0 <= r < len(self.held) and r not in named and 0 <= t <= 64 * self.table.shape[1]
            named.add(r)
            need = max(0, -(-t // 64) - int(self.held[r])) if ok else 0
            wanted += need
            ok = ok and (need == 0 or wanted <= short)
            status.append(int(ok))
            for _ in range(need if ok else 0):
                page = int(self.free.pop())
                self.table[r, self.held[r]] = page
                self.held[r] += 1
                self.refs[page] = 1
        return status

    def release(self, rows):
        gone = []
        for r in rows:
            if not 0 <= r < len(self.held):
                continue
            for page in self.table[r, :self.held[r]]:
                self.refs[page] -= 1
                if self.refs[page] == 0:
                    gone.append(int(page))
            self.held[r] = self.lens[r] = 0
        self.free += sorted(gone, reverse=True)

    def compact(self):
        used = np.nonzero(self.refs > 0)[0]
        live = len(used)
        src, dst = used[used >= live], np.setdiff1d(np.arange(live), used)
        self.copy(list(zip(src.tolist(), dst.tolist())))
        names = dict(zip(src.tolist(), dst.tolist()))
        for r in range(len(self.held)):
            for j in range(self.held[r]):
                self.table[r, j] = names.get(int(self.table[r, j]), self.table[r, j])
        self.refs[dst] = self.refs[src]
        self.refs[src] = 0
        self.free = list(range(len(self.refs) - 1, live - 1, -1))
