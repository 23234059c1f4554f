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
