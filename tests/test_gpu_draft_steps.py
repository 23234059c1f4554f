"""Steps of speculative decoding over a head pool, every call as a serving loop makes it: pages are reserved, drafted tokens
appended in every layer, attended as a tree, the accepted ones committed; requests are forked and freed between the steps,
the pool is compacted, and a decode reads what is left."""
import numpy as np
import pytest
import torch

import quantized_kv_paged_gb300 as q
from tests import heads_ref as R
from tests import tree_ref as T

pytestmark = pytest.mark.gpu

LAYERS, ROWS, ROW_PAGES, PAGES = 3, 6, 9, 40


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()


class Steps:
    """What the host decides in advance: who drafts how many tokens in which tree, which paths are accepted, and when
    requests begin, fork and end."""

    def __init__(self, seed, heads, kv_heads, dim, cache, steps=5):
        rng = np.random.default_rng(seed)
        self.dims, self.cache, self.steps = (heads, kv_heads, dim), cache, []
        lens = np.array([0, 0, 0, 0, 0, 0])
        lens[:4] = [61, 128, 5, 200]
        self.first = lens.copy()
        indptr = (np.arange(ROWS + 1) * ROW_PAGES).astype(np.int32)
        self.indptr, self.indptr_host = i32(indptr), indptr
        gen = torch.Generator(device="cuda").manual_seed(seed)
        for s in range(steps):
            alive = [0, 2, 3, 4, 5] if s > 2 else [0, 1, 2, 3]
            drafted = np.zeros(ROWS, int)
            drafted[alive] = rng.integers(1, 40, len(alive))
            tok = np.concatenate([[0], np.cumsum(drafted)])
            paths = T.random_paths(rng, drafted)
            n = int(tok[-1])
            accepted, count = np.zeros((ROWS, 8), int), np.zeros(ROWS, int)
            for r in alive:
                best = max((paths[i] for i in range(tok[r], tok[r + 1])), key=len)[:int(rng.integers(0, 9))]
                accepted[r, :len(best)], count[r] = best, len(best)
            depth = np.array([len(p) for p in paths])
            pos = np.concatenate([lens[r] + depth[tok[r]:tok[r + 1]] - 1 for r in range(ROWS)])
            full = (lens + drafted).astype(np.int32)
            args = (indptr, full, tok.astype(np.int32), heads, kv_heads, dim, cache)
            ws = torch.full((max(256, q.gqa_tree_plan(*args).workspace_bytes),), 0x5A, dtype=torch.uint8, device="cuda")
            mask = T.masks_of(paths, 2)
            self.steps.append(dict(
                alive=i32(alive), want=i32(full[alive]), host=(lens.copy(), full, tok, paths, accepted, count), plan=q.gqa_tree_plan(*args, workspace=ws),
                ws=ws, tok=i32(tok), mask=i32(mask.view(np.int32)), pos=torch.from_numpy(pos.astype(np.int64)).cuda(), path=i32(accepted), count=i32(count),
                k=torch.randn((LAYERS, n, kv_heads, dim), generator=gen, device="cuda").bfloat16(), v=torch.randn((LAYERS, n, kv_heads, dim), generator=gen, device="cuda").bfloat16(),
                q=torch.randn((LAYERS, n, heads, dim), generator=gen, device="cuda").bfloat16()))
            lens = lens + count
            if s == 2:
                lens[4], lens[5], lens[1] = lens[0], lens[3], 0
        self.lens = lens
        self.cs = torch.from_numpy(R.table(400, dim)).cuda()
        args = (indptr, lens.astype(np.int32), heads, kv_heads, dim, cache)
        self.dws = torch.empty(q.gqa_decode_plan(*args).workspace_bytes, dtype=torch.uint8, device="cuda")
        self.dplan = q.gqa_decode_plan(*args, workspace=self.dws)
        self.query = torch.randn((ROWS, heads, dim), generator=gen, device="cuda").bfloat16()
        self.pool0 = torch.randint(0, 0x70, (LAYERS, PAGES, 2, kv_heads, 64, dim), generator=gen, device="cuda", dtype=torch.uint8)

    def buffers(self):
        heads, kv_heads, dim = self.dims
        b = dict(codes=[torch.empty_like(self.pool0[i]) for i in range(LAYERS)], scale=[torch.empty((PAGES, 2, kv_heads), device="cuda") for _ in range(LAYERS)],
                 table=torch.empty((ROWS, ROW_PAGES), dtype=torch.int32, device="cuda"), held=i32(np.zeros(ROWS)), lens=i32(np.zeros(ROWS)),
                 refs=i32(np.zeros(PAGES)), free=i32(np.zeros(PAGES)), count=i32([0]), klen=i32(np.zeros(ROWS)),
                 ws=torch.zeros(q.kv_pages_workspace(PAGES, ROWS, ROWS), dtype=torch.uint8, device="cuda"), status=i32(np.full(ROWS, 9)),
                 out=[[torch.zeros_like(s["q"][0]) for _ in range(LAYERS)] for s in self.steps], q=[torch.zeros_like(s["q"][0]) for s in self.steps],
                 lse=[[torch.zeros(s["q"].shape[1:3], device="cuda") for _ in range(LAYERS)] for s in self.steps],
                 done=torch.zeros_like(self.query), done_lse=torch.zeros(self.query.shape[:2], device="cuda"),
                 all=i32(np.arange(ROWS)), begin=i32(self.first), pairs=(i32([0, 3]), i32([4, 5])), ended=i32([1]))
        return b

    def run(self, b, after=lambda *a: None):
        """`after` is called behind every call."""
        state = [b[x] for x in ("table", "held", "lens", "refs", "free", "count")]
        flat = b["table"].view(-1)
        for i in range(LAYERS):
            b["codes"][i].copy_(self.pool0[i])
            b["scale"][i].fill_(0.01)
        for x in ("held", "lens", "refs"):
            b[x].zero_()
        b["free"].copy_(torch.arange(PAGES, device="cuda", dtype=torch.int32))
        b["count"].fill_(PAGES)
        b["table"].fill_(-1)
        q.kv_pages_grow(*state, b["all"], b["begin"], b["status"], b["ws"])
        b["lens"].copy_(b["begin"])
        pools = b["codes"] + b["scale"]
        for i, s in enumerate(self.steps):
            q.kv_pages_grow(*state, s["alive"], s["want"], b["status"][:len(s["alive"])], b["ws"])
            after("grow", i)
            for l in range(LAYERS):
                q.gqa_append_rope(s["k"][l], s["v"][l], s["tok"], b["lens"], self.indptr, flat, self.cs, q.ROPE_HALVES, b["codes"][l], b["scale"][l],
                                  self.cache, q=s["q"][l], q_out=b["q"][i], positions=s["pos"])
                after("append", i, l)
                q.gqa_tree_run(s["plan"], b["q"][i], b["codes"][l], b["scale"][l], flat, s["mask"], 0.1, b["out"][i][l], b["lse"][i][l], s["ws"])
                after("tree", i, l)
            q.gqa_tree_commit(b["codes"], b["scale"], self.cache, b["lens"], self.indptr, flat, s["path"], s["count"])
            after("commit", i)
            b["lens"].add_(s["count"])
            if i == 2:
                q.kv_pages_fork(pools, *state, *b["pairs"], b["status"][:2], b["ws"])
                after("fork", i)
                q.kv_pages_free(*state, b["ended"], b["ws"])
                after("free", i)
        q.kv_pages_compact(pools, *state, b["ws"])
        after("compact", 0)
        q.gqa_decode_run(self.dplan, self.query, b["codes"][1], b["scale"][1], flat, 0.1, b["done"], b["done_lse"], self.dws)
        after("decode", 0)

    def bits(self, b):
        flat = b["codes"] + b["scale"] + [b[x] for x in ("table", "held", "lens", "refs", "free", "count", "done", "done_lse")]
        flat += [t for s in b["out"] for t in s] + [t for s in b["lse"] for t in s]
        return [t.view(torch.uint8).cpu() for t in flat]


def host(b):
    return [(c.cpu().numpy().copy(), s.cpu().numpy().copy()) for c, s in zip(b["codes"], b["scale"])]


@pytest.mark.parametrize("heads,kv_heads,dim,cache", [(8, 2, 128, q.CACHE_E4M3), (4, 4, 64, q.CACHE_INT8), (6, 1, 256, q.CACHE_E4M3)])
def test_every_step_and_all_of_them_unsynchronised_and_captured(qkvp, heads, kv_heads, dim, cache):
    w = Steps(heads * dim, heads, kv_heads, dim, cache)
    b, before = w.buffers(), {}

    def look(call, i, l=0):
        torch.cuda.synchronize()
        s = w.steps[i]
        lens, full, tok, paths, path, count = s["host"]
        ids = b["table"].cpu().numpy().reshape(-1)
        if call == "grow":
            assert (b["status"][:len(s["alive"])] == 1).all()
        elif call == "tree":
            codes, scale = b["codes"][l].cpu().numpy(), b["scale"][l].cpu().numpy()
            ref = T.attend(R.bf16_to_f32(b["q"][i].cpu()), codes, scale, cache, w.indptr_host, ids, full, tok, paths, 0.1)
            R.check_attend(b["out"][i][l], b["lse"][i][l], ref, int(full.max()) + 64, dim)
            before[l] = codes.copy(), scale.copy()
        elif call == "commit":
            for (c, x), (gc, gs) in zip(before.values(), host(b)):
                T.commit(c, x, cache, lens, w.indptr_host, ids, path, count)
                assert np.array_equal(gc, c) and np.array_equal(gs.view(np.int32), x.view(np.int32))
        elif call == "fork":
            assert (b["status"][:2] == 1).all()
        elif call == "decode":
            assert b["lens"].tolist() == w.lens.tolist()
            ref = R.attend(R.bf16_to_f32(w.query.cpu()), b["codes"][1].cpu().numpy(), b["scale"][1].cpu().numpy(), cache, w.indptr_host, ids, w.lens, 0.1)
            R.check_attend(b["done"], b["done_lse"], ref, int(w.lens.max()) + 64, dim)
    w.run(b, look)
    want = w.bits(b)
    for _ in range(3):
        w.run(b)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(want, w.bits(b)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w.run(b)
    for _ in range(3):
        for t in b["done"], b["done_lse"], *b["out"][0]:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(want, w.bits(b)))
