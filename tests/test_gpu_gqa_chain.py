"""Appends and decodes that overlap their launches: what one writes the next reads."""
import numpy as np
import pytest
import torch

import quantized_kv_paged_gb300 as q
from tests import heads_ref as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("batch,heads,kv_heads,dim", [(3, 16, 2, 128), (40, 8, 8, 64)])
def test_steps_back_to_back(qkvp, batch, heads, kv_heads, dim):
    """Steps of one append and two decodes, q_out and the tables reused, with nothing between the launches: the bits of
    the same steps with a synchronisation behind every call."""
    steps, per = 60, 4
    gen = torch.Generator(device="cuda").manual_seed(batch)
    cs = torch.from_numpy(R.table(steps + 200, dim)).cuda()
    held = torch.randint(0, 130, (batch,), generator=gen, device="cuda", dtype=torch.int32)
    lens = [(held.cpu().numpy() + i + 1).astype(np.int32) for i in range(steps)]
    indptr = (np.arange(batch + 1) * per).astype(np.int32)
    ids = torch.randperm(batch * per, generator=gen, device="cuda").to(torch.int32)
    new = [[torch.randn((batch, h, dim), generator=gen, device="cuda").bfloat16() for h in (kv_heads, kv_heads, heads)] for _ in range(steps)]
    tok, dptr = torch.arange(batch + 1, dtype=torch.int32, device="cuda"), torch.from_numpy(indptr).cuda()
    plans = []
    for n in lens:
        for kw in (dict(), dict(window=50, sinks=3)):
            args = (indptr, n, heads, kv_heads, dim, q.CACHE_E4M3)
            ws = torch.empty(q.gqa_decode_plan(*args, **kw).workspace_bytes, dtype=torch.uint8, device="cuda")
            plans.append((q.gqa_decode_plan(*args, workspace=ws, **kw), ws))

    def run(wait):
        codes = torch.zeros((batch * per, 2, kv_heads, 64, dim), dtype=torch.uint8, device="cuda")
        scale = torch.zeros((batch * per, 2, kv_heads), device="cuda")
        # caches that hold something: the tokens before the first step
        at = torch.randint(0, 0x70, codes.shape, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda", dtype=torch.uint8)
        codes.copy_(at)
        scale.fill_(0.01)
        klen, table = held.clone(), torch.empty_like(ids)
        q_out = torch.empty((batch, heads, dim), dtype=torch.bfloat16, device="cuda")
        outs = torch.empty((steps, 2, batch, heads, dim), dtype=torch.bfloat16, device="cuda")
        lse = torch.empty((steps, 2, batch, heads), device="cuda")
        torch.cuda.synchronize()
        for i, (k, v, query) in enumerate(new):
            table.copy_(ids)
            q.gqa_append_rope(k, v, tok, klen, dptr, table, cs, q.ROPE_HALVES, codes, scale, q.CACHE_E4M3, q=query, q_out=q_out)
            if wait:
                torch.cuda.synchronize()
            for j in range(2):
                p, ws = plans[2 * i + j]
                q.gqa_decode_run(p, q_out, codes, scale, table, 0.1, outs[i, j], lse[i, j], ws)
                if wait:
                    torch.cuda.synchronize()
            klen.add_(1)
        torch.cuda.synchronize()
        return outs, lse, codes, scale

    want = run(True)
    for _ in range(5):
        for a, b in zip(run(False), want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
