"""The appends with nothing, or nothing that has a place, to append."""
import numpy as np
import pytest
import torch

import quantized_kv_paged_gb300 as q
from tests import heads_ref as R

pytestmark = pytest.mark.gpu


def _i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_steps_without_tokens(qkvp):
    """A step of no tokens with its queries: every tensor of it is empty. Nothing is written."""
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")          # noqa: E731
    none = torch.zeros(0, dtype=torch.int64, device="cuda")
    cs = torch.from_numpy(R.table(100, 64)).cuda()
    pool = torch.full((2, 64, 576), 0x5A, dtype=torch.uint8, device="cuda")
    q.mla_append_rope(bf(0, 512), bf(0, 64), none, none, cs, q.ROPE_PAIRS, pool, None, q.KV_FP8_E4M3, q_pe=bf(0, 16, 64), q=bf(0, 16, 576))
    codes, scale = torch.full((2, 2, 1, 64, 64), 0x5A, dtype=torch.uint8, device="cuda"), torch.full((2, 2, 1), 3.0, device="cuda")
    q.gqa_append_rope(bf(0, 1, 64), bf(0, 1, 64), _i32(0, 0), _i32(5), _i32(0, 2), _i32(0, 1), cs, q.ROPE_HALVES, codes, scale, q.CACHE_E4M3,
                      q=bf(0, 4, 64), q_out=bf(0, 4, 64))
    torch.cuda.synchronize()
    assert (pool == 0x5A).all() and (codes == 0x5A).all() and (scale == 3).all()


def test_tokens_without_any_page(qkvp):
    """An empty page table: no token has a page, so nothing is stored, and the queries are rotated all the same."""
    rng = np.random.default_rng(2)
    k, query = (R.to_bf16(rng.standard_normal((5, h, 64)).astype(np.float32)) for h in (1, 4))
    cs = R.table(100, 64)
    codes, scale = torch.full((2, 2, 1, 64, 64), 0x5A, dtype=torch.uint8, device="cuda"), torch.full((2, 2, 1), 3.0, device="cuda")
    q_out = torch.empty((5, 4, 64), dtype=torch.bfloat16, device="cuda")
    q.gqa_append_rope(k.cuda(), k.cuda(), _i32(0, 2, 5), _i32(7, 0), _i32(0, 0, 0), _i32(), torch.from_numpy(cs).cuda(), q.ROPE_HALVES, codes, scale,
                      q.CACHE_E4M3, q=query.cuda(), q_out=q_out)
    torch.cuda.synchronize()
    assert (codes == 0x5A).all() and (scale == 3).all()
    want = np.stack([R.rotate(x, cs[p], R.HALVES) for x, p in zip(R.bf16_to_f32(query), (7, 8, 0, 1, 2))])
    assert torch.equal(q_out.cpu().view(torch.int16), R.to_bf16(want).view(torch.int16))


@pytest.mark.parametrize("n", [40, 1100])
def test_slots_named_twice_leave_the_other_rows_right(qkvp, n):
    """Every third token goes to slot 7: that row may hold anything, every other row and all queries are as they should be."""
    rng = np.random.default_rng(n)
    c_kv, k_pe, q_pe = (R.to_bf16(rng.standard_normal(s).astype(np.float32)) for s in ((n, 512), (n, 64), (n, 2, 64)))
    cs = torch.from_numpy(R.table(n, 64)).cuda()
    slots = 64 + np.arange(n)
    twice = slots.copy()
    twice[::3] = 7
    got = []
    for s in (slots, twice):
        pool = torch.full((2 + n // 64 + 1, q.PAGE_BYTES_FP8_PER_TOKEN), 0x5A, dtype=torch.uint8, device="cuda")
        query = torch.zeros((n, 2, 576), dtype=torch.bfloat16, device="cuda")
        q.mla_append_rope(c_kv.cuda(), k_pe.cuda(), torch.from_numpy(s).cuda(), torch.arange(n, device="cuda"), cs, q.ROPE_HALVES, pool, None,
                          q.KV_FP8_PER_TOKEN, q_pe=q_pe.cuda(), q=query)
        torch.cuda.synchronize()
        rows = torch.cat([pool[:, :64 * 576].reshape(-1, 576), pool[:, 64 * 576:].reshape(-1, 4)], 1).cpu()
        got.append((rows, query.cpu()))
    assert torch.equal(got[0][1].view(torch.int16), got[1][1].view(torch.int16))
    once, again = got[0][0], got[1][0]
    single = np.arange(n) % 3 != 0
    assert torch.equal(once[slots[single]], again[slots[single]])
    untouched = np.setdiff1d(np.arange(len(again)), np.concatenate([slots[single], [7]]))
    assert (again[untouched] == 0x5A).all()
