"""The appends' forms for many tokens, bit for bit: latent rows together with query heads in one warp (1,024 tokens and more),
and pages of several heads to a CTA (300 pages times KV heads and more)."""
import numpy as np
import pytest
import torch

import quantized_kv_paged_gb300 as q
from tests import heads_ref as R
from tests.test_gpu_rope_append import Pool, _bf16, _f32_rows_quantized, _i32, _same, _table

pytestmark = pytest.mark.gpu

WIDTH = {q.KV_FP8_E4M3: 576, q.KV_NVFP4: 288, q.KV_FP8_PER_TOKEN: 576}


def _latent(n, heads, kv, style, seed, in_place=False):
    """One append of n rows into a larger pool; every byte of the pool, the scales and q is compared. NVFP4 rows repeat
    every 97 tokens (their restatement goes block by block); places and query heads are all different."""
    rng = np.random.default_rng(seed)
    distinct = 97 if kv == q.KV_NVFP4 else n
    of = np.arange(n) % distinct
    g = 0.37 if kv == q.KV_NVFP4 else 1.0
    c_kv, k_pe, pos = _bf16(rng, distinct, 512), _bf16(rng, distinct, 64), rng.integers(0, 3000, distinct)
    c_kv[3, 17], k_pe[4, 9], c_kv[5], k_pe[5] = float("nan"), float("inf"), 0.0, 0.0
    pos[0], pos[6], pos[7] = 2999, 3000, -1                        # the last row, and two that are skipped
    cs = R.table(3000, 64)
    pages = n // 64 + 3
    slots = rng.permutation(pages * 64)[:n].astype(np.int64)
    slots[1], slots[2], slots[n - 1] = -1, pages * 64, 1 << 40     # skipped, their queries are not
    qbuf = _bf16(rng, n, max(heads, 1), 576)
    q_pe = qbuf[:, :, 512:] if in_place else _bf16(rng, n, max(heads, 1), 64)
    width = WIDTH[kv] * 64 + (256 if kv == q.KV_FP8_PER_TOKEN else 0)
    pool = torch.full((pages, width), 0x5A, dtype=torch.uint8, device="cuda")
    scale = torch.full((pages, 64, 36), 0x33, dtype=torch.uint8, device="cuda") if kv == q.KV_NVFP4 else None
    dev_q = qbuf.cuda()
    dev_pe = dev_q[:, :, 512:] if in_place else q_pe.cuda()
    q.mla_append_rope(c_kv[of].cuda(), k_pe[of].cuda(), torch.from_numpy(slots).cuda(), torch.from_numpy(pos[of]).cuda(), torch.from_numpy(cs).cuda(),
                      style, pool, scale, kv, q_pe=dev_pe if heads else None, q=dev_q if heads else None, global_scale=g)
    torch.cuda.synchronize()
    good = (pos >= 0) & (pos < 3000)
    at = cs[np.where(good, pos, 0)]
    codes, sc = _f32_rows_quantized(np.concatenate([R.bf16_to_f32(c_kv), R.rotate(R.bf16_to_f32(k_pe), at, style)], 1), kv, g)
    want, want_scale = np.full((pages, width), 0x5A, np.uint8), np.full((pages, 64, 36), 0x33, np.uint8)
    kept = np.nonzero(good[of] & (slots >= 0) & (slots < pages * 64))[0]
    page, off = np.divmod(slots[kept], 64)
    rows = np.arange(WIDTH[kv])
    want[page[:, None], off[:, None] * WIDTH[kv] + rows] = codes[of[kept]]
    if kv == q.KV_FP8_PER_TOKEN:
        bits = np.where(np.isnan(sc), np.uint32(0x7FC00000), sc.view(np.uint32)).astype(np.uint32)
        want[page[:, None], 64 * 576 + 4 * off[:, None] + np.arange(4)] = bits[of[kept]].view(np.uint8).reshape(-1, 4)
    elif kv == q.KV_NVFP4:
        want_scale[page, off] = sc[of[kept]]
    bad = np.argwhere(pool.cpu().numpy() != want)
    assert bad.size == 0, (len(bad), bad[:5].tolist())
    if kv == q.KV_NVFP4:
        assert np.array_equal(scale.cpu().numpy(), want_scale)
    if heads:
        ref = qbuf.clone()
        turned = R.to_bf16(R.rotate(R.bf16_to_f32(q_pe), at[of][:, None], style))
        ref[:, :, 512:] = torch.where(torch.from_numpy(good[of])[:, None, None], turned, qbuf[:, :, 512:])
        _same(dev_q, ref.view(torch.int16).numpy())


@pytest.mark.parametrize("kv", [q.KV_FP8_E4M3, q.KV_NVFP4, q.KV_FP8_PER_TOKEN])
@pytest.mark.parametrize("style", [q.ROPE_PAIRS, q.ROPE_HALVES])
@pytest.mark.parametrize("n,heads", [(1023, 17), (1024, 4), (1500, 16), (1024, 17), (1500, 33), (1201, 128), (2100, 0)])
def test_latent_rows_of_a_prompt(qkvp, kv, style, n, heads):
    _latent(n, heads, kv, style, seed=n + heads + kv)


@pytest.mark.parametrize("style", [q.ROPE_PAIRS, q.ROPE_HALVES])
@pytest.mark.parametrize("heads", [16, 40])
def test_latent_rows_of_a_prompt_rotate_queries_in_place(qkvp, heads, style):
    _latent(1100, heads, q.KV_FP8_E4M3, style, seed=heads, in_place=True)


@pytest.mark.parametrize("cache", [R.E4M3, R.INT8])
@pytest.mark.parametrize("dim,rot,kv_heads,style", [(64, 32, 16, R.PAIRS), (128, 128, 7, R.HALVES), (128, 0, 8, R.HALVES), (256, 64, 5, R.HALVES),
                                                    (64, 64, 9, R.HALVES)])
def test_several_heads_of_a_page(qkvp, cache, dim, rot, kv_heads, style):
    """Ragged chunks, 63 pages counted as busy: a CTA takes 63 * 2 * kv_heads / 300 heads, two (5, 7), three (8, 9) or six
    (16), the last part but for 9 fewer. Heads next to one another hold NaN, infinities and zeros, started pages have
    scales that grow, are 0 or are kept; some tokens are skipped, and rows behind the last request are padding."""
    rng = np.random.default_rng(dim + rot + kv_heads + cache)
    new, held = [1003, 0, 2050, 700], [37, 5, 64, 130]
    tok = np.concatenate([[0], np.cumsum(new)])
    n = int(tok[-1]) + 29
    counts = [(a + b + 63) // 64 for a, b in zip(new, held)]
    pool = Pool(rng, sum(counts) + 2, kv_heads, dim, cache)
    indptr, ids = _table(rng, len(pool.codes), counts)
    ids[indptr[2] + 9] = len(pool.codes)                           # a page out of the pool, in the middle of a request
    first = ids[indptr[[0, 3]] + [0, 2]]                           # started pages of requests 0 and 3
    pool.scale[first[0], :, 0], pool.codes[first[0], :, 0] = 0.0, 0
    pool.scale[first[1], :, kv_heads - 1] = 1e-12
    pool.scale[first[0], :, kv_heads - 1] = 100.0
    pool.dev_scale.copy_(torch.from_numpy(pool.scale))
    pool.dev_codes.copy_(torch.from_numpy(pool.codes))
    k, v = R.bf16_to_f32(_bf16(rng, n, kv_heads, dim, gain=5)), R.bf16_to_f32(_bf16(rng, n, kv_heads, dim, gain=5))
    for x in (k, v):
        x[5, 0, 3], x[6, 1, 4], x[7, 2, 5], x[8, 2, 6] = np.nan, np.inf, -np.inf, np.nan
        x[1100:1260, 1:3] = 0.0                                    # whole pages of zeros in two heads
        x[2000, 3], x[2001, 4] = np.nan, np.inf
        x[tok[3] + 3, kv_heads - 1] = 3e38
        x[tok[-1]:] = np.nan
    k, v = R.to_bf16(k), R.to_bf16(v)
    cs = R.table(2200, rot) if rot else None
    pos = np.concatenate([h + np.arange(m) for m, h in zip(new, held)] + [np.zeros(29, np.int64)])
    if rot:
        pos[[0, 40, 1500, 1501, 3052]] = [2200, -1, 1 << 40, 5000, -7]
    query = _bf16(rng, n, 3, dim)
    q_out = torch.full((n, 3, dim), 7.0, dtype=torch.bfloat16, device="cuda")
    q.gqa_append_rope(k.cuda(), v.cuda(), _i32(tok), _i32(held), _i32(indptr), _i32(ids), torch.from_numpy(cs).cuda() if rot else None, style,
                      pool.dev_codes, pool.dev_scale, cache, q=query.cuda(), q_out=q_out, positions=torch.from_numpy(pos).cuda())
    R.append_heads(R.bf16_to_f32(k), R.bf16_to_f32(v), tok, held, indptr, ids, cs, style, pool.codes, pool.scale, cache, positions=pos)
    pool.check()
    want = torch.full((n, 3, dim), 7.0, dtype=torch.bfloat16)
    keep = np.nonzero((pos[:tok[-1]] >= 0) & (pos[:tok[-1]] < 2200))[0]
    turned = R.bf16_to_f32(query[keep])
    want[keep] = R.to_bf16(R.rotate(turned, cs[pos[keep]][:, None], style) if rot else turned)
    _same(q_out, want.view(torch.int16).numpy())


def test_search_over_more_requests_than_two_rounds_find(qkvp):
    """70,000 requests, one in ten with a token: three rounds of 256 probes, of 274, 2 and 1 requests apart."""
    rng = np.random.default_rng(17)
    batch = 70000
    new, held = (rng.random(batch) < 0.1).astype(np.int64), rng.integers(0, 64, batch)
    new[[0, batch - 1]] = 1
    tok = np.concatenate([[0], np.cumsum(new)])
    n = int(tok[-1])
    pool = Pool(rng, n + 1, 1, 64, R.INT8)
    indptr, ids = _table(rng, n + 1, new)
    k, v = _bf16(rng, n, 1, 64), _bf16(rng, n, 1, 64)
    q.gqa_append_rope(k.cuda(), v.cuda(), _i32(tok), _i32(held), _i32(indptr), _i32(ids), None, R.HALVES, pool.dev_codes, pool.dev_scale, R.INT8)
    R.append_heads(R.bf16_to_f32(k), R.bf16_to_f32(v), tok, held, indptr, ids, None, R.HALVES, pool.codes, pool.scale, R.INT8)
    pool.check()
