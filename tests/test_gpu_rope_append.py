"""The appends with rotation against their plain restatement, bit for bit: codes, scales and queries."""
import numpy as np
import pytest
import torch

import oracle
import quantized_kv_paged_gb300 as q
from tests import heads_ref as R

pytestmark = pytest.mark.gpu


def _bf16(rng, *shape, gain=4.0):
    return R.to_bf16((rng.standard_normal(shape) * np.exp2(rng.uniform(-gain, gain, shape[:1] + (1,) * (len(shape) - 1)))).astype(np.float32))


def _same(got: torch.Tensor, want: np.ndarray):
    got = got.cpu().view(torch.int16).numpy() if got.dtype == torch.bfloat16 else got.cpu().numpy()
    assert got.shape == want.shape
    bad = np.argwhere(got.view(np.uint8) != want.view(np.uint8)) if got.dtype.itemsize == 1 else np.argwhere(got != want)
    assert bad.size == 0, (len(bad), bad[:5].tolist())


def _f32_rows_quantized(rows, kv, g):
    """Latent rows float32 [n, 576] -> (codes, scale) by the header's formulas."""
    if kv == q.KV_FP8_E4M3:
        return oracle.encode_array(rows, 1), None
    if kv == q.KV_FP8_PER_TOKEN:
        amax = np.abs(rows).max(1)
        scale = np.where(np.isnan(rows).any(1), np.float32(np.nan), amax / np.float32(448)).astype(np.float32)
        with np.errstate(all="ignore"):
            x = np.where(scale[:, None] == 0, rows, rows / scale[:, None])
        return oracle.encode_array(x, 1), scale
    data, scale = np.zeros((len(rows), 288), np.uint8), np.zeros((len(rows), 36), np.uint8)
    for i, row in enumerate(rows):
        for b in range(36):
            data[i, 8 * b:8 * b + 8], scale[i, b] = oracle.nvfp4_block(row[16 * b:16 * b + 16], g)
    return data, scale


@pytest.mark.parametrize("kv", [q.KV_FP8_E4M3, q.KV_NVFP4, q.KV_FP8_PER_TOKEN])
@pytest.mark.parametrize("style", [q.ROPE_PAIRS, q.ROPE_HALVES])
@pytest.mark.parametrize("n,heads", [(1, 16), (7, 33), (130, 4), (65, 0), (3, 128)])
def test_mla_append_rope_bit_exact(qkvp, kv, style, n, heads):
    rng = np.random.default_rng(1000 * kv + 10 * n + style)
    g = 0.37 if kv == q.KV_NVFP4 else 1.0
    c_kv, wide = _bf16(rng, n, 640), _bf16(rng, n, 576)
    wide[0, 515] = 0.0
    if n > 5:
        c_kv[3, 17], wide[4, 512 + 9], c_kv[5] = float("nan"), float("inf"), 0.0
        wide[5] = 0.0
    cs = R.table(5000, 64)
    pos = rng.integers(0, 5000, n)
    pos[0] = 4999
    slots = rng.permutation(4 * 64)[:n].astype(np.int64)
    if n > 5:
        slots[1], slots[2], pos[6] = -1, 4 * 64, 5000              # skipped: no slot, past the pool, past the table
    q_pe, qbuf = _bf16(rng, n, max(heads, 1), 200), _bf16(rng, n, max(heads, 1), 576)
    skip = (slots < 0) | (slots >= 256) | (pos < 0) | (pos >= 5000)
    width = {q.KV_FP8_E4M3: 64 * 576, q.KV_NVFP4: 64 * 288, q.KV_FP8_PER_TOKEN: q.PAGE_BYTES_FP8_PER_TOKEN}[kv]
    pool = torch.full((4, width), 0x5A, dtype=torch.uint8, device="cuda")
    scale = torch.full((4, 64, 36), 0x33, dtype=torch.uint8, device="cuda") if kv == q.KV_NVFP4 else None
    dev_q = qbuf.cuda()
    q.mla_append_rope(c_kv.cuda()[:, 64:576], wide.cuda()[:, 512:], torch.from_numpy(slots).cuda(), torch.from_numpy(pos).cuda(),
                      torch.from_numpy(cs).cuda(), style, pool, scale, kv, q_pe=q_pe.cuda()[:, :, 8:72] if heads else None,
                      q=dev_q if heads else None, global_scale=g)
    torch.cuda.synchronize()
    rows = np.concatenate([R.bf16_to_f32(c_kv[:, 64:576]), np.zeros((n, 64), np.float32)], 1)
    pe = R.bf16_to_f32(wide[:, 512:])
    for i in range(n):
        if 0 <= pos[i] < 5000:
            rows[i, 512:] = R.rotate(pe[i], cs[pos[i]], style)
    codes, sc = _f32_rows_quantized(rows, kv, g)
    want = np.full((4, width), 0x5A, np.uint8)
    want_scale = np.full((4, 64, 36), 0x33, np.uint8)
    for i in np.nonzero(~skip)[0]:
        p, o = divmod(int(slots[i]), 64)
        w = codes.shape[1]
        want[p, o * w:(o + 1) * w] = codes[i]
        if kv == q.KV_FP8_PER_TOKEN:
            want[p, 64 * 576 + 4 * o:64 * 576 + 4 * o + 4] = sc[i:i + 1].view(np.uint8)
        elif kv == q.KV_NVFP4:
            want_scale[p, o] = sc[i]
    got = pool.cpu().numpy()
    if kv == q.KV_FP8_PER_TOKEN:                                    # the NaN scale has one pattern
        f = want[:, 64 * 576:].view(np.uint32)
        f[(f & 0x7FFFFFFF) > 0x7F800000] = 0x7FC00000
    bad = np.argwhere(got != want)
    assert bad.size == 0, (len(bad), bad[:5].tolist())
    if kv == q.KV_NVFP4:
        assert np.array_equal(scale.cpu().numpy(), want_scale)
    if heads:
        ref = qbuf.clone()
        for i in range(n):
            if 0 <= pos[i] < 5000:
                ref[i, :, 512:] = R.to_bf16(R.rotate(R.bf16_to_f32(q_pe[i, :, 8:72]), cs[pos[i]], style))
        _same(dev_q, ref.view(torch.int16).numpy())


def test_mla_append_rope_in_place_query(qkvp):
    rng = np.random.default_rng(5)
    n, heads = 9, 20
    qbuf, cs, pos = _bf16(rng, n, heads, 576), R.table(300, 64), rng.integers(0, 300, n)
    for style in (q.ROPE_PAIRS, q.ROPE_HALVES):
        dev = qbuf.cuda()
        pool = torch.zeros((1, 64 * 576), dtype=torch.uint8, device="cuda")
        q.mla_append_rope(_bf16(rng, n, 512).cuda(), _bf16(rng, n, 64).cuda(), torch.arange(n, device="cuda"), torch.from_numpy(pos).cuda(),
                          torch.from_numpy(cs).cuda(), style, pool, None, q.KV_FP8_E4M3, q_pe=dev[:, :, 512:], q=dev)
        ref = qbuf.clone()
        for i in range(n):
            ref[i, :, 512:] = R.to_bf16(R.rotate(R.bf16_to_f32(qbuf[i, :, 512:]), cs[pos[i]], style))
        _same(dev, ref.view(torch.int16).numpy())


class Pool:
    """A head pool on the GPU and its host twin, filled with codes and scales that a cache could hold."""

    def __init__(self, rng, pages, heads, dim, cache, fill=None):
        x = rng.standard_normal((pages, 2, heads, 64, dim)).astype(np.float32)
        self.scale = (np.abs(x).max((3, 4)) / R.QMAX[cache]).astype(np.float32)
        self.codes = R.encode(x / self.scale[..., None, None], cache)
        if fill is not None:
            self.codes[:], self.scale[:] = fill
        self.dev_codes, self.dev_scale = torch.from_numpy(self.codes).cuda(), torch.from_numpy(self.scale).cuda()

    def check(self):
        torch.cuda.synchronize()
        assert np.array_equal(self.dev_scale.cpu().numpy(), self.scale, equal_nan=True), np.argwhere(self.dev_scale.cpu().numpy() != self.scale)[:5].tolist()
        _same(self.dev_codes, self.codes)


def _table(rng, pages, counts):
    indptr = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    return indptr, rng.permutation(pages)[:indptr[-1]].astype(np.int32)


def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()


CASES = [
    # new tokens per request, cached before
    ([1], [0]), ([1, 1, 1, 1, 1], [63, 64, 0, 130, 1]), ([5, 0, 3, 1], [62, 9, 64, 127]), ([64, 65, 63], [0, 63, 1]),
    ([200, 1, 0, 333], [100, 5, 7, 0]), ([0, 0, 2], [0, 4, 30]), ([700], [0]),
    # few tokens for many requests, one of them with most of two pages
    ([1] * 20 + [70] + [0, 1] * 10 + [2] * 12, list(range(53))),
]


@pytest.mark.parametrize("dim,rot", [(64, 64), (64, 32), (128, 128), (128, 96), (128, 0), (256, 256), (256, 16)])
@pytest.mark.parametrize("cache", [R.E4M3, R.INT8])
@pytest.mark.parametrize("style", [R.HALVES, R.PAIRS])
def test_gqa_append_rope_bit_exact(qkvp, dim, rot, cache, style):
    rng = np.random.default_rng(dim + rot + 7 * cache + style)
    cs = R.table(1200, rot) if rot else None
    dev_cs = torch.from_numpy(cs).cuda() if rot else None
    for kv_heads, heads, (new, held) in zip((1, 2, 3, 4, 2, 1, 8, 2), (1, 14, 7, 0, 32, 5, 16, 4), CASES):
        n = sum(new)
        counts = [(a + b + 63) // 64 + 1 for a, b in zip(new, held)]
        pages = sum(counts) + 2
        pool = Pool(rng, pages, kv_heads, dim, cache)
        indptr, ids = _table(rng, pages, counts)
        # projections with room to both sides, strong tokens that make scales grow
        qkv = _bf16(rng, n, (heads + 2 * kv_heads) * dim + 24, gain=5)
        cut = lambda t, a, h: t[:, 8 + a * dim:8 + (a + h) * dim].unflatten(1, (h, dim))       # noqa: E731
        dq, dk, dv = (cut(qkv.cuda(), a, h) for a, h in ((0, heads), (heads, kv_heads), (heads + kv_heads, kv_heads)))
        tok = np.concatenate([[0], np.cumsum(new)])
        q_out = torch.full((n, heads, dim), 7.0, dtype=torch.bfloat16, device="cuda")
        use = heads > 0
        q.gqa_append_rope(dk, dv, _i32(tok), _i32(held), _i32(indptr), _i32(ids), dev_cs, style, pool.dev_codes, pool.dev_scale, cache,
                          q=dq if use else None, q_out=q_out if use else None)
        k, v = R.bf16_to_f32(cut(qkv, heads, kv_heads)), R.bf16_to_f32(cut(qkv, heads + kv_heads, kv_heads))
        R.append_heads(k, v, tok, held, indptr, ids, cs, style, pool.codes, pool.scale, cache)
        pool.check()
        if use:
            qf = R.bf16_to_f32(cut(qkv, 0, heads))
            want = qf.copy()
            if rot:
                at = np.concatenate([h + np.arange(m) for m, h in zip(new, held)])
                for i in range(n):
                    want[i] = R.rotate(qf[i], cs[at[i]], style)
            _same(q_out, R.to_bf16(want).view(torch.int16).numpy())


@pytest.mark.parametrize("cache", [R.E4M3, R.INT8])
def test_gqa_append_special_values_and_zero_blocks(qkvp, cache):
    """NaN, infinities, an all-zero block, a block whose scale is 0 and a scale that has to grow a long way."""
    rng = np.random.default_rng(3)
    pool = Pool(rng, 6, 1, 64, cache)
    pool.scale[2, :, 0], pool.scale[4, 0, 0] = 0.0, 1e-37
    pool.codes[2], pool.codes[5, 1] = 0, 0xFF if cache == R.E4M3 else 0x81
    pool.dev_codes.copy_(torch.from_numpy(pool.codes))
    pool.dev_scale.copy_(torch.from_numpy(pool.scale))
    new, held = [10, 3, 2, 4, 1], [0, 60, 5, 20, 63]
    k = R.bf16_to_f32(_bf16(rng, 20, 1, 64))
    v = R.bf16_to_f32(_bf16(rng, 20, 1, 64))
    k[1, 0, 5], k[2, 0, 6], k[3, 0, 7], v[4, 0, 0] = np.nan, np.inf, -np.inf, np.nan
    v[0:10] = 0.0
    v[13:15], k[13] = 0.0, 0.0
    v[19, 0, :] = 3.3e38
    k, v = R.bf16_to_f32(R.to_bf16(k)), R.bf16_to_f32(R.to_bf16(v))
    tok = np.concatenate([[0], np.cumsum(new)])
    indptr, ids = np.array([0, 1, 2, 3, 4, 5], np.int32), np.array([0, 1, 2, 4, 5], np.int32)
    held[1] = 60 - 0
    new[1] = 3
    q.gqa_append_rope(R.to_bf16(k).cuda(), R.to_bf16(v).cuda(), _i32(tok), _i32(held), _i32(indptr), _i32(ids), None, R.HALVES, pool.dev_codes,
                      pool.dev_scale, cache)
    R.append_heads(k, v, tok, held, indptr, ids, None, R.HALVES, pool.codes, pool.scale, cache)
    pool.check()


@pytest.mark.parametrize("n_pad", [0, 37])
def test_gqa_append_skips_padding_bad_pages_and_positions(qkvp, n_pad):
    """Rows behind the last sequence, pages outside the list, the table or the pool, positions past the table:
    nothing of them is written; the query of a token with a bad page is rotated all the same."""
    rng = np.random.default_rng(8 + n_pad)
    new, held = [3, 70, 2, 5], [10, 60, 0, 3]
    tok = np.concatenate([[0], np.cumsum(new)])
    n = tok[-1] + n_pad
    pool = Pool(rng, 8, 2, 64, R.E4M3)
    indptr = np.array([0, 1, 3, 4, 5], np.int32)                    # request 1 needs 3 pages, has 2
    ids = np.array([5, 2, 7, 8, -1], np.int32)                      # requests 2 and 3: out of the pool
    cs = R.table(100, 64)
    k, v, qq = _bf16(rng, n, 2, 64), _bf16(rng, n, 2, 64), _bf16(rng, n, 4, 64)
    pos = rng.integers(0, 100, n)
    pos[1], pos[5], pos[tok[2] + 1] = 100, -1, 1 << 40
    q_out = torch.full((n, 4, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    q.gqa_append_rope(k.cuda(), v.cuda(), _i32(tok), _i32(held), _i32(indptr), _i32(ids), torch.from_numpy(cs).cuda(), R.PAIRS, pool.dev_codes,
                      pool.dev_scale, R.E4M3, q=qq.cuda(), q_out=q_out, positions=torch.from_numpy(pos).cuda())
    R.append_heads(R.bf16_to_f32(k), R.bf16_to_f32(v), tok, held, indptr, ids, cs, R.PAIRS, pool.codes, pool.scale, R.E4M3, positions=pos)
    pool.check()
    want = np.full((n, 4, 64), 9.0, np.float32)
    for i in range(tok[-1]):
        if 0 <= pos[i] < 100:
            want[i] = R.rotate(R.bf16_to_f32(qq[i]), cs[pos[i]], R.PAIRS)
    _same(q_out, R.to_bf16(want).view(torch.int16).numpy())


def test_gqa_append_many_requests_and_in_place_query(qkvp):
    """1,500 requests (the search over requests takes three rounds), zero-length ones among them."""
    rng = np.random.default_rng(11)
    batch = 1500
    for lo, hi in ((0, 1), (0, 3)):
        new, held = rng.integers(lo, hi + 1, batch), rng.integers(0, 200, batch)
        tok = np.concatenate([[0], np.cumsum(new)])
        n = int(tok[-1])
        counts = (new + held + 63) // 64
        pool = Pool(rng, int(counts.sum()) + 1, 1, 64, R.INT8)
        indptr, ids = _table(rng, len(pool.codes), counts)
        cs = R.table(300, 64)
        k, v, qq = _bf16(rng, n, 1, 64), _bf16(rng, n, 1, 64), _bf16(rng, n, 3, 64)
        dq = qq.cuda()
        q.gqa_append_rope(k.cuda(), v.cuda(), _i32(tok), _i32(held), _i32(indptr), _i32(ids), torch.from_numpy(cs).cuda(), R.HALVES, pool.dev_codes,
                          pool.dev_scale, R.INT8, q=dq, q_out=dq)
        R.append_heads(R.bf16_to_f32(k), R.bf16_to_f32(v), tok, held, indptr, ids, cs, R.HALVES, pool.codes, pool.scale, R.INT8)
        pool.check()
        want = R.bf16_to_f32(qq)
        at = np.concatenate([h + np.arange(m) for m, h in zip(new, held)])
        for i in range(n):
            want[i] = R.rotate(want[i], cs[at[i]], R.HALVES)
        _same(dq, R.to_bf16(want).view(torch.int16).numpy())


def test_captured_append_follows_the_device_lengths(qkvp):
    """A captured step replays with new tokens and lengths: the same bytes as eager calls, on another stream."""
    rng = np.random.default_rng(21)
    batch, kv_heads, dim = 5, 2, 128
    held = np.array([0, 63, 64, 10, 200])
    counts = (held + 8 + 63) // 64 + 1
    pool = Pool(rng, int(counts.sum()), kv_heads, dim, R.E4M3)
    indptr, ids = _table(rng, len(pool.codes), counts)
    cs = R.table(400, dim)
    k = torch.zeros((batch, kv_heads, dim), dtype=torch.bfloat16, device="cuda")
    v, qq, q_out = torch.zeros_like(k), torch.zeros((batch, 8, dim), dtype=torch.bfloat16, device="cuda"), torch.zeros((batch, 8, dim), dtype=torch.bfloat16, device="cuda")
    tok, klen, dptr, dids, dcs = _i32(np.arange(batch + 1)), _i32(held), _i32(indptr), _i32(ids), torch.from_numpy(cs).cuda()
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        q.gqa_append_rope(k, v, tok, klen, dptr, dids, dcs, R.HALVES, pool.dev_codes, pool.dev_scale, R.E4M3, q=qq, q_out=q_out)
    for step in range(4):
        hk, hv, hq = _bf16(rng, batch, kv_heads, dim), _bf16(rng, batch, kv_heads, dim), _bf16(rng, batch, 8, dim)
        k.copy_(hk)
        v.copy_(hv)
        qq.copy_(hq)
        klen.copy_(torch.from_numpy(held + step))
        graph.replay()
        R.append_heads(R.bf16_to_f32(hk), R.bf16_to_f32(hv), np.arange(batch + 1), held + step, indptr, ids, cs, R.HALVES, pool.codes, pool.scale, R.E4M3)
        pool.check()
        want = np.stack([R.rotate(R.bf16_to_f32(hq[i]), cs[held[i] + step], R.HALVES) for i in range(batch)])
        _same(q_out, R.to_bf16(want).view(torch.int16).numpy())
