"""Decode attention over the 8-bit head pool against its definition in 64 bits, under the bounds derived in
heads_ref.check_attend."""
import numpy as np
import pytest
import torch

import quantized_kv_paged_gb300 as q
import synth
from tests import heads_ref as R
from tests.helpers import compare

pytestmark = pytest.mark.gpu

RAGGED = [1, 0, 63, 64, 65, 127, 128, 129, 1000, 33, 2500]


class Batch:
    """A ragged batch over a scattered pool whose unused slots and pages hold NaN codes (E4M3), extreme codes
    (INT8) and NaN scales, and whose page-table entries of pages that no query sees are no page ids."""

    def __init__(self, lens, heads, kv_heads, dim, cache, window=0, sinks=0, seed=0, v_spread=2.0, q_gain=1.0):
        rng = np.random.default_rng(seed)
        self.lens, self.heads, self.kv_heads, self.dim, self.cache = np.array(lens, np.int32), heads, kv_heads, dim, cache
        self.window, self.sinks = window, sinks
        counts = (self.lens + 63) // 64 + rng.integers(0, 2, len(lens))
        self.indptr = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        pages = int(self.indptr[-1]) + 3
        self.ids = rng.permutation(pages)[:self.indptr[-1]].astype(np.int32)
        bad = 0xFF if cache == R.E4M3 else 0x80
        self.codes = np.full((pages, 2, kv_heads, 64, dim), bad, np.uint8)
        self.scale = np.full((pages, 2, kv_heads), np.nan, np.float32)
        visible = np.zeros(int(self.indptr[-1]), bool)
        for r, n in enumerate(self.lens):
            for t0 in range(0, int(n), 64):
                page, c = self.ids[self.indptr[r] + t0 // 64], min(64, int(n) - t0)
                x = rng.standard_normal((2, kv_heads, c, dim)).astype(np.float32)
                x[0, :, :, ::29] *= 5
                x[1] *= np.exp2(rng.uniform(-v_spread, v_spread, (kv_heads, 1, 1)))
                s = np.abs(x).max((2, 3)) / R.QMAX[cache]
                self.codes[page, :, :, :c], self.scale[page] = R.encode(x / s[..., None, None], cache), s
                t = np.arange(t0, t0 + c)
                visible[self.indptr[r] + t0 // 64] = window == 0 or bool(((t >= n - window) | (t < sinks)).any())
        self.q = R.to_bf16(rng.standard_normal((len(lens), heads, dim)).astype(np.float32) * q_gain)
        self.hidden = ~visible
        self.ids[self.hidden] = rng.choice([-1, -2 ** 31, pages, 2 ** 31 - 1], int(self.hidden.sum()))
        self.sm_scale = dim ** -0.5

    def run(self, num_sms=0, min_splits=0, lse=True, stream=None):
        p, ws = self.plan(num_sms, min_splits)
        self.dev = dict(q=self.q.cuda(), codes=torch.from_numpy(self.codes).cuda(), scale=torch.from_numpy(self.scale).cuda(),
                        ids=torch.from_numpy(self.ids).cuda())
        out = torch.full((len(self.lens) + 1, self.heads, self.dim), 5.0, dtype=torch.bfloat16, device="cuda")
        l = torch.full((len(self.lens) + 1, self.heads), 5.0, dtype=torch.float32, device="cuda")
        torch.cuda.synchronize()
        q.gqa_decode_run(p, self.dev["q"], self.dev["codes"], self.dev["scale"], self.dev["ids"], self.sm_scale, out[:-1], l[:-1] if lse else None, ws, stream=stream)
        torch.cuda.synchronize()
        assert int(ws[p.status_offset:p.status_offset + 4].view(torch.int32).item()) == 0
        assert (out[-1] == 5).all() and (l[-1] == 5).all()         # rows behind the last sequence
        return out[:-1], l[:-1], p

    def plan(self, num_sms=0, min_splits=0):
        args = (self.indptr, self.lens, self.heads, self.kv_heads, self.dim, self.cache)
        kw = dict(window=self.window, sinks=self.sinks, num_sms=num_sms, min_splits=min_splits)
        ws = torch.full((max(256, q.gqa_decode_plan(*args, **kw).workspace_bytes),), 0xA5, dtype=torch.uint8, device="cuda")
        return q.gqa_decode_plan(*args, workspace=ws, **kw), ws

    def ref(self):
        return R.attend(R.bf16_to_f32(self.q), self.codes, self.scale, self.cache, self.indptr, self.ids, self.lens, self.sm_scale,
                        self.window, self.sinks)

    def check(self, **kw):
        out, lse, p = self.run(**kw)
        print(R.check_attend(out, lse, self.ref(), int(self.lens.max()), self.dim), p.as_dict())
        return p


@pytest.mark.parametrize("cache", [R.E4M3, R.INT8])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (8, 1), (10, 2), (32, 2), (7, 7), (37, 1), (40, 8)])
def test_ragged_batch(qkvp, cache, dim, heads, kv_heads):
    Batch(RAGGED, heads, kv_heads, dim, cache, seed=heads + dim).check()


@pytest.mark.parametrize("cache", [R.E4M3, R.INT8])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (64, 0), (65, 63), (100, 64), (130, 65), (900, 4), (5000, 0), (33, 200)])
def test_window_and_sinks(qkvp, cache, dim, window, sinks):
    Batch(RAGGED, 8, 2, dim, cache, window, sinks, seed=window + sinks).check()


@pytest.mark.parametrize("num_sms,min_splits", [(1, 0), (3, 0), (152, 0), (40, 300), (1, 100000)])
@pytest.mark.parametrize("heads,kv_heads,dim", [(16, 2, 128), (40, 2, 64), (4, 4, 256)])
def test_splits_are_joined(qkvp, num_sms, min_splits, heads, kv_heads, dim):
    p = Batch([4000, 1, 700, 0, 65], heads, kv_heads, dim, R.E4M3, seed=num_sms).check(num_sms=num_sms, min_splits=min_splits)
    assert min_splits == 0 or p.num_split_groups > 0


@pytest.mark.parametrize("cache", [R.E4M3, R.INT8])
def test_long_request_many_splits(qkvp, cache):
    p = Batch([40001], 8, 1, 128, cache, seed=4).check()
    assert p.max_group_segments > 16


@pytest.mark.parametrize("q_gain", [1e-30, 1e-3, 30.0, 3e4])
def test_query_magnitudes(qkvp, q_gain):
    """From queries far below FP16's range (uniform weights) to logits in the millions (one token takes all)."""
    Batch([300, 64, 17], 12, 2, 128, R.E4M3, seed=2, q_gain=q_gain).check()


@pytest.mark.parametrize("cache", [R.E4M3, R.INT8])
def test_value_scales_far_apart(qkvp, cache):
    """V block scales over 36 binades, one block all zero: a block's weight in the sum does not depend on
    where it comes."""
    for seed in range(3):
        b = Batch([1500, 640], 8, 2, 128, cache, seed=seed, v_spread=18.0)
        for e in (0, 3, 7):
            b.scale[b.ids[e], 1], b.codes[b.ids[e], 1] = 0.0, 0
        b.check(num_sms=2 if seed else 0)


@pytest.mark.parametrize("cache", [R.E4M3, R.INT8])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("heads,kv_heads", [(8, 2), (32, 2)])
@pytest.mark.parametrize("steps,heavy", [([-110, 0], 0), ([0, -110], 0), ([-115, -20, 75], 0), ([60, -60, 0], 0), ([-110, 0], -110),
                                         ([-115, -20, 75], -115), ([75, -20, -115], -115)])
def test_value_scales_over_all_exponents(qkvp, cache, dim, heads, kv_heads, steps, heavy):
    """V block scales more than 2^90 apart, in every order; `heavy`: the pages of these scales take nearly all
    of the weight (keys 64 times as large). The reference's exponents, up to 2^7, are held to 2^-18, which the bound's e,
    at least 2 * 72 * 2^-24 * dot with a dot above 2, exceeds."""
    b = Batch([900, 200, 70], heads, kv_heads, dim, cache, seed=dim + heads)
    for r, n in enumerate(b.lens):
        for i in range((int(n) + 63) // 64):
            e = steps[i % len(steps)]
            b.scale[b.ids[b.indptr[r] + i], 1] *= np.float32(2.0 ** e)
            if heavy and e == heavy:
                b.scale[b.ids[b.indptr[r] + i], 0] *= np.float32(64)
    ref = b.ref()
    assert np.isfinite(ref[0]).all() and (ref[3] > 2).all()
    for num_sms in (0, 1):
        out, lse, _ = b.run(num_sms=num_sms)
        R.check_attend(out, lse, ref, 900, dim)


def test_zero_scale_keys_and_equal_logits(qkvp):
    b = Batch([900], 8, 1, 64, R.INT8, seed=5)
    b.scale[:, 0][~np.isnan(b.scale[:, 0])] = 0.0
    out, lse, _ = b.run()
    R.check_attend(out, lse, b.ref(), 900, 64)
    assert np.allclose(lse.cpu().numpy(), np.log(900), atol=2e-6)


def test_page_ids_out_of_the_pool_are_not_seen(qkvp):
    b = Batch([640, 300, 70], 8, 2, 128, R.E4M3, seed=6)
    b.ids[b.indptr[0] + np.array([0, 4, 9])] = [-1, 2 ** 31 - 1, len(b.codes)]
    b.ids[b.indptr[2]:b.indptr[3]] = -5                            # a whole request
    p = b.check()
    assert p.batch == 3
    b.check(num_sms=1)


def test_without_lse_and_on_another_stream(qkvp):
    b = Batch(RAGGED, 16, 4, 64, R.INT8, seed=9)
    s = torch.cuda.Stream()
    out, _, _ = b.run()
    out2, lse2, _ = b.run(lse=False, stream=s)
    assert torch.equal(out, out2) and (lse2 == 5).all()


def test_repeats_bit_for_bit_and_in_graphs(qkvp):
    """One plan, many runs: equal bits from eager calls, a captured graph, and after other runs used the
    workspace. Planning is refused during capture."""
    b = Batch([3000, 64, 700, 0, 5], 32, 4, 128, R.E4M3, seed=12)
    out, lse, _ = b.run()
    p, ws = b.plan()
    d = b.dev
    o, l = torch.empty_like(out), torch.empty_like(lse)

    def step():
        q.gqa_decode_run(p, d["q"], d["codes"], d["scale"], d["ids"], b.sm_scale, o, l, ws)

    for _ in range(20):
        step()
        assert torch.equal(o, out) and torch.equal(l, lse)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        step()
        step()
        st = q.gqa_decode_plan(b.indptr, b.lens, 32, 4, 128, R.E4M3, workspace=ws, raise_on_error=False).status
    assert st == q.QKVP_E_UNSUPPORTED
    for _ in range(3):
        o.fill_(float("nan"))
        l.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, out) and torch.equal(l, lse)


def test_two_streams_at_once(qkvp):
    """Two batches with plans and workspaces of their own, run many times on two streams side by side."""
    bs = [Batch([3000, 700, 65], 16, 2, 128, R.E4M3, seed=50), Batch([900] * 30, 16, 8, 64, R.INT8, 200, 5, seed=51)]
    want = [b.run()[:2] for b in bs]
    plans = [b.plan() for b in bs]
    outs = [(torch.empty_like(w[0]), torch.empty_like(w[1])) for w in want]
    streams = [torch.cuda.Stream() for _ in bs]
    torch.cuda.synchronize()
    for _ in range(50):
        for b, (p, ws), (o, l), st in zip(bs, plans, outs, streams):
            q.gqa_decode_run(p, b.dev["q"], b.dev["codes"], b.dev["scale"], b.dev["ids"], b.sm_scale, o, l, ws, stream=st)
    torch.cuda.synchronize()
    for (o, l), (wo, wl) in zip(outs, want):
        assert torch.equal(o, wo) and torch.equal(l, wl)


def test_offsets_past_32_bits(qkvp):
    """Pages at the end of a 6 GiB pool: appended to and attended, at offsets past 2^32."""
    kv_heads, dim, heads, n = 8, 256, 16, 300
    pages = (6 << 30) // (2 * kv_heads * 64 * dim)
    codes = torch.empty((pages, 2, kv_heads, 64, dim), dtype=torch.uint8, device="cuda")
    scale = torch.zeros((pages, 2, kv_heads), device="cuda")
    ids = np.array([pages - 1, pages - 7, 0, pages - 2, pages // 2, pages - 3], np.int32)
    rng = np.random.default_rng(60)
    k, v = (R.to_bf16(rng.standard_normal((n, kv_heads, dim)).astype(np.float32)) for _ in range(2))
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")          # noqa: E731
    dids = torch.from_numpy(ids).cuda()
    q.gqa_append_rope(k.cuda(), v.cuda(), i32(0, n), i32(0), i32(0, len(ids)), dids, None, R.HALVES, codes, scale, R.E4M3)
    used = ids[:(n + 63) // 64].astype(np.int64)
    small_codes, small_scale = np.zeros((6, 2, kv_heads, 64, dim), np.uint8), np.zeros((6, 2, kv_heads), np.float32)
    R.append_heads(R.bf16_to_f32(k), R.bf16_to_f32(v), [0, n], [0], [0, 6], np.arange(6), None, R.HALVES, small_codes, small_scale, R.E4M3)
    for i, page in enumerate(used):
        c = min(64, n - 64 * i)
        assert np.array_equal(codes[page, :, :, :c].cpu().numpy(), small_codes[i, :, :, :c])
        assert np.array_equal(scale[page].cpu().numpy(), small_scale[i])
    query = R.to_bf16(rng.standard_normal((1, heads, dim)).astype(np.float32))
    args = ([0, 6], [n], heads, kv_heads, dim, R.E4M3)
    ws = torch.empty(q.gqa_decode_plan(*args).workspace_bytes, dtype=torch.uint8, device="cuda")
    p = q.gqa_decode_plan(*args, workspace=ws)
    out, lse = torch.empty((1, heads, dim), dtype=torch.bfloat16, device="cuda"), torch.empty((1, heads), device="cuda")
    q.gqa_decode_run(p, query.cuda(), codes, scale, dids, 0.1, out, lse, ws)
    torch.cuda.synchronize()
    ref = R.attend(R.bf16_to_f32(query), small_codes, small_scale, R.E4M3, [0, 6], np.arange(6), [n], 0.1)
    R.check_attend(out, lse, ref, n, dim)


def test_first_call_of_a_process_is_captured(qkvp):
    """No eager call goes before: kernel set-up inside a capture, append and decode in one graph."""
    code = """
import torch, quantized_kv_paged_gb300 as q
dev = "cuda"
codes, scale = torch.zeros((4, 2, 1, 64, 64), dtype=torch.uint8, device=dev), torch.zeros((4, 2, 1), device=dev)
i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=dev)
k = torch.randn((100, 1, 64), device=dev).bfloat16()
query, out = torch.randn((1, 2, 64), device=dev).bfloat16(), torch.zeros((1, 2, 64), device=dev).bfloat16()
tok, held, ptr, ids = i32(0, 100), i32(0), i32(0, 2), i32(3, 1)
args = ([0, 2], [100], 2, 1, 64, q.CACHE_E4M3)
ws = torch.empty(q.gqa_decode_plan(*args).workspace_bytes, dtype=torch.uint8, device=dev)
plan = q.gqa_decode_plan(*args, workspace=ws)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g, stream=torch.cuda.Stream()):
    q.gqa_append_rope(k, k, tok, held, ptr, ids, None, q.ROPE_HALVES, codes, scale, q.CACHE_E4M3)
    q.gqa_decode_run(plan, query, codes, scale, ids, 0.125, out, None, ws)
g.replay()
torch.cuda.synchronize()
kv = (codes.view(torch.float8_e4m3fn).float() * scale[..., None, None])[[3, 1], 0, 0].reshape(-1, 64)[:100]
want = torch.softmax(query[0].float() @ kv.T * 0.125, 1) @ kv
assert (out[0].float() - want).abs().max() < 0.02, (out, want)
print("captured first: ok")
"""
    import subprocess
    import sys
    from tests.conftest import ROOT
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured first: ok" in r.stdout, r.stdout + r.stderr


def test_nan_in_a_visible_key_reaches_its_head_only(qkvp):
    b = Batch([500, 90], 8, 2, 64, R.E4M3, seed=13)
    b.codes[b.ids[1], 0, 1, 5, 3] = 0x7F
    out, lse, _ = b.run()
    assert torch.isnan(out[0, 4:]).all() and torch.isnan(lse[0, 4:]).all()
    assert torch.isfinite(out[0, :4]).all() and torch.isfinite(out[1]).all()


def test_serving_steps_end_to_end(qkvp):
    """Prefill chunks, then decode steps, as a serving loop calls them: append with rotation, plan, decode with
    a full and a windowed layer. The cache's bytes equal the restatement's, the outputs its attention."""
    rng = np.random.default_rng(30)
    batch, heads, kv_heads, dim, max_pos = 3, 8, 2, 64, 2000
    cs = R.table(max_pos, dim)
    dcs = torch.from_numpy(cs).cuda()
    lens = np.zeros(batch, np.int64)
    indptr = (np.arange(batch + 1) * 12).astype(np.int32)
    ids = rng.permutation(40)[:36].astype(np.int32)
    codes, scale = np.full((40, 2, kv_heads, 64, dim), 0xFF, np.uint8), np.full((40, 2, kv_heads), np.nan, np.float32)
    dcodes, dscale, dids, dptr = torch.from_numpy(codes).cuda(), torch.from_numpy(scale).cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(indptr).cuda()
    for new in ([130, 1, 300], [70, 64, 0], [1, 1, 1], [1, 1, 1], [1, 1, 1]):
        n = sum(new)
        k, v, qq = (R.to_bf16(rng.standard_normal((n, h, dim)).astype(np.float32) * np.exp2(rng.uniform(0, 3, (n, 1, 1)))) for h in (kv_heads, kv_heads, heads))
        tok = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        q_out = torch.empty((n, heads, dim), dtype=torch.bfloat16, device="cuda")
        q.gqa_append_rope(k.cuda(), v.cuda(), torch.from_numpy(tok).cuda(), torch.from_numpy(lens.astype(np.int32)).cuda(), dptr, dids, dcs, R.HALVES, dcodes,
                          dscale, R.E4M3, q=qq.cuda(), q_out=q_out)
        R.append_heads(R.bf16_to_f32(k), R.bf16_to_f32(v), tok, lens, indptr, ids, cs, R.HALVES, codes, scale, R.E4M3)
        lens += new
        assert np.array_equal(dcodes.cpu().numpy(), codes) and np.array_equal(dscale.cpu().numpy(), scale, equal_nan=True)
        last = torch.from_numpy(np.maximum(tok[1:] - 1, 0)).cuda().long()
        query = q_out[last]
        for window, sinks in ((0, 0), (100, 3)):
            args = (indptr, lens.astype(np.int32), heads, kv_heads, dim, q.CACHE_E4M3)
            ws = torch.empty(max(256, q.gqa_decode_plan(*args, window=window, sinks=sinks).workspace_bytes), dtype=torch.uint8, device="cuda")
            p = q.gqa_decode_plan(*args, window=window, sinks=sinks, workspace=ws)
            out, lse = torch.empty_like(query), torch.empty((batch, heads), device="cuda")
            q.gqa_decode_run(p, query, dcodes, dscale, dids, 0.125, out, lse, ws)
            torch.cuda.synchronize()
            ref = R.attend(R.bf16_to_f32(query), codes, scale, R.E4M3, indptr, ids, lens, 0.125, window, sinks)
            R.check_attend(out, lse, ref, int(lens.max()), dim)


@pytest.mark.parametrize("kv", [q.KV_FP8_E4M3, q.KV_NVFP4, q.KV_FP8_PER_TOKEN])
def test_latent_append_then_mla_decode(qkvp, kv):
    """The latent path in one run: rotate, quantize and append every token, rotate the query into q, decode;
    against the FP64 oracle on a pool appended from the same rows by the oracle."""
    import oracle
    rng = np.random.default_rng(40)
    lens, heads = [130, 64, 5], 16
    w = synth.build_workload("latent_rope", lens, heads=heads, pool_pages=8, seed=3, device="cuda")
    n = sum(lens)
    cs = R.table(4000, 64)
    pos = np.concatenate([1000 * r + np.arange(m) for r, m in enumerate(lens)])
    slots = w.slots.cpu().numpy()
    c_kv, k_pe = (R.to_bf16(rng.standard_normal((n, d)).astype(np.float32)) for d in (512, 64))
    q_pe = R.to_bf16(rng.standard_normal((3, heads, 64)).astype(np.float32))
    width = {q.KV_FP8_E4M3: (64, 576), q.KV_NVFP4: (64, 288), q.KV_FP8_PER_TOKEN: (q.PAGE_BYTES_FP8_PER_TOKEN,)}[kv]
    pool = torch.full((w.num_pages, *width), 0xFF, dtype=torch.uint8, device="cuda")
    scale = torch.full((w.num_pages, 64, 36), 0x7F, dtype=torch.uint8, device="cuda") if kv == q.KV_NVFP4 else None
    dcs = torch.from_numpy(cs).cuda()
    at = np.concatenate([[0], np.cumsum(lens)])
    last = at[1:] - 1
    query = w.q.clone()
    keep = np.setdiff1d(np.arange(n), last)
    for rows, qp, qb in ((keep, None, None), (last, q_pe.cuda(), query)):
        idx = torch.from_numpy(rows)
        q.mla_append_rope(c_kv[idx].cuda(), k_pe[idx].cuda(), torch.from_numpy(slots[rows]).cuda(), torch.from_numpy(pos[rows]).cuda(), dcs, q.ROPE_PAIRS,
                          pool, scale, kv, q_pe=qp, q=qb)
    plan = q.mla_decode_plan(w.kv_indptr, w.kv_len, heads, kv)
    ws = torch.empty(max(plan.workspace_bytes, 256), dtype=torch.uint8, device="cuda")
    plan = q.mla_decode_plan(w.kv_indptr, w.kv_len, heads, kv, workspace=ws)
    out, lse = torch.empty((3, heads, 512), dtype=torch.bfloat16, device="cuda"), torch.empty((3, heads), device="cuda")
    q.mla_decode_run(plan, query, pool, scale, w.num_pages, torch.from_numpy(w.kv_indices).cuda(), w.sm_scale, 1.0, out, lse, ws)
    torch.cuda.synchronize()
    # the oracle attends the appended bytes; the rotation and codes themselves are held bit for bit elsewhere
    qb = w.q.cpu().clone()
    for r in range(3):
        qb[r, :, 512:] = R.to_bf16(R.rotate(R.bf16_to_f32(q_pe[r]), cs[pos[last[r]]], R.PAIRS))
    assert torch.equal(query.cpu().view(torch.int16), qb.view(torch.int16))
    hp = (pool.cpu().numpy(), scale.cpu().numpy() if scale is not None else None)
    o_ref, l_ref = oracle.mla_decode(qb.view(torch.int16).numpy().view(np.uint16), hp[0], hp[1], kv, 64, w.num_pages, w.kv_indptr, w.kv_indices,
                                     w.kv_len, w.sm_scale, 1.0)
    compare(out.float().cpu().numpy().reshape(-1, 512), lse.cpu().numpy().reshape(-1), o_ref, l_ref, raw=True)
