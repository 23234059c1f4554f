"""Attention of drafted tokens over a head pool, against 64 bits."""
import numpy as np
import pytest
import torch

import quantized_kv_paged_gb300 as q
from tests import heads_ref as R
from tests.tree_ref import Batch

pytestmark = pytest.mark.gpu

# (cached, drafted, heads, KV heads, dim): from one token to lengths that cross pages anywhere, 1 to 600 rows on a KV head
SHAPES = [
    ([0], [1], 1, 1, 64),
    ([5], [3], 4, 2, 128),
    ([63, 64, 65], [1, 2, 7], 8, 2, 64),
    ([60, 0, 700, 64], [9, 33, 1, 64], 8, 4, 128),
    ([130, 3], [40, 70], 7, 1, 128),
    ([300, 0, 127], [5, 66, 31], 6, 3, 256),
    ([1000, 513], [20, 130], 10, 2, 64),
    ([200, 90, 0], [64, 256, 100], 4, 2, 128),
    ([2500], [37], 16, 1, 128),
    ([0, 64, 0], [0, 2, 0], 2, 2, 128),
]


def check(b, out, lse, ref):
    return R.check_attend(out, lse, ref, int(b.lens.max()) + 64, b.dims[2])


@pytest.mark.parametrize("cache", [q.CACHE_E4M3, q.CACHE_INT8])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_trees(qkvp, shape, cache):
    cached, drafted, heads, kv_heads, dim = shape
    b = Batch(len(cached) * 7 + dim, cached, drafted, heads, kv_heads, dim, cache, extra_words=1)
    out, lse, _ = b.run(q, dim ** -0.5)
    check(b, out, lse, b.reference(dim ** -0.5))


@pytest.mark.parametrize("shape", SHAPES[2:8], ids=str)
def test_chains_and_masks_of_chains(qkvp, shape):
    cached, drafted, heads, kv_heads, dim = shape
    b = Batch(3, cached, drafted, heads, kv_heads, dim, q.CACHE_E4M3, chain=True)
    out, lse, _ = b.run(q, 0.1, chain=True)
    check(b, out, lse, b.reference(0.1))
    again, lse2, _ = b.run(q, 0.1)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16)) and torch.equal(lse, lse2)


@pytest.mark.parametrize("splits", [3, 17, 60])
@pytest.mark.parametrize("heads,kv_heads,dim,drafted", [(4, 1, 128, 9), (8, 2, 64, 50), (3, 1, 256, 50), (10, 2, 128, 40)])
def test_splits_and_joins(qkvp, splits, heads, kv_heads, dim, drafted):
    b = Batch(splits, [3900, 1], [drafted, drafted], heads, kv_heads, dim, q.CACHE_INT8)
    out, lse, plan = b.run(q, dim ** -0.5, min_splits=splits)
    assert plan.num_joins > 0
    check(b, out, lse, b.reference(dim ** -0.5))


@pytest.mark.parametrize("window,sinks", [(40, 0), (64, 4), (100, 70), (200, 1), (1000, 130), (10 ** 9, 5), (2 ** 31 - 1, 2 ** 31 - 1)])
@pytest.mark.parametrize("heads,kv_heads,dim,cache", [(8, 2, 64, q.CACHE_INT8), (4, 1, 128, q.CACHE_E4M3), (2, 1, 256, q.CACHE_E4M3)])
def test_windows(qkvp, window, sinks, heads, kv_heads, dim, cache):
    b = Batch(window % 1000 + sinks % 1000, [700, 64, 0, 333, 190], [40, 1, 17, 40, 39], heads, kv_heads, dim, cache)
    out, lse, _ = b.run(q, dim ** -0.5, window=window, sinks=sinks)
    check(b, out, lse, b.reference(dim ** -0.5, window, sinks))


def test_window_of_a_chain_of_one_is_the_decode(qkvp):
    """One drafted token a request is the decode's question: the same tokens, the same formulas."""
    b = Batch(5, [700, 64, 0, 333], [1, 1, 1, 1], 8, 2, 128, q.CACHE_E4M3, chain=True)
    for kw in (dict(), dict(window=100, sinks=7)):
        out, lse, _ = b.run(q, 0.09, chain=True, **kw)
        ref = R.attend(R.bf16_to_f32(b.q), b.codes, b.scale, b.cache, b.indptr, b.ids, b.lens, 0.09, **kw)
        check(b, out, lse, ref)


@pytest.mark.parametrize("cached", [0, 70])
def test_rows_that_see_nothing(qkvp, cached):
    """Drafted tokens whose mask is empty: with nothing cached their rows are 0 and -inf."""
    b = Batch(11, [cached, cached], [40, 5], 8, 2, 128, q.CACHE_E4M3, empty=0.5)
    assert any(not p for p in b.paths)
    out, lse, _ = b.run(q, 0.1)
    check(b, out, lse, b.reference(0.1))


@pytest.mark.parametrize("sm_scale", [-0.2, 0.0, 3.0])
def test_scales_of_any_sign(qkvp, sm_scale):
    b = Batch(12, [130, 20], [9, 30], 8, 2, 64, q.CACHE_INT8)
    out, lse, _ = b.run(q, sm_scale)
    check(b, out, lse, b.reference(sm_scale))


def test_bad_pages_are_not_seen(qkvp):
    b = Batch(13, [500, 100], [12, 40], 8, 2, 128, q.CACHE_E4M3)
    b.ids[[1, 4]] = [-1, b.pages]
    b.ids[-2] = 2 ** 31 - 1
    out, lse, _ = b.run(q, 0.1)
    check(b, out, lse, b.reference(0.1))


@pytest.mark.parametrize("window", [0, 64])
@pytest.mark.parametrize("splits", [0, 9])
def test_nan_where_it_is_not_seen(qkvp, splits, window):
    """NaN codes in K and V of a drafted token reach the rows that see it and no other; unused slots hold NaN, too."""
    b = Batch(14, [200, 63], [30, 20], 8, 2, 128, q.CACHE_E4M3)
    clean = b.reference(0.1, window, 4 if window else 0)

    def slot(r, t):
        return int(b.ids[b.indptr[r] + t // 64]), t % 64
    # behind the last token, and the pages that no request has
    for r in range(2):
        page, off = slot(r, int(b.lens[r]) - 1)
        b.codes[page, :, :, off + 1:] = 0x7F
    used = {int(b.ids[b.indptr[r] + p]) for r in range(2) for p in range((int(b.lens[r]) + 63) // 64)}
    for page in set(range(b.pages)) - used:
        b.codes[page], b.scale[page] = 0xFF, np.nan
    # V of drafted token 7 of request 0 in one dim, K of token 11
    page, off = slot(0, 207)
    b.codes[page, 1, 0, off, 5] = 0x7F
    page, off = slot(0, 211)
    b.codes[page, 0, 1, off, 9] = 0xFF
    out, lse, _ = b.run(q, 0.1, min_splits=splits, window=window, sinks=4 if window else 0)
    o, l = out.float().cpu(), lse.cpu()
    for i, path in enumerate(b.paths[:30]):
        v_bad, k_bad = 7 in path, 11 in path
        assert torch.isnan(o[i, :4, 5]).all() == v_bad and not torch.isnan(o[i, :4, :5]).any() and not torch.isnan(o[i, :4, 6:]).any()
        assert torch.isnan(o[i, 4:]).all() == k_bad and torch.isnan(o[i, 4:]).any() == k_bad and torch.isnan(l[i, 4:]).all() == k_bad
    # every other row as without them
    bad = np.array([7 in p or 11 in p for p in b.paths[:30]] + [False] * 20)
    keep = np.nonzero(~bad)[0]
    R.check_attend(out[torch.from_numpy(keep).cuda()], lse[torch.from_numpy(keep).cuda()], tuple(x[keep] for x in clean), 400, 128)


@pytest.mark.parametrize("apart", [4, 30, 100])
def test_v_scales_far_apart(qkvp, apart):
    """V's scales 2^apart from page to page, growing, shrinking and mixed, with pages of zeros between them."""
    rng = np.random.default_rng(apart)
    for order in range(3):
        b = Batch(15 + order, [500], [30], 8, 2, 128, q.CACHE_INT8)
        n = int(b.indptr[-1])
        e = np.linspace(-apart / 2, apart / 2, n)
        e = e if order == 0 else e[::-1] if order == 1 else rng.permutation(e)
        b.scale[b.ids, 1] = np.exp2(np.round(e)).astype(np.float32)[:, None] * b.scale[b.ids, 1]
        if order == 2:
            b.scale[b.ids[3], 1] = 0
        # logits that make up for it: the largest weights lie in the pages of the smallest scales
        b.scale[b.ids, 0] *= np.float32(1.0)
        out, lse, _ = b.run(q, 0.05)
        check(b, out, lse, b.reference(0.05))


def test_zero_scales(qkvp):
    b = Batch(16, [130], [20], 8, 2, 128, q.CACHE_E4M3)
    b.scale[b.ids[0]] = 0
    b.scale[b.ids[2], 0] = 0
    out, lse, _ = b.run(q, 0.1)
    check(b, out, lse, b.reference(0.1))
    b.scale[:] = 0
    out, lse, _ = b.run(q, 0.1)
    assert (out == 0).all()


def test_large_and_tiny_queries(qkvp):
    b = Batch(17, [130], [20], 8, 2, 128, q.CACHE_INT8)
    b.q[:, 0] *= 2.0 ** 20
    b.q[:, 3] *= 2.0 ** -30
    b.q[:, 5] = 0
    out, lse, _ = b.run(q, 2.0 ** -18)
    check(b, out, lse, b.reference(2.0 ** -18))


def test_without_lse_and_on_another_stream(qkvp):
    b = Batch(18, [900, 7], [30, 3], 8, 2, 128, q.CACHE_E4M3)
    want, _, _ = b.run(q, 0.1)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        out, _, _ = b.run(q, 0.1, lse=False)
    assert torch.equal(out.view(torch.int16), want.view(torch.int16))


def test_captured_and_replayed(qkvp):
    """A captured step replays over new queries, masks and cache contents, bit for bit the eager call."""
    b = Batch(19, [900, 77], [33, 50], 8, 2, 128, q.CACHE_E4M3)
    plan, ws = b.plan(q)
    n = int(b.tok[-1])
    mask, ids = torch.from_numpy(b.mask.view(np.int32)).cuda(), torch.from_numpy(b.ids).cuda()
    codes, scale, qq = torch.from_numpy(b.codes).cuda(), torch.from_numpy(b.scale).cuda(), b.q.cuda()
    out, lse = torch.empty_like(qq), torch.empty((n, 8), device="cuda")

    def call():
        q.gqa_tree_run(plan, qq, codes, scale, ids, mask, 0.1, out, lse, ws)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for i in range(3):
        qq.copy_(torch.randn(qq.shape, generator=torch.Generator(device="cuda").manual_seed(i), device="cuda"))
        mask[5] = mask[7 + i]
        scale.mul_(1.25)
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone(), lse.clone()
        out.zero_()
        call()
        torch.cuda.synchronize()
        assert torch.equal(got[0].view(torch.int16), out.view(torch.int16)) and torch.equal(got[1], lse)


@pytest.mark.parametrize("sms", [1, 2, 5])
@pytest.mark.parametrize("heads,kv_heads,dim,window", [(8, 2, 128, 0), (8, 4, 64, 300), (3, 1, 256, 0)])
def test_few_workers_with_many_segments(qkvp, sms, heads, kv_heads, dim, window):
    """One worker goes through segments of every kind: 1 to 128 rows, one to many pages, split ones and whole ones."""
    b = Batch(20 + sms, [700, 3, 0, 64, 129, 1500, 1, 63], [40, 1, 64, 33, 2, 7, 150, 65], heads, kv_heads, dim, q.CACHE_E4M3, empty=0.1)
    for splits in (0, 30):
        out, lse, plan = b.run(q, dim ** -0.5, window=window, sinks=5 if window else 0, num_sms=sms, min_splits=splits)
        assert plan.num_workers == sms
        check(b, out, lse, b.reference(dim ** -0.5, window, 5 if window else 0))


def test_queries_that_hold_no_number_stay_in_their_rows(qkvp):
    """The other rows are as near to 64 bits as ever. (Not the same bits: rows of a warp share the choice of when their
    running maximum is renewed, which moves roundings.)"""
    b = Batch(21, [200, 30], [20, 9], 8, 2, 128, q.CACHE_E4M3)
    ref = b.reference(0.1)
    b.q[3, 2, 5], b.q[7, 0, 0], b.q[28, 7, 127] = float("nan"), float("inf"), float("-inf")
    out, lse, _ = b.run(q, 0.1)
    bad = np.zeros(lse.shape, bool)
    bad[3, 2] = bad[7, 0] = bad[28, 7] = True
    assert not torch.isfinite(lse.cpu()[torch.from_numpy(bad)]).any()
    keep = torch.from_numpy(~bad).cuda()
    R.check_attend(out[keep], lse[keep], tuple(x[~bad] for x in ref), int(b.lens.max()) + 64, 128)


def test_mask_bits_behind_the_last_drafted_token_do_not_count(qkvp):
    b = Batch(22, [100, 64, 0], [5, 40, 33], 4, 2, 64, q.CACHE_INT8, extra_words=2)
    want, lse, _ = b.run(q, 0.1)
    for r, n in enumerate(b.drafted):
        for i in range(b.tok[r], b.tok[r + 1]):
            for k in range(n, 32 * b.words):
                b.mask[i, k // 32] |= np.uint32(1 << (k % 32))
    out, lse2, _ = b.run(q, 0.1)
    assert torch.equal(out.view(torch.int16), want.view(torch.int16)) and torch.equal(lse2, lse)


def test_pages_past_32_bits(qkvp):
    """A pool of 5 GB whose used pages begin behind 2^32 bytes, decoded, committed and copied."""
    b = Batch(23, [300, 90], [20, 33], 16, 8, 128, q.CACHE_E4M3, spare=3)
    pages, first = 40000, 40000 - b.pages
    codes, scale = torch.zeros((pages, 2, 8, 64, 128), dtype=torch.uint8, device="cuda"), torch.zeros((pages, 2, 8), device="cuda")
    codes[first:], scale[first:] = torch.from_numpy(b.codes), torch.from_numpy(b.scale)
    assert first * codes[0].numel() > 2 ** 32
    want, want_lse, _ = b.run(q, 0.1)
    plan, ws = b.plan(q)
    out, lse, ids = torch.zeros_like(want), torch.zeros_like(want_lse), torch.from_numpy(b.ids + first).to(torch.int32).cuda()
    q.gqa_tree_run(plan, b.q.cuda(), codes, scale, ids, torch.from_numpy(b.mask.view(np.int32)).cuda(), 0.1, out, lse, ws)
    assert torch.equal(out.view(torch.int16), want.view(torch.int16)) and torch.equal(lse, want_lse)
    from tests import tree_ref as T
    i32 = lambda x: torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()          # noqa: E731
    path, n = np.array([[0, 3, 5, 19], [1, 2, 30, 0]]), np.array([4, 3])
    q.gqa_tree_commit([codes], [scale], b.cache, i32(b.cached), i32(b.indptr), ids, i32(path), i32(n))
    T.commit(b.codes, b.scale, b.cache, b.cached, b.indptr, b.ids, path, n)
    assert np.array_equal(codes[first:].cpu().numpy(), b.codes) and np.array_equal(scale[first:].cpu().numpy(), b.scale)
    q.kv_pages_copy([codes, scale], i32([pages - 1, first]), i32([1, pages - 2]))
    assert np.array_equal(codes[1].cpu().numpy(), b.codes[-1]) and np.array_equal(codes[pages - 2].cpu().numpy(), b.codes[0])
    assert not codes[2:first].any()


def test_two_streams_at_once(qkvp):
    jobs = [Batch(24 + i, [900, 77, 1300], [33, 50, 64], 8, 2, 128, q.CACHE_E4M3) for i in range(2)]
    want = [b.run(q, 0.1)[:2] for b in jobs]
    streams, held = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for b in jobs:
        plan, ws = b.plan(q)
        held.append((plan, b.q.cuda(), torch.from_numpy(b.codes).cuda(), torch.from_numpy(b.scale).cuda(), torch.from_numpy(b.ids).cuda(),
                     torch.from_numpy(b.mask.view(np.int32)).cuda(), ws))
    outs = [(torch.zeros_like(o), torch.zeros_like(l)) for o, l in want]
    torch.cuda.synchronize()
    for _ in range(4):
        for s, (plan, qq, codes, scale, ids, mask, ws), (o, l) in zip(streams, held, outs):
            q.gqa_tree_run(plan, qq, codes, scale, ids, mask, 0.1, o, l, ws, stream=s.cuda_stream)
    torch.cuda.synchronize()
    for (o, l), (wo, wl) in zip(outs, want):
        assert torch.equal(o.view(torch.int16), wo.view(torch.int16)) and torch.equal(l, wl)


@pytest.mark.parametrize("cache", [q.CACHE_E4M3, q.CACHE_INT8])
@pytest.mark.parametrize("cached,drafted,heads,kv_heads,dim,copies", [
    ([8000, 7001], [4, 1], 8, 1, 128, 4), ([4000], [1], 1, 1, 64, 4), ([4001, 3444, 2555], [9, 16, 0], 4, 2, 64, 4), ([14900], [32], 1, 1, 256, 4),
    ([12000, 12097], [9, 3], 8, 2, 128, 2), ([5000, 4600], [33, 2], 1, 1, 64, 2), ([5000], [8], 16, 2, 64, 2), ([5000], [13], 10, 2, 64, 1),
    ([14800], [12], 10, 2, 256, 1)])
def test_copies_of_few_rows(qkvp, cached, drafted, heads, kv_heads, dim, copies, cache):
    b = Batch(30 + dim + copies, cached, drafted, heads, kv_heads, dim, cache, empty=0.1)
    for kw, splits in ((dict(), dict(num_sms=1)), (dict(), dict(num_sms=2)), (dict(), dict(num_sms=1, min_splits=2)),
                       (dict(window=max(cached) - 70, sinks=70), dict(num_sms=1))):
        out, lse, plan = b.run(q, dim ** -0.5, **kw, **splits)
        assert plan.row_copies == copies, (plan.total_pages, plan.num_segments)
        check(b, out, lse, b.reference(dim ** -0.5, **kw))
    out, lse, plan = b.run(q, dim ** -0.5, min_splits=40)
    assert plan.row_copies == 1                # short segments
    check(b, out, lse, b.reference(dim ** -0.5))


@pytest.mark.parametrize("drafted,dim", [(6, 128), (12, 64)])
def test_copies_of_few_rows_with_nan_and_v_scales_far_apart(qkvp, drafted, dim):
    """A NaN V code reaches the rows that see it whichever copy has the token, V's scales differ within a copy's tokens, and
    rows that see nothing but a few tokens have copies that see none."""
    b = Batch(40 + drafted, [4800], [drafted], 4, 1, dim, q.CACHE_E4M3, chain=True)
    rng = np.random.default_rng(drafted)
    b.scale[b.ids, 1] *= np.exp2(rng.integers(-40, 41, len(b.ids))).astype(np.float32)[:, None]
    want = b.reference(0.1)
    out, lse, plan = b.run(q, 0.1, num_sms=1)
    assert plan.row_copies > 1
    check(b, out, lse, want)
    page, off = int(b.ids[4802 // 64]), 4802 % 64
    b.codes[page, 1, 0, off, 5] = 0x7F
    out, lse, _ = b.run(q, 0.1, num_sms=1)
    o = out.float().cpu()
    assert torch.isnan(o[2:, :, 5]).all() and not torch.isnan(o[:2]).any() and not torch.isnan(o[2:, :, :5]).any() and not torch.isnan(o[2:, :, 6:]).any()
    keep = torch.arange(2).cuda()
    R.check_attend(out[keep], lse[keep], tuple(x[:2] for x in want), 4900, dim)
    few = Batch(44, [4800], [drafted], 4, 1, dim, q.CACHE_INT8)
    few.ids[:75] = -1                          # pages outside the pool: the drafted tokens alone are left
    out, lse, plan = few.run(q, 0.1, num_sms=1)
    assert plan.row_copies > 1
    check(few, out, lse, few.reference(0.1))


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_pools_on_16_byte_boundaries(qkvp, dim):
    """Codes need 16-byte alignment and no more; the bits are those of a pool on a larger boundary."""
    b = Batch(60 + dim, [700, 5, 64], [20, 3, 40], 4, 2, dim, q.CACHE_E4M3)
    want, lse, _ = b.run(q, 0.1)
    plan, ws = b.plan(q)
    flat = torch.zeros(b.codes.size + 64, dtype=torch.uint8, device="cuda")
    codes = flat[16:16 + b.codes.size].view(b.codes.shape)
    assert codes.data_ptr() % 32 == 16
    codes.copy_(torch.from_numpy(b.codes))
    out, lse2 = torch.zeros_like(want), torch.zeros_like(lse)
    q.gqa_tree_run(plan, b.q.cuda(), codes, torch.from_numpy(b.scale).cuda(), torch.from_numpy(b.ids).cuda(), torch.from_numpy(b.mask.view(np.int32)).cuda(),
                   0.1, out, lse2, ws)
    assert torch.equal(out.view(torch.int16), want.view(torch.int16)) and torch.equal(lse2, lse)
