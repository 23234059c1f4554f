"""The rotated appends' and the head-pool decode's argument checks and plans, without a GPU."""
import ctypes

import numpy as np
import pytest
import torch

import quantized_kv_paged_gb300 as q


@pytest.fixture(scope="module")
def lib():
    from quantized_kv_paged_gb300 import build
    build.build()
    return q.load()


def plan(indptr, lens, heads=32, kv_heads=8, dim=128, cache=q.CACHE_E4M3, sms=152, **kw):
    return q.gqa_decode_plan(np.asarray(indptr, np.int32), np.asarray(lens, np.int32), heads, kv_heads, dim, cache,
                             num_sms=sms, raise_on_error=False, **kw)


def table(lens, spare=0):
    return np.concatenate([[0], np.cumsum([(n + 63) // 64 + spare for n in lens])]).astype(np.int32)


def test_plan_refuses_bad_arguments(lib):
    lens = [100]
    ptr = table(lens)
    assert plan(ptr, lens).status == q.QKVP_OK
    for kw, want in ((dict(dim=96), q.QKVP_E_UNSUPPORTED), (dict(cache=3), q.QKVP_E_UNSUPPORTED),
                     (dict(heads=30), q.QKVP_E_UNSUPPORTED), (dict(heads=0), q.QKVP_E_UNSUPPORTED),
                     (dict(kv_heads=0), q.QKVP_E_UNSUPPORTED), (dict(kv_heads=257, heads=257), q.QKVP_E_UNSUPPORTED),
                     (dict(page_size=32), q.QKVP_E_UNSUPPORTED), (dict(window=-1), q.QKVP_E_INVALID),
                     (dict(window=4, sinks=-1), q.QKVP_E_INVALID), (dict(sinks=4), q.QKVP_E_INVALID),
                     (dict(min_splits=-1), q.QKVP_E_INVALID)):
        assert plan(ptr, lens, **kw).status == want, kw
    assert plan([1, 3], lens).status == q.QKVP_E_INVALID
    assert plan([0, 1], lens).status == q.QKVP_E_INVALID          # 100 tokens on one page
    assert plan([0, 2], [-1]).status == q.QKVP_E_INVALID
    with pytest.raises(ValueError):
        plan([0, 2], [5, 5])


@pytest.mark.parametrize("length,window,sinks,pages,tokens", [
    (0, 0, 0, 0, 0), (1, 0, 0, 1, 1), (64, 0, 0, 1, 64), (65, 0, 0, 2, 65),
    (1000, 1000, 0, 16, 1000), (1000, 999, 0, 16, 999), (1000, 1, 0, 1, 1), (1000, 40, 0, 1, 40),
    (1000, 41, 0, 2, 41), (1000, 1, 1, 2, 2), (1000, 1, 64, 2, 65), (1000, 1, 65, 3, 66),
    (1000, 100, 5000, 16, 1000), (1000, 900, 99, 16, 999), (1000, 900, 100, 16, 1000), (129, 2, 128, 3, 129),
    (40, 10, 3, 1, 13), (200, 2 ** 31 - 1, 7, 4, 200)])
def test_plan_counts_visible_pages_and_tokens(lib, length, window, sinks, pages, tokens):
    p = plan(table([length]), [length], heads=4, kv_heads=2, window=window, sinks=sinks)
    assert p.status == q.QKVP_OK and (p.total_pages, p.total_tokens) == (pages, tokens)
    assert p.num_segments >= 2


def test_plan_balances_and_sizes(lib):
    lens = [32768] * 44
    p = plan(table(lens), lens, heads=64)
    assert p.total_tokens == 44 * 32768 and p.total_pages == 44 * 512
    mean = p.total_pages * 8 / p.num_workers
    assert mean <= p.max_worker_pages <= 1.1 * mean
    assert p.num_partials <= 2 * p.num_workers + 44 * 8
    assert p.workspace_bytes >= p.table_bytes + p.num_partials * 16 * (128 + 1) * 4
    one = plan([0, 16384], [1 << 20], heads=32, kv_heads=4, min_splits=1000)
    assert one.num_segments >= 1000 and one.num_split_groups == 4
    many = plan(table([64]), [64], heads=40, kv_heads=1)          # three passes of 16, 16 and 8 heads
    assert many.num_segments == 3
    none = plan([0], [])
    assert none.status == q.QKVP_OK and none.num_segments == 0


def test_plan_reports_the_workspace_it_needs(lib):
    lens = np.array([5000], np.int32)
    ptr, p = table(lens), q.gqa_plan()
    st = lib.gqa_decode_plan(ptr.ctypes.data, lens.ctypes.data, 1, 32, 8, 128, 64, 1, 0, 0, 152, 0, ctypes.c_void_p(256),
                             64, None, ctypes.byref(p))
    assert st == q.QKVP_E_WORKSPACE and p.workspace_bytes > 64 and p.magic == 0


def test_run_refuses_before_any_launch(lib):
    L = lib
    p = plan(table([100]), [100])
    ok = dict(plan=ctypes.byref(p), q=16, kv=128, scale=16, pages=4, idx=16, sm=0.1, out=16, lse=4, ws=256, n=1 << 30)

    def run(**kw):
        a = dict(ok, **kw)
        return L.gqa_decode_run(a["plan"], a["q"], a["kv"], a["scale"], a["pages"], a["idx"], a["sm"], a["out"], a["lse"], a["ws"], a["n"], None)

    assert run() == q.QKVP_E_INVALID                               # a size query is no plan: nothing was uploaded
    p.magic = 0x716b76702d677161
    for kw, want in ((dict(plan=None), q.QKVP_E_INVALID), (dict(ws=None), q.QKVP_E_WORKSPACE), (dict(n=8), q.QKVP_E_WORKSPACE),
                     (dict(ws=128), q.QKVP_E_WORKSPACE), (dict(q=None), q.QKVP_E_INVALID), (dict(q=8), q.QKVP_E_INVALID),
                     (dict(out=None), q.QKVP_E_INVALID), (dict(out=8), q.QKVP_E_INVALID), (dict(lse=2), q.QKVP_E_INVALID),
                     (dict(kv=None), q.QKVP_E_INVALID), (dict(kv=64), q.QKVP_E_INVALID), (dict(scale=None), q.QKVP_E_INVALID),
                     (dict(scale=2), q.QKVP_E_INVALID), (dict(idx=None), q.QKVP_E_INVALID), (dict(pages=-1), q.QKVP_E_INVALID),
                     (dict(sm=float("nan")), q.QKVP_E_INVALID), (dict(sm=float("inf")), q.QKVP_E_INVALID),
                     (dict(pages=1 << 40), q.QKVP_E_UNSUPPORTED)):
        assert run(**kw) == want, kw


GQA = dict(k=16, ks=256, v=16, vs=256, n=4, tok=4, klen=4, batch=1, ptr=4, idx=4, nnz=9, pos=None, cs=16, mp=100, rot=64, style=0,
           hk=2, d=128, kv=16, sc=4, cache=1, ps=64, pages=9, q=16, qs=512, h=4, qo=32)


@pytest.mark.parametrize("kw,want", [
    (dict(n=-1), "I"), (dict(batch=-1), "I"), (dict(nnz=-1), "I"), (dict(pages=-1), "I"), (dict(mp=-1), "I"), (dict(h=-1), "I"),
    (dict(d=80), "U"), (dict(cache=0), "U"), (dict(ps=16), "U"), (dict(hk=0), "U"), (dict(hk=257), "U"), (dict(style=2), "U"),
    (dict(rot=8), "U"), (dict(rot=144), "U"), (dict(rot=-16), "U"), (dict(rot=0), "I"), (dict(cs=None), "I"), (dict(cs=8), "I"),
    (dict(k=None), "I"), (dict(k=8), "I"), (dict(ks=248), "I"), (dict(ks=260), "I"), (dict(v=None), "I"), (dict(vs=255), "I"),
    (dict(tok=None), "I"), (dict(klen=None), "I"), (dict(ptr=None), "I"), (dict(idx=None), "I"), (dict(kv=None), "I"), (dict(kv=8), "I"),
    (dict(sc=None), "I"), (dict(pos=4), "I"), (dict(q=None), "I"), (dict(qo=None), "I"), (dict(h=0), "I"), (dict(q=8), "I"),
    (dict(qs=504), "I"), (dict(q=32, qs=1024), "I"), (dict(n=1 << 40), "U"), (dict(mp=1 << 40), "U"), (dict(pages=1 << 60), "I")])
def test_gqa_append_refusals(lib, kw, want):
    a = dict(GQA, **kw)
    st = lib.gqa_append_rope(a["k"], a["ks"], a["v"], a["vs"], a["n"], a["tok"], a["klen"], a["batch"], a["ptr"], a["idx"], a["nnz"],
                             a["pos"], a["cs"], a["mp"], a["rot"], a["style"], a["hk"], a["d"], a["kv"], a["sc"], a["cache"], a["ps"],
                             a["pages"], a["q"], a["qs"], a["h"], a["qo"], None)
    assert st == {"I": q.QKVP_E_INVALID, "U": q.QKVP_E_UNSUPPORTED}[want]


MLA = dict(c=16, cs=512, p=16, ps=576, n=4, slot=8, pos=8, tab=16, mp=9, style=1, qp=16, qt=4096, qh=128, h=16, q=32, kv=16, sc=None,
           dt=1, g=1.0, page=64, pages=4)


@pytest.mark.parametrize("kw,want", [
    (dict(n=-1), "I"), (dict(pages=-1), "I"), (dict(mp=-1), "I"), (dict(h=-1), "I"), (dict(dt=3), "U"), (dict(style=5), "U"),
    (dict(page=32), "U"), (dict(sc=16), "I"), (dict(g=2.0), "I"), (dict(dt=2), "I"), (dict(dt=2, sc=16, g=0.0), "I"),
    (dict(dt=2, sc=16, g=float("inf")), "I"), (dict(dt=2, sc=8), "I"), (dict(qp=None), "I"), (dict(q=None), "I"), (dict(h=0), "I"),
    (dict(c=None), "I"), (dict(c=8), "I"), (dict(cs=504), "I"), (dict(cs=516), "I"), (dict(p=None), "I"), (dict(ps=56), "I"),
    (dict(ps=65), "I"), (dict(slot=None), "I"), (dict(slot=4), "I"), (dict(pos=None), "I"), (dict(tab=None), "I"), (dict(tab=8), "I"),
    (dict(kv=None), "I"), (dict(kv=8), "I"), (dict(q=8), "I"), (dict(qt=4097), "I"), (dict(qh=60), "I"), (dict(h=5000), "U")])
def test_mla_append_refusals(lib, kw, want):
    a = dict(MLA, **kw)
    st = lib.mla_append_rope(a["c"], a["cs"], a["p"], a["ps"], a["n"], a["slot"], a["pos"], a["tab"], a["mp"], a["style"], a["qp"], a["qt"],
                             a["qh"], a["h"], a["q"], a["kv"], a["sc"], a["dt"], a["g"], a["page"], a["pages"], None)
    assert st == {"I": q.QKVP_E_INVALID, "U": q.QKVP_E_UNSUPPORTED}[want]


def test_nothing_to_do_is_fine(lib):
    a = dict(GQA, n=0)
    assert lib.gqa_append_rope(a["k"], a["ks"], a["v"], a["vs"], 0, a["tok"], a["klen"], 1, a["ptr"], a["idx"], 9, None, a["cs"], 100, 64, 0, 2,
                               128, a["kv"], a["sc"], 1, 64, 9, a["q"], 512, 4, a["qo"], None) == q.QKVP_OK
    assert lib.mla_append_rope(16, 512, 16, 576, 0, 8, 8, 16, 9, 1, None, 0, 0, 0, None, 16, None, 1, 1.0, 64, 4, None) == q.QKVP_OK


def test_binding_refuses_wrong_tensors(lib):
    """Shapes, types and layouts are checked before devices, so CPU tensors show each check's own error; right
    ones are refused for not being on the GPU."""
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)          # noqa: E731
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)            # noqa: E731
    pool, scale = torch.zeros((4, 2, 2, 64, 128), dtype=torch.uint8), torch.zeros((4, 2, 2))
    cs = torch.zeros((10, 64))
    good = dict(k=bf(3, 2, 128), v=bf(3, 2, 128), tok_indptr=i32(2), kv_len=i32(1), kv_indptr=i32(2), kv_indices=i32(4), cos_sin=cs,
                rope_style=q.ROPE_HALVES, kv_data=pool, kv_scale=scale, cache_dtype=q.CACHE_E4M3)
    with pytest.raises(ValueError, match="current CUDA device"):
        q.gqa_append_rope(**good)
    for kw in (dict(k=bf(3, 2, 64)), dict(k=torch.zeros((3, 2, 128))), dict(v=bf(4, 2, 128)), dict(v=bf(3, 128, 2).transpose(1, 2)),
               dict(k=bf(3, 4, 128)[:, ::2]), dict(tok_indptr=i32(3)), dict(kv_len=torch.zeros(1, dtype=torch.int64)),
               dict(kv_scale=scale[:2]), dict(kv_data=pool[:, :, :, :32]), dict(cos_sin=cs.double()), dict(cos_sin=cs.T),
               dict(positions=torch.zeros(3, dtype=torch.int32)), dict(q=bf(3, 4, 128)), dict(q=bf(2, 4, 128), q_out=bf(3, 4, 128)),
               dict(q=bf(3, 4, 128), q_out=bf(3, 8, 128)[:, ::2])):
        with pytest.raises(ValueError) as e:
            q.gqa_append_rope(**dict(good, **kw))
        assert "current CUDA device" not in str(e.value), kw
    mla = dict(c_kv=bf(3, 512), k_pe=bf(3, 576)[:, 512:], slot_mapping=torch.zeros(3, dtype=torch.int64),
               positions=torch.zeros(3, dtype=torch.int64), cos_sin=cs, rope_style=q.ROPE_PAIRS,
               kv_data=torch.zeros((2, 64, 576), dtype=torch.uint8), kv_scale=None, kv_dtype=q.KV_FP8_E4M3)
    with pytest.raises(ValueError, match="current CUDA device"):
        q.mla_append_rope(**mla)
    for kw in (dict(c_kv=bf(3, 576)), dict(k_pe=bf(2, 64)), dict(positions=torch.zeros(3, dtype=torch.int32)), dict(cos_sin=torch.zeros(10, 32)),
               dict(q=bf(3, 4, 576)), dict(q_pe=bf(3, 2, 64), q=bf(3, 4, 576)), dict(q_pe=bf(3, 4, 64), q=bf(3, 4, 640)[..., :576])):
        with pytest.raises(ValueError) as e:
            q.mla_append_rope(**dict(mla, **kw))
        assert "current CUDA device" not in str(e.value), kw
    p = plan(table([100]), [100], heads=4, kv_heads=2)
    run = dict(plan=p, q=bf(1, 4, 128), kv_data=pool, kv_scale=scale, kv_indices=i32(2), sm_scale=0.1, out=bf(1, 4, 128), lse=None,
               workspace=torch.zeros(1 << 16, dtype=torch.uint8))
    with pytest.raises(ValueError, match="current CUDA device"):
        q.gqa_decode_run(**run)
    for kw in (dict(q=bf(2, 4, 128)), dict(q=bf(1, 4, 256)[..., ::2]), dict(kv_data=pool[..., :64]), dict(kv_scale=torch.zeros((4, 4))),
               dict(out=torch.zeros((1, 4, 128))), dict(lse=torch.zeros((1, 2))), dict(kv_indices=torch.zeros(2, dtype=torch.int64)),
               dict(kv_indices=i32(1))):
        with pytest.raises(ValueError) as e:
            q.gqa_decode_run(**dict(run, **kw))
        assert "current CUDA device" not in str(e.value), kw


@pytest.mark.parametrize("kv,row,scales", [(q.KV_FP8_E4M3, 576, 0), (q.KV_NVFP4, 288, 36), (q.KV_FP8_PER_TOKEN, 580, 0)])
def test_binding_refuses_latent_pools_that_do_not_hold_the_pages(lib, kv, row, scales):
    """Slots are checked against the page count on the device, so the pool's bytes have to be there: strided,
    short and missing ones are refused. A pool of the right size is refused for not being on the GPU."""
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)          # noqa: E731
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)             # noqa: E731
    i64 = torch.zeros(2, dtype=torch.int64)
    good = dict(c_kv=bf(2, 512), k_pe=bf(2, 64), slot_mapping=i64, positions=i64, cos_sin=torch.zeros((10, 64)), rope_style=q.ROPE_PAIRS,
                kv_data=u8(3, 64, row), kv_scale=u8(3, 64, scales) if scales else None, kv_dtype=kv)
    with pytest.raises(ValueError, match="current CUDA device"):
        q.mla_append_rope(**good)
    with pytest.raises(ValueError, match="current CUDA device"):
        q.mla_append_rope(**dict(good, num_pages=2))
    bad = [dict(num_pages=4), dict(kv_data=u8(3, 64, row + 8)[..., :row]), dict(kv_data=u8(3, 32, row)), dict(kv_data=u8(6, 64, row)[::2])]
    if scales:
        bad += [dict(kv_scale=u8(2, 64, scales)), dict(kv_scale=u8(3, 64, scales + 4)[..., :scales])]
    for kw in bad:
        with pytest.raises(ValueError, match="pages"):
            q.mla_append_rope(**dict(good, **kw))
