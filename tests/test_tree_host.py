"""Argument checks and plans of the tree attention, the commit of paths and the pages of a cache, without a GPU."""
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


I, U, W, OK = q.QKVP_E_INVALID, q.QKVP_E_UNSUPPORTED, q.QKVP_E_WORKSPACE, q.QKVP_OK
LONGEST = 2 ** 31 - 1


def table(lens, spare=0):
    return np.concatenate([[0], np.cumsum([(n + 63) // 64 + spare for n in lens])]).astype(np.int32)


def plan(lens, drafted, heads=32, kv_heads=8, dim=128, cache=q.CACHE_E4M3, sms=152, ptr=None, **kw):
    tok = np.concatenate([[0], np.cumsum(drafted)]).astype(np.int32)
    return q.gqa_tree_plan(table(lens) if ptr is None else np.asarray(ptr, np.int32), np.asarray(lens, np.int32), tok, heads, kv_heads, dim, cache,
                           num_sms=sms, raise_on_error=False, **kw)


@pytest.mark.parametrize("kw,want", [
    (dict(), OK), (dict(dim=96), U), (dict(dim=0), U), (dict(cache=0), U), (dict(cache=7), U), (dict(heads=30), U), (dict(heads=0), U),
    (dict(kv_heads=0), U), (dict(kv_heads=257, heads=257), U), (dict(page_size=32), U), (dict(window=-1), I), (dict(window=64, sinks=-1), I),
    (dict(sinks=4), I), (dict(window=4), U), (dict(window=5), OK), (dict(window=5, sinks=LONGEST), OK), (dict(window=LONGEST, sinks=LONGEST), OK),
    (dict(min_splits=-1), I), (dict(sms=65537), I), (dict(ptr=[1, 3]), I), (dict(ptr=[0, 1]), I), (dict(lens=[-1]), I), (dict(lens=[4]), I),
    (dict(lens=[5]), OK), (dict(drafted=[-1]), I), (dict(lens=[257], drafted=[257]), U), (dict(lens=[256], drafted=[256]), OK),
    (dict(drafted=[0]), OK)])
def test_plan_refusals(lib, kw, want):
    a = dict(dict(lens=[100], drafted=[5]), **kw)
    if a["lens"] == [-1]:
        a["ptr"] = [0, 2]
    assert plan(**a).status == want


def test_plan_refuses_a_token_table_that_does_not_fit(lib):
    lens = np.array([100, 100], np.int32)
    for tok in ([1, 3, 5], [0, 5, 3], [0, -1, 3]):
        assert q.gqa_tree_plan(table(lens), lens, np.array(tok, np.int32), 8, 2, 64, q.CACHE_INT8, num_sms=4, raise_on_error=False).status == I
    with pytest.raises(ValueError):
        q.gqa_tree_plan(table(lens), lens, np.array([0, 5], np.int32), 8, 2, 64, q.CACHE_INT8, num_sms=4)
    p = q.qkvp_tree_plan()
    ptr, tok = table(lens), np.array([0, 2, 4], np.int32)
    args = [ptr.ctypes.data, lens.ctypes.data, tok.ctypes.data, 2, 8, 2, 64, 64, q.CACHE_INT8, 0, 0, 4, 0, None, 0, None, ctypes.byref(p)]
    assert lib.gqa_tree_plan(*args) == OK and p.magic == 0
    for i in (0, 1, 2, 16):
        assert lib.gqa_tree_plan(*[None if j == i else a for j, a in enumerate(args)]) == I
    assert lib.gqa_tree_plan(*args[:13], 256, 64, None, args[16]) == W and p.workspace_bytes > 64 and p.magic == 0


@pytest.mark.parametrize("length,drafted,window,sinks,pages", [
    (1, 1, 0, 0, 1), (64, 64, 0, 0, 1), (65, 1, 0, 0, 2), (1000, 1, 0, 0, 16), (1000, 200, 0, 0, 16),
    (1000, 1, 1, 0, 1), (1000, 10, 10, 0, 1), (1000, 40, 40, 0, 2), (1000, 20, 100, 0, 3), (1000, 20, 100, 1, 4), (1000, 20, 100, 128, 5),
    (1000, 20, 970, 0, 16), (1000, 20, 960, 0, 16), (1000, 20, LONGEST, 9, 16), (LONGEST - 63, 256, 256, 0, 8)])
def test_plan_reads_the_visible_pages(lib, length, drafted, window, sinks, pages):
    """The earliest page is that of token length - drafted - window: with one path token the window reaches that far."""
    p = plan([length], [drafted], heads=4, kv_heads=2, window=window, sinks=sinks)
    assert p.status == OK and p.total_pages == pages
    first = max(0, length - drafted - window) // 64
    assert not window or first >= (length + 63) // 64 - pages


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("sms", [1, 7, 152])
def test_plan_covers_balances_and_sizes(lib, dim, sms):
    rng = np.random.default_rng(dim + sms)
    drafted = rng.integers(0, 257, 40)
    lens = rng.integers(0, 9000, 40) + drafted
    p = plan(lens, drafted, heads=24, kv_heads=4, dim=dim, sms=sms)
    blocks = [-(-int(t) * 6 // 128) for t in drafted]
    assert p.status == OK and p.num_workers == sms and p.num_tokens == drafted.sum() and p.max_drafted == drafted.max()
    assert p.total_pages == sum((int(n) + 63) // 64 for n, t in zip(lens, drafted) if t)
    work = sum(4 * b * ((int(n) + 63) // 64) for n, b in zip(lens, blocks))
    assert 4 * sum(blocks) <= p.num_segments <= 4 * sum(blocks) + sms
    assert p.max_worker_pages >= work / sms >= p.min_worker_pages
    # a started segment counts as up to 16 pages, so no worker is further from the mean than what its segments count
    assert p.max_worker_pages <= work / sms + 16 * (p.num_segments / sms + 1) + 1
    assert p.num_partials <= 2 * p.num_joins + 2 * sms
    assert p.partial_o_offset >= p.table_bytes and p.partial_lse_offset >= p.partial_o_offset + p.num_partials * 128 * dim * 4
    assert p.workspace_bytes >= p.partial_lse_offset + p.num_partials * 128 * 4 and p.status_offset + 4 <= p.table_bytes
    for x in (p.partial_o_offset, p.partial_lse_offset, p.table_bytes):
        assert x % 256 == 0


def test_plan_of_nothing_and_of_much(lib):
    for lens, drafted in (([], []), ([0, 100], [0, 0])):
        p = plan(lens, drafted)
        assert p.status == OK and (p.num_tokens, p.num_segments, p.num_joins) == (0, 0, 0)
    few = plan([32768] * 44, [4] * 44, heads=64)
    assert (few.row_copies, few.num_joins) == (4, 352) and few.num_partials == few.num_segments
    assert plan([32768] * 44, [5] * 44, heads=64).row_copies == 2 and plan([500] * 44, [4] * 44, heads=64).row_copies == 1
    assert plan([32768] * 44, [8] * 44, heads=64, dim=64).row_copies == 2 and plan([32768] * 44, [8] * 44, heads=64, dim=256).row_copies == 1
    assert plan([32768] * 44, [9] * 44, heads=64).row_copies == 1
    assert plan([1 << 20], [8], heads=8, kv_heads=1, min_splits=100, ptr=[0, 16384]).max_join_segments >= 100
    assert plan([LONGEST], [1], ptr=[0, 1 << 25]).status == U
    assert plan([LONGEST], [1], ptr=[0, 1 << 25], window=1, heads=1, kv_heads=1).status in (OK, U)
    many = [60] * 70000
    assert plan(many, [60] * 70000, heads=256, kv_heads=256).status == U      # more row blocks than the plan addresses


def test_run_refuses_before_any_launch(lib):
    p = plan([100], [5])
    ok = dict(plan=ctypes.byref(p), q=16, kv=128, scale=16, pages=4, idx=16, mask=4, words=1, sm=0.1, out=16, lse=4, ws=256, n=1 << 40)

    def run(**kw):
        a = dict(ok, **kw)
        return lib.gqa_tree_run(a["plan"], a["q"], a["kv"], a["scale"], a["pages"], a["idx"], a["mask"], a["words"], a["sm"], a["out"], a["lse"],
                                a["ws"], a["n"], None)
    assert run() == I                                              # a size query is no plan: nothing was uploaded
    p.magic = magic()
    for kw, want in ((dict(plan=None), I), (dict(ws=None), W), (dict(n=8), W), (dict(ws=128), W), (dict(q=None), I), (dict(q=8), I),
                     (dict(out=None), I), (dict(out=8), I), (dict(lse=2), I), (dict(kv=None), I), (dict(kv=8), I), (dict(scale=None), I),
                     (dict(scale=2), I), (dict(idx=None), I), (dict(idx=2), I), (dict(mask=2), I), (dict(words=0), I), (dict(mask=None), I),
                     (dict(words=-1), I), (dict(pages=-1), I), (dict(sm=float("nan")), I), (dict(sm=float("-inf")), I), (dict(pages=1 << 60), I)):
        assert run(**kw) == want, kw
    p.magic ^= 1
    assert run() == I


def magic():
    import os
    import re
    from tests.conftest import ROOT
    with open(os.path.join(ROOT, "quantized_kv_paged_gb300", "csrc", "qkvp_internal.h")) as f:
        return int(re.search(r"kTreeMagic\s*=\s*(0x[0-9A-Fa-f]+)", f.read()).group(1), 16)


def pointers(*p):
    return (ctypes.c_void_p * len(p))(*p)


COMMIT = dict(kv=pointers(16, 32), sc=pointers(4, 8), layers=2, klen=4, batch=1, ptr=4, idx=4, nnz=9, path=4, plen=4, mp=8, hk=2, d=128, cache=1,
              ps=64, pages=9)


@pytest.mark.parametrize("kw,want", [
    (dict(layers=-1), I), (dict(batch=-1), I), (dict(nnz=-1), I), (dict(mp=-1), I), (dict(pages=-1), I), (dict(d=80), U), (dict(cache=0), U),
    (dict(ps=16), U), (dict(hk=0), U), (dict(hk=257), U), (dict(layers=129), U), (dict(mp=257), U), (dict(kv=None), I), (dict(sc=None), I),
    (dict(klen=None), I), (dict(klen=2), I), (dict(ptr=None), I), (dict(idx=None), I), (dict(idx=2), I), (dict(path=None), I), (dict(path=6), I),
    (dict(plen=None), I), (dict(kv=pointers(16, 0)), I), (dict(kv=pointers(8, 16)), I), (dict(sc=pointers(4, 2)), I), (dict(sc=pointers(0, 4)), I),
    (dict(pages=1 << 60), I), (dict(layers=0, kv=None, sc=None), OK), (dict(batch=0, klen=None), OK), (dict(mp=0, path=None), OK)])
def test_commit_refusals(lib, kw, want):
    a = dict(COMMIT, **kw)
    assert lib.gqa_tree_commit(a["kv"], a["sc"], a["layers"], a["klen"], a["batch"], a["ptr"], a["idx"], a["nnz"], a["path"], a["plen"], a["mp"],
                               a["hk"], a["d"], a["cache"], a["ps"], a["pages"], None) == want


def pools(*pairs):
    return (ctypes.c_int64 * (2 * len(pairs)))(*[x for p in pairs for x in p])


def state(**kw):
    a = dict(dict(table=4, held=4, lens=4, refs=4, free_list=4, free_count=4, rows=3, row_pages=5, num_pages=20), **kw)
    return q.qkvp_page_state(*a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(n=-1), I), (dict(pages=-1), I), (dict(pages=1 << 31), U), (dict(src=None), I), (dict(dst=None), I), (dict(src=2), I), (dict(p=None), I),
    (dict(p=pools((0, 64))), I), (dict(p=pools((2, 64))), I), (dict(p=pools((16, 0))), I), (dict(p=pools((16, -4))), I), (dict(p=pools((16, 6))), I),
    (dict(p=pools((16, 1 << 31))), U), (dict(p=pools((16, 1 << 62)), pages=8), I), (dict(count=257, p=pools(*[(16, 64)] * 257)), U),
    (dict(count=-1), I), (dict(n=0, src=None, dst=None), OK), (dict(count=0, p=None), OK)])
def test_copy_refusals(lib, kw, want):
    a = dict(dict(p=pools((16, 64)), count=1, src=4, dst=4, n=3, pages=20), **kw)
    assert lib.kv_pages_copy(a["p"], a["count"], a["src"], a["dst"], a["n"], a["pages"], None) == want


@pytest.mark.parametrize("kw,want", [
    (dict(table=None), I), (dict(held=None), I), (dict(lens=None), I), (dict(refs=None), I), (dict(free_list=None), I), (dict(free_count=None), I),
    (dict(table=2), I), (dict(held=6), I), (dict(lens=1), I), (dict(refs=2), I), (dict(free_list=2), I), (dict(free_count=2), I), (dict(rows=-1), I),
    (dict(row_pages=-1), I), (dict(num_pages=-1), I), (dict(num_pages=1 << 31), U)])
def test_states_that_are_refused(lib, kw, want):
    s, big, p = state(**kw), 1 << 40, pools((16, 64))
    r = ctypes.byref(s)
    assert lib.kv_pages_fork(p, 1, r, 4, 4, 1, 4, 256, big, None) == want
    assert lib.kv_pages_grow(r, 4, 4, 1, 4, 256, big, None) == want
    assert lib.kv_pages_free(r, 4, 1, 256, big, None) == want
    assert lib.kv_pages_compact(p, 1, r, 256, big, None) == want


def test_lists_and_workspaces_that_are_refused(lib):
    s, p = state(), pools((16, 64))
    r, need = ctypes.byref(s), q.kv_pages_workspace(20, 3, 4)
    fork = dict(p=p, count=1, s=r, a=4, b=4, n=4, st=4, ws=256, size=need)
    for kw, want in ((dict(s=None), I), (dict(a=None), I), (dict(b=2), I), (dict(st=None), I), (dict(n=-1), I), (dict(ws=None), W), (dict(ws=128), W),
                     (dict(size=need - 1), W), (dict(n=10 ** 6), W), (dict(p=pools((16, 6))), I), (dict(n=0, a=None, b=None, st=None), OK)):
        a = dict(fork, **kw)
        assert lib.kv_pages_fork(a["p"], a["count"], a["s"], a["a"], a["b"], a["n"], a["st"], a["ws"], a["size"], None) == want, kw
        if "p" not in kw:
            assert lib.kv_pages_grow(a["s"], a["a"], a["b"], a["n"], a["st"], a["ws"], a["size"], None) == want, kw
        if not {"p", "b", "st"} & set(kw) or kw.get("n") == 0:
            assert lib.kv_pages_free(a["s"], a["a"], a["n"], a["ws"], a["size"], None) == want, kw
    assert lib.kv_pages_compact(p, 1, r, 256, 16, None) == W and lib.kv_pages_compact(p, 1, None, 256, need, None) == I
    empty = state(num_pages=0, refs=None, free_list=None)
    assert lib.kv_pages_compact(p, 1, ctypes.byref(empty), 256, 1 << 20, None) == OK


def test_workspace_sizes(lib):
    size = ctypes.c_uint64()
    assert lib.kv_pages_workspace(5, 5, 5, None) == I
    for args, want in (((-1, 1, 1), I), ((1, -1, 1), I), ((1, 1, -1), I), ((1 << 31, 1, 1), U), ((LONGEST, LONGEST, LONGEST), OK)):
        assert lib.kv_pages_workspace(*args, ctypes.byref(size)) == want
    assert size.value >= 3 * 4 * LONGEST
    assert q.kv_pages_workspace(100, 10, 5) <= q.kv_pages_workspace(100, 10, 500) <= q.kv_pages_workspace(100, 1000, 500)
    with pytest.raises(q.QkvpError if hasattr(q, "QkvpError") else Exception):
        q.kv_pages_workspace(-1, 1, 1)


def refuses(call, good, bad):
    """Layouts are checked before devices: right tensors are refused for not being on the GPU, wrong ones for what they are."""
    with pytest.raises(ValueError, match="current CUDA device"):
        call(**good)
    for kw in bad:
        with pytest.raises(ValueError) as e:
            call(**dict(good, **kw))
        assert "current CUDA device" not in str(e.value), kw


def test_bindings_refuse_wrong_tensors(lib):
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)          # noqa: E731
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)            # noqa: E731
    pool, scale = torch.zeros((4, 2, 2, 64, 128), dtype=torch.uint8), torch.zeros((4, 2, 2))
    p = plan([100], [40], heads=4, kv_heads=2)
    refuses(q.gqa_tree_run, dict(plan=p, q=bf(40, 4, 128), kv_data=pool, kv_scale=scale, kv_indices=i32(2), tree_mask=i32(40, 2), sm_scale=0.1,
                                 out=bf(40, 4, 128), lse=torch.zeros((40, 4)), workspace=torch.zeros(1 << 20, dtype=torch.uint8)),
            [dict(q=bf(39, 4, 128)), dict(q=bf(40, 4, 256)[..., ::2]), dict(q=torch.zeros((40, 4, 128))), dict(kv_data=pool[..., :64]),
             dict(kv_scale=torch.zeros((4, 4))), dict(out=torch.zeros((40, 4, 128))), dict(lse=torch.zeros((40, 2))), dict(kv_indices=i32(1)),
             dict(kv_indices=torch.zeros(2, dtype=torch.int64)), dict(tree_mask=i32(40, 1)), dict(tree_mask=i32(39, 2)), dict(tree_mask=i32(40, 4)[:, ::2]),
             dict(tree_mask=torch.zeros((40, 2), dtype=torch.int64)), dict(kv_data=torch.zeros((4, 2, 4, 64, 128), dtype=torch.uint8), kv_scale=torch.zeros((4, 2, 4)))])
    refuses(q.gqa_tree_commit, dict(kv_data=[pool, pool], kv_scale=[scale, scale], cache_dtype=q.CACHE_E4M3, kv_len=i32(3), kv_indptr=i32(4),
                                    kv_indices=i32(9), path=i32(3, 5), path_len=i32(3)),
            [dict(kv_data=[pool]), dict(kv_data=[pool, pool[:2]]), dict(kv_data=[pool, pool.float()]), dict(kv_scale=[scale, scale.double()]),
             dict(kv_scale=[scale, scale[:, :1]]), dict(kv_scale=[torch.zeros((4, 2, 4))[..., ::2]] * 2), dict(kv_indptr=i32(3)), dict(path=i32(2, 5)),
             dict(path=i32(3, 10)[:, ::2]), dict(path_len=i32(4)), dict(kv_len=torch.zeros(3, dtype=torch.int64)),
             dict(kv_data=[pool, pool.as_strided((2, 4, 2, 64, 128), pool.stride())])])
    st = dict(table=i32(3, 5), held=i32(3), lens=i32(3), refs=i32(20), free_list=i32(20), free_count=i32(1))
    ws, buf = torch.zeros(1 << 12, dtype=torch.uint8), [torch.zeros((20, 64)), torch.zeros((20, 2, 8), dtype=torch.uint8)]
    bad = [dict(table=i32(3, 10)[:, ::2]), dict(table=i32(15)), dict(held=i32(4)), dict(lens=torch.zeros(3)), dict(free_list=i32(21)), dict(free_count=i32(2)),
           dict(refs=i32(21))]
    bad_pools = [dict(pools=[torch.zeros((20, 64)), torch.zeros((19, 64))]), dict(pools=[torch.zeros((20, 64))[:, ::2]]), dict(pools=[torch.zeros(())]),
                 dict(pools=[torch.zeros((20, 0))]), dict(pools=[torch.zeros((1, 64)).expand(20, 64)])]
    # pools are looked at last, so the others have to be right and on the device: these show their own errors alone
    refuses(q.kv_pages_fork, dict(pools=buf, parents=i32(2), children=i32(2), status=i32(2), workspace=ws, **st),
            bad + [dict(parents=i32(3)), dict(children=i32(4)[::2]), dict(status=torch.zeros(2))])
    refuses(q.kv_pages_grow, dict(rows=i32(2), tokens=i32(2), status=i32(2), workspace=ws, **st), bad + [dict(tokens=i32(1)), dict(rows=torch.zeros(2))])
    refuses(q.kv_pages_free, dict(rows=i32(2), workspace=ws, **st), bad + [dict(rows=i32(4)[::2])])
    refuses(q.kv_pages_compact, dict(pools=buf, workspace=ws, **st), bad)
    refuses(q.kv_pages_copy, dict(pools=buf, src=i32(2), dst=i32(2)), [dict(src=i32(3)), dict(dst=torch.zeros(2)), dict(src=i32(4)[::2])])
    for kw in bad_pools:
        with pytest.raises(ValueError, match="pool"):
            q.kv_pages_copy(**dict(dict(pools=buf, src=i32(2), dst=i32(2)), **kw))
    with pytest.raises(ValueError, match="contiguous"):
        q.kv_pages_grow(rows=i32(2), tokens=i32(2), status=i32(2), workspace=ws[::2], **st)


@pytest.mark.parametrize("name", ["tree.cu", "tree_commit.cu", "pages.cu"])
def test_overlapped_kernels_read_by_ordinary_loads(name):
    """As for the decode: what the kernel before may still write is not read through the read-only path."""
    import os
    from tests.conftest import ROOT
    with open(os.path.join(ROOT, "quantized_kv_paged_gb300", "csrc", name)) as f:
        text = f.read()
    assert "launch_overlapped(" in text and "wait_for_previous()" in text
    assert not [w for w in ("__ldg(", "ldg_nc", "ld.global.nc", "__restrict__") if w in text]
