"""Page tables, counts, the free list and copies: exact against lists on the host."""
import numpy as np
import pytest
import torch

import quantized_kv_paged_gb300 as q
from tests.tree_ref import Pages

pytestmark = pytest.mark.gpu


def pools_of(rng, pages, sizes):
    return [rng.integers(0, 256, (pages, b), dtype=np.uint8) for b in sizes]


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


def work(pages, rows, n):
    return torch.zeros(q.kv_pages_workspace(pages, rows, n), dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("sizes", [(64,), (36864, 4), (37120, 18432, 2304, 12, 4096, 4112, 8192 + 36), (131072, 64) * 3])
@pytest.mark.parametrize("n", [0, 1, 37])
def test_copies(qkvp, sizes, n):
    rng = np.random.default_rng(n + len(sizes))
    pages = 2 * n + 5
    pools = pools_of(rng, pages, sizes)
    order = rng.permutation(pages)
    src, dst = order[:n].copy(), order[n:2 * n].copy()
    if n > 10:
        src[3], dst[5], src[6] = -1, pages, 2 ** 31 - 1
        dst[7] = src[7]
    d = [torch.from_numpy(p).cuda() for p in pools]
    q.kv_pages_copy(d, dev(src), dev(dst))
    torch.cuda.synchronize()
    for p, got in zip(pools, d):
        old = p.copy()
        for s, t in zip(src, dst):
            if 0 <= s < pages and 0 <= t < pages:
                p[t] = old[s]
        assert np.array_equal(got.cpu().numpy(), p)


def test_copies_of_unaligned_pools_leave_their_neighbours(qkvp):
    """Pools that start 4 bytes off a 16-byte boundary, and what lies around them."""
    whole = torch.arange(8 * 4100 + 64, device="cuda").to(torch.uint8)
    pool = whole[4:4 + 8 * 4100].view(8, 4100)
    want = whole.clone()
    want[4:4 + 8 * 4100].view(8, 4100)[6] = pool[1]
    q.kv_pages_copy([pool], dev([1]), dev([6]))
    assert torch.equal(whole, want)


@pytest.mark.parametrize("seed", range(6))
def test_a_life_of_calls(qkvp, seed):
    """Forks, growth, frees and compactions in any order on one state and one workspace, some of them refused."""
    rng = np.random.default_rng(seed)
    rows, row_pages = [(9, 6), (40, 11), (1500, 3), (3, 200), (64, 20), (25, 8)][seed]
    held = [int(rng.integers(0, row_pages + 1)) if rng.random() < 0.5 else 0 for _ in range(rows)]
    pages = sum(held) + [4, 30, 300, 100, 1, 70000][seed]
    s = Pages(rng, rows, row_pages, pages, held, pools_of(rng, pages, (32, 20) if pages > 50000 else (272, 36)))
    state, pools = s.state(), [torch.from_numpy(p).cuda() for p in s.pools]
    limit = 2 * rows + 3
    ws = work(pages, rows, limit)
    for step in range(14):
        n = int(rng.integers(1, limit + 1)) if step % 3 else int(rng.integers(1, 4))
        kind = ["fork", "grow", "free", "fork", "compact", "grow", "free"][step % 7]
        a = rng.integers(-1, rows + 1, n)
        if kind == "fork":
            # children that are empty, as a caller picks them, and some that are not
            empty = np.nonzero(s.held == 0)[0]
            b = np.where(rng.random(n) < 0.8, rng.permutation(np.resize(empty, n)) if len(empty) else -1, rng.integers(-1, rows + 1, n))
            status = dev(np.full(n, 9))
            q.kv_pages_fork(pools, *state, dev(a), dev(b), status, ws)
            assert status.tolist() == s.fork(a.tolist(), b.tolist())
        elif kind == "grow":
            t = rng.integers(-1, 64 * row_pages + 2, n)
            t = np.where(rng.random(n) < 0.3, rng.integers(0, 129, n), t)
            status = dev(np.full(n, 9))
            q.kv_pages_grow(*state, dev(a), dev(t), status, ws)
            assert status.tolist() == s.grow(a.tolist(), t.tolist())
        elif kind == "free":
            a = a[:max(1, n // 4)]
            q.kv_pages_free(*state, dev(a), ws)
            s.release(a.tolist())
        else:
            q.kv_pages_compact(pools, *state, ws)
            s.compact()
        s.same(state, pools)
    head = ws[:256 + 4 * rows]
    assert not head[:4].any() and not head[256:].any()


def test_empty_lists_and_states(qkvp):
    rng = np.random.default_rng(1)
    s = Pages(rng, 3, 4, 20, [2, 0, 3], pools_of(rng, 20, (64,)))
    state, pools = s.state(), [torch.from_numpy(p).cuda() for p in s.pools]
    none, ws = dev([]), work(20, 3, 0)
    q.kv_pages_fork(pools, *state, none, none, none, ws)
    q.kv_pages_grow(*state, none, none, none, ws)
    q.kv_pages_free(*state, none, ws)
    q.kv_pages_copy([], dev([1]), dev([2]))
    s.same(state, pools)
    q.kv_pages_compact([], *state, ws)      # bookkeeping alone
    pools_before = [p.copy() for p in s.pools]
    s.compact()
    s.pools = pools_before
    s.same(state, pools)


def test_free_pages_run_out_to_the_last(qkvp):
    rng = np.random.default_rng(2)
    s = Pages(rng, 6, 4, 7, [1, 0, 0, 0, 0, 0], pools_of(rng, 7, (64,)))
    s.lens[0] = 40
    state, pools = s.state(), [torch.from_numpy(p).cuda() for p in s.pools]
    ws = work(7, 6, 8)
    st = dev([0] * 5)
    q.kv_pages_grow(*state, dev([1, 2, 3, 4, 5]), dev([128, 192, 64, 0, 64]), st, ws)
    assert st.tolist() == s.grow([1, 2, 3, 4, 5], [128, 192, 64, 0, 64]) == [1, 1, 1, 1, 0]
    s.same(state, pools)
    q.kv_pages_fork(pools, *state, dev([0]), dev([5]), st[:1], ws)
    assert st[:1].tolist() == s.fork([0], [5]) == [0]
    q.kv_pages_free(*state, dev([2, 2]), ws)
    s.release([2])
    q.kv_pages_fork(pools, *state, dev([0]), dev([5]), st[:1], ws)
    assert st[:1].tolist() == s.fork([0], [5]) == [1]
    s.same(state, pools)


def test_a_state_that_does_not_add_up_faults_nothing(qkvp):
    """Ids outside the pool in tables and the free list, counts and lengths that are wrong: nothing outside is touched."""
    rng = np.random.default_rng(3)
    s = Pages(rng, 8, 5, 30, [3, 4, 0, 0, 5, 0, 2, 0], pools_of(rng, 30, (64,)))
    state, pools = s.state(), [torch.from_numpy(p).cuda() for p in s.pools]
    guard = [t.clone() for t in pools]
    table, held, lens, refs, free, count = state
    table[0, :2] = dev([-4, 2 ** 31 - 1])
    held[4] = 100
    lens[6] = 10 ** 6
    free[int(count) - 1] = 1000
    count.fill_(29)
    ws = work(30, 8, 8)
    st = dev([0] * 4)
    q.kv_pages_fork(pools, *state, dev([0, 6, 1, 4]), dev([2, 3, 5, 7]), st, ws)
    q.kv_pages_grow(*state, dev([2, 5]), dev([300, 320]), st[:2], ws)
    q.kv_pages_free(*state, dev([0, 4, 1, 2]), ws)
    q.kv_pages_compact(pools, *state, ws)
    torch.cuda.synchronize()
    assert 0 <= int(count) <= 30 and [p.shape for p in guard] == [p.shape for p in pools]


def test_captured_and_replayed(qkvp):
    rng = np.random.default_rng(5)
    s = Pages(rng, 6, 4, 40, [3, 2, 0, 0, 0, 0], pools_of(rng, 40, (4160, 32)))
    state, pools = s.state(), [torch.from_numpy(p).cuda() for p in s.pools]
    ws = work(40, 6, 4)
    parents, children, tokens, st = dev([0, 0, 1, 1]), dev([2, 3, 4, 5]), dev([200, 10, 256, 0]), dev([0] * 4)

    def step():
        q.kv_pages_fork(pools, *state, parents, children, st, ws)
        q.kv_pages_grow(*state, children, tokens, st, ws)
        q.kv_pages_free(*state, children, ws)
        q.kv_pages_compact(pools, *state, ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for picks in ([0, 0, 1, 1], [1, 0, 0, 0], [0, 1, 0, 1]):
        parents.copy_(dev(picks))
        graph.replay()
        torch.cuda.synchronize()
        s.fork(picks, [2, 3, 4, 5])
        s.grow([2, 3, 4, 5], [200, 10, 256, 0])
        s.release([2, 3, 4, 5])
        s.compact()
        s.same(state, pools)


def test_pages_of_latent_pools(qkvp):
    """Every cache layout of the library has its page first, so its codes and scales are pools like any other."""
    rng = np.random.default_rng(9)
    shapes = [(12, 64, 576), (12, 64, 288), (12, 64, 36), (12, 64, 580), (12, 2, 3, 64, 128)]
    host = [rng.integers(0, 256, s, dtype=np.uint8) for s in shapes] + [rng.standard_normal((12, 2, 3)).astype(np.float32)]
    d = [torch.from_numpy(x).cuda() for x in host]
    d.append(torch.randn((12, 64, 576), device="cuda").bfloat16())
    last = d[-1].clone()
    q.kv_pages_copy(d, dev([0, 3, 7]), dev([11, 2, 6]))
    for x, got in zip(host, d):
        x[[11, 2, 6]] = x[[0, 3, 7]]
        assert np.array_equal(got.cpu().numpy(), x)
    last[[11, 2, 6]] = last[[0, 3, 7]]
    assert torch.equal(d[-1], last)
