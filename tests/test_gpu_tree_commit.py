"""Committing accepted paths: bytes and scales against the header's arithmetic."""
import numpy as np
import pytest
import torch

import quantized_kv_paged_gb300 as q
from tests import heads_ref as R
from tests import tree_ref as T

pytestmark = pytest.mark.gpu


def layers_of(rng, n, pages, heads, dim, cache, spread):
    out = []
    for _ in range(n):
        x = rng.standard_normal((pages, 2, heads, 64, dim)).astype(np.float32) * np.exp2(rng.uniform(-spread, spread, (pages, 2, heads, 1, 1))).astype(np.float32)
        scale = (np.abs(x).max((3, 4)) / R.QMAX[cache]).astype(np.float32)
        out.append((R.encode(x / scale[..., None, None], cache).reshape(x.shape), scale))
    return out


def run(layers, cache, kv_len, indptr, ids, path, path_len, stream=None):
    dev = [(torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda()) for c, s in layers]
    q.gqa_tree_commit([c for c, _ in dev], [s for _, s in dev], cache, *(torch.from_numpy(np.asarray(x, np.int32)).cuda() for x in (
        kv_len, indptr, ids, path, path_len)))
    torch.cuda.synchronize()
    for (c, s), (gc, gs) in zip(layers, dev):
        T.commit(c, s, cache, kv_len, indptr, ids, path, path_len)
        assert np.array_equal(gs.cpu().numpy().view(np.int32), s.view(np.int32))
        bad = gc.cpu().numpy() != c
        assert not bad.any(), np.argwhere(bad)[:4].tolist()


@pytest.mark.parametrize("cache", [q.CACHE_E4M3, q.CACHE_INT8])
@pytest.mark.parametrize("heads,dim,layers,max_path", [(1, 64, 1, 1), (3, 64, 2, 40), (2, 128, 3, 9), (5, 128, 1, 256), (2, 256, 2, 70)])
def test_paths(qkvp, cache, heads, dim, layers, max_path):
    rng = np.random.default_rng(heads * dim + max_path)
    batch, per = 7, 7
    kv_len = rng.integers(0, 130, batch)
    kv_len[:3] = [63, 64, 0]
    path, path_len = np.zeros((batch, max_path), np.int64), rng.integers(0, max_path + 1, batch)
    path_len[1] = max_path
    for r in range(batch):
        most = per * 64 - kv_len[r] if r % 2 else min(max_path + 3, per * 64 - kv_len[r])
        path[r, :path_len[r]] = np.sort(rng.choice(min(256, most) if max_path < 200 else most, path_len[r], replace=False))
    ids = rng.permutation(batch * per + 2)[:batch * per]
    run(layers_of(rng, layers, batch * per + 2, heads, dim, cache, 2), cache, kv_len, np.arange(batch + 1) * per, ids, path, path_len)


def test_paths_that_stay_or_are_refused(qkvp):
    """In their place already, empty, out of order, out of range, outside the table or the pool: nothing changes."""
    rng = np.random.default_rng(4)
    paths = [[0, 1, 2, 3], [0, 1, 2, 3], [1, 1, 2, 3], [3, 2, 5, 6], [-1, 0, 1, 2], [0, 1, 2, 200], [0, 5, 9, 70], [2, 3, 4, 5], [2 ** 31 - 1, 0, 0, 0]]
    path_len = [4, 0, 4, 4, 4, 4, 4, -3, 1]
    batch, per = len(paths), 3
    ids = np.arange(batch * per)[::-1].copy()
    ids[6 * per + 1] = batch * per              # request 6's second page is not in the pool
    layers = layers_of(rng, 2, batch * per, 2, 64, q.CACHE_INT8, 1)
    before = [(c.copy(), s.copy()) for c, s in layers]
    run(layers, q.CACHE_INT8, [60] * batch, np.arange(batch + 1) * per, ids, np.array(paths), path_len)
    for (c, s), (c0, s0) in zip(layers, before):
        assert np.array_equal(c, c0) and np.array_equal(s, s0)
    run(layers, q.CACHE_INT8, [60] * batch, np.arange(batch + 1) * per, ids, np.array(paths), [5] * batch)
    assert np.array_equal(layers[0][0], before[0][0])


@pytest.mark.parametrize("cache", [q.CACHE_E4M3, q.CACHE_INT8])
def test_growing_blocks_zero_scales_and_nan(qkvp, cache):
    """Tokens from a page 2^-20 to 2^20 times as strong, blocks of scale 0, and NaN codes among what moves."""
    rng = np.random.default_rng(6)
    batch, per = 6, 3
    layers = layers_of(rng, 1, batch * per, 2, 128, cache, 0)
    codes, scale = layers[0]
    ids = np.arange(batch * per)
    for r, f in enumerate([2.0 ** -20, 2.0 ** 20, 1.5, 1.0, 0.0, 2.0 ** 3]):
        scale[ids[r * per + 1]] *= np.float32(f)
    scale[ids[3 * per]], codes[ids[3 * per]] = 0, 0
    if cache == q.CACHE_E4M3:
        codes[ids[2 * per + 1], :, :, 3, 7] = 0x7F
        codes[ids[2 * per + 1], :, :, 4] = 0xFF
    path = np.array([[1, 5, 7, 9, 70]] * batch)
    run(layers, cache, [58, 59, 60, 61, 62, 63], np.arange(batch + 1) * per, ids, path, [5] * batch)


def test_captured_and_replayed(qkvp):
    rng = np.random.default_rng(8)
    c0, s0 = layers_of(rng, 1, 9, 2, 64, q.CACHE_E4M3, 1)[0]
    ids, indptr = torch.arange(9, dtype=torch.int32, device="cuda"), torch.tensor([0, 3, 6, 9], dtype=torch.int32, device="cuda")
    kv_len, n = torch.tensor([10, 60, 63], dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    path = torch.zeros((3, 4), dtype=torch.int32, device="cuda")
    codes, scale = torch.from_numpy(c0).cuda(), torch.from_numpy(s0).cuda()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q.gqa_tree_commit([codes], [scale], q.CACHE_E4M3, kv_len, indptr, ids, path, n)
    for new, length in (([[1, 3, 5, 6], [0, 2, 9, 11], [4, 5, 6, 30]], [4, 3, 4]), ([[2, 0, 0, 0], [7, 8, 9, 10], [0, 1, 2, 5]], [1, 4, 4])):
        codes.copy_(torch.from_numpy(c0))
        scale.copy_(torch.from_numpy(s0))
        path.copy_(torch.tensor(new))
        n.copy_(torch.tensor(length))
        graph.replay()
        torch.cuda.synchronize()
        c, s = c0.copy(), s0.copy()
        T.commit(c, s, q.CACHE_E4M3, kv_len.tolist(), indptr.tolist(), ids.tolist(), np.array(new), length)
        assert np.array_equal(codes.cpu().numpy(), c) and np.array_equal(scale.cpu().numpy(), s)


@pytest.mark.parametrize("cache", [q.CACHE_E4M3, q.CACHE_INT8])
def test_scales_at_the_ends_of_the_range(qkvp, cache):
    """Values past FP32's range do not count towards a block's amax; subnormal, negative, infinite and NaN scales of the pages
    that tokens come from (a block that takes them has a scale that is not negative)."""
    rng = np.random.default_rng(11)
    big = [3e38, 3.4e38 / R.QMAX[cache], 2.7e36, 1e37, -3e36, 2e-45, np.inf, np.nan, -0.25, 1e-38]
    batch, per = 2 * len(big), 2
    layers = layers_of(rng, 2, batch * per, 2, 64, cache, 0)
    codes, scale = layers[0]
    codes[1::2, :, :, :3] = rng.integers(0, 256, codes[1::2, :, :, :3].shape, dtype=np.uint8)      # every code, -128 and NaN too
    ids = np.arange(batch * per)
    for r in range(batch):
        scale[2 * r + 1] = np.float32(big[r % len(big)])
        scale[2 * r] *= np.float32(1 if r < len(big) else 1e-38)
    path = np.array([[3, 6, 8]] * batch)
    run(layers, cache, [58 + r % 4 for r in range(batch)], np.arange(batch + 1) * per, ids, path, [3] * batch)


def test_two_streams_at_once(qkvp):
    """Two pools committed on two streams, more layers than one warp's share, with nothing between the calls."""
    rng = np.random.default_rng(12)
    batch, per, layers = 5, 4, 40
    ids, indptr, kv_len = np.arange(batch * per), np.arange(batch + 1) * per, np.array([0, 63, 64, 100, 128])
    path, n = np.array([[1, 2, 4, 8, 16, 40]] * batch), [6, 5, 4, 6, 0]
    streams, jobs = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for i in range(2):
        host = layers_of(rng, layers, batch * per, 3, 128, q.CACHE_E4M3, 2)
        jobs.append((host, [(torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda()) for c, s in host]))
    args = [torch.from_numpy(np.asarray(x, np.int32)).cuda() for x in (kv_len, indptr, ids, path, n)]
    torch.cuda.synchronize()
    for s, (_, dev) in zip(streams, jobs):
        q.gqa_tree_commit([c for c, _ in dev], [x for _, x in dev], q.CACHE_E4M3, *args, stream=s.cuda_stream)
    torch.cuda.synchronize()
    for host, dev in jobs:
        for (c, s), (gc, gs) in zip(host, dev):
            T.commit(c, s, q.CACHE_E4M3, kv_len, indptr, ids, path, n)
            assert np.array_equal(gc.cpu().numpy(), c) and np.array_equal(gs.cpu().numpy(), s)
