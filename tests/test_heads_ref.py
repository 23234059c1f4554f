"""The plain restatements that the head-pool tests compare with, checked on their own (CPU)."""
import numpy as np
import pytest
import torch

from tests import heads_ref as R


@pytest.mark.parametrize("style", [R.HALVES, R.PAIRS])
def test_rotation_is_a_rotation(style):
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 128)).astype(np.float32)
    cs = R.table(100001, 64)
    for p in (0, 1, 777, 100000):
        y = R.rotate(x, cs[p], style)
        assert np.array_equal(y[:, 64:], x[:, 64:])
        # two roundings of products and one of the sum, each half a step of values up to sqrt(2) |pair|
        ref = R.rotate64(x, cs[p], style)
        a, b = R.pairs_of(64, style)
        size = np.hypot(x[:, a], x[:, b])
        for i in (a, b):
            assert (np.abs(y - ref)[:, i] <= 4 * 2.0 ** -24 * size).all()
        if p == 0:
            assert np.array_equal(y, x)


def _stream(rng, n, heads, dim, gain):
    return (rng.standard_normal((n, heads, dim)) * np.exp2(gain * rng.random((n, 1, 1)))).astype(np.float32)


@pytest.mark.parametrize("cache", [R.E4M3, R.INT8])
def test_append_one_by_one_stays_within_a_step(cache):
    """64 tokens of growing size appended one at a time: every element of the finished block within one step
    (INT8) or within its rounding and what subnormal codes lose (E4M3) of the final scale."""
    rng = np.random.default_rng(1)
    k = _stream(rng, 64, 1, 64, 8) * np.exp2(np.arange(64) / 6)[:, None, None].astype(np.float32)
    codes, scale = np.zeros((1, 2, 1, 64, 64), np.uint8), np.zeros((1, 2, 1), np.float32)
    for t in range(64):
        R.append_heads(k[t:t + 1], k[t:t + 1], [0, 1], [t], [0, 1], np.array([0]), None, R.HALVES, codes, scale, cache)
    got = R.dequant(codes, scale, cache)[0, 1, 0]
    s = float(scale[0, 1, 0])
    err = np.abs(got - k[:, 0])
    if cache == R.INT8:
        assert (err <= s * (1 + 1e-6)).all()
    else:
        # normal codes are exact under growth; below 2^-6 each of the growths rounds once, by half of 2^-9
        assert (err <= np.maximum(np.abs(k[:, 0]) * 2.0 ** -4, s * 2.0 ** -9 * 1.01)).all()
    assert np.abs(k).max() / float(R.QMAX[cache]) <= s < 2 * np.abs(k).max() / float(R.QMAX[cache]) * (1 + 1e-6)


def test_attend_matches_torch_float64():
    rng = np.random.default_rng(2)
    k = rng.standard_normal((200, 2, 64)).astype(np.float32)
    codes, scale = np.zeros((4, 2, 2, 64, 64), np.uint8), np.zeros((4, 2, 2), np.float32)
    R.append_heads(k, -k, [0, 200], [0], [0, 4], np.array([2, 0, 3, 1]), None, R.HALVES, codes, scale, R.E4M3)
    q = rng.standard_normal((1, 6, 64)).astype(np.float32)
    vals = R.dequant(codes, scale, R.E4M3)
    rows = [vals[[2, 0, 3, 1][t // 64], :, :, t % 64] for t in range(200)]
    kk = torch.from_numpy(np.stack([x[0] for x in rows], 1)).repeat_interleave(3, 0)      # [H][n][D]
    vv = torch.from_numpy(np.stack([x[1] for x in rows], 1)).repeat_interleave(3, 0)
    qq = torch.from_numpy(q[0].astype(np.float64))[:, None]
    for window, sinks in ((0, 0), (70, 0), (1, 0), (100, 5), (150, 100)):
        t = torch.arange(200)
        mask = (t >= 200 - window) | (t < sinks) if window else t >= 0
        want = torch.nn.functional.scaled_dot_product_attention(qq, kk, vv, attn_mask=mask[None, None], scale=0.3)[:, 0]
        got = R.attend(q, codes, scale, R.E4M3, [0, 4], [2, 0, 3, 1], [200], 0.3, window, sinks)
        assert np.allclose(got[0][0], want.numpy(), rtol=1e-12, atol=1e-12)
