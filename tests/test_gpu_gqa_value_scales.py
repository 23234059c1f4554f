"""Decode over head pools whose V block scales and logits go their own ways: scales that rise or fall by many
powers of two, several times within a request, with logits that make up for it, or do not."""
import numpy as np
import pytest
import torch

import quantized_kv_paged_gb300 as q
from tests import heads_ref as R

pytestmark = pytest.mark.gpu

# Requests as lists of pages: (log2 of the V block's scale, or None for a scale of 0, and the tokens' base-2 logit).
# Within a page the logits differ by up to 2/64 of that.
RISING = [
    [(0, 0), (-60, 68), (28, -28), (56, -56)],
    [(-62 + 25 * i, -25 * i) for i in range(6)],
    [(-110 + 27 * i, -27 * i) for i in range(9)],
    [(-100 + 25 * i, 0) for i in range(8)],
    [(-100 + 50 * i, 20 * i) for i in range(5)],
    [(-126, 0), (-99, -27)],                          # sums that are small BF16 numbers
]
FALLING = [[step for step in reversed(row)] for row in RISING]
APART = [
    [(100, -1000), (0, 0)], [(0, 0), (100, -1000)],   # the larger block has no weight at all
    [(61, -90), (0, 0), (-61, 90)], [(90, 0), (-90, 181), (90, 1), (-90, 180)],
    [(None, 40), (0, 0), (3, -2)], [(0, 0), (-20, 1), (None, 60), (None, -30), (4, 2)], [(-35, 0), (-50, 14), (None, 3)],
    [(None, 50), (-100, 40), (100, -150)], [(None, 0), (None, 5)], [(20, 0), (None, 30), (-80, 31), (None, 1)],
    [(3, 0), (-2, 4), (5, -3), (0, 1), (-30, 2), (1, 3)],
]


class Requests:
    """One KV head. Dim 0 of the keys carries the logit, dim 1 its variety; the query heads take it at different gains."""

    def __init__(self, rows, heads, dim, cache, repeat=1, copies=1, seed=0, v_codes=None, window=0, sinks=0):
        rng = np.random.default_rng(seed)
        self.heads, self.dim, self.cache, self.sm_scale = heads, dim, cache, float(np.log(2))
        self.see = dict(window=window, sinks=sinks)
        rows = [[p for p in row for _ in range(repeat)] for row in rows for _ in range(copies)]
        self.lens = np.array([64 * len(r) - (11 * i) % 40 for i, r in enumerate(rows)], np.int32)
        self.indptr = np.concatenate([[0], np.cumsum([len(r) for r in rows])]).astype(np.int32)
        pages = int(self.indptr[-1])
        self.ids = rng.permutation(pages).astype(np.int32)
        self.scale = np.zeros((pages, 2, 1), np.float32)
        values = np.zeros((pages, 2, 1, 64, dim), np.float32)
        for entry, (v, z) in enumerate(p for row in rows for p in row):
            page = self.ids[entry]
            sign = rng.choice([-1.0, 1.0], 64)
            values[page, 0, 0, :, 0], values[page, 0, 0, :, 1] = np.sign(z) or 1.0, sign
            self.scale[page, 0, 0] = abs(z) or 2.0 ** -10
            values[page, 1, 0] = rng.standard_normal((64, dim)) * 20 if v_codes is None else v_codes
            self.scale[page, 1, 0] = 0.0 if v is None else 2.0 ** v * (1.0 if v_codes is not None else rng.uniform(1.0, 1.9))
        self.codes = R.encode(values, cache)
        gains = np.array([1.0, -1.0, 0.0, 0.5, 1.0, 0.03125, -0.25, 0.9375])[np.arange(heads) % 8]
        query = np.zeros((len(rows), heads, dim), np.float32)
        query[:, :, 0], query[:, :, 1] = gains, gains / 64
        self.q = R.to_bf16(query)

    def run(self, num_sms):
        args = (self.indptr, self.lens, self.heads, 1, self.dim, self.cache)
        ws = torch.full((q.gqa_decode_plan(*args, num_sms=num_sms, **self.see).workspace_bytes,), 0xA5, dtype=torch.uint8, device="cuda")
        p = q.gqa_decode_plan(*args, num_sms=num_sms, workspace=ws, **self.see)
        out = torch.full((len(self.lens), self.heads, self.dim), 5.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((len(self.lens), self.heads), 5.0, device="cuda")
        dev = [x.cuda() for x in (self.q, torch.from_numpy(self.codes), torch.from_numpy(self.scale), torch.from_numpy(self.ids))]
        q.gqa_decode_run(p, *dev, self.sm_scale, out, lse, ws)
        again, lse2 = torch.empty_like(out), torch.empty_like(lse)
        for _ in range(3):
            q.gqa_decode_run(p, *dev, self.sm_scale, again, lse2, ws)
            assert torch.equal(out.view(torch.int16), again.view(torch.int16)) and torch.equal(lse, lse2)
        assert int(ws[p.status_offset:p.status_offset + 4].view(torch.int32).item()) == 0
        return out.float().cpu().double().numpy(), lse.cpu().double().numpy(), p

    def check(self, num_sms):
        """heads_ref.check_attend's bounds, but for two terms. Weights that FP16 holds as subnormals are off by 2^-25
        against a largest product of a weight and a V scale (not a largest weight) of at least 2^6: n 2^-31 of that
        product, and twice as much with the scales' mantissas, times the largest code. Weights below 2^-70 of the
        largest may count as zero. And the exponents of weights add scales' exponents and logits of up to 2^9 each, in
        four sums that round by up to 2^-15: 2^-13 in all."""
        out, lse, p = self.run(num_sms)
        for r, n in enumerate(self.lens):
            t = R.seen(int(n), **self.see)
            page = self.ids[self.indptr[r] + t // 64]
            k, code = (R.decode(self.codes[page, i, 0, t % 64], self.cache) for i in (0, 1))
            sk, sv = (self.scale[page, i, 0].astype(np.float64) for i in (0, 1))
            query = R.bf16_to_f32(self.q[r]).astype(np.float64)
            z = query @ (k * sk[:, None]).T * self.sm_scale
            dot = (np.abs(query) @ np.abs(k * sk[:, None]).T).max(1) * self.sm_scale
            m = z.max(1, keepdims=True)
            w = np.exp(z - m)
            total = w.sum(1, keepdims=True)
            w /= total
            v = code * sv[:, None]
            want, size, want_lse = w @ v, w @ np.abs(v), (m + np.log(total))[:, 0]
            e = 2 * (self.dim + 8) * 2.0 ** -24 * dot + 2.0 ** -20 + n * 2.0 ** -23 + 2.0 ** -13
            tol = 2.0 ** -8 * np.abs(want) + ((e + 2.0 ** -11)[:, None] * size * (1 + 2.0 ** -8) +
                                             (n * 2.0 ** -30 * (w * sv).max(1)[:, None] + n * 2.0 ** -70 * sv.max()) * np.abs(code).max() + 2.0 ** -133)
            bad = ~(np.abs(out[r] - want) <= tol)
            assert not bad.any(), (r, int(bad.sum()), np.argwhere(bad)[:3].tolist(), out[r][bad][:3], want[bad][:3])
            far = ~(np.abs(lse[r] - want_lse) <= e + 2.0 ** -22 * np.abs(want_lse) + 2.0 ** -20)
            assert not far.any(), (r, lse[r][far], want_lse[far])
        return p


@pytest.mark.parametrize("num_sms,repeat,copies,team", [(1, 1, 4, 1), (152, 1, 1, 4), (4, 4, 1, 4)])
@pytest.mark.parametrize("rows", [RISING, FALLING, APART], ids=["rising", "falling", "apart"])
@pytest.mark.parametrize("heads", [5, 16])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("cache", [R.E4M3, R.INT8])
def test_scales_and_logits_that_go_apart(qkvp, cache, dim, heads, rows, num_sms, repeat, copies, team):
    p = Requests(rows, heads, dim, cache, repeat, copies, seed=dim + heads).check(num_sms)
    assert p.warps_per_worker == team or num_sms == 4


@pytest.mark.parametrize("num_sms,copies", [(1, 3), (152, 1)])
@pytest.mark.parametrize("dim,heads", [(64, 16), (128, 5), (256, 16)])
def test_scales_that_go_apart_behind_a_window(qkvp, dim, heads, num_sms, copies):
    Requests(RISING + APART, heads, dim, R.E4M3, 3, copies, seed=dim, window=333, sinks=70).check(num_sms)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_scales_at_the_top_of_the_range(qkvp, dim):
    """V scales next to 2^128 behind a logit that just does not move the softmax's reference."""
    top = float(np.log2(np.float64(np.finfo(np.float32).max)))
    b = Requests([[(top, 0), (top, z)] for z in (7.875, 7.9375, 8, 8.0625)], 8, dim, R.E4M3, v_codes=0.25)
    b.codes[:, 0, :, :, 1] = 0                        # equal logits within a page
    b.scale[:, 0][b.scale[:, 0] == 2.0 ** -10] = 0.0  # the first page's are 0, the second's up to 8 for head 0
    b.scale[:, 1] = np.finfo(np.float32).max
    b.check(1)
    b.check(152)
