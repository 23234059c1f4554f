"""Plain restatements of the rotated appends and of the head-pool decode, for the tests: numpy loops over
requests, pages and heads. The appends follow the header's FP32 arithmetic (one rounding per operation), so
their bytes are compared exactly; the decode is in 64 bits."""
from __future__ import annotations

import numpy as np
import torch

import oracle

PAGE = 64
HALVES, PAIRS = 0, 1
E4M3, INT8 = 1, 2
QMAX = {E4M3: np.float32(448.0), INT8: np.float32(127.0)}
E4M3_VALUES = np.array([oracle.e4m3_value(c) for c in range(256)])


def bf16_to_f32(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().float().numpy()


def to_bf16(x: np.ndarray) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16)


def table(max_pos: int, rot: int, base: float = 10000.0) -> np.ndarray:
    inv = base ** (-np.arange(0, rot, 2) / max(rot, 1))
    ang = np.arange(max_pos)[:, None] * inv
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


def pairs_of(rot: int, style: int):
    i = np.arange(rot // 2)
    return (i, i + rot // 2) if style == HALVES else (2 * i, 2 * i + 1)


def rotate(x: np.ndarray, cs: np.ndarray, style: int) -> np.ndarray:
    """x [..., D] float32 rotated by the table row cs [r] over its first r dims."""
    a, b = pairs_of(cs.shape[-1], style)
    c, s = np.split(cs, 2, -1)
    out = x.copy()
    with np.errstate(all="ignore"):
        out[..., a], out[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    return out


def rotate64(x, cs, style):
    a, b = pairs_of(cs.shape[-1], style)
    w = cs[:cs.shape[0] // 2].astype(np.float64) + 1j * cs[cs.shape[0] // 2:].astype(np.float64)
    out = x.astype(np.float64).copy()
    z = (out[..., a] + 1j * out[..., b]) * w
    out[..., a], out[..., b] = z.real, z.imag
    return out


def encode(x: np.ndarray, cache: int) -> np.ndarray:
    x = np.asarray(x, np.float32)
    if cache == E4M3:
        return oracle.encode_array(x, 1)
    return np.where(np.isnan(x), 0, np.clip(np.rint(np.nan_to_num(x, nan=0.0)), -127, 127)).astype(np.int8).view(np.uint8)


def decode(codes: np.ndarray, cache: int) -> np.ndarray:
    return E4M3_VALUES[codes] if cache == E4M3 else codes.view(np.int8).astype(np.float64)


def append_heads(k, v, tok_indptr, kv_len, kv_indptr, kv_indices, cs, style, codes, scale, cache, positions=None):
    """k, v float32 [n, Hkv, D]; codes [pages, 2, Hkv, 64, D] uint8 and scale [pages, 2, Hkv] float32 are
    changed in place. cs [max_pos, r] or None."""
    n, pages, heads = k.shape[0], codes.shape[0], codes.shape[2]
    for r in range(len(kv_len)):
        t0, t1, held = min(int(tok_indptr[r]), n), min(int(tok_indptr[r + 1]), n), int(kv_len[r])
        done = 0
        while done < t1 - t0:
            local, first = divmod(held + done, PAGE)
            count = min(PAGE - first, t1 - t0 - done)
            rows = np.arange(t0 + done, t0 + done + count)
            at = held + done + np.arange(count)
            done += count
            entry = int(kv_indptr[r]) + local
            if entry >= int(kv_indptr[r + 1]) or entry >= len(kv_indices) or not 0 <= kv_indices[entry] < pages:
                continue
            page = int(kv_indices[entry])
            pos = at if positions is None else positions[rows]
            keep = np.ones(count, bool) if cs is None else (pos >= 0) & (pos < cs.shape[0])
            for kind in range(2):
                for h in range(heads):
                    x = (k if kind == 0 else v)[rows, h].copy()
                    if kind == 0 and cs is not None:
                        for i in np.nonzero(keep)[0]:
                            x[i] = rotate(x[i], cs[pos[i]], style)
                    fin = np.abs(x[keep])[np.isfinite(x[keep])]
                    need = np.float32(fin.max() if fin.size else 0.0) / QMAX[cache]
                    old, block = scale[page, kind, h], codes[page, kind, h]
                    if first == 0 or not old > 0:
                        new = need
                    else:
                        new, shrink = old, np.float32(1)
                        while new < need:
                            new, shrink = new * np.float32(2), shrink * np.float32(0.5)
                        if shrink != 1:
                            block[:first] = encode(decode(block[:first], cache).astype(np.float32) * shrink, cache)
                    scale[page, kind, h] = new
                    with np.errstate(all="ignore"):
                        block[first + np.nonzero(keep)[0]] = encode(x[keep] / new if new != 0 else x[keep], cache)


def dequant(codes, scale, cache):
    """[pages, 2, Hkv, 64, D] float64."""
    return decode(codes, cache) * scale.astype(np.float64)[..., None, None]


def seen(length: int, window: int, sinks: int) -> np.ndarray:
    t = np.arange(length)
    return t if window == 0 else t[(t >= length - window) | (t < sinks)]


def attend(q, codes, scale, cache, kv_indptr, kv_indices, kv_len, sm_scale, window=0, sinks=0):
    """q float32 [B, H, D]. Returns out, lse and, for error bounds, sum p |v|, max_t sum_d |q_d k_d| sm_scale
    and the largest visible |v|, all in 64 bits."""
    batch, heads, dim = q.shape
    pages, kv_heads = codes.shape[0], codes.shape[2]
    group = heads // kv_heads
    out, absout = np.zeros((batch, heads, dim)), np.zeros((batch, heads, dim))
    lse, dot, vmax = np.full((batch, heads), -np.inf), np.zeros((batch, heads)), np.zeros((batch, heads))
    for r in range(batch):
        t = seen(int(kv_len[r]), window, sinks)
        page = np.asarray(kv_indices)[int(kv_indptr[r]) + t // PAGE].astype(np.int64)
        ok = (page >= 0) & (page < pages)
        t, page = t[ok], page[ok]
        if not t.size:
            continue
        for h in range(kv_heads):
            k, v = (decode(codes[page, i, h, t % PAGE], cache) * scale[page, i, h].astype(np.float64)[:, None] for i in (0, 1))
            sl = slice(h * group, (h + 1) * group)
            qq = q[r, sl].astype(np.float64)
            z = qq @ k.T * sm_scale
            m = z.max(1, keepdims=True)
            p = np.exp(z - m)
            total = p.sum(1, keepdims=True)
            out[r, sl], absout[r, sl] = p @ v / total, p @ np.abs(v) / total
            lse[r, sl] = (m + np.log(total))[:, 0]
            dot[r, sl] = (np.abs(qq) @ np.abs(k).T).max(1) * abs(sm_scale)
            vmax[r, sl] = np.abs(v).max()
    return out, lse, absout, dot, vmax


def check_attend(out: torch.Tensor, lse: torch.Tensor, ref, n: int, dim: int):
    """The kernel's bf16 out and float lse against attend()'s, element by element.

    z: D products, exact in FP32 (FP16 operands), summed in FP32, then two FP32 products: off by at most
    (D + 8) 2^-24 times sum |q k| sm_scale (dot). exp2 is good to 2^-21. So a weight is off by the factor
    1 + e, e = 2 (D + 8) 2^-24 dot + 2^-20 (numerator and denominator), the weight in the second product by
    half an FP16 step more, 2^-11, or 2^-25 absolute against a largest weight of at least 2^6 where it is
    subnormal; the sums of n terms add n 2^-23. The output is rounded to BF16, half a step: 2^-8 relative
    to its value covers it."""
    o_ref, l_ref, absout, dot, vmax = ref
    o = out.float().cpu().double().numpy()
    l = lse.cpu().double().numpy()
    e = 2 * (dim + 8) * 2.0 ** -24 * dot + 2.0 ** -20 + n * 2.0 ** -23
    tol = 2.0 ** -8 * np.abs(o_ref) + (e + 2.0 ** -11)[..., None] * absout * (1 + 2.0 ** -8) + (n * 2.0 ** -31 * vmax)[..., None] + 2.0 ** -133
    empty = np.isneginf(l_ref)
    assert np.array_equal(np.isneginf(l), empty) and not np.isnan(l).any()
    assert (o[empty] == 0).all()
    bad = np.abs(o - o_ref) > tol
    assert not bad.any(), (int(bad.sum()), float((np.abs(o - o_ref) / tol).max()), np.argwhere(bad)[:4].tolist())
    d = np.abs(l[~empty] - l_ref[~empty])
    lt = (e + 2.0 ** -22 * np.abs(np.where(empty, 0, l_ref)) + 2.0 ** -20)[~empty]
    assert (d <= lt).all(), float((d / lt).max())
    return float((np.abs(o - o_ref) / tol).max()), float((d / lt).max()) if d.size else 0.0
