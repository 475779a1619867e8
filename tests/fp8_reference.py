"""64-bit reference of the block-scaled e4m3 operators, with error bounds.

Everything is numpy in float64; where the definition rounds a step to fp32
(scale, reciprocal, scaled value), the float64 result of that one step is
rounded to fp32, which is the correctly rounded fp32 result (a quotient or
product of fp32 numbers has at most 48 bits, or is far enough from a tie).

Bounds.  u = 2^-24 is half a step of fp32, eps(t) / 2 half a step of the output
type.  A product sums, for each block, 128 exact products in the tensor cores'
fp32 (at most a full step, 2u, per addition, whether it rounds or truncates),
multiplies by a scale product (3u: two roundings of scales and one fused
multiply-add) and adds the blocks in fp32 (u per addition, and as many more for
sums that are split between blocks of threads and joined).  With S the sum of
the terms' magnitudes the error is at most (2 * 128 + 3 + 2 * KB + 160) u S, and
the output adds eps / 2 of the result (and half the smallest fp16 step).
"""
from __future__ import annotations

import numpy as np
import torch

U = 2.0 ** -24
TINY = 2.0 ** -126


def f32(v):
    return np.asarray(v, dtype=np.float64).astype(np.float32).astype(np.float64)


def e4m3_round(v):
    """Nearest e4m3 value, ties to even, saturating; and the step at v."""
    v = np.asarray(v, dtype=np.float64)
    e = np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -6)))
    step = np.exp2(np.minimum(e, 8) - 3)
    return np.clip(np.rint(v / step) * step, -448.0, 448.0), step


def blocks(x, axis=-1):
    """x with its last axis padded by zeros and split in blocks of 128."""
    K = x.shape[-1]
    kb = -(-K // 128)
    p = np.zeros(x.shape[:-1] + (kb * 128,))
    p[..., :K] = x
    return p.reshape(x.shape[:-1] + (kb, 128))


def quantize(x):
    """(codes, scales) of the last axis of finite values that are fp32 already."""
    b = blocks(x)
    s = np.maximum(f32(np.abs(b).max(-1) / 448.0), TINY)
    q, _ = e4m3_round(f32(b * f32(1.0 / s)[..., None]))
    return q.reshape(x.shape[:-1] + (-1,))[..., : x.shape[-1]], s


def quantize_weight(W):
    """(codes N x K, scales) of a K x N weight in 128 x 128 blocks."""
    K, N = W.shape
    nb, kb = -(-N // 128), -(-K // 128)
    p = np.zeros((nb * 128, kb * 128))
    p[:N, :K] = W.T
    p = p.reshape(nb, 128, kb, 128)
    s = np.maximum(f32(np.abs(p).max((1, 3)) / 448.0), TINY)
    q, _ = e4m3_round(f32(p * f32(1.0 / s)[:, None, :, None]))
    return q.reshape(nb * 128, kb * 128)[:N, :K], s


def row_values(q, s):
    return q * np.repeat(s, 128, -1)[..., : q.shape[-1]]


def weight_values(q, s):
    return q * np.repeat(np.repeat(s, 128, -1), 128, -2)[..., : q.shape[-2], : q.shape[-1]]


def product(xv, wv):
    """(X W^T, bound of its fp32 error) of dequantised values."""
    kb = -(-xv.shape[-1] // 128)
    y = xv @ wv.T
    return y, (2 * 128 + 3 + 2 * kb + 160) * U * (np.abs(xv) @ np.abs(wv).T)


def out_bound(y, err, dtype):
    """Bound of a 16-bit output whose fp32 value is within err of y."""
    half = torch.finfo(dtype).eps / 2
    return err + half * (np.abs(y) + err) + (2.0 ** -25 if dtype == torch.float16 else 0.0)


def check(got, y, bound, what="Y"):
    got = got.detach().double().cpu().numpy()
    assert got.shape == y.shape, (got.shape, y.shape)
    bad = ~(np.abs(got - y) <= bound)
    if bad.any():
        i = np.unravel_index(int(np.argmax(np.where(bad, np.abs(got - y) / np.maximum(bound, 1e-300), 0))), y.shape)
        raise AssertionError(f"{what}: {int(bad.sum())} of {y.size} outside the bound; worst at {i}: got {got[i]}, "
                             f"want {y[i]}, bound {bound[i]}")


def route(X, R, top_k, renorm):
    """(ids, weights) of each token, ties to the lower index; NaN scores last."""
    l = X @ R.T
    key = np.where(np.isnan(l), -np.inf, l)
    ids = np.argsort(-key, axis=1, kind="stable")[:, :top_k]
    top = np.take_along_axis(l, ids[:, :1], 1)
    p = np.exp(np.take_along_axis(l, ids, 1) - top)
    p = p / (p.sum(1, keepdims=True) if renorm else np.exp(l - top).sum(1, keepdims=True))
    return ids, p


def moe(X, R, gate, up, down, top_k, renorm):
    """(Y, bound of its fp32 error, ids, weights); gate, up, down: dequantised
    E x N x K.

    The bound follows the layer: the fp32 errors dg, du of the two products;
    h = silu(g) u with |silu'| <= 1.1 and 8 roundings; the scale of a block has
    the relative error of its largest |h|; a code lies between those of the
    scaled value less and plus its error (rounding is monotonic); then the
    second product, the weights (32 roundings cover exp, sum and division)
    and the sum over the experts."""
    T, H = X.shape
    ids, p = route(X, R, top_k, renorm)
    q, s = quantize(X)
    xv = row_values(q, s)
    y, err = np.zeros((T, H)), np.zeros((T, H))
    for e in np.unique(ids):
        t, j = np.nonzero(ids == e)
        g, dg = product(xv[t], gate[e])
        u, du = product(xv[t], up[e])
        sg = g / (1 + np.exp(-g))
        h = sg * u
        dh = 1.1 * np.abs(u) * dg + np.abs(sg) * du + 1.1 * dg * du + 8 * U * np.abs(h)
        hb, dhb = blocks(h), blocks(dh)
        amax = np.abs(hb).max(-1)
        damax = dhb.max(-1) / np.maximum(amax, 1e-300) + U
        hs = np.maximum(amax / 448.0, TINY)
        v = hb / hs[..., None]
        dv = dhb / hs[..., None] + np.abs(v) * (damax[..., None] + 4 * U)
        c = e4m3_round(v)[0]
        # rounding is monotonic: the code of a value within dv of v lies between those of v - dv and v + dv
        off = np.maximum(e4m3_round(v + dv)[0] - c, c - e4m3_round(v - dv)[0])
        dc = (off + np.abs(c) * damax[..., None]) * hs[..., None]
        I = h.shape[-1]
        hv = (c * hs[..., None]).reshape(len(t), -1)[:, :I]
        dhv = dc.reshape(len(t), -1)[:, :I]
        ye, dye = product(hv, down[e])
        dye = dye + dhv @ np.abs(down[e]).T
        w = p[t, j][:, None]
        np.add.at(y, t, ye * w)
        np.add.at(err, t, (dye + 36 * U * np.abs(ye) + U * top_k * (np.abs(hv) @ np.abs(down[e]).T)) * w)
    return y, err, ids, p
