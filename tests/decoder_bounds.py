"""Error bounds of the decoder operators against the fp64 oracle, from the arithmetic alone.

U = 2^-24 is half a step of fp32; HALF half a step of a tensor's type.  An fp32 sum whose longest chain of additions has n
terms is off by at most n U times the sum of magnitudes.  A row of the norm is summed by chains of at most 32 terms a
lane, 6 lane steps and 16 waves: 64 covers them (ROW).
"""
import numpy as np
import torch

from encoder_bounds import HALF, U, close, f64  # noqa: F401

ROW = 64
KINDS = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


def norm_bounds(h, weight, ref, dtype, gy=None, gh=None):
    """Bounds of y, rstd, gx and gw for h [rows, C] in fp64."""
    w = np.ones(h.shape[1]) if weight is None else np.abs(weight)
    r = ref["rstd"]
    # the mean is off by (ROW + 2) U of itself, its root by half of that, plus the root's and the quotient's rounding
    er = ((ROW + 2) / 2 + 3) * U
    res = dict(rstd=er * r)
    ey = (er + 3 * U) * np.abs(ref["y"])
    res["y"] = ey + HALF[dtype] * (np.abs(ref["y"]) + ey)
    if gy is None:
        return res
    g, a = np.abs(gy), np.abs(h)
    rc = r[:, None]
    dot = (g * w * a).mean(axis=1)[:, None]
    # u: one rounding; the dot ROW + 2 more and its three factors; r three times; the difference and the product
    e = rc * g * w * (er + 4 * U) + rc ** 3 * a * dot * (3 * er + (ROW + 12) * U)
    size = rc * (g * w + rc ** 2 * a * dot) + (0 if gh is None else np.abs(gh))
    e = e + 4 * U * size
    res["gx"] = e + HALF[dtype] * (np.abs(ref["gx"]) + e)
    # every row's term is off by r's error and two roundings; chains of all rows, teams and workgroups at most
    terms = (g * a * rc).sum(axis=0)
    res["gw"] = (er + (h.shape[0] + 64) * U) * terms
    return res


def attention_bounds(q, ref, scale, cap, dtype):
    """Bounds of out [B, T, Hq, D].  Codes are exact in the products; fp32 queries and all weights go in as parts that leave
    2^-24 (fp32) or 2^-17 (bf16) of them."""
    B, T, Hq, D = q.shape
    low = 2 * U if dtype == torch.float32 else 2.0 ** -17
    out = np.zeros_like(q, dtype=np.float64)
    for b in range(B):
        k, v, p, s = ref["k"][b], ref["v"][b], ref["p"][b], ref["s"][b]
        n, Hk = k.shape[0], k.shape[1]
        G = Hq // Hk
        for h in range(Hq):
            mag = scale * (np.abs(q[b, :, h]) @ np.abs(k[:, h // G]).T)
            # three parts of D products; four factors; the cap's tanh (a few U of the cap); base 2 and the maximum's shift
            es = (3 * D + 16) * U * mag + 8 * U * cap + 8 * U * np.abs(s[h])
            es = np.where(ref["seen"][b], es, 0.0).max(axis=1, initial=0.0) + 8 * U * np.abs(s[h]).max(axis=1, initial=0.0)
            rel = 2 * es + 2 * (n + 64) * U + low
            out[b, :, h] = rel[:, None] * (p[h] @ np.abs(v[:, h // G])) * 1.01
            # a weight (or a part of one) under fp32's smallest normal number counts as nothing: the sum of the weights is 1
            # at least, so that is under 2^-126 of each value, once for the weight and once for each of three parts
            out[b, :, h] += 4 * 2.0 ** -126 * np.where(ref["seen"][b][:, :, None], np.abs(v[None, :, h // G]), 0).sum(axis=1)
    want = np.abs(ref["out"])
    return out + HALF[dtype] * (want + out)
