"""Error bounds of the attention without allowances for values rounded to bf16 inside it.

U = 2^-24 is half a step of fp32.  Against the fp64 oracle a result may be off by
- its own rounding to its type (finfo(type).eps / 2 of the value);
- what fp32 scores, exponentials and sums of the lengths at hand are off by;
- for bf16 tensors 2^-16 of every factor of the second products, which are sums of two bf16: the first is off by at most
  2^-8 of the value and the second by at most 2^-8 of that rest.
A capped score is off by a few U of itself (of 64 where a bf16 score is capped at no more than that): not of the cap.
The row sums of output gradient times output are those of the exact output for bf16 tensors; fp32 ones may take them from
the fp32 output (half a step of it).
"""
import numpy as np
import torch

from encoder_bounds import HALF, U, f64
import oracle.encoder as enc

TWO_PARTS = 2.0 ** -16
# fp32 and bf16 end at 2^-126: a weight, its product and its second part may each be flushed to zero below that, wherever the
# largest weight of a row is 1 or more (they are taken around a maximum that is never above the row's)
TINY = 2.0 ** -124


def oracle(q, k, v, how, go=None):
    """The oracle's results and the bounds of out, gq, gk, gv and gslope."""
    a = {n: (f64(t) if torch.is_tensor(t) and t.is_floating_point() else t.cpu().numpy() if torch.is_tensor(t) else t)
         for n, t in how.items()}
    a["cap"] = a.get("cap") or 0.0
    gn = None if go is None else f64(go)
    ref = enc.attention(f64(q), f64(k), f64(v), go=gn, **a)
    return ref, bounds(f64(q), f64(k), f64(v), ref, a, q.dtype, gn)


def bounds(q, k, v, ref, how, dtype, go=None):
    B, Tq, Hq, D = q.shape
    Tk, Hk = k.shape[1:3]
    G = Hq // Hk
    half, cap = HALF[dtype], how["cap"]
    low = TWO_PARTS if dtype == torch.bfloat16 else 0.0
    scale = abs(how.get("scale") or D ** -0.5)
    seen = ref["vis"].any(axis=1)[:, :, None, None]
    ka, va = np.where(seen, np.abs(k), 0.0), np.where(seen, np.abs(v), 0.0)
    res = {n: np.zeros_like(x) for n, x in (("out", q), ("gq", q), ("gk", k), ("gv", v))}
    res["gslope"] = np.zeros((B, Tq, Hq))
    for b in range(B):
        for h in range(Hq):
            kb, vb, vis = ka[b, :, h // G], va[b, :, h // G], ref["vis"][b]
            mag = scale * (np.abs(q[b, :, h]) @ kb.T)
            es = (D + 8) * U * mag + 4 * U * np.abs(ref["s"][b, h])
            if cap:
                es = es + 8 * U * np.minimum(cap, np.maximum(mag, 64.0 if low else 0.0))
            if "dist" in ref:
                es = es + 16 * U * np.abs(how["slope"][b, :, h, None]) * (
                    ref["dist"][b] + np.abs(how["pos_q"][b]).sum(-1)[:, None])
            es = np.where(vis, es, 0.0)
            es = es + U * np.abs(ref["s"][b, h]).max(initial=0.0)
            p = ref["p"][b, h]
            # the weights' own errors and those of their sum
            rel = 2 * es.max(axis=1, keepdims=True, initial=0.0) + 2 * (Tk + 16) * U
            pv = p @ vb
            eo = (rel + low) * pv * 1.01 + TINY * vb.sum(axis=0)
            o = np.abs(ref["out"][b, :, h])
            res["out"][b, :, h] = eo + half * (o + eo)
            if go is None:
                continue
            ga = np.abs(go[b, :, h])
            lse = ref["lse"][b, h]
            relp = 2 * rel + 4 * U * (1 + np.abs(np.where(np.isfinite(lse), lse, 0)))[:, None]
            edp = (D + 4) * U * (ga @ vb.T)
            dp, ds = np.abs(ref["dp"][b, h]), np.abs(ref["ds"][b, h])
            mean = (p * dp).sum(-1, keepdims=True)
            span = dp + mean
            if low:       # delta as the sum over the keys itself
                edelta = (p * (relp * span + edp)).sum(-1, keepdims=True) + (Tk + D + 16) * U * mean
            else:
                edelta = (ga * res["out"][b, :, h]).sum(-1, keepdims=True) + (D + 4) * U * (ga * o).sum(-1, keepdims=True)
            eds = p * (edelta + edp) + relp * p * span + TINY * (1 + span)
            sum_ds = np.abs(ref["dsc"][b, h]) + eds * 1.01
            edsc = (eds + low * ds) * 1.02 + (16 * U + 4 * es) * ds
            if "dist" in ref:
                d = ref["dist"][b]
                chain = 4 * (Tk + 16) * U
                egs = ((relp + chain) * p * span * d + p * edp * d).sum(-1)
                egs += (p * d).sum(-1) * ((relp + chain) * p * span + p * edp).sum(-1)
                egs += 2 * (relp.max(initial=0.0) + (Tk + 16) * U) * (edelta[:, 0] * (p * d).sum(-1))
                if low:
                    egs += edelta[:, 0] * (p * d).sum(-1)
                res["gslope"][b, :, h] = egs
            acc = 2 * (max(Tk, Tq * G) + 16) * U
            g = np.abs(ref["gq"][b, :, h])
            e = scale * ((edsc + acc * sum_ds) @ kb)
            res["gq"][b, :, h] = e + half * (g + e)
            res["gk"][b, :, h // G] += scale * ((edsc + acc * sum_ds).T @ np.abs(q[b, :, h]))
            res["gv"][b, :, h // G] += ((relp + low + acc) * p * 1.01 + TINY).T @ ga
    if go is not None:
        res["gk"] += half * (np.abs(ref["gk"]) + res["gk"])
        res["gv"] += half * (np.abs(ref["gv"]) + res["gv"])
    return res
