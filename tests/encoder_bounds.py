"""Error bounds of the encoder operators against the fp64 oracle, from the arithmetic alone.

U = 2^-24 is half a step of fp32.  A rounding to a tensor's type is off by at most finfo(type).eps / 2 of the value.
An fp32 sum whose longest chain of additions has n terms is off by at most n U times the sum of magnitudes; CHAIN
bounds the chains of the norm kernels at the tested sizes (16 pieces of a thread, 8 channels of a piece, up to 128
terms of a lane's share of the workgroup's sums, 6 lane steps and the merge of at most 64 chunks, which lanes share
where there are more).
"""
import numpy as np
import torch

import oracle.encoder as enc

U = 2.0 ** -24
CHAIN = 256
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def f64(t):
    return t.detach().double().cpu().numpy()


def close(name, got, ref, bound):
    got = f64(got)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    err = np.abs(got - ref)
    bad = ~(err <= bound)
    worst = float((err / np.maximum(bound, 1e-300)).max(initial=0.0)) if not bad.any() else None
    print(f"[bound] {name}: max|d|={err.max(initial=0.0):.3e} share of the bound={worst}", flush=True)
    assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.size} outside, first at {np.argwhere(bad)[0]}: " \
                          f"{got[tuple(np.argwhere(bad)[0])]} against {ref[tuple(np.argwhere(bad)[0])]}"


def norm_bounds(x, groups, weight, bias, kind, ref, gy, dtype):
    """Bounds of y, gx, gw, gb (the gradients with gy) and of z."""
    I, S, C = x.shape
    G, cg = groups, C // groups
    w = np.ones(C) if weight is None else np.abs(weight)
    b = np.zeros(C) if bias is None else np.abs(bias)
    spread = lambda a: np.repeat(a, cg, axis=-1)[:, None, :]       # [I, G] -> [I, 1, C]
    mean, rstd = spread(np.abs(ref["mean"])), spread(ref["rstd"])
    size = spread(np.abs(x).reshape(I, S, G, cg).mean(axis=(1, 3)))
    xh = np.abs(ref["xh"])
    # mean off by CHAIN U size, x - mean by U (|x| + |mean|), rstd by (CHAIN + 8) U
    exh = U * (rstd * ((CHAIN + 4) * size + 4 * (np.abs(x) + mean)) + (CHAIN + 8) * xh)
    ez = w * exh + 4 * U * (w * (xh + rstd * mean) + b)
    # |act'| <= 1.13; the exponential's argument and result are off by (|z| + 8) U
    y = np.abs(ref["y"])
    ey = 1.13 * ez + U * (np.abs(ref["z"]) + 8) * 2 * (y + np.abs(ref["z"]) * (kind != "none")) + HALF[dtype] * y
    ey = ey + HALF[dtype] * ey
    res = dict(y=ey, z=ez)
    if gy is not None:
        g = np.abs(gy)
        # |act''| <= 1.0 (SiLU 0.5, GELU 0.8); the derivative itself is off by (|z| + 8) 4 U
        edz = g * (ez * (kind in ("silu", "gelu")) + 4 * U * (np.abs(ref["z"]) + 8))
        if kind == "relu":      # the derivative jumps where z may round across zero
            edz = edz + g * (np.abs(ref["z"]) <= ez)
        dz = np.abs(ref["dz"])
        u, eu = dz * w, edz * w + 2 * U * dz * w
        gm = lambda a: spread(a.reshape(I, S, G, cg).mean(axis=(1, 3)))
        em1 = gm(eu) + 2 * CHAIN * U * gm(u)
        em2 = gm(eu * xh + u * exh) + 2 * CHAIN * U * gm(u * xh)
        m2 = gm(u * xh)
        egx = rstd * (eu + em1 + xh * em2 + exh * m2 + 4 * U * (u + gm(u) + xh * m2)) \
            + (CHAIN + 8) * U * rstd * (u + gm(u) + xh * m2)
        res["gx"] = egx + HALF[dtype] * (np.abs(ref["gx"]) + egx)
        res["gb"] = (edz + 4 * CHAIN * U * dz).sum(axis=(0, 1))
        res["gw"] = (edz * xh + dz * exh + 4 * CHAIN * U * dz * xh).sum(axis=(0, 1))
    return res


def attention_bounds(q, k, v, ref, how, dtype, go=None, split=False):
    """Bounds of out (and of gq, gk, gv, gslope with go).  Probabilities are relative to their own size: a score
    off by e moves them by 2 e, the sum of Tk weights by Tk U."""
    B, Tq, Hq, D = q.shape
    Tk, Hk = k.shape[1:3]
    G = Hq // Hk
    half = HALF[dtype]
    cap = how.get("cap") or 0.0
    scale = abs(how.get("scale") or D ** -0.5)
    vis = ref["vis"].any(axis=1)                                        # [B, Tk]
    kk = np.where(vis[:, :, None, None], np.abs(k), 0.0)
    vv = np.where(vis[:, :, None, None], np.abs(v), 0.0)
    res = {n: np.zeros_like(a) for n, a in (("out", q), ("gq", q), ("gk", k), ("gv", k))}
    res["lse"] = np.zeros((B, Hq, Tq))
    res["gslope"] = np.zeros((B, Tq, Hq))
    for b in range(B):
        for h in range(Hq):
            # products of D terms and the running maximum's shift; the cap's tanh and the distance a few U each
            mag = scale * (np.abs(q[b, :, h]) @ kk[b, :, h // G].T)
            es = (D + 8) * U * mag + 8 * U * cap + 4 * U * np.abs(ref["s"][b, h])
            if "dist" in ref:
                es = es + 16 * U * np.abs(how["slope"][b, :, h, None]) * (
                    ref["dist"][b] + np.abs(how["pos_q"][b]).sum(-1)[:, None])
            es = np.where(ref["vis"][b], es, 0.0)
            es = es + U * np.abs(ref["s"][b, h]).max(initial=0.0)
            p = ref["p"][b, h]
            rel = 2 * es.max(axis=1, keepdims=True, initial=0.0) + 2 * (Tk + 16) * U
            va = vv[b, :, h // G]
            pv = p @ va
            # bf16 probabilities are rounded before their product
            low = half if dtype == torch.bfloat16 else 0.0
            eo = (rel + low) * pv * 1.01
            res["out"][b, :, h] = eo + half * (np.abs(ref["out"][b, :, h]) + eo)
            res["lse"][b, h] = rel[:, 0] + 4 * U * (1 + np.abs(np.where(np.isfinite(ref["lse"][b, h]), ref["lse"][b, h], 0)))
            if go is None:
                continue
            ga = np.abs(go[b, :, h])
            edelta = (ga * res["out"][b, :, h]).sum(-1, keepdims=True) + (D + 4) * U * (ga * np.abs(ref["out"][b, :, h])).sum(-1, keepdims=True)
            edp = (D + 4) * U * (ga @ va.T)
            ds, dp = np.abs(ref["ds"][b, h]), np.abs(ref["dp"][b, h])
            # p from the rounded lse: rel again, and U |lse|
            relp = 2 * rel + 4 * U * (1 + np.abs(np.where(np.isfinite(ref["lse"][b, h]), ref["lse"][b, h], 0)))[:, None]
            span = dp + (p * dp).sum(-1, keepdims=True)
            eds = p * (edelta + edp) + relp * p * span
            sum_ds = np.abs(ref["dsc"][b, h]) + eds * 1.01
            edsc = (eds + low * ds) * 1.02 + (16 * U + 4 * es) * ds
            # the slope's gradient carries the probabilities' sum instead of the rounded delta
            if "dist" in ref:
                d = ref["dist"][b]
                egs = ((relp + 4 * (Tk + 16) * U) * p * span * d + p * edp * d).sum(-1)
                egs += (p * d).sum(-1) * ((relp + 4 * (Tk + 16) * U) * p * span + p * edp).sum(-1)
                egs += 2 * (relp.max(initial=0.0) + (Tk + 16) * U) * (edelta[:, 0] * (p * d).sum(-1))
                res["gslope"][b, :, h] = egs
            acc = 2 * (max(Tk, Tq * G) + 16) * U
            gq = np.abs(ref["gq"][b, :, h])
            e = scale * ((edsc + acc * sum_ds) @ kk[b, :, h // G])
            res["gq"][b, :, h] = e + half * (gq + e)
            res["gk"][b, :, h // G] += scale * ((edsc + acc * sum_ds).T @ np.abs(q[b, :, h]))
            res["gv"][b, :, h // G] += ((relp + low + acc) * p * 1.01).T @ ga
    if go is not None:
        res["gk"] += half * (np.abs(ref["gk"]) + res["gk"])
        res["gv"] += half * (np.abs(ref["gv"]) + res["gv"])
    return res


def oracle_attention(q, k, v, how, go=None):
    a = {n: (f64(t) if torch.is_tensor(t) and t.is_floating_point() else t.cpu().numpy() if torch.is_tensor(t) else t)
         for n, t in how.items()}
    if a.get("slope") is not None and a["slope"].ndim == 1:
        a["slope"] = np.broadcast_to(a["slope"], (q.shape[0], q.shape[1], q.shape[2]))
    a["cap"] = a.get("cap") or 0.0
    qn, kn, vn = f64(q), f64(k), f64(v)
    ref = enc.attention(qn, kn, vn, go=None if go is None else f64(go), **a)
    bounds = attention_bounds(qn, kn, vn, ref, a, q.dtype, None if go is None else f64(go))
    return ref, bounds
