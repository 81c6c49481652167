"""CPU oracle for the encoder operators (group norm with an activation, rotary positions, attention), numpy float64.

TEST INFRASTRUCTURE ONLY.  Nothing in the product path may import this module.  It shares no code with the HIP path.

Layouts follow the library: maps [images, pixels, C]; queries [B, Tq, Hq, D]; keys and values [B, Tk, Hk, D].
The attention functions also return what error bounds need (probabilities and score gradients).
"""
from __future__ import annotations

import math
from typing import Dict, Optional, Tuple

import numpy as np

_erf = np.vectorize(math.erf, otypes=[np.float64])


def activation(z: np.ndarray, kind: str) -> Tuple[np.ndarray, np.ndarray]:
    """act(z) and its derivative (a ReLU's at 0 is 0)."""
    if kind == "none":
        return z, np.ones_like(z)
    if kind == "relu":
        return np.where(z > 0, z, 0.0), np.where(z > 0, 1.0, 0.0)
    if kind == "silu":
        with np.errstate(over="ignore"):
            s = 1.0 / (1.0 + np.exp(-z))
        return z * s, s + z * s * (1.0 - s)
    if kind == "gelu":
        cdf = 0.5 * (1.0 + _erf(z / math.sqrt(2.0)))
        return z * cdf, cdf + z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    raise ValueError(kind)


def group_norm(x: np.ndarray, groups: int, weight, bias, eps: float, kind: str, gy: Optional[np.ndarray] = None
               ) -> Dict[str, np.ndarray]:
    """x [I, S, C]; returns y, mean and rstd [I, G], and with gy the gradients gx, gw, gb."""
    x = np.asarray(x, np.float64)
    I, S, C = x.shape
    w = np.ones(C) if weight is None else np.asarray(weight, np.float64)
    b = np.zeros(C) if bias is None else np.asarray(bias, np.float64)
    xg = x.reshape(I, S, groups, C // groups)
    mean = xg.mean(axis=(1, 3))
    var = ((xg - mean[:, None, :, None]) ** 2).mean(axis=(1, 3))
    rstd = 1.0 / np.sqrt(var + eps)
    xh = ((xg - mean[:, None, :, None]) * rstd[:, None, :, None]).reshape(I, S, C)
    z = xh * w + b
    y, da = activation(z, kind)
    out = dict(y=y, z=z, xh=xh, mean=mean, rstd=rstd)
    if gy is not None:
        dz = np.asarray(gy, np.float64) * da
        u = (dz * w).reshape(I, S, groups, C // groups)
        xhg = xh.reshape(u.shape)
        m1 = u.mean(axis=(1, 3), keepdims=True)
        m2 = (u * xhg).mean(axis=(1, 3), keepdims=True)
        gx = rstd[:, None, :, None] * (u - m1 - xhg * m2)
        out.update(dz=dz, gx=gx.reshape(I, S, C), gw=(dz * xh).sum(axis=(0, 1)), gb=dz.sum(axis=(0, 1)))
    return out


def rotary(x: np.ndarray, pos: np.ndarray, freqs: np.ndarray, interleaved: bool, inverse: bool = False) -> np.ndarray:
    """x [B, T, H, D], pos [B, T, A], freqs [A, P]."""
    x = np.asarray(x, np.float64)
    P = freqs.shape[1]
    theta = np.asarray(pos, np.float64) @ np.asarray(freqs, np.float64)
    if inverse:
        theta = -theta
    c, s = np.cos(theta)[:, :, None], np.sin(theta)[:, :, None]
    y = x.copy()
    i1 = np.arange(P) * 2 if interleaved else np.arange(P)
    i2 = i1 + 1 if interleaved else i1 + P
    y[..., i1] = x[..., i1] * c - x[..., i2] * s
    y[..., i2] = x[..., i2] * c + x[..., i1] * s
    return y


def visible(B, Tq, Tk, doc_q=None, doc_k=None, causal=False, prefix=None) -> np.ndarray:
    """[B, Tq, Tk] bool: query i sees key j."""
    vis = np.ones((B, Tq, Tk), bool)
    if causal:
        i, j = np.arange(Tq)[:, None], np.arange(Tk)[None, :]
        for b in range(B):
            vis[b] &= (j <= i + Tk - Tq) | (j < (0 if prefix is None else int(prefix[b])))
    if doc_q is not None:
        dq, dk = np.asarray(doc_q)[:, :, None], np.asarray(doc_k)[:, None, :]
        vis &= (dq == dk) & (dq >= 0)
    return vis


def attention(q, k, v, *, scale=None, cap=0.0, pos_q=None, pos_k=None, slope=None, doc_q=None, doc_k=None,
              causal=False, prefix=None, go=None) -> Dict[str, np.ndarray]:
    """out, lse [B, Hq, Tq], p and s [B, Hq, Tq, Tk]; with go also gq, gk, gv, gslope, dp and ds."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    B, Tq, Hq, D = q.shape
    Tk, Hk = k.shape[1:3]
    G = Hq // Hk
    scale = D ** -0.5 if scale is None else scale
    vis = visible(B, Tq, Tk, doc_q, doc_k, causal, prefix)
    dist = None
    if pos_q is not None:
        d = np.asarray(pos_q, np.float64)[:, :, None] - np.asarray(pos_k, np.float64)[:, None]
        dist = np.where(vis, np.sqrt((d * d).sum(-1)), 0.0)
    out = np.zeros((B, Tq, Hq, D))
    lse = np.full((B, Hq, Tq), -np.inf)
    P = np.zeros((B, Hq, Tq, Tk))
    S = np.zeros((B, Hq, Tq, Tk))
    grads = {}
    if go is not None:
        go = np.asarray(go, np.float64)
        grads = dict(gq=np.zeros_like(q), gk=np.zeros_like(k), gv=np.zeros_like(v), dp=np.zeros_like(P),
                     ds=np.zeros_like(P), dsc=np.zeros_like(P))
        if dist is not None:
            grads["gslope"] = np.zeros((B, Tq, Hq))
    for b in range(B):
        seen_k = vis[b].any(axis=0)
        for h in range(Hq):
            # keys that no query sees hold anything
            kk = np.where(seen_k[:, None], k[b, :, h // G], 0.0)
            vv = np.where(seen_k[:, None], v[b, :, h // G], 0.0)
            s = scale * (q[b, :, h] @ kk.T)
            th = np.tanh(s / cap) if cap else None
            if cap:
                s = cap * th
            if dist is not None:
                s = s - np.asarray(slope, np.float64)[b, :, h, None] * dist[b]
            S[b, h] = np.where(vis[b], s, 0.0)
            if Tk == 0:
                continue
            masked = np.where(vis[b], s, -np.inf)
            m = masked.max(axis=1, keepdims=True)
            m = np.where(np.isfinite(m), m, 0.0)
            e = np.where(vis[b], np.exp(masked - m), 0.0)
            l = e.sum(axis=1, keepdims=True)
            with np.errstate(divide="ignore"):
                lse[b, h] = np.where(l[:, 0] > 0, m[:, 0] + np.log(l[:, 0]), -np.inf)
            p = e / np.where(l > 0, l, 1.0)
            P[b, h] = p
            out[b, :, h] = p @ vv
            if go is not None:
                g = go[b, :, h]
                dp = g @ vv.T
                ds = p * (dp - (p * dp).sum(axis=1, keepdims=True))
                grads["dp"][b, h], grads["ds"][b, h] = dp, ds
                if dist is not None:
                    grads["gslope"][b, :, h] = -(ds * dist[b]).sum(axis=1)
                dsc = ds * (1.0 - th * th) if cap else ds
                dsc = np.where(vis[b], dsc, 0.0)
                grads["dsc"][b, h] = dsc
                grads["gq"][b, :, h] = scale * (dsc @ kk)
                grads["gk"][b, :, h // G] += scale * (dsc.T @ q[b, :, h])
                grads["gv"][b, :, h // G] += p.T @ g
    res = dict(out=out, lse=lse, p=P, s=S, vis=vis, **grads)
    if dist is not None:
        res["dist"] = dist
    return res
