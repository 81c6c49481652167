"""CPU oracle for the decoder operators (root-mean-square norm, numbers in 8 bits, token cache, attention over it), numpy
float64.

TEST INFRASTRUCTURE ONLY.  Nothing in the product path may import this module.  It shares no code with the HIP path.

The cache is kept as the library lays it out: k [pages, Hk, 64, Dp] and v [pages, Hk, Dp, 64] code bytes (uint8),
k_scale and v_scale [pages, Hk, 64] float32.
"""
from __future__ import annotations

from typing import Dict, Optional, Tuple

import numpy as np

PAGE = 64
MOST = {"int8": 127.0, "e4m3": 448.0}


# ---- root-mean-square norm

def rms_norm(h: np.ndarray, weight: Optional[np.ndarray], eps: float, gy: Optional[np.ndarray] = None,
             gh: Optional[np.ndarray] = None) -> Dict[str, np.ndarray]:
    """h [rows, C] (the residual already added); with gy the gradients gx and gw too."""
    h = np.asarray(h, np.float64)
    w = np.ones(h.shape[1]) if weight is None else np.asarray(weight, np.float64)
    r = 1.0 / np.sqrt((h * h).mean(axis=1) + eps)
    out = dict(y=h * r[:, None] * w, rstd=r)
    if gy is not None:
        u = np.asarray(gy, np.float64) * w
        dot = (u * h).mean(axis=1)
        gx = r[:, None] * (u - h * (r * r * dot)[:, None])
        out.update(gx=gx if gh is None else gx + gh, gw=(gy * h * r[:, None]).sum(axis=0), u=u)
    return out


# ---- numbers in 8 bits

def numbers(kind: str) -> np.ndarray:
    """What each of the 256 bytes stands for (e4m3: sign, four bits of exponent with bias 7, three of mantissa)."""
    b = np.arange(256)
    if kind == "int8":
        return np.where(b < 128, b, b - 256).astype(np.float64)
    e, m = (b >> 3) & 15, b & 7
    x = np.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * 2.0 ** (e - 7.0))
    x = np.where((b & 127) == 127, np.nan, x)
    return np.where(b < 128, x, -x)


def _ladder(kind: str):
    """The format's numbers from 0 up to the largest, and the bytes of the positive ones; neighbours differ in the byte's
    last bit, so the even byte is the even number."""
    bytes_ = np.arange(128 if kind == "int8" else 127)
    return numbers(kind)[bytes_], bytes_


def codes(x: np.ndarray, scale: np.ndarray, kind: str) -> np.ndarray:
    """The bytes of the numbers nearest to x / scale, ties to the even one."""
    up, bytes_ = _ladder(kind)
    q = np.abs(np.asarray(x, np.float64) / np.asarray(scale, np.float64))
    q = np.minimum(q, MOST[kind])
    hi = np.clip(np.searchsorted(up, q), 1, len(up) - 1)
    down, above = q - up[hi - 1], up[hi] - q
    at = np.where((above < down) | ((above == down) & (hi % 2 == 0)), hi, hi - 1)
    neg = np.signbit(x)
    if kind == "int8":
        return np.where(neg, -bytes_[at], bytes_[at]).astype(np.int64).astype(np.uint8)
    return np.where(neg, bytes_[at] + 128, bytes_[at]).astype(np.uint8)


def row_codes(x: np.ndarray, kind: str) -> Tuple[np.ndarray, np.ndarray]:
    """(bytes [..., D], scale [...] float32) of rows of fp32 (or narrower) numbers."""
    top = np.abs(x).max(axis=-1).astype(np.float32)
    bad = ~np.isfinite(x).all(axis=-1)
    with np.errstate(invalid="ignore"):
        scale = np.maximum(top / np.float32(MOST[kind]), np.float32(2.0 ** -126))
    scale = np.where(bad, np.float32(1), scale)
    clean = np.where(bad[..., None], 0.0, x)
    return codes(clean, scale[..., None], kind), np.where(bad, np.float32(np.nan), scale).astype(np.float32)


# ---- token cache

class Cache:
    def __init__(self, pages: int, Hk: int, D: int, kind: str):
        Dp = -(-D // 16) * 16
        self.k = np.zeros((pages, Hk, PAGE, Dp), np.uint8)
        self.v = np.zeros((pages, Hk, Dp, PAGE), np.uint8)
        self.k_scale = np.zeros((pages, Hk, PAGE), np.float32)
        self.v_scale = np.zeros((pages, Hk, PAGE), np.float32)
        self.pages, self.D, self.kind = pages, D, kind

    def place(self, table, start, pos):
        """(page, slot) of a sequence's token, or None."""
        if start < 0 or pos // PAGE >= len(table):
            return None
        page = int(table[pos // PAGE])
        return (page, pos % PAGE) if 0 <= page < self.pages else None

    def write(self, k, v, table, start, count=None) -> None:
        B, T = k.shape[:2]
        for b in range(B):
            for t in range(T if count is None else min(T, max(0, int(count[b])))):
                at = self.place(table[b], int(start[b]), int(start[b]) + t)
                if at is None:
                    continue
                page, slot = at
                kc, ks = row_codes(k[b, t], self.kind)
                vc, vs = row_codes(v[b, t], self.kind)
                self.k[page, :, slot] = 0
                self.v[page, :, :, slot] = 0
                self.k[page, :, slot, :self.D] = kc
                self.v[page, :, :self.D, slot] = vc
                self.k_scale[page, :, slot], self.v_scale[page, :, slot] = ks, vs

    def token(self, page: int, slot: int):
        n = numbers(self.kind)
        k = n[self.k[page, :, slot, :self.D]] * self.k_scale[page, :, slot, None].astype(np.float64)
        v = n[self.v[page, :, :self.D, slot]] * self.v_scale[page, :, slot, None].astype(np.float64)
        return k, v

    def read(self, table, start, T, count=None):
        B, Hk = len(table), self.k.shape[1]
        k, v = np.zeros((B, T, Hk, self.D)), np.zeros((B, T, Hk, self.D))
        for b in range(B):
            for t in range(T if count is None else min(T, max(0, int(count[b])))):
                at = self.place(table[b], int(start[b]), int(start[b]) + t)
                if at is not None:
                    k[b, t], v[b, t] = self.token(*at)
        return k, v


# ---- attention over the cache

def attention(q: np.ndarray, cache: Cache, table, start, drafts: str, count=None, bits=None,
              scale: Optional[float] = None, cap: float = 0.0) -> Dict[str, list]:
    """q [B, T, Hq, D]; drafts: "none", "chain" or "tree" (bits [B, T, T] booleans).  Returns out, and per sequence what
    error bounds need: the tokens' keys and values k, v [n, Hk, D], which of them a query sees [T, n], probabilities p and
    scores s [Hq, T, n]."""
    B, T, Hq, D = q.shape
    Hk = cache.k.shape[1]
    G = Hq // Hk
    scale = D ** -0.5 if scale is None else scale
    res = dict(out=np.zeros_like(q, dtype=np.float64), k=[], v=[], seen=[], p=[], s=[])
    for b in range(B):
        n0 = int(start[b])
        rows = 0 if n0 < 0 else (T if count is None else min(T, max(0, int(count[b]))))
        places, seen = [], []
        for pos in range(max(0, min(n0 + (0 if drafts == "none" else rows), len(table[b]) * PAGE))):
            at = cache.place(table[b], n0, pos)
            if at is None:
                continue
            j = pos - n0
            col = np.zeros(T, bool)
            for t in range(rows):
                col[t] = j < 0 or (drafts == "chain" and j <= t) or (drafts == "tree" and bool(bits[b][t][j]))
            places.append(at)
            seen.append(col)
        n = len(places)
        kv = [cache.token(*at) for at in places]
        k = np.stack([x[0] for x in kv]) if n else np.zeros((0, Hk, D))
        v = np.stack([x[1] for x in kv]) if n else np.zeros((0, Hk, D))
        vis = np.stack(seen, axis=1) if n else np.zeros((T, 0), bool)
        ps, ss = np.zeros((Hq, T, n)), np.zeros((Hq, T, n))
        for h in range(Hq):
            with np.errstate(invalid="ignore"):
                s = scale * (q[b, :, h].astype(np.float64) @ k[:, h // G].T)
            if cap:
                s = cap * np.tanh(s / cap)
            s = np.where(vis, s, -np.inf)
            m = s.max(axis=1, initial=-np.inf)
            e = np.where(vis, np.exp(s - np.where(np.isfinite(m), m, 0.0)[:, None]), 0.0)
            total = e.sum(axis=1)
            p = e / np.where(total == 0, 1.0, total)[:, None]
            ps[h], ss[h] = p, np.where(vis, s, 0.0)
            for t in range(T):
                at = np.flatnonzero(vis[t])
                res["out"][b, t, h] = p[t, at] @ v[at, h // G]
        for name, x in (("k", k), ("v", v), ("seen", vis), ("p", ps), ("s", ss)):
            res[name].append(x)
    return res
