"""PyTorch-facing calls of the decoder operators: argument marshalling only.

Root-mean-square norm with the residual's addition (and an output in 8 bits), the token cache in 8 bits, and attention
of query tokens, trees of drafted ones among others, over that cache.  ``camera_bev_view_amd.ops`` re-exports them beside
the encoder operators.
"""
from __future__ import annotations

import ctypes
import functools
import struct
from typing import Optional, Sequence, Tuple

import torch
from torch.autograd.function import once_differentiable

from . import _lib
from .encoder import (_DTYPES, _check_apart, _check_plain, _check_sizes, _check_values, _collapse, _data, _device,
                      _raw_stream, _scratch)

_CODES = {torch.int8: _lib.FBEV_CODES_INT8, torch.float8_e4m3fn: _lib.FBEV_CODES_E4M3}
_PAGE = _lib.FBEV_CACHE_PAGE
_F32, _I32 = torch.float32, torch.int32
_set = object.__setattr__

# A call's own time counts where a step of serving is a few small ones: descriptors are packed as bytes (a tenth of a
# ctypes structure's time; the layouts are the structures' of _lib) and go as plain pointers.
_pack_rms = struct.Struct("@6qif").pack
_pack_cache = struct.Struct("@4i4P").pack
_pack_rows = struct.Struct("@3i4x3P").pack
_pack_attention = struct.Struct("@3i4x3qP2f").pack
_pack_strides = struct.Struct("@3q").pack
_P, _I, _Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
_ARGS = {"fbev_rms_norm_forward": [_P, _P, _I, _P, _P, _P, _P, _P, _P],
         "fbev_rms_norm_codes": [_P, _P, _I, _P, _P, _I, _I, _P, _P, _P, _P],
         "fbev_rms_norm_backward": [_P, _P, _P, _I, _P, _P, _P, _P, _P, _P, _Z, _P],
         "fbev_cache_write": [_P, _P, _P, _P, _I, _P, _P, _P],
         "fbev_cache_read": [_P, _P, _I, _P, _P, _P],
         "fbev_cache_attention": [_P, _P, _P, _P, _I, _P, _P, _Z, _P]}


@functools.lru_cache(maxsize=None)
def _function(name: str):
    fn = _lib.load()[name]              # a handle of its own: the library's takes structures
    fn.argtypes, fn.restype = _ARGS[name], _I
    return fn


def _call(name: str, dev: torch.device, *args) -> None:
    """The library's ``name``(*args, stream) on the current stream of ``dev``, with that device current."""
    fn, index = _function(name), dev.index
    if _device() == index:
        status = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(dev):
            status = fn(*args, _raw_stream(index))
    if status:
        _lib.check(status)


class _NoBackward(torch.autograd.Function):
    """The result of a call without a backward, as a part of its inputs' graph: a gradient that arrives there is an error
    and not lost."""

    @staticmethod
    def forward(ctx, name, result, *inputs):
        ctx.name = name
        return result.view_as(result)

    @staticmethod
    def backward(ctx, grad):
        raise RuntimeError(f"{ctx.name} has no backward: call it under torch.no_grad() or on detached tensors")


def _without_backward(name: str, result: torch.Tensor, *inputs: Optional[torch.Tensor]) -> torch.Tensor:
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in inputs):
        return _NoBackward.apply(name, result, *inputs)
    return result


# ---- root-mean-square norm

@functools.lru_cache(maxsize=1024)
def _rms_scratch(rows: int, C: int, dtype: int) -> int:
    lib, need = _lib.load(), ctypes.c_size_t()
    _lib.check(lib.fbev_rms_norm_workspace(_lib.RmsDesc(rows, 1, (0, 0), (0, 0), C, 0.0), dtype, ctypes.byref(need)))
    return need.value


def _rows(x: torch.Tensor, other: Optional[torch.Tensor]):
    """(outer, inner, x's strides of them, other's strides): how to walk the rows of both, or None."""
    lead = x.dim() - 1
    for t in (x, other):
        if t is not None and t.shape[-1] > 1 and t.stride(-1) != 1:
            return None
    if lead == 2:                       # two strides as they are (the library joins them where it can)
        return (*x.shape[:2], *x.stride()[:2], *((0, 0) if other is None else other.stride()[:2]))
    for cut in range(lead, -1, -1):
        strides = []
        for t in (x, other):
            if t is None:
                strides += [0, 0]
                continue
            so, si = _collapse(t.shape[:cut], t.stride()[:cut]), _collapse(t.shape[cut:lead], t.stride()[cut:lead])
            if so is None or si is None:
                break
            strides += [so, si]
        if len(strides) == 4:
            outer = inner = 1
            for n in x.shape[:cut]:
                outer *= n
            for n in x.shape[cut:lead]:
                inner *= n
            return (outer, inner, *strides)
    return None


def _rms_desc(x: torch.Tensor, residual: Optional[torch.Tensor], weight, eps: float):
    """(x, residual, rows, C, packed descriptor); x and residual copied where two strides do not walk their rows."""
    shape, dev = x.shape, x.device
    if not shape:
        raise ValueError("x must be [..., C]")
    if not x.is_cuda:
        raise ValueError("x must be a device tensor")
    if x.dtype not in _DTYPES:
        raise ValueError(f"x must be float32 or bfloat16, got {x.dtype}")
    if residual is not None and (residual.shape != shape or residual.dtype != x.dtype or residual.device != dev):
        raise ValueError(f"residual must be a {x.dtype} tensor of shape {list(shape)} on {dev}")
    C = shape[-1]
    _check_sizes(C)
    if weight is not None and not (weight.shape == (C,) and weight.dtype == _F32 and weight.device == dev
                                   and weight.is_contiguous()):
        _check_plain("weight", weight, (C,), _F32, dev)
    if x.is_contiguous() and (residual is None or residual.is_contiguous()):
        rows = x.numel() // C if C else 0
        return x, residual, rows, C, _pack_rms(rows, 1, C, 0, C, 0, C, eps)
    walk = _rows(x, residual)
    if walk is None:
        return _rms_desc(x.contiguous(), None if residual is None else residual.contiguous(), weight, eps)
    return x, residual, walk[0] * walk[1], C, _pack_rms(*walk, C, eps)


def rms_norm_forward(x: torch.Tensor, weight: Optional[torch.Tensor] = None, *,
                     residual: Optional[torch.Tensor] = None, eps: float = 1e-6, out: Optional[torch.Tensor] = None,
                     h_out: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """fbev_rms_norm_forward on rows of channels x [..., C] (fp32 or bf16): h = x + residual (like x; rounded once), y = h
    weight / sqrt(mean h^2 + eps).  ``weight`` [C] is contiguous fp32.  Rows may lie at two strides (heads of a packed
    projection); other layouts are copied first.  ``h_out`` may be x or residual themselves, where contiguous.
    Returns (y, h, rstd [...] fp32); h is x without a residual.  The backward takes h and rstd.  Results are no part of a
    graph: rms_norm and rms_norm_add are the differentiable calls."""
    dev = x.device
    x, residual, _, _, rd = _rms_desc(x, residual, weight, eps)
    if out is None:
        y = torch.empty_like(x, memory_format=torch.contiguous_format)
    else:
        y = out
        _check_plain("out", out, x.shape, x.dtype, dev)
        _check_apart("out", out, x, residual, weight, h_out)
    h = _sum_out(h_out, x, residual, weight)
    rstd = torch.empty(x.shape[:-1], dtype=_F32, device=dev)
    _call("fbev_rms_norm_forward", dev, _data(x), _data(residual), _DTYPES[x.dtype], rd, _data(weight), _data(y),
          None if residual is None else _data(h), _data(rstd))
    return y, h, rstd


def _sum_out(h_out, x, residual, weight) -> torch.Tensor:
    if residual is None:
        if h_out is not None:
            raise ValueError("h_out comes with a residual")
        return x
    if h_out is None:
        return torch.empty_like(x, memory_format=torch.contiguous_format)
    _check_plain("h_out", h_out, x.shape, x.dtype, x.device)
    for t in (x, residual):
        if not (t.data_ptr() == h_out.data_ptr() and t.is_contiguous()):
            _check_apart("h_out, unless it is x or residual itself,", h_out, t)
    _check_apart("h_out", h_out, weight)
    return h_out


def rms_norm_codes(x: torch.Tensor, weight: Optional[torch.Tensor] = None, *,
                   residual: Optional[torch.Tensor] = None, eps: float = 1e-6,
                   codes: torch.dtype = torch.float8_e4m3fn, block: int = 128, h_out: Optional[torch.Tensor] = None
                   ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """fbev_rms_norm_codes: rms_norm_forward with y in 8 bits (``codes``: torch.int8 or torch.float8_e4m3fn) and a scale for each ``block``
    channels (32, 64 or 128; 0: one for the row).  Returns (codes like x, scales [..., blocks] fp32, h): a code stands for
    code * scale.  Forward only: a gradient that reaches scales or h is an error."""
    if codes not in _CODES:
        raise ValueError(f"codes must be torch.int8 or torch.float8_e4m3fn, got {codes}")
    dev = x.device
    x, residual, _, C, rd = _rms_desc(x, residual, weight, eps)
    _check_sizes(block)
    out = torch.empty_like(x, dtype=codes, memory_format=torch.contiguous_format)
    blocks = -(-C // block) if 0 < block < C else 1
    scales = torch.empty(*x.shape[:-1], blocks, dtype=_F32, device=dev)         # (a tuple takes 0.35 us longer)
    h = _sum_out(h_out, x, residual, weight)
    _call("fbev_rms_norm_codes", dev, _data(x), _data(residual), _DTYPES[x.dtype], rd, _data(weight), _CODES[codes],
          block, _data(out), _data(scales), None if residual is None else _data(h))
    if x.requires_grad or (residual is not None and residual.requires_grad) or (weight is not None and weight.requires_grad):
        scales = _without_backward("rms_norm_codes", scales, x, residual, weight)
        if residual is not None:
            h = _without_backward("rms_norm_codes", h, x, residual, weight)
    return out, scales, h


def rms_norm_backward(grad_y: torch.Tensor, h: torch.Tensor, rstd: torch.Tensor,
                      weight: Optional[torch.Tensor] = None, *, grad_h: Optional[torch.Tensor] = None,
                      with_weight: bool = True, workspace: Optional[torch.Tensor] = None
                      ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """fbev_rms_norm_backward: (grad_x, which is the residual's gradient too, contiguous; grad_weight [C] fp32, or None
    without ``with_weight``) from dL/dy, the forward's h and rstd, and ``grad_h``, dL/dh from elsewhere (the residual stream)."""
    dev = h.device
    h, _, rows, C, rd = _rms_desc(h, None, weight, 0.0)
    for name, g in (("grad_y", grad_y), ("grad_h", grad_h)):
        if g is not None and (g.shape != h.shape or g.dtype != h.dtype or g.device != dev):
            raise ValueError(f"{name} must be a {h.dtype} tensor of shape {list(h.shape)} on {dev}")
    grad_y = grad_y.contiguous()
    grad_h = None if grad_h is None else grad_h.contiguous()
    _check_plain("rstd", rstd, h.shape[:-1], torch.float32, dev)
    gx = torch.empty_like(h, memory_format=torch.contiguous_format)
    gw = torch.empty(C, dtype=_F32, device=dev) if with_weight else None
    need = _rms_scratch(rows, C, _DTYPES[h.dtype]) if with_weight else 0
    workspace, have = _scratch(need, workspace, dev)
    _call("fbev_rms_norm_backward", dev, _data(grad_y), _data(grad_h), _data(h), _DTYPES[h.dtype], rd, _data(weight),
          _data(rstd), _data(gx), _data(gw), _data(workspace), have)
    return gx, gw


class RmsNorm(torch.autograd.Function):
    """Autograd wrapper of the root-mean-square norm; with a residual it returns (y, x + residual)."""

    @staticmethod
    def forward(ctx, x, residual, weight, eps):
        y, h, rstd = rms_norm_forward(x, weight, residual=residual, eps=eps)
        ctx.save_for_backward(h, rstd, weight)
        ctx.set_materialize_grads(False)
        ctx.both = residual is not None
        return (y, h) if ctx.both else y

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_y, grad_h=None):
        h, rstd, weight = ctx.saved_tensors
        want = ctx.needs_input_grad
        if grad_y is None:
            return grad_h if want[0] else None, grad_h if want[1] else None, None, None
        gx, gw = rms_norm_backward(grad_y, h, rstd, weight, grad_h=grad_h, with_weight=want[2])
        return gx if want[0] else None, gx if want[1] else None, gw, None


def rms_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, *, eps: float = 1e-6) -> torch.Tensor:
    """Differentiable x weight / sqrt(mean x^2 + eps) over the last dimension (see rms_norm_forward)."""
    return RmsNorm.apply(x, None, weight, eps)


def rms_norm_add(x: torch.Tensor, residual: torch.Tensor, weight: Optional[torch.Tensor] = None, *,
                 eps: float = 1e-6) -> Tuple[torch.Tensor, torch.Tensor]:
    """Differentiable (rms_norm(h), h) of h = x + residual: a layer's output joins the residual stream and is normalised
    for the next one."""
    return RmsNorm.apply(x, residual, weight, eps)


# ---- token cache

class TokenCache:
    """Keys and values of many sequences in 8 bits, in pages of 64 tokens: codes k [pages, Hk, 64, Dp] and v [pages, Hk,
    Dp, 64] (torch.int8 or torch.float8_e4m3fn; Dp: D rounded up to a multiple of 16, zeros behind D) and k_scale, v_scale
    [pages, Hk, 64] fp32, contiguous tensors of one device.  Which page belongs to which sequence is the caller's table.

    The tensors are its own from then on: they can be written in place but not replaced, and a call on a cache whose tensors
    have been resized or given other memory is refused.  A larger cache is a new one; deep and pickled copies have tensors of their own."""

    __slots__ = ("_held",)

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor, D: int):
        shape, dtype, dev = k.shape, k.dtype, k.device
        if len(shape) != 4 or dtype not in _CODES:
            raise ValueError(f"k must be [pages, Hk, {_PAGE}, Dp] of torch.int8 or torch.float8_e4m3fn")
        if not k.is_cuda:
            raise ValueError("k must be a device tensor")
        pages, Hk, Dp = shape[0], shape[1], -(-D // 16) * 16
        _check_sizes(pages, Hk, D)
        side = (pages, Hk, _PAGE)
        if not (shape == (pages, Hk, _PAGE, Dp) and k.is_contiguous()
                and v.shape == (pages, Hk, Dp, _PAGE) and v.is_contiguous() and v.dtype == dtype and v.device == dev
                and k_scale.shape == side and k_scale.is_contiguous() and k_scale.dtype == _F32
                and k_scale.device == dev and v_scale.shape == side and v_scale.is_contiguous()
                and v_scale.dtype == _F32 and v_scale.device == dev):
            for name, t, want, kind in (("k", k, (pages, Hk, _PAGE, Dp), dtype), ("v", v, (pages, Hk, Dp, _PAGE), dtype),
                                        ("k_scale", k_scale, side, _F32), ("v_scale", v_scale, side, _F32)):
                _check_plain(name, t, want, kind, dev)
        # addresses and sizes as they are now, and where to ask for them again
        a, b, c, d = look = k.data_ptr, v.data_ptr, k_scale.data_ptr, v_scale.data_ptr
        where, n = (a(), b(), c(), d()), pages * Hk * _PAGE
        _set(self, "_held", (k, v, k_scale, v_scale, D, Hk, pages, dev, _pack_cache(pages, Hk, D, _CODES[dtype], *where),
                             (*where, n * Dp, n * Dp, n, n), (*look, k.numel, v.numel, k_scale.numel, v_scale.numel)))

    def __setattr__(self, name, value):
        raise AttributeError(f"a TokenCache is fixed once made: {name} cannot be set (make a new one)")

    def __reduce__(self):
        return TokenCache, self._held[:5]

    k = property(lambda self: self._held[0])
    v = property(lambda self: self._held[1])
    k_scale = property(lambda self: self._held[2])
    v_scale = property(lambda self: self._held[3])
    D = property(lambda self: self._held[4])
    Hk = property(lambda self: self._held[5])
    pages = property(lambda self: self._held[6])
    device = property(lambda self: self._held[7])

    @property
    def desc(self) -> bytes:
        """The packed descriptor, for a call at once: its addresses have been looked at again."""
        return _cache_desc(self._held)


def _cache_desc(held) -> bytes:
    _, _, _, _, _, _, _, _, desc, where, (a, b, c, d, e, f, g, h) = held
    if where != (a(), b(), c(), d(), e(), f(), g(), h()):
        raise ValueError("the cache's tensors have been resized or moved: make a new TokenCache of them")
    return desc


def token_cache(pages: int, Hk: int, D: int, *, codes: torch.dtype = torch.float8_e4m3fn, device="cuda") -> TokenCache:
    """An empty cache of ``pages`` pages for ``Hk`` key heads of ``D`` channels."""
    Dp = -(-D // 16) * 16
    if codes not in _CODES:
        raise ValueError(f"codes must be torch.int8 or torch.float8_e4m3fn, got {codes}")
    return TokenCache(torch.zeros((pages, Hk, _PAGE, Dp), dtype=torch.uint8, device=device).view(codes),
                      torch.zeros((pages, Hk, Dp, _PAGE), dtype=torch.uint8, device=device).view(codes),
                      torch.zeros((pages, Hk, _PAGE), dtype=torch.float32, device=device),
                      torch.zeros((pages, Hk, _PAGE), dtype=torch.float32, device=device), D)


def _cache_rows(dev, table, start, count, B: int, T: int) -> bytes:
    shape = table.shape
    if len(shape) != 2 or shape[0] != B:
        raise ValueError(f"table must be [B={B}, pages of a sequence], got {tuple(shape)}")
    _check_sizes(B, T, shape[1])
    if not (table.dtype == _I32 and table.device == dev and table.is_contiguous()
            and start.dtype == _I32 and start.device == dev and start.shape == (B,) and start.is_contiguous()
            and (count is None or count.dtype == _I32 and count.device == dev and count.shape == (B,)
                 and count.is_contiguous())):
        for name, t, want in (("table", table, shape), ("start", start, (B,)), ("count", count, (B,))):
            if t is not None:
                _check_plain(name, t, want, _I32, dev)
    return _pack_rows(B, T, shape[1], table.data_ptr(), start.data_ptr(), 0 if count is None else count.data_ptr())


def cache_write(cache: TokenCache, k: torch.Tensor, v: torch.Tensor, table: torch.Tensor, start: torch.Tensor, *,
                count: Optional[torch.Tensor] = None) -> None:
    """fbev_cache_write: rows k, v [B,T,Hk,D] (fp32 or bf16) become the tokens start[b] .. start[b] + count[b] (T without
    ``count``) of their sequences, whose pages ``table`` [B,W] names (all int32).  Padding and rows without a page are
    dropped.  No token may be written twice in a call.  The cache holds no gradients: what k and v were made from gets none."""
    held = cache._held
    _, _, _, _, D, Hk, _, dev, _, _, _ = held
    shape, dtype = k.shape, k.dtype
    if not (len(shape) == 4 and dtype in _DTYPES and k.device == dev and v.dtype == dtype and v.device == dev):
        _check_values("k", k, 4, dev)
        _check_values("v", v, 4, dev, dtype)
    if v.shape != shape or shape[2] != Hk or shape[3] != D:
        raise ValueError(f"k {tuple(shape)} and v {tuple(v.shape)} must be [B, T, Hk={Hk}, D={D}]")
    ks, vs = k.stride(), v.stride()
    if D > 1 and (ks[3] != 1 or vs[3] != 1):
        k, v = k.contiguous(), v.contiguous()
        ks, vs = k.stride(), v.stride()
    cr = _cache_rows(dev, table, start, count, shape[0], shape[1])
    _call("fbev_cache_write", dev, _cache_desc(held), cr, k.data_ptr(), v.data_ptr(), _DTYPES[dtype],
          _pack_strides(*ks[:3]), _pack_strides(*vs[:3]))


def cache_read(cache: TokenCache, table: torch.Tensor, start: torch.Tensor, T: int, *,
               count: Optional[torch.Tensor] = None, dtype: torch.dtype = torch.bfloat16
               ) -> Tuple[torch.Tensor, torch.Tensor]:
    """fbev_cache_read: (k, v) [B,T,Hk,D] of ``dtype``, what the codes of the tokens start[b] .. start[b] + T stand for; zeros
    from count[b] on and where there is no page."""
    if dtype not in _DTYPES:
        raise ValueError(f"dtype must be float32 or bfloat16, got {dtype}")
    held = cache._held
    _, _, _, _, D, Hk, _, dev, _, _, _ = held
    shape = table.shape
    B = shape[0] if shape else 0
    cr = _cache_rows(dev, table, start, count, B, T)
    k = torch.empty(B, T, Hk, D, dtype=dtype, device=dev)
    v = torch.empty_like(k)
    _call("fbev_cache_read", dev, _cache_desc(held), cr, _DTYPES[dtype], k.data_ptr(), v.data_ptr())
    return k, v


# ---- attention over the cache

@functools.lru_cache(maxsize=1024)
def _cache_attention_scratch(B: int, T: int, W: int, Hq: int, Hk: int, D: int, dtype: int) -> int:
    lib, need = _lib.load(), ctypes.c_size_t()
    cd = _lib.CacheDesc(0, Hk, D, 0, None, None, None, None)
    cr = _lib.CacheRows(B, T, W, 16, 16, None)            # not dereferenced
    ad = _lib.CacheAttentionDesc(Hq, _lib.FBEV_DRAFT_NONE, 0, (0, 0, 0), None, 1.0, 0.0)
    _lib.check(lib.fbev_cache_attention_workspace(cd, cr, ad, dtype, ctypes.byref(need)))
    return need.value


def tree_ancestors(parents: Sequence, *, device="cuda") -> torch.Tensor:
    """The ``ancestors`` of cache_attention from each drafted token's parent among them (-1: none, it follows the cache):
    [T] parents give [1, T, words], [B, T] give [B, T, words] (int64 bits).  A token sees its ancestors and itself.  Made on
    the host: parents on the device are waited for, so a captured step takes ancestors made before it."""
    rows = parents.tolist() if torch.is_tensor(parents) else [list(p) if hasattr(p, "__len__") else p for p in parents]
    shape = tuple(getattr(parents, "shape", ()))        # of a tensor or an array: a batch of none still has its T
    if len(shape) != 2 and (not rows or not isinstance(rows[0], list)):
        rows = [rows]
    T = shape[1] if len(shape) == 2 else len(rows[0])
    if any(len(r) != T for r in rows):
        raise ValueError("every tree must have the same number of tokens")
    words, out = max(1, -(-T // 64)), []
    for r in rows:
        masks = []
        for j, p in enumerate(r):
            if not -1 <= p < j:
                raise ValueError(f"token {j} has parent {p}: a parent comes before its children (-1: none)")
            masks.append((masks[p] if p >= 0 else 0) | 1 << j)
        cut = [[m >> 64 * w & (1 << 64) - 1 for w in range(words)] for m in masks]
        out.append([[x - (1 << 64) if x >> 63 else x for x in m] for m in cut])
    return torch.tensor(out, dtype=torch.int64).reshape(len(rows), T, words).to(device)


def cache_attention(q: torch.Tensor, cache: TokenCache, table: torch.Tensor, start: torch.Tensor, *,
                    count: Optional[torch.Tensor] = None, ancestors: Optional[torch.Tensor] = None,
                    drafted: bool = True, scale: Optional[float] = None, cap: Optional[float] = None,
                    out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """fbev_cache_attention: queries q [B,T,Hq,D] (fp32 or bf16; Hq a multiple of the cache's Hk) over the tokens of their
    sequences, out [B,T,Hq,D].

    Every query sees the start[b] tokens of the cache.  The call's own tokens, written to the cache before as start[b] ..
    start[b] + T, are seen up to the query's own (a prompt, a single token), or as ``ancestors`` [B or 1,T,words] int64 says: bit j % 64
    of word j / 64 for token j (a tree of drafted tokens; see tree_ancestors), or not at all when not ``drafted``
    (queries that are not tokens of the cache).  Tokens and queries from count[b] on are padding; they, and queries that
    see nothing, get zeros.  ``scale``: 1 / sqrt(D) unless given; ``cap``: scores become cap tanh(score / cap) (0 or None:
    no cap).  Forward only: the cache holds no gradients, and one that reaches the result of a q that requires them is an
    error."""
    held = cache._held
    _, _, _, _, held_D, Hk, _, dev, _, _, _ = held
    shape, dtype = q.shape, q.dtype
    if not (len(shape) == 4 and dtype in _DTYPES and q.device == dev):
        _check_values("q", q, 4, dev)
    B, T, Hq, D = shape
    if D != held_D:
        raise ValueError(f"q {tuple(q.shape)} must have the cache's D={held_D} channels")
    if Hq >= 1 << 31:
        _check_sizes(Hq)
    qs = q.stride()
    if D > 1 and qs[3] != 1:
        q = q.contiguous()
        qs = q.stride()
    cr = _cache_rows(dev, table, start, count, B, T)
    mode, words = (_lib.FBEV_DRAFT_CHAIN if drafted else _lib.FBEV_DRAFT_NONE), 0
    if ancestors is not None:
        if not drafted:
            raise ValueError("ancestors come with drafted tokens")
        if ancestors.dtype != torch.int64 or ancestors.device != dev or ancestors.dim() != 3 \
                or ancestors.shape[0] not in (1, B) or ancestors.shape[1] != T or ancestors.shape[2] * 64 < T:
            raise ValueError(f"ancestors must be an int64 tensor of shape [{B} or 1, {T}, words >= {-(-T // 64)}] on {dev}")
        if ancestors.shape[0] != B:
            ancestors = ancestors.expand(B, T, ancestors.shape[2])
        ancestors = ancestors.contiguous()
        mode, words = _lib.FBEV_DRAFT_TREE, ancestors.shape[2]
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    else:
        _check_plain("out", out, q.shape, q.dtype, dev)
        _check_apart("out", out, q, *held[:4], table, start, count, ancestors, workspace)
    if scale is None:
        scale = D ** -0.5 if D else 1.0
    dt = _DTYPES[dtype]
    ad = _pack_attention(Hq, mode, words, *qs[:3], _data(ancestors) or 0, scale, cap or 0.0)
    workspace, have = _scratch(_cache_attention_scratch(B, T, table.shape[1], Hq, Hk, D, dt), workspace, dev)
    _call("fbev_cache_attention", dev, _cache_desc(held), cr, ad, q.data_ptr(), dt, out.data_ptr(), _data(workspace), have)
    return _without_backward("cache_attention", out, q) if q.requires_grad else out
