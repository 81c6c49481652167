"""PyTorch-facing calls of the encoder operators: argument marshalling only.

Group norm with an activation on channels-last maps, rotary positions with several axes, and attention between
queries, BEV cells and tokens.  Each operator has a forward and a backward call and a differentiable function;
``camera_bev_view_amd.ops`` re-exports them beside the view transforms.
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional, Sequence, Tuple

import torch
from torch.autograd.function import once_differentiable

from . import _lib

_DTYPES = {torch.float32: _lib.FBEV_DTYPE_F32, torch.bfloat16: _lib.FBEV_DTYPE_BF16}
_byref = ctypes.byref


_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream      # current_stream().cuda_stream without the Stream object


def _data(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _call(name: str, dev: torch.device, *args) -> None:
    """The library's ``name``(*args, stream) on the current stream of ``dev``, with that device current."""
    fn = getattr(_lib.load(), name)
    if _device() == dev.index:
        status = fn(*args, _raw_stream(dev.index))
    else:
        with torch.cuda.device(dev):
            status = fn(*args, _raw_stream(dev.index))
    if status:
        _lib.check(status)


# Workspace sizes depend on the sizes alone: asked once for each.

@functools.lru_cache(maxsize=1024)
def _norm_scratch(images: int, pixels: int, C: int, groups: int, dtype: int, backward: int) -> int:
    lib, need = _lib.load(), ctypes.c_size_t()
    nd = _lib.NormDesc(images, pixels, 0, 0, C, groups, 0, 0.0)
    _lib.check(lib.fbev_group_norm_workspace(nd, dtype, backward, _byref(need)))
    return need.value


@functools.lru_cache(maxsize=1024)
def _attention_scratch(B: int, Tq: int, Tk: int, Hq: int, Hk: int, D: int, dims: int, backward: int) -> int:
    lib, need = _lib.load(), ctypes.c_size_t()
    z = (0, 0, 0)
    ad = _lib.AttentionDesc(B, Tq, Tk, Hq, Hk, D, z, z, z, 1.0, 0.0, dims, 0, None, None, None, None, None, None)
    _lib.check(lib.fbev_attention_workspace(ad, backward, _byref(need)))
    return need.value


def _check_values(name: str, x: torch.Tensor, ndim: int, device=None, dtype=None) -> None:
    if x.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions, got {tuple(x.shape)}")
    if not x.is_cuda or (device is not None and x.device != device):
        raise ValueError(f"{name} must be a device tensor" + (f" on {device}" if device is not None else ""))
    if x.dtype not in _DTYPES if dtype is None else x.dtype != dtype:
        raise ValueError(f"{name} must be " + (f"{dtype}" if dtype is not None else "float32 or bfloat16")
                         + f", got {x.dtype}")


def _check_plain(name: str, x: torch.Tensor, shape, dtype, device) -> None:
    if tuple(x.shape) != tuple(shape) or x.dtype != dtype or not x.is_contiguous() or x.device != device:
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {list(shape)} on {device}")


def _scratch(need: int, workspace: Optional[torch.Tensor], device) -> Tuple[Optional[torch.Tensor], int]:
    if workspace is not None and (workspace.dtype != torch.uint8 or not workspace.is_contiguous()
                                  or workspace.device != device):
        raise ValueError(f"workspace must be a contiguous uint8 tensor on {device}")
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=device) if need else None
    return workspace, 0 if workspace is None else workspace.numel()


def _check_sizes(*sizes: int) -> None:
    if max(sizes) >= 1 << 31:                         # the descriptors' 32-bit fields would cut them short
        raise ValueError(f"sizes must be below 2^31, got {max(sizes)}")


def _walk(t: torch.Tensor):
    """The tensor's bytes as (count, stride) dimensions, widest stride first, without those that stay in place."""
    es = t.element_size()
    dims = [(n, s * es) for n, s in zip(t.shape, t.stride()) if n > 1 and s > 0]
    return sorted(dims + [(es, 1)], key=lambda d: -d[1])


def _extent(dims) -> int:
    return sum((n - 1) * s for n, s in dims) + 1


def _disjoint(off: int, a, b) -> bool:
    """Whether walk b, begun `off` bytes behind walk a, shares no byte with it.  Exact where one steps over the other's
    inner dimensions (slices of packed tensors); False where that takes more than comparing extents."""
    if off >= _extent(a) or -off >= _extent(b):
        return True
    if not a or not b:
        return False                                  # a single byte within the other's extent
    step = max(a[0][1], b[0][1])
    if step <= 1:
        return False
    inner_a, inner_b = a[a[0][1] == step:], b[b[0][1] == step:]
    if _extent(inner_a) > step or _extent(inner_b) > step:
        return False
    off %= step                                       # of any two blocks that can meet
    return _disjoint(off, inner_a, inner_b) and _disjoint(off - step, inner_a, inner_b)


def _steps_over(dims) -> bool:
    """Whether every dimension steps over those inside it: no byte is walked twice."""
    return all(dims[i][1] >= _extent(dims[i + 1:]) for i in range(len(dims) - 1))


def _overlap(x: torch.Tensor, y: torch.Tensor) -> bool:
    if x.numel() == 0 or y.numel() == 0:
        return False
    return not _disjoint(y.data_ptr() - x.data_ptr(), _walk(x), _walk(y))


def _check_apart(name: str, out: torch.Tensor, *others: Optional[torch.Tensor]) -> None:
    """Refuses an output on memory that another workgroup may still read (or write)."""
    if any(x is not None and _overlap(out, x) for x in others):
        raise ValueError(f"{name} must not overlap another tensor of the call")


# ---- group norm with an activation

def _collapse(shape: Sequence[int], stride: Sequence[int]) -> Optional[int]:
    """The one stride that walks these dimensions as a single one, or None."""
    one, size = None, 1
    for n, s in zip(reversed(shape), reversed(stride)):
        if n == 1:
            continue
        if one is None:
            one = s
        elif s != one * size:
            return None
        size *= n
    return 0 if one is None else one


def _norm_desc(x: torch.Tensor, groups: int, eps: float, activation: str, image_dims: Optional[int]):
    if x.dim() < 2:
        raise ValueError(f"x must be [images..., pixels..., C], got {tuple(x.shape)}")
    if not x.is_cuda:
        raise ValueError("x must be a device tensor")
    if x.dtype not in _DTYPES:
        raise ValueError(f"x must be float32 or bfloat16, got {x.dtype}")
    if activation not in _lib.FBEV_ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(_lib.FBEV_ACTIVATIONS)}, got {activation!r}")
    lead = (2 if x.dim() == 5 else 1) if image_dims is None else image_dims
    if not 0 <= lead < x.dim():
        raise ValueError(f"image_dims={lead} does not fit a tensor of {x.dim()} dimensions")
    shape, stride = x.shape, x.stride()
    _check_sizes(shape[-1], groups)
    si, sp = _collapse(shape[:lead], stride[:lead]), _collapse(shape[lead:-1], stride[lead:-1])
    if si is None or sp is None or (shape[-1] > 1 and stride[-1] != 1):
        x = x.contiguous()
        stride = x.stride()
        si, sp = _collapse(shape[:lead], stride[:lead]), _collapse(shape[lead:-1], stride[lead:-1])
    images = pixels = 1
    for n in shape[:lead]:
        images *= n
    for n in shape[lead:-1]:
        pixels *= n
    return x, _lib.NormDesc(images, pixels, si, sp, shape[-1], groups, _lib.FBEV_ACTIVATIONS[activation], eps)


def _check_affine(C: int, weight, bias, device) -> None:
    for name, p in (("weight", weight), ("bias", bias)):
        if p is not None:
            _check_plain(name, p, (C,), torch.float32, device)


def group_norm_forward(x: torch.Tensor, groups: int, weight: Optional[torch.Tensor] = None,
                       bias: Optional[torch.Tensor] = None, *, eps: float = 1e-5, activation: str = "none",
                       image_dims: Optional[int] = None, out: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """fbev_group_norm_forward on channels-last maps x [images..., pixels..., C] (fp32 or bf16; the first
    ``image_dims`` dimensions count images: two of [B,N,H,W,C], one otherwise).  ``activation``: "none", "relu",
    "silu" or "gelu".  ``weight`` and ``bias`` [C] are contiguous fp32.  Maps whose channels are not contiguous (a permuted
    [B,C,X,Y]) or whose pixels have more than one stride are copied first.  Returns (y like x, contiguous; stats
    [images, groups, 2] fp32: mean and 1 / sqrt(var + eps))."""
    dev = x.device
    x, nd = _norm_desc(x, groups, eps, activation, image_dims)
    _check_affine(nd.C, weight, bias, dev)
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=dev)
    else:
        _check_plain("out", out, x.shape, x.dtype, dev)
        _check_apart("out", out, x, weight, bias, workspace)
    stats = torch.empty((nd.images, max(groups, 0), 2), dtype=torch.float32, device=dev)
    dt = _DTYPES[x.dtype]
    workspace, have = _scratch(_norm_scratch(nd.images, nd.pixels, nd.C, groups, dt, 0), workspace, dev)
    _call("fbev_group_norm_forward", dev, _data(x), dt, nd, _data(weight), _data(bias), _data(out), _data(stats),
          _data(workspace), have)
    return out, stats


def group_norm_backward(grad_y: torch.Tensor, x: torch.Tensor, stats: torch.Tensor, groups: int,
                        weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None, *,
                        activation: str = "none", image_dims: Optional[int] = None, with_params: bool = True,
                        workspace: Optional[torch.Tensor] = None):
    """fbev_group_norm_backward: (grad_x like x, contiguous; grad_weight [C], grad_bias [C] fp32, or None without
    ``with_params``) from dL/dy and the forward's inputs and stats."""
    dev = x.device
    x, nd = _norm_desc(x, groups, 0.0, activation, image_dims)
    _check_affine(nd.C, weight, bias, dev)
    if grad_y.shape != x.shape or grad_y.dtype != x.dtype or grad_y.device != dev:
        raise ValueError(f"grad_y must be a {x.dtype} tensor of shape {list(x.shape)} on {dev}")
    grad_y = grad_y.contiguous()
    _check_plain("stats", stats, (nd.images, groups, 2), torch.float32, dev)
    gx = torch.empty(x.shape, dtype=x.dtype, device=dev)
    gw = gb = None
    if with_params:
        gw = torch.empty(nd.C, dtype=torch.float32, device=dev)
        gb = torch.empty(nd.C, dtype=torch.float32, device=dev)
    dt = _DTYPES[x.dtype]
    workspace, have = _scratch(_norm_scratch(nd.images, nd.pixels, nd.C, groups, dt, 1), workspace, dev)
    _call("fbev_group_norm_backward", dev, _data(grad_y), _data(x), dt, nd, _data(weight), _data(bias), _data(stats),
          _data(gx), _data(gw), _data(gb), _data(workspace), have)
    return gx, gw, gb


class GroupNormAct(torch.autograd.Function):
    """Autograd wrapper of the group norm with an activation."""

    @staticmethod
    def forward(ctx, x, weight, bias, groups, eps, activation, image_dims):
        y, stats = group_norm_forward(x, groups, weight, bias, eps=eps, activation=activation, image_dims=image_dims)
        ctx.save_for_backward(x, weight, bias, stats)
        ctx.meta = (groups, activation, image_dims)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_y):
        x, weight, bias, stats = ctx.saved_tensors
        groups, activation, image_dims = ctx.meta
        want = ctx.needs_input_grad
        gx, gw, gb = group_norm_backward(grad_y, x, stats, groups, weight, bias, activation=activation,
                                         image_dims=image_dims, with_params=want[1] or want[2])
        return gx, gw if want[1] else None, gb if want[2] else None, None, None, None, None


def group_norm_act(x: torch.Tensor, groups: int, weight: Optional[torch.Tensor] = None,
                   bias: Optional[torch.Tensor] = None, *, eps: float = 1e-5, activation: str = "silu",
                   image_dims: Optional[int] = None) -> torch.Tensor:
    """Differentiable act(group_norm(x) * weight + bias) on channels-last maps (see group_norm_forward)."""
    return GroupNormAct.apply(x, weight, bias, groups, eps, activation, image_dims)


# ---- rotary positions

def rotary_freqs(pairs: Sequence[int], base: float = 10000.0, *, device=None) -> torch.Tensor:
    """A frequency table [axes, sum(pairs)]: axis a turns its own pairs[a] pairs of channels, the i-th by
    base^(-i / pairs[a]) radians a unit, and leaves the others alone."""
    table = torch.zeros((len(pairs), sum(pairs)), dtype=torch.float64)
    at = 0
    for a, n in enumerate(pairs):
        if n > 0:
            table[a, at:at + n] = base ** (-torch.arange(n, dtype=torch.float64) / n)
        at += n
    return table.float().to(device)


def _rotary(q, k, pos, freqs, interleaved, inverse, q_out, k_out):
    ref = q if q is not None else k
    if ref is None:
        raise ValueError("q or k must be given")
    dev, dtype = ref.device, ref.dtype
    for name, x in (("q", q), ("k", k)):
        if x is not None:
            _check_values(name, x, 4, dev, dtype)
            if x.shape[3] != ref.shape[3] or x.shape[:2] != ref.shape[:2]:
                raise ValueError(f"q {tuple(q.shape)} and k {tuple(k.shape)} disagree on tokens or channels")
    if dtype not in _DTYPES:
        raise ValueError(f"q and k must be float32 or bfloat16, got {dtype}")
    B, T, _, D = ref.shape
    if pos.dim() != 3 or tuple(pos.shape[:2]) != (B, T):
        raise ValueError(f"pos must be [B={B}, T={T}, axes], got {tuple(pos.shape)}")
    if freqs.dim() != 2 or freqs.shape[0] != pos.shape[2]:
        raise ValueError(f"freqs must be [axes={pos.shape[2]}, pairs], got {tuple(freqs.shape)}")
    for name, x in (("pos", pos), ("freqs", freqs)):
        if x.dtype != torch.float32 or x.device != dev:
            raise ValueError(f"{name} must be a float32 tensor on {dev}")
    _check_sizes(B, T, D, 0 if q is None else q.shape[2], 0 if k is None else k.shape[2], *freqs.shape)
    pos, freqs = pos.contiguous(), freqs.contiguous()
    outs = []
    ins = []
    for name, x, out in (("q", q, q_out), ("k", k, k_out)):
        if x is None:
            ins.append(None)
            outs.append(None)
            continue
        if x.shape[3] > 1 and x.stride(3) != 1:
            if out is x:
                raise ValueError(f"{name} is rotated in place: its channels must be contiguous")
            x = x.contiguous()
        if out is None:
            out = torch.empty(x.shape, dtype=dtype, device=dev)
        elif out.shape != x.shape or out.dtype != dtype or out.device != dev or \
                (x.shape[3] > 1 and out.stride(3) != 1):
            raise ValueError(f"{name}_out must be a {dtype} tensor of shape {list(x.shape)} on {dev}, "
                             "channels contiguous")
        elif out.numel() and any(s == 0 and n > 1 for n, s in zip(out.shape, out.stride())):
            raise ValueError(f"{name}_out must not be a broadcast tensor")
        elif not _steps_over(_walk(out)):
            raise ValueError(f"{name}_out must not overlap itself")
        elif out.data_ptr() != x.data_ptr() or out.stride() != x.stride():
            _check_apart(f"{name}_out, unless it is {name} itself,", out, x)
        ins.append(x)
        outs.append(out)
    for given, name, out, other in ((q_out, "q_out", outs[0], 1), (k_out, "k_out", outs[1], 0)):
        if given is not None and out is not None:
            _check_apart(name, out, ins[other], outs[other], pos, freqs)
    none = (0, 0, 0, 0)
    strides = [none if x is None else x.stride() for x in ins + outs]
    rd = _lib.RotaryDesc(B, T, D, pos.shape[2], freqs.shape[1], 0 if q is None else q.shape[2],
                         0 if k is None else k.shape[2], bool(interleaved), bool(inverse), strides[0][:3],
                         strides[1][:3], strides[2][:3], strides[3][:3])
    _call("fbev_rotary", dev, _data(ins[0]), _data(ins[1]), _DTYPES[dtype], rd, _data(pos), _data(freqs),
          _data(outs[0]), _data(outs[1]))
    return outs[0], outs[1]


def rotary_forward(q: Optional[torch.Tensor], k: Optional[torch.Tensor], pos: torch.Tensor, freqs: torch.Tensor, *,
                   interleaved: bool = False, q_out: Optional[torch.Tensor] = None,
                   k_out: Optional[torch.Tensor] = None):
    """fbev_rotary: queries [B,T,Hq,D] and keys [B,T,Hk,D] (fp32 or bf16, either may be None) turned by
    theta = pos [B,T,axes] . freqs [axes,pairs] (fp32; angles in double).  Pair i is channels (i, i + pairs), or
    (2i, 2i + 1) when ``interleaved``.  ``q_out`` / ``k_out`` may be q / k themselves (slices of a packed tensor among
    them), but share no memory with anything else of the call.  Returns (q', k')."""
    return _rotary(q, k, pos, freqs, interleaved, False, q_out, k_out)


def rotary_backward(grad_q: Optional[torch.Tensor], grad_k: Optional[torch.Tensor], pos: torch.Tensor,
                    freqs: torch.Tensor, *, interleaved: bool = False, q_out: Optional[torch.Tensor] = None,
                    k_out: Optional[torch.Tensor] = None):
    """The gradients with respect to rotary_forward's q and k: fbev_rotary by the opposite angles."""
    return _rotary(grad_q, grad_k, pos, freqs, interleaved, True, q_out, k_out)


class RotaryAxes(torch.autograd.Function):
    """Autograd wrapper of the rotary positions; positions and frequencies are constants."""

    @staticmethod
    def forward(ctx, q, k, pos, freqs, interleaved):
        ctx.save_for_backward(pos, freqs)
        ctx.interleaved = interleaved
        return rotary_forward(q, k, pos, freqs, interleaved=interleaved)

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_q, grad_k):
        pos, freqs = ctx.saved_tensors
        want = ctx.needs_input_grad
        gq, gk = grad_q if want[0] else None, grad_k if want[1] else None
        if gq is not None or gk is not None:
            gq, gk = rotary_backward(gq, gk, pos, freqs, interleaved=ctx.interleaved)
        return gq, gk, None, None, None


def rotary_axes(q: Optional[torch.Tensor], k: Optional[torch.Tensor], pos: torch.Tensor, freqs: torch.Tensor, *,
                interleaved: bool = False):
    """Differentiable rotary_forward."""
    return RotaryAxes.apply(q, k, pos, freqs, interleaved)


# ---- attention

def _attention_desc(q, k, v, scale, cap, pos_q, pos_k, slope, doc_q, doc_k, causal, prefix):
    """Checks the arguments; returns (q, k, v, descriptor, tensors the descriptor points into)."""
    _check_values("q", q, 4)
    dev, dtype = q.device, q.dtype
    _check_values("k", k, 4, dev, dtype)
    _check_values("v", v, 4, dev, dtype)
    B, Tq, Hq, D = q.shape
    Tk, Hk = k.shape[1], k.shape[2]
    if k.shape[0] != B or k.shape[3] != D or v.shape != k.shape:
        raise ValueError(f"k {tuple(k.shape)} and v {tuple(v.shape)} must be [B={B}, Tk, Hk, D={D}]")
    _check_sizes(B, Tq, Tk, Hq, Hk, D)
    if D > 1:
        q = q if q.stride(3) == 1 else q.contiguous()
        k = k if k.stride(3) == 1 else k.contiguous()
        v = v if v.stride(3) == 1 else v.contiguous()
    dims = 0
    keep = []
    bias = (pos_q, pos_k, slope)
    if any(x is not None for x in bias):
        if any(x is None for x in bias):
            raise ValueError("pos_q, pos_k and slope come together")
        dims = pos_q.shape[-1]
        if slope.dim() == 1:
            slope = slope.expand(B, Tq, slope.shape[0])
        for name, x, shape in (("pos_q", pos_q, (B, Tq, dims)), ("pos_k", pos_k, (B, Tk, dims)),
                               ("slope", slope, (B, Tq, Hq))):
            if tuple(x.shape) != shape or x.dtype != torch.float32 or x.device != dev:
                raise ValueError(f"{name} must be a float32 tensor of shape {list(shape)} on {dev}")
        if not 1 <= dims <= 3:
            raise ValueError(f"positions have {dims} axes, 1 to 3 are supported")
        pos_q, pos_k, slope = pos_q.contiguous(), pos_k.contiguous(), slope.contiguous()
        keep += [pos_q, pos_k, slope]
    if (doc_q is None) != (doc_k is None):
        raise ValueError("doc_q and doc_k come together")
    if doc_q is not None:
        for name, x, shape in (("doc_q", doc_q, (B, Tq)), ("doc_k", doc_k, (B, Tk))):
            if tuple(x.shape) != shape or x.dtype != torch.int32 or x.device != dev:
                raise ValueError(f"{name} must be an int32 tensor of shape {list(shape)} on {dev}")
        doc_q, doc_k = doc_q.contiguous(), doc_k.contiguous()
        keep += [doc_q, doc_k]
    if prefix is not None:
        if not causal:
            raise ValueError("prefix needs causal=True")
        if tuple(prefix.shape) != (B,) or prefix.dtype != torch.int32 or prefix.device != dev:
            raise ValueError(f"prefix must be an int32 tensor of shape [{B}] on {dev}")
        prefix = prefix.contiguous()
        keep.append(prefix)
    if scale is None:
        scale = D ** -0.5 if D else 1.0
    ad = _lib.AttentionDesc(B, Tq, Tk, Hq, Hk, D, q.stride()[:3], k.stride()[:3], v.stride()[:3], scale, cap or 0.0,
                            dims, bool(causal), _data(pos_q), _data(pos_k), _data(slope), _data(doc_q), _data(doc_k),
                            _data(prefix))
    return q, k, v, ad, keep


def attention_forward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, *, scale: Optional[float] = None,
                      cap: Optional[float] = None, pos_q: Optional[torch.Tensor] = None,
                      pos_k: Optional[torch.Tensor] = None, slope: Optional[torch.Tensor] = None,
                      doc_q: Optional[torch.Tensor] = None, doc_k: Optional[torch.Tensor] = None,
                      causal: bool = False, prefix: Optional[torch.Tensor] = None,
                      out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None
                      ) -> Tuple[torch.Tensor, torch.Tensor]:
    """fbev_attention_forward on q [B,Tq,Hq,D], k and v [B,Tk,Hk,D] (fp32 or bf16; Hq a multiple of Hk).

    ``scale``: 1 / sqrt(D) unless given.  ``cap``: scores become cap tanh(score / cap) (0 or None: no cap).
    ``pos_q`` [B,Tq,n], ``pos_k`` [B,Tk,n] (n = 1 .. 3) with ``slope`` [B,Tq,Hq] or [Hq], all fp32: scores lose
    slope times the Euclidean distance of the two positions.  ``doc_q`` [B,Tq], ``doc_k`` [B,Tk] int32: only keys of
    the query's own document are seen, negative ones (padding) by none.  ``causal``: key j is seen by query i when
    j <= i + Tk - Tq, or j < ``prefix`` [B] (int32).  Queries that see no key get zeros.
    Returns (out [B,Tq,Hq,D], stats [B,Hq,Tq,2] fp32): the softmax's m and l, sum_j exp(s_j) = 2^m l, which the
    backward takes (m = -inf, l = 0 where no key is seen)."""
    q, k, v, ad, keep = _attention_desc(q, k, v, scale, cap, pos_q, pos_k, slope, doc_q, doc_k, causal, prefix)
    dev = q.device
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=dev)
    else:
        _check_plain("out", out, q.shape, q.dtype, dev)
        _check_apart("out", out, q, k, v, *keep, workspace)
    stats = torch.empty((ad.B, ad.Hq, ad.Tq, 2), dtype=torch.float32, device=dev)
    workspace, have = _scratch(_attention_scratch(ad.B, ad.Tq, ad.Tk, ad.Hq, ad.Hk, ad.D, ad.dims, 0), workspace, dev)
    _call("fbev_attention_forward", dev, _data(q), _data(k), _data(v), _DTYPES[q.dtype], ad, _data(out), _data(stats),
          _data(workspace), have)
    del keep
    return out, stats


def attention_backward(grad_out: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor,
                       stats: torch.Tensor, *, scale: Optional[float] = None, cap: Optional[float] = None,
                       pos_q: Optional[torch.Tensor] = None, pos_k: Optional[torch.Tensor] = None,
                       slope: Optional[torch.Tensor] = None, doc_q: Optional[torch.Tensor] = None,
                       doc_k: Optional[torch.Tensor] = None, causal: bool = False,
                       prefix: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """fbev_attention_backward: (grad_q, grad_k, grad_v, grad_slope [B,Tq,Hq] fp32 or None without positions) from
    dL/dout and the forward's inputs, out and stats."""
    q, k, v, ad, keep = _attention_desc(q, k, v, scale, cap, pos_q, pos_k, slope, doc_q, doc_k, causal, prefix)
    dev, dtype = q.device, q.dtype
    if grad_out.shape != q.shape or grad_out.dtype != dtype or grad_out.device != dev:
        raise ValueError(f"grad_out must be a {dtype} tensor of shape {list(q.shape)} on {dev}")
    grad_out = grad_out.contiguous()
    _check_plain("out", out, q.shape, dtype, dev)
    _check_plain("stats", stats, (ad.B, ad.Hq, ad.Tq, 2), torch.float32, dev)
    gq = torch.empty(q.shape, dtype=dtype, device=dev)
    gk = torch.empty(k.shape, dtype=dtype, device=dev)
    gv = torch.empty(v.shape, dtype=dtype, device=dev)
    gslope = torch.empty((ad.B, ad.Tq, ad.Hq), dtype=torch.float32, device=dev) if ad.dims else None
    workspace, have = _scratch(_attention_scratch(ad.B, ad.Tq, ad.Tk, ad.Hq, ad.Hk, ad.D, ad.dims, 1), workspace, dev)
    _call("fbev_attention_backward", dev, _data(grad_out), _data(q), _data(k), _data(v), _DTYPES[dtype], ad,
          _data(out), _data(stats), _data(gq), _data(gk), _data(gv), _data(gslope), _data(workspace), have)
    del keep
    return gq, gk, gv, gslope


class QueryAttention(torch.autograd.Function):
    """Autograd wrapper of the attention: gradients for q, k, v and the slopes; positions and masks are constants."""

    @staticmethod
    def forward(ctx, q, k, v, slope, scale, cap, pos_q, pos_k, doc_q, doc_k, causal, prefix):
        out, stats = attention_forward(q, k, v, scale=scale, cap=cap, pos_q=pos_q, pos_k=pos_k, slope=slope,
                                       doc_q=doc_q, doc_k=doc_k, causal=causal, prefix=prefix)
        ctx.save_for_backward(q, k, v, slope, pos_q, pos_k, doc_q, doc_k, prefix, out, stats)
        ctx.meta = (scale, cap, causal)
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_out):
        q, k, v, slope, pos_q, pos_k, doc_q, doc_k, prefix, out, stats = ctx.saved_tensors
        scale, cap, causal = ctx.meta
        gq, gk, gv, gs = attention_backward(grad_out, q, k, v, out, stats, scale=scale, cap=cap, pos_q=pos_q,
                                            pos_k=pos_k, slope=slope, doc_q=doc_q, doc_k=doc_k, causal=causal,
                                            prefix=prefix)
        return (gq, gk, gv, gs) + (None,) * 8


def query_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, *, scale: Optional[float] = None,
                    cap: Optional[float] = None, pos_q: Optional[torch.Tensor] = None,
                    pos_k: Optional[torch.Tensor] = None, slope: Optional[torch.Tensor] = None,
                    doc_q: Optional[torch.Tensor] = None, doc_k: Optional[torch.Tensor] = None, causal: bool = False,
                    prefix: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Differentiable attention_forward: gradients for q, k, v and slope (a [Hq] slope gets its sum)."""
    if slope is not None and slope.dim() == 1:
        slope = slope.expand(q.shape[0], q.shape[1], slope.shape[0])
    return QueryAttention.apply(q, k, v, slope, scale, cap, pos_q, pos_k, doc_q, doc_k, causal, prefix)
