"""CPU: the encoder operators refuse bad arguments on the host, before anything reaches a device."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

from camera_bev_view_amd import _lib, ops

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000          # never dereferenced: every call below fails validation first
INVALID, UNSUPPORTED = _lib.FBEV_ERR_INVALID_ARGUMENT, _lib.FBEV_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def norm(lib, x=FAKE, dtype=0, images=2, pixels=50, C=32, groups=4, act=2, eps=1e-5, si=1600, sp=32, y=FAKE, stats=FAKE,
         ws=FAKE, have=1 << 30):
    nd = _lib.NormDesc(images, pixels, si, sp, C, groups, act, eps)
    return lib.fbev_group_norm_forward(x, dtype, nd, None, None, y, stats, ws, have, None)


def norm_bwd(lib, gy=FAKE, x=FAKE, images=2, pixels=50, C=32, groups=4, stats=FAKE, gx=FAKE, gw=FAKE, ws=FAKE,
             have=1 << 30):
    nd = _lib.NormDesc(images, pixels, pixels * C, C, C, groups, 0, 0.0)
    return lib.fbev_group_norm_backward(gy, x, 0, nd, None, None, stats, gx, gw, None, ws, have, None)


def rotary(lib, q=FAKE, k=FAKE, dtype=0, B=1, T=5, D=32, axes=3, pairs=16, hq=2, hk=1, pos=FAKE, freqs=FAKE, qo=FAKE,
           ko=FAKE, stride=(320, 64, 32)):
    rd = _lib.RotaryDesc(B, T, D, axes, pairs, hq, hk, 0, 0, stride, stride, stride, stride)
    return lib.fbev_rotary(q, k, dtype, rd, pos, freqs, qo, ko, None)


def attn_desc(B=1, Tq=4, Tk=6, Hq=4, Hk=2, D=32, stride=(1024, 128, 32), scale=0.1, cap=0.0, dims=0, causal=0,
              pos_q=FAKE, pos_k=FAKE, slope=FAKE, doc_q=None, doc_k=None, prefix=None):
    return _lib.AttentionDesc(B, Tq, Tk, Hq, Hk, D, stride, stride, stride, scale, cap, dims, causal, pos_q, pos_k,
                              slope, doc_q, doc_k, prefix)


def attn(lib, q=FAKE, k=FAKE, v=FAKE, dtype=0, out=FAKE, stats=FAKE, ws=FAKE, have=1 << 30, **kw):
    return lib.fbev_attention_forward(q, k, v, dtype, attn_desc(**kw), out, stats, ws, have, None)


def attn_bwd(lib, go=FAKE, q=FAKE, k=FAKE, v=FAKE, dtype=0, out=FAKE, stats=FAKE, gq=FAKE, gk=FAKE, gv=FAKE, gs=None,
             ws=FAKE, have=1 << 30, **kw):
    return lib.fbev_attention_backward(go, q, k, v, dtype, attn_desc(**kw), out, stats, gq, gk, gv, gs, ws, have, None)


@pytest.mark.parametrize("call,kw,status,text", [
    (norm, dict(dtype=7), UNSUPPORTED, "dtype"),
    (norm, dict(images=-1), INVALID, "images"),
    (norm, dict(groups=5), INVALID, "multiple of groups"),
    (norm, dict(groups=0), INVALID, "groups"),
    (norm, dict(act=9), INVALID, "activation"),
    (norm, dict(eps=float("nan")), INVALID, "eps"),
    (norm, dict(eps=-1.0), INVALID, "eps"),
    (norm, dict(sp=-1), INVALID, "stride"),
    (norm, dict(x=None), INVALID, "non-NULL"),
    (norm, dict(stats=None), INVALID, "non-NULL"),
    (norm, dict(pixels=1 << 20, ws=None), INVALID, "workspace"),
    (norm, dict(pixels=1 << 20, have=8), INVALID, "workspace"),
    (norm, dict(pixels=1 << 20, ws=FAKE + 8), INVALID, "16-byte"),
    (norm, dict(C=8192, groups=1), UNSUPPORTED, "pieces"),
    (norm, dict(pixels=1 << 32), UNSUPPORTED, "2^40"),
    (norm_bwd, dict(gy=None), INVALID, "non-NULL"),
    (norm_bwd, dict(gx=None), INVALID, "non-NULL"),
    (norm_bwd, dict(ws=None), INVALID, "workspace"),
    (rotary, dict(dtype=2), UNSUPPORTED, "dtype"),
    (rotary, dict(T=-1), INVALID, "negative size"),
    (rotary, dict(axes=0), INVALID, "axes"),
    (rotary, dict(axes=9), INVALID, "axes"),
    (rotary, dict(pairs=17), INVALID, "pairs"),
    (rotary, dict(pairs=0), INVALID, "pairs"),
    (rotary, dict(D=8192, pairs=4096), UNSUPPORTED, "pairs"),
    (rotary, dict(q=None), INVALID, "NULL"),
    (rotary, dict(ko=None), INVALID, "NULL"),
    (rotary, dict(pos=None), INVALID, "pos"),
    (rotary, dict(stride=(-1, 1, 1)), INVALID, "stride"),
    (attn, dict(dtype=3), UNSUPPORTED, "dtype"),
    (attn, dict(Hq=3), INVALID, "multiple"),
    (attn, dict(Hk=0), INVALID, "bad size"),
    (attn, dict(D=129), UNSUPPORTED, "FBEV_MAX_HEAD_DIM"),
    (attn, dict(Tq=-1), INVALID, "bad size"),
    (attn, dict(scale=float("inf")), INVALID, "scale"),
    (attn, dict(cap=-1.0), INVALID, "cap"),
    (attn, dict(scale=1e-20), UNSUPPORTED, "scale"),
    (attn, dict(scale=-1e20), UNSUPPORTED, "scale"),
    (attn, dict(cap=1e-30), UNSUPPORTED, "cap"),
    (attn, dict(dims=4), INVALID, "dims"),
    (attn, dict(dims=2, slope=None), INVALID, "slope"),
    (attn, dict(doc_q=FAKE), INVALID, "together"),
    (attn, dict(prefix=FAKE), INVALID, "causal"),
    (attn, dict(stride=(1, -1, 1)), INVALID, "stride"),
    (attn, dict(q=None), INVALID, "q is NULL"),
    (attn, dict(v=None), INVALID, "k and v"),
    (attn, dict(out=None), INVALID, "out"),
    (attn, dict(Tk=1 << 20, ws=None), INVALID, "workspace"),
    (attn, dict(Tk=1 << 30), UNSUPPORTED, "keys"),
    (attn, dict(B=1 << 20, Tq=1 << 20), UNSUPPORTED, "tiles"),
    (attn_bwd, dict(go=None), INVALID, "non-NULL"),
    (attn_bwd, dict(gk=None), INVALID, "non-NULL"),
    (attn_bwd, dict(gs=FAKE), INVALID, "grad_slope"),
    (attn_bwd, dict(have=4), INVALID, "workspace"),
    (attn_bwd, dict(stats=FAKE + 4), INVALID, "8-byte"),
])
def test_refusals(lib, call, kw, status, text):
    assert call(lib, **kw) == status
    assert text in lib.fbev_last_error().decode()


def test_null_descriptors_and_sizes(lib):
    n = ctypes.c_size_t()
    assert lib.fbev_group_norm_workspace(None, 0, 0, ctypes.byref(n)) == INVALID
    assert lib.fbev_attention_workspace(None, 0, ctypes.byref(n)) == INVALID
    assert lib.fbev_attention_workspace(attn_desc(), 0, None) == INVALID
    assert lib.fbev_rotary(FAKE, FAKE, 0, None, FAKE, FAKE, FAKE, FAKE, None) == INVALID
    # nothing to do needs no buffers
    assert norm(lib, images=0, x=None, y=None, stats=None, ws=None, have=0) == 0
    assert rotary(lib, T=0, q=None, k=None, pos=None, freqs=None, qo=None, ko=None) == 0
    assert attn(lib, B=0, q=None, k=None, v=None, out=None, stats=None, ws=None, have=0) == 0
    assert attn(lib, Tq=0, q=None, out=None, stats=None, ws=None, have=0) == 0
    # few rows over many keys need a workspace, many rows none
    assert lib.fbev_attention_workspace(attn_desc(Tq=1, Tk=40000), 0, ctypes.byref(n)) == 0 and n.value > 0
    assert lib.fbev_attention_workspace(attn_desc(B=64, Tq=4000, Tk=4000), 0, ctypes.byref(n)) == 0 and n.value == 0


def test_binding_refuses_host_tensors_and_mismatched_arguments():
    x = torch.zeros((2, 5, 8))
    with pytest.raises(ValueError, match="device tensor"):
        ops.group_norm_forward(x, 2)
    with pytest.raises(ValueError, match="device tensor"):
        ops.attention_forward(torch.zeros((1, 2, 1, 8)), torch.zeros((1, 2, 1, 8)), torch.zeros((1, 2, 1, 8)))
    with pytest.raises(ValueError, match="device tensor"):
        ops.rotary_forward(torch.zeros((1, 2, 1, 8)), None, torch.zeros((1, 2, 1)), torch.zeros((1, 4)))
    with pytest.raises(ValueError, match="must be given"):
        ops.rotary_forward(None, None, torch.zeros((1, 2, 1)), torch.zeros((1, 4)))


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"),
                    reason="needs g++ and the ROCm headers")
def test_host_layer_under_asan_and_ubsan(tmp_path):
    san = os.path.join(ROOT, "tests", "sanitize")
    exe = str(tmp_path / "fbev_encoder_sanitize")
    src = os.path.join(ROOT, "camera_bev_view_amd", "csrc")
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
           "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-fno-omit-frame-pointer",
           os.path.join(src, "encoder_api.cpp"), os.path.join(src, "flashbev_api.cpp"),
           os.path.join(san, "launch_stubs.cpp"), os.path.join(san, "encoder_harness.cpp"), "-o", exe, "-lpthread"]
    build = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert build.returncode == 0, build.stderr[-4000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:halt_on_error=1:verify_asan_link_order=0",
               UBSAN_OPTIONS="print_stacktrace=1")
    res = subprocess.run([exe], capture_output=True, text=True, timeout=120, env=env)
    assert res.returncode == 0 and res.stdout.strip().endswith("ok"), res.stdout[-4000:] + res.stderr[-4000:]
