"""CPU: the decoder operators refuse bad arguments on the host, before anything reaches a device."""
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


def rms(lib, x=FAKE, res=None, dtype=0, outer=6, inner=1, C=40, eps=1e-6, xs=(40, 0), rs=(40, 0), y=FAKE, h=None,
        rstd=FAKE):
    return lib.fbev_rms_norm_forward(x, res, dtype, _lib.RmsDesc(outer, inner, xs, rs, C, eps), None, y, h, rstd, None)


def rms_codes(lib, codes=1, block=32, out=FAKE, scales=FAKE, C=256):
    return lib.fbev_rms_norm_codes(FAKE, None, 1, _lib.RmsDesc(6, 1, (C, 0), (0, 0), C, 1e-6), None, codes, block, out,
                                   scales, None, None)


def rms_bwd(lib, gy=FAKE, h=FAKE, rstd=FAKE, gx=FAKE, gw=FAKE, ws=FAKE, have=1 << 30, dtype=0):
    return lib.fbev_rms_norm_backward(gy, None, h, dtype, _lib.RmsDesc(6, 1, (40, 0), (0, 0), 40, 0.0), None, rstd, gx,
                                      gw, ws, have, None)


def cache(pages=4, Hk=2, D=40, codes=0, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE):
    return _lib.CacheDesc(pages, Hk, D, codes, k, v, ks, vs)


def rows(B=3, T=5, W=2, table=FAKE, start=FAKE, count=None):
    return _lib.CacheRows(B, T, W, table, start, count)


def split(kw):
    mine = {n: kw.pop(n) for n in list(kw) if n in ("pages", "Hk", "D", "codes", "kc", "vc", "ks", "vs")}
    for name, to in (("kc", "k"), ("vc", "v")):
        if name in mine:
            mine[to] = mine.pop(name)
    return cache(**mine), rows(**{n: kw.pop(n) for n in list(kw) if n in ("B", "T", "W", "table", "start", "count")}), kw


def write(lib, **kw):
    cd, cr, kw = split(kw)
    s = (ctypes.c_int64 * 3)(*kw.get("stride", (400, 80, 40)))
    return lib.fbev_cache_write(cd, cr, kw.get("k", FAKE), kw.get("v", FAKE), kw.get("dtype", 0), s,
                                None if kw.get("no_stride") else s, None)


def read(lib, **kw):
    cd, cr, kw = split(kw)
    return lib.fbev_cache_read(cd, cr, kw.get("dtype", 0), FAKE, FAKE, None)


def attn(lib, **kw):
    cd, cr, kw = split(kw)
    ad = _lib.CacheAttentionDesc(kw.get("Hq", 4), kw.get("drafts", 1), kw.get("words", 0),
                                 kw.get("stride", (800, 160, 40)), kw.get("ancestors"), kw.get("scale", 0.1),
                                 kw.get("cap", 0.0))
    return lib.fbev_cache_attention(cd, cr, ad, kw.get("q", FAKE), kw.get("dtype", 0), kw.get("out", FAKE),
                                    kw.get("ws", FAKE), kw.get("have", 1 << 40), None)


@pytest.mark.parametrize("call,kw,status,text", [
    (rms, dict(dtype=5), UNSUPPORTED, "dtype"),
    (rms, dict(outer=-1), INVALID, "outer"),
    (rms, dict(C=0), INVALID, "C=0"),
    (rms, dict(C=16385), UNSUPPORTED, "FBEV_MAX_RMS_CHANNELS"),
    (rms, dict(eps=float("nan")), INVALID, "eps"),
    (rms, dict(eps=-1e-6), INVALID, "eps"),
    (rms, dict(xs=(-1, 0)), INVALID, "stride"),
    (rms, dict(outer=1 << 20, inner=1 << 12), UNSUPPORTED, "rows"),
    (rms, dict(x=None), INVALID, "non-NULL"),
    (rms, dict(y=None), INVALID, "non-NULL"),
    (rms, dict(res=FAKE), INVALID, "together"),
    (rms, dict(h=FAKE), INVALID, "together"),
    (rms_codes, dict(codes=2), INVALID, "codes"),
    (rms_codes, dict(block=16), INVALID, "block"),
    (rms_codes, dict(block=-1), INVALID, "block"),
    (rms_codes, dict(block=96), INVALID, "block"),
    (rms_codes, dict(scales=None), INVALID, "scales"),
    (rms_codes, dict(out=None), INVALID, "non-NULL"),
    (rms_bwd, dict(gy=None), INVALID, "non-NULL"),
    (rms_bwd, dict(rstd=None), INVALID, "non-NULL"),
    (rms_bwd, dict(gx=None), INVALID, "non-NULL"),
    (rms_bwd, dict(ws=None), INVALID, "workspace"),
    (rms_bwd, dict(have=8), INVALID, "workspace"),
    (rms_bwd, dict(ws=FAKE + 4), INVALID, "16-byte"),
    (rms_bwd, dict(dtype=-1), UNSUPPORTED, "dtype"),
    (write, dict(pages=-1), INVALID, "bad size"),
    (write, dict(Hk=0), INVALID, "bad size"),
    (write, dict(T=-1), INVALID, "bad size"),
    (write, dict(D=129), UNSUPPORTED, "FBEV_MAX_HEAD_DIM"),
    (write, dict(codes=7), INVALID, "codes"),
    (write, dict(W=(1 << 24) + 1), UNSUPPORTED, "pages a sequence"),
    (write, dict(kc=None), INVALID, "non-NULL"),
    (write, dict(vc=FAKE + 8), INVALID, "aligned"),
    (write, dict(ks=FAKE + 4), INVALID, "aligned"),
    (write, dict(table=None), INVALID, "table"),
    (write, dict(start=None), INVALID, "start"),
    (write, dict(stride=(1, -1, 1)), INVALID, "stride"),
    (write, dict(no_stride=True), INVALID, "stride"),
    (write, dict(k=None), INVALID, "k and v"),
    (write, dict(dtype=9), UNSUPPORTED, "dtype"),
    (write, dict(B=1 << 20, T=1 << 20), UNSUPPORTED, "2^31"),
    (read, dict(dtype=2), UNSUPPORTED, "dtype"),
    (read, dict(vs=None), INVALID, "non-NULL"),
    (read, dict(B=-2), INVALID, "bad size"),
    (attn, dict(Hq=3), INVALID, "multiple"),
    (attn, dict(Hq=0), INVALID, "multiple"),
    (attn, dict(drafts=3), INVALID, "drafts"),
    (attn, dict(drafts=2, T=65, words=1, ancestors=FAKE), INVALID, "words"),
    (attn, dict(drafts=2, words=1), INVALID, "ancestors"),
    (attn, dict(drafts=2, words=1, ancestors=FAKE + 4), INVALID, "8-byte"),
    (attn, dict(scale=float("inf")), INVALID, "scale"),
    (attn, dict(scale=1e-20), UNSUPPORTED, "scale"),
    (attn, dict(cap=-1.0), INVALID, "cap"),
    (attn, dict(cap=1e20), UNSUPPORTED, "cap"),
    (attn, dict(stride=(-1, 1, 1)), INVALID, "stride"),
    (attn, dict(q=None), INVALID, "q and out"),
    (attn, dict(out=None), INVALID, "q and out"),
    (attn, dict(dtype=2), UNSUPPORTED, "dtype"),
    (attn, dict(T=1 << 29), UNSUPPORTED, "rows"),
    (attn, dict(B=1 << 20, T=1 << 10), UNSUPPORTED, "tiles"),
    (attn, dict(B=1 << 22, T=1), UNSUPPORTED, "tiles"),
    (attn, dict(B=1 << 16, T=1 << 10, Hq=2, Hk=2, D=40), UNSUPPORTED, "tiles"),
    (attn, dict(W=1000, ws=None), INVALID, "workspace"),
    (attn, dict(W=1000, have=16), INVALID, "workspace"),
    (attn, dict(W=1000, ws=FAKE + 8), INVALID, "16-byte"),
])
def test_refusals(lib, call, kw, status, text):
    assert call(lib, **dict(kw)) == status
    assert text in lib.fbev_last_error().decode()


def test_null_descriptors_and_empty_calls(lib):
    n = ctypes.c_size_t()
    assert lib.fbev_rms_norm_forward(FAKE, None, 0, None, None, FAKE, None, None, None) == INVALID
    assert lib.fbev_rms_norm_workspace(None, 0, ctypes.byref(n)) == INVALID
    assert lib.fbev_cache_read(None, rows(), 0, FAKE, FAKE, None) == INVALID
    assert lib.fbev_cache_read(cache(), None, 0, FAKE, FAKE, None) == INVALID
    assert lib.fbev_cache_attention(cache(), rows(), None, FAKE, 0, FAKE, FAKE, 0, None) == INVALID
    ad = _lib.CacheAttentionDesc(4, 0, 0, (1, 1, 1), None, 0.1, 0.0)
    assert lib.fbev_cache_attention_workspace(cache(), rows(), ad, 0, None) == INVALID
    # nothing to do needs no buffers
    assert rms(lib, outer=0, x=None, y=None, rstd=None) == 0
    assert lib.fbev_rms_norm_backward(None, None, None, 0, _lib.RmsDesc(0, 1, (0, 0), (0, 0), 40, 0.0), None, None, None,
                                      None, None, 0, None) == 0
    empty = dict(pages=0, kc=None, vc=None, ks=None, vs=None)
    assert write(lib, **empty) == 0 and write(lib, B=0, table=None, start=None, k=None, v=None) == 0
    assert write(lib, T=0, table=None, start=None) == 0 and write(lib, W=0, table=None) == 0
    assert read(lib, T=0) == 0 and attn(lib, B=0, q=None, out=None, ws=None, have=0) == 0
    assert lib.fbev_cache_read(cache(), rows(), 0, None, None, None) == 0
    # the most workgroups of one launch
    assert lib.fbev_cache_attention_workspace(cache(), rows(B=(1 << 22) - 1, T=1), ad, 0, ctypes.byref(n)) == 0
    # few rows over many tokens need a workspace, many rows none
    assert lib.fbev_cache_attention_workspace(cache(), rows(T=1, W=1000), ad, 0, ctypes.byref(n)) == 0 and n.value > 0
    assert lib.fbev_cache_attention_workspace(cache(), rows(B=300, T=640, W=9), ad, 0, ctypes.byref(n)) == 0
    assert n.value == 0


def test_binding_refuses_host_tensors_and_mismatched_arguments():
    x = torch.zeros((2, 5, 8))
    with pytest.raises(ValueError, match="device tensor"):
        ops.rms_norm_forward(x)
    with pytest.raises(ValueError, match="device tensor"):
        ops.rms_norm_codes(x)
    with pytest.raises(ValueError, match="codes"):
        ops.rms_norm_codes(x, codes=torch.uint8)
    with pytest.raises(ValueError, match="device tensor"):
        ops.token_cache(2, 1, 16, device="cpu")
    with pytest.raises(ValueError, match="codes"):
        ops.token_cache(2, 1, 16, codes=torch.float8_e5m2, device="cpu")


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"),
                    reason="needs g++ and the ROCm headers")
def test_host_layer_under_asan_and_ubsan(tmp_path):
    san = os.path.join(ROOT, "tests", "sanitize")
    exe = str(tmp_path / "fbev_decoder_sanitize")
    src = os.path.join(ROOT, "camera_bev_view_amd", "csrc")
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
           "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-fno-omit-frame-pointer",
           os.path.join(src, "decoder_api.cpp"), os.path.join(src, "flashbev_api.cpp"),
           os.path.join(san, "launch_stubs.cpp"), os.path.join(san, "decoder_harness.cpp"), "-o", exe, "-lpthread"]
    build = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert build.returncode == 0, build.stderr[-4000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:halt_on_error=1:verify_asan_link_order=0",
               UBSAN_OPTIONS="print_stacktrace=1")
    res = subprocess.run([exe], capture_output=True, text=True, timeout=120, env=env)
    assert res.returncode == 0 and res.stdout.strip().endswith("ok"), res.stdout[-4000:] + res.stderr[-4000:]
