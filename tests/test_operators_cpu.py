"""Refusals of the norm, clipping and few-token entry points (CPU only: the
checks run before any device work, so pointers are never dereferenced)."""
import ctypes
import os

import pytest
import torch

import dropless_top_moe_b200 as moe
from dropless_top_moe_b200._lib import (MOE_BF16, MOE_ERR_INVALID_ARG as INV, MOE_ERR_UNSUPPORTED as UNS,
                                        MOE_ERR_WORKSPACE as WS, MOE_F32, load)

bf, f32 = torch.bfloat16, torch.float32
BIG = 1 << 40
A, B, C, D, E_ = (0x100000000 * (i + 1) for i in range(5))   # aligned, far apart, never dereferenced


@pytest.fixture(scope="module")
def lib():
    from dropless_top_moe_b200.build import build
    build()
    return load()


def z(*shape, dtype=bf):
    return torch.zeros(*shape, dtype=dtype)


def test_norm_refuses(lib):
    def fwd(x=A, r=B, w=C, N=16, H=128, dt=MOE_BF16, eps=1e-6, h=D, y=E_):
        return lib.moe_add_rms_norm(x, r, w, N, H, dt, eps, h, y, None)
    assert fwd(x=None) == INV and fwd(w=None) == INV and fwd(y=None) == INV
    assert fwd(h=None) == INV                          # a residual needs somewhere to keep the sum
    assert fwd(x=A + 2) == INV and fwd(h=D + 8) == INV
    assert fwd(dt=2) == INV and fwd(N=-1) == INV and fwd(H=0) == INV
    assert fwd(eps=-1.0) == INV and fwd(eps=float("nan")) == INV
    assert fwd(H=12) == UNS and fwd(H=6, dt=MOE_F32) == UNS
    assert fwd(H=16392) == UNS and fwd(H=8196, dt=MOE_F32) == UNS
    assert fwd(h=E_) == INV                            # both outputs the same
    assert fwd(y=A + 256) == INV and fwd(h=B + 16) == INV and fwd(y=C - 256) == INV   # partial overlaps


def test_norm_backward_refuses(lib):
    def bwd(dy=A, h=B, w=C, dh=None, N=16, H=128, dt=MOE_BF16, eps=1e-6, dx=D, dw=E_, ws=6 * A, n=BIG):
        return lib.moe_add_rms_norm_bwd(dy, h, w, dh, N, H, dt, eps, dx, dw, ws, n, None)
    assert bwd(dy=None) == INV and bwd(h=None) == INV and bwd(w=None) == INV
    assert bwd(dx=None) == INV and bwd(dw=None) == INV
    assert bwd(ws=None) == WS and bwd(n=256) == WS
    assert bwd(dx=A + 16) == INV and bwd(dw=C) == INV and bwd(dw=D + 256) == INV
    assert bwd(H=4) == UNS and bwd(eps=-0.5) == INV and bwd(dh=A + 1) == INV
    size = lib.moe_add_rms_norm_bwd_workspace_size
    assert size(16, 12, MOE_BF16) == 0 and size(-1, 128, MOE_BF16) == 0
    last = 0
    for N in (0, 1, 2, 100, 148, 500, 3000, 1 << 20, 2 ** 31 - 1):     # never less for more rows
        assert size(N, 2048, MOE_F32) >= max(last, 256)
        last = size(N, 2048, MOE_F32)


def test_clip_refuses(lib):
    def clip(ptrs=(A, B), outs=None, sizes=(100, 100), dts=(MOE_F32, MOE_BF16), max_norm=1.0, norm=C, ws=D, n=BIG):
        k = len(ptrs)
        return lib.moe_clip_grad_norm((ctypes.c_void_p * k)(*ptrs),
                                      None if outs is None else (ctypes.c_void_p * k)(*outs),
                                      (ctypes.c_int64 * k)(*sizes), (ctypes.c_int32 * k)(*dts), k, max_norm, norm,
                                      ws, n, None)
    assert clip(ptrs=(A, None)) == INV and clip(ptrs=(A + 2, B)) == INV and clip(ptrs=(A, B + 1)) == INV
    assert clip(sizes=(100, -1)) == INV and clip(dts=(0, 7)) == INV
    assert clip(max_norm=-1.0) == INV and clip(max_norm=float("nan")) == INV
    assert clip(norm=None) == INV and clip(ws=None) == WS and clip(n=300) == WS and clip(ws=D + 4) == INV
    assert clip(ptrs=(A, A)) == INV                           # the same gradient twice
    assert clip(ptrs=(A, A + 396)) == INV                     # its last element shared
    assert clip(outs=(C, C + 200)) == INV                     # outputs that overlap
    assert clip(outs=(A + 16, C)) == INV                      # an output over its own gradient, shifted
    assert clip(outs=(B, C)) == INV                           # an output over another gradient
    assert clip(outs=(C, None)) == INV and clip(outs=(C + 1, D)) == INV
    assert lib.moe_clip_grad_norm(None, None, None, None, 3, 1.0, C, D, BIG, None) == INV
    assert lib.moe_clip_grad_norm(None, None, None, None, -1, 1.0, C, D, BIG, None) == INV
    assert lib.moe_clip_grad_norm_workspace_size(-1) == 0
    assert lib.moe_clip_grad_norm_workspace_size(769) > lib.moe_clip_grad_norm_workspace_size(768) > 256


def test_binding_checks_the_norms_tensors():
    x, w = z(4, 128), z(128)
    with pytest.raises(ValueError, match="x"):
        moe.moe_add_rms_norm(z(2, 4, 128), w)
    with pytest.raises(ValueError, match="weight"):
        moe.moe_add_rms_norm(x, z(64))
    with pytest.raises(TypeError, match="weight"):
        moe.moe_add_rms_norm(x, z(128, dtype=f32))
    with pytest.raises(ValueError, match="residual"):
        moe.moe_add_rms_norm(x, w, residual=z(5, 128))
    with pytest.raises(ValueError, match="h"):
        moe.moe_add_rms_norm(x, w, h=z(4, 128))
    with pytest.raises(TypeError, match="dtype"):
        moe.moe_add_rms_norm(z(4, 128, dtype=torch.float16), z(128, dtype=torch.float16))
    with pytest.raises(ValueError, match="CUDA"):
        moe.moe_add_rms_norm(x, w)
    with pytest.raises(ValueError, match="dh"):
        moe.moe_add_rms_norm_bwd(x, x, w, dh=z(4, 64))
    with pytest.raises(ValueError, match="dweight"):
        moe.moe_add_rms_norm_bwd(x, x, w, dweight=z(64))
    with pytest.raises(ValueError, match="CUDA"):
        moe.moe_add_rms_norm_bwd(x, x, w)


def test_binding_checks_the_gradients():
    with pytest.raises(ValueError, match="CUDA"):
        moe.moe_clip_grad_norm([z(4)], 1.0)
    with pytest.raises(TypeError, match="dtype"):
        moe.moe_clip_grad_norm([z(4, dtype=torch.float64)], 1.0)
    with pytest.raises(ValueError, match="outs"):
        moe.moe_clip_grad_norm([z(4)], 1.0, outs=[])
    with pytest.raises(ValueError, match=r"outs\[0\]"):
        moe.moe_clip_grad_norm([z(4)], 1.0, outs=[z(5)])
    with pytest.raises(TypeError, match=r"outs\[0\]"):
        moe.moe_clip_grad_norm([z(4)], 1.0, outs=[z(4, dtype=f32)])
    with pytest.raises(TypeError, match="norm"):
        moe.moe_clip_grad_norm([z(4)], 1.0, norm=z(1))


def test_few_token_layer_refuses(lib):
    def dec(x=A, W_r=B, W1=C, W3=D, W2=E_, N=16, H=128, E=4, K=2, F=256, dt=MOE_BF16, y=6 * A, top=7 * A, w=8 * A,
            ws=9 * A, n=BIG):
        return lib.moe_layer_decode(x, W_r, W1, W3, W2, N, H, E, K, F, dt, y, top, w, ws, n, None)
    for k in ("x", "W_r", "W1", "W3", "W2", "y", "top", "w"):
        assert dec(**{k: None}) == INV, k
        assert dec(**{k: 10 * A + 4}) == INV, k
    assert dec(ws=None) == WS and dec(n=1000) == WS and dec(ws=9 * A + 8) == INV
    assert dec(dt=5) == INV and dec(N=-1) == INV and dec(K=5) == INV and dec(K=0) == INV and dec(F=0) == INV
    assert dec(N=lib.moe_decode_max_tokens() + 1) == UNS
    assert dec(H=192) == UNS and dec(F=100) == UNS and dec(E=257) == UNS and dec(E=64, K=33) == UNS
    assert dec(dt=MOE_F32, H=130) == UNS and dec(F=(1 << 16) + 128) == UNS
    size = lib.moe_layer_decode_workspace_size
    assert size(16, 192, 4, 2, 256, MOE_BF16) == 0 and size(129, 128, 4, 2, 256, MOE_BF16) == 0
    for dt in (MOE_BF16, MOE_F32):                       # one workspace serves every smaller batch
        for H, E, K, F in ((128, 4, 2, 256), (4096, 64, 4, 2048), (7168, 256, 8, 2048), (4096, 8, 2, 14336)):
            last = 0
            for N in range(0, 129):
                assert size(N, H, E, K, F, dt) >= max(last, 256), (N, H)
                last = size(N, H, E, K, F, dt)


def test_binding_checks_the_few_token_layers_tensors():
    with pytest.raises(moe.MoEError):
        moe.MoEDecodeLayer(8, 100, 4, 2, 256)
    with pytest.raises(TypeError, match="dtype"):
        moe.MoEDecodeLayer(8, 128, 4, 2, 256, dtype=torch.float16)


def test_norm_refuses_shared_memory_in_a_single_row_too(lib):
    """A row of weight or dweight is as large as x or dx are when there is one row."""
    def fwd(N, x=A, r=B, w=C, h=D, y=E_):
        return lib.moe_add_rms_norm(x, r, w, N, 128, MOE_BF16, 1e-6, h, y, None)

    def bwd(N, dy=A, h=B, w=C, dh=None, dx=D, dw=E_):
        return lib.moe_add_rms_norm_bwd(dy, h, w, dh, N, 128, MOE_BF16, 1e-6, dx, dw, 6 * A, BIG, None)
    for N in (2, 1):
        assert fwd(N, h=C) == INV and fwd(N, y=C) == INV, N
        assert bwd(N, dw=D) == INV, N                               # dx and dweight the same
        assert bwd(N, dx=C) == INV and bwd(N, dw=C) == INV, N
        assert bwd(N, dw=A) == INV and bwd(N, dw=B) == INV and bwd(N, dh=7 * A, dw=7 * A) == INV, N
    assert bwd(0, dw=C) == INV


def test_few_token_tickets_cover_their_line(tmp_path):
    """tests/c_api/decode_line.cpp: the plain arithmetic of decode_line.cuh, run on the CPU."""
    import shutil
    import subprocess
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    exe = str(tmp_path / "decode_line")
    subprocess.run([cxx, "-std=c++17", "-O2", "-Wall", "-Wextra", "-Werror", "-x", "c++",
                    "-I", os.path.join(root, "dropless_top_moe_b200", "csrc"),
                    os.path.join(root, "tests", "c_api", "decode_line.cpp"), "-o", exe], check=True)
    res = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert res.returncode == 0, res.stdout[-2000:]


def test_clip_refuses_a_norm_or_workspace_inside_a_gradient(lib):
    """Both are written by the call: a block would scale, or sum, what another has overwritten."""
    def clip(norm, ws, outs=None):
        k = 2
        return lib.moe_clip_grad_norm((ctypes.c_void_p * k)(A, B), None if outs is None else (ctypes.c_void_p * k)(*outs),
                                      (ctypes.c_int64 * k)(100, 100), (ctypes.c_int32 * k)(MOE_F32, MOE_BF16), k, 1.0,
                                      norm, ws, BIG, None)
    size = lib.moe_clip_grad_norm_workspace_size(2)
    assert clip(A, D) == INV and clip(A + 396, D) == INV and clip(B + 196, D) == INV
    assert clip(C, A) == INV and clip(C, A + 384) == INV and clip(C, A - size + 16) == INV and clip(C, B - 256) == INV
    for outs in ((D, E_), (A, E_)):
        assert clip(E_ + 100, 9 * A, outs) == INV and clip(outs[0] + 4, 9 * A, outs) == INV
        assert clip(9 * A, E_ + 192, outs) == INV and clip(9 * A, outs[0] - 256, outs) == INV
        assert clip(B + 8, 9 * A, outs) == INV                       # a gradient that is only read


def test_handover_selftest_refuses(lib):
    st = lib.moe_selftest_handover_timeout
    assert st(None, BIG, 10 ** 6, A, None) == INV and st(A, BIG, 10 ** 6, None, None) == INV
    assert st(A + 4, BIG, 10 ** 6, B, None) == INV and st(A, 1000, 10 ** 6, B, None) == WS
    assert st(A, BIG, 10, B, None) == INV and st(A, BIG, 2 * 10 ** 9, B, None) == INV
