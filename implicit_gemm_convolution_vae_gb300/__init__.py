"""Python binding of ``libvae_igemm.so``, the sm_103a image-VAE decoder hot path.

Argument marshalling only: every step of the computation runs in the CUDA
library through its C ABI (``include/vae_igemm.h``); PyTorch provides the
device memory and the stream. There is no CPU fallback: if the library is
not built, or no sm_103a device is present, calls raise ``VaeError``.

Layouts follow the C ABI: activations NHWC, conv weights f16
``[cout][3][3][cin]`` (3x3) or ``[cout][cin]`` (1x1), streams f32, conv
inputs f16.
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import Optional

import numpy as np

from .build import LIB_PATH, build  # noqa: F401  (build is re-exported)

__all__ = [
    "VaeError", "lib", "version", "last_error", "sync_status", "set_wait_timeout_ns",
    "selftest_wait_timeout", "conv3x3_nhwc", "conv3x3_nhwc_rms", "conv3x3_nhwc_gn", "conv3x3_gn_workspace_bytes", "groupnorm_apply",
    "conv1x1", "rmsnorm_silu", "groupnorm_silu",
    "groupnorm_workspace_bytes", "cast_f16", "mid_attention", "mid_attention_workspace_bytes",
    "layernorm", "layernorm_backward", "layernorm_backward_workspace_bytes", "RopePlan", "rope",
    "attention", "attention_workspace_bytes", "attention_backward", "attention_backward_workspace_bytes",
    "Decoder", "DecodeGraph", "pack_conv3x3", "pack_conv1x1",
    "UPSAMPLE2X", "PAD_REPLICATE", "PAD_REFLECT", "DOWNSAMPLE2X", "EPI_SILU", "OUT_F16", "FAMILY_GN", "FAMILY_RMS",
    "NORM_GROUP", "NORM_RMS",
]

UPSAMPLE2X, PAD_REPLICATE, EPI_SILU, OUT_F16, UPSAMPLE_T2X, UPSAMPLE2X_SUBPIXEL = 1, 2, 16, 32, 64, 128
PAD_REFLECT, DOWNSAMPLE2X = 256, 512
FAMILY_GN, FAMILY_RMS = 0, 1
NORM_GROUP, NORM_RMS = 0, 1

STATUS_NAMES = {0: "VAE_OK", -1: "VAE_ERR_ARG", -2: "VAE_ERR_SHAPE", -3: "VAE_ERR_ALIGN",
                -4: "VAE_ERR_NOMEM", -5: "VAE_ERR_CUDA", -6: "VAE_ERR_DEVICE_TIMEOUT",
                -7: "VAE_ERR_UNSUPPORTED"}


class VaeError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{STATUS_NAMES.get(code, code)}: {msg}")
        self.code = code


_LIB = None
_P = ctypes.c_void_p
_I = ctypes.c_int
_F = ctypes.c_float
_SZ = ctypes.c_size_t

# Every exported function with its argument types (restype int unless noted).
SIGNATURES = {
    "vae_version": ([], ctypes.c_char_p),
    "vae_last_error": ([], ctypes.c_char_p),
    "vae_sync_status": ([_P], _I),
    "vae_set_wait_timeout_ns": ([ctypes.c_ulonglong], _I),
    "vae_selftest_wait_timeout": ([ctypes.c_ulonglong, _P], _I),
    "vae_conv3x3_nhwc": ([_P, _I, _I, _I, _I, _P, _P, _P, _P, _I, _F, ctypes.c_uint, _P], _I),
    "vae_conv3d_causal_ndhwc": ([_P, _I, _I, _I, _I, _I, _P, _P, _P, _P, _I, _F, ctypes.c_uint, _P], _I),
    "vae_pack_subpixel_weights": ([_P, _I, _I, _P, _P], _I),
    "vae_conv1x1": ([_P, _I, _I, _P, _P, _P, _P, _I, _F, ctypes.c_uint, _P], _I),
    "vae_conv3x3_nhwc_rms": ([_P, _I, _I, _I, _I, _P, _P, _P, _I, _F, ctypes.c_uint, _P, _I, _P, _P], _I),
    "vae_conv3x3_gn_workspace_bytes": ([_I, _I, _I, _I, _I, ctypes.c_uint], _SZ),
    "vae_conv3x3_nhwc_gn": ([_P, _I, _I, _I, _I, _P, _P, _P, _P, _I, _F, ctypes.c_uint, _I, _F, _P, _P, _SZ, _P], _I),
    "vae_groupnorm_apply": ([_P, _I, _I, _I, _I, _P, _P, _P, _I, _F, _P, _P], _I),
    "vae_rmsnorm_silu": ([_P, _I, _I, _P, _P, _I, _F, _P, _P], _I),
    "vae_groupnorm_workspace_bytes": ([_I, _I, _I, _I], _SZ),
    "vae_groupnorm_silu": ([_P, _I, _I, _I, _I, _F, _P, _P, _P, _I, _F, _P, _P, _SZ, _P], _I),
    "vae_groupnorm_silu_static": ([_P, _I, _I, _I, _I, _F, _P, _P, _P, _I, _F, _P, _P], _I),
    "vae_cast_f16": ([_P, _SZ, _I, _P, _F, _P, _P], _I),
    "vae_mid_attention_workspace_bytes": ([_I, _I, _I], _SZ),
    "vae_mid_attention": ([_P, _I, _I, _I, _I, _F, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P], _I),
    "vae_layernorm": ([_P, _I, _I, _I, _P, _P, _F, _P, _I, _P], _I),
    "vae_layernorm_backward_workspace_bytes": ([_I, _I], _SZ),
    "vae_layernorm_backward": ([_P, _I, _P, _I, _I, _I, _P, _F, _P, _P, _P, _P, _SZ, _P], _I),
    "vae_rope_plan_init": ([_P, _I, _P, ctypes.c_double, _I], _I),
    "vae_rope": ([_P, _I, _I, _I, _I, _I, _P, _P, _I, _I, _P, _I, _P, _P, _P], _I),
    "vae_attention_workspace_bytes": ([_P], _SZ),
    "vae_attention": ([_P, _P, _P, _P, _P, _P, _P, _SZ, _P], _I),
    "vae_attention_backward_workspace_bytes": ([_P], _SZ),
    "vae_attention_backward": ([_P] * 11 + [_SZ, _P], _I),
    "vae_decoder_create": ([_P, ctypes.POINTER(_P)], _I),
    "vae_decoder_destroy": ([_P], _I),
    "vae_decode_workspace": ([_P, _I, _I, _P, ctypes.POINTER(_SZ)], _I),
    "vae_decode": ([_P, _P, _I, _I, _P, _P, _P, _SZ, _P], _I),
    "vae_decode_host": ([_P, _P, _I, _I, _P, _P, _P, _SZ, _P], _I),
    "vae_decode_profile": ([_P, _P, _I, ctypes.POINTER(_I)], _I),
    "vae_decode_graph_create": ([_P, _P, _I, _I, _P, _P, _P, _SZ, _P, ctypes.POINTER(_P)], _I),
    "vae_decode_graph_launch": ([_P, _P], _I),
    "vae_decode_graph_destroy": ([_P], _I),
}


def lib():
    """The loaded library (raises if it was not built)."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise VaeError(-5, f"{os.path.basename(LIB_PATH)} is not built; run "
                               "`python -m implicit_gemm_convolution_vae_gb300.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in SIGNATURES.items():
            fn = getattr(L, name, None)
            if fn is None:
                continue
            fn.argtypes = args
            fn.restype = res
        _LIB = L
    return _LIB


def version() -> str:
    return lib().vae_version().decode()


def last_error() -> str:
    return lib().vae_last_error().decode()


def _check(rc: int):
    if rc != 0:
        raise VaeError(rc, last_error())


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream=None) -> int:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _need(t, dtype, name, ndim=None):
    import torch
    if t is None:
        return
    if not t.is_cuda:
        raise VaeError(-1, f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise VaeError(-1, f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise VaeError(-1, f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise VaeError(-2, f"{name} must have {ndim} dims, got {t.dim()}")


def sync_status(stream=None) -> int:
    """Synchronise the stream; raises VaeError(VAE_ERR_DEVICE_TIMEOUT) if a device wait ran out."""
    rc = lib().vae_sync_status(_stream(stream))
    _check(rc)
    return rc


def set_wait_timeout_ns(ns: int) -> None:
    _check(lib().vae_set_wait_timeout_ns(int(ns)))


def selftest_wait_timeout(timeout_ns: int = 1_000_000, stream=None) -> int:
    """Runs the bounded-wait self test; returns its status code (expected -6)."""
    return lib().vae_selftest_wait_timeout(int(timeout_ns), _stream(stream))


def pack_subpixel_weights(w, stream=None):
    """f16 [cout][3][3][cin] -> the up conv's sub-pixel weights f16 [cout][16][cin] (device)."""
    import torch
    _need(w, torch.float16, "w", 4)
    cout, _, _, cin = w.shape
    ws = torch.empty((cout, 16, cin), dtype=torch.float16, device=w.device)
    _check(lib().vae_pack_subpixel_weights(_ptr(w), cout, cin, _ptr(ws), _stream(stream)))
    return ws


def conv3x3_nhwc(x, w, bias=None, residual=None, out=None, oscale: float = 1.0, upsample: bool = False,
                 replicate: bool = False, silu: bool = False, out_f16: bool = False, subpixel: bool = False,
                 reflect: bool = False, down: bool = False, stream=None):
    """3x3 implicit-GEMM conv. x f16 [n][h][w][cin]; w f16 [cout][3][3][cin], or with
    ``subpixel`` (an up conv) the summed weights [cout][16][cin] of pack_subpixel_weights.
    ``reflect``: mirror padding; ``down``: the encoder's far-side-padded stride-2
    downsample (output [n][h//2][w//2][cout])."""
    import torch
    _need(x, torch.float16, "x", 4)
    _need(w, torch.float16, "w", 3 if subpixel else 4)
    _need(bias, torch.float32, "bias", 1)
    n, h, wd, cin = x.shape
    cout = w.shape[0]
    if tuple(w.shape[1:]) != ((16, cin) if subpixel else (3, 3, cin)):
        raise VaeError(-2, f"w has the wrong shape {tuple(w.shape)}")
    H, W = (2 * h, 2 * wd) if upsample else ((h // 2, wd // 2) if down else (h, wd))
    odt = torch.float16 if out_f16 else torch.float32
    if out is None:
        out = torch.empty((n, H, W, cout), dtype=odt, device=x.device)
    _need(out, odt, "out")
    _need(residual, torch.float32, "residual")
    for t, nm in ((out, "out"), (residual, "residual")):
        if t is not None and t.numel() != n * H * W * cout:
            raise VaeError(-2, f"{nm} must hold [n][{H}][{W}][{cout}], got {tuple(t.shape)}")
    flags = (UPSAMPLE2X if upsample else 0) | (PAD_REPLICATE if replicate else 0) | \
            (EPI_SILU if silu else 0) | (OUT_F16 if out_f16 else 0) | (UPSAMPLE2X_SUBPIXEL if subpixel else 0) | \
            (PAD_REFLECT if reflect else 0) | (DOWNSAMPLE2X if down else 0)
    _check(lib().vae_conv3x3_nhwc(_ptr(x), n, h, wd, cin, _ptr(w), _ptr(bias), _ptr(residual), _ptr(out),
                                  cout, float(oscale), flags, _stream(stream)))
    return out


def conv3x3_nhwc_gn(x, w, groups: int, bias=None, residual=None, out=None, oscale: float = 1.0,
                    upsample: bool = False, replicate: bool = False, reflect: bool = False, down: bool = False,
                    silu: bool = False, eps: float = 1e-6, workspace=None, stream=None):
    """3x3 conv (f32 output) that also returns the GroupNorm statistics of its
    output: (y [n][H][W][cout] f32, stats [n][groups][2] f32 = (mean, rstd))."""
    import torch
    _need(x, torch.float16, "x", 4)
    _need(w, torch.float16, "w", 4)
    _need(bias, torch.float32, "bias", 1)
    n, h, wd, cin = x.shape
    cout = w.shape[0]
    if tuple(w.shape[1:]) != (3, 3, cin):
        raise VaeError(-2, f"w has the wrong shape {tuple(w.shape)}")
    H, W = (2 * h, 2 * wd) if upsample else ((h // 2, wd // 2) if down else (h, wd))
    if out is None:
        out = torch.empty((n, H, W, cout), dtype=torch.float32, device=x.device)
    _need(out, torch.float32, "out")
    _need(residual, torch.float32, "residual")
    for t, nm in ((out, "out"), (residual, "residual")):
        if t is not None and t.numel() != n * H * W * cout:
            raise VaeError(-2, f"{nm} must hold [n][{H}][{W}][{cout}], got {tuple(t.shape)}")
    flags = (UPSAMPLE2X if upsample else 0) | (PAD_REPLICATE if replicate else 0) | (EPI_SILU if silu else 0) | \
            (PAD_REFLECT if reflect else 0) | (DOWNSAMPLE2X if down else 0)
    need = conv3x3_gn_workspace_bytes(n, h, wd, cout, groups, flags)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=x.device)
    stats = torch.empty((n, groups, 2), dtype=torch.float32, device=x.device)
    _check(lib().vae_conv3x3_nhwc_gn(_ptr(x), n, h, wd, cin, _ptr(w), _ptr(bias), _ptr(residual), _ptr(out), cout,
                                     float(oscale), flags, int(groups), float(eps), _ptr(stats), _ptr(workspace),
                                     workspace.numel(), _stream(stream)))
    return out, stats


def conv3x3_nhwc_rms(x, w, gamma, bias=None, out=None, y=None, oscale: float = 1.0, silu: bool = True,
                     replicate: bool = False, reflect: bool = False, down: bool = False, stream=None):
    """3x3 conv with RMS_norm(+SiLU) of each output pixel in its epilogue: f16
    [n][H][W][cout] (and, if ``y`` is given, the f32 conv output into it)."""
    import torch
    _need(x, torch.float16, "x", 4)
    _need(w, torch.float16, "w", 4)
    _need(gamma, torch.float32, "gamma", 1)
    _need(bias, torch.float32, "bias", 1)
    n, h, wd, cin = x.shape
    cout = w.shape[0]
    if tuple(w.shape[1:]) != (3, 3, cin):
        raise VaeError(-2, f"w has the wrong shape {tuple(w.shape)}")
    H, W = (h // 2, wd // 2) if down else (h, wd)
    if out is None:
        out = torch.empty((n, H, W, cout), dtype=torch.float16, device=x.device)
    _need(out, torch.float16, "out")
    _need(y, torch.float32, "y")
    for t, nm in ((out, "out"), (y, "y")):
        if t is not None and t.numel() != n * H * W * cout:
            raise VaeError(-2, f"{nm} must hold [n][{H}][{W}][{cout}], got {tuple(t.shape)}")
    flags = (PAD_REPLICATE if replicate else 0) | (PAD_REFLECT if reflect else 0) | (DOWNSAMPLE2X if down else 0)
    _check(lib().vae_conv3x3_nhwc_rms(_ptr(x), n, h, wd, cin, _ptr(w), _ptr(bias), _ptr(y), cout, float(oscale),
                                      flags, _ptr(gamma), 1 if silu else 0, _ptr(out), _stream(stream)))
    return out


def conv3x3_gn_workspace_bytes(n: int, h: int, w: int, cout: int, groups: int, flags: int = 0) -> int:
    return int(lib().vae_conv3x3_gn_workspace_bytes(n, h, w, cout, groups, flags))


def groupnorm_apply(x, groups: int, stats, gamma, beta, silu: bool = False, out_scale: float = 1.0, out=None,
                    stream=None):
    """GroupNorm from precomputed statistics. x f32 [n][hw][c] -> f16 [n][hw][c]."""
    import torch
    _need(x, torch.float32, "x", 3)
    _need(stats, torch.float32, "stats")
    _need(gamma, torch.float32, "gamma", 1)
    _need(beta, torch.float32, "beta", 1)
    n, hw, c = x.shape
    if stats.numel() != n * groups * 2:
        raise VaeError(-2, f"stats must hold [n][{groups}][2], got {tuple(stats.shape)}")
    if out is None:
        out = torch.empty((n, hw, c), dtype=torch.float16, device=x.device)
    _need(out, torch.float16, "out")
    _check(lib().vae_groupnorm_apply(_ptr(x), n, hw, c, groups, _ptr(stats), _ptr(gamma), _ptr(beta),
                                     1 if silu else 0, float(out_scale), _ptr(out), _stream(stream)))
    return out


def conv3d_causal_ndhwc(x, w, bias=None, residual=None, out=None, oscale: float = 1.0, upsample: bool = False,
                        t_upsample: bool = False, replicate: bool = False, silu: bool = False,
                        out_f16: bool = False, stream=None):
    """3x3x3 causal conv over frames. x f16 [n][f][h][w][cin]; w f16 [cout][3][3][3][cin]."""
    import torch
    _need(x, torch.float16, "x", 5)
    _need(w, torch.float16, "w", 5)
    _need(bias, torch.float32, "bias", 1)
    n, f, h, wd, cin = x.shape
    cout = w.shape[0]
    if tuple(w.shape[1:]) != (3, 3, 3, cin):
        raise VaeError(-2, f"w must be [cout][3][3][3][{cin}], got {tuple(w.shape)}")
    F = 2 * f - 1 if t_upsample else f
    H, W = (2 * h, 2 * wd) if upsample else (h, wd)
    odt = torch.float16 if out_f16 else torch.float32
    if out is None:
        out = torch.empty((n, F, H, W, cout), dtype=odt, device=x.device)
    _need(out, odt, "out")
    _need(residual, torch.float32, "residual")
    flags = (UPSAMPLE2X if upsample else 0) | (UPSAMPLE_T2X if t_upsample else 0) | \
            (PAD_REPLICATE if replicate else 0) | (EPI_SILU if silu else 0) | (OUT_F16 if out_f16 else 0)
    _check(lib().vae_conv3d_causal_ndhwc(_ptr(x), n, f, h, wd, cin, _ptr(w), _ptr(bias), _ptr(residual), _ptr(out),
                                         cout, float(oscale), flags, _stream(stream)))
    return out


def conv1x1(x, w, bias=None, residual=None, out=None, oscale: float = 1.0, silu: bool = False,
            out_f16: bool = False, stream=None):
    """1x1 conv (GEMM). x f16 [m][cin]; w f16 [cout][cin]."""
    import torch
    _need(x, torch.float16, "x", 2)
    _need(w, torch.float16, "w", 2)
    _need(bias, torch.float32, "bias", 1)
    m, cin = x.shape
    cout = w.shape[0]
    odt = torch.float16 if out_f16 else torch.float32
    if out is None:
        out = torch.empty((m, cout), dtype=odt, device=x.device)
    _need(out, odt, "out")
    _need(residual, torch.float32, "residual")
    flags = (EPI_SILU if silu else 0) | (OUT_F16 if out_f16 else 0)
    _check(lib().vae_conv1x1(_ptr(x), m, cin, _ptr(w), _ptr(bias), _ptr(residual), _ptr(out), cout,
                             float(oscale), flags, _stream(stream)))
    return out


def rmsnorm_silu(x, gamma, bias_in=None, silu: bool = False, out_scale: float = 1.0, out=None, stream=None):
    """Per-pixel RMS_norm. x f32 [m][c] -> f16 [m][c]."""
    import torch
    _need(x, torch.float32, "x", 2)
    _need(gamma, torch.float32, "gamma", 1)
    _need(bias_in, torch.float32, "bias_in", 1)
    m, c = x.shape
    if out is None:
        out = torch.empty((m, c), dtype=torch.float16, device=x.device)
    _need(out, torch.float16, "out")
    _check(lib().vae_rmsnorm_silu(_ptr(x), m, c, _ptr(bias_in), _ptr(gamma), int(silu), float(out_scale),
                                  _ptr(out), _stream(stream)))
    return out


def groupnorm_workspace_bytes(n: int, hw: int, c: int, groups: int) -> int:
    return int(lib().vae_groupnorm_workspace_bytes(n, hw, c, groups))


def groupnorm_silu(x, groups: int, gamma, beta, eps: float = 1e-6, bias_in=None, silu: bool = False,
                   out_scale: float = 1.0, out=None, workspace=None, stream=None):
    """GroupNorm. x f32 [n][hw][c] -> f16 [n][hw][c]."""
    import torch
    _need(x, torch.float32, "x", 3)
    _need(gamma, torch.float32, "gamma", 1)
    _need(beta, torch.float32, "beta", 1)
    _need(bias_in, torch.float32, "bias_in", 1)
    n, hw, c = x.shape
    if out is None:
        out = torch.empty((n, hw, c), dtype=torch.float16, device=x.device)
    _need(out, torch.float16, "out")
    nb = groupnorm_workspace_bytes(n, hw, c, groups)
    if workspace is None:
        workspace = torch.empty(max(nb, 16), dtype=torch.uint8, device=x.device)
    _check(lib().vae_groupnorm_silu(_ptr(x), n, hw, c, groups, float(eps), _ptr(bias_in), _ptr(gamma),
                                    _ptr(beta), int(silu), float(out_scale), _ptr(out), _ptr(workspace),
                                    workspace.numel() * workspace.element_size(), _stream(stream)))
    return out


def cast_f16(x, c: int, bias=None, scale: float = 1.0, out=None, stream=None):
    """(x + bias[c]) * scale -> f16, elementwise over a [.., c] f32 tensor."""
    import torch
    _need(x, torch.float32, "x")
    _need(bias, torch.float32, "bias", 1)
    if out is None:
        out = torch.empty(x.shape, dtype=torch.float16, device=x.device)
    _need(out, torch.float16, "out")
    _check(lib().vae_cast_f16(_ptr(x), x.numel(), c, _ptr(bias), float(scale), _ptr(out), _stream(stream)))
    return out


def mid_attention_workspace_bytes(m: int, c: int, groups: int = 32) -> int:
    return int(lib().vae_mid_attention_workspace_bytes(m, c, groups))


def mid_attention(x, norm_kind: int, gamma, beta, wq, bq, wk, bk, wv, bv, wo, bo, groups: int = 32,
                  eps: float = 1e-6, workspace=None, stream=None):
    """In-place mid self-attention on x f32 [m][c]; w* f16 [c][c], b* f32 [c]."""
    import torch
    _need(x, torch.float32, "x", 2)
    for nm, t in (("wq", wq), ("wk", wk), ("wv", wv), ("wo", wo)):
        _need(t, torch.float16, nm, 2)
    m, c = x.shape
    nb = mid_attention_workspace_bytes(m, c, groups)
    if workspace is None:
        workspace = torch.empty(max(nb, 16), dtype=torch.uint8, device=x.device)
    _check(lib().vae_mid_attention(_ptr(x), m, c, int(norm_kind), groups, float(eps), _ptr(gamma), _ptr(beta),
                                   _ptr(wq), _ptr(bq), _ptr(wk), _ptr(bk), _ptr(wv), _ptr(bv), _ptr(wo),
                                   _ptr(bo), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                   _stream(stream)))
    return x


# ───────────────────────── operators on latent tokens ─────────────────────────
#
# Small calls are bound by what happens on the host, so this part builds no
# temporary ctypes objects and asks PyTorch for each thing once.

_T = None  # torch, once a call needs it


class _Torch:
    """What the calls below take from torch, looked up once."""

    def __init__(self):
        import torch
        self.torch, self.empty, self.zeros = torch, torch.empty, torch.zeros
        self.f32, self.i32, self.u8 = torch.float32, torch.int32, torch.uint8
        self.device, self.stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
        self.types = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}


def _torch():
    global _T
    if _T is None:
        _T = _Torch()
    return _T


def _type(dt, name):
    """The C ABI's element type of a torch dtype."""
    code = _T.types.get(dt)
    if code is None:
        raise VaeError(-1, f"{name} must be float32, float16 or bfloat16, got {dt}")
    return code


def _device_of(named):
    """The index of the device that the given tensors (pairs of a name and a tensor or None) share."""
    index = None
    for name, t in named:
        if t is not None:
            i = t.get_device()
            if i != index:
                if i < 0:
                    raise VaeError(-1, f"{name} must be a CUDA tensor")
                if index is not None:
                    raise VaeError(-1, f"{name} is on cuda:{i}, the others on cuda:{index}")
                index = i
    return index


class _On:
    """Makes the tensors' device the current one for a call, and ``stream``, where one is given, the
    current stream, so that what the call allocates and fills belongs to the stream that it runs on."""

    def __init__(self, index, stream):
        import torch
        if stream is not None and stream.device.index != index:
            raise VaeError(-1, f"the stream is on {stream.device}, the tensors on cuda:{index}")
        self.device = torch.cuda.device(index)
        self.stream = None if stream is None else torch.cuda.stream(stream)

    def __enter__(self):
        self.device.__enter__()
        if self.stream is not None:
            self.stream.__enter__()

    def __exit__(self, *exc):
        if self.stream is not None:
            self.stream.__exit__(*exc)
        self.device.__exit__(*exc)


def _call(index, stream, f, *args):
    """f(*args, raw stream) on the tensors' device and the given or current stream."""
    T = _T or _torch()
    if stream is None and index == T.device():
        return f(*args, T.stream(index))
    with _On(index, stream):
        return f(*args, T.stream(index))


def _given(**tensors):
    for name, t in tensors.items():
        if t is None:
            raise VaeError(-1, f"{name} is needed")


_INT = (1 << 31) - 1  # the C ABI's sizes; ctypes would cut a larger one off without a word


def _sizes(**sizes):
    for name, n in sizes.items():
        if n > _INT:
            raise VaeError(-2, f"{name} must be below 2^31, got {n}")


def _tensor(t, name, dtype, shape):
    """Checks a tensor's type, shape and that it is contiguous."""
    if t.dtype is dtype and t.shape == shape and t.is_contiguous():
        return
    if t.dtype is not dtype:
        raise VaeError(-1, f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise VaeError(-2, f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    raise VaeError(-1, f"{name} must be contiguous")


def _work(workspace):
    """(pointer, bytes) of a workspace tensor or None."""
    if workspace is None:
        return None, 0
    if not workspace.is_contiguous():
        raise VaeError(-1, "workspace must be contiguous")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def layernorm(x, gamma=None, beta=None, eps: float = 1e-6, out_dtype=None, out=None, stream=None):
    """Layer norm of each row of x [m][c] (f32, f16 or bf16); gamma, beta f32 [c] or None.
    The result has ``out_dtype`` (default: x's), or is written into ``out``."""
    if x is None:
        _given(x=x)
    index = _device_of((("x", x), ("gamma", gamma), ("beta", beta), ("out", out)))
    return _call(index, stream, _layernorm, x, gamma, beta, eps, out_dtype, out)


def _layernorm(x, gamma, beta, eps, out_dtype, out, stream):
    if x.dim() != 2:
        raise VaeError(-2, f"x must have 2 dims, got {x.dim()}")
    shape = x.shape
    m, c = shape
    if m > _INT or c > _INT:
        _sizes(m=m, c=c)
    _tensor(x, "x", x.dtype, shape)
    if gamma is not None:
        _tensor(gamma, "gamma", _T.f32, (c,))
    if beta is not None:
        _tensor(beta, "beta", _T.f32, (c,))
    if out is None:
        out = _T.empty(shape, dtype=out_dtype or x.dtype, device=x.device)
    else:
        _tensor(out, "out", out_dtype or out.dtype, shape)
    _check(lib().vae_layernorm(x.data_ptr(), _type(x.dtype, "x"), m, c, _ptr(gamma), _ptr(beta), eps, out.data_ptr(),
                               _type(out.dtype, "out"), stream))
    return out


def layernorm_backward_workspace_bytes(m: int, c: int) -> int:
    _sizes(m=m, c=c)
    return int(lib().vae_layernorm_backward_workspace_bytes(m, c))


def layernorm_backward(dy, x, gamma=None, eps: float = 1e-6, weight_grads: bool = True, dx=None, dgamma=None,
                       dbeta=None, workspace=None, stream=None):
    """The gradient of layernorm at x [m][c] for dy [m][c]: (dx of x's type, dgamma, dbeta f32 [c]);
    with ``weight_grads`` False the last two are None and not computed."""
    if dy is None or x is None:
        _given(dy=dy, x=x)
    index = _device_of((("dy", dy), ("x", x), ("gamma", gamma), ("dx", dx), ("dgamma", dgamma), ("dbeta", dbeta),
                        ("workspace", workspace)))
    return _call(index, stream, _layernorm_backward, dy, x, gamma, eps, weight_grads, dx, dgamma, dbeta, workspace)


def _layernorm_backward(dy, x, gamma, eps, weight_grads, dx, dgamma, dbeta, workspace, stream):
    if x.dim() != 2:
        raise VaeError(-2, f"x must have 2 dims, got {x.dim()}")
    shape = x.shape
    m, c = shape
    if m > _INT or c > _INT:
        _sizes(m=m, c=c)
    _tensor(x, "x", x.dtype, shape)
    _tensor(dy, "dy", dy.dtype, shape)
    if gamma is not None:
        _tensor(gamma, "gamma", _T.f32, (c,))
    if dx is None:
        dx = _T.torch.empty_like(x)
    else:
        _tensor(dx, "dx", x.dtype, shape)
    if weight_grads:
        if dgamma is None:
            dgamma = _T.empty((c,), dtype=_T.f32, device=x.device)
        else:
            _tensor(dgamma, "dgamma", _T.f32, (c,))
        if dbeta is None:
            dbeta = _T.empty((c,), dtype=_T.f32, device=x.device)
        else:
            _tensor(dbeta, "dbeta", _T.f32, (c,))
        if workspace is None:
            workspace = _T.empty(max(lib().vae_layernorm_backward_workspace_bytes(m, c), 16), dtype=_T.u8,
                                    device=x.device)
    elif dgamma is not None or dbeta is not None:
        raise VaeError(-1, "dgamma and dbeta need weight_grads")
    _check(lib().vae_layernorm_backward(dy.data_ptr(), _type(dy.dtype, "dy"), x.data_ptr(), _type(x.dtype, "x"), m, c,
                                        _ptr(gamma), eps, dx.data_ptr(), _ptr(dgamma), _ptr(dbeta), *_work(workspace),
                                        stream))
    return dx, dgamma, dbeta


class _RopePlan(ctypes.Structure):
    _fields_ = [("naxes", _I), ("pairs", _I), ("interleaved", _I), ("turns_hi", _F * 128), ("turns_lo", _F * 128),
                ("axis", ctypes.c_ubyte * 128)]


class RopePlan:
    """The pairs and frequencies of a rotary embedding: ``axes`` channels per axis (even numbers),
    ``theta`` the base, pairs (2p, 2p + 1) when ``interleaved``, else (p, p + R/2)."""

    def __init__(self, axes, theta: float = 10000.0, interleaved: bool = True):
        self.axes = tuple(int(a) for a in axes)
        _sizes(axes=max((abs(a) for a in self.axes), default=0))
        self._plan = _RopePlan()
        dims = (_I * max(1, len(self.axes)))(*self.axes)
        _check(lib().vae_rope_plan_init(ctypes.byref(self._plan), len(self.axes), dims, float(theta),
                                        int(bool(interleaved))))
        self._at = ctypes.addressof(self._plan)


_STRIDES = struct.Struct("=3q")


def _strides3(t, name):
    """The {batch, token, head} strides of a [b][n][heads][d] tensor whose channels are contiguous."""
    st = t.stride()
    if st[3] != 1 and t.shape[3] > 1:
        raise VaeError(-1, f"{name}'s last dim must be contiguous")
    return st[:3]


def rope(x, positions, plan: RopePlan, inverse: bool = False, out=None, stream=None):
    """Turns the pairs of x [b][s][h][d] (strides free, channels contiguous) by their angles at
    ``positions`` [s][axes] or [b][s][axes] (f32 or int32); ``inverse`` turns back (the gradient).
    ``out`` may be x."""
    if x is None or positions is None or plan is None:
        _given(x=x, positions=positions, plan=plan)
    index = _device_of((("x", x), ("positions", positions), ("out", out)))
    return _call(index, stream, _rope, x, positions, plan, inverse, out)


def _rope(x, positions, plan, inverse, out, stream):
    if x.dim() != 4:
        raise VaeError(-2, f"x must have 4 dims, got {x.dim()}")
    shape = x.shape
    b, s, h, d = shape
    if b > _INT or s > _INT or h > _INT or d > _INT:
        _sizes(b=b, s=s, h=h, d=d)
    ints = positions.dtype == _T.i32
    if not ints and positions.dtype != _T.f32:
        raise VaeError(-1, f"positions must be float32 or int32, got {positions.dtype}")
    pb = positions.shape[0] if positions.dim() == 3 else 1
    na = len(plan.axes)
    _tensor(positions, "positions", positions.dtype, (pb, s, na) if positions.dim() == 3 else (s, na))
    if out is None:
        out = _T.empty(shape, dtype=x.dtype, device=x.device)
    elif out.shape != shape:
        raise VaeError(-2, f"out must be {tuple(shape)}, got {tuple(out.shape)}")
    elif out.dtype != x.dtype:
        raise VaeError(-1, f"out must be {x.dtype}, got {out.dtype}")
    _check(lib().vae_rope(x.data_ptr(), _type(x.dtype, "x"), b, s, h, d, _STRIDES.pack(*_strides3(x, "x")),
                          positions.data_ptr(), ints, pb, plan._at, bool(inverse), out.data_ptr(),
                          _STRIDES.pack(*_strides3(out, "out")), stream))
    return out


# struct vae_attention_desc: type .. d, scale, block, fill, the two lengths, eight times three strides
_DESC = struct.Struct("=7if2i2Q24q")
_NO_STRIDES = (0,) * 12


def _attention_args(q, k, v, scale, q_len, k_len, block, fill):
    """The desc's fields up to v's strides; checks q, k, v and the lengths."""
    dtype = q.dtype
    for t, nm in ((q, "q"), (k, "k"), (v, "v")):
        if t.dim() != 4:
            raise VaeError(-2, f"{nm} must have 4 dims, got {t.dim()}")
        if t.dtype != dtype:
            raise VaeError(-1, f"{nm} must be {dtype}, got {t.dtype}")
    b, sq, hq, d = q.shape
    kshape = k.shape
    _, sk, hkv, _ = kshape
    if b > _INT or sq > _INT or sk > _INT or hq > _INT or hkv > _INT or d > _INT:
        _sizes(b=b, sq=sq, sk=sk, hq=hq, hkv=hkv, d=d)
    if kshape[0] != b or kshape[3] != d:
        raise VaeError(-2, f"k must be {(b, sk, hkv, d)}, got {tuple(kshape)}")
    if v.shape != kshape:
        raise VaeError(-2, f"v must be {tuple(kshape)}, got {tuple(v.shape)}")
    if not 0 <= block < 1 << 31:
        raise VaeError(-1, f"block must be >= 0 and fit 31 bits, got {block}")
    if q_len is not None:
        _tensor(q_len, "q_len", _T.i32, (b,))
    if k_len is not None:
        _tensor(k_len, "k_len", _T.i32, (b,))
    return (_type(dtype, "q"), b, sq, sk, hq, hkv, d, 1.0 / d ** 0.5 if scale is None else scale, block, fill,
            0 if q_len is None else q_len.data_ptr(), 0 if k_len is None else k_len.data_ptr(), *_strides3(q, "q"),
            *_strides3(k, "k"), *_strides3(v, "v"))


def _like(t, ref, name, lens):
    """``t`` checked against ``ref``'s shape and type, or a new dense tensor (zeros where ``lens`` leaves
    rows unwritten)."""
    if t is None:
        return (_T.empty if lens is None else _T.zeros)(ref.shape, dtype=ref.dtype, device=ref.device)
    if t.shape != ref.shape:
        raise VaeError(-2, f"{name} must be {tuple(ref.shape)}, got {tuple(t.shape)}")
    if t.dtype != ref.dtype:
        raise VaeError(-1, f"{name} must be {ref.dtype}, got {t.dtype}")
    return t


def _dense(n, h, d):
    return n * h * d, h * d, d


def attention_workspace_bytes(b: int, sq: int, sk: int, hq: int, hkv: int, d: int, block: int = 0) -> int:
    _sizes(b=b, sq=sq, sk=sk, hq=hq, hkv=hkv, d=d, block=block)
    q, k = _dense(sq, hq, d), _dense(sk, hkv, d)
    return int(lib().vae_attention_workspace_bytes(_DESC.pack(1, b, sq, sk, hq, hkv, d, 1.0, block, 0, 0, 0, *q, *k, *k, *q,
                                                              *_NO_STRIDES)))


def attention(q, k, v, scale: Optional[float] = None, q_len=None, k_len=None, block: int = 0, out=None, lse=None,
              workspace=None, stream=None):
    """Multi-head attention of q [b][sq][hq][d] over k, v [b][sk][hkv][d] (f16 or bf16, strides free,
    channels contiguous; scale default 1/sqrt(d)). q_len, k_len int32 [b]: the valid rows of a padded
    batch. block 0: every valid key; block > 0: the keys of the query's own block of that many
    positions and of the earlier ones (1: causal). Returns (o, lse f32 [b][hq][sq]); rows behind q_len
    are left as they were in ``out`` and ``lse``, 0 and -inf in new ones."""
    if q is None or k is None or v is None:
        _given(q=q, k=k, v=v)
    index = _device_of((("q", q), ("k", k), ("v", v), ("q_len", q_len), ("k_len", k_len), ("out", out), ("lse", lse),
                        ("workspace", workspace)))
    return _call(index, stream, _attention, q, k, v, scale, q_len, k_len, block, out, lse, workspace)


def _attention(q, k, v, scale, q_len, k_len, block, out, lse, workspace, stream):
    # new tensors are filled behind the lengths by the kernels; beside one that the caller gave, beforehand
    fill = out is None and lse is None
    args = _attention_args(q, k, v, scale, q_len, k_len, block, fill)
    b, sq, hq, _ = q.shape
    out = _like(out, q, "out", None if fill else q_len)
    if lse is not None:
        _tensor(lse, "lse", _T.f32, (b, hq, sq))
    elif fill or q_len is None:
        lse = _T.empty((b, hq, sq), dtype=_T.f32, device=q.device)
    else:
        lse = _T.torch.full((b, hq, sq), -float("inf"), dtype=_T.f32, device=q.device)
    desc = _DESC.pack(*args, *_strides3(out, "out"), *_NO_STRIDES)
    L = lib()
    if workspace is None:
        nb = L.vae_attention_workspace_bytes(desc)
        workspace = _T.empty(nb, dtype=_T.u8, device=q.device) if nb else None
    _check(L.vae_attention(desc, q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                           *_work(workspace), stream))
    return out, lse


def attention_backward_workspace_bytes(b: int, sq: int, sk: int, hq: int, hkv: int, d: int, block: int = 0) -> int:
    _sizes(b=b, sq=sq, sk=sk, hq=hq, hkv=hkv, d=d, block=block)
    q, k = _dense(sq, hq, d), _dense(sk, hkv, d)
    return int(lib().vae_attention_backward_workspace_bytes(
        _DESC.pack(1, b, sq, sk, hq, hkv, d, 1.0, block, 0, 0, 0, *q, *k, *k, *q, *q, *q, *k, *k)))


def attention_backward(do, q, k, v, o, lse, scale: Optional[float] = None, q_len=None, k_len=None, block: int = 0,
                       dq=None, dk=None, dv=None, workspace=None, stream=None):
    """The gradient of attention for do [b][sq][hq][d], from o and lse of the same call: (dq, dk, dv).
    Rows behind q_len and k_len are left as they were, 0 in new tensors."""
    if do is None or q is None or k is None or v is None or o is None or lse is None:
        _given(do=do, q=q, k=k, v=v, o=o, lse=lse)
    index = _device_of((("do", do), ("q", q), ("k", k), ("v", v), ("o", o), ("lse", lse), ("q_len", q_len),
                        ("k_len", k_len), ("dq", dq), ("dk", dk), ("dv", dv), ("workspace", workspace)))
    return _call(index, stream, _attention_backward, do, q, k, v, o, lse, scale, q_len, k_len, block, dq, dk, dv,
                 workspace)


def _attention_backward(do, q, k, v, o, lse, scale, q_len, k_len, block, dq, dk, dv, workspace, stream):
    fill = dq is None and dk is None and dv is None
    args = _attention_args(q, k, v, scale, q_len, k_len, block, fill)
    b, sq, hq, _ = q.shape
    _like(do, q, "do", None)
    _like(o, q, "o", None)
    _tensor(lse, "lse", _T.f32, (b, hq, sq))
    q_fill, k_fill = (None, None) if fill else (q_len, k_len)
    dq = _like(dq, q, "dq", q_fill)
    dk, dv = _like(dk, k, "dk", k_fill), _like(dv, k, "dv", k_fill)
    desc = _DESC.pack(*args, *_strides3(o, "o"), *_strides3(do, "do"), *_strides3(dq, "dq"), *_strides3(dk, "dk"),
                      *_strides3(dv, "dv"))
    L = lib()
    if workspace is None:
        workspace = _T.empty(max(L.vae_attention_backward_workspace_bytes(desc), 16), dtype=_T.u8,
                                device=q.device)
    _check(L.vae_attention_backward(desc, do.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                                    lse.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), *_work(workspace),
                                    stream))
    return dq, dk, dv


# ───────────────────────────── weight layouts ─────────────────────────────

def pack_conv3x3(w_oihw: np.ndarray) -> np.ndarray:
    """OIHW [cout][cin][3][3] -> the kernel's [cout][3][3][cin] (a permutation)."""
    return np.ascontiguousarray(np.asarray(w_oihw).transpose(0, 2, 3, 1))


def pack_conv3d(w_oidhw: np.ndarray) -> np.ndarray:
    """OIDHW [cout][cin][3][3][3] -> the kernel's [cout][3][3][3][cin] (a permutation)."""
    return np.ascontiguousarray(np.asarray(w_oidhw).transpose(0, 2, 3, 4, 1))


def pack_conv1x1(w_oihw: np.ndarray) -> np.ndarray:
    """OIHW [cout][cin][1][1] -> [cout][cin]."""
    w = np.asarray(w_oihw)
    return np.ascontiguousarray(w.reshape(w.shape[0], w.shape[1]))


# ───────────────────────────── whole decoder ─────────────────────────────

class _ConvDesc(ctypes.Structure):
    _fields_ = [("w", _P), ("b", _P), ("cout", _I), ("cin", _I), ("k", _I)]


class _NormDesc(ctypes.Structure):
    _fields_ = [("gamma", _P), ("beta", _P)]


class _ResnetDesc(ctypes.Structure):
    _fields_ = [("norm1", _NormDesc), ("conv1", _ConvDesc), ("norm2", _NormDesc), ("conv2", _ConvDesc),
                ("shortcut", _ConvDesc)]


class _AttnDesc(ctypes.Structure):
    _fields_ = [("norm", _NormDesc), ("q", _ConvDesc), ("k", _ConvDesc), ("v", _ConvDesc), ("o", _ConvDesc)]


class _UpDesc(ctypes.Structure):
    _fields_ = [("resnets", ctypes.POINTER(_ResnetDesc)), ("n_resnets", _I), ("up", _ConvDesc),
                ("in_dim", _I), ("out_dim", _I), ("ft", _I)]


class _DecoderDesc(ctypes.Structure):
    _fields_ = [("family", _I), ("latent_channels", _I), ("scaling", _F), ("shift", _F), ("groups", _I),
                ("eps", _F), ("dupup", _I), ("post_quant", _ConvDesc), ("conv_in", _ConvDesc),
                ("mid_res1", _ResnetDesc), ("mid_attn", _AttnDesc), ("mid_res2", _ResnetDesc),
                ("ups", ctypes.POINTER(_UpDesc)), ("n_ups", _I), ("norm_out", _NormDesc),
                ("conv_out", _ConvDesc)]


DECODE_PROFILE = 1
DECODE_NO_FUSION = 2
DECODE_FUSE_NORM = 4
DECODE_SUBPIXEL_UP = 8
DECODE_PROFILE_FULLRES = 16
STAGE_NAMES = {0: "conv3x3", 1: "conv1x1", 2: "norm", 3: "cast", 4: "attention", 5: "layout", 6: "copy"}


class StageRecord(ctypes.Structure):
    _fields_ = [("kind", _I), ("launches", _I), ("h", _I), ("w", _I), ("cin", _I), ("cout", _I),
                ("flops", ctypes.c_double), ("bytes", ctypes.c_double), ("ms", ctypes.c_float)]


class DecodeOpts(ctypes.Structure):
    _fields_ = [("band_from", _I), ("nbands", _I), ("band_rows", _I), ("guard_log2", _I),
                ("flags", ctypes.c_uint)]


class Decoder:
    """A decoder handle built from a host description.

    ``desc`` is any object with the attributes of ``vae_decoder_desc``
    (family "gn"/"rms", conv_in, mid_res1, mid_attn, mid_res2, ups,
    norm_out, conv_out, post_quant, latent_channels, scaling, shift, groups,
    eps, dupup), whose convs carry ``w`` (f16 OIHW numpy) and ``b`` (f32) and
    whose norms carry ``gamma`` / ``beta``. The library copies the weights to
    the current device in its own layouts.
    """

    def __init__(self, desc):
        self._keep = []
        d = _DecoderDesc()
        d.family = FAMILY_GN if desc.family == "gn" else FAMILY_RMS
        d.latent_channels = int(desc.latent_channels)
        d.scaling = float(getattr(desc, "scaling", 1.0))
        d.shift = float(getattr(desc, "shift", 0.0))
        d.groups = int(getattr(desc, "groups", 32))
        d.eps = float(getattr(desc, "eps", 1e-6))
        d.dupup = int(bool(getattr(desc, "dupup", False)))
        d.post_quant = self._conv(getattr(desc, "post_quant", None))
        d.conv_in = self._conv(desc.conv_in)
        d.mid_res1 = self._resnet(desc.mid_res1)
        a = desc.mid_attn
        d.mid_attn = _AttnDesc(self._norm(a.norm), self._conv(a.q), self._conv(a.k), self._conv(a.v),
                               self._conv(a.o))
        d.mid_res2 = self._resnet(desc.mid_res2)
        ups = (_UpDesc * len(desc.ups))()
        for i, u in enumerate(desc.ups):
            res = (_ResnetDesc * max(1, len(u.resnets)))()
            for j, r in enumerate(u.resnets):
                res[j] = self._resnet(r)
            self._keep.append(res)
            ups[i] = _UpDesc(ctypes.cast(res, ctypes.POINTER(_ResnetDesc)), len(u.resnets), self._conv(u.up),
                             int(u.in_dim), int(u.out_dim), int(getattr(u, "ft", 1)))
        self._keep.append(ups)
        d.ups = ctypes.cast(ups, ctypes.POINTER(_UpDesc))
        d.n_ups = len(desc.ups)
        d.norm_out = self._norm(desc.norm_out)
        d.conv_out = self._conv(desc.conv_out)
        self.nch = int(desc.conv_out.w.shape[0])
        self.latent_channels = d.latent_channels
        self.n_up = sum(1 for u in desc.ups if u.up is not None)
        h = _P()
        _check(lib().vae_decoder_create(ctypes.byref(d), ctypes.byref(h)))
        self._h = h
        self._keep = None  # the library copied everything

    def _arr(self, a, dtype):
        if a is None:
            return None
        a = np.ascontiguousarray(np.asarray(a, dtype=dtype))
        self._keep.append(a)
        return a.ctypes.data

    def _conv(self, c):
        if c is None:
            return _ConvDesc(None, None, 0, 0, 0)
        w = np.asarray(c.w, dtype=np.float16)
        return _ConvDesc(self._arr(w.view(np.uint16), np.uint16), self._arr(c.b, np.float32),
                         int(w.shape[0]), int(w.shape[1]), int(w.shape[2]))

    def _norm(self, n):
        return _NormDesc(self._arr(n.gamma, np.float32), self._arr(getattr(n, "beta", None), np.float32))

    def _resnet(self, r):
        return _ResnetDesc(self._norm(r.norm1), self._conv(r.conv1), self._norm(r.norm2), self._conv(r.conv2),
                           self._conv(r.shortcut))

    @staticmethod
    def opts(band_from: int = 0, nbands: int = 0, band_rows: int = 0, guard_log2: int = 8,
             profile=False, fuse: Optional[bool] = None, subpixel: bool = False) -> DecodeOpts:
        """profile: False, True (events around every stage) or "fullres" (only around
        the full-resolution ResNet convs). fuse: None (the library's default:
        separate norms), True (a ResNet's second RMS_norm fused into its first
        conv wherever one CTA holds a pixel's channels), False (separate norms)."""
        prof = (DECODE_PROFILE if profile else 0) | (DECODE_PROFILE_FULLRES if profile == "fullres" else 0)
        fz = 0 if fuse is None else (DECODE_FUSE_NORM if fuse else DECODE_NO_FUSION)
        return DecodeOpts(band_from, nbands, band_rows, guard_log2,
                          prof | fz | (DECODE_SUBPIXEL_UP if subpixel else 0))

    def profile(self):
        """Stage records of the most recent profiled decode, as dicts (synchronises)."""
        n = _I()
        _check(lib().vae_decode_profile(self._h, None, 0, ctypes.byref(n)))
        arr = (StageRecord * max(1, n.value))()
        _check(lib().vae_decode_profile(self._h, ctypes.cast(arr, _P), n.value, ctypes.byref(n)))
        return [{"kind": STAGE_NAMES.get(r.kind, r.kind), "launches": r.launches, "h": r.h, "w": r.w,
                 "cin": r.cin, "cout": r.cout, "flops": r.flops, "bytes": r.bytes, "ms": r.ms}
                for r in arr[:n.value]]

    def workspace_bytes(self, h0: int, w0: int, opts: Optional[DecodeOpts] = None) -> int:
        n = _SZ()
        _check(lib().vae_decode_workspace(self._h, h0, w0, ctypes.byref(opts) if opts else None,
                                          ctypes.byref(n)))
        return int(n.value)

    def graph(self, z, out, workspace, opts: Optional[DecodeOpts] = None, stream=None) -> "DecodeGraph":
        """Capture the decode of ``z`` into ``out`` (both CUDA, fixed from now on) as a
        CUDA graph; ``DecodeGraph.launch()`` replays it. Runs one eager decode first."""
        import torch
        _need(z, torch.float32, "z", 3)
        _need(out, torch.float32, "out", 3)
        zc, h0, w0 = z.shape
        g = _P()
        _check(lib().vae_decode_graph_create(self._h, _ptr(z), h0, w0, _ptr(out), ctypes.byref(opts) if opts else None,
                                             _ptr(workspace), workspace.numel(), _stream(stream), ctypes.byref(g)))
        return DecodeGraph(g, (z, out, workspace))

    def decode(self, z, out=None, opts: Optional[DecodeOpts] = None, workspace=None, stream=None):
        """z f32 [zc][h0][w0] (CUDA) -> out f32 [nch][h0<<ups][w0<<ups] (CUDA)."""
        import torch
        _need(z, torch.float32, "z", 3)
        zc, h0, w0 = z.shape
        H, W = h0 << self.n_up, w0 << self.n_up
        if out is None:
            out = torch.empty((self.nch, H, W), dtype=torch.float32, device=z.device)
        _need(out, torch.float32, "out", 3)
        if workspace is None:
            workspace = torch.empty(max(self.workspace_bytes(h0, w0, opts), 16), dtype=torch.uint8,
                                    device=z.device)
        _check(lib().vae_decode(self._h, _ptr(z), h0, w0, _ptr(out), ctypes.byref(opts) if opts else None,
                                _ptr(workspace), workspace.numel(), _stream(stream)))
        return out

    def decode_host(self, z_host: np.ndarray, out_host: np.ndarray, workspace, opts=None, stream=None):
        """End-to-end call with host (ideally pinned) buffers; synchronises the stream."""
        zc, h0, w0 = z_host.shape
        _check(lib().vae_decode_host(self._h, z_host.ctypes.data if isinstance(z_host, np.ndarray)
                                     else z_host.data_ptr(), h0, w0,
                                     out_host.ctypes.data if isinstance(out_host, np.ndarray)
                                     else out_host.data_ptr(),
                                     ctypes.byref(opts) if opts else None, _ptr(workspace), workspace.numel(),
                                     _stream(stream)))
        return out_host

    def close(self):
        if getattr(self, "_h", None):
            lib().vae_decoder_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class DecodeGraph:
    """A captured decode (see ``Decoder.graph``); keeps its buffers alive."""

    def __init__(self, handle, keep):
        self._g = handle
        self._keep = keep

    def launch(self, stream=None):
        _check(lib().vae_decode_graph_launch(self._g, _stream(stream)))

    def __del__(self):
        if getattr(self, "_g", None) is not None and _LIB is not None:
            lib().vae_decode_graph_destroy(self._g)
            self._g = None
