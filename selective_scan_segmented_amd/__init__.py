"""selective_scan_segmented_amd -- SF-Mamba's folded, segmented selective scan on MI355X.

The compute lives in ``libsfm.so`` (hand-written HIP kernels for gfx950 behind
the C ABI declared in ``include/sfm.h``).  This module is the thin Python
binding: it checks tensors, passes their device pointers and the current HIP
stream, and turns non-zero status codes into exceptions.  Every step runs in
the library's kernels; there is no fallback -- if ``libsfm.so`` is missing the
first call raises.

`stream` (a torch.cuda.Stream; None: the current one) is where a call's kernels run.  What the call allocates comes
from that stream's memory pool.  What the caller passes has to be ready there, and to live until the call's kernels
are through; what it returns has to be waited for as any work of that stream.

Functions keep the C names:
  sfm_selective_scan_fwd, sfm_dwconv1d_fold, sfm_aux_pad_swap, sfm_pick_b1,
  sfm_gated_delta_fwd, sfm_gated_delta_bwd, sfm_gated_delta_step, sfm_group_norm_fwd, sfm_group_norm_bwd
"""
from __future__ import annotations

import ctypes
import os

__all__ = ["sfm_selective_scan_fwd", "sfm_selective_scan_fwd_ex", "sfm_selective_scan_fwd_ws",
           "sfm_selective_scan_fwd_ws_size", "sfm_selective_scan_bwd",
           "sfm_selective_scan_bwd_workspace_size", "sfm_dwconv1d_fold", "sfm_aux_pad_swap", "sfm_aux_pad_bwd",
           "sfm_aux_pad_bwd_ex",
           "sfm_gated_delta_fwd", "sfm_gated_delta_fwd_ws_size", "sfm_gated_delta_bwd",
           "sfm_gated_delta_bwd_ws_size", "sfm_gated_delta_step", "sfm_group_norm_fwd",
           "sfm_group_norm_bwd", "sfm_group_norm_ws_size",
           "sfm_pick_b1", "sfm_scan_plan_string", "sfm_version", "library_path", "load_library", "SFMError"]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIBPATH = os.path.join(_HERE, "libsfm.so")
_lib = None

SFM_F32, SFM_BF16 = 0, 1
SFM_AUX_PAD, SFM_AUX_SWAP = 0, 1
_ACT = {None: 0, "none": 0, "silu": 1, 0: 0, 1: 1}


class SFMError(RuntimeError):
    pass


def library_path() -> str:
    return _LIBPATH


def load_library():
    """Load libsfm.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIBPATH):
        raise ImportError(f"libsfm.so not found at {_LIBPATH}; build it with "
                          "`python -m selective_scan_segmented_amd.build`")
    lib = ctypes.CDLL(_LIBPATH)
    vp, i64, ci, fp = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_void_p
    lib.sfm_selective_scan_fwd.argtypes = [vp, vp, fp, vp, vp, fp, fp, ci, fp, fp, ci, ci, ci, vp,
                                           i64, i64, i64, i64, i64, ci, vp]
    lib.sfm_selective_scan_fwd_ex.argtypes = [vp, vp, fp, vp, vp, fp, fp, ci, fp, fp, ci, ci, ci, vp,
                                              i64, i64, i64, i64, i64, ci, ci, vp]
    lib.sfm_selective_scan_fwd_ws.argtypes = [vp, vp, fp, vp, vp, fp, fp, ci, fp, fp, ci, ci, ci, vp,
                                              i64, i64, i64, i64, i64, ci, ci, vp, i64, vp]
    lib.sfm_selective_scan_fwd_noalloc.argtypes = [vp, vp, fp, vp, vp, fp, fp, ci, fp, fp, ci, ci, ci, vp,
                                                   i64, i64, i64, i64, i64, ci, ci, vp]
    lib.sfm_selective_scan_fwd_ws_size.argtypes = [i64, i64, i64, i64, i64, ci, ci, ci,
                                                   ctypes.POINTER(ctypes.c_int64)]
    lib.sfm_dwconv1d_fold.argtypes = [vp, fp, fp, vp, i64, i64, i64, i64, ci, ci, ci, ci, vp]
    lib.sfm_selective_scan_bwd.argtypes = [vp, vp, fp, vp, vp, fp, fp, ci, fp, fp, ci, ci, ci, vp,
                                           vp, vp, fp, fp, fp, fp, fp, fp, fp,
                                           i64, i64, i64, i64, i64, ci, ci, vp, i64, vp]
    lib.sfm_selective_scan_bwd_workspace_size.argtypes = [i64, i64, i64, i64, i64, ci, ci, ci,
                                                          ctypes.POINTER(ctypes.c_int64)]
    lib.sfm_aux_pad_bwd.argtypes = [vp, vp, i64, i64, i64, ci, vp]
    lib.sfm_aux_pad_bwd_ex.argtypes = [vp, vp, i64, i64, i64, ci, ci, vp]
    lib.sfm_aux_pad_swap.argtypes = [vp, vp, i64, i64, i64, ci, ci, vp]
    lib.sfm_pick_b1.argtypes = [i64, i64, i64, i64, ctypes.POINTER(ctypes.c_int64)]
    lib.sfm_scan_plan_string.argtypes = [i64, i64, i64, i64, i64, ci, ci, ci, ctypes.c_char_p, i64]
    f32 = ctypes.c_float
    pi64 = ctypes.POINTER(ctypes.c_int64)
    lib.sfm_gated_delta_fwd.argtypes = [vp] * 9 + [i64] * 10 + [f32, ci, ci, vp, i64, vp]
    lib.sfm_gated_delta_fwd_ws_size.argtypes = [i64] * 6 + [ci, ci, pi64]
    lib.sfm_gated_delta_step.argtypes = [vp] * 8 + [i64] * 9 + [f32, ci, ci, vp]
    lib.sfm_group_norm_fwd.argtypes = [vp] * 6 + [i64] * 4 + [f32, ci, ci, vp, i64, vp]
    lib.sfm_group_norm_bwd.argtypes = [vp] * 9 + [i64] * 4 + [ci, ci, vp, i64, vp]
    lib.sfm_group_norm_fwd_ws_size.argtypes = [i64] * 4 + [ci, pi64]
    lib.sfm_group_norm_bwd_ws_size.argtypes = [i64] * 4 + [ci, ci, pi64]
    lib.sfm_gated_delta_bwd.argtypes = [vp] * 15 + [i64] * 10 + [f32, ci, ci, vp, i64, vp]
    lib.sfm_gated_delta_bwd_ws_size.argtypes = [i64] * 7 + [ci, ci, pi64]
    for f in ("sfm_gated_delta_fwd", "sfm_gated_delta_fwd_ws_size", "sfm_gated_delta_step", "sfm_gated_delta_bwd",
              "sfm_gated_delta_bwd_ws_size", "sfm_group_norm_fwd",
              "sfm_group_norm_bwd", "sfm_group_norm_fwd_ws_size", "sfm_group_norm_bwd_ws_size"):
        getattr(lib, f).restype = ctypes.c_int
    for f in ("sfm_selective_scan_fwd", "sfm_selective_scan_fwd_ex", "sfm_selective_scan_fwd_ws",
              "sfm_selective_scan_fwd_ws_size", "sfm_dwconv1d_fold", "sfm_aux_pad_swap",
              "sfm_pick_b1", "sfm_version", "sfm_scan_plan_string", "sfm_selective_scan_bwd",
              "sfm_selective_scan_bwd_workspace_size", "sfm_aux_pad_bwd", "sfm_aux_pad_bwd_ex"):
        getattr(lib, f).restype = ctypes.c_int
    lib.sfm_status_string.argtypes = [ctypes.c_int]
    lib.sfm_status_string.restype = ctypes.c_char_p
    lib.sfm_last_error.restype = ctypes.c_char_p
    _lib = lib
    return lib


def _check(rc: int, name: str):
    if rc != 0:
        lib = load_library()
        raise SFMError(f"{name}: {lib.sfm_status_string(rc).decode()} ({rc}): {lib.sfm_last_error().decode()}")


def sfm_version() -> int:
    return load_library().sfm_version()


_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:  # (an import statement costs a call of its own time: 0.2 us)
        import torch
        _torch_module = torch
    return _torch_module


def _io_code(t) -> int:
    torch = _torch()
    if t.dtype == torch.float32:
        return SFM_F32
    if t.dtype == torch.bfloat16:
        return SFM_BF16
    raise TypeError(f"io tensors must be float32 or bfloat16, got {t.dtype}")


def _dev(t, name, dtype=None, shape=None):
    torch = _torch()
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise TypeError(f"{name} must be a GPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    if stream is not None:
        return stream.cuda_stream
    torch = _torch()
    try:  # the current stream's handle without a Stream object around it (a third of a small call's host time)
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    except AttributeError:
        return torch.cuda.current_stream().cuda_stream


def _new(shape, dtype, device, stream):
    """A tensor for a call on `stream` (None: the current one).

    It comes from that stream's own pool: a block of another pool may still be read or written there by kernels that
    `stream` does not wait for, such as an earlier call's whose workspace it was.  The caller has it on the current
    stream, so its memory is not handed out again before that stream is past its free either."""
    torch = _torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(device))
    return t


def _scratch(size, device, stream):
    """A workspace for a call on `stream`: from its pool, and nothing that the caller has on another one."""
    torch = _torch()
    if stream is None:
        return torch.empty(size, dtype=torch.uint8, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(size, dtype=torch.uint8, device=device)


def _new_like(t, stream):
    """_new of a contiguous tensor's shape and type, in less host time."""
    return _torch().empty_like(t) if stream is None else _new(t.shape, t.dtype, t.device, stream)


SFM_FUSE_PAD, SFM_FUSE_SWAP, SFM_LAYOUT_BLD = 1, 2, 4
SFM_NOALLOC_SCRATCH_BYTES = 32 << 20  # static scratch of sfm_selective_scan_fwd_noalloc (include/sfm.h)


def sfm_selective_scan_fwd(u, delta, A, Bm, Cm, Dskip=None, delta_bias=None, delta_softplus=True,
                           conv_w=None, conv_b=None, conv_pad_left=1, conv_act=None, y=None, B2=1,
                           stream=None):
    """Folded, segmented selective scan (see include/sfm.h).

    u, delta: [B, D, L]; A: [D, N] float32; Bm, Cm: [B, N, L]; io dtype float32 or bfloat16.
    With conv_w ([D, K] float32) ``u`` is the conv input and the boundary-masked conv is fused.
    B2 samples form one folded row (B1 = B / B2).  Returns y [B, D, L] (allocated if None).
    """
    return sfm_selective_scan_fwd_ex(u, delta, A, Bm, Cm, Dskip, delta_bias, delta_softplus, conv_w, conv_b,
                                     conv_pad_left, conv_act, y, B2, 0, stream)


def sfm_selective_scan_fwd_ex(u, delta, A, Bm, Cm, Dskip=None, delta_bias=None, delta_softplus=True,
                              conv_w=None, conv_b=None, conv_pad_left=1, conv_act=None, y=None, B2=1,
                              flags=0, stream=None):
    """sfm_selective_scan_fwd with the aux pad (flags & SFM_FUSE_PAD: u is the unpadded
    [B, D, L-2] stage input) and/or the aux swap of y (flags & SFM_FUSE_SWAP) fused in.
    flags & SFM_LAYOUT_BLD: channel-last tensors, u/delta/y [B, L, D] (u [B, L-2, D] with
    the pad), Bm/Cm [B, L, N]."""
    return _fwd_ex(u, delta, A, Bm, Cm, Dskip, delta_bias, delta_softplus, conv_w, conv_b, conv_pad_left,
                   conv_act, y, B2, flags, stream, False)


def _fwd_ex(u, delta, A, Bm, Cm, Dskip, delta_bias, delta_softplus, conv_w, conv_b, conv_pad_left, conv_act, y,
            B2, flags, stream, workspace):
    """Argument marshalling of the fused forward entry points (workspace False:
    sfm_selective_scan_fwd_ex; "noalloc": sfm_selective_scan_fwd_noalloc; else
    sfm_selective_scan_fwd_ws)."""
    torch = _torch()
    io = _io_code(u)
    cl = bool(flags & SFM_LAYOUT_BLD)
    if cl:
        B, XL, D = u.shape
    else:
        B, D, XL = u.shape
    L = XL + 2 if flags & SFM_FUSE_PAD else XL
    N = A.shape[1]
    if B % B2:
        raise ValueError(f"B2={B2} must divide B={B}")
    tl = (lambda a, b_: (B, b_, a)) if cl else (lambda a, b_: (B, a, b_))  # [B, a, b] in this layout
    _dev(u, "u")
    _dev(delta, "delta", u.dtype, tl(D, L))
    _dev(A, "A", torch.float32, (D, N))
    _dev(Bm, "Bm", u.dtype, tl(N, L))
    _dev(Cm, "Cm", u.dtype, tl(N, L))
    _dev(Dskip, "Dskip", torch.float32, (D,))
    _dev(delta_bias, "delta_bias", torch.float32, (D,))
    K = 0
    if conv_w is not None:
        _dev(conv_w, "conv_w", torch.float32)
        if conv_w.dim() != 2 or conv_w.shape[0] != D:
            raise ValueError("conv_w must be [D, K]")
        K = conv_w.shape[1]
        _dev(conv_b, "conv_b", torch.float32, (D,))
    if y is None:
        y = _new(tl(D, L), u.dtype, u.device, stream)
    _dev(y, "y", u.dtype, tl(D, L))
    args = (_ptr(u), _ptr(delta), _ptr(A), _ptr(Bm), _ptr(Cm), _ptr(Dskip), _ptr(delta_bias),
            int(bool(delta_softplus)), _ptr(conv_w), _ptr(conv_b), K, int(conv_pad_left), _ACT[conv_act], _ptr(y),
            B // B2, B2, D, N, L, io, int(flags))
    if workspace is False:
        rc = load_library().sfm_selective_scan_fwd_ex(*args, _stream(stream))
    elif isinstance(workspace, str) and workspace == "noalloc":
        rc = load_library().sfm_selective_scan_fwd_noalloc(*args, _stream(stream))
    else:
        need = sfm_selective_scan_fwd_ws_size(B // B2, B2, D, N, L, K, "bf16" if io == SFM_BF16 else "f32",
                                              int(flags))
        if workspace is None:
            workspace = _scratch(max(need, 16), u.device, stream)
        _dev(workspace, "workspace")
        rc = load_library().sfm_selective_scan_fwd_ws(*args, _ptr(workspace),
                                                      workspace.numel() * workspace.element_size(),
                                                      _stream(stream))
    _check(rc, "sfm_selective_scan_fwd")
    return y


def sfm_selective_scan_fwd_ws(u, delta, A, Bm, Cm, Dskip=None, delta_bias=None, delta_softplus=True,
                              conv_w=None, conv_b=None, conv_pad_left=1, conv_act=None, y=None, B2=1,
                              flags=0, workspace=None, stream=None):
    """sfm_selective_scan_fwd_ex with a device workspace (a uint8 GPU tensor of at least
    sfm_selective_scan_fwd_ws_size() bytes; allocated here when None): rows too long
    for the in-LDS carries are split along L across the whole GPU."""
    return _fwd_ex(u, delta, A, Bm, Cm, Dskip, delta_bias, delta_softplus, conv_w, conv_b, conv_pad_left,
                   conv_act, y, B2, flags, stream, workspace)


def sfm_selective_scan_fwd_noalloc(u, delta, A, Bm, Cm, Dskip=None, delta_bias=None, delta_softplus=True,
                                   conv_w=None, conv_b=None, conv_pad_left=1, conv_act=None, y=None, B2=1,
                                   flags=0, stream=None):
    """sfm_selective_scan_fwd_ws without a workspace argument: the library's static
    per-GPU scratch array stands in for it (see include/sfm.h for its limit).  ``y``
    must be passed by callers that cannot allocate (else it is allocated here)."""
    return _fwd_ex(u, delta, A, Bm, Cm, Dskip, delta_bias, delta_softplus, conv_w, conv_b, conv_pad_left,
                   conv_act, y, B2, flags, stream, "noalloc")


def sfm_selective_scan_fwd_ws_size(B1: int, B2: int, D: int, N: int, L: int, conv_k: int = 4,
                                   io: str = "bf16", flags: int = 0) -> int:
    """Workspace bytes sfm_selective_scan_fwd_ws needs (host only; 0: the regular forward runs)."""
    out = ctypes.c_int64(0)
    _check(load_library().sfm_selective_scan_fwd_ws_size(B1, B2, D, N, L, conv_k,
                                                         SFM_BF16 if io == "bf16" else SFM_F32, flags,
                                                         ctypes.byref(out)),
           "sfm_selective_scan_fwd_ws_size")
    return int(out.value)


def sfm_selective_scan_bwd_workspace_size(B1: int, B2: int, D: int, N: int, L: int, conv_k: int = 4,
                                          io: str = "bf16", flags: int = 0) -> int:
    """Workspace bytes sfm_selective_scan_bwd needs (host only)."""
    out = ctypes.c_int64(0)
    _check(load_library().sfm_selective_scan_bwd_workspace_size(B1, B2, D, N, L, conv_k,
                                                                SFM_BF16 if io == "bf16" else SFM_F32, flags,
                                                                ctypes.byref(out)),
           "sfm_selective_scan_bwd_workspace_size")
    return int(out.value)


def sfm_selective_scan_bwd(u, delta, A, Bm, Cm, dy, Dskip=None, delta_bias=None, delta_softplus=True,
                           conv_w=None, conv_b=None, conv_pad_left=1, conv_act=None, B2=1, flags=0,
                           workspace=None, grads=None, stream=None):
    """Gradients of sfm_selective_scan_fwd_ex for upstream dy (see include/sfm.h).

    Returns a dict: du (padded layout [B, D, L], io), ddelta (io), dA, dBm, dCm,
    dDskip, ddelta_bias, dconv_w, dconv_b (float32).  `grads` may hold
    preallocated tensors under those names; `workspace` a uint8 GPU tensor of at
    least sfm_selective_scan_bwd_workspace_size() bytes.  flags & SFM_LAYOUT_BLD:
    channel-last tensors ([B, L, D] and [B, L, N], gradients likewise)."""
    torch = _torch()
    io = _io_code(u)
    cl = bool(flags & SFM_LAYOUT_BLD)
    if cl:
        B, XL, D = u.shape
    else:
        B, D, XL = u.shape
    L = XL + 2 if flags & SFM_FUSE_PAD else XL
    N = A.shape[1]
    if B % B2:
        raise ValueError(f"B2={B2} must divide B={B}")
    tl = (lambda a, b_: (B, b_, a)) if cl else (lambda a, b_: (B, a, b_))  # [B, a, b] in this layout
    _dev(u, "u")
    for t, name, shape in ((delta, "delta", tl(D, L)), (Bm, "Bm", tl(N, L)), (Cm, "Cm", tl(N, L)),
                           (dy, "dy", tl(D, L))):
        _dev(t, name, u.dtype, shape)
    _dev(A, "A", torch.float32, (D, N))
    _dev(Dskip, "Dskip", torch.float32, (D,))
    _dev(delta_bias, "delta_bias", torch.float32, (D,))
    K = 0
    if conv_w is not None:
        _dev(conv_w, "conv_w", torch.float32)
        if conv_w.dim() != 2 or conv_w.shape[0] != D:
            raise ValueError("conv_w must be [D, K]")
        K = conv_w.shape[1]
        _dev(conv_b, "conv_b", torch.float32, (D,))
    g = dict(grads or {})
    f32 = dict(dtype=torch.float32, device=u.device)
    shapes = dict(du=(tl(D, L), u.dtype), ddelta=(tl(D, L), u.dtype), dA=((D, N), torch.float32),
                  dBm=(tl(N, L), torch.float32), dCm=(tl(N, L), torch.float32))
    if Dskip is not None:
        shapes["dDskip"] = ((D,), torch.float32)
    if delta_bias is not None:
        shapes["ddelta_bias"] = ((D,), torch.float32)
    if conv_w is not None:
        shapes["dconv_w"] = ((D, K), torch.float32)
        if conv_b is not None:
            shapes["dconv_b"] = ((D,), torch.float32)
    for k, (shape, dt) in shapes.items():
        if g.get(k) is None:
            g[k] = _new(shape, dt, u.device, stream)
        _dev(g[k], k, dt, shape)
    need = sfm_selective_scan_bwd_workspace_size(B // B2, B2, D, N, L, K, "bf16" if io == SFM_BF16 else "f32",
                                                 flags)
    if workspace is None:
        workspace = _scratch(max(need, 16), u.device, stream)
    _dev(workspace, "workspace")
    rc = load_library().sfm_selective_scan_bwd(
        _ptr(u), _ptr(delta), _ptr(A), _ptr(Bm), _ptr(Cm), _ptr(Dskip), _ptr(delta_bias), int(bool(delta_softplus)),
        _ptr(conv_w), _ptr(conv_b), K, int(conv_pad_left), _ACT[conv_act], _ptr(dy),
        _ptr(g["du"]), _ptr(g["ddelta"]), _ptr(g["dA"]), _ptr(g["dBm"]), _ptr(g["dCm"]), _ptr(g.get("dDskip")),
        _ptr(g.get("ddelta_bias")), _ptr(g.get("dconv_w")), _ptr(g.get("dconv_b")),
        B // B2, B2, D, N, L, io, int(flags), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _stream(stream))
    _check(rc, "sfm_selective_scan_bwd")
    return g


def sfm_aux_pad_bwd(gpad, gx=None, stream=None):
    """Gradient of the aux pad: gpad [B, D, T+2] -> gx [B, D, T]."""
    return sfm_aux_pad_bwd_ex(gpad, gx, 0, stream)


def sfm_aux_pad_bwd_ex(gpad, gx=None, flags=0, stream=None):
    """Gradient of the aux pad; flags & SFM_LAYOUT_BLD: gpad [B, T+2, D] -> gx [B, T, D]."""
    io = _io_code(gpad)
    cl = bool(flags & SFM_LAYOUT_BLD)
    if cl:
        B, L, D = gpad.shape
        shape = (B, L - 2, D)
    else:
        B, D, L = gpad.shape
        shape = (B, D, L - 2)
    _dev(gpad, "gpad")
    if gx is None:
        gx = _new(shape, gpad.dtype, gpad.device, stream)
    _dev(gx, "gx", gpad.dtype, shape)
    _check(load_library().sfm_aux_pad_bwd_ex(_ptr(gpad), _ptr(gx), B, D, L - 2, io, int(flags), _stream(stream)),
           "sfm_aux_pad_bwd")
    return gx


def sfm_dwconv1d_fold(x, w, bias=None, pad_left=1, act=None, out=None, B2=1, stream=None):
    """Boundary-masked depthwise conv1d over folded rows: x [B, D, L], w [D, K] float32."""
    torch = _torch()
    io = _io_code(x)
    B, D, L = x.shape
    if B % B2:
        raise ValueError(f"B2={B2} must divide B={B}")
    _dev(x, "x")
    _dev(w, "w", torch.float32)
    if w.dim() != 2 or w.shape[0] != D:
        raise ValueError("w must be [D, K]")
    _dev(bias, "bias", torch.float32, (D,))
    if out is None:
        out = _new_like(x, stream)
    _dev(out, "out", x.dtype, (B, D, L))
    rc = load_library().sfm_dwconv1d_fold(_ptr(x), _ptr(w), _ptr(bias), _ptr(out), B // B2, B2, D, L, w.shape[1],
                                          int(pad_left), _ACT[act], io, _stream(stream))
    _check(rc, "sfm_dwconv1d_fold")
    return out


def sfm_aux_pad_swap(inp, out=None, mode="pad", stream=None):
    """mode 'pad': [B, D, T] -> [B, D, T+2] with mean-initialised ends;
    mode 'swap': [B, D, L] -> ends exchanged (in place when ``out is inp``)."""
    io = _io_code(inp)
    B, D, n = inp.shape
    _dev(inp, "in")
    if mode == "pad":
        T, code = n, SFM_AUX_PAD
        if out is None:
            out = _new((B, D, T + 2), inp.dtype, inp.device, stream)
        _dev(out, "out", inp.dtype, (B, D, T + 2))
    elif mode == "swap":
        T, code = n - 2, SFM_AUX_SWAP
        if out is None:
            out = _new_like(inp, stream)
        _dev(out, "out", inp.dtype, (B, D, n))
    else:
        raise ValueError(f"mode must be 'pad' or 'swap', got {mode!r}")
    rc = load_library().sfm_aux_pad_swap(_ptr(inp), _ptr(out), B, D, T, code, io, _stream(stream))
    _check(rc, "sfm_aux_pad_swap")
    return out


def sfm_scan_plan_string(B1: int, B2: int, D: int, N: int, L: int, conv_k: int = 4, io: str = "bf16",
                         flags: int = 0) -> str:
    """The launch plan sfm_selective_scan_fwd(_ex) would use for these sizes (host only)."""
    buf = ctypes.create_string_buffer(256)
    _check(load_library().sfm_scan_plan_string(B1, B2, D, N, L, conv_k, SFM_BF16 if io == "bf16" else SFM_F32,
                                               flags, buf, 256), "sfm_scan_plan_string")
    return buf.value.decode()


def sfm_pick_b1(B: int, L: int, D: int, N: int) -> int:
    """Adaptive B1 from the offline table (host only); B2 = B // result."""
    out = ctypes.c_int64(0)
    _check(load_library().sfm_pick_b1(B, L, D, N, ctypes.byref(out)), "sfm_pick_b1")
    return int(out.value)


# ---------------------------------------------------------------- the gated delta rule
def _want(t, name, dtype, shape):
    """_dev for the usual case in one look: a contiguous GPU tensor of this type and shape (or None)."""
    if t is not None and not (t.is_cuda and t.dtype is dtype and t.shape == shape and t.is_contiguous()):
        _dev(t, name, dtype, shape)


SFM_DELTA_L2NORM = 1


def _tokens(t, name, heads, width, dtype, lead):
    """Checks a [*lead, heads, width] tensor whose heads are contiguous and whose tokens
    are evenly strided (a slice of a wider projection is fine); returns the token stride."""
    shape = lead + (heads, width)
    if t.shape == shape and t.dtype is dtype and t.is_cuda and t.is_contiguous():
        return heads * width
    if not t.is_cuda:
        raise TypeError(f"{name} must be a GPU tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    st = t.stride()
    single = len(lead) == 2 and lead[1] == 1  # rows of one token: the tokens are the rows'
    ld = st[0] if single else st[-3]
    if (width > 1 and st[-1] != 1) or (heads > 1 and st[-2] != width) or \
            (len(lead) == 2 and not single and lead[0] > 1 and st[0] != lead[1] * ld) or \
            (ld < heads * width and lead.numel() > 1):
        raise ValueError(f"{name}: heads must be contiguous and tokens evenly strided, got strides {st}")
    return max(ld, heads * width)


def _delta_args(q, k, v, g, beta, packed, form="[B, L, heads, size]"):
    """Checks shared by the gated delta rule's functions; returns the sizes and strides."""
    io = _io_code(q)
    shape, wide = q.shape, v.shape
    dims = form.count(",") + 1
    if len(shape) != dims or len(wide) != dims:
        raise ValueError(f"q, k and v must be {form}, got q {tuple(shape)} and v {tuple(wide)}")
    lead, Hk, dk, H, dv = shape[:-2], shape[-2], shape[-1], wide[-2], wide[-1]
    if packed and lead[0] != 1:
        raise ValueError("packed rows (offsets) are one batch entry: [1, tokens, heads, size]")
    dtype = q.dtype
    ldq = _tokens(q, "q", Hk, dk, dtype, lead)
    ldk = _tokens(k, "k", Hk, dk, dtype, lead)
    ldv = _tokens(v, "v", H, dv, dtype, lead)
    heads = lead + (H,)
    _want(g, "g", dtype, heads)
    _want(beta, "beta", dtype, heads)
    return io, lead, Hk, H, dk, dv, ldq, ldk, ldv


def _rows(lead, offsets, max_len):
    if offsets is None:
        return lead[0], lead[1], lead[0] * lead[1]
    torch = _torch()
    _dev(offsets, "offsets", torch.int32)
    if offsets.dim() != 1 or offsets.numel() < 2:
        raise ValueError("offsets must be int32 [rows + 1]")
    L = lead[1] if max_len is None else int(max_len)
    if L == 0 and lead[1] == 0:
        L = 1  # (rows that are all empty: the longest's bound, which has to be positive)
    return offsets.numel() - 1, L, lead[1]


def sfm_gated_delta_fwd_ws_size(rows: int, L: int, tokens: int, H: int, dk: int, dv: int, want_state: bool = False,
                                io: str = "bf16") -> int:
    """Workspace bytes sfm_gated_delta_fwd needs (host only)."""
    out = ctypes.c_int64(0)
    _check(load_library().sfm_gated_delta_fwd_ws_size(rows, L, tokens, H, dk, dv, int(bool(want_state)),
                                                      SFM_BF16 if io == "bf16" else SFM_F32, ctypes.byref(out)),
           "sfm_gated_delta_fwd_ws_size")
    return int(out.value)


def sfm_gated_delta_fwd(q, k, v, g, beta, h0=None, offsets=None, max_len=None, scale=None, l2norm=False, o=None,
                        return_state=False, state=None, workspace=None, stream=None):
    """The gated delta rule over whole rows (see include/sfm.h).

    q, k: [B, L, Hk, dk]; v: [B, L, H, dv]; g (log decay), beta: [B, L, H]; float32 or bfloat16.
    h0: [B, H, dk, dv] float32 states before the rows, or None.  offsets (int32 [rows + 1] on the
    GPU): packed rows, tensors [1, tokens, ...]; max_len bounds the longest row (None: unknown, and planned as
    no more than four times the average: give it where one row is far longer).  scale defaults to
    dk ** -0.5; l2norm divides q and k by their length.  Tokens of no row, and those past max_len in
    one, are not written: a new output holds anything there.  Returns o [B, L, H, dv], and with
    return_state the states after the rows.  `state`, if given, takes those in either case (h0
    itself is allowed)."""
    torch = _torch()
    io, lead, Hk, H, dk, dv, ldq, ldk, ldv = _delta_args(q, k, v, g, beta, offsets is not None)
    rows, L, tokens = _rows(lead, offsets, max_len)
    _want(h0, "h0", torch.float32, (rows, H, dk, dv))
    if o is not None:
        _want(o, "o", q.dtype, lead + (H, dv))
    else:
        o = _new_like(v, stream) if v.is_contiguous() else _new(lead + (H, dv), q.dtype, q.device, stream)
    if state is not None:
        _want(state, "state", torch.float32, (rows, H, dk, dv))
    elif return_state:
        state = _new((rows, H, dk, dv), torch.float32, q.device, stream)
    need = 0 if L <= 64 else sfm_gated_delta_fwd_ws_size(rows, L, tokens, H, dk, dv, state is not None, "bf16" if io else "f32")
    if workspace is None and need:
        workspace = _scratch(need, q.device, stream)
    _dev(workspace, "workspace")
    rc = load_library().sfm_gated_delta_fwd(
        _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(h0), _ptr(o), _ptr(state), _ptr(offsets), rows, L,
        tokens, Hk, H, dk, dv, ldq, ldk, ldv, dk ** -0.5 if scale is None else scale, io,
        SFM_DELTA_L2NORM if l2norm else 0, _ptr(workspace),
        0 if workspace is None else workspace.numel() * workspace.element_size(), _stream(stream))
    _check(rc, "sfm_gated_delta_fwd")
    return (o, state) if return_state else o


def sfm_gated_delta_bwd_ws_size(rows: int, L: int, tokens: int, Hk: int, H: int, dk: int, dv: int,
                                want_dh0: bool = False, io: str = "bf16") -> int:
    """Workspace bytes sfm_gated_delta_bwd needs (host only)."""
    out = ctypes.c_int64(0)
    _check(load_library().sfm_gated_delta_bwd_ws_size(rows, L, tokens, Hk, H, dk, dv, int(bool(want_dh0)),
                                                      SFM_BF16 if io == "bf16" else SFM_F32, ctypes.byref(out)),
           "sfm_gated_delta_bwd_ws_size")
    return int(out.value)


def sfm_gated_delta_bwd(q, k, v, g, beta, do, h0=None, dstate=None, offsets=None, max_len=None, scale=None,
                        l2norm=False, grads=None, workspace=None, stream=None):
    """Gradients of sfm_gated_delta_fwd (same arguments) for do, the gradient of o, and dstate, that of the
    states after the rows (float32, None: zero).  Returns a dict with dq, dk, dv, dg, dbeta and, with h0,
    dh0 (float32); `grads` may hold preallocated tensors under those names, dh0 also without h0.
    Tokens that the forward does not write get no gradients: a new tensor holds anything there."""
    torch = _torch()
    io, lead, Hk, H, dk, dv, ldq, ldk, ldv = _delta_args(q, k, v, g, beta, offsets is not None)
    rows, L, tokens = _rows(lead, offsets, max_len)
    _want(h0, "h0", torch.float32, (rows, H, dk, dv))
    _want(dstate, "dstate", torch.float32, (rows, H, dk, dv))
    _want(do, "do", q.dtype, lead + (H, dv))
    out = dict(grads or {})
    for name, like in (("dq", q), ("dk", k), ("dv", v), ("dg", g), ("dbeta", beta), ("dh0", h0)):
        if like is None:  # (dh0 of states that were zero: only where the caller gives a tensor for it)
            _want(out.get(name), name, torch.float32, (rows, H, dk, dv))
        elif out.get(name) is not None:
            _want(out[name], name, like.dtype, like.shape)
        else:
            out[name] = _new_like(like, stream) if like.is_contiguous() else _new(like.shape, like.dtype, q.device, stream)
    need = sfm_gated_delta_bwd_ws_size(rows, L, tokens, Hk, H, dk, dv, out.get("dh0") is not None, "bf16" if io else "f32")
    if workspace is None:
        workspace = _scratch(need, q.device, stream)
    _dev(workspace, "workspace")
    rc = load_library().sfm_gated_delta_bwd(
        _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(h0), _ptr(do), _ptr(dstate), _ptr(out["dq"]),
        _ptr(out["dk"]), _ptr(out["dv"]), _ptr(out["dg"]), _ptr(out["dbeta"]), _ptr(out.get("dh0")), _ptr(offsets),
        rows, L, tokens, Hk, H, dk, dv, ldq, ldk, ldv, dk ** -0.5 if scale is None else scale, io,
        SFM_DELTA_L2NORM if l2norm else 0, _ptr(workspace), workspace.numel() * workspace.element_size(),
        _stream(stream))
    _check(rc, "sfm_gated_delta_bwd")
    return out


def sfm_gated_delta_step(q, k, v, g, beta, state, slots=None, scale=None, l2norm=False, o=None, stream=None):
    """One token of each request: q, k [R, Hk, dk]; v [R, H, dv]; g, beta [R, H]; state [pool, H, dk, dv]
    float32, updated in place; slots int32 [R] (row r's state; outside the pool: padding) or None
    (state r).  Returns o [R, H, dv]."""
    torch = _torch()
    io, lead, Hk, H, dk, dv, ldq, ldk, ldv = _delta_args(q, k, v, g, beta, False, "[R, heads, size]")
    rows = lead[0]
    _dev(state, "state", torch.float32)
    if state.dim() != 4 or state.shape[1:] != (H, dk, dv):
        raise ValueError(f"state must have shape (pool, {H}, {dk}, {dv}), got {tuple(state.shape)}")
    _want(slots, "slots", torch.int32, (rows,))
    if o is not None:
        _want(o, "o", q.dtype, (rows, H, dv))
    else:
        o = _new_like(v, stream) if v.is_contiguous() else _new((rows, H, dv), q.dtype, q.device, stream)
    rc = load_library().sfm_gated_delta_step(
        _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(state), _ptr(slots), _ptr(o), rows, state.shape[0],
        Hk, H, dk, dv, ldq, ldk, ldv, dk ** -0.5 if scale is None else scale, io,
        SFM_DELTA_L2NORM if l2norm else 0, _stream(stream))
    _check(rc, "sfm_gated_delta_step")
    return o


# ---------------------------------------------------------------- group norm, channels last
def sfm_group_norm_ws_size(N: int, L: int, C: int, G: int, io: str = "bf16", backward: bool = False,
                           want_weights: bool = True) -> int:
    """Workspace bytes of sfm_group_norm_fwd, or with `backward` of sfm_group_norm_bwd (host only)."""
    out = ctypes.c_int64(0)
    code = SFM_BF16 if io == "bf16" else SFM_F32
    lib = load_library()
    _check(lib.sfm_group_norm_bwd_ws_size(N, L, C, G, int(bool(want_weights)), code, ctypes.byref(out)) if backward
           else lib.sfm_group_norm_fwd_ws_size(N, L, C, G, code, ctypes.byref(out)), "sfm_group_norm_ws_size")
    return int(out.value)


def _norm_sizes(x):
    """[N, ..., C] -> N, tokens, C."""
    if x.dim() < 2:
        raise ValueError("x must be [N, ..., C]")
    N, C = x.shape[0], x.shape[-1]
    return N, x.numel() // max(1, N * C), C


def sfm_group_norm_fwd(x, num_groups, weight=None, bias=None, eps=1e-5, act=None, y=None, mean=None, rstd=None,
                       workspace=None, stream=None):
    """Group norm of channel-last x [N, ..., C] over num_groups groups of neighbouring channels, then
    act (None or 'silu').  weight, bias: [C] float32 or None.  Returns y and the float32 [N, G]
    mean and rstd that sfm_group_norm_bwd takes."""
    torch = _torch()
    io = _io_code(x)
    N, L, C = _norm_sizes(x)
    _dev(x, "x")
    _want(weight, "weight", torch.float32, (C,))
    _want(bias, "bias", torch.float32, (C,))
    if y is None:
        y = _new_like(x, stream)
    else:
        _want(y, "y", x.dtype, x.shape)
    if mean is None:
        mean = _new((N, num_groups), torch.float32, x.device, stream)
    else:
        _want(mean, "mean", torch.float32, (N, num_groups))
    if rstd is None:
        rstd = _new_like(mean, stream)
    else:
        _want(rstd, "rstd", torch.float32, (N, num_groups))
    need = sfm_group_norm_ws_size(N, L, C, num_groups, "bf16" if io else "f32")
    if workspace is None and need:
        workspace = _scratch(need, x.device, stream)
    _dev(workspace, "workspace")
    rc = load_library().sfm_group_norm_fwd(
        _ptr(x), _ptr(weight), _ptr(bias), _ptr(y), _ptr(mean), _ptr(rstd), N, L, C, num_groups, eps, _ACT[act], io,
        _ptr(workspace), 0 if workspace is None else workspace.numel() * workspace.element_size(), _stream(stream))
    _check(rc, "sfm_group_norm_fwd")
    return y, mean, rstd


def sfm_group_norm_bwd(dy, x, mean, rstd, weight=None, bias=None, act=None, grads=None, workspace=None, stream=None):
    """Gradients of sfm_group_norm_fwd for upstream dy: a dict with dx and, for the weight and bias
    given, dw and db (float32).  `grads` may hold preallocated tensors under those names."""
    torch = _torch()
    io = _io_code(x)
    N, L, C = _norm_sizes(x)
    _dev(x, "x")
    _want(dy, "dy", x.dtype, x.shape)
    _dev(mean, "mean", torch.float32)
    if mean.dim() != 2 or mean.shape[0] != N:
        raise ValueError(f"mean must be [{N}, groups], got {tuple(mean.shape)}")
    G = mean.shape[1]
    _want(rstd, "rstd", torch.float32, (N, G))
    _want(weight, "weight", torch.float32, (C,))
    _want(bias, "bias", torch.float32, (C,))
    out = dict(grads or {})
    for name, like in (("dx", x), ("dw", weight), ("db", bias)):
        if out.get(name) is not None:
            _want(out[name], name, *((x.dtype, x.shape) if name == "dx" else (torch.float32, (C,))))
        elif like is not None:
            out[name] = _new_like(like, stream)
    need = sfm_group_norm_ws_size(N, L, C, G, "bf16" if io else "f32", True,
                                  out.get("dw") is not None or out.get("db") is not None)
    if workspace is None and need:
        workspace = _scratch(need, x.device, stream)
    _dev(workspace, "workspace")
    rc = load_library().sfm_group_norm_bwd(
        _ptr(dy), _ptr(x), _ptr(mean), _ptr(rstd), _ptr(weight), _ptr(bias), _ptr(out["dx"]), _ptr(out.get("dw")),
        _ptr(out.get("db")), N, L, C, G, _ACT[act], io, _ptr(workspace),
        0 if workspace is None else workspace.numel() * workspace.element_size(), _stream(stream))
    _check(rc, "sfm_group_norm_bwd")
    return out
