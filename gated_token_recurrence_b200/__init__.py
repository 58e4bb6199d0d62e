"""Python binding of libgtr.so (key-only gated linear attention forward, sm_100a).

Argument marshalling only: every step of the computation runs in the CUDA
kernels of ``libgtr.so``.  PyTorch supplies device memory and streams.  There
is no CPU fallback: importing this package fails if the library is missing.

    import gated_token_recurrence_b200 as gtr
    out = gtr.gla_fwd(q, k, v, log_gamma, grid=(H, W), direction=gtr.L2R)

Tensors are [B, L, heads, d] (log_gamma fp32 [B, L, heads, d_k]), contiguous,
on the current CUDA device.  See include/gtr.h for the full contract.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Tuple

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgtr.so")

L2R, R2L, T2B, B2T = 0, 1, 2, 3
F32, F16, BF16 = 0, 1, 2
PATH_AUTO, PATH_SPLIT, PATH_FUSED, PATH_FUSED_SEQUENTIAL = 0, 1, 2, 3
PATHS = {"auto": PATH_AUTO, "split": PATH_SPLIT, "fused": PATH_FUSED,
         "fused_sequential": PATH_FUSED_SEQUENTIAL}
STATUS = {0: "GTR_OK", 1: "GTR_ERR_INVALID_ARG", 2: "GTR_ERR_UNSUPPORTED", 3: "GTR_ERR_CUDA",
          4: "GTR_ERR_TIMEOUT", 5: "GTR_ERR_WORKSPACE", 6: "GTR_ERR_RANGE"}

# every symbol include/gtr.h declares
EXPORTED = ("gtr_gla_fwd", "gtr_gla_fwd_f16", "gtr_gla_fwd_bf16", "gtr_gla_fwd_f32",
            "gtr_gla_workspace_bytes", "gtr_gla_fwd_ex", "gtr_gla_fwd_host",
            "gtr_gla_read_error", "gtr_gla_plan", "gtr_gla_workspace_init", "gtr_status_string",
            "gtr_version", "gtr_gla_fwd_noalloc", "gtr_gla_block_fwd", "gtr_sswiglu_dwconv",
            "gtr_gla_workspace_debug", "gtr_ssm_conv", "gtr_ssm_scan", "gtr_ssm_step", "gtr_block_norm")


class GTRError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__(f"{what}: {STATUS.get(status, status)}" if what else STATUS.get(status, str(status)))


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"libgtr.so not found at {LIB_PATH}; build it with "
            "`python gated_token_recurrence_b200/build.py` (nvcc, sm_100a)")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    fwd_args = [vp] * 5 + [i] * 7
    lib.gtr_gla_fwd.argtypes = fwd_args + [i, i, vp]
    for name in ("gtr_gla_fwd_f16", "gtr_gla_fwd_bf16", "gtr_gla_fwd_f32"):
        getattr(lib, name).argtypes = fwd_args + [vp]
    lib.gtr_gla_fwd_ex.argtypes = fwd_args + [i, i, i, vp, sz, vp]
    lib.gtr_gla_fwd_host.argtypes = fwd_args + [i, i, vp]
    lib.gtr_gla_fwd_noalloc.argtypes = fwd_args + [i, i, vp]
    f = ctypes.c_float
    lib.gtr_gla_block_fwd.argtypes = [vp] * 7 + [i, f, vp, vp, f, vp] + [i] * 10 + [vp, sz, vp]
    lib.gtr_sswiglu_dwconv.argtypes = [vp] * 5 + [i] * 5 + [vp]
    q = ctypes.c_int64
    lib.gtr_ssm_conv.argtypes = [vp, q, vp, vp, vp, vp, vp, vp] + [i] * 8 + [vp]
    ssm = [vp, q, vp, q, vp, vp, q, vp, q, vp, q, vp, vp, i, vp, vp]
    lib.gtr_ssm_scan.argtypes = ssm + [vp, vp] + [i] * 8 + [vp]
    lib.gtr_ssm_step.argtypes = ssm + [vp] + [i] * 5 + [vp]
    lib.gtr_block_norm.argtypes = [vp] * 5 + [i, i, vp, f, vp, vp, i, q, i, i, i, vp]
    lib.gtr_gla_workspace_debug.argtypes = [vp, i, ctypes.c_uint, vp]
    lib.gtr_gla_workspace_bytes.argtypes = [i] * 8
    lib.gtr_gla_workspace_bytes.restype = sz
    lib.gtr_gla_read_error.argtypes = [vp, vp]
    lib.gtr_gla_workspace_init.argtypes = [vp, sz, vp]
    lib.gtr_gla_plan.argtypes = [i] * 7 + [ctypes.POINTER(i), ctypes.POINTER(i)]
    lib.gtr_status_string.argtypes = [i]
    lib.gtr_status_string.restype = ctypes.c_char_p
    lib.gtr_version.argtypes = []
    for name in ("gtr_gla_fwd", "gtr_gla_fwd_f16", "gtr_gla_fwd_bf16", "gtr_gla_fwd_f32",
                 "gtr_gla_fwd_ex", "gtr_gla_fwd_host", "gtr_gla_read_error", "gtr_gla_plan",
                 "gtr_gla_workspace_init", "gtr_version", "gtr_gla_fwd_noalloc", "gtr_gla_block_fwd",
                 "gtr_sswiglu_dwconv", "gtr_gla_workspace_debug", "gtr_ssm_conv", "gtr_ssm_scan",
                 "gtr_ssm_step", "gtr_block_norm"):
        getattr(lib, name).restype = ctypes.c_int
    return lib


lib = _load()


_CODES: dict = {}


def _dtype_code(t) -> int:
    if not _CODES:
        import torch
        _CODES.update({torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16})
    return _CODES[t.dtype]


def default_out_dtype(in_dtype):
    """fp16 -> fp16, bf16 -> fp32, fp32 -> fp32."""
    import torch
    return torch.float16 if in_dtype == torch.float16 else torch.float32


def _check(st: int, what: str):
    if st != 0:
        raise GTRError(st, what)


def _stream_handle(stream) -> int:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream)


def _shape(q, v, grid):
    B, L, heads, d_k = q.shape
    H, W = grid
    if H * W != L:
        raise ValueError(f"grid {H}x{W} does not match L={L}")
    return B, heads, H, W, d_k, v.shape[-1]


def workspace_bytes(B: int, heads: int, H: int, W: int, d_k: int = 64, d_v: int = 64,
                    in_dtype: int = F16, path: str = "auto") -> int:
    return int(lib.gtr_gla_workspace_bytes(B, heads, H, W, d_k, d_v, in_dtype, PATHS[path]))


def new_workspace(B: int, heads: int, H: int, W: int, d_k: int = 64, d_v: int = 64,
                  in_dtype: int = F16, path: str = "auto", device=None):
    """A zeroed uint8 CUDA tensor sized for :func:`gla_fwd` with ``workspace=``."""
    import torch
    n = max(256, workspace_bytes(B, heads, H, W, d_k, d_v, in_dtype, path))
    return torch.zeros(n, dtype=torch.uint8, device=device)


def gla_fwd(q, k, v, log_gamma, grid: Tuple[int, int], direction: int = L2R, out=None,
            path: str = "auto", workspace=None, stream=None):
    """Forward pass on CUDA tensors; returns ``out`` ([B, L, heads, d_v]).

    ``workspace`` (a uint8 CUDA tensor of at least :func:`workspace_bytes`,
    zeroed before its first use - see :func:`new_workspace`) selects the
    caller-managed-workspace entry (no allocation, capturable);
    without it the library's cached per-device workspace is used, and ``path``
    must then be "auto".
    """
    import torch
    B, heads, H, W, d_k, d_v = _shape(q, v, grid)
    if out is None:
        out = torch.empty((B, H * W, heads, d_v), dtype=default_out_dtype(q.dtype), device=q.device)
    for t in (q, k, v, log_gamma, out):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("gla_fwd takes contiguous CUDA tensors")
    if log_gamma.dtype != torch.float32:
        raise ValueError("log_gamma must be float32")
    if not (q.dtype == k.dtype == v.dtype):
        raise ValueError("q, k, v must share a dtype")
    args = (q.data_ptr(), k.data_ptr(), v.data_ptr(), log_gamma.data_ptr(), out.data_ptr(),
            B, heads, H, W, d_k, d_v, int(direction), _dtype_code(q), _dtype_code(out))
    s = _stream_handle(stream)
    if workspace is None and path == "auto":
        _check(lib.gtr_gla_fwd(*args, s), "gtr_gla_fwd")
    else:
        if workspace is None:
            workspace = new_workspace(B, heads, H, W, d_k, d_v, _dtype_code(q), path, q.device)
        _check(lib.gtr_gla_fwd_ex(*args, PATHS[path], workspace.data_ptr(), workspace.numel(), s),
               "gtr_gla_fwd_ex")
    return out


def gla_block_fwd(q, k, v, grid: Tuple[int, int], direction: int = L2R, log_gamma=None,
                  gate_z=None, gate_w2=None, gate_b=None, gate_tau: float = 16.0,
                  out_gate=None, norm_w=None, norm_eps: float = 1e-6, out=None, path: str = "auto",
                  workspace=None, stream=None):
    """The GLA token mixer of a GTR block (``gtr_gla_block_fwd``) on CUDA tensors.

    Gates: either ``log_gamma`` [B, L, heads, d_k] fp32, or the low-rank producer
    ``gate_z`` [B, L, r] fp32 with ``gate_w2`` [r, heads*d_k] and ``gate_b`` [heads*d_k]
    (log gamma = logsigmoid(z W2 + b) / gate_tau).  With ``out_gate`` [B, L, heads, d_v]
    (input dtype) and ``norm_w`` [d_v] fp32 the output is RMSNorm(o) * norm_w * SiLU(out_gate).
    """
    import torch
    B, heads, H, W, d_k, d_v = _shape(q, v, grid)
    if out is None:
        out = torch.empty((B, H * W, heads, d_v), dtype=default_out_dtype(q.dtype), device=q.device)
    tensors = [t for t in (q, k, v, log_gamma, gate_z, gate_w2, gate_b, out_gate, norm_w, out) if t is not None]
    for t in tensors:
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("gla_block_fwd takes contiguous CUDA tensors")
    for t in (log_gamma, gate_z, gate_w2, gate_b, norm_w):
        if t is not None and t.dtype != torch.float32:
            raise ValueError("gates, gate factors and the norm weight are float32")
    ptr = lambda t: None if t is None else t.data_ptr()
    rank = 0 if gate_z is None else int(gate_z.shape[-1])
    ws, wsb = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel())
    st = lib.gtr_gla_block_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), ptr(log_gamma), ptr(gate_z),
                               ptr(gate_w2), ptr(gate_b), rank, float(gate_tau), ptr(out_gate), ptr(norm_w),
                               float(norm_eps), out.data_ptr(), B, heads, H, W, d_k, d_v, int(direction),
                               _dtype_code(q), _dtype_code(out), PATHS[path], ws, wsb, _stream_handle(stream))
    _check(st, "gtr_gla_block_fwd")
    return out


def sswiglu_dwconv(xg, xv, conv_w, conv_b, grid: Tuple[int, int], out=None, stream=None):
    """SiLU(xg) * DWConv3x3(xv) on CUDA tensors ([B, L, C], L = H * W; conv_w [C, 3, 3] fp32,
    conv_b [C] fp32 or None) through ``gtr_sswiglu_dwconv``."""
    import torch
    B, L, C = xv.shape
    H, W = grid
    if H * W != L or xg.shape != xv.shape or xg.dtype != xv.dtype:
        raise ValueError("xg and xv must both be [B, H*W, C] of one dtype")
    if out is None:
        out = torch.empty_like(xv)
    for t in (xg, xv, conv_w, out) + (() if conv_b is None else (conv_b,)):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("sswiglu_dwconv takes contiguous CUDA tensors")
    st = lib.gtr_sswiglu_dwconv(xg.data_ptr(), xv.data_ptr(), conv_w.data_ptr(),
                                None if conv_b is None else conv_b.data_ptr(), out.data_ptr(), B, H, W, C,
                                _dtype_code(xv), _stream_handle(stream))
    _check(st, "gtr_sswiglu_dwconv")
    return out


# ---------------------------------------------------------------- selective SSM, block norm
# These calls are a few microseconds long, so the checks in front of them are written for the
# common case: one comparison of shape, type and device per tensor, strides looked at only
# where a tensor is not contiguous.
def _here(t):
    """The current device's index and its current stream's handle, for a call on tensor t."""
    import torch
    if not t.is_cuda:
        raise ValueError("expected CUDA tensors")
    dev = torch.cuda.current_device()
    return dev, torch._C._cuda_getCurrentRawStream(dev)


def _type_error(what, t, shape, dtype):
    return ValueError(f"{what}: expected a CUDA tensor {dtype} {tuple(shape)} on the current device, "
                      f"got {t.dtype} {tuple(t.shape)} on {t.device}")


def _whole(what, t, shape, dtype, dev):
    """The address of a contiguous tensor of this shape and type (None passes)."""
    if t is None:
        return None
    if t.shape != shape or t.dtype != dtype or t.get_device() != dev:
        raise _type_error(what, t, shape, dtype)
    if not t.is_contiguous():
        raise ValueError(f"{what}: must be contiguous")
    return t.data_ptr()


def _row_distance(what, t, tokens: int) -> int:
    """The distance between the rows of consecutive tokens of a tensor whose first `tokens` (1 or
    2) axes are batch and token axes; a row itself (the other 1 or 2 axes) is contiguous."""
    shape, stride = t.shape, t.stride()
    width = shape[-1]
    if (width != 1 and stride[-1] != 1) or (
            len(shape) - tokens == 2 and shape[tokens] != 1 and stride[tokens] != width):
        raise ValueError(f"{what}: the values of one token must be contiguous")
    if shape[tokens - 1] != 1:
        ld = stride[tokens - 1]
        if tokens == 2 and shape[0] != 1 and stride[0] != shape[1] * ld:
            raise ValueError(f"{what}: consecutive tokens must be evenly spaced")
        return ld
    if shape[0] != 1:
        return stride[0]
    unit = 16 // t.element_size()  # one token in all: any valid distance
    return -(-width * (shape[tokens] if len(shape) - tokens == 2 else 1) // unit) * unit


def _rows(what, t, shape, dtype, dev, tokens: int, width: int):
    """(address, distance between tokens) of a tensor that may be a column range of wider rows."""
    if t.shape != shape or t.dtype != dtype or t.get_device() != dev:
        raise _type_error(what, t, shape, dtype)
    return t.data_ptr(), (width if t.is_contiguous() else _row_distance(what, t, tokens))


def _grid_of(L, grid):
    H, W = grid
    if H * W != L:
        raise ValueError(f"grid {H}x{W} does not match L={L}")
    return H, W


def ssm_conv(x, w, bias, grid: Tuple[int, int], direction: int = L2R, silu: bool = True, state=None,
             state_out=None, lengths=None, out=None, stream=None):
    """Short causal depthwise convolution along the scan (``gtr_ssm_conv``); returns ``out``.

    ``x`` [B, L, C] (L = H * W; may be a column range of wider rows), ``w`` [C, K] fp32 with
    K = 2, 3 or 4, ``bias`` [C] fp32 or None.  ``state`` [B, K-1, C] holds the inputs before the
    first token (None: zeros); the last K-1 inputs are written to ``state_out``, which may be
    ``state``.  For a single new token per sequence the grid is (1, 1).  ``lengths`` [B] int32:
    tokens of each sequence of a padded batch; outputs behind them are left as they were.
    """
    import torch
    dev, here = _here(x)
    B, L, C = x.shape
    H, W = _grid_of(L, grid)
    K = w.shape[-1]
    ty, f32 = x.dtype, torch.float32
    px, ld = _rows("x", x, (B, L, C), ty, dev, 2, C)
    if out is None:
        out = torch.empty((B, L, C), dtype=ty, device=x.device)
    st = (B, K - 1, C)
    _check(lib.gtr_ssm_conv(px, ld, _whole("w", w, (C, K), f32, dev),
                            _whole("bias", bias, (C,), f32, dev),
                            _whole("state", state, st, ty, dev),
                            _whole("state_out", state_out, st, ty, dev),
                            _whole("lengths", lengths, (B,), torch.int32, dev),
                            _whole("out", out, (B, L, C), ty, dev), B, H, W, C, K, int(direction), 1 if silu else 0,
                            _dtype_code(x), here if stream is None else stream.cuda_stream), "gtr_ssm_conv")
    return out


def _ssm_inputs(u, dt, A, Bm, Cm, z, skip, dt_bias, lead, dev):
    """The arguments that a scan and a step share; ``lead`` is (B, L) or (B,)."""
    D, N = A.shape
    G = Bm.shape[-2]
    ty, f32, k = u.dtype, A.dtype, len(lead)
    rows, groups = (*lead, D), (*lead, G, N)
    pu, lu = _rows("u", u, rows, ty, dev, k, D)
    pd, ldt = _rows("dt", dt, rows, ty, dev, k, D)
    pb, lb = _rows("Bm", Bm, groups, ty, dev, k, G * N)
    pc, lc = _rows("Cm", Cm, groups, ty, dev, k, G * N)
    pz, lz = (None, 0) if z is None else _rows("z", z, rows, ty, dev, k, D)
    if _dtype_code(A) != F32:
        raise ValueError("A: must be float32")
    return ((pu, lu, pd, ldt, _whole("A", A, (D, N), f32, dev), pb, lb, pc, lc, pz, lz,
             _whole("skip", skip, (D,), f32, dev), _whole("dt_bias", dt_bias, (D,), f32, dev)), D, N, G)


def ssm_scan(u, dt, A, Bm, Cm, grid: Tuple[int, int], direction: int = L2R, skip=None, z=None, dt_bias=None,
             softplus: bool = True, state=None, state_out=None, lengths=None, out=None, stream=None):
    """Selective state space scan over a prompt (``gtr_ssm_scan``); returns ``out`` [B, L, D].

    ``u``, ``dt`` and the optional gate ``z`` [B, L, D], ``Bm`` and ``Cm`` [B, L, G, N] (each may
    be a column range of wider rows), ``A`` [D, N], ``skip`` and ``dt_bias`` [D] fp32.  ``state``
    [B, D, N] fp32 is h before the first token (None: zeros); h after the last is written to
    ``state_out``, which may be ``state``.  ``lengths`` as for :func:`ssm_conv`.
    """
    import torch
    dev, here = _here(u)
    B, L, D = u.shape
    H, W = _grid_of(L, grid)
    args, D, N, G = _ssm_inputs(u, dt, A, Bm, Cm, z, skip, dt_bias, (B, L), dev)
    if out is None:
        out = torch.empty((B, L, D), dtype=u.dtype, device=u.device)
    st = (B, D, N)
    _check(lib.gtr_ssm_scan(*args, 1 if softplus else 0, _whole("state", state, st, A.dtype, dev),
                            _whole("state_out", state_out, st, A.dtype, dev),
                            _whole("lengths", lengths, (B,), torch.int32, dev),
                            _whole("out", out, (B, L, D), u.dtype, dev), B, H, W, D, N, G, int(direction),
                            _dtype_code(u), here if stream is None else stream.cuda_stream), "gtr_ssm_scan")
    return out


def ssm_step(u, dt, A, Bm, Cm, state, skip=None, z=None, dt_bias=None, softplus: bool = True, state_out=None,
             out=None, stream=None):
    """Selective scan of one new token per sequence (``gtr_ssm_step``); returns ``out`` [B, D].

    ``u``, ``dt``, ``z`` [B, D], ``Bm`` and ``Cm`` [B, G, N]; the states ``state`` [B, D, N] fp32 are
    updated in place, or written to ``state_out`` where it is given.
    """
    dev, here = _here(u)
    B, D = u.shape
    args, D, N, G = _ssm_inputs(u, dt, A, Bm, Cm, z, skip, dt_bias, (B,), dev)
    if out is None:
        import torch
        out = torch.empty((B, D), dtype=u.dtype, device=u.device)
    st = (B, D, N)
    ps = _whole("state", state, st, A.dtype, dev)
    _check(lib.gtr_ssm_step(*args, 1 if softplus else 0, ps,
                            ps if state_out is None else _whole("state_out", state_out, st, A.dtype, dev),
                            _whole("out", out, (B, D), u.dtype, dev), B, D, N, G, _dtype_code(u),
                            here if stream is None else stream.cuda_stream), "gtr_ssm_step")
    return out


def block_norm(y, h, post_w=None, pre_w=None, gate=None, gate_silu: bool = False, scale=None, eps: float = 1e-6,
               h_out=None, n_out=None, stream=None):
    """The norms around a block with its gate, residual scale and residual stream (``gtr_block_norm``).

    h' = h + scale * act(gate) * RMSNorm(y) * post_w and n = RMSNorm(h') * pre_w; returns (h', n),
    n None without ``pre_w``.  ``y`` [B, L, C]; ``h`` [B, L, C] of the same type or fp32; ``gate``
    [B, C] or [B, L, C]; ``post_w``, ``pre_w``, ``scale`` [C] fp32.  ``h_out`` may be ``h`` and ``n_out``
    may be ``y``.
    """
    import torch
    dev, here = _here(y)
    B, L, C = rows = y.shape
    ty, f32 = y.dtype, torch.float32
    if h_out is None:
        h_out = torch.empty_like(h)
    if pre_w is None:
        if n_out is not None:
            raise ValueError("block_norm: n_out without pre_w")
    elif n_out is None:
        n_out = torch.empty_like(y)
    per_token = gate is not None and gate.dim() == 3
    _check(lib.gtr_block_norm(_whole("y", y, rows, ty, dev), _whole("h", h, rows, h.dtype, dev),
                              _whole("post_w", post_w, (C,), f32, dev),
                              _whole("pre_w", pre_w, (C,), f32, dev),
                              _whole("gate", gate, rows if per_token else (B, C), ty, dev),
                              1 if per_token else 0, 1 if gate_silu else 0,
                              _whole("scale", scale, (C,), f32, dev), eps,
                              _whole("h_out", h_out, rows, h.dtype, dev),
                              _whole("n_out", n_out, rows, ty, dev), B, L, C, _dtype_code(y), _dtype_code(h),
                              here if stream is None else stream.cuda_stream), "gtr_block_norm")
    return h_out, n_out


def gla_fwd_host(q, k, v, log_gamma, out, grid: Tuple[int, int], direction: int = L2R,
                 stream=None):
    """Forward pass on HOST (CPU, ideally pinned) tensors through ``gtr_gla_fwd_host``.

    The library copies the inputs in, runs, copies ``out`` back and synchronises.
    """
    B, heads, H, W, d_k, d_v = _shape(q, v, grid)
    for t in (q, k, v, log_gamma, out):
        if t.is_cuda or not t.is_contiguous():
            raise ValueError("gla_fwd_host takes contiguous CPU tensors")
    st = lib.gtr_gla_fwd_host(q.data_ptr(), k.data_ptr(), v.data_ptr(), log_gamma.data_ptr(),
                              out.data_ptr(), B, heads, H, W, d_k, d_v, int(direction),
                              _dtype_code(q), _dtype_code(out), _stream_handle(stream))
    _check(st, "gtr_gla_fwd_host")
    return out


def plan(B: int, heads: int, H: int, W: int, d_k: int = 64, d_v: int = 64,
         in_dtype: int = F16) -> Tuple[str, int]:
    """(path name, kernel launches per call) that the dispatcher picks for this problem."""
    path, launches = ctypes.c_int(0), ctypes.c_int(0)
    _check(lib.gtr_gla_plan(B, heads, H, W, d_k, d_v, in_dtype, ctypes.byref(path),
                            ctypes.byref(launches)), "gtr_gla_plan")
    name = {v: k for k, v in PATHS.items()}[path.value]
    return name, launches.value


def read_error(workspace=None, stream=None) -> int:
    """Synchronise and return (and clear) the device error word; 0 = none."""
    ptr = None if workspace is None else workspace.data_ptr()
    return int(lib.gtr_gla_read_error(ptr, _stream_handle(stream)))


def status_string(st: int) -> str:
    return lib.gtr_status_string(int(st)).decode()


def version() -> int:
    return int(lib.gtr_version())
