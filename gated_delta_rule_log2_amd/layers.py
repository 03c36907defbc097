"""The operators around the recurrence in a layer: the short causal convolution, the RMS norm
with the residual's addition, and the selective state space scan that takes the recurrence's
place in some layers; each for prompts, for single tokens and for gradients.

As in the rest of the package the work is the HIP library's (C ABI in include/kda.h); the
functions here check and marshal torch tensors, run on the current HIP stream of the
tensors' device, and have no CPU fallback.  They neither synchronise nor copy to the host,
except that a packed call without ``cu_seqlens_host`` reads its offsets (as chunk_kda does).

    y, state = short_conv(x, weight, bias, activation="silu", output_final_state=True)
    y = short_conv_step(x_t, state, weight, bias, activation="silu")
    y, state = chunk_ssm(x, dt, A_log, B, C, output_final_state=True)
    y = ssm_step(x_t, dt_t, A_log, B_t, C_t, state)
    y, h = rms_norm(x, weight, residual)
    q, scales, h = rms_norm_fp8(x, weight, residual, group_size=128)
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import KDAContractError, KDARuntimeError, _abi, _check_tensor, _dtype_code, _ptr, _raise, library

_byref = ctypes.byref
# the current stream's handle without a Stream object around it (a single token's call is all overhead)
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _refuse(code: str, msg: str):
    raise KDAContractError(_abi.STATUS[code], msg)


def _device(t: torch.Tensor, what: str) -> torch.device:
    if t.device.type != "cuda":
        raise KDARuntimeError(_abi.KDA_ERR_HIP, f"{what} runs on a HIP device; got a CPU tensor")
    return t.device


def _call(fn, dev: torch.device, *args) -> None:
    """fn(*args, stream) with the tensors' device current."""
    if dev.index == torch.cuda.current_device():
        rc = fn(*args, _raw_stream(dev.index))
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, _raw_stream(dev.index))
    if rc != _abi.KDA_OK:
        _raise(rc, library())


def _size(fn, desc) -> int:
    n = ctypes.c_size_t(0)
    rc = fn(_byref(desc), _byref(n))
    if rc != _abi.KDA_OK:
        _raise(rc, library())
    return n.value


def _scratch(nbytes: int, dev: torch.device) -> torch.Tensor:
    """A call's own workspace, from torch's caching allocator: ordered with the stream, and a
    captured graph's is the graph's alone."""
    return torch.empty(nbytes, dtype=torch.uint8, device=dev)


def _check_place(t: torch.Tensor, name: str, shape: tuple, dev: torch.device, dtype) -> None:
    if t.shape != shape:
        _refuse("KDA_ERR_SHAPE", f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != dev:
        _refuse("KDA_ERR_SHAPE", f"{name} must be on {dev}")
    if dtype is not None and t.dtype != dtype:
        _refuse("KDA_ERR_DTYPE", f"{name} must be {dtype}")


def _token_stride(t: torch.Tensor, name: str, shape: tuple, dev: torch.device, dtype=None) -> int:
    """Elements between two tokens of t [B, T, ...]: its inner dimensions are contiguous and
    its tokens evenly spaced (a slice of a projection's output is)."""
    _check_place(t, name, shape, dev, dtype)
    B, T = shape[:2]
    stride, inner, ok = t.stride(), 1, True
    for i in range(len(shape) - 1, 1, -1):
        ok = ok and (shape[i] == 1 or stride[i] == inner)
        inner *= shape[i]
    step = stride[1] if T > 1 else stride[0] if B > 1 else inner
    ok = ok and step >= inner and (B == 1 or T <= 1 or stride[0] == T * step)
    if not ok and t.numel() > 0:
        _refuse("KDA_ERR_SHAPE", f"{name} must be contiguous within a token and its tokens evenly spaced")
    return max(step, inner)


def _row_stride(t: torch.Tensor, name: str, shape: tuple, dev: torch.device, dtype=None) -> int:
    """The same of one token for each row, t [rows, ...]."""
    _check_place(t, name, shape, dev, dtype)
    if t.is_contiguous():
        return t.numel() // shape[0]
    return _token_stride(t.unsqueeze(1), name, (shape[0], 1, *shape[1:]), dev, dtype)


class _Offsets:
    """Packed offsets: the host's copy (kept alive) and the device's, or none."""

    def __init__(self, cu_seqlens, cu_seqlens_host, B: int, dev: torch.device):
        self.host = self.dev = self.host_ptr = None
        self.N = B
        if cu_seqlens is None and cu_seqlens_host is None:
            return
        given = cu_seqlens if cu_seqlens is not None else cu_seqlens_host
        host = cu_seqlens_host if cu_seqlens_host is not None else cu_seqlens
        if given.dim() != 1 or given.numel() < 2 or host.shape != given.shape or given.is_floating_point():
            _refuse("KDA_ERR_VARLEN", "cu_seqlens must be a 1-D integer tensor of at least two offsets, and "
                                      "cu_seqlens_host its copy")
        self.host = host.detach().to("cpu", torch.int64).contiguous()
        self.dev = given.to(device=dev, dtype=torch.int64).contiguous()
        self.N = self.host.numel() - 1
        self.host_ptr = ctypes.cast(self.host.data_ptr(), ctypes.POINTER(ctypes.c_int64))


def _slots(slots, rows: int, pool: int, dev: torch.device):
    if slots is not None:
        _check_tensor(slots, "slots", (rows,), dev, torch.int32)
    elif pool < rows:
        _refuse("KDA_ERR_SHAPE", f"without slots the state must hold a row for each of the {rows} tokens")


# ------------------------------------------------------------------------------------- short convolution
def _conv_desc(B, T, x, weight, bias, activation, step, num_seqs, host_ptr, dy=None):
    if activation not in (None, "silu"):
        _refuse("KDA_ERR_UNSUPPORTED", f"activation must be None or 'silu', got {activation!r}")
    D, W, dev = x.shape[-1], weight.shape[1], x.device
    _check_tensor(weight, "weight", (D, W), dev)
    _check_tensor(bias, "bias", (D,), dev, weight.dtype)
    code = _dtype_code(x, "x")
    return _abi.KdaConvDesc(B, T, D, W, num_seqs, host_ptr, code, _dtype_code(weight, "weight"),
                            code if dy is None else _dtype_code(dy, "dy"), _abi.CONV_SILU if activation else 0, step)


def _conv_shapes(x, weight, dims, what):
    if x.dim() != dims or weight.dim() != 2 or x.shape[0] < 1:
        _refuse("KDA_ERR_SHAPE", "x must be [B, T, D] (a step [rows, D]) and weight [D, W]")
    if not 2 <= weight.shape[1] <= 4:
        _refuse("KDA_ERR_UNSUPPORTED", f"the convolution's width must be 2, 3 or 4, got {weight.shape[1]}")
    return _device(x, what)


def short_conv(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
               activation: Optional[str] = None, initial_state: Optional[torch.Tensor] = None,
               output_final_state: bool = False, cu_seqlens: Optional[torch.Tensor] = None, *,
               cu_seqlens_host: Optional[torch.Tensor] = None):
    """Causal convolution of every channel over its last W tokens, with an optional bias and
    SiLU: y_t = act(bias + sum_w weight[:, w] x_{t-W+1+w}).  Returns (y, final_state or None).

    x [B, T, D] float32 or bfloat16, possibly a view whose tokens are evenly spaced; weight
    [D, W] (W = 2, 3, 4) and bias [D] float32 or bfloat16; initial_state / final_state
    [N, W - 1, D] in x's dtype: a sequence's last W - 1 inputs, oldest first (N = B, or
    len(cu_seqlens) - 1 with B = 1).  cu_seqlens_host: a CPU copy of cu_seqlens, which spares
    the call the wait for the offsets (needed under graph capture).
    """
    dev = _conv_shapes(x, weight, 3, "short_conv")
    B, T, D = x.shape
    offsets = _Offsets(cu_seqlens, cu_seqlens_host, B, dev)
    d = _conv_desc(B, T, x, weight, bias, activation, _token_stride(x, "x", x.shape, dev), offsets.N, offsets.host_ptr)
    states = (offsets.N, d.W - 1, D)
    _check_tensor(initial_state, "initial_state", states, dev, x.dtype)
    y = torch.empty((B, T, D), dtype=x.dtype, device=dev)
    ht = torch.empty(states, dtype=x.dtype, device=dev) if output_final_state else None
    _call(library().kda_short_conv_fwd, dev, _byref(d), _ptr(x), _ptr(weight), _ptr(bias), _ptr(initial_state),
          _ptr(offsets.dev), _ptr(y), _ptr(ht))
    return y, ht


def short_conv_bwd(x: torch.Tensor, weight: torch.Tensor, dy: torch.Tensor, bias: Optional[torch.Tensor] = None,
                   activation: Optional[str] = None, initial_state: Optional[torch.Tensor] = None,
                   dht: Optional[torch.Tensor] = None, cu_seqlens: Optional[torch.Tensor] = None, *,
                   cu_seqlens_host: Optional[torch.Tensor] = None) -> dict:
    """Gradients of <dy, y> + <dht, final_state> for short_conv's inputs: dx and dh0 in x's
    dtype (dh0 where an initial_state is given), dweight and dbias (with a bias) in float32.
    dy has x's shape, in x's dtype or float32; dht the final state's shape and x's dtype.
    """
    dev = _conv_shapes(x, weight, 3, "short_conv_bwd")
    B, T, D = x.shape
    offsets = _Offsets(cu_seqlens, cu_seqlens_host, B, dev)
    d = _conv_desc(B, T, x, weight, bias, activation, _token_stride(x, "x", x.shape, dev), offsets.N, offsets.host_ptr, dy)
    states = (offsets.N, d.W - 1, D)
    _check_tensor(dy, "dy", (B, T, D), dev)
    _check_tensor(initial_state, "initial_state", states, dev, x.dtype)
    _check_tensor(dht, "dht", states, dev, x.dtype)
    lib = library()
    ws = _scratch(_size(lib.kda_short_conv_bwd_workspace_size, d), dev)
    out = {"dx": torch.empty((B, T, D), dtype=x.dtype, device=dev),
           "dweight": torch.empty((D, d.W), dtype=torch.float32, device=dev)}
    if bias is not None:
        out["dbias"] = torch.empty((D,), dtype=torch.float32, device=dev)
    if initial_state is not None:
        out["dh0"] = torch.empty(states, dtype=x.dtype, device=dev)
    _call(lib.kda_short_conv_bwd, dev, _byref(d), _ptr(x), _ptr(weight), _ptr(bias), _ptr(initial_state),
          _ptr(offsets.dev), _ptr(dy), _ptr(dht), _ptr(out["dx"]), _ptr(out["dweight"]), _ptr(out.get("dbias")),
          _ptr(out.get("dh0")), _ptr(ws), ws.numel())
    return out


def short_conv_step(x: torch.Tensor, state: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
                    activation: Optional[str] = None, slots: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One token of each row: y [rows, D] from x [rows, D] and the rows' states, which move on
    in place.  state [pool, W - 1, D] in x's dtype; slots [rows] int32 names each row's state
    (row b's is b without it).  A slot below 0 or past the pool marks a padding row: y is 0
    there and no state is touched.  Rows must not share a slot.
    """
    if x.dim() == 2 and x.shape[0] == 0:
        return torch.empty_like(x)
    dev = _conv_shapes(x, weight, 2, "short_conv_step")
    rows, D = x.shape
    d = _conv_desc(rows, 1, x, weight, bias, activation, _row_stride(x, "x", x.shape, dev), rows, None)
    pool = state.shape[0]
    _check_tensor(state, "state", (pool, d.W - 1, D), dev, x.dtype)
    _slots(slots, rows, pool, dev)
    y = torch.empty((rows, D), dtype=x.dtype, device=dev)
    _call(library().kda_short_conv_step, dev, _byref(d), x.data_ptr(), weight.data_ptr(), _ptr(bias), state.data_ptr(),
          _ptr(slots), pool, y.data_ptr())
    return y


# --------------------------------------------------------------------------------------------- RMS norm
def _norm_desc(x, weight, eps, group_size, what):
    dev = _device(x, what)
    if x.dim() < 1 or x.shape[-1] < 1:
        _refuse("KDA_ERR_SHAPE", "x must be [..., D]")
    D = x.shape[-1]
    _check_tensor(weight, "weight", (D,), dev)
    if not x.is_contiguous():
        _refuse("KDA_ERR_SHAPE", "x must be contiguous")
    return _abi.KdaNormDesc(x.numel() // D, D, group_size, _dtype_code(x, "x"), _dtype_code(weight, "weight"), eps), dev


def rms_norm(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None, eps: float = 1e-6):
    """RMS norm of the last dimension with the residual's addition in front: h = x + residual
    (rounded to x's dtype), y = h / sqrt(mean(h^2) + eps) * weight.  Returns (y, h); h is x
    itself without a residual.  x, residual [..., D] float32 or bfloat16, weight [D] either.
    """
    d, dev = _norm_desc(x, weight, eps, 0, "rms_norm")
    _check_tensor(residual, "residual", x.shape, dev, x.dtype)
    y = torch.empty_like(x)
    h = x if residual is None else torch.empty_like(x)
    _call(library().kda_rms_norm_fwd, dev, _byref(d), _ptr(x), _ptr(residual), _ptr(weight), _ptr(y),
          None if residual is None else _ptr(h))
    return y, h


def rms_norm_fp8(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None, eps: float = 1e-6,
                 group_size: int = 0):
    """rms_norm with its output in 8 bits for a projection in 8 bits: returns (q, scales, h)
    with y = q * scales over groups of group_size values (0: the row): q [..., D]
    float8_e4m3fn, scales [..., D / group_size] float32 (max|y| of the group / 448).
    group_size: 0, or a power of two from 8 to 512 that divides D.
    """
    d, dev = _norm_desc(x, weight, eps, group_size, "rms_norm_fp8")
    _check_tensor(residual, "residual", x.shape, dev, x.dtype)
    if group_size < 0 or (group_size and d.D % group_size):
        _refuse("KDA_ERR_UNSUPPORTED", f"group_size {group_size} must divide D = {d.D}")
    q = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=dev)
    scales = torch.empty((*x.shape[:-1], d.D // group_size if group_size else 1), dtype=torch.float32, device=dev)
    h = x if residual is None else torch.empty_like(x)
    _call(library().kda_rms_norm_fp8, dev, _byref(d), _ptr(x), _ptr(residual), _ptr(weight), _ptr(q), _ptr(scales),
          None if residual is None else _ptr(h))
    return q, scales, h


def rms_norm_bwd(h: torch.Tensor, weight: torch.Tensor, dy: torch.Tensor, dh: Optional[torch.Tensor] = None,
                 eps: float = 1e-6) -> dict:
    """Gradients of <dy, y> + <dh, h>: dx (h's dtype; x and the residual each have it) and
    dweight (float32).  h is what rms_norm returned; dy, and dh where a gradient arrives at
    the residual stream, have its shape and dtype.
    """
    d, dev = _norm_desc(h, weight, eps, 0, "rms_norm_bwd")
    _check_tensor(dy, "dy", h.shape, dev, h.dtype)
    _check_tensor(dh, "dh", h.shape, dev, h.dtype)
    lib = library()
    ws = _scratch(_size(lib.kda_rms_norm_bwd_workspace_size, d), dev)
    dx = torch.empty_like(h)
    dweight = torch.empty((d.D,), dtype=torch.float32, device=dev)
    _call(lib.kda_rms_norm_bwd, dev, _byref(d), _ptr(h), _ptr(weight), _ptr(dy), _ptr(dh), _ptr(dx), _ptr(dweight),
          _ptr(ws), ws.numel())
    return {"dx": dx, "dweight": dweight}


# ------------------------------------------------------------------------------- state space scan
def _ssm_desc(x, dt, A_log, B, C, D, dt_bias, softplus, num_seqs, host_ptr, what):
    dev, (H, P), (G, N) = x.device, x.shape[-2:], B.shape[-2:]
    if x.dim() == 4:
        (nb, T), stride = x.shape[:2], _token_stride
    else:
        nb, T, stride = x.shape[0], 1, _row_stride
    lead = x.shape[:-2]
    if A_log is None:
        _refuse("KDA_ERR_MISSING_A_LOG", f"{what} needs A_log")
    for t, name in ((A_log, "A_log"), (D, "D"), (dt_bias, "dt_bias")):
        _check_tensor(t, name, (H,), dev, torch.float32)
    return _abi.KdaSsmDesc(nb, T, H, G, N, P, num_seqs, host_ptr, _dtype_code(x, "x"), _dtype_code(dt, "dt"),
                           _abi.SSM_SOFTPLUS if softplus else 0, stride(x, "x", x.shape, dev),
                           stride(dt, "dt", (*lead, H), dev), stride(B, "B", (*lead, G, N), dev, x.dtype),
                           stride(C, "C", (*lead, G, N), dev, x.dtype))


def _ssm_shapes(x, dt, B, C, dims, what):
    if x.dim() != dims or B.dim() != dims or C.dim() != dims or dt.dim() != dims - 1 or x.shape[0] < 1:
        _refuse("KDA_ERR_SHAPE", "x must be [B, T, H, P], dt [B, T, H], and B, C [B, T, G, N] (a step has no T)")
    if 0 in x.shape[-2:] or 0 in B.shape[-2:]:
        _refuse("KDA_ERR_SHAPE", "x, B and C must have heads and channels")
    return _device(x, what)


def chunk_ssm(x: torch.Tensor, dt: torch.Tensor, A_log: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
              D: Optional[torch.Tensor] = None, dt_bias: Optional[torch.Tensor] = None,
              use_softplus_in_kernel: bool = False, initial_state: Optional[torch.Tensor] = None,
              output_final_state: bool = False, cu_seqlens: Optional[torch.Tensor] = None, *,
              cu_seqlens_host: Optional[torch.Tensor] = None):
    """The selective state space scan: per head, with the step d_t = dt_t + dt_bias (through a
    softplus with use_softplus_in_kernel) and A = -exp(A_log),

        S_t = exp(d_t A) S_{t-1} + d_t B_t x_t^T;    y_t = S_t^T C_t + D x_t

    Returns (y, final_state or None).  x [B, T, H, P], B, C [B, T, G, N] (head h uses group
    h / (H / G)) in one of float32 and bfloat16, dt [B, T, H] in either; each may be a view
    whose tokens are evenly spaced.  A_log, D, dt_bias [H] float32; N and P multiples of 32 up
    to 128.  initial_state / final_state [N_seq, H, N, P] float32 (N_seq = B, or
    len(cu_seqlens) - 1 with B = 1).  cu_seqlens_host as short_conv.
    """
    dev = _ssm_shapes(x, dt, B, C, 4, "chunk_ssm")
    offsets = _Offsets(cu_seqlens, cu_seqlens_host, x.shape[0], dev)
    d = _ssm_desc(x, dt, A_log, B, C, D, dt_bias, use_softplus_in_kernel, offsets.N, offsets.host_ptr,
                  "chunk_ssm")
    states = (offsets.N, d.H, d.N, d.P)
    _check_tensor(initial_state, "initial_state", states, dev, torch.float32)
    lib = library()
    ws = _scratch(_size(lib.kda_ssm_fwd_workspace_size, d), dev)
    y = torch.empty(x.shape, dtype=x.dtype, device=dev)
    ht = torch.empty(states, dtype=torch.float32, device=dev) if output_final_state else None
    _call(lib.kda_ssm_fwd, dev, _byref(d), _ptr(x), _ptr(dt), _ptr(A_log), _ptr(B), _ptr(C), _ptr(D), _ptr(dt_bias),
          _ptr(initial_state), _ptr(offsets.dev), _ptr(y), _ptr(ht), _ptr(ws), ws.numel())
    return y, ht


def chunk_ssm_bwd(x: torch.Tensor, dt: torch.Tensor, A_log: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
                  dy: torch.Tensor, dht: Optional[torch.Tensor] = None, D: Optional[torch.Tensor] = None,
                  dt_bias: Optional[torch.Tensor] = None, use_softplus_in_kernel: bool = False,
                  initial_state: Optional[torch.Tensor] = None, cu_seqlens: Optional[torch.Tensor] = None, *,
                  cu_seqlens_host: Optional[torch.Tensor] = None) -> dict:
    """Gradients of <dy, y> + <dht, final_state> for chunk_ssm's inputs: dx, dB, dC in x's
    dtype, ddt in dt's, dA_log, and dD, ddt_bias, dh0 where D, dt_bias, an initial_state are
    given, in float32.  dy has x's shape and dtype (contiguous), dht the final state's.
    """
    dev = _ssm_shapes(x, dt, B, C, 4, "chunk_ssm_bwd")
    offsets = _Offsets(cu_seqlens, cu_seqlens_host, x.shape[0], dev)
    d = _ssm_desc(x, dt, A_log, B, C, D, dt_bias, use_softplus_in_kernel, offsets.N, offsets.host_ptr,
                  "chunk_ssm_bwd")
    states = (offsets.N, d.H, d.N, d.P)
    _check_tensor(dy, "dy", x.shape, dev, x.dtype)
    _check_tensor(initial_state, "initial_state", states, dev, torch.float32)
    _check_tensor(dht, "dht", states, dev, torch.float32)
    lib = library()
    ws = _scratch(_size(lib.kda_ssm_bwd_workspace_size, d), dev)
    f32 = dict(dtype=torch.float32, device=dev)
    out = {"dx": torch.empty(x.shape, dtype=x.dtype, device=dev), "ddt": torch.empty(dt.shape, dtype=dt.dtype, device=dev),
           "dA_log": torch.empty((d.H,), **f32), "dB": torch.empty(B.shape, dtype=x.dtype, device=dev),
           "dC": torch.empty(C.shape, dtype=x.dtype, device=dev)}
    if D is not None:
        out["dD"] = torch.empty((d.H,), **f32)
    if dt_bias is not None:
        out["ddt_bias"] = torch.empty((d.H,), **f32)
    if initial_state is not None:
        out["dh0"] = torch.empty(states, **f32)
    _call(lib.kda_ssm_bwd, dev, _byref(d), _ptr(x), _ptr(dt), _ptr(A_log), _ptr(B), _ptr(C), _ptr(D), _ptr(dt_bias),
          _ptr(initial_state), _ptr(offsets.dev), _ptr(dy), _ptr(dht), _ptr(out["dx"]), _ptr(out["ddt"]),
          _ptr(out["dA_log"]), _ptr(out["dB"]), _ptr(out["dC"]), _ptr(out.get("dD")), _ptr(out.get("ddt_bias")),
          _ptr(out.get("dh0")), _ptr(ws), ws.numel())
    return out


def ssm_step(x: torch.Tensor, dt: torch.Tensor, A_log: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
             state: torch.Tensor, D: Optional[torch.Tensor] = None, dt_bias: Optional[torch.Tensor] = None,
             use_softplus_in_kernel: bool = False, slots: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One token of each row: y [rows, H, P] from x [rows, H, P], dt [rows, H], B, C [rows, G, N]
    and the rows' states, updated in place.  state [pool, H, N, P] float32; slots as
    short_conv_step.
    """
    if x.dim() == 3 and x.shape[0] == 0:
        return torch.empty_like(x)
    dev = _ssm_shapes(x, dt, B, C, 3, "ssm_step")
    rows = x.shape[0]
    d = _ssm_desc(x, dt, A_log, B, C, D, dt_bias, use_softplus_in_kernel, rows, None, "ssm_step")
    pool = state.shape[0]
    _check_tensor(state, "state", (pool, d.H, d.N, d.P), dev, torch.float32)
    _slots(slots, rows, pool, dev)
    y = torch.empty(x.shape, dtype=x.dtype, device=dev)
    _call(library().kda_ssm_step, dev, _byref(d), x.data_ptr(), dt.data_ptr(), A_log.data_ptr(), B.data_ptr(), C.data_ptr(),
          _ptr(D), _ptr(dt_bias), state.data_ptr(), _ptr(slots), pool, y.data_ptr())
    return y
