"""The operators around the gated delta rule in a linear-attention layer.

Same names and arguments as the C entry points of ``include/gdr.h``, on torch
tensors; work is enqueued on the current stream of the tensors' device.

``gdr_causal_conv_fwd`` / ``gdr_causal_conv_bwd`` / ``gdr_causal_conv_step``
    Short causal convolution (2 to 4 taps) with SiLU: prompts, gradient, one new token.
``gdr_step``
    The gated delta rule for one new token of each row.
``gdr_ssm_scan_fwd`` / ``gdr_ssm_step``
    Selective state space scan: prompts, one new token (inference).
``gdr_rms_norm_fwd`` / ``gdr_rms_norm_bwd``
    Root-mean-square norm with the residual's addition, a gate, an 8-bit output with scales.
``gdr_linear_scan_fwd`` / ``gdr_linear_scan_bwd`` / ``gdr_linear_scan_step``
    Gated linear recurrence of one decay per channel: prompts, gradient, one new token.
``gdr_block_norm_fwd`` / ``gdr_block_norm_bwd``
    The norm behind a block with its gate and scale, the residual's addition, and the norm before the next block.
``gdr_quantize_rows`` / ``gdr_matmul_i8``
    Rows in 8-bit integers with one scale each, and their product with such a weight (inference).
``causal_conv`` / ``rms_norm`` / ``linear_scan`` / ``block_norm``
    Differentiable through ``torch.autograd``.

Operands called "strided" may be slices of a wider row, such as the parts of a
fused projection's output.  ``cu_seqlens`` on the device is taken as it is (int32,
non-decreasing; nothing is copied to the host, so the calls can be captured into
a graph); on the host it is checked and copied.  Tokens that belong to no sequence
get zero rows.  ``slots`` name each row's state in the pool: a row whose slot is out
of range, or was named by an earlier row, is padding and gets a zero row.

Where gradients are recorded, the entry points other than the ``_bwd`` ones refuse
inputs that require one: ``causal_conv``, ``rms_norm``, ``linear_scan`` and
``block_norm`` are the calls that give it.  The ``_bwd`` ones return plain values.

These four can be captured with their backward, as any differentiable call of
torch: on leaves that no eager graph alive was built from.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch
from torch.autograd.function import once_differentiable

from . import GDR_BF16, GDR_F32, GdrError, _Shape, load_library

_i32, _i64, _f32, _vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p


class _ConvShape(ctypes.Structure):
    _fields_ = [("B", _i32), ("T", _i32), ("D", _i32), ("W", _i32), ("num_seqs", _i32), ("dtype", ctypes.c_int),
                ("activation", ctypes.c_int), ("x_stride", _i64)]


class _SsmShape(ctypes.Structure):
    _fields_ = [("B", _i32), ("T", _i32), ("H", _i32), ("G", _i32), ("P", _i32), ("N", _i32), ("num_seqs", _i32),
                ("dtype", ctypes.c_int), ("dt_softplus", _i32), ("x_stride", _i64), ("dt_stride", _i64),
                ("b_stride", _i64), ("c_stride", _i64)]


class _NormShape(ctypes.Structure):
    _fields_ = [("rows", _i64), ("inner", _i32), ("dim", _i32), ("dtype", ctypes.c_int), ("eps", _f32), ("quant", _i32),
                ("x_outer", _i64), ("x_inner", _i64), ("r_outer", _i64), ("r_inner", _i64), ("g_outer", _i64),
                ("g_inner", _i64)]


class _LinearScanShape(ctypes.Structure):
    _fields_ = [("B", _i32), ("T", _i32), ("D", _i32), ("num_seqs", _i32), ("dtype", ctypes.c_int), ("x_stride", _i64),
                ("r_stride", _i64), ("i_stride", _i64)]


class _BlockNormShape(ctypes.Structure):
    _fields_ = [("rows", _i64), ("dim", _i32), ("dtype", ctypes.c_int), ("eps", _f32), ("x_stride", _i64),
                ("residual_stride", _i64), ("gate_stride", _i64)]


class _QuantizeShape(ctypes.Structure):
    _fields_ = [("rows", _i64), ("dim", _i32), ("dtype", ctypes.c_int), ("x_stride", _i64), ("q_stride", _i64)]


class _MatmulI8Shape(ctypes.Structure):
    _fields_ = [("M", _i32), ("N", _i32), ("K", _i32), ("dtype", ctypes.c_int), ("x_stride", _i64), ("w_stride", _i64)]


_SIGNATURES = {
    "gdr_causal_conv_fwd": (_ConvShape, 8),
    "gdr_causal_conv_bwd": (_ConvShape, 12, ctypes.c_size_t, 1),
    "gdr_causal_conv_step": (_ConvShape, 4, _i32, 3),
    "gdr_step": (_Shape, 1, _i64, 1, _i64, 1, _i64, 2, _f32, 1, _i32, 3),
    "gdr_ssm_scan_fwd": (_SsmShape, 12, ctypes.c_size_t, 1),
    "gdr_ssm_step": (_SsmShape, 8, _i32, 3),
    "gdr_rms_norm_fwd": (_NormShape, 8),
    "gdr_rms_norm_bwd": (_NormShape, 9, ctypes.c_size_t, 1),
    "gdr_causal_conv_bwd_workspace_size": (_ConvShape,),
    "gdr_ssm_scan_fwd_workspace_size": (_SsmShape,),
    "gdr_rms_norm_bwd_workspace_size": (_NormShape,),
    "gdr_linear_scan_fwd": (_LinearScanShape, 9, ctypes.c_size_t, 1),
    "gdr_linear_scan_bwd": (_LinearScanShape, 14, ctypes.c_size_t, 1),
    "gdr_linear_scan_step": (_LinearScanShape, 5, _i32, 3),
    "gdr_block_norm_fwd": (_BlockNormShape, 9),
    "gdr_block_norm_bwd": (_BlockNormShape, 15, ctypes.c_size_t, 1),
    "gdr_quantize_rows": (_QuantizeShape, 4),
    "gdr_matmul_i8": (_MatmulI8Shape, 7),
    "gdr_linear_scan_fwd_workspace_size": (_LinearScanShape,),
    "gdr_linear_scan_bwd_workspace_size": (_LinearScanShape,),
    "gdr_block_norm_bwd_workspace_size": (_BlockNormShape,),
}
_entries = {}


def _entry(name):
    """The library's entry point, its prototype set (a number in the signature: that many pointers)."""
    fn = _entries.get(name)
    if fn is None:
        fn = getattr(load_library(), name)
        shape, *rest = _SIGNATURES[name]
        fn.argtypes = [ctypes.POINTER(shape)]
        for r in rest:
            fn.argtypes += [_vp] * r if isinstance(r, int) else [r]
        fn.restype = ctypes.c_size_t if name.endswith("_size") else ctypes.c_int
        _entries[name] = fn
    return fn


_device, _raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
# The steps write to their states behind torch's back: told so, autograd refuses a
# backward pass that kept such a state, instead of reading the new one.
_changed = torch._C._increment_version


def _call(index, fn, shape, *args):
    """Calls an entry point with the tensors' device current and its current stream last."""
    if _device() == index:
        rc = fn(shape, *args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            rc = fn(shape, *args, _raw_stream(index))
    if rc:
        raise GdrError(f"libgdr status {rc}: {load_library().gdr_last_error().decode()}")


def _bytes(name, shape) -> int:
    n = _entry(name)(shape)
    if n == 0:
        raise GdrError(f"libgdr status -1: {load_library().gdr_last_error().decode()}")
    return n


def _workspace(workspace, n, index):
    if workspace is None:
        return torch.empty(n, device=index, dtype=torch.uint8)
    if workspace.get_device() != index or workspace.dtype != torch.uint8 or not workspace.is_contiguous() or workspace.numel() < n:
        raise GdrError(f"workspace must be a contiguous uint8 tensor of at least {n} bytes on device {index}")
    return workspace


def _code(t) -> int:
    if t.dtype is torch.bfloat16:
        return GDR_BF16
    if t.dtype is torch.float32:
        return GDR_F32
    raise GdrError(f"unsupported dtype {t.dtype} (bfloat16 or float32)")


# The checks below run on every call of a serving step: one test of what is
# expected first, and what is wrong with the tensor only where that fails.
def _refuse(t, name, shape, dtype, index, contiguous=True):
    if tuple(t.shape) != shape:
        raise GdrError(f"shape mismatch: {name} is {tuple(t.shape)}, expected {shape}")
    if t.dtype != dtype:
        raise GdrError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise GdrError(f"{name} must be a device tensor")
    if t.get_device() != index:
        raise GdrError(f"{name} is on {t.device}, expected device {index}")
    if contiguous and not t.is_contiguous():
        raise GdrError(f"{name} must be contiguous")


def _dense(t, name, shape, dtype, index):
    """Pointer of a contiguous device tensor of this shape and type (None stays None)."""
    if t is None:
        return None
    if t.shape != shape or t.dtype is not dtype or t.get_device() != index or index < 0 or not t.is_contiguous():
        _refuse(t, name, shape, dtype, index)
    return t.data_ptr()


def _rows_of(t, name, shape, dtype, index, lead):
    """(pointer, token stride) of a tensor whose last dimensions are dense and whose first `lead` ones (batch, token)
    have one stride."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != index or index < 0:
        _refuse(t, name, shape, dtype, index, False)
    if t.is_contiguous():
        return t.data_ptr(), 0
    st = t.stride()
    width = 1
    for n, s in zip(reversed(shape[lead:]), reversed(st[lead:])):
        if n != 1 and s != width:
            raise GdrError(f"{name}: the values of a token must be contiguous")
        width *= n
    if lead == 1:
        token, tokens = (st[0] if shape[0] > 1 else 0), shape[0]
    else:
        B, T = shape[:2]
        token, tokens = (st[1] if T > 1 else st[0] if B > 1 else 0), B * T
        if B > 1 and T > 1 and st[0] != T * token:
            raise GdrError(f"{name}: batch and token must have one stride")
    if token == 0 and tokens > 1:   # 0 stands for dense in the library
        raise GdrError(f"{name}: rows overlap (expanded tensor): call .contiguous()")
    return t.data_ptr(), token


_MOST = 0x7fffffff   # the library's sizes are 32-bit integers, and ctypes cuts what is longer off without a word


def _too_long(**sizes):
    raise GdrError(f"{next(name for name, n in sizes.items() if n > _MOST)} must be below 2^31")


def _offsets(cu_seqlens, B, T, dev):
    """(device int32 tensor or None, number of sequences)."""
    if cu_seqlens is None:
        return None, B
    if B != 1:
        raise GdrError("packed mode (cu_seqlens) requires B == 1")
    cu = cu_seqlens if isinstance(cu_seqlens, torch.Tensor) else torch.as_tensor(cu_seqlens)
    if cu.dim() != 1 or cu.numel() < 2 or cu.dtype not in (torch.int32, torch.int64):
        raise GdrError("cu_seqlens must be a 1-D int32 or int64 tensor of at least two offsets")
    if cu.numel() > _MOST:
        _too_long(offsets=cu.numel())
    if cu.is_cuda:
        if cu.device != dev:
            raise GdrError(f"cu_seqlens is on {cu.device}, expected {dev}")
    else:
        if cu[0] < 0 or cu[-1] > T or (cu[1:] < cu[:-1]).any():
            raise GdrError("cu_seqlens must be non-decreasing, within [0, T]")
    if cu.dtype != torch.int32 or not cu.is_cuda or not cu.is_contiguous():
        cu = cu.to(device=dev, dtype=torch.int32).contiguous()
    return cu, cu.numel() - 1


_grad_enabled = torch._C.is_grad_enabled if hasattr(torch._C, "is_grad_enabled") else torch.is_grad_enabled


def _no_gradient(name, instead=None):
    raise GdrError(f"{name} offers no gradient: call it under torch.no_grad(), or detach its inputs" if instead is None else
                   f"{name} records no gradient: call {instead}, or call it under torch.no_grad()")


def _ptr(t):
    return None if t is None else t.data_ptr()


def _pool(state, name, tail, dtype, index, rows, slots):
    if state.dim() != 1 + len(tail):
        raise GdrError(f"shape mismatch: {name} is {tuple(state.shape)}, expected (slots, {', '.join(map(str, tail))})")
    n = state.shape[0]
    if state.shape[1:] != tail or state.dtype is not dtype or state.get_device() != index or index < 0 or not state.is_contiguous():
        _refuse(state, name, (n, *tail), dtype, index)
    ptr = state.data_ptr()
    if n < 1 or (slots is None and n < rows):
        raise GdrError(f"{name} holds {n} slots for {rows} rows")
    # int32 slots name none behind the 2^31 - 1st, and ctypes would cut a longer pool's size off
    return ptr, n if n < _MOST else _MOST, _dense(slots, "slots", (rows,), torch.int32, index)


_ACT = {None: 0, "none": 0, "silu": 1}


def _activation(activation):
    if activation not in _ACT:
        raise GdrError(f"unknown activation {activation!r} (None or 'silu')")
    return _ACT[activation]


# ------------------------------------------------------------ convolution --
def _conv_args(x, weight, bias, cu_seqlens, activation):
    if x.dim() != 3 or weight.dim() != 2:
        raise GdrError("x must be [B, T, D] and weight [D, W]")
    B, T, D = x.shape
    W = weight.shape[1]
    if B > _MOST or T > _MOST or D > _MOST:
        _too_long(B=B, T=T, D=D)
    act, code, dev, ty = _activation(activation), _code(x), x.get_device(), x.dtype
    xp, xs = _rows_of(x, "x", (B, T, D), ty, dev, 2)
    wp = _dense(weight, "weight", (D, W), ty, dev)
    bp = _dense(bias, "bias", (D,), ty, dev)
    cu, N = _offsets(cu_seqlens, B, T, x.device)
    return _ConvShape(B, T, D, W, N, code, act, xs), xp, wp, bp, cu, N, dev


def gdr_causal_conv_fwd(x, weight, bias=None, initial_state=None, cu_seqlens=None, *, activation="silu",
                        output_final_state=False):
    """y = act(causal convolution of x): x [B, T, D] (strided), weight [D, W], initial_state [N, W - 1, D].
    Returns (y, final_state or None)."""
    if _grad_enabled() and (x.requires_grad or weight.requires_grad or (bias is not None and bias.requires_grad)
                            or (initial_state is not None and initial_state.requires_grad)):
        _no_gradient("gdr_causal_conv_fwd", "causal_conv")
    sh, xp, wp, bp, cu, N, dev = _conv_args(x, weight, bias, cu_seqlens, activation)
    state = (N, sh.W - 1, sh.D)
    hp = _dense(initial_state, "initial_state", state, x.dtype, dev)
    y = torch.empty(x.shape, device=dev, dtype=x.dtype)
    ht = torch.empty(state, device=dev, dtype=x.dtype) if output_final_state else None
    _call(dev, _entry("gdr_causal_conv_fwd"), sh, xp, wp, bp, hp, _ptr(cu), y.data_ptr(), _ptr(ht))
    return y, ht


def gdr_causal_conv_bwd(x, weight, bias, dy, initial_state=None, dht=None, cu_seqlens=None, *, activation="silu",
                        workspace=None):
    """Backward of gdr_causal_conv_fwd.  Returns (dx, dw, db, dh0); db is None without a bias, dh0 without an
    initial state."""
    sh, xp, wp, bp, cu, N, dev = _conv_args(x, weight, bias, cu_seqlens, activation)
    state = (N, sh.W - 1, sh.D)
    hp = _dense(initial_state, "initial_state", state, x.dtype, dev)
    dyp = _dense(dy, "dy", tuple(x.shape), x.dtype, dev)
    dhp = _dense(dht, "dht", state, x.dtype, dev)
    dx = torch.empty(x.shape, device=dev, dtype=x.dtype)
    dw = torch.empty_like(weight)
    db = None if bias is None else torch.empty_like(bias)
    dh0 = None if initial_state is None else torch.empty_like(initial_state)
    ws = _workspace(workspace, _bytes("gdr_causal_conv_bwd_workspace_size", sh), dev)
    _call(dev, _entry("gdr_causal_conv_bwd"), sh, xp, wp, bp, hp, _ptr(cu), dyp, dhp, dx.data_ptr(), dw.data_ptr(), _ptr(db),
          _ptr(dh0), ws.data_ptr(), ws.numel())
    return dx, dw, db, dh0


def gdr_causal_conv_step(x, state, weight, bias=None, *, slots=None, activation="silu"):
    """One new token per row: x [rows, D] (strided), state [slots, W - 1, D] moves on in place.  Returns y [rows, D]."""
    if x.dim() != 2 or weight.dim() != 2:
        raise GdrError("x must be [rows, D] and weight [D, W]")
    if _grad_enabled() and (x.requires_grad or state.requires_grad or weight.requires_grad
                            or (bias is not None and bias.requires_grad)):
        _no_gradient("gdr_causal_conv_step")
    rows, D = x.shape
    W = weight.shape[1]
    if rows > _MOST or D > _MOST:
        _too_long(rows=rows, D=D)
    act, code, dev, ty = _activation(activation), _code(x), x.get_device(), x.dtype
    xp, xs = _rows_of(x, "x", (rows, D), ty, dev, 1)
    wp = _dense(weight, "weight", (D, W), ty, dev)
    bp = _dense(bias, "bias", (D,), ty, dev)
    sp, n, lp = _pool(state, "state", (W - 1, D), ty, dev, rows, slots)
    y = torch.empty(rows, D, device=dev, dtype=ty) if xs else torch.empty_like(x)
    if rows:
        _call(dev, _entry("gdr_causal_conv_step"), _ConvShape(rows, 1, D, W, 0, code, act, xs), xp, wp, bp, sp, n, lp, y.data_ptr())
        _changed((state,))
    return y


class _ConvFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, initial_state, cu_seqlens, activation, output_final_state):
        cu, _ = _offsets(cu_seqlens, x.shape[0], x.shape[1], x.device) if x.dim() == 3 else (None, 0)
        y, ht = gdr_causal_conv_fwd(x, weight, bias, initial_state, cu, activation=activation,
                                    output_final_state=output_final_state)
        ctx.save_for_backward(x, weight, bias, initial_state, cu)
        ctx.activation = activation
        ctx.set_materialize_grads(False)
        return y, ht

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dht):
        x, weight, bias, h0, cu = ctx.saved_tensors
        if dy is None and dht is None:
            return (None,) * 7
        dy = torch.zeros(x.shape, device=x.device, dtype=x.dtype) if dy is None else dy.contiguous()
        dht = None if dht is None else dht.contiguous()
        dx, dw, db, dh0 = gdr_causal_conv_bwd(x, weight, bias, dy, h0, dht, cu, activation=ctx.activation)
        return dx, dw, db, dh0, None, None, None


def causal_conv(x, weight, bias=None, initial_state=None, output_final_state=False, cu_seqlens=None, activation="silu"):
    """High-level call: returns (y, final_state or None); differentiable."""
    return _ConvFunction.apply(x, weight, bias, initial_state, cu_seqlens, activation, output_final_state)


# ------------------------------------------------------ gated delta rule --
def gdr_step(q, k, v, g, beta, state, scale=None, *, slots=None):
    """One new token per row of the gated delta rule: q, k [rows, Hq, K], v [rows, Hv, V] (strided), g, beta [rows, Hv]
    fp32, state [slots, Hv, K, V] fp32, in place.  Returns o [rows, Hv, V]."""
    if q.dim() != 3 or v.dim() != 3:
        raise GdrError("q and v must be 3-D: [rows, Hq, K] and [rows, Hv, V]")
    if _grad_enabled() and (q.requires_grad or k.requires_grad or v.requires_grad or g.requires_grad
                            or beta.requires_grad or state.requires_grad):
        _no_gradient("gdr_step")
    rows, Hq, K = q.shape
    Hv, V = v.shape[1], v.shape[2]
    code, dev, dt = _code(q), q.get_device(), q.dtype
    qp, qs = _rows_of(q, "q", (rows, Hq, K), dt, dev, 1)
    kp, ks = _rows_of(k, "k", (rows, Hq, K), dt, dev, 1)
    vp, vs = _rows_of(v, "v", (rows, Hv, V), dt, dev, 1)
    gp = _dense(g, "g", (rows, Hv), torch.float32, dev)
    bp = _dense(beta, "beta", (rows, Hv), torch.float32, dev)
    sp, n, lp = _pool(state, "state", (Hv, K, V), torch.float32, dev, rows, slots)
    o = torch.empty(rows, Hv, V, device=dev, dtype=dt) if vs else torch.empty_like(v)
    if rows:
        _call(dev, _entry("gdr_step"), _Shape(rows, 1, Hq, Hv, K, V, 0, code), qp, qs, kp, ks, vp, vs, gp, bp,
              K ** -0.5 if scale is None else float(scale), sp, n, lp, o.data_ptr())
        _changed((state,))
    return o


# -------------------------------------------------------------------- scan --
def gdr_ssm_scan_fwd(x, dt, A, B, C, D=None, dt_bias=None, initial_state=None, cu_seqlens=None, *, dt_softplus=True,
                     output_final_state=False, workspace=None):
    """Selective state space scan: x [batch, T, H, P], dt [batch, T, H], B, C [batch, T, G, N] (strided); A, D, dt_bias
    [H] fp32; initial_state [N_seqs, H, N, P] fp32.  Returns (y, final_state or None).  No gradient."""
    if x.dim() != 4 or B.dim() != 4:
        raise GdrError("x and B must be 4-D: [batch, T, H, P] and [batch, T, G, N]")
    if _grad_enabled() and any(t is not None and t.requires_grad for t in (x, dt, A, B, C, D, dt_bias, initial_state)):
        _no_gradient("gdr_ssm_scan_fwd")
    b, T, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    code, dev, ty = _code(x), x.get_device(), x.dtype
    xp, xs = _rows_of(x, "x", (b, T, H, P), ty, dev, 2)
    dp, ds = _rows_of(dt, "dt", (b, T, H), ty, dev, 2)
    Bp, bs = _rows_of(B, "B", (b, T, G, N), ty, dev, 2)
    Cp, cs = _rows_of(C, "C", (b, T, G, N), ty, dev, 2)
    Ap = _dense(A, "A", (H,), torch.float32, dev)
    Dp = _dense(D, "D", (H,), torch.float32, dev)
    ip = _dense(dt_bias, "dt_bias", (H,), torch.float32, dev)
    cu, S = _offsets(cu_seqlens, b, T, x.device)
    hp = _dense(initial_state, "initial_state", (S, H, N, P), torch.float32, dev)
    sh = _SsmShape(b, T, H, G, P, N, S, code, 1 if dt_softplus else 0, xs, ds, bs, cs)
    y = torch.empty((b, T, H, P), device=dev, dtype=ty)
    ht = torch.empty((S, H, N, P), device=dev, dtype=torch.float32) if output_final_state else None
    ws = _workspace(workspace, _bytes("gdr_ssm_scan_fwd_workspace_size", sh), dev)
    _call(dev, _entry("gdr_ssm_scan_fwd"), sh, xp, dp, Ap, Bp, Cp, Dp, ip, hp, _ptr(cu), y.data_ptr(), _ptr(ht), ws.data_ptr(),
          ws.numel())
    return y, ht


def gdr_ssm_step(x, dt, A, B, C, state, D=None, dt_bias=None, *, slots=None, dt_softplus=True):
    """One new token per row of the scan: x [rows, H, P], dt [rows, H], B, C [rows, G, N] (strided), state
    [slots, H, N, P] fp32, in place.  Returns y [rows, H, P]."""
    if x.dim() != 3 or B.dim() != 3:
        raise GdrError("x and B must be 3-D: [rows, H, P] and [rows, G, N]")
    if _grad_enabled() and any(t is not None and t.requires_grad for t in (x, dt, A, B, C, state, D, dt_bias)):
        _no_gradient("gdr_ssm_step")
    rows, H, P = x.shape
    G, N = B.shape[1], B.shape[2]
    code, dev, ty = _code(x), x.get_device(), x.dtype
    xp, xs = _rows_of(x, "x", (rows, H, P), ty, dev, 1)
    dp, ds = _rows_of(dt, "dt", (rows, H), ty, dev, 1)
    Bp, bs = _rows_of(B, "B", (rows, G, N), ty, dev, 1)
    Cp, cs = _rows_of(C, "C", (rows, G, N), ty, dev, 1)
    Ap = _dense(A, "A", (H,), torch.float32, dev)
    Dp = _dense(D, "D", (H,), torch.float32, dev)
    ip = _dense(dt_bias, "dt_bias", (H,), torch.float32, dev)
    sp, n, lp = _pool(state, "state", (H, N, P), torch.float32, dev, rows, slots)
    y = torch.empty(rows, H, P, device=dev, dtype=ty) if xs else torch.empty_like(x)
    if rows:
        _call(dev, _entry("gdr_ssm_step"), _SsmShape(rows, 1, H, G, P, N, 0, code, 1 if dt_softplus else 0, xs, ds, bs, cs),
              xp, dp, Ap, Bp, Cp, Dp, ip, sp, n, lp, y.data_ptr())
        _changed((state,))
    return y


# -------------------------------------------------------------------- norm --
def _norm_rows(t, name, shape, dtype, index):
    """(pointer, outer stride, inner stride) of [..., inner, dim] rows; all leading dimensions have one stride."""
    if t is None:
        return None, 0, 0
    if t.shape != shape or t.dtype is not dtype or t.get_device() != index or index < 0:
        _refuse(t, name, shape, dtype, index, False)
    if t.is_contiguous():
        return t.data_ptr(), 0, 0
    st = t.stride()
    if shape[-1] != 1 and st[-1] != 1:
        raise GdrError(f"{name}: the values of a row must be contiguous")
    if len(shape) == 2:
        outer, inner = st[0], 0
    else:
        inner, width = (st[-2] if shape[-2] > 1 else 0), None
        outer = 0
        for n, s in zip(reversed(shape[:-2]), reversed(st[:-2])):
            if n == 1:
                continue
            if width is None:
                outer, width = s, s * n
            elif s != width:
                raise GdrError(f"{name}: the leading dimensions must have one stride")
            else:
                width *= n
    if outer == 0 and inner == 0:
        raise GdrError(f"{name}: rows overlap (expanded tensor): call .contiguous()")
    return t.data_ptr(), outer, inner


def _norm_shape(x):
    if x.dim() < 2:
        raise GdrError("x must be [..., dim] with at least two dimensions")
    shape = x.shape
    dim = shape[-1]
    if dim > _MOST:
        _too_long(dim=dim)
    rows = x.numel() // dim if dim else 0
    return shape, rows, (shape[-2] if len(shape) > 2 and rows else 1), dim


def gdr_rms_norm_fwd(x, weight, residual=None, gate=None, *, eps=1e-6, quant=False):
    """y = rms_norm(x + residual) * weight * silu(gate) over the last dimension; x, residual and gate [..., dim]
    (strided).  Returns (y, scales, h): with quant, y is float8_e4m3fn and scales [..., ceil(dim / 128)] fp32 hold one
    scale for each 128 values; h is the sum x + residual (None without a residual)."""
    if _grad_enabled() and (x.requires_grad or weight.requires_grad or (residual is not None and residual.requires_grad)
                            or (gate is not None and gate.requires_grad)):
        _no_gradient("gdr_rms_norm_fwd", "rms_norm")
    shape, rows, inner, dim = _norm_shape(x)
    code, dev, dt = _code(x), x.get_device(), x.dtype
    xp, xo, xi = _norm_rows(x, "x", shape, dt, dev)
    rp, ro, ri = _norm_rows(residual, "residual", shape, dt, dev)
    gp, go, gi = _norm_rows(gate, "gate", shape, dt, dev)
    wp = _dense(weight, "weight", (dim,), dt, dev)
    y = torch.empty(*shape, device=dev, dtype=torch.float8_e4m3fn if quant else dt)
    scales = torch.empty(*shape[:-1], (dim + 127) // 128, device=dev, dtype=torch.float32) if quant else None
    h = torch.empty(*shape, device=dev, dtype=dt) if residual is not None else None
    sh = _NormShape(rows, inner, dim, code, eps, 1 if quant else 0, xo, xi, ro, ri, go, gi)
    _call(dev, _entry("gdr_rms_norm_fwd"), sh, xp, rp, gp, wp, y.data_ptr(), _ptr(scales), _ptr(h))
    return y, scales, h


def gdr_rms_norm_bwd(h, weight, dy, gate=None, dres=None, *, eps=1e-6, workspace=None):
    """Backward of gdr_rms_norm_fwd at h = x + residual; dres is the gradient of h from elsewhere.  Returns
    (dh, dw, dgate); dh is the gradient of x and of residual, dgate is None without a gate."""
    shape, rows, inner, dim = _norm_shape(h)
    code, dev, dt = _code(h), h.get_device(), h.dtype
    hp, ho, hi = _norm_rows(h, "h", shape, dt, dev)
    gp, go, gi = _norm_rows(gate, "gate", shape, dt, dev)
    wp = _dense(weight, "weight", (dim,), dt, dev)
    dyp = _dense(dy, "dy", shape, dt, dev)
    drp = _dense(dres, "dres", shape, dt, dev)
    dh = torch.empty(shape, device=dev, dtype=dt)
    dw = torch.empty((dim,), device=dev, dtype=dt)
    dgate = torch.empty(shape, device=dev, dtype=dt) if gate is not None else None
    sh = _NormShape(rows, inner, dim, code, eps, 0, ho, hi, 0, 0, go, gi)
    ws = _workspace(workspace, _bytes("gdr_rms_norm_bwd_workspace_size", sh), dev)
    _call(dev, _entry("gdr_rms_norm_bwd"), sh, hp, gp, wp, dyp, drp, dh.data_ptr(), dw.data_ptr(), _ptr(dgate), ws.data_ptr(),
          ws.numel())
    return dh, dw, dgate


class _NormFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, gate, eps):
        y, _, h = gdr_rms_norm_fwd(x, weight, residual, gate, eps=eps)
        ctx.save_for_backward(x if h is None else h, weight, gate)
        ctx.eps, ctx.added = eps, h is not None
        ctx.set_materialize_grads(False)
        return y, h

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dres):
        h, weight, gate = ctx.saved_tensors
        if dy is None:
            return (dres, None, dres if ctx.added else None, None, None)
        dh, dw, dgate = gdr_rms_norm_bwd(h, weight, dy.contiguous(), gate, None if dres is None else dres.contiguous(),
                                         eps=ctx.eps)
        return dh, dw, (dh if ctx.added else None), dgate, None


def rms_norm(x, weight, residual: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None, eps=1e-6):
    """High-level call: returns (y, h or None) with h = x + residual; differentiable."""
    return _NormFunction.apply(x, weight, residual, gate, eps)


# ------------------------------------------------------- linear recurrence --
def _linear_scan_args(x, r, i, A, cu_seqlens):
    if x.dim() != 3:
        raise GdrError("x must be [B, T, D]")
    shape = tuple(x.shape)
    B, T, D = shape
    if B > _MOST or T > _MOST or D > _MOST:
        _too_long(B=B, T=T, D=D)
    code, dev, ty = _code(x), x.get_device(), x.dtype
    xp, xs = _rows_of(x, "x", shape, ty, dev, 2)
    rp, rs = _rows_of(r, "r", shape, ty, dev, 2)
    ip, ist = _rows_of(i, "i", shape, ty, dev, 2)
    Ap = _dense(A, "A", (D,), torch.float32, dev)
    cu, N = _offsets(cu_seqlens, B, T, x.device)
    return _LinearScanShape(B, T, D, N, code, xs, rs, ist), (xp, rp, ip, Ap), cu, N, dev


def gdr_linear_scan_fwd(x, r, i, A, initial_state=None, cu_seqlens=None, *, output_final_state=False, workspace=None):
    """h = a h + sqrt(1 - a^2) sigmoid(i) x with a = exp(A sigmoid(r)), token by token: x, r, i [B, T, D] (strided), A [D]
    fp32, initial_state [N, D] fp32.  Returns (y, final_state or None)."""
    if _grad_enabled() and (x.requires_grad or r.requires_grad or i.requires_grad or A.requires_grad
                            or (initial_state is not None and initial_state.requires_grad)):
        _no_gradient("gdr_linear_scan_fwd", "linear_scan")
    sh, ptrs, cu, N, dev = _linear_scan_args(x, r, i, A, cu_seqlens)
    hp = _dense(initial_state, "initial_state", (N, sh.D), torch.float32, dev)
    y = torch.empty(*x.shape, device=dev, dtype=x.dtype)
    ht = torch.empty(N, sh.D, device=dev, dtype=torch.float32) if output_final_state else None
    ws = _workspace(workspace, _bytes("gdr_linear_scan_fwd_workspace_size", sh), dev)
    _call(dev, _entry("gdr_linear_scan_fwd"), sh, *ptrs, hp, _ptr(cu), y.data_ptr(), _ptr(ht), ws.data_ptr(), ws.numel())
    return y, ht


def gdr_linear_scan_bwd(x, r, i, A, dy, initial_state=None, dht=None, cu_seqlens=None, *, workspace=None):
    """Backward of gdr_linear_scan_fwd.  Returns (dx, dr, di, dA, dh0); dh0 is None without an initial state."""
    sh, ptrs, cu, N, dev = _linear_scan_args(x, r, i, A, cu_seqlens)
    hp = _dense(initial_state, "initial_state", (N, sh.D), torch.float32, dev)
    dyp = _dense(dy, "dy", tuple(x.shape), x.dtype, dev)
    dhp = _dense(dht, "dht", (N, sh.D), torch.float32, dev)
    dx, dr, di = (torch.empty(x.shape, device=dev, dtype=x.dtype) for _ in range(3))
    dA = torch.empty((sh.D,), device=dev, dtype=torch.float32)
    dh0 = None if initial_state is None else torch.empty((N, sh.D), device=dev, dtype=torch.float32)
    ws = _workspace(workspace, _bytes("gdr_linear_scan_bwd_workspace_size", sh), dev)
    _call(dev, _entry("gdr_linear_scan_bwd"), sh, *ptrs, hp, _ptr(cu), dyp, dhp, dx.data_ptr(), dr.data_ptr(), di.data_ptr(),
          dA.data_ptr(), _ptr(dh0), ws.data_ptr(), ws.numel())
    return dx, dr, di, dA, dh0


def gdr_linear_scan_step(x, r, i, A, state, *, slots=None):
    """One new token per row: x, r, i [rows, D] (strided), A [D] fp32, state [slots, D] fp32, in place.  Returns y
    [rows, D]."""
    if x.dim() != 2:
        raise GdrError("x must be [rows, D]")
    if _grad_enabled() and (x.requires_grad or r.requires_grad or i.requires_grad or A.requires_grad or state.requires_grad):
        _no_gradient("gdr_linear_scan_step")
    shape = x.shape
    rows, D = shape
    if rows > _MOST or D > _MOST:
        _too_long(rows=rows, D=D)
    code, dev, ty = _code(x), x.get_device(), x.dtype
    xp, xs = _rows_of(x, "x", shape, ty, dev, 1)
    rp, rs = _rows_of(r, "r", shape, ty, dev, 1)
    ip, ist = _rows_of(i, "i", shape, ty, dev, 1)
    Ap = _dense(A, "A", (D,), torch.float32, dev)
    sp, n, lp = _pool(state, "state", (D,), torch.float32, dev, rows, slots)
    y = torch.empty(rows, D, device=dev, dtype=ty) if xs else torch.empty_like(x)
    if rows:
        _call(dev, _entry("gdr_linear_scan_step"), _LinearScanShape(rows, 1, D, 0, code, xs, rs, ist), xp, rp, ip, Ap, sp, n, lp,
              y.data_ptr())
        _changed((state,))
    return y


class _LinearScanFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, r, i, A, initial_state, cu_seqlens, output_final_state):
        cu, _ = _offsets(cu_seqlens, x.shape[0], x.shape[1], x.device) if x.dim() == 3 else (None, 0)
        y, ht = gdr_linear_scan_fwd(x, r, i, A, initial_state, cu, output_final_state=output_final_state)
        ctx.save_for_backward(x, r, i, A, initial_state, cu)
        ctx.set_materialize_grads(False)
        return y, ht

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dht):
        x, r, i, A, h0, cu = ctx.saved_tensors
        if dy is None and dht is None:
            return (None,) * 7
        dy = torch.zeros(x.shape, device=x.device, dtype=x.dtype) if dy is None else dy.contiguous()
        dht = None if dht is None else dht.contiguous()
        dx, dr, di, dA, dh0 = gdr_linear_scan_bwd(x, r, i, A, dy, h0, dht, cu)
        return dx, dr, di, dA, dh0, None, None


def linear_scan(x, r, i, A, initial_state=None, output_final_state=False, cu_seqlens=None):
    """High-level call: returns (y, final_state or None); differentiable."""
    return _LinearScanFunction.apply(x, r, i, A, initial_state, cu_seqlens, output_final_state)


# ------------------------------------------------------- norms of a block --
def _flat_rows(t, name, shape, dtype, index):
    """(pointer, row stride) of [..., dim] rows that have one stride (0: dense)."""
    if t is None:
        return None, 0
    if t.shape != shape or t.dtype is not dtype or t.get_device() != index or index < 0:
        _refuse(t, name, shape, dtype, index, False)
    if t.is_contiguous():
        return t.data_ptr(), 0
    st = t.stride()
    if shape[-1] != 1 and st[-1] != 1:
        raise GdrError(f"{name}: the values of a row must be contiguous")
    stride = width = None
    for n, s in zip(reversed(shape[:-1]), reversed(st[:-1])):
        if n == 1:
            continue
        if stride is None:
            stride, width = s, s * n
        elif s != width:
            raise GdrError(f"{name}: the leading dimensions must have one stride")
        else:
            width *= n
    if stride is not None and stride < shape[-1]:
        raise GdrError(f"{name}: rows overlap (expanded tensor): call .contiguous()")
    return t.data_ptr(), stride or 0


def _block_norm_args(x, post_weight, h, pre_weight, gate, scale, eps, h_name):
    if x.dim() < 2:
        raise GdrError("x must be [..., dim] with at least two dimensions")
    shape = x.shape
    dim = shape[-1]
    if dim > _MOST:
        _too_long(dim=dim)
    rows = x.numel() // dim if dim else 0
    code, dev, ty = _code(x), x.get_device(), x.dtype
    xp, xs = _flat_rows(x, "x", shape, ty, dev)
    hp, hs = _flat_rows(h, h_name, shape, ty, dev)
    gp, gs = _flat_rows(gate, "gate", shape, ty, dev)
    post = _dense(post_weight, "post_weight", (dim,), ty, dev)
    pre = _dense(pre_weight, "pre_weight", (dim,), ty, dev)
    sp = _dense(scale, "scale", (dim,), ty, dev)
    return _BlockNormShape(rows, dim, code, eps, xs, hs, gs), (xp, hp, gp, post, pre, sp), dev


def gdr_block_norm_fwd(x, post_weight, residual, pre_weight, gate=None, scale=None, *, eps=1e-6):
    """h = residual + scale * rms_norm(x) * post_weight * silu(gate), y = rms_norm(h) * pre_weight, over the last dimension;
    x, residual and gate [..., dim] (strided), weights and scale [dim].  Returns (y, h)."""
    if _grad_enabled() and (x.requires_grad or post_weight.requires_grad or residual.requires_grad or pre_weight.requires_grad
                            or (gate is not None and gate.requires_grad) or (scale is not None and scale.requires_grad)):
        _no_gradient("gdr_block_norm_fwd", "block_norm")
    sh, ptrs, dev = _block_norm_args(x, post_weight, residual, pre_weight, gate, scale, eps, "residual")
    y = torch.empty(*x.shape, device=dev, dtype=x.dtype)
    h = torch.empty_like(y)
    _call(dev, _entry("gdr_block_norm_fwd"), sh, *ptrs, y.data_ptr(), h.data_ptr())
    return y, h


def gdr_block_norm_bwd(x, post_weight, h, pre_weight, dy, gate=None, scale=None, dres=None, *, eps=1e-6, workspace=None):
    """Backward of gdr_block_norm_fwd at its x and h; dres is the gradient of h from elsewhere.  Returns (dx, dh, dpost,
    dpre, dgate, dscale); dh is the gradient of residual, dgate and dscale are None without a gate or scale."""
    sh, ptrs, dev = _block_norm_args(x, post_weight, h, pre_weight, gate, scale, eps, "h")
    shape, ty, dim = tuple(x.shape), x.dtype, sh.dim
    dyp = _dense(dy, "dy", shape, ty, dev)
    drp = _dense(dres, "dres", shape, ty, dev)
    dx, dh = torch.empty(shape, device=dev, dtype=ty), torch.empty(shape, device=dev, dtype=ty)
    dgate = None if gate is None else torch.empty(shape, device=dev, dtype=ty)
    dpost, dpre = torch.empty((dim,), device=dev, dtype=ty), torch.empty((dim,), device=dev, dtype=ty)
    dscale = None if scale is None else torch.empty((dim,), device=dev, dtype=ty)
    ws = _workspace(workspace, _bytes("gdr_block_norm_bwd_workspace_size", sh), dev)
    _call(dev, _entry("gdr_block_norm_bwd"), sh, *ptrs, dyp, drp, dx.data_ptr(), dh.data_ptr(), _ptr(dgate), dpost.data_ptr(),
          dpre.data_ptr(), _ptr(dscale), ws.data_ptr(), ws.numel())
    return dx, dh, dpost, dpre, dgate, dscale


class _BlockNormFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, post_weight, residual, pre_weight, gate, scale, eps):
        y, h = gdr_block_norm_fwd(x, post_weight, residual, pre_weight, gate, scale, eps=eps)
        ctx.save_for_backward(x, post_weight, h, pre_weight, gate, scale)
        ctx.eps = eps
        ctx.set_materialize_grads(False)
        return y, h

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dres):
        x, post, h, pre, gate, scale = ctx.saved_tensors
        if dy is None and dres is None:
            return (None,) * 7
        dy = torch.zeros(x.shape, device=x.device, dtype=x.dtype) if dy is None else dy.contiguous()
        dres = None if dres is None else dres.contiguous()
        dx, dh, dpost, dpre, dgate, dscale = gdr_block_norm_bwd(x, post, h, pre, dy, gate, scale, dres, eps=ctx.eps)
        return dx, dpost, dh, dpre, dgate, dscale, None


def block_norm(x, post_weight, residual, pre_weight, gate: Optional[torch.Tensor] = None,
               scale: Optional[torch.Tensor] = None, eps=1e-6):
    """High-level call: returns (y, h); differentiable."""
    return _BlockNormFunction.apply(x, post_weight, residual, pre_weight, gate, scale, eps)


# ------------------------------------------------------ products in 8 bits --
def gdr_quantize_rows(x):
    """Rows of x [..., K] (strided) in 8-bit integers.  Returns (q, scales): q [..., K] int8, its rows at multiples of 16
    bytes (a slice of a wider tensor where K is none), scales [...] fp32."""
    if x.dim() < 1 or x.shape[-1] < 1:
        raise GdrError("x must be [..., K] with K positive")
    if _grad_enabled() and x.requires_grad:
        _no_gradient("gdr_quantize_rows")
    shape = x.shape
    K = shape[-1]
    if K > _MOST:
        _too_long(K=K)
    code, dev = _code(x), x.get_device()
    xp, xs = _flat_rows(x, "x", shape, x.dtype, dev)
    pad = -(-K // 16) * 16
    q = torch.empty(*shape[:-1], pad, device=dev, dtype=torch.int8)
    scales = torch.empty(shape[:-1], device=dev, dtype=torch.float32)
    _call(dev, _entry("gdr_quantize_rows"), _QuantizeShape(x.numel() // K, K, code, xs, pad), xp, q.data_ptr(), scales.data_ptr())
    return (q if pad == K else q[..., :K]), scales


def _i8_rows(t, name, shape, index):
    """(pointer, row stride) of int8 rows at multiples of 16 bytes."""
    ptr, stride = _flat_rows(t, name, shape, torch.int8, index)
    K = shape[-1]
    if K % 16 == 0:
        return ptr, stride
    pad = -(-K // 16) * 16
    rows = t.numel() // K
    if rows == 0:
        return ptr, 0
    if stride == 0 and rows > 1:
        raise GdrError(f"{name}: rows of {K} values must be at multiples of 16 bytes (pad the rows and slice)")
    stride = stride or pad
    # the last row is read up to the end of its last 16 bytes
    if t.storage_offset() + (rows - 1) * stride + pad > t.untyped_storage().nbytes():
        raise GdrError(f"{name}: the last row's storage must reach to a multiple of 16 bytes")
    return ptr, stride


def gdr_matmul_i8(q, scales, weight, weight_scales, bias=None, *, dtype=torch.bfloat16):
    """y[m, n] = (q[m] . weight[n]) scales[m] weight_scales[n] + bias[n]: q [..., K] and weight [N, K] int8 with rows at
    multiples of 16 bytes, scales [...], weight_scales [N] and bias [N] fp32.  Returns y [..., N] of the dtype."""
    if q.dim() < 1 or weight.dim() != 2:
        raise GdrError("q must be [..., K] and weight [N, K]")
    if _grad_enabled() and (scales.requires_grad or weight_scales.requires_grad or (bias is not None and bias.requires_grad)):
        _no_gradient("gdr_matmul_i8")
    shape = q.shape
    N, K = weight.shape
    if K < 1 or shape[-1] != K:
        raise GdrError(f"shape mismatch: q is {tuple(shape)}, weight {tuple(weight.shape)}")
    M = q.numel() // K
    if M > _MOST or N > _MOST or K > _MOST:
        _too_long(M=M, N=N, K=K)
    code = GDR_BF16 if dtype is torch.bfloat16 else GDR_F32 if dtype is torch.float32 else None
    if code is None:
        raise GdrError(f"unsupported dtype {dtype} (bfloat16 or float32)")
    dev = q.get_device()
    qp, qs = _i8_rows(q, "q", shape, dev)
    wp, ws = _i8_rows(weight, "weight", weight.shape, dev)
    sp = _dense(scales, "scales", shape[:-1], torch.float32, dev)
    wsp = _dense(weight_scales, "weight_scales", (N,), torch.float32, dev)
    bp = _dense(bias, "bias", (N,), torch.float32, dev)
    y = torch.empty(*shape[:-1], N, device=dev, dtype=dtype)
    _call(dev, _entry("gdr_matmul_i8"), _MatmulI8Shape(M, N, K, code, qs, ws), qp, sp, wp, wsp, bp, y.data_ptr())
    return y
