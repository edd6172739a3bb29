"""Python face of the operators inside a gated feed-forward block
(include/fp8ffn.h).

  * both projections, the activation and their product in one call, dense or
    per expert: ``fp8_block_gemm_gated``, ``fp8_block_grouped_gemm_gated`` and,
    with the result quantized and the projections kept in 8 bits,
    ``fp8_block_gemm_gated_quant_1x128``,
    ``fp8_block_grouped_gemm_gated_quant_1x128``;
  * its gradient from the kept projections: ``fp8_gated_grad``,
    ``fp8_gated_grad_quant_1x128``, ``fp8_gated_grad_quant``;
  * 8-bit checkpoints read back and turned: ``fp8_dequant_act_1x128``,
    ``fp8_requant_act_128x1_t``;
  * the input gradient per expert: ``fp8_block_grouped_gemm_dgrad``.

``_pow2`` forms take and write power-of-two scales.  As in ``moe``: argument
marshalling only, outputs and workspaces are allocated when not given, shapes
are checked before anything is launched, outputs and workspaces must not share
memory with inputs or each other, no autograd graph is built, and work goes to
``stream`` or to the current stream of the tensors' device.
"""
from __future__ import annotations

import ctypes

import torch

from . import binding
from .binding import Fp8Error
from .moe import (_BF16, _CODES, _F32, _INT, _U8, _WIDE, _dense, _disjoint, _dtype, _Place, _ptr,
                  _rows, _tensor, _workspace_tensor)

FP8_ACT_SILU = 0
FP8_ACT_GELU_TANH = 1

_ACTIVATIONS = {"silu": FP8_ACT_SILU, "gelu_tanh": FP8_ACT_GELU_TANH, FP8_ACT_SILU: FP8_ACT_SILU,
                FP8_ACT_GELU_TANH: FP8_ACT_GELU_TANH}

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I = ctypes.c_int
_Z = ctypes.c_size_t
_GATED = ([_P, _P, _P, _P, _I, _I64, _I64, _I64, _P, _I, _P, _Z, _P], _I)
_GATED_QUANT = ([_P, _P, _P, _P, _I, _I64, _I64, _I64, _P, _P, _P, _P, _P, _Z, _P], _I)
_GROUPED = ([_P, _P, _P, _P, _P, _I64, _I, _I64, _I64, _I64, _P, _I, _P, _Z, _P], _I)
_GROUPED_QUANT = ([_P, _P, _P, _P, _P, _I64, _I, _I64, _I64, _I64, _P, _P, _P, _P, _P, _Z, _P],
                  _I)
_GRAD = [_P, _I, _I64, _P, _I64, _P, _I, _I64, _I64]
_GRAD_QUANT = (_GRAD + [_P, _P, _P, _P, _P, _P, _P], _I)
_REQUANT = ([_P, _P, _I64, _I64, _P, _P, _P], _I)
_DGRAD = ([_P, _P, _P, _P, _P, _I64, _I64, _P, _I, _I64, _I64, _P], _I)
_SIGNATURES = {
    "fp8_block_gemm_gated": _GATED,
    "fp8_block_gemm_gated_pow2": _GATED,
    "fp8_block_gemm_gated_quant_1x128": _GATED_QUANT,
    "fp8_block_gemm_gated_quant_1x128_pow2": _GATED_QUANT,
    "fp8_gated_gemm_workspace_bytes": ([_I64, _I64, _I64], _Z),
    "fp8_grouped_gated_gemm_workspace_bytes": ([_I64, _I64, _I64, _I64], _Z),
    "fp8_block_grouped_gemm_gated": _GROUPED,
    "fp8_block_grouped_gemm_gated_pow2": _GROUPED,
    "fp8_block_grouped_gemm_gated_quant_1x128": _GROUPED_QUANT,
    "fp8_block_grouped_gemm_gated_quant_1x128_pow2": _GROUPED_QUANT,
    "fp8_gated_grad": (_GRAD + [_P, _I, _P], _I),
    "fp8_gated_grad_quant": _GRAD_QUANT,
    "fp8_gated_grad_quant_pow2": _GRAD_QUANT,
    "fp8_dequant_act_1x128": ([_P, _P, _I64, _I64, _P, _I, _P], _I),
    "fp8_requant_act_128x1_t": _REQUANT,
    "fp8_requant_act_128x1_t_pow2": _REQUANT,
    "fp8_block_grouped_gemm_dgrad": _DGRAD,
    "fp8_block_grouped_gemm_dgrad_pow2": _DGRAD,
}

_functions = {}


def _fn(name):
    f = _functions.get(name)
    if f is None:
        f = getattr(binding.lib(), name)
        f.argtypes, f.restype = _SIGNATURES[name]
        _functions[name] = f
    return f


def _call(name, *args):
    f = _functions.get(name) or _fn(name)
    status = f(*args)
    if status:
        raise Fp8Error(status, name)


def _activation(activation):
    try:
        return _ACTIVATIONS[activation]
    except (KeyError, TypeError):
        raise ValueError(f"unsupported activation {activation}") from None


def _multiple(n, name):
    if n % 128:
        raise ValueError(f"{name} must be a multiple of 128, got {n}")


def _product(x, x_scales, w, w_scales, group_offsets, x_name, x_axis, w_axes):
    """Checks the operands of a product: x [rows][x_axis], w [w_axes] (one more
    axis in front per expert); returns (rows, x's width, w's last two sizes)."""
    _tensor(x, x_name, _U8)
    if x.dim() != 2:
        raise ValueError(f"{x_name} must be 2-dimensional, got shape {tuple(x.shape)}")
    if not x.is_contiguous():
        raise ValueError(f"{x_name} must be contiguous")
    _tensor(w, "w", _U8)
    lead = 0 if group_offsets is None else 1
    if w.dim() != 2 + lead:
        raise ValueError(f"w must have shape ({'experts, ' if lead else ''}{w_axes}), got "
                         f"{tuple(w.shape)}")
    if not w.is_contiguous():
        raise ValueError("w must be contiguous")
    rows, width = x.shape
    _multiple(width, x_axis)
    for n in w.shape[lead:]:
        _multiple(n, "w's sizes")
    _dense(x_scales, f"{x_name}_scales", (rows, width // 128), _F32)
    _dense(w_scales, "w_scales", (*w.shape[:lead], w.shape[-2] // 128, w.shape[-1] // 128), _F32)
    if lead:
        _dense(group_offsets, "group_offsets", (w.shape[0] + 1,), _INT)
    return rows, width, w.shape[-2], w.shape[-1]


def _gated_operands(a, a_scales, w, w_scales, group_offsets):
    """(M, I, K) of a gated product."""
    M, K, two, inner = _product(a, a_scales, w, w_scales, group_offsets, "a", "K", "2 I, K")
    if inner != K:
        raise ValueError(f"w must have {K} columns, got {inner}")
    if two % 256:
        raise ValueError(f"w must have two parts of a multiple of 128 rows, got {two} rows")
    return M, two // 2, K


def fp8_gated_gemm_workspace_bytes(rows: int, inner: int, width: int) -> int:
    return int(_fn("fp8_gated_gemm_workspace_bytes")(rows, inner, width))


def fp8_grouped_gated_gemm_workspace_bytes(rows: int, experts: int, inner: int,
                                           width: int) -> int:
    return int(_fn("fp8_grouped_gated_gemm_workspace_bytes")(rows, experts, inner, width))


_PRODUCT = "a a_scales w w_scales group_offsets"


def _gated(name, a, a_scales, w, w_scales, group_offsets, activation, out_dtype, out, workspace,
           stream):
    act = _activation(activation)
    dtype = _dtype(out_dtype)
    M, I, K = _gated_operands(a, a_scales, w, w_scales, group_offsets)
    inputs = (a, a_scales, w, w_scales, group_offsets)
    if out is not None:
        _dense(out, "out", (M, I), (dtype,))
    if workspace is not None:
        _workspace_tensor(workspace)
    if out is not None or workspace is not None:
        _disjoint("out workspace", (out, workspace), _PRODUCT, inputs)
    with _Place(stream, _PRODUCT + " out workspace", *inputs, out, workspace) as p:
        if out is None:
            out = p.empty((M, I), dtype)
        if group_offsets is None:
            ws, ws_bytes = p.workspace(workspace, fp8_gated_gemm_workspace_bytes(M, I, K))
            _call(name, a.data_ptr(), a_scales.data_ptr(), w.data_ptr(), w_scales.data_ptr(), act,
                  M, I, K, out.data_ptr(), _CODES[dtype], ws, ws_bytes, p.handle)
        else:
            ws, ws_bytes = p.workspace(
                workspace, fp8_grouped_gated_gemm_workspace_bytes(M, w.shape[0], I, K))
            _call(name, a.data_ptr(), a_scales.data_ptr(), w.data_ptr(), w_scales.data_ptr(),
                  group_offsets.data_ptr(), w.shape[0], act, M, I, K, out.data_ptr(),
                  _CODES[dtype], ws, ws_bytes, p.handle)
    return out


def _gated_quant(name, a, a_scales, w, w_scales, group_offsets, activation, checkpoint, q, scales,
                 h, h_scales, workspace, stream):
    act = _activation(activation)
    M, I, K = _gated_operands(a, a_scales, w, w_scales, group_offsets)
    inputs = (a, a_scales, w, w_scales, group_offsets)
    if not checkpoint and (h is not None or h_scales is not None):
        raise ValueError("h or h_scales given without checkpoint")
    for what, t, shape, dtypes in (("q", q, (M, I), _U8), ("scales", scales, (M, I // 128), _F32),
                                   ("h", h, (M, 2 * I), _U8),
                                   ("h_scales", h_scales, (M, I // 64), _F32)):
        if t is not None:
            _dense(t, what, shape, dtypes)
    _workspace_tensor(workspace)
    _disjoint("q scales h h_scales workspace", (q, scales, h, h_scales, workspace), _PRODUCT,
              inputs)
    with _Place(stream, _PRODUCT + " q scales h h_scales workspace", *inputs, q, scales, h,
                h_scales, workspace) as p:
        if q is None:
            q = p.empty((M, I), torch.uint8)
        if scales is None:
            scales = p.empty((M, I // 128), torch.float32)
        if checkpoint:
            if h is None:
                h = p.empty((M, 2 * I), torch.uint8)
            if h_scales is None:
                h_scales = p.empty((M, I // 64), torch.float32)
        if group_offsets is None:
            ws, ws_bytes = p.workspace(workspace, fp8_gated_gemm_workspace_bytes(M, I, K))
            _call(name, a.data_ptr(), a_scales.data_ptr(), w.data_ptr(), w_scales.data_ptr(), act,
                  M, I, K, q.data_ptr(), scales.data_ptr(), _ptr(h), _ptr(h_scales), ws, ws_bytes,
                  p.handle)
        else:
            ws, ws_bytes = p.workspace(
                workspace, fp8_grouped_gated_gemm_workspace_bytes(M, w.shape[0], I, K))
            _call(name, a.data_ptr(), a_scales.data_ptr(), w.data_ptr(), w_scales.data_ptr(),
                  group_offsets.data_ptr(), w.shape[0], act, M, I, K, q.data_ptr(),
                  scales.data_ptr(), _ptr(h), _ptr(h_scales), ws, ws_bytes, p.handle)
    return q, scales, h, h_scales


def fp8_block_gemm_gated(a, a_scales, w, w_scales, activation="silu", out_dtype="bf16", out=None,
                         workspace=None, stream=None):
    """out [M][I] = act(g) u with [g | u] = a w^T: a E4M3 [M][K] with a_scales
    [M][K/128], w E4M3 [2 I][K] (the gate's rows first) with w_scales [2 I /
    128][K/128]; activation "silu" or "gelu_tanh".  K and I are multiples of
    128."""
    return _gated("fp8_block_gemm_gated", a, a_scales, w, w_scales, None, activation, out_dtype,
                  out, workspace, stream)


def fp8_block_gemm_gated_pow2(a, a_scales, w, w_scales, activation="silu", out_dtype="bf16",
                              out=None, workspace=None, stream=None):
    """As fp8_block_gemm_gated, for power-of-two scales."""
    return _gated("fp8_block_gemm_gated_pow2", a, a_scales, w, w_scales, None, activation,
                  out_dtype, out, workspace, stream)


def fp8_block_gemm_gated_quant_1x128(a, a_scales, w, w_scales, activation="silu",
                                     checkpoint=False, q=None, scales=None, h=None, h_scales=None,
                                     workspace=None, stream=None):
    """As fp8_block_gemm_gated with the result quantized 1x128 from its fp32
    values, and with ``checkpoint`` the projections too: (q uint8 [M][I] E4M3,
    scales fp32 [M][I/128], h uint8 [M][2 I] E4M3 of [g | u], h_scales fp32 [M][2
    I / 128]), h and h_scales None without it."""
    return _gated_quant("fp8_block_gemm_gated_quant_1x128", a, a_scales, w, w_scales, None,
                        activation, checkpoint, q, scales, h, h_scales, workspace, stream)


def fp8_block_gemm_gated_quant_1x128_pow2(a, a_scales, w, w_scales, activation="silu",
                                          checkpoint=False, q=None, scales=None, h=None,
                                          h_scales=None, workspace=None, stream=None):
    """As fp8_block_gemm_gated_quant_1x128, power-of-two scales in and out."""
    return _gated_quant("fp8_block_gemm_gated_quant_1x128_pow2", a, a_scales, w, w_scales, None,
                        activation, checkpoint, q, scales, h, h_scales, workspace, stream)


def _offsets(group_offsets):
    _tensor(group_offsets, "group_offsets", _INT)
    return group_offsets


def fp8_block_grouped_gemm_gated(a, a_scales, w, w_scales, group_offsets, activation="silu",
                                 out_dtype="bf16", out=None, workspace=None, stream=None):
    """fp8_block_gemm_gated per expert over expert-sorted rows: a [T][K], w
    [E][2 I][K], w_scales [E][2 I / 128][K/128], group_offsets int32 [E+1] on the
    GPU.  Rows outside every expert's range are left as they are."""
    return _gated("fp8_block_grouped_gemm_gated", a, a_scales, w, w_scales,
                  _offsets(group_offsets), activation, out_dtype, out, workspace, stream)


def fp8_block_grouped_gemm_gated_pow2(a, a_scales, w, w_scales, group_offsets, activation="silu",
                                      out_dtype="bf16", out=None, workspace=None, stream=None):
    """As fp8_block_grouped_gemm_gated, for power-of-two scales."""
    return _gated("fp8_block_grouped_gemm_gated_pow2", a, a_scales, w, w_scales,
                  _offsets(group_offsets), activation, out_dtype, out, workspace, stream)


def fp8_block_grouped_gemm_gated_quant_1x128(a, a_scales, w, w_scales, group_offsets,
                                             activation="silu", checkpoint=False, q=None,
                                             scales=None, h=None, h_scales=None,
                                             workspace=None, stream=None):
    """fp8_block_gemm_gated_quant_1x128 per expert (see
    fp8_block_grouped_gemm_gated)."""
    return _gated_quant("fp8_block_grouped_gemm_gated_quant_1x128", a, a_scales, w, w_scales,
                        _offsets(group_offsets), activation, checkpoint, q, scales, h, h_scales,
                        workspace, stream)


def fp8_block_grouped_gemm_gated_quant_1x128_pow2(a, a_scales, w, w_scales, group_offsets,
                                                  activation="silu", checkpoint=False, q=None,
                                                  scales=None, h=None, h_scales=None,
                                                  workspace=None, stream=None):
    """As fp8_block_grouped_gemm_gated_quant_1x128, power-of-two scales in and
    out."""
    return _gated_quant("fp8_block_grouped_gemm_gated_quant_1x128_pow2", a, a_scales, w, w_scales,
                        _offsets(group_offsets), activation, checkpoint, q, scales, h, h_scales,
                        workspace, stream)


# ---- gradient of the activation and the product -----------------------------------

def _grad_inputs(da, h, h_scales):
    """(M, I, row stride of da, of h)."""
    ld_da = _rows(da, "da", _WIDE)
    M, I = da.shape
    _multiple(I, "da's width")
    ld_h = _rows(h, "h", _BF16 if h_scales is None else _U8, (M, 2 * I))
    if h_scales is not None:
        _dense(h_scales, "h_scales", (M, I // 64), _F32)
    return M, I, ld_da, ld_h


def fp8_gated_grad(da, h, h_scales=None, activation="silu", out_dtype="bf16", dh=None,
                   stream=None):
    """dh [M][2 I] = [da u act'(g) | da act(g)] from da [M][I] (bf16 or fp32) and
    the projections h = [g | u] [M][2 I], uint8 E4M3 with h_scales [M][2 I / 128]
    (what fp8_block_gemm_gated_quant_1x128 kept) or bf16 without."""
    act, dtype = _activation(activation), _dtype(out_dtype)
    M, I, ld_da, ld_h = _grad_inputs(da, h, h_scales)
    if dh is not None:
        _dense(dh, "dh", (M, 2 * I), (dtype,))
        _disjoint("dh", (dh,), "da h h_scales", (da, h, h_scales))
    with _Place(stream, "da h h_scales dh", da, h, h_scales, dh) as p:
        if dh is None:
            dh = p.empty((M, 2 * I), dtype)
        _call("fp8_gated_grad", da.data_ptr(), _CODES[da.dtype], ld_da, h.data_ptr(), ld_h,
              _ptr(h_scales), act, M, I, dh.data_ptr(), _CODES[dtype], p.handle)
    return dh


_TURNED = "q scales q_t scales_t a_t a_scales_t"


def _grad_quant(name, turned, da, h, h_scales, activation, outputs, stream):
    act = _activation(activation)
    M, I, ld_da, ld_h = _grad_inputs(da, h, h_scales)
    G = (M + 127) // 128
    shapes = ((M, 2 * I), (M, I // 64), (2 * I, M), (2 * I, G), (I, M), (I, G))
    wanted = 6 if turned else 2
    for what, t, shape, dtypes in zip(_TURNED.split(), outputs, shapes, (_U8, _F32) * 3):
        if t is not None:
            _dense(t, what, shape, dtypes)
    _disjoint(_TURNED, outputs, "da h h_scales", (da, h, h_scales))
    with _Place(stream, "da h h_scales " + _TURNED, da, h, h_scales, *outputs) as p:
        outs = [p.empty(shapes[i], torch.float32 if i % 2 else torch.uint8)
                if outputs[i] is None and i < wanted else outputs[i] for i in range(6)]
        _call(name, da.data_ptr(), _CODES[da.dtype], ld_da, h.data_ptr(), ld_h, _ptr(h_scales),
              act, M, I, *(_ptr(t) for t in outs), p.handle)
    return tuple(outs[:wanted])


def fp8_gated_grad_quant_1x128(da, h, h_scales=None, activation="silu", q=None, scales=None,
                               stream=None):
    """fp8_gated_grad quantized 1x128 from its fp32 values, for the input
    gradient: (q uint8 [M][2 I], scales fp32 [M][2 I / 128])."""
    return _grad_quant("fp8_gated_grad_quant", False, da, h, h_scales, activation,
                       (q, scales, None, None, None, None), stream)


def fp8_gated_grad_quant_1x128_pow2(da, h, h_scales=None, activation="silu", q=None, scales=None,
                                    stream=None):
    """As fp8_gated_grad_quant_1x128 with power-of-two scales out."""
    return _grad_quant("fp8_gated_grad_quant_pow2", False, da, h, h_scales, activation,
                       (q, scales, None, None, None, None), stream)


def fp8_gated_grad_quant(da, h, h_scales=None, activation="silu", q=None, scales=None, q_t=None,
                         scales_t=None, a_t=None, a_scales_t=None, stream=None):
    """All that the products of a backward pass take, in one pass: (q [M][2 I],
    scales [M][2 I / 128]: fp8_gated_grad quantized 1x128, for the input
    gradient; q_t [2 I][M], scales_t [2 I][ceil(M/128)]: the same in 128x1 groups
    and transposed, a_t [I][M], a_scales_t [I][ceil(M/128)]: act(g) u so, for the
    weight gradients)."""
    return _grad_quant("fp8_gated_grad_quant", True, da, h, h_scales, activation,
                       (q, scales, q_t, scales_t, a_t, a_scales_t), stream)


def fp8_gated_grad_quant_pow2(da, h, h_scales=None, activation="silu", q=None, scales=None,
                              q_t=None, scales_t=None, a_t=None, a_scales_t=None, stream=None):
    """As fp8_gated_grad_quant with power-of-two scales out."""
    return _grad_quant("fp8_gated_grad_quant_pow2", True, da, h, h_scales, activation,
                       (q, scales, q_t, scales_t, a_t, a_scales_t), stream)


# ---- 8-bit checkpoints ---------------------------------------------------------------

def _stored(q, scales):
    _tensor(q, "q", _U8)
    if q.dim() != 2:
        raise ValueError(f"q must be 2-dimensional, got shape {tuple(q.shape)}")
    if not q.is_contiguous():
        raise ValueError("q must be contiguous")
    M, K = q.shape
    _dense(scales, "scales", (M, (K + 127) // 128), _F32)
    return M, K


def fp8_dequant_act_1x128(q, scales, out_dtype="bf16", x=None, stream=None):
    """x [M][K] of out_dtype: what E4M3 q [M][K] with 1x128 scales
    [M][ceil(K/128)] stands for."""
    dtype = _dtype(out_dtype)
    M, K = _stored(q, scales)
    if x is not None:
        _dense(x, "x", (M, K), (dtype,))
        _disjoint("x", (x,), "q scales", (q, scales))
    with _Place(stream, "q scales x", q, scales, x) as p:
        if x is None:
            x = p.empty((M, K), dtype)
        _call("fp8_dequant_act_1x128", q.data_ptr(), scales.data_ptr(), M, K, x.data_ptr(),
              _CODES[dtype], p.handle)
    return x


def _requant(name, q, scales, q_t, scales_t, stream):
    M, K = _stored(q, scales)
    G = (M + 127) // 128
    if q_t is not None:
        _dense(q_t, "q_t", (K, M), _U8)
    if scales_t is not None:
        _dense(scales_t, "scales_t", (K, G), _F32)
    _disjoint("q_t scales_t", (q_t, scales_t), "q scales", (q, scales))
    with _Place(stream, "q scales q_t scales_t", q, scales, q_t, scales_t) as p:
        if q_t is None:
            q_t = p.empty((K, M), torch.uint8)
        if scales_t is None:
            scales_t = p.empty((K, G), torch.float32)
        _call(name, q.data_ptr(), scales.data_ptr(), M, K, q_t.data_ptr(), scales_t.data_ptr(),
              p.handle)
    return q_t, scales_t


def fp8_requant_act_128x1_t(q, scales, q_t=None, scales_t=None, stream=None):
    """E4M3 q [M][K] with 1x128 scales, turned for a weight gradient: (q_t uint8
    [K][M], scales_t fp32 [K][ceil(M/128)]), as fp8_quant_act_128x1_t gives them
    for the values that q and scales stand for."""
    return _requant("fp8_requant_act_128x1_t", q, scales, q_t, scales_t, stream)


def fp8_requant_act_128x1_t_pow2(q, scales, q_t=None, scales_t=None, stream=None):
    """As fp8_requant_act_128x1_t with power-of-two scales out."""
    return _requant("fp8_requant_act_128x1_t_pow2", q, scales, q_t, scales_t, stream)


# ---- input gradient per expert ---------------------------------------------------------

def _grouped_dgrad(name, dy, dy_scales, w, w_scales, group_offsets, out_dtype, dx, stream):
    dtype = _dtype(out_dtype)
    T, N, inner, K = _product(dy, dy_scales, w, w_scales, _offsets(group_offsets), "dy", "N",
                              "N, K")
    if inner != N:
        raise ValueError(f"w must have {N} rows per expert, got {inner}")
    inputs = (dy, dy_scales, w, w_scales, group_offsets)
    if dx is not None:
        _dense(dx, "dx", (T, K), (dtype,))
        _disjoint("dx", (dx,), "dy dy_scales w w_scales group_offsets", inputs)
    with _Place(stream, "dy dy_scales w w_scales group_offsets dx", *inputs, dx) as p:
        if dx is None:
            dx = p.empty((T, K), dtype)
        _call(name, dy.data_ptr(), dy_scales.data_ptr(), w.data_ptr(), w_scales.data_ptr(),
              group_offsets.data_ptr(), w.shape[0], T, dx.data_ptr(), _CODES[dtype], N, K,
              p.handle)
    return dx


def fp8_block_grouped_gemm_dgrad(dy, dy_scales, w, w_scales, group_offsets, out_dtype="bf16",
                                 dx=None, stream=None):
    """dx [T][K] = dy [T][N] W[e] for the rows of each expert e: dy E4M3 with
    scales [T][N/128], w the forward weights E4M3 [E][N][K] with scales
    [E][N/128][K/128], read transposed inside the product; group_offsets int32
    [E+1] on the GPU.  Rows outside every expert's range are left as they
    are."""
    return _grouped_dgrad("fp8_block_grouped_gemm_dgrad", dy, dy_scales, w, w_scales,
                          group_offsets, out_dtype, dx, stream)


def fp8_block_grouped_gemm_dgrad_pow2(dy, dy_scales, w, w_scales, group_offsets,
                                      out_dtype="bf16", dx=None, stream=None):
    """As fp8_block_grouped_gemm_dgrad, for power-of-two scales."""
    return _grouped_dgrad("fp8_block_grouped_gemm_dgrad_pow2", dy, dy_scales, w, w_scales,
                          group_offsets, out_dtype, dx, stream)
