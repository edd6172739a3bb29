"""Python face of the operators around the expert products (include/fp8moe.h).

  * tokens sorted by expert and back: ``fp8_moe_sort``, ``fp8_moe_dispatch``,
    ``fp8_moe_dispatch_quant_1x128``, the two in one call
    (``fp8_moe_sort_dispatch``, ``fp8_moe_sort_dispatch_quant_1x128``),
    ``fp8_moe_combine`` and the gradients ``fp8_moe_dispatch_grad`` and
    ``fp8_moe_combine_grad``;
  * norms round a block with its gate and residual scale:
    ``fp8_norm_residual``, ``fp8_norm_residual_quant_1x128``,
    ``fp8_norm_residual_grad``;
  * 4-bit weights: ``fp8_w4_quant_1x128``, ``fp8_w4_quant_1x32``,
    ``fp8_w4_matvec``, ``fp8_w4_grouped_matvec``.

Results carry no autograd graph, whatever the inputs' ``requires_grad``: the
gradients are the ``_grad`` calls.

As in ``binding``: argument marshalling only, outputs and workspaces are
allocated when not given, and shapes are checked before anything is launched,
because the kernels index every buffer by the sizes they are given; outputs
and workspaces must not share memory with inputs or each other (but a new
residual stream or sum may be written over the old one).  Input matrices may
have any row stride (``x[:, :h]``, ``x.expand(t, -1)``) as long as a row's
values are adjacent; everything else must be contiguous.

Work goes to ``stream``, or to the current stream of the tensors' device.
With a ``stream`` of its own, outputs and workspaces are allocated on that
stream, and every tensor is recorded on it, so that memory freed while the
work is pending is not handed out again before it is done.
"""
from __future__ import annotations

import ctypes

import torch

from . import binding
from .binding import FP8_OUT_BF16, FP8_OUT_F32, Fp8Error

FP8_W4_F32_1X128 = 0
FP8_W4_E8M0_1X32 = 1

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I = ctypes.c_int
_F = ctypes.c_float
_Z = ctypes.c_size_t
_NORM = [_P, _I, _I64, _P, _I, _I64, _P, _P, _P, _I, _I64, _I64, _I64, _I, _F, _F, _F, _P, _P]
_SORT_QUANT = [_P, _I64, _I64, _I64, _P, _I, _I64, _I64, _P, _P, _P, _P, _P, _P, _Z, _P]
_DISPATCH_QUANT = [_P, _I64, _I64, _I64, _P, _I64, _P, _P, _I64, _P]
_SIGNATURES = {
    "fp8_moe_sort": ([_P, _I, _I64, _I64, _I64, _P, _P, _P, _P, _Z, _P], _I),
    "fp8_moe_sort_workspace_bytes": ([_I64, _I64, _I64], _Z),
    "fp8_moe_dispatch": ([_P, _I, _I64, _P, _I64, _I64, _I64, _I64, _P, _I64, _P, _P, _I64, _P],
                         _I),
    "fp8_moe_dispatch_quant_1x128": (_DISPATCH_QUANT, _I),
    "fp8_moe_dispatch_quant_1x128_pow2": (_DISPATCH_QUANT, _I),
    "fp8_moe_sort_dispatch": ([_P, _I, _I64, _I64, _I64, _P, _I, _I64, _I64, _P, _P, _P, _P, _P,
                               _Z, _P], _I),
    "fp8_moe_sort_dispatch_quant_1x128": (_SORT_QUANT, _I),
    "fp8_moe_sort_dispatch_quant_1x128_pow2": (_SORT_QUANT, _I),
    "fp8_moe_dispatch_grad": ([_P, _I, _I64, _I64, _P, _I64, _I64, _I64, _P, _I, _P], _I),
    "fp8_moe_combine": ([_P, _I, _I64, _I64, _P, _P, _I64, _I64, _I64, _P, _I64, _P, _I, _P],
                        _I),
    "fp8_moe_combine_grad": ([_P, _I64, _P, _I64, _I, _I64, _P, _P, _I64, _I64, _I64, _P, _P,
                              _P], _I),
    "fp8_norm_residual": (_NORM + [_P, _P, _P], _I),
    "fp8_norm_residual_quant_1x128": (_NORM + [_P, _P, _P, _P, _P], _I),
    "fp8_norm_residual_quant_1x128_pow2": (_NORM + [_P, _P, _P, _P, _P], _I),
    "fp8_norm_residual_grad": ([_P, _I64, _P, _I64, _P, _I, _I64, _P, _I, _I64, _P, _P, _P, _P,
                                _P, _I, _I64, _I64, _I64, _I, _F, _F, _P, _P, _P, _P, _P, _P,
                                _Z, _P], _I),
    "fp8_norm_residual_grad_workspace_bytes": ([_I64, _I64, _I64], _Z),
    "fp8_w4_quant_1x128": ([_P, _I64, _I64, _P, _P, _P], _I),
    "fp8_w4_quant_1x32": ([_P, _I64, _I64, _P, _P, _P], _I),
    "fp8_w4_matvec": ([_P, _I64, _P, _P, _I, _I64, _I64, _I64, _P, _I, _P], _I),
    "fp8_w4_grouped_matvec": ([_P, _I64, _P, _P, _I, _P, _I64, _I64, _I64, _I64, _P, _I, _P],
                              _I),
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


_CODES = {torch.float32: FP8_OUT_F32, torch.bfloat16: FP8_OUT_BF16}
_NAMES = {"f32": torch.float32, "bf16": torch.bfloat16, FP8_OUT_F32: torch.float32,
          FP8_OUT_BF16: torch.bfloat16, torch.float32: torch.float32,
          torch.bfloat16: torch.bfloat16}


def _dtype(out_dtype):
    try:
        return _NAMES[out_dtype]
    except (KeyError, TypeError):
        raise ValueError(f"unsupported out_dtype {out_dtype}") from None


def _tensor(t, name, dtypes):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")


def _dense(t, name, shape, dtypes):
    """A contiguous tensor of that shape and type."""
    _tensor(t, name, dtypes)
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _rows(t, name, dtypes, shape=None):
    """A matrix whose rows are contiguous, any stride between them; returns
    that stride."""
    _tensor(t, name, dtypes)
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-dimensional, got shape {tuple(t.shape)}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.stride(1) != 1 and t.shape[1] > 1 and t.shape[0] > 0:
        raise ValueError(f"{name} must have adjacent values in a row")
    return t.stride(0)


def _disjoint(out_names, outputs, in_names, inputs):
    """Refuse an output (or workspace) whose memory is an input's or another
    output's: workgroups read inputs while others have begun to write.
    Tensors or None, the outputs contiguous; names in one string each."""
    given, top = [], 0
    for i, t in enumerate(outputs):
        if t is None:
            continue
        a0 = t.data_ptr()
        a1 = a0 + t.nbytes
        if a0 == a1:
            continue
        for b0, b1, j in given:
            if a0 < b1 and b0 < a1:
                _shared(out_names, i, out_names, j)
        given.append((a0, a1, i))
        top = a1 if a1 > top else top
    if not given:
        return
    for j, t in enumerate(inputs):
        if t is None:
            continue
        b0 = t.data_ptr()
        if b0 >= top:  # behind every output
            continue
        size = t.nbytes
        if size == 0:
            continue
        b1 = b0 + (size if t.is_contiguous() else t.element_size() * (
            1 + sum((n - 1) * s for n, s in zip(t.shape, t.stride()))))
        for a0, a1, i in given:
            if b0 < a1 and a0 < b1:
                _shared(out_names, i, in_names, j)


def _shared(names, i, others, j):
    raise ValueError(f"{names.split()[i]} must not share memory with {others.split()[j]}")


def _plain_empty(shape, strides, dtype):
    return torch.empty_strided(shape, strides, dtype=dtype, device="cuda")


# A call on few tokens takes as long on the host as on the GPU.  These are what
# torch's own compiled programs call: the current stream's handle without a
# Stream object (0.1 us against 2), an allocation on the current device without
# torch.empty's argument parsing (0.8 us against 1.6).
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch.cuda.current_device
try:
    from torch._C._dynamo.guards import _empty_strided_cuda as _empty
except ImportError:
    _empty = _plain_empty


class _Place:
    """Where a call runs: checks that every tensor is on one GPU, makes that
    device and the stream current while outputs are allocated and the work is
    enqueued, and gives the stream's handle."""

    __slots__ = ("device", "stream", "handle", "tensors", "outer", "scratch")

    def __init__(self, stream, names, *tensors):
        device = None
        for t in tensors:
            if t is None:
                continue
            if not t.is_cuda:
                raise ValueError(f"{self._name(names, tensors, t)} must be on the GPU")
            if device is None:
                device = t.device
            elif t.device != device:
                raise ValueError(f"{self._name(names, tensors, t)} must be on {device}, got "
                                 f"{t.device}")
        if stream is not None and stream.device != device:
            raise ValueError(f"stream must be on {device}, got {stream.device}")
        self.device = device
        self.stream = stream
        self.tensors = tensors

    @staticmethod
    def _name(names, tensors, t):
        return next(n for n, u in zip(names.split(), tensors) if u is t)

    def __enter__(self):
        self.outer = None
        index = self.device.index
        if self.stream is not None:
            self.outer = torch.cuda.stream(self.stream)
            self.outer.__enter__()
            for t in self.tensors:
                if t is not None:
                    t.record_stream(self.stream)
        elif index != _current_device():
            self.outer = torch.cuda.device(self.device)
            self.outer.__enter__()
        self.handle = _raw_stream(index)
        return self

    def empty(self, shape, dtype):
        """A contiguous tensor of `shape` (a plain tuple) on the call's device,
        which is current inside `with`."""
        if len(shape) == 2:
            return _empty(shape, (shape[1], 1), dtype)
        if len(shape) == 1:
            return _empty(shape, (1,), dtype)
        strides, step = [], 1
        for n in reversed(shape):
            strides.append(step)
            step *= n
        return _empty(shape, tuple(reversed(strides)), dtype)

    def workspace(self, given, nbytes):
        """(pointer, bytes) of the workspace, allocated if it is needed and
        not given; keeps it alive until the work is enqueued."""
        if given is None:
            if nbytes == 0:
                return None, 0
            given = self.scratch = _empty((nbytes,), (1,), torch.uint8)
        return given.data_ptr(), given.numel() * given.element_size()

    def __exit__(self, *exc):
        if self.outer is not None:
            self.outer.__exit__(*exc)
        return False


def _ptr(t):
    return None if t is None else t.data_ptr()


_INT = (torch.int32,)
_IDS = (torch.int32, torch.int64)
_F32 = (torch.float32,)
_BF16 = (torch.bfloat16,)
_WIDE = (torch.bfloat16, torch.float32)
_U8 = (torch.uint8,)
_MAX_EXPERTS = 1024


def _workspace_tensor(workspace):
    if workspace is not None:
        if not isinstance(workspace, torch.Tensor):
            raise TypeError("workspace must be a torch.Tensor")
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")


# ---- tokens sorted by expert and back -------------------------------------------

def _check_ids(expert_ids, num_experts, group_offsets, slot_row, row_slot, workspace):
    _tensor(expert_ids, "expert_ids", _IDS)
    if expert_ids.dim() != 2:
        raise ValueError("expert_ids must be 2-dimensional, got shape "
                         f"{tuple(expert_ids.shape)}")
    if not expert_ids.is_contiguous():
        raise ValueError("expert_ids must be contiguous")
    if not 1 <= num_experts <= _MAX_EXPERTS:
        raise ValueError(f"num_experts must be 1 to {_MAX_EXPERTS}, got {num_experts}")
    if group_offsets is not None:
        _dense(group_offsets, "group_offsets", (num_experts + 1,), _INT)
    if slot_row is not None:
        _dense(slot_row, "slot_row", expert_ids.shape, _INT)
    if row_slot is not None:
        _dense(row_slot, "row_slot", (expert_ids.numel(),), _INT)
    _workspace_tensor(workspace)


_PLAN = "group_offsets slot_row row_slot workspace"


def _plan(place, expert_ids, num_experts, group_offsets, slot_row, row_slot):
    if group_offsets is None:
        group_offsets = place.empty((num_experts + 1,), torch.int32)
    if slot_row is None:
        slot_row = place.empty(tuple(expert_ids.shape), torch.int32)
    if row_slot is None:
        row_slot = place.empty((expert_ids.numel(),), torch.int32)
    return group_offsets, slot_row, row_slot


def fp8_moe_sort_workspace_bytes(tokens: int, top_k: int, num_experts: int) -> int:
    return int(_fn("fp8_moe_sort_workspace_bytes")(tokens, top_k, num_experts))


def fp8_moe_sort(expert_ids, num_experts, group_offsets=None, slot_row=None, row_slot=None,
                 workspace=None, stream=None):
    """expert_ids [T][k] (int32 or int64; an id outside [0, num_experts) drops
    its slot) -> (group_offsets int32 [num_experts + 1], slot_row int32 [T][k]
    (-1 for a dropped slot), row_slot int32 [T k] (-1 past the kept rows))."""
    _check_ids(expert_ids, num_experts, group_offsets, slot_row, row_slot, workspace)
    T, k = expert_ids.shape
    _disjoint(_PLAN, (group_offsets, slot_row, row_slot, workspace), "expert_ids", (expert_ids,))
    with _Place(stream, "expert_ids group_offsets slot_row row_slot workspace",
                expert_ids, group_offsets, slot_row, row_slot, workspace) as p:
        plan = _plan(p, expert_ids, num_experts, group_offsets, slot_row, row_slot)
        ws, ws_bytes = p.workspace(workspace, fp8_moe_sort_workspace_bytes(T, k, num_experts))
        _call("fp8_moe_sort", expert_ids.data_ptr(), expert_ids.element_size(), T, k, num_experts,
              plan[0].data_ptr(), plan[1].data_ptr(), plan[2].data_ptr(), ws, ws_bytes, p.handle)
    return plan


def _slots(slot_row, tokens=None):
    """(T, k) of a plan, whose T is `tokens` unless the plan itself says it."""
    _tensor(slot_row, "slot_row", _INT)
    if slot_row.dim() != 2 or tokens not in (None, slot_row.shape[0]):
        raise ValueError(f"slot_row must have shape ({'T' if tokens is None else tokens}, top_k), "
                         f"got {tuple(slot_row.shape)}")
    if not slot_row.is_contiguous():
        raise ValueError("slot_row must be contiguous")
    return slot_row.shape


def _row_matrix(t, name, width, dtypes):
    _tensor(t, name, dtypes)
    if t.dim() != 2 or t.shape[1] != width:
        raise ValueError(f"{name} must have shape (rows, {width}), got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


_COPIED = (torch.uint8, torch.int8, torch.float8_e4m3fn, torch.float8_e5m2, torch.float16,
           torch.bfloat16, torch.float32)


def fp8_moe_dispatch(x, slot_row, scales=None, xs=None, xs_scales=None, stream=None):
    """xs[slot_row[t, j]] = x[t], bit for bit, for x [T][H] of 1, 2 or 4-byte
    values.  With ``scales`` [T][G] fp32 (quantized rows) they travel with
    their rows and (xs, xs_scales) is returned, else xs.  xs has T k rows
    unless given; rows that no slot names are left as they are."""
    ldx = _rows(x, "x", _COPIED)
    T, H = x.shape
    _, k = _slots(slot_row, T)
    if xs is not None:
        _row_matrix(xs, "xs", H, (x.dtype,))
    rows = T * k if xs is None else xs.shape[0]
    G = ld_scales = 0
    if scales is not None:
        ld_scales = _rows(scales, "scales", _F32)
        G = scales.shape[1]
        if scales.shape[0] != T:
            raise ValueError(f"scales must have {T} rows, got {scales.shape[0]}")
        if xs_scales is not None:
            _dense(xs_scales, "xs_scales", (rows, G), _F32)
    elif xs_scales is not None:
        raise ValueError("xs_scales given without scales")
    _disjoint("xs xs_scales", (xs, xs_scales), "x slot_row scales", (x, slot_row, scales))
    with _Place(stream, "x slot_row scales xs xs_scales",
                x, slot_row, scales, xs, xs_scales) as p:
        if xs is None:
            xs = p.empty((rows, H), x.dtype)
        if scales is not None and xs_scales is None:
            xs_scales = p.empty((rows, G), torch.float32)
        _call("fp8_moe_dispatch", x.data_ptr(), x.element_size(), ldx, _ptr(scales), ld_scales, T,
              H, G, slot_row.data_ptr(), k, xs.data_ptr(), _ptr(xs_scales), rows, p.handle)
    return xs if scales is None else (xs, xs_scales)


def _dispatch_quant(name, x, slot_row, q, scales, stream):
    ldx = _rows(x, "x", _BF16)
    T, H = x.shape
    _, k = _slots(slot_row, T)
    G = (H + 127) // 128
    if q is not None:
        _row_matrix(q, "q", H, _U8)
    elif scales is not None:
        _row_matrix(scales, "scales", G, _F32)
    rows = q.shape[0] if q is not None else scales.shape[0] if scales is not None else T * k
    if scales is not None:
        _dense(scales, "scales", (rows, G), _F32)
    _disjoint("q scales", (q, scales), "x slot_row", (x, slot_row))
    with _Place(stream, "x slot_row q scales",
                x, slot_row, q, scales) as p:
        if q is None:
            q = p.empty((rows, H), torch.uint8)
        if scales is None:
            scales = p.empty((rows, G), torch.float32)
        _call(name, x.data_ptr(), ldx, T, H, slot_row.data_ptr(), k, q.data_ptr(),
              scales.data_ptr(), rows, p.handle)
    return q, scales


def fp8_moe_dispatch_quant_1x128(x, slot_row, q=None, scales=None, stream=None):
    """The gather of fp8_moe_dispatch with the 1x128 quantizer in it: x bf16
    [T][H] -> (q uint8 [T k][H] E4M3, scales fp32 [T k][ceil(H/128)])."""
    return _dispatch_quant("fp8_moe_dispatch_quant_1x128", x, slot_row, q, scales, stream)


def fp8_moe_dispatch_quant_1x128_pow2(x, slot_row, q=None, scales=None, stream=None):
    """As fp8_moe_dispatch_quant_1x128 with power-of-two scales."""
    return _dispatch_quant("fp8_moe_dispatch_quant_1x128_pow2", x, slot_row, q, scales, stream)


def fp8_moe_sort_dispatch(x, expert_ids, num_experts, group_offsets=None, slot_row=None,
                          row_slot=None, xs=None, workspace=None, stream=None):
    """fp8_moe_sort and fp8_moe_dispatch in one call: (group_offsets, slot_row,
    row_slot, xs [T k][H])."""
    ldx = _rows(x, "x", _COPIED)
    _check_ids(expert_ids, num_experts, group_offsets, slot_row, row_slot, workspace)
    (T, H), (ids_T, k) = x.shape, expert_ids.shape
    if ids_T != T:
        raise ValueError(f"expert_ids must have {T} rows, got {ids_T}")
    if xs is not None:
        _dense(xs, "xs", (T * k, H), (x.dtype,))
    _disjoint(_PLAN + " xs", (group_offsets, slot_row, row_slot, workspace, xs), "x expert_ids",
              (x, expert_ids))
    with _Place(stream, "x expert_ids group_offsets slot_row row_slot xs workspace",
                x, expert_ids, group_offsets, slot_row, row_slot, xs, workspace) as p:
        plan = _plan(p, expert_ids, num_experts, group_offsets, slot_row, row_slot)
        if xs is None:
            xs = p.empty((T * k, H), x.dtype)
        ws, ws_bytes = p.workspace(workspace, fp8_moe_sort_workspace_bytes(T, k, num_experts))
        _call("fp8_moe_sort_dispatch", x.data_ptr(), x.element_size(), ldx, T, H,
              expert_ids.data_ptr(), expert_ids.element_size(), k, num_experts,
              plan[0].data_ptr(), plan[1].data_ptr(), plan[2].data_ptr(), xs.data_ptr(), ws,
              ws_bytes, p.handle)
    return plan + (xs,)


def _sort_dispatch_quant(name, x, expert_ids, num_experts, group_offsets, slot_row, row_slot, q,
                         scales, workspace, stream):
    ldx = _rows(x, "x", _BF16)
    _check_ids(expert_ids, num_experts, group_offsets, slot_row, row_slot, workspace)
    (T, H), (ids_T, k) = x.shape, expert_ids.shape
    if ids_T != T:
        raise ValueError(f"expert_ids must have {T} rows, got {ids_T}")
    G = (H + 127) // 128
    if q is not None:
        _dense(q, "q", (T * k, H), _U8)
    if scales is not None:
        _dense(scales, "scales", (T * k, G), _F32)
    _disjoint(_PLAN + " q scales", (group_offsets, slot_row, row_slot, workspace, q, scales),
              "x expert_ids", (x, expert_ids))
    with _Place(stream, "x expert_ids group_offsets slot_row row_slot q scales workspace",
                x, expert_ids, group_offsets, slot_row, row_slot, q, scales, workspace) as p:
        plan = _plan(p, expert_ids, num_experts, group_offsets, slot_row, row_slot)
        if q is None:
            q = p.empty((T * k, H), torch.uint8)
        if scales is None:
            scales = p.empty((T * k, G), torch.float32)
        ws, ws_bytes = p.workspace(workspace, fp8_moe_sort_workspace_bytes(T, k, num_experts))
        _call(name, x.data_ptr(), ldx, T, H, expert_ids.data_ptr(), expert_ids.element_size(), k,
              num_experts, plan[0].data_ptr(), plan[1].data_ptr(), plan[2].data_ptr(),
              q.data_ptr(), scales.data_ptr(), ws, ws_bytes, p.handle)
    return plan + (q, scales)


def fp8_moe_sort_dispatch_quant_1x128(x, expert_ids, num_experts, group_offsets=None,
                                      slot_row=None, row_slot=None, q=None, scales=None,
                                      workspace=None, stream=None):
    """fp8_moe_sort and fp8_moe_dispatch_quant_1x128 in one call:
    (group_offsets, slot_row, row_slot, q, scales)."""
    return _sort_dispatch_quant("fp8_moe_sort_dispatch_quant_1x128", x, expert_ids, num_experts,
                                group_offsets, slot_row, row_slot, q, scales, workspace, stream)


def fp8_moe_sort_dispatch_quant_1x128_pow2(x, expert_ids, num_experts, group_offsets=None,
                                           slot_row=None, row_slot=None, q=None, scales=None,
                                           workspace=None, stream=None):
    """As fp8_moe_sort_dispatch_quant_1x128 with power-of-two scales."""
    return _sort_dispatch_quant("fp8_moe_sort_dispatch_quant_1x128_pow2", x, expert_ids,
                                num_experts, group_offsets, slot_row, row_slot, q, scales,
                                workspace, stream)


def fp8_moe_dispatch_grad(dxs, slot_row, dx=None, out_dtype=None, stream=None):
    """dx[t] = sum over j of dxs[slot_row[t, j]] (dropped slots give nothing):
    dxs [R][H] bf16 or fp32 -> dx [T][H] of out_dtype (dxs's own unless
    given)."""
    ld = _rows(dxs, "dxs", _WIDE)
    T, k = _slots(slot_row)
    R, H = dxs.shape
    dtype = _dtype(out_dtype) if out_dtype is not None else dx.dtype if isinstance(
        dx, torch.Tensor) else dxs.dtype
    if dx is not None:
        _dense(dx, "dx", (T, H), tuple(d for d in _WIDE if d == dtype) or _WIDE)
        _disjoint("dx", (dx,), "dxs slot_row", (dxs, slot_row))
    with _Place(stream, "dxs slot_row dx",
                dxs, slot_row, dx) as p:
        if dx is None:
            dx = p.empty((T, H), dtype)
        _call("fp8_moe_dispatch_grad", dxs.data_ptr(), _CODES[dxs.dtype], ld, R,
              slot_row.data_ptr(), T, k, H, dx.data_ptr(), _CODES[dtype], p.handle)
    return dx


def fp8_moe_combine(ys, slot_row, weights=None, residual=None, out=None, out_dtype=None,
                    stream=None):
    """out[t] = residual[t] + sum over j of weights[t, j] ys[slot_row[t, j]]:
    ys [R][H] bf16 or fp32, weights fp32 [T][k] (ones without), residual and
    out [T][H] of out_dtype (ys's own unless given; residual may be out
    itself)."""
    ld = _rows(ys, "ys", _WIDE)
    T, k = _slots(slot_row)
    R, H = ys.shape
    dtype = _dtype(out_dtype) if out_dtype is not None else out.dtype if isinstance(
        out, torch.Tensor) else ys.dtype
    if weights is not None:
        _dense(weights, "weights", (T, k), _F32)
    ld_residual = 0
    if residual is not None:
        ld_residual = _rows(residual, "residual", (dtype,), (T, H))
    if out is not None:
        _dense(out, "out", (T, H), tuple(d for d in _WIDE if d == dtype) or _WIDE)
        same = (residual is not None and residual.data_ptr() == out.data_ptr()
                and ld_residual == H)
        _disjoint("out", (out,), "ys slot_row weights residual",
                  (ys, slot_row, weights, None if same else residual))
    with _Place(stream, "ys slot_row weights residual out",
                ys, slot_row, weights, residual, out) as p:
        if out is None:
            out = p.empty((T, H), dtype)
        _call("fp8_moe_combine", ys.data_ptr(), _CODES[ys.dtype], ld, R, slot_row.data_ptr(),
              _ptr(weights), T, k, H, _ptr(residual), ld_residual, out.data_ptr(), _CODES[dtype],
              p.handle)
    return out


def fp8_moe_combine_grad(dout, ys, slot_row, weights=None, dys=None, dweights=None,
                         stream=None):
    """Gradient of fp8_moe_combine: dys[slot_row[t, j]] = weights[t, j] dout[t]
    (rows that no slot names are left as they are) and dweights[t, j] = <dout[t],
    ys[slot_row[t, j]]>, 0 for a dropped slot.  (dys [R][H], dweights fp32
    [T][k])."""
    ld_dout = _rows(dout, "dout", _WIDE)
    T, H = dout.shape
    _, k = _slots(slot_row, T)
    ld_ys = _rows(ys, "ys", (dout.dtype,))
    R = ys.shape[0]
    if ys.shape[1] != H:
        raise ValueError(f"ys must have shape (rows, {H}), got {tuple(ys.shape)}")
    if weights is not None:
        _dense(weights, "weights", (T, k), _F32)
    if dys is not None:
        _dense(dys, "dys", (R, H), (dout.dtype,))
    if dweights is not None:
        _dense(dweights, "dweights", (T, k), _F32)
    _disjoint("dys dweights", (dys, dweights), "dout ys slot_row weights",
              (dout, ys, slot_row, weights))
    with _Place(stream, "dout ys slot_row weights dys dweights",
                dout, ys, slot_row, weights, dys, dweights) as p:
        if dys is None:
            dys = p.empty((R, H), dout.dtype)
        if dweights is None:
            dweights = p.empty((T, k), torch.float32)
        _call("fp8_moe_combine_grad", dout.data_ptr(), ld_dout, ys.data_ptr(), ld_ys,
              _CODES[dout.dtype], R, slot_row.data_ptr(), _ptr(weights), T, k, H, dys.data_ptr(),
              dweights.data_ptr(), p.handle)
    return dys, dweights


# ---- norms before and after a block ------------------------------------------------

def _norm_params(H, T, w_post, gate, w_pre):
    """(type code of the parameters, gate rows)."""
    dtype = None
    for name, t in (("w_post", w_post), ("gate", gate), ("w_pre", w_pre)):
        if t is None:
            continue
        _tensor(t, name, _WIDE if dtype is None else (dtype,))
        dtype = t.dtype
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if name != "gate":
            if t.shape != (H,):
                raise ValueError(f"{name} must have shape ({H},), got {tuple(t.shape)}")
        elif t.dim() not in (1, 2) or t.shape[-1] != H:
            raise ValueError(f"gate must have shape ({H},) or (rows, {H}), got {tuple(t.shape)}")
    rows = 1 if gate is None or gate.dim() == 1 else gate.shape[0]
    if gate is not None and (rows < 1 or T % rows):
        raise ValueError(f"gate's {rows} rows must divide the {T} tokens")
    return _CODES[dtype or torch.float32], rows


def _stream_types(y):
    return _F32 if y.dtype == torch.float32 else _WIDE


def _norm(name, quant, y, r, w_post, gate, w_pre, post_norm, residual_scale, branch_scale, eps,
          r_out, n, q, scales, rstd_post, rstd_pre, stream):
    ldy = _rows(y, "y", _WIDE)
    T, H = y.shape
    ldr = _rows(r, "r", _stream_types(y), (T, H))
    code, gate_rows = _norm_params(H, T, w_post, gate, w_pre)
    G = (H + 127) // 128
    if r_out is not None:
        _dense(r_out, "r_out", (T, H), (r.dtype,))
    if n is not None:
        _dense(n, "n", (T, H), (y.dtype,))
    if q is not None:
        _dense(q, "q", (T, H), _U8)
    if scales is not None:
        _dense(scales, "scales", (T, G), _F32)
    for what, t in (("rstd_post", rstd_post), ("rstd_pre", rstd_pre)):
        if t is not None:
            _dense(t, what, (T,), _F32)
    same = r_out is not None and r_out.data_ptr() == r.data_ptr() and ldr == H
    _disjoint("r_out n q scales rstd_post rstd_pre", (r_out, n, q, scales, rstd_post, rstd_pre),
              "y r w_post gate w_pre", (y, None if same else r, w_post, gate, w_pre))
    with _Place(stream, "y r w_post gate w_pre r_out n q scales rstd_post rstd_pre",
                y, r, w_post, gate, w_pre, r_out, n, q, scales, rstd_post, rstd_pre) as p:
        if r_out is None:
            r_out = p.empty((T, H), r.dtype)
        if quant:
            if q is None:
                q = p.empty((T, H), torch.uint8)
            if scales is None:
                scales = p.empty((T, G), torch.float32)
        elif n is None:
            n = p.empty((T, H), y.dtype)
        if rstd_post is None and post_norm:
            rstd_post = p.empty((T,), torch.float32)
        if rstd_pre is None:
            rstd_pre = p.empty((T,), torch.float32)
        args = (y.data_ptr(), _CODES[y.dtype], ldy, r.data_ptr(), _CODES[r.dtype], ldr,
                _ptr(w_post), _ptr(gate), _ptr(w_pre), code, T, H, gate_rows, int(post_norm),
                residual_scale, branch_scale, eps, r_out.data_ptr(), _ptr(n))
        if quant:
            args += (q.data_ptr(), scales.data_ptr())
        _call(name, *args, _ptr(rstd_post), _ptr(rstd_pre), p.handle)
    return r_out, n, q, scales, rstd_post, rstd_pre


def fp8_norm_residual(y, r, w_post=None, gate=None, w_pre=None, *, post_norm=True,
                      residual_scale=1.0, branch_scale=1.0, eps=1e-6, r_out=None, n=None,
                      rstd_post=None, rstd_pre=None, stream=None):
    """u = y rstd_post w_post (y itself without post_norm), r_out =
    residual_scale r + branch_scale gate u, n = r_out rstd_pre w_pre, rstd = 1 /
    sqrt(mean of squares + eps) over each token's H channels.

    y [T][H] bf16 or fp32; r [T][H] bf16 or fp32 (fp32 with fp32 y); w_post,
    w_pre [H] and gate [H] or [rows][H] (rows dividing T: each row serves T /
    rows tokens in turn), all fp32 or all bf16, None for ones.  Returns (r_out,
    n, rstd_post, rstd_pre), rstd_post None without post_norm; r_out may be r."""
    out = _norm("fp8_norm_residual", False, y, r, w_post, gate, w_pre, post_norm, residual_scale,
                branch_scale, eps, r_out, n, None, None, rstd_post, rstd_pre, stream)
    return out[0], out[1], out[4], out[5]


def fp8_norm_residual_quant_1x128(y, r, w_post=None, gate=None, w_pre=None, *, post_norm=True,
                                  residual_scale=1.0, branch_scale=1.0, eps=1e-6, r_out=None,
                                  n=None, q=None, scales=None, rstd_post=None, rstd_pre=None,
                                  stream=None):
    """As fp8_norm_residual with n quantized 1x128 from its fp32 values: (r_out,
    q uint8 [T][H] E4M3, scales fp32 [T][ceil(H/128)], rstd_post, rstd_pre).
    With ``n`` given it is written too (for a router, say)."""
    out = _norm("fp8_norm_residual_quant_1x128", True, y, r, w_post, gate, w_pre, post_norm,
                residual_scale, branch_scale, eps, r_out, n, q, scales, rstd_post, rstd_pre,
                stream)
    return out[0], out[2], out[3], out[4], out[5]


def fp8_norm_residual_quant_1x128_pow2(y, r, w_post=None, gate=None, w_pre=None, *,
                                       post_norm=True, residual_scale=1.0, branch_scale=1.0,
                                       eps=1e-6, r_out=None, n=None, q=None, scales=None,
                                       rstd_post=None, rstd_pre=None, stream=None):
    """As fp8_norm_residual_quant_1x128 with power-of-two scales."""
    out = _norm("fp8_norm_residual_quant_1x128_pow2", True, y, r, w_post, gate, w_pre, post_norm,
                residual_scale, branch_scale, eps, r_out, n, q, scales, rstd_post, rstd_pre,
                stream)
    return out[0], out[2], out[3], out[4], out[5]


def fp8_norm_residual_grad_workspace_bytes(tokens: int, width: int, gate_rows: int = 1) -> int:
    return int(_fn("fp8_norm_residual_grad_workspace_bytes")(tokens, width, gate_rows))


def fp8_norm_residual_grad(dn, dr_out, y, r_out, rstd_post, rstd_pre, w_post=None, gate=None,
                           w_pre=None, *, post_norm=True, residual_scale=1.0, branch_scale=1.0,
                           dy=None, dr=None, workspace=None, stream=None):
    """Gradient of fp8_norm_residual from dn (of n; None for zero) and dr_out (of
    r_out; None for zero), with the forward's y, r_out and rstd's: (dy, dr,
    dw_post, dgate, dw_pre), the last three fp32 and None where the forward had
    no such parameter (dgate [H] or [rows][H] as gate)."""
    ldy = _rows(y, "y", _WIDE)
    T, H = y.shape
    if dn is None and dr_out is None:
        raise ValueError("one of dn and dr_out must be given")
    ld_dn = ld_dr = ld_r = 0
    if dn is not None:
        ld_dn = _rows(dn, "dn", (y.dtype,), (T, H))
        _dense(rstd_pre, "rstd_pre", (T,), _F32)
    ld_r = _rows(r_out, "r_out", _stream_types(y), (T, H))
    if dr_out is not None:
        ld_dr = _rows(dr_out, "dr_out", (r_out.dtype,), (T, H))
    if post_norm:
        _dense(rstd_post, "rstd_post", (T,), _F32)
    else:
        rstd_post = w_post = None
    code, gate_rows = _norm_params(H, T, w_post, gate, w_pre)
    if dy is not None:
        _dense(dy, "dy", (T, H), (y.dtype,))
    if dr is not None:
        _dense(dr, "dr", (T, H), (r_out.dtype,))
    _workspace_tensor(workspace)
    _disjoint("dy dr workspace", (dy, dr, workspace),
              "dn dr_out y r_out rstd_post rstd_pre w_post gate w_pre",
              (dn, dr_out, y, r_out, rstd_post, rstd_pre if dn is not None else None, w_post, gate,
               w_pre))
    with _Place(stream, "dn dr_out y r_out rstd_post rstd_pre w_post gate w_pre dy dr workspace",
                dn, dr_out, y, r_out, rstd_post, rstd_pre, w_post, gate, w_pre, dy, dr,
                workspace) as p:
        if dy is None:
            dy = p.empty((T, H), y.dtype)
        if dr is None:
            dr = p.empty((T, H), r_out.dtype)
        dw_post = p.empty((H,), torch.float32) if w_post is not None else None
        dw_pre = p.empty((H,), torch.float32) if w_pre is not None else None
        dgate = p.empty(tuple(gate.shape), torch.float32) if gate is not None else None
        ws, ws_bytes = p.workspace(
            workspace, fp8_norm_residual_grad_workspace_bytes(T, H, gate_rows))
        _call("fp8_norm_residual_grad", _ptr(dn), ld_dn, _ptr(dr_out), ld_dr, y.data_ptr(),
              _CODES[y.dtype], ldy, r_out.data_ptr(), _CODES[r_out.dtype], ld_r, _ptr(rstd_post),
              _ptr(rstd_pre), _ptr(w_post), _ptr(gate), _ptr(w_pre), code, T, H, gate_rows,
              int(post_norm), residual_scale, branch_scale, dy.data_ptr(), dr.data_ptr(),
              _ptr(dw_post), _ptr(dgate), _ptr(dw_pre), ws, ws_bytes, p.handle)
    return dy, dr, dw_post, dgate, dw_pre


# ---- 4-bit weights -------------------------------------------------------------------

def _w4_quant(name, w, group, scale_type, codes, scales, stream):
    _tensor(w, "w", _BF16)
    if w.dim() < 2:
        raise ValueError(f"w must have shape (..., N, K), got {tuple(w.shape)}")
    if not w.is_contiguous():
        raise ValueError("w must be contiguous")
    lead, K = w.shape[:-1], w.shape[-1]
    N = lead.numel()
    code_shape = (*lead, (K + 1) // 2)
    scale_shape = (*lead, (K + group - 1) // group)
    if codes is not None:
        _dense(codes, "codes", code_shape, _U8)
    if scales is not None:
        _dense(scales, "scales", scale_shape, (scale_type,))
    _disjoint("codes scales", (codes, scales), "w", (w,))
    with _Place(stream, "w codes scales",
                w, codes, scales) as p:
        if codes is None:
            codes = p.empty(code_shape, torch.uint8)
        if scales is None:
            scales = p.empty(scale_shape, scale_type)
        _call(name, w.data_ptr(), N, K, codes.data_ptr(), scales.data_ptr(), p.handle)
    return codes, scales


def fp8_w4_quant_1x128(w, codes=None, scales=None, stream=None):
    """w bf16 [..., N, K] -> (codes uint8 [..., N, ceil(K/2)], two E2M1 codes a
    byte, scales fp32 [..., N, ceil(K/128)] = amax / 6)."""
    return _w4_quant("fp8_w4_quant_1x128", w, 128, torch.float32, codes, scales, stream)


def fp8_w4_quant_1x32(w, codes=None, scales=None, stream=None):
    """w bf16 [..., N, K] -> (codes uint8 [..., N, ceil(K/2)], two E2M1 codes a
    byte, scales uint8 [..., N, ceil(K/32)], E8M0: the smallest power of two that
    is at least amax / 6)."""
    return _w4_quant("fp8_w4_quant_1x32", w, 32, torch.uint8, codes, scales, stream)


def _w4_operands(x, codes, scales, lead):
    ldx = _rows(x, "x", _BF16)
    K = x.shape[1]
    _tensor(codes, "codes", _U8)
    if codes.dim() != lead + 2 or codes.shape[-1] != (K + 1) // 2:
        raise ValueError(f"codes must have shape ({'experts, ' if lead else ''}N, "
                         f"{(K + 1) // 2}), got {tuple(codes.shape)}")
    if not codes.is_contiguous():
        raise ValueError("codes must be contiguous")
    _tensor(scales, "scales", (torch.float32, torch.uint8))
    kind, group = ((FP8_W4_F32_1X128, 128) if scales.dtype == torch.float32
                   else (FP8_W4_E8M0_1X32, 32))
    _dense(scales, "scales", (*codes.shape[:-1], (K + group - 1) // group), (scales.dtype,))
    return ldx, kind


def fp8_w4_matvec(x, codes, scales, out_dtype="bf16", y=None, stream=None):
    """y [M][N] = x [M][K] times the 4-bit weights of fp8_w4_quant_1x128 (fp32
    scales) or fp8_w4_quant_1x32 (uint8 E8M0 scales), codes [N][ceil(K/2)]; x
    bf16, used as it is.  Made for few rows (up to 16 at a pass over the
    weights)."""
    dtype = _dtype(out_dtype)
    ldx, kind = _w4_operands(x, codes, scales, 0)
    (M, K), N = x.shape, codes.shape[0]
    if y is not None:
        _dense(y, "y", (M, N), (dtype,))
        _disjoint("y", (y,), "x codes scales", (x, codes, scales))
    with _Place(stream, "x codes scales y",
                x, codes, scales, y) as p:
        if y is None:
            y = p.empty((M, N), dtype)
        _call("fp8_w4_matvec", x.data_ptr(), ldx, codes.data_ptr(), scales.data_ptr(), kind, M, N,
              K, y.data_ptr(), _CODES[dtype], p.handle)
    return y


def fp8_w4_grouped_matvec(x, codes, scales, group_offsets, out_dtype="bf16", y=None,
                          stream=None):
    """Row r of expert e (rows [group_offsets[e], group_offsets[e+1]) of x
    [R][K]) times the expert's 4-bit weights: codes [E][N][ceil(K/2)], scales
    [E][N][...] -> y [R][N].  Rows outside every expert's range are left as they
    are."""
    dtype = _dtype(out_dtype)
    ldx, kind = _w4_operands(x, codes, scales, 1)
    (R, K), (E, N) = x.shape, codes.shape[:2]
    _dense(group_offsets, "group_offsets", (E + 1,), _INT)
    if y is not None:
        _dense(y, "y", (R, N), (dtype,))
        _disjoint("y", (y,), "x codes scales group_offsets", (x, codes, scales, group_offsets))
    with _Place(stream, "x codes scales group_offsets y",
                x, codes, scales, group_offsets, y) as p:
        if y is None:
            y = p.empty((R, N), dtype)
        _call("fp8_w4_grouped_matvec", x.data_ptr(), ldx, codes.data_ptr(), scales.data_ptr(),
              kind, group_offsets.data_ptr(), E, R, N, K, y.data_ptr(), _CODES[dtype], p.handle)
    return y
