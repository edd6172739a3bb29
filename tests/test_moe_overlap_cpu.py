"""Outputs and workspaces of the operators around the expert products that
share memory with an input or with each other are refused before anything is
launched: a workgroup may read an input after another has begun to write."""
import pytest
import torch

from fp8_fine_grained_token_amd import moe as M

BF, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


def new(dtype, *shape):
    return torch.zeros(shape, dtype=dtype)


def over(t, dtype, *shape, at=0):
    """A tensor of that type and shape in t's memory, `at` bytes in."""
    size = torch.Size(shape).numel() * dtype.itemsize
    raw = torch.empty(0, dtype=U8).set_(t.untyped_storage())
    start = t.storage_offset() * t.element_size() + at
    return raw[start:start + size].view(dtype).reshape(shape)


# every output (and workspace) of each call, on memory of the call's inputs and
# of its other outputs
T, K, E, H = 4, 3, 5, 256
BIG = 1 << 14  # bytes: room for every output anywhere in it


def sort(ids, **kw):
    return M.fp8_moe_sort(ids, E, **kw)


PLAN = {"group_offsets": (I32, E + 1), "slot_row": (I32, T, K), "row_slot": (I32, T * K),
        "workspace": (U8, 64)}
Q = {"q": (U8, T * K, H), "scales": (F32, T * K, H // 128)}
NORM = {"r_out": (BF, T, H), "n": (BF, T, H), "rstd_post": (F32, T), "rstd_pre": (F32, T)}
NORM_Q = dict(NORM, q=(U8, T, H), scales=(F32, T, H // 128))
NORM_IN = {"y": (BF, T, H), "r": (BF, T, H), "w_post": (F32, H), "gate": (F32, H),
           "w_pre": (F32, H)}

CALLS = {
    "sort": (sort, {"ids": (I32, T, K)}, PLAN),
    "dispatch": (M.fp8_moe_dispatch,
                 {"x": (U8, T, H), "slot_row": (I32, T, K), "scales": (F32, T, 2)},
                 {"xs": (U8, T * K, H), "xs_scales": (F32, T * K, 2)}),
    "dispatch_quant": (M.fp8_moe_dispatch_quant_1x128, {"x": (BF, T, H), "slot_row": (I32, T, K)},
                       Q),
    "dispatch_quant_pow2": (M.fp8_moe_dispatch_quant_1x128_pow2,
                            {"x": (BF, T, H), "slot_row": (I32, T, K)}, Q),
    "sort_dispatch": (lambda x, ids, **kw: M.fp8_moe_sort_dispatch(x, ids, E, **kw),
                      {"x": (BF, T, H), "ids": (I32, T, K)}, dict(PLAN, xs=(BF, T * K, H))),
    "sort_dispatch_quant": (
        lambda x, ids, **kw: M.fp8_moe_sort_dispatch_quant_1x128(x, ids, E, **kw),
        {"x": (BF, T, H), "ids": (I32, T, K)}, dict(PLAN, **Q)),
    "sort_dispatch_quant_pow2": (
        lambda x, ids, **kw: M.fp8_moe_sort_dispatch_quant_1x128_pow2(x, ids, E, **kw),
        {"x": (BF, T, H), "ids": (I32, T, K)}, dict(PLAN, **Q)),
    "dispatch_grad": (M.fp8_moe_dispatch_grad, {"dxs": (BF, T * K, H), "slot_row": (I32, T, K)},
                      {"dx": (BF, T, H)}),
    "combine": (M.fp8_moe_combine,
                {"ys": (BF, T * K, H), "slot_row": (I32, T, K), "weights": (F32, T, K)},
                {"out": (BF, T, H)}),
    "combine_grad": (M.fp8_moe_combine_grad,
                     {"dout": (BF, T, H), "ys": (BF, T * K, H), "slot_row": (I32, T, K),
                      "weights": (F32, T, K)},
                     {"dys": (BF, T * K, H), "dweights": (F32, T, K)}),
    "norm": (M.fp8_norm_residual, NORM_IN, NORM),
    "norm_quant": (M.fp8_norm_residual_quant_1x128, NORM_IN, NORM_Q),
    "norm_quant_pow2": (M.fp8_norm_residual_quant_1x128_pow2, NORM_IN, NORM_Q),
    "norm_grad": (M.fp8_norm_residual_grad,
                  {"dn": (BF, T, H), "dr_out": (BF, T, H), "y": (BF, T, H), "r_out": (BF, T, H),
                   "rstd_post": (F32, T), "rstd_pre": (F32, T), "w_post": (F32, H),
                   "gate": (F32, H), "w_pre": (F32, H)},
                  {"dy": (BF, T, H), "dr": (BF, T, H), "workspace": (U8, 64)}),
    "w4_quant_1x128": (M.fp8_w4_quant_1x128, {"w": (BF, T, H)},
                       {"codes": (U8, T, H // 2), "scales": (F32, T, H // 128)}),
    "w4_quant_1x32": (M.fp8_w4_quant_1x32, {"w": (BF, T, H)},
                      {"codes": (U8, T, H // 2), "scales": (U8, T, H // 32)}),
    "w4_matvec": (M.fp8_w4_matvec, {"x": (BF, T, H), "codes": (U8, 8, H // 2),
                                    "scales": (F32, 8, H // 128)}, {"y": (BF, T, 8)}),
    "w4_grouped_matvec": (M.fp8_w4_grouped_matvec,
                          {"x": (BF, T, H), "codes": (U8, E, 8, H // 2),
                           "scales": (F32, E, 8, H // 128), "group_offsets": (I32, E + 1)},
                          {"y": (BF, T, 8)}),
}
PAIRS = [(call, out, other) for call, (_, ins, outs) in CALLS.items() for out in outs
         for other in list(ins) + [o for o in outs if o != out]]


@pytest.mark.parametrize("call,out,other", PAIRS, ids=["-".join(p) for p in PAIRS])
def test_shared_memory_is_refused(call, out, other):
    fn, ins, outs = CALLS[call]
    args = {name: new(*spec) for name, spec in ins.items()}
    given, spec, whole = {}, ins.get(other) or outs[other], new(U8, BIG)
    (args if other in ins else given)[other] = over(whole, *spec)
    size = torch.Size(spec[1:]).numel() * spec[0].itemsize
    # on the other's first byte, and on its last bytes
    for at in (0, (size - 1) // 8 * 8):
        if (out, other, at) == ("r_out", "r", 0):
            continue  # the new stream may be the old one, but no part of it
        given[out] = over(whole, *outs[out], at=at)
        with pytest.raises(ValueError, match="share memory"):
            fn(*args.values(), **given)


@pytest.mark.parametrize("call", list(CALLS))
def test_separate_and_adjacent_memory_is_not(call):
    # every output given, one right behind the other in one allocation: the
    # call gets as far as asking for the GPU
    fn, ins, outs = CALLS[call]
    args = {name: new(*spec) for name, spec in ins.items()}
    whole, at, given = new(U8, 8 * BIG), 0, {}
    for name, spec in outs.items():
        given[name] = over(whole, *spec, at=at)
        at += -(-torch.Size(spec[1:]).numel() * spec[0].itemsize // 8) * 8
    with pytest.raises(ValueError, match="on the GPU"):
        fn(*args.values(), **given)


def test_the_stream_and_the_sum_may_be_written_in_place():
    r, y = new(BF, T, H), new(BF, T, H)
    with pytest.raises(ValueError, match="on the GPU"):
        M.fp8_norm_residual(y, r, r_out=r)
    with pytest.raises(ValueError, match="share memory"):
        M.fp8_norm_residual(y, r, r_out=r, n=r)
    with pytest.raises(ValueError, match="on the GPU"):
        M.fp8_moe_combine(new(BF, T * K, H), new(I32, T, K), residual=r, out=r)
    with pytest.raises(ValueError, match="share memory"):
        M.fp8_moe_combine(new(BF, T * K, H), new(I32, T, K), residual=r[:1].expand(T, H), out=r)
