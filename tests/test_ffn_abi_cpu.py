"""Contract of the operators inside a gated feed-forward block that needs no
GPU: the library exports what include/fp8ffn.h declares, bad arguments are
refused with the documented status before anything is launched, and the Python
layer refuses tensors the kernels could not index (every call here fails
validation or is a documented no-op)."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

from fp8_fine_grained_token_amd import binding as B
from fp8_fine_grained_token_amd import ffn as L

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A, ODD, N = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10001), ctypes.c_void_p(0)
A2, A4, A8 = ctypes.c_void_p(0x10002), ctypes.c_void_p(0x10004), ctypes.c_void_p(0x10008)
F32, BF16 = B.FP8_OUT_F32, B.FP8_OUT_BF16
BIG = 1 << 31


def call(name, *args):
    return L._fn(name)(*args)


def declared():
    text = open(os.path.join(ROOT, "include", "fp8ffn.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return set(re.findall(r"\b(fp8_[a-z0-9_]+)\s*\(", text))


def test_every_declared_symbol_is_exported_and_bound():
    assert declared() == set(L._SIGNATURES)
    import fp8_fine_grained_token_amd as F
    for name in declared():
        assert hasattr(B.lib(), name), name
        assert getattr(F, name) is getattr(L, name)
    for name in F._FFN:
        assert getattr(F, name) is getattr(L, name) and name in dir(F)


def test_header_is_plain_c():
    # a C99 program that includes all three headers and names every function
    program = "#include \"fp8ffn.h\"\n#include \"fp8moe.h\"\n#include \"fp8blk.h\"\n" + "".join(
        f"void *p{i} = (void *)&{n};\n" for i, n in enumerate(sorted(declared())))
    r = subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-fsyntax-only", "-x", "c",
                        "-I" + os.path.join(ROOT, "include"), "-"], input=program, text=True,
                       capture_output=True)
    assert r.returncode == 0, r.stderr


# ---- status codes of the C entries ------------------------------------------------

def gated(suffix="", a=A, sa=A, w=A, sw=A, act=0, M=4, I=256, K=128, out=A, t=BF16, ws=N, wsb=0):
    return call("fp8_block_gemm_gated" + suffix, a, sa, w, sw, act, M, I, K, out, t, ws, wsb, N)


def gated_q(suffix="", a=A, sa=A, w=A, sw=A, act=0, M=4, I=256, K=128, q=A, s=A, h=N, hs=N, ws=N,
            wsb=0):
    return call("fp8_block_gemm_gated_quant_1x128" + suffix, a, sa, w, sw, act, M, I, K, q, s, h,
                hs, ws, wsb, N)


def grouped(suffix="", a=A, sa=A, w=A, sw=A, off=A, E=3, act=0, T=4, I=256, K=128, out=A, t=BF16,
            ws=N, wsb=0):
    return call("fp8_block_grouped_gemm_gated" + suffix, a, sa, w, sw, off, E, act, T, I, K, out,
                t, ws, wsb, N)


def grouped_q(suffix="", a=A, sa=A, w=A, sw=A, off=A, E=3, act=0, T=4, I=256, K=128, q=A, s=A,
              h=N, hs=N, ws=N, wsb=0):
    return call("fp8_block_grouped_gemm_gated_quant_1x128" + suffix, a, sa, w, sw, off, E, act, T,
                I, K, q, s, h, hs, ws, wsb, N)


@pytest.mark.parametrize("suffix", ["", "_pow2"])
def test_gated_product_errors(suffix):
    for go in (gated, gated_q, grouped, grouped_q):
        rows = "T" if go in (grouped, grouped_q) else "M"
        assert go(suffix, act=2) == go(suffix, act=-1) == B.FP8_ERR_DTYPE
        for bad in (dict(I=-128), dict(K=-128), {rows: -1}, dict(I=192), dict(K=64), dict(I=64),
                    {rows: BIG}, dict(I=BIG // 2), dict(K=1 << 24), {rows: 1 << 30, "K": 1 << 20},
                    {rows: 1 << 28, "I": 1 << 12}):
            assert go(suffix, **bad) == B.FP8_ERR_SHAPE, bad
        assert go(suffix, K=0) == B.FP8_ERR_SHAPE
        for what in ("a", "sa", "w", "sw"):
            assert go(suffix, **{what: N}) == B.FP8_ERR_NULL, what
        for what, at in (("a", A8), ("w", A8), ("sa", A2), ("sw", A2)):
            assert go(suffix, **{what: at}) == B.FP8_ERR_ALIGN, what
        # no rows or no columns: nothing to do, whatever the pointers
        assert go(suffix, **{rows: 0}, a=N, w=N) == go(suffix, I=0, a=N) == B.FP8_OK
        assert go(suffix, **{rows: 0}, K=0) == B.FP8_OK
    for go in (gated, grouped):
        assert go(suffix, out=N) == B.FP8_ERR_NULL
        assert go(suffix, out=A8) == B.FP8_ERR_ALIGN
        assert go(suffix, t=2) == B.FP8_ERR_DTYPE
    for go in (gated_q, grouped_q):
        assert go(suffix, q=N) == go(suffix, s=N) == B.FP8_ERR_NULL
        assert go(suffix, h=A) == go(suffix, hs=A) == B.FP8_ERR_NULL
        assert go(suffix, q=A8) == go(suffix, s=A2) == B.FP8_ERR_ALIGN
        assert go(suffix, h=A8, hs=A) == go(suffix, h=A, hs=A2) == B.FP8_ERR_ALIGN
    for go in (gated, gated_q, grouped, grouped_q):
        assert go(suffix, ws=A) == go(suffix, wsb=256) == B.FP8_ERR_WORKSPACE
        assert go(suffix, ws=A8, wsb=256) == B.FP8_ERR_WORKSPACE
    for go in (grouped, grouped_q):
        assert go(suffix, off=N) == B.FP8_ERR_NULL and go(suffix, off=A2) == B.FP8_ERR_ALIGN
        for E in (0, -1, 1 << 20):
            assert go(suffix, E=E) == B.FP8_ERR_SHAPE
        assert go(suffix, E=0, T=0) == B.FP8_OK


def test_workspace_of_sizes_out_of_range():
    for sizes in ((-1, 128, 128), (1, 64, 128), (1, 128, 64), (0, 128, 128), (1, 0, 128),
                  (1, 128, 0), (1, BIG // 2, 128), (BIG, 128, 128), (1, 128, 1 << 24)):
        assert L.fp8_gated_gemm_workspace_bytes(*sizes) == 0, sizes
        rows, inner, width = sizes
        assert L.fp8_grouped_gated_gemm_workspace_bytes(rows, 4, inner, width) == 0, sizes
    for experts in (0, -1, 1 << 20):
        assert L.fp8_grouped_gated_gemm_workspace_bytes(4, experts, 128, 128) == 0


def test_plans_that_take_a_workspace():
    # K in parts as long as the 64 x 64 tiles of the parts, at most, are about what
    # runs at once: with more of them the one-kernel plan is faster
    need = L.fp8_grouped_gated_gemm_workspace_bytes
    for K in (512, 2304, 7168):
        assert need(1000, 8, 768, K) > 0 and need(1000, 4, 768, K) > 0
        assert need(1000, 4, 1024, K) == need(1600, 16, 512, K) == 0
        # few rows: 32-row tiles
        assert L.fp8_gated_gemm_workspace_bytes(17, 16384, K) > 0
        assert L.fp8_gated_gemm_workspace_bytes(17, 16512, K) == 0
        assert need(150, 16, 1024, K) > 0 and need(20, 32, 1024, K) > 0
        assert need(100, 8, 2048, K) == need(500, 32, 512, K) == 0
        # 64-row tiles as the other plan
        assert need(500, 16, 512, K) > 0 and need(1600, 64, 128, K) > 0
        assert need(900, 32, 384, K) == need(400, 8, 1408, K) == 0


def test_gated_grad_errors():
    def dense(da=A, dt=BF16, ld=256, h=A, ldh=512, hs=A, act=0, M=4, I=256, dh=A, t=BF16):
        return call("fp8_gated_grad", da, dt, ld, h, ldh, hs, act, M, I, dh, t, N)

    def quant(suffix="", da=A, dt=BF16, ld=256, h=A, ldh=512, hs=A, act=0, M=4, I=256, q=A, s=A,
              qt=A, st=A, at=A, as_=A):
        return call("fp8_gated_grad_quant" + suffix, da, dt, ld, h, ldh, hs, act, M, I, q, s, qt,
                    st, at, as_, N)

    def quant_pow2(**kw):
        return quant("_pow2", **kw)

    for go in (dense, quant, quant_pow2):
        assert go(act=2) == go(dt=2) == B.FP8_ERR_DTYPE
        for bad in (dict(M=-1), dict(I=-128), dict(I=64), dict(I=200), dict(M=BIG),
                    dict(I=BIG // 2), dict(M=1 << 30, I=1 << 9), dict(ld=-1), dict(ldh=-1),
                    dict(ld=1 << 39), dict(ldh=1 << 39), dict(M=1 << 28, I=128)):
            assert go(**bad) == B.FP8_ERR_SHAPE, bad
        assert go(da=N) == go(h=N) == B.FP8_ERR_NULL
        assert go(da=ODD) == go(da=A2, dt=F32) == B.FP8_ERR_ALIGN
        assert go(hs=A2) == go(h=ODD, hs=N) == B.FP8_ERR_ALIGN
        assert go(M=0, da=N, h=N) == go(I=0, da=N, h=N) == B.FP8_OK
    assert dense(dh=N) == B.FP8_ERR_NULL and dense(t=2) == B.FP8_ERR_DTYPE
    assert dense(dh=ODD) == dense(dh=A2, t=F32) == B.FP8_ERR_ALIGN
    for go in (quant, quant_pow2):
        for pair in (("q", "s"), ("qt", "st"), ("at", "as_")):
            for one in pair:  # one of a pair alone
                assert go(**{one: N}) == B.FP8_ERR_NULL
        assert go(q=N, s=N, qt=N, st=N, at=N, as_=N) == B.FP8_ERR_NULL
        assert go(q=A4) == go(s=A2) == go(st=A2) == go(as_=A2) == B.FP8_ERR_ALIGN


def test_gated_grad_limit():
    # 16 threads to a row's 128 columns in workgroups of 256: from M I / 128 =
    # 2^28 - 15 on the last workgroup is work-item 2^32 (rows may share their
    # memory: ld 0)
    for M, I in (((1 << 28) - 1, 128), ((1 << 28) - 15, 128), ((1 << 27) - 7, 256)):
        for name, rest in (("fp8_gated_grad", (A, BF16)),
                           ("fp8_gated_grad_quant", (A, A, N, N, N, N)),
                           ("fp8_gated_grad_quant_pow2", (A, A, A, A, A, A))):
            assert call(name, A, BF16, 0, A, 0, A, 0, M, I, *rest, N) == B.FP8_ERR_SHAPE, (M, I)


def test_checkpoint_errors():
    def read(q=A, s=A, M=4, K=300, x=A, t=BF16):
        return call("fp8_dequant_act_1x128", q, s, M, K, x, t, N)

    def turn(q=A, s=A, M=4, K=300, x=A, t=A, suffix=""):
        return call("fp8_requant_act_128x1_t" + suffix, q, s, M, K, x, t, N)

    def turn_pow2(**kw):
        return turn(suffix="_pow2", **kw)

    for go in (read, turn, turn_pow2):
        for bad in (dict(M=-1), dict(K=-1), dict(M=BIG), dict(K=BIG), dict(M=1 << 30, K=1 << 10),
                    dict(M=1 << 20, K=1 << 19)):
            assert go(**bad) == B.FP8_ERR_SHAPE, bad
        assert go(q=N) == go(s=N) == go(x=N) == B.FP8_ERR_NULL
        assert go(s=A2) == B.FP8_ERR_ALIGN
        assert go(M=0, q=N) == go(K=0, x=N) == B.FP8_OK
    assert read(t=2) == B.FP8_ERR_DTYPE
    assert read(x=ODD) == read(x=A2, t=F32) == B.FP8_ERR_ALIGN
    assert turn(t=N) == B.FP8_ERR_NULL and turn(t=A2) == B.FP8_ERR_ALIGN


def test_checkpoint_limits():
    # M ceil(K/8) below 2^32 - 256, ceil(M/128) ceil(K/128) below 2^23, of which
    # the second keeps a row's fp32 values below 2^32 bytes
    for M, K in ((1, 1 << 30), (128, (1 << 30) - 127), (BIG - 1, 9), ((1 << 31) - 128, 16),
                 (129, 1 << 29)):
        for name, rest in (("fp8_dequant_act_1x128", (A, F32, N)),
                           ("fp8_dequant_act_1x128", (A, BF16, N)),
                           ("fp8_requant_act_128x1_t", (A, A, N)),
                           ("fp8_requant_act_128x1_t_pow2", (A, A, N))):
            assert call(name, A, A, M, K, *rest) == B.FP8_ERR_SHAPE, (M, K, name)


@pytest.mark.parametrize("suffix", ["", "_pow2"])
def test_grouped_dgrad_errors(suffix):
    def go(dy=A, sdy=A, w=A, sw=A, off=A, E=3, T=4, dx=A, t=BF16, n=256, k=128):
        return call("fp8_block_grouped_gemm_dgrad" + suffix, dy, sdy, w, sw, off, E, T, dx, t, n,
                    k, N)
    assert go(t=2) == B.FP8_ERR_DTYPE
    for bad in (dict(T=-1), dict(n=-128), dict(k=-128), dict(n=64), dict(k=64), dict(T=BIG),
                dict(n=1 << 24), dict(n=1 << 17, k=1 << 15), dict(E=0), dict(E=-1),
                dict(E=1 << 20), dict(n=0), dict(T=1 << 30, n=1 << 12)):
        assert go(**bad) == B.FP8_ERR_SHAPE, bad
    for what in ("dy", "sdy", "w", "sw", "off", "dx"):
        assert go(**{what: N}) == B.FP8_ERR_NULL, what
    for what, at in (("dy", A8), ("w", A8), ("dx", A8), ("sdy", A2), ("sw", A2), ("off", A2)):
        assert go(**{what: at}) == B.FP8_ERR_ALIGN, what
    assert go(T=0, dy=N) == go(k=0, w=N) == go(T=0, E=0) == B.FP8_OK


# ---- the Python layer ----------------------------------------------------------------

BF, FP, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
M, I, K, E = 4, 256, 384, 3
OPERANDS = {"a": (U8, M, K), "a_scales": (FP, M, K // 128), "w": (U8, 2 * I, K),
            "w_scales": (FP, 2 * I // 128, K // 128)}
GROUPED = {"a": (U8, M, K), "a_scales": (FP, M, K // 128), "w": (U8, E, 2 * I, K),
           "w_scales": (FP, E, 2 * I // 128, K // 128), "group_offsets": (I32, E + 1)}
OUT = {"out": (BF, M, I)}
QUANT = {"q": (U8, M, I), "scales": (FP, M, I // 128)}
KEPT = dict(QUANT, h=(U8, M, 2 * I), h_scales=(FP, M, I // 64))
GRAD = {"da": (BF, M, I), "h": (U8, M, 2 * I), "h_scales": (FP, M, I // 64)}
ROWS = {"q": (U8, M, 2 * I), "scales": (FP, M, I // 64)}
TURNED = dict(ROWS, q_t=(U8, 2 * I, M), scales_t=(FP, 2 * I, 1), a_t=(U8, I, M),
              a_scales_t=(FP, I, 1))
STORED = {"q": (U8, M, 300), "scales": (FP, M, 3)}
DGRAD = {"dy": (U8, M, 2 * I), "dy_scales": (FP, M, I // 64), "w": (U8, E, 2 * I, K),
         "w_scales": (FP, E, 2 * I // 128, K // 128), "group_offsets": (I32, E + 1)}
WORK = {"workspace": (U8, 64)}


def kept(fn):
    return lambda *args, **kw: fn(*args, checkpoint=True, **kw)


CALLS = {}
for s_ in ("", "_pow2"):
    CALLS["gated" + s_] = (getattr(L, "fp8_block_gemm_gated" + s_), OPERANDS, dict(OUT, **WORK))
    CALLS["gated_quant" + s_] = (kept(getattr(L, "fp8_block_gemm_gated_quant_1x128" + s_)),
                                 OPERANDS, dict(KEPT, **WORK))
    CALLS["grouped" + s_] = (getattr(L, "fp8_block_grouped_gemm_gated" + s_), GROUPED,
                             dict(OUT, **WORK))
    CALLS["grouped_quant" + s_] = (
        kept(getattr(L, "fp8_block_grouped_gemm_gated_quant_1x128" + s_)), GROUPED,
        dict(KEPT, **WORK))
    CALLS["grad_rows" + s_] = (getattr(L, "fp8_gated_grad_quant_1x128" + s_), GRAD, ROWS)
    CALLS["grad_quant" + s_] = (getattr(L, "fp8_gated_grad_quant" + s_), GRAD, TURNED)
    CALLS["requant" + s_] = (getattr(L, "fp8_requant_act_128x1_t" + s_), STORED,
                             {"q_t": (U8, 300, M), "scales_t": (FP, 300, 1)})
    CALLS["dgrad" + s_] = (getattr(L, "fp8_block_grouped_gemm_dgrad" + s_), DGRAD,
                           {"dx": (BF, M, K)})
CALLS["grad"] = (L.fp8_gated_grad, GRAD, {"dh": (BF, M, 2 * I)})
CALLS["dequant"] = (L.fp8_dequant_act_1x128, STORED, {"x": (BF, M, 300)})


def new(dtype, *shape):
    return torch.zeros(shape, dtype=dtype)


def given(specs):
    return {name: new(*spec) for name, spec in specs.items()}


@pytest.mark.parametrize("name", list(CALLS))
def test_good_arguments_get_as_far_as_asking_for_the_gpu(name):
    fn, ins, outs = CALLS[name]
    with pytest.raises(ValueError, match="on the GPU"):
        fn(*given(ins).values())
    with pytest.raises(ValueError, match="on the GPU"):
        fn(*given(ins).values(), **given(outs))


def variants(spec):
    """Tensors that are not of that shape and type."""
    dtype, *shape = spec
    yield torch.float64, shape
    yield dtype, [*shape[:-1], shape[-1] + 128]
    yield dtype, [shape[0] + 1, *shape[1:]]
    yield dtype, [1, *shape]
    yield dtype, shape[1:]


BAD = [(call, arg, v) for call, (_, ins, outs) in CALLS.items()
       for arg in list(ins) + [o for o in outs if o != "workspace"] for v in range(5)]


@pytest.mark.parametrize("name,arg,v", BAD, ids=["-".join(map(str, b)) for b in BAD])
def test_wrong_shapes_and_types_are_refused(name, arg, v):
    fn, ins, outs = CALLS[name]
    args, outs_given = given(ins), given(outs)
    where = args if arg in ins else outs_given
    dtype, shape = list(variants((ins.get(arg) or outs[arg])))[v]
    where[arg] = torch.zeros(shape, dtype=dtype)
    with pytest.raises((ValueError, TypeError)) as e:
        fn(*args.values(), **outs_given)
    assert "on the GPU" not in str(e.value)
    where[arg] = None if arg not in ("h_scales",) else "x"
    if arg in ins:
        with pytest.raises((ValueError, TypeError)) as e:
            fn(*args.values(), **outs_given)
        assert "on the GPU" not in str(e.value)


STRIDED = {("grad", "da"), ("grad", "h"), ("grad_rows", "da"), ("grad_rows", "h"),
           ("grad_quant", "da"), ("grad_quant", "h"), ("grad_rows_pow2", "da"),
           ("grad_rows_pow2", "h"), ("grad_quant_pow2", "da"), ("grad_quant_pow2", "h")}


@pytest.mark.parametrize("name", list(CALLS))
def test_strides(name):
    # rows apart only where the call says so, values of a row apart nowhere
    fn, ins, outs = CALLS[name]
    for arg, (dtype, *shape) in {**ins, **outs}.items():
        if len(shape) < 2:
            continue
        for axis in (len(shape) - 1, 0):
            if shape[axis] == 1 or arg == "workspace":
                continue
            args, outs_given = given(ins), given(outs)
            wide = list(shape)
            wide[axis] *= 2
            if axis == 0 and len(shape) == 2:  # a part of wider rows
                t = torch.zeros((shape[0], 2 * shape[1]), dtype=dtype)[:, :shape[1]]
            else:
                t = torch.zeros(wide, dtype=dtype)
                t = t[::2] if axis == 0 else t[..., ::2]
            if t.is_contiguous():
                continue
            (args if arg in ins else outs_given)[arg] = t
            ok = axis == 0 and (name, arg) in STRIDED
            with pytest.raises(ValueError, match="on the GPU" if ok else "contiguous|adjacent"):
                fn(*args.values(), **outs_given)


def over(whole, spec, at=0):
    dtype, *shape = spec
    size = torch.Size(shape).numel() * dtype.itemsize
    return whole[at:at + size].view(dtype).reshape(shape)


PAIRS = [(call, out, other) for call, (_, ins, outs) in CALLS.items() for out in outs
         for other in list(ins) + [o for o in outs if o != out]]


@pytest.mark.parametrize("name,out,other", PAIRS, ids=["-".join(p) for p in PAIRS])
def test_shared_memory_is_refused(name, out, other):
    fn, ins, outs = CALLS[name]
    args, whole = given(ins), new(U8, 1 << 22)
    spec = ins.get(other) or outs[other]
    size = torch.Size(spec[1:]).numel() * spec[0].itemsize
    for at in (0, (size - 1) // 8 * 8):
        outs_given = {}
        (args if other in ins else outs_given)[other] = over(whole, spec)
        outs_given[out] = over(whole, outs[out], at)
        with pytest.raises(ValueError, match="share memory"):
            fn(*args.values(), **outs_given)


def test_other_refusals():
    args = given(OPERANDS)
    with pytest.raises(ValueError, match="activation"):
        L.fp8_block_gemm_gated(*args.values(), activation="relu")
    with pytest.raises(ValueError, match="activation"):
        L.fp8_gated_grad(*given(GRAD).values(), activation=None)
    with pytest.raises(ValueError, match="out_dtype"):
        L.fp8_block_gemm_gated(*args.values(), out_dtype="f16")
    with pytest.raises(ValueError, match="without checkpoint"):
        L.fp8_block_gemm_gated_quant_1x128(*args.values(), h=new(U8, M, 2 * I))
    with pytest.raises(TypeError, match="workspace"):
        L.fp8_block_gemm_gated(*args.values(), workspace=5)
    with pytest.raises(ValueError, match="workspace"):
        L.fp8_block_gemm_gated(*args.values(), workspace=new(U8, 8, 8)[:, :4])
    # three blocks of 128 rows are not two halves
    args["w"], args["w_scales"] = new(U8, 384, K), new(FP, 3, 3)
    with pytest.raises(ValueError, match="two parts"):
        L.fp8_block_gemm_gated(*args.values())
    # bf16 projections have no scales, and 8-bit ones need them
    with pytest.raises(TypeError, match="h must be"):
        L.fp8_gated_grad(new(BF, M, I), new(U8, M, 2 * I))
    with pytest.raises(TypeError, match="h must be"):
        L.fp8_gated_grad(new(BF, M, I), new(BF, M, 2 * I), new(FP, M, I // 64))
