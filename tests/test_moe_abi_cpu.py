"""Contract of the operators around the expert products that needs no GPU:
the library exports what include/fp8moe.h declares, bad arguments are refused
with the documented status before anything is launched, and the Python layer
refuses tensors the kernels could not index (every call here fails validation
or is a documented no-op)."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

from fp8_fine_grained_token_amd import binding as B
from fp8_fine_grained_token_amd import moe as M

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A, ODD = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10001)
N = ctypes.c_void_p(0)
F32, BF16 = B.FP8_OUT_F32, B.FP8_OUT_BF16
BIG = 1 << 31


def call(name, *args):
    return M._fn(name)(*args)


def declared():
    text = open(os.path.join(ROOT, "include", "fp8moe.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return set(re.findall(r"\b(fp8_[a-z0-9_]+)\s*\(", text))


def test_every_declared_symbol_is_exported_and_bound():
    assert declared() == set(M._SIGNATURES)
    for name in declared():
        assert hasattr(B.lib(), name), name
    import fp8_fine_grained_token_amd as F
    for name in declared():
        assert getattr(F, name) is getattr(M, name)


def test_header_is_plain_c():
    # a C99 program that includes the header and names every function
    names = sorted(declared())
    program = "#include \"fp8moe.h\"\n" + "".join(
        f"void *p{i} = (void *)&{n};\n" for i, n in enumerate(names))
    r = subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-fsyntax-only", "-x", "c",
                        "-I" + os.path.join(ROOT, "include"), "-"], input=program, text=True,
                       capture_output=True)
    assert r.returncode == 0, r.stderr


def sort(ids=A, b=8, T=4, k=2, E=8, off=A, sr=A, rs=A, ws=N, wsb=0):
    return call("fp8_moe_sort", ids, b, T, k, E, off, sr, rs, ws, wsb, N)


def test_sort_errors():
    assert sort(b=2) == B.FP8_ERR_DTYPE
    assert sort(T=-1) == sort(k=-1) == sort(E=0) == sort(E=1025) == B.FP8_ERR_SHAPE
    assert sort(T=1 << 20, k=1 << 11) == B.FP8_ERR_SHAPE
    assert sort(ids=N) == sort(off=N) == sort(sr=N) == sort(rs=N) == B.FP8_ERR_NULL
    assert sort(off=N, T=0) == B.FP8_ERR_NULL
    assert sort(ids=ctypes.c_void_p(0x10004)) == B.FP8_ERR_ALIGN
    assert sort(off=ODD) == sort(sr=ODD) == sort(rs=ODD) == B.FP8_ERR_ALIGN
    need = M.fp8_moe_sort_workspace_bytes(1000, 8, 64)
    assert need > 0 and M.fp8_moe_sort_workspace_bytes(1, 8, 64) == 0
    assert sort(T=1000, k=8, E=64) == B.FP8_ERR_WORKSPACE
    assert sort(T=1000, k=8, E=64, ws=A, wsb=need - 1) == B.FP8_ERR_WORKSPACE
    assert sort(T=1000, k=8, E=64, ws=ODD, wsb=need) == B.FP8_ERR_WORKSPACE
    assert M.fp8_moe_sort_workspace_bytes(-1, 8, 64) == 0


def test_dispatch_errors():
    def go(x=A, b=2, ld=64, xs_=N, T=4, H=64, G=0, sr=A, k=2, xs=A, xss=N, R=8, lds=0):
        return call("fp8_moe_dispatch", x, b, ld, xs_, lds, T, H, G, sr, k, xs, xss, R, N)
    assert go(b=3) == B.FP8_ERR_DTYPE
    assert go(T=-1) == go(H=-1) == go(k=-1) == go(R=-1) == go(ld=-1) == B.FP8_ERR_SHAPE
    assert go(T=BIG) == go(H=BIG) == go(R=BIG) == go(T=1 << 20, k=1 << 11) == B.FP8_ERR_SHAPE
    assert go(ld=1 << 39) == B.FP8_ERR_SHAPE
    assert go(xs_=A, xss=A, G=-1) == B.FP8_ERR_SHAPE
    assert go(x=N) == go(sr=N) == go(xs=N) == go(xs_=A, G=2) == go(xss=A) == B.FP8_ERR_NULL
    assert go(x=ODD) == go(xs=ODD) == go(sr=ODD) == B.FP8_ERR_ALIGN
    assert go(x=N, sr=N, xs=N, T=0) == go(x=N, xs=N, H=0) == B.FP8_OK

    for name in ("fp8_moe_dispatch_quant_1x128", "fp8_moe_dispatch_quant_1x128_pow2"):
        def quant(x=A, ld=64, T=4, H=64, sr=A, k=2, q=A, s=A, R=8):
            return call(name, x, ld, T, H, sr, k, q, s, R, N)
        assert quant(H=-1) == quant(ld=-1) == B.FP8_ERR_SHAPE
        assert quant(x=N) == quant(sr=N) == quant(q=N) == quant(s=N) == B.FP8_ERR_NULL
        assert quant(x=ODD) == quant(s=ODD) == B.FP8_ERR_ALIGN
        assert quant(T=0, x=N, sr=N) == B.FP8_OK


def test_sort_dispatch_errors():
    def go(x=A, b=2, ld=64, T=4, H=64, ids=A, ib=8, k=2, E=8, xs=A):
        return call("fp8_moe_sort_dispatch", x, b, ld, T, H, ids, ib, k, E, A, A, A, xs, N, 0, N)
    assert go(b=8) == go(ib=3) == B.FP8_ERR_DTYPE
    assert go(T=-1) == go(H=-1) == go(E=0) == go(ld=-2) == B.FP8_ERR_SHAPE
    assert go(x=N) == go(ids=N) == go(xs=N) == B.FP8_ERR_NULL
    assert go(x=ODD) == go(xs=ODD) == B.FP8_ERR_ALIGN
    for name in ("fp8_moe_sort_dispatch_quant_1x128", "fp8_moe_sort_dispatch_quant_1x128_pow2"):
        def quant(x=A, ld=64, T=4, H=64, ids=A, ib=8, k=2, E=8, q=A, s=A):
            return call(name, x, ld, T, H, ids, ib, k, E, A, A, A, q, s, N, 0, N)
        assert quant(ib=3) == B.FP8_ERR_DTYPE
        assert quant(H=-1) == quant(E=2000) == B.FP8_ERR_SHAPE
        assert quant(x=N) == quant(q=N) == quant(s=N) == B.FP8_ERR_NULL
        assert quant(T=3000, k=4) == B.FP8_ERR_WORKSPACE


def test_combine_errors():
    def go(ys=A, it=BF16, ld=64, R=8, sr=A, w=A, T=4, k=2, H=64, res=N, ldr=0, out=A, ot=BF16):
        return call("fp8_moe_combine", ys, it, ld, R, sr, w, T, k, H, res, ldr, out, ot, N)
    assert go(it=2) == go(ot=-1) == B.FP8_ERR_DTYPE
    assert go(T=-1) == go(R=-1) == go(H=-1) == go(ld=-1) == go(res=A, ldr=-1) == B.FP8_ERR_SHAPE
    assert go(ys=N) == go(sr=N) == go(out=N) == B.FP8_ERR_NULL
    assert go(ys=ODD) == go(out=ODD) == go(res=ODD) == go(w=ODD) == B.FP8_ERR_ALIGN
    assert go(T=0, ys=N, out=N, sr=N) == B.FP8_OK
    assert call("fp8_moe_dispatch_grad", N, BF16, 64, 8, A, 4, 2, 64, A, BF16, N) == B.FP8_ERR_NULL

    def grad(d=A, ld=64, ys=A, ldy=64, t=BF16, R=8, sr=A, w=A, T=4, k=2, H=64, dys=A, dw=A):
        return call("fp8_moe_combine_grad", d, ld, ys, ldy, t, R, sr, w, T, k, H, dys, dw, N)
    assert grad(t=5) == B.FP8_ERR_DTYPE
    assert grad(ld=-1) == grad(ldy=-1) == grad(k=-1) == B.FP8_ERR_SHAPE
    assert grad(d=N) == grad(ys=N) == grad(sr=N) == B.FP8_ERR_NULL
    assert grad(d=ODD) == grad(dys=ODD) == grad(dw=ODD) == grad(w=ODD) == B.FP8_ERR_ALIGN
    assert grad(dys=N, dw=N) == grad(T=0, d=N) == B.FP8_OK


def test_norm_errors():
    def go(name="fp8_norm_residual", y=A, yt=BF16, ldy=64, r=A, rt=BF16, ldr=64, wp=A, g=A, wq=A,
           pt=F32, T=4, H=64, gr=1, out=A, tail=(A, A, A)):
        return call(name, y, yt, ldy, r, rt, ldr, wp, g, wq, pt, T, H, gr, 1, 1.0, 1.0, 1e-6, out,
                    *tail, N)
    assert go(yt=2) == go(rt=2) == go(pt=2) == go(yt=F32, rt=BF16) == B.FP8_ERR_DTYPE
    assert go(T=-1) == go(H=-1) == go(H=32769) == go(ldy=-1) == go(ldr=-1) == B.FP8_ERR_SHAPE
    assert go(gr=0) == go(gr=3) == go(gr=-1) == B.FP8_ERR_SHAPE
    assert go(y=N) == go(r=N) == go(out=N) == B.FP8_ERR_NULL
    assert go(y=ODD) == go(r=ODD) == go(wp=ODD) == go(g=ODD) == go(out=ODD) == B.FP8_ERR_ALIGN
    assert go(tail=(ODD, A, A)) == go(tail=(A, ODD, A)) == B.FP8_ERR_ALIGN
    assert go(T=0, y=N, r=N, out=N) == B.FP8_OK
    for name in ("fp8_norm_residual_quant_1x128", "fp8_norm_residual_quant_1x128_pow2"):
        assert go(name, tail=(N, N, A, A, A)) == go(name, tail=(N, A, N, A, A)) == B.FP8_ERR_NULL
        assert go(name, tail=(N, A, ODD, A, A)) == B.FP8_ERR_ALIGN

    need = M.fp8_norm_residual_grad_workspace_bytes(4, 64, 1)
    assert need > 0 and M.fp8_norm_residual_grad_workspace_bytes(4, 64, 3) == 0

    def grad(dn=A, dro=A, y=A, yt=BF16, r=A, rt=BF16, s1=A, s2=A, wp=A, g=A, T=4, H=64, gr=1,
             post=1, dy=A, dr=A, dwp=A, dg=A, dwq=A, ws=A, wsb=need, ld=64):
        return call("fp8_norm_residual_grad", dn, ld, dro, 64, y, yt, 64, r, rt, 64, s1, s2, wp,
                    g, A, F32, T, H, gr, post, 1.0, 1.0, dy, dr, dwp, dg, dwq, ws, wsb, N)
    assert grad(yt=9) == grad(yt=F32, rt=BF16) == B.FP8_ERR_DTYPE
    assert grad(T=-1) == grad(H=40000) == grad(gr=3) == grad(ld=-1) == B.FP8_ERR_SHAPE
    assert grad(y=N) == grad(dy=N) == grad(dr=N) == grad(s1=N) == grad(s2=N) == B.FP8_ERR_NULL
    assert grad(r=N) == grad(g=N) == grad(post=0) == B.FP8_ERR_NULL
    assert grad(ws=N) == grad(wsb=need - 1) == grad(ws=ODD) == B.FP8_ERR_WORKSPACE
    assert grad(dy=ODD) == grad(dwp=ODD) == grad(dn=ODD) == B.FP8_ERR_ALIGN


def test_w4_errors():
    for name in ("fp8_w4_quant_1x128", "fp8_w4_quant_1x32"):
        assert call(name, A, -1, 64, A, A, N) == call(name, A, 4, BIG, A, A, N) == B.FP8_ERR_SHAPE
        assert call(name, N, 4, 64, A, A, N) == call(name, A, 4, 64, A, N, N) == B.FP8_ERR_NULL
        assert call(name, ODD, 4, 64, A, A, N) == B.FP8_ERR_ALIGN
        assert call(name, N, 0, 64, N, N, N) == B.FP8_OK

    def go(x=A, ld=64, c=A, s=A, kind=0, R=2, n=8, K=64, y=A, t=BF16):
        return call("fp8_w4_matvec", x, ld, c, s, kind, R, n, K, y, t, N)
    assert go(kind=2) == go(t=4) == B.FP8_ERR_DTYPE
    assert go(R=-1) == go(n=-1) == go(K=-1) == go(ld=-1) == go(n=BIG) == B.FP8_ERR_SHAPE
    assert go(x=N) == go(c=N) == go(s=N) == go(y=N) == B.FP8_ERR_NULL
    assert go(x=ODD) == go(s=ODD) == go(y=ODD) == B.FP8_ERR_ALIGN
    assert go(R=0, x=N, y=N) == go(n=0, y=N) == B.FP8_OK

    def grouped(off=A, E=3, R=2, n=8):
        return call("fp8_w4_grouped_matvec", A, 64, A, A, 1, off, E, R, n, 64, A, BF16, N)
    assert grouped(E=-1) == grouped(E=0) == grouped(E=65536) == B.FP8_ERR_SHAPE
    assert grouped(off=N) == B.FP8_ERR_NULL and grouped(off=ODD) == B.FP8_ERR_ALIGN
    assert grouped(R=0, off=N) == B.FP8_OK


def test_widest_rows():
    # one past the documented limits: expert-ordered rows below 2^28 values,
    # 4-bit rows below 2^24
    H, K = 1 << 28, 1 << 24
    assert call("fp8_moe_combine", A, BF16, H, 8, A, A, 4, 2, H, N, 0, A, BF16,
                N) == B.FP8_ERR_SHAPE
    assert call("fp8_moe_combine_grad", A, H, A, H, BF16, 8, A, A, 4, 2, H, A, A,
                N) == B.FP8_ERR_SHAPE
    assert call("fp8_moe_dispatch_grad", A, BF16, H, 8, A, 4, 2, H, A, BF16, N) == B.FP8_ERR_SHAPE
    for suffix in ("", "_pow2"):
        assert call("fp8_moe_dispatch_quant_1x128" + suffix, A, H, 4, H, A, 2, A, A, 8,
                    N) == B.FP8_ERR_SHAPE
    assert call("fp8_w4_matvec", A, K, A, A, 1, 2, 8, K, A, BF16, N) == B.FP8_ERR_SHAPE
    assert call("fp8_w4_grouped_matvec", A, K, A, A, 1, A, 3, 2, 8, K, A, BF16,
                N) == B.FP8_ERR_SHAPE


# ---- the Python layer: refused before anything is launched ---------------------

def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def f32(*shape):
    return torch.zeros(shape)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


REFUSED = [
    (ValueError, "on the GPU", lambda: M.fp8_moe_sort(i32(4, 2), 8)),
    (TypeError, "expert_ids", lambda: M.fp8_moe_sort(f32(4, 2), 8)),
    (ValueError, "num_experts", lambda: M.fp8_moe_sort(i32(4, 2), 0)),
    (ValueError, "2-dimensional", lambda: M.fp8_moe_sort(i32(8), 4)),
    (ValueError, "contiguous", lambda: M.fp8_moe_sort(i32(4, 4)[:, :2], 4)),
    (ValueError, "slot_row must have", lambda: M.fp8_moe_sort(i32(4, 2), 8, slot_row=i32(2, 4))),
    (ValueError, "group_offsets must", lambda: M.fp8_moe_sort(i32(4, 2), 8, group_offsets=i32(8))),
    (ValueError, "slot_row must have", lambda: M.fp8_moe_dispatch(bf(4, 8), i32(3, 2))),
    (TypeError, "x must be", lambda: M.fp8_moe_dispatch(torch.zeros(4, 8, dtype=torch.int64),
                                                        i32(4, 2))),
    (ValueError, "adjacent", lambda: M.fp8_moe_dispatch(bf(8, 4).t(), i32(4, 2))),
    (ValueError, "xs_scales given", lambda: M.fp8_moe_dispatch(bf(4, 8), i32(4, 2),
                                                               xs_scales=f32(8, 1))),
    (ValueError, "scales must have 4", lambda: M.fp8_moe_dispatch(u8(4, 8), i32(4, 2),
                                                                  scales=f32(3, 1))),
    (ValueError, "xs must have", lambda: M.fp8_moe_dispatch(bf(4, 8), i32(4, 2), xs=bf(8, 9))),
    (TypeError, "x must be", lambda: M.fp8_moe_dispatch_quant_1x128(f32(4, 8), i32(4, 2))),
    (ValueError, "scales must have", lambda: M.fp8_moe_dispatch_quant_1x128(
        bf(4, 200), i32(4, 2), q=u8(8, 200), scales=f32(8, 1))),
    (ValueError, "expert_ids must have 4", lambda: M.fp8_moe_sort_dispatch(bf(4, 8), i32(5, 2), 3)),
    (ValueError, "q must have", lambda: M.fp8_moe_sort_dispatch_quant_1x128_pow2(
        bf(4, 8), i32(4, 2), 3, q=u8(4, 8))),
    (ValueError, "weights must have", lambda: M.fp8_moe_combine(bf(8, 8), i32(4, 2), f32(4, 3))),
    (TypeError, "residual must be", lambda: M.fp8_moe_combine(bf(8, 8), i32(4, 2),
                                                              residual=f32(4, 8))),
    (ValueError, "unsupported out_dtype", lambda: M.fp8_moe_combine(bf(8, 8), i32(4, 2),
                                                                    out_dtype="f16")),
    (ValueError, "out must have", lambda: M.fp8_moe_combine(bf(8, 8), i32(4, 2), out=bf(4, 9))),
    (TypeError, "ys must be", lambda: M.fp8_moe_combine_grad(bf(4, 8), f32(8, 8), i32(4, 2))),
    (ValueError, "ys must have", lambda: M.fp8_moe_combine_grad(bf(4, 8), bf(8, 9), i32(4, 2))),
    (ValueError, "r must have", lambda: M.fp8_norm_residual(bf(4, 8), bf(4, 9))),
    (TypeError, "r must be", lambda: M.fp8_norm_residual(f32(4, 8), bf(4, 8))),
    (ValueError, "w_post must have", lambda: M.fp8_norm_residual(bf(4, 8), bf(4, 8), f32(9))),
    (TypeError, "gate must be", lambda: M.fp8_norm_residual(bf(4, 8), bf(4, 8), f32(8), bf(8))),
    (ValueError, "divide", lambda: M.fp8_norm_residual(bf(4, 8), bf(4, 8), None, f32(3, 8))),
    (ValueError, "one of dn", lambda: M.fp8_norm_residual_grad(None, None, bf(4, 8), bf(4, 8),
                                                               f32(4), f32(4))),
    (ValueError, "rstd_pre must", lambda: M.fp8_norm_residual_grad(
        bf(4, 8), None, bf(4, 8), bf(4, 8), f32(4), f32(5))),
    (TypeError, "rstd_post", lambda: M.fp8_norm_residual_grad(
        bf(4, 8), None, bf(4, 8), bf(4, 8), None, f32(4))),
    (ValueError, "codes must have", lambda: M.fp8_w4_matvec(bf(2, 64), u8(8, 31), f32(8, 1))),
    (ValueError, "scales must have", lambda: M.fp8_w4_matvec(bf(2, 64), u8(8, 32), u8(8, 1))),
    (ValueError, "codes must have", lambda: M.fp8_w4_grouped_matvec(bf(2, 64), u8(8, 32),
                                                                    f32(8, 1), i32(2))),
    (ValueError, "group_offsets must", lambda: M.fp8_w4_grouped_matvec(
        bf(2, 64), u8(3, 8, 32), f32(3, 8, 1), i32(3))),
    (ValueError, "w must have", lambda: M.fp8_w4_quant_1x32(bf(64))),
]


@pytest.mark.parametrize("kind,text,make", REFUSED, ids=[str(i) for i in range(len(REFUSED))])
def test_python_layer_refuses(kind, text, make):
    with pytest.raises(kind, match=text):
        make()


def test_outputs_must_not_overlap_inputs():
    buf = bf(12, 8)
    with pytest.raises(ValueError, match="share memory"):
        M.fp8_moe_dispatch(buf[:4], i32(4, 2), xs=buf[2:10])
    with pytest.raises(ValueError, match="share memory"):
        M.fp8_moe_combine(buf[:8], i32(4, 2), out=buf[4:8])
    with pytest.raises(ValueError, match="share memory"):
        M.fp8_norm_residual(buf[:4], buf[4:8], n=buf[6:10])
    with pytest.raises(ValueError, match="share memory"):
        M.fp8_norm_residual(buf[:4], buf[4:8], r_out=buf[5:9])
