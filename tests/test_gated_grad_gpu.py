"""Gradient of the activation and the product, and 8-bit checkpoints, on the
GPU.

The fp32 gradient is compared with the formulas in 64 bits (and those with
differences of the 64-bit activation); every other form is the same fp32 values
rounded or quantized, so it is compared with the fp32 result bit for bit.  (a =
act(g) u comes in fp32 as the du of da = u, the same product.)
"""
import numpy as np
import pytest

import fp8_fine_grained_token_amd as F
from fp8_fine_grained_token_amd import binding as B

from .ffn_util import ACTS, act64, quantized, same_quantized, sigmoid_error
from .gpu_util import U32, e4m3_lut, host, torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    t = torch()
    if not t.cuda.is_available():
        pytest.skip("no GPU")
    B.lib()
    yield
    t.cuda.synchronize()


def inputs(seed, M, I, da_type="bf16", kept="e4m3", sigma=3.0, pow2=False):
    """(da, h, h_scales) on the GPU and (da, h) as fp32 numpy."""
    t = torch()
    rng = np.random.default_rng(seed)
    da = rng.standard_normal((M, I), dtype=np.float32)
    h = rng.standard_normal((M, 2 * I), dtype=np.float32) * np.float32(sigma)
    h[rng.random((M, 2 * I)) < 0.02] *= 30
    da = t.from_numpy(da).cuda().to(t.bfloat16 if da_type == "bf16" else t.float32)
    if kept == "e4m3":
        q, s = quantized(h, pow2)
        h = t.from_numpy(np.ascontiguousarray(q)).cuda()
        s = t.from_numpy(s).cuda()
        hf = (e4m3_lut()[q].astype(np.float32) * np.repeat(s.cpu().numpy(), 128, 1))
        return da, h, s, host(da), hf
    h = t.from_numpy(h).cuda().to(t.bfloat16)
    return da, h, None, host(da), host(h)


def check_grad(dh, da, h, act):
    """fp32 dh against the formulas.  With s off by e(s) relatively, 1 - s by
    s e(s) + 2^-24: act = g s by (e(s) + 2^-24) |act|; t = s (1 - s) by e(s) t + s
    (s e(s) + 2^-24) + 2^-24 t; g z' of GELU by 4 roundings; the sum s + g z' t
    and the products round once each."""
    I = da.shape[1]
    g, u, d = h[:, :I].astype(np.float64), h[:, I:].astype(np.float64), da.astype(np.float64)
    a, slope, z, s, gz = act64(g, act)
    e = sigmoid_error(z, s, act)
    with np.errstate(over="ignore"):
        r = 1 / (1 + np.exp(z))
    tau = s * r
    dt = e * tau + s * (s * e + U32) + 2 * U32 * tau
    dslope = s * e + gz * (dt + 5 * U32 * tau) + U32 * (s + gz * tau)
    dg, du = d * u * slope, d * a
    tiny = (np.abs(d) + 1) * (np.abs(u) + 1) * (np.abs(g) + 1) ** 3 * 2.0 ** -120
    b_dg = np.abs(d * u) * (dslope * (1 + 3 * U32) + 3 * U32 * np.abs(slope)) + tiny
    b_du = np.abs(du) * (e + 3 * U32) + tiny
    for what, got, want, bound in (("dg", dh[:, :I], dg, b_dg), ("du", dh[:, I:], du, b_du)):
        bad = np.abs(got - want) > bound
        assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4], got[bad][:4],
                               want[bad][:4])


SIZES = [(1, 128), (2, 384), (7, 128), (8, 256), (127, 128), (128, 128), (129, 256), (333, 640),
         (1000, 128)]


@pytest.mark.parametrize("da_type", ["bf16", "f32"])
@pytest.mark.parametrize("kept", ["e4m3", "bf16"])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,I", SIZES)
def test_against_the_formulas(M, I, act, kept, da_type):
    t = torch()
    da, h, s, da_np, h_np = inputs(M * 7 + I, M, I, da_type, kept)
    dh = F.fp8_gated_grad(da, h, s, act, out_dtype="f32")
    check_grad(host(dh), da_np, h_np, act)
    assert t.equal(F.fp8_gated_grad(da, h, s, act), dh.bfloat16())
    # a in fp32
    u = t.from_numpy(np.ascontiguousarray(h_np[:, I:])).cuda()
    a = F.fp8_gated_grad(u, h, s, act, out_dtype="f32")[:, I:].contiguous()
    dh, a = host(dh), host(a)
    for pow2 in (False, True):
        suffix = "_pow2" if pow2 else ""
        rows = getattr(F, "fp8_gated_grad_quant_1x128" + suffix)(da, h, s, act)
        same_quantized(*rows, dh, pow2, "rows")
        every = getattr(F, "fp8_gated_grad_quant" + suffix)(da, h, s, act)
        same_quantized(*every[:2], dh, pow2, "rows of all")
        same_quantized(*every[2:4], np.ascontiguousarray(dh.T), pow2, "turned")
        same_quantized(*every[4:], np.ascontiguousarray(a.T), pow2, "a turned")


@pytest.mark.parametrize("act", ACTS)
def test_formulas_against_differences(act):
    # what the tests hold the kernels to is the derivative of a
    rng = np.random.default_rng(0)
    g, u, da = (rng.standard_normal(2000) * 3 for _ in range(3))
    a, slope, *_ = act64(g, act)
    eps = 1e-6
    up, down = act64(g + eps, act)[0], act64(g - eps, act)[0]
    assert np.allclose(da * u * (up - down) / (2 * eps), da * u * slope, rtol=1e-7, atol=1e-7)
    assert np.allclose(da * (a * (u + eps) - a * (u - eps)) / (2 * eps), da * a, rtol=1e-7,
                       atol=1e-7)


@pytest.mark.parametrize("act", ACTS)
def test_kernel_against_differences(act):
    # fp32 gradient of sum(da a) against central differences in 64 bits, every
    # column shifted by itself: off by the kernel's few roundings and, for a
    # step of 1e-4, third derivatives below 2 times 1e-8 / 6
    da, h, s, da_np, h_np = inputs(11, 5, 128, "f32", "bf16", sigma=2.0)
    h_np = np.clip(h_np, -8, 8)
    h = torch().from_numpy(h_np).cuda().bfloat16()
    dh = host(F.fp8_gated_grad(da, h, None, act, out_dtype="f32"))
    g, u, d = (x.astype(np.float64) for x in (h_np[:, :128], h_np[:, 128:], da_np))
    eps = 1e-4
    dg = d * u * (act64(g + eps, act)[0] - act64(g - eps, act)[0]) / (2 * eps)
    du = d * (act64(g, act)[0] * (u + eps) - act64(g, act)[0] * (u - eps)) / (2 * eps)
    scale = np.abs(d) * (np.abs(u) + np.abs(g) + 1)
    assert (np.abs(dh[:, :128] - dg) <= scale * (1e-8 + 40 * U32)).all()
    assert (np.abs(dh[:, 128:] - du) <= scale * (1e-8 + 40 * U32)).all()


@pytest.mark.parametrize("da_type", ["bf16", "f32"])
@pytest.mark.parametrize("act", ACTS)
def test_shut_gates_of_large_products(act, da_type):
    # da u is past the largest fp32 value, da u act'(g) is not: 0 where the gate
    # is shut, finite where it nearly is
    t = torch()
    I = 128
    gates = np.array([-300.0, -120.0, -90.0, -20.0, -6.0, -4.5], np.float32)
    h_np = np.repeat(gates, 2)[:, None].repeat(2 * I, 1)
    da_np = np.full((12, I), 2.0 ** 64, np.float32)
    h_np[:, I:] = 2.0 ** 66
    da_np[1::2] *= -1
    da = t.from_numpy(da_np).cuda().to(t.bfloat16 if da_type == "bf16" else t.float32)
    h = t.from_numpy(h_np).cuda().bfloat16()
    want = da_np.astype(np.float64) * h_np[:, I:] * act64(h_np[:, :I], act)[1]
    assert np.abs(want).max() < 2.0 ** 127 and np.abs(want).max() > 0
    dh = F.fp8_gated_grad(da, h, None, act, out_dtype="f32")
    assert t.isfinite(dh).all()
    check_grad(host(dh), da_np, h_np, act)
    for pow2 in ("", "_pow2"):
        for part in getattr(F, "fp8_gated_grad_quant" + pow2)(da, h, None, act)[1::2]:
            assert t.isfinite(part).all()


@pytest.mark.parametrize("kept", ["e4m3", "bf16"])
@pytest.mark.parametrize("da_type", ["bf16", "f32"])
def test_strides_and_alignments(kept, da_type):
    # rows apart, the first value on any element's alignment, one row repeated
    t = torch()
    M, I = 137, 256
    da, h, s, _, _ = inputs(3, M, I, da_type, kept)
    want = F.fp8_gated_grad_quant(da, h, s)
    dense = F.fp8_gated_grad(da, h, s, out_dtype="f32")
    for pad, first in ((5, 1), (8, 8), (3, 0)):
        wide_da = t.full((M, I + pad + first), float("nan"), dtype=da.dtype, device="cuda")
        wide_h = t.full((M, 2 * I + pad + first), 0x7F if kept == "e4m3" else float("nan"),
                        dtype=h.dtype, device="cuda")
        x, y = wide_da[:, first:first + I], wide_h[:, first:first + 2 * I]
        x.copy_(da)
        y.copy_(h)
        for a, b in zip(F.fp8_gated_grad_quant(x, y, s), want):
            assert t.equal(a, b)
        assert t.equal(F.fp8_gated_grad(x, y, s, out_dtype="f32"), dense)
    one = da[:1].expand(M, I)
    assert t.equal(F.fp8_gated_grad(one, h, s), F.fp8_gated_grad(one.contiguous(), h, s))


@pytest.mark.parametrize("M", [1, 13, 200])
def test_some_of_the_parts_and_given_outputs(M):
    # each pair alone through the C entry, and outputs given by the caller
    import ctypes
    from fp8_fine_grained_token_amd import ffn as L
    t = torch()
    I = 256
    da, h, s, _, _ = inputs(5, M, I)
    want = F.fp8_gated_grad_quant(da, h, s)
    stream = ctypes.c_void_p(t.cuda.current_stream().cuda_stream)
    for parts in ((0,), (1,), (2,), (0, 2), (1, 2), (0, 1)):
        outs = [t.full_like(x, 5) for x in want]
        L._call("fp8_gated_grad_quant", da.data_ptr(), 1, I, h.data_ptr(), 2 * I, s.data_ptr(), 0,
                M, I, *(x.data_ptr() if i // 2 in parts else None for i, x in enumerate(outs)),
                stream)
        for i, (x, y) in enumerate(zip(outs, want)):
            assert t.equal(x, y) if i // 2 in parts else (x == 5).all(), (parts, i)
    outs = [t.full_like(x, 5) for x in want]
    for x, y, z in zip(F.fp8_gated_grad_quant(da, h, s, "silu", *outs), want, outs):
        assert x is z and t.equal(x, y)
    dh = t.zeros((M, 2 * I), device="cuda")
    assert F.fp8_gated_grad(da, h, s, out_dtype="f32", dh=dh) is dh


def test_outputs_on_odd_addresses():
    # transposed bytes and fp32 results on the alignment of one element
    t = torch()
    M, I = 77, 128
    da, h, s, _, _ = inputs(6, M, I)
    want = F.fp8_gated_grad_quant(da, h, s)
    raw = t.zeros(2 * I * M + 64, dtype=t.uint8, device="cuda")
    q_t = raw[3:3 + 2 * I * M].view(2 * I, M)
    a_raw = t.zeros(I * M + 64, dtype=t.uint8, device="cuda")
    a_t = a_raw[1:1 + I * M].view(I, M)
    got = F.fp8_gated_grad_quant(da, h, s, q_t=q_t, a_t=a_t)
    for x, y in zip(got, want):
        assert t.equal(x, y)
    assert not raw[:3].any() and not raw[3 + 2 * I * M:].any()
    assert not a_raw[:1].any() and not a_raw[1 + I * M:].any()
    dh = t.zeros(M * 2 * I + 1, device="cuda")[1:].view(M, 2 * I)
    F.fp8_gated_grad(da, h, s, out_dtype="f32", dh=dh)
    assert t.equal(dh, F.fp8_gated_grad(da, h, s, out_dtype="f32"))
    bf = t.zeros(M * 2 * I + 1, dtype=t.bfloat16, device="cuda")[1:].view(M, 2 * I)
    assert t.equal(F.fp8_gated_grad(da, h, s, dh=bf), F.fp8_gated_grad(da, h, s))


@pytest.mark.parametrize("act", ACTS)
def test_nan_and_infinity(act):
    # they reach their own column's outputs as the formulas have it, and the
    # scale groups that hold those
    t = torch()
    M, I = 140, 256
    da, h, _, _, _ = inputs(7, M, I, "f32", "bf16")
    clean = host(F.fp8_gated_grad(da, h, None, act, out_dtype="f32"))
    h[3, 5] = float("nan")       # g
    h[7, I + 200] = float("inf")  # u
    h[9, 130] = float("inf")      # g: act' = 1, act = g
    h[11, 131] = float("-inf")    # g: act' = 0, act = -inf 0
    h[20, 9] = 3e38               # g^3 overflows: still act' = 1
    h[21, 9] = -3e38              # act' = 0, act = -0
    da[15, 40] = float("nan")
    got = host(F.fp8_gated_grad(da, h, None, act, out_dtype="f32"))
    touched = {(3, 5), (7, 200), (9, 130), (11, 131), (20, 9), (21, 9), (15, 40)}
    same = (got == clean)
    for r, c in touched:
        same[r, c] = same[r, I + c] = True
    assert same.all(), np.argwhere(~same)[:5]
    d, u = host(da), host(h)[:, I:]
    assert np.isnan(got[3, 5]) and np.isnan(got[3, I + 5])
    assert np.isinf(got[7, 200]) and got[7, I + 200] == clean[7, I + 200]
    assert got[9, 130] == d[9, 130] * u[9, 130] and np.isinf(got[9, I + 130])
    assert got[11, 131] == 0 and np.isnan(got[11, I + 131])
    assert got[20, 9] == d[20, 9] * u[20, 9] and got[21, 9] == 0 and got[21, I + 9] == 0
    assert np.isnan(got[15, 40]) and np.isnan(got[15, I + 40])
    u32 = t.from_numpy(np.ascontiguousarray(u)).cuda()
    a = host(F.fp8_gated_grad(u32, h, None, act, out_dtype="f32")[:, I:].contiguous())
    for pow2 in (False, True):
        every = getattr(F, "fp8_gated_grad_quant" + ("_pow2" if pow2 else ""))(da, h, None, act)
        same_quantized(*every[:2], got, pow2)
        same_quantized(*every[2:4], np.ascontiguousarray(got.T), pow2)
        same_quantized(*every[4:], np.ascontiguousarray(a.T), pow2)


def test_nan_in_an_8_bit_checkpoint():
    t = torch()
    M, I = 130, 128
    da, h, s, _, _ = inputs(8, M, I)
    h[2, 7], s[5, 1] = 0x7F, float("inf")  # a NaN code of g, an infinite scale of u
    dh = host(F.fp8_gated_grad(da, h, s, out_dtype="f32"))
    assert np.isnan(dh[2, 7]) and np.isnan(dh[2, I + 7]) and not np.isnan(dh[2, 8])
    live = np.ones(M, bool)
    live[[2, 5]] = False
    assert np.isfinite(dh[live]).all() and not np.isfinite(dh[5, :I]).all()
    assert np.isfinite(dh[5, I:]).all()
    same_quantized(*F.fp8_gated_grad_quant(da, h, s)[2:4], np.ascontiguousarray(dh.T))


def test_no_rows_and_no_columns():
    t = torch()
    for M, I in ((0, 128), (3, 0)):
        da = t.zeros((M, I), dtype=t.bfloat16, device="cuda")
        h = t.zeros((M, 2 * I), dtype=t.bfloat16, device="cuda")
        assert F.fp8_gated_grad(da, h).shape == (M, 2 * I)
        every = F.fp8_gated_grad_quant(da, h)
        assert every[2].shape == (2 * I, M) and every[5].shape == (I, (M + 127) // 128)
    q, s = t.zeros((0, 5), dtype=t.uint8, device="cuda"), t.zeros((0, 1), device="cuda")
    assert F.fp8_dequant_act_1x128(q, s).shape == (0, 5)
    assert F.fp8_requant_act_128x1_t(q, s)[0].shape == (5, 0)


# ---- 8-bit checkpoints ---------------------------------------------------------------

def stored(seed, M, K, pow2=False):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((M, K), dtype=np.float32) * np.exp(rng.standard_normal((M, 1)) * 4)
    q, s = quantized(x.astype(np.float32), pow2)
    value = e4m3_lut()[q].astype(np.float32) * np.repeat(s, 128, 1)[:, :K]
    t = torch()
    return t.from_numpy(np.ascontiguousarray(q)).cuda(), t.from_numpy(s).cuda(), value


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("M,K", [(1, 1), (5, 3), (3, 7), (2, 8), (4, 9), (3, 127), (2, 128),
                                 (9, 129), (1, 1000), (130, 1001), (127, 256), (129, 384),
                                 (300, 135), (1, 7168)])
def test_read_back_and_turned(M, K, pow2):
    t = torch()
    q, s, value = stored(M + K, M, K, pow2)
    x = F.fp8_dequant_act_1x128(q, s, out_dtype="f32")
    assert (host(x).view(np.uint32) == value.view(np.uint32)).all()
    assert t.equal(F.fp8_dequant_act_1x128(q, s), x.bfloat16())
    for suffix in ("", "_pow2"):
        q_t, s_t = getattr(F, "fp8_requant_act_128x1_t" + suffix)(q, s)
        same_quantized(q_t, s_t, np.ascontiguousarray(value.T), suffix != "")


def test_turned_is_the_quantizer_of_the_values():
    # on values that bf16 holds exactly, the 128x1 quantizer's own bytes
    t = torch()
    x = (t.randint(-7, 8, (256, 384), device="cuda") * 0.5).bfloat16()
    q, s = F.fp8_quant_act_1x128_pow2(x)
    assert t.equal(F.fp8_dequant_act_1x128(q, s), x)
    for suffix in ("", "_pow2"):
        want = getattr(F, "fp8_quant_act_128x1_t" + suffix)(x)
        for a, b in zip(getattr(F, "fp8_requant_act_128x1_t" + suffix)(q, s), want):
            assert t.equal(a, b)


def test_every_code_and_extreme_scales():
    t = torch()
    codes = np.arange(256, dtype=np.uint8).reshape(2, 128)
    lut = e4m3_lut().copy()
    lut[[0x7F, 0xFF]] = np.nan
    for scale in (1.0, 2.0 ** -126, 2.0 ** -140, 1e38, 0.0, np.inf, np.nan):
        q = t.from_numpy(codes).cuda()
        s = t.full((2, 1), scale, device="cuda")
        with np.errstate(all="ignore"):
            want = lut[codes].astype(np.float32) * np.float32(scale)
        got = host(F.fp8_dequant_act_1x128(q, s, out_dtype="f32"))
        assert ((got == want) | (np.isnan(got) & np.isnan(want))).all(), scale
        same_quantized(*F.fp8_requant_act_128x1_t(q, s), np.ascontiguousarray(want.T))


def test_read_back_and_turned_on_odd_addresses():
    t = torch()
    M, K = 37, 203
    q, s, _ = stored(4, M, K)
    want_x, want = F.fp8_dequant_act_1x128(q, s), F.fp8_requant_act_128x1_t(q, s)
    raw = t.full((M * K + 9,), 0x7F, dtype=t.uint8, device="cuda")
    src = raw[5:5 + M * K].view(M, K)
    src.copy_(q)
    out = t.zeros(M * K + 3, dtype=t.bfloat16, device="cuda")
    assert t.equal(F.fp8_dequant_act_1x128(src, s, x=out[1:1 + M * K].view(M, K)), want_x)
    assert out[0] == 0 and not out[1 + M * K:].any()
    back = t.zeros(M * K + 3, dtype=t.uint8, device="cuda")
    q_t, s_t = F.fp8_requant_act_128x1_t(src, s, q_t=back[1:1 + M * K].view(K, M))
    assert t.equal(q_t, want[0]) and t.equal(s_t, want[1])
    assert back[0] == 0 and not back[1 + M * K:].any()
