"""What the tests of the gated feed-forward operators share: the 1x128 rule
on fp32 values, the activation in 64 bits, operands."""
import ctypes

import numpy as np

from fp8_fine_grained_token_amd import ffn as L

from .gpu_util import U32, torch

ACTS = ("silu", "gelu_tanh")


def quantized(x, pow2=False):
    """(E4M3 bytes, scales) of fp32 numpy x [rows][cols] in groups of 128 along
    cols, by the rule of fp8_quant_act_1x128 (or its _pow2 form): the scale is
    amax / 448 in fp32 (the smallest power of two that is no smaller, 2^-126 at
    least), the code the E4M3 value nearest to the fp32 quotient x / scale."""
    t = torch()
    rows, cols = x.shape
    G = (cols + 127) // 128
    g = np.zeros((rows, G * 128), np.float32)
    g[:, :cols] = x
    g = g.reshape(rows, G, 128)
    with np.errstate(all="ignore"):
        amax = np.abs(g).max(axis=2)  # NaN if there is one
        bad = ~np.isfinite(amax)
        if pow2:
            m, e = np.frexp(amax.astype(np.float64))  # amax = m 2^e, 448 = 0.875 2^9
            e = np.where(m > 0.875, e - 8, e - 9)
            s = np.ldexp(1.0, np.where(amax > 0, np.maximum(e, -126), -126)).astype(np.float32)
        else:
            s = amax / np.float32(448)
        # a scale that rounds to 0 has nothing to divide by: codes +0, as for
        # a group of zeros
        v = np.where(((amax > 0) & (s > 0))[..., None], g / s[..., None], np.float32(0))
    v = np.clip(v, -448, 448)
    q = t.from_numpy(np.ascontiguousarray(v)).to(t.float8_e4m3fn).view(t.uint8).numpy()
    q = np.where(bad[..., None], np.uint8(0x7F), q)
    s = np.where(bad, amax, s)
    return q.reshape(rows, G * 128)[:, :cols], s


def same_quantized(got_q, got_s, x, pow2=False, what=""):
    """Bytes and scales are bit for bit what the rule gives for fp32 x."""
    q, s = quantized(x, pow2)
    gs, gq = got_s.cpu().numpy(), got_q.cpu().numpy()
    same = (gs.view(np.uint32) == s.view(np.uint32)) | (np.isnan(gs) & np.isnan(s))
    assert same.all(), (what, "scales", np.argwhere(~same)[:4], gs[~same][:4], s[~same][:4])
    assert (gq == q).all(), (what, "bytes", np.argwhere(gq != q)[:4], gq[gq != q][:4],
                             q[gq != q][:4])


def act64(g, kind):
    """(act(g), act'(g), z, sigmoid(z), |z'| g) in 64 bits."""
    g = g.astype(np.float64)
    if kind == "silu":
        z, dz = g, np.ones_like(g)
    else:
        c = 2 * np.sqrt(2 / np.pi)
        z, dz = c * (g + 0.044715 * g ** 3), c * (1 + 3 * 0.044715 * g ** 2)
    with np.errstate(over="ignore"):
        s, r = 1 / (1 + np.exp(-z)), 1 / (1 + np.exp(z))
    return g * s, s + g * dz * s * r, z, s, np.abs(g * dz)


def sigmoid_error(z, s, kind):
    """Bound on the relative error of the kernels' sigmoid(z) = 1 / (1 + e), e =
    2^h, h = z times -log2(e).  log2(e) is off by less than 2^-26 and the product
    rounds by 2^-24, so e is off by ln 2 |h| 1.25 2^-24 = 1.25 |z| 2^-24, and by
    another ulp (2^-23) of the exponential; in s that shows by the factor e / (1
    + e) = 1 - s.  1 + e rounds once (2^-24), the reciprocal is within 1 ulp
    (2^-23).  For GELU z itself carries five roundings (two constants, product,
    fused multiply-add, product), 5 |z| 2^-24 in the exponent.  5 of the 2.5 ulps
    that do not grow with z are allowed."""
    rel = 5 * 2.0 ** -23
    return rel + (1.5 if kind == "silu" else 7.5) * U32 * np.abs(z) * (1 - s)


def operands(seed, M, I, K, pow2=False, experts=0, sigma=1.0):
    """(a, a_scales, w, w_scales) on the GPU from random data."""
    import fp8_fine_grained_token_amd as F
    t = torch()
    g = t.Generator(device="cuda").manual_seed(seed)
    x = t.randn((M, K), generator=g, device="cuda")
    x *= t.where(t.rand(K, generator=g, device="cuda") < 0.01, 30.0, 1.0)
    w = t.randn((max(1, experts) * 2 * I, K), generator=g, device="cuda") * (sigma * K ** -0.5)
    qa = F.fp8_quant_act_1x128_pow2 if pow2 else F.fp8_quant_act_1x128
    qw = F.fp8_quant_weight_128x128_pow2 if pow2 else F.fp8_quant_weight_128x128
    a, sa = qa(x.to(t.bfloat16))
    w, sw = qw(w.to(t.bfloat16))
    if experts:
        w, sw = w.view(experts, 2 * I, K), sw.view(experts, 2 * I // 128, K // 128)
    return a, sa, w, sw


def without_workspace(name, a, sa, w, sw, act, quant=False, out_dtype="f32", offsets=None,
                      outs=None):
    """The C entry without a workspace: out, or (q, scales, h, h_scales);
    `offsets` for a grouped one."""
    t = torch()
    M, K = a.shape
    I = w.shape[-2] // 2
    stream = ctypes.c_void_p(t.cuda.current_stream().cuda_stream)
    head = [a.data_ptr(), sa.data_ptr(), w.data_ptr(), sw.data_ptr()]
    if offsets is not None:
        head += [offsets.data_ptr(), w.shape[0]]
    head += [L._ACTIVATIONS[act], M, I, K]
    if quant:
        outs = outs or (t.empty((M, I), dtype=t.uint8, device="cuda"),
                        t.empty((M, I // 128), device="cuda"),
                        t.empty((M, 2 * I), dtype=t.uint8, device="cuda"),
                        t.empty((M, I // 64), device="cuda"))
        L._call(name, *head, *(o.data_ptr() for o in outs), None, 0, stream)
        return outs
    out = outs if outs is not None else t.empty(
        (M, I), dtype=t.float32 if out_dtype == "f32" else t.bfloat16, device="cuda")
    L._call(name, *head, out.data_ptr(), 0 if out.dtype == t.float32 else 1, None, 0, stream)
    return out
