"""Norms round a block with gate and residual scale, on the GPU against the
formulas in 64-bit numpy.

Tolerances come from the arithmetic.  A row's sum of H squares is taken by
threads of at most 32 values in sequence and a tree over them (at most 11
levels and 16 waves): off by at most 60 roundings relatively, so a reciprocal
root by at most 34 2^-24.  Every other value is a few FP32 operations on such
terms; their magnitudes, summed without cancellation, times 64 2^-24 bound
them, and the result is rounded once to its type.
"""
import numpy as np
import pytest

import oracle
from fp8_fine_grained_token_amd import binding as B
from fp8_fine_grained_token_amd import moe as M

from .gpu_util import U32, U_BF16, e4m3_lut, host, torch

pytestmark = pytest.mark.gpu

TYPES = [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    t = torch()
    if not t.cuda.is_available():
        pytest.skip("no GPU")
    B.lib()
    yield
    t.cuda.synchronize()


def dt(name):
    return torch().bfloat16 if name == "bf16" else torch().float32


def draw(rng, shape, dtype, sigma=1.0, mean=0.0):
    a = rng.standard_normal(shape, dtype=np.float32) * np.float32(sigma) + np.float32(mean)
    return torch().from_numpy(a).to(dt(dtype)).cuda()


def f64(t):
    return t.detach().double().cpu().numpy()


def close(got, want, magnitudes, terms=64):
    u = U_BF16 if got.dtype == torch().bfloat16 else U32
    g = f64(got)
    bound = terms * U32 * magnitudes
    bound = bound + u * (np.abs(want) + bound) + 2.0 ** -126
    assert np.isfinite(g).all()
    bad = np.abs(g - want) > bound
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4], g[bad][:4], want[bad][:4])


class Case:
    """Operands of one call (inputs with a row stride) and the formulas."""

    def __init__(self, seed, T, H, ytype, rtype, gates, post, params="f32", weights=True,
                 alpha=0.9, beta=0.7, eps=1e-5):
        rng = np.random.default_rng(seed)
        self.T, self.H, self.post, self.alpha, self.beta, self.eps = T, H, post, alpha, beta, eps
        pad = lambda d, s=1.0: draw(rng, (T, H + 5), d, s)[:, 2:2 + H]  # noqa: E731
        self.y, self.r = pad(ytype, 3.0), pad(rtype)
        self.dn, self.dr_out = pad(ytype), pad(rtype)
        self.w_post = draw(rng, (H,), params, 0.2, 1.0) if weights and post else None
        self.w_pre = draw(rng, (H,), params, 0.2, 1.0) if weights else None
        self.gate = draw(rng, (gates, H), params, 0.5, 0.3) if gates else None
        self.kw = dict(post_norm=post, residual_scale=alpha, branch_scale=beta)
        self.w1 = f64(self.w_post) if self.w_post is not None else np.ones(H)
        self.w2 = f64(self.w_pre) if self.w_pre is not None else np.ones(H)
        self.g = (np.repeat(f64(self.gate), T // gates, axis=0) if gates else np.ones((T, H)))

    def args(self):
        return self.y, self.r, self.w_post, self.gate, self.w_pre

    def forward(self, y=None, r=None, w1=None, w2=None, g=None):
        y = f64(self.y) if y is None else y
        r = f64(self.r) if r is None else r
        w1 = self.w1 if w1 is None else w1
        w2 = self.w2 if w2 is None else w2
        g = self.g if g is None else g
        rs1 = 1 / np.sqrt((y * y).mean(1) + self.eps) if self.post else None
        u = y * rs1[:, None] * w1 if self.post else y
        out = self.alpha * r + self.beta * g * u
        mag = np.abs(self.alpha * r) + np.abs(self.beta * g * u)
        rs2 = 1 / np.sqrt((out * out).mean(1) + self.eps)
        return out, mag, out * rs2[:, None] * w2, rs1, rs2


SIZES = [(1, 7168), (1, 1), (5, 8), (3, 129), (33, 64), (20, 500), (7, 513), (4, 1001), (2, 8200),
         (2, 16385), (1, 32768), (6, 2048)]


@pytest.mark.parametrize("ytype,rtype", TYPES)
@pytest.mark.parametrize("T,H", SIZES)
def test_forward(T, H, ytype, rtype):
    c = Case(H + T, T, H, ytype, rtype, 1 if T % 2 else 0, H != 513)
    out, mag, n, rs1, rs2 = c.forward()
    r_out, got_n, rstd_post, rstd_pre = M.fp8_norm_residual(*c.args(), eps=c.eps, **c.kw)
    close(r_out, out, mag)
    # n carries r_out's error relative to its own terms
    close(got_n, n, np.abs(c.w2) * rs2[:, None] * mag + np.abs(n) * (
        1 + (mag / np.sqrt((out * out).mean(1) + c.eps)[:, None]).mean(1, keepdims=True)))
    close(rstd_pre, rs2, rs2 * (1 + (mag * mag).mean(1) / ((out * out).mean(1) + c.eps)))
    if c.post:
        close(rstd_post, rs1, rs1)
    else:
        assert rstd_post is None


@pytest.mark.parametrize("T,H,gates,params,post,weights", [
    (12, 640, 3, "bf16", True, True), (12, 640, 12, "f32", True, True),
    (12, 72, 4, "f32", False, True), (700, 40, 7, "bf16", True, False),
    (3000, 16, 2, "f32", True, True), (2200, 520, 1100, "f32", True, True)])
def test_forward_gates_and_parameters(T, H, gates, params, post, weights):
    c = Case(T + H, T, H, "bf16", "f32", gates, post, params, weights)
    out, mag, n, _, rs2 = c.forward()
    r_out, got_n, _, _ = M.fp8_norm_residual(*c.args(), eps=c.eps, **c.kw)
    close(r_out, out, mag)
    close(got_n, n, np.abs(c.w2) * rs2[:, None] * mag + 3 * np.abs(n) * (
        mag / np.sqrt((out * out).mean(1) + c.eps)[:, None]).mean(1, keepdims=True))


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("T,H", [(1, 7168), (300, 128), (40, 1001), (9, 40), (5, 2056)])
def test_quantized_from_the_unrounded_value(T, H, pow2):
    # with fp32 y, n is the fp32 value that is quantized: bytes and scales
    # follow from it exactly
    c = Case(T * H, T, H, "f32", "f32", 1, True)
    t = torch()
    n = t.empty((T, H), device="cuda")
    c.y[0, : min(H, 128)] = 0
    c.r[0, : min(H, 128)] = 0  # an all-zero group (or row)
    fn = M.fp8_norm_residual_quant_1x128_pow2 if pow2 else M.fp8_norm_residual_quant_1x128
    r_out, q, s, _, _ = fn(*c.args(), eps=c.eps, n=n, **c.kw)
    ref, ref_n, _, _ = M.fp8_norm_residual(*c.args(), eps=c.eps, **c.kw)
    assert t.equal(r_out, ref) and t.equal(n, ref_n)
    nn, q, s = host(n), host(q), host(s)
    lut = e4m3_lut()
    for g in range(s.shape[1]):
        part = nn[:, 128 * g:128 * g + 128]
        amax = np.abs(part).max(1)
        if pow2:
            want = np.exp2(np.ceil(np.log2(np.maximum(amax.astype(np.float64), 2.0 ** -200) / 448)))
            want = np.maximum(want, 2.0 ** -126).astype(np.float32)
        else:
            want = amax / np.float32(448)
        assert np.array_equal(s[:, g], want)
        with np.errstate(invalid="ignore", divide="ignore"):
            v = np.where(amax[:, None] > 0, part / want[:, None], np.float32(0)).astype(np.float32)
        code = oracle.e4m3_encode(v)
        assert np.array_equal(lut[q[:, 128 * g:128 * g + 128]], lut[code])


def test_in_place_stream_and_no_pre_norm():
    t = torch()
    c = Case(3, 50, 300, "bf16", "f32", 1, True)
    r_out, n, _, _ = M.fp8_norm_residual(*c.args(), eps=c.eps, **c.kw)
    r = c.r.contiguous()
    M.fp8_norm_residual(c.y, r, *c.args()[2:], eps=c.eps, r_out=r, **c.kw)
    assert t.equal(r, r_out)
    lib = B.lib()
    out = t.empty_like(r_out)
    w = [x.data_ptr() for x in (c.w_post, c.gate, c.w_pre)]
    st = M._fn("fp8_norm_residual")(
        c.y.data_ptr(), 1, c.y.stride(0), c.r.data_ptr(), 0, c.r.stride(0), *w, 0, 50, 300, 1, 1,
        c.alpha, c.beta, c.eps, out.data_ptr(), None, None, None,
        t.cuda.current_stream().cuda_stream)
    assert st == 0 and lib is not None and t.equal(out, r_out)


def test_cancelling_residual_keeps_its_digits():
    # the branch takes the stream back almost whole: the statistics are of the
    # sum itself, not of its parts' sums
    t = torch()
    rng = np.random.default_rng(1)
    y = draw(rng, (4, 512), "f32")
    r = -y * (1 + 2.0 ** -10)
    r_out, n, _, rs2 = M.fp8_norm_residual(y, r, post_norm=False, eps=1e-12)
    out = f64(y) + f64(r)
    want = 1 / np.sqrt((out * out).mean(1) + 1e-12)
    assert np.abs(f64(rs2) / want - 1).max() < 64 * U32


def gradients(c, r_out, rs1, rs2, use_dn=True, use_dr=True):
    """The formulas from the stored tensors, and the magnitudes of their terms."""
    y, H = f64(c.y), c.H
    rs2 = rs2[:, None]
    rh = f64(r_out) * rs2
    dn = f64(c.dn) * use_dn
    A = dn * c.w2
    dr_out = f64(c.dr_out) * use_dr
    D = dr_out + rs2 * (A - rh * (A * rh).mean(1, keepdims=True))
    Dm = np.abs(dr_out) + rs2 * (np.abs(A) + np.abs(rh) * np.abs(A * rh).mean(1, keepdims=True))
    yh = y * rs1[:, None] if c.post else y
    du, dum = c.beta * c.g * D, np.abs(c.beta * c.g) * Dm
    if c.post:
        Bv, Bm = du * c.w1, dum * np.abs(c.w1)
        dy = rs1[:, None] * (Bv - yh * (Bv * yh).mean(1, keepdims=True))
        dym = rs1[:, None] * (Bm + np.abs(yh) * (Bm * np.abs(yh)).mean(1, keepdims=True))
    else:
        dy, dym = du, dum
    gates = 1 if c.gate is None else c.gate.shape[0]
    dg = (c.beta * D * yh * c.w1).reshape(gates, -1, H).sum(1)
    dgm = (np.abs(c.beta * yh * c.w1) * Dm).reshape(gates, -1, H).sum(1)
    return {"dr": (c.alpha * D, np.abs(c.alpha) * Dm), "dy": (dy, dym),
            "dw_post": ((du * yh).sum(0), (dum * np.abs(yh)).sum(0)), "dgate": (dg, dgm),
            "dw_pre": ((dn * rh).sum(0), np.abs(dn * rh).sum(0))}


def check_gradients(c, use_dn=True, use_dr=True, rows_in_a_row=64):
    r_out, _, rs1, rs2 = M.fp8_norm_residual(*c.args(), eps=c.eps, **c.kw)
    got = M.fp8_norm_residual_grad(c.dn if use_dn else None, c.dr_out if use_dr else None, c.y,
                                   r_out, rs1, rs2, c.w_post, c.gate, c.w_pre, **c.kw)
    want = gradients(c, r_out, f64(rs1) if c.post else None, f64(rs2), use_dn, use_dr)
    for name, g in zip(("dy", "dr", "dw_post", "dgate", "dw_pre"), got):
        has = {"dw_post": c.w_post, "dgate": c.gate, "dw_pre": c.w_pre}.get(name, c.y)
        if has is None:
            assert g is None
            continue
        # a parameter's gradient adds T terms: runs of rows one after the
        # other, then a tree of sums
        terms = 64 if name in ("dy", "dr") else 64 + rows_in_a_row + c.T // 64
        close(g, want[name][0], want[name][1], terms)


@pytest.mark.parametrize("ytype,rtype", TYPES)
@pytest.mark.parametrize("T,H", SIZES + [(600, 136), (1300, 24), (530, 1032)])
def test_gradient_against_formula(T, H, ytype, rtype):
    check_gradients(Case(H * 2 + T, T, H, ytype, rtype, 0 if T % 3 == 0 else 1, H != 513))


@pytest.mark.parametrize("T,H,gates,params,post,weights", [
    (12, 640, 3, "bf16", True, True), (12, 640, 12, "f32", True, True),
    (12, 72, 4, "f32", False, True), (700, 40, 7, "bf16", True, False),
    (3000, 16, 2, "f32", True, True), (2200, 520, 1100, "f32", True, True),
    (1500, 1040, 2, "f32", True, True), (3000, 48, 1000, "f32", True, True),
    (1026, 264, 513, "f32", False, True), (4096, 24, 4096, "bf16", True, True)])
def test_gradient_gates_and_parameters(T, H, gates, params, post, weights):
    c = Case(T * 7 + H, T, H, "bf16", "f32", gates, post, params, weights)
    check_gradients(c)


@pytest.mark.parametrize("use_dn,use_dr", [(True, False), (False, True)])
@pytest.mark.parametrize("H", [96, 1500])
def test_gradient_with_one_incoming(use_dn, use_dr, H):
    check_gradients(Case(H, 70, H, "bf16", "bf16", 2, True), use_dn, use_dr)


def test_gradient_of_no_tokens_is_zero():
    t = torch()
    e = t.empty((0, 256), device="cuda")
    z = t.empty(0, device="cuda")
    w = t.ones(256, device="cuda")
    dy, dr, dw_post, dgate, dw_pre = M.fp8_norm_residual_grad(e, e, e, e, z, z, w, w.clone(), w)
    assert dy.shape == dr.shape == (0, 256)
    for g in (dw_post, dgate, dw_pre):
        assert g.shape == (256,) and not g.any()
    r_out, n, _, _ = M.fp8_norm_residual(e, e, w, w, w)
    assert r_out.shape == n.shape == (0, 256)


def test_gradient_against_differences():
    # central differences of the 64-bit formula along random directions; fp32
    # tensors, so that rounding of the stored values (2^-24) stays below the
    # differences' own error (step^2)
    c = Case(11, 24, 200, "f32", "f32", 3, True)
    rng = np.random.default_rng(12)
    r_out, _, rs1, rs2 = M.fp8_norm_residual(*c.args(), eps=c.eps, **c.kw)
    dy, dr, dw_post, dgate, dw_pre = M.fp8_norm_residual_grad(
        c.dn, c.dr_out, c.y, r_out, rs1, rs2, c.w_post, c.gate, c.w_pre, **c.kw)
    dn, dro = f64(c.dn), f64(c.dr_out)

    def loss(**k):
        out, _, n, _, _ = c.forward(**k)
        return (out * dro).sum() + (n * dn).sum()

    step = 1e-5
    gate = f64(c.gate)
    for name, grad, base in (("y", dy, f64(c.y)), ("r", dr, f64(c.r)), ("w1", dw_post, c.w1),
                             ("w2", dw_pre, c.w2), ("g", dgate, gate)):
        d = rng.standard_normal(base.shape)
        wide = (lambda v: np.repeat(v, 8, axis=0)) if name == "g" else (lambda v: v)  # noqa: E731
        num = (loss(**{name: wide(base + step * d)}) - loss(**{name: wide(base - step * d)})) / (
            2 * step)
        g = f64(grad)
        assert abs(num - (g * d).sum()) < 2e-6 * np.linalg.norm(g) * np.linalg.norm(d), name
