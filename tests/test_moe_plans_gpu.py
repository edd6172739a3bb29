"""Every form that the launch rules of the operators around the expert products
can choose, on the GPU against 64-bit formulas: the forms for many rows, wide
rows and many column tiles, which small cases do not reach.

Bounds are those of the operators' other tests: n FP32 operations on a sum are
off by at most n 2^-24 of the sum of the magnitudes, and a result is rounded
once to its type.
"""
import numpy as np
import pytest

import oracle
from fp8_fine_grained_token_amd import binding as B
from fp8_fine_grained_token_amd import moe as M

from .gpu_util import U32, U_BF16, host, torch

pytestmark = pytest.mark.gpu


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


def draw(seed, shape, dtype="bf16", sigma=1.0, mean=0.0):
    t = torch()
    g = t.Generator(device="cuda").manual_seed(seed)
    return (t.randn(shape, generator=g, device="cuda") * sigma + mean).to(dt(dtype))


def cuda(a):
    return torch().from_numpy(np.ascontiguousarray(a)).cuda()


def close(got, want, magnitudes, terms, what=""):
    """got within `terms` FP32 roundings of the magnitudes and the one rounding
    to its type (64-bit tensors on the device)."""
    u = U_BF16 if got.dtype == torch().bfloat16 else U32
    bound = terms * U32 * magnitudes
    bound = bound + u * (want.abs() + bound) + 2.0 ** -126
    bad = ~((got.double() - want).abs() <= bound)
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:4].tolist(), got[bad][:4].tolist(),
                           want[bad][:4].tolist())


# ---- 4-bit products ----------------------------------------------------------------

def weights(seed, lead, K, kind):
    """Random codes, scales within a factor of 16 and the weights they stand
    for in 64 bits, one expert at a time."""
    t = torch()
    g = t.Generator(device="cuda").manual_seed(seed)
    codes = t.randint(0, 256, (*lead, (K + 1) // 2), generator=g, device="cuda", dtype=t.uint8)
    if kind == "f32":
        scales = t.rand((*lead, (K + 127) // 128), generator=g, device="cuda") + 0.1
    else:
        scales = t.randint(123, 128, (*lead, (K + 31) // 32), generator=g, device="cuda",
                           dtype=t.uint8)
    return codes, scales


def wide(codes, scales, K):
    t = torch()
    table = t.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6],
                     dtype=t.float64, device="cuda")
    w = table[t.stack((codes & 15, codes >> 4), dim=-1).reshape(codes.shape[0], -1).int()][:, :K]
    k = t.arange(K, device="cuda")
    if scales.dtype == t.uint8:
        return w * t.exp2(scales[:, k // 32].double() - 127)
    return w * scales[:, k // 128].double()


def check_product(y, x, w):
    x, K = x.double(), x.shape[1]
    close(y, x @ w.t(), x.abs() @ w.abs().t(), K)
    # far inside that bound a typical sum is off by some sqrt(K) roundings of
    # its own size: a lost or doubled block would show
    if y.dtype == torch().float32:
        want = x @ w.t()
        assert float((y.double() - want).norm() / want.norm()) < 2 * K ** 0.5 * U32


# stretches of K side by side: one (2, 6, 7 and 8 blocks a wave), two and four
# (one and two blocks); several column tiles a wave, the last one in part, with
# K in one, four and eight parts and one to three passes of rows; K past what
# the waves hold (65, 129 and 144 blocks), one and several tiles a wave
PRODUCTS = [(12, 70, 2048), (16, 37, 6144), (16, 70, 7168), (9, 33, 8192), (8, 41, 2101),
            (8, 300, 7168), (1, 300, 4096), (4, 300, 7168), (3, 33, 8192), (2, 41, 2112),
            (1, 4, 1100), (1, 40003, 1000), (5, 33000, 1024), (20, 9001, 4096), (7, 5001, 7168),
            (33, 4500, 6100), (1, 4099, 8192), (2, 4500, 8320), (17, 4200, 16500),
            (1, 4200, 18432), (5, 30, 18400)]


@pytest.mark.parametrize("kind", ["f32", "e8m0"])
@pytest.mark.parametrize("rows,N,K", PRODUCTS)
def test_products(rows, N, K, kind):
    codes, scales = weights(N + K, (N,), K, kind)
    x = draw(K, (rows, K + 1))[:, 1:]
    w = wide(codes, scales, K)
    check_product(M.fp8_w4_matvec(x, codes, scales, out_dtype="f32"), x, w)
    check_product(M.fp8_w4_matvec(x, codes, scales), x, w)


# 24 experts, six of them with rows (one row to three passes): several column
# tiles a wave, N not in whole tiles, K of seven, six and eight blocks a wave
# and in chunks
@pytest.mark.parametrize("kind", ["f32", "e8m0"])
@pytest.mark.parametrize("N,K", [(4100, 7168), (4096, 6144), (4090, 1000), (2050, 8320)])
def test_expert_products(N, K, kind):
    t = torch()
    E, counts = 24, {0: 1, 5: 37, 6: 16, 11: 17, 20: 5, 23: 3}
    n = np.array([counts.get(e, 0) for e in range(E)])
    off = np.concatenate(([0], np.cumsum(n))).astype(np.int32)
    codes, scales = weights(N + K, (E, N), K, kind)
    x = draw(K, (int(off[-1]) + 1, K))
    y = t.full((x.shape[0], N), 9.0, device="cuda")
    M.fp8_w4_grouped_matvec(x, codes, scales, cuda(off), out_dtype="f32", y=y)
    for e in counts:
        a, b = off[e], off[e + 1]
        check_product(y[a:b], x[a:b], wide(codes[e], scales[e], K))
    assert bool((y[-1] == 9).all())


# ---- tokens by expert ----------------------------------------------------------------

def plan(seed, T, k, E, drop):
    """A sorted plan with dropped slots: the sort of the library, which has
    tests of its own."""
    t = torch()
    g = t.Generator(device="cuda").manual_seed(seed)
    ids = t.randint(0, E, (T, k), generator=g, device="cuda")
    ids[t.rand((T, k), generator=g, device="cuda") < drop] = -1
    return M.fp8_moe_sort(ids, E)[1]


def scattered(rows, slot_row, to):
    """rows [T][...] put where slot_row says, into a copy of `to`."""
    want = to.clone()
    for j in range(slot_row.shape[1]):
        kept = slot_row[:, j] >= 0
        want[slot_row[kept, j].long()] = rows[kept]
    return want


# at least 2^19 vectors of 16 bytes: four a thread; odd ends, rows in several
# workgroups' stretches, scales with wide and with narrow planes
@pytest.mark.parametrize("dtype,T,k,H,G", [
    ("uint8", 8400, 2, 1001, 8), ("uint8", 2400, 3, 7168, 56), ("bfloat16", 4200, 3, 1001, 0),
    ("bfloat16", 8300, 2, 520, 2), ("float32", 2110, 4, 1001, 0), ("bfloat16", 220, 2, 20003, 0),
    ("uint8", 270, 9, 33000, 258)])
def test_gather_of_many_vectors(dtype, T, k, H, G):
    t = torch()
    slot_row = plan(H, T, k, 16, 0.25)
    g = t.Generator(device="cuda").manual_seed(T)
    size = getattr(t, dtype).itemsize
    bits = t.randint(0, 256, (T, (H + 2) * size), generator=g, device="cuda", dtype=t.uint8)
    x = bits.view(getattr(t, dtype))[:, 1:1 + H]
    kept = t.full((T * k, H * size), 0xA5, device="cuda", dtype=t.uint8)
    want = scattered(x.contiguous().view(t.uint8), slot_row, kept)
    xs = kept.clone().view(x.dtype)
    if G:
        s = draw(5, (T, G + 3), "f32")[:, 1:1 + G]
        ss = t.full((T * k, G), -1.0, device="cuda")
        want_s = scattered(s, slot_row, ss)
        M.fp8_moe_dispatch(x, slot_row, scales=s, xs=xs, xs_scales=ss)
        assert t.equal(ss, want_s)
    else:
        M.fp8_moe_dispatch(x, slot_row, xs=xs)
    assert t.equal(xs.view(t.uint8), want)


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("T,k,H", [(4200, 3, 1001), (8300, 2, 520), (600, 2, 7168),
                                   (210, 2, 20003)])
def test_quantized_gather_of_many_vectors(T, k, H, pow2):
    t = torch()
    slot_row = plan(H, T, k, 16, 0.25)
    x = draw(H, (T, H + 3))[:, 1:1 + H]
    x[5] = 0
    x[T // 2, :H // 2] *= 1e-38
    bits = host(x.contiguous().view(t.int16)).view(np.uint16)
    q, s = (oracle.quant_act_1x128_pow2 if pow2 else oracle.quant_act_1x128)(bits)
    q0 = t.full((T * k, H), 0x5A, device="cuda", dtype=t.uint8)
    s0 = t.full((T * k, (H + 127) // 128), -3.0, device="cuda")
    want_q, want_s = scattered(cuda(q), slot_row, q0), scattered(cuda(s), slot_row, s0)
    gather = M.fp8_moe_dispatch_quant_1x128_pow2 if pow2 else M.fp8_moe_dispatch_quant_1x128
    gather(x, slot_row, q=q0, scales=s0)
    assert t.equal(q0, want_q) and t.equal(s0.view(t.int32), want_s.view(t.int32))


# at least 2^19 vectors of eight values with one to four slots (several vectors
# a thread), with less than 96 MiB of rows and, the last three, with more
@pytest.mark.parametrize("dtype,out_dtype", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"),
                                             ("f32", "bf16")])
@pytest.mark.parametrize("T,k,H", [(4300, 1, 1001), (8300, 2, 520), (4300, 3, 1001),
                                   (4300, 4, 1001), (13200, 2, 2000), (6700, 4, 2001),
                                   (26300, 1, 2003)])
def test_weighted_sum_of_many_vectors(T, k, H, dtype, out_dtype):
    t = torch()
    slot_row = plan(T, T, k, 16, 0.2)
    ys, w = draw(1, (T * k, H), dtype), draw(2, (T, k), "f32")
    res, dout = draw(3, (T, H), out_dtype), draw(4, (T, H), dtype)
    out = M.fp8_moe_combine(ys, slot_row, w, residual=res, out_dtype=out_dtype)
    want, mags = res.double(), res.double().abs()
    for j in range(k):
        kept = (slot_row[:, j] >= 0)[:, None]
        term = ys[slot_row[:, j].clamp(min=0).long()].double() * w[:, j, None].double() * kept
        want += term
        mags += term.abs_()
    close(out, want, mags, k + 1)
    if out_dtype != dtype:
        return
    dys, dw = M.fp8_moe_combine_grad(dout, ys, slot_row, w, dys=t.zeros_like(ys))
    for j in range(k):
        kept = slot_row[:, j] >= 0
        rows = slot_row[kept, j].long()
        products = ys[rows].double() * dout[kept].double()
        close(dw[kept, j], products.sum(1), products.abs().sum(1), 8 * -(-H // 512) + 30)
        assert not dw[~kept, j].any()
        term = w[kept, j, None].double() * dout[kept].double()
        close(dys[rows], term, term.abs(), 1)


# ---- norms: workgroups of several rows -----------------------------------------------

class Norms:
    """Operands and the formulas in 64 bits on the device, with the magnitudes
    of their terms."""

    def __init__(self, T, H, y_type, r_type, gates, post=True, seed=0):
        self.T, self.H, self.post, self.alpha, self.beta, self.eps = T, H, post, 0.9, 0.7, 1e-5
        self.y, self.r = draw(seed + 1, (T, H + 5), y_type, 3.0)[:, 2:2 + H], draw(seed + 2, (T, H),
                                                                                 r_type)
        self.dn, self.dr_out = draw(seed + 3, (T, H), y_type), draw(seed + 4, (T, H), r_type)
        self.w_post = draw(seed + 5, (H,), "f32", 0.2, 1.0) if post else None
        self.w_pre = draw(seed + 6, (H,), "f32", 0.2, 1.0)
        self.gate = draw(seed + 7, (gates, H), "f32", 0.5, 0.3) if gates else None
        self.kw = dict(post_norm=post, residual_scale=self.alpha, branch_scale=self.beta)
        t = torch()
        self.w1 = self.w_post.double() if post else t.ones(H, dtype=t.float64, device="cuda")
        self.w2 = self.w_pre.double()
        self.g = (self.gate.double().repeat_interleave(T // gates, dim=0) if gates
                  else t.ones((1, H), dtype=t.float64, device="cuda"))

    def args(self):
        return self.y, self.r, self.w_post, self.gate, self.w_pre

    def check_forward(self, r_out, n, rstd_post, rstd_pre):
        y, r = self.y.double(), self.r.double()
        rs1 = (y.square().mean(1) + self.eps).rsqrt()
        u = y * rs1[:, None] * self.w1 if self.post else y
        out = self.alpha * r + self.beta * self.g * u
        mag = (self.alpha * r).abs() + (self.beta * self.g * u).abs()
        ms = out.square().mean(1) + self.eps
        rs2 = ms.rsqrt()
        # 64 roundings: a row's sum is off by at most 60 and its root by 34, the
        # rest are a few operations; n carries the stream's error too
        close(r_out, out, mag, 64, "r_out")
        close(rstd_pre, rs2, rs2 * (1 + mag.square().mean(1) / ms), 64, "rstd_pre")
        if self.post:
            close(rstd_post, rs1, rs1, 64, "rstd_post")
        if n is not None:
            want = out * rs2[:, None] * self.w2
            close(n, want, self.w2.abs() * rs2[:, None] * mag
                  + want.abs() * (1 + (mag * rs2[:, None]).mean(1, keepdim=True)), 64, "n")

    def check_gradient(self, r_out, rs1, rs2, got):
        H = self.H
        y, s2 = self.y.double(), rs2.double()[:, None]
        rh, dn, e = r_out.double() * s2, self.dn.double(), self.dr_out.double()
        A = dn * self.w2
        D = e + s2 * (A - rh * (A * rh).mean(1, keepdim=True))
        Dm = e.abs() + s2 * (A.abs() + rh.abs() * (A * rh).abs().mean(1, keepdim=True))
        yh = y * rs1.double()[:, None] if self.post else y
        bg = self.beta * self.g
        dy, dym = bg * D, bg.abs() * Dm
        gates = 1 if self.gate is None else self.gate.shape[0]
        dg = (self.beta * D * yh * self.w1).reshape(gates, -1, H).sum(1)
        dgm = ((self.beta * yh * self.w1).abs() * Dm).reshape(gates, -1, H).sum(1)
        dw, dwm = (dy * yh).sum(0), (dym * yh.abs()).sum(0)
        if self.post:
            s1, Bv, Bm = rs1.double()[:, None], dy * self.w1, dym * self.w1.abs()
            dy = s1 * (Bv - yh * (Bv * yh).mean(1, keepdim=True))
            dym = s1 * (Bm + yh.abs() * (Bm * yh.abs()).mean(1, keepdim=True))
        # a parameter's gradient adds T terms: runs of rows one after the other,
        # then a tree of sums
        many = 128 + self.T // 64
        close(got[0], dy, dym, 64, "dy")
        close(got[1], self.alpha * D, self.alpha * Dm, 64, "dr")
        if self.post:
            close(got[2], dw, dwm, many, "dw_post")
        if self.gate is not None:
            close(got[3], dg, dgm, many, "dgate")
        close(got[4], (dn * rh).sum(0), (dn * rh).abs().sum(0), many, "dw_pre")


# two rows and more a workgroup of four to 16 waves, one and two vectors a
# thread, rows that are read again; gates that change inside a workgroup's rows
@pytest.mark.parametrize("T,H,y_type,r_type,gates,post", [
    (2300, 1500, "bf16", "bf16", 1, True), (1100, 4001, "bf16", "bf16", 1, True),
    (1100, 4001, "f32", "f32", 550, True), (1100, 7168, "bf16", "f32", 1, True),
    (1101, 7168, "bf16", "bf16", 3, True), (1100, 7168, "bf16", "bf16", 0, False),
    (1100, 9000, "bf16", "f32", 220, True), (700, 16384, "f32", "f32", 1, False),
    (2100, 16392, "bf16", "bf16", 2, True)])
def test_norms_of_many_rows(T, H, y_type, r_type, gates, post):
    t = torch()
    c = Norms(T, H, y_type, r_type, gates, post)
    first = M.fp8_norm_residual(*c.args(), eps=c.eps, **c.kw)
    c.check_forward(*first)
    # in place, and quantized in place
    r = c.r.clone()
    got = M.fp8_norm_residual(c.y, r, *c.args()[2:], eps=c.eps, r_out=r, **c.kw)
    for a, b in zip(got, first):
        assert (a is None and b is None) or t.equal(a, b)
    # the fp32 values that are quantized come from the fp32 form of y
    n = t.empty((T, H), device="cuda")
    y32, r32 = c.y.float(), c.r.float()
    for fn, pow2 in ((M.fp8_norm_residual_quant_1x128, False),
                     (M.fp8_norm_residual_quant_1x128_pow2, True)):
        out32, q32, s32, _, _ = fn(y32, r32, *c.args()[2:], eps=c.eps, n=n, **c.kw)
        r.copy_(c.r)
        out, q, s, _, _ = fn(c.y, r, *c.args()[2:], eps=c.eps, r_out=r, **c.kw)
        assert t.equal(out, first[0]) and t.equal(out32.to(out.dtype), out)
        assert t.equal(q, q32) and t.equal(s, s32)
        check_codes(n, q, s, pow2)


def check_codes(n, q, s, pow2):
    """Scales and E4M3 codes of fp32 n, by torch on the host."""
    t = torch()
    n, q, s = n.cpu(), q.cpu(), s.cpu()
    T, H = n.shape
    G = s.shape[1]
    grouped = t.nn.functional.pad(n, (0, 128 * G - H)).reshape(T, G, 128)
    amax = grouped.abs().amax(2)
    want = amax / t.tensor(448.0)
    if pow2:
        # the smallest power of two that is at least amax / 448, from 2^-126 on
        want = t.exp2(t.ceil(t.log2(amax.double().clamp(min=2.0 ** -200) / 448))).clamp(
            min=2.0 ** -126).float()
    assert t.equal(s, want)
    codes = (grouped / want[:, :, None]).reshape(T, -1)[:, :H].to(t.float8_e4m3fn).view(t.uint8)
    assert t.equal(q, codes)


# two rows and more a workgroup in every build; members that share a gate row,
# and members of several whole ones; rows whose means are found first (H > 8192)
@pytest.mark.parametrize("T,H,y_type,r_type,gates,post", [
    (1100, 1500, "bf16", "bf16", 1, True), (1030, 2500, "bf16", "bf16", 1, True),
    (1030, 2500, "f32", "f32", 515, True), (600, 4001, "bf16", "f32", 3, True),
    (1024, 4001, "bf16", "bf16", 512, True), (600, 7168, "bf16", "bf16", 1, True),
    (1101, 7168, "bf16", "f32", 3, True), (1024, 7168, "f32", "f32", 512, True),
    (700, 7168, "bf16", "bf16", 0, False), (600, 9000, "bf16", "bf16", 1, True),
    (1024, 9000, "bf16", "f32", 512, True), (1101, 9001, "bf16", "bf16", 3, False),
    (2100, 8200, "f32", "f32", 7, True)])
def test_gradients_of_many_rows(T, H, y_type, r_type, gates, post):
    c = Norms(T, H, y_type, r_type, gates, post, seed=10)
    r_out, _, rs1, rs2 = M.fp8_norm_residual(*c.args(), eps=c.eps, **c.kw)
    got = M.fp8_norm_residual_grad(c.dn, c.dr_out, c.y, r_out, rs1, rs2, c.w_post, c.gate, c.w_pre,
                                   **c.kw)
    c.check_gradient(r_out, rs1, rs2, got)


@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("H", [5, 40, 1500, 4001, 9000])
def test_gradient_left_out_is_zero(H, post):
    t = torch()
    c = Norms(24, H, "bf16", "f32", 3, post, seed=20)
    r_out, _, rs1, rs2 = M.fp8_norm_residual(*c.args(), eps=c.eps, **c.kw)

    def grad(dn, dr_out, rs2):
        return M.fp8_norm_residual_grad(dn, dr_out, c.y, r_out, rs1, rs2, c.w_post, c.gate,
                                        c.w_pre, **c.kw)

    for got, want in ((grad(None, c.dr_out, None), grad(t.zeros_like(c.dn), c.dr_out, rs2)),
                      (grad(c.dn, None, rs2), grad(c.dn, t.zeros_like(c.dr_out), rs2))):
        for a, b in zip(got, want):
            assert (a is None and b is None) or t.equal(a, b)
