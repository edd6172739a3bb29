"""Infinities and NaN in the operators around the expert products, on the GPU:
they show where the formulas have them and nowhere else.

A call on clean operands stands beside each: what a non-finite value must not
reach has to be equal to it bit for bit.
"""
import numpy as np
import pytest

from fp8_fine_grained_token_amd import binding as B
from fp8_fine_grained_token_amd import moe as M

from .gpu_util import e4m3_lut, host, torch

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    t = torch()
    if not t.cuda.is_available():
        pytest.skip("no GPU")
    B.lib()
    yield
    t.cuda.synchronize()


def draw(seed, shape, dtype="bf16", sigma=1.0, mean=0.0):
    t = torch()
    v = np.random.default_rng(seed).standard_normal(shape, dtype=np.float32) * np.float32(sigma)
    return t.from_numpy(v + np.float32(mean)).to(
        t.bfloat16 if dtype == "bf16" else t.float32).cuda()


def cuda(a):
    return torch().from_numpy(np.ascontiguousarray(a)).cuda()


@pytest.mark.parametrize("bad", [INF, -INF])
@pytest.mark.parametrize("H", [300, 1001, 9003, 17001])
def test_infinite_parameter_is_counted_once(H, bad):
    # in the columns that a row's last vector shares with the one before it:
    # the new stream is infinite there, so its reciprocal root is 0 (not NaN)
    # and the finite columns of n are 0
    t = torch()
    T, at = 3, H - 6
    y, r = draw(1, (T, H), "f32", mean=4.0), draw(2, (T, H), "f32")
    for gate, w_post in ((True, False), (False, True)):
        p = draw(3, (H,), "f32", 0.1, 1.0)
        p[at] = bad
        r_out, n, _, rstd = M.fp8_norm_residual(y, r, p if w_post else None, p if gate else None)
        assert t.equal(rstd, t.zeros_like(rstd))
        assert r_out[:, at].isinf().all() and n[:, at].isnan().all()
        r_out[:, at] = n[:, at] = 0
        assert r_out.isfinite().all() and not n.any()


@pytest.mark.parametrize("bad", [INF, NAN])
@pytest.mark.parametrize("H", [5, 300, 2500, 9000])
def test_gradient_without_post_norm_is_blind_to_y(H, bad):
    # y enters only the gate's gradient, in its own column
    t = torch()
    T = 6
    y, dn = draw(1, (T, H)), draw(2, (T, H))
    r_out, dr_out = draw(3, (T, H), "f32"), draw(4, (T, H), "f32")
    gate, w = draw(5, (H,), "f32", 0.3, 1.0), draw(6, (H,), "f32", 0.1, 1.0)
    rstd = 1 / r_out.square().mean(1).sqrt()

    def grad(dn, dr_out):
        return M.fp8_norm_residual_grad(dn, dr_out, y, r_out, None, rstd, None, gate, w,
                                        post_norm=False, branch_scale=0.7)

    for which in ((dn, dr_out), (None, dr_out), (dn, None)):
        y[2, H // 2] = 1.0
        clean = grad(*which)
        y[2, H // 2] = bad
        got = grad(*which)
        for name, a, b in zip(("dy", "dr", "dw_post", "dgate", "dw_pre"), got, clean):
            if name == "dgate":
                assert not a[H // 2].isfinite()
                a[H // 2] = b[H // 2]
            assert (a is None and b is None) or t.equal(a, b), name


def check_quantized(x, q, s, q0, s0, bad_groups, rows):
    """Groups of `rows` ([slots] -> row) of x: NaN or infinite scale and NaN
    read back for the (token, group) pairs of bad_groups, every other group
    equal to the clean call's (q0, s0)."""
    q, s, q0, s0 = host(q).copy(), host(s).copy(), host(q0), host(s0)
    nan_code = (np.arange(256) & 0x7F) == 0x7F
    for tok, g, want in bad_groups:
        for r in rows[tok]:
            at = slice(128 * g, min(128 * g + 128, q.shape[1]))
            assert np.isnan(s[r, g]) if np.isnan(want) else s[r, g] == INF, (tok, g, s[r, g])
            codes = q[r, at]
            with np.errstate(invalid="ignore"):
                back = np.where(nan_code[codes], NAN, e4m3_lut()[codes]) * s[r, g]
            assert np.isnan(back).all(), (tok, g, codes)
            q[r, at], s[r, g] = q0[r, at], s0[r, g]
    assert np.array_equal(q, q0) and np.array_equal(s.view(np.uint32), s0.view(np.uint32))


# the last one takes several vectors a thread
@pytest.mark.parametrize("suffix", ["", "_pow2"])
@pytest.mark.parametrize("T,k,H", [(1, 2, 1001), (9, 3, 5), (40, 2, 640), (4200, 2, 1001)])
def test_gather_keeps_nonfinite_groups(T, k, H, suffix):
    t = torch()
    E, G = 4, (H + 127) // 128
    ids = cuda(np.random.default_rng(T).integers(0, E, (T, k)))
    _, slot_row, _ = M.fp8_moe_sort(ids, E)
    x = draw(H, (T, H))
    if T > 2:
        x[1] = 0  # an all-zero row beside them
    rows = host(slot_row)
    tok = min(2, T - 1)
    bad = [(tok, 0, NAN), (tok, G - 1, INF)] if G > 1 else [(tok, 0, NAN)]
    gather = getattr(M, "fp8_moe_dispatch_quant_1x128" + suffix)
    both = getattr(M, "fp8_moe_sort_dispatch_quant_1x128" + suffix)
    q0, s0 = gather(x, slot_row)
    for put in (NAN, -NAN):
        x[tok, 3] = put
        if G > 1:
            x[tok, H - 2] = -INF
        q, s = gather(x, slot_row)
        check_quantized(x, q, s, q0, s0, bad, rows)
        _, _, _, q, s = both(x, ids, E)
        check_quantized(x, q, s, q0, s0, bad, rows)
    x[tok, 3] = INF
    q, s = gather(x, slot_row)
    check_quantized(x, q, s, q0, s0, [(tok, 0, INF)] + bad[1:], rows)
    assert t.equal(both(x, ids, E)[4], s)


@pytest.mark.parametrize("suffix", ["", "_pow2"])
@pytest.mark.parametrize("H,back", [(5, 2), (300, 2), (1001, 2), (1027, 6), (7168, 2), (16387, 6)])
def test_norm_keeps_nonfinite_groups(H, back, suffix):
    # a weight of the second norm: one group of every row (with `back` 6 a group
    # whose last columns the next group's only vector reads too)
    T, at = 3, H - back
    y, r = draw(1, (T, H)), draw(2, (T, H), "f32")
    w = draw(3, (H,), "f32", 0.1, 1.0)
    quant = getattr(M, "fp8_norm_residual_quant_1x128" + suffix)
    r0, q0, s0, _, rs0 = quant(y, r, None, None, w)
    for put in (NAN, INF):
        bad = w.clone()
        bad[at] = put
        r1, q, s, _, rs = quant(y, r, None, None, bad)
        assert torch().equal(r1, r0) and torch().equal(rs, rs0)
        check_quantized(None, q, s, q0, s0, [(i, at // 128, put) for i in range(T)],
                        [[i] for i in range(T)])


# K in whole and in part blocks of 128, and more blocks than the waves' parts
# of a row come to: 300 (3 blocks), 1000, 1100 (9), 5120 (40), 8200 (65)
@pytest.mark.parametrize("rows", [1, 12])
@pytest.mark.parametrize("kind", ["f32", "e8m0"])
@pytest.mark.parametrize("K", [20, 100, 300, 1000, 1100, 2300, 5120, 8200])
def test_a_nonfinite_scale_stays_in_its_output(K, kind, rows):
    t = torch()
    N, group = 70, 128 if kind == "f32" else 32
    rng = np.random.default_rng(K)
    codes = cuda(rng.integers(0, 256, (N, (K + 1) // 2), dtype=np.uint8))
    G = (K + group - 1) // group
    if kind == "f32":
        scales, bads = cuda(rng.random((N, G), dtype=np.float32) + 0.5), (NAN, INF, -INF)
    else:
        scales, bads = cuda(rng.integers(120, 130, (N, G), dtype=np.uint8)), (255,)
    x = draw(K, (rows, K))
    clean = M.fp8_w4_matvec(x, codes, scales, out_dtype="f32")
    w3, c3 = t.stack([codes] * 3), t.stack([scales] * 3)
    off = t.tensor([0, 0, rows, rows], dtype=t.int32, device="cuda")
    for bad in bads:
        s = scales.clone()
        s[10] = s[33, 0] = bad
        y = M.fp8_w4_matvec(x, codes, s, out_dtype="f32")
        assert not y[:, [10, 33]].isfinite().any()
        y[:, [10, 33]] = clean[:, [10, 33]]
        assert t.equal(y, clean)
        # the experts on both sides
        s3 = c3.clone()
        s3[0] = s3[2] = bad
        assert t.equal(M.fp8_w4_grouped_matvec(x, w3, s3, off, out_dtype="f32"), clean)


@pytest.mark.parametrize("K,N", [(6, 2), (64, 40), (1000, 40), (8200, 24)])
def test_ends_of_the_e8m0_range(K, N):
    # one-hot rows of x read single weights; x keeps the product in range.
    # Low bytes: weights down to 2^-128, subnormal in bf16 and fp32.
    t = torch()
    rng = np.random.default_rng(K)
    value = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])
    at = rng.choice(K, min(K, 16), replace=False)
    for byte, far in ((0, 90), (1, 90), (2, 90), (250, -90), (251, -90), (252, -90), (253, -90),
                      (254, -90)):
        c = rng.integers(0, 16, (N, K + K % 2))
        if byte > 252:  # weights below 2^128: up to 3 2^126, 1.5 2^127
            c = np.where((c & 7) > (5 if byte == 253 else 3), c & 8, c)
        packed = (c[:, 0::2] | c[:, 1::2] << 4).astype(np.uint8)
        scales = np.full((N, (K + 31) // 32), byte, np.uint8)
        x = t.zeros((at.size, K), dtype=t.bfloat16, device="cuda")
        x[t.arange(at.size), t.from_numpy(at)] = 2.0 ** far
        y = M.fp8_w4_matvec(x, cuda(packed), cuda(scales), out_dtype="f32")
        want = value[c[:, at]].T * 2.0 ** (byte - 127 + far)
        assert np.array_equal(y.double().cpu().numpy(), want), byte
        if byte > 252:  # 6 * 2^126 and more is past every type
            packed[5 % N, 0] = 0x77
            assert not M.fp8_w4_matvec(x, cuda(packed), cuda(scales))[:, 5 % N].isfinite().any()


@pytest.mark.parametrize("bad", [NAN, INF, -INF])
@pytest.mark.parametrize("kind", ["f32", "e8m0"])
@pytest.mark.parametrize("K", [20, 300, 1000])
def test_weight_quantizer_marks_nonfinite_groups(K, kind, bad):
    # the group's scale is NaN or infinite (E8M0: the NaN byte), so that a
    # product with the row is NaN; the other groups are as ever
    t = torch()
    N, group = 40, 128 if kind == "f32" else 32
    quant = M.fp8_w4_quant_1x128 if kind == "f32" else M.fp8_w4_quant_1x32
    w = draw(K, (N, K), sigma=0.02)
    codes0, scales0 = quant(w)
    g = (K - 1) // group
    w[7, K - 2] = bad
    codes, scales = quant(w)
    if kind == "e8m0":
        assert int(scales[7, g]) == 255
    else:
        assert scales[7, g].isnan() if np.isnan(bad) else scales[7, g] == INF
    scales[7, g] = scales0[7, g]
    codes[7, group * g // 2:] = codes0[7, group * g // 2:]
    assert t.equal(codes, codes0) and t.equal(scales, scales0)
    x = draw(K + 1, (3, K))
    x[1] = 0
    clean = M.fp8_w4_matvec(x, codes0, scales0, out_dtype="f32")
    y = M.fp8_w4_matvec(x, *quant(w), out_dtype="f32")
    assert y[:, 7].isnan().all()
    y[:, 7] = clean[:, 7]
    assert t.equal(y, clean)


def test_weights_at_the_end_of_the_range():
    # bf16 reaches 1.99 * 2^127: with E8M0 scales 1.75 * 2^127 rounds to 2^128
    t = torch()
    w = draw(1, (40, 96))
    w[3, 40], w[5, 40], w[7, 70] = 1.5 * 2.0 ** 127, 1.73 * 2.0 ** 127, 1.75 * 2.0 ** 127
    codes, scales = M.fp8_w4_quant_1x32(w)
    assert scales[[3, 5, 7], [1, 1, 2]].tolist() == [252, 253, 253]
    x = t.zeros((2, 96), dtype=t.bfloat16, device="cuda")
    x[0, 40] = 2.0 ** -100
    y = M.fp8_w4_matvec(x, codes, scales, out_dtype="f32")
    assert y[0, 3] == y[0, 5] == 1.5 * 2.0 ** 27 and not y[:, 7].isfinite().any()
    y[:, 7] = 0
    assert y.isfinite().all()
