"""4-bit weights on the GPU: the quantizer bit for bit, the products against
64-bit numpy.

A product of a row of x with a row of weights adds K FP32 terms; every order
of adding them is off by at most K 2^-24 of the sum of the magnitudes, and a
typical one by about sqrt(K) 2^-24 of the result's own size, which is checked
as a relative Frobenius error.  The output is rounded once to its type.
"""
import numpy as np
import pytest

from fp8_fine_grained_token_amd import binding as B
from fp8_fine_grained_token_amd import moe as M

from .gpu_util import U32, U_BF16, host, torch

pytestmark = pytest.mark.gpu

E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    t = torch()
    if not t.cuda.is_available():
        pytest.skip("no GPU")
    B.lib()
    yield
    t.cuda.synchronize()


def cuda(a):
    return torch().from_numpy(np.ascontiguousarray(a)).cuda()


def bf16(seed, shape, sigma=1.0):
    t = torch()
    return t.from_numpy(np.random.default_rng(seed).standard_normal(shape, dtype=np.float32)
                        * np.float32(sigma)).to(t.bfloat16).cuda()


def f64(t):
    return t.detach().double().cpu().numpy()


def unpack(codes, K):
    both = np.stack((codes & 15, codes >> 4), axis=-1).reshape(*codes.shape[:-1], -1)
    return both[..., :K]


def weights64(codes, scales, K):
    codes, scales = host(codes), host(scales)
    if scales.dtype == np.uint8:
        s = np.repeat(np.exp2(scales.astype(np.float64) - 127), 32, axis=-1)
    else:
        s = np.repeat(scales.astype(np.float64), 128, axis=-1)
    return E2M1[unpack(codes, K)] * s[..., :K]


def nearest_even(v):
    """E2M1 magnitude codes of float32 |v| by search over the eight values."""
    grid = E2M1[:8]
    d = np.abs(v.astype(np.float64)[..., None] - grid)
    best = d.min(-1, keepdims=True)
    tie = d == best
    even = np.where(tie & (np.arange(8) % 2 == 0), np.arange(8), 99).min(-1)
    first = tie.argmax(-1)
    return np.where(even < 99, np.where(tie.sum(-1) > 1, even, first), first)


@pytest.mark.parametrize("N,K", [(64, 256), (5, 1), (3, 129), (33, 1000), (7, 31), (2, 7168),
                                 (16, 33)])
@pytest.mark.parametrize("kind", ["f32", "e8m0"])
def test_quantizer(N, K, kind):
    t = torch()
    w = bf16(N + K, (N, K), 0.02)
    if K >= 129 and N > 2:
        w[0, :128] = 0
        w[1, :64] = -0.0
        w[-1, :32] = 2.0 ** -133 * 3          # bf16 subnormals
        w[-1, 32:64] = 3.0e38
        w[2, :16] = t.tensor([0.25, -0.75, 1.25, 1.75, 2.5, -3.5, 5.0, 6.0] * 2)  # ties
        w[2, 16:128] = 0
    codes, scales = (M.fp8_w4_quant_1x128 if kind == "f32" else M.fp8_w4_quant_1x32)(w)
    assert codes.shape == (N, (K + 1) // 2)
    x = w.float().cpu().numpy()
    group = 128 if kind == "f32" else 32
    c = host(codes)
    if K % 2:
        assert not (c[:, -1] >> 4).any()
    c = unpack(c, K)
    s = host(scales)
    for g in range(s.shape[1]):
        part = x[:, g * group:(g + 1) * group]
        amax = np.abs(part).max(1)
        if kind == "f32":
            want = amax / np.float32(6)
            with np.errstate(invalid="ignore", divide="ignore"):
                v = np.where(want[:, None] > 0, part / want[:, None], np.float32(0))
        else:
            E = np.ceil(np.log2(np.maximum(amax.astype(np.float64), 2.0 ** -200) / 6))
            E = np.maximum(E, -127)
            want = (E + 127).astype(np.uint8)
            v = part.astype(np.float64) / np.exp2(E)[:, None]
        assert np.array_equal(s[:, g], want)
        sign = np.where(amax[:, None] > 0, np.signbit(part) * 8, 0)
        assert np.array_equal(c[:, g * group:(g + 1) * group], nearest_even(np.abs(v)) + sign)


def check(y, x, w):
    u = U_BF16 if y.dtype == torch().bfloat16 else U32
    K = x.shape[1]
    want, mag = x @ w.T, np.abs(x) @ np.abs(w).T
    bound = K * U32 * mag
    bound = bound + u * (np.abs(want) + bound) + 2.0 ** -126
    g = f64(y)
    assert np.isfinite(g).all()
    bad = np.abs(g - want) > bound
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4], g[bad][:4], want[bad][:4])
    norm = np.linalg.norm(mag) / 8  # the result's typical size, without its cancellation
    if norm and y.dtype == torch().float32:
        assert np.linalg.norm(g - want) <= 4e-6 * norm


SIZES = [(1, 2048, 7168), (1, 1, 1), (1, 3, 2), (2, 16, 32), (3, 17, 33), (4, 37, 128), (5, 1037, 1000),
         (7, 64, 129), (8, 100, 4096), (9, 50, 511), (15, 33, 640), (16, 256, 2049), (17, 40, 320),
         (33, 130, 260), (100, 20, 96), (1, 16, 8200), (6, 8, 70000)]


@pytest.mark.parametrize("kind", ["f32", "e8m0"])
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("rows,N,K", SIZES)
def test_matvec(rows, N, K, kind, out):
    w = bf16(N, (N, K), 0.02)
    codes, scales = (M.fp8_w4_quant_1x128 if kind == "f32" else M.fp8_w4_quant_1x32)(w)
    x = bf16(K, (rows, K + 9))[:, 3:3 + K]  # rows with a stride, off alignment
    x[:, ::17] *= 50
    y = M.fp8_w4_matvec(x, codes, scales, out_dtype=out)
    check(y, f64(x), weights64(codes, scales, K))


def test_scale_of_each_group_reaches_its_channels():
    # scales 2^10 apart from group to group and row to row
    N, K, rows = 40, 1100, 6
    rng = np.random.default_rng(3)
    codes = cuda(rng.integers(0, 256, (N, K // 2), dtype=np.uint8))
    x = bf16(4, (rows, K))
    s = np.exp2(10.0 * ((np.arange(N)[:, None] + np.arange(9)) % 5) - 20).astype(np.float32) * 1.37
    check(M.fp8_w4_matvec(x, codes, cuda(s), out_dtype="f32"), f64(x),
          weights64(codes, cuda(s), K))
    e = (127 + 10 * ((np.arange(N)[:, None] + np.arange(35)) % 5) - 20).astype(np.uint8)
    check(M.fp8_w4_matvec(x, codes, cuda(e), out_dtype="f32"), f64(x),
          weights64(codes, cuda(e), K))


def test_every_code_and_channel():
    # one-hot rows read single weights: every code at every place of a byte
    N, K = 32, 512
    rng = np.random.default_rng(5)
    c = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
    codes, scales = cuda(c), cuda(np.full((N, K // 128), 1.0, np.float32))
    t = torch()
    for k0 in range(0, K, 16):
        x = t.zeros((16, K), dtype=t.bfloat16, device="cuda")
        x[t.arange(16), t.arange(k0, k0 + 16)] = 1
        y = f64(M.fp8_w4_matvec(x, codes, scales, out_dtype="f32"))
        assert np.array_equal(y, E2M1[unpack(c, K)][:, k0:k0 + 16].T)


def test_nonfinite_rows_stay_in_their_row():
    t = torch()
    codes, scales = M.fp8_w4_quant_1x128(bf16(1, (70, 300)))
    x = bf16(2, (5, 300))
    clean = M.fp8_w4_matvec(x, codes, scales)
    x[2, 7] = float("nan")
    x[4, 9] = float("inf")
    y = M.fp8_w4_matvec(x, codes, scales)
    for m in (0, 1, 3):
        assert t.equal(y[m], clean[m])
    assert y[2].isnan().all()


def test_empty_sizes():
    t = torch()
    codes, scales = M.fp8_w4_quant_1x128(bf16(1, (7, 0)))
    y = M.fp8_w4_matvec(bf16(2, (3, 0)), codes, scales)
    assert y.shape == (3, 7) and not y.any()
    codes, scales = M.fp8_w4_quant_1x32(bf16(1, (7, 64)))
    assert M.fp8_w4_matvec(bf16(2, (0, 64)), codes, scales).shape == (0, 7)
    off = t.zeros(3, dtype=t.int32, device="cuda")
    codes, scales = M.fp8_w4_quant_1x32(bf16(1, (2, 7, 64)))
    assert M.fp8_w4_grouped_matvec(bf16(2, (0, 64)), codes, scales, off).shape == (0, 7)


GROUPS = [([5, 0, 1, 18], 40, 256), ([0, 0, 3], 17, 1000), ([1] * 9, 33, 129), ([40], 20, 64),
          ([0, 16, 17, 0, 2], 100, 640), ([3, 2, 8, 4, 1, 0, 12], 64, 4096)]


@pytest.mark.parametrize("kind", ["f32", "e8m0"])
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("counts,N,K", GROUPS)
def test_grouped(counts, N, K, kind, out):
    t = torch()
    E, R = len(counts), sum(counts) + 2  # the last two rows are nobody's
    w = bf16(R, (E, N, K), 0.02)
    codes, scales = (M.fp8_w4_quant_1x128 if kind == "f32" else M.fp8_w4_quant_1x32)(w)
    x = bf16(K, (R, K + 1))[:, 1:]
    off = np.concatenate(([0], np.cumsum(counts))).astype(np.int32)
    y = t.full((R, N), 9.0, dtype=t.bfloat16 if out == "bf16" else t.float32, device="cuda")
    M.fp8_w4_grouped_matvec(x, codes, scales, cuda(off), out_dtype=out, y=y)
    w64, x64 = weights64(codes, scales, K), f64(x)
    for e in range(E):
        if counts[e]:
            check(y[off[e]:off[e + 1]], x64[off[e]:off[e + 1]], w64[e])
    assert bool((y[-2:] == 9).all())


def test_grouped_offsets_are_made_safe():
    # beyond the rows, negative and decreasing offsets: clamped, never
    # overlapping
    t = torch()
    E, N, K, R = 5, 24, 96, 10
    codes, scales = M.fp8_w4_quant_1x32(bf16(1, (E, N, K)))
    x = bf16(2, (R, K))
    off = np.array([-4, 3, 2, 50, 7, 90], np.int32)
    y = t.full((R, N), 9.0, device="cuda")
    M.fp8_w4_grouped_matvec(x, codes, scales, cuda(off), out_dtype="f32", y=y)
    w64, x64 = weights64(codes, scales, K), f64(x)
    check(y[:3], x64[:3], w64[0])    # [-4, 3) -> [0, 3)
    check(y[3:], x64[3:], w64[2])    # [2, 50) -> [3, 10); the rest is taken


def test_grouped_equals_dense_and_every_run():
    t = torch()
    codes, scales = M.fp8_w4_quant_1x128(bf16(1, (3, 130, 700)))
    x = bf16(2, (12, 700))
    off = cuda(np.array([0, 4, 4, 12], np.int32))
    y = M.fp8_w4_grouped_matvec(x, codes, scales, off, out_dtype="f32")
    for _ in range(2):
        assert t.equal(M.fp8_w4_grouped_matvec(x, codes, scales, off, out_dtype="f32"), y)
    s = t.cuda.Stream()
    s.wait_stream(t.cuda.current_stream())
    z = M.fp8_w4_grouped_matvec(x, codes, scales, off, out_dtype="f32", stream=s)
    t.cuda.current_stream().wait_stream(s)
    assert t.equal(z, y)


def test_codes_past_2_gib():
    # the last expert's codes begin past 2^31 bytes: 64-bit offsets
    t = torch()
    E, N, K = 9, 65536, 8192
    codes = t.zeros((E, N, K // 2), dtype=t.uint8, device="cuda")
    codes[-1, -1] = 0x22  # ones
    scales = t.full((E, N, K // 32), 127, dtype=t.uint8, device="cuda")
    off = t.zeros(E + 1, dtype=t.int32, device="cuda")
    off[-1] = 2
    x = t.ones((2, K), dtype=t.bfloat16, device="cuda")
    y = M.fp8_w4_grouped_matvec(x, codes, scales, off, out_dtype="f32")
    assert bool((y[:, -1] == K).all()) and not y[:, :-1].any()
