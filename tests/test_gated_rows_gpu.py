"""Rows that are not a call's, and rows that hold NaN, reach no other row of the
products of a gated feed-forward block, whichever plan runs; and more experts
than the offsets of one wave's pass or than the split plan takes."""
import numpy as np
import pytest

import fp8_fine_grained_token_amd as F
from fp8_fine_grained_token_amd import binding as B

from .ffn_util import operands, without_workspace
from .gpu_util import torch
from .test_gated_gemm_gpu import offsets_of, sentinels, suffix

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    t = torch()
    if not t.cuda.is_available():
        pytest.skip("no GPU")
    B.lib()
    yield
    t.cuda.synchronize()


def poisoned(a, sa, rows):
    """Copies whose `rows` hold NaN codes and NaN scales."""
    a, sa = a.clone(), sa.clone()
    a[rows], sa[rows] = 0x7F, float("nan")
    return a, sa


# registers, 32-row and 64-row parts, 32-row, 64-row and 256-row tiles
DENSE = [(3, 256, 1152), (30, 128, 2304), (300, 256, 2304), (20, 32768, 128), (1000, 2048, 128),
         (2305, 4096, 128)]


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("M,I,K", DENSE)
def test_a_row_of_nan(M, I, K, pow2):
    t = torch()
    a, sa, w, sw = operands(M, M, I, K, pow2)
    call = getattr(F, "fp8_block_gemm_gated_quant_1x128" + suffix(pow2))
    plain = getattr(F, "fp8_block_gemm_gated" + suffix(pow2))
    want, out = call(a, sa, w, sw, checkpoint=True), plain(a, sa, w, sw)
    bad = [M // 2]
    rest = [r for r in range(M) if r not in bad]
    ap, sap = poisoned(a, sa, bad)
    for x, y in zip(call(ap, sap, w, sw, checkpoint=True), want):
        assert t.equal(x[rest], y[rest])
    got = plain(ap, sap, w, sw)
    assert t.equal(got[rest], out[rest]) and t.isnan(got[bad]).all()


# 32-row and 64-row parts, 32-row, 64-row and 128-row tiles
@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("first,counts,spare,I,K", [
    (2, [9, 0, 5], 3, 128, 2304), (5, [50, 0, 90], 7, 128, 2304),
    (3, [20, 0, 33, 1] * 10, 9, 768, 128), (6, [30, 70, 0, 40] * 4, 21, 1152, 128),
    (1, [300, 0, 129, 257], 70, 1024, 128)])
def test_rows_of_no_expert(first, counts, spare, I, K, pow2):
    # rows before the first expert's and behind the last one's, of NaN
    t = torch()
    E, n = len(counts), sum(counts)
    T = first + n + spare
    a, sa, w, sw = operands(5, T, I, K, pow2, experts=E)
    off = offsets_of(counts) + first
    outside = list(range(first)) + list(range(first + n, T))
    inside = slice(first, first + n)
    ap, sap = poisoned(a, sa, outside)
    name = "fp8_block_grouped_gemm_gated"
    results = []
    for x, s in ((a, sa), (ap, sap)):
        out = t.full((T, I), 7.0, device="cuda").bfloat16()
        getattr(F, name + suffix(pow2))(x, s, w, sw, off, out=out)
        kept = sentinels(T, I)
        getattr(F, name + "_quant_1x128" + suffix(pow2))(x, s, w, sw, off, "silu", True, *kept)
        assert (out[outside] == 7).all() and all((k[outside] == 9).all() for k in kept)
        results.append((out, *kept))
    for x, y in zip(*results):
        assert t.equal(x, y)
    assert not t.isnan(results[1][0][inside]).any()
    # the input gradient, on x's rows as dy (N = K of the product, its K = I)
    w2, sw2 = w[:, :K].contiguous(), sw[:, :K // 128].contiguous()
    if 2 * I >= K and K == 128:
        dxs = []
        for x, s in ((a, sa), (ap, sap)):
            dx = t.full((T, K), 7.0, device="cuda")
            getattr(F, "fp8_block_grouped_gemm_dgrad" + suffix(pow2))(x, s, w2, sw2, off, "f32", dx)
            assert (dx[outside] == 7).all()
            dxs.append(dx)
        assert t.equal(*dxs) and not t.isnan(dxs[1][inside]).any()


@pytest.mark.parametrize("E", [65, 1024, 1025, 3001])
def test_many_experts(E):
    t = torch()
    I, K = 128, 256
    rng = np.random.default_rng(E)
    counts = np.zeros(E, int)
    counts[rng.choice(E, 40, replace=False)] = rng.integers(1, 5, 40)
    counts[-1] = 2
    T = int(counts.sum())
    a, sa, w, sw = operands(7, T, I, K, experts=E)
    off = offsets_of(counts)
    q, s, h, hs = F.fp8_block_grouped_gemm_gated_quant_1x128(a, sa, w, sw, off, checkpoint=True)
    out = F.fp8_block_grouped_gemm_gated(a, sa, w, sw, off, out_dtype="f32")
    dx = F.fp8_block_grouped_gemm_dgrad(a, sa, w, sw, off, "f32")
    ends = off.tolist()
    for e in np.nonzero(counts)[0]:
        i, j = ends[e], ends[e + 1]
        one = offsets_of([j - i])
        args = (a[i:j].contiguous(), sa[i:j].contiguous(), w[e:e + 1].contiguous(),
                sw[e:e + 1].contiguous(), one)
        # without a workspace both run on 32-row tiles with the same sums
        got = without_workspace("fp8_block_grouped_gemm_gated", a, sa, w, sw, "silu", offsets=off)
        assert t.equal(got[i:j], without_workspace("fp8_block_grouped_gemm_gated", *args[:4],
                                                   "silu", offsets=one))
        assert t.equal(dx[i:j], F.fp8_block_grouped_gemm_dgrad(*args, "f32"))
        assert (out[i:j] - got[i:j]).norm() <= 1e-6 * got[i:j].norm()
    assert t.isfinite(out).all() and t.isfinite(s).all() and t.isfinite(hs).all()
