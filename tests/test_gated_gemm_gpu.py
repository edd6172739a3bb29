"""Gated products on the GPU.

A product without a workspace adds the same K blocks in the same order as
fp8_block_gemm without one, so its projections are fp8_block_gemm's bit for bit:
the checkpoint is compared with the 1x128 rule on those, the quantized result
with the rule on the fp32 result, and the fp32 result with the activation in 64
bits of those projections (tolerance from the arithmetic, see ffn_util).
Against the binary64 product of the operands the bound is the GEMM's own,
carried through the activation, whose slope is at most 1.13.
"""
import ctypes

import numpy as np
import pytest

import fp8_fine_grained_token_amd as F
import oracle
from fp8_fine_grained_token_amd import binding as B
from fp8_fine_grained_token_amd import ffn as L

from .ffn_util import (ACTS, act64, operands, same_quantized, sigmoid_error, without_workspace)
from .gpu_util import U32, U_BF16, e4m3_lut, gemm_error_bound, host, log, tile_rows, torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    t = torch()
    if not t.cuda.is_available():
        pytest.skip("no GPU")
    B.lib()
    yield
    t.cuda.synchronize()


def suffix(pow2):
    return "_pow2" if pow2 else ""


def plain_product(a, sa, w, sw, pow2):
    """[g | u] in fp32 from fp8_block_gemm without a workspace."""
    t = torch()
    (M, K), N = a.shape, w.shape[0]
    c = t.empty((M, N), device="cuda")
    name = "fp8_block_gemm" + suffix(pow2)
    st = getattr(B.lib(), name)(
        *(ctypes.c_void_p(x.data_ptr()) for x in (a, sa, w, sw, c)), 0, M, N, K, None, 0,
        ctypes.c_void_p(t.cuda.current_stream().cuda_stream))
    assert st == 0
    return c


def check_act(out, h, act):
    """fp32 out against act(g) u of fp32 h in 64 bits."""
    I = out.shape[1]
    g, u = h[:, :I].astype(np.float64), h[:, I:].astype(np.float64)
    a, _, z, s, _ = act64(g, act)
    want = a * u
    # g s and (g s) u round once each; a sigmoid below 2^-126 may be 0
    bound = np.abs(want) * (sigmoid_error(z, s, act) + 3 * U32)
    bound += (np.abs(g) + 1) * (np.abs(u) + 1) * 2.0 ** -125
    bad = np.abs(out - want) > bound
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4], out[bad][:4], want[bad][:4])


# rows, inner width, K: one value of each kind of edge; 4097 x 2048 and 2305 x
# 4096 fill the card with 256-row tiles, whose last has one row
SHAPES = [(1, 128, 128), (1, 256, 1152), (3, 384, 128), (16, 128, 7168), (17, 640, 256),
          (64, 256, 640), (127, 128, 1280), (128, 128, 128), (129, 384, 384), (300, 640, 896),
          (257, 1024, 256), (1000, 2048, 256), (1100, 4096, 128), (4097, 2048, 128),
          (2305, 4096, 384)]


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,I,K", SHAPES)
def test_parts_against_the_plain_product(M, I, K, act, pow2):
    a, sa, w, sw = operands(M + K, M, I, K, pow2)
    h = host(plain_product(a, sa, w, sw, pow2))
    name = "fp8_block_gemm_gated"
    out = without_workspace(name + suffix(pow2), a, sa, w, sw, act)
    check_act(host(out), h, act)
    bf16 = without_workspace(name + suffix(pow2), a, sa, w, sw, act, out_dtype="bf16")
    assert torch().equal(bf16, out.to(torch().bfloat16))
    q, s, hq, hs = without_workspace(name + "_quant_1x128" + suffix(pow2), a, sa, w, sw, act,
                                     quant=True)
    same_quantized(q, s, host(out), pow2, "a")
    same_quantized(hq, hs, h, pow2, "h")


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("M", [33, 64, 65, 128, 129])
def test_many_columns_against_the_plain_product(M, pow2):
    # 64-row, 128-row and 256-row tiles of one row of tiles
    I = 32768
    a, sa, w, sw = operands(M, M, I, 128, pow2)
    h = host(plain_product(a, sa, w, sw, pow2))
    name = "fp8_block_gemm_gated"
    out = without_workspace(name + suffix(pow2), a, sa, w, sw, "silu")
    check_act(host(out), h, "silu")
    q, s, hq, hs = without_workspace(name + "_quant_1x128" + suffix(pow2), a, sa, w, sw, "silu",
                                     quant=True)
    same_quantized(q, s, host(out), pow2, "a")
    same_quantized(hq, hs, h, pow2, "h")


def exact_product(a, sa, w, sw, rows):
    """[g | u] of some rows in binary64 and the bound on the kernels' fp32."""
    qa, s = a.cpu().numpy(), sa.cpu().numpy()
    qw, ws = w.cpu().numpy(), sw.cpu().numpy()
    lut = e4m3_lut()
    x = lut[qa[rows]] * np.repeat(s[rows].astype(np.float64), 128, axis=1)
    y = lut[qw] * np.repeat(np.repeat(ws.astype(np.float64), 128, 0), 128, 1)
    return x @ y.T, gemm_error_bound(qa, s, qw, ws, rows, splits=64)


def carried(h, b, act):
    """act(g) u of binary64 h and a bound on it for an h off by at most b."""
    I = h.shape[1] // 2
    g, u, bg, bu = h[:, :I], h[:, I:], b[:, :I], b[:, I:]
    a, _, z, s, _ = act64(g, act)
    want = a * u
    bound = 1.13 * bg * (np.abs(u) + bu) + np.abs(a) * bu
    return want, bound + (np.abs(want) + bound) * (sigmoid_error(z, s, act) + 3 * U32) + 2.0 ** -120


def check_kept(q, s, want, bound, pow2=False):
    """Quantized values against binary64 values that the kernel's are within
    `bound` of: its scale is its maximum over 448 (or up to twice that), and a
    code is off by half a step: 2^-4 of the value, or 2^-10 scales near 0."""
    v, sc = e4m3_lut()[q], np.repeat(s.astype(np.float64), 128, axis=1)[:, :q.shape[1]]
    off = bound + (np.abs(want) + bound) * 2.0 ** -4 * 1.001 + sc * 2.0 ** -10 * 1.001
    bad = np.abs(v * sc - want) > off
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4])
    rows, cols = want.shape
    top = np.abs(want).reshape(rows, cols // 128, 128).max(2)
    slack = bound.reshape(rows, cols // 128, 128).max(2)
    most = 2.0 if pow2 else 1.0
    assert (s * 448.0 <= most * (top + slack) * (1 + 4 * U32)).all()
    assert (s * 448.0 >= (top - slack) * (1 - 4 * U32)).all()


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("M,I,K,act", [
    (1, 256, 1152, "silu"), (2, 2048, 7168, "silu"), (16, 512, 7168, "gelu_tanh"),
    (17, 512, 2304, "silu"), (48, 256, 4096, "silu"), (64, 384, 640, "gelu_tanh"),
    (65, 512, 7168, "silu"), (100, 1024, 7168, "silu"), (256, 1024, 7168, "gelu_tanh"),
    (300, 640, 896, "silu"), (1025, 512, 512, "silu"), (4097, 2048, 256, "gelu_tanh")])
def test_against_binary64(M, I, K, act, pow2):
    # whichever plan the call takes, through the Python layer (which gives it
    # the workspace that it asks for)
    a, sa, w, sw = operands(7 * M + I, M, I, K, pow2)
    rows = tile_rows(M, 64, 1) if M > 300 else np.arange(M)
    h, b = exact_product(a, sa, w, sw, rows)
    want, bound = carried(h, b, act)
    log(f"  workspace {L.fp8_gated_gemm_workspace_bytes(M, I, K)}")
    name = "fp8_block_gemm_gated"
    out = host(getattr(F, name + suffix(pow2))(a, sa, w, sw, act, out_dtype="f32"))[rows]
    assert (np.abs(out - want) <= bound).all(), np.abs(out - want).max()
    bf16 = host(getattr(F, name + suffix(pow2))(a, sa, w, sw, act))[rows]
    assert (np.abs(bf16 - want) <= bound + U_BF16 * (np.abs(want) + bound)).all()
    call = getattr(F, name + "_quant_1x128" + suffix(pow2))
    q, s, hq, hs = (x.cpu().numpy()[rows] for x in call(a, sa, w, sw, act, checkpoint=True))
    check_kept(q, s, want, bound, pow2)
    check_kept(hq, hs, h, b, pow2)
    again = call(a, sa, w, sw, act)
    assert again[2] is None and again[3] is None
    assert (again[0].cpu().numpy()[rows] == q).all() and (again[1].cpu().numpy()[rows] == s).all()


@pytest.mark.parametrize("M", [1, 40, 200])
def test_given_outputs_and_workspaces(M):
    t = torch()
    I, K = 512, 2304
    a, sa, w, sw = operands(5, M, I, K)
    want = F.fp8_block_gemm_gated_quant_1x128(a, sa, w, sw, checkpoint=True)
    need = L.fp8_gated_gemm_workspace_bytes(M, I, K)
    # a workspace of garbage, exactly as large as asked for, between guards
    raw = t.full((need + 512,), 0xFF, dtype=t.uint8, device="cuda")
    outs = [t.full_like(x, 77) for x in want]
    got = F.fp8_block_gemm_gated_quant_1x128(
        a, sa, w, sw, "silu", True, *outs, workspace=raw[256:256 + need] if need else None)
    for x, y, z in zip(want, got, outs):
        assert t.equal(x, y) and y is z
    assert (raw[:256] == 0xFF).all() and (raw[256 + need:] == 0xFF).all()
    # one that is too small: the plan without, close to the other
    if need:
        small = t.empty(256, dtype=t.uint8, device="cuda")
        x = F.fp8_block_gemm_gated(a, sa, w, sw, out_dtype="f32", workspace=small)
        assert t.equal(x, without_workspace("fp8_block_gemm_gated", a, sa, w, sw, "silu"))


def test_no_rows_and_no_columns():
    t = torch()
    a, sa, w, sw = operands(1, 4, 128, 256)
    assert F.fp8_block_gemm_gated(a[:0], sa[:0], w, sw).shape == (0, 128)
    q, s, h, hs = F.fp8_block_gemm_gated_quant_1x128(a[:0], sa[:0], w, sw, checkpoint=True)
    assert q.shape == (0, 128) and s.shape == (0, 1) and h.shape == (0, 256)
    assert F.fp8_block_gemm_gated(a, sa, w[:0], sw[:0]).shape == (4, 0)
    off = t.zeros(2, dtype=t.int32, device="cuda")
    assert F.fp8_block_grouped_gemm_gated(a[:0], sa[:0], w[None], sw[None], off).shape == (0, 128)


@pytest.mark.parametrize("act", ACTS)
def test_zero_and_saturated_gates(act):
    # rows of zeros, gates far into both tails: exact zeros, u or g u
    t = torch()
    M, I, K = 40, 128, 256
    a, sa, w, sw = operands(2, M, I, K, sigma=400.0)
    a[3] = 0
    sa[5] = 0
    for M_ in (M, 1):
        out = F.fp8_block_gemm_gated(a[:M_], sa[:M_], w, sw, act, out_dtype="f32")
        q, s, h, hs = F.fp8_block_gemm_gated_quant_1x128(a[:M_], sa[:M_], w, sw, act,
                                                         checkpoint=True)
        assert t.isfinite(out).all() and t.isfinite(s).all() and t.isfinite(hs).all()
    out = host(F.fp8_block_gemm_gated(a, sa, w, sw, act, out_dtype="f32"))
    q, s, h, hs = F.fp8_block_gemm_gated_quant_1x128(a, sa, w, sw, act, checkpoint=True)
    for r in (3, 5):
        assert (out[r] == 0).all() and (q[r] & 0x7F == 0).all() and s[r, 0] == 0
        assert (h[r] & 0x7F == 0).all() and (hs[r] == 0).all()
    check_act(host(without_workspace("fp8_block_gemm_gated", a, sa, w, sw, act)),
              host(plain_product(a, sa, w, sw, False)), act)


def offsets_of(counts):
    return torch().tensor(np.concatenate(([0], np.cumsum(counts))).astype(np.int32)).cuda()


GROUPS = [([1], 0, 128, 128), ([5, 0, 1, 129, 0], 3, 256, 384), ([0, 0, 0], 4, 128, 128),
          ([128, 256, 64, 300], 0, 384, 640), ([2] * 70 + [0] * 3, 1, 128, 256),
          ([700, 3, 1], 11, 1024, 256), ([9, 0, 40], 2, 256, 2304),
          ([40, 0, 129, 1, 300], 5, 256, 384), ([64, 64], 0, 128, 1280),
          ([30, 70, 1, 40], 4, 1408, 256), ([3] * 40, 2, 2048, 256),
          ([20, 40, 0, 33, 7, 1, 31, 32], 9, 4096, 128)]


def sentinels(T, I):
    t = torch()
    return (t.full((T, I), 9, dtype=t.uint8, device="cuda"), t.full((T, I // 128), 9.0).cuda(),
            t.full((T, 2 * I), 9, dtype=t.uint8, device="cuda"), t.full((T, I // 64), 9.0).cuda())


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("counts,spare,I,K",
                         [c for c in GROUPS if sum(c[0]) + c[1] > 24 * len(c[0])])
def test_grouped_against_dense(counts, spare, I, K, pow2):
    # without a workspace (and with more than 24 rows to an expert on average)
    # each expert's rows are the dense product, bit for bit; rows behind the last
    # expert's stay as they were
    t = torch()
    E, T = len(counts), sum(counts) + spare
    a, sa, w, sw = operands(3, T, I, K, pow2, experts=E)
    off = offsets_of(counts)
    name = "fp8_block_grouped_gemm_gated"
    args = (a, sa, w, sw, "gelu_tanh")
    out = without_workspace(name + suffix(pow2), *args, offsets=off,
                            outs=t.full((T, I), 7.0, device="cuda"))
    bf = without_workspace(name + suffix(pow2), *args, offsets=off,
                           outs=t.full((T, I), 7.0, device="cuda").bfloat16())
    outs = without_workspace(name + "_quant_1x128" + suffix(pow2), *args, quant=True, offsets=off,
                             outs=sentinels(T, I))
    ends = off.tolist()
    for e, (i, j) in enumerate(zip(ends, ends[1:])):
        if i == j:
            continue
        args = (a[i:j].contiguous(), sa[i:j].contiguous(), w[e], sw[e], "gelu_tanh")
        want = without_workspace("fp8_block_gemm_gated" + suffix(pow2), *args)
        assert t.equal(out[i:j], want) and t.equal(bf[i:j], want.bfloat16())
        for x, y in zip(outs, without_workspace("fp8_block_gemm_gated_quant_1x128" + suffix(pow2),
                                                *args, quant=True)):
            assert t.equal(x[i:j], y)
    n = sum(counts)
    assert (out[n:] == 7).all() and (bf[n:] == 7).all() and all((x[n:] == 9).all() for x in outs)


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("counts,spare,I,K", GROUPS)
def test_grouped_against_binary64(counts, spare, I, K, pow2):
    # whichever plan the call takes
    t = torch()
    E, T = len(counts), sum(counts) + spare
    a, sa, w, sw = operands(6, T, I, K, pow2, experts=E)
    off = offsets_of(counts)
    log(f"  workspace {L.fp8_grouped_gated_gemm_workspace_bytes(T, E, I, K)}")
    bare = without_workspace("fp8_block_grouped_gemm_gated" + suffix(pow2), a, sa, w, sw, "silu",
                             offsets=off, outs=t.full((T, I), 7.0, device="cuda"))
    name = "fp8_block_grouped_gemm_gated"
    out = t.full((T, I), 7.0, device="cuda")
    assert getattr(F, name + suffix(pow2))(a, sa, w, sw, off, out_dtype="f32", out=out) is out
    bf = t.full((T, I), 7.0, device="cuda").bfloat16()
    getattr(F, name + suffix(pow2))(a, sa, w, sw, off, out=bf)
    assert t.equal(bf, out.bfloat16())
    kept = sentinels(T, I)
    getattr(F, name + "_quant_1x128" + suffix(pow2))(a, sa, w, sw, off, "silu", True, *kept)
    n = sum(counts)
    assert (out[n:] == 7).all() and all((x[n:] == 9).all() for x in kept)
    assert (bare[n:] == 7).all()
    same_quantized(kept[0][:n], kept[1][:n], host(out[:n]), pow2)
    q, s, h, hs = (x.cpu().numpy() for x in kept)
    out, bare = host(out), host(bare)
    ends = off.tolist()
    for e, (i, j) in enumerate(zip(ends, ends[1:])):
        if i < j:
            want_h, b = exact_product(a, sa, w[e], sw[e], np.arange(i, j))
            want, bound = carried(want_h, b, "silu")
            assert (np.abs(out[i:j] - want) <= bound).all()
            assert (np.abs(bare[i:j] - want) <= bound).all()
            check_kept(q[i:j], s[i:j], want, bound, pow2)
            check_kept(h[i:j], hs[i:j], want_h, b, pow2)


@pytest.mark.parametrize("T,I", [(300, 128), (300, 2048), (5, 256)])
def test_grouped_offsets_out_of_order(T, I):
    # any offsets are made ranges within the rows, each row at most one
    # expert's: those of the plain grouped product, whose sums are within the
    # GEMM's bound of this one's (with a workspace and without)
    t = torch()
    E, K = 4, 256
    a, sa, w, sw = operands(4, T, I, K, experts=E)
    for off in ([0, 400, 100, -5, 300], [50, 20, 200, 200, 1 << 30], [-7, 128, 64, 290, 10],
                [1 << 30, 5, 3, 2, 1], [2, 2, 2, 2, 4]):
        off = t.tensor(off, dtype=t.int32).cuda()
        h = t.full((T, 2 * I), float("nan"), device="cuda")
        F.fp8_block_grouped_gemm(a, sa, w, sw, off, out_dtype="f32", c=h)
        live = ~t.isnan(h[:, 0])
        out = without_workspace("fp8_block_grouped_gemm_gated", a, sa, w, sw, "silu", offsets=off,
                                outs=t.full((T, I), float("nan"), device="cuda"))
        assert t.equal(t.isnan(out).all(1), ~live) and not t.isnan(out[live]).any()
        if T > 24 * E:  # FP8 products, the plain call's bit for bit
            check_act(host(out[live]), host(h[live]), "silu")
        split = t.full((T, I), float("nan"), device="cuda")
        F.fp8_block_grouped_gemm_gated(a, sa, w, sw, off, out_dtype="f32", out=split)
        assert t.equal(t.isnan(split).all(1), ~live) and not t.isnan(split[live]).any()
        if live.any():
            want = host(h[live]).astype(np.float64)
            want = act64(want[:, :I], "silu")[0] * want[:, I:]
            for x in (out, split):  # a row of another expert's weights is off by 1
                assert np.linalg.norm(host(x[live]) - want) < 1e-3 * np.linalg.norm(want)


# ---- input gradient per expert ---------------------------------------------------

@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("out_dtype", ["f32", "bf16"])
@pytest.mark.parametrize("counts,spare,N,K", [
    ([1], 0, 128, 128), ([5, 0, 1, 129, 0], 3, 384, 256), ([0, 0], 2, 128, 384),
    ([128, 256, 64, 300], 0, 640, 384), ([2] * 70, 1, 256, 128), ([700, 3], 11, 1152, 640),
    # 128 x 128, 64 x 256 and 128 x 256 tiles, the last two with half a column tile
    ([300, 200, 1, 500], 5, 384, 2048), ([20, 0, 65, 7] * 10, 3, 640, 1152),
    ([700, 3, 900], 0, 256, 4224)])
def test_grouped_dgrad_against_dense(counts, spare, N, K, out_dtype, pow2):
    t = torch()
    E, T = len(counts), sum(counts) + spare
    g = t.Generator(device="cuda").manual_seed(8)
    dy, sdy = getattr(F, "fp8_quant_act_1x128" + suffix(pow2))(
        t.randn((T, N), generator=g, device="cuda").bfloat16())
    w, sw = getattr(F, "fp8_quant_weight_128x128" + suffix(pow2))(
        (t.randn((E * N, K), generator=g, device="cuda") / N ** 0.5).bfloat16())
    w, sw = w.view(E, N, K), sw.view(E, N // 128, K // 128)
    off = offsets_of(counts)
    dx = t.full((T, K), 7.0, device="cuda").to(t.float32 if out_dtype == "f32" else t.bfloat16)
    call = getattr(F, "fp8_block_grouped_gemm_dgrad" + suffix(pow2))
    assert call(dy, sdy, w, sw, off, out_dtype, dx) is dx
    ends = off.tolist()
    for e, (i, j) in enumerate(zip(ends, ends[1:])):
        if i < j:
            q, s = dy[i:j].contiguous(), sdy[i:j].contiguous()
            want = getattr(F, "fp8_block_gemm_dgrad" + suffix(pow2))(q, s, w[e], sw[e], out_dtype)
            assert t.equal(dx[i:j], want)
    assert (dx[sum(counts):] == 7).all()
    if out_dtype == "f32" and not pow2 and T > 5:
        i, j = ends[0], ends[1]
        if i < j:
            lut = e4m3_lut()
            x = lut[dy[i:j].cpu().numpy()] * np.repeat(sdy[i:j].double().cpu().numpy(), 128, 1)
            qw, ws = w[0].t().contiguous().cpu().numpy(), sw[0].t().contiguous().cpu().numpy()
            y = lut[qw] * np.repeat(np.repeat(ws.astype(np.float64), 128, 0), 128, 1)
            b = gemm_error_bound(dy[i:j].cpu().numpy(), sdy[i:j].cpu().numpy(), qw, ws)
            assert (np.abs(host(dx[i:j]) - x @ y.T) <= b).all()


def test_grouped_dgrad_no_rows():
    t = torch()
    w, sw = t.zeros((2, 128, 256), dtype=t.uint8, device="cuda"), t.ones((2, 1, 2), device="cuda")
    off = t.zeros(3, dtype=t.int32, device="cuda")
    dy, s = t.zeros((0, 128), dtype=t.uint8, device="cuda"), t.ones((0, 1), device="cuda")
    assert F.fp8_block_grouped_gemm_dgrad(dy, s, w, sw, off).shape == (0, 256)


def test_oracle_product_is_the_same_definition():
    # the helper's binary64 product against the C oracle's
    a, sa, w, sw = operands(9, 5, 128, 256)
    h, _ = exact_product(a, sa, w, sw, np.arange(5))
    want = oracle.block_gemm(a.cpu().numpy(), sa.cpu().numpy(), w.cpu().numpy(), sw.cpu().numpy())
    assert np.allclose(h, want, rtol=1e-12, atol=1e-12)
