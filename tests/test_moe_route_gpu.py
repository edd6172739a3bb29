"""Tokens sorted by expert and back, on the GPU against plain 64-bit numpy.

Integers, copied rows, E4M3 bytes and their scales must be equal.  Sums are
compared value by value with a bound derived from the arithmetic: a sum of n
FP32 fused multiply-adds is off by at most n 2^-24 of the sum of the
magnitudes, and the result is rounded once to its type (half a unit in the
last place: 2^-8 of a bf16 value, 2^-24 of an FP32 one).
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


def routing(seed, T, k, E, drop=0.0, wide=True):
    rng = np.random.default_rng(seed)
    p = np.arange(1, E + 1) ** -1.1
    ids = rng.choice(E, (T, k), p=p / p.sum())
    gone = rng.random((T, k)) < drop
    junk = rng.choice([-1, E, -E - 7, 2 ** 31 - 1] + ([2 ** 40, -2 ** 40, 2 ** 32] if wide else []),
                      (T, k))
    return np.where(gone, junk, ids).astype(np.int64 if wide else np.int32)


def plan_of(ids, E):
    flat = ids.reshape(-1).astype(np.int64)
    key = np.where((flat >= 0) & (flat < E), flat, E)
    order = np.argsort(key, kind="stable")
    offsets = np.searchsorted(key[order], np.arange(E + 1)).astype(np.int32)
    row_slot = np.where(np.arange(flat.size) < offsets[-1], order, -1).astype(np.int32)
    slot_row = np.full(flat.size, -1, np.int32)
    slot_row[order[:offsets[-1]]] = np.arange(offsets[-1], dtype=np.int32)
    return offsets, slot_row.reshape(ids.shape), row_slot


def cuda(a):
    return torch().from_numpy(np.ascontiguousarray(a)).cuda()


def draw(seed, shape, dtype="bf16", sigma=1.0):
    t = torch()
    v = t.from_numpy(np.random.default_rng(seed).standard_normal(shape, dtype=np.float32) * sigma)
    return v.to(t.bfloat16 if dtype == "bf16" else t.float32).cuda()


def f64(t):
    return t.detach().double().cpu().numpy()


def close(got, want, magnitudes, terms):
    """Each value within `terms` FP32 roundings of its magnitudes and the one
    rounding to its type."""
    u = U_BF16 if got.dtype == torch().bfloat16 else U32
    g = f64(got)
    bound = terms * U32 * magnitudes
    bound = bound + u * (np.abs(want) + bound) + 2.0 ** -126
    assert np.isfinite(g).all()
    bad = np.abs(g - want) > bound
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4], g[bad][:4], want[bad][:4])


SORTS = [(1, 1, 1, 0.0), (1, 8, 32, 0.0), (3, 2, 1024, 0.0), (256, 8, 32, 0.0), (64, 64, 64, 0.0),
         (4097, 1, 7, 0.1), (1037, 3, 10, 0.34), (1500, 6, 1000, 0.0), (5000, 8, 2, 0.0),
         (40, 5, 16, 1.0), (20000, 4, 256, 0.5), (63, 3, 5, 0.0), (4096, 1, 3, 0.9)]


@pytest.mark.parametrize("wide", [True, False])
@pytest.mark.parametrize("T,k,E,drop", SORTS)
def test_sort(T, k, E, drop, wide):
    ids = routing(T + k + E, T, k, E, drop, wide)
    want = plan_of(ids, E)
    got = M.fp8_moe_sort(cuda(ids), E)
    for g, w in zip(got, want):
        assert np.array_equal(host(g), w)


def test_sort_of_nothing_and_many_runs():
    t = torch()
    off, slot_row, row_slot = M.fp8_moe_sort(t.empty((0, 8), dtype=t.int64, device="cuda"), 5)
    assert host(off).tolist() == [0] * 6 and slot_row.shape == (0, 8) and row_slot.numel() == 0
    # more slots than 512 runs of 4096: longer runs
    ids = routing(9, 300001, 7, 61, 0.2)
    for g, w in zip(M.fp8_moe_sort(cuda(ids), 61), plan_of(ids, 61)):
        assert np.array_equal(host(g), w)


@pytest.mark.parametrize("dtype", ["uint8", "float8_e4m3fn", "bfloat16", "float16", "float32"])
@pytest.mark.parametrize("T,k,H,strided", [(1, 8, 7168, False), (1, 1, 1, False), (37, 3, 1001, True),
                                           (130, 2, 16, False), (33, 4, 2049, True),
                                           (5, 12, 129, False)])
def test_dispatch_copies_rows(T, k, H, strided, dtype):
    t = torch()
    ids = routing(H, T, k, 9, 0.3)
    off, slot_row, _ = plan_of(ids, 9)
    bits = np.random.default_rng(T).integers(0, 256, (T, (H + 5) * 4), dtype=np.uint8)
    full = cuda(bits).view(getattr(t, dtype))
    # rows with a stride that start one element into an allocation
    x = full[:, 1:1 + H] if strided else full[:, :H].contiguous()
    xs = cuda(np.full((T * k, H * x.element_size()), 0xA5, np.uint8)).view(x.dtype)
    M.fp8_moe_dispatch(x, cuda(slot_row), xs=xs)
    raw = host(x.contiguous().view(t.uint8))
    want = np.full((T * k, H * x.element_size()), 0xA5, np.uint8)
    for (tok, j), r in np.ndenumerate(slot_row):
        if r >= 0:
            want[r] = raw[tok]
    assert np.array_equal(host(xs.view(t.uint8)), want)


def test_dispatch_repeated_row_scales_and_few_rows():
    t = torch()
    T, k, H, G = 50, 3, 640, 5
    _, slot_row, _ = plan_of(routing(4, T, k, 6, 0.2), 6)
    q = cuda(np.random.default_rng(5).integers(0, 255, (T, H), dtype=np.uint8))
    s = draw(6, (T, 2 * G), "f32")[:, 3:3 + G]
    # 100 rows only: slots of later rows are dropped
    xs = t.zeros((100, H), dtype=t.uint8, device="cuda")
    ss = t.zeros((100, G), device="cuda")
    M.fp8_moe_dispatch(q, cuda(slot_row), scales=s, xs=xs, xs_scales=ss)
    qn, sn = host(q), host(s.contiguous())
    wq, ws = np.zeros((100, H), np.uint8), np.zeros((100, G), np.float32)
    for (tok, j), r in np.ndenumerate(slot_row):
        if 0 <= r < 100:
            wq[r], ws[r] = qn[tok], sn[tok]
    assert np.array_equal(host(xs), wq) and np.array_equal(host(ss), ws)
    one = draw(7, (1, H))
    got = M.fp8_moe_dispatch(one.expand(T, H), cuda(np.abs(slot_row)))  # stride 0
    assert t.equal(got[int(slot_row[0, 0])], one[0])


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("T,k,H", [(1, 8, 7168), (300, 2, 640), (37, 3, 1001), (70, 4, 5),
                                   (9, 1, 2050)])
def test_dispatch_quantizes_as_the_quantizer(T, k, H, pow2):
    ids = routing(H + 1, T, k, 11, 0.25)
    _, slot_row, _ = plan_of(ids, 11)
    x = draw(T, (T, H + 3))[:, 1:1 + H]
    x[0, :] = 0
    x[-1, : H // 2] *= 1e-38
    bits = host(x.contiguous().view(torch().int16)).view(np.uint16)
    qo, so = (oracle.quant_act_1x128_pow2 if pow2 else oracle.quant_act_1x128)(bits)
    q0 = cuda(np.full((T * k, H), 0x5A, np.uint8))
    s0 = cuda(np.full((T * k, (H + 127) // 128), -3, np.float32))
    suffix = "_pow2" if pow2 else ""
    q, s = getattr(M, "fp8_moe_dispatch_quant_1x128" + suffix)(x, cuda(slot_row), q=q0, scales=s0)
    wq = np.full((T * k, H), 0x5A, np.uint8)
    ws = np.full(s0.shape, -3, np.float32)
    for (tok, j), r in np.ndenumerate(slot_row):
        if r >= 0:
            wq[r], ws[r] = qo[tok], so[tok]
    assert np.array_equal(host(q), wq)
    assert np.array_equal(host(s).view(np.uint32), ws.view(np.uint32))
    # sort and gather in one call: the same plan and rows
    q1, s1 = cuda(np.full((T * k, H), 0x5A, np.uint8)), cuda(np.full(s0.shape, -3, np.float32))
    got = getattr(M, "fp8_moe_sort_dispatch_quant_1x128" + suffix)(x, cuda(ids), 11, q=q1,
                                                                   scales=s1)
    for g, w in zip(got[:3], plan_of(ids, 11)):
        assert np.array_equal(host(g), w)
    assert np.array_equal(host(got[3]), wq)
    assert np.array_equal(host(got[4]).view(np.uint32), ws.view(np.uint32))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,k,E,H,drop", [(1, 8, 32, 7168, 0.0), (0, 4, 3, 64, 0.0),
                                          (700, 8, 300, 96, 0.2), (515, 8, 16, 1001, 0.5),
                                          (8, 3, 4, 0, 0.0), (2000, 3, 1024, 40, 0.0),
                                          (4, 80, 100, 33, 0.1), (60, 20, 24, 130, 0.3)])
def test_sort_and_dispatch_in_one_call(T, k, E, H, drop, dtype):
    t = torch()
    ids = routing(T + H, T, k, E, drop)
    x = draw(T + 1, (T, H), dtype)
    xs = t.full((T * k, H), 7.0, dtype=x.dtype, device="cuda")
    got = M.fp8_moe_sort_dispatch(x, cuda(ids), E, xs=xs)
    want = plan_of(ids, E)
    for g, w in zip(got[:3], want):
        assert np.array_equal(host(g), w)
    ref = np.full((T * k, H), 7.0)
    kept = want[2][:want[0][-1]]
    ref[:kept.size] = f64(x)[kept // k]
    assert np.array_equal(f64(got[3]), ref)


COMBINES = [(1, 8, 32, 7168, 0.0), (1, 1, 1, 1, 0.0), (300, 3, 10, 1001, 0.34),
            (129, 9, 12, 640, 0.2), (33, 17, 20, 129, 0.5), (20, 2, 4, 2056, 1.0),
            (7, 0, 3, 40, 0.0), (515, 8, 64, 64, 0.0)]


@pytest.mark.parametrize("dtype,out_dtype", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"),
                                             ("f32", "bf16")])
@pytest.mark.parametrize("T,k,E,H,drop", COMBINES)
def test_combine(T, k, E, H, drop, dtype, out_dtype):
    t = torch()
    _, slot_row, _ = plan_of(routing(T * 3 + k, T, k, E, drop), E)
    R = T * k
    ys = draw(H, (R, H + 7), dtype)[:, 3:3 + H]
    w = draw(H + 1, (T, k), "f32")
    # what stands in rows and weights of dropped slots must not matter
    w[cuda(slot_row) < 0] = float("nan")
    used = np.zeros(R, bool)
    used[slot_row[slot_row >= 0]] = True
    ys[cuda(~used)] = float("inf")
    res = draw(H + 2, (T, H), out_dtype)
    sums, mags = np.zeros((T, H)), np.zeros((T, H))
    yn, wn = f64(ys), f64(w)
    for (tok, j), r in np.ndenumerate(slot_row):
        if r >= 0:
            sums[tok] += wn[tok, j] * yn[r]
            mags[tok] += np.abs(wn[tok, j] * yn[r])
    s = cuda(slot_row)
    close(M.fp8_moe_combine(ys, s, w, out_dtype=out_dtype), sums, mags, k + 1)
    rn = f64(res)
    close(M.fp8_moe_combine(ys, s, w, residual=res, out_dtype=out_dtype), sums + rn,
          mags + np.abs(rn), k + 1)
    M.fp8_moe_combine(ys, s, w, residual=res, out=res)  # in place
    close(res, sums + rn, mags + np.abs(rn), k + 1)
    # the gather's gradient: the same sum with weights of one
    plain, pmag = np.zeros((T, H)), np.zeros((T, H))
    for (tok, j), r in np.ndenumerate(slot_row):
        if r >= 0:
            plain[tok] += yn[r]
            pmag[tok] += np.abs(yn[r])
    close(M.fp8_moe_dispatch_grad(ys, s, out_dtype=out_dtype), plain, pmag, k + 1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,k,E,H,drop", COMBINES + [(64, 4, 8, 16, 0.0), (3, 2, 2, 20000, 0.0)])
def test_combine_grad_against_formula(T, k, E, H, drop, dtype):
    t = torch()
    _, slot_row, _ = plan_of(routing(T * 5 + k, T, k, E, drop), E)
    R = T * k
    dout = draw(H + 3, (T, H + 2), dtype)[:, 1:1 + H]
    ys, w = draw(H + 4, (R, H), dtype), draw(H + 5, (T, k), "f32")
    w[cuda(slot_row) < 0] = float("nan")
    dys0 = t.full((R, H), 11.0, dtype=ys.dtype, device="cuda")
    dys, dw = M.fp8_moe_combine_grad(dout, ys, cuda(slot_row), w, dys=dys0)
    dn, yn, wn = f64(dout), f64(ys), f64(w)
    want_dys = np.full((R, H), 11.0)
    want_dw, mag_dw = np.zeros((T, k)), np.zeros((T, k))
    for (tok, j), r in np.ndenumerate(slot_row):
        if r >= 0:
            want_dys[r] = wn[tok, j] * dn[tok]
            want_dw[tok, j] = (dn[tok] * yn[r]).sum()
            mag_dw[tok, j] = np.abs(dn[tok] * yn[r]).sum()
    close(dys, want_dys, np.abs(want_dys), 1)
    # a thread adds at most 8 ceil(H / 512) products in a row, then the
    # threads are added in a tree and across at most 16 waves
    close(dw, want_dw, mag_dw, 8 * -(-H // 512) + 30)
    one_dys, one_dw = M.fp8_moe_combine_grad(dout, ys, cuda(slot_row))
    close(one_dw, want_dw, mag_dw, 8 * -(-H // 512) + 30)
    kept = slot_row[slot_row >= 0]
    tok = np.nonzero(slot_row >= 0)[0]
    assert np.array_equal(f64(one_dys)[kept], dn[tok])


@pytest.mark.parametrize("dtype,T,k,H", [("bf16", 9000, 6, 1001), ("bf16", 18000, 3, 1000),
                                         ("bf16", 30000, 2, 1001), ("f32", 2100, 5, 2500)])
def test_many_rows(dtype, T, k, H):
    # more than 96 MiB of rows, and few and many slots a token
    t = torch()
    E = 16
    _, slot_row, _ = plan_of(routing(T, T, k, E, 0.1), E)
    s = cuda(slot_row)
    ys, w, dout = draw(1, (T * k, H), dtype), draw(2, (T, k), "f32"), draw(3, (T, H), dtype)
    out = M.fp8_moe_combine(ys, s, w)
    dys, dw = M.fp8_moe_combine_grad(dout, ys, s, w, dys=t.zeros_like(ys))
    want_dys = t.zeros(T * k, H, dtype=t.float64, device="cuda")
    sums = t.zeros(T, H, dtype=t.float64, device="cuda")
    mags, dots, dot_mags = sums.clone(), w.double() * 0, w.double() * 0
    for j in range(k):
        kept = (s[:, j] >= 0).double()[:, None]
        rows = s[:, j].clamp(min=0).long()
        terms = ys[rows].double() * kept * w[:, j, None].double()
        sums += terms
        mags += terms.abs()
        products = ys[rows].double() * kept * dout.double()
        dots[:, j], dot_mags[:, j] = products.sum(1), products.abs().sum(1)
        at = s[:, j] >= 0
        want_dys[rows[at]] = w[at, j, None].double() * dout[at].double()
    close(out, f64(sums), f64(mags), k + 1)
    # a thread adds 8 ceil(H / 512) products at most, then a tree of threads
    close(dw, f64(dots), f64(dot_mags), 8 * -(-H // 512) + 30)
    close(dys, f64(want_dys), f64(want_dys.abs()), 1)


def test_gradients_against_differences():
    # the maps are linear in ys, w and x, so a difference quotient of any step
    # has no truncation error: only FP32 rounding (about sqrt(n) 2^-24)
    t = torch()
    T, k, E, H = 60, 4, 7, 260
    ids = cuda(routing(8, T, k, E, 0.25))
    _, slot_row, _ = M.fp8_moe_sort(ids, E)
    ys, w = draw(1, (T * k, H), "f32"), draw(2, (T, k), "f32")
    dout, d_ys, d_w = draw(3, (T, H), "f32"), draw(4, (T * k, H), "f32"), draw(5, (T, k), "f32")

    def loss(ys, w):
        return float((M.fp8_moe_combine(ys, slot_row, w).double() * dout.double()).sum())

    dys, dw = M.fp8_moe_combine_grad(dout, ys, slot_row, w, dys=t.zeros_like(ys))
    step = 0.5
    scale = float(dout.norm() * ys.norm())
    num = (loss(ys + step * d_ys, w) - loss(ys - step * d_ys, w)) / (2 * step)
    assert abs(num - float((dys.double() * d_ys.double()).sum())) < 1e-5 * scale
    num = (loss(ys, w + step * d_w) - loss(ys, w - step * d_w)) / (2 * step)
    assert abs(num - float((dw.double() * d_w.double()).sum())) < 1e-5 * scale

    x, d_x, dxs = draw(6, (T, H), "f32"), draw(7, (T, H), "f32"), draw(8, (T * k, H), "f32")

    def gathered(x):
        xs = M.fp8_moe_dispatch(x, slot_row, xs=t.zeros((T * k, H), device="cuda"))
        return float((xs.double() * dxs.double()).sum())

    num = (gathered(x + step * d_x) - gathered(x - step * d_x)) / (2 * step)
    dx = M.fp8_moe_dispatch_grad(dxs, slot_row)
    assert abs(num - float((dx.double() * d_x.double()).sum())) < 1e-5 * scale


def test_same_result_every_run_and_on_another_stream():
    t = torch()
    T, k, E, H = 513, 8, 32, 1000
    ids, x = cuda(routing(3, T, k, E)), draw(9, (T, H))
    w, ys = draw(10, (T, k), "f32"), draw(11, (T * k, H))

    def chain(stream=None):
        off, slot_row, row_slot, q, s = M.fp8_moe_sort_dispatch_quant_1x128(x, ids, E,
                                                                            stream=stream)
        out = M.fp8_moe_combine(ys, slot_row, w, stream=stream)
        dys, dw = M.fp8_moe_combine_grad(out, ys, slot_row, w, stream=stream)
        return off, slot_row, row_slot, q, s, out, dys, dw

    first = chain()
    other = t.cuda.Stream()
    for _ in range(3):
        other.wait_stream(t.cuda.current_stream())
        again = chain(other)
        t.cuda.current_stream().wait_stream(other)
        for a, b in zip(first, again):
            assert t.equal(a, b)


def test_rows_past_32_bit_offsets():
    # 2^31 bytes and more between the first row and the last: row offsets are
    # 64-bit
    t = torch()
    T, H = 300, 8192
    R = 140000  # 140000 x 8192 bf16 = 2.3 GB
    ys = t.zeros((R, H), dtype=t.bfloat16, device="cuda")
    rows = np.linspace(0, R - 1, T).astype(np.int32)[:, None]
    vals = draw(1, (T, H))
    ys[cuda(rows[:, 0].astype(np.int64))] = vals
    out = M.fp8_moe_combine(ys, cuda(rows))
    assert t.equal(out, vals)
    xs = t.zeros((R, H), dtype=t.bfloat16, device="cuda")
    M.fp8_moe_dispatch(vals, cuda(rows), xs=xs)
    assert t.equal(xs, ys)
