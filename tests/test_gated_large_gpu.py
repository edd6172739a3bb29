"""Operators of a gated feed-forward block on matrices whose offsets pass 32
bits: the last rows (or the last expert's) are bit for bit those of a call on
them alone."""
import pytest

import fp8_fine_grained_token_amd as F
from fp8_fine_grained_token_amd import binding as B

from .ffn_util import without_workspace
from .gpu_util import torch

pytestmark = pytest.mark.gpu

M, I = 530_001, 4096          # [M][2 I] has more than 2^32 elements
START = M // 128 * 128 - 128  # a group's first row
E, K = 80, 7168               # and [E][2 I][K] too


@pytest.fixture(autouse=True)
def _gpu():
    t = torch()
    if not t.cuda.is_available():
        pytest.skip("no GPU")
    B.lib()
    yield
    t.cuda.synchronize()
    t.cuda.empty_cache()


def codes(*shape):
    """Random finite E4M3 bytes."""
    t = torch()
    q = t.randint(0, 127, shape, dtype=t.uint8, device="cuda")
    q[..., ::3] |= 0x80
    return q


def uniform(*shape):
    return torch().rand(shape, device="cuda") + 0.5


def test_checkpoint():
    t = torch()
    h, s = codes(M, 2 * I), uniform(M, I // 64)
    x = F.fp8_dequant_act_1x128(h, s)
    assert t.equal(x[START:], F.fp8_dequant_act_1x128(h[START:], s[START:]))
    del x
    q, sq = F.fp8_requant_act_128x1_t(h, s)
    wq, ws = F.fp8_requant_act_128x1_t(h[START:], s[START:])
    assert t.equal(q[:, START:], wq) and t.equal(sq[:, START // 128:], ws)


@pytest.mark.parametrize("out_dtype", ["f32", "bf16"])
def test_wide_row(out_dtype):
    # the widest row there may be, whose fp32 values end just below 2^32 bytes,
    # against the same groups as many short rows
    t = torch()
    wide, cut = (1 << 30) - 131, (1 << 30) - (1 << 20)
    q, s = codes(1, wide), uniform(1, (wide + 127) // 128)
    x = t.full((1, wide), 7.0, device="cuda").to(t.float32 if out_dtype == "f32" else t.bfloat16)
    F.fp8_dequant_act_1x128(q, s, out_dtype=out_dtype, x=x)
    parts = F.fp8_dequant_act_1x128(q[:, :cut].view(-1, 1 << 20),
                                    s[:, :cut // 128].view(-1, 1 << 13), out_dtype=out_dtype)
    assert t.equal(x[0, :cut], parts.view(-1))
    tail = F.fp8_dequant_act_1x128(q[:, cut:].contiguous(), s[:, cut // 128:].contiguous(),
                                   out_dtype=out_dtype)
    assert t.equal(x[:, cut:], tail)
    del x, parts
    q_t, _ = F.fp8_requant_act_128x1_t(q, s)
    assert t.equal(q_t[cut:], F.fp8_requant_act_128x1_t(q[:, cut:].contiguous(),
                                                        s[:, cut // 128:].contiguous())[0])


def test_gradient():
    t = torch()
    h, s = codes(M, 2 * I), uniform(M, I // 64) * 2.0 ** -6
    da = t.empty((M, I), dtype=t.bfloat16, device="cuda").normal_()
    tail = (da[START:], h[START:], s[START:])
    dh = F.fp8_gated_grad(da, h, s)
    assert t.equal(dh[START:], F.fp8_gated_grad(*tail))
    del dh
    q, sq = F.fp8_gated_grad_quant_1x128(da, h, s)
    wq, ws = F.fp8_gated_grad_quant_1x128(*tail)
    assert t.equal(q[START:], wq) and t.equal(sq[START:], ws)
    del q, sq
    got, want = F.fp8_gated_grad_quant(da, h, s), F.fp8_gated_grad_quant(*tail)
    for i, (g, w) in enumerate(zip(got, want)):
        cut = g[START:] if i < 2 else g[:, START // 128 if i % 2 else START:]
        assert t.equal(cut, w), i


def test_product():
    t = torch()
    a, sa, w, sw = codes(M, 128), uniform(M, 1), codes(2 * I, 128), uniform(I // 64, 1)
    name = "fp8_block_gemm_gated_quant_1x128"
    got = without_workspace(name, a, sa, w, sw, "silu", quant=True)
    want = without_workspace(name, a[START:], sa[START:], w, sw, "silu", quant=True)
    for g, v in zip(got, want):
        assert t.equal(g[START:], v)


@pytest.mark.parametrize("rows", [2, 30, 80])  # 32-row, 64-row and 128-row tiles
def test_experts(rows):
    t = torch()
    w, sw = codes(E, 2 * I, K), uniform(E, I // 64, K // 128) * 2.0 ** -12
    a, sa = codes(E * rows, K), uniform(E * rows, K // 128)
    off = t.arange(0, (E + 1) * rows, rows, dtype=t.int32, device="cuda")
    one = t.tensor([0, rows], dtype=t.int32, device="cuda")
    name = "fp8_block_grouped_gemm_gated_quant_1x128"
    got = without_workspace(name, a, sa, w, sw, "silu", quant=True, offsets=off)
    want = without_workspace(name, a[-rows:], sa[-rows:], w[-1:], sw[-1:], "silu", quant=True,
                             offsets=one)
    for g, v in zip(got, want):
        assert t.equal(g[-rows:], v)
    dy, sdy = codes(E * rows, 2 * I), uniform(E * rows, I // 64)
    dx = F.fp8_block_grouped_gemm_dgrad(dy, sdy, w, sw, off)
    assert t.equal(dx[-rows:], F.fp8_block_grouped_gemm_dgrad(dy[-rows:], sdy[-rows:], w[-1:],
                                                              sw[-1:], one))
