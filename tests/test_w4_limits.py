"""Sizes that the 4-bit products take up to the documented limits: many output
columns, and many experts with many columns, whose launches stay small because
a workgroup takes several column tiles."""
import ctypes

import numpy as np
import pytest

from fp8_fine_grained_token_amd import binding as B
from fp8_fine_grained_token_amd import moe as M

from .gpu_util import torch

A, N = ctypes.c_void_p(0x10000), ctypes.c_void_p(0)


def test_sizes_below_the_limits_are_not_refused():
    # with no result to write to, a call within the limits gets as far as that
    def dense(n, k):
        return M._fn("fp8_w4_matvec")(A, k, A, A, 1, 2, n, k, N, B.FP8_OUT_BF16, N)

    def grouped(e, n, k):
        return M._fn("fp8_w4_grouped_matvec")(A, k, A, A, 1, A, e, 8, n, k, N, B.FP8_OUT_BF16, N)

    assert dense(1 << 26, 64) == dense((1 << 31) - 1, 1) == B.FP8_ERR_NULL
    assert grouped(8192, 8192, 64) == grouped(65535, 8192, 1024) == B.FP8_ERR_NULL
    assert dense(1 << 31, 1) == dense(1 << 20, 1 << 20) == B.FP8_ERR_SHAPE
    assert grouped(65536, 8, 64) == grouped(65535, 8192, 4096) == B.FP8_ERR_SHAPE


@pytest.fixture
def gpu():
    t = torch()
    if not t.cuda.is_available():
        pytest.skip("no GPU")
    B.lib()
    yield t
    t.cuda.synchronize()


def e2m1(t, code):
    return t.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6],
                    device="cuda")[code.int()]


@pytest.mark.gpu
def test_many_columns(gpu):
    # two channels: every result is exact in fp32
    t, n = gpu, (1 << 26) + 5
    codes = t.randint(0, 256, (n, 1), dtype=t.uint8, device="cuda")
    scales = t.randint(125, 130, (n, 1), dtype=t.uint8, device="cuda")
    x = t.tensor([[1.5, -2.0]], dtype=t.bfloat16, device="cuda")
    y = M.fp8_w4_matvec(x, codes, scales, out_dtype="f32")
    want = e2m1(t, codes & 15) * 1.5 - e2m1(t, codes >> 4) * 2.0
    assert t.equal(y[0], (want * t.exp2(scales.float() - 127))[:, 0])


@pytest.mark.gpu
def test_many_experts_of_many_columns(gpu):
    # 1 GiB of codes; rows with a single channel, so that results are exact
    t, E, n, K = gpu, 8192, 8192, 32
    codes = t.randint(0, 256, (E, n, K // 2), dtype=t.uint8, device="cuda")
    scales = t.randint(125, 130, (E, n, 1), dtype=t.uint8, device="cuda")
    rows = [0, 1, 1, 77, 4095, 4096, 8190, 8191]  # each row's expert
    off = np.searchsorted(rows, np.arange(E + 1)).astype(np.int32)
    x = t.zeros((8, K), dtype=t.bfloat16, device="cuda")
    for i in range(8):
        x[i, 3 * i] = 1.0 + i
    y = M.fp8_w4_grouped_matvec(x, codes, scales, t.from_numpy(off).cuda(), out_dtype="f32")
    for i, e in enumerate(rows):
        c = codes[e, :, 3 * i // 2]
        w = e2m1(t, c >> 4 if 3 * i % 2 else c & 15) * t.exp2(scales[e, :, 0].float() - 127)
        assert t.equal(y[i], w * (1.0 + i)), i
