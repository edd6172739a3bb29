"""FP8BLK_LOG for the products of a gated feed-forward block: every call prints
the plan that it launches, as the other GEMMs do.  The flag is read once per
process, so the calls run in a child process.
"""
import os
import subprocess
import sys

import pytest

from .gpu_util import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import sys
sys.path.insert(0, %r)
import torch
import fp8_fine_grained_token_amd as F
from tests.ffn_util import operands, without_workspace
quant = F.fp8_block_gemm_gated_quant_1x128
grouped = F.fp8_block_grouped_gemm_gated_quant_1x128_pow2
F.fp8_block_gemm_gated(*operands(1, 1, 256, 256))
quant(*operands(1, 3, 256, 256))
quant(*operands(1, 30, 256, 1024))
F.fp8_block_gemm_gated_pow2(*operands(1, 200, 256, 1024, True))
without_workspace("fp8_block_gemm_gated", *operands(1, 30, 256, 256), "silu")
quant(*operands(1, 20, 32768, 128))
quant(*operands(1, 129, 32768, 128))
for rows, inner in ((2, 640), (20, 8192), (60, 8192), (70, 8192)):
    off = torch.tensor([0, rows, 2 * rows], dtype=torch.int32, device="cuda")
    grouped(*operands(1, 2 * rows, inner, 128, True, experts=2), off)
a, sa, w, sw = operands(1, 40, 128, 256, experts=2)
off = torch.tensor([0, 0, 40], dtype=torch.int32, device="cuda")
F.fp8_block_grouped_gemm_dgrad(a, sa, w, sw, off)
torch.cuda.synchronize()
print("child done", flush=True)
""" % ROOT

EXPECT = [
    "block_gemm_gated M=1 N=512 K=256 tiles=16x16 in registers ksplit=1",
    "block_gemm_gated_quant_1x128 M=3 N=512 K=256 tiles=16x16 in registers + sums ksplit=1",
    "block_gemm_gated_quant_1x128 M=30 N=512 K=1024 tiles=32x64 parts + sums ksplit=2",
    "block_gemm_gated_pow2 M=200 N=512 K=1024 tiles=64x64 parts + sums ksplit=2",
    "block_gemm_gated M=30 N=512 K=256 tiles=64x256 ksplit=1",
    "block_gemm_gated_quant_1x128 M=20 N=65536 K=128 tiles=32x256 ksplit=1",
    "block_gemm_gated_quant_1x128 M=129 N=65536 K=128 tiles=256x256 ksplit=1",
    "block_grouped_gemm_gated_quant_1x128_pow2 M=4 N=1280 K=128 tiles=32x64 parts + sums ksplit=1",
    "block_grouped_gemm_gated_quant_1x128_pow2 M=40 N=16384 K=128 tiles=32x256 ksplit=1",
    "block_grouped_gemm_gated_quant_1x128_pow2 M=120 N=16384 K=128 tiles=64x256 ksplit=1",
    "block_grouped_gemm_gated_quant_1x128_pow2 M=140 N=16384 K=128 tiles=128x256 ksplit=1",
    "block_grouped_gemm_dgrad M=40 N=256 K=256 tiles=64x128 per expert ksplit=1",
]


@pytest.mark.parametrize("on", [True, False])
def test_plan_lines(on):
    t = torch()
    if not t.cuda.is_available():
        pytest.skip("no GPU")
    env = dict(os.environ)
    env.pop("FP8BLK_LOG", None)
    if on:
        env["FP8BLK_LOG"] = "1"
    r = subprocess.run([sys.executable, "-c", CHILD], capture_output=True, text=True, env=env,
                       timeout=120)
    assert r.returncode == 0, r.stderr[-3000:]
    assert "child done" in r.stdout
    lines = [ln for ln in r.stderr.splitlines() if ln.startswith("fp8blk: ")]
    print("\n".join(lines))
    assert len(lines) == (len(EXPECT) if on else 0), lines
    for line, want in zip(lines, EXPECT):
        assert want in line, (line, want)
