"""Products of a gated feed-forward block run once with the released library
and once with the race-check build (see poison_cases and
test_gated_poison_gpu).  Each case covers one tile kind and pipeline.

Run as a script (python tests/gated_poison_cases.py OUT.npz) it computes every
case with whatever library FP8BLK_LIB names and saves the outputs.
"""
import os
import sys

import numpy as np

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

# rows, inner width, K: 256-row tiles, 128-row tiles, 64-row tiles, K in parts
# on 64-row and on 32-row tiles, 32-row tiles
DENSE = {"big": (2305, 4096, 384), "mid": (4097, 512, 1152), "half": (1000, 2048, 1280),
         "parts": (300, 256, 2304), "row_parts": (30, 128, 2304), "few": (3, 256, 1152),
         "row": (20, 32768, 640)}
# rows of each expert, inner width, K: 32-row, 64-row and 128-row tiles, K in
# parts on 64-row and on 32-row tiles
GROUPED = {"rows": ([20, 0, 33, 1] * 10, 2048, 1152), "half": ([30, 70, 0, 40] * 4, 2048, 1152),
           "mid": ([300, 0, 129, 257], 2048, 640), "parts": ([50, 0, 90], 128, 2304),
           "row_parts": ([9, 0, 5], 128, 2304)}
# rows of each expert, inner dimension, columns: 64 x 128, 128 x 128, 64 x 256 and
# 128 x 256 tiles
DGRAD = {"small": ([300, 0, 129, 1, 257, 70], 1280, 512), "short": ([300, 200, 1, 500], 1280, 2048),
         "half": ([20, 0, 65, 7] * 10, 1280, 1152), "mid": ([700, 3, 900], 1280, 4224)}


def run_cases():
    import torch
    import fp8_fine_grained_token_amd as F

    out = {}

    def keep(name, *tensors):
        torch.cuda.synchronize()
        for i, x in enumerate(tensors):
            out[f"{name}_{i}"] = x.contiguous().view(torch.uint8).cpu().numpy().copy()

    def operands(seed, M, I, K, E, pow2):
        g = torch.Generator(device="cuda").manual_seed(seed)
        end = "_pow2" if pow2 else ""
        x = torch.randn((M, K), generator=g, device="cuda").to(torch.bfloat16)
        w = (torch.randn((max(1, E) * 2 * I, K), generator=g, device="cuda")
             * K ** -0.5).to(torch.bfloat16)
        a, sa = getattr(F, "fp8_quant_act_1x128" + end)(x)
        w, sw = getattr(F, "fp8_quant_weight_128x128" + end)(w)
        if E:
            w, sw = w.view(E, 2 * I, K), sw.view(E, 2 * I // 128, K // 128)
        return a, sa, w, sw

    for pow2 in (False, True):
        end = "_pow2" if pow2 else ""
        for name, (M, I, K) in DENSE.items():
            ops = operands(1, M, I, K, 0, pow2)
            keep(name + end, *getattr(F, "fp8_block_gemm_gated_quant_1x128" + end)(
                *ops, checkpoint=True))
        for name, (counts, I, K) in GROUPED.items():
            E = len(counts)
            ops = operands(2, sum(counts), I, K, E, pow2)
            off = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).cuda()
            keep("grouped_" + name + end,
                 *getattr(F, "fp8_block_grouped_gemm_gated_quant_1x128" + end)(
                     *ops, off, checkpoint=True))
        for name, (counts, N, K) in DGRAD.items():
            dy, s, _, _ = operands(3, sum(counts), 128, N, 0, pow2)
            _, _, w, sw = operands(4, 1, N // 2, K, len(counts), pow2)
            off = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).cuda()
            keep("grouped_dgrad_" + name + end, getattr(F, "fp8_block_grouped_gemm_dgrad" + end)(
                dy, s, w, sw, off, out_dtype="f32"))
    return out


if __name__ == "__main__":
    res = run_cases()
    np.savez(sys.argv[1], **res)
    print("cases done:", ", ".join(sorted(res)), flush=True)
