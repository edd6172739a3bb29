"""The operators around the expert products used together: the example block
against fp32 torch, and inside a captured HIP graph.

The example's distances are those of its number formats.  E4M3 keeps 4
significant bits: an operand is off by about 2^-5 / sqrt(3) = 1.8% of itself,
so a product of two quantized operands by 2.6% and the two products of an
expert (with the activation between them) by about 4%; E2M1 keeps 2 bits,
about 11% an operand, and the two products are off by about 16%.  Twice those
is allowed; anything misplaced is off by 100%.
"""
import importlib.util
import os

import numpy as np
import pytest

from fp8_fine_grained_token_amd import binding as B
from fp8_fine_grained_token_amd import moe as M

from .gpu_util import log, torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    t = torch()
    if not t.cuda.is_available():
        pytest.skip("no GPU")
    B.lib()
    yield
    t.cuda.synchronize()


def example():
    spec = importlib.util.spec_from_file_location(
        "moe_block", os.path.join(ROOT, "examples", "moe_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("sizes", [dict(), dict(width=256, inner=128, experts=5, top_k=3,
                                                tokens=37, decoded=1)])
def test_example_block(sizes):
    for what, far in example().main(**sizes).items():
        log(f"  {what}: {far:.4f}")
        limit = 0.32 if "4 bits" in what else 0.08
        assert far < limit, what


def test_graph_of_a_decode_step():
    # norm, sort and gather, 4-bit products and the weighted sum captured once
    # and replayed on fresh inputs, every replay against the eager chain
    t = torch()
    m = example()
    block = m.MoeBlock(512, 256, 6, 2)
    tokens = 5
    y, r = (t.randn(tokens, 512, device="cuda").to(t.bfloat16) for _ in range(2))
    ids = t.zeros((tokens, 2), dtype=t.int64, device="cuda")
    weights = t.full((tokens, 2), 0.5, device="cuda")

    def step():
        r_out, q, s, rs1, rs2 = M.fp8_norm_residual_quant_1x128(y, r, block.w_post, block.gate,
                                                                block.w_pre)
        _, n, _, _ = M.fp8_norm_residual(y, r, block.w_post, block.gate, block.w_pre)
        off, slot_row, row_slot, xs = M.fp8_moe_sort_dispatch(n, ids, 6)
        qs, ss = M.fp8_moe_dispatch(q, slot_row, scales=s)
        h = M.fp8_w4_grouped_matvec(xs, *block.up_w4, off)
        ys = M.fp8_w4_grouped_matvec(h[:, :256].contiguous(), *block.down_w4, off)
        out = M.fp8_moe_combine(ys, slot_row, weights, residual=r_out)
        dys, dw = M.fp8_moe_combine_grad(out, ys, slot_row, weights)
        dn = M.fp8_moe_dispatch_grad(dys, slot_row)
        grads = M.fp8_norm_residual_grad(dn, out, y, r_out, rs1, rs2, block.w_post, block.gate,
                                         block.w_pre)
        return (r_out, qs, ss, off, slot_row, row_slot, ys, out, dys, dw, dn) + grads

    def fresh(seed):
        g = np.random.default_rng(seed)
        y.copy_(t.from_numpy(g.standard_normal((tokens, 512), dtype=np.float32)))
        r.copy_(t.from_numpy(g.standard_normal((tokens, 512), dtype=np.float32)))
        ids.copy_(t.from_numpy(g.integers(0, 6, (tokens, 2))))
        weights.copy_(t.from_numpy(g.random((tokens, 2), dtype=np.float32)))

    fresh(0)
    s = t.cuda.Stream()
    s.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(s):
        step()
    t.cuda.current_stream().wait_stream(s)
    t.cuda.synchronize()
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        outs = step()
    for seed in range(1, 5):
        fresh(seed)
        t.cuda.synchronize()
        graph.replay()
        t.cuda.synchronize()
        for i, (a, b) in enumerate(zip(outs, step())):
            assert t.equal(a, b), (seed, i)


def test_large_sort_in_a_graph():
    # the two-launch sort, its counts in a workspace of the caller's
    t = torch()
    T, k, E = 3000, 5, 100
    ids = t.randint(0, E, (T, k), device="cuda")
    ws = t.empty(M.fp8_moe_sort_workspace_bytes(T, k, E), dtype=t.uint8, device="cuda")
    M.fp8_moe_sort(ids, E, workspace=ws)
    t.cuda.synchronize()
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        outs = M.fp8_moe_sort(ids, E, workspace=ws)
    for seed in range(3):
        t.manual_seed(seed)
        ids.copy_(t.randint(-1, E + 1, (T, k), device="cuda"))
        graph.replay()
        t.cuda.synchronize()
        for a, b in zip(outs, M.fp8_moe_sort(ids, E)):
            assert t.equal(a, b)
