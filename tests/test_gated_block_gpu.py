"""The operators of a gated feed-forward block run together: a training step
against autograd in fp32, in captured graphs, on other streams and two at once.

Distances from fp32 are those of the number formats.  E4M3 keeps 4 significant
bits: an operand is off by about 2^-5 / sqrt(3) = 1.8% of itself, a product of
two by 2.6%; errors of different origin add as squares.  g and u are off by
2.6% each, so act(g) u by 3.7% (silu and gelu keep relative errors within about
their size here), kept in 8 bits by 3.2% and act(g) u from them by 4.5%.
  result: act(g) u 3.7%, its rounding and the weights' 2.6%: 4.5%
  dh: the product 2.6%, the kept g and u 3.2% each: 5.2%
  dx: dh, its rounding and the weights' 2.6%: 5.8%
  dW up: dh and its rounding 5.5%, x rounded twice 2.6%: 6.1%
  dW down: dy 1.8%, act(g) u from the kept values 4.5%, its rounding: 5.2%
Twice those is allowed (power-of-two scales reach no further: a group's values
use the same 4 bits); anything misplaced is off by 100%.
"""
import numpy as np
import pytest

import fp8_fine_grained_token_amd as F
from fp8_fine_grained_token_amd import binding as B

from .ffn_util import ACTS
from .gpu_util import log, torch

pytestmark = pytest.mark.gpu

LIMITS = {"y": 0.09, "dx": 0.116, "dw_up": 0.122, "dw_down": 0.104}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    t = torch()
    if not t.cuda.is_available():
        pytest.skip("no GPU")
    B.lib()
    yield
    t.cuda.synchronize()


def forms(pow2):
    """A function's form for these scales."""
    return lambda name: getattr(F, name + ("_pow2" if pow2 else ""))


class Block:
    """y = (act(g) u) w_down^T, [g | u] = x w_up^T, with 8-bit products."""

    def __init__(self, width, inner, act, pow2, seed=0):
        t = torch()
        g = t.Generator(device="cuda").manual_seed(seed)
        self.f, self.act, self.inner = forms(pow2), act, inner
        self.up = (t.randn((2 * inner, width), generator=g, device="cuda")
                   * width ** -0.5).to(t.bfloat16)
        self.down = (t.randn((width, inner), generator=g, device="cuda")
                     * inner ** -0.5).to(t.bfloat16)
        self.up8 = self.f("fp8_quant_weight_128x128")(self.up)
        self.down8 = self.f("fp8_quant_weight_128x128")(self.down)

    def forward(self, x):
        f = self.f
        q, s = f("fp8_quant_act_1x128")(x)
        a, a_s, h, h_s = f("fp8_block_gemm_gated_quant_1x128")(
            q, s, *self.up8, activation=self.act, checkpoint=True)
        return f("fp8_block_gemm")(a, a_s, *self.down8), (q, s, h, h_s)

    def backward(self, dy, saved):
        """(dx, dw_up, dw_down); the weight gradients where the products take
        the rows (a multiple of 128)."""
        f, (q, s, h, h_s) = self.f, saved
        da = f("fp8_block_gemm_dgrad")(*f("fp8_quant_act_1x128")(dy), *self.down8)
        if dy.shape[0] % 128:
            dh = f("fp8_gated_grad_quant_1x128")(da, h, h_s, activation=self.act)
            return f("fp8_block_gemm_dgrad")(*dh, *self.up8), None, None
        g, g_s, g_t, g_ts, a_t, a_ts = f("fp8_gated_grad_quant")(da, h, h_s, activation=self.act)
        x_t = f("fp8_requant_act_128x1_t")(q, s)
        dw_up = f("fp8_block_gemm_wgrad")(g_t, g_ts, *x_t)
        dw_down = f("fp8_block_gemm_wgrad")(*f("fp8_quant_act_128x1_t")(dy), a_t, a_ts)
        return f("fp8_block_gemm_dgrad")(g, g_s, *self.up8), dw_up, dw_down

    def plain(self, x, dy):
        t = torch()
        act = (t.nn.functional.silu if self.act == "silu" else
               lambda v: t.nn.functional.gelu(v, approximate="tanh"))
        x, up, down = (v.float().requires_grad_() for v in (x, self.up, self.down))
        h = x @ up.t()
        y = (act(h[:, :self.inner]) * h[:, self.inner:]) @ down.t()
        return (y.detach(),) + t.autograd.grad(y, (x, up, down), dy.float())


def rows(seed, n, width):
    t = torch()
    g = t.Generator(device="cuda").manual_seed(seed)
    return t.randn((n, width), generator=g, device="cuda").to(t.bfloat16)


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,width,inner", [(1, 256, 128), (77, 640, 384), (256, 512, 256),
                                           (384, 1024, 1408), (1920, 256, 640)])
def test_training_step(M, width, inner, act, pow2):
    b = Block(width, inner, act, pow2)
    x, dy = rows(1, M, width), rows(2, M, width)
    y, saved = b.forward(x)
    got = (y,) + b.backward(dy, saved)
    for (what, limit), a, w in zip(LIMITS.items(), got, b.plain(x, dy)):
        if a is None:
            continue
        far = float((a.float() - w).norm() / w.norm())
        log(f"  {M} x {width} x {inner} {act}: {what} {far:.4f}")
        # a single row has few values to average over
        assert far < (limit if M > 1 else 1.5 * limit), what


@pytest.mark.parametrize("M,width,inner", [(4, 256, 384), (128, 1024, 256), (256, 512, 2048)])
def test_step_in_a_graph(M, width, inner):
    # captured once, replayed on fresh inputs with other work in between, every
    # replay against the eager step
    t = torch()
    b = Block(width, inner, "silu", False)
    x, dy = rows(1, M, width), rows(2, M, width)

    def step():
        y, saved = b.forward(x)
        dx, dw_up, dw_down = b.backward(dy, saved)
        kept = F.fp8_dequant_act_1x128(saved[2], saved[3])
        dh = F.fp8_gated_grad(dy.repeat(1, -(-inner // width))[:, :inner], kept)
        return [v for v in (y, *saved, dx, dw_up, dw_down, kept, dh) if v is not None]

    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(side):
        step()
    t.cuda.current_stream().wait_stream(side)
    t.cuda.synchronize()
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        outs = step()
    for seed in range(3, 7):
        x.copy_(rows(seed, M, width))
        dy.copy_(rows(seed + 10, M, width))
        t.cuda.synchronize()
        graph.replay()
        t.cuda.synchronize()
        for i, (a, w) in enumerate(zip(outs, step())):
            assert t.equal(a, w), (seed, i)


def grouped_step(xs, dys, up8, down8, offsets, outs):
    """Grouped forward and backward into the given outputs; the rows behind the
    last expert's stay as they are."""
    q, s = F.fp8_quant_act_1x128(xs)
    F.fp8_block_grouped_gemm_gated_quant_1x128(q, s, *up8, offsets, checkpoint=True, q=outs["q"],
                                               scales=outs["s"], h=outs["h"],
                                               h_scales=outs["h_s"])
    F.fp8_block_grouped_gemm(outs["q"], outs["s"], *down8, offsets, c=outs["y"])
    F.fp8_block_grouped_gemm_dgrad(*F.fp8_quant_act_1x128(dys), *down8, offsets, dx=outs["da"])
    dh = F.fp8_gated_grad_quant_1x128(outs["da"], outs["h"], outs["h_s"])
    F.fp8_block_grouped_gemm_dgrad(*dh, *up8, offsets, dx=outs["dx"])
    return outs


@pytest.mark.parametrize("T,E,width,inner", [(40, 6, 256, 128), (400, 4, 512, 640),
                                             (300, 9, 1024, 1152)])
def test_grouped_step_in_a_graph(T, E, width, inner):
    # expert ranges that change between replays, some empty, with rows behind
    # the last one's
    t = torch()
    g = t.Generator(device="cuda").manual_seed(3)

    def weights(n, k):
        w = (t.randn((E * n, k), generator=g, device="cuda") * k ** -0.5).to(t.bfloat16)
        q, s = F.fp8_quant_weight_128x128(w)
        return q.view(E, n, k), s.view(E, n // 128, k // 128)

    up8, down8 = weights(2 * inner, width), weights(width, inner)
    xs, dys = rows(1, T, width), rows(2, T, width)
    offsets = t.zeros(E + 1, dtype=t.int32, device="cuda")

    def blank():
        # zeros, so that rows of no expert hold values that the chain may read
        z = {"q": (T, inner), "h": (T, 2 * inner)}
        f = {"s": (T, inner // 128), "h_s": (T, inner // 64)}
        b = {"y": (T, width), "da": (T, inner), "dx": (T, width)}
        return {k: t.zeros(v, dtype=d, device="cuda") for part, d in (
            (z, t.uint8), (f, t.float32), (b, t.bfloat16)) for k, v in part.items()}

    def fresh(seed):
        r = np.random.default_rng(seed)
        used = int(r.integers(T // 2, T + 1))
        cuts = np.sort(r.integers(0, used + 1, E - 1))
        off = np.concatenate([[0], cuts, [used]])
        off[2] = off[1]  # an expert without rows
        offsets.copy_(t.from_numpy(off.astype(np.int32)))
        xs.copy_(rows(seed, T, width))
        dys.copy_(rows(seed + 50, T, width))
        t.cuda.synchronize()
        return used

    fresh(10)
    outs = blank()
    grouped_step(xs, dys, up8, down8, offsets, outs)
    t.cuda.synchronize()
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        grouped_step(xs, dys, up8, down8, offsets, outs)
    for seed in range(11, 16):
        used = fresh(seed)
        for v in outs.values():
            v.zero_()
        t.cuda.synchronize()
        graph.replay()
        t.cuda.synchronize()
        want = grouped_step(xs, dys, up8, down8, offsets, blank())
        for k, v in outs.items():
            assert t.equal(v, want[k]), (seed, k)
            assert not v[used:].any(), (seed, k, "rows of no expert")
        assert outs["dx"][:used].abs().sum() > 0


@pytest.mark.parametrize("M", [1, 40, 300])
def test_other_streams_and_two_at_once(M):
    # stream= and the current stream; two calls in flight have workspaces of
    # their own
    t = torch()
    K, I = 2048, 512
    b = Block(K, I, "silu", False)
    xs = [F.fp8_quant_act_1x128(rows(i, M, K)) for i in range(2)]
    want = [F.fp8_block_gemm_gated_quant_1x128(*x, *b.up8, checkpoint=True) for x in xs]
    da = rows(9, M, I)
    grads = [F.fp8_gated_grad_quant(da, w[2], w[3]) for w in want]
    t.cuda.synchronize()
    streams = [t.cuda.Stream() for _ in range(2)]
    got, got_grads = [[], []], [[], []]
    for _ in range(8):
        for i, s in enumerate(streams):
            if i:
                r = F.fp8_block_gemm_gated_quant_1x128(*xs[i], *b.up8, checkpoint=True, stream=s)
                got_grads[i].append(F.fp8_gated_grad_quant(da, r[2], r[3], stream=s))
            else:
                with t.cuda.stream(s):
                    r = F.fp8_block_gemm_gated_quant_1x128(*xs[i], *b.up8, checkpoint=True)
                    got_grads[i].append(F.fp8_gated_grad_quant(da, r[2], r[3]))
            got[i].append(r)
    t.cuda.synchronize()
    for i in range(2):
        for r, d in zip(got[i], got_grads[i]):
            assert all(t.equal(a, w) for a, w in zip(r, want[i]))
            assert all(t.equal(a, w) for a, w in zip(d, grads[i]))
