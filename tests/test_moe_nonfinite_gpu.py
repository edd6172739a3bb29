"""Infinities and NaN in the operators around the expert products, on the GPU:
they show where the formulas have them and nowhere else.

A call on clean operands stands beside each: what a non-finite value must not
reach has to be equal to it bit for bit.
"""
import numpy as np
import pytest

from fp8_fine_grained_token_amd import binding as B
from fp8_fine_grained_token_amd import moe as M

from .gpu_util import e4m3_lut, host, torch

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    t = torch()
    if not t.cuda.is_available():
        pytest.skip("no GPU")
    B.lib()
    yield
    t.cuda.synchronize()


def draw(seed, shape, dtype="bf16", sigma=1.0, mean=0.0):
    t = torch()
    v = np.random.default_rng(seed).standard_normal(shape, dtype=np.float32) * np.float32(sigma)
    return t.from_numpy(v + np.float32(mean)).to(
        t.bfloat16 if dtype == "bf16" else t.float32).cuda()


def cuda(a):
    return torch().from_numpy(np.ascontiguousarray(a)).cuda()


@pytest.mark.parametrize("bad", [INF, -INF])
@pytest.mark.parametrize("H", [300, 1001, 9003, 17001])
def test_infinite_parameter_is_counted_once(H, bad):
    # in the columns that a row's last vector shares with the one before it:
    # the new stream is infinite there, so its reciprocal root is 0 (not NaN)
    # and the finite columns of n are 0
    t = torch()
    T, at = 3, H - 6
    y, r = draw(1, (T, H), "f32", mean=4.0), draw(2, (T, H), "f32")
    for gate, w_post in ((True, False), (False, True)):
        p = draw(3, (H,), "f32", 0.1, 1.0)
        p[at] = bad
        r_out, n, _, rstd = M.fp8_norm_residual(y, r, p if w_post else None, p if gate else None)
        assert t.equal(rstd, t.zeros_like(rstd))
        assert r_out[:, at].isinf().all() and n[:, at].isnan().all()
        r_out[:, at] = n[:, at] = 0
        assert r_out.isfinite().all() and not n.any()


@pytest.mark.parametrize("bad", [INF, NAN])
@pytest.mark.parametrize("H", [5, 300, 2500, 9000])
def test_gradient_without_post_norm_is_blind_to_y(H, bad):
    # y enters only the gate's gradient, in its own column
    t = torch()
    T = 6
    y, dn = draw(1, (T, H)), draw(2, (T, H))
    r_out, dr_out = draw(3, (T, H), "f32"), draw(4, (T, H), "f32")
    gate, w = draw(5, (H,), "f32", 0.3, 1.0), draw(6, (H,), "f32", 0.1, 1.0)
    rstd = 1 / r_out.square().mean(1).sqrt()

    def grad(dn, dr_out):
        return M.fp8_norm_residual_grad(dn, dr_out, y, r_out, None, rstd, None, gate, w,
                                        post_norm=False, branch_scale=0.7)

    for which in ((dn, dr_out), (None, dr_out), (dn, None)):
        y[2, H // 2] = 1.0
        clean = grad(*which)
        y[2, H // 2] = bad
        got = grad(*which)
        for name, a, b in zip(("dy", "dr", "dw_post", "dgate", "dw_pre"), got, clean):
            if name == "dgate":
                assert not a[H // 2].isfinite()
                a[H // 2] = b[H // 2]
            assert (a is None and b is None) or t.equal(a, b), name
