"""The norms' gradients at the ends of the range that moe_residual_norm takes:
rows whose squares come near fp32's largest number, rows of zeros under an eps
near its smallest.

The bounds are those of test_gpu_norm: they are relative to the terms that enter
each value, and no term here leaves fp32's normal numbers. Sums of squares stay
below 3e38 (16384 values of 1e17), factors r between 1e-17 and 1e18, and what
is taken off, n mean(q n), has the size of q.
"""
import pytest
import torch

import test_gpu_norm as N

pytestmark = pytest.mark.gpu

SHAPES = [(40, 64, "f32"), (40, 64, "bf16"), (40, 2048, "bf16"), (24, 8200, "bf16"), (24, 16384, "bf16"),
          (24, 4100, "f32")]


@pytest.mark.parametrize("where", ["stream", "branch", "both"])
@pytest.mark.parametrize("T,d,dtype", SHAPES)
def test_rows_of_large_values(T, d, dtype, where):
    # The gradient through the stream is left out: beside it the norm's own,
    # 1 / rms in size, would not show.
    cfg, dt, t, (du, _) = N.make(T, d, dtype, 7, alpha=0.75, beta=1.25, seed=3)
    size = torch.tensor([1.0, 1e13, 1e14, 1e15, 1e16, 5e16], device="cuda").repeat(T)[:T, None]
    unit = lambda v: v.float() / v.float().square().mean(1, keepdim=True).sqrt()
    if where != "branch":
        t["h"] = (unit(t["h"]) * size).to(dt)
    if where != "stream":
        t["y"] = (unit(t["y"]) * size).to(dt)
    h_out, u = N.forward(cfg, dt, t)
    N.check_forward(cfg, dt, t, h_out, u)
    N.check_backward(cfg, dt, t, du, None, h_out, N.backward(cfg, dt, t, du, None, h_out))


@pytest.mark.parametrize("eps", [1e-12, 1e-27, 1e-30, 1e-36])
@pytest.mark.parametrize("T,d,dtype", SHAPES)
def test_zero_and_small_rows_under_a_small_eps(T, d, dtype, eps):
    cfg, dt, t, (du, dh) = N.make(T, d, dtype, 3, eps=eps, seed=5)
    t["h"][2], t["y"][2] = 0, 0                # both norms of zeros
    t["y"][6] = 0                              # the branch's alone
    t["h"][9], t["y"][9] = t["h"][9] * 1e-15, 0
    t["y"][13] *= 1e-15
    h_out, u = N.forward(cfg, dt, t)
    assert (h_out[2] == 0).all() and (u[2] == 0).all()
    N.check_forward(cfg, dt, t, h_out, u)
    N.check_backward(cfg, dt, t, du, dh, h_out, N.backward(cfg, dt, t, du, dh, h_out))
