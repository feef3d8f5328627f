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


@pytest.fixture
def freed():
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("T,gt", [(2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31 - 1, 2 ** 30 + 5), (2 ** 30 + 77, 2 ** 30 + 76)])
def test_as_many_tokens_as_an_int_counts(T, gt, freed):
    """The first and last tokens, those around the gate rows' border and those
    around a run's; every other gradient is zero, so that the sums are of a few
    terms each and the bounds those of a small batch."""
    d = 8
    g = torch.Generator(device="cuda").manual_seed(1)
    at = sorted({0, 1, 518217, 518218, T // 2, gt - 1, min(gt, T - 1), T - 4, T - 2, T - 1})
    gates = -(-T // gt)
    cfg, small = N.NormConfig(T=T, d=d, gate_tokens=gt), N.NormConfig(T=len(at), d=d, gate_tokens=1)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)
    hs, ys, dus, gate, wp, wn = rn(len(at), d), rn(len(at), d), rn(len(at), d), rn(gates, d), 1 + 0.2 * rn(d), 1 + 0.2 * rn(d)
    rows = torch.tensor(at, device="cuda")
    h, y = torch.zeros(T, d, device="cuda", dtype=torch.bfloat16), torch.zeros(T, d, device="cuda", dtype=torch.bfloat16)
    h[rows], y[rows] = hs, ys
    # A gate row a token, repeated, in place of rows shared by 2^30 tokens.
    rep = gate[rows // gt].contiguous()
    t = dict(h=hs, y=ys, w_post=wp, gate=rep, w_pre=wn)
    h1, u1 = N.forward(small, torch.bfloat16, t)
    want = N.backward(small, torch.bfloat16, t, dus, None, h1)
    B = N.B
    B.moe_residual_norm(cfg, h, y, wp, gate, wn, h, y)                  # in place: u over y
    assert torch.equal(h[rows], h1) and torch.equal(y[rows], u1)
    y.zero_()
    y[rows] = ys
    du = torch.zeros(T, d, device="cuda", dtype=torch.bfloat16)
    du[rows] = dus
    dwp, dg, dwn = torch.empty_like(wp), torch.empty_like(gate), torch.empty_like(wn)
    B.moe_residual_norm_backward(cfg, h, y, wp, gate, wn, du, None, None, du, dwp, dg, dwn,
                                 B.alloc_norm_backward_workspace(cfg))
    assert torch.equal(du[rows], want["dy"])                            # a row by itself
    # Each sum once more in its run's order: 10 terms, and the rounding to bf16.
    near = lambda a, b: (a.double() - b.double()).abs() <= 2 ** -8 * (a.double().abs() + b.double().abs()) + 1e-30
    assert near(dwp, want["dw_post"]).all() and near(dwn, want["dw_pre"]).all()
    by_gate = torch.zeros(gates, d, device="cuda", dtype=torch.float64).index_add_(0, rows // gt, want["dgate"].double())
    room = torch.zeros(gates, d, device="cuda", dtype=torch.float64).index_add_(0, rows // gt, want["dgate"].double().abs())
    # Each token's part was rounded to bf16 above, and the sum is here, off by 2^-8 of what it came to.
    assert ((dg.double() - by_gate).abs() <= 2 ** -8 * (room + by_gate.abs() + 2 ** -8 * room) + 1e-30).all()


@pytest.mark.parametrize("d,dtype", [(64, "f32"), (2048, "bf16"), (8200, "bf16"), (16384, "bf16")])
def test_a_branch_without_a_norm_passes_its_gradient_whatever_its_values(d, dtype):
    # dy = beta gate dh' then: no value of y enters it, nor dh.
    cfg, dt, t, (_, dh) = N.make(12, d, dtype, 3, post=False, pre=False, alpha=0.5, beta=2.0)
    h_out, _ = N.forward(cfg, dt, t)
    o = N.backward(cfg, dt, t, None, dh, h_out, dgate=1)
    N.check_backward(cfg, dt, t, None, dh, h_out, o)
    y = t["y"].clone()
    y[2, 5], y[7, 0], y[9] = float("inf"), float("nan"), -float("inf")
    o2 = N.backward(cfg, dt, dict(t, y=y), None, dh, h_out, dgate=1)
    assert torch.equal(o2["dy"], o["dy"]) and torch.equal(o2["dh"], o["dh"])
