"""The operators around the block together, as a model uses them: a layer
served on 4-bit weights, and a training step from norm to weight update.

Training in fp32, end to end against the fp64 oracles chained the same way.
Each part alone is held to a relative L2 error of 1e-5 (block and backward) or
less (norms); a chain passes the error of one part through the next ones, six
of them with factors of order one: 1e-4. Serving in bf16 compares every part
with its oracle on the part's own inputs, within that part's bounds.
"""
import numpy as np
import pytest
import torch

import gpu_harness as H
import oracle.layer_oracle as lo
import oracle.moe_oracle as orc
from mixture_experts_ffn_sigmoid_b200 import binding as B
from mixture_experts_ffn_sigmoid_b200.inputs import GATE_SIGMOID, MoEConfig, NormConfig, OrthoConfig, make_inputs

pytestmark = pytest.mark.gpu
f64 = H.f64


def near(got, want, tol, what):
    got = f64(got)
    assert np.isfinite(got).all(), what
    rel = np.linalg.norm(got - want) / np.linalg.norm(want)
    assert rel <= tol, (what, rel)


@pytest.mark.parametrize("f_shared", [0, 40])
def test_training_step(f_shared):
    cfg = MoEConfig("layer", T=77, d=200, E=12, k=3, f=72, dtype="f32", gate_mode=GATE_SIGMOID, route_scale=1.5,
                    f_shared=f_shared, bias="uniform")
    T, d = cfg.T, cfg.d
    inp = make_inputs(cfg, "cuda", seed=2)
    g = torch.Generator(device="cuda").manual_seed(8)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")
    n0 = NormConfig(T=T, d=d, dtype="f32")
    n1 = NormConfig(T=T, d=d, dtype="f32", gate_tokens=16, alpha=0.9, beta=0.7)
    h0, w0, wp, wn, gate = rn(T, d), 1 + 0.2 * rn(d), 1 + 0.2 * rn(d), 1 + 0.2 * rn(d), rn(n1.n_gates, d)
    dh1, du1 = rn(T, d), rn(T, d)
    new = lambda t: torch.empty_like(t)

    # Forward: norm, block, residual norm.
    u0, y, h1, u1 = (new(h0) for _ in range(4))
    B.moe_residual_norm(n0, h0, None, None, None, w0, None, u0)
    ws = B.alloc_backward_workspace(cfg)
    B.moe_forward_train(cfg, u0, inp["w_router"], inp["bias"], inp["w1"], inp["w3"], inp["w2"], inp["ws1"], inp["ws3"],
                        inp["ws2"], y, ws)
    B.moe_residual_norm(n1, h0, y, wp, gate, wn, h1, u1)
    # Backward.
    dh, dy, dwp, dg, dwn = new(h0), new(h0), new(wp), new(gate), new(wn)
    B.moe_residual_norm_backward(n1, h1, y, wp, gate, wn, du1, dh1, dh, dy, dwp, dg, dwn,
                                 B.alloc_norm_backward_workspace(n1))
    du0, dr = new(h0), new(inp["w_router"])
    d1, d3, d2 = new(inp["w1"]), new(inp["w3"]), new(inp["w2"])
    s1, s3, s2 = (new(inp[n]) if f_shared else None for n in ("ws1", "ws3", "ws2"))
    B.moe_backward_saved(cfg, u0, inp["w_router"], inp["w1"], inp["w3"], inp["w2"], inp["ws1"], inp["ws3"], inp["ws2"],
                         dy, du0, dr, d1, d3, d2, s1, s3, s2, ws)
    assert B.moe_get_device_error(ws) == B.MOE_OK
    dh0, dw0 = new(h0), new(w0)
    B.moe_residual_norm_backward(n0, h0, None, None, None, w0, du0, dh, dh0, None, None, None, dw0,
                                 B.alloc_norm_backward_workspace(n0))

    # The same in fp64, for the GPU's choice of experts.
    idx = H.gpu_route(cfg, dict(inp, x=u0))["idx"].cpu().numpy()
    a = {n: f64(v) for n, v in dict(inp, h0=h0, w0=w0, wp=wp, wn=wn, gate=gate, dh1=dh1, du1=du1).items()}
    k1 = dict(gate_tokens=16, eps=float(np.float32(1e-6)), alpha=float(np.float32(0.9)), beta=float(np.float32(0.7)))
    k0 = dict(eps=k1["eps"])
    _, U0 = lo.residual_norm(a["h0"], None, None, None, a["w0"], **k0)
    r = orc.route(U0, a["w_router"], a["bias"], cfg.k, cfg.gate_mode, 1, 1, cfg.route_scale)
    gates = orc.gate_values(r["logits"], r["scores"], idx.astype(np.int64), cfg.gate_mode, cfg.route_scale)
    Y = orc.expert_outputs(U0, idx, gates, a["w1"], a["w3"], a["w2"], a["ws1"], a["ws3"], a["ws2"])
    H1, U1 = lo.residual_norm(a["h0"], Y, a["wp"], a["gate"], a["wn"], **k1)
    for got, want, what in ((u0, U0, "u0"), (y, Y, "y"), (h1, H1, "h1"), (u1, U1, "u1")):
        near(got, want, 1e-4, what)
    gn = lo.residual_norm_backward(H1, Y, a["wp"], a["gate"], a["wn"], a["du1"], a["dh1"], **k1)
    gb = orc.moe_backward(U0, a["w_router"], a["bias"], a["w1"], a["w3"], a["w2"], cfg.k, cfg.gate_mode, gn["dy"], 1, 1,
                          cfg.route_scale, a["ws1"], a["ws3"], a["ws2"], idx=idx)
    g0 = lo.residual_norm_backward(a["h0"], None, None, None, a["w0"], gb["dx"], gn["dh"], **k0)
    for got, want, what in ((dwp, gn["dw_post"], "dw_post"), (dg, gn["dgate"], "dgate"), (dwn, gn["dw_pre"], "dw_pre"),
                            (du0, gb["dx"], "dx"), (dr, gb["dw_router"], "dw_router"), (d1, gb["dw1"], "dw1"),
                            (d3, gb["dw3"], "dw3"), (d2, gb["dw2"], "dw2"), (dh0, g0["dh"], "dh0"),
                            (dw0, g0["dw_pre"], "dw0")):
        near(got, want, 1e-4, what)

    # The expert matrices' update by Muon: an expert no token chose stays but for decay.
    oc = OrthoConfig(n=cfg.E, rows=cfg.f, cols=d, dtype="f32")
    mom, w1 = torch.zeros_like(inp["w1"]), inp["w1"].clone()
    wo = B.alloc_ortho_workspace(oc)
    B.moe_muon_step(oc, d1, mom, w1, wo, lr=0.1, mu=0.95, nesterov=True, weight_decay=0.1)
    assert B.moe_get_device_error(wo) == B.MOE_OK
    assert torch.equal(mom, d1)
    per = [tuple(float(np.float32(v)) for v in lo.MUON_COEFFS)] * 5
    for e in range(cfg.E):
        u = 1.95 * f64(d1[e])
        x = lo.newton_schulz(u, per) if np.abs(u).max() > 0 else np.zeros_like(u)
        # 2 e0 of the fp16 products (a few 1e-3 of X's norm) times the step
        e0 = np.linalg.norm(lo.newton_schulz(u, per, stored=lo.half_64) - x)
        want = (1 - 0.01) * a["w1"][e] - 0.1 * x
        assert np.linalg.norm(f64(w1[e]) - want) <= 0.1 * 2 * e0 + 1e-6 * np.linalg.norm(want)


@pytest.mark.parametrize("T", [1, 24, 200])
@pytest.mark.parametrize("in_place", [False, True])
def test_serving_layer_on_4_bit_weights(T, in_place):
    cfg = MoEConfig("layer w4", T=T, d=512, E=16, k=4, f=256, f_shared=128, bias="uniform", gate_mode=GATE_SIGMOID,
                    route_scale=2.5)
    inp = make_inputs(cfg, "cuda", seed=5)
    q = {n: B.W4Matrix.quantize(inp[n], 64) for n in ("w1", "w3", "w2", "ws1", "ws3", "ws2")}
    block = B.MoEBlock(cfg, {**inp, **q}, "cuda")
    g = torch.Generator(device="cuda").manual_seed(3)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)
    h, wp, wn, gate = inp["x"], (1 + 0.2 * rn(512)), (1 + 0.2 * rn(512)), rn(1, 512)
    norm = NormConfig(T=T, d=512, gate_tokens=T, alpha=1.0, beta=0.5)
    u = torch.empty_like(h)
    B.moe_residual_norm(norm, h, None, None, None, wn, None, u)
    y = block.forward(u)
    h0, u0 = h.clone(), u.clone()
    h1, u1 = block.step(h, u, norm, wp, gate, wn, *((h, u) if in_place else ()))
    assert (h1 is h) == in_place and (in_place or (torch.equal(h, h0) and torch.equal(u, u0)))
    kw = dict(gate_tokens=T, eps=float(np.float32(1e-6)), alpha=1.0, beta=0.5)
    _, U = lo.residual_norm(f64(h0), None, None, None, f64(wn), **kw)
    near(u0, U, 2.0 ** -8, "u")
    H1, U1 = lo.residual_norm(f64(h0), f64(y), f64(wp), f64(gate), f64(wn), **kw)
    near(h1, H1, 2.0 ** -8, "h1")          # one rounding to bf16: 2^-8 of a value at most
    near(u1, U1, 2.0 ** -8, "u1")
    # The block itself, on the input that the norm gave it.
    dense = {n: lo.w4_dense(m.q.cpu().numpy(), f64(m.scale), None, 64) for n, m in q.items()}
    ref = orc.route(f64(u0), f64(inp["w_router"]), f64(inp["bias"]), cfg.k, cfg.gate_mode, 1, 1, cfg.route_scale)
    ok = ~orc.near_tie_tokens(ref, cfg.k, 1, 1, H.NEAR_TIE_EPS)
    want = orc.expert_outputs(f64(u0), ref["idx"], ref["gates"], dense["w1"], dense["w3"], dense["w2"], dense["ws1"],
                              dense["ws3"], dense["ws2"])
    H.compare_outputs(cfg, f64(y)[ok], want[ok])
