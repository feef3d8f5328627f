"""moe_residual_norm and its gradients on the GPU against the fp64 oracle.

Bounds, per value. A result is rounded once to its type: half a step,
eps(type) / 2 of its size. Before that everything is fp32: each product or sum
is off by 2^-24 of its size, and the factors r(v) by at most half of the
relative error of a sum of squares (all positive, so one unit per addition on
the way: up to 16 in a thread, 10 in the two shuffle trees) plus rsqrtf's two
units. 40 units of 2^-24 of the absolute terms that enter a value cover this;
sums over T tokens add one unit of their absolute terms per addition.
"""
import numpy as np
import pytest
import torch

import oracle.layer_oracle as lo
from mixture_experts_ffn_sigmoid_b200 import binding as B
from mixture_experts_ffn_sigmoid_b200.inputs import NormConfig

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
C = 40


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def make(T, d, dtype, gate_tokens, post=True, gate=True, pre=True, branch=True, seed=0, **kw):
    cfg = NormConfig(T=T, d=d, dtype=dtype, gate_tokens=gate_tokens, **kw)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")
    t = dict(h=(rn(T, d) * torch.exp(rn(T, 1))).to(dt), y=(rn(T, d) * torch.exp(rn(T, 1))).to(dt) if branch else None,
             w_post=(1 + 0.3 * rn(d)).to(dt) if post else None, gate=rn(cfg.n_gates, d).to(dt) if gate else None,
             w_pre=(1 + 0.3 * rn(d)).to(dt) if pre else None)
    return cfg, dt, t, (rn(T, d).to(dt) if pre else None, rn(T, d).to(dt))


def kwargs(cfg):
    return dict(gate_tokens=cfg.gate_tokens, eps=float(np.float32(cfg.eps)), alpha=float(np.float32(cfg.alpha)),
                beta=float(np.float32(cfg.beta)), w_offset=float(np.float32(cfg.w_offset)))


def within(got, want, bound, what):
    got = f64(got)
    assert np.isfinite(got).all(), what
    over = np.abs(got - want) - bound
    at = int(over.argmax())
    assert over.flat[at] <= 0, f"{what}: {got.flat[at]} for {want.flat[at]} at {np.unravel_index(at, want.shape)}, " \
                               f"allowed {bound.flat[at]:.3e}"


def forward(cfg, dt, t):
    h_out = torch.full((cfg.T, cfg.d), float("nan"), dtype=dt, device="cuda") if t["y"] is not None else None
    u = torch.full((cfg.T, cfg.d), float("nan"), dtype=dt, device="cuda") if t["w_pre"] is not None else None
    B.moe_residual_norm(cfg, t["h"], t["y"], t["w_post"], t["gate"], t["w_pre"], h_out, u)
    return h_out, u


def check_forward(cfg, dt, t, h_out, u):
    kw, e = kwargs(cfg), half_step(dt)
    a = {n: f64(v) for n, v in t.items()}
    ref, ref_u = lo.residual_norm(a["h"], a["y"], a["w_post"], a["gate"], a["w_pre"], **kw)
    size = np.abs(kw["alpha"] * a["h"]) + np.abs(ref - kw["alpha"] * a["h"]) if t["y"] is not None else np.abs(ref) * 0
    tiny = 1e-38
    if h_out is not None:
        within(h_out, ref, e * np.abs(ref) + C * U * size + tiny, "h_out")
    if u is not None:
        # The stream's own error passes through the norm: by its value, and by
        # the row's mean square (the error's norm over the row's).
        eh = C * U * size
        r = 1 / np.sqrt((ref ** 2).mean(-1, keepdims=True) + kw["eps"])
        row = np.linalg.norm(eh, axis=-1, keepdims=True) * r / np.sqrt(cfg.d)
        within(u, ref_u, e * np.abs(ref_u) + (C * U + row) * np.abs(ref_u)
               + eh * r * np.abs(a["w_pre"] + kw["w_offset"]) + tiny, "u")


def backward(cfg, dt, t, du, dh_out, h_out, ws=None, **skip):
    like = lambda v: None if v is None else torch.full_like(v, float("nan"))
    o = dict(dh=like(h_out), dy=like(t["y"]), dw_post=like(t["w_post"]), dgate=like(t["gate"]), dw_pre=like(t["w_pre"]))
    for n in skip:
        o[n] = None
    ws = B.alloc_norm_backward_workspace(cfg) if ws is None else ws
    B.moe_residual_norm_backward(cfg, h_out, t["y"], t["w_post"], t["gate"], t["w_pre"], du, dh_out, o["dh"], o["dy"],
                                 o["dw_post"], o["dgate"], o["dw_pre"], ws)
    return o


def check_backward(cfg, dt, t, du, dh_out, h_out, o):
    kw, e = kwargs(cfg), half_step(dt)
    a = {n: f64(v) for n, v in t.items()}
    H, gdu, gdh = f64(h_out), f64(du), f64(dh_out)
    ref = lo.residual_norm_backward(H, a["y"], a["w_post"], a["gate"], a["w_pre"], gdu, gdh, **kw)
    T, off, tiny = cfg.T, kw["w_offset"], 1e-38
    # Absolute terms of dH, carried on to what is computed from it.
    A = np.zeros((T, cfg.d)) if gdh is None else np.abs(gdh)
    if gdu is not None:
        r = 1 / np.sqrt((H ** 2).mean(-1, keepdims=True) + kw["eps"])
        n, q = np.abs(H * r), np.abs(gdu * (a["w_pre"] + off))
        A = A + r * (q + n * (q * n).mean(-1, keepdims=True))
        if o["dw_pre"] is not None:
            within(o["dw_pre"], ref["dw_pre"], e * np.abs(ref["dw_pre"]) + (C + T) * U * (np.abs(gdu) * n).sum(0) + tiny,
                   "dw_pre")
    scale = abs(kw["alpha"]) if t["y"] is not None else 1.0
    if o["dh"] is not None:
        within(o["dh"], ref["dh"], e * np.abs(ref["dh"]) + C * U * scale * A + tiny, "dh")
    if t["y"] is None:
        return
    G = np.abs(lo.gate_rows(a["gate"], T, cfg.gate_tokens, cfg.d)) * abs(kw["beta"])
    if t["w_post"] is None:
        ry, w = 1.0, 1.0
        Ady = G * A
        z = np.abs(a["y"])
    else:
        ry = 1 / np.sqrt((a["y"] ** 2).mean(-1, keepdims=True) + kw["eps"])
        w = np.abs(a["w_post"] + off)
        z, p = np.abs(a["y"] * ry), G * A * w
        Ady = ry * (p + z * (p * z).mean(-1, keepdims=True))
    # Twice: dH's error and then as many operations again.
    if o["dy"] is not None:
        within(o["dy"], ref["dy"], e * np.abs(ref["dy"]) + 2 * C * U * Ady + tiny, "dy")
    if o["dw_post"] is not None:
        within(o["dw_post"], ref["dw_post"], e * np.abs(ref["dw_post"]) + (2 * C + T) * U * (G * A * z).sum(0) + tiny,
               "dw_post")
    if o["dgate"] is not None:
        abs_terms = np.zeros_like(ref["dgate"])
        np.add.at(abs_terms, np.arange(T) // cfg.gate_tokens, abs(kw["beta"]) * A * z * w)
        within(o["dgate"], ref["dgate"], e * np.abs(ref["dgate"]) + (2 * C + T) * U * abs_terms + tiny, "dgate")


SHAPES = [  # T, d, dtype, gate_tokens
    (1, 8, "bf16", 1), (1, 4, "f32", 1), (2, 64, "bf16", 2), (5, 200, "bf16", 3), (33, 100, "f32", 1),
    (32, 2048, "bf16", 32), (150, 7168, "bf16", 7), (333, 1000, "f32", 37), (1200, 264, "bf16", 1200),
    (700, 8192, "bf16", 512), (301, 8200, "bf16", 100), (160, 16384, "bf16", 1), (301, 4100, "f32", 299),
    (150, 8192, "f32", 2 ** 31 - 1), (5000, 40, "bf16", 11),
]


@pytest.mark.parametrize("T,d,dtype,gt", SHAPES)
def test_forward_and_backward_on_every_shape(T, d, dtype, gt):
    cfg, dt, t, (du, dh) = make(T, d, dtype, gt, alpha=0.75, beta=1.25)
    h_out, u = forward(cfg, dt, t)
    check_forward(cfg, dt, t, h_out, u)
    check_backward(cfg, dt, t, du, dh, h_out, backward(cfg, dt, t, du, dh, h_out))


@pytest.mark.parametrize("branch,post,gate,pre,use_dh", [
    (True, False, True, True, True), (True, True, False, True, True), (True, True, True, False, True),
    (True, False, False, False, True), (True, False, False, True, False), (True, True, True, True, False),
    (False, False, False, True, True), (False, False, False, True, False)])
@pytest.mark.parametrize("dtype,d", [("bf16", 520), ("f32", 260)])
def test_forward_and_backward_with_parts_absent(branch, post, gate, pre, use_dh, dtype, d):
    cfg, dt, t, (du, dh) = make(67, d, dtype, 9, post, gate, pre, branch, alpha=-0.5, beta=2.0, w_offset=1.0)
    dh = dh if use_dh else None
    h_out, u = forward(cfg, dt, t)
    check_forward(cfg, dt, t, h_out, u)
    saved = h_out if branch else t["h"]
    check_backward(cfg, dt, t, du, dh, saved, backward(cfg, dt, t, du, dh, saved))


@pytest.mark.parametrize("skip", ["dh", "dy", "dw_post", "dgate", "dw_pre"])
def test_unwanted_gradients_are_left_out(skip):
    cfg, dt, t, (du, dh) = make(70, 256, "bf16", 16)
    h_out, _ = forward(cfg, dt, t)
    o = backward(cfg, dt, t, du, dh, h_out, **{skip: 1})
    assert o[skip] is None
    check_backward(cfg, dt, t, du, dh, h_out, o)


def test_rows_are_independent_and_rows_behind_the_last_stay():
    cfg, dt, t, _ = make(40, 512, "bf16", 1)
    h_out, u = forward(cfg, dt, t)
    poisoned = {n: None if v is None else v.clone() for n, v in t.items()}
    poisoned["h"][3], poisoned["y"][7], poisoned["y"][9] = float("nan"), float("inf"), 0.0
    big = [torch.full((44, 512), 7.0, dtype=dt, device="cuda") for _ in range(2)]
    B.moe_residual_norm(cfg, poisoned["h"], poisoned["y"], t["w_post"], t["gate"], t["w_pre"], *big)
    keep = [i for i in range(40) if i not in (3, 7, 9)]
    assert torch.equal(big[0][keep], h_out[keep]) and torch.equal(big[1][keep], u[keep])
    assert torch.isnan(big[0][3]).all() and torch.isnan(big[1][7]).all()
    assert torch.equal(big[0][9], poisoned["h"][9])      # a branch of zeros adds nothing
    assert (big[0][40:] == 7).all() and (big[1][40:] == 7).all()


def test_zero_rows_have_zero_norm_and_finite_gradients():
    cfg, dt, t, (du, dh) = make(6, 64, "f32", 2)
    t["h"][2] = 0
    t["y"][2] = 0
    h_out, u = forward(cfg, dt, t)
    assert (u[2] == 0).all()
    check_backward(cfg, dt, t, du, dh, h_out, backward(cfg, dt, t, du, dh, h_out))


@pytest.mark.parametrize("dtype,d", [("bf16", 2048), ("bf16", 8200), ("f32", 1000)])
def test_in_place_forms_give_the_same_bits(dtype, d):
    cfg, dt, t, (du, dh) = make(400, d, dtype, 64)
    h_out, u = forward(cfg, dt, t)
    h2, y2 = t["h"].clone(), t["y"].clone()
    B.moe_residual_norm(cfg, h2, y2, t["w_post"], t["gate"], t["w_pre"], h2, y2)
    assert torch.equal(h2, h_out) and torch.equal(y2, u)
    o = backward(cfg, dt, t, du, dh, h_out)
    dh2, du2, w = dh.clone(), du.clone(), {n: torch.empty_like(o[n]) for n in ("dw_post", "dgate", "dw_pre")}
    ws = B.alloc_norm_backward_workspace(cfg)
    B.moe_residual_norm_backward(cfg, h_out, t["y"], t["w_post"], t["gate"], t["w_pre"], du2, dh2, dh2, du2,
                                 w["dw_post"], w["dgate"], w["dw_pre"], ws)
    assert torch.equal(dh2, o["dh"]) and torch.equal(du2, o["dy"])
    for n, v in w.items():        # and the sums do not depend on timing
        assert torch.equal(v, o[n]), n


def test_graph_replay_and_other_streams():
    cfg, dt, t, (du, dh) = make(300, 1024, "bf16", 50)
    h_out, u = forward(cfg, dt, t)
    o = backward(cfg, dt, t, du, dh, h_out)
    ws = B.alloc_norm_backward_workspace(cfg)
    out = {n: torch.zeros_like(v) for n, v in dict(o, h_out=h_out, u=u).items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def step(stream=None):
        B.moe_residual_norm(cfg, t["h"], t["y"], t["w_post"], t["gate"], t["w_pre"], out["h_out"], out["u"], stream)
        B.moe_residual_norm_backward(cfg, out["h_out"], t["y"], t["w_post"], t["gate"], t["w_pre"], du, dh, out["dh"],
                                     out["dy"], out["dw_post"], out["dgate"], out["dw_pre"], ws, stream)

    step(side)
    side.synchronize()
    for n, v in dict(o, h_out=h_out, u=u).items():
        assert torch.equal(out[n], v), n
        out[n].zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    for n, v in dict(o, h_out=h_out, u=u).items():
        assert torch.equal(out[n], v), n


def test_no_tokens():
    cfg, dt, t, _ = make(4, 64, "bf16", 2)
    cfg = NormConfig(T=0, d=64, gate_tokens=2)
    dw = [torch.full((64,), 3.0, dtype=dt, device="cuda") for _ in range(2)]
    B.moe_residual_norm(cfg, None, t["y"], None, None, t["w_pre"], None, None)
    B.moe_residual_norm_backward(cfg, None, t["y"], t["w_post"], None, t["w_pre"], None, None, None, None, dw[0], None,
                                 dw[1], B.alloc_norm_backward_workspace(cfg))
    assert (dw[0] == 0).all() and (dw[1] == 0).all()


def test_tensors_of_another_kind_are_refused():
    cfg, dt, t, _ = make(4, 64, "bf16", 2)
    out = [torch.empty_like(t["h"]) for _ in range(2)]
    with pytest.raises(ValueError):
        B.moe_residual_norm(cfg, t["h"].t().contiguous().t(), t["y"], None, None, t["w_pre"], *out)
    with pytest.raises(ValueError):
        B.moe_residual_norm(cfg, t["h"].float(), t["y"], None, None, t["w_pre"], *out)
    with pytest.raises(B.MoEError) as e:      # one array for both results
        B.moe_residual_norm(cfg, t["h"], t["y"], None, None, t["w_pre"], out[0], out[0])
    assert e.value.status == B.MOE_ERR_INVALID_ARG
