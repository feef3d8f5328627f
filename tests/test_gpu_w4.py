"""4-bit expert weights on the GPU against the fp64 oracle.

Bounds of the expert FFN. A token row runs in fp16 under a
power of two for the row, a part of it under 1/16 besides: exact, but for values
below 2^-17 16 / 2^14 = 2^-27 of the row's largest magnitude, which are off by at
most 2^-25 16 / 2^14 = 2^-35 of that. The codes are
exact, so every product of a group is exact, and each addition is off by at
most one unit of 2^-23 (the tensor cores' adder may truncate) of the absolute
terms. A group's sum, and the zero point times its activations' sum that comes
off it, have terms of at most 15 |x| and G / 8 + 8 additions in a row; their
difference, scaled, takes at most K / 16 + 16 more over |W| |x|. SiLU's slope is below 1.1, its fp32 evaluation
good to 2^-20. The intermediate is rounded to bf16 (2^-8 of its size at most),
passes through |W2|, and the result is rounded once more.

In the 2-norm of a segment, 2^-7: each of the two roundings moves a value by at
most 2^-8 of its size. Where one entry h_j makes up the row (a segment can be a
single row of a narrow expert), y is W2's column j times h_j, and the rounding
of h_j moves all of y by up to 2^-8, the last rounding by 2^-8 more. Where many
entries share the row their errors are independent and add up to less,
2^-8 / sqrt(3) each.
"""
import numpy as np
import pytest
import torch

import gpu_harness as H
import oracle.layer_oracle as lo
import oracle.moe_oracle as orc
from mixture_experts_ffn_sigmoid_b200 import binding as B
from mixture_experts_ffn_sigmoid_b200.inputs import GATE_SIGMOID, MoEConfig, make_inputs

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


# ------------------------------------------------------------- quantisation
def quantize_rule(w, group, zeros):
    """(codes, scale, zero) by the documented rule, in IEEE fp32 on the CPU."""
    g = w.cpu().float().unflatten(-1, (-1, group))
    if zeros:
        lo_, hi = g.amin(-1, keepdim=True).clamp(max=0), g.amax(-1, keepdim=True).clamp(min=0)
        scale = ((hi - lo_) * torch.tensor(1.0 / 15.0, dtype=torch.float32)).to(BF)
        step = torch.where(scale > 0, scale.float(), 1.0)
        zero = torch.round(-lo_ / step).clamp(0, 15)
    else:
        scale = (g.abs().amax(-1, keepdim=True) * torch.tensor(1.0 / 7.0, dtype=torch.float32)).to(BF)
        step = torch.where(scale > 0, scale.float(), 1.0)
        zero = torch.full_like(step, 8.0)
    code = (torch.round(g / step) + zero).clamp(0, 15)
    return code.flatten(-2).to(torch.uint8), scale.squeeze(-1), zero.squeeze(-1).to(torch.uint8)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("rows,groups", [(1, 1), (3, 5), (257, 3), (1000, 13)])
def test_quantize_and_back(group, zeros, dtype, rows, groups):
    K = group * groups
    g = torch.Generator(device="cuda").manual_seed(rows + group)
    w = (torch.randn(rows, K, generator=g, device="cuda") * 0.1 + (0.05 if zeros else 0.0)).to(dtype)
    w[0, :group] = 0.0                                   # a group of zeros
    if rows > 2:
        w[1] = w[1].abs() + 0.01                         # one sign only
        w[2] *= 1e-30
    m = B.W4Matrix.quantize(w, group, zeros)
    code, scale, zero = quantize_rule(w, group, zeros)
    q = m.q.cpu()
    assert torch.equal(torch.stack([q & 15, q >> 4], -1).flatten(-2), code)
    assert torch.equal(m.scale.cpu(), scale)
    if zeros:
        assert torch.equal(m.zero.cpu(), zero)
    for out in (torch.float32, BF):
        back = torch.full((rows, K), float("nan"), device="cuda", dtype=out)
        B.moe_w4_dequantize(m, back)
        want = lo.w4_dense(m.q.cpu().numpy(), f64(m.scale), m.zero.cpu().numpy() if zeros else None, group)
        assert torch.equal(back.cpu(), torch.from_numpy(want).to(out))   # exact products, rounded once
    # Half a step of the scale, and what the scale's own rounding (2^-8) can
    # push past the last code: 2^-8 of 7 or 15 steps; the zero point's rounding
    # moves the ends of the range by another half step.
    err = np.abs(want - f64(w)) / np.maximum(np.repeat(f64(m.scale), group, -1), 1e-38)
    err[2:3] = 0 if rows > 2 else err[2:3]               # 1e-31 scales: bf16 subnormals hold few bits
    assert err[:, :].max() <= (0.5 + 0.5 + 15 / 256 if zeros else 0.5 + 7 / 256) + 1e-5


def test_quantize_marks_groups_that_are_not_finite():
    w = torch.ones(4, 128, device="cuda")
    w[1, 5], w[2, 70] = float("nan"), float("inf")
    m = B.W4Matrix.quantize(w, 64, False)
    assert torch.isnan(m.scale[1, 0]) and torch.isnan(m.scale[2, 1])
    assert torch.isfinite(m.scale.float()).sum() == 6


# ------------------------------------------------------------------ experts
def random_w4(g, *shape, group, zeros):
    *lead, K = shape
    q = torch.randint(0, 256, (*lead, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = ((0.5 + torch.rand(*lead, K // group, generator=g, device="cuda")) / (4.6 * K ** 0.5)).to(BF)
    z = torch.randint(0, 16, (*lead, K // group), generator=g, device="cuda", dtype=torch.uint8) if zeros else None
    return B.W4Matrix(q, s, z, group)


def dense(m, e=None):
    pick = (lambda t: None if t is None else t.cpu().numpy()) if e is None else \
        (lambda t: None if t is None else t[e].cpu().numpy())
    s = f64(m.scale if e is None else m.scale[e])
    return lo.w4_dense(pick(m.q), s, pick(m.zero), m.group)


def make(T, d, E, k, f, fs, group, zeros, seed=0, skew=0.0):
    cfg = MoEConfig("w4", T=T, d=d, E=E, k=k, f=f, f_shared=fs)
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, d, generator=g, device="cuda").to(BF)
    w = [random_w4(g, *s, group=group, zeros=zeros) for s in ((E, f, d), (E, f, d), (E, d, f))]
    ws = [random_w4(g, *s, group=group, zeros=zeros) for s in ((fs, d), (fs, d), (d, fs))] if fs else [None] * 3
    score = torch.rand(T, E, generator=g, device="cuda") - skew * torch.arange(E, device="cuda")
    flat = score.topk(k, dim=1).indices.sort(dim=1).values.reshape(-1)
    perm_src = (torch.argsort(flat, stable=True) // k).to(torch.int32)
    counts = torch.bincount(flat, minlength=E)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    return cfg, x, w, ws, perm_src, offsets


def scales(m, e=None):
    """The scale of every weight."""
    return np.repeat(f64(m.scale if e is None else m.scale[e]), m.group, axis=-1)


def check_rows(got, x, w1, w3, w2, what, s1, s3, s2, group):
    y, a, b, h = lo.swiglu_rows(x, w1, w3, w2)
    units = lambda K: (K / 16 + 16) * 2.0 ** -23
    K, f = x.shape[1], h.shape[1]
    in_group = (group / 8 + 8) * 2.0 ** -23 * 2 * 15
    split = lambda v, w: 2.0 ** -35 * np.abs(v).max(-1, keepdims=True) * np.abs(w).sum(-1)
    ea, eb = (units(K) * (np.abs(x) @ np.abs(w).T) + in_group * (np.abs(x) @ s.T) + split(x, w)
              for w, s in ((w1, s1), (w3, s3)))
    eh = 1.1 * ea * (np.abs(b) + eb) + np.abs(h) / np.maximum(np.abs(b), 1e-300) * eb + (2.0 ** -8 + 2.0 ** -20) * np.abs(h)
    ey = eh @ np.abs(w2).T + units(f) * (np.abs(h) @ np.abs(w2).T) + in_group * (np.abs(h) @ s2.T) + split(h, w2) + 2.0 ** -8 * np.abs(y) + 1e-38
    got = f64(got)
    assert np.isfinite(got).all(), what
    assert (np.abs(got - y) <= ey).all(), (what, (np.abs(got - y) - ey).max())
    rel = np.linalg.norm(got - y) / np.linalg.norm(y)
    assert rel <= 2.0 ** -7, (what, rel)


def run_experts(cfg, x, w, ws, perm_src, offsets, packed=False, workspace=None, stream=None):
    R = cfg.T * cfg.k
    y = torch.full((R, cfg.d), float("nan"), device="cuda", dtype=BF)
    ys = torch.full((cfg.T, cfg.d), float("nan"), device="cuda", dtype=BF) if cfg.f_shared else None
    wk = B.alloc_workspace(cfg) if workspace is None else workspace
    rows = x[perm_src.long()].contiguous() if packed else x
    B.moe_expert_swiglu_w4(cfg, rows, None if packed else perm_src, offsets, *w, x if cfg.f_shared else None, *ws, y, ys,
                           wk, stream)
    assert B.moe_get_device_error(wk, stream) == B.MOE_OK
    return y, ys


def check_experts(cfg, x, w, ws, perm_src, offsets, y, ys, experts=None):
    off, xp = offsets.tolist(), f64(x)[perm_src.cpu().numpy()]
    for e in range(cfg.E) if experts is None else experts:
        if off[e] < off[e + 1]:
            check_rows(y[off[e]:off[e + 1]], xp[off[e]:off[e + 1]], *[dense(m, e) for m in w], f"expert {e}",
                       *[scales(m, e) for m in w], w[0].group)
    if ys is not None:
        check_rows(ys, f64(x), *[dense(m) for m in ws], "shared", *[scales(m) for m in ws], w[0].group)


CASES = [  # T, d, E, k, f, f_shared, group, zeros
    (1, 32, 1, 1, 32, 0, 32, False), (1, 128, 4, 2, 128, 128, 128, True), (2, 96, 3, 3, 160, 32, 32, True),
    (7, 416, 5, 2, 224, 0, 32, False), (8, 256, 8, 1, 384, 64, 64, False), (9, 192, 2, 1, 448, 0, 64, True),
    (17, 640, 2, 2, 256, 128, 128, False), (31, 2048, 16, 4, 768, 0, 128, False), (40, 512, 300, 8, 64, 64, 64, True),
    (33, 1152, 4, 3, 640, 384, 128, True), (100, 320, 6, 2, 96, 96, 32, False), (300, 256, 4, 2, 256, 128, 64, False),
    (5, 7168, 4, 2, 2048, 256, 128, False), (24, 4096, 3, 1, 1536, 0, 32, True),
    (11, 14336, 2, 1, 96, 0, 32, False), (3, 16384, 2, 2, 64, 64, 32, True), (64, 2048, 4, 2, 512, 0, 128, False),
]


@pytest.mark.parametrize("T,d,E,k,f,fs,group,zeros", CASES)
def test_experts(T, d, E, k, f, fs, group, zeros):
    a = make(T, d, E, k, f, fs, group, zeros)
    check_experts(*a, *run_experts(*a))


@pytest.mark.parametrize("T,d,f,fs", [(1, 2048, 32, 32), (2, 1024, 64, 0), (9, 2048, 32, 128)])
def test_the_intermediate_adds_little_to_the_result_s_rounding(T, d, f, fs):
    """A narrow expert's row can rest on one intermediate value, whose rounding
    then moves all of it: by at most fp16's half step, 2^-11 of it (bf16's would
    be 2^-8). Rounding the result leaves an rms error of 0.42 2^-8 (mantissas
    spread over a binade), so the first is at most r = 2^-3 / 0.42 = 0.30 of it.
    Over d >= 1024 values the two errors' correlation c is within 4 / sqrt(d) =
    0.125 (four sigma): together sqrt(1 + r^2 + 2 r c) = 1.08 at most; fp32's
    2^-15 disappears beside that."""
    cfg, x, w, ws, perm_src, offsets = make(T, d, 4, 2, f, fs, 32, True, seed=11)
    y, ys = run_experts(cfg, x, w, ws, perm_src, offsets)
    off, xp = offsets.tolist(), f64(x)[perm_src.cpu().numpy()]
    for e in range(4):
        if off[e] < off[e + 1]:
            want = lo.swiglu_rows(xp[off[e]:off[e + 1]], *[dense(m, e) for m in w])[0]
            got = f64(y[off[e]:off[e + 1]])
            once = f64(torch.from_numpy(want).to(BF))
            for i in range(len(want)):
                assert np.linalg.norm(got[i] - want[i]) <= 1.08 * np.linalg.norm(once[i] - want[i])


@pytest.mark.parametrize("T,skew", [(20, 1.0), (70, 1.0)])
def test_experts_on_skewed_routing_and_packed_rows(T, skew):
    # Every token takes experts 0 and 1, the others have no rows.
    a = make(T, 384, 12, 2, 256, 128, 128, True, seed=4, skew=skew)
    y, ys = run_experts(*a)
    check_experts(*a, y, ys)
    y2, ys2 = run_experts(*a, packed=True)
    assert torch.equal(y, y2) and torch.equal(ys, ys2)


def test_rows_behind_the_last_segment_stay_and_infinities_stay_in_their_row():
    cfg, x, w, ws, perm_src, offsets = make(12, 256, 4, 2, 128, 0, 64, False, seed=2)
    y, _ = run_experts(cfg, x, w, ws, perm_src, offsets)
    short = offsets.clone()
    short[-1] = short[-2] = min(int(offsets[-2]), 20)
    out = torch.full((30, 256), 5.0, device="cuda", dtype=BF)
    xi = x.clone()
    xi[3, 7], xi[4, 9] = float("inf"), float("nan")
    wk = B.alloc_workspace(cfg)
    B.moe_expert_swiglu_w4(cfg, xi, perm_src, short, *w, None, *ws, out, None, wk)
    n = int(short[-1])
    assert (out[n:] == 5).all()
    clean = (perm_src[:n] != 3) & (perm_src[:n] != 4)
    assert torch.equal(out[:n][clean], y[:n][clean])
    assert not torch.isfinite(out[:n][~clean].float()).all(dim=1).any()


@pytest.mark.parametrize("scale", [1e-38, 1e-30, 3e-3, 1.0, 1e3, 1e28])
def test_rows_of_any_magnitude(scale):
    # Row by row another size, one row of zeros, one of a single large value;
    # the largest stay where the products themselves are finite.
    cfg, x, w, ws, perm_src, offsets = make(10, 512, 4, 2, 128, 0, 64, True, seed=7)
    rows = torch.tensor([1, 2, 4, 0.5, 1e-2, 0, 1, 1, 30, 1e-4], device="cuda")[:, None]
    xs = (x.float() * rows * scale)
    xs[6] = 0
    xs[6, 100] = scale
    xs = xs.to(BF)
    xp, off = xs[perm_src.long()], offsets.tolist()
    wk = B.alloc_workspace(cfg)
    # h grows with the square of x: only the pre-activations' scale is kept
    # apart here, by weights w3 whose scale undoes it.
    w3 = B.W4Matrix(w[1].q, (w[1].scale.float() / scale).to(BF) if scale in (1e3, 1e28) else w[1].scale, w[1].zero, 64)
    ww = [w[0], w3, w[2]]
    y = torch.full((20, 512), float("nan"), device="cuda", dtype=BF)
    B.moe_expert_swiglu_w4(cfg, xs, perm_src, offsets, *ww, None, *ws, y, None, wk)
    for e in range(4):
        if off[e] < off[e + 1]:
            with np.errstate(over="ignore"):
                want, a, b, h = lo.swiglu_rows(f64(xp[off[e]:off[e + 1]]), *[dense(m, e) for m in ww])
            got = f64(y[off[e]:off[e + 1]])
            assert np.isfinite(got).all()
            # Relative to each row's largest result: two roundings to bf16 (as
            # above), the split and SiLU's fp32 evaluation stay below 2^-6 of
            # it; below 1e-37 bf16 and fp32 have subnormal numbers only.
            room = 2.0 ** -6 * np.abs(want).max(-1, keepdims=True) + 1e-37
            assert (np.abs(got - want) <= room).all(), e


def test_bad_tables_are_reported():
    cfg, x, w, ws, perm_src, offsets = make(6, 128, 4, 2, 128, 0, 64, False)
    wk, y = B.alloc_workspace(cfg), torch.zeros(12, 128, device="cuda", dtype=BF)
    bad_rows, bad_off = perm_src.clone(), offsets.clone()
    bad_rows[3] = 6
    bad_off[2] = 10 ** 6
    for p, o in ((bad_rows, offsets), (perm_src, bad_off), (perm_src - 5, offsets)):
        B.moe_expert_swiglu_w4(cfg, x, p, o, *w, None, *ws, y, None, wk)
        assert B.moe_get_device_error(wk) == B.MOE_ERR_INVALID_ARG
    B.moe_expert_swiglu_w4(cfg, x, perm_src, offsets, *w, None, *ws, y, None, wk)
    assert B.moe_get_device_error(wk) == B.MOE_OK       # a good call writes the word anew


def test_graph_replay_and_two_streams():
    a, b = make(16, 512, 8, 2, 256, 128, 64, True), make(3, 1024, 16, 4, 384, 0, 128, False, seed=9)
    want = [run_experts(*v) for v in (a, b)]
    side = [torch.cuda.Stream() for _ in range(2)]
    wss = [B.alloc_workspace(v[0]) for v in (a, b)]
    torch.cuda.synchronize()
    for _ in range(3):
        got = [run_experts(*v, workspace=w, stream=s) for v, w, s in zip((a, b), wss, side)]
    torch.cuda.synchronize()
    for (y, ys), (y0, ys0) in zip(got, want):
        assert torch.equal(y, y0) and (ys is None or torch.equal(ys, ys0))
    cfg, x, w, ws, perm_src, offsets = a
    y, ys = torch.zeros(32, 512, device="cuda", dtype=BF), torch.zeros(16, 512, device="cuda", dtype=BF)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.moe_expert_swiglu_w4(cfg, x, perm_src, offsets, *w, x, *ws, y, ys, wss[0])
    for _ in range(5):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want[0][0]) and torch.equal(ys, want[0][1])


# -------------------------------------------------------------- whole block
@pytest.mark.parametrize("T,E", [(1, 16), (32, 16), (150, 16), (24, 288)])
def test_block_on_quantised_weights(T, E):
    cfg = MoEConfig("w4 block", T=T, d=512, E=E, k=4, f=256, gate_mode=GATE_SIGMOID, n_groups=4, topk_groups=2,
                    route_scale=2.5, f_shared=128, bias="uniform")
    inp = make_inputs(cfg, "cuda", seed=1)
    q = {n: B.W4Matrix.quantize(inp[n], 64, zero_points=n in ("w3", "ws1")) for n in ("w1", "w3", "w2", "ws1", "ws3", "ws2")}
    block = B.MoEBlock(cfg, {**inp, **q}, "cuda")
    y = block.forward(inp["x"])
    assert B.moe_get_device_error(block.workspace(T)) == B.MOE_OK
    ref = H.oracle_route(cfg, inp)
    ok = ~orc.near_tie_tokens(ref, cfg.k, cfg.n_groups, cfg.topk_groups, H.NEAR_TIE_EPS)
    d = {n: dense(m) for n, m in q.items()}
    want = orc.expert_outputs(f64(inp["x"]), ref["idx"], ref["gates"], d["w1"], d["w3"], d["w2"], d["ws1"], d["ws3"],
                              d["ws2"])
    H.compare_outputs(cfg, f64(y)[ok], want[ok])


def test_no_tokens():
    cfg, x, w, ws, perm_src, offsets = make(4, 128, 4, 2, 128, 0, 64, False)
    c = B.make_config(cfg, T=0)
    B.moe_expert_swiglu_w4(c, None, None, offsets, *w, None, *ws, None, None, B.alloc_workspace(cfg))
    m = B.W4Matrix.quantize(torch.empty(0, 128, device="cuda"), 64)
    B.moe_w4_dequantize(m, torch.empty(0, 128, device="cuda"))
