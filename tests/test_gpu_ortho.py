"""Newton-Schulz orthogonalisation and the Muon step on the GPU against the
fp64 oracle.

Bounds. What the kernels keep between products is rounded to fp16 (2^-11 of a
value at most), nothing else loses more than fp32 does. How far such roundings
carry depends on the spectrum: the oracle follows them in fp64 with the same
roundings at the same places (``stored=half_64``) and so gives the size e0 of
their effect for each input. The kernels' roundings are as large but fall
differently where fp32 sums differ in the last bits, so their error is another
draw of the same size: 2 e0 is allowed in the 2-norm. For matrices of fewer
than 4096 entries e0 is itself a small sample; three roundings a step, each
2^-11 at most, are allowed besides. The result's bf16 rounding adds 2^-8 at
most, 2^-8 / sqrt(3) over many entries.
"""
import numpy as np
import pytest
import torch

import oracle.layer_oracle as lo
from mixture_experts_ffn_sigmoid_b200 import binding as B
from mixture_experts_ffn_sigmoid_b200.inputs import OrthoConfig

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def f64(t):
    return t.detach().cpu().double().numpy()


def gradients(n, rows, cols, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")
    return (1e-3 * (rn(n, rows, cols) * torch.exp(0.3 * rn(n, rows, 1)) + rn(n, rows, 1) * rn(n, 1, cols))) \
        .to(torch.float32 if dtype == "f32" else BF)


def allowed(u, coeffs, eps, want):
    """2-norm allowance before the result's own rounding, relative to want."""
    e0 = np.linalg.norm(lo.newton_schulz(u, coeffs, eps, lo.half_64) - want) / np.linalg.norm(want)
    return 2 * e0 + (3 * len(coeffs) * 2.0 ** -11 if want.size < 4096 else 0.0), want.size < 4096


def run(cfg, g, coeffs=None, o=None, ws=None, stream=None):
    o = torch.full((cfg.n, cfg.rows, cfg.cols), float("nan"), device="cuda", dtype=BF) if o is None else o
    ws = B.alloc_ortho_workspace(cfg) if ws is None else ws
    B.moe_orthogonalize(cfg, g, o, ws, coeffs, stream)
    assert B.moe_get_device_error(ws, stream) == B.MOE_OK
    return o


def check(cfg, g, o, coeffs=None, matrices=None):
    per = [lo.MUON_COEFFS] * cfg.steps if coeffs is None else coeffs
    per = [tuple(float(np.float32(v)) for v in t) for t in per]
    for i in range(cfg.n) if matrices is None else matrices:
        u, got = f64(g[i]), f64(o[i])
        want = lo.newton_schulz(u, per, float(np.float32(cfg.eps)))
        assert np.isfinite(got).all()
        tol, small = allowed(u, per, cfg.eps, want)
        rel = np.linalg.norm(got - want) / np.linalg.norm(want)
        assert rel <= tol + 2.0 ** -8 / (1 if small else 3 ** 0.5), (i, rel, tol)


CASES = [(1, 1, 1), (2, 1, 7), (2, 7, 1), (3, 8, 8), (1, 63, 65), (2, 65, 63), (3, 100, 300), (2, 300, 100),
         (5, 128, 128), (1, 257, 513), (1, 513, 257), (2, 256, 1024), (1, 600, 1999), (1, 1031, 520), (2, 768, 768),
         (1, 5, 3001), (2, 128, 512), (1, 512, 128), (1, 129, 512), (1, 128, 513), (1, 97, 449), (1, 8, 8)]


@pytest.mark.parametrize("n,rows,cols", CASES)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_orthogonalize(n, rows, cols, dtype):
    cfg = OrthoConfig(n=n, rows=rows, cols=cols, dtype=dtype)
    g = gradients(n, rows, cols, dtype)
    check(cfg, g, run(cfg, g))


@pytest.mark.parametrize("n,rows,cols", [(3, 1024, 1100), (8, 700, 720), (4, 640, 777), (60, 130, 140), (2, 1500, 1300)])
def test_every_way_of_tiling(n, rows, cols):
    # Squares by 128 x 128 tiles with and without mirrored ones, by pairs'
    # 256 x 256, and X's products by either.
    cfg = OrthoConfig(n=n, rows=rows, cols=cols)
    g = gradients(n, rows, cols, "bf16", seed=6)
    check(cfg, g, run(cfg, g), matrices=[0, n - 1])


def test_large_stack_in_groups():
    # 8 tiles of each of 74 pairs are one group: the stack takes two.
    cfg = OrthoConfig(n=700, rows=16, cols=24)
    g = gradients(700, 16, 24, "bf16")
    o = run(cfg, g)
    check(cfg, g, o, matrices=[0, 1, 349, 350, 351, 698, 699])
    assert torch.isfinite(o.float()).all()
    assert B.ortho_workspace_size(cfg) == B.ortho_workspace_size(OrthoConfig(n=350, rows=16, cols=24))


@pytest.mark.parametrize("rows,cols", [(9, 400), (13, 415), (300, 12), (76, 8), (15, 1433), (1723, 16)])
def test_few_rows_keep_the_diagonals(rows, cols):
    """Over few rows the roundings of B's diagonal would not average out. The
    weights of a step from zero, in fp32, are X itself; over 64 matrices its
    error is that of the same roundings in fp64 with the diagonals whole (A's
    too up to 512 columns): 64 squares of errors have a mean that is within
    1.5 of another 64's unless single ones dominate, 1.5 in the error itself."""
    n = 64
    cfg = OrthoConfig(n=n, rows=rows, cols=cols, dtype="f32")
    g = gradients(n, rows, cols, "f32", seed=9)
    w = torch.zeros(n, rows, cols, device="cuda")
    B.moe_muon_step(cfg, g, torch.zeros_like(w), w, B.alloc_ortho_workspace(cfg), lr=1.0, mu=0.0, weight_decay=0.0)
    per = [tuple(float(np.float32(v)) for v in lo.MUON_COEFFS)] * 5
    got, same = [], []
    for i in range(n):
        u = f64(g[i])
        want = lo.newton_schulz(u, per, float(np.float32(cfg.eps)))
        whole = lo.half_64_off_diagonal
        near = lo.newton_schulz(u, per, cfg.eps, lo.half_64, whole if max(rows, cols) <= 512 else None, whole)
        got.append(np.linalg.norm(-f64(w[i]) - want) / np.linalg.norm(want))
        same.append(np.linalg.norm(near - want) / np.linalg.norm(want))
    rms = lambda v: float(np.sqrt(np.mean(np.square(v))))
    assert rms(got) <= 1.5 * rms(same), (rms(got), rms(same))


@pytest.mark.parametrize("steps", [1, 2, 3, 8])
def test_steps_and_coefficients(steps):
    cfg = OrthoConfig(n=2, rows=200, cols=136, steps=steps)
    g = gradients(2, 200, 136, "bf16", seed=3)
    check(cfg, g, run(cfg, g))
    coeffs = [(1.5, -0.5, 0.0) if k % 2 else (2.0, -1.5, 0.5) for k in range(steps)]
    check(cfg, g, run(cfg, g, coeffs), coeffs)
    same = run(cfg, g, (1.5, -0.5, 0.0))
    assert torch.equal(same, run(cfg, g, [(1.5, -0.5, 0.0)] * steps))


def test_singular_values_come_near_one():
    cfg = OrthoConfig(n=1, rows=256, cols=1024, dtype="f32")
    g = torch.randn(1, 256, 1024, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    s = np.linalg.svd(f64(run(cfg, g)[0]), compute_uv=False)
    # The polynomial maps singular values of a random matrix of this shape
    # (0.03 to 0.1 after scaling to norm 1) into [0.68, 1.21] in five steps;
    # bf16 entries move one by at most 2^-8 of the norm of a row block, 0.06.
    assert s.min() > 0.6 and s.max() < 1.3


def test_zero_and_broken_matrices_stay_apart():
    cfg = OrthoConfig(n=4, rows=96, cols=160, dtype="f32")
    g = gradients(4, 96, 160, "f32")
    o = run(cfg, g)
    g2 = g.clone()
    g2[1] = 0
    g2[2, 5, 7] = float("nan")
    o2 = run(cfg, g2)
    assert torch.equal(o2[0], o[0]) and torch.equal(o2[3], o[3])
    assert (o2[1] == 0).all() and not torch.isfinite(o2[2].float()).all()


@pytest.mark.parametrize("rows,cols", [(130, 264), (264, 130), (77, 41)])
def test_result_over_the_gradients_and_rows_behind(rows, cols):
    cfg = OrthoConfig(n=3, rows=rows, cols=cols)
    g = gradients(3, rows, cols, "bf16")
    o = run(cfg, g)
    buf = torch.full((4, rows, cols), 9.0, device="cuda", dtype=BF)
    buf[:3] = g
    run(cfg, buf, o=buf)
    assert torch.equal(buf[:3], o) and (buf[3] == 9).all()


def test_graph_replay_and_streams():
    cfg, cfg2 = OrthoConfig(n=4, rows=256, cols=384), OrthoConfig(n=2, rows=500, cols=120, dtype="f32")
    g, g2 = gradients(4, 256, 384, "bf16"), gradients(2, 500, 120, "f32")
    o, o2 = run(cfg, g), run(cfg2, g2)
    side = [torch.cuda.Stream() for _ in range(2)]
    wss = [B.alloc_ortho_workspace(c) for c in (cfg, cfg2)]
    torch.cuda.synchronize()
    got = [[torch.zeros_like(o), torch.zeros_like(o2)] for _ in range(1)][0]
    for _ in range(4):
        for c, gg, out, ws, st in zip((cfg, cfg2), (g, g2), got, wss, side):
            B.moe_orthogonalize(c, gg, out, ws, None, st)
    torch.cuda.synchronize()
    assert torch.equal(got[0], o) and torch.equal(got[1], o2)
    got[0].zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.moe_orthogonalize(cfg, g, got[0], wss[0])
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], o)


# --------------------------------------------------------------------- Muon
@pytest.mark.parametrize("n,rows,cols", [(1, 3, 5), (2, 130, 264), (3, 264, 130), (2, 77, 41), (1, 41, 1027)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("wdtype", [torch.float32, BF])
@pytest.mark.parametrize("nesterov", [False, True])
def test_muon_step(n, rows, cols, dtype, wdtype, nesterov):
    cfg = OrthoConfig(n=n, rows=rows, cols=cols, dtype=dtype)
    g = gradients(n, rows, cols, dtype)
    gen = torch.Generator(device="cuda").manual_seed(5)
    mom = 2e-3 * torch.randn(n, rows, cols, generator=gen, device="cuda")
    w = (torch.randn(n, rows, cols, generator=gen, device="cuda") / cols ** 0.5).to(wdtype)
    m0, w0 = mom.clone(), w.clone()
    ws = B.alloc_ortho_workspace(cfg)
    lr, mu, decay, scale = 0.05, 0.9, 0.1, 1.7
    B.moe_muon_step(cfg, g, mom, w, ws, lr=lr, mu=mu, nesterov=nesterov, weight_decay=decay, scale=scale)
    assert B.moe_get_device_error(ws) == B.MOE_OK
    f = lambda v: float(np.float32(v))
    per = [tuple(f(v) for v in lo.MUON_COEFFS)] * 5
    half = torch.finfo(wdtype).eps / 2
    for i in range(n):
        m, u = lo.muon_direction(f64(g[i]), f64(m0[i]), f(mu), nesterov)
        assert (np.abs(f64(mom[i]) - m) <= 2 * 2.0 ** -24 * (np.abs(f(mu) * f64(m0[i])) + np.abs(f64(g[i])))).all()
        x = lo.newton_schulz(u, per, f(cfg.eps))
        tol, _ = allowed(u, per, cfg.eps, x)
        keep, step = 1 - f(lr) * f(decay), f(lr) * f(scale)
        want = keep * f64(w0[i]) - step * x
        # X's error times the step, the weight's rounding, and fp32's on the
        # way (keep, step, product and sum: one unit each).
        size = keep * np.abs(f64(w0[i])) + step * np.abs(x)
        room = step * tol * np.linalg.norm(x) + half * np.linalg.norm(want) + 4 * 2.0 ** -24 * np.linalg.norm(size)
        assert np.linalg.norm(f64(w[i]) - want) <= room


def test_muon_steps_follow_each_other_like_the_pieces():
    # The step equals momentum, moe_orthogonalize and the update by hand.
    cfg = OrthoConfig(n=2, rows=192, cols=320, dtype="f32")
    ws = B.alloc_ortho_workspace(cfg)
    mom = torch.zeros(2, 192, 320, device="cuda")
    w = torch.randn(2, 192, 320, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2)) / 18
    for k in range(3):
        g = gradients(2, 192, 320, "f32", seed=k)
        u = g + 0.95 * (0.95 * mom + g)
        o = run(cfg, u.contiguous())
        want = f64(w) - 0.02 * f64(o)
        B.moe_muon_step(cfg, g, mom, w, ws, lr=0.02)
        # The same products on inputs that differ by fp32 roundings, which can
        # turn fp16 roundings: each side within 2e-3 of the exact X (the bound
        # above at this shape), and o rounded to bf16 besides.
        assert np.linalg.norm(f64(w) - want) <= 0.02 * (2 * 2e-3 + 2.0 ** -8) * np.linalg.norm(f64(o))


def test_no_matrices():
    cfg = B.make_ortho_config(n=0, rows=8, cols=8)
    ws = B.alloc_ortho_workspace(cfg)
    B.moe_orthogonalize(cfg, None, None, ws)
