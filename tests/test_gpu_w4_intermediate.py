"""The SwiGLU intermediate between the two launches of the 4-bit experts: eleven
significant bits, under a power of two for every eight neighbours.

Bounds, per value: those of test_gpu_w4 with the intermediate's own term. A
value is off by half a step of fp16, 2^-11 of it, or, below 2^-14 of the largest
of its eight, by 2^-25 of that one (raised by 2^-11 before its exponent is
taken). Eight neighbours are eight consecutive rows of W1 and W3.

In the 2-norm of a segment: the result's rounding to bf16 alone leaves an rms
error of 0.42 2^-8 (mantissas spread over a binade). The intermediate's, where
one value makes up a row, moves all of it by 2^-11, which is r = 2^-3 / 0.42 =
0.30 of that, where many do by less. Over n values the two errors' correlation
is within 4 / sqrt(n) (four sigma), 0.5 over 64: together at most sqrt(1 + 0.30^2
+ 2 0.30 0.5) = 1.18 of the first; fp32's part, 2^-15, disappears beside the rest
of 1.2. An intermediate of bf16's eight bits would leave 1.41.
"""
import numpy as np
import pytest
import torch

import oracle.layer_oracle as lo
import test_gpu_w4 as W
from mixture_experts_ffn_sigmoid_b200 import binding as B

pytestmark = pytest.mark.gpu
f64 = W.f64


def check_rows(got, x, ms, what, e=None):
    w1, w3, w2 = (W.dense(m, e) for m in ms)
    s1, s3, s2 = (W.scales(m, e) for m in ms)
    group = ms[0].group
    y, a, b, h = lo.swiglu_rows(x, w1, w3, w2)
    units = lambda K: (K / 16 + 16) * 2.0 ** -23
    K, f = x.shape[1], h.shape[1]
    in_group = (group / 8 + 8) * 2.0 ** -23 * 2 * 15
    split = lambda v, w: 2.0 ** -35 * np.abs(v).max(-1, keepdims=True) * np.abs(w).sum(-1)
    ea, eb = (units(K) * (np.abs(x) @ np.abs(w).T) + in_group * (np.abs(x) @ s.T) + split(x, w)
              for w, s in ((w1, s1), (w3, s3)))
    largest = np.repeat(np.abs(h).reshape(len(h), -1, 8).max(-1), 8, axis=-1)
    eh = 1.1 * ea * (np.abs(b) + eb) + np.abs(h) / np.maximum(np.abs(b), 1e-300) * eb \
        + (2.0 ** -11 + 2.0 ** -20) * np.abs(h) + 1.001 * 2.0 ** -25 * largest
    ey = eh @ np.abs(w2).T + units(f) * (np.abs(h) @ np.abs(w2).T) + in_group * (np.abs(h) @ s2.T) + split(h, w2) \
        + 2.0 ** -8 * np.abs(y) + 1e-38
    got = f64(got)
    assert np.isfinite(got).all(), what
    assert (np.abs(got - y) <= ey).all(), (what, (np.abs(got - y) - ey).max())
    return got, y


def check(cfg, x, w, ws, perm_src, offsets, y, ys, norm=True):
    off, xp = offsets.tolist(), f64(x)[perm_src.cpu().numpy()]
    parts = [(y[off[e]:off[e + 1]], xp[off[e]:off[e + 1]], w, f"expert {e}", e) for e in range(cfg.E) if off[e] < off[e + 1]]
    if ys is not None:
        parts.append((ys, f64(x), ws, "shared", None))
    for part in parts:
        got, want = check_rows(*part)
        if norm and got.size >= 64:
            once = f64(torch.from_numpy(want).to(torch.bfloat16))
            assert np.linalg.norm(got - want) <= 1.2 * np.linalg.norm(once - want), part[3]


@pytest.mark.parametrize("T,d,E,k,f,fs,group,zeros", W.CASES)
def test_eleven_bits_on_every_shape(T, d, E, k, f, fs, group, zeros):
    a = W.make(T, d, E, k, f, fs, group, zeros, seed=21)
    check(*a, *W.run_experts(*a))


@pytest.mark.parametrize("T,spread", [(6, 6), (30, 12), (6, 20)])
def test_neighbours_of_very_different_size(T, spread):
    # W3's rows, and with them the intermediate's values, differ by powers of
    # two up to 2^(2 spread) from one to the next.
    cfg, x, w, ws, perm_src, offsets = a = W.make(T, 256, 4, 2, 192, 64, 32, True, seed=5)
    g = torch.Generator(device="cuda").manual_seed(7)
    for m in (w[1], ws[1]):
        m.scale.mul_(torch.exp2(torch.randint(-spread, spread + 1, m.scale.shape[:-1], generator=g, device="cuda"))[..., None])
    check(*a, *W.run_experts(*a), norm=False)


def test_an_intermediate_that_overflows_stays_in_its_row():
    cfg, x, w, ws, perm_src, offsets = W.make(9, 256, 3, 2, 128, 128, 64, False, seed=3)
    y, ys = W.run_experts(cfg, x, w, ws, perm_src, offsets)
    big = x.clone()
    big[4] *= 1e30                              # finite, its square is not
    out, outs = torch.empty_like(y), torch.empty_like(ys)
    B.moe_expert_swiglu_w4(cfg, big, perm_src, offsets, *w, big, *ws, out, outs, B.alloc_workspace(cfg))
    hit = perm_src == 4
    assert torch.equal(out[~hit], y[~hit]) and torch.isnan(out[hit].float()).all()
    rest = torch.arange(9, device="cuda") != 4
    assert torch.equal(outs[rest], ys[rest]) and torch.isnan(outs[4].float()).all()


@pytest.mark.parametrize("T,d,E,k,f,fs,zeros", [
    (200, 256, 3, 1, 256, 128, False), (197, 384, 3, 1, 128, 0, True), (71, 512, 2, 2, 384, 128, True),
    (64, 128, 1, 1, 128, 0, False), (77, 16384, 1, 1, 128, 128, False), (65, 128, 1, 1, 16384, 0, True)])
def test_sixteen_rows_a_pass(T, d, E, k, f, fs, zeros):
    # Groups of 128 and 64 rows a segment or more; the widest rows fit eight or fewer at a time.
    a = W.make(T, d, E, k, f, fs, 128, zeros, seed=31)
    check(*a, *W.run_experts(*a))
