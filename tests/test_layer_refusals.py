"""Argument checks of the operators around the block, on the CPU: every refusal
comes before a device is touched, so the addresses here are never read."""
import ctypes

import pytest
import torch

from mixture_experts_ffn_sigmoid_b200 import binding as B
from mixture_experts_ffn_sigmoid_b200 import build as build_mod
from mixture_experts_ffn_sigmoid_b200.inputs import NormConfig

FAKE, ODD = 0x10000, 0x10008
BIG = 1 << 40


@pytest.fixture(scope="module", autouse=True)
def built_library():
    build_mod.build()
    return B.lib()


def norm(**kw):
    return B.make_norm_config(**{**dict(T=8, d=64, dtype="bf16", gate_tokens=4), **kw})


def call_norm(cfg, h=FAKE, y=FAKE + 4096, w_post=FAKE, gate=FAKE, w_pre=FAKE, h_out=FAKE, u=FAKE + 4096):
    return B.lib().moe_residual_norm(ctypes.byref(cfg) if cfg else None, h, y, w_post, gate, w_pre, h_out, u, None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), B.MOE_ERR_INVALID_ARG), (dict(d=0), B.MOE_ERR_INVALID_ARG), (dict(gate_tokens=0), B.MOE_ERR_INVALID_ARG),
    (dict(eps=0.0), B.MOE_ERR_INVALID_ARG), (dict(eps=float("nan")), B.MOE_ERR_INVALID_ARG),
    (dict(alpha=float("inf")), B.MOE_ERR_INVALID_ARG), (dict(beta=float("nan")), B.MOE_ERR_INVALID_ARG),
    (dict(w_offset=float("inf")), B.MOE_ERR_INVALID_ARG), (dict(d=100), B.MOE_ERR_MISALIGNED),
    (dict(d=102, dtype="f32"), B.MOE_ERR_MISALIGNED), (dict(d=16392), B.MOE_ERR_UNSUPPORTED),
    (dict(d=8196, dtype="f32"), B.MOE_ERR_UNSUPPORTED)])
def test_norm_settings(kw, status):
    c = norm(**kw)
    assert call_norm(c) == status
    assert B.lib().moe_residual_norm_backward_workspace_size(ctypes.byref(c)) == 0
    assert B.lib().moe_residual_norm_backward(ctypes.byref(c), *[FAKE] * 13, BIG, None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(y=None), B.MOE_ERR_INVALID_ARG),                     # a branch's weights without a branch
    (dict(y=None, w_post=None, gate=None, h_out=None, w_pre=None, u=None), B.MOE_ERR_INVALID_ARG),
    (dict(y=None, w_post=None, gate=None), B.MOE_ERR_INVALID_ARG),   # h_out without a branch
    (dict(w_pre=None), B.MOE_ERR_INVALID_ARG), (dict(u=None), B.MOE_ERR_INVALID_ARG),
    (dict(h=None), B.MOE_ERR_INVALID_ARG), (dict(h_out=None), B.MOE_ERR_INVALID_ARG),
    (dict(u=FAKE), B.MOE_ERR_INVALID_ARG),
    (dict(h=ODD), B.MOE_ERR_MISALIGNED), (dict(y=ODD), B.MOE_ERR_MISALIGNED), (dict(w_post=ODD), B.MOE_ERR_MISALIGNED),
    (dict(gate=ODD), B.MOE_ERR_MISALIGNED), (dict(w_pre=ODD), B.MOE_ERR_MISALIGNED),
    (dict(h_out=ODD), B.MOE_ERR_MISALIGNED), (dict(u=ODD), B.MOE_ERR_MISALIGNED)])
def test_norm_pointers(kw, status):
    assert call_norm(norm(), **kw) == status


def test_norm_null_settings_and_no_tokens():
    assert call_norm(None) == B.MOE_ERR_INVALID_ARG
    assert call_norm(norm(T=0), h=None, h_out=None, u=None) == B.MOE_OK


NAMES = ("h_out", "y", "w_post", "gate", "w_pre", "du", "dh_out", "dh", "dy", "dw_post", "dgate", "dw_pre", "ws")


@pytest.mark.parametrize("kw,status", [
    (dict(y=None), B.MOE_ERR_INVALID_ARG), (dict(w_post=None), B.MOE_ERR_INVALID_ARG),
    (dict(gate=None), B.MOE_ERR_INVALID_ARG), (dict(w_pre=None), B.MOE_ERR_INVALID_ARG),
    (dict(du=None), B.MOE_ERR_INVALID_ARG), (dict(h_out=None), B.MOE_ERR_INVALID_ARG),
    (dict(w_pre=None, dw_pre=None, du=None, dh_out=None), B.MOE_ERR_INVALID_ARG),   # no gradient arrives
    (dict(dh=FAKE, dy=FAKE), B.MOE_ERR_INVALID_ARG), (dict(ws=None), B.MOE_ERR_INVALID_ARG),
    *[({n: ODD}, B.MOE_ERR_MISALIGNED) for n in NAMES]])
def test_norm_backward_pointers(kw, status):
    c = norm()
    a = {n: FAKE + 4096 * i for i, n in enumerate(NAMES)}
    a.update(kw)
    assert B.lib().moe_residual_norm_backward(ctypes.byref(c), *[a[n] for n in NAMES], BIG, None) == status


@pytest.mark.parametrize("one,other", [("dw_post", "dw_pre"), ("dgate", "dy"), ("dgate", "dh"), ("dh", "dw_pre"), ("dgate", "dw_post")])
def test_norm_backward_outputs_are_distinct(one, other):
    a = {n: FAKE + 4096 * i for i, n in enumerate(NAMES)}
    a[one] = a[other]
    assert B.lib().moe_residual_norm_backward(ctypes.byref(norm()), *[a[n] for n in NAMES], BIG, None) == B.MOE_ERR_INVALID_ARG


def test_norm_backward_workspace_must_be_large_enough():
    c = norm()
    need = B.norm_backward_workspace_size(c)
    assert need > 0
    args = [FAKE + 4096 * i for i in range(13)]
    assert B.lib().moe_residual_norm_backward(ctypes.byref(c), *args, need - 1, None) == B.MOE_ERR_WORKSPACE_TOO_SMALL


bf = torch.bfloat16


@pytest.mark.parametrize("name,bad", [
    ("h", torch.zeros(7, 64, dtype=bf)), ("h", torch.zeros(8, 64)), ("y", torch.zeros(7, 64, dtype=bf)),
    ("gate", torch.zeros(1, 64, dtype=bf)), ("w_post", torch.zeros(63, dtype=bf)), ("w_pre", torch.zeros(64)),
    ("h_out", torch.zeros(7, 64, dtype=bf)), ("u", torch.zeros(8, 63, dtype=bf)), ("h", None), ("h_out", None)])
def test_norm_binding_refuses_short_or_wrong_tensors(name, bad):
    a = dict(h=torch.zeros(8, 64, dtype=bf), y=torch.zeros(8, 64, dtype=bf), w_post=torch.zeros(64, dtype=bf),
             gate=torch.zeros(2, 64, dtype=bf), w_pre=torch.zeros(64, dtype=bf), h_out=torch.zeros(8, 64, dtype=bf),
             u=torch.zeros(8, 64, dtype=bf))
    cfg = NormConfig(T=8, d=64, gate_tokens=4)
    with pytest.raises(ValueError, match="CUDA"):     # well-formed CPU tensors get as far as the device check
        B.moe_residual_norm(cfg, **a)
    a[name] = bad
    with pytest.raises(ValueError, match=name):
        B.moe_residual_norm(cfg, **a)


# ------------------------------------------------------------- 4-bit weights
def w4(q=FAKE, scale=FAKE, zero=None):
    return ctypes.byref(B.CW4Matrix(q, scale, zero))


@pytest.mark.parametrize("rows,K,dtype,group,status", [
    (-1, 128, 0, 64, B.MOE_ERR_INVALID_ARG), (4, 0, 0, 64, B.MOE_ERR_INVALID_ARG), (4, 100, 0, 64, B.MOE_ERR_INVALID_ARG),
    (4, 128, 2, 64, B.MOE_ERR_INVALID_ARG), (4, 128, 0, 16, B.MOE_ERR_INVALID_ARG), (4, 128, 0, 0, B.MOE_ERR_INVALID_ARG),
    (1 << 60, 128, 0, 64, B.MOE_ERR_UNSUPPORTED), (0, 128, 0, 64, B.MOE_OK)])
def test_w4_matrix_shapes(rows, K, dtype, group, status):
    L = B.lib()
    assert L.moe_w4_quantize(rows, K, dtype, group, FAKE, w4(), None) == status
    assert L.moe_w4_dequantize(rows, K, dtype, group, w4(), FAKE, None) == status


@pytest.mark.parametrize("m,w,status", [
    (None, FAKE, B.MOE_ERR_INVALID_ARG), (w4(q=None), FAKE, B.MOE_ERR_INVALID_ARG),
    (w4(scale=None), FAKE, B.MOE_ERR_INVALID_ARG), (w4(q=ODD), FAKE, B.MOE_ERR_MISALIGNED),
    (w4(scale=ODD), FAKE, B.MOE_ERR_MISALIGNED), (w4(zero=ODD), FAKE, B.MOE_ERR_MISALIGNED), (w4(), None, B.MOE_ERR_INVALID_ARG), (w4(), ODD, B.MOE_ERR_MISALIGNED)])
def test_w4_matrix_pointers(m, w, status):
    L = B.lib()
    assert L.moe_w4_quantize(4, 128, 0, 64, w, m, None) == status
    assert L.moe_w4_dequantize(4, 128, 0, 64, m, w, None) == status


def moe_cfg(**kw):
    return B.CConfig(**{**dict(T=8, d=128, E=4, k=2, f=256, dtype=B.MOE_DTYPE_BF16, gate_mode=0, n_groups=1, topk_groups=1,
                               route_scale=1.0, f_shared=128), **kw})


def call_experts_w4(cfg, group=64, **kw):
    a = dict(x=FAKE, perm_src=FAKE, off=FAKE, w1=w4(), w3=w4(), w2=w4(), xs=FAKE, ws1=w4(), ws3=w4(), ws2=w4(), y=FAKE,
             ys=FAKE, ws=FAKE, n=BIG)
    a.update(kw)
    return B.lib().moe_expert_swiglu_w4(ctypes.byref(cfg), group, *[a[n] for n in (
        "x", "perm_src", "off", "w1", "w3", "w2", "xs", "ws1", "ws3", "ws2", "y", "ys", "ws", "n")], None)


def call_forward_w4(cfg, group=64, **kw):
    a = dict(x=FAKE, wr=FAKE, bias=None, w1=w4(), w3=w4(), w2=w4(), ws1=w4(), ws3=w4(), ws2=w4(), y=FAKE, ws=FAKE, n=BIG)
    a.update(kw)
    return B.lib().moe_forward_w4(ctypes.byref(cfg), group, *[a[n] for n in (
        "x", "wr", "bias", "w1", "w3", "w2", "ws1", "ws3", "ws2", "y", "ws", "n")], None)


@pytest.mark.parametrize("kw,group,status", [
    (dict(k=5), 64, B.MOE_ERR_INVALID_ARG), ({}, 16, B.MOE_ERR_INVALID_ARG), ({}, 256, B.MOE_ERR_INVALID_ARG),
    (dict(dtype=B.MOE_DTYPE_F32), 64, B.MOE_ERR_UNSUPPORTED), (dict(d=96), 64, B.MOE_ERR_UNSUPPORTED),
    (dict(f=288), 64, B.MOE_ERR_UNSUPPORTED), (dict(f=16448), 64, B.MOE_ERR_UNSUPPORTED), (dict(f_shared=96), 64, B.MOE_ERR_UNSUPPORTED)])
def test_w4_experts_settings(kw, group, status):
    assert call_experts_w4(moe_cfg(**kw), group) == status
    assert call_forward_w4(moe_cfg(**kw), group) == status


@pytest.mark.parametrize("kw,status", [
    *[({n: None}, B.MOE_ERR_INVALID_ARG) for n in ("x", "w1", "w3", "w2", "ws1", "ws3", "ws2", "y", "ws")],
    (dict(x=ODD), B.MOE_ERR_MISALIGNED), (dict(w2=w4(q=ODD)), B.MOE_ERR_MISALIGNED),
    (dict(ws1=w4(scale=None)), B.MOE_ERR_INVALID_ARG), (dict(y=ODD), B.MOE_ERR_MISALIGNED),
    (dict(n=1000), B.MOE_ERR_WORKSPACE_TOO_SMALL)])
def test_w4_experts_pointers(kw, status):
    assert call_experts_w4(moe_cfg(), **kw) == status
    assert call_forward_w4(moe_cfg(), **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(off=None), B.MOE_ERR_INVALID_ARG), (dict(xs=None), B.MOE_ERR_INVALID_ARG), (dict(ys=None), B.MOE_ERR_INVALID_ARG),
    (dict(off=FAKE + 2), B.MOE_ERR_MISALIGNED), (dict(perm_src=FAKE + 1), B.MOE_ERR_MISALIGNED)])
def test_w4_expert_tables(kw, status):
    assert call_experts_w4(moe_cfg(), **kw) == status


def test_w4_outputs_are_distinct():
    assert call_experts_w4(moe_cfg(), y=FAKE + 4096, ys=FAKE + 4096) == B.MOE_ERR_INVALID_ARG


def test_w4_no_tokens():
    assert call_experts_w4(moe_cfg(T=0), x=None, y=None) == B.MOE_OK
    assert call_forward_w4(moe_cfg(T=0), x=None, y=None) == B.MOE_OK


def test_w4_matrix_binding():
    u8 = torch.uint8
    with pytest.raises(ValueError, match="group"):
        B.W4Matrix(torch.zeros(4, 64, dtype=u8), torch.zeros(4, 8, dtype=bf), group=16)
    with pytest.raises(ValueError, match="q"):
        B.W4Matrix(torch.zeros(4, 64), torch.zeros(4, 2, dtype=bf), group=64)
    with pytest.raises(ValueError, match="scale"):
        B.W4Matrix(torch.zeros(4, 64, dtype=u8), torch.zeros(4, 3, dtype=bf), group=64)
    with pytest.raises(ValueError, match="zero"):
        B.W4Matrix(torch.zeros(4, 64, dtype=u8), torch.zeros(4, 2, dtype=bf), torch.zeros(4, 1, dtype=u8), group=64)
    with pytest.raises(ValueError, match="whole groups"):
        B.W4Matrix.empty(4, 100, group=64, device="cpu")
    m = B.W4Matrix.empty(4, 128, group=64, zero_points=True, device="cpu")
    assert (m.rows, m.K, m.zero.shape) == (4, 128, (4, 2))
    with pytest.raises(ValueError, match="CUDA"):
        B.moe_w4_quantize(torch.zeros(4, 128), m)
    with pytest.raises(ValueError, match="elements"):
        B.moe_w4_quantize(torch.zeros(3, 128), m)
    with pytest.raises(ValueError, match="dtype"):
        B.moe_w4_dequantize(m, torch.zeros(4, 128, dtype=torch.float16))


def test_w4_matrix_keeps_its_tensors():
    m = B.W4Matrix.empty(4, 128, group=64, device="cpu")
    for name in ("q", "scale", "zero"):
        with pytest.raises(AttributeError):
            setattr(m, name, None)


def test_w4_block_binding():
    from mixture_experts_ffn_sigmoid_b200.inputs import MoEConfig
    cfg = MoEConfig("c", T=2, d=128, E=4, k=2, f=64)
    make = lambda *s, group=64: B.W4Matrix.empty(*s, group=group, device="cpu")
    a = dict(x=torch.zeros(2, 128, dtype=bf), w_router=torch.zeros(4, 128, dtype=bf), bias=None, w1=make(4, 64, 128),
             w3=make(4, 64, 128), w2=make(4, 128, 64), ws1=None, ws3=None, ws2=None, y=torch.zeros(2, 128, dtype=bf),
             workspace=torch.zeros(8, dtype=torch.uint8))
    with pytest.raises(ValueError, match="CUDA"):
        B.moe_forward_w4(cfg, **a)
    for name, bad in (("w1", make(3, 64, 128)), ("w2", make(4, 64, 128)), ("w3", make(4, 64, 128, group=128))):
        with pytest.raises(ValueError, match=name):
            B.moe_forward_w4(cfg, **{**a, name: bad})
    with pytest.raises(TypeError, match="w1"):
        B.moe_forward_w4(cfg, **{**a, "w1": torch.zeros(4, 64, 128)})


# --------------------------------------------------------- orthogonalisation
def ortho(**kw):
    return B.make_ortho_config(**{**dict(n=2, rows=64, cols=96), **kw})


def call_ortho(c, coeffs=None, g=FAKE, o=FAKE, ws=FAKE, n=BIG):
    return B.lib().moe_orthogonalize(ctypes.byref(c) if c else None, coeffs, g, o, ws, n, None)


def call_muon(c, coeffs=None, g=FAKE, m=FAKE, w=FAKE, wd=0, lr=0.1, mu=0.9, decay=0.0, scale=1.0, ws=FAKE, n=BIG):
    return B.lib().moe_muon_step(ctypes.byref(c) if c else None, coeffs, g, m, w, wd, lr, mu, 1, decay, scale, ws, n, None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), B.MOE_ERR_INVALID_ARG), (dict(rows=0), B.MOE_ERR_INVALID_ARG), (dict(cols=-4), B.MOE_ERR_INVALID_ARG),
    (dict(steps=0), B.MOE_ERR_INVALID_ARG), (dict(steps=65), B.MOE_ERR_INVALID_ARG), (dict(eps=0.0), B.MOE_ERR_INVALID_ARG),
    (dict(eps=float("inf")), B.MOE_ERR_INVALID_ARG), (dict(rows=65537), B.MOE_ERR_UNSUPPORTED),
    (dict(cols=65537), B.MOE_ERR_UNSUPPORTED)])
def test_ortho_settings(kw, status):
    c = ortho(**kw)
    assert B.ortho_workspace_size(c) == 0
    assert call_ortho(c) == status and call_muon(c) == status


def test_ortho_pointers_and_workspace():
    c, bad, odd = ortho(), B.MOE_ERR_INVALID_ARG, B.MOE_ERR_MISALIGNED
    assert call_ortho(None) == bad and call_muon(None) == bad
    for kw in (dict(g=None), dict(o=None), dict(ws=None)):
        assert call_ortho(c, **kw) == bad
    for kw in (dict(g=ODD), dict(o=ODD), dict(ws=ODD)):
        assert call_ortho(c, **kw) == odd
    for kw in (dict(g=None), dict(m=None), dict(w=None), dict(ws=None), dict(wd=2), dict(lr=float("nan")),
               dict(mu=float("inf")), dict(decay=float("nan")), dict(scale=float("inf"))):
        assert call_muon(c, **kw) == bad
    for kw in (dict(g=ODD), dict(m=ODD), dict(w=ODD)):
        assert call_muon(c, **kw) == odd
    need = B.ortho_workspace_size(c)
    assert need > 0 and call_ortho(c, n=need - 1) == B.MOE_ERR_WORKSPACE_TOO_SMALL
    assert call_muon(c, n=need - 1) == B.MOE_ERR_WORKSPACE_TOO_SMALL
    assert call_ortho(ortho(n=0), g=None, o=None) == B.MOE_OK


def test_ortho_arrays_that_must_be_distinct():
    f32, bad = ortho(dtype="f32"), B.MOE_ERR_INVALID_ARG
    assert call_ortho(f32, g=FAKE, o=FAKE) == bad            # o is half as wide: a matrix's result in another's gradient
    a, b = FAKE + 4096, FAKE + 8192
    for kw in (dict(g=a, m=a, w=b), dict(g=a, m=b, w=a), dict(g=b, m=a, w=a)):
        assert call_muon(f32, **kw) == bad


def test_ortho_eps_below_what_fp32_squares_hold():
    for eps in (1e-13, 1e-30):
        assert B.ortho_workspace_size(ortho(eps=eps)) == 0 and call_ortho(ortho(eps=eps)) == B.MOE_ERR_INVALID_ARG
    assert B.ortho_workspace_size(ortho(eps=1e-11)) > 0


@pytest.mark.parametrize("abc,ok", [
    ((1.5, -0.5, 0.0), True), ((2.0, -1.5, 0.5), True), ((float("nan"), 0.0, 0.0), False),
    ((3.0, 0.0, 0.0), False),          # 3^5 of the largest singular value
    ((1.0, 600.0, -600.0), False)])
def test_coefficients_that_leave_the_range_are_refused(abc, ok):
    c = ortho()
    arr = (ctypes.c_float * 15)(*abc * 5)
    # A good set gets as far as the missing gradients.
    assert call_ortho(c, arr, g=None if ok else FAKE) == B.MOE_ERR_INVALID_ARG
    if ok:
        assert call_ortho(c, arr, g=ODD) == B.MOE_ERR_MISALIGNED


def test_ortho_binding():
    z = lambda dt=bf: torch.zeros(2, 64, 96, dtype=dt)
    from mixture_experts_ffn_sigmoid_b200.inputs import OrthoConfig
    c, ws = OrthoConfig(n=2, rows=64, cols=96), torch.zeros(8, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        B.moe_orthogonalize(c, z(), z(), ws)
    with pytest.raises(ValueError, match="g"):
        B.moe_orthogonalize(c, z(torch.float32), z(), ws)
    with pytest.raises(ValueError, match="o"):
        B.moe_orthogonalize(c, z(), z()[:1], ws)
    with pytest.raises(ValueError, match="coeffs"):
        B.moe_orthogonalize(c, z(), z(), ws, coeffs=[(1.0, 2.0, 3.0)] * 2)
    with pytest.raises(ValueError, match="momentum"):
        B.moe_muon_step(c, z(), z(), z(), ws, lr=0.1)
    with pytest.raises(ValueError, match="weight"):
        B.moe_muon_step(c, z(), z(torch.float32), z(torch.float16), ws, lr=0.1)
