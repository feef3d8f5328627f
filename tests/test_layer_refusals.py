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
