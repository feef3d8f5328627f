"""Stacks worked through in groups, and stacks of matrices that stay on chip, which
run all together; bounds as in test_gpu_ortho."""
import pytest
import torch

import test_gpu_ortho as N
from mixture_experts_ffn_sigmoid_b200 import binding as B
from mixture_experts_ffn_sigmoid_b200.inputs import OrthoConfig

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,cols", [(16, 520), (600, 12)])
def test_large_stack_in_groups(rows, cols):
    # 8 tiles of each of 74 pairs are one group: the stack takes two.
    cfg = OrthoConfig(n=700, rows=rows, cols=cols)
    assert B.ortho_workspace_size(cfg) == B.ortho_workspace_size(OrthoConfig(n=350, rows=rows, cols=cols))
    g = N.gradients(700, rows, cols, "bf16")
    o = N.run(cfg, g)
    N.check(cfg, g, o, matrices=[0, 1, 349, 350, 351, 698, 699])
    assert torch.isfinite(o.float()).all()


@pytest.mark.parametrize("n,rows,cols", [(2000, 24, 16), (1500, 128, 40)])
def test_large_stack_on_chip(n, rows, cols):
    cfg = OrthoConfig(n=n, rows=rows, cols=cols)
    g = N.gradients(n, rows, cols, "bf16", seed=4)
    before = g.clone()
    o = N.run(cfg, g)
    assert torch.equal(g, before)
    N.check(cfg, g, o, matrices=[0, 1, 591, 592, 593, n // 2, n - 1])
    assert torch.isfinite(o.float()).all()
