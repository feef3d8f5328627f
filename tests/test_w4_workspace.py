"""The block's workspace, which every entry point shares, holds nothing that only
the 4-bit experts use: it grows with f by the intermediate alone."""
import pytest

from mixture_experts_ffn_sigmoid_b200 import binding as B
from mixture_experts_ffn_sigmoid_b200.inputs import MoEConfig


@pytest.mark.parametrize("dtype,es", [("bf16", 2), ("f32", 4)])
@pytest.mark.parametrize("T,d,k", [(4096, 4096, 2), (128, 256, 1)])
@pytest.mark.parametrize("f_shared", [0, 1024])
def test_workspace_grows_with_f_by_the_intermediate(T, d, k, f_shared, dtype, es):
    size = lambda f, fs: B.workspace_size(MoEConfig("w", T=T, d=d, E=8, k=k, f=f, f_shared=fs, dtype=dtype))
    for f in (4096, 14336):
        assert size(f, f_shared) - size(256, f_shared) == T * k * (f - 256) * es
    if f_shared:
        assert size(256, 2 * f_shared) - size(256, f_shared) == T * f_shared * es
