"""The workspace of the norms' gradients up to the largest token count, without a GPU."""
import pytest

from mixture_experts_ffn_sigmoid_b200 import binding as B
from mixture_experts_ffn_sigmoid_b200.inputs import NormConfig


@pytest.mark.parametrize("T", [2 ** 30, 2 ** 31 - 3000, 2 ** 31 - 2, 2 ** 31 - 1])
@pytest.mark.parametrize("d", [8, 7168])
def test_workspace_of_many_tokens(T, d):
    # Four fp32 rows a run; runs are bounded by the GPU's CTA slots (16 an SM
    # at most), and enough tokens fill nearly all of them.
    size, some = B.norm_backward_workspace_size(NormConfig(T=T, d=d)), B.norm_backward_workspace_size(NormConfig(T=2 ** 20, d=d))
    assert size % (16 * d) == 0
    assert 0.9 * some <= size <= 16 * d * 16 * 256
