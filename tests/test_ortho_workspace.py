"""The scratch of the Newton-Schulz products, without a GPU."""
import pytest

from mixture_experts_ffn_sigmoid_b200 import binding as B
from mixture_experts_ffn_sigmoid_b200.inputs import OrthoConfig


@pytest.mark.parametrize("rows,cols", [(1, 1), (128, 512), (512, 128), (40, 300)])
@pytest.mark.parametrize("n", [1, 592, 100000])
def test_matrices_that_stay_on_chip_need_the_error_word_alone(n, rows, cols):
    assert B.ortho_workspace_size(OrthoConfig(n=n, rows=rows, cols=cols)) <= 1024


@pytest.mark.parametrize("rows,cols", [(129, 129), (16, 520), (520, 16)])
def test_others_need_both_x_and_the_squares(rows, cols):
    # Two of X and two of m x m in fp16, a matrix, up to a group's size.
    m, n = min(rows, cols), max(rows, cols)
    size = lambda count: B.ortho_workspace_size(OrthoConfig(n=count, rows=rows, cols=cols))
    assert size(100) >= 100 * (4 * m * n + 4 * m * m)
    assert size(100) > size(10) and size(40000) <= 700 * size(1)
