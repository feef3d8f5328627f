"""The oracle of the operators around the block, held against hand values and
differences on the CPU."""
import numpy as np
import pytest

import oracle.layer_oracle as lo


def test_residual_norm_by_hand():
    # y = (3, 4): mean square 12.5; without eps the norm is (3, 4) / sqrt(12.5).
    h, y = np.array([[1.0, -1.0]]), np.array([[3.0, 4.0]])
    out, u = lo.residual_norm(h, y, np.array([1.0, 2.0]), np.array([[0.5, -1.0]]), np.array([2.0, 1.0]),
                              gate_tokens=1, eps=0.0, alpha=2.0, beta=10.0)
    r = 1 / np.sqrt(12.5)
    want = np.array([2.0 + 10 * 0.5 * 3 * r, -2.0 - 10 * 4 * r * 2])
    assert np.allclose(out[0], want, rtol=1e-15)
    assert np.allclose(u[0], want / np.sqrt((want ** 2).mean()) * [2, 1], rtol=1e-15)


@pytest.mark.parametrize("post,gate,pre,offset", [(1, 1, 1, 0.0), (1, 1, 1, 1.0), (0, 1, 1, 0.0), (1, 0, 1, 0.0),
                                                  (1, 1, 0, 0.0), (0, 0, 1, 0.0)])
def test_residual_norm_backward_against_differences(post, gate, pre, offset):
    rng = np.random.default_rng(3)
    T, d = 5, 6
    kw = dict(gate_tokens=2, eps=1e-3, alpha=0.7, beta=1.3, w_offset=offset)
    p = dict(h=rng.standard_normal((T, d)), y=rng.standard_normal((T, d)),
             w_post=rng.standard_normal(d) if post else None, gate=rng.standard_normal((3, d)) if gate else None,
             w_pre=rng.standard_normal(d) if pre else None)
    du, dh = rng.standard_normal((T, d)), rng.standard_normal((T, d))

    def loss(**q):
        out, u = lo.residual_norm(**q, **kw)
        return (out * dh).sum() + (0.0 if u is None else (u * du).sum())

    out, _ = lo.residual_norm(**p, **kw)
    g = lo.residual_norm_backward(out, p["y"], p["w_post"], p["gate"], p["w_pre"], du if pre else None, dh, **kw)
    for name, v in p.items():
        if v is None:
            assert g["d" + name] is None
            continue
        step = rng.standard_normal(v.shape)
        e = 1e-5
        diff = (loss(**{**p, name: v + e * step}) - loss(**{**p, name: v - e * step})) / (2 * e)
        want = (g["d" + name] * step).sum()
        # A central difference is off by e^2 times a third derivative of order
        # one, and by rounding of order 1e-15 / e.
        assert abs(diff - want) <= 1e-7 * max(1.0, abs(want)), name


def test_newton_schulz_acts_on_singular_values():
    rng = np.random.default_rng(0)
    for shape in ((4, 7), (7, 4), (5, 5)):
        u = rng.standard_normal(shape)
        left, s, right = np.linalg.svd(u, full_matrices=False)
        s = s / (np.sqrt((s * s).sum()) + 1e-7)
        coeffs = [lo.MUON_COEFFS, (1.5, -0.5, 0.0), (2.0, -1.5, 0.5)]
        for a, b, c in coeffs:
            s = a * s + b * s ** 3 + c * s ** 5
        assert np.allclose(lo.newton_schulz(u, coeffs), (left * s) @ right, rtol=0, atol=1e-13)


def test_swiglu_rows_and_w4_dense_by_hand():
    q, scale = np.array([[0x98, 0x07]], dtype=np.uint8), np.array([[0.5, 2.0]])
    assert np.array_equal(lo.w4_dense(q, scale, None, 2), [[0.0, 0.5, -2.0, -16.0]])
    assert np.array_equal(lo.w4_dense(q, scale, np.array([[8, 7]], dtype=np.uint8), 2), [[0.0, 0.5, 0.0, -14.0]])
    y, a, b, h = lo.swiglu_rows(np.array([[1.0]]), np.array([[2.0]]), np.array([[3.0]]), np.array([[4.0]]))
    assert np.allclose(y, 4 * 3 * 2 / (1 + np.exp(-2.0)))
