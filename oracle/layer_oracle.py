"""CPU oracle of what stands around the expert block, in plain numpy fp64.

Test infrastructure, as ``moe_oracle``: written from the definitions, sharing
no code with the CUDA path.

* ``residual_norm`` and ``residual_norm_backward``: the norms before and after
  a block with its gate and residual scale (Sparse MoE FFN note, eq. 12: the
  residual around the block).
"""
from __future__ import annotations

import numpy as np


# ----------------------------------------------------------- residual norms
def rms_norm(v, w, eps, w_offset=0.0):
    """v / sqrt(mean(v^2) + eps) * (w + w_offset), rows on the last axis."""
    return v / np.sqrt((v * v).mean(axis=-1, keepdims=True) + eps) * (w + w_offset)


def gate_rows(gate, T, gate_tokens, d):
    """The gate row of every token, [T, d] (ones without a gate)."""
    if gate is None:
        return np.ones((T, d))
    return gate[np.arange(T) // gate_tokens]


def residual_norm(h, y, w_post, gate, w_pre, *, gate_tokens=1, eps=1e-6, alpha=1.0, beta=1.0, w_offset=0.0):
    """(h_out, u); u None without w_pre. y None: h_out is h."""
    T, d = h.shape
    if y is None:
        out = h
    else:
        z = y if w_post is None else rms_norm(y, w_post, eps, w_offset)
        out = alpha * h + beta * gate_rows(gate, T, gate_tokens, d) * z
    return out, None if w_pre is None else rms_norm(out, w_pre, eps, w_offset)


def rms_norm_backward(v, w, dz, eps, w_offset=0.0):
    """(dv, dw) of rms_norm: dv = r (q - n mean(q n)), n = v r, q = dz (w + w_offset)."""
    r = 1.0 / np.sqrt((v * v).mean(axis=-1, keepdims=True) + eps)
    n, q = v * r, dz * (w + w_offset)
    return r * (q - n * (q * n).mean(axis=-1, keepdims=True)), (dz * n).sum(axis=0)


def residual_norm_backward(h_out, y, w_post, gate, w_pre, du, dh_out, *, gate_tokens=1, eps=1e-6, alpha=1.0,
                           beta=1.0, w_offset=0.0):
    """dict of dh, dy, dw_post, dgate, dw_pre (None where there is no such input)."""
    T, d = (h_out if h_out is not None else y).shape
    total = np.zeros((T, d)) if dh_out is None else dh_out.copy()
    out = dict(dy=None, dw_post=None, dgate=None, dw_pre=None)
    if w_pre is not None:
        dv, out["dw_pre"] = rms_norm_backward(h_out, w_pre, du, eps, w_offset)
        total += dv
    if y is None:
        out["dh"] = total
        return out
    out["dh"] = alpha * total
    z = y if w_post is None else rms_norm(y, w_post, eps, w_offset)
    dz = beta * gate_rows(gate, T, gate_tokens, d) * total
    if gate is not None:
        out["dgate"] = np.zeros_like(gate)
        np.add.at(out["dgate"], np.arange(T) // gate_tokens, beta * total * z)
    if w_post is None:
        out["dy"] = dz
    else:
        out["dy"], out["dw_post"] = rms_norm_backward(y, w_post, dz, eps, w_offset)
    return out


# ------------------------------------------------------------ 4-bit weights
def w4_dense(q, scale, zero, group):
    """Dense fp64 values of 4-bit codes: q bytes [..., K/2] (even k low), scale
    and zero [..., K/group], zero None: 8."""
    code = np.empty((*q.shape[:-1], 2 * q.shape[-1]))
    code[..., 0::2], code[..., 1::2] = q & 15, q >> 4
    z = 8.0 if zero is None else np.repeat(zero.astype(np.float64), group, axis=-1)
    return np.repeat(scale, group, axis=-1) * (code - z)


def swiglu_rows(x, w1, w3, w2):
    """(y, a, b, h) of W2 (SiLU(W1 x) * W3 x) for rows x."""
    a, b = x @ w1.T, x @ w3.T
    h = a / (1.0 + np.exp(-a)) * b
    return h @ w2.T, a, b, h


# --------------------------------------------------------- orthogonalisation
MUON_COEFFS = (3.4445, -4.7750, 2.0315)


def newton_schulz(u, coeffs, eps=1e-7, stored=lambda v: v, stored_a=None, stored_b=None):
    """X of the Newton-Schulz steps for one matrix u; coeffs [(a, b, c)] per
    step. ``stored`` rounds what an implementation keeps between products (X,
    A = X X^T and a I + b A + c A^2): the identity gives the exact result.
    stored_a and stored_b take its place for the two products."""
    if u.shape[0] > u.shape[1]:
        return newton_schulz(u.T, coeffs, eps, stored, stored_a, stored_b).T
    x = stored(u / (np.sqrt((u * u).sum()) + eps))
    for k, (a, b, c) in enumerate(coeffs):
        g = (stored_a or stored)(x @ x.T)
        x = (stored_b or stored)(a * np.eye(len(g)) + b * g + c * (g @ g)) @ x
        if k + 1 < len(coeffs):
            x = stored(x)
    return x


def half_64(v):
    """v rounded to IEEE half precision at 64 times its size."""
    return (v * 64.0).astype(np.float16).astype(np.float64) / 64.0


def half_64_off_diagonal(v):
    """half_64 but for the diagonal, which stays."""
    return half_64(v) + np.diag(np.diag(v - half_64(v)))


def muon_direction(g, momentum, mu, nesterov):
    """(new momentum, U)."""
    m = mu * momentum + g
    return m, g + mu * m if nesterov else m
