"""Offsets past 31 and 32 bits: the last rows, experts and matrices of large
arrays against a call on them alone, which the other tests hold to the oracle."""
import pytest
import torch

from mixture_experts_ffn_sigmoid_b200 import binding as B
from mixture_experts_ffn_sigmoid_b200.inputs import MoEConfig, NormConfig, OrthoConfig

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(autouse=True)
def freed():
    yield
    torch.cuda.empty_cache()


def noise(seed, *shape, dtype=BF):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda", dtype=dtype)


def test_norm_and_backward():
    T, d, n = 330_000, 7168, 9                                  # 2.4e9 elements
    cfg, one = NormConfig(T=T, d=d, gate_tokens=T), NormConfig(T=n, d=d, gate_tokens=n)
    w, gate = 1 + 0.1 * noise(1, d), noise(2, 1, d)
    h, y = noise(3, T, d), noise(4, T, d)
    hs, ys = h[-n:].clone(), y[-n:].clone()
    want = [torch.empty_like(hs) for _ in range(2)]
    B.moe_residual_norm(one, hs, ys, w, gate, w, *want)
    B.moe_residual_norm(cfg, h, y, w, gate, w, h, y)            # in place
    assert torch.equal(h[-n:], want[0]) and torch.equal(y[-n:], want[1])
    du, dh = noise(5, T, d), noise(6, T, d)
    part = [t[-n:].clone() for t in (h, y, du, dh)]
    dws = torch.empty(d, device="cuda", dtype=BF)
    out = [torch.empty_like(part[0]) for _ in range(2)]
    B.moe_residual_norm_backward(one, part[0], part[1], w, gate, w, part[2], part[3], *out, dws, None, None,
                                 B.alloc_norm_backward_workspace(one))
    B.moe_residual_norm_backward(cfg, h, y, w, gate, w, du, dh, dh, du, dws, None, None,
                                 B.alloc_norm_backward_workspace(cfg))
    assert torch.equal(dh[-n:], out[0]) and torch.equal(du[-n:], out[1])


def test_quantize_and_back():
    rows, K = 270_000, 16384                                    # 4.4e9 weights
    w = noise(7, rows, K)
    m = B.W4Matrix.quantize(w, 128, True)
    last = B.W4Matrix.quantize(w[-3:].contiguous(), 128, True)
    for a, b in ((m.q, last.q), (m.scale, last.scale), (m.zero, last.zero)):
        assert torch.equal(a[-3:], b)
    B.moe_w4_dequantize(m, w)
    back = torch.empty(3, K, device="cuda", dtype=BF)
    B.moe_w4_dequantize(last, back)
    assert torch.equal(w[-3:], back)


def test_experts_w4():
    E, d, f, T, k = 160, 16384, 2048, 6, 2                      # 2.7e9 bytes of codes a matrix
    g = torch.Generator(device="cuda").manual_seed(8)

    def w4(*s):
        q = torch.randint(0, 256, (*s[:-1], s[-1] // 2), generator=g, device="cuda", dtype=torch.uint8)
        sc = ((0.5 + torch.rand(*s[:-1], s[-1] // 64, generator=g, device="cuda")) / (4.6 * s[-1] ** 0.5)).to(BF)
        return B.W4Matrix(q, sc, None, 64)

    w = [w4(E, f, d), w4(E, f, d), w4(E, d, f)]
    tail = [B.W4Matrix(m.q[-2:].contiguous(), m.scale[-2:].contiguous(), None, 64) for m in w]
    x = noise(9, T, d)
    src = torch.arange(T * k, device="cuda", dtype=torch.int32) % T
    out = []
    for n, ws in ((E, w), (2, tail)):
        cfg = MoEConfig("large", T=T, d=d, E=n, k=k, f=f)
        off = torch.zeros(n + 1, device="cuda", dtype=torch.int32)
        off[-2], off[-1] = 5, T * k                             # five rows for the last expert but one
        y, work = torch.full((T * k, d), float("nan"), device="cuda", dtype=BF), B.alloc_workspace(cfg)
        B.moe_expert_swiglu_w4(cfg, x, src, off, *ws, None, None, None, None, y, None, work)
        assert B.moe_get_device_error(work) == B.MOE_OK
        out.append(y)
    # The work is split differently: sums of the same terms in fp32, rounded to bf16 twice.
    assert torch.isfinite(out[0].float()).all()
    assert (out[0].float() - out[1].float()).norm() <= 2.0 ** -7 * out[1].float().norm()


def test_orthogonalize():
    n, m = 40, 8192                                             # 2.7e9 elements
    g = noise(10, n, m, m)
    cfg, one = OrthoConfig(n=n, rows=m, cols=m, steps=1), OrthoConfig(n=1, rows=m, cols=m, steps=1)
    o, last = torch.empty_like(g), torch.empty(1, m, m, device="cuda", dtype=BF)
    B.moe_orthogonalize(cfg, g, o, B.alloc_ortho_workspace(cfg))
    B.moe_orthogonalize(one, g[-1:], last, B.alloc_ortho_workspace(one))
    # fp16 roundings may turn where tiles are split differently: the bound of two such results.
    assert (o[-1:].float() - last.float()).norm() <= 2.0 ** -7 * last.float().norm()
