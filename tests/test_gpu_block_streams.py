"""MoEBlock and W4Matrix on a stream that is not torch's current one: what they
allocate belongs to that stream, so that neither side's work runs into memory
that the other still uses. The current stream is held up by a spin of some
milliseconds, or the block's stream is, so that the order in time is known."""
import pytest
import torch

from mixture_experts_ffn_sigmoid_b200 import binding as B
from mixture_experts_ffn_sigmoid_b200.inputs import GATE_SIGMOID, MoEConfig, NormConfig, make_inputs

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
SPIN = 50_000_000          # cycles: 25 ms or more


def layer(w4, T=48, d=1024):
    cfg = MoEConfig("streams", T=T, d=d, E=8, k=2, f=256, gate_mode=GATE_SIGMOID, bias="uniform")
    inp = make_inputs(cfg, "cuda", seed=4)
    if w4:
        inp.update({n: B.W4Matrix.quantize(inp[n], 64) for n in ("w1", "w3", "w2")})
    g = torch.Generator(device="cuda").manual_seed(6)
    w = [(1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(BF) for _ in range(2)]
    u = torch.randn(T, d, generator=g, device="cuda").to(BF)
    return B.MoEBlock(cfg, inp, "cuda"), inp["x"], u, NormConfig(T=T, d=d), w


@pytest.mark.parametrize("as_handle", [False, True])
@pytest.mark.parametrize("w4", [False, True])
def test_the_block_s_output_is_not_given_away_while_the_norm_reads_it(w4, as_handle, monkeypatch):
    block, h, u, norm, (wp, wn) = layer(w4)
    want = block.step(h, u, norm, wp, None, wn)
    torch.cuda.synchronize()
    seen = []
    run = B.moe_residual_norm

    def spy(cfg, h, y, *rest):
        seen.append((y.data_ptr(), y.numel() * y.element_size()))
        return run(cfg, h, y, *rest)

    monkeypatch.setattr(B, "moe_residual_norm", spy)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.empty_cache()                   # no spare blocks: the first free one is y's
    with torch.cuda.stream(side):
        torch.cuda._sleep(SPIN)
    got = block.step(h, u, norm, wp, None, wn, stream=side.cuda_stream if as_handle else side)
    new = [torch.full_like(h, float("nan")) for _ in range(4)]      # on the current stream, at once
    (at, size), = seen
    assert not any(t.data_ptr() < at + size and at < t.data_ptr() + size for t in new)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("call", ["step", "forward", "quantize"])
def test_results_do_not_land_in_memory_that_the_current_stream_still_reads(call):
    block, h, u, norm, (wp, wn) = layer(False)
    w = torch.randn(48, 4096, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda")
    side = torch.cuda.Stream()
    run = {"step": lambda: block.step(h, u, norm, wp, None, wn, stream=side),
           "forward": lambda: block.forward(u, stream=side),
           "quantize": lambda: B.W4Matrix.quantize(w, 64, stream=side)}[call]
    run()                                      # what is made once is made
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    old = [torch.full_like(h, 3.0) for _ in range(6)]
    kept = [torch.empty_like(h) for _ in range(6)]
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda._sleep(SPIN)
    for k, o in zip(kept, old):                # waits for the spin
        k.copy_(o)
    del o, old                                 # free for what the current stream does next
    out = run()
    torch.cuda.synchronize()
    assert all((k == 3.0).all() for k in kept)
    del out


def test_a_workspace_made_on_first_use_belongs_to_the_stream():
    block, h, u, norm, (wp, wn) = layer(False)
    size = B.workspace_size(B.make_config(block.cfg, 48))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    old, kept = torch.full((size,), 7, device="cuda", dtype=torch.uint8), torch.empty(size, device="cuda", dtype=torch.uint8)
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda._sleep(SPIN)
    kept.copy_(old)
    del old
    y = block.forward(u, stream=side)
    torch.cuda.synchronize()
    assert (kept == 7).all()
    assert torch.equal(y, block.forward(u))
