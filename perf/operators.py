"""Measured cases of the operators around the expert block, and their plain forms.

Four operators, each in the sizes that the block's own workloads give it:

* ``norm`` / ``norm_backward``: the RMS norms after and before a block, with the
  branch's gate and the residual scale in between, and the gradients;
* ``experts_w4``: the routed and shared experts of a decode batch on 4-bit
  weights with group scales;
* ``quantize_w4``: a weight matrix into that 4-bit form and back;
* ``orthogonalize``: Newton-Schulz products over a stack of expert gradients,
  bare or as the whole Muon update of momentum and weights.

``run`` is one pass: torch's elementary operations in 32 bits where ``own`` is
false, this repository's entry points where it is true. ``exact`` is the same
from the definitions, in 64 bits.
"""
import math

import torch

own = False

NS_STEPS = 5
NS_COEFFS = (3.4445, -4.7750, 2.0315)
NORM_EPS = 1e-6
NS_EPS = 1e-7


# ------------------------------------------------------------------- cases
def _norm(name, T, d, dtype, gate_tokens, alpha, backward=False):
    """gate_tokens: tokens that share one gate row; 0: no gate."""
    return {"name": name, "op": "norm_backward" if backward else "norm", "T": T, "d": d, "dtype": dtype,
            "gate_tokens": gate_tokens, "alpha": alpha}


def _experts(name, T, d, E, k, f, f_shared, group, zeros):
    return {"name": name, "op": "experts_w4", "T": T, "d": d, "E": E, "k": k, "f": f, "f_shared": f_shared,
            "group": group, "zeros": zeros}


def _quant(name, rows, K, dtype, group, zeros):
    return {"name": name, "op": "quantize_w4", "rows": rows, "K": K, "dtype": dtype, "group": group, "zeros": zeros}


def _ortho(name, n, rows, cols, dtype, step):
    """step: the whole Muon update, else the bare orthogonalisation."""
    return {"name": name, "op": "orthogonalize", "n": n, "rows": rows, "cols": cols, "dtype": dtype, "step": step}


def listed():
    return [
        # One decode step of the fine-grained layer: 32 tokens, latency counts.
        _norm("norm decode 32x2048", 32, 2048, "bf16", 0, 1.0),
        # A prompt through the DeepSeek-V3-shaped layer, one learned gate per channel.
        _norm("norm prompt 4096x7168", 4096, 7168, "bf16", 4096, 1.0),
        # The same batch's backward pass, the gate conditioned on sequences of 512 tokens.
        _norm("norm backward 4096x7168", 4096, 7168, "bf16", 512, 1.0, True),
        # fp32 parity training: an odd batch, a width off every tile, ragged last gate.
        _norm("norm backward fp32 1111x1000", 1111, 1000, "f32", 37, 0.9, True),
        # A single sequence's decode step: eight experts, one row each.
        _experts("experts w4 1 token", 1, 2048, 128, 8, 768, 0, 128, False),
        # The decode workload: 32 tokens over 128 fine-grained experts.
        _experts("experts w4 decode", 32, 2048, 128, 8, 768, 0, 128, False),
        # DeepSeek-V3 widths with the shared expert, an eighth of the experts; AWQ-like zero points.
        _experts("experts w4 wide", 24, 7168, 32, 8, 2048, 2048, 64, True),
        # Quantising eight DeepSeek-V3 gate matrices at load time.
        _quant("quantize w4 16384x7168", 16384, 7168, "bf16", 128, False),
        # A small fp32 layer, an odd number of rows.
        _quant("quantize w4 fp32 1001x416", 1001, 416, "f32", 32, True),
        # The tiny fp32 layer's eight experts: launch latency counts.
        _ortho("orthogonalize 8x256x128", 8, 256, 128, "f32", False),
        # A Muon step on eight experts' gate matrices at DeepSeek-V3 widths.
        _ortho("muon 8x2048x7168", 8, 2048, 7168, "bf16", True),
        # Two Mixtral-shaped gate matrices, taller than wide.
        _ortho("orthogonalize 2x14336x4096", 2, 14336, 4096, "bf16", False),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def _ortho_flops(n, rows, cols):
    m, c = min(rows, cols), max(rows, cols)
    return NS_STEPS * n * (3.0 * m * m * c + 1.0 * m * m * m)


def draw(rng):
    op = rng.choice(["norm", "norm_backward", "experts_w4", "quantize_w4", "orthogonalize"])
    if op in ("norm", "norm_backward"):
        T, d = _log_int(rng, 1, 4096), _log_int(rng, 64, 7168, 8)
        dtype = rng.choice(["bf16", "f32"])
        if dtype == "f32":
            T = min(T, 2048)
        gate = rng.choice([0, 1, T, rng.randint(1, T)])
        c = _norm("", T, d, dtype, gate, rng.choice([1.0, 0.5, 1.25]), op == "norm_backward")
    elif op == "experts_w4":
        group = rng.choice([32, 64, 128])
        E = rng.choice([8, 16, 32, 64, 128])
        d, f = _log_int(rng, 256, 4096, 128), _log_int(rng, 128, 1536, 128)
        c = _experts("", _log_int(rng, 1, 128), d, E, rng.randint(1, 8), f,
                     rng.choice([0, 0, _log_int(rng, 128, 1024, 128)]), group, rng.random() < 0.5)
    elif op == "quantize_w4":
        group = rng.choice([32, 64, 128])
        c = _quant("", _log_int(rng, 1, 8192), group * _log_int(rng, 1, 4096 // group), rng.choice(["bf16", "f32"]),
                   group, rng.random() < 0.5)
    else:
        n, rows, cols = rng.randint(1, 8), _log_int(rng, 8, 4096), _log_int(rng, 8, 4096)
        c = _ortho("", n, rows, cols, rng.choice(["bf16", "f32"]), rng.random() < 0.5)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs
def _dt(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def _gates(case):
    return -(-case["T"] // case["gate_tokens"]) if case["gate_tokens"] else 0


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*shape, std=1.0, dtype=torch.float32):
        return torch.randn(shape, generator=g, device="cuda").mul_(std).to(dtype)

    def rand(*shape):
        return torch.rand(shape, generator=g, device="cuda")

    s = {"case": case}
    op = case["op"]
    if op in ("norm", "norm_backward"):
        T, d, dt = case["T"], case["d"], _dt(case)
        # Residual streams spread over orders of magnitude from token to token.
        size = torch.exp(randn(T, 1))
        s["h"] = (randn(T, d) * size).to(dt)
        s["y"] = (randn(T, d) * 0.3 * torch.exp(randn(T, 1))).to(dt)
        s["w_post"] = (1 + randn(d, std=0.2)).to(dt)
        s["w_pre"] = (1 + randn(d, std=0.2)).to(dt)
        s["gate"] = randn(_gates(case), d, std=0.5, dtype=dt) if case["gate_tokens"] else None
        if op == "norm":
            s["out"] = [torch.empty_like(s["h"]) for _ in range(2)]                 # h_out, u
        else:
            s["du"], s["dh_out"] = randn(T, d, dtype=dt), randn(T, d, dtype=dt)
            s["out"] = [torch.empty_like(s["h"]) for _ in range(2)]                 # dh, dy
            s["dw"] = [torch.empty_like(s["w_pre"]) for _ in range(2)]              # dw_post, dw_pre
            s["dgate"] = torch.empty_like(s["gate"]) if s["gate"] is not None else None
    elif op == "experts_w4":
        T, d, E, k, f, fs, G = (case[n] for n in ("T", "d", "E", "k", "f", "f_shared", "group"))

        def w4(*shape):
            rows, K = shape[:-1], shape[-1]
            q = torch.randint(0, 256, (*rows, K // 2), generator=g, device="cuda", dtype=torch.uint8)
            # Codes spread over +-7.5 steps: a step that gives weights of variance 1/K.
            scale = ((0.5 + rand(*rows, K // G)) / (4.6 * math.sqrt(K))).to(torch.bfloat16)
            z = torch.randint(5, 11, (*rows, K // G), generator=g, device="cuda", dtype=torch.uint8) \
                if case["zeros"] else None
            return q, scale, z

        s["x"] = randn(T, d, dtype=torch.bfloat16)
        s["w"] = [w4(E, f, d), w4(E, f, d), w4(E, d, f)]
        s["ws"] = [w4(fs, d), w4(fs, d), w4(d, fs)] if fs else None
        # The routing that moe_route and moe_permute leave behind.
        idx = (rand(T, E) + 0.3 * rand(E)).topk(k, dim=1).indices.sort(dim=1).values
        flat = idx.reshape(-1)
        order = torch.argsort(flat, stable=True)
        s["perm_src"] = (order // k).to(torch.int32)
        counts = torch.bincount(flat, minlength=E)
        s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        s["out"] = [torch.empty(T * k, d, device="cuda", dtype=torch.bfloat16),
                    torch.empty(T, d, device="cuda", dtype=torch.bfloat16) if fs else None]
    elif op == "quantize_w4":
        rows, K, G = case["rows"], case["K"], case["group"]
        s["w"] = (randn(rows, K) * torch.exp(0.5 * randn(rows, 1)) / math.sqrt(K)
                  + (0.5 / math.sqrt(K) if case["zeros"] else 0.0)).to(_dt(case))
        s["q"] = torch.empty(rows, K // 2, device="cuda", dtype=torch.uint8)
        s["scale"] = torch.empty(rows, K // G, device="cuda", dtype=torch.bfloat16)
        s["zero"] = torch.empty(rows, K // G, device="cuda", dtype=torch.uint8) if case["zeros"] else None
        s["back"] = torch.empty_like(s["w"])
    else:
        n, rows, cols = case["n"], case["rows"], case["cols"]
        # A gradient's spectrum: noise over rows and columns of different
        # sizes, and one direction that stands out.
        grad = randn(n, rows, cols) * torch.exp(0.3 * randn(n, rows, 1)) * torch.exp(0.3 * randn(n, 1, cols))
        grad += 2.0 * randn(n, rows, 1) * randn(n, 1, cols)
        s["g"] = grad.mul_(1e-3).to(_dt(case))
        if case["step"]:
            s["momentum"] = randn(n, rows, cols, std=2e-3)
            s["weight"] = randn(n, rows, cols, std=1.0 / math.sqrt(cols), dtype=torch.bfloat16)
            s["lr"], s["mu"], s["decay"] = 0.02, 0.95, 0.01
            s["scale"] = math.sqrt(max(1.0, rows / cols))
        else:
            s["o"] = torch.empty(n, rows, cols, device="cuda", dtype=torch.bfloat16)
    return s


# ------------------------------------------------- this repository's calls
def _own(s):
    from mixture_experts_ffn_sigmoid_b200 import binding as B

    case, op = s["case"], s["case"]["op"]
    if "cfg" not in s:   # what a user's program builds once and keeps
        if op in ("norm", "norm_backward"):
            s["cfg"] = B.make_norm_config(T=case["T"], d=case["d"], dtype=case["dtype"],
                                          gate_tokens=max(1, case["gate_tokens"]), eps=NORM_EPS, alpha=case["alpha"],
                                          beta=0.8, w_offset=0.0)
            if op == "norm_backward":
                s["workspace"] = B.alloc_norm_backward_workspace(s["cfg"])
        elif op == "experts_w4":
            from mixture_experts_ffn_sigmoid_b200.inputs import MoEConfig
            s["cfg"] = B.make_config(MoEConfig("w4", T=case["T"], d=case["d"], E=case["E"], k=case["k"], f=case["f"],
                                               f_shared=case["f_shared"]))
            s["workspace"] = B.alloc_workspace(s["cfg"])
            s["w4"] = [B.W4Matrix(*m, group=case["group"]) for m in s["w"]]
            s["ws4"] = [B.W4Matrix(*m, group=case["group"]) for m in s["ws"]] if s["ws"] else [None] * 3
        elif op == "quantize_w4":
            s["cfg"] = B.W4Matrix(s["q"], s["scale"], s["zero"], group=case["group"])
        else:
            s["cfg"] = B.make_ortho_config(n=case["n"], rows=case["rows"], cols=case["cols"], dtype=case["dtype"],
                                           steps=NS_STEPS, eps=NS_EPS)
            s["workspace"] = B.alloc_ortho_workspace(s["cfg"])
    if op == "norm":
        B.moe_residual_norm(s["cfg"], s["h"], s["y"], s["w_post"], s["gate"], s["w_pre"], *s["out"])
        return s["out"]
    if op == "norm_backward":
        B.moe_residual_norm_backward(s["cfg"], s["h"], s["y"], s["w_post"], s["gate"], s["w_pre"], s["du"],
                                     s["dh_out"], *s["out"], s["dw"][0], s["dgate"], s["dw"][1], s["workspace"])
        return [*s["out"], s["dw"][0], s["dgate"], s["dw"][1]]
    if op == "experts_w4":
        B.moe_expert_swiglu_w4(s["cfg"], s["x"], s["perm_src"], s["offsets"], *s["w4"],
                               s["x"] if s["ws"] else None, *s["ws4"], *s["out"], s["workspace"])
        return s["out"]
    if op == "quantize_w4":
        B.moe_w4_quantize(s["w"], s["cfg"])
        B.moe_w4_dequantize(s["cfg"], s["back"])
        return [s["back"], s["scale"]]
    if case["step"]:
        B.moe_muon_step(s["cfg"], s["g"], s["momentum"], s["weight"], s["workspace"], lr=s["lr"], mu=s["mu"],
                        nesterov=True, weight_decay=s["decay"], scale=s["scale"])
        return [s["momentum"], s["weight"]]
    B.moe_orthogonalize(s["cfg"], s["g"], s["o"], s["workspace"])
    return s["o"]


# -------------------------------------------------------------- plain forms
def _rms(v):
    return torch.rsqrt(v.square().mean(dim=-1, keepdim=True) + NORM_EPS)


def _gate_rows(s, v):
    """The gate's row of every token, in v's type."""
    case = s["case"]
    if s["gate"] is None:
        return torch.ones((), device="cuda", dtype=v)
    return s["gate"].to(v).repeat_interleave(case["gate_tokens"], dim=0)[:case["T"]]


def _plain_norm(s):
    dt, f = s["h"].dtype, torch.float32
    y = s["y"].to(f)
    h = s["case"]["alpha"] * s["h"].to(f) + 0.8 * _gate_rows(s, f) * (y * _rms(y) * s["w_post"].to(f))
    return [h.to(dt), (h * _rms(h) * s["w_pre"].to(f)).to(dt)]


def _plain_norm_backward(s):
    case, dt, f = s["case"], s["h"].dtype, torch.float32
    h, y, du, gate = s["h"].to(f), s["y"].to(f), s["du"].to(f), _gate_rows(s, f)
    rh, ry = _rms(h), _rms(y)
    nh, ny = h * rh, y * ry
    dn = du * s["w_pre"].to(f)
    dH = s["dh_out"].to(f) + rh * (dn - nh * (dn * nh).mean(dim=-1, keepdim=True))
    dz = 0.8 * gate * dH
    dm = dz * s["w_post"].to(f)
    dy = ry * (dm - ny * (dm * ny).mean(dim=-1, keepdim=True))
    dgate = None
    if s["gate"] is not None:
        per = 0.8 * dH * ny * s["w_post"].to(f)
        per = torch.cat([per, per.new_zeros(_gates(case) * case["gate_tokens"] - case["T"], case["d"])])
        dgate = per.view(_gates(case), case["gate_tokens"], case["d"]).sum(dim=1).to(dt)
    return [(case["alpha"] * dH).to(dt), dy.to(dt), (dz * ny).sum(dim=0).to(dt), dgate, (du * nh).sum(dim=0).to(dt)]


def _plain_dense(m, group):
    q, scale, zero = m
    codes = torch.stack([q & 15, q >> 4], dim=-1).flatten(-2).float()
    codes = codes.unflatten(-1, (-1, group))
    z = 8.0 if zero is None else zero.float().unsqueeze(-1)
    return ((codes - z) * scale.float().unsqueeze(-1)).flatten(-2)


def _plain_ffn(x, w, group):
    """x [..., T, d] through every expert of w: [..., T, d]."""
    a = x @ _plain_dense(w[0], group).transpose(-1, -2)
    b = x @ _plain_dense(w[1], group).transpose(-1, -2)
    return (a * torch.sigmoid(a) * b) @ _plain_dense(w[2], group).transpose(-1, -2)


def _plain_experts(s):
    case = s["case"]
    x, src = s["x"].float(), s["perm_src"].long()
    row = torch.arange(case["T"] * case["k"], device="cuda", dtype=torch.int32)
    expert = torch.searchsorted(s["offsets"][1:], row, right=True)
    if case["T"] * case["k"] < case["E"]:   # few rows: each with its expert's weights
        w = [[None if t is None else t[expert] for t in m] for m in s["w"]]
        y_perm = _plain_ffn(x[src].unsqueeze(1), w, case["group"]).squeeze(1)
    else:                                   # every token through every expert
        y_perm = _plain_ffn(x, s["w"], case["group"])[expert, src]
    return [y_perm.to(torch.bfloat16), _plain_ffn(x, s["ws"], case["group"]).to(torch.bfloat16) if s["ws"] else None]


def _plain_quantize(s):
    case = s["case"]
    w = s["w"].float().unflatten(-1, (-1, case["group"]))
    if case["zeros"]:
        lo, hi = w.amin(-1, keepdim=True).clamp(max=0), w.amax(-1, keepdim=True).clamp(min=0)
        scale = ((hi - lo) / 15.0).to(torch.bfloat16)
        step = torch.where(scale > 0, scale.float(), 1.0)
        zero = torch.round(-lo / step).clamp(0, 15)
    else:
        scale = (w.abs().amax(-1, keepdim=True) / 7.0).to(torch.bfloat16)
        step = torch.where(scale > 0, scale.float(), 1.0)
        zero = 8.0
    code = (torch.round(w / step) + zero).clamp(0, 15)
    return [((code - zero) * scale.float()).flatten(-2).to(s["w"].dtype), scale.squeeze(-1)]


def _plain_newton_schulz(u):
    a, b, c = NS_COEFFS
    tall = u.shape[1] > u.shape[2]
    x = u.transpose(1, 2) if tall else u
    x = x / (x.square().sum(dim=(1, 2), keepdim=True).sqrt() + NS_EPS)
    for _ in range(NS_STEPS):
        p = x @ x.transpose(1, 2)
        x = a * x + (b * p + c * (p @ p)) @ x
    return x.transpose(1, 2) if tall else x


def _plain_orthogonalize(s):
    if not s["case"]["step"]:
        return _plain_newton_schulz(s["g"].float()).to(torch.bfloat16)
    g = s["g"].float()
    s["momentum"].mul_(s["mu"]).add_(g)
    o = _plain_newton_schulz(g + s["mu"] * s["momentum"])
    w = s["weight"].float() * (1 - s["lr"] * s["decay"]) - s["lr"] * s["scale"] * o
    s["weight"].copy_(w)
    return [s["momentum"], s["weight"]]


PLAIN = {"norm": _plain_norm, "norm_backward": _plain_norm_backward, "experts_w4": _plain_experts,
         "quantize_w4": _plain_quantize, "orthogonalize": _plain_orthogonalize}


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["case"]["op"]](state)


# --------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op in ("norm", "norm_backward"):
        T, d, es = case["T"], case["d"], 4 if case["dtype"] == "f32" else 2
        small = (2 + _gates(case)) * d * es
        if op == "norm":            # reads h, y; writes h_out, u
            return {"bytes": 4 * T * d * es + small, "flops": 12.0 * T * d}
        return {"bytes": 6 * T * d * es + 2 * small, "flops": 30.0 * T * d}
    if op == "experts_w4":
        T, d, E, k, f, fs, G = (case[n] for n in ("T", "d", "E", "k", "f", "f_shared", "group"))
        touched = E * (1.0 - (1.0 - k / E) ** T)   # expected over uniform routing
        weights = 3.0 * d * f * touched + 3.0 * d * fs
        per = 0.5 + (3.0 if case["zeros"] else 2.0) / G
        rows = T * k + (T if fs else 0)
        return {"bytes": weights * per + 2.0 * T * d + 2.0 * rows * d + 4.0 * (T * k + E + 1),
                "flops": 6.0 * d * (T * k * f + T * fs)}
    if op == "quantize_w4":
        n, es = case["rows"] * case["K"], 4 if case["dtype"] == "f32" else 2
        packed = n * (0.5 + (3.0 if case["zeros"] else 2.0) / case["group"])
        return {"bytes": 2.0 * n * es + 2.0 * packed, "flops": 6.0 * n}
    n, r, c = case["n"], case["rows"], case["cols"]
    es = 4 if case["dtype"] == "f32" else 2
    moved = n * r * c * (es + (8 + 4 if case["step"] else 2))
    # Both squares are symmetric: half of each, and the full last product.
    return {"bytes": float(moved), "flops": _ortho_flops(n, r, c)}


# -------------------------------------------------------------------- exact
def exact(case, seed):
    s = prepare(case, seed)
    op, D = case["op"], torch.float64
    if op in ("norm", "norm_backward"):
        T, d = case["T"], case["d"]
        h, y, wp, wn = (s[n].to(D) for n in ("h", "y", "w_post", "w_pre"))
        rows = torch.arange(T, device="cuda") // max(1, case["gate_tokens"])
        c = 0.8 * (s["gate"].to(D)[rows] if s["gate"] is not None else torch.ones(T, d, device="cuda", dtype=D))
        sy = ((y * y).sum(1, keepdim=True) / d + NORM_EPS).sqrt()
        z = y / sy
        if op == "norm":
            out = case["alpha"] * h + c * z * wp
            return [out, out / ((out * out).sum(1, keepdim=True) / d + NORM_EPS).sqrt() * wn]
        # d(v / s)_j = dv_j / s - v_j (v . dv) / (d s^3)
        sh = ((h * h).sum(1, keepdim=True) / d + NORM_EPS).sqrt()
        du, q = s["du"].to(D), s["du"].to(D) * wn
        total = s["dh_out"].to(D) + q / sh - h * (h * q).sum(1, keepdim=True) / (d * sh ** 3)
        p = total * c * wp
        dy = p / sy - y * (y * p).sum(1, keepdim=True) / (d * sy ** 3)
        dgate = None
        if s["gate"] is not None:
            dgate = torch.zeros(_gates(case), d, device="cuda", dtype=D).index_add_(0, rows, 0.8 * total * z * wp)
        return [case["alpha"] * total, dy, (total * c * z).sum(0), dgate, (du * h / sh).sum(0)]
    if op == "experts_w4":
        G = case["group"]

        def dense(m):
            q, scale, zero = m
            w = torch.empty(*q.shape[:-1], 2 * q.shape[-1], device="cuda", dtype=D)
            w[..., 0::2], w[..., 1::2] = q.bitwise_and(15).to(D), q.bitwise_right_shift(4).to(D)
            w -= 8 if zero is None else zero.to(D).repeat_interleave(G, dim=-1)
            return w.mul_(scale.to(D).repeat_interleave(G, dim=-1))

        def ffn(x, w1, w3, w2):
            a, b = x @ w1.T, x @ w3.T
            return (a / (1 + torch.exp(-a)) * b) @ w2.T

        x, off = s["x"].to(D), s["offsets"].tolist()
        xp = x[s["perm_src"].long()]
        y = torch.empty(case["T"] * case["k"], case["d"], device="cuda", dtype=D)
        for e in range(case["E"]):
            if off[e] < off[e + 1]:
                one = [dense(tuple(None if t is None else t[e] for t in m)) for m in s["w"]]
                y[off[e]:off[e + 1]] = ffn(xp[off[e]:off[e + 1]], *one)
        return [y, ffn(x, *[dense(m) for m in s["ws"]]) if s["ws"] else None]
    if op == "quantize_w4":
        # Which code a weight next to a border takes is the 32-bit division's
        # and the scale's rounding's to say: no value of its own in 64 bits.
        return None
    u = s["g"].to(D)
    m = None
    if case["step"]:
        m = s["mu"] * s["momentum"].to(D) + u
        u = u + s["mu"] * m
    a, b, c = NS_COEFFS
    x = u / (torch.linalg.vector_norm(u, dim=(1, 2), keepdim=True) + NS_EPS)
    small = x.shape[1] <= x.shape[2]
    for _ in range(NS_STEPS):
        gram = torch.einsum("nij,nkj->nik", x, x) if small else torch.einsum("nji,njk->nik", x, x)
        poly = b * gram + c * torch.einsum("nij,njk->nik", gram, gram)
        poly.diagonal(dim1=1, dim2=2).add_(a)
        x = torch.einsum("nij,njk->nik", poly, x) if small else torch.einsum("nij,njk->nik", x, poly)
    if not case["step"]:
        return x
    return [m, (1 - s["lr"] * s["decay"]) * s["weight"].to(D) - s["lr"] * s["scale"] * x]
