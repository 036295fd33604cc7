"""The gated block's training calls and its calls on 4-bit weights as a user's
program makes them, and their plain forms.

Kinds of case:

  train       swiglu_gated_mlp_train: the block, keeping Gate and Up
  mlp_back    swiglu_gated_mlp_backward: gradients of the whole block
  gated_back  swiglu_fused_gemm_backward: gradients of the SwiGLU stage
  down_back   swiglu_down_proj_backward: gradients of the down projection, the
              weight's in 32 bits and added to what earlier batches left
  mx4_gated   swiglu_fused_gemm_mx4: Gate and Up with 4-bit weights
  mx4_down    swiglu_down_proj_mx4: the down projection with 4-bit weights
  mx4_mlp     swiglu_gated_mlp_mx4: the block with 4-bit weights
  mx4_quant   swiglu_quantize_mx4, then swiglu_dequantize_mx4

4-bit weights: codes of 1 sign, 2 exponent and 1 mantissa bits, the even k in
a byte's low half, with one power of two (its exponent plus 127) for each group
of 32 consecutive k.

With ``own`` false, ``run`` computes them from elementary torch operations in
32 bits; with ``own`` true it calls the library.  ``exact`` computes them in 64
bits.  By definition the block's H and the gradient by Gate and Up are rounded
to bf16, and what follows them is computed from the rounded values.
"""
import math

import torch

own = False


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # a training step's forward pass over a small model's micro-batch
        {"name": "train_small", "kind": "train", "M": 512, "K": 896, "N": 4864},
        # the same over long sequences of a middling model
        {"name": "train_long", "kind": "train", "M": 8192, "K": 1536, "N": 8960},
        # the SwiGLU stage's gradients of a few tokens: a short, ragged sample
        {"name": "gated_back_few", "kind": "gated_back", "M": 33, "K": 896, "N": 4872},
        # the down projection's, the weight's summed over micro-batches
        {"name": "down_back_sum", "kind": "down_back", "M": 4099, "K": 1536, "N": 8960},
        # gradients of an ordinary micro-batch
        {"name": "mlp_back", "kind": "mlp_back", "M": 2048, "K": 1536, "N": 8960},
        # gradients of long sequences of a large model
        {"name": "mlp_back_long", "kind": "mlp_back", "M": 8192, "K": 5120, "N": 13824},
        # one token of one request
        {"name": "mx4_gated_one", "kind": "mx4_gated", "M": 1, "K": 3584, "N": 18944},
        # one token through a small model's block: latency
        {"name": "mx4_mlp_one", "kind": "mx4_mlp", "M": 1, "K": 896, "N": 4864},
        # one token each of some requests, through a large model's block
        {"name": "mx4_mlp_requests", "kind": "mx4_mlp", "M": 24, "K": 8192, "N": 29568},
        # a prompt
        {"name": "mx4_gated_prompt", "kind": "mx4_gated", "M": 2048, "K": 3584, "N": 18944},
        # laying out a weight once: a small model's, and an odd count of rows
        {"name": "mx4_quant", "kind": "mx4_quant", "M": 9728, "K": 896, "N": 0},
        {"name": "mx4_quant_odd", "kind": "mx4_quant", "M": 37889, "K": 3616, "N": 0},
    ]


def _spread(rng, low, high):
    """A whole number from low to high, even over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 1)))))))


KINDS = ("train", "mlp_back", "gated_back", "down_back", "mx4_gated", "mx4_down", "mx4_mlp",
         "mx4_quant")


def draw(rng):
    kind = rng.choice(KINDS)
    if kind == "mx4_quant":
        K = 32 * _spread(rng, 2, 256)
        return {"kind": kind, "M": _spread(rng, 1, (1 << 27) // K), "K": K, "N": 0}
    if kind.startswith("mx4"):
        K, N = 32 * _spread(rng, 16, 256), 32 * _spread(rng, 16, 600)
        most = 2048
    else:
        K, N = 8 * _spread(rng, 64, 1024), 8 * _spread(rng, 64, 2048)
        # the largest listed case multiplies and adds 6 * 8192 * 5120 * 13824 times
        most = 3 * 8192 * 5120 * 13824 // (6 * K * N)
    return {"kind": kind, "M": _spread(rng, 1, min(8192, most)), "K": K, "N": N}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
DEVICE = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16


def _normal(g, shape, std=1.0, dtype=BF16):
    return (torch.randn(shape, generator=g, device=DEVICE, dtype=F32) * std).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed))
    kind, M, K, N = case["kind"], case["M"], case["K"], case["N"]
    s = {"kind": kind}
    if kind == "mx4_quant":
        # rows of a weight differ in size
        rows = torch.exp(torch.randn(M, 1, generator=g, device=DEVICE))
        s["X"] = (torch.randn(M, K, generator=g, device=DEVICE) * rows / math.sqrt(K)).to(BF16)
        return s
    # the scratch that a user's program keeps for these calls
    s["workspace"] = torch.empty(128 << 20, dtype=torch.uint8, device=DEVICE)
    if kind.startswith("mx4"):
        s["X"] = _normal(g, (M, N if kind == "mx4_down" else K))
        if kind != "mx4_down":
            s["Wq"], s["Ws"] = _quantize(_normal(g, (2 * N, K), 1.0 / math.sqrt(K)))
        if kind != "mx4_gated":
            s["W3q"], s["W3s"] = _quantize(_normal(g, (K, N), 1.0 / math.sqrt(N)))
        return s
    if kind != "down_back":
        s["A"] = _normal(g, (M, K))
        s["W_fused"] = _normal(g, (2 * N, K), 1.0 / math.sqrt(K))
    if kind != "gated_back":
        s["W3t"] = _normal(g, (K, N), 1.0 / math.sqrt(N))
    if kind == "train":
        return s
    if kind != "down_back":
        # what a forward pass kept: Gate and Up are about normal
        s["GU"] = _normal(g, (M, 2 * N))
    if kind == "gated_back":
        s["dH"] = _normal(g, (M, N), 0.1)
        return s
    s["dOut"] = _normal(g, (M, K), 0.1)
    if kind == "mlp_back":
        gate, up = s["GU"][:, 0::2].float(), s["GU"][:, 1::2].float()
        s["H"] = (gate / (1.0 + torch.exp(-gate)) * up).to(BF16)
    else:
        s["H"] = _normal(g, (M, N), 0.5)
        s["sum"] = _normal(g, (K, N), 2.0, F32)
    return s


# ---------------------------------------------------------------------------
# plain forms: elementary torch operations in 32 bits, rounded once at the end
# ---------------------------------------------------------------------------
def _silu_parts(g):
    """SiLU and its derivative."""
    sig = 1.0 / (1.0 + torch.exp(-g))
    return g * sig, sig * (1.0 + g * (1.0 - sig))


def _plain_train(s):
    a, w = s["A"].float(), s["W_fused"].float()
    gu = a @ w.t()
    h = (_silu_parts(gu[:, 0::2])[0] * gu[:, 1::2]).to(BF16)
    out = (h.float() @ s["W3t"].float().t()).to(BF16)
    return out, h, gu.to(BF16)


def _plain_d_gu(dh, gu):
    """The gradient by Gate and Up, interleaved as they are, in bf16."""
    gu = gu.float()
    silu, slope = _silu_parts(gu[:, 0::2])
    return torch.stack((dh * gu[:, 1::2] * slope, dh * silu), dim=2).reshape(gu.shape).to(BF16)


def _plain_stage(dh, s):
    d_gu = _plain_d_gu(dh, s["GU"])
    d = d_gu.float()
    return (d @ s["W_fused"].float()).to(BF16), (d.t() @ s["A"].float()).to(BF16), d_gu


def _plain_backward(s):
    if s["kind"] == "gated_back":
        return _plain_stage(s["dH"].float(), s)
    d_out = s["dOut"].float()
    dh = d_out @ s["W3t"].float()
    dw3 = d_out.t() @ s["H"].float()
    if s["kind"] == "down_back":
        return dh.to(BF16), dw3 + s["sum"]
    da, dw, d_gu = _plain_stage(dh, s)
    return da, dw, dw3.to(BF16), d_gu


def _power(n):
    """2^n in 64 bits for whole n, from its exponent bits."""
    return ((n.to(torch.int64) + 1023) << 52).view(torch.float64)


def _quantize(x):
    """Codes [rows, K / 2] and scales [rows, K / 32] of bf16 x: the largest
    magnitude of a group lies in [4, 8) of its scale (from the exponent bits;
    groups of tiny values keep scale 0), nearest code, ties to the even one."""
    rows, k = x.shape
    bits = x.contiguous().view(torch.int16).to(torch.int32) & 0x7FFF
    exponent = (bits.view(rows, k // 32, 32).max(dim=2).values >> 7)
    scale = torch.where(exponent == 255, exponent, (exponent - 2).clamp(min=0))
    v = x.double().view(rows, k // 32, 32).abs() * _power(127 - scale)[:, :, None]
    # borders between neighbouring codes; a tie goes to the even code
    code = torch.zeros(v.shape, dtype=torch.uint8, device=x.device)
    for n, (border, tie_up) in enumerate(((0.25, False), (0.75, True), (1.25, False), (1.75, True),
                                          (2.5, False), (3.5, True), (5.0, False))):
        code += (v >= border if tie_up else v > border).to(torch.uint8)
    code |= (x.view(rows, k // 32, 32).view(torch.int16) < 0).to(torch.uint8) << 3
    code[scale == 255] = 0
    code = code.view(rows, k)
    return code[:, 0::2] | (code[:, 1::2] << 4), scale.to(torch.uint8)


def _values(q, s):
    """The numbers that codes and scales stand for."""
    rows, half = q.shape
    code = torch.stack((q & 15, q >> 4), dim=2).view(rows, 2 * half)
    e, m = ((code >> 1) & 3).float(), (code & 1).float()
    v = torch.where(e == 0, m * 0.5, torch.where(e == 1, 1.0, torch.where(e == 2, 2.0, 4.0)) * (1.0 + m * 0.5))
    v = torch.where(code >= 8, -v, v).view(rows, half // 16, 32)
    size = torch.where(s == 255, float("nan"), _power(s.to(torch.int64) - 127))
    return (v * size[:, :, None]).float().view(rows, 2 * half)


def _plain_mx4(s):
    kind = s["kind"]
    if kind == "mx4_quant":
        q, sc = _quantize(s["X"])
        return _values(q, sc).to(BF16), sc
    h = s["X"].float()
    if kind != "mx4_down":
        gu = h @ _values(s["Wq"], s["Ws"]).t()
        h = (_silu_parts(gu[:, 0::2])[0] * gu[:, 1::2]).to(BF16)
        if kind == "mx4_gated":
            return h
    out = (h.float() @ _values(s["W3q"], s["W3s"]).t()).to(BF16)
    return out if kind == "mx4_down" else (out, h)


def _plain(s):
    if s["kind"] == "train":
        return _plain_train(s)
    return _plain_mx4(s) if s["kind"].startswith("mx4") else _plain_backward(s)


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------
def _own(s):
    from gated_mlp_gemm_amd import swiglu as sw
    kind, ws = s["kind"], s.get("workspace")
    if kind == "train":
        return sw.swiglu_gated_mlp_train(s["A"], s["W_fused"], s["W3t"], workspace=ws)
    if kind == "mlp_back":
        return sw.swiglu_gated_mlp_backward(s["dOut"], s["A"], s["W_fused"], s["W3t"], s["H"],
                                            s["GU"], workspace=ws)
    if kind == "gated_back":
        return sw.swiglu_fused_gemm_backward(s["dH"], s["A"], s["W_fused"], s["GU"], workspace=ws)
    if kind == "down_back":
        return sw.swiglu_down_proj_backward(s["dOut"], s["H"], s["W3t"], dW3t_add=s["sum"],
                                            workspace=ws)
    if kind == "mx4_gated":
        return sw.swiglu_fused_gemm_mx4(s["X"], s["Wq"], s["Ws"], workspace=ws)
    if kind == "mx4_down":
        return sw.swiglu_down_proj_mx4(s["X"], s["W3q"], s["W3s"], workspace=ws)
    if kind == "mx4_mlp":
        return sw.swiglu_gated_mlp_mx4(s["X"], s["Wq"], s["Ws"], s["W3q"], s["W3s"], workspace=ws)
    q, sc = sw.swiglu_quantize_mx4(s["X"])
    return sw.swiglu_dequantize_mx4(q, sc), sc


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    kind, M, K, N = case["kind"], case["M"], case["K"], case["N"]
    if kind == "mx4_quant":
        # codes and scales written; they are read again for the values in the same pass
        return {"bytes": M * K * 4 + M * K // 32, "flops": 4 * M * K}
    wide, narrow, product = 2 * M * N, 2 * M * K, 2 * M * N * K
    if kind.startswith("mx4"):
        weight = K * N * 17 // 32                     # of one K x N matrix: 4 bits, 8 a group
        parts = {"mx4_gated": 2, "mx4_down": 1, "mx4_mlp": 3}[kind]
        rows = narrow + wide + (narrow if kind == "mx4_mlp" else 0)
        return {"bytes": parts * weight + rows, "flops": parts * product}
    weight = 2 * K * N
    if kind == "train":
        return {"bytes": 3 * weight + 2 * narrow + 3 * wide, "flops": 3 * product}
    if kind == "mlp_back":
        # dOut, A, weights, H, GU; dA, the weights' gradients, the gradient by GU
        return {"bytes": 6 * weight + 3 * narrow + 5 * wide, "flops": 6 * product}
    if kind == "gated_back":
        return {"bytes": 4 * weight + 2 * narrow + 5 * wide, "flops": 4 * product}
    return {"bytes": weight + 8 * K * N + narrow + 2 * wide, "flops": 2 * product}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def _exact_swiglu(x, w_gate, w_up):
    gate, up = x @ w_gate.t(), x @ w_up.t()
    return gate, up, gate * torch.sigmoid(gate) * up


def _exact_d_gu(dh, gu):
    gu = gu.double()
    gate, up = gu[:, 0::2], gu[:, 1::2]
    sig = torch.sigmoid(gate)
    d = torch.empty_like(gu)
    d[:, 0::2] = dh * up * (sig + gate * sig * torch.sigmoid(-gate))
    d[:, 1::2] = dh * gate * sig
    return d


LADDER = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _sizes(device):
    """What each scale stands for."""
    return torch.tensor([2.0 ** (n - 127) for n in range(255)] + [math.nan], dtype=torch.float64,
                        device=device)


def _exact_weight(q, s):
    """[rows, K] in 64 bits, by a table of the sixteen codes."""
    table = torch.tensor(LADDER + tuple(-v for v in LADDER), dtype=torch.float64, device=q.device)
    out = torch.empty(q.shape[0], 2 * q.shape[1], dtype=torch.float64, device=q.device)
    out[:, 0::2] = table[(q % 16).int()]
    out[:, 1::2] = table[(q // 16).int()]
    size = _sizes(q.device)[s.int()]
    return out * torch.repeat_interleave(size, 32, dim=1)


def _exact_quantized(x):
    """The value nearest to each number on its group's ladder, and the scales."""
    rows, k = x.shape
    v = x.double().view(rows, -1, 32)
    top = v.abs().amax(dim=2)
    _, e = torch.frexp(top)                                       # top in [2^(e-1), 2^e)
    scale = torch.where(top > 0, e - 1 - 2 + 127, 0).clamp(min=0)
    size = _sizes(x.device)[scale]
    ladder = torch.tensor(LADDER, dtype=torch.float64, device=x.device)
    u = v.abs() / size[:, :, None]
    below = torch.searchsorted(ladder, u.contiguous(), right=True) - 1
    above = (below + 1).clamp(max=7)
    low, high = u - ladder[below], ladder[above] - u
    up = (above > below) & ((high < low) | ((high == low) & (above % 2 == 0)))
    code = torch.where(up, above, below)
    return (torch.sign(v) * ladder[code] * size[:, :, None]).view(rows, k), scale.to(torch.uint8)


def exact(case, seed):
    s = prepare(case, seed)
    kind = s["kind"]
    if kind == "mx4_quant":
        return _exact_quantized(s["X"])
    if kind == "train":
        w = s["W_fused"].double()
        gate, up, h = _exact_swiglu(s["A"].double(), w[0::2], w[1::2])
        out = h.to(BF16).double() @ s["W3t"].double().t()
        return out, h, torch.stack((gate, up), dim=2).view(h.shape[0], -1)
    if kind.startswith("mx4"):
        x = s["X"].double()
        if kind == "mx4_down":
            return x @ _exact_weight(s["W3q"], s["W3s"]).t()
        w = _exact_weight(s["Wq"], s["Ws"])
        h = _exact_swiglu(x, w[0::2], w[1::2])[2]
        del w
        if kind == "mx4_gated":
            return h
        return h.to(BF16).double() @ _exact_weight(s["W3q"], s["W3s"]).t(), h
    if kind == "down_back":
        d_out = s["dOut"].double()
        return d_out @ s["W3t"].double(), s["H"].double().t().mm(d_out).t() + s["sum"].double()
    dh = s["dH"].double() if kind == "gated_back" else s["dOut"].double() @ s["W3t"].double()
    d_gu = _exact_d_gu(dh, s["GU"])
    d = d_gu.to(BF16).double()
    da = d @ s["W_fused"].double()
    dw = s["A"].double().t().mm(d).t()
    if kind == "gated_back":
        return da, dw, d_gu
    return da, dw, s["H"].double().t().mm(s["dOut"].double()).t(), d_gu
