"""The router and the low-rank adapter calls as a user's program makes them, and
their plain forms.

Five kinds of case:

  route        swiglu_route: softmax, top-k, counts and balance loss
  route_train  the same, then swiglu_route_backward: the gradient by the logits
  gated        swiglu_fused_gemm_lora: Gate and Up with each row's adapters
  down         swiglu_down_proj_lora: the down projection with each row's adapter
  mlp          swiglu_route, then swiglu_gated_mlp_lora on what it picked

With ``own`` false, ``run`` computes them from elementary torch operations in
32 bits; with ``own`` true it calls the library.  ``exact`` computes them in 64
bits, adapter by adapter and slot by slot.
"""
import math

import torch

own = False


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one token choosing among a few adapters: latency
        {"name": "route_one", "kind": "route", "M": 1, "E": 8, "k": 2, "dtype": "fp32",
         "masked": False, "normalize": True},
        # a prompt batch over many experts, raw probabilities as weights
        {"name": "route_prompt", "kind": "route", "M": 8192, "E": 64, "k": 4, "dtype": "bf16",
         "masked": True, "normalize": False},
        # a training batch, forward and gradient
        {"name": "route_train", "kind": "route_train", "M": 16384, "E": 128, "k": 8,
         "dtype": "fp32", "masked": True, "normalize": True},
        # the same with odd counts and short logits
        {"name": "route_train_odd", "kind": "route_train", "M": 4099, "E": 61, "k": 3,
         "dtype": "bf16", "masked": True, "normalize": False},
        # one token of one request
        {"name": "gated_one", "kind": "gated", "M": 1, "K": 896, "N": 4864, "L": 8, "r": 16,
         "J": 1, "rows": "mixed"},
        # one token each of many requests
        {"name": "gated_requests", "kind": "gated", "M": 64, "K": 3584, "N": 18944, "L": 32,
         "r": 16, "J": 1, "rows": "mixed"},
        # the prompts of a few requests, one after the other
        {"name": "gated_prompts", "kind": "gated", "M": 2048, "K": 1536, "N": 8960, "L": 8,
         "r": 32, "J": 1, "rows": "runs"},
        # a mixture of low-rank experts, two a row
        {"name": "gated_mixture", "kind": "gated", "M": 512, "K": 3584, "N": 18944, "L": 8,
         "r": 16, "J": 2, "rows": "mixed"},
        # a ragged decode batch through the down projection
        {"name": "down_requests_odd", "kind": "down", "M": 33, "K": 8960, "N": 1536, "L": 16,
         "r": 8, "J": 1, "rows": "mixed"},
        # long prompts of several requests through the down projection
        {"name": "down_prompts_long", "kind": "down", "M": 8192, "K": 13824, "N": 5120, "L": 16,
         "r": 64, "J": 1, "rows": "runs"},
        # the whole block on a decode batch, adapters picked by the router
        {"name": "mlp_mixture_small", "kind": "mlp", "M": 128, "K": 896, "N": 4864, "L": 8,
         "r": 16, "J": 2, "rows": "mixed"},
        # the whole block on a prompt batch
        {"name": "mlp_mixture", "kind": "mlp", "M": 2048, "K": 1536, "N": 8960, "L": 8, "r": 16,
         "J": 2, "rows": "mixed"},
    ]


def _spread(rng, low, high):
    """A whole number from low to high, even over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 1)))))))


def draw(rng):
    kind = rng.choice(("route", "route_train", "gated", "down", "mlp"))
    if kind.startswith("route"):
        E = _spread(rng, 2, 256)
        return {"kind": kind, "M": _spread(rng, 1, 16384), "E": E, "k": rng.randint(1, min(8, E)),
                "dtype": rng.choice(("bf16", "fp32")), "masked": rng.random() < 0.5,
                "normalize": rng.random() < 0.5}
    K, N = 8 * _spread(rng, 64, 1024), 8 * _spread(rng, 64, 2048)
    r = 8 * rng.randint(1, 8)
    L = _spread(rng, 1, 32)
    J = rng.randint(1, min(4, L)) if kind != "down" and rng.random() < 0.6 else 1
    # the products of the largest listed case hold 8192 * 13824 * 5120 multiply-adds
    most = 8192 * 13824 * 5120 // (K * N * {"gated": 2, "down": 1, "mlp": 3}[kind]) // 2
    return {"kind": kind, "M": _spread(rng, 1, min(8192, most)), "K": K, "N": N, "L": L, "r": r,
            "J": J, "rows": rng.choice(("mixed", "runs")) if J == 1 and kind != "mlp" else "mixed"}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
DEVICE = "cuda:0"
NEG_INF = float("-inf")


def _normal(g, shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device=DEVICE, dtype=torch.float32) * std).to(dtype)


def _logits(g, M, E, dtype, masked):
    """Router logits: a drift per expert, some experts closed to some rows
    (-inf), and a row of padding now and then (valid = 0)."""
    z = torch.randn(M, E, generator=g, device=DEVICE) * 1.5
    z = z + torch.randn(E, generator=g, device=DEVICE) * 0.5
    valid = None
    if masked:
        closed = torch.rand(M, E, generator=g, device=DEVICE) < 0.05
        z = torch.where(closed, torch.full_like(z, NEG_INF), z)
        valid = (torch.rand(M, generator=g, device=DEVICE) >= 0.07).to(torch.uint8)
    return z.to(torch.float32 if dtype == "fp32" else torch.bfloat16), valid


def _request_ids(g, M, L, rows):
    """One adapter a row: each row its own, or runs of rows of one request;
    about one row (or run) in ten has none (-1)."""
    if rows == "mixed":
        ids = torch.randint(0, L, (M, 1), generator=g, device=DEVICE)
        none = torch.rand(M, 1, generator=g, device=DEVICE) < 0.1
        # at least one row has an adapter
        none[M // 2] = False
    else:
        runs = max(1, min(M, 12))
        cut = torch.sort(torch.randint(0, M, (runs,), generator=g, device=DEVICE)).values
        run = torch.searchsorted(cut, torch.arange(M, device=DEVICE), right=True)
        of_run = torch.randint(0, L, (runs + 1,), generator=g, device=DEVICE)
        none_run = torch.rand(runs + 1, generator=g, device=DEVICE) < 0.1
        ids, none = of_run[run][:, None], none_run[run][:, None]
    return torch.where(none, torch.full_like(ids, -1), ids).to(torch.int32)


def _adapters(g, L, parts, K, N, r):
    """Adapter table beside a [parts * N, K] weight: A [L, parts r, K],
    B [L, parts N, r] (Gate and Up rows interleaved when parts is 2), scale [L]."""
    return {"A": _normal(g, (L, parts * r, K), 1.0 / math.sqrt(K)),
            "B": _normal(g, (L, parts * N, r), 0.5 / math.sqrt(r)),
            "scale": torch.rand(L, generator=g, device=DEVICE) * 1.5 + 0.5}


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed))
    M, kind = case["M"], case["kind"]
    s = {"kind": kind}
    if kind.startswith("route"):
        s["logits"], s["valid"] = _logits(g, M, case["E"], case["dtype"], case["masked"])
        s["k"], s["normalize"] = case["k"], case["normalize"]
        if kind == "route_train":
            s["d_weights"] = torch.randn(M, case["k"], generator=g, device=DEVICE)
            s["d_loss"] = torch.rand((), generator=g, device=DEVICE) * 0.02 + 0.01
        return s
    K, N, L, r, J = case["K"], case["N"], case["L"], case["r"], case["J"]
    s["X"] = _normal(g, (M, K))
    if kind == "down":
        s["W3t"] = _normal(g, (N, K), 1.0 / math.sqrt(K))
        s["down"] = _adapters(g, L, 1, K, N, r)
    else:
        s["W_fused"] = _normal(g, (2 * N, K), 1.0 / math.sqrt(K))
        s["gate_up"] = _adapters(g, L, 2, K, N, r)
    if kind == "mlp":
        s["W3t"] = _normal(g, (K, N), 1.0 / math.sqrt(N))
        s["down"] = _adapters(g, L, 1, N, K, r)
        s["logits"], s["valid"] = _logits(g, M, L, "fp32", False)
        s["k"], s["normalize"] = J, True
    elif J == 1:
        s["ids"], s["weights"] = _request_ids(g, M, L, case["rows"]), None
    else:
        z, _ = _logits(g, M, L, "fp32", False)
        order = torch.sort(z, dim=1, descending=True, stable=True)
        s["ids"] = order.indices[:, :J].to(torch.int32).contiguous()
        s["weights"] = torch.softmax(order.values[:, :J], dim=1).contiguous()
    # the scratch that a serving program keeps for these calls
    s["workspace"] = torch.empty((128 << 20) + 64 * M * J * 2 * r, dtype=torch.uint8, device=DEVICE)
    return s


# ---------------------------------------------------------------------------
# plain forms: elementary torch operations in 32 bits, rounded once at the end
# ---------------------------------------------------------------------------
def _plain_probs(s):
    """Softmax of every row that routes (zeros elsewhere), and which rows do."""
    z = s["logits"].float()
    top = z.max(dim=1, keepdim=True).values
    live = top[:, 0] > NEG_INF
    if s["valid"] is not None:
        live = live & (s["valid"] != 0)
    e = torch.exp(z - torch.where(live[:, None], top, torch.zeros_like(top)))
    p = torch.where(live[:, None], e / e.sum(dim=1, keepdim=True), torch.zeros_like(z))
    return z, p, live


def _plain_route(s):
    z, p, live = _plain_probs(s)
    k, E = s["k"], z.shape[1]
    order = torch.sort(z, dim=1, descending=True, stable=True)     # ties: the lowest index first
    ids, vals = order.indices[:, :k], order.values[:, :k]
    picked = live[:, None] & (vals > NEG_INF)
    w = torch.where(picked, torch.gather(p, 1, ids), torch.zeros_like(vals))
    if s["normalize"]:
        e = torch.where(picked, torch.exp(vals - vals[:, :1]), torch.zeros_like(vals))
        w = torch.where(picked, e / e.sum(dim=1, keepdim=True), torch.zeros_like(e))
    hit = (ids[:, :, None] == torch.arange(E, device=z.device)) & picked[:, :, None]
    per_expert = hit.sum(dim=(0, 1))
    rows = live.sum()
    # column sums over many rows: in 64 bits
    mean_p = p.double().sum(dim=0) / rows.clamp(min=1)
    share = per_expert.double() / per_expert.sum().clamp(min=1)
    loss = (E * (share * mean_p).sum()).float()
    counts = torch.cat([per_expert, rows[None]]).to(torch.int32)
    return torch.where(picked, ids, torch.full_like(ids, -1)).to(torch.int32), w, counts, loss


def _plain_route_backward(s, ids, w, counts):
    z, p, live = _plain_probs(s)
    E = z.shape[1]
    n, per_expert = counts[E].float().clamp(min=1), counts[:E].float()
    g = s["d_loss"] * E * per_expert / (per_expert.sum().clamp(min=1) * n)
    hit = (ids[:, :, None] == torch.arange(E, device=z.device)).float()      # [M, k, E]
    dw = s["d_weights"]
    if s["normalize"]:
        dz = p * (g - (p * g).sum(dim=1, keepdim=True))
        dv = w * (dw - (w * dw).sum(dim=1, keepdim=True))
        dz = dz + (hit * dv[:, :, None]).sum(dim=1)
    else:
        G = g + (hit * dw[:, :, None]).sum(dim=1)
        dz = p * (G - (p * G).sum(dim=1, keepdim=True))
    return torch.where(live[:, None], dz, torch.zeros_like(dz)).to(s["logits"].dtype)


def _plain_shares(ids, weights, scale):
    """How much of each adapter each row takes: [M, L]."""
    hit = (ids[:, :, None] == torch.arange(scale.numel(), device=ids.device)).float()
    if weights is not None:
        hit = hit * weights[:, :, None]
    return hit.sum(dim=1) * scale


def _plain_delta(x, a, b, shares):
    """sum over adapters of shares * (x a^T) b^T; a [L, r, K], b [L, N, r]."""
    L, r, K = a.shape
    t = (x @ a.reshape(L * r, K).t()).view(-1, L, r) * shares[:, :, None]
    return t.reshape(-1, L * r) @ b.permute(0, 2, 1).reshape(L * r, -1)


def _plain_gated(x, w_fused, ad, ids, weights):
    """SiLU(gate) * up in 32 bits."""
    x, w = x.float(), w_fused.float()
    a, b, r = ad["A"].float(), ad["B"].float(), ad["B"].shape[2]
    shares = _plain_shares(ids, weights, ad["scale"])
    gate = x @ w[0::2].t() + _plain_delta(x, a[:, :r], b[:, 0::2], shares)
    up = x @ w[1::2].t() + _plain_delta(x, a[:, r:], b[:, 1::2], shares)
    return gate / (1.0 + torch.exp(-gate)) * up


def _plain_down(h, w3t, ad, ids, weights):
    h = h.float()
    shares = _plain_shares(ids, weights, ad["scale"])
    return h @ w3t.float().t() + _plain_delta(h, ad["A"].float(), ad["B"].float(), shares)


def _plain(s):
    kind, bf16 = s["kind"], torch.bfloat16
    if kind == "route":
        return _plain_route(s)
    if kind == "route_train":
        ids, w, counts, loss = _plain_route(s)
        return ids, w, counts, loss, _plain_route_backward(s, ids, w, counts)
    if kind == "gated":
        return _plain_gated(s["X"], s["W_fused"], s["gate_up"], s["ids"], s["weights"]).to(bf16)
    if kind == "down":
        return _plain_down(s["X"], s["W3t"], s["down"], s["ids"], s["weights"]).to(bf16)
    ids, w, counts, loss = _plain_route(s)
    h = _plain_gated(s["X"], s["W_fused"], s["gate_up"], ids, w).to(bf16)
    out = _plain_down(h, s["W3t"], s["down"], ids, w).to(bf16)
    return out, h, ids, w, counts, loss


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------
def _own(s):
    from gated_mlp_gemm_amd import swiglu as sw
    kind = s["kind"]
    if kind in ("route", "route_train", "mlp"):
        ids, w, counts, loss = sw.swiglu_route(s["logits"], s["k"], valid=s["valid"],
                                               normalize=s["normalize"])
        if kind == "route":
            return ids, w, counts, loss
        if kind == "route_train":
            d_logits = sw.swiglu_route_backward(s["logits"], ids, w, counts,
                                                d_weights=s["d_weights"], d_loss=s["d_loss"],
                                                valid=s["valid"], normalize=s["normalize"])
            return ids, w, counts, loss, d_logits

    def adapters(t):
        return sw.SwigluLora(t["A"], t["B"], t["scale"])

    if kind == "gated":
        return sw.swiglu_fused_gemm_lora(s["X"], s["W_fused"], adapters(s["gate_up"]), s["ids"],
                                         s["weights"], workspace=s["workspace"])
    if kind == "down":
        return sw.swiglu_down_proj_lora(s["X"], s["W3t"], adapters(s["down"]), s["ids"],
                                        s["weights"], workspace=s["workspace"])
    out, h = sw.swiglu_gated_mlp_lora(s["X"], s["W_fused"], s["W3t"], adapters(s["gate_up"]),
                                      adapters(s["down"]), ids, w, workspace=s["workspace"])
    return out, h, ids, w, counts, loss


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def _route_work(M, E, k, size, masked, train):
    b = M * E * size + (M if masked else 0) + 8 * M * k + 4 * (E + 2)
    f = 6 * M * E
    if train:
        # the logits are read again for the gradient in the same pass: counted once
        b += M * E * size + 4 * M * k + 4
        f += 8 * M * E
    return b, f


def work(case):
    M, kind = case["M"], case["kind"]
    if kind.startswith("route"):
        b, f = _route_work(M, case["E"], case["k"], 4 if case["dtype"] == "fp32" else 2,
                           case["masked"], kind == "route_train")
        return {"bytes": b, "flops": f}
    K, N, L, r, J = case["K"], case["N"], case["L"], case["r"], case["J"]
    used = min(L, M * J)
    b = f = 0
    if kind in ("gated", "mlp"):
        b += 2 * (M * K + 2 * N * K + M * N + used * 2 * r * (K + N)) + 8 * M * J
        f += 4 * M * N * K + 4 * M * J * r * (K + N)
    if kind == "down":
        b += 2 * (M * K + N * K + M * N + used * r * (K + N)) + 8 * M * J
        f += 2 * M * N * K + 2 * M * J * r * (K + N)
    if kind == "mlp":
        b += 2 * (N * K + M * K + used * r * (K + N))
        f += 2 * M * N * K + 2 * M * J * r * (K + N)
        rb, rf = _route_work(M, L, J, 4, False, False)
        b, f = b + rb, f + rf
    return {"bytes": b, "flops": f}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def _exact_route(s):
    z = s["logits"].double()
    M, E = z.shape
    live = ~torch.isneginf(z).all(dim=1)
    if s["valid"] is not None:
        live &= s["valid"].bool()
    p = torch.zeros_like(z)
    p[live] = torch.softmax(z[live], dim=1)
    left = z.clone()
    ids = torch.full((M, s["k"]), -1, dtype=torch.int64, device=z.device)
    w = torch.zeros(M, s["k"], dtype=torch.float64, device=z.device)
    at = torch.arange(M, device=z.device)
    index = torch.arange(E, device=z.device)
    for j in range(s["k"]):
        best = left.max(dim=1).values
        # the lowest index among the largest
        first = torch.where(left == best[:, None], index, E).min(dim=1).values.clamp(max=E - 1)
        take = live & (best > NEG_INF)
        ids[take, j] = first[take]
        w[take, j] = p[at, first][take]
        left[at, first] = NEG_INF
    if s["normalize"]:
        w = w / w.sum(dim=1, keepdim=True).clamp(min=1e-300)
    counts = torch.bincount(ids[ids >= 0], minlength=E)
    n = int(live.sum())
    total = int(counts.sum())
    loss = E * (counts.double() / max(total, 1) * p.sum(dim=0) / max(n, 1)).sum()
    return p, live, ids, w, counts, n, total, loss


def _exact_d_logits(s, p, live, ids, w, counts, n, total):
    """By the softmax's Jacobian, a matrix a row, in pieces of the rows."""
    M, E = p.shape
    d_p = (s["d_loss"].double() * E * counts.double() / (max(total, 1) * max(n, 1))).expand(M, E)
    dw = torch.where(ids >= 0, s["d_weights"].double(), 0.0)
    safe = ids.clamp(min=0)
    out = torch.zeros_like(p)
    if s["normalize"]:
        # w_j = p_j / q with q = sum of the picked p
        q = torch.where(ids >= 0, torch.gather(p, 1, safe), 0.0).sum(dim=1, keepdim=True)
        q = torch.where(q > 0, q, torch.ones_like(q))
        d_picked = (dw - (w * dw).sum(dim=1, keepdim=True)) / q
    else:
        d_picked = dw
    d_p = d_p.clone().scatter_add_(1, safe, torch.where(ids >= 0, d_picked, 0.0))
    step = max(1, (1 << 26) // (E * E))
    for m in range(0, M, step):
        q = p[m:m + step]
        jac = torch.diag_embed(q) - q[:, :, None] * q[:, None, :]
        out[m:m + step] = (jac * d_p[m:m + step, None, :]).sum(dim=2)
    out[~live] = 0.0
    return out


def _exact_product(x, w, ad, part, parts, ids, weights):
    """x w[part::parts]^T and, adapter by adapter, the rows that take it."""
    w, a = w[part::parts], ad["A"]
    r = a.shape[1] // parts
    y = x @ w.double().t()
    for n in range(a.shape[0]):
        take = (ids == n)
        share = take.double() if weights is None else torch.where(take, weights.double(), 0.0)
        rows = take.any(dim=1).nonzero()[:, 0]
        if rows.numel() == 0:
            continue
        t = x[rows] @ a[n, part * r:(part + 1) * r].double().t()
        d = t @ ad["B"][n, part::parts].double().t()
        y[rows] += d * (share[rows].sum(dim=1) * ad["scale"][n].double())[:, None]
    return y


def _exact_gated(x, s, ids, weights):
    gate = _exact_product(x, s["W_fused"], s["gate_up"], 0, 2, ids, weights)
    up = _exact_product(x, s["W_fused"], s["gate_up"], 1, 2, ids, weights)
    return gate * torch.sigmoid(gate) * up


def exact(case, seed):
    s = prepare(case, seed)
    kind = s["kind"]
    if kind.startswith("route"):
        p, live, ids, w, counts, n, total, loss = _exact_route(s)
        every = torch.cat([counts, torch.tensor([n], device=counts.device)])
        if kind == "route":
            return ids, w, every, loss
        return ids, w, every, loss, _exact_d_logits(s, p, live, ids, w, counts, n, total)
    if kind == "gated":
        return _exact_gated(s["X"].double(), s, s["ids"], s["weights"])
    if kind == "down":
        return _exact_product(s["X"].double(), s["W3t"], s["down"], 0, 1, s["ids"], s["weights"])
    _, _, ids, w, counts, n, _, loss = _exact_route(s)
    h = _exact_gated(s["X"].double(), s, ids, w)
    # the block rounds its intermediate to bf16 by definition
    out = _exact_product(h.to(torch.bfloat16).double(), s["W3t"], s["down"], 0, 1, ids, w)
    return out, h, ids, w, torch.cat([counts, torch.tensor([n], device=counts.device)]), loss
