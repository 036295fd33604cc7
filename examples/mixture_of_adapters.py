"""A gated MLP block with a mixture of low-rank adapters, from its router on
(needs an MI355X):

    python examples/mixture_of_adapters.py

The router picks two of eight adapters a token and weighs them
(``swiglu_route``); the block takes them beside its Gate, Up and down
projections (``swiglu_gated_mlp_lora``).  Then a few steps on the router alone:
its balance loss and a loss on its weights, with the gradient by the logits
from ``swiglu_route_backward``.  Last, one token of one request that brought its
own adapter.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from gated_mlp_gemm_amd import swiglu as sw  # noqa: E402

TOKENS, WIDTH, HIDDEN = 512, 896, 4864
ADAPTERS, RANK, PICKS = 8, 16, 2


def weight(rows, cols, std, dev):
    return (torch.randn(rows, cols, device=dev) * std).to(torch.bfloat16)


def tables(dev):
    """The adapters' tables beside Gate and Up, and beside the down projection."""
    a_up = weight(ADAPTERS * 2 * RANK, WIDTH, WIDTH ** -0.5, dev).view(ADAPTERS, 2 * RANK, WIDTH)
    # B's Gate and Up rows interleave as the packed weight's do: the same packer
    b_up = sw.swiglu_pack_weights_nk(weight(ADAPTERS * HIDDEN, RANK, 0.1, dev),
                                     weight(ADAPTERS * HIDDEN, RANK, 0.1, dev))
    a_down = weight(ADAPTERS * RANK, HIDDEN, HIDDEN ** -0.5, dev).view(ADAPTERS, RANK, HIDDEN)
    b_down = weight(ADAPTERS * WIDTH, RANK, 0.1, dev).view(ADAPTERS, WIDTH, RANK)
    scale = torch.full((ADAPTERS,), 2.0, device=dev)
    return (sw.SwigluLora(a_up, b_up.view(ADAPTERS, 2 * HIDDEN, RANK), scale),
            sw.SwigluLora(a_down, b_down, scale))


def main():
    torch.manual_seed(0)
    dev = torch.device("cuda:0")
    w_fused = sw.swiglu_pack_weights_nk(weight(HIDDEN, WIDTH, WIDTH ** -0.5, dev),
                                        weight(HIDDEN, WIDTH, WIDTH ** -0.5, dev))
    w_down = weight(WIDTH, HIDDEN, HIDDEN ** -0.5, dev)
    gate_up, down = tables(dev)
    x = weight(TOKENS, WIDTH, 1.0, dev)
    router = torch.randn(ADAPTERS, WIDTH, device=dev) * WIDTH ** -0.5
    workspace = sw.make_lora_workspace(TOKENS, HIDDEN, WIDTH, PICKS, RANK, dev)

    logits = x.float() @ router.t()
    ids, weights, counts, loss = sw.swiglu_route(logits, PICKS)
    out, _ = sw.swiglu_gated_mlp_lora(x, w_fused, w_down, gate_up, down, ids, weights,
                                      workspace=workspace)
    plain, _ = sw.swiglu_gated_mlp(x, w_fused, w_down, variant="auto")
    change = (out.float() - plain.float()).norm() / plain.float().norm()
    print(f"picks of each adapter {counts[:-1].tolist()}, balance loss {loss.item():.4f}")
    print(f"the adapters change the block's output by {change.item():.3f} of its norm")

    # the router's own training: even use, and more weight on the first pick
    for step in range(20):
        logits = x.float() @ router.t()
        ids, weights, counts, loss = sw.swiglu_route(logits, PICKS)
        d_weights = torch.zeros_like(weights)
        d_weights[:, 0] = -1.0 / TOKENS
        d_logits = sw.swiglu_route_backward(logits, ids, weights, counts, d_weights=d_weights,
                                            d_loss=torch.ones((), device=dev))
        if step % 19 == 0:
            print(f"step {step:2d}: balance loss {loss.item():.4f}, "
                  f"first pick's weight {weights[:, 0].mean().item():.4f}")
        router -= 2.0 * (d_logits.t() @ x.float())

    # one token of one request, with adapter 3 of the table and no router
    token, _ = sw.swiglu_gated_mlp_lora(x[:1], w_fused, w_down, gate_up, down,
                                        torch.tensor([[3]], dtype=torch.int32, device=dev))
    print(f"one token with adapter 3: norm {token.float().norm().item():.3f}")


if __name__ == "__main__":
    main()
