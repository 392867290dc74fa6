"""A mixture-of-experts layer on this library, for decoding and for training.

    python -m combine_ep_layout_04_amd.examples.moe_layer [tokens]

* ``decode``: router, layout, the gated first product and the second product
  with 4-bit weights (the tokens are read through the layout's ``src``, so they
  are not dispatched), and the weighted sum back in token order.  Everything
  is launched without a look at the device's results, so it can be captured
  into a graph.
* ``train_step``: router, layout, the rows sorted by expert, a gated expert of
  torch products per segment, the weighted sum, and the gradients of all of it
  back to the tokens, the router's weight and the experts' weights.
"""

from __future__ import annotations

import sys
import time

import torch

from .. import ep


def decode(x, gate_weight, w13: ep.W4Weights, w2: ep.W4Weights, num_topk: int, *, bias=None,
           score: str = "sigmoid", num_groups: int = 1, topk_groups: int = 1, group_top: int = 1,
           scale: float = 1.0):
    """x [T, H] (bf16 / fp16) through a router ``gate_weight`` [E, H] and E
    experts of 4-bit weights: ``w13`` gated [E, 2I, H], ``w2`` [E, H, I]."""
    E = gate_weight.shape[0]
    logits = x @ gate_weight.t()
    idx, w, _ = ep.ep_router(logits, num_topk, score=score, bias=bias, num_groups=num_groups,
                             topk_groups=topk_groups, group_top=group_top, scale=scale)
    _, offsets, slot, src, _ = ep.ep_layout(idx, E, want_invalid=False)
    rows = slot.numel()
    h = ep.ep_expert_matmul_w4(x, w13, offsets, src=src, rows=rows)
    y = ep.ep_expert_matmul_w4(h, w2, offsets)
    return ep.ep_unpermute(y, slot, w)


def train_step(x, gate_weight, w13, w2, num_topk: int, grad_out, *, score: str = "softmax",
               grad_probs_of=None):
    """Forward and backward of a layer with experts of full weights ``w13``
    [E, 2I, H] and ``w2`` [E, H, I].  ``grad_probs_of(probs, counts)`` gives
    the gradient of a loss on the scores (load balancing), or None.

    Returns (out, grad_x, grad_gate_weight, grad_w13, grad_w2)."""
    E = gate_weight.shape[0]
    logits = x @ gate_weight.t()
    idx, w, probs = ep.ep_router(logits, num_topk, score=score, want_probs=grad_probs_of is not None)
    counts, offsets, slot, _, _ = ep.ep_layout(idx, E)
    rows = ep.ep_permute(x, slot)
    # the experts, by torch, with a graph of their own whose leaves are each
    # expert's rows and weights
    bounds = offsets.tolist()
    leaves = [[t.detach().requires_grad_() for t in (rows[bounds[e]:bounds[e + 1]], w13[e], w2[e])]
              for e in range(E)]
    with torch.enable_grad():
        parts = []
        for r, a, b in leaves:
            gate, up = (r @ a.t()).chunk(2, 1)
            parts.append((torch.nn.functional.silu(gate) * up) @ b.t())
        y = torch.cat(parts)
    out = ep.ep_unpermute(y.detach(), slot, w)

    grad_y, grad_w = ep.ep_unpermute_backward(grad_out, slot, w, y.detach())
    grads = torch.autograd.grad(y, [t for leaf in leaves for t in leaf], grad_y[:bounds[E]])
    grad_rows = torch.cat(grads[0::3])
    grad_w13, grad_w2 = torch.stack(grads[1::3]), torch.stack(grads[2::3])
    grad_x, _ = ep.ep_permute_backward(grad_rows, slot)
    grad_probs = None if grad_probs_of is None else grad_probs_of(probs, counts)
    grad_logits = ep.ep_router_backward(logits, idx, grad_w, grad_probs, score=score)
    grad_x += grad_logits @ gate_weight
    return out, grad_x, grad_logits.t() @ x, grad_w13, grad_w2


def random_w4(E, N, K, *, group_size=128, gated=False, dtype=torch.bfloat16, device="cuda:0"):
    """Random packed weights of about unit gain (a stand-in for loaded ones)."""
    codes = torch.randint(0, 256, (E, N, K // 2), dtype=torch.uint8, device=device)
    scales = (torch.rand(E, N, (K + group_size - 1) // group_size, device=device) + 0.5) / (4.6 * K ** 0.5)
    return ep.ep_w4_pack(codes, scales.to(dtype), group_size=group_size, gated=gated)


def main(tokens: int = 4):
    dev, E, k, H, I = "cuda:0", 64, 4, 2048, 1408
    torch.manual_seed(0)
    x = torch.randn(tokens, H, device=dev).bfloat16()
    gate = (torch.randn(E, H, device=dev) / H ** 0.5).bfloat16()
    w13, w2 = random_w4(E, 2 * I, H, gated=True), random_w4(E, H, I)
    bias = torch.zeros(E, device=dev)

    def step():
        return decode(x, gate, w13, w2, k, bias=bias)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):           # once outside the capture
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for name, run in (("eager", step), ("graph", graph.replay)):
        run()
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        for _ in range(100):
            run()
        torch.cuda.synchronize()
        print(f"decode, {tokens} tokens, {E} experts, top {k}, {H} x {I}, 4 bit, {name}: "
              f"{(time.perf_counter() - t0) * 1e4:.1f} us a layer", flush=True)
    assert torch.equal(out, step())

    f13 = torch.randn(E, 2 * I, H, device=dev).bfloat16() / H ** 0.5
    f2 = torch.randn(E, H, I, device=dev).bfloat16() / I ** 0.5
    xt = torch.randn(512, H, device=dev).bfloat16()

    def balance(probs, counts):             # of E * sum_e mean(probs_e) * share_e
        return (counts.float() * (E / (counts.sum() * probs.shape[0]))).expand_as(probs).contiguous()
    grads = train_step(xt, gate, f13, f2, k, torch.randn_like(xt), grad_probs_of=balance)
    print("train step, 512 tokens: " + ", ".join(str(tuple(g.shape)) for g in grads), flush=True)


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 4)
