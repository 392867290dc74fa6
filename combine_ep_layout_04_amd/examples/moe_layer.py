"""A mixture-of-experts layer on this library, for decoding and for training.

    python -m combine_ep_layout_04_amd.examples.moe_layer [tokens]

* ``decode``: router, layout, the gated first product and the second product
  with weights of 4 bits, 8 bits or full width (the tokens are read through the
  layout's ``src``, so they are not dispatched), and the weighted sum back in
  token order.  Everything is launched without a look at the device's results,
  so it can be captured into a graph.
* ``train_step``: router, layout, the rows sorted by expert, the gated block
  and the second product of every expert, the weighted sum, and the gradients
  of all of it back to the tokens, the router's weight and the experts'
  weights.  In bf16 and fp16 nothing waits for the device's results; in fp32
  the experts are torch products per segment.
"""

from __future__ import annotations

import sys
import time
from typing import NamedTuple

import torch

from .. import ep


class Fp8Weights(NamedTuple):
    """8-bit expert weights: E4M3 codes [E, N, K] and a scale per 128 x 128."""
    codes: torch.Tensor
    scales: torch.Tensor


def cast_rows(x):
    """Each row of x (bf16) in 8 bits: codes and a scale per 128 channels."""
    alone = torch.arange(x.shape[0], dtype=torch.int32, device=x.device).reshape(-1, 1)
    codes, scales, _ = ep.ep_dispatch(x, alone, fp8=True)
    return codes, scales


def experts(x, w13, w2, offsets, src):
    """The experts' rows of tokens ``x``: both products, by the weights' kind."""
    if isinstance(w13, ep.W4Weights):
        h = ep.ep_expert_matmul_w4(x, w13, offsets, src=src)
        return ep.ep_expert_matmul_w4(h, w2, offsets)
    if isinstance(w13, Fp8Weights):
        h = ep.ep_expert_matmul_fp8(*cast_rows(x), *w13, offsets, gated=True, src=src)
        return ep.ep_expert_matmul_fp8(*cast_rows(h), *w2, offsets)
    h, _ = ep.ep_expert_glu(x, w13, offsets, src=src)
    return ep.ep_expert_matmul(h, w2, offsets)


def decode(x, gate_weight, w13, w2, num_topk: int, *, bias=None,
           score: str = "sigmoid", num_groups: int = 1, topk_groups: int = 1, group_top: int = 1,
           scale: float = 1.0):
    """x [T, H] (bf16 / fp16) through a router ``gate_weight`` [E, H] and E
    experts: ``w13`` gated [E, 2I, H], ``w2`` [E, H, I], both ep.W4Weights,
    Fp8Weights (bf16 tokens) or tensors of x's type."""
    E = gate_weight.shape[0]
    logits = x @ gate_weight.t()
    idx, w, _ = ep.ep_router(logits, num_topk, score=score, bias=bias, num_groups=num_groups,
                             topk_groups=topk_groups, group_top=group_top, scale=scale)
    _, offsets, slot, src, _ = ep.ep_layout(idx, E, want_invalid=False)
    return ep.ep_unpermute(experts(x, w13, w2, offsets, src), slot, w)


def _expert_rows(rows, w13, w2, offsets):
    """(y, backward) of the experts' two products on rows by expert; backward
    gives the gradients of rows, w13 and w2 from that of y."""
    if rows.dtype != torch.float32:
        h, pre = ep.ep_expert_glu(rows, w13, offsets, want_pre=True)
        y = ep.ep_expert_matmul(h, w2, offsets)

        def backward(grad_y):
            grad_h, grad_w2 = ep.ep_expert_matmul_backward(grad_y, h, w2, offsets)
            return (*ep.ep_expert_glu_backward(grad_h, pre, rows, w13, offsets), grad_w2)
        return y, backward
    # by torch, with a graph of their own whose leaves are each expert's rows
    # and weights
    E = w13.shape[0]
    bounds = offsets.tolist()
    leaves = [[t.detach().requires_grad_() for t in (rows[bounds[e]:bounds[e + 1]], w13[e], w2[e])]
              for e in range(E)]
    with torch.enable_grad():
        parts = []
        for r, a, b in leaves:
            gate, up = (r @ a.t()).chunk(2, 1)
            parts.append((torch.nn.functional.silu(gate) * up) @ b.t())
        y = torch.cat(parts)

    def backward(grad_y):
        grads = torch.autograd.grad(y, [t for leaf in leaves for t in leaf], grad_y[:bounds[E]])
        return torch.cat(grads[0::3]), torch.stack(grads[1::3]), torch.stack(grads[2::3])
    return y.detach(), backward


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
    y, backward = _expert_rows(rows, w13, w2, offsets)
    out = ep.ep_unpermute(y, slot, w)

    grad_y, grad_w = ep.ep_unpermute_backward(grad_out, slot, w, y)
    grad_rows, grad_w13, grad_w2 = backward(grad_y)
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


def random_fp8(E, N, K, *, device="cuda:0"):
    """Random 8-bit weights of about unit gain."""
    w = torch.randn(E, N, K, device=device).clamp_(-4, 4) * 64
    return Fp8Weights(w.to(torch.float8_e4m3fn).view(torch.uint8),
                      torch.full((E, (N + 127) // 128, (K + 127) // 128), 1 / (64 * K ** 0.5), device=device))


def main(tokens: int = 4):
    dev, E, k, H, I = "cuda:0", 64, 4, 2048, 1408
    torch.manual_seed(0)
    x = torch.randn(tokens, H, device=dev).bfloat16()
    gate = (torch.randn(E, H, device=dev) / H ** 0.5).bfloat16()
    bias = torch.zeros(E, device=dev)
    f13 = torch.randn(E, 2 * I, H, device=dev).bfloat16() / H ** 0.5
    f2 = torch.randn(E, H, I, device=dev).bfloat16() / I ** 0.5
    for bits, w13, w2 in ((4, random_w4(E, 2 * I, H, gated=True), random_w4(E, H, I)),
                          (8, random_fp8(E, 2 * I, H), random_fp8(E, H, I)), (16, f13, f2)):
        time_decode(bits, x, gate, w13, w2, k, bias)
    xt = torch.randn(512, H, device=dev).bfloat16()

    def balance(probs, counts):             # of E * sum_e mean(probs_e) * share_e
        return (counts.float() * (E / (counts.sum() * probs.shape[0]))).expand_as(probs).contiguous()
    grads = train_step(xt, gate, f13, f2, k, torch.randn_like(xt), grad_probs_of=balance)
    print("train step, 512 tokens: " + ", ".join(str(tuple(g.shape)) for g in grads), flush=True)


def time_decode(bits, x, gate, w13, w2, k, bias):
    (tokens, H), E = x.shape, gate.shape[0]

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
        print(f"decode, {tokens} tokens, {E} experts, top {k}, width {H}, {bits} bit, {name}: "
              f"{(time.perf_counter() - t0) * 1e4:.1f} us a layer", flush=True)
    assert torch.equal(out, step())


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 4)
