"""The 64-bit forms of the router, row movement and 4-bit weights
(oracle/moe.py) against hand-worked values, differences and torch."""

import numpy as np
import pytest
import torch

from oracle import moe


def test_router_by_hand():
    logits = np.log(np.array([[1.0, 2.0, 3.0, 4.0]]))
    idx, w, p = moe.router(logits, 2)
    assert idx.tolist() == [[3, 2]]
    np.testing.assert_allclose(p, [[0.1, 0.2, 0.3, 0.4]], rtol=1e-15)
    np.testing.assert_allclose(w, [[4 / 7, 3 / 7]], rtol=1e-15)
    _, w, _ = moe.router(logits, 2, renormalize=False, scale=2.0)
    np.testing.assert_allclose(w, [[0.8, 0.6]], rtol=1e-15)


def test_router_bias_steers_the_choice_only():
    logits = np.zeros((1, 4))
    idx, w, _ = moe.router(logits, 1, "sigmoid", bias=[0, 0, 0.1, 0], renormalize=False)
    assert idx.tolist() == [[2]] and w[0, 0] == 0.5


def test_router_groups_and_ties():
    # group ratings by the two best sigmoid values: (0.5 + 0.5), (s(2) + s(-9))
    logits = np.array([[0.0, 0.0, 2.0, -9.0]])
    idx, _, _ = moe.router(logits, 2, "sigmoid", num_groups=2, topk_groups=1, group_top=2)
    assert idx.tolist() == [[0, 1]]
    idx, _, _ = moe.router(logits, 2, "sigmoid", num_groups=2, topk_groups=1, group_top=1)
    assert idx.tolist() == [[2, 3]]


def test_router_masked_rows():
    logits = np.array([[-np.inf, 1.0, np.nan], [-np.inf] * 3])
    idx, w, p = moe.router(logits, 2)
    assert idx.tolist() == [[1, -1], [-1, -1]]
    assert w.tolist() == [[1.0, 0.0], [0.0, 0.0]] and p.tolist() == [[0, 1, 0], [0, 0, 0]]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("probs", [True, False])
def test_router_backward_against_differences(score, renorm, probs):
    rng = np.random.default_rng(7)
    T, E, k = 3, 9, 4
    logits = rng.normal(size=(T, E))
    logits[1, 2] = -np.inf
    idx, _, _ = moe.router(logits, k, score)
    gw = rng.normal(size=(T, k))
    gp = rng.normal(size=(T, E)) if probs else None

    def loss(l):
        p = moe._scores(l, score)
        s = np.take_along_axis(p, idx, 1)
        w = 1.5 * (s / s.sum(1, keepdims=True) if renorm else s)
        return (w * gw).sum() + (0.0 if gp is None else (p * gp).sum())

    got = moe.router_backward(logits, idx, gw, gp, score, renorm, 1.5)
    h = 1e-5
    for t in range(T):
        for e in range(E):
            if logits[t, e] == -np.inf:
                assert got[t, e] == 0.0
                continue
            up, dn = logits.copy(), logits.copy()
            up[t, e] += h
            dn[t, e] -= h
            # central differences: h^2 of the third derivative (< 10 here)
            # plus the values' rounding over h
            assert abs((loss(up) - loss(dn)) / (2 * h) - got[t, e]) < 1e-8


def test_movement_against_torch_autograd():
    rng = np.random.default_rng(3)
    T, k, H = 5, 3, 4
    slot = rng.permutation(T * k).reshape(T, k).astype(np.int32)
    slot[1, 1] = -1
    x, w, y = rng.normal(size=(T, H)), rng.normal(size=(T, k)), rng.normal(size=(T * k, H))
    ok = torch.from_numpy(slot >= 0)
    at = torch.from_numpy(np.maximum(slot, 0)).long()
    tx, tw, ty = (torch.from_numpy(a).requires_grad_() for a in (x, w, y))
    out = (torch.where(ok, tw, 0.0)[:, :, None] * ty[at]).sum(1)
    np.testing.assert_allclose(moe.unpermute(y, slot, w), out.detach().numpy(), atol=1e-14)
    g = torch.from_numpy(rng.normal(size=(T, H)))
    gy, gw = torch.autograd.grad((out * g).sum(), (ty, tw))
    np.testing.assert_allclose(moe.permute(g.numpy(), slot, w, T * k), gy.numpy(), atol=1e-14)
    np.testing.assert_allclose(moe.pair_dots(g.numpy(), y, slot)[0], gw.numpy(), atol=1e-14)
    rows = torch.zeros(T * k, H, dtype=torch.float64)
    rows = rows.index_put((at[ok],), (tw[:, :, None] * tx[:, None, :])[ok])
    gr = torch.from_numpy(rng.normal(size=(T * k, H)))
    gx, gw = torch.autograd.grad((rows * gr).sum(), (tx, tw))
    np.testing.assert_allclose(moe.unpermute(gr.numpy(), slot, w), gx.numpy(), atol=1e-14)
    np.testing.assert_allclose(moe.pair_dots(x, gr.numpy(), slot)[0], gw.numpy(), atol=1e-14)


def test_w4_by_hand():
    codes = np.array([[[0x21, 0xF8]]], dtype=np.uint8)            # codes 1, 2, 8, 15
    scales = np.array([[[0.5, 2.0]]])
    assert moe.w4_dequantize(codes, scales, None, 2).tolist() == [[[-3.5, -3.0, 0.0, 14.0]]]
    zeros = np.array([[[1, 15]]], dtype=np.uint8)
    assert moe.w4_dequantize(codes, scales, zeros, 2).tolist() == [[[0.0, 0.5, -14.0, 0.0]]]
