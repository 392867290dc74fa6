"""ep_router_backward with sigmoid scores whose chosen logits lie so far below
0 that a score has no fp32 value: the forward's weights are ordinary numbers
there, and so are their gradients."""

import numpy as np
import pytest
import torch

from combine_ep_layout_04_amd import ep
from oracle import moe

from moe_util import DEV, TYPES, U, check, f64, rounded, wide

pytestmark = pytest.mark.gpu

# T, E, k: each split of a row over lanes
SHAPES = [(9, 8, 2), (33, 16, 16), (20, 60, 4), (1030, 128, 6), (17, 128, 8), (2050, 256, 8), (6, 256, 40),
          (5, 700, 10)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("level", [-60.0, -86.0, -95.0, -110.0, -300.0, -690.0])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda c: "-".join(map(str, c)))
def test_backward(shape, level, dtype):
    T, E, k = shape
    rng = np.random.default_rng(int(-level))
    a = level + rng.normal(size=(T, E)) * 3.0
    a[1] = np.where(np.arange(E) % 3 == 0, a[1], a[1] * 0.5)    # some far below the others
    a[2, : E // 2] = -np.inf
    a[3] = -np.inf
    l = torch.from_numpy(a).to(TYPES[dtype]).double().numpy()
    idx, _, _ = moe.router(l, k, "sigmoid")
    gw = rng.normal(size=(T, k)).astype(np.float32)
    gp = rng.normal(size=(T, E)).astype(np.float32)
    logits, ti, tw = wide(l, dtype), torch.from_numpy(idx).to(DEV), torch.from_numpy(gw).to(DEV)
    p = moe._scores(l, "sigmoid")
    valid = idx >= 0
    at = np.where(valid, idx, 0)
    s = np.where(valid, np.take_along_axis(p, at, 1), 0.0)
    tot = s.sum(1, keepdims=True)
    r = s / np.where(tot > 0, tot, 1.0)
    g = np.where(valid, np.abs(gw) * 1.5, 0.0)
    size = np.zeros((T, E))
    np.add.at(size, (np.arange(T)[:, None], at), r * (g + (r * g).sum(1, keepdims=True)))
    # the exponent's argument, at most 110 where exp is not 0, carries a
    # rounding; k + 96 operations; the gradient of scores below 2^-126 may be 0
    for probs in (None, gp):
        got = ep.ep_router_backward(logits, ti, tw, None if probs is None else torch.from_numpy(gp).to(DEV),
                                    score="sigmoid", scale=1.5)
        ref = moe.router_backward(l, idx, gw, probs, "sigmoid", True, 1.5)
        assert np.abs(ref[0]).max() > 0.01                      # nothing vanishes in the definition
        err = size * (k + 96 + 110) * U + 2.0 ** -126 * (1 + np.abs(gp))
        if probs is not None:
            err = err + p * np.abs(gp) * 96 * U
        check(got, ref, rounded(ref, err, dtype), f"probs={probs is not None}")


def test_backward_where_the_weights_are_zero():
    # below about -709.78 every score is 0 in the 64 bits of the forward, and
    # so are its weights; the gradient follows it on both sides
    l = torch.tensor([[-709.5, -709.75, -800.0], [-709.8125, -710.0, -9999.0]], device=DEV)
    idx, w, _ = ep.ep_router(l, 2, score="sigmoid")
    g = torch.tensor([[1.0, -1.0], [1.0, -1.0]], device=DEV)
    got = ep.ep_router_backward(l, idx, g, score="sigmoid")
    assert bool((w[0] > 0.4).all()) and bool((w[1] == 0).all())
    assert float(got[0, 0]) > 0.4 and float(got[0, 1]) < -0.4 and bool((got[1] == 0).all())


def test_backward_against_differences():
    # a step in one logit changes the forward's sum(w g) by the gradient times
    # the step, around -95
    T, E, k = 5, 12, 3
    rng = np.random.default_rng(2)
    l = np.round((-95.0 + rng.normal(size=(T, E))) * 1024) / 1024      # steps of 2^-7 are exact
    logits = torch.from_numpy(l.astype(np.float32)).to(DEV)
    gw = torch.from_numpy(rng.normal(size=(T, k)).astype(np.float32)).to(DEV)
    idx, _, _ = ep.ep_router(logits, k, score="sigmoid")
    g = f64(ep.ep_router_backward(logits, idx, gw, score="sigmoid"))
    h = 2.0 ** -7
    for e in range(E):
        side = []
        for d in (h, -h):
            x = logits.clone()
            x[:, e] += d
            i, w, _ = ep.ep_router(x, k, score="sigmoid")
            side.append(((w.double() * gw.double()).sum(1), (i == idx).all(1)))
        (a, sa), (b, sb) = side
        same = (sa & sb).cpu().numpy()
        # h^2/6 of a third derivative below 30, and fp32 roundings of weights
        # of size 1 over h
        assert np.all(np.abs(f64((a - b) / (2 * h)) - g[:, e])[same] < 30 * h * h / 6 + 30 * U / h)
