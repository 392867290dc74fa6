"""ep_router and its backward on logits of +inf: sigmoid scores are 1; softmax
scores of that row are NaN as the formula's are, and never reach another row."""

import itertools

import numpy as np
import pytest
import torch

from combine_ep_layout_04_amd import ep
from oracle import moe

from moe_util import DEV, TYPES, U, check, f64, wide

pytestmark = pytest.mark.gpu

INF = float("inf")
# T, E, k, groups, topk_groups: each split of a row over lanes
SHAPES = [(9, 8, 3, 2, 1), (33, 16, 4, 4, 2), (20, 60, 4, 5, 2), (1030, 128, 6, 8, 3), (17, 130, 8, 10, 4),
          (2050, 256, 8, 8, 4), (6, 256, 12, 8, 4), (5, 700, 10, 7, 2)]


def make(rng, T, E, dtype):
    """Rows 0, 3, ... of ordinary logits, the others with one or two of +inf;
    some logits masked."""
    a = rng.normal(size=(T, E)) * 2.0
    a[rng.random((T, E)) < 0.2] = -INF
    a[:, 1] = 0.5
    hit = np.arange(T) % 3 != 0
    a[hit, rng.integers(2, E, T)[hit]] = INF
    a[np.arange(T) % 3 == 2, E // 2] = INF
    return torch.from_numpy(a).to(TYPES[dtype]).double().numpy(), hit


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("mode", ["plain", "groups", "groups by two", "bias", "bias and groups"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda c: "-".join(map(str, c)))
def test_forward(shape, mode, dtype):
    T, E, k, groups, tg = shape
    rng = np.random.default_rng(4)
    l, hit = make(rng, T, E, dtype)
    bias = (rng.random(E) * 0.2 - 0.1).astype(np.float32) if "bias" in mode else None
    kw = dict(num_groups=groups if "groups" in mode else 1, topk_groups=tg if "groups" in mode else 1,
              group_top=2 if "two" in mode or mode == "bias and groups" else 1)
    logits = wide(l, dtype)
    tb = None if bias is None else torch.from_numpy(bias).to(DEV)
    tol = (110 + 64) * U
    for score, renorm in itertools.product(("softmax", "sigmoid"), (True, False)):
        idx, w, p = ep.ep_router(logits, k, score=score, bias=tb, renormalize=renorm, want_probs=True, **kw)
        with np.errstate(all="ignore"):
            ri, rw, rp = moe.router(l, k, score, bias, kw["num_groups"], kw["topk_groups"],
                                    kw["group_top"], renorm)
        assert np.array_equal(idx.cpu().numpy(), ri)
        gw, gp, gi = f64(w), f64(p), idx.cpu().numpy()
        fine = ~hit if score == "softmax" else np.ones(T, dtype=bool)
        check(w[torch.from_numpy(fine).to(DEV)], rw[fine], np.abs(rw[fine]) * tol + 2.0 ** -126, "weights")
        check(p[torch.from_numpy(fine).to(DEV)], rp[fine], rp[fine] * tol + 2.0 ** -126, "probs")
        if score == "softmax":
            masked = l == -INF
            assert np.all(np.isnan(gp[hit][~masked[hit]])) and np.all(gp[hit][masked[hit]] == 0)
            # values that are NaN leave no expert; by logit the +inf is first
            # and the weights are NaN
            if bias is not None or kw["group_top"] == 2:
                assert np.all(gi[hit] == -1) and np.all(gw[hit] == 0)
            else:
                first = np.argmax(l[hit] == INF, axis=1)
                assert np.array_equal(gi[hit][:, 0], first)
                assert np.all(np.isnan(gw[hit]) == (gi[hit] >= 0))


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda c: "-".join(map(str, c)))
def test_backward(shape, dtype):
    T, E, k, _, _ = shape
    rng = np.random.default_rng(5)
    l, hit = make(rng, T, E, dtype)
    logits = wide(l, dtype)
    gw = torch.randn(T, k, device=DEV)
    gp = torch.randn(T, E, device=DEV)
    masked = l == -INF
    for score, renorm, probs in itertools.product(("softmax", "sigmoid"), (True, False), (True, False)):
        idx, _, _ = ep.ep_router(logits, k, score=score)
        got = f64(ep.ep_router_backward(logits, idx, gw, gp if probs else None, score=score,
                                        renormalize=renorm))
        assert np.all(got[masked] == 0)
        if score == "sigmoid":                                  # a score of 1 does not move
            assert np.all(np.isfinite(got)) and np.all(got[l == INF] == 0)
            continue
        assert np.all(np.isfinite(got[~hit]))
        if probs or not renorm:
            assert np.all(np.isnan(got[hit][~masked[hit]]))
        else:
            chosen = np.zeros((T, E), dtype=bool)
            i = idx.cpu().numpy()
            for t in range(T):
                chosen[t, i[t][i[t] >= 0]] = True
            assert np.all(np.isnan(got[hit][chosen[hit]])) and np.all(got[hit][~chosen[hit]] == 0)
