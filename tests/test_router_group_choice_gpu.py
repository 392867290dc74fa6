"""ep_router with groups rated by two values and no bias: groups are rated by
their scores, experts chosen by their logits, also where scores are equal
(sigmoid of large logits is 1, softmax far below the largest logit is 0)."""

import numpy as np
import pytest
import torch

from combine_ep_layout_04_amd import ep
from oracle import moe

from moe_util import DEV, TYPES, U, check, wide

pytestmark = pytest.mark.gpu

SHAPES = [
    # T, E, k, groups, topk_groups, pad: each split of a row over lanes
    (9, 8, 4, 2, 1, 0), (33, 16, 8, 4, 2, 3), (40, 24, 7, 3, 2, 0), (37, 64, 8, 8, 3, 1),
    (21, 128, 8, 8, 4, 0), (1030, 128, 8, 4, 2, 0), (17, 256, 8, 8, 4, 0), (2050, 256, 8, 8, 4, 0),
    (13, 130, 9, 10, 4, 2), (11, 512, 16, 16, 4, 0),
]


def saturated(rng, T, E, groups):
    """Per row some groups of large whole logits (a score of exactly 1 in 64
    bits from 38 on), the others of ordinary ones."""
    per = E // groups
    a = rng.normal(size=(T, E)) * 2.0
    for t in range(T):
        for g in range(groups):
            if rng.random() < 0.5:
                a[t, g * per:(g + 1) * per] = 38.0 + rng.permutation(per) % 200
    return a


def far_below(rng, T, E, dtype):
    """Ordinary logits, most of them 10000 lower: scores of exactly 0."""
    step = {"bf16": 64.0, "fp16": 8.0, "fp32": 1.0 / 128}[dtype]
    low = -10000.0 - step * np.stack([rng.permutation(E) for _ in range(T)])
    return np.where(rng.random((T, E)) < 0.8, low, rng.normal(size=(T, E)))


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda c: "-".join(map(str, c)))
def test_choice_by_logit(shape, score, dtype):
    T, E, k, groups, tg, pad = shape
    rng = np.random.default_rng(11)
    a = saturated(rng, T, E, groups) if score == "sigmoid" else far_below(rng, T, E, dtype)
    a[T // 2, rng.random(E) < 0.5] = -np.inf                    # masked ones stay out
    l = torch.from_numpy(a).to(TYPES[dtype]).double().numpy()
    logits = wide(l, dtype, pad)
    # as far as the exponent's argument reaches, 64 for sums over lanes and
    # the functions' own errors
    for renorm in (True, False):
        idx, w, _ = ep.ep_router(logits, k, score=score, num_groups=groups, topk_groups=tg,
                                 group_top=2, renormalize=renorm)
        ri, rw, _ = moe.router(l, k, score, None, groups, tg, 2, renorm)
        gi = idx.cpu().numpy()
        assert np.array_equal(gi, ri), f"{np.argwhere(gi != ri)[:3]}"
        check(w, rw, np.abs(rw) * (110 + 64) * U + 2.0 ** -126, "weights")


def test_choice_by_hand():
    l = torch.tensor([[38.0, 40.0, 50.0, 45.0, -1.0, 0.0, 1.0, 2.0]], device=DEV)
    idx, w, _ = ep.ep_router(l, 2, score="sigmoid", num_groups=2, topk_groups=1, group_top=2)
    assert idx.tolist() == [[2, 3]] and w.tolist() == [[0.5, 0.5]]
    # neighbouring fp32 logits whose scores are the same
    l = torch.full((1, 8), 25.0, device=DEV)
    l[0, 3] = torch.nextafter(l[0, 3], l[0, 3] + 1)
    idx, _, _ = ep.ep_router(l, 1, score="sigmoid", num_groups=2, topk_groups=1, group_top=2)
    assert idx.tolist() == [[3]]


def test_a_bias_of_zeros_still_chooses_by_value():
    # with a bias the definition compares values: equal scores tie
    l = torch.tensor([[38.0, 40.0, 50.0, 45.0, -1.0, 0.0, 1.0, 2.0]], device=DEV)
    idx, _, _ = ep.ep_router(l, 2, score="sigmoid", bias=torch.zeros(8, device=DEV), num_groups=2,
                             topk_groups=1, group_top=2)
    assert idx.tolist() == [[0, 1]]
