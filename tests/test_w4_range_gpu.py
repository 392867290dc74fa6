"""ep_expert_matmul_w4 over the whole range of bf16: rows of x near its largest
and its smallest values, where the product itself is an ordinary number."""

import numpy as np
import pytest
import torch

from combine_ep_layout_04_amd import ep
from oracle import moe

from moe_util import DEV, TYPES, U, check, f64, rounded

pytestmark = pytest.mark.gpu


SIZES = [
    (127, -120), (123, -117), (121, -115),      # sums of (16 + code) x past fp32's largest
    (100, -95), (0, -6), (-100, 95),
    (-114, 108), (-120, 114), (-124, 118),      # products of a part of x below fp32's smallest normal
    (126, -6), (-114, -6),                      # results near the ends too
]
WEIGHTS = [(128, False, False), (64, True, False), (32, False, False), (32, True, True), (128, True, True)]


# not gated where the activation's product would leave the range
@pytest.mark.parametrize("x_exp,s_exp,group,zeros,gated", [
    s + w for s in SIZES for w in WEIGHTS if not w[2] or abs(s[0] + s[1]) <= 20])
@pytest.mark.parametrize("T", [3, 40])
def test_range(x_exp, s_exp, group, zeros, gated, T):
    N, K = 50, 288
    rng = np.random.default_rng(7)
    ng = (K + group - 1) // group
    codes = rng.integers(0, 256, (1, N, K // 2)).astype(np.uint8)
    s = torch.from_numpy((rng.random((1, N, ng)) + 0.5) * 2.0 ** (s_exp - 3)).bfloat16()
    z = rng.integers(0, 16, (1, N, ng)).astype(np.uint8) if zeros else None
    # magnitudes of 2^x_exp and one octave down, all of one sign in row 1
    x = (rng.random((T, K)) + 1.0) * 2.0 ** (x_exp - 1) * np.where(rng.random((T, K)) < 0.5, -1.0, 1.0)
    x[1] = np.abs(x[1])
    x = torch.from_numpy(x).bfloat16()
    W = ep.ep_w4_pack(torch.from_numpy(codes).to(DEV), s.to(DEV),
                      None if z is None else torch.from_numpy(z).to(DEV), group_size=group, gated=gated)
    got = ep.ep_expert_matmul_w4(x.to(DEV), W)
    xs = f64(x)
    deq = moe.w4_dequantize(codes, f64(s), z, group)[0]
    out = xs @ deq.T
    # each product enters fp32 sums as (16 + code) x and leaves as (16 + zero)
    # x: at most 62 scale |x| in sums of at most 128 terms a group
    size = np.abs(xs) @ (f64(s)[0][:, np.arange(K) // group] * 62.0).T
    err = size * (128 + K / 128 + 8) * U
    if gated:
        h = N // 2
        g, u, eg, eu = out[:, :h], out[:, h:], err[:, :h], err[:, h:]
        out = moe.silu(g) * u
        err = 1.1 * np.abs(u) * eg + np.abs(moe.silu(g)) * eu + 1.1 * eg * eu \
            + np.abs(out) * (np.abs(g) + 8) * 2 * U
    largest = torch.finfo(torch.bfloat16).max
    assert np.abs(out).max() < largest * 0.9
    check(got, out, rounded(out, err, "bf16"), f"2^{x_exp}")
    # and no looser than the result's own rounding over the whole
    norm = np.linalg.norm
    if not gated:
        assert norm(f64(got) - out) <= norm(np.abs(out)) * 2.0 ** -8
