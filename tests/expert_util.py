"""64-bit forms and error bounds of the experts' products.

Bounds count roundings: a sum of K products held in fp32 is off by at most
2 K 2^-24 sum |terms| (products of 16-bit values are exact in fp32; 2 for an
addition that cuts instead of rounding), the activation by a few fp32
operations, and a result rounded to 16 bits by half a step."""

import numpy as np
import torch

from moe_util import U

HALF = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}      # eps / 2: half a step, relative
SMALL = {"bf16": 2.0 ** -134, "fp16": 2.0 ** -25}   # half the smallest subnormal


def sigmoid(v):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-v))


def product(x, W):
    """(x W^T, its error bound in fp32) for x [n, K], W [N, K]."""
    return x @ W.T, 2.0 * (x.shape[1] + 8) * U * (np.abs(x) @ np.abs(W).T)


def glu(y, err):
    """silu(gate) * up of the halves of y, and its error bound."""
    h = y.shape[1] // 2
    g, u, eg, eu = y[:, :h], y[:, h:], err[:, :h], err[:, h:]
    s = sigmoid(g)
    f = g * s * u
    # |silu'| <= 1.1; the exponential's argument is rounded (|g| roundings)
    return f, 1.1 * np.abs(u) * eg + np.abs(g * s) * eu + 1.1 * eg * eu + np.abs(f) * (np.abs(g) + 8) * 2 * U


def glu_gradient(dh, pre, dtype):
    """d of gate and up [n, N] from dh [n, N/2] and pre [n, N], and its error
    bound: fp32 operations, then rounded to dtype."""
    h = pre.shape[1] // 2
    g, u = pre[:, :h], pre[:, h:]
    s = sigmoid(g)
    es = (np.abs(g) + 8) * 2 * U                    # relative error of s
    inner = 1.0 + g * (1.0 - s)
    dg, du = dh * u * s * inner, dh * g * s
    eg = np.abs(dh * u * s) * (es * np.abs(inner) + np.abs(g) * (s * es + 2 * U) + 8 * U * (1 + np.abs(g)))
    eu = np.abs(du) * (es + 4 * U)
    d, e = np.concatenate([dg, du], 1), np.concatenate([eg, eu], 1)
    return d, e + HALF[dtype] * (np.abs(d) + e) + SMALL[dtype]


def ragged(rng, E, rows, empty=()):
    """Rows per expert around `rows`, none for the experts in `empty`."""
    n = rng.integers(max(1, rows - rows // 3), rows + rows // 3 + 1, E)
    n[list(empty)] = 0
    return n


def segments(counts, device, align=1):
    """(counts, offsets) tensors of segments that start on multiples of align."""
    starts = np.concatenate([[0], np.cumsum((counts + align - 1) // align * align)])
    return (torch.from_numpy(counts.astype(np.int32)).to(device),
            torch.from_numpy(starts.astype(np.int32)).to(device))
