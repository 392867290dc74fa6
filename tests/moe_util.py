"""Helpers of the router, row movement and 4-bit product tests.

Tolerances count roundings: half a step of the result's type (relative
finfo.eps / 2, or half the smallest subnormal), plus 2^-24 per fp32 operation
on the sizes of what is added up."""

import numpy as np
import torch

DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
U = 2.0 ** -24
# half the smallest positive value
TINY = {"bf16": 2.0 ** -134, "fp16": 2.0 ** -25, "fp32": 2.0 ** -150}


def f64(t: torch.Tensor) -> np.ndarray:
    return t.double().cpu().numpy()


def half_step(ref: np.ndarray, dtype: str) -> np.ndarray:
    return np.abs(ref) * torch.finfo(TYPES[dtype]).eps / 2 + TINY[dtype]


def rounded(ref: np.ndarray, err: np.ndarray, dtype: str) -> np.ndarray:
    """Allowed distance of a result rounded to dtype from a value within err of ref."""
    return err + half_step(np.abs(ref) + err, dtype)


def check(got: torch.Tensor, ref: np.ndarray, tol: np.ndarray, what: str):
    g = f64(got)
    assert g.shape == ref.shape, (what, g.shape, ref.shape)
    bad = ~(np.abs(g - ref) <= tol)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} beyond the tolerance, first at "
                             f"{i}: got {g[i]!r} want {ref[i]!r} +- {np.broadcast_to(tol, ref.shape)[i]!r}")


def wide(a: np.ndarray, dtype: str, pad: int = 0, shift: int = 0) -> torch.Tensor:
    """a on the device in dtype, inside a NaN-filled buffer: `shift` elements
    from its start, rows `pad` elements apart beyond their width."""
    n, h = a.shape
    buf = torch.full((n * (h + pad) + shift + 1,), float("nan"), dtype=TYPES[dtype], device=DEV)
    v = buf[shift:shift + n * (h + pad)].view(n, h + pad)[:, :h]
    v.copy_(torch.from_numpy(a))
    return v


def routing(rng, T, E, k, masked=0.0, skew=False):
    p = np.arange(1, E + 1, dtype=float) ** (-1.5 if skew else 0.0)
    if k <= E:
        key = rng.gumbel(size=(T, E)) + np.log(p)
        idx = np.argsort(-key, axis=1)[:, :k].astype(np.int64)
    else:
        idx = rng.integers(0, E, (T, k)).astype(np.int64)
    idx[rng.random((T, k)) < masked] = -1
    return idx
