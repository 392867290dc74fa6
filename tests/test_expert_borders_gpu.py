"""The borders between the kernels for few rows and the tiles, at exact row
counts, and what either does with 8-bit products that cancel."""

import numpy as np
import pytest
import torch

from combine_ep_layout_04_amd import ep

from expert_util import glu, product, segments
from moe_util import DEV, TYPES, check, f64, rounded

pytestmark = pytest.mark.gpu

# experts, outputs, rows an expert up to which the kernels for few rows go: 64
# with up to 32 tiles of 256 outputs, 32 with up to 128, else 8
BORDERS = [(1, 256, 64), (2, 4096, 64), (3, 4096, 32), (16, 1024, 32), (16, 2048, 32), (17, 2048, 8), (16, 2560, 8)]


def few_rows(R, E, N):
    hold = min(R, E)
    tiles = hold * N // 256
    return R // hold <= (8 if tiles > 128 else 32 if tiles > 32 else 64)


SIDES = [(E, N, each) for E, N, last in BORDERS for each in (last, last + 1)]


def test_sides():
    for E, N, last in BORDERS:
        assert few_rows(E * last, E, N) and not few_rows(E * (last + 1), E, N)


@pytest.mark.parametrize("E,N,each", SIDES)
def test_8_bits_that_cancel(E, N, each):
    """Two large products that cancel and a small one, all of one 8.  Few rows:
    the sum is within the roundings of fp32, 2 K 2^-24 of the terms' sizes; tiles
    may drop of each product what lies 2^-13 below the largest."""
    K = 16
    v = torch.zeros(2, K)                       # of x and of the weights
    v[:, 0], v[:, 1] = 448.0, torch.tensor([-448.0, 448.0])
    v[:, 2] = torch.tensor([2.0, 4.0])
    c = v.to(torch.float8_e4m3fn).view(torch.uint8).to(DEV)
    R = E * each
    _, off = segments(np.full(E, each), DEV)
    got = ep.ep_expert_matmul_fp8(c[0].expand(R, K).contiguous(), torch.ones(R, 1, device=DEV),
                                  c[1].expand(E, N, K).contiguous(), torch.ones(E, -(-N // 128), 1, device=DEV), off)
    terms = 2 * 448.0 ** 2 + 8
    tol = 2 * (K + 8) * 2.0 ** -24 * terms if few_rows(R, E, N) else 7 * 2.0 ** -13 * 448.0 ** 2
    assert tol < 8 or not few_rows(R, E, N)
    assert bool(((got.double() - 8).abs() <= tol + 2.0 ** -8 * 8).all())


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("E,N,each", SIDES)
def test_8_bits(E, N, each, gated):
    """All codes; few rows without an allowance for what tiles drop."""
    K, R = 272, E * each
    rng = np.random.default_rng(4)

    def codes(*shape):
        c = torch.from_numpy(rng.integers(0, 256, shape).astype(np.uint8))
        c[~torch.isfinite(c.view(torch.float8_e4m3fn).float())] = 0
        return c.to(DEV), c.view(torch.float8_e4m3fn).double().numpy()
    cx, vx = codes(R, K)
    cw, vw = codes(E, N, K)
    xs = (np.exp(rng.normal(size=(R, 3))) / 448).astype(np.float32)
    ws = (np.exp(rng.normal(size=(E, -(-N // 128), 3))) / 448 / K ** 0.5).astype(np.float32)
    _, off = segments(np.full(E, each), DEV)
    got = ep.ep_expert_matmul_fp8(cx, torch.from_numpy(xs).to(DEV), cw, torch.from_numpy(ws).to(DEV), off, gated=gated,
                                  dtype=torch.float16)
    x = vx * xs.astype(np.float64).repeat(128, 1)[:, :K]
    for e in range(0, E, 5):
        at = slice(e * each, (e + 1) * each)
        w = vw[e] * ws[e].astype(np.float64).repeat(128, 0)[:N].repeat(128, 1)[:, :K]
        ref, err = product(x[at], w)
        if not few_rows(R, E, N):
            top = [np.abs(v).reshape(len(v), -1, 8).max(2) for v in (x[at], w)]
            err = err + 7 * 2.0 ** -13 * (top[0] @ top[1].T)
        if gated:
            ref, err = glu(ref, err)
        check(got[at], ref, rounded(ref, err, "fp16"), f"expert {e}")


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("E,N,each", SIDES)
@pytest.mark.parametrize("dtype,K", [("bf16", 200), ("fp16", 131)])
def test_16_bits(E, N, each, dtype, K, gated):
    R = E * each
    g = torch.Generator(device=DEV).manual_seed(6)
    x = torch.randn(R, K, generator=g, device=DEV).to(TYPES[dtype])
    w = (torch.randn(E, N, K, generator=g, device=DEV) / K ** 0.5).to(TYPES[dtype])
    _, off = segments(np.full(E, each), DEV)
    got = ep.ep_expert_glu(x, w, off)[0] if gated else ep.ep_expert_matmul(x, w, off)
    for e in range(0, E, 5):
        at = slice(e * each, (e + 1) * each)
        ref, err = product(f64(x[at]), f64(w[e]))
        if gated:
            ref, err = glu(ref, err)
        check(got[at], ref, rounded(ref, err, dtype), f"expert {e}")


def test_dispatched_rows_without_allowance():
    """Rows as the dispatch casts them, few an expert: nothing is dropped."""
    T, H, E, k, N = 70, 384, 4, 2, 96
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn(T, H, generator=g, device=DEV).bfloat16()
    idx = torch.rand(T, E, generator=g, device=DEV).argsort(1)[:, :k].contiguous()
    _, offsets, slot, _, _ = ep.ep_layout(idx, E)
    assert few_rows(T * k, E, N)
    q, s, _ = ep.ep_dispatch(x, slot, fp8=True)
    cw = torch.randint(0, 0x70, (E, N, H), generator=g, device=DEV, dtype=torch.uint8)
    ws = torch.rand(E, 1, H // 128, generator=g, device=DEV) / 448
    got = ep.ep_expert_matmul_fp8(q, s, cw, ws, offsets, dtype=torch.float16)
    xv = f64(q.view(torch.float8_e4m3fn).float()) * f64(s).repeat(128, 1)
    wv = f64(cw.view(torch.float8_e4m3fn).float()) * f64(ws).repeat(N, 1).repeat(128, 2)
    off = offsets.tolist()
    for e in range(E):
        a, b = off[e], off[e + 1]
        ref, err = product(xv[a:b], wv[e])
        check(got[a:b], ref, rounded(ref, err, "fp16"), f"expert {e}")
