"""ep_expert_matmul_fp8 against the 64-bit form on the decoded values."""

import numpy as np
import pytest
import torch

from combine_ep_layout_04_amd import ep

from expert_util import glu, product, ragged, segments
from moe_util import DEV, TYPES, check, rounded

pytestmark = pytest.mark.gpu

CODES = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}

CASES = [
    # rows an expert (about), E, K, N, format, scales, columns, gated, dtype, gather, align
    (1, 1, 16, 1, "e4m3", "fp32", False, False, "bf16", False, 1),
    (1, 1, 2048, 999, "e5m2", "ue8m0", False, False, "fp16", False, 1),
    (1, 9, 1408, 260, "e4m3", "fp32", False, True, "bf16", True, 1),
    (7, 5, 144, 300, "e4m3", "ue8m0", True, True, "bf16", True, 1),
    (12, 300, 128, 32, "e5m2", "fp32", True, False, "bf16", False, 1),
    (28, 3, 656, 130, "e4m3", "fp32", False, False, "fp16", True, 1),
    (25, 2, 112, 34, "e5m2", "ue8m0", False, True, "fp16", False, 1),
    (60, 4, 512, 256, "e4m3", "fp32", False, True, "bf16", False, 1),
    (100, 3, 208, 300, "e4m3", "fp32", True, False, "bf16", True, 1),
    (70, 3, 640, 420, "e5m2", "ue8m0", False, True, "bf16", True, 1),      # halves of 210: two scales a tile
    (130, 2, 96, 130, "e4m3", "fp32", True, True, "fp16", True, 1),
    (300, 2, 384, 512, "e4m3", "fp32", False, True, "bf16", True, 1),
    (260, 3, 272, 500, "e5m2", "fp32", True, False, "fp16", False, 1),
    (500, 1, 1040, 768, "e4m3", "ue8m0", False, False, "bf16", False, 1),
    (220, 2, 256, 202, "e4m3", "fp32", False, True, "bf16", False, 1),
    (6, 40, 272, 1030, "e5m2", "fp32", True, False, "fp16", True, 1),      # many experts: few rows, tiles from 9 on
    (14, 16, 272, 2560, "e4m3", "fp32", False, True, "bf16", True, 1),
    (20, 40, 144, 1000, "e4m3", "ue8m0", False, False, "fp16", False, 1),
    (64, 1, 528, 300, "e4m3", "fp32", False, True, "bf16", False, 1),      # one expert: few rows up to 64
    (20, 4, 128, 64, "e4m3", "fp32", False, True, "bf16", False, 32),
    (200, 4, 128, 256, "e4m3", "fp32", False, True, "bf16", True, 128),
]


def codes(rng, n, k, fmt):
    """Random finite codes (all of them, subnormal and largest included)."""
    c = rng.integers(0, 256, (n, k)).astype(np.uint8)
    v = torch.from_numpy(c).view(CODES[fmt]).double().numpy()
    c[~np.isfinite(v)] = 0
    return c, torch.from_numpy(c).view(CODES[fmt]).double().numpy()


def aligned(x, w):
    """What the matrix cores' 8-bit instructions drop: they line up each 8
    products by the largest exponent and keep 13 bits below it, so each of 7
    products is off by less than 2^-13 of the largest one (of at most the
    product of the largest factors)."""
    def largest(v):
        return np.abs(v).reshape(len(v), -1, 8).max(2)
    return 7 * 2.0 ** -13 * (largest(x) @ largest(w).T)


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_product(case):
    each, E, K, N, fmt, scale, columns, gated, dtype, gather, align = case
    rng = np.random.default_rng(7)
    n = ragged(rng, E, each, empty=[E // 2] if E > 2 else [])
    counts, offsets = segments(n, DEV, align)
    off = offsets.cpu().numpy()
    R = int(off[E]) + (5 if each > 1 else 0)
    M = max(1, R // 2) if gather else R
    B = (K + 127) // 128
    cx, vx = codes(rng, M, K, fmt)
    cw, vw = codes(rng, E * N, K, "e4m3")
    cw, vw = cw.reshape(E, N, K), vw.reshape(E, N, K)
    big = {"e4m3": 448.0, "e5m2": 57344.0}[fmt]
    xs = np.exp(rng.normal(size=(M, B))).astype(np.float32) / np.float32(big)
    if scale == "ue8m0":
        held = (np.floor(np.log2(xs)) + 127).astype(np.uint8)
        xs = np.exp2(held.astype(np.float64) - 127)
    else:
        held = xs
    ws = (np.exp(rng.normal(size=(E, (N + 127) // 128, B))) / 448 / np.sqrt(K)).astype(np.float32)
    src = rng.integers(0, M, R).astype(np.int32) if gather else None
    pad = 16 if align > 1 else 0
    tx = torch.full((M, K + pad), 0x7F, dtype=torch.uint8, device=DEV)[:, :K]
    tx.copy_(torch.from_numpy(cx))
    ts = torch.from_numpy(held).to(DEV)
    if columns:
        hold = torch.zeros(B, (M + 15) // 16 * 16, dtype=ts.dtype, device=DEV)
        hold[:, :M] = ts.t()
        ts = hold.t()[:M]
    M_out = N // 2 if gated else N
    buf = torch.full((R + 2, M_out + 3), 7.0, dtype=TYPES[dtype], device=DEV)
    kw = dict(fmt=fmt, gated=gated, src=None if src is None else torch.from_numpy(src).to(DEV), rows=R,
              counts=counts if align > 1 else None, dtype=TYPES[dtype])
    tw, tws = torch.from_numpy(cw).to(DEV), torch.from_numpy(ws).to(DEV)
    got = ep.ep_expert_matmul_fp8(tx, ts, tw, tws, offsets, out=buf[:, :M_out], **kw)
    used = np.zeros(R, bool)
    for e in range(E):
        used[off[e]:off[e] + n[e]] = True
    used = torch.from_numpy(used).to(DEV)
    assert bool((buf[:R][~used] == 7.0).all()) and bool((buf[R:] == 7.0).all())
    assert bool((buf[:, M_out:] == 7.0).all())
    x = vx * xs.astype(np.float64).repeat(128, 1)[:, :K]
    for e in range(E):
        a, b = off[e], off[e] + n[e]
        if a == b:
            continue
        w = vw[e] * ws[e].astype(np.float64).repeat(128, 0)[:N].repeat(128, 1)[:, :K]
        xe = x[a:b] if src is None else x[src[a:b]]
        ref, err = product(xe, w)
        # the tiles: with many of them from 9 rows an expert on, else from 33
        if R // min(R, E) > (8 if min(R, E) * N // 256 > 128 else 32):
            err += aligned(xe, w)
        if gated:
            ref, err = glu(ref, err)
        check(got[a:b], ref, rounded(ref, err, dtype), f"expert {e}")
    again = ep.ep_expert_matmul_fp8(tx, ts, tw, tws, offsets, **kw)
    assert torch.equal(again[used].view(torch.int16), got[:R][used].contiguous().view(torch.int16))


@pytest.mark.parametrize("scale,fmt", [("fp32", "e4m3"), ("pow2", "e4m3"), ("ue8m0", "e4m3"), ("fp32", "e5m2")])
@pytest.mark.parametrize("columns", [False, True])
def test_takes_what_the_dispatch_writes(scale, fmt, columns):
    """Rows cast by ep_dispatch, through the layout's offsets, row-major and
    column-major scales."""
    T, H, E, k, N = 70, 384, 4, 2, 96
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn(T, H, generator=g, device=DEV).bfloat16()
    idx = torch.rand(T, E, generator=g, device=DEV).argsort(1)[:, :k].contiguous()
    _, offsets, slot, src, _ = ep.ep_layout(idx, E)
    R = T * k
    ld = (R + 15) // 16 * 16
    q, s, _ = ep.ep_dispatch(x, slot, fp8=True, fmt=fmt, scale=scale, scale_ld=ld if columns else 0)
    rows = s.t()[:R] if columns else s
    cw, _ = codes(np.random.default_rng(1), E * N, H, "e4m3")
    w = torch.from_numpy(cw.reshape(E, N, H)).to(DEV)
    ws = torch.rand(E, 1, H // 128, generator=g, device=DEV) / 448
    got = ep.ep_expert_matmul_fp8(q, rows, w, ws, offsets, fmt=fmt)
    # the tokens cast once each, read through src, give the same bits
    alone = torch.arange(T, dtype=torch.int32, device=DEV).reshape(T, 1)
    tq, tscale, _ = ep.ep_dispatch(x, alone, fp8=True, fmt=fmt, scale=scale)
    also = ep.ep_expert_matmul_fp8(tq, tscale, w, ws, offsets, fmt=fmt, src=src)
    assert torch.equal(got.view(torch.int16), also.view(torch.int16))
    v = q.cpu().view(CODES[fmt]).double().numpy()
    f = np.exp2(rows.cpu().double().numpy() - 127) if scale == "ue8m0" else rows.cpu().double().numpy()
    xv = v * f.repeat(128, 1)
    wv = w.cpu().view(CODES["e4m3"]).double().numpy() * ws.cpu().double().numpy().repeat(N, 1).repeat(128, 2)
    off = offsets.cpu().numpy()
    for e in range(E):
        a, b = off[e], off[e + 1]
        ref, err = product(xv[a:b], wv[e])
        err += aligned(xv[a:b], wv[e])
        check(got[a:b], ref, rounded(ref, err, "bf16"), f"expert {e}")


@pytest.mark.parametrize("each", [3, 40, 250])
def test_exact_sums(each):
    """Small whole numbers and powers of two as scales: the result is exact,
    to the bit, in every kernel."""
    E, K, N = 2, 272, 160
    rng = np.random.default_rng(11)
    x = rng.integers(-2, 3, (each * E, K)).astype(np.float64)
    w = rng.integers(-1, 2, (E, N, K)).astype(np.float64)
    B = 3
    bx = rng.integers(126, 129, (each * E, B)).astype(np.uint8)
    ws = np.exp2(rng.integers(-1, 2, (E, 2, B))).astype(np.float32)
    cx = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).to(DEV)
    cw = torch.from_numpy(w).to(torch.float8_e4m3fn).view(torch.uint8).to(DEV)
    _, off = segments(np.array([each] * E), DEV)
    got = ep.ep_expert_matmul_fp8(cx, torch.from_numpy(bx).to(DEV), cw, torch.from_numpy(ws).to(DEV), off,
                                  dtype=torch.float16)
    xv = x * np.exp2(bx.astype(np.float64) - 127).repeat(128, 1)[:, :K]
    for e in range(E):
        wv = w[e] * ws[e].astype(np.float64).repeat(128, 0)[:N].repeat(128, 1)[:, :K]
        ref = torch.from_numpy(xv[e * each:(e + 1) * each] @ wv.T)      # multiples of 1/4 below 2^13
        assert torch.equal(got[e * each:(e + 1) * each].cpu(), ref.half())


@pytest.mark.parametrize("each", [3, 40, 250])
def test_special_scales_and_codes(each):
    """A NaN code, an infinite scale (byte 255) and the smallest one (byte 0)
    reach their own rows only."""
    K, N = 256, 64
    one = 0x38
    x = torch.full((each, K), one, dtype=torch.uint8, device=DEV)
    x[0, 5] = 0x7F
    s = torch.full((each, 2), 127, dtype=torch.uint8, device=DEV)
    s[1, 0], s[2] = 255, 0
    w = torch.full((1, N, K), one, dtype=torch.uint8, device=DEV)
    ws = torch.full((1, 1, 2), 2.0 ** 20, device=DEV)
    got = ep.ep_expert_matmul_fp8(x, s, w, ws)
    assert bool(torch.isnan(got[0]).all()) and bool(torch.isinf(got[1]).all())
    assert bool((got[2] == 2.0 ** (-127 + 20 + 8)).all()) and bool((got[3:] == 2.0 ** 28).all())


def test_no_rows():
    x = torch.empty(0, 128, dtype=torch.uint8, device=DEV)
    w = torch.zeros(2, 16, 128, dtype=torch.uint8, device=DEV)
    off = torch.zeros(3, dtype=torch.int32, device=DEV)
    out = ep.ep_expert_matmul_fp8(x, torch.empty(0, 1, device=DEV), w, torch.ones(2, 1, 1, device=DEV), off)
    assert out.shape == (0, 16)
