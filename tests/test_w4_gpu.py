"""ep_w4_pack and ep_expert_matmul_w4 against the 64-bit product with the
unpacked weights."""

import numpy as np
import pytest
import torch

from combine_ep_layout_04_amd import ep
from oracle import moe

from moe_util import DEV, TYPES, U, check, f64, rounded, routing, wide

pytestmark = pytest.mark.gpu

CASES = [
    # T, E, k, K, N, group, dtype, zeros, gated, gather, pad, shift
    (1, 1, 1, 32, 1, 32, "bf16", False, False, False, 0, 0),
    (1, 1, 1, 4096, 1000, 128, "fp16", True, False, False, 0, 0),
    (2, 4, 2, 64, 16, 64, "fp16", True, False, True, 0, 0),
    (3, 8, 2, 96, 17, 32, "bf16", False, False, True, 3, 1),
    (1, 256, 8, 160, 30, 128, "bf16", False, True, True, 0, 0),
    (5, 8, 3, 288, 33, 256, "fp16", True, False, False, 1, 0),
    (16, 8, 8, 128, 48, 32, "bf16", True, True, True, 0, 0),
    (17, 1, 1, 512, 50, 64, "fp16", False, True, False, 0, 3),
    (40, 2, 1, 544, 66, 128, "bf16", True, False, True, 0, 0),
    (65, 1, 1, 256, 130, 128, "bf16", False, False, False, 0, 0),
    (70, 2, 2, 192, 40, 32, "fp16", True, True, False, 8, 0),
    (130, 3, 2, 1056, 70, 384, "bf16", False, True, True, 0, 0),
    (300, 16, 2, 320, 36, 64, "bf16", True, False, True, 0, 0),
    (64, 1000, 3, 64, 20, 32, "fp16", False, False, True, 0, 0),
    (2, 3, 2, 2080, 100, 1024, "fp16", True, True, False, 0, 0),
]


def make(rng, E, N, K, group, dtype, zeros):
    ng = (K + group - 1) // group
    codes = rng.integers(0, 256, (E, N, K // 2)).astype(np.uint8)
    s = torch.from_numpy((rng.random((E, N, ng)) + 0.25) / np.sqrt(K) / 4).to(TYPES[dtype])
    z = rng.integers(0, 16, (E, N, ng)).astype(np.uint8) if zeros else None
    return codes, s, z


def product(x, W, gated, size_terms):
    """(result, error bound before rounding) of rows x [n, K] with W [N, K].

    Each product enters the sums as (16 + code) x, and the 16 + zero leaves
    again: at most 31 and 31 times scale |x|, in fp32 sums of at most 128
    terms a group and one term a group, and a few operations more."""
    out = x @ W.T
    ab = size_terms
    K = x.shape[1]
    err = ab * 2.0 * (128 + K / 128 + 8) * U
    if not gated:
        return out, err
    h = W.shape[0] // 2
    g, u, eg, eu = out[:, :h], out[:, h:], err[:, :h], err[:, h:]
    f = moe.silu(g) * u
    # |silu'| <= 1.1; the exponential's argument carries |g| roundings
    return f, 1.1 * np.abs(u) * eg + np.abs(moe.silu(g)) * eu + eg * eu * 1.1 + np.abs(f) * (np.abs(g) + 8) * 2 * U


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_product(case):
    T, E, k, K, N, group, dtype, zeros, gated, gather, pad, shift = case
    rng = np.random.default_rng(3)
    codes, s, z = make(rng, E, N, K, group, dtype, zeros)
    idx = routing(rng, T, E, k, 0.1 if T > 2 else 0.0, skew=T > 20)
    counts, offsets, slot, src, _ = ep.ep_layout(torch.from_numpy(idx).to(DEV), E)
    R = T * k
    n = int(offsets[E])
    x = torch.from_numpy(rng.normal(size=(T if gather else R, K))).to(TYPES[dtype]).double().numpy()
    tx = wide(x, dtype, pad, shift)
    if not gather:
        tx[n:] = float("nan")                    # rows of no expert
    W = ep.ep_w4_pack(torch.from_numpy(codes).to(DEV), s.to(DEV),
                      None if z is None else torch.from_numpy(z).to(DEV), group_size=group, gated=gated)
    M = N // 2 if gated else N
    out = torch.full((R + 3, M + pad), 7.0, dtype=TYPES[dtype], device=DEV)
    got = ep.ep_expert_matmul_w4(tx, W, offsets, src=src if gather else None, rows=R, out=out[:, :M])
    assert bool((out[n:] == 7.0).all()) and bool((out[:, M:] == 7.0).all())
    deq = moe.w4_dequantize(codes, f64(s), z, group)
    scale = f64(s)[:, :, np.arange(K) // group] * 62.0
    off, rows = offsets.cpu().numpy(), src.cpu().numpy()
    for e in range(E):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        xe = x[rows[a:b]] if gather else x[a:b]
        ref, err = product(xe, deq[e], gated, np.abs(xe) @ scale[e].T)
        check(got[a:b], ref, rounded(ref, err, dtype), f"expert {e}")
    # the same bits every time, and with the counts given
    again = ep.ep_expert_matmul_w4(tx, W, offsets, src=src if gather else None, rows=R, counts=counts)
    assert torch.equal(again[:n].view(torch.int16), got[:n].contiguous().view(torch.int16))


@pytest.mark.parametrize("group,dtype,zeros,gated", [
    (128, "bf16", False, False), (128, "fp16", True, True), (64, "bf16", True, False),
    (32, "fp16", False, True), (32, "bf16", True, False)])
@pytest.mark.parametrize("T,E,k,N", [
    # few rows an expert: over 32768 blocks of 16 outputs, over 4096, over
    # 1536, over 512, below
    (64, 16, 4, 16400), (16, 16, 4, 4008), (16, 16, 4, 1400), (16, 16, 4, 500), (2, 2, 1, 72),
    # over 16 rows an expert: over 16384, 6144, 4096, 1536, below
    (200, 4, 2, 16408), (200, 4, 2, 8008), (200, 4, 2, 5000), (200, 4, 2, 1800), (200, 4, 2, 200),
])
def test_every_split(T, E, k, N, group, dtype, zeros, gated):
    K = 96 if N > 2000 else 416
    rng = np.random.default_rng(N)
    codes, s, z = make(rng, E, N, K, group, dtype, zeros)
    idx = routing(rng, T, E, k)
    _, offsets, _, src, _ = ep.ep_layout(torch.from_numpy(idx).to(DEV), E)
    x = torch.from_numpy(rng.normal(size=(T, K))).to(TYPES[dtype])
    W = ep.ep_w4_pack(torch.from_numpy(codes).to(DEV), s.to(DEV),
                      None if z is None else torch.from_numpy(z).to(DEV), group_size=group, gated=gated)
    got = ep.ep_expert_matmul_w4(x.to(DEV), W, offsets, src=src)
    xs, off, rows = f64(x), offsets.cpu().numpy(), src.cpu().numpy()
    deq = moe.w4_dequantize(codes, f64(s), z, group)
    for e in range(E):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        xe = xs[rows[a:b]]
        ref, err = product(xe, deq[e], gated,
                           np.abs(xe) @ (f64(s)[e][:, np.arange(K) // group] * 62.0).T)
        check(got[a:b], ref, rounded(ref, err, dtype), f"expert {e}")


def test_one_expert_needs_no_offsets():
    rng = np.random.default_rng(8)
    codes, s, z = make(rng, 1, 70, 256, 128, "bf16", False)
    W = ep.ep_w4_pack(torch.from_numpy(codes).to(DEV), s.to(DEV))
    deq = moe.w4_dequantize(codes, f64(s), None, 128)[0]
    for T in (1, 2, 15, 16, 17, 33, 64, 65, 200):
        x = torch.from_numpy(rng.normal(size=(T, 256))).bfloat16()
        got = ep.ep_expert_matmul_w4(x.to(DEV), W)
        xe = f64(x)
        ref, err = product(xe, deq, False, np.abs(xe) @ (f64(s)[0][:, np.arange(256) // 128] * 62.0).T)
        check(got, ref, rounded(ref, err, "bf16"), f"T={T}")


@pytest.mark.parametrize("alignment,capacity", [(16, 0), (1, 40)])
def test_padded_layouts(alignment, capacity):
    T, E, k, K, N = 50, 6, 2, 128, 24
    rng = np.random.default_rng(9)
    codes, s, _ = make(rng, E, N, K, 128, "fp16", False)
    W = ep.ep_w4_pack(torch.from_numpy(codes).to(DEV), s.to(DEV))
    idx = torch.from_numpy(routing(rng, T, E, k, 0.1)).to(DEV)
    R = ep.layout_max_rows(T, k, E, alignment, capacity)
    counts, offsets, slot, src, _ = ep.ep_layout(idx, E, alignment=alignment, capacity=capacity)
    x = torch.randn(T, K, device=DEV).half()
    out = torch.full((R, N), 7.0, dtype=torch.float16, device=DEV)
    ep.ep_expert_matmul_w4(x, W, offsets, src=src, counts=counts, rows=R, out=out)
    deq = moe.w4_dequantize(codes, f64(s), None, 128)
    c, o, r = counts.cpu().numpy(), offsets.cpu().numpy(), src.cpu().numpy()
    untouched = np.ones(R, dtype=bool)
    for e in range(E):
        a, b = o[e], o[e] + c[e]
        untouched[a:b] = False
        if a == b:
            continue
        xe = f64(x)[r[a:b]]
        ref, err = product(xe, deq[e], False, np.abs(xe) @ (f64(s)[e][:, np.arange(K) // 128] * 62.0).T)
        check(out[a:b], ref, rounded(ref, err, "fp16"), f"expert {e}")
    assert bool((out[torch.from_numpy(untouched).to(DEV)] == 7.0).all())


def test_an_infinity_stays_in_its_row():
    K, N = 160, 20
    rng = np.random.default_rng(1)
    codes, s, _ = make(rng, 1, N, K, 128, "bf16", False)
    W = ep.ep_w4_pack(torch.from_numpy(codes).to(DEV), s.to(DEV))
    x = torch.randn(4, K, device=DEV).bfloat16()
    x[1, 7], x[2, 150] = float("inf"), float("nan")
    got = ep.ep_expert_matmul_w4(x, W)
    assert bool(torch.isfinite(got[[0, 3]].float()).all())
    assert not bool(torch.isfinite(got[[1, 2]].float()).any())
    assert torch.equal(got[:1], ep.ep_expert_matmul_w4(x[:1], W))


def test_counts_and_offsets_past_the_rows_are_bounded():
    # offsets that claim more rows than the buffers have: only those within
    W = ep.ep_w4_pack(torch.zeros(2, 16, 32, dtype=torch.uint8, device=DEV),
                      torch.ones(2, 16, 1, dtype=torch.bfloat16, device=DEV), group_size=64)
    x = torch.ones(8, 64, device=DEV).bfloat16()
    offsets = torch.tensor([0, 6, 60], dtype=torch.int32, device=DEV)
    out = torch.full((12, 16), 7.0, device=DEV).bfloat16()
    ep.ep_expert_matmul_w4(x, W, offsets, rows=8, out=out)
    assert bool((out[:8] == -512).all()) and bool((out[8:] == 7).all())


def test_weights_past_32_bits():
    # 3.2 GB of packed weights, the last experts chosen
    E, N, K = 96, 4096, 16384
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GiB free")
    g = torch.Generator(device=DEV).manual_seed(3)
    codes = torch.randint(0, 256, (E, N, K // 2), generator=g, device=DEV, dtype=torch.uint8)
    s = (torch.rand(E, N, K // 128, generator=g, device=DEV) / 512).bfloat16()
    W = ep.ep_w4_pack(codes, s)
    assert W.packed.numel() > 1 << 31
    idx = torch.tensor([[E - 1, 0, E - 2]], dtype=torch.int64, device=DEV)
    _, offsets, _, src, _ = ep.ep_layout(idx, E)
    x = torch.randn(1, K, generator=g, device=DEV).bfloat16()
    got = ep.ep_expert_matmul_w4(x, W, offsets, src=src)
    for r, e in enumerate((0, E - 2, E - 1)):
        deq = moe.w4_dequantize(codes[e:e + 1].cpu().numpy(), f64(s[e:e + 1]), None, 128)[0]
        xe = f64(x)
        ref, err = product(xe, deq, False, np.abs(xe) @ (f64(s[e])[:, np.arange(K) // 128] * 62.0).T)
        check(got[r:r + 1], ref, rounded(ref, err, "bf16"), f"expert {e}")


def test_refuses():
    codes = torch.zeros(2, 8, 32, dtype=torch.uint8, device=DEV)
    s = torch.ones(2, 8, 1, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(TypeError, match="scales"):
        ep.ep_w4_pack(codes, s.float(), group_size=64)
    with pytest.raises(ValueError, match="scales must be"):
        ep.ep_w4_pack(codes, s, group_size=32)
    with pytest.raises(ValueError, match="invalid"):
        ep.ep_w4_pack(codes, s, group_size=48)
    with pytest.raises(ValueError, match="invalid"):
        ep.ep_w4_pack(codes[:, :7].contiguous(), s[:, :7].contiguous(), group_size=64, gated=True)
    W = ep.ep_w4_pack(codes, s, group_size=64)
    x = torch.zeros(3, 64, device=DEV).bfloat16()
    offsets = torch.tensor([0, 1, 3], dtype=torch.int32, device=DEV)
    with pytest.raises(TypeError, match="x must be"):
        ep.ep_expert_matmul_w4(x.half(), W, offsets)
    with pytest.raises(ValueError, match="columns"):
        ep.ep_expert_matmul_w4(x[:, :32], W, offsets)
    with pytest.raises(ep.EpError, match="offsets"):
        ep.ep_expert_matmul_w4(x, W)
    with pytest.raises(ep.EpError, match="rows"):
        ep.ep_expert_matmul_w4(x, W, offsets, rows=4)
    with pytest.raises(ValueError, match="out has"):
        ep.ep_expert_matmul_w4(x, W, offsets, out=torch.empty(2, 8, device=DEV).bfloat16())
