"""ep_expert_matmul_w4 where every sum is exact, so that the result has to be
the definition's, rounded once, to the bit: one wrong code, scale, zero point
or row of x shows at any width.  And random products held to the rounding of
their type over the whole result."""

import pytest
import torch

from combine_ep_layout_04_amd import ep

from moe_util import DEV, TYPES, U

pytestmark = pytest.mark.gpu


def make(g, E, N, K, group, zeros, dtype, exact):
    ng = (K + group - 1) // group
    codes = torch.randint(0, 256, (E, N, K // 2), generator=g, dtype=torch.uint8, device=DEV)
    if exact:       # powers of two
        s = 2.0 ** torch.randint(-8, -4, (E, N, ng), generator=g, device=DEV).double()
    else:
        s = (torch.rand(E, N, ng, generator=g, device=DEV, dtype=torch.float64) + 0.5) / (4.6 * K ** 0.5)
    s = s.to(TYPES[dtype])
    z = torch.randint(0, 16, (E, N, ng), generator=g, dtype=torch.uint8, device=DEV) if zeros else None
    return codes, s, z


def dequantized(codes, s, z, group):
    """One expert's [N, K] in 64 bits."""
    N, half = codes.shape
    q = torch.stack([codes & 15, codes >> 4], 2).reshape(N, 2 * half).double()
    at = torch.arange(2 * half, device=DEV) // group
    q -= 8.0 if z is None else z.double()[:, at]
    return q, s.double()[:, at]


def layout(g, T, E, k):
    idx = torch.rand(T, E, generator=g, device=DEV).argsort(1)[:, :k].contiguous()
    _, offsets, _, src, _ = ep.ep_layout(idx, E)
    return offsets, src


SHAPES = [
    # T, E, k, N, K: wide products, then each split of ep_w4.hip
    (1, 1, 1, 40, 4096), (3, 1, 1, 33, 16384), (1, 4, 2, 70, 65536), (40, 1, 1, 50, 16384), (130, 3, 2, 24, 8192),
    (64, 16, 4, 16400, 160), (16, 16, 4, 4008, 544), (16, 16, 4, 1400, 544), (16, 16, 4, 500, 1056), (2, 2, 1, 72, 2080),
    (200, 4, 2, 16408, 160), (200, 4, 2, 8008, 544), (200, 4, 2, 5000, 544), (200, 4, 2, 1800, 1056), (200, 4, 2, 200, 2080),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("group,zeros", [(32, True), (64, False), (128, True), (128, False), (1024, True)])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda c: "-".join(map(str, c)))
def test_exact(shape, group, zeros, dtype):
    T, E, k, N, K = shape
    g = torch.Generator(device=DEV).manual_seed(N + K)
    codes, s, z = make(g, E, N, K, group, zeros, dtype, True)
    # whole numbers: sums of (16 + code) x within a group of 128 stay whole
    # and below 2^14, sums of scale (code - zero) x a multiple of 2^-8 and
    # below 65536 * 15 * 2 / 32 < 2^16: 24 bits in all
    x = torch.randint(-2, 3, (T, K), generator=g, device=DEV).to(TYPES[dtype])
    offsets, src = layout(g, T, E, k)
    W = ep.ep_w4_pack(codes, s, z, group_size=group)
    got = ep.ep_expert_matmul_w4(x, W, offsets, src=src)
    for e in range(E):
        a, b = int(offsets[e]), int(offsets[e + 1])
        if a == b:
            continue
        q, sc = dequantized(codes[e], s[e], None if z is None else z[e], group)
        ref = x[src[a:b].long()].double() @ (q * sc).t()
        assert torch.equal(got[a:b], ref.to(TYPES[dtype])), e


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("group,zeros,gated", [(128, False, False), (32, True, False), (64, False, True),
                                               (128, True, True)])
@pytest.mark.parametrize("T,E,k,N,K", [(1, 1, 1, 400, 4096), (1, 2, 1, 200, 16384), (40, 1, 1, 300, 16384),
                                       (70, 4, 2, 100, 4096)])
def test_rounding_over_the_whole(T, E, k, N, K, group, zeros, gated, dtype):
    g = torch.Generator(device=DEV).manual_seed(5)
    codes, s, z = make(g, E, N, K, group, zeros, dtype, False)
    x = torch.randn(T, K, generator=g, device=DEV).to(TYPES[dtype])
    offsets, src = layout(g, T, E, k)
    got = ep.ep_expert_matmul_w4(x, ep.ep_w4_pack(codes, s, z, group_size=group, gated=gated), offsets,
                                 src=src).double()
    ref, spread = torch.empty_like(got), torch.empty_like(got)
    for e in range(E):
        a, b = int(offsets[e]), int(offsets[e + 1])
        q, sc = dequantized(codes[e], s[e], None if z is None else z[e], group)
        rows = x[src[a:b].long()].double()
        r = rows @ (q * sc).t()
        # the root of the sum of squares of what is added up, 62 scale |x|
        # each: roundings of 128 terms a group, each at most U of a partial
        # sum, which stays within 16 times that root of random signs
        p = (rows * rows) @ (62.0 * sc).square().t()
        p = p.sqrt() * 16
        if gated:
            n = N // 2
            gate, up = r[:, :n], r[:, n:]
            act = gate * torch.sigmoid(gate)
            ref[a:b] = act * up
            p = 1.1 * up.abs() * p[:, :n] + act.abs() * p[:, n:] + ref[a:b].abs() * (gate.abs() + 8)
            spread[a:b] = p
        else:
            ref[a:b], spread[a:b] = r, p
    half = ref.abs() * torch.finfo(TYPES[dtype]).eps / 2
    tiny = torch.finfo(TYPES[dtype]).smallest_normal * torch.finfo(TYPES[dtype]).eps / 2
    assert (got - ref).norm() <= (half + tiny + spread * U).norm()
    # the bound is the type's rounding, not the allowance for fp32 sums
    assert (spread * U).norm() < 0.5 * half.norm()
