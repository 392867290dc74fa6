"""The experts' products at the ends of what a call may have."""

import pytest
import torch

from combine_ep_layout_04_amd import ep

from moe_util import DEV

pytestmark = pytest.mark.gpu


def small(shape, most, seed):
    """Whole numbers up to `most`: their products' sums below are exact."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randint(-most, most + 1, shape, generator=g, device=DEV).float()


@pytest.mark.parametrize("kind", ["bf16", "8 bits"])
def test_most_rows(kind):
    """2^31 - 1 rows, all but three of them one expert's."""
    R, first, M, K = (1 << 31) - 1, 3, 7, 16
    x, w = small((M, K), 2, 1), small((2, 1, K), 1, 2)
    table = (x.double() @ w[:, 0].double().t()).t().bfloat16()      # of 16 terms up to 2: exact
    src = torch.arange(R, dtype=torch.int32, device=DEV).remainder_(M)
    off = torch.tensor([0, first, R], dtype=torch.int32, device=DEV)
    out = torch.full((R, 1), 77.0, dtype=torch.bfloat16, device=DEV)
    if kind == "bf16":
        ep.ep_expert_matmul(x.bfloat16(), w.bfloat16(), off, src=src, out=out)
    else:
        codes = [t.to(torch.float8_e4m3fn).view(torch.uint8) for t in (x, w)]
        ep.ep_expert_matmul_fp8(codes[0], torch.ones(M, 1, device=DEV), codes[1], torch.ones(2, 1, 1, device=DEV),
                                off, src=src, out=out)
    assert torch.equal(out[:first, 0], table[0][src[:first].long()])
    step = 1 << 28
    for a in range(first, R, step):
        b = min(a + step, R)
        assert torch.equal(out[a:b, 0], table[1].index_select(0, src[a:b])), a


@pytest.mark.parametrize("kind", ["bf16", "8 bits"])
def test_all_experts_of_the_widest_output(kind):
    """1024 experts of 2^20 outputs, a row each: more than 2^32 threads."""
    E, N, K = 1024, 1 << 20, 16 if kind == "8 bits" else 8
    x = small((E, K), 2, 3)
    some = small((61, K), 1, 4)         # weights' rows; which of them an output takes: (expert + output) % 61
    x8 = x.to(torch.float8_e4m3fn).view(torch.uint8)
    held = some.to(torch.float8_e4m3fn).view(torch.uint8) if kind == "8 bits" else some.bfloat16()
    w = torch.empty(E, N, K, dtype=held.dtype, device=DEV)
    at = torch.arange(N, device=DEV)
    for e in range(E):
        w[e] = held[(e + at) % 61]
    off = torch.arange(E + 1, dtype=torch.int32, device=DEV)
    if kind == "8 bits":
        got = ep.ep_expert_matmul_fp8(x8, torch.ones(E, 1, device=DEV), w, torch.ones(E, N // 128, 1, device=DEV), off)
    else:
        got = ep.ep_expert_matmul(x.bfloat16(), w, off)
    table = (x.double() @ some.double().t()).bfloat16()             # exact
    for e in range(E):
        assert torch.equal(got[e], table[e][(e + at) % 61]), e


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("each", [3, 500])
def test_range_of_the_gated_gradient(dtype, each):
    """The gradient of gate and up is of the rows' type between the activation
    and the products: in fp16 infinite past 65504 and 0 below 2^-25, also where
    the sums over it are neither; bf16 has the range of fp32."""
    K, half = 16, 8
    w = torch.full((1, 2 * half, K), 2.0 ** -10, dtype=dtype, device=DEV)
    x = torch.full((each, K), 1024.0, dtype=dtype, device=DEV)
    pre = torch.zeros(each, 2 * half, dtype=dtype, device=DEV)
    for g, up, d in ((32768.0, 8.0, 2.0 ** 17), (2.0 ** -24, 2.0 ** -3, 2.0 ** -28)):
        # gate 0: d_gate = g up / 2, d_up = 0; in one row, so all sums are exact
        grad = torch.zeros(each, half, dtype=dtype, device=DEV)
        grad[0] = g
        pre[:, half:] = up
        gr, gw = ep.ep_expert_glu_backward(grad, pre, x, w, weights_dtype=torch.float32)
        if dtype == torch.float16:
            d = float("inf") if d > 1 else 0.0
        assert bool((gr[0] == half * d * 2.0 ** -10).all()) and bool((gw[0, :half] == d * 1024).all())
        assert bool((gr[1:] == 0).all()) and bool((gw[0, half:] == 0).all())
