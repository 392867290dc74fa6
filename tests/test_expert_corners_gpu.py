"""Corners of the experts' products: no choice left, no rows, the widest inputs,
more experts than one look at their offsets finds, halves of one output."""

import numpy as np
import pytest
import torch

from combine_ep_layout_04_amd import ep

from expert_util import glu, glu_gradient, product, ragged, segments
from moe_util import DEV, TYPES, check, f64, rounded

pytestmark = pytest.mark.gpu


def values(g, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device=DEV).to(dtype)


def generator(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


@pytest.mark.parametrize("R", [3, 300, 3000])
@pytest.mark.parametrize("N,K", [(64, 72), (62, 67)])
def test_every_choice_masked(R, N, K):
    """All rows lie behind the last expert: nothing is written but zeros of the
    weights' gradients, whatever the rows hold."""
    E = 4
    g = generator(1)
    x, w = torch.full((R, K), float("nan"), dtype=torch.bfloat16, device=DEV), values(g, E, N, K)
    grad = torch.full((R, N), float("nan"), dtype=torch.bfloat16, device=DEV)
    off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)

    def buf(cols):
        return torch.full((R, cols), 7.0, dtype=torch.bfloat16, device=DEV)
    outs = [ep.ep_expert_matmul(x, w, off, out=buf(N)), *ep.ep_expert_glu(x, w, off, out=buf(N // 2), pre=buf(N))]
    for wide in (torch.bfloat16, torch.float32):
        gr, gw = ep.ep_expert_matmul_backward(grad, x, w, off, grad_rows=buf(K), weights_dtype=wide)
        hr, hw = ep.ep_expert_glu_backward(grad[:, :N // 2], grad, x, w, off, grad_rows=buf(K), weights_dtype=wide)
        outs += [gr, hr]
        assert bool((gw == 0).all()) and bool((hw == 0).all())
    codes = torch.full((R, 64), 0x7F, dtype=torch.uint8, device=DEV)
    for gated in (False, True):
        outs.append(ep.ep_expert_matmul_fp8(codes, torch.ones(R, 1, device=DEV), codes[:1].expand(E, N, 64).contiguous(),
                                            torch.ones(E, 1, 1, device=DEV), off, gated=gated,
                                            out=buf(N // 2 if gated else N)))
    for o in outs:
        assert bool((o == 7.0).all())


@pytest.mark.parametrize("wide", [torch.bfloat16, torch.float32])
def test_no_rows_of_odd_widths(wide):
    E, N, K = 3, 34, 67
    x, w = torch.empty(0, K, dtype=torch.bfloat16, device=DEV), values(generator(2), E, N, K)
    off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    for gr, gw in (ep.ep_expert_matmul_backward(x.new_empty(0, N), x, w, off, weights_dtype=wide),
                   ep.ep_expert_glu_backward(x.new_empty(0, N // 2), x.new_empty(0, N), x, w, off, weights_dtype=wide)):
        assert gr.shape == (0, K) and gw.dtype == wide and bool((gw == 0).all())


@pytest.mark.parametrize("each", [2, 100, 400])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_widest_inputs(each, dtype):
    """65536 inputs (and, for the gradients, that many columns)."""
    K, N = 65536, 34
    g = generator(3)
    x, w = values(g, each, K, dtype=TYPES[dtype]), (values(g, 1, N, K) / 256).to(TYPES[dtype])
    y, err = product(f64(x), f64(w[0]))
    check(ep.ep_expert_matmul(x, w), y, rounded(y, err, dtype), "product")
    out, pre = ep.ep_expert_glu(x, w, want_pre=True)
    check(pre, y, rounded(y, err, dtype), "pre")
    f, ferr = glu(y, err)
    check(out, f, rounded(f, ferr, dtype), "gated")
    dh = values(g, each, N // 2, dtype=TYPES[dtype])
    gr, gw = ep.ep_expert_glu_backward(dh, pre, x, w)
    d, ed = glu_gradient(f64(dh), f64(pre), dtype)
    ref, err = product(d, f64(w[0]).T)
    check(gr, ref, rounded(ref, err + ed @ np.abs(f64(w[0])), dtype), "rows")
    ref, err = product(d.T, f64(x).T)
    check(gw[0], ref, rounded(ref, err + ed.T @ np.abs(f64(x)), dtype), "weights")


@pytest.mark.parametrize("each", [2, 100])
def test_widest_inputs_in_8_bits(each):
    K, N = 65536, 34
    g = generator(4)
    codes = [torch.randint(0, 256, (n, K), generator=g, device=DEV, dtype=torch.uint8) for n in (each, N)]
    for c in codes:
        c[~torch.isfinite(c.view(torch.float8_e4m3fn).float())] = 0
    xs, ws = (torch.rand(n, 512, generator=g, device=DEV) / 448 for n in (each, 1))
    v = [f64(c.view(torch.float8_e4m3fn).float()) * f64(s).repeat(128, 1) for c, s in zip(codes, (xs, ws))]
    got = ep.ep_expert_matmul_fp8(codes[0], xs, codes[1][None].contiguous(), ws[None].contiguous())
    ref, err = product(*v)
    if each > 64:
        top = [np.abs(a).reshape(len(a), -1, 8).max(2) for a in v]
        err = err + 7 * 2.0 ** -13 * (top[0] @ top[1].T)
    check(got, ref, rounded(ref, err, "bf16"), "product")


@pytest.mark.parametrize("each,N", [(3, 64), (20, 512), (70, 512)])
def test_many_experts(each, N):
    """700 experts, every seventh without rows: their offsets are looked at 256
    at a time, by the kernels for few rows and by the tiles."""
    E, K = 700, 80
    rng = np.random.default_rng(5)
    n = ragged(rng, E, each, empty=range(0, E, 7))
    _, off = segments(n, DEV)
    at = off.cpu().numpy()
    R = int(at[E])
    g = generator(6)
    x, w, d = values(g, R, K), values(g, E, N, K), values(g, R, N)
    got = ep.ep_expert_matmul(x, w, off)
    gr, gw = ep.ep_expert_matmul_backward(d, x, w, off)
    cx, cw = (torch.randint(0, 0x70, s, generator=g, device=DEV, dtype=torch.uint8) for s in ((R, K), (E, N, K)))
    q = ep.ep_expert_matmul_fp8(cx, torch.ones(R, 1, device=DEV), cw, torch.ones(E, -(-N // 128), 1, device=DEV), off)
    for e in list(range(0, E, 41)) + [254, 255, 256, 257, 511, 512, 513, E - 1]:
        s = slice(at[e], at[e + 1])
        ref, err = product(f64(x[s]), f64(w[e]))
        check(got[s], ref, rounded(ref, err, "bf16"), f"expert {e}")
        ref, err = product(f64(d[s]), f64(w[e]).T)
        check(gr[s], ref, rounded(ref, err, "bf16"), f"rows of expert {e}")
        ref, err = product(f64(d[s]).T, f64(x[s]).T) if n[e] else (np.zeros((N, K)),) * 2
        check(gw[e], ref, rounded(ref, err, "bf16"), f"weights of expert {e}")
        v = [f64(c.view(torch.float8_e4m3fn).float()) for c in (cx[s], cw[e])]
        ref, err = product(*v)
        top = [np.abs(a).reshape(len(a), K // 8, 8).max(2) for a in v]
        check(q[s], ref, rounded(ref, err + 7 * 2.0 ** -13 * (top[0] @ top[1].T), "bf16"), f"8 bits, expert {e}")


@pytest.mark.parametrize("each", [1, 20, 70, 200])
@pytest.mark.parametrize("half", [1, 15, 17, 129])
def test_8_bit_halves_of_few_outputs(each, half):
    E, K = 2, 144
    g = generator(7)
    cx, cw = (torch.randint(0, 0x60, s, generator=g, device=DEV, dtype=torch.uint8)
              for s in ((E * each, K), (E, 2 * half, K)))
    cw[:, :half] |= 0x80                                            # gates below 0 too
    ws = torch.rand(E, -(-2 * half // 128), 2, generator=g, device=DEV) / 1000
    xs = torch.rand(E * each, 2, generator=g, device=DEV)
    _, off = segments(np.array([each] * E), DEV)
    got = ep.ep_expert_matmul_fp8(cx, xs, cw, ws, off, gated=True, dtype=torch.float16)
    for e in range(E):
        s = slice(e * each, (e + 1) * each)
        x = f64(cx[s].view(torch.float8_e4m3fn).float()) * f64(xs[s]).repeat(128, 1)[:, :K]
        w = f64(cw[e].view(torch.float8_e4m3fn).float()) * f64(ws[e]).repeat(128, 0)[:2 * half].repeat(128, 1)[:, :K]
        y, err = product(x, w)
        if each > 64:
            top = [np.abs(a).reshape(len(a), -1, 8).max(2) for a in (x, w)]
            err = err + 7 * 2.0 ** -13 * (top[0] @ top[1].T)
        ref, err = glu(y, err)
        check(got[s], ref, rounded(ref, err, "fp16"), f"expert {e}")
