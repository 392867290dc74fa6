"""The experts' products in a layer (examples/moe_layer.py) against 64-bit
forms, on side streams, overlapping, captured into graphs, and past 32 bits."""

import numpy as np
import pytest
import torch

from combine_ep_layout_04_amd import ep
from combine_ep_layout_04_amd.examples import moe_layer
from oracle import moe

from expert_util import product, segments
from moe_util import DEV, check, f64, rounded

pytestmark = pytest.mark.gpu


def full_weights(E, I, H, dtype=torch.bfloat16, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return tuple((torch.randn(E, N, K, generator=g, device=DEV) / K ** 0.5).to(dtype)
                 for N, K in ((2 * I, H), (H, I)))


def layer(x, gate, d13, d2, k, score):
    """The layer in 64 bits, its experts chosen by the bf16 logits."""
    idx, w, _ = moe.router(f64(x @ gate.t()), k, score, None, 1, 1, 1)
    I = d2.shape[2]
    ref = np.zeros(x.shape)
    for t in range(len(ref)):
        for j in range(k):
            a = d13[idx[t, j]] @ f64(x)[t]
            ref[t] += w[t, j] * (d2[idx[t, j]] @ (moe.silu(a[:I]) * a[I:]))
    return ref


@pytest.mark.parametrize("T", [1, 7, 300])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_decode_full_width(T, dtype):
    E, k, H, I = 6, 2, 264, 96
    w13, w2 = full_weights(E, I, H, dtype)
    x = torch.randn(T, H, device=DEV).to(dtype)
    gate = (torch.randn(E, H, device=DEV) / H ** 0.5).to(dtype)
    got = f64(moe_layer.decode(x, gate, w13, w2, k))
    ref = layer(x, gate, f64(w13), f64(w2), k, "sigmoid")
    # three roundings (hidden, rows, result), each half a step of its value
    # at most, so well below three of the norm
    assert np.linalg.norm(got - ref) < 3 * torch.finfo(dtype).eps / 2 * np.linalg.norm(ref) * 1.5


@pytest.mark.parametrize("T", [1, 7, 300])
def test_decode_8_bit(T):
    E, k, H, I = 6, 2, 256, 128
    w13, w2 = moe_layer.random_fp8(E, 2 * I, H), moe_layer.random_fp8(E, H, I)
    d13, d2 = (f64(w.codes.view(torch.float8_e4m3fn).float()) * f64(w.scales).repeat(128, 1).repeat(128, 2)
               for w in (w13, w2))
    x = torch.randn(T, H, device=DEV).bfloat16()
    gate = (torch.randn(E, H, device=DEV) / H ** 0.5).bfloat16()
    got = f64(moe_layer.decode(x, gate, w13, w2, k))
    ref = layer(x, gate, d13, d2, k, "sigmoid")
    # two casts to E4M3 of what goes into a product (half a step is 2^-4 at
    # most; a sum's error is at random below that of its norm), and the
    # activation's slope of 1.1 with both factors off
    assert np.linalg.norm(got - ref) < (2.2 + 1) * 2.0 ** -4 * np.linalg.norm(ref)


@pytest.mark.parametrize("T", [24, 700])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_train_step(T, dtype):
    """All gradients of the layer in 16 bits, against double precision and the
    same choice of experts."""
    E, k, H, I = 4, 2, 136, 48
    g = torch.Generator(device=DEV).manual_seed(1)
    x, gate = (torch.randn(s, generator=g, device=DEV) / d for s, d in (((T, H), 1), ((E, H), H ** 0.5)))
    w13, w2 = full_weights(E, I, H, dtype)
    x, gate, go = x.to(dtype), gate.to(dtype), torch.randn(T, H, generator=g, device=DEV).to(dtype)
    got = moe_layer.train_step(x, gate, w13, w2, k, go)
    idx = ep.ep_router(x @ gate.t(), k)[0].cpu()
    leaves = [t.cpu().double().requires_grad_() for t in (x, gate, w13, w2)]
    xd, gd, ad, bd = leaves
    p = torch.softmax(xd @ gd.t(), 1)
    w = p.gather(1, idx)
    w = w / w.sum(1, keepdim=True)
    out = 0
    for j in range(k):
        for e in range(E):
            at = idx[:, j] == e
            a = xd @ ad[e].t()
            y = (torch.nn.functional.silu(a[:, :I]) * a[:, I:]) @ bd[e].t()
            out = out + torch.where(at, w[:, j], 0.0)[:, None] * y
    ref = (out,) + torch.autograd.grad((out * go.cpu().double()).sum(), leaves)
    for name, a, b in zip(("out", "grad_x", "grad_gate", "grad_w13", "grad_w2"), got, ref):
        # at most ten roundings of half a step from input to gradient (logits,
        # rows, pre, hidden, y, their gradients), each relative to what it rounds
        err, size = np.linalg.norm(f64(a) - b.detach().numpy()), float(b.norm())
        assert err < 10 * torch.finfo(dtype).eps / 2 * size, (name, err / size)


def everything(s, stream=None):
    """Every call of the set on one set of inputs."""
    kw = dict(stream=stream)
    x, w13, w2, off, src = s["x"], s["w13"], s["w2"], s["offsets"], s["src"]
    h, pre = ep.ep_expert_glu(x, w13, off, src=src, want_pre=True, **kw)
    y = ep.ep_expert_matmul(h, w2, off, **kw)
    gh, gw2 = ep.ep_expert_matmul_backward(y, h, w2, off, **kw)
    gr, gw13 = ep.ep_expert_glu_backward(gh, pre, x, w13, off, src=src, weights_dtype=torch.float32, **kw)
    q = ep.ep_expert_matmul_fp8(s["q"], s["qs"], s["wq"], s["wqs"], off, gated=True, src=src, **kw)
    return h, pre, y, gh, gw2, gr, gw13, q


def state(each=40, E=5, H=256, I=96, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    w13, w2 = full_weights(E, I, H, seed=seed)
    n = np.full(E, each)
    n[1] = 0
    _, off = segments(n, DEV)
    R = int(n.sum())
    wq = moe_layer.random_fp8(E, 2 * I, H)
    s = dict(offsets=off, w13=w13, w2=w2, wq=wq.codes, wqs=wq.scales, x=torch.empty(R, H, device=DEV).bfloat16(),
             src=torch.randint(0, R, (R,), generator=g, device=DEV, dtype=torch.int32),
             q=torch.empty(R, H, dtype=torch.uint8, device=DEV), qs=torch.empty(R, H // 128, device=DEV))
    refill(s, seed)
    return s


def refill(s, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    s["x"].copy_(torch.randn(s["x"].shape, generator=g, device=DEV))
    q, qs = moe_layer.cast_rows(s["x"])
    s["q"].copy_(q)
    s["qs"].copy_(qs)


def equal(a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


SIZES = [3, 40, 300]        # rows an expert: every kind of kernel


@pytest.mark.parametrize("each", SIZES)
def test_side_stream(each):
    s = state(each)
    ref = [t.clone() for t in everything(s)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        side.wait_stream(torch.cuda.current_stream())
        got = everything(s, stream)
        side.synchronize()
        assert equal(got, ref)
    with torch.cuda.stream(side):
        got = everything(s)
    side.synchronize()
    assert equal(got, ref)


@pytest.mark.parametrize("each", SIZES)
def test_two_streams_at_once(each):
    a, b = state(each, seed=1), state(each + 7, H=384, seed=2)
    ref = [[t.clone() for t in everything(s)] for s in (a, b)]
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    got = [None, None]
    for _ in range(3):
        for i, s in enumerate((a, b)):
            with torch.cuda.stream(streams[i]):
                got[i] = everything(s)
        torch.cuda.synchronize()
        assert equal(got[0], ref[0]) and equal(got[1], ref[1])


@pytest.mark.parametrize("each", SIZES)
def test_graph_replays(each):
    s = state(each)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        everything(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = everything(s)
    for seed in (2, 3, 4):
        refill(s, seed)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        ref = everything(s)
        torch.cuda.synchronize()
        assert equal(got, ref), seed


@pytest.mark.parametrize("each", [2, 40, 300])
def test_rows_far_past_32_bits(each):
    """Rows of x and of the results beyond 2^32 bytes, picked by src and in
    place."""
    K, N, ld = 64, 48, 1 << 20
    rows = (5 << 30) // (2 * ld)                  # 5 GiB of rows 2 MiB apart
    buf = torch.empty(rows, ld, dtype=torch.bfloat16, device=DEV)
    x = buf[:, :K]
    x.copy_(torch.randn(rows, K, device=DEV))
    w = torch.randn(1, N, K, device=DEV).bfloat16()
    src = torch.arange(rows - each, rows, dtype=torch.int32, device=DEV)
    near = x[-each:].contiguous()
    ref, err = product(f64(near), f64(w[0]))
    got = ep.ep_expert_matmul(x, w, src=src)
    check(got, ref, rounded(ref, err, "bf16"), "src")
    out = torch.empty(rows, ld, dtype=torch.bfloat16, device=DEV)
    whole = ep.ep_expert_matmul(x, w, out=out[:, :N])
    check(whole[-each:], ref, rounded(ref, err, "bf16"), "rows in place")
    del out
    g = torch.randn(each, N, device=DEV).bfloat16()
    gr, gw = ep.ep_expert_matmul_backward(g, x, w, src=src)
    ref, err = product(f64(g).T, f64(near).T)
    check(gw[0], ref, rounded(ref, err, "bf16"), "weights")
    # 8 bits
    codes = buf.view(torch.uint8)[:, :K]
    q, qs = moe_layer.cast_rows(torch.cat([near, near], 1))
    codes[-each:] = q[:, :K]
    scales = torch.ones(rows, 1, device=DEV)
    scales[-each:] = qs
    wq = moe_layer.random_fp8(1, N, K)
    got = ep.ep_expert_matmul_fp8(codes, scales, wq.codes, wq.scales, src=src)
    also = ep.ep_expert_matmul_fp8(q[:, :K].contiguous(), qs, wq.codes, wq.scales)
    if each < 33:       # the same kernel; the others sum in the same order too
        assert torch.equal(got, also)
    v = f64(q[:, :K].contiguous().view(torch.float8_e4m3fn).float()) * f64(qs)
    ref, err = product(v, f64(wq.codes[0].view(torch.float8_e4m3fn).float()) * f64(wq.scales)[0, 0, 0])
    err = err + 7 * 2.0 ** -13 * np.abs(v).max(1)[:, None] * 256 * f64(wq.scales)[0, 0, 0] * K / 8
    check(got, ref, rounded(ref, err, "bf16"), "8 bits")


def test_halves_of_weights_far_apart():
    """Gate and up more than 2^32 bytes apart."""
    K, half, each = 32768, 66000, 40
    w = torch.empty(1, 2 * half, K, dtype=torch.bfloat16, device=DEV)
    w[:, :, 64:] = 0
    w[:, :, :64] = torch.randn(2 * half, 64, device=DEV) / 8
    x = torch.randn(each, K, device=DEV).bfloat16()
    out, _ = ep.ep_expert_glu(x, w)
    for n in (0, 31999, half - 64):
        near = torch.cat([w[0, n:n + 64, :64], w[0, half + n:half + n + 64, :64]])[None].contiguous()
        small, _ = ep.ep_expert_glu(x[:, :64].contiguous(), near)
        # the same terms and zeros, in sums of another length: a rounding each
        assert torch.allclose(out[:, n:n + 64].float(), small.float(), rtol=2.0 ** -7, atol=2.0 ** -10)
