"""ep_expert_matmul, ep_expert_glu and their backwards against the 64-bit
forms."""

import numpy as np
import pytest
import torch

from combine_ep_layout_04_amd import ep

from expert_util import glu, glu_gradient, product, ragged, segments
from moe_util import DEV, TYPES, U, check, f64, rounded, wide

pytestmark = pytest.mark.gpu

CASES = [
    # rows an expert (about), E, K, N, dtype, gather, pad, shift, align
    # single rows, and rows of a plain matrix-vector product
    (1, 1, 1, 2, "bf16", False, 0, 0, 1),
    (1, 1, 8, 16, "fp16", False, 0, 0, 1),
    (1, 1, 2048, 1000, "bf16", False, 0, 0, 1),
    (1, 8, 300, 34, "fp16", True, 0, 0, 1),
    # few rows: up to 16 and up to 32 an expert
    (5, 3, 136, 66, "bf16", True, 8, 0, 1),
    (12, 7, 1999, 100, "fp16", True, 3, 1, 1),
    (14, 300, 64, 32, "bf16", False, 0, 0, 1),
    (24, 5, 1000, 258, "bf16", False, 0, 3, 1),
    (30, 2, 129, 18, "fp16", True, 1, 0, 1),
    # tiles of 128 x 128
    (50, 4, 512, 256, "bf16", False, 0, 0, 1),
    (100, 3, 200, 130, "fp16", True, 8, 0, 1),
    (130, 2, 72, 514, "bf16", True, 0, 0, 1),
    # the same off 16 bytes: odd widths, odd strides, odd starts
    (60, 3, 333, 70, "bf16", True, 0, 0, 1),
    (90, 2, 64, 128, "fp16", False, 3, 0, 1),
    (150, 1, 128, 62, "bf16", False, 8, 1, 1),
    # tiles of 256 x 256
    (300, 2, 320, 512, "bf16", True, 0, 0, 1),
    (257, 3, 72, 258, "fp16", False, 8, 0, 1),
    (700, 1, 1000, 770, "bf16", False, 0, 0, 1),
    # few rows of many experts: 64 outputs a workgroup, and tiles from 9 rows on
    (6, 40, 200, 1026, "bf16", True, 0, 0, 1),
    (7, 40, 135, 1030, "fp16", False, 1, 0, 1),
    (14, 16, 264, 2560, "bf16", True, 0, 0, 1),
    (20, 40, 131, 1000, "fp16", False, 3, 1, 1),
    # up to 64 rows of one expert
    (64, 1, 520, 300, "bf16", False, 0, 0, 1),
    (47, 1, 264, 258, "fp16", True, 1, 0, 1),
    # segments with gaps
    (20, 4, 96, 48, "bf16", False, 0, 0, 32),
    (100, 4, 96, 48, "bf16", True, 0, 0, 64),
    (260, 3, 104, 100, "fp16", False, 0, 0, 128),
]


class Case:
    def __init__(self, case, seed=5):
        each, E, K, N, self.dtype, gather, pad, shift, align = case
        rng = np.random.default_rng(seed)
        n = ragged(rng, E, each, empty=[E // 2] if E > 2 else [])
        if E > 4:
            n[1] = 1
        self.E, self.K, self.N, self.n = E, K, N, n
        self.counts, self.offsets = segments(n, DEV, align)
        self.off = self.offsets.cpu().numpy()
        # a few rows behind the last segment
        self.R = R = int(self.off[E]) + (3 if each > 1 else 0)
        dt = TYPES[self.dtype]

        def values(*shape):
            return torch.from_numpy(rng.normal(size=shape)).to(dt).double().numpy()
        T = max(1, R // 2)
        self.x = values(T if gather else R, K)
        self.src = rng.integers(0, T, R).astype(np.int32) if gather else None
        self.w = values(E, N, K) / np.sqrt(K)
        self.w = torch.from_numpy(self.w).to(dt).double().numpy()
        # rows of no expert hold NaN
        self.used = np.zeros(R, bool)
        for e in range(E):
            self.used[self.off[e]:self.off[e] + n[e]] = True
        self.tx = wide(self.x, self.dtype, pad, shift)
        if not gather:
            self.tx[torch.from_numpy(~self.used).to(DEV)] = float("nan")
        self.tw = torch.from_numpy(self.w).to(dt).to(DEV)
        self.tsrc = None if self.src is None else torch.from_numpy(self.src).to(DEV)
        self.pad, self.shift = pad, shift
        self.grad = values(R, N)
        self.pre = values(R, N)
        self.kw = dict(src=self.tsrc, counts=self.counts if align > 1 else None)

    def rows(self, e):
        a, b = self.off[e], self.off[e] + self.n[e]
        return slice(a, b), (self.x[a:b] if self.src is None else self.x[self.src[a:b]])

    def holder(self, cols):
        """A buffer of 7.0 and the columns of it that a call may write."""
        buf = torch.full((self.R + 2, cols + self.pad), 7.0, dtype=TYPES[self.dtype], device=DEV)
        return buf, buf[:, :cols]

    def untouched(self, buf, cols):
        used = torch.from_numpy(self.used).to(DEV)
        assert bool((buf[:self.R][~used] == 7.0).all()) and bool((buf[self.R:] == 7.0).all())
        assert bool((buf[:, cols:] == 7.0).all())

    def gradient(self, a):
        t = wide(a, self.dtype, self.pad, self.shift)
        t[torch.from_numpy(~self.used).to(DEV)] = float("nan")
        return t


def bits_equal(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_matmul(case):
    c = Case(case)
    buf, out = c.holder(c.N)
    got = ep.ep_expert_matmul(c.tx, c.tw, c.offsets, rows=c.R, out=out, **c.kw)
    c.untouched(buf, c.N)
    for e in range(c.E):
        at, x = c.rows(e)
        if len(x):
            ref, err = product(x, c.w[e])
            check(got[at], ref, rounded(ref, err, c.dtype), f"expert {e}")
    again = ep.ep_expert_matmul(c.tx, c.tw, c.offsets, rows=c.R, **c.kw)
    used = torch.from_numpy(c.used).to(DEV)
    assert bits_equal(again[used], got[:c.R][used])


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_glu(case):
    c = Case(case)
    buf, out = c.holder(c.N // 2)
    pbuf, pre = c.holder(c.N)
    got, kept = ep.ep_expert_glu(c.tx, c.tw, c.offsets, rows=c.R, out=out, pre=pre, **c.kw)
    c.untouched(buf, c.N // 2)
    c.untouched(pbuf, c.N)
    for e in range(c.E):
        at, x = c.rows(e)
        if len(x):
            y, err = product(x, c.w[e])
            check(kept[at], y, rounded(y, err, c.dtype), f"pre of expert {e}")
            ref, err = glu(y, err)
            check(got[at], ref, rounded(ref, err, c.dtype), f"expert {e}")
    again, none = ep.ep_expert_glu(c.tx, c.tw, c.offsets, rows=c.R, **c.kw)
    used = torch.from_numpy(c.used).to(DEV)
    assert none is None and bits_equal(again[used], got[:c.R][used])


def check_backward(c, d, ed, got_rows, got_weights, wide_dtype):
    for e in range(c.E):
        at, x = c.rows(e)
        if len(x):
            ref, err = product(d[at], c.w[e].T)
            check(got_rows[at], ref, rounded(ref, err + ed[at] @ np.abs(c.w[e]), c.dtype), f"rows of expert {e}")
        ref, err = product(d[at].T, x.T) if len(x) else (np.zeros((c.N, c.K)),) * 2
        err = err + ed[at].T @ np.abs(x)
        check(got_weights[e], ref, rounded(ref, err, wide_dtype), f"weights of expert {e}")


@pytest.mark.parametrize("wide_w", [False, True])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_matmul_backward(case, wide_w):
    c = Case(case)
    buf, out = c.holder(c.K)
    g = c.gradient(c.grad)
    kw = dict(c.kw, weights_dtype=torch.float32 if wide_w else None)
    gr, gw = ep.ep_expert_matmul_backward(g, c.tx, c.tw, c.offsets, grad_rows=out, **kw)
    c.untouched(buf, c.K)
    check_backward(c, c.grad, np.zeros_like(c.grad), gr, gw, "fp32" if wide_w else c.dtype)
    r2, none = ep.ep_expert_matmul_backward(g, c.tx, c.tw, c.offsets, want_weights=False, **kw)
    none2, w2 = ep.ep_expert_matmul_backward(g, c.tx, c.tw, c.offsets, want_rows=False, **kw)
    used = torch.from_numpy(c.used).to(DEV)
    assert none is None and none2 is None
    assert bits_equal(r2[used], gr[:c.R][used]) and bits_equal(w2, gw)


@pytest.mark.parametrize("wide_w", [False, True])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_glu_backward(case, wide_w):
    c = Case(case)
    buf, out = c.holder(c.K)
    dh = c.grad[:, :c.N // 2]
    g, p = c.gradient(dh), c.gradient(c.pre)
    kw = dict(c.kw, weights_dtype=torch.float32 if wide_w else None)
    gr, gw = ep.ep_expert_glu_backward(g, p, c.tx, c.tw, c.offsets, grad_rows=out, **kw)
    c.untouched(buf, c.K)
    d, ed = glu_gradient(dh, c.pre, c.dtype)
    check_backward(c, d, ed, gr, gw, "fp32" if wide_w else c.dtype)
    need = ep.ep_expert_backward_workspace_size(c.R, c.N, c.K, True, c.tsrc is not None)
    work = torch.empty(need, dtype=torch.uint8, device=DEV)
    none, w2 = ep.ep_expert_glu_backward(g, p, c.tx, c.tw, c.offsets, want_rows=False, workspace=work, **kw)
    assert none is None and bits_equal(w2, gw)


def test_gradients_against_differences():
    """The gated block's and the product's gradients are those of their
    forward: directional differences of the 64-bit forms."""
    c = Case((40, 2, 96, 64, "fp16", False, 0, 0, 1))
    rng = np.random.default_rng(1)
    at, x = c.rows(0)
    v, dw = rng.normal(size=x.shape), rng.normal(size=c.w[0].shape)
    dh, h = c.grad[at][:, :c.N // 2], 1e-5

    def value(x, w, gated):
        y = x @ w.T
        return float((glu(y, 0 * y)[0] * dh).sum() if gated else (y * c.grad[at]).sum())
    for gated in (True, False):
        if gated:
            _, pre = ep.ep_expert_glu(c.tx, c.tw, c.offsets, rows=c.R, want_pre=True)
            gr, gw = ep.ep_expert_glu_backward(c.gradient(c.grad[:, :c.N // 2]), pre, c.tx, c.tw, c.offsets,
                                               weights_dtype=torch.float32)
        else:
            gr, gw = ep.ep_expert_matmul_backward(c.gradient(c.grad), c.tx, c.tw, c.offsets,
                                                  weights_dtype=torch.float32)
        by_x = (value(x + h * v, c.w[0], gated) - value(x - h * v, c.w[0], gated)) / (2 * h)
        by_w = (value(x, c.w[0] + h * dw, gated) - value(x, c.w[0] - h * dw, gated)) / (2 * h)
        gx, gww = f64(gr[at]), f64(gw[0])
        # each gradient entry is off by less than 2^-10 of the sum of the sizes
        # of its terms (pre, d and the result are rounded to 2^-11 each; the
        # slopes of the activation's factors are below 2)
        terms = np.abs(c.grad[at]) * 3
        terms = terms[:, :c.N // 2].repeat(2, 1) * (1 + np.abs(f64(pre[at])).max()) if gated else terms
        lim_x = float((terms @ np.abs(c.w[0]) * np.abs(v)).sum()) * 2.0 ** -9
        lim_w = float((terms.T @ np.abs(x) * np.abs(dw)).sum()) * 2.0 ** -9
        assert abs((gx * v).sum() - by_x) < lim_x and abs((gww * dw).sum() - by_w) < lim_w
        assert lim_x < 0.5 * np.abs(gx * v).sum() and lim_w < 0.5 * np.abs(gww * dw).sum()


def test_no_rows():
    for dt in (torch.bfloat16, torch.float16):
        x, w = torch.empty(0, 64, dtype=dt, device=DEV), torch.randn(3, 32, 64, device=DEV).to(dt)
        off = torch.zeros(4, dtype=torch.int32, device=DEV)
        assert ep.ep_expert_matmul(x, w, off).shape == (0, 32)
        assert ep.ep_expert_glu(x, w, off, want_pre=True)[1].shape == (0, 32)
        gr, gw = ep.ep_expert_matmul_backward(x.new_empty(0, 32), x, w, off)
        assert gr.shape == (0, 64) and bool((gw == 0).all())
        gr, gw = ep.ep_expert_glu_backward(x.new_empty(0, 16), x.new_empty(0, 32), x, w, off)
        assert gr.shape == (0, 64) and bool((gw == 0).all())


@pytest.mark.parametrize("rows", [3, 60, 300])
def test_bad_sources_read_row_zero_and_bad_offsets_stay_inside(rows):
    """src outside x reads row 0; offsets past num_rows reach nothing."""
    E, K, N = 2, 64, 32
    x = torch.randn(7, K, device=DEV).bfloat16()
    w = torch.randn(E, N, K, device=DEV).bfloat16()
    src = torch.full((rows * E,), -1, dtype=torch.int32, device=DEV)
    src[::2] = 1 << 30
    off = torch.tensor([0, rows, 2 * rows], dtype=torch.int32, device=DEV)
    good = torch.zeros_like(src)
    assert bits_equal(ep.ep_expert_matmul(x, w, off, src=src), ep.ep_expert_matmul(x, w, off, src=good))
    g = torch.randn(rows * E, N, device=DEV).bfloat16()
    for a, b in zip(ep.ep_expert_matmul_backward(g, x, w, off, src=src),
                    ep.ep_expert_matmul_backward(g, x, w, off, src=good)):
        assert bits_equal(a, b)
    buf = torch.full((2 * rows + 8, N), 7.0, dtype=torch.bfloat16, device=DEV)
    far = torch.tensor([0, rows, 1 << 30], dtype=torch.int32, device=DEV)
    got = ep.ep_expert_matmul(x, w, far, src=good, out=buf, rows=2 * rows)
    assert bool((buf[2 * rows:] == 7.0).all())
    assert bits_equal(got[:2 * rows], ep.ep_expert_matmul(x, w, off, src=good))


@pytest.mark.parametrize("each", [4, 40, 300])
def test_special_values_stay_in_their_rows(each):
    """An infinity or a NaN in a row of x reaches that row of the result only."""
    E, K, N = 2, 72, 64
    x = torch.randn(each * E, K, device=DEV).bfloat16()
    w = torch.randn(E, N, K, device=DEV).bfloat16()
    _, off = segments(np.array([each] * E), DEV)
    ref = ep.ep_expert_matmul(x, w, off)
    y = x.clone()
    y[1, K - 1], y[each, 0] = float("inf"), float("nan")
    got = ep.ep_expert_matmul(y, w, off)
    keep = torch.ones(each * E, dtype=torch.bool, device=DEV)
    keep[1] = keep[each] = False
    assert bits_equal(got[keep], ref[keep])
    assert bool(torch.isinf(got[1]).all()) and bool(torch.isnan(got[each]).all())


def test_saturated_gates():
    """Gates far from 0: silu is the gate itself, or 0."""
    K = 32
    x = torch.zeros(4, K, device=DEV).bfloat16()
    x[:, 0] = 1.0
    w = torch.zeros(1, 32, K, device=DEV).bfloat16()
    for i, v in enumerate([3e38, -3e38, 500.0, -500.0, 88.0, -88.0, 0.0, -0.0]):
        w[0, i, 0] = v
    w[0, 16:, 0] = 0.5
    got = ep.ep_expert_glu(x, w)[0].float()
    want = torch.tensor([3e38, 0, 500, 0, 88, 0, 0, 0], device=DEV).bfloat16().float() * 0.5
    assert torch.allclose(got[0, :8], want, rtol=2.0 ** -8, atol=1e-35)
    pre = torch.cat([w[0, :16, 0], w[0, 16:, 0]]).expand(4, 32).contiguous()
    gr, gw = ep.ep_expert_glu_backward(torch.ones(4, 16, device=DEV).bfloat16(), pre, x, w)
    # four rows of silu(3e38) = 3e38 sum to 1.2e39, past the largest bf16
    # (3.4e38): that entry of the up half is infinite, and no other
    assert float(gw[0, 16, 0]) == float("inf")
    gw[0, 16, 0] = 0.0
    assert bool(torch.isfinite(gw).all())
    # the up half's gradient is silu(gate), the gate's up times 1 or 0
    assert float(gw[0, 16 + 2, 0]) == 2000.0 and float(gw[0, 2, 0]) == 2.0 and float(gw[0, 3, 0]) == 0.0
