"""Arguments the experts' products refuse, on the host before any launch (fake
pointers, so only where no GPU is visible), and tensors the binding refuses."""

import pytest
import torch

from combine_ep_layout_04_amd import ep

FAKE = 0x100000
no_gpu = pytest.mark.skipif(torch.cuda.device_count() > 0,
                            reason="fake pointers must never reach a launch on a real GPU")


def call(name, base, over):
    a = dict(base)
    assert set(over) <= set(a)
    a.update(over)
    return getattr(ep.lib(), name)(*a.values(), None)


MATMUL = dict(x=FAKE, dtype=0, ldx=64, M=8, src=None, w=FAKE, E=2, N=32, K=64, offsets=FAKE, counts=None, R=8,
              out=FAKE, ldo=32)
SHAPES = [
    (dict(dtype=2), 1), (dict(dtype=-1), 1), (dict(E=0), 1), (dict(E=1025), 1), (dict(N=0), 1),
    (dict(N=(1 << 20) + 2, ), 1), (dict(K=0), 1), (dict(K=65537), 1), (dict(R=-1), 1), (dict(R=1 << 31), 1),
    (dict(offsets=None), 1), (dict(E=1, offsets=None, counts=FAKE), 1), (dict(offsets=FAKE + 2), 1),
    (dict(counts=FAKE + 1), 1),
]


@no_gpu
@pytest.mark.parametrize("over,code", SHAPES + [
    (dict(x=None), 1), (dict(x=FAKE + 1), 1), (dict(ldx=63), 1), (dict(M=0), 1), (dict(M=7), 1),
    (dict(src=FAKE + 2), 1), (dict(w=None), 1), (dict(w=FAKE + 1), 1), (dict(out=None), 1),
    (dict(out=FAKE + 1), 1), (dict(ldo=31), 1),
    (dict(R=(1 << 31) - 1, M=1 << 31, N=1 << 20, ldo=1 << 20), 2),
])
def test_matmul_rejects(over, code):
    assert call("ep_expert_matmul", MATMUL, over) == code, ep.last_error()
    assert ep.last_error()


GLU = dict(MATMUL, ldo=16, pre=None, ldp=0)


@no_gpu
@pytest.mark.parametrize("over,code", SHAPES + [
    (dict(N=33), 1), (dict(x=None), 1), (dict(w=None), 1), (dict(out=None), 1), (dict(ldo=15), 1),
    (dict(pre=FAKE + 1, ldp=32), 1), (dict(pre=FAKE, ldp=31), 1), (dict(M=7), 1),
])
def test_glu_rejects(over, code):
    assert call("ep_expert_glu", GLU, over) == code, ep.last_error()
    assert ep.last_error()


BACKWARD = dict(g=FAKE, dtype=0, ldg=32, x=FAKE, ldx=64, M=8, src=None, w=FAKE, E=2, N=32, K=64, offsets=FAKE,
                counts=None, R=8, gr=FAKE, ldgr=64, gw=FAKE, gwt=0, work=None, bytes=0)
GRADS = SHAPES + [
    (dict(g=None), 1), (dict(g=FAKE + 1), 1), (dict(gr=None, gw=None), 1), (dict(gwt=1), 1),
    (dict(dtype=1, gwt=0), 1), (dict(gw=FAKE + 1), 1), (dict(gwt=2, gw=FAKE + 2), 1), (dict(x=None), 1),
    (dict(ldx=63), 1), (dict(M=7), 1), (dict(src=FAKE + 2), 1), (dict(w=None), 1), (dict(gr=FAKE + 1), 1),
    (dict(ldgr=63), 1), (dict(R=0, gw=FAKE + 1), 1),
]


@no_gpu
@pytest.mark.parametrize("over,code", GRADS + [
    (dict(ldg=31), 1), (dict(src=FAKE), 1), (dict(src=FAKE, work=FAKE, bytes=1023), 1),
    (dict(src=FAKE, work=FAKE + 8, bytes=1024), 1), (dict(N=30), 1), (dict(K=63), 1),
    (dict(R=(1 << 31) - 1, M=1 << 31, N=1 << 20, ldg=1 << 20), 2),
])
def test_matmul_backward_rejects(over, code):
    assert call("ep_expert_matmul_backward", BACKWARD, over) == code, ep.last_error()
    assert ep.last_error()


GLU_B = dict(g=FAKE, dtype=0, ldg=16, pre=FAKE, ldp=32, x=FAKE, ldx=64, M=8, src=None, w=FAKE, E=2, N=32, K=64,
             offsets=FAKE, counts=None, R=8, gr=FAKE, ldgr=64, gw=FAKE, gwt=0, work=FAKE, bytes=512)


@no_gpu
@pytest.mark.parametrize("over,code", GRADS + [
    (dict(N=33), 1), (dict(ldg=15), 1), (dict(pre=None), 1), (dict(pre=FAKE + 1), 1), (dict(ldp=31), 1),
    (dict(work=None), 1), (dict(work=FAKE + 8), 1), (dict(bytes=511), 1),
    (dict(R=(1 << 31) - 1, M=1 << 31, N=1 << 20, ldg=1 << 19, ldp=1 << 20, bytes=1 << 62), 2),
])
def test_glu_backward_rejects(over, code):
    assert call("ep_expert_glu_backward", GLU_B, over) == code, ep.last_error()
    assert ep.last_error()


def test_workspace_size():
    size = ep.ep_expert_backward_workspace_size
    assert size(8, 32, 64) == size(0, 32, 64) == 0
    assert size(8, 32, 64, gated=True) == 512 and size(8, 32, 64, gathered=True) == 1024
    assert size(3, 34, 64) == 3 * 40 * 2 and size(3, 32, 65) == 3 * 72 * 2
    assert size(3, 34, 65, gated=True, gathered=True) == 3 * (40 + 72) * 2
    assert size(-1, 33, 64) == size(8, 33, 64, gated=True) == size(8, 0, 63) == size(8, 33, 0) == 0
    assert size(1 << 31, 33, 64) == size(8, (1 << 20) + 1, 63) == size(8, 33, 65537) == 0
    assert size((1 << 31) - 1, 1 << 20, 65535, gated=True) == ((1 << 31) - 1) * ((1 << 21) + (1 << 17))


FP8 = dict(x=FAKE, fmt=1, ldx=128, M=8, xs=FAKE, sf=0, sr=1, sb=8, src=None, w=FAKE, ws=FAKE, E=2, N=32, K=128,
           gated=0, offsets=FAKE, counts=None, R=8, out=FAKE, dtype=0, ldo=32)


@no_gpu
@pytest.mark.parametrize("over,code", SHAPES + [
    (dict(fmt=0), 1), (dict(fmt=3), 1), (dict(sf=3), 1), (dict(sf=-1), 1), (dict(N=33, gated=1), 1),
    (dict(K=120), 1), (dict(x=None), 1), (dict(x=FAKE + 8), 1), (dict(ldx=112), 1), (dict(ldx=136), 1),
    (dict(M=0), 1), (dict(M=7), 1), (dict(xs=None), 1), (dict(xs=FAKE + 2), 1), (dict(sr=-1), 1),
    (dict(sb=-1), 1), (dict(src=FAKE + 2), 1), (dict(w=None), 1), (dict(w=FAKE + 8), 1), (dict(ws=None), 1),
    (dict(ws=FAKE + 2), 1), (dict(out=None), 1), (dict(out=FAKE + 1), 1), (dict(ldo=31), 1),
    (dict(gated=1, ldo=15), 1), (dict(R=(1 << 31) - 1, M=1 << 31, N=1 << 20, ldo=1 << 20), 2),
])
def test_fp8_rejects(over, code):
    assert call("ep_expert_matmul_fp8", FP8, over) == code, ep.last_error()
    assert ep.last_error()


@no_gpu
def test_no_rows_reads_nothing():
    null = dict(R=0, x=None, w=None, out=None, M=0)
    assert call("ep_expert_matmul", MATMUL, null) == 0
    assert call("ep_expert_glu", GLU, null) == 0
    assert call("ep_expert_matmul_fp8", FP8, dict(null, xs=None, ws=None)) == 0
    assert call("ep_expert_matmul_backward", BACKWARD, dict(R=0, g=None, x=None, w=None, gw=None, src=FAKE)) == 0
    assert call("ep_expert_glu_backward", GLU_B, dict(R=0, g=None, x=None, w=None, gw=None, work=None)) == 0


def test_binding_refuses_host_tensors_and_types():
    x, w = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(1, 6, 8, dtype=torch.bfloat16)
    for f in (ep.ep_expert_matmul, ep.ep_expert_glu):
        with pytest.raises(ValueError, match="device tensor"):
            f(x, w)
        with pytest.raises(TypeError, match="bfloat16 or float16"):
            f(x.float(), w)
    with pytest.raises(ValueError, match="device tensor"):
        ep.ep_expert_matmul_backward(torch.zeros(4, 6).bfloat16(), x, w)
    with pytest.raises(TypeError, match="uint8"):
        ep.ep_expert_matmul_fp8(x, x, w, w)
    with pytest.raises(ValueError, match="unknown fmt"):
        ep.ep_expert_matmul_fp8(x, x, w, w, fmt="e3m4")


@pytest.mark.gpu
def test_binding_refuses_shapes():
    d = "cuda:0"
    x, w = torch.zeros(4, 8, device=d).bfloat16(), torch.zeros(2, 6, 8, device=d).bfloat16()
    off = torch.zeros(3, dtype=torch.int32, device=d)
    src = torch.zeros(4, dtype=torch.int32, device=d)
    g, h, p = x.new_zeros(4, 6), x.new_zeros(4, 3), x.new_zeros(4, 6)
    bad = [
        (TypeError, lambda: ep.ep_expert_matmul(x, w.half(), off)),
        (ValueError, lambda: ep.ep_expert_matmul(x, w[0], off)),
        (ValueError, lambda: ep.ep_expert_matmul(x[:, :7], w, off)),
        (ValueError, lambda: ep.ep_expert_matmul(x, w.transpose(1, 2), off)),
        (ValueError, lambda: ep.ep_expert_matmul(x, w, off[:2])),
        (TypeError, lambda: ep.ep_expert_matmul(x, w, off.long())),
        (ValueError, lambda: ep.ep_expert_matmul(x, w, off, src=src, rows=5)),
        (ep.EpError, lambda: ep.ep_expert_matmul(x, w, off, rows=5)),
        (ValueError, lambda: ep.ep_expert_matmul(x, w, off, out=x.new_zeros(3, 6))),
        (ValueError, lambda: ep.ep_expert_matmul(x, w, off, out=x.new_zeros(4, 5))),
        (ep.EpError, lambda: ep.ep_expert_matmul(x, w)),
        (ValueError, lambda: ep.ep_expert_glu(x, w[:, :5].contiguous(), off)),
        (ValueError, lambda: ep.ep_expert_glu(x, w, off, pre=x.new_zeros(4, 5))),
        (ValueError, lambda: ep.ep_expert_matmul_backward(g[:, :5], x, w, off)),
        (ValueError, lambda: ep.ep_expert_matmul_backward(g, x[:3], w, off)),
        (ValueError, lambda: ep.ep_expert_matmul_backward(g, x, w, off, src=src[:3])),
        (ValueError, lambda: ep.ep_expert_matmul_backward(g, x, w, off, want_rows=False, want_weights=False)),
        (TypeError, lambda: ep.ep_expert_matmul_backward(g, x, w, off, weights_dtype=torch.float16)),
        (ValueError, lambda: ep.ep_expert_matmul_backward(g, x, w, off, grad_weights=w.new_zeros(2, 6, 7))),
        (ValueError, lambda: ep.ep_expert_matmul_backward(g, x, w, off, grad_rows=x.new_zeros(3, 8))),
        (ValueError, lambda: ep.ep_expert_glu_backward(h, p[:3], x, w, off)),
        (ValueError, lambda: ep.ep_expert_glu_backward(g, p, x, w, off)),
        (ValueError, lambda: ep.ep_expert_glu_backward(h, p, x, w, off, workspace=torch.zeros(
            63, dtype=torch.uint8, device=d))),
    ]
    q, s = torch.zeros(4, 16, dtype=torch.uint8, device=d), torch.ones(4, 1, device=d)
    wq, ws = torch.zeros(2, 6, 16, dtype=torch.uint8, device=d), torch.ones(2, 1, 1, device=d)
    bad += [
        (ValueError, lambda: ep.ep_expert_matmul_fp8(q[:, :8], s, wq, ws, off)),
        (TypeError, lambda: ep.ep_expert_matmul_fp8(q, s.half(), wq, ws, off)),
        (ValueError, lambda: ep.ep_expert_matmul_fp8(q, s[:3], wq, ws, off)),
        (ValueError, lambda: ep.ep_expert_matmul_fp8(q, s, wq, ws[:1], off)),
        (TypeError, lambda: ep.ep_expert_matmul_fp8(q, s, wq, ws, off, dtype=torch.float32)),
        (ValueError, lambda: ep.ep_expert_matmul_fp8(q, s, wq[:, :5].contiguous(), ws, off, gated=True)),
        (ValueError, lambda: ep.ep_expert_matmul_fp8(q.t(), s, wq, ws, off)),
        (ValueError, lambda: ep.ep_expert_matmul_fp8(q, s.cpu(), wq, ws, off)),
    ]
    for kind, f in bad:
        with pytest.raises(kind):
            f()
