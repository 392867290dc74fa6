"""Arguments the router, row movement and 4-bit product calls refuse, on the
host before any launch (fake pointers, so only where no GPU is visible)."""

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


ROUTER = dict(logits=FAKE, dtype=0, T=4, E=8, ld=8, k=2, score=0, bias=None, groups=1, tg=1, gt=1,
              renorm=1, scale=1.0, idx=FAKE, w=FAKE, probs=None)


@no_gpu
@pytest.mark.parametrize("over,code", [
    (dict(dtype=3), 1), (dict(dtype=-1), 1), (dict(T=-1), 1), (dict(k=0), 1), (dict(k=65, E=80, ld=80), 1),
    (dict(E=0), 1), (dict(E=1025, ld=1025), 1), (dict(ld=7), 1), (dict(score=2), 1),
    (dict(groups=3), 1), (dict(groups=0), 1), (dict(E=128, ld=128, groups=128), 1),
    (dict(groups=2, tg=3), 1), (dict(groups=2, tg=0), 1), (dict(gt=0), 1), (dict(gt=3), 1),
    (dict(k=9), 1), (dict(groups=4, tg=1, k=3), 1), (dict(T=1 << 30), 2),
    (dict(logits=None), 1), (dict(idx=None), 1), (dict(w=None), 1),
    (dict(logits=FAKE + 1), 1), (dict(dtype=2, logits=FAKE + 2), 1), (dict(bias=FAKE + 2), 1),
    (dict(idx=FAKE + 4), 1), (dict(w=FAKE + 2), 1), (dict(probs=FAKE + 4), 1),
])
def test_router_rejects(over, code):
    assert call("ep_router", ROUTER, over) == code, ep.last_error()
    assert ep.last_error()


ROUTER_B = dict(logits=FAKE, dtype=0, T=4, E=8, ld=8, k=2, score=0, renorm=1, scale=1.0, idx=FAKE,
                gw=FAKE, gp=None, gl=FAKE)


@no_gpu
@pytest.mark.parametrize("over,code", [
    (dict(dtype=5), 1), (dict(T=-1), 1), (dict(k=0), 1), (dict(E=1025, ld=1025), 1), (dict(ld=7), 1),
    (dict(score=-1), 1), (dict(logits=None), 1), (dict(idx=None), 1), (dict(gw=None), 1),
    (dict(gl=None), 1), (dict(gp=FAKE + 2), 1), (dict(gl=FAKE + 1), 1), (dict(idx=FAKE + 4), 1),
])
def test_router_backward_rejects(over, code):
    assert call("ep_router_backward", ROUTER_B, over) == code, ep.last_error()
    assert ep.last_error()


PERMUTE = dict(x=FAKE, dtype=0, T=4, H=7, ldx=7, k=2, slot=FAKE, w=None, rows=FAKE, ldr=7, R=8,
               counts=None, offsets=None, E=0)
ROWS_BAD = [
    (dict(dtype=3), 1), (dict(T=-1), 1), (dict(k=0), 1), (dict(k=65), 1), (dict(H=0), 1),
    (dict(H=65537), 1), (dict(R=-1), 1), (dict(R=1 << 31), 1), (dict(T=1 << 30, k=2), 2),
    (dict(T=(1 << 30) - 1, k=2, H=4096), 2), (dict(slot=None), 1), (dict(slot=FAKE + 2), 1),
    (dict(w=FAKE + 2), 1),
]


@no_gpu
@pytest.mark.parametrize("over,code", ROWS_BAD + [
    (dict(x=None), 1), (dict(x=FAKE + 1), 1), (dict(dtype=2, x=FAKE + 2), 1), (dict(ldx=6), 1),
    (dict(rows=None), 1), (dict(ldr=6), 1), (dict(rows=FAKE + 1), 1), (dict(counts=FAKE), 1),
    (dict(offsets=FAKE), 1), (dict(counts=FAKE, offsets=FAKE), 1),
    (dict(counts=FAKE, offsets=FAKE, E=1025), 1), (dict(counts=FAKE, offsets=FAKE + 2, E=8), 1),
])
def test_permute_rejects(over, code):
    base = dict(PERMUTE)
    if over.get("H", 0) > 7:
        base.update(ldx=1 << 17, ldr=1 << 17)
    assert call("ep_permute", base, over) == code, ep.last_error()
    assert ep.last_error()


PERMUTE_B = dict(g=FAKE, dtype=0, T=4, H=7, ldg=7, R=8, k=2, slot=FAKE, w=FAKE, x=FAKE, ldx=7, gx=FAKE,
                 ldgx=7, gw=FAKE)


@no_gpu
@pytest.mark.parametrize("over,code", [(o, c) for o, c in ROWS_BAD if o.get("H", 0) <= 7] + [
    (dict(g=None), 1), (dict(ldg=6), 1), (dict(x=None), 1), (dict(ldx=6), 1), (dict(gx=None), 1),
    (dict(ldgx=6), 1), (dict(gw=FAKE + 2), 1), (dict(g=FAKE + 1), 1),
])
def test_permute_backward_rejects(over, code):
    assert call("ep_permute_backward", PERMUTE_B, over) == code, ep.last_error()
    assert ep.last_error()


UNPERMUTE = dict(y=FAKE, dtype=0, T=4, H=7, ldy=7, R=8, k=2, slot=FAKE, w=None, out=FAKE, ldo=7)


@no_gpu
@pytest.mark.parametrize("over,code", [(o, c) for o, c in ROWS_BAD if o.get("H", 0) <= 7] + [
    (dict(y=None), 1), (dict(ldy=6), 1), (dict(out=None), 1), (dict(ldo=6), 1), (dict(out=FAKE + 1), 1),
])
def test_unpermute_rejects(over, code):
    assert call("ep_unpermute", UNPERMUTE, over) == code, ep.last_error()
    assert ep.last_error()


UNPERMUTE_B = dict(g=FAKE, dtype=0, T=4, H=7, ldg=7, k=2, slot=FAKE, w=FAKE, y=FAKE, ldy=7, gy=FAKE,
                   ldgy=7, R=8, gw=FAKE, counts=None, offsets=None, E=0)


@no_gpu
@pytest.mark.parametrize("over,code", [(o, c) for o, c in ROWS_BAD if o.get("H", 0) <= 7] + [
    (dict(g=None), 1), (dict(ldg=6), 1), (dict(y=None), 1), (dict(ldy=6), 1), (dict(gy=None), 1),
    (dict(ldgy=6), 1), (dict(gw=FAKE + 2), 1), (dict(counts=FAKE), 1),
])
def test_unpermute_backward_rejects(over, code):
    assert call("ep_unpermute_backward", UNPERMUTE_B, over) == code, ep.last_error()
    assert ep.last_error()


PACK = dict(codes=FAKE, scales=FAKE, zeros=None, dtype=0, E=2, N=8, K=64, G=32, gated=0, packed=FAKE,
            bytes=1 << 20)
W4_BAD = [
    (dict(dtype=2), 1), (dict(E=0), 1), (dict(E=1025), 1), (dict(N=0), 1), (dict(N=(1 << 20) + 1), 1),
    (dict(N=7, gated=1), 1), (dict(K=0), 1), (dict(K=48), 1), (dict(K=65568), 1), (dict(G=0), 1),
    (dict(G=16), 1), (dict(G=96), 1), (dict(G=192), 1), (dict(packed=None), 1), (dict(packed=FAKE + 128), 1),
    (dict(bytes=100), 1),
]


@no_gpu
@pytest.mark.parametrize("over,code", W4_BAD + [
    (dict(codes=None), 1), (dict(scales=None), 1), (dict(scales=FAKE + 1), 1),
])
def test_w4_pack_rejects(over, code):
    assert call("ep_w4_pack", PACK, over) == code, ep.last_error()
    assert ep.last_error()


MATMUL = dict(x=FAKE, dtype=0, ldx=64, xrows=4, src=None, packed=FAKE, bytes=1 << 20, E=2, N=8, K=64,
              G=32, zeros=0, gated=0, offsets=FAKE, counts=None, R=4, out=FAKE, ldo=8)


@no_gpu
@pytest.mark.parametrize("over,code", [(o, c) for o, c in W4_BAD] + [
    (dict(R=-1), 1), (dict(R=1 << 31), 1), (dict(offsets=None), 1), (dict(E=1, offsets=None, counts=FAKE), 1),
    (dict(x=None), 1), (dict(ldx=63), 1), (dict(out=None), 1), (dict(ldo=7), 1), (dict(xrows=3), 1),
    (dict(xrows=0, src=FAKE), 1), (dict(src=FAKE + 2), 1), (dict(offsets=FAKE + 2), 1),
    (dict(x=FAKE + 1), 1),
    (dict(R=(1 << 31) - 1, xrows=(1 << 31) - 1, N=1 << 20, ldo=1 << 20, bytes=1 << 40), 2),
])
def test_expert_matmul_w4_rejects(over, code):
    base = dict(MATMUL)
    if over.get("K", 0) > 64:
        base["ldx"] = 1 << 17
    assert call("ep_expert_matmul_w4", base, over) == code, ep.last_error()
    assert ep.last_error()


def test_no_tokens_and_no_rows_are_noops():
    L = ep.lib()
    assert L.ep_router(None, 0, 0, 8, 8, 2, 0, None, 1, 1, 1, 1, 1.0, None, None, None, None) == 0
    assert L.ep_router_backward(None, 0, 0, 8, 8, 2, 0, 1, 1.0, None, None, None, None, None) == 0
    assert L.ep_permute(None, 0, 0, 7, 7, 2, None, None, None, 7, 0, None, None, 0, None) == 0
    assert L.ep_permute_backward(None, 0, 0, 7, 7, 0, 2, None, None, None, 7, None, 7, None, None) == 0
    assert L.ep_unpermute(None, 0, 0, 7, 7, 0, 2, None, None, None, 7, None) == 0
    assert L.ep_expert_matmul_w4(None, 0, 64, 0, None, None, 0, 2, 8, 64, 32, 0, 0, FAKE, None, 0,
                                 None, 8, None) == 0
    assert ep.last_error() == ""


def test_packed_size():
    # tiles of 16 rows x 128 k (1 KiB), 16-bit scales per row block and group,
    # padded to 256 bytes; groups under 128 padded to whole tiles
    def up(n):
        return (n + 255) // 256 * 256
    assert ep.ep_w4_packed_size(1, 16, 128, 128) == 1024 + up(32)
    assert ep.ep_w4_packed_size(2, 17, 160, 128) == 2 * 2 * 2 * 1024 + up(2 * 2 * 2 * 32)
    assert ep.ep_w4_packed_size(2, 17, 160, 32) == 2 * 2 * 2 * 1024 + up(2 * 2 * 8 * 32)
    assert ep.ep_w4_packed_size(2, 17, 160, 32, True) == \
        2 * 2 * 2 * 1024 + up(2 * 2 * 8 * 32) + up(2 * 2 * 8 * 16)
    assert ep.ep_w4_packed_size(1, 34, 128, 256, False, True) == 4 * 1024 + up(4 * 32)
    assert ep.ep_w4_packed_size(1, 33, 128, 128, False, True) == 0
    assert ep.ep_w4_packed_size(1, 16, 130, 128) == 0
    assert ep.ep_w4_packed_size(0, 16, 128, 128) == 0


def test_binding_refuses_host_tensors_and_types():
    x = torch.zeros(4, 8)
    slot = torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="device tensor"):
        ep.ep_router(x, 2)
    with pytest.raises(TypeError, match="bfloat16"):
        ep.ep_router(x.int(), 2)
    with pytest.raises(TypeError):
        ep.ep_permute([[1.0]], slot)
    with pytest.raises(ValueError, match="device tensor"):
        ep.ep_unpermute(x, slot)
    with pytest.raises(ValueError, match="device tensor"):
        ep.ep_w4_pack(torch.zeros(1, 8, 16, dtype=torch.uint8), torch.zeros(1, 8, 1, dtype=torch.float16),
                      group_size=32)
    with pytest.raises(TypeError, match="uint8"):
        ep.ep_w4_pack(x, x)
