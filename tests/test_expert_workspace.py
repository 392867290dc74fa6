"""The backward's workspace without the weights' gradient: no rows of x are
laid out, so none is asked for them."""

import pytest
import torch

from combine_ep_layout_04_amd import ep

from moe_util import DEV

FAKE = 0x100000


@pytest.mark.skipif(torch.cuda.device_count() > 0, reason="fake pointers must never reach a launch on a real GPU")
@pytest.mark.parametrize("K,src", [(64, FAKE), (63, None), (63, FAKE)])
def test_rows_alone_need_none_for_x(K, src):
    """Accepted: without a device the launch fails, after all checks."""
    def plain(gw, work, size):
        return ep.lib().ep_expert_matmul_backward(FAKE, 0, 32, FAKE, K, 8, src, FAKE, 2, 32, K, FAKE, None, 8, FAKE, K,
                                                  gw, 0, work, size, None)

    def gated(gw, work, size):
        return ep.lib().ep_expert_glu_backward(FAKE, 0, 16, FAKE, 32, FAKE, K, 8, src, FAKE, 2, 32, K, FAKE, None, 8,
                                               FAKE, K, gw, 0, work, size, None)
    assert plain(None, None, 0) == 3 and plain(FAKE, None, 0) == 1
    assert gated(None, FAKE, 512) == 3 and gated(None, FAKE, 511) == 1 and gated(FAKE, FAKE, 512) == 1


@pytest.mark.gpu
@pytest.mark.parametrize("each", [3, 40, 300])
@pytest.mark.parametrize("K,gathered", [(64, True), (63, False), (63, True)])
def test_rows_alone(each, K, gathered):
    """The rows' gradient with the smaller workspace has the bits of the call
    for both, which lays x out."""
    E, N = 3, 80
    R = E * each
    g = torch.Generator(device=DEV).manual_seed(1)
    x, w, grad, pre = (torch.randn(s, generator=g, device=DEV).bfloat16()
                       for s in ((R, K), (E, N, K), (R, N), (R, N)))
    off = torch.arange(0, R + 1, each, dtype=torch.int32, device=DEV)
    src = torch.randint(0, R, (R,), generator=g, device=DEV, dtype=torch.int32) if gathered else None
    for gated in (False, True):
        def call(**kw):
            if gated:
                return ep.ep_expert_glu_backward(grad[:, :N // 2], pre, x, w, off, src=src, **kw)
            return ep.ep_expert_matmul_backward(grad, x, w, off, src=src, **kw)
        both, _ = call()
        size = ep.ep_expert_backward_workspace_size(R, N, 8, gated)
        assert size == (R * N * 2 if gated else 0)
        held = torch.full((size + 64,), 7, dtype=torch.uint8, device=DEV)
        alone, none = call(want_weights=False, workspace=held[:size])
        assert none is None and torch.equal(alone.view(torch.int16), both.view(torch.int16))
        assert bool((held[size:] == 7).all())
        torch.cuda.synchronize()
        before = torch.cuda.memory_stats()["requested_bytes.all.allocated"]
        call(want_weights=False)
        asked = torch.cuda.memory_stats()["requested_bytes.all.allocated"] - before
        assert asked == R * K * 2 + size        # the gradient, and no rows of x
