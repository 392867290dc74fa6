"""What the measured HBM traffic of bench.py hangs on: the headers that go into
the digest of the dispatch, combine and layout kernels hold nothing of the
router, the row movement and the 4-bit products, so that working on these does
not make the counters of those stale."""

import os
import re

import bench

CSRC = os.path.join(bench.ROOT, "combine_ep_layout_04_amd", "csrc")


def code(name):
    with open(os.path.join(CSRC, name), encoding="utf-8") as fh:
        return bench._code_only(fh.read())


def test_digest_headers_hold_nothing_of_the_layer():
    names = set(re.findall(r"struct (\w+) \{", code("ep_layer.h")))
    names |= set(re.findall(r"\b(\w+)\(", code("ep_layer.h")))
    assert {"RouterArgs", "MoveArgs", "W4Args", "launch_router", "launch_move_rows", "launch_w4"} <= names
    for header in ("ep_internal.h", "ep_device.h", "ep_cast.h"):
        assert not names & set(re.findall(r"\w+", code(header))), header
        assert "ep_layer.h" not in code(header)
    # and of their sources only the ones that the layer is made of include it
    users = {f for f in os.listdir(CSRC) if f.endswith(".hip") and '"ep_layer.h"' in code(f)}
    assert users == {"ep_api.hip", "ep_router.hip", "ep_permute.hip", "ep_w4.hip"}
    assert not users & set(bench.KERNEL_SOURCES.values())
