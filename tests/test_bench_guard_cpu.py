"""The hash that tells a counter summary is stale covers the code that it was taken on."""
import os
import re

import pytest

import bench

SIGNATURES = {"kda.h", "kda_internal.h"}     # declarations: no device code


def local_headers(path):
    found = set()
    for name in re.findall(r'#include "([^"]+)"', open(path).read()):
        inner = os.path.join(bench.CSRC, name)
        if name not in SIGNATURES and name not in found:
            found |= {name} | local_headers(inner)
    return found


@pytest.mark.parametrize("op", sorted(bench.KERNEL_SOURCES))
def test_hash_covers_every_header_with_device_code(op):
    listed = {os.path.basename(p) for p in bench.KERNEL_SOURCES[op]}
    assert f"{op}.hip" in listed
    assert local_headers(os.path.join(bench.CSRC, f"{op}.hip")) <= listed
