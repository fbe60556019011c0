"""The recorded DRAM traffic of the large GEMMs is valid for the sources that it was captured on: its key has to cover
every file that is compiled into the kernel."""
import json
import os
import re

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "bit_nf4_quantized_08_b200", "csrc")


def _includes(name, seen):
    """name and what it includes from its own folder, and so on."""
    if name in seen:
        return seen
    seen.add(name)
    with open(os.path.join(CSRC, name)) as f:
        for inc in re.findall(r'^#include "([^"]+)"', f.read(), re.M):
            if os.path.exists(os.path.join(CSRC, inc)) and "/" not in inc:  # (the ABI header holds no kernel code)
                _includes(inc, seen)
    return seen


@pytest.mark.parametrize("kind", ["fwd_gemm", "dx_gemm"])
def test_traffic_key_covers_the_kernel_s_sources(kind):
    with open(os.path.join(ROOT, "profiles", "traffic.json")) as f:
        entry = json.load(f)[kind]
    # gemm_pair.cuh holds the kernel, linear.cuh its schedules and launches
    assert set(entry["files"]) == _includes("gemm_pair.cuh", set()) | {"linear.cuh"}
