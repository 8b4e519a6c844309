"""The paged cache's kernels compile for sm_103a without register spills, but for two whose register
budgets are fixed by their warps: the 64-row variant of the few-row attention (18 warps, 96 registers) and
the prompt attention (registers moved between warpgroups).  Those stay below a bound."""

import tempfile

import pytest
from test_build_resources import NVCC, _resources
import os

pytestmark = pytest.mark.skipif(not os.path.exists(NVCC), reason="nvcc not found")


@pytest.mark.parametrize("src", ["kv_tables.cu", "kv_append.cu", "kv_few.cu", "kv_prompt.cu"])
def test_spills(src):
    with tempfile.TemporaryDirectory() as tmp:
        _, kernels = _resources(src, tmp)
    assert kernels
    for name, spills in kernels.items():
        bound = 0
        if "k_attn_few" in name and "ELi64EEEv" in name:
            bound = 320
        elif "k_attn_prompt" in name:
            bound = 32
        assert max(spills) <= bound, (name, spills)
