"""The paged cache's sources: no constant or device function that nothing uses, and the register spills that
the kernels have and no more (the 64-row few-row attention has 18 warps on 96 registers a thread)."""

import glob
import os
import re
import tempfile

import pytest
from test_build_resources import NVCC, _resources

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_fp8_mixture_gb300", "csrc")


def test_everything_defined_is_used():
    files = sorted(glob.glob(os.path.join(CSRC, "kv_*")))
    text = {f: re.sub(r"//[^\n]*", "", open(f).read()) for f in files}
    every = "\n".join(text.values())
    defined = set(re.findall(r"\bconstexpr \w+ (k\w+) =", every))
    defined |= set(re.findall(r"__device__ __forceinline__ [\w ]+?\b(\w+)\(", every))
    assert len(defined) > 60
    assert [n for n in sorted(defined) if len(re.findall(rf"\b{n}\b", every)) < 2] == []


@pytest.mark.skipif(not os.path.exists(NVCC), reason="nvcc not found")
@pytest.mark.parametrize("src", ["kv_few.cu", "kv_prompt.cu"])
def test_spills_are_those_known(src):
    with tempfile.TemporaryDirectory() as tmp:
        _, kernels = _resources(src, tmp)
    assert kernels
    for name, spills in kernels.items():
        known = "k_attn_few" in name and "ELi64EEEv" in name
        assert max(spills) <= (216 if known else 0), (name, spills)
