"""Stream order of kernels that are launched as programmatic dependents, read from
their sources (CPU).  Such a kernel starts before the one in front of it has ended;
`griddepcontrol.wait` covers that one alone.  So each of them has to execute the wait
somewhere, or a kernel behind it could run beside the one in front of it."""
import glob
import os
import re

import pytest

from paged_kv_decode_ns_gb300 import _build

# file with the launch -> (file with the kernel, kernels)
LAUNCHED_EARLY = {
    "paged_decode_launch.cuh": ("paged_decode.cuh", ["paged_decode_kernel"]),
    "tc_prefill.cu": ("tc_prefill.cu", ["tc_prefill_kernel"]),
    "span_attn.cuh": ("span_attn.cuh", ["span_attn_kernel", "span_join_kernel"]),
    "kv_gather.cu": ("kv_gather.cu", ["kv_gather_kernel"]),
    "verify_drafts.cu": ("verify_drafts.cu", ["verify_kernel"]),
}


def source(name):
    with open(os.path.join(_build.CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def kernel_body(name, kernel):
    m = re.search(r"__global__[^;{]*?\b" + kernel + r"\s*\(.*?\n}\n", source(name), re.S)
    assert m, f"{kernel} not found in {name}"
    return m.group(0)


def test_every_early_launch_is_listed():
    found = {os.path.basename(p) for p in glob.glob(os.path.join(_build.CSRC, "*"))
             if os.path.isfile(p) and "ProgrammaticStreamSerialization" in source(os.path.basename(p))}
    assert found == set(LAUNCHED_EARLY)


@pytest.mark.parametrize("launch", sorted(LAUNCHED_EARLY))
def test_kernels_launched_early_wait_for_the_grid_in_front(launch):
    name, kernels = LAUNCHED_EARLY[launch]
    for kernel in kernels:
        assert "grid_dependency_wait()" in kernel_body(name, kernel), kernel


@pytest.mark.parametrize("name", ["span_attn.cuh", "kv_gather.cu", "verify_drafts.cu"])
def test_loads_behind_the_wait_are_coherent(name):
    """What the grid in front writes changes while such a kernel is resident, so its reads may not go
    through the read-only path (the decode reads its planning arrays before the wait, by contract)."""
    text = source(name)
    assert "__ldg" not in text and "__restrict__" not in text and "ld.global.nc" not in text
