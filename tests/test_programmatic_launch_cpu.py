"""Kernels launched while the stream's previous kernel still drains see its
results only after griddepcontrol.wait.  A pointer that promises the memory
to be constant and unaliased (const __restrict__, __ldg) lets the compiler load
before the wait, so none of their sources may use one."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mlp_gemms_gb300", "csrc")


def _text(path):
    with open(path) as f:
        return re.sub(r"//[^\n]*", "", f.read())


SOURCES = {os.path.basename(p): _text(p) for p in sorted(glob.glob(os.path.join(CSRC, "*.cu")))}
KERNELS = sorted({(name, k) for name, text in SOURCES.items() for k in re.findall(r"\blaunch_pdl\((\w+)", text)})


def test_programmatic_kernels_are_found():
    assert {k for _, k in KERNELS} >= {"ckpt_fwd_kernel", "ckpt_bwd_kernel", "ckpt_colsum_kernel", "skinny_kernel",
                                       "ragged_kernel", "ragged_split_kernel", "wgrad_sum_kernel"}


@pytest.mark.parametrize("name,kernel", KERNELS, ids=lambda v: v)
def test_programmatic_kernels_make_no_read_only_promise(name, kernel):
    params = re.findall(r"\b%s\(((?:[^()]|\([^()]*\))*)\)\s*\{" % kernel, SOURCES[name])
    assert len(params) == 1, "definition of %s" % kernel
    assert "__restrict" not in params[0]


@pytest.mark.parametrize("name", sorted({name for name, _ in KERNELS}))
def test_programmatic_sources_use_no_read_only_loads(name):
    assert not re.search(r"\b__ldg\s*\(", SOURCES[name])
