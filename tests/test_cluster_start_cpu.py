"""A block of a cluster may touch another's shared memory only once that one is
known to run: every function that reads, writes or arrives at another block's
memory has a cluster barrier before the first such access."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mlp_gemms_gb300", "csrc")
REMOTE = re.compile(r"\b(?:leader_addr|peer_addr|cta_addr|st_cluster_u32|arrive_on_leader\w*)\(|mapa\.shared::cluster|"
                    r"\b(?:ld|st)\.shared::cluster")


def _functions():
    """(file, first line, text) of the functions that hold a cluster barrier."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        with open(path) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        line = 1
        for body in re.split(r"(?<=\n\}\n)", text):
            if "cluster_sync_all();" in body:
                yield os.path.basename(path), line, body
            line += body.count("\n")


FUNCTIONS = list(_functions())


def test_clustered_kernels_are_found():
    assert {f for f, _, body in FUNCTIONS if REMOTE.search(body)} == {
        "ckpt.cu", "gemm_kernel.cuh", "gemm_pair.cu", "norm.cu", "ragged.cu"}


@pytest.mark.parametrize("name,line,body", FUNCTIONS, ids=["%s:%d" % f[:2] for f in FUNCTIONS])
def test_a_barrier_before_the_first_remote_access(name, line, body):
    remote = REMOTE.search(body)
    if remote is not None:
        assert body.index("cluster_sync_all();") < remote.start()
