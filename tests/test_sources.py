"""Rules that every kernel of the library keeps, read from its sources."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "decode_gemm_e8_b200", "csrc")


def _sources():
    files = sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh")) +
                   glob.glob(os.path.join(CSRC, "*.h")))
    assert len(files) > 10
    return {os.path.basename(f): open(f).read() for f in files}


def test_no_copy_is_multicast_to_a_cluster():
    """Every bulk and tensor copy fills the shared memory of its own CTA: one library serves
    every rank of a run on several GPUs.  (A commit signals barriers and copies nothing.)"""
    for name, text in _sources().items():
        text = re.sub(r'"\s*\n\s*"', "", text)   # an instruction may be cut into several literals
        for line in text.splitlines():
            if "multicast::cluster" in line:
                assert "tcgen05.commit" in line and "cp.async" not in line, (name, line)
