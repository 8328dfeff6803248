"""What the CUDA sources may not hold, read as text."""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_no_tma_load_with_cluster_multicast():
    """The library is also loaded by the ranks of a job on several GPUs, where such a load is not to be used:
    CTAs that want the same tile read it through L2."""
    files = [f for e in ("cu", "cuh", "h") for f in glob.glob(os.path.join(ROOT, "speculative_decoding_verify_ragged_gb300", "csrc", "*." + e))]
    assert len(files) > 10
    for path in files:
        with open(path) as f:
            # PTX strings may be split over lines: an instruction ends at its ';' or its operand list
            for ins in re.findall(r"cp\.async\.bulk[^;\[(]*", f.read()):
                assert ".multicast" not in ins, (os.path.basename(path), ins)
