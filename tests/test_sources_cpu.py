"""Where the library's sources keep what (CPU only)."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "entropy_active_span_gb300", "csrc")


def test_lm_head_sources_hold_the_lm_head_alone():
    """bench.py knows the build of a captured DRAM figure by the text of these four
    files: an operator's declaration or entry point in one of them would cast off
    every figure although no LM-head kernel changed."""
    for f in ("eas_gemm_tc.cu", "eas_device.cuh", "eas_kernels.h", "eas_api.cu"):
        found = re.search(r"rmsnorm|embed_|clip_grad|launch_overlapped",
                          open(os.path.join(CSRC, f)).read())
        assert found is None, (f, found)
