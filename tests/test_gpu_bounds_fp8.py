"""The bounds-checking build on the e4m3 and expert kernels: no index check fails and the results are
those of libhq.so, bit for bit."""

import os
import subprocess
import sys

import pytest
import torch

import bounds_workload_fp8

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_bounds_build_finds_no_violation_and_changes_no_bit(cuda_device, tmp_path):
    import post_weight_quantization_tcgen05_b200 as hq
    ref, words = bounds_workload_fp8.run_all(hq)
    assert all(w == 0 for w in words.values())
    out = tmp_path / "bounds.pt"
    r = subprocess.run([sys.executable, os.path.join(ROOT, "tests", "bounds_workload_fp8.py"), str(out)],
                       env=dict(os.environ, HQ_LIBRARY="libhq_bounds.so"), cwd=ROOT, capture_output=True, text=True,
                       timeout=600)
    assert r.returncode == 0, r.stdout + r.stderr
    res = torch.load(out)
    assert res["library"] == "libhq_bounds.so" and res["enabled"] is True
    bad = {k: (w >> 16, w & 0xFFFF) for k, w in res["words"].items() if w != 0}
    assert not bad, f"index checks failed (file tag, line): {bad}"
    for k, v in ref.items():
        assert torch.equal(v, res["outputs"][k]), k
