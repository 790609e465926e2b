"""The e4m3 products on the GPU where their kernels' warps, CTAs and clusters meet."""

import pytest
import torch

from test_gpu_fp8 import IMPLS, TYPES, hq, small_integers  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("impl", ["few16", "few64"])
@pytest.mark.parametrize("M,N,K", [(1, 1, 1024), (2, 33, 2000), (17, 200, 2000), (70, 481, 1537), (9, 5000, 1000)])
def test_clusters_whose_last_columns_split_a_warp(hq, cuda_device, M, N, K, impl):  # noqa: F811
    """K is split over clusters of CTAs and N ends inside a warp's columns: exact sums, the same in every
    one of many calls."""
    a, sa = small_integers(1, M, K, 1)
    w, sw = small_integers(2, N, K, 128)
    sa = sa.t().contiguous()
    ref = ((a[:, :K].double() * sa.double().t().repeat_interleave(128, 1)[:, :K])
           @ (w[:, :K].double() * sw.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]).t())
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for dt in ("f32", "bf16"):
        Y = torch.full((50, M, N), float("nan"), dtype=TYPES[dt], device="cuda")
        for y in Y:
            hq.hq_debug_fp8_gemm_impl(a, sa, None, w, sw, K, y, IMPLS[impl], dev_status=status)
        assert (Y == ref.float().to(TYPES[dt])).all()
    assert status.item() == 0
