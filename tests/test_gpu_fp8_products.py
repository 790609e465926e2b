"""The e4m3 products on the GPU where their kernels' warps, CTAs and clusters meet."""

import pytest
import torch

from test_gpu_fp8 import IMPLS, TYPES, activations, hq, quantise_blocks, quantise_rows, small_integers  # noqa: F401

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


@pytest.mark.parametrize("M,N,K", [(1, 640, 1024), (5, 384, 5120), (24, 2000, 1537), (100, 2048, 640), (700, 5000, 300),
                                   (3000, 2600, 1024)])
def test_layers_that_take_turns_in_one_workspace(hq, cuda_device, M, N, K):  # noqa: F811
    """Activations 2^12 apart in size, one after the other through the same workspace without a wait, a
    product starting while its rows are still quantised: each result is that of the two steps apart."""
    w, sw = quantise_blocks(hq, activations(1, N, K, "bf16"))
    ws = hq.alloc_workspace(hq.hq_fp8_linear_workspace_bytes(M, K))
    X = [activations(2 + i, M, K, "bf16") * 2.0 ** (12 * i - 6) for i in range(2)]
    want = [torch.empty((M, N), device="cuda") for _ in X]
    for x, y in zip(X, want):
        hq.hq_fp8_gemm(*quantise_rows(hq, x), w, sw, K, y)
    Y = torch.full((40, M, N), float("nan"), device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    for i, y in enumerate(Y):
        hq.hq_fp8_linear(X[i % 2], w, sw, y, ws, dev_status=status)
    for i in range(2):
        assert (Y[i::2] == want[i]).all(), i
    assert status.item() == 0


# (kernel, sizes of the experts' runs or None, M, N, K): every CTA has blocks enough to refill each of stages 0 .. 3
TIMEOUTS = [("single", None, 300, 300, 1024), ("pair", None, 600, 520, 1024), ("few16", None, 5, 300, 16384),
            ("few64", None, 70, 300, 8192), ("few16", [5, 0, 3], 8, 300, 2000), ("few64", [40, 1], 41, 130, 1000),
            ("pair", [300, 2, 298], 600, 520, 1024)]


@pytest.mark.parametrize("stage", [0, 3])
@pytest.mark.parametrize("impl,sizes,M,N,K", TIMEOUTS)
def test_a_wait_that_runs_out_is_reported_and_the_stream_stays_usable(hq, cuda_device, impl, sizes, M, N, K, stage):  # noqa: F811
    """The bounded-wait failure path, made to run: the MMA issuer never releases one operand stage, so
    the wait to refill it runs out (limit 1e6 cycles, about half a millisecond).  The call reports
    HQ_ERR_TIMEOUT through its status word and returns, the peers of a pair or a cluster with it; the next
    calls on the same stream compute the right Y."""
    E = len(sizes) if sizes else 1
    a, sa = small_integers(1, M, K, 1)
    w, sw = small_integers(2, E * N, K, 1)
    sw = sw.view(E, N, -1)[:, ::128].contiguous()
    A = a[:, :K].double() * sa.double().repeat_interleave(128, 1)[:, :K]
    ref = torch.empty((M, N), device="cuda")
    ends = [0]
    for e, n in enumerate(sizes or [M]):
        ends.append(ends[-1] + n)
        W = w.view(E, N, -1)[e, :, :K].double() * sw[e].double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
        ref[ends[-2]:ends[-1]] = (A[ends[-2]:ends[-1]] @ W.t()).float()
    offsets = torch.tensor(ends, dtype=torch.int32, device="cuda") if sizes else None
    args = (a, sa.t().contiguous(), offsets, *((w.view(E, N, -1), sw) if sizes else (w, sw[0])), K)
    Y = torch.zeros((M, N), device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    hq.hq_debug_fp8_gemm_timeout(*args, Y, IMPLS[impl], status, wait_limit_cycles=1_000_000, withhold_stage=stage)
    torch.cuda.synchronize()
    assert status.item() == hq.HQ_ERR_TIMEOUT
    # the same kernel with the short limit and nothing withheld finishes normally, and so does an ordinary call
    status.zero_()
    for call in (lambda: hq.hq_debug_fp8_gemm_timeout(*args, Y, IMPLS[impl], status, wait_limit_cycles=1_000_000),
                 lambda: hq.hq_debug_fp8_gemm_impl(*args, Y, IMPLS[impl], dev_status=status)):
        Y.fill_(float("nan"))
        call()
        assert torch.equal(Y, ref) and status.item() == 0
