"""Every kernel of the e4m3 product with the scales that quantised values have, against the fp64 oracle:
dense, and with experts whose weights have several blocks of 128 rows, each with scales of its own."""

import numpy as np
import pytest
import torch

import oracle
from gpu_helpers import to_np64
from test_gpu_fp8 import IMPLS, TYPES, activations, check_product, gen, hq, quantise_blocks, quantise_rows, values  # noqa: F401

pytestmark = pytest.mark.gpu


def uneven_weights(seed, E, N, K):
    """Weights whose blocks of 128 x 128 differ in size by powers of e."""
    g = gen(seed)
    each = torch.exp(torch.randn((E, -(-N // 128), -(-K // 128)), generator=g, device="cuda"))
    W = torch.randn((E, N, K), generator=g, device="cuda")
    return W * each.repeat_interleave(128, 1)[:, :N].repeat_interleave(128, 2)[:, :, :K]


@pytest.mark.parametrize("impl", list(IMPLS))
@pytest.mark.parametrize("M,N,K,out", [(3, 300, 1000, "f32"), (600, 520, 1537, "f32"), (600, 520, 1537, "bf16"),
                                       (2900, 3400, 400, "bf16"), (257, 129, 5120, "f32")])
def test_every_kernel_with_real_scales(hq, cuda_device, M, N, K, out, impl):  # noqa: F811
    a, sa = quantise_rows(hq, activations(M, M, K, "bf16"))
    w, sw = quantise_blocks(hq, uneven_weights(N, 1, N, K)[0])
    ref, size = oracle.fp8_product(values(a, K), to_np64(sa).T, values(w, K), to_np64(sw))
    Y = torch.full((M, N), float("nan"), dtype=TYPES[out], device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    hq.hq_debug_fp8_gemm_impl(a, sa, None, w, sw, K, Y, IMPLS[impl], dev_status=status)
    check_product(Y, ref, size, K, impl)
    assert status.item() == 0


@pytest.mark.parametrize("impl", list(IMPLS))
@pytest.mark.parametrize("sizes,gaps,N,K,out", [([5, 0, 130, 1], (2, 3), 390, 520, "f32"), ([257, 0, 1, 255, 256], (0, 9), 640, 260, "bf16"),
                                                ([300, 512, 3, 700], (1, 0), 1100, 400, "f32")])
def test_every_kernel_on_experts_with_real_scales(hq, cuda_device, sizes, gaps, N, K, out, impl):  # noqa: F811
    E = len(sizes)
    ends = np.cumsum([gaps[0], *sizes])
    rows = int(ends[-1]) + gaps[1]
    a, sa = quantise_rows(hq, activations(rows, rows, K, "bf16"))
    w, sw = quantise_blocks(hq, uneven_weights(N, E, N, K))
    assert sw.unique().numel() == sw.numel()  # no two blocks have the same scale
    offsets = torch.tensor(ends, dtype=torch.int32, device="cuda")
    Y = torch.full((rows, N), 7.0, dtype=TYPES[out], device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    hq.hq_debug_fp8_gemm_impl(a, sa, offsets, w, sw, K, Y, IMPLS[impl], dev_status=status)
    ref, size = np.full((rows, N), 7.0), np.zeros((rows, N))
    oracle.fp8_expert_product(values(a, K), to_np64(sa).T, ends, [values(w[e], K) for e in range(E)], to_np64(sw), ref, size)
    check_product(Y, ref, size, K, impl)
    assert (Y[:ends[0]] == 7).all() and (Y[ends[-1]:] == 7).all()
    # an expert alone, by the same kernel, has the same bits
    for e in range(E):
        part = slice(ends[e], ends[e + 1])
        if sizes[e] > 0:
            Z = torch.empty((sizes[e], N), dtype=Y.dtype, device="cuda")
            hq.hq_debug_fp8_gemm_impl(a[part].contiguous(), sa[:, part].contiguous(),
                                      torch.tensor([0, sizes[e]], dtype=torch.int32, device="cuda"), w[e:e + 1], sw[e:e + 1],
                                      K, Z, IMPLS[impl], dev_status=status)
            assert torch.equal(Z, Y[part])
    assert status.item() == 0
