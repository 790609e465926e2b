"""Layers of experts: calibration and the quantised product.

A router sends each token to `top` of E experts (ids int32 [T, top]; an id outside [0, E) is a
dropped choice).  hq_expert_sort and hq_expert_dispatch lay the tokens' rows out by expert, so that

* calibration sums one Hessian for each expert from its own tokens: `expert_hessians`.  The Hessian
  is a sum over tokens ("hipfire-calib-data" dataset card: full Hessians XX^T), so chunks add up and
  every expert's matrix goes through hq_gptq_quantize like any other layer's;
* the e4m3 layer runs as one product over all experts' rows, and the outputs return weighted to
  token order: `expert_linear`.

Every arithmetic step runs in the library's kernels; this module only allocates and calls.
"""

from __future__ import annotations

import torch


def sort_tokens(hq, ids, E: int):
    """(offsets [E + 1], order [T * top], position [T, top]) of hq_expert_sort, newly allocated."""
    T, top = ids.shape
    offsets, order, position = hq.expert_sort_outputs(T, top, E, ids.device)
    workspace = hq.alloc_workspace(hq.hq_expert_sort_workspace_bytes(T, top, E), ids.device)
    hq.hq_expert_sort(ids, E, offsets, order, position, workspace)
    return offsets, order, position


def expert_hessians(hq, X, ids, H, dev_status=None) -> list[int]:
    """H [E, K, K] (fp32, lower triangles) += each expert's sum of x^T x over the tokens X [T, K]
    sent to it; returns the tokens of each expert (what hq_imatrix divides by).  A token that names
    an expert twice counts twice.  Reads the offsets back, so it waits for the sort."""
    (T, K), top, E = X.shape, ids.shape[1], H.shape[0]
    offsets, _, position = sort_tokens(hq, ids, E)
    rows = torch.empty((T * top, K), dtype=X.dtype, device=X.device)
    hq.hq_expert_dispatch(X, position, rows)
    ends = offsets.tolist()
    for e in range(E):
        if ends[e] < ends[e + 1]:
            hq.hq_hessian_accumulate(H[e], rows[ends[e]:ends[e + 1]], dev_status)
    return [ends[e + 1] - ends[e] for e in range(E)]


def expert_linear(hq, X, ids, weights, w_codes, w_scales, Y, dev_status=None) -> None:
    """Y [T, N] = sum_j weights[t, j] (X[t] W_e^T), e = ids[t, j], with the experts' weights as
    hq_fp8_quantize_blocks makes them (codes [E, N, pitch]); X [T, K] is quantised on the way.
    weights fp32 [T, top] or None (all ones).  The experts' outputs are kept in Y's dtype."""
    (T, K), (E, N) = X.shape, w_codes.shape[:2]
    top = ids.shape[1]
    offsets, _, position = sort_tokens(hq, ids, E)
    codes, scales = hq.fp8_rows_outputs(T * top, K, X.device)
    hq.hq_expert_dispatch_fp8(X, position, codes, scales)
    rows = torch.empty((T * top, N), dtype=Y.dtype, device=X.device)
    hq.hq_fp8_expert_gemm(codes, scales, offsets, w_codes, w_scales, K, rows, dev_status)
    hq.hq_expert_combine(rows, position, weights, Y)
