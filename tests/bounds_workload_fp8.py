"""A run of the e4m3 and expert kernels on small seeded inputs for the bounds-checking build: every call
is followed by a read of the bounds word.  Imported by tests/test_gpu_bounds_fp8.py (with libhq.so) and
run as a script in a child process with HQ_LIBRARY=libhq_bounds.so:

    HQ_LIBRARY=libhq_bounds.so python tests/bounds_workload_fp8.py OUT.pt
"""

from __future__ import annotations

import os
import sys

import torch


def _gen(seed: int) -> torch.Generator:
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def run_all(hq) -> tuple[dict, dict]:
    """(outputs, bounds words after each call)."""
    out, words = {}, {}

    def mark(name, **tensors):
        torch.cuda.synchronize()
        words[name] = hq.hq_debug_bounds_status()[1]
        out.update({f"{name}.{k}": v.view(torch.uint8) if v.element_size() == 1 else v for k, v in tensors.items()})

    hq.hq_debug_bounds_status()  # clear
    for dt in (torch.bfloat16, torch.float32):
        for M, N, K in ((1, 200, 300), (3, 130, 128), (40, 264, 257), (300, 390, 520), (700, 1030, 130)):
            tag = f"{dt}_{M}x{N}x{K}"
            X = torch.randn((M, K), device="cuda", generator=_gen(M)).to(dt)
            W = torch.randn((N, K), device="cuda", generator=_gen(N)).to(dt)
            a, sa = hq.fp8_rows_outputs(M, K)
            hq.hq_fp8_quantize_rows(X, a, sa)
            mark("rows_" + tag, codes=a, scales=sa)
            w, sw = hq.fp8_blocks_outputs(N, K)
            hq.hq_fp8_quantize_blocks(W, w, sw)
            mark("blocks_" + tag, codes=w, scales=sw)
            Y = torch.empty((M, N), dtype=dt, device="cuda")
            hq.hq_fp8_linear(X, w, sw, Y, hq.alloc_workspace(hq.hq_fp8_linear_workspace_bytes(M, K)))
            mark("linear_" + tag, Y=Y)
            for impl in (1, 2, 3, 4):
                Z = torch.empty_like(Y)
                hq.hq_debug_fp8_gemm_impl(a, sa, None, w, sw, K, Z, impl)
                mark(f"gemm{impl}_" + tag, Y=Z)
    for T, top, E, K in ((5, 3, 4, 131), (600, 8, 40, 264), (3000, 2, 7, 64)):
        tag = f"{T}x{top}x{E}x{K}"
        ids = torch.randint(-1, E + 1, (T, top), device="cuda", generator=_gen(T)).to(torch.int32)
        off, order, pos = (t.fill_(-7) for t in hq.expert_sort_outputs(T, top, E))
        hq.hq_expert_sort(ids, E, off, order, pos, hq.alloc_workspace(hq.hq_expert_sort_workspace_bytes(T, top, E)))
        mark("sort_" + tag, offsets=off, order=order, position=pos)
        X = torch.randn((T, K), device="cuda", generator=_gen(K)).to(torch.bfloat16)
        w = torch.rand((T, top), device="cuda", generator=_gen(top))
        rows = torch.zeros((T * top, K), dtype=X.dtype, device="cuda")
        hq.hq_expert_dispatch(X, pos, rows)
        codes, scales = hq.fp8_rows_outputs(T * top, K)
        codes.view(torch.uint8).zero_(), scales.zero_()
        hq.hq_expert_dispatch_fp8(X, pos, codes, scales)
        mark("dispatch_" + tag, rows=rows, codes=codes, scales=scales)
        W = torch.randn((E, 96, K), device="cuda", generator=_gen(E)).to(torch.bfloat16)
        wc, ws = hq.fp8_blocks_outputs(96, K, E)
        hq.hq_fp8_quantize_blocks(W, wc, ws)
        Y = torch.zeros((T * top, 96), dtype=torch.bfloat16, device="cuda")
        hq.hq_fp8_expert_gemm(codes, scales, off, wc, ws, K, Y)
        mark("product_" + tag, Y=Y)
        Z, dr, dw = torch.empty_like(X), torch.zeros_like(rows), torch.zeros_like(w)
        hq.hq_expert_combine(rows, pos, w, Z)
        hq.hq_expert_combine_backward(X, rows, pos, w, dr, dw)
        mark("combine_" + tag, Y=Z, d_rows=dr, d_weights=dw)
    return {k: v.cpu() for k, v in out.items()}, words


if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    import post_weight_quantization_tcgen05_b200 as hq_mod
    outputs, bound_words = run_all(hq_mod)
    torch.save({"outputs": outputs, "words": bound_words, "enabled": hq_mod.hq_debug_bounds_status()[0],
                "library": os.path.basename(hq_mod._LIB_PATH)}, sys.argv[1])
