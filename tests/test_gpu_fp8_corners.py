"""Calls of the e4m3 layers that are allowed and seldom made: operands past 2^31 elements in every kernel,
tokens at any address and with values that are no numbers, graphs replayed at once."""

import pytest
import torch

from test_gpu_fp8 import FP8, IMPLS, TYPES, activations, gen, hq, quantise_blocks, quantise_rows, small_integers  # noqa: F401

pytestmark = pytest.mark.gpu


def test_weights_past_2_to_the_31_elements(hq, cuda_device):  # noqa: F811
    """The last of five experts begins past 2^31 elements: its codes, its scales and its rows' products are
    what they are for it alone."""
    E, N, K = 5, 65536, 8192
    assert (E - 1) * N * K >= 2 ** 31
    W = torch.zeros((E, N, K), dtype=torch.bfloat16, device="cuda")
    W[-1] = torch.randn((N, K), generator=gen(1), device="cuda", dtype=torch.bfloat16)
    w, sw = quantise_blocks(hq, W)
    alone, s_alone = quantise_blocks(hq, W[-1:].clone())
    del W
    assert torch.equal(w[-1:].view(torch.uint8), alone.view(torch.uint8)) and torch.equal(sw[-1:], s_alone)
    assert not sw[:-1].any() and not w[:-1].view(torch.uint8).any()
    ends = [0, 2, 2, 5, 6, 300]
    offsets = torch.tensor(ends, dtype=torch.int32, device="cuda")
    own = torch.tensor([0, 294], dtype=torch.int32, device="cuda")
    a, sa = quantise_rows(hq, activations(2, 300, K, "bf16"))
    for impl in IMPLS.values():
        Y, Z = (torch.full((rows, N), float("nan"), dtype=torch.bfloat16, device="cuda") for rows in (300, 294))
        hq.hq_debug_fp8_gemm_impl(a, sa, offsets, w, sw, K, Y, impl)
        hq.hq_debug_fp8_gemm_impl(a[6:].contiguous(), sa[:, 6:].contiguous(), own, alone, s_alone, K, Z, impl)
        assert torch.equal(Y[6:], Z) and Z.any() and not Y[:6].any()


@pytest.mark.parametrize("impl", list(IMPLS))
@pytest.mark.parametrize("experts", [False, True])
def test_results_past_2_to_the_31_elements(hq, cuda_device, impl, experts):  # noqa: F811
    M, N, K = 16500, 131080, 16
    assert M * N > 2 ** 31
    a, sa = small_integers(1, M, K, 1)
    w, sw = small_integers(2, N, K, 128)
    Y = torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda")
    offsets = torch.tensor([0, M - 200, M - 200, M - 3], dtype=torch.int32, device="cuda") if experts else None
    lead = 3 if experts else 1
    ws, ss = (w.view(torch.uint8).expand(lead, N, K).contiguous().view(FP8), sw.expand(lead, *sw.shape).contiguous())
    hq.hq_debug_fp8_gemm_impl(a, sa.t().contiguous(), offsets, ws if experts else w, ss if experts else sw, K, Y, IMPLS[impl])
    W = (w.double() * sw.double().repeat_interleave(128, 0)[:N]).t()
    last = M - 3 if experts else M
    for r in (slice(0, 40), slice(M - 230, last)):
        assert torch.equal(Y[r], ((a[r].double() * sa[r].double()) @ W).float().to(torch.bfloat16))
    if experts:
        assert (Y[last:] == 7).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M", [1, 3, 4, 5, 40])
@pytest.mark.parametrize("K", [1, 17, 255, 1000, 2048, 5121])
def test_layers_of_tokens_at_any_address(hq, cuda_device, M, K, dtype):  # noqa: F811
    """One to four tokens are quantised by the product's kernel, more by one of their own: neither depends
    on where the tokens lie, nor reads what lies around them."""
    N = 200
    w, sw = quantise_blocks(hq, activations(1, N, K, dtype))
    X = activations(M, M, K, dtype)
    ws = hq.alloc_workspace(hq.hq_fp8_linear_workspace_bytes(M, K))
    want = torch.empty((M, N), device="cuda")
    hq.hq_fp8_gemm(*quantise_rows(hq, X), w, sw, K, want)
    for at in (0, 1, 2, 3, 5):
        around = torch.full((M * K + 16,), float("nan"), dtype=X.dtype, device="cuda")
        x = around[at:at + M * K].view(M, K).copy_(X)
        Y = torch.full((M, N), float("nan"), device="cuda")
        hq.hq_fp8_linear(x, w, sw, Y, ws)
        assert torch.equal(Y, want), at


@pytest.mark.parametrize("M", [1, 2, 4, 6, 30, 100])
def test_layers_of_tokens_that_are_no_numbers(hq, cuda_device, M):  # noqa: F811
    """A NaN or an infinity reaches its own token's results and no other's; a token of zeros gives zeros."""
    N, K = 260, 700
    w, sw = quantise_blocks(hq, activations(1, N, K, "bf16"))
    X = activations(2, M, K, "bf16")
    ws = hq.alloc_workspace(hq.hq_fp8_linear_workspace_bytes(M, K))
    Y, Z = (torch.empty((M, N), device="cuda") for _ in range(2))
    hq.hq_fp8_linear(X, w, sw, Y, ws)
    for bad in (float("nan"), float("inf"), -float("inf")):
        for r in {0, M - 1}:
            X2 = X.clone()
            X2[r, K - 1] = bad
            hq.hq_fp8_linear(X2, w, sw, Z, ws)
            others = [i for i in range(M) if i != r]
            assert not Z[r].isfinite().any() and torch.equal(Z[others], Y[others])
    X2 = X.clone()
    X2[M // 2] = -0.0
    hq.hq_fp8_linear(X2, w, sw, Z, ws)
    assert (Z[M // 2] == 0).all()


def test_two_graphs_of_layers_replayed_at_once(hq, cuda_device):  # noqa: F811
    """Two graphs, each a chain of layers through a workspace of its own, replayed over and over on streams of
    their own: each layer reads what the one before wrote, and rewrites the workspace that it read."""
    sizes = (512, 1100, 384, 2000)
    graphs, keep = [], []
    for M in (3, 700):
        ws = hq.alloc_workspace(max(hq.hq_fp8_linear_workspace_bytes(M, k) for k in sizes))
        layers = [quantise_blocks(hq, activations(i, n, k, "bf16") / k) for i, (k, n) in enumerate(zip(sizes, sizes[1:]))]
        acts = [activations(M, M, sizes[0], "bf16")] + [torch.empty((M, n), dtype=torch.bfloat16, device="cuda") for n in sizes[1:]]

        def run():
            for (w, sw), x, y in zip(layers, acts, acts[1:]):
                hq.hq_fp8_linear(x, w, sw, y, ws)
        run()
        want = [a.clone() for a in acts]
        torch.cuda.synchronize()
        g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(g):
            for _ in range(10):
                run()
        graphs.append((g, s))
        keep.append((ws, layers, acts, want))
    for _ in range(20):
        for g, s in graphs:
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for _, _, acts, want in keep:
        assert all(torch.equal(a, b) for a, b in zip(acts, want)) and want[-1].any()
