"""The e4m3 layers on the GPU against the fp64 oracle: quantisers bit for bit, products within the
rounding of their sums."""

import numpy as np
import pytest
import torch

import oracle
from gpu_helpers import to_np64

pytestmark = pytest.mark.gpu

FP8 = torch.float8_e4m3fn
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def hq():
    import post_weight_quantization_tcgen05_b200 as m
    return m


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def activations(seed, M, K, dtype):
    """Channels of uneven size, as activations have them."""
    g = gen(seed)
    s = torch.exp(torch.randn(K, generator=g, device="cuda"))
    return (torch.randn((M, K), generator=g, device="cuda") * s).to(TYPES[dtype])


def quantise_rows(hq, X):
    codes, scales = hq.fp8_rows_outputs(*X.shape)
    codes.view(torch.uint8).fill_(0xAA)
    hq.hq_fp8_quantize_rows(X, codes, scales)
    return codes, scales


def quantise_blocks(hq, W):
    codes, scales = hq.fp8_blocks_outputs(W.shape[-2], W.shape[-1], W.shape[0] if W.dim() == 3 else None)
    codes.view(torch.uint8).fill_(0xAA)
    hq.hq_fp8_quantize_blocks(W, codes, scales)
    return codes, scales


def values(codes, K):
    return oracle.e4m3_decode(codes.view(torch.uint8).cpu().numpy())[..., :K]


def tolerance(y, size, K, dtype):
    """What rounding can do to Y, from the sum `size` of its terms' magnitudes.  The products of two
    e4m3 values are exact; a tensor-core step adds 32 of them and the running sum, each cut at no less
    than 2^-23 of the largest: four steps a block, 4 * 33 * 2^-23 of the block's magnitudes.  Each
    block's sum is scaled by a product of scales (one rounding) and added in fp32 (one more), and
    the K / 128 blocks' sums are added up: ceil(K / 128) + 1 roundings of 2^-24.  The output rounds
    once more: half a step of its type."""
    own = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}[dtype]
    return size * (132 * 2.0 ** -23 + (-(-K // 128) + 1) * 2.0 ** -24) * (1 + own) + np.abs(y) * own


def check_product(Y, ref, size, K, what=""):
    err = np.abs(to_np64(Y) - ref)
    tol = tolerance(ref, size, K, Y.dtype)
    assert np.all(err <= tol), f"{what}: worst {np.max(err / np.maximum(tol, 1e-300)):.2f} of the tolerance"


# ------------------------------------------------------------------ quantisers

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,K", [(1, 1), (1, 16), (3, 127), (2, 128), (5, 129), (8, 512), (9, 520), (17, 1000), (64, 5120),
                                 (1, 17408), (33, 1537)])
def test_rows_match_the_oracle_bit_for_bit(hq, cuda_device, M, K, dtype):
    X = activations(M * 7 + K, M, K, dtype)
    codes, scales = quantise_rows(hq, X)
    c, s = oracle.fp8_quantize(to_np64(X), 1)
    assert np.array_equal(to_np64(scales), s.T)
    assert np.array_equal(values(codes, K), c)
    assert not codes.view(torch.uint8)[:, K:].any()  # the padding of a row is zeros


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("E,N,K", [(1, 1, 1), (1, 128, 128), (2, 130, 200), (3, 64, 1000), (1, 257, 129), (1, 384, 640)])
def test_blocks_match_the_oracle_bit_for_bit(hq, cuda_device, E, N, K, dtype):
    W = (torch.randn((E, N, K), generator=gen(E + N + K), device="cuda") * 0.02).to(TYPES[dtype])
    codes, scales = quantise_blocks(hq, W)
    for e in range(E):
        c, s = oracle.fp8_quantize(to_np64(W[e]), 128)
        assert np.array_equal(to_np64(scales[e]), s)
        assert np.array_equal(values(codes[e], K), c)
    assert not codes.view(torch.uint8)[..., K:].any()
    one, s_one = quantise_blocks(hq, W[E - 1])
    assert torch.equal(one.view(torch.uint8), codes[E - 1].view(torch.uint8)) and torch.equal(s_one, scales[E - 1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_of_any_alignment(hq, cuda_device, dtype):
    """A base that is not 16-byte aligned, with rows that are multiples of 16 bytes."""
    store = activations(3, 1, 6 * 256 + 1, dtype).reshape(-1)
    X = store[1:].view(6, 256)
    assert X.is_contiguous() and X.data_ptr() % 16 != 0
    for f in (quantise_rows, quantise_blocks):
        (c, s), (c2, s2) = f(hq, X), f(hq, X.clone())
        assert torch.equal(c.view(torch.uint8), c2.view(torch.uint8)) and torch.equal(s, s2)


def test_rows_of_special_values(hq, cuda_device):
    X = torch.zeros((8, 256), device="cuda")
    X[1, 3] = 2.0 ** -110           # below the smallest scale's range
    X[2, 5] = -3e38                 # near the largest fp32
    X[3] = -0.0
    X[4, 200] = float("nan")
    X[4, :128] = 1.0                # the NaN's row, another block
    X[5, 7] = float("inf")
    X[6, 1], X[6, 2] = 1.0, -448.0
    X[7, 0], X[7, 1] = 1e-44, -1e-44  # subnormal
    codes, scales = quantise_rows(hq, X)
    q = values(codes, 256) * np.repeat(to_np64(scales).T, 128, 1)
    c, s = oracle.fp8_quantize(to_np64(X), 1)
    for r in (0, 1, 2, 3, 6, 7):
        assert np.array_equal(to_np64(scales)[:, r], s[r]) and np.array_equal(values(codes, 256)[r], c[r]), r
    assert np.all(q[0] == 0) and np.all(q[3] == 0) and scales[0, 0] == 0
    # 1.0 comes back as 448 fp32(1 / 448): the quotient's one rounding, at most 2^-24 of it
    assert np.all(np.abs(q[4, :128] - 1.0) <= 2.0 ** -24) and np.all(np.isnan(q[4, 128:]))
    assert not np.any(np.isfinite(q[5, :128])) and np.all(q[5, 128:] == 0)


# ------------------------------------------------------------------ products

def small_integers(seed, rows, K, block_rows):
    """Codes of -2 .. 2 and scales that are powers of two: every sum below is exact in fp32."""
    g = gen(seed)
    codes = torch.zeros((rows, -(-K // 16) * 16), device="cuda")
    codes[:, :K] = torch.randint(-2, 3, (rows, K), generator=g, device="cuda").float()
    n = -(-rows // block_rows)
    scales = 2.0 ** torch.randint(-2, 2, (n, -(-K // 128)), generator=g, device="cuda").float()
    return codes.to(FP8), scales


SHAPES = [(1, 1, 1), (1, 128, 128), (2, 3, 17), (7, 130, 129), (128, 128, 128), (129, 257, 300), (100, 64, 1000),
          (300, 520, 136), (1, 5120, 640), (16, 1000, 1537), (257, 384, 2048), (64, 272, 5120)]


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product_of_small_integers_is_exact(hq, cuda_device, M, N, K, out):
    """|codes| <= 2, |scales| between 1/4 and 2: the terms are multiples of 2^-4 and at most 16 each,
    their sums below 2^17 for K <= 5120: 21 bits, exact in fp32; a bf16 output rounds once."""
    a, sa = small_integers(1, M, K, 1)
    w, sw = small_integers(2, N, K, 128)
    Y = torch.full((M, N), float("nan"), dtype=TYPES[out], device="cuda")
    hq.hq_fp8_gemm(a, sa.t().contiguous(), w, sw, K, Y)
    ref, _ = oracle.fp8_product(values(a, K), to_np64(sa), values(w, K), to_np64(sw))
    want = torch.from_numpy(ref).float().to(TYPES[out])
    assert torch.equal(Y.cpu(), want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_linear_and_gemm_against_the_oracle(hq, cuda_device, M, N, K, dtype):
    X = activations(M + N + K, M, K, dtype)
    W = (torch.randn((N, K), generator=gen(5), device="cuda") * 0.02).to(TYPES[dtype])
    w, sw = quantise_blocks(hq, W)
    a, sa = quantise_rows(hq, X)
    Y = torch.full((M, N), float("nan"), dtype=TYPES[dtype], device="cuda")
    ws = hq.alloc_workspace(hq.hq_fp8_linear_workspace_bytes(M, K))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    hq.hq_fp8_linear(X, w, sw, Y, ws, dev_status=status)
    ref, size = oracle.fp8_product(values(a, K), to_np64(sa).T, values(w, K), to_np64(sw))
    check_product(Y, ref, size, K, "linear")
    Y2 = torch.full_like(Y, float("nan"))
    hq.hq_fp8_gemm(a, sa, w, sw, K, Y2, dev_status=status)
    assert torch.equal(Y, Y2)
    assert status.item() == 0
    # bytes past column K are not part of the matrix
    junk, wjunk = a.view(torch.uint8).clone(), w.view(torch.uint8).clone()
    junk[:, K:], wjunk[:, K:] = 0x7F, 0x7F
    hq.hq_fp8_gemm(junk, sa, wjunk, sw, K, Y2)
    assert torch.equal(Y, Y2)


def test_many_tiles_and_both_types(hq, cuda_device):
    """More tiles than SMs, with rows and columns that fill no whole tile."""
    M, N, K = 2900, 3400, 400
    X, W = activations(1, M, K, "bf16"), activations(2, N, K, "bf16")
    a, sa = quantise_rows(hq, X)
    w, sw = quantise_blocks(hq, W)
    ref, size = oracle.fp8_product(values(a, K), to_np64(sa).T, values(w, K), to_np64(sw))
    for dt in ("bf16", "f32"):
        Y = torch.full((M, N), float("nan"), dtype=TYPES[dt], device="cuda")
        hq.hq_fp8_gemm(a, sa, w, sw, K, Y)
        check_product(Y, ref, size, K, dt)


def test_a_row_s_result_does_not_depend_on_the_others(hq, cuda_device):
    M, N, K = 200, 300, 700
    X = activations(4, M, K, "bf16")
    w, sw = quantise_blocks(hq, activations(5, N, K, "bf16"))
    Y, Z = (torch.empty((M, N), dtype=torch.float32, device="cuda") for _ in range(2))
    ws = hq.alloc_workspace(hq.hq_fp8_linear_workspace_bytes(M, K))
    hq.hq_fp8_linear(X, w, sw, Y, ws)
    X2 = X.clone()
    X2[3, 5], X2[150] = float("nan"), float("inf")
    hq.hq_fp8_linear(X2, w, sw, Z, ws)
    others = [r for r in range(M) if r not in (3, 150)]
    assert torch.equal(Y[others], Z[others])
    assert Z[3].isnan().all() and not Z[150].isfinite().any()
    # a NaN in a weight reaches the columns of its block of 128 only
    W2 = activations(5, N, K, "bf16")
    W2[130, 0] = float("nan")
    w2, sw2 = quantise_blocks(hq, W2)
    hq.hq_fp8_linear(X, w2, sw2, Z, ws)
    assert Z[:, 128:256].isnan().all() and torch.equal(Z[:, :128], Y[:, :128]) and torch.equal(Z[:, 256:], Y[:, 256:])


def test_unaligned_output(hq, cuda_device):
    M, N, K = 40, 256, 256
    X, W = activations(6, M, K, "bf16"), activations(7, N, K, "bf16")
    a, sa = quantise_rows(hq, X)
    w, sw = quantise_blocks(hq, W)
    for dt in ("bf16", "f32"):
        Y = torch.empty((M, N), dtype=TYPES[dt], device="cuda")
        hq.hq_fp8_gemm(a, sa, w, sw, K, Y)
        store = torch.full((M * N + 3,), -1.0, dtype=TYPES[dt], device="cuda")
        hq.hq_fp8_gemm(a, sa, w, sw, K, store[1:1 + M * N].view(M, N))
        assert torch.equal(store[1:1 + M * N].view(M, N), Y)
        assert store[0] == -1 and (store[1 + M * N:] == -1).all()


def expert_case(seed, sizes, gaps, N, K):
    """(offsets, rows): ranges of `sizes` rows; `gaps`: rows before the first and after the last."""
    g = np.cumsum([gaps[0], *sizes])
    return torch.tensor(g, dtype=torch.int32, device="cuda"), int(g[-1]) + gaps[1]


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("sizes,gaps,N,K", [([1], (0, 0), 64, 64), ([0, 5, 0, 0, 130, 1, 0], (0, 0), 130, 200),
                                            ([3, 0, 300], (2, 5), 257, 300), ([128, 128], (0, 3), 128, 128),
                                            ([0, 0, 0], (0, 7), 64, 64), ([11] * 20, (0, 1), 200, 1000),
                                            ([700, 2, 900], (1, 0), 384, 512)])
def test_expert_product_against_the_oracle(hq, cuda_device, sizes, gaps, N, K, out):
    E = len(sizes)
    offsets, rows = expert_case(0, sizes, gaps, N, K)
    X = activations(rows + N, rows, K, "bf16")
    W = (torch.randn((E, N, K), generator=gen(9), device="cuda") * 0.02).to(torch.bfloat16)
    a, sa = quantise_rows(hq, X)
    w, sw = quantise_blocks(hq, W)
    Y = torch.full((rows, N), 7.0, dtype=TYPES[out], device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    hq.hq_fp8_expert_gemm(a, sa, offsets, w, sw, K, Y, dev_status=status)
    off = offsets.tolist()
    ref, size = np.full((rows, N), 7.0), np.zeros((rows, N))
    oracle.fp8_expert_product(values(a, K), to_np64(sa).T, off, [values(w[e], K) for e in range(E)], to_np64(sw), ref, size)
    check_product(Y, ref, size, K)
    assert (Y[:off[0]] == 7).all() and (Y[off[-1]:] == 7).all()  # rows of no expert stay as they were
    assert status.item() == 0
    # each expert alone gives the same bits
    for e in range(E):
        if off[e] < off[e + 1]:
            part = slice(off[e], off[e + 1])
            Z = torch.empty((off[e + 1] - off[e], N), dtype=TYPES[out], device="cuda")
            hq.hq_fp8_gemm(a[part].contiguous(), sa[:, part].contiguous(), w[e], sw[e], K, Z)
            tol = torch.from_numpy(tolerance(ref[part], size[part], K, Y.dtype)).cuda()
            assert ((Z.double() - Y[part].double()).abs() <= 2 * tol).all()


def test_offsets_that_leave_the_rows_are_cut(hq, cuda_device):
    """Device data that a program got wrong: ranges are cut to the rows, inverted ones are empty."""
    N, K, rows = 128, 128, 40
    a, sa = quantise_rows(hq, activations(1, rows, K, "bf16"))
    w, sw = quantise_blocks(hq, activations(2, 3 * N, K, "bf16").view(3, N, K))
    Y = torch.full((rows, N), 7.0, device="cuda")
    hq.hq_fp8_expert_gemm(a, sa, torch.tensor([-5, 10, 4, 900], dtype=torch.int32, device="cuda"), w, sw, K, Y)
    # expert 0: rows 0..9, expert 1: none (10 > 4), expert 2: rows 4..39
    A = values(a, K) * to_np64(sa).T
    W = [values(w[e], K) * to_np64(sw[e]) for e in range(3)]
    assert np.allclose(to_np64(Y[:4]), (A @ W[0].T)[:4], rtol=1e-4, atol=1e-3)
    assert np.allclose(to_np64(Y[10:]), (A @ W[2].T)[10:], rtol=1e-4, atol=1e-3)
    Y.fill_(7.0)
    hq.hq_fp8_expert_gemm(a, sa, torch.tensor([50, 60, 70, 80], dtype=torch.int32, device="cuda"), w, sw, K, Y)
    assert (Y == 7).all()


def test_many_experts(hq, cuda_device):
    E, N, K = 1024, 32, 64
    sizes = torch.randint(0, 3, (E,), generator=gen(1), device="cuda").tolist()
    offsets, rows = expert_case(0, sizes, (0, 2), N, K)
    a, sa = small_integers(3, rows, K, 1)
    w, sw = small_integers(4, E * N, K, N)
    Y = torch.full((rows, N), 7.0, device="cuda")
    hq.hq_fp8_expert_gemm(a, sa.t().contiguous(), offsets, w.view(E, N, -1), sw.view(E, 1, 1), K, Y)
    off = offsets.tolist()
    A, W = values(a, K) * to_np64(sa), values(w, K).reshape(E, N, K) * to_np64(sw).reshape(E, 1, 1)
    ref = np.full((rows, N), 7.0)
    for e in range(E):
        ref[off[e]:off[e + 1]] = A[off[e]:off[e + 1]] @ W[e].T
    assert np.array_equal(to_np64(Y), ref)


# ------------------------------------------------------------------ streams, graphs

@pytest.mark.parametrize("M,N,K", [(1, 640, 1024), (300, 640, 1024)])
def test_linear_on_a_side_stream_and_in_a_graph(hq, cuda_device, M, N, K):
    X = activations(1, M, K, "bf16")
    w, sw = quantise_blocks(hq, activations(2, N, K, "bf16"))
    ws = hq.alloc_workspace(hq.hq_fp8_linear_workspace_bytes(M, K))
    Y = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    hq.hq_fp8_linear(X, w, sw, Y, ws)
    want = Y.clone()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    Y.fill_(0)
    s.wait_stream(torch.cuda.current_stream())
    hq.hq_fp8_linear(X, w, sw, Y, ws, stream=s)
    s.synchronize()
    assert torch.equal(Y, want)
    X2 = activations(3, M, K, "bf16")
    want2 = torch.empty_like(Y)
    hq.hq_fp8_linear(X2, w, sw, want2, ws)
    graph, x = torch.cuda.CUDAGraph(), X.clone()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        hq.hq_fp8_linear(x, w, sw, Y, ws)
    for src, ref in ((X2, want2), (X, want), (X2, want2)):
        x.copy_(src)
        graph.replay()
        assert torch.equal(Y, ref)


@pytest.mark.parametrize("M,N,K", [(294, 256, 6043), (130, 100, 2000), (700, 300, 4096), (40, 4000, 700), (512, 1024, 640)])
def test_few_tiles_of_many_rows(hq, cuda_device, M, N, K):
    """More rows than a serving step but few tiles: K is split, and the layer is the product of the
    quantised rows bit for bit."""
    X, W = activations(1, M, K, "bf16"), activations(2, N, K, "bf16") * 0.02
    w, sw = quantise_blocks(hq, W)
    a, sa = quantise_rows(hq, X)
    Y, Z = (torch.full((M, N), float("nan"), device="cuda") for _ in range(2))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    hq.hq_fp8_gemm(a, sa, w, sw, K, Y, dev_status=status)
    hq.hq_fp8_linear(X, w, sw, Z, hq.alloc_workspace(hq.hq_fp8_linear_workspace_bytes(M, K)), dev_status=status)
    assert torch.equal(Y, Z) and status.item() == 0
    ref, size = oracle.fp8_product(*oracle.fp8_quantize(to_np64(X), 1), *oracle.fp8_quantize(to_np64(W), 128))
    check_product(Y, ref, size, K)


def test_linears_of_different_kernels_at_once(hq, cuda_device):
    """Layers of one token, 24, 64, 300 and 2000 rows on streams of their own, over and over: kernels that
    share the SMs' tensor memory, with clusters and without, give what each gives alone."""
    N, K = 2048, 1536
    w, sw = quantise_blocks(hq, activations(2, N, K, "bf16"))
    sets = []
    for M in (1, 24, 64, 300, 2000, 1):
        X = activations(M, M, K, "bf16")
        ws = hq.alloc_workspace(hq.hq_fp8_linear_workspace_bytes(M, K))
        Y = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
        hq.hq_fp8_linear(X, w, sw, Y, ws)
        sets.append((X, ws, Y.clone(), Y.fill_(0), torch.cuda.Stream()))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    for _ in range(30):
        for X, ws, _, Y, s in sets:
            hq.hq_fp8_linear(X, w, sw, Y, ws, dev_status=status, stream=s)
    torch.cuda.synchronize()
    assert status.item() == 0
    for X, _, want, Y, _ in sets:
        assert torch.equal(Y, want), X.shape


# ------------------------------------------------------------------ the kernels one by one

IMPLS = {"single": 1, "pair": 2, "few16": 3, "few64": 4}


@pytest.mark.parametrize("impl", list(IMPLS))
@pytest.mark.parametrize("M,N,K", SHAPES + [(2900, 3400, 400), (512, 17408, 256), (16, 5120, 5120), (5, 17408, 640), (64, 4000, 1536),
                                             (300, 8, 200), (4000, 4096, 100), (3000, 5000, 129)])
def test_every_kernel_on_one_weight(hq, cuda_device, M, N, K, impl):
    a, sa = small_integers(1, M, K, 1)
    w, sw = small_integers(2, N, K, 128)
    sa = sa.t().contiguous()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ref = ((a[:, :K].double() * sa.double().t().repeat_interleave(128, 1)[:, :K])
           @ (w[:, :K].double() * sw.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]).t())
    for dt in ("f32", "bf16"):
        Y = torch.full((M, N), float("nan"), dtype=TYPES[dt], device="cuda")
        hq.hq_debug_fp8_gemm_impl(a, sa, None, w, sw, K, Y, IMPLS[impl], dev_status=status)
        assert torch.equal(Y, ref.float().to(TYPES[dt]))
    assert status.item() == 0


@pytest.mark.parametrize("impl", list(IMPLS))
@pytest.mark.parametrize("sizes,gaps,N,K", [([1], (0, 0), 64, 64), ([0, 5, 0, 0, 130, 1, 0], (0, 0), 130, 200),
                                            ([3, 0, 300], (2, 5), 257, 300), ([0, 0, 0], (0, 7), 64, 64),
                                            ([700, 2, 900], (1, 0), 384, 512), ([257, 0, 1, 255, 256] * 8, (0, 9), 640, 260),
                                            ([130, 3, 0, 40] * 40, (0, 0), 900, 128)])
def test_every_kernel_on_experts(hq, cuda_device, sizes, gaps, N, K, impl):
    E = len(sizes)
    offsets, rows = expert_case(0, sizes, gaps, N, K)
    a, sa = small_integers(3, rows, K, 1)
    w, sw = small_integers(4, E * N, K, N)  # one row of scales for each expert's N rows
    sw = sw[:, None].expand(E, -(-N // 128), -1).contiguous()
    Y = torch.full((rows, N), 7.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    hq.hq_debug_fp8_gemm_impl(a, sa.t().contiguous(), offsets, w.view(E, N, -1), sw, K, Y, IMPLS[impl], dev_status=status)
    A = a[:, :K].double() * sa.double().repeat_interleave(128, 1)[:, :K]
    ref = torch.full((rows, N), 7.0, dtype=torch.float64, device="cuda")
    off = offsets.tolist()
    for e in range(E):
        W = w.view(E, N, -1)[e, :, :K].double() * sw[e, 0].double().repeat_interleave(128)[:K]
        ref[off[e]:off[e + 1]] = A[off[e]:off[e + 1]] @ W.t()
    assert torch.equal(Y.double(), ref)
    assert status.item() == 0


@pytest.mark.parametrize("impl", list(IMPLS))
def test_offsets_whose_ranges_overlap_stay_inside_y(hq, cuda_device, impl):
    """Device data that a program got wrong: four of the eight experts name all rows.  Every entry of Y is
    what it was or one of those experts' results, and nothing beside Y is written."""
    E, rows, N, K = 8, 1500, 132, 128
    a, sa = small_integers(1, rows, K, 1)
    w, sw = small_integers(2, E * N, K, N)
    sw = sw[:, None].expand(E, 2, -1).contiguous()
    offsets = torch.tensor([0, rows] * 4 + [0], dtype=torch.int32, device="cuda")
    around = torch.full((rows + 600, N), 0.5, device="cuda")
    Y = around[300:300 + rows]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    hq.hq_debug_fp8_gemm_impl(a, sa.t().contiguous(), offsets, w.view(E, N, -1), sw, K, Y, IMPLS[impl], dev_status=status)
    A = a[:, :K].double() * sa.double()
    known = Y == 0.5
    for e in range(0, E, 2):
        known |= Y.double() == A @ (w.view(E, N, -1)[e, :, :K].double() * sw[e, 0, 0].double()).t()
    assert known.all() and (around[:300] == 0.5).all() and (around[300 + rows:] == 0.5).all()
    assert status.item() == 0


# ------------------------------------------------------------------ offsets past 32 bits

def test_more_than_2_to_the_31_elements(hq, cuda_device):
    """X, its codes and Y each have more than 2^31 elements: the last rows are what a call of their own
    makes of them."""
    M, N, K = 265_000, 8200, 8192
    assert M * K > 2 ** 31 and M * N > 2 ** 31
    few = activations(1, 300, K, "bf16")
    X = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    X[-300:] = few
    a, sa = quantise_rows(hq, X)
    del X
    b, sb = quantise_rows(hq, few)
    assert torch.equal(a.view(torch.uint8)[-300:], b.view(torch.uint8)) and torch.equal(sa[:, -300:], sb)
    assert not sa[:, :-300].any()
    w, sw = quantise_blocks(hq, activations(2, N, K, "bf16"))
    Y = torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda")
    hq.hq_fp8_gemm(a, sa, w, sw, K, Y)
    Z = torch.empty((300, N), dtype=torch.bfloat16, device="cuda")
    # the same kernel as for the long call, so that the same sums are taken
    hq.hq_debug_fp8_gemm_impl(b, sb, None, w, sw, K, Z, IMPLS["pair"])
    assert torch.equal(Y[-300:], Z)
    assert not Y[:-300].any()


def test_a_first_call_under_capture(cuda_device):
    """A process whose first call of the kernels is captured into a graph."""
    import os
    import subprocess
    import sys
    code = """
import torch, post_weight_quantization_tcgen05_b200 as hq
torch.cuda.init()
X = torch.ones((300, 256), device="cuda"); w, sw = hq.fp8_blocks_outputs(384, 256); Y = torch.zeros((300, 384), device="cuda")
W = torch.ones((384, 256), device="cuda"); ws = hq.alloc_workspace(hq.hq_fp8_linear_workspace_bytes(300, 256))
x = torch.ones((1, 256), device="cuda"); y = torch.zeros((1, 384), device="cuda")
torch.cuda.synchronize(); g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    hq.hq_fp8_quantize_blocks(W, w, sw)
    hq.hq_fp8_linear(X, w, sw, Y, ws)
    hq.hq_fp8_linear(x, w, sw, y, ws)
g.replay(); torch.cuda.synchronize()
# 1.0 is quantised to 448 with the scale fp32(1 / 448)
assert (Y - 256).abs().max() < 256 * 2 ** -20 and (y - 256).abs().max() < 256 * 2 ** -20, (Y.max(), y.max())
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr


def test_a_first_call_of_the_pairs_under_capture(cuda_device):
    """The same for rows enough that pairs of CTAs run."""
    import os
    import subprocess
    import sys
    code = """
import torch, post_weight_quantization_tcgen05_b200 as hq
torch.cuda.init()
X = torch.ones((4000, 256), device="cuda"); W = torch.ones((4096, 256), device="cuda"); Y = torch.zeros((4000, 4096), device="cuda")
w, sw = hq.fp8_blocks_outputs(4096, 256); ws = hq.alloc_workspace(hq.hq_fp8_linear_workspace_bytes(4000, 256))
torch.cuda.synchronize(); g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    hq.hq_fp8_quantize_blocks(W, w, sw)
    hq.hq_fp8_linear(X, w, sw, Y, ws)
g.replay(); torch.cuda.synchronize()
assert (Y - 256).abs().max() < 256 * 2 ** -20, Y.max()
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr


def test_linear_is_the_gemm_of_the_quantised_rows_in_any_order_of_first_calls(cuda_device):
    """How K is split must not depend on which of the two a process calls first."""
    import os
    import subprocess
    import sys
    code = """
import torch, post_weight_quantization_tcgen05_b200 as hq
for M, N, K in ((1, 200, 300), (2, 200, 300), (1, 5120, 640), (4, 1000, 1000), (1, 640, 5120), (16, 640, 2000)):
    g = torch.Generator(device="cuda"); g.manual_seed(M + N)
    X = torch.randn((M, K), device="cuda", generator=g); W = torch.randn((N, K), device="cuda", generator=g)
    w, sw = hq.fp8_blocks_outputs(N, K); hq.hq_fp8_quantize_blocks(W, w, sw)
    Y, Z = torch.empty((M, N), device="cuda"), torch.empty((M, N), device="cuda")
    hq.hq_fp8_linear(X, w, sw, Y, hq.alloc_workspace(hq.hq_fp8_linear_workspace_bytes(M, K)))
    a, sa = hq.fp8_rows_outputs(M, K); hq.hq_fp8_quantize_rows(X, a, sa)
    hq.hq_fp8_gemm(a, sa, w, sw, K, Z)
    assert torch.equal(Y, Z), (M, N, K)
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
