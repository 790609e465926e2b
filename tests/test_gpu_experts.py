"""Tokens by expert and back on the GPU against the fp64 oracle: the sort exactly, the copies bit for
bit, sums and gradients within their roundings; then calibration and the quantised layer through them."""

import numpy as np
import pytest
import torch

import oracle
from gpu_helpers import H_REL_FRO, rel_fro, to_np64

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


@pytest.fixture(scope="module")
def hq():
    import post_weight_quantization_tcgen05_b200 as m
    return m


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def choices(seed, T, top, E, drop=0.1):
    """Uneven choices, some dropped, by ids below and above the range; a token may repeat an expert."""
    g = gen(seed)
    ids = (torch.rand((T, top), generator=g, device="cuda") ** 2 * E).to(torch.int32)
    away = torch.rand((T, top), generator=g, device="cuda") < drop
    wrong = torch.tensor([-1, E, -2 ** 31, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    pick = torch.randint(0, 4, (T, top), generator=g, device="cuda")
    return torch.where(away, wrong[pick], ids)


def sort(hq, ids, E):
    T, top = ids.shape
    offsets, order, position = (t.fill_(-77) for t in hq.expert_sort_outputs(T, top, E))
    ws = hq.alloc_workspace(hq.hq_expert_sort_workspace_bytes(T, top, E))
    hq.hq_expert_sort(ids, E, offsets, order, position, ws)
    return offsets, order, position


def check_sort(ids, E, offsets, order, position):
    flat = ids.cpu().numpy().reshape(-1).astype(np.int64)
    key = np.where((flat >= 0) & (flat < E), flat, E)
    ref = np.argsort(key, kind="stable")
    ends = np.searchsorted(key[ref], np.arange(E + 1))
    n = ends[-1]
    assert np.array_equal(offsets.cpu().numpy(), ends)
    assert np.array_equal(order.cpu().numpy()[:n], ref[:n])
    assert (order[n:] == -77).all()  # rows behind the last are left as they were
    place = np.full(flat.size, -1, np.int64)
    place[ref[:n]] = np.arange(n)
    assert np.array_equal(position.cpu().numpy().reshape(-1), place)


# ------------------------------------------------------------------ sort

@pytest.mark.parametrize("T,top,E,drop", [(1, 1, 1, 0.0), (1, 1, 1, 1.0), (1, 8, 4, 0.2), (7, 3, 5, 0.1), (64, 8, 48, 0.02),
                                          (100, 1, 1024, 0.1), (1023, 8, 256, 0.1), (1024, 8, 64, 0.0), (1025, 8, 64, 0.5),
                                          (5000, 6, 1024, 0.1), (40000, 8, 160, 0.05), (300, 2, 513, 1.0),
                                          (8193, 1, 2, 0.0), (70000, 7, 1, 0.3)])
def test_sort(hq, cuda_device, T, top, E, drop):
    ids = choices(T + E, T, top, E, drop)
    out = sort(hq, ids, E)
    check_sort(ids, E, *out)
    if T * top <= 512:
        off, order, position = oracle.expert_sort(ids.cpu().numpy(), E)
        assert np.array_equal(out[0].cpu().numpy(), off) and np.array_equal(out[2].cpu().numpy(), position)
        assert np.array_equal(out[1].cpu().numpy()[:len(order)], order)
    again = sort(hq, ids, E)
    assert all(torch.equal(a, b) for a, b in zip(out, again))


def test_sort_without_tokens(hq, cuda_device):
    offsets, _, _ = sort(hq, torch.empty((0, 4), dtype=torch.int32, device="cuda"), 9)
    assert offsets.tolist() == [0] * 10


def test_sorts_of_two_streams_and_a_graph(hq, cuda_device):
    """Two calls at once, each with its own workspace, and a captured one replayed on new ids."""
    T, top, E = 20000, 4, 100
    sets = [choices(s, T, top, E) for s in (1, 2)]
    outs = [[t.fill_(-77) for t in hq.expert_sort_outputs(T, top, E)] for _ in sets]
    work = [hq.alloc_workspace(hq.hq_expert_sort_workspace_bytes(T, top, E)) for _ in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(3):
        for ids, out, ws, s in zip(sets, outs, work, streams):
            hq.hq_expert_sort(ids, E, *out, ws, stream=s)
    torch.cuda.synchronize()
    for ids, out in zip(sets, outs):
        check_sort(ids, E, *out)
    ids, graph = sets[0].clone(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hq.hq_expert_sort(ids, E, *outs[0], work[0])
    ids.copy_(sets[1])
    outs[0][1].fill_(-77)
    graph.replay()
    check_sort(sets[1], E, *outs[0])


# ------------------------------------------------------------------ rows

ROWS = [(1, 1, 1, 1), (1, 8, 4, 5), (5, 3, 2, 8), (7, 2, 3, 131), (64, 8, 48, 640), (33, 4, 9, 1000), (300, 1, 7, 264),
        (20, 11, 6, 2056), (3, 8, 8, 5120), (40, 17, 5, 33)]


def a_case(hq, T, top, E, K, dtype, seed=0):
    ids = choices(seed + T + K, T, top, E, 0.15)
    offsets, order, position = sort(hq, ids, E)
    X = torch.randn((T, K), generator=gen(seed + 1), device="cuda").to(TYPES[dtype])
    w = torch.rand((T, top), generator=gen(seed + 2), device="cuda") - 0.3
    return offsets, order, position, X, w


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,top,E,K", ROWS)
def test_dispatch(hq, cuda_device, T, top, E, K, dtype):
    offsets, order, position, X, _ = a_case(hq, T, top, E, K, dtype)
    n = int(offsets[-1])
    rows = torch.full((T * top, K), 7.0, dtype=X.dtype, device="cuda")
    hq.hq_expert_dispatch(X, position, rows)
    assert torch.equal(rows[:n], X[order[:n].long() // top])
    assert (rows[n:] == 7).all()
    # quantised on the way: what quantising the rows gives, and nothing behind the last
    codes, scales = hq.fp8_rows_outputs(T * top, K)
    codes.view(torch.uint8).fill_(0xAA)
    scales.fill_(-1)
    hq.hq_expert_dispatch_fp8(X, position, codes, scales)
    ref, ref_s = hq.fp8_rows_outputs(T * top, K)
    hq.hq_fp8_quantize_rows(rows, ref, ref_s)
    assert torch.equal(codes.view(torch.uint8)[:n], ref.view(torch.uint8)[:n])
    assert torch.equal(scales[:, :n], ref_s[:, :n])
    assert (codes.view(torch.uint8)[n:] == 0xAA).all() and (scales[:, n:] == -1).all()


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,top,E,K", ROWS)
def test_combine(hq, cuda_device, T, top, E, K, dtype, weighted):
    offsets, _, position, _, w = a_case(hq, T, top, E, K, dtype)
    rows = torch.randn((T * top, K), generator=gen(5), device="cuda").to(TYPES[dtype])
    rows[int(offsets[-1]):] = float("nan")         # what no choice names is not read
    w = torch.where(position < 0, float("nan"), w)  # nor is the weight of a dropped choice
    Y = torch.full((T, K), float("nan"), dtype=TYPES[dtype], device="cuda")
    hq.hq_expert_combine(rows, position, w if weighted else None, Y)
    pos, r, wn = position.cpu().numpy(), to_np64(rows), to_np64(w)
    ref = oracle.expert_combine(r, pos, wn if weighted else None)
    size = oracle.expert_combine(np.abs(r), pos, np.abs(wn) if weighted else None)
    # top fused multiply-adds in fp32, then the rounding to the output's type
    tol = size * top * 2.0 ** -24 + (np.abs(ref) + size * top * 2.0 ** -24) * HALF_STEP[dtype]
    assert np.all(np.abs(to_np64(Y) - ref) <= tol)
    empty = (position < 0).all(1)
    assert (Y[empty] == 0).all()  # a token whose choices are all dropped


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,top,E,K", ROWS)
def test_combine_backward(hq, cuda_device, T, top, E, K, dtype):
    offsets, _, position, dY, w = a_case(hq, T, top, E, K, dtype)
    n = int(offsets[-1])
    rows = torch.randn((T * top, K), generator=gen(5), device="cuda").to(TYPES[dtype])
    rows[n:] = float("nan")
    w = torch.where(position < 0, float("nan"), w)
    d_rows = torch.full_like(rows, 7.0)
    d_w = torch.full_like(w, 7.0)
    hq.hq_expert_combine_backward(dY, rows, position, w, d_rows, d_w)
    pos, r, wn, g = position.cpu().numpy(), to_np64(rows), to_np64(w), to_np64(dY)
    ref_r, ref_w = oracle.expert_combine_backward(g, r, pos, wn, np.full(r.shape, 7.0))
    _, size = oracle.expert_combine_backward(np.abs(g), np.abs(r), pos, wn, np.full(r.shape, 7.0))
    # one product in fp32 and one rounding to the rows' type
    assert np.all(np.abs(to_np64(d_rows) - ref_r) <= np.abs(ref_r) * (2.0 ** -24 + HALF_STEP[dtype]) * (1 + 2.0 ** -8))
    assert (d_rows[n:] == 7).all()
    # at most K additions in fp32, in any order
    assert np.all(np.abs(to_np64(d_w) - ref_w) <= size * K * 2.0 ** -24 + 1e-300)
    assert (d_w[position < 0] == 0).all()
    # the dispatch's gradient is the unweighted sum of a token's rows
    dX = torch.empty_like(dY)
    hq.hq_expert_combine(d_rows, position, None, dX)
    dr = to_np64(d_rows)
    ref = oracle.expert_combine(dr, pos, None)
    size = oracle.expert_combine(np.abs(dr), pos, None)
    assert np.all(np.abs(to_np64(dX) - ref) <= size * top * 2.0 ** -23 + np.abs(ref) * HALF_STEP[dtype] * (1 + 2.0 ** -8))


def test_gradients_against_differences(hq, cuda_device):
    """<dY, combine(rows, w)> is linear in rows and in w: a step of a power of two along a random
    direction changes it by that step times the gradient's product, but for fp32 rounding."""
    T, top, E, K = 24, 4, 5, 96
    _, _, position, dY, w = a_case(hq, T, top, E, K, "f32", seed=3)
    rows = torch.randn((T * top, K), generator=gen(8), device="cuda")
    d_rows, d_w = torch.zeros_like(rows), torch.zeros_like(w)
    hq.hq_expert_combine_backward(dY, rows, position, w, d_rows, d_w)

    def loss(r, v):
        Y = torch.empty((T, K), device="cuda")
        hq.hq_expert_combine(r.contiguous(), position, v.contiguous(), Y)
        return float((dY.double() * Y.double()).sum())

    step = 2.0 ** -3
    for x, dx, f in ((rows, d_rows, lambda r: loss(r, w)), (w, d_w, lambda v: loss(rows, v))):
        u = torch.randn(x.shape, generator=gen(9), device="cuda")
        diff = (f(x + step * u) - f(x - step * u)) / (2 * step)
        want = float((u.double() * dx.double()).sum())
        # each of the T K outputs carries top + 1 roundings of 2^-24 of about 2 in size, twice, over 2 steps
        bound = float(dY.abs().sum()) * 4 * (top + 1) * 2.0 ** -24 / step * 4
        assert abs(diff - want) <= bound, (diff, want, bound)


@pytest.mark.parametrize("offset", [1, 2])
def test_rows_that_are_not_16_byte_aligned(hq, cuda_device, offset):
    T, top, E, K = 9, 3, 4, 256
    offsets, order, position, X, w = a_case(hq, T, top, E, K, "bf16")
    n = int(offsets[-1])
    away = lambda t: torch.cat([t.reshape(-1)[:offset], t.reshape(-1)])[offset:].view(t.shape)  # noqa: E731
    Xu = away(X)
    assert Xu.data_ptr() % 16 != 0
    rows, rows_u = (torch.zeros((T * top, K), dtype=X.dtype, device="cuda") for _ in range(2))
    hq.hq_expert_dispatch(X, position, rows)
    hq.hq_expert_dispatch(Xu, position, rows_u)
    assert torch.equal(rows, rows_u)
    (c, s), (cu, su) = hq.fp8_rows_outputs(T * top, K), hq.fp8_rows_outputs(T * top, K)
    hq.hq_expert_dispatch_fp8(X, position, c, s)
    hq.hq_expert_dispatch_fp8(Xu, position, cu, su)
    assert torch.equal(c.view(torch.uint8)[:n], cu.view(torch.uint8)[:n]) and torch.equal(s[:, :n], su[:, :n])
    Y, Yu = torch.empty_like(X), torch.empty_like(X)
    hq.hq_expert_combine(rows, position, w, Y)
    hq.hq_expert_combine(away(rows), position, w, Yu)
    assert torch.equal(Y, Yu)
    out = [(torch.zeros_like(rows), torch.zeros_like(w)) for _ in range(2)]
    hq.hq_expert_combine_backward(X, rows, position, w, *out[0])
    hq.hq_expert_combine_backward(Xu, rows, position, w, *out[1])
    assert torch.equal(out[0][0], out[1][0])
    assert (out[0][1] - out[1][1]).abs().max() <= K * 2.0 ** -23 * 16 * K  # sums of K terms in another order


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("K", [2, 31, 32, 33, 127, 129, 255, 257, 1023, 1025, 2050])
def test_rows_of_odd_widths(hq, cuda_device, K, dtype):
    """Widths around what a warp takes of a row that is not made of 16-byte vectors, more choices than are
    handled at once."""
    test_dispatch(hq, cuda_device, 19, 9, 4, K, dtype)
    test_combine(hq, cuda_device, 19, 9, 4, K, dtype, True)
    test_combine_backward(hq, cuda_device, 19, 9, 4, K, dtype)


def test_positions_out_of_range_count_as_dropped(hq, cuda_device):
    """Device data that a program got wrong is not followed out of the rows."""
    T, top, K = 4, 2, 64
    position = torch.tensor([[0, 8], [2, -9], [2 ** 31 - 1, 5], [-2 ** 31, 7]], dtype=torch.int32, device="cuda")
    good = torch.where((position >= 0) & (position < T * top), position, -1)
    X = torch.randn((T, K), generator=gen(1), device="cuda")
    w = torch.rand((T, top), generator=gen(2), device="cuda")
    rows = [torch.full((T * top, K), 7.0, device="cuda") for _ in range(2)]
    fp8 = [hq.fp8_rows_outputs(T * top, K) for _ in range(2)]
    Y, d = [torch.empty_like(X) for _ in range(2)], [(torch.full_like(rows[0], 7.0), torch.empty_like(w)) for _ in range(2)]
    for k, p in enumerate((position, good)):
        hq.hq_expert_dispatch(X, p, rows[k])
        fp8[k][0].view(torch.uint8).fill_(1)
        fp8[k][1].fill_(1)
        hq.hq_expert_dispatch_fp8(X, p, *fp8[k])
        hq.hq_expert_combine(rows[k], p, w, Y[k])
        hq.hq_expert_combine_backward(X, rows[k], p, w, *d[k])
    assert torch.equal(rows[0], rows[1]) and torch.equal(Y[0], Y[1])
    assert torch.equal(fp8[0][0].view(torch.uint8), fp8[1][0].view(torch.uint8)) and torch.equal(fp8[0][1], fp8[1][1])
    assert torch.equal(d[0][0], d[1][0]) and torch.equal(d[0][1], d[1][1])


def test_rows_past_2_to_the_31_elements(hq, cuda_device):
    T, top, E, K = 70_000, 4, 5, 8192
    assert T * top * K > 2 ** 31
    ids = choices(3, T, top, E)
    offsets, order, position = sort(hq, ids, E)
    n = int(offsets[-1])
    X = torch.randn((T, K), generator=gen(1), device="cuda").to(torch.bfloat16)
    w = torch.rand((T, top), generator=gen(2), device="cuda")
    rows = torch.empty((T * top, K), dtype=X.dtype, device="cuda")
    hq.hq_expert_dispatch(X, position, rows)
    some = torch.cat([torch.arange(0, 50), torch.arange(n - 50, n)]).cuda()
    assert torch.equal(rows[some], X[order[some].long() // top])
    Y, dX = torch.empty_like(X), torch.empty_like(X)
    hq.hq_expert_combine(rows, position, None, Y)  # a power of two of a bf16 value where all choices are kept
    kept = (position >= 0).sum(1)
    assert torch.equal(Y[kept == 4], (X[kept == 4].float() * 4).to(X.dtype))
    assert torch.equal(Y[kept == 0], torch.zeros_like(X[kept == 0]))
    d_rows, d_w = torch.empty_like(rows), torch.empty_like(w)
    hq.hq_expert_combine_backward(X, rows, position, w, d_rows, d_w)
    t = order[some].long() // top
    assert torch.equal(d_rows[some], (X[t].float() * w.reshape(-1)[order[some].long()][:, None]).to(X.dtype))
    sq = (X[t].double() ** 2).sum(1)
    assert ((d_w.reshape(-1)[order[some].long()] - sq).abs() <= sq * K * 2.0 ** -24).all()
    del d_rows, dX, Y
    codes, scales = hq.fp8_rows_outputs(T * top, K)
    hq.hq_expert_dispatch_fp8(X, position, codes, scales)
    ref, ref_s = hq.fp8_rows_outputs(100, K)
    hq.hq_fp8_quantize_rows(rows[some].contiguous(), ref, ref_s)
    assert torch.equal(codes.view(torch.uint8)[some], ref.view(torch.uint8)) and torch.equal(scales[:, some], ref_s)


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("K", [256, 100])
def test_hessians_of_experts(hq, cuda_device, K):
    from post_weight_quantization_tcgen05_b200 import experts
    T, top, E = 900, 3, 6
    ids = choices(4, T, top, E)
    ids[ids == 3] = 0  # an expert without tokens
    X = torch.randn((T, K), generator=gen(2), device="cuda").to(torch.bfloat16)
    H = torch.zeros((E, K, K), device="cuda")
    half = T // 2
    counts = [experts.expert_hessians(hq, X[s].contiguous(), ids[s].contiguous(), H) for s in (slice(0, half), slice(half, T))]
    low = np.tril(np.ones((K, K), bool))
    for e in range(E):
        named = (ids == e).sum(1).cpu().numpy()
        assert counts[0][e] + counts[1][e] == named.sum()
        ref = oracle.hessian(np.repeat(to_np64(X), named, 0)) if named.any() else np.zeros((K, K))
        if named.any():
            assert rel_fro(to_np64(H[e])[low], ref[low]) < H_REL_FRO
        else:
            assert not H[e].any()


@pytest.mark.parametrize("T,top,E,K,N,dtype", [(1, 2, 4, 256, 384, "bf16"), (37, 4, 6, 300, 200, "bf16"),
                                               (37, 4, 6, 300, 200, "f32"), (500, 8, 16, 640, 512, "bf16")])
def test_expert_layer(hq, cuda_device, T, top, E, K, N, dtype):
    from post_weight_quantization_tcgen05_b200 import experts
    ids = choices(T, T, top, E)
    X = torch.randn((T, K), generator=gen(2), device="cuda").to(TYPES[dtype])
    W = (torch.randn((E, N, K), generator=gen(3), device="cuda") * 0.05).to(TYPES[dtype])
    w = torch.rand((T, top), generator=gen(4), device="cuda")
    wc, ws = hq.fp8_blocks_outputs(N, K, E)
    hq.hq_fp8_quantize_blocks(W, wc, ws)
    Y = torch.full((T, N), float("nan"), dtype=TYPES[dtype], device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    experts.expert_linear(hq, X, ids, w, wc, ws, Y, dev_status=status)
    assert status.item() == 0
    a, sa = oracle.fp8_quantize(to_np64(X), 1)
    ref, size, i, wn = np.zeros((T, N)), np.zeros((T, N)), ids.cpu().numpy(), to_np64(w)
    for e in range(E):
        c, s = oracle.fp8_quantize(to_np64(W[e]), 128)
        y, m = oracle.fp8_product(a, sa, c, s)
        each = np.where(i == e, wn, 0.0).sum(1)[:, None]
        ref += each * y
        size += each * m
    # the product's roundings, its output's, the top products of the sum and the last rounding
    blocks = -(-K // 128)
    tol = size * (132 * 2.0 ** -23 + (blocks + 1 + top + 1) * 2.0 ** -24 + HALF_STEP[dtype] * 1.01) + np.abs(ref) * HALF_STEP[dtype]
    assert np.all(np.abs(to_np64(Y) - ref) <= tol)


class Layer:
    """Buffers of an expert layer, forward and backward, in one place: what a graph holds on to."""

    def __init__(self, hq, T, top, E, K, N):
        self.hq, self.E, self.K = hq, E, K
        bf16 = dict(dtype=torch.bfloat16, device="cuda")
        self.X, self.dY = torch.zeros((T, K), **bf16), torch.zeros((T, N), **bf16)
        self.ids = torch.full((T, top), -1, dtype=torch.int32, device="cuda")
        self.w = torch.zeros((T, top), device="cuda")
        self.sorted = hq.expert_sort_outputs(T, top, E)
        self.ws = hq.alloc_workspace(hq.hq_expert_sort_workspace_bytes(T, top, E))
        self.codes, self.scales = hq.fp8_rows_outputs(T * top, K)
        # zeros, as rows that no choice names are left alone
        self.rows, self.d_rows = torch.zeros((T * top, N), **bf16), torch.zeros((T * top, N), **bf16)
        self.Y, self.dw = torch.empty((T, N), **bf16), torch.empty((T, top), device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def fill(self, seed, drop):
        T, top = self.ids.shape
        self.X.copy_(torch.randn(self.X.shape, generator=gen(seed), device="cuda"))
        self.dY.copy_(torch.randn(self.dY.shape, generator=gen(seed + 1), device="cuda"))
        self.w.copy_(torch.rand((T, top), generator=gen(seed + 2), device="cuda"))
        self.ids.copy_(choices(seed, T, top, self.E, drop))

    def run(self, wc, ws, stream=None):
        hq, (offsets, order, position) = self.hq, self.sorted
        hq.hq_expert_sort(self.ids, self.E, offsets, order, position, self.ws, stream=stream)
        hq.hq_expert_dispatch_fp8(self.X, position, self.codes, self.scales, stream=stream)
        hq.hq_fp8_expert_gemm(self.codes, self.scales, offsets, wc, ws, self.K, self.rows, self.status, stream=stream)
        hq.hq_expert_combine(self.rows, position, self.w, self.Y, stream=stream)
        hq.hq_expert_combine_backward(self.dY, self.rows, position, self.w, self.d_rows, self.dw, stream=stream)

    def results(self):
        """Y, the weights' gradient, and each choice's row of the rows' gradient (zero if dropped)."""
        position = self.sorted[2].long()
        d = self.d_rows[position.clamp(min=0)] * (position >= 0)[..., None]
        return self.Y.clone(), self.dw.clone(), d


@pytest.mark.parametrize("T,top,E,K,N", [(5, 2, 7, 272, 200), (300, 8, 12, 640, 384), (4000, 4, 9, 384, 512)])
def test_expert_layer_replayed_and_on_two_streams(hq, cuda_device, T, top, E, K, N):
    W = (torch.randn((E, N, K), generator=gen(3), device="cuda") * 0.05).to(torch.bfloat16)
    wc, ws = hq.fp8_blocks_outputs(N, K, E)
    hq.hq_fp8_quantize_blocks(W, wc, ws)
    layers, drops, want = [Layer(hq, T, top, E, K, N) for _ in range(2)], (0.0, 0.2, 1.0, 0.5), []
    for seed, drop in enumerate(drops):
        layers[0].fill(10 * seed, drop)
        layers[0].run(wc, ws)
        want.append(layers[0].results())
    assert not want[2][0].any() and not want[2][1].any()  # all choices dropped: zeros
    assert want[0][0].any() and want[3][2].any()
    # captured once, replayed on other tokens and choices
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        layers[0].run(wc, ws)
    for seed in (1, 2, 0, 3):
        layers[0].fill(10 * seed, drops[seed])
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(layers[0].results(), want[seed]))
    # two calls at once, each with buffers of its own
    streams = [torch.cuda.Stream() for _ in layers]
    for layer, seed in zip(layers, (0, 1)):
        layer.fill(10 * seed, drops[seed])
    torch.cuda.synchronize()
    for _ in range(5):
        for layer, s in zip(layers, streams):
            layer.run(wc, ws, stream=s)
    torch.cuda.synchronize()
    for layer, seed in zip(layers, (0, 1)):
        assert all(torch.equal(a, b) for a, b in zip(layer.results(), want[seed]))
        assert layer.status.item() == 0


def test_expert_layer_without_tokens_and_an_expert_named_by_every_choice(hq, cuda_device):
    from post_weight_quantization_tcgen05_b200 import experts
    E, K, N, T, top = 3, 256, 128, 5, 4
    W = (torch.randn((E, N, K), generator=gen(3), device="cuda") * 0.05).to(torch.bfloat16)
    wc, ws = hq.fp8_blocks_outputs(N, K, E)
    hq.hq_fp8_quantize_blocks(W, wc, ws)
    none = torch.empty((0, K), dtype=torch.bfloat16, device="cuda")
    experts.expert_linear(hq, none, torch.empty((0, top), dtype=torch.int32, device="cuda"), None, wc, ws,
                          torch.empty((0, N), dtype=torch.bfloat16, device="cuda"))
    # every choice of every token is the same expert: four equal rows a token, whose sum is exact
    X = torch.randn((T, K), generator=gen(2), device="cuda").to(torch.bfloat16)
    Y, one = torch.empty((T, N), dtype=torch.bfloat16, device="cuda"), torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
    ids = torch.full((T, top), 1, dtype=torch.int32, device="cuda")
    experts.expert_linear(hq, X, ids, None, wc, ws, Y)
    experts.expert_linear(hq, X, ids[:, :1].contiguous(), None, wc, ws, one)
    assert one.any() and torch.equal(Y, 4 * one)
