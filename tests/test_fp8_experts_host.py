"""The e4m3 layers and the expert layout without a GPU: the oracle against what its definitions
fix, the refusals of the C ABI and of the binding, and the order of the calls in experts.py."""

import ctypes
import types

import numpy as np
import pytest
import torch

import oracle
from post_weight_quantization_tcgen05_b200 import experts


@pytest.fixture(scope="module")
def hq():
    import post_weight_quantization_tcgen05_b200 as m
    return m


# ------------------------------------------------------------------ oracle

def test_e4m3_values_and_rounding():
    v = oracle.e4m3_decode(np.arange(256))
    assert np.array_equal(v, torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy(),
                          equal_nan=True)
    fin = np.unique(v[np.isfinite(v)])
    assert fin.max() == 448 and fin[fin > 0].min() == 2.0 ** -9
    assert np.array_equal(oracle.e4m3_round(fin), fin)
    # a rounding is never further from x than any other value is
    x = np.concatenate([np.linspace(-460, 460, 4001), np.linspace(-0.03, 0.03, 4001), (fin[1:] + fin[:-1]) / 2])
    r = oracle.e4m3_round(x)
    assert np.array_equal(np.abs(r - x), np.min(np.abs(x[:, None] - fin[None]), axis=1))
    # between two neighbours, the one with an even last bit
    mid = (fin[1:] + fin[:-1]) / 2
    byte = {float(a): b for b, a in enumerate(v) if np.isfinite(a)}
    assert all(byte[float(a)] % 2 == 0 for a in oracle.e4m3_round(mid) if a != 0)
    assert oracle.e4m3_round(np.inf) == 448 and oracle.e4m3_round(-1e9) == -448 and np.isnan(oracle.e4m3_round(np.nan))


def test_quantiser_of_the_oracle():
    g = np.random.RandomState(0)
    x = g.randn(130, 300).astype(np.float32) * np.exp(g.randn(300))[None].astype(np.float32)
    for rows in (1, 128):
        c, s = oracle.fp8_quantize(x, rows)
        assert s.shape == (130 if rows == 1 else 2, 3)
        q = oracle.fp8_dequantize(c, s, rows)
        top = np.repeat(np.repeat(s * 448, rows, 0)[:130], 128, 1)[:, :300]
        # half a step of e4m3 relative to the value, or half its smallest step, plus the fp32 roundings
        assert np.all(np.abs(q - x) <= np.maximum(np.abs(x) * 2.0 ** -4, top / 448 * 2.0 ** -10) + np.abs(x) * 2.0 ** -22)
        assert np.abs(c).max() == 448  # every block's largest value takes the largest code
    c, s = oracle.fp8_quantize(np.zeros((2, 5)), 1)
    assert not c.any() and not s.any()
    c, s = oracle.fp8_quantize(np.full((1, 3), 2.0 ** -110), 1)
    assert s[0, 0] == np.float32(2.0 ** -100 / 448) and np.all(c == oracle.e4m3_round(448 * 2.0 ** -10))


def test_product_of_the_oracle_by_hand():
    a, sa = np.array([[1.0, 2.0, -3.0]]), np.array([[0.5]])
    w, sw = np.array([[2.0, 0.0, 1.0], [0.0, -1.0, 4.0]]), np.array([[2.0]])
    y, size = oracle.fp8_product(a, sa, w, sw)
    assert np.array_equal(y, [[-1.0, -14.0]]) and np.array_equal(size, [[5.0, 14.0]])


def test_sort_of_the_oracle_by_hand():
    offsets, order, position = oracle.expert_sort(np.array([[2, 0], [0, -1], [2, 2], [7, 0]]), 3)
    assert offsets.tolist() == [0, 3, 3, 6]
    assert order.tolist() == [1, 2, 7, 0, 4, 5]
    assert position.tolist() == [[3, 0], [1, -1], [4, 5], [-1, 2]]


def test_combine_gradients_of_the_oracle_against_differences():
    g = np.random.RandomState(1)
    _, order, pos = oracle.expert_sort(g.randint(-1, 3, (5, 3)), 3)
    rows, w, dY = g.randn(15, 4), g.randn(5, 3), g.randn(5, 4)
    d_rows, d_w = oracle.expert_combine_backward(dY, rows, pos, w, np.zeros((15, 4)))
    loss = lambda r, v: float(np.sum(dY * oracle.expert_combine(r, pos, v)))  # noqa: E731
    h = 1e-6
    for x, dx, f in ((rows, d_rows, lambda r: loss(r, w)), (w, d_w, lambda v: loss(rows, v))):
        for i in np.ndindex(x.shape):
            up, down = x.copy(), x.copy()
            up[i] += h
            down[i] -= h
            # the loss is linear in each: the difference is its gradient but for rounding
            assert abs((f(up) - f(down)) / (2 * h) - dx[i]) < 1e-8


# ------------------------------------------------------------------ refusals

def test_sizes(hq):
    assert [hq.hq_fp8_pitch(k) for k in (0, 1, 16, 17, 5120)] == [0, 16, 16, 32, 5120]
    assert hq.hq_fp8_linear_workspace_bytes(0, 128) == 0
    assert hq.hq_fp8_linear_workspace_bytes(3, 130) >= 3 * 144 + 2 * 3 * 4
    assert hq.hq_fp8_linear_workspace_bytes(-1, 128) == hq.hq_fp8_linear_workspace_bytes(1, 0) == 0
    assert hq.hq_expert_sort_workspace_bytes(64, 8, 48) > 0
    assert hq.hq_expert_sort_workspace_bytes(1, 0, 4) == hq.hq_expert_sort_workspace_bytes(1, 1, 0) == 0
    assert hq.hq_expert_sort_workspace_bytes(1, 1, 1025) == hq.hq_expert_sort_workspace_bytes(1 << 28, 8, 4) == 0


def test_bad_arguments_are_refused_before_a_launch(hq):
    L, p, odd, none = hq.lib, ctypes.c_void_p(4096), ctypes.c_void_p(4097), None  # never dereferenced
    bad, unsup, ws = hq.HQ_ERR_INVALID, hq.HQ_ERR_UNSUPPORTED, hq.HQ_ERR_WORKSPACE
    big = 1 << 62

    assert L.hq_fp8_quantize_rows(none, 1, 0, 8, none, none, none) == hq.HQ_OK  # no rows: nothing to do
    for args, want in (((none, 1, 2, 8, p, p), bad), ((p, 1, 2, 8, none, p), bad), ((p, 1, 2, 8, p, none), bad),
                       ((p, 2, 2, 8, p, p), bad), ((p, 1, -1, 8, p, p), bad), ((p, 1, 2, 0, p, p), bad),
                       ((odd, 1, 2, 8, p, p), bad), ((p, 1, 2, 8, ctypes.c_void_p(4104), p), bad),
                       ((p, 1, 2, 8, p, odd), bad), ((p, 1, big, 8, p, p), unsup), ((p, 1, 2, big, p, p), unsup)):
        assert L.hq_fp8_quantize_rows(*args, none) == want, args

    for args, want in (((none, 1, 1, 2, 8, p, p), bad), ((p, 1, 0, 2, 8, p, p), bad), ((p, 1, 1, 0, 8, p, p), bad),
                       ((p, 7, 1, 2, 8, p, p), bad), ((p, 1, 1025, 2, 8, p, p), unsup), ((p, 1, 1, big, 8, p, p), unsup),
                       ((p, 1, 1024, 1 << 22, 8, p, p), unsup), ((p, 0, 1, 2, 8, ctypes.c_void_p(4104), p), bad)):
        assert L.hq_fp8_quantize_blocks(*args, none) == want, args

    def gemm(a=p, sa=p, M=2, w=p, sw=p, N=4, K=8, y=p, dt=1):
        return L.hq_fp8_gemm(a, sa, M, w, sw, N, K, y, dt, none, none)
    assert gemm(M=0, a=none, y=none) == hq.HQ_OK
    for kw in ({"a": none}, {"sa": none}, {"w": none}, {"sw": none}, {"y": none}, {"M": -1}, {"N": 0}, {"K": 0}, {"dt": 2},
               {"a": ctypes.c_void_p(4104)}, {"w": ctypes.c_void_p(4104)}, {"y": odd}, {"sa": odd}, {"sw": odd}):
        assert gemm(**kw) == bad, kw
    for kw in ({"M": big}, {"N": big}, {"K": big}):
        assert gemm(**kw) == unsup, kw

    def linear(x=p, dt=1, M=2, w=p, N=4, K=8, y=p, work=p, nbytes=1 << 20):
        return L.hq_fp8_linear(x, dt, M, w, p, N, K, y, 1, work, nbytes, none, none)
    assert linear(M=0, work=none, nbytes=0) == hq.HQ_OK
    assert linear(x=none) == linear(dt=3) == linear(w=none) == linear(y=none) == linear(K=0) == linear(x=odd) == bad
    assert linear(work=none) == linear(nbytes=8) == linear(work=ctypes.c_void_p(4096 + 128)) == ws

    def expert(rows=2, off=p, E=3, N=4, K=8):
        return L.hq_fp8_expert_gemm(p, p, rows, off, p, p, E, N, K, p, 1, none, none)
    assert expert(rows=0, off=none) == hq.HQ_OK
    assert expert(off=none) == expert(off=odd) == expert(E=0) == bad
    assert expert(E=1025) == expert(E=1024, N=1 << 22) == unsup

    def sort(ids=p, T=2, top=2, E=4, off=p, order=p, pos=p, work=p, nbytes=1 << 20):
        return L.hq_expert_sort(ids, T, top, E, off, order, pos, work, nbytes, none)
    assert sort(ids=none) == sort(off=none) == sort(order=none) == sort(pos=none) == sort(ids=odd) == bad
    assert sort(T=-1) == sort(top=0) == sort(E=0) == bad
    assert sort(E=1025) == sort(T=1 << 28, top=8) == sort(T=big, top=big) == unsup
    assert sort(work=none) == sort(nbytes=8) == sort(work=ctypes.c_void_p(4104)) == ws

    for f, n in ((lambda *a: L.hq_expert_dispatch(a[0], a[1], a[2], 8, a[3], a[4], p, none), "dispatch"),
                 (lambda *a: L.hq_expert_dispatch_fp8(a[0], a[1], a[2], 8, a[3], a[4], p, p, none), "dispatch_fp8"),
                 (lambda *a: L.hq_expert_combine(a[0], a[1], a[2], 8, a[3], a[4], none, p, none), "combine"),
                 (lambda *a: L.hq_expert_combine_backward(a[0], p, a[1], a[2], 8, a[3], a[4], p, p, p, none), "backward")):
        assert f(none, 1, 0, none, 2) == hq.HQ_OK, n
        for a in ((none, 1, 2, p, 2), (p, 2, 2, p, 2), (p, 1, -1, p, 2), (p, 1, 2, none, 2), (p, 1, 2, p, 0),
                  (odd, 1, 2, p, 2), (p, 1, 2, odd, 2)):
            assert f(*a) == bad, (n, a)
        assert f(p, 1, 1 << 28, p, 8) == unsup, n
    assert L.hq_expert_combine_backward(p, p, 1, 2, 8, p, 2, none, p, p, none) == bad  # the forward's weights


def test_binding_refuses_wrong_shapes_types_and_places(hq):
    X, fp8 = torch.zeros((3, 130), dtype=torch.bfloat16), torch.float8_e4m3fn
    codes, scales = torch.zeros((3, 144), dtype=torch.uint8).view(fp8), torch.zeros((2, 3))
    with pytest.raises(ValueError, match="CUDA"):
        hq.hq_fp8_quantize_rows(X, codes, scales)
    with pytest.raises(ValueError, match="codes"):
        hq.hq_fp8_quantize_rows(X, codes[:, :130], scales)
    with pytest.raises(ValueError, match="scales"):
        hq.hq_fp8_quantize_rows(X, codes, scales.t())
    with pytest.raises(ValueError, match="codes"):
        hq.hq_fp8_quantize_rows(X, codes.float(), scales)
    with pytest.raises(ValueError, match="scales"):
        hq.hq_fp8_quantize_blocks(X, codes, torch.zeros((1, 3)))
    with pytest.raises(ValueError, match="w_scales"):
        hq.hq_fp8_gemm(codes, scales, codes, torch.zeros((1, 1)), 130, torch.zeros((3, 3)))
    with pytest.raises(ValueError, match="offsets"):
        hq.hq_fp8_expert_gemm(codes, scales, torch.zeros(2, dtype=torch.int64), codes[None], torch.zeros((1, 1, 2)), 130,
                              torch.zeros((3, 3)))
    ids = torch.zeros((3, 2), dtype=torch.int64)
    out = hq.expert_sort_outputs(3, 2, 4, "cpu")
    with pytest.raises(ValueError, match="ids"):
        hq.hq_expert_sort(ids, 4, *out, torch.zeros(1024, dtype=torch.uint8))
    with pytest.raises(ValueError, match="rows"):
        hq.hq_expert_dispatch(X, out[2], torch.zeros((6, 130)))
    with pytest.raises(ValueError, match="weights"):
        hq.hq_expert_combine(torch.zeros((6, 5)), out[2], torch.zeros((3, 3)), torch.zeros((3, 5)))


# ------------------------------------------------------------------ experts.py

def test_the_header_names_the_binding_s_limit(hq):
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    m = re.search(r"#define\s+HQ_MAX_EXPERTS\s+(\d+)", open(os.path.join(root, "include", "hq.h")).read())
    assert m and int(m.group(1)) == hq.HQ_MAX_EXPERTS


def test_expert_hessians_feeds_each_expert_its_rows():
    def sort(ids, E, offsets, order, position, workspace):
        off, o, p = oracle.expert_sort(ids.numpy(), E)
        offsets.copy_(torch.from_numpy(off))
        order[:len(o)] = torch.from_numpy(o).int()
        position.copy_(torch.from_numpy(p))

    def dispatch(X, position, rows):
        for t in range(X.shape[0]):
            for j in range(position.shape[1]):
                if position[t, j] >= 0:
                    rows[position[t, j]] = X[t]

    def accumulate(H, X, dev_status=None):
        H += X.t() @ X

    import post_weight_quantization_tcgen05_b200 as real
    hq = types.SimpleNamespace(hq_expert_sort=sort, hq_expert_dispatch=dispatch, hq_hessian_accumulate=accumulate,
                               hq_expert_sort_workspace_bytes=real.hq_expert_sort_workspace_bytes,
                               expert_sort_outputs=real.expert_sort_outputs, alloc_workspace=real.alloc_workspace)
    g = torch.Generator()
    g.manual_seed(3)
    X = torch.randn((20, 6), generator=g, dtype=torch.float64)
    ids = torch.randint(-1, 3, (20, 2), generator=g, dtype=torch.int32)
    ids[ids == 1] = 0  # nothing for expert 1
    H = torch.ones((3, 6, 6), dtype=torch.float64)
    counts = experts.expert_hessians(hq, X, ids, H)
    for e in range(3):
        named = (ids == e).sum(1).double()
        assert counts[e] == int(named.sum())
        assert torch.allclose(H[e], 1 + (X * named[:, None]).t() @ X)
    assert counts[1] == 0
