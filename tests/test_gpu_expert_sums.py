"""The sums and gradients of the experts' rows where every term counts: whole numbers, whose sums are
exact, and real values within the roundings that the kernel's own order of summation allows."""

import pytest
import torch

from test_gpu_experts import TYPES, a_case, gen, hq  # noqa: F401

pytestmark = pytest.mark.gpu

WIDTHS = [1, 8, 33, 255, 1000, 2056, 5119, 5120, 5121, 8191, 8192, 17408]


def shifted(t):
    """The same values from a base that is one element past a 16-byte boundary."""
    return torch.cat([t.reshape(-1)[:1], t.reshape(-1)])[1:].view(t.shape)


def terms(position, dY, rows):
    """dY[t] * rows[position[t, j]] in 64 bits, zeros for dropped choices."""
    kept = (position >= 0)[..., None]
    return torch.where(kept, dY.double()[:, None] * rows.double()[position.clamp(min=0).long()], 0.0)


def gradients(hq, dY, rows, position, w):  # noqa: F811
    d_rows, d_w = torch.full_like(rows, 7.0), torch.full_like(w, 7.0)
    hq.hq_expert_combine_backward(dY, rows, position, w, d_rows, d_w)
    return d_rows, d_w


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("K", WIDTHS)
@pytest.mark.parametrize("T,top,E", [(7, 3, 4), (5, 9, 6)])
def test_sums_and_gradients_of_whole_numbers_are_exact(hq, cuda_device, T, top, E, K, dtype):  # noqa: F811
    """Values of 1 .. 2 in size, weights that are powers of two: the weights' gradients are sums of K
    whole numbers up to 4, below 2^24, so that a term left out or taken twice shows."""
    _, _, position, _, w = a_case(hq, T, top, E, K, dtype)
    g = gen(K)

    def whole(shape):
        v = torch.randint(1, 3, shape, generator=g, device="cuda") * (torch.randint(0, 2, shape, generator=g, device="cuda") * 2 - 1)
        return v.to(TYPES[dtype])
    dY, rows = whole((T, K)), whole((T * top, K))
    w = 2.0 ** torch.randint(-2, 3, w.shape, generator=g, device="cuda").float()
    kept = (position >= 0)[..., None]
    at = position.clamp(min=0).long()
    for move in (lambda t: t, shifted):
        d_rows, d_w = gradients(hq, move(dY), move(rows), position, w)
        assert torch.equal(d_w.double(), terms(position, dY, rows).sum(2))
        want = torch.full_like(rows, 7.0)
        want[position[position >= 0].long()] = (w[..., None] * dY.float()[:, None])[position >= 0].to(rows.dtype)
        assert torch.equal(d_rows, want)
        Y = torch.full_like(dY, float("nan"))
        hq.hq_expert_combine(move(rows), position, w, Y)
        # at most 9 terms, multiples of 2^-2 up to 8: exact in fp32, rounded once
        assert torch.equal(Y, torch.where(kept, w[..., None] * rows.float()[at], 0.0).sum(1).to(dY.dtype))


def depth(K, dtype, aligned):
    """Additions that one term of a weight's gradient goes through: those of its thread (16-byte vectors, or
    four values 32 apart where rows are not made of them, dealt out to 32 .. 256 threads in powers of two),
    5 over the lanes of a warp, 8 over the warps at most."""
    size = 2 if dtype == "bf16" else 4
    whole = aligned and K * size % 16 == 0
    each = 16 // size if whole else 4
    vectors = K // each if whole else -(-K // 128) * 32
    threads = 32
    while threads < 256 and threads < vectors:
        threads *= 2
    return -(-vectors // threads) * each + 5 + 8


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("K", WIDTHS)
def test_gradients_within_the_order_of_summation(hq, cuda_device, K, dtype):  # noqa: F811
    """Each addition rounds by 2^-24 of a partial sum, which is no larger than the sum of the terms'
    magnitudes; the factor covers the products of such roundings."""
    T, top, E = 12, 5, 7
    _, _, position, dY, w = a_case(hq, T, top, E, K, dtype, seed=11)
    rows = torch.randn((T * top, K), generator=gen(5), device="cuda").to(TYPES[dtype])
    t = terms(position, dY, rows)
    for move, aligned in ((lambda v: v, True), (shifted, False)):
        _, d_w = gradients(hq, move(dY), move(rows), position, w)
        tol = t.abs().sum(2) * depth(K, dtype, aligned) * 2.0 ** -24 * (1 + 2.0 ** -10)
        assert ((d_w.double() - t.sum(2)).abs() <= tol).all()
