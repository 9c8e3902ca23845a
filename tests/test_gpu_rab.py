"""GPU tests of the bucketed position bias and its gradient: values exact, the
gradient against 64-bit sums (fp32 sums of n terms: n 2^-24 of the sum of their
magnitudes), and through the attention that reads the table."""
import pytest
import torch

import pointwise_attention_b200 as pa

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def rnd(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(DEV)


def buckets(thr, L):
    d = torch.arange(L)
    return torch.searchsorted(thr.long(), d, right=True).to(DEV)


CASES = [(1, 1, (1, 1, 5)), (3, 2, (8, 4, 64)), (2, 7, (32, 16, 128)), (4, 100, (32, 16, 64)),
         (1, 513, (128, 1, 500)), (8, 1000, (128, 64, 70)), (5, 4096, (64, 32, 2048)),
         (2, 4097, (2, 1, 4096)), (3, 30011, (100, 10, 20000)), (1, 70000, (32, 16, 300))]


@pytest.mark.parametrize("H,L,b", CASES)
def test_forward_and_backward(H, L, b):
    thr = pa.hstu_pos_bucket_thresholds(*b)
    nb = b[0]
    table = rnd(H + L, H, nb)
    k = buckets(thr, L)
    want = torch.cat([torch.zeros(H, L - 1, device=DEV), table[:, k]], dim=1)
    assert torch.equal(pa.hstu_rab_bucket_fwd(table, L, thr), want)
    g = rnd(L, H, 2 * L - 1)
    g[:, :L - 1] = float("nan")        # entries of later keys are not read
    got = pa.hstu_rab_bucket_bwd(g, nb, thr)
    gd = g[:, L - 1:].double()
    ref = torch.zeros(H, nb, dtype=torch.float64, device=DEV).index_add_(1, k, gd)
    mag = torch.zeros(H, nb, dtype=torch.float64, device=DEV).index_add_(1, k, gd.abs())
    n = torch.bincount(k, minlength=nb).double() + 2
    assert bool(((got.double() - ref).abs() <= mag * n * 2.0 ** -24).all())
    assert torch.equal(got, pa.hstu_rab_bucket_bwd(g, nb, thr))


def test_any_ascending_thresholds_and_unaligned_output():
    """Empty buckets, thresholds past the table, an output off 16 bytes."""
    thr = torch.tensor([1, 1, 5, 40, 40, 41, 1000], dtype=torch.int32)
    H, L = 3, 61
    table = rnd(1, H, 8)
    k = buckets(thr, L)
    want = torch.cat([torch.zeros(H, L - 1, device=DEV), table[:, k]], dim=1)
    buf = torch.full((H * (2 * L - 1) + 2,), 9.0, device=DEV)
    out = buf[1:-1].view(H, 2 * L - 1)
    pa.hstu_rab_bucket_fwd(table, L, thr, out=out)
    assert torch.equal(out, want) and float(buf[0]) == 9.0 and float(buf[-1]) == 9.0
    g = rnd(2, H, 2 * L - 1)
    d = pa.hstu_rab_bucket_bwd(g, 8, thr)
    assert bool((d[:, [1, 4, 7]] == 0).all())
    assert pa.hstu_rab_bucket_bwd(g[:0], 8, thr).shape == (0, 8)


def test_through_the_attention():
    """Forward and backward of the attention with a table made from buckets:
    the buckets' gradient is that of the loss, against differences in fp32
    attention (steps of 1e-2 on values of order one: quadratic terms of the
    loss, a smooth function, cancel in central differences; what is left is
    about step^2 and fp32 rounding over the step)."""
    T, H, D, nb, L = 90, 2, 32, 8, 64
    off = torch.tensor([0, 50, 50, 90], dtype=torch.int32, device=DEV)
    q, k, v = (0.3 * rnd(s, T, H, D) for s in (1, 2, 3))
    u, dy = rnd(4, T, H * D), rnd(5, T, H * D)
    thr = pa.hstu_pos_bucket_thresholds(nb, 4, 40)
    table = 0.2 * rnd(6, H, nb)

    def forward(t):
        rab = pa.hstu_rab_bucket_fwd(t, L, thr)
        y, saved = pa.hstu_attn_fwd(q, k, v, u, off, 50, rab_pos=rab, save_for_backward=True)
        return y, saved, rab

    y, saved, rab = forward(table)
    g = pa.hstu_attn_bwd(dy, q, k, v, u, off, 50, saved, rab_pos=rab)
    d = pa.hstu_rab_bucket_bwd(g["d_rab_pos"], nb, thr)
    step = 1e-2
    for h, b in ((0, 0), (0, 3), (1, 5), (1, 7)):
        e = torch.zeros_like(table)
        e[h, b] = step
        hi, lo = (float((forward(table + s * e)[0].double() * dy.double()).sum()) for s in (1, -1))
        num = (hi - lo) / (2 * step)
        assert abs(num - float(d[h, b])) <= 2e-3 * max(1.0, float(d.abs().max()))
