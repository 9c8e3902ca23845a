"""GPU tests of calls whose elements lie past 32 bits, and of the few-candidate
kernel with more heads than a CTA has warps.

What lies far away is compared bit by bit with the same data close by.
"""
import pytest
import torch

import pointwise_attention_b200 as pa

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16


def rnd(seed, *shape, dtype=BF16, std=1.0):
    return (std * torch.randn(*shape, generator=torch.Generator().manual_seed(seed))).to(dtype).to(DEV)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def score(cache, lens, first, cands, H, time):
    B, T, C = len(lens), sum(lens), sum(cands)
    off, coff = ([sum(x[:b]) for b in range(B + 1)] for x in (lens, cands))
    kw = dict(first_rows=i32(first), total_tokens=T,
              rab_pos=rnd(9, H, 2 * max(lens) + 1, dtype=F32, std=0.3))
    if time:
        kw.update(timestamps=1_700_000_000 + 700 * torch.arange(T, device=DEV),
                  cand_timestamps=1_700_000_000 + 700 * T + 900 * torch.arange(C, device=DEV),
                  rab_time=rnd(10, H, 128, dtype=F32, std=0.3))
    ws = pa.hstu_cand_kv4_workspace(B, H, max(lens), C, max(cands), DEV)
    y = pa.hstu_cand_kv4_fwd(cache, i32(off), max(lens), rnd(3, C, H, 128, std=128 ** -0.5),
                             rnd(4, C, H, 128, std=128 ** -0.5), rnd(5, C, H, 128),
                             rnd(6, C, H * 128), i32(coff), max(cands), workspace=ws, **kw)
    assert pa.hstu_attn_check(ws) == 0
    return y


@pytest.mark.parametrize("H,R", [(8, (1 << 23) + 333), (3, 23_000_001)])
def test_cache_rows_past_32_bits(H, R):
    """Codes of more than 2^32 bytes: rows at the cache's end written, read back
    and scored against, with an odd number of heads too."""
    lens = [301, 77]
    T = sum(lens)
    assert R * H * 64 > 1 << 32
    k, v = rnd(1, T, H, 128, std=128 ** -0.5), rnd(2, T, H, 128)
    near = pa.hstu_kv4_pack(k, v)
    cache = tuple(torch.empty((R, H, n), dtype=d, device=DEV)
                  for n, d in ((64, torch.uint8), (4, BF16)) * 2)
    first = [R - T, R - lens[1]]
    rows = torch.arange(R - T, R, dtype=torch.int32, device=DEV)
    pa.hstu_kv4_pack(k, v, cache=cache, rows=rows)
    for a, b in zip(cache, near):
        assert torch.equal(a[R - T:], b)
    for a, b in zip(pa.hstu_kv4_unpack(cache, rows=rows), pa.hstu_kv4_unpack(near)):
        assert torch.equal(a, b)
    for cands in ([2, 5], [40, 130]):
        for time in (False, True):
            assert torch.equal(score(cache, lens, first, cands, H, time),
                               score(near, lens, [0, lens[0]], cands, H, time))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("E", [257, 512])
def test_rows_past_32_bits(dtype, E):
    """The last rows of more than 2^32 bytes, as those rows alone."""
    T, n = (1 << 32) // (E * (2 if dtype == BF16 else 4)) + 1001, 600
    x = torch.empty((T, E), dtype=dtype, device=DEV)
    x[:-n] = 0
    x[-n:] = rnd(1, n, E, dtype=dtype)
    w = 1 + rnd(2, E, dtype=F32, std=0.1)
    near = x[-n:].clone()
    got = pa.hstu_rmsnorm_fwd(x, weight=w, quant=True, save_rstd=True)
    want = pa.hstu_rmsnorm_fwd(near, weight=w, quant=True, save_rstd=True)
    for key in ("q8", "scale", "rstd"):
        assert torch.equal(got[key][-n:].view(torch.uint8), want[key].view(torch.uint8))
    del got
    rstd = torch.ones(T, device=DEV)
    rstd[-n:] = want["rstd"]
    dx, dw = pa.hstu_rmsnorm_bwd(x, x, rstd, weight=w)
    dx1, dw1 = pa.hstu_rmsnorm_bwd(near, near, want["rstd"], weight=w)
    assert torch.equal(dx[-n:], dx1) and bool((dx[:-n:100_003] == 0).all())
    # rows of zeros add nothing; the others' sums are taken in another order
    terms = (near.double().square() * want["rstd"].double()[:, None]).sum(0)
    assert bool(((dw - dw1).abs().double() <= 2 * n * 2.0 ** -24 * terms).all())


@pytest.mark.parametrize("time", [False, True])
@pytest.mark.parametrize("H", [9, 11, 15, 16])
def test_few_candidates_with_many_heads(H, time):
    """Up to 16 candidates with heads in two groups of CTAs, empty histories and
    users without candidates among them, against the formula in 64 bits."""
    lens, cands = [333, 0, 47, 160], [1, 3, 0, 12]
    B, T, C = 4, sum(lens), sum(cands)
    off, coff = ([sum(x[:b]) for b in range(B + 1)] for x in (lens, cands))
    k, v = rnd(1, T, H, 128, std=128 ** -0.5), rnd(2, T, H, 128)
    cache = pa.hstu_kv4_pack(k, v)
    kh, vh = (t.double() for t in pa.hstu_kv4_unpack(cache))
    y = score(cache, lens, off[:-1], cands, H, time).double()
    q, kc = (rnd(s, C, H, 128, std=128 ** -0.5).double() for s in (3, 4))
    vc, u = rnd(5, C, H, 128).double(), rnd(6, C, H * 128).double()
    L = max(lens) + 1
    rab = rnd(9, H, 2 * L - 1, dtype=F32, std=0.3).double()
    rt = rnd(10, H, 128, dtype=F32, std=0.3).double()
    thr = torch.from_numpy(pa.hstu_time_bucket_thresholds(128)).to(DEV)
    silu = lambda x: x / (1.0 + torch.exp(-x))
    want, tol = [], []
    for b in range(B):
        n = lens[b]
        for c in range(coff[b], coff[b + 1]):
            s = slice(off[b], off[b + 1])
            x = torch.einsum("hd,nhd->hn", q[c], kh[s]) + rab[:, [L - 1 + n - j for j in range(n)]]
            mag = torch.einsum("hd,nhd->hn", q[c].abs(), kh[s].abs())
            x0 = (q[c] * kc[c]).sum(-1) + rab[:, L - 1]
            if time:
                dt = 700 * T + 900 * c - 700 * torch.arange(off[b], off[b + 1], device=DEV)
                x = x + rt[:, torch.searchsorted(thr, dt, right=True)]
                x0 = x0 + rt[:, 0]
            a, a0 = silu(x), silu(x0)
            o = torch.einsum("hn,nhd->hd", a, vh[s]) + a0[:, None] * vc[c]
            # a weight in two bf16 parts, its score and its exponential in fp32;
            # fp32 sums of n terms
            da = a.abs() * (2.0 ** -16 + 2.0 ** -20) + 1.1 * (mag + x.abs() + 1) * 132 * 2.0 ** -24
            do = (torch.einsum("hn,nhd->hd", da, vh[s].abs()) +
                  torch.einsum("hn,nhd->hd", a.abs(), vh[s].abs()) * (n + 8) * 2.0 ** -24 +
                  (a0.abs() + 1)[:, None] * vc[c].abs() * 2.0 ** -16)
            o, do = o.flatten() / (n + 1), do.flatten() / (n + 1)
            r = 1.0 / torch.sqrt(o.var(correction=0) + 1e-5)
            xh = (o - o.mean()) * r
            dx = 1.05 * r * (do + do.mean() + xh.abs() * (xh.abs() * do).mean()) + xh.abs() * 2.0 ** -16
            g = silu(u[c])
            want.append(xh * g)
            tol.append(dx * g.abs() + (xh * g).abs() * (2.0 ** -8 + 2.0 ** -16) + 1e-30)
    want, tol = torch.stack(want), torch.stack(tol)
    assert torch.isfinite(y).all()
    assert bool(((y - want).abs() <= tol).all()), float(((y - want).abs() / tol).max())
