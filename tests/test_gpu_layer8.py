"""GPU tests of the new operators in a run, as a user would chain them."""
import pytest
import torch

import pointwise_attention_b200 as pa

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16 = torch.bfloat16


def rnd(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(DEV)


def test_serving_run():
    """Histories: norm to 8 bits, projection, attention with a bucketed table,
    output projection, keys and values into the 4-bit cache; candidates: the
    same norm and projection, scored against the cache.  The scores equal those
    of the bf16 scoring over the cache's values up to both kernels' roundings
    of the attention weights (each a few bf16 half steps: bf16 arithmetic on
    pairs there), the bound of the bf16 scoring's own tests."""
    B, H, E = 3, 4, 512
    lens, cands = [300, 40, 129], [5, 1, 20]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    off, coff = i32([0, 300, 340, 469]), i32([0, 5, 6, 26])
    T, C = 469, 26
    w8, ws = pa.hstu_quant_rows(rnd(1, 2048, E) / E ** 0.5)
    w_out = (rnd(2, E, 512) / 512 ** 0.5).to(BF16)
    gain = 1.0 + 0.1 * rnd(3, E)
    thr = pa.hstu_pos_bucket_thresholds(32, 16, 256)
    rab = pa.hstu_rab_bucket_fwd(0.3 * rnd(4, H, 32), 301, thr)
    x, cx = rnd(5, T, E).to(BF16), rnd(6, C, E).to(BF16)

    def project(rows):
        n = pa.hstu_rmsnorm_fwd(rows, weight=gain, quant=True)
        return pa.hstu_uvqk_fp8_fwd(n["q8"], n["scale"], w8, ws, H, 128, 128, act=1)

    p, c = project(x), project(cx)
    y, _ = pa.hstu_attn_fwd(p["q"], p["k"], p["v"], p["u"], off, 300, rab_pos=rab)
    z, _ = pa.hstu_out_fwd(y, w_out, x)
    nxt = pa.hstu_rmsnorm_fwd(z, residual=x, weight=gain, quant=True)
    assert torch.isfinite(nxt["scale"]).all() and nxt["q8"].shape == (T, E)
    cache = pa.hstu_kv4_pack(p["k"], p["v"])
    got = pa.hstu_cand_kv4_fwd(cache, off, 300, c["q"], c["k"], c["v"], c["u"], coff, 20,
                               rab_pos=rab)
    kh, vh = pa.hstu_kv4_unpack(cache)
    want = pa.hstu_cand_fwd(kh, vh, off, 300, c["q"], c["k"], c["v"], c["u"], coff, 20,
                            rab_pos=rab)
    scale = float(want.float().abs().max())
    err = (got.float() - want.float()).abs()
    assert float(err.max()) <= 1e-2 * scale and float(err.mean()) <= 1e-3 * scale


def test_training_run_gradients_flow_to_buckets_and_norm():
    """Norm, projection (plain, fp32), attention with a bucketed table; backward
    to the table's buckets, the norm's weight and the input, against
    differences along one random direction of each.  fp32 throughout: the loss
    is of order ten and good to about 1e-5, the step 2e-2, so differences are
    good to about 1e-3; the directional derivatives are of order one."""
    T, E, H, D, L, nb = 70, 48, 2, 16, 64, 12
    off = torch.tensor([0, 45, 70], dtype=torch.int32, device=DEV)
    x, res = rnd(1, T, E), rnd(2, T, E)
    gain, w = 1.0 + 0.1 * rnd(3, E), rnd(4, 4 * H * D, E) / E ** 0.5
    table, c = 0.3 * rnd(5, H, nb), 0.1 * rnd(6, T, H * D)
    thr = pa.hstu_pos_bucket_thresholds(nb, 6, 50)

    def forward(x, gain, table):
        n = pa.hstu_rmsnorm_fwd(x, residual=res, weight=gain, save_rstd=True)
        p = n["y"] @ w.t()
        u, v, q, k = (t.contiguous() for t in p.split(H * D, dim=1))
        v, q, k = (t.view(T, H, D) for t in (v, q, k))
        rab = pa.hstu_rab_bucket_fwd(table, L, thr)
        y, saved = pa.hstu_attn_fwd(q, k, v, u, off, 45, rab_pos=rab, save_for_backward=True)
        return n, (q, k, v, u), rab, y, saved

    n, (q, k, v, u), rab, y, saved = forward(x, gain, table)
    g = pa.hstu_attn_bwd(c, q, k, v, u, off, 45, saved, rab_pos=rab)
    d_table = pa.hstu_rab_bucket_bwd(g["d_rab_pos"], nb, thr)
    dp = torch.cat([g["du"], g["dv"].flatten(1), g["dq"].flatten(1), g["dk"].flatten(1)], dim=1)
    dx, d_gain = pa.hstu_rmsnorm_bwd(dp @ w, n["h"], n["rstd"], weight=gain)
    loss = lambda *a: float((forward(*a)[3].double() * c.double()).sum())
    step = 2e-2
    for i, (value, grad) in enumerate(((x, dx), (gain, d_gain), (table, d_table))):
        direction = rnd(10 + i, *value.shape)
        direction /= direction.norm()
        args = [x, gain, table]
        hi, lo = list(args), list(args)
        hi[i], lo[i] = value + step * direction, value - step * direction
        num = (loss(*hi) - loss(*lo)) / (2 * step)
        want = float((grad.double() * direction.double()).sum())
        assert abs(num - want) <= 3e-3 * max(1.0, float(grad.norm())), (i, num, want)
