"""CPU tests of the row, bucket, 8-bit projection and 4-bit cache entry points:
bad arguments are refused synchronously with the documented status, and the
bucket thresholds are those of the formula.

Every refused case passes placeholder device addresses and breaks one rule, so
the library returns before it touches them.
"""
import ctypes
import math

import pytest
import torch

INV, UNS, WS = 1, 2, 5
FAKE = 0x7F0000000000   # placeholder device address, 256-byte aligned; never dereferenced


@pytest.fixture(scope="module")
def pa():
    from pointwise_attention_b200 import build
    build.build()
    import pointwise_attention_b200 as pa
    return pa


def vp(x):
    return None if x is None else ctypes.c_void_p(x)


def call(fn, args, change):
    args = dict(args)
    args.update(change)
    return fn(*[vp(v) if isinstance(v, int) and k.startswith("p_") else v
                for k, v in args.items()])


RMS = dict(dt=1, T=4, E=64, p_x=FAKE, p_res=None, p_w=None, eps=1e-6, p_h=None, p_y=FAKE,
           p_q8=None, p_s=None, p_rstd=None, p_stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(dt=2), INV), (dict(T=-1), INV), (dict(E=0), INV), (dict(p_x=None), INV),
    (dict(p_y=None), INV), (dict(eps=0.0), INV), (dict(eps=float("nan")), INV),
    (dict(eps=float("inf")), INV), (dict(p_q8=FAKE), INV), (dict(p_s=FAKE), INV),
    (dict(p_h=FAKE), INV), (dict(p_x=FAKE + 1), INV), (dict(p_y=FAKE + 1), INV),
    (dict(p_w=FAKE + 2), INV), (dict(p_rstd=FAKE + 2), INV), (dict(E=16385), UNS),
    (dict(dt=0, p_x=FAKE + 2), INV), (dict(T=2 ** 31 - 1), UNS)])
def test_rmsnorm_fwd_refusals(pa, change, want):
    assert call(pa.load_library().hstu_rmsnorm_fwd, RMS, change) == want


BWD = dict(dt=1, T=4, E=64, p_dy=FAKE, p_h=FAKE, p_r=FAKE, p_w=None, p_dres=None, p_dx=FAKE,
           p_dw=FAKE, p_ws=FAKE, bytes=1 << 20, p_stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(dt=7), INV), (dict(T=-1), INV), (dict(E=-3), INV), (dict(p_dy=None), INV),
    (dict(p_h=None), INV), (dict(p_r=None), INV), (dict(p_dx=None), INV),
    (dict(p_dres=FAKE + 1), INV), (dict(p_dw=FAKE + 1), INV), (dict(E=20000), UNS),
    (dict(p_ws=None), WS), (dict(p_ws=FAKE + 16), WS), (dict(bytes=255), WS)])
def test_rmsnorm_bwd_refusals(pa, change, want):
    assert call(pa.load_library().hstu_rmsnorm_bwd, BWD, change) == want


QR = dict(dt=0, T=4, E=64, p_x=FAKE, p_q8=FAKE, p_s=FAKE, p_stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(dt=-1), INV), (dict(T=-2), INV), (dict(E=0), INV), (dict(p_x=None), INV),
    (dict(p_q8=None), INV), (dict(p_s=None), INV), (dict(p_x=FAKE + 2), INV),
    (dict(E=16400), UNS)])
def test_quant_rows_refusals(pa, change, want):
    assert call(pa.load_library().hstu_quant_rows, QR, change) == want


UV = dict(T=4, E=64, H=2, dqk=128, dv=128, act=1, p_x=FAKE, p_xs=FAKE, p_w=FAKE, p_ws_=FAKE,
          p_b=None, p_u=FAKE, p_v=FAKE, p_q=FAKE, p_k=FAKE, p_ws=FAKE, bytes=256, p_stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(T=-1), INV), (dict(H=0), INV), (dict(act=2), INV), (dict(p_x=None), INV),
    (dict(p_xs=None), INV), (dict(p_w=FAKE + 8), INV), (dict(p_b=FAKE + 4), INV),
    (dict(p_k=None), INV), (dict(E=24), UNS), (dict(H=1), UNS), (dict(dqk=64), UNS),
    (dict(T=8388481), UNS), (dict(p_ws=None), WS), (dict(bytes=128), WS)])
def test_uvqk_fp8_refusals(pa, change, want):
    assert call(pa.load_library().hstu_uvqk_fp8_fwd, UV, change) == want


def test_empty_calls_enqueue_nothing(pa):
    lib = pa.load_library()
    assert call(lib.hstu_rmsnorm_fwd, RMS, dict(T=0, p_x=None, p_y=None)) == 0
    assert call(lib.hstu_rmsnorm_bwd, BWD, dict(T=0, p_dw=None)) == 0
    assert call(lib.hstu_quant_rows, QR, dict(T=0, p_x=None)) == 0
    assert call(lib.hstu_uvqk_fp8_fwd, UV, dict(T=0, p_x=None)) == 0
    assert call(lib.hstu_kv4_pack, KV, dict(T=0, p_k=None)) == 0
    assert call(lib.hstu_kv4_unpack, UNKV, dict(T=0, p_k=None)) == 0


KV = dict(T=4, H=2, p_k=FAKE, p_v=FAKE, p_rows=None, R=4, p_kc=FAKE, p_ks=FAKE, p_vc=FAKE,
          p_vs=FAKE, p_ws=FAKE, bytes=256, p_stream=None)
UNKV = dict(T=4, H=2, p_kc=FAKE, p_ks=FAKE, p_vc=FAKE, p_vs=FAKE, p_rows=None, R=4, p_k=FAKE,
            p_v=FAKE, p_ws=FAKE, bytes=256, p_stream=None)


@pytest.mark.parametrize("which", ["pack", "unpack"])
@pytest.mark.parametrize("change,want", [
    (dict(T=-1), INV), (dict(H=0), INV), (dict(R=-1), INV), (dict(R=3), INV),
    (dict(p_k=None), INV), (dict(p_vc=None), INV), (dict(p_ks=FAKE + 8), INV),
    (dict(p_rows=FAKE + 2), INV), (dict(H=65537), UNS), (dict(p_rows=FAKE, p_ws=None), WS),
    (dict(p_ws=FAKE + 128), WS), (dict(bytes=255), WS)])
def test_kv4_refusals(pa, which, change, want):
    lib = pa.load_library()
    if which == "pack":
        assert call(lib.hstu_kv4_pack, KV, change) == want
    else:
        assert call(lib.hstu_kv4_unpack, UNKV, change) == want


def test_rab_bucket_refusals(pa):
    lib = pa.load_library()
    thr = (ctypes.c_int32 * 127)(*range(1, 128))
    ok = dict(H=2, L=100, NB=8, thr=thr, p_in=FAKE, p_out=FAKE, p_stream=None)
    bad = [dict(H=-1), dict(L=0), dict(NB=0), dict(NB=129), dict(thr=None), dict(p_in=None),
           dict(p_out=FAKE + 2), dict(L=2 ** 30 + 1),
           dict(thr=(ctypes.c_int32 * 127)(0, *range(2, 128))),
           dict(thr=(ctypes.c_int32 * 127)(5, 4, *range(6, 131)))]
    for fn in (lib.hstu_rab_bucket_fwd, lib.hstu_rab_bucket_bwd):
        for change in bad:
            assert call(fn, ok, change) == INV, change
        assert call(fn, ok, dict(H=65536)) == UNS
        assert call(fn, ok, dict(H=0, p_in=None, p_out=None)) == 0


def problem(pa, **kw):
    p = pa.hstu_problem_t()
    base = dict(dtype=1, batch=2, total_tokens=64, max_seq_len=48, num_heads=4, d_qk=128, d_v=128,
                offsets=FAKE, ln_eps=1e-5)
    base.update(kw)
    for k, v in base.items():
        setattr(p, k, v)
    return p


CAND = dict(p_kc=FAKE, p_ks=FAKE, p_vc=FAKE, p_vs=FAKE, R=64, p_first=None, p_co=FAKE, C=6, mc=4,
            p_cts=None, p_q=FAKE, p_k=FAKE, p_v=FAKE, p_u=FAKE, p_y=FAKE, p_ws=FAKE,
            bytes=1 << 30, p_stream=None)


@pytest.mark.parametrize("prob,change,want", [
    ({}, dict(C=-1), INV), ({}, dict(mc=0), INV), ({}, dict(R=63), INV), ({}, dict(R=-1), INV),
    ({}, dict(p_co=None), INV), ({}, dict(p_q=None), INV), ({}, dict(p_y=FAKE + 4), INV),
    ({}, dict(p_kc=None), INV), ({}, dict(p_vs=FAKE + 8), INV),
    (dict(rab_pos=FAKE, rab_pos_len=48), {}, INV),
    (dict(rab_time=FAKE, num_time_buckets=8, timestamps=FAKE), {}, INV),
    (dict(rab_time=FAKE, num_time_buckets=8), dict(p_cts=FAKE), INV),
    (dict(batch=-1), {}, INV), (dict(ln_eps=0.0), {}, INV), (dict(dtype=0), {}, UNS),
    (dict(d_v=64), {}, UNS), (dict(num_heads=17), {}, UNS),
    (dict(batch=1 << 20, max_seq_len=1 << 20, total_tokens=64), dict(mc=1 << 12), UNS),
    ({}, dict(p_ws=None), WS), ({}, dict(p_ws=FAKE + 64), WS), ({}, dict(bytes=4096), WS)])
def test_cand_kv4_refusals(pa, prob, change, want):
    lib = pa.load_library()
    p = problem(pa, **prob)
    fn = lambda *a: lib.hstu_cand_kv4_fwd(ctypes.byref(p), *a)
    assert call(fn, CAND, change) == want


def test_cand_kv4_workspace_sizes(pa):
    size = pa.load_library().hstu_cand_kv4_workspace_size
    for bad in [(-1, 4, 10, 4, 2), (1, 0, 10, 4, 2), (1, 17, 10, 4, 2), (1, 4, -1, 4, 2),
                (1, 4, 10, -1, 2), (1, 4, 10, 4, -1)]:
        assert size(*bad) == 0
    assert size(2, 4, 100, 6, 4) > 256 + 6 * 4 * 512 - 1
    assert size(0, 4, 0, 0, 0) >= 256


def test_cand_kv4_workspace_serves_smaller_calls(pa):
    """The size of a call is never above that of a call with larger sizes."""
    import random
    size = pa.load_library().hstu_cand_kv4_workspace_size
    rng = random.Random(1)
    for _ in range(4000):
        H = rng.randint(1, 16)
        m = int(2 ** rng.uniform(0, 10))
        big = [int(2 ** rng.uniform(0, 9)), H, int(2 ** rng.uniform(0, 14)), 0, m]
        big[3] = rng.randint(1, big[0] * m)
        small = [rng.randint(0, big[0]), H, rng.randint(0, big[2]), rng.randint(0, big[3]),
                 rng.randint(0, m)]
        assert size(*small) <= size(*big), (small, big)


def buckets_by_formula(nb, exact, far, d):
    """bucket(d) in rational arithmetic: the largest k with
    d^n >= exact^(n-j) far^j, j = k - exact."""
    if d < exact:
        return min(d, nb - 1)
    n = nb - exact
    k = exact
    while k < nb - 1 and d ** n >= exact ** (n - (k + 1 - exact)) * far ** (k + 1 - exact):
        k += 1
    return min(k, nb - 1)


@pytest.mark.parametrize("nb,exact,far", [(1, 1, 5), (2, 1, 2), (32, 16, 128), (32, 16, 4096),
                                          (64, 32, 65536), (128, 1, 2 ** 31 - 1), (7, 7, 0),
                                          (10, 8, 9), (128, 64, 65)])
def test_pos_bucket_thresholds(pa, nb, exact, far):
    thr = pa.hstu_pos_bucket_thresholds(nb, exact, far).tolist()
    assert len(thr) == nb - 1 and thr == sorted(thr)
    probe = sorted({x + e for x in thr for e in (-1, 0, 1)} | {0, 1, exact, max(far, 1)})
    for d in probe:
        if 0 <= d < 2 ** 31:
            assert sum(t <= d for t in thr) == buckets_by_formula(nb, exact, far, d), d


@pytest.mark.parametrize("args", [(0, 1, 5), (129, 1, 5), (8, 0, 5), (8, 9, 5), (8, 4, 4)])
def test_pos_bucket_thresholds_refusals(pa, args):
    with pytest.raises(pa.HSTUError):
        pa.hstu_pos_bucket_thresholds(*args)


def test_host_tensors_are_refused(pa):
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        pa.hstu_rmsnorm_fwd(x)
    with pytest.raises(ValueError):
        pa.hstu_quant_rows(x)
    with pytest.raises(ValueError):
        pa.hstu_rab_bucket_fwd(x, 10, torch.arange(1, 64, dtype=torch.int32))
    with pytest.raises(ValueError):
        pa.hstu_kv4_pack(x, x)


def test_thresholds_of_the_logarithmic_formula_agree_with_floating_point(pa):
    """Away from borders the floating-point form gives the same buckets."""
    thr = pa.hstu_pos_bucket_thresholds(32, 16, 4096).tolist()
    for d in range(16, 6000, 7):
        x = math.log(d / 16) / math.log(4096 / 16) * 16
        if abs(x - round(x)) > 1e-6:
            assert sum(t <= d for t in thr) == min(31, 16 + math.floor(x))
