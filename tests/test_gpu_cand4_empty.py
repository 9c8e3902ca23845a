"""GPU tests of scoring against the 4-bit cache with nothing in one of its
places: no users, no cache rows, tensors longer than what they hold."""
import pytest
import torch

import pointwise_attention_b200 as pa

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16 = torch.bfloat16
H = 4


def rnd(seed, *shape, std=1.0):
    return (std * torch.randn(*shape, generator=torch.Generator().manual_seed(seed))).to(BF16).to(DEV)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def candidates(C):
    return (rnd(3, C, H, 128, std=128 ** -0.5), rnd(4, C, H, 128, std=128 ** -0.5),
            rnd(5, C, H, 128), rnd(6, C, H * 128))


@pytest.mark.parametrize("slots", [False, True])
@pytest.mark.parametrize("time", [False, True])
def test_no_users(slots, time):
    """An empty batch over a cache that holds rows: an empty result."""
    cache = pa.hstu_kv4_pack(rnd(1, 50, H, 128), rnd(2, 50, H, 128))
    none = torch.zeros(0, dtype=torch.int64, device=DEV)
    kw = dict(timestamps=none, cand_timestamps=none, rab_time=torch.zeros(H, 8, device=DEV)) if time else {}
    y = pa.hstu_cand_kv4_fwd(cache, i32([0]), 40, *candidates(0), i32([0]), 0,
                             first_rows=i32([]) if slots else None, **kw)
    assert y.shape == (0, H * 128)


@pytest.mark.parametrize("slots", [False, True])
@pytest.mark.parametrize("cands", [[2, 0, 3], [30, 0, 20]])
def test_a_cache_without_rows(cands, slots):
    """Users that are all new: each candidate sees itself alone, as against a
    cache that has rows; a history in such a cache is reported."""
    C = sum(cands)
    coff = i32([0, cands[0], cands[0], C])
    rab = torch.randn(H, 21, generator=torch.Generator().manual_seed(9)).to(DEV)
    kw = dict(first_rows=i32([0, 0, 0]) if slots else None, rab_pos=rab)
    full = pa.hstu_kv4_pack(rnd(1, 8, H, 128), rnd(2, 8, H, 128))
    args = (*candidates(C), coff, max(cands))
    want = pa.hstu_cand_kv4_fwd(full, i32([0, 0, 0, 0]), 10, *args, **kw)
    empty = pa.hstu_kv4_cache(0, H, DEV)
    assert torch.equal(pa.hstu_cand_kv4_fwd(empty, i32([0, 0, 0, 0]), 10, *args, **kw), want)
    ws = pa.hstu_cand_kv4_workspace(3, H, 10, C, max(cands), DEV)
    pa.hstu_cand_kv4_fwd(empty, i32([0, 5, 5, 5]), 10, *args, workspace=ws, **kw)
    assert pa.hstu_attn_check(ws) == pa._binding.HSTU_ERR_INVALID_ARG


def test_timestamps_longer_than_the_cache():
    """A timestamp buffer of a fixed size over a cache of the batch's rows."""
    cache = pa.hstu_kv4_pack(rnd(1, 60, H, 128), rnd(2, 60, H, 128))
    ts = 1_700_000_000 + 100 * torch.arange(200, device=DEV)
    rab = torch.randn(H, 128, generator=torch.Generator().manual_seed(9)).to(DEV)
    args = (cache, i32([0, 25, 60]), 40, *candidates(7), i32([0, 3, 7]), 4)
    kw = dict(cand_timestamps=ts[60:67].clone(), rab_time=rab)
    want = pa.hstu_cand_kv4_fwd(*args, timestamps=ts[:60].clone(), **kw)
    assert torch.equal(pa.hstu_cand_kv4_fwd(*args, timestamps=ts, **kw), want)
