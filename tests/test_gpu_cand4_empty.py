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
