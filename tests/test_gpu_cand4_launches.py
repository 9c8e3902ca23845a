"""GPU tests of scoring against the 4-bit cache as the chain of kernels that it
is: calls one behind another on one workspace, each of which starts its kernels
beside the ones before."""
import pytest
import torch

import pointwise_attention_b200 as pa

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16 = torch.bfloat16


def rnd(seed, *shape, std=1.0):
    return (std * torch.randn(*shape, generator=torch.Generator().manual_seed(seed))).to(BF16).to(DEV)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Batch:
    """Users of equal histories and candidates, time plans of their own."""

    def __init__(self, seed, B, n, m, H):
        g = torch.Generator().manual_seed(seed)
        self.B, self.n, self.m, self.H = B, n, m, H
        T, C = B * n, B * m
        self.cache = pa.hstu_kv4_pack(rnd(seed, T, H, 128, std=128 ** -0.5), rnd(seed + 1, T, H, 128))
        self.off, self.coff = i32([n * b for b in range(B + 1)]), i32([m * b for b in range(B + 1)])
        self.first = self.off[:-1].clone()
        self.q, self.k = (rnd(seed + s, C, H, 128, std=128 ** -0.5) for s in (2, 3))
        self.v, self.u = rnd(seed + 4, C, H, 128), rnd(seed + 5, C, H * 128)
        step = int(torch.randint(1, 4000, (1,), generator=g))
        self.ts = 1_700_000_000 + torch.cumsum(torch.randint(0, step, (T,), generator=g), 0).to(DEV)
        self.cts = int(self.ts[-1]) + torch.randint(0, 90000, (C,), generator=g).to(DEV)
        self.rab_time = torch.randn(H, 128, generator=g).to(DEV)

    def call(self, ws, first=None):
        return pa.hstu_cand_kv4_fwd(self.cache, self.off, self.n, self.q, self.k, self.v, self.u,
                                    self.coff, self.m, first_rows=self.first if first is None else first,
                                    total_tokens=self.B * self.n, timestamps=self.ts,
                                    cand_timestamps=self.cts, rab_time=self.rab_time, workspace=ws)

    def workspace(self):
        return pa.hstu_cand_kv4_workspace(self.B, self.H, self.n, self.B * self.m, self.m, DEV)


def test_time_plans_are_those_of_the_call():
    """Two batches in turn on one workspace, back to back: the plans and bucket
    bytes that a call reads are its own, not the ones before at their place."""
    a, b = Batch(1, 6, 700, 130, 4), Batch(11, 6, 700, 130, 4)
    want = [x.call(x.workspace()) for x in (a, b)]
    ws = a.workspace()
    torch.cuda.synchronize()
    got = [x.call(ws) for _ in range(10) for x in (a, b)]
    assert pa.hstu_attn_check(ws) == 0
    for i, y in enumerate(got):
        assert torch.equal(y, want[i % 2]), i


@pytest.mark.parametrize("m", [4, 130])
def test_a_call_behind_one_that_reports_every_user(m):
    """A call whose users all begin outside the cache writes nothing and is
    reported; the call behind it on the workspace is not touched by what its
    kernels still do."""
    bad, good = Batch(21, 8, 3000, m, 4), Batch(31, 8, 3000, m, 4)
    want = good.call(good.workspace())
    ws = good.workspace()
    nowhere = torch.full_like(bad.first, bad.cache[0].shape[0])
    torch.cuda.synchronize()
    for _ in range(20):
        bad.call(ws, first=nowhere)
        got = good.call(ws)
        assert pa.hstu_attn_check(ws) == pa._binding.HSTU_ERR_INVALID_ARG
        assert torch.equal(got, want)


@pytest.mark.parametrize("m", [4, 130])
def test_a_call_behind_one_without_candidates(m):
    """No user has a candidate: nothing is written, and the next call is whole."""
    none, good = Batch(41, 5, 2000, m, 4), Batch(51, 5, 2000, m, 4)
    want = good.call(good.workspace())
    ws = good.workspace()
    none.coff = torch.zeros_like(none.coff)
    torch.cuda.synchronize()
    for _ in range(20):
        none.call(ws)
        assert torch.equal(good.call(ws), want)
    assert pa.hstu_attn_check(ws) == 0
