"""GPU tests of scoring against the 4-bit cache from candidate buffers of a
fixed size, of which a call fills a part: the rows of nobody cost nothing and
change nothing, and the sums stay in the workspace that the size query gives."""
import os
import subprocess
import sys

import pytest
import torch

import pointwise_attention_b200 as pa

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16 = torch.bfloat16
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def rnd(seed, *shape, std=1.0):
    return (std * torch.randn(*shape, generator=torch.Generator().manual_seed(seed))).to(BF16).to(DEV)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Served:
    """Histories in a cache and a buffer of `room` candidates, of which those
    from `first` on are the users'."""

    def __init__(self, lens, cands, H, room, first=0, time=True):
        self.lens, self.cands, self.H, self.room, self.time = lens, cands, H, room, time
        T = sum(lens)
        self.cache = pa.hstu_kv4_pack(rnd(1, T, H, 128, std=128 ** -0.5), rnd(2, T, H, 128))
        self.off = i32([sum(lens[:b]) for b in range(len(lens) + 1)])
        self.coff = [first + sum(cands[:b]) for b in range(len(cands) + 1)]
        self.q, self.k = (rnd(s, room, H, 128, std=128 ** -0.5) for s in (3, 4))
        self.v, self.u = rnd(5, room, H, 128), rnd(6, room, H * 128)
        g = torch.Generator().manual_seed(7)
        self.rab_pos = (0.3 * torch.randn(H, 2 * max(lens) + 1, generator=g)).to(DEV)
        self.ts = self.cts = self.rab_time = None
        if time:
            self.ts = 1_700_000_000 + torch.cumsum(torch.randint(0, 900, (T,), generator=g), 0).to(DEV)
            self.cts = 1_700_000_000 + 450 * T + torch.randint(0, 90000, (room,), generator=g).to(DEV)
            self.rab_time = (0.3 * torch.randn(H, 128, generator=g)).to(DEV)

    def call(self, lo=0, hi=None, coff=None, workspace=None, y=None):
        s = slice(lo, hi)
        coff = [c - lo for c in self.coff] if coff is None else coff
        cut = lambda t: None if t is None else t[s].contiguous()
        return pa.hstu_cand_kv4_fwd(
            self.cache, self.off, max(self.lens), cut(self.q), cut(self.k), cut(self.v),
            cut(self.u), i32(coff), max(self.cands), timestamps=self.ts,
            cand_timestamps=cut(self.cts), rab_pos=self.rab_pos, rab_time=self.rab_time,
            workspace=workspace, y=y)

    def guarded(self):
        """A workspace of exactly the queried size with known bytes behind it."""
        n = pa.hstu_cand_kv4_workspace(len(self.lens), self.H, max(self.lens), self.room,
                                       max(self.cands), DEV).numel()
        whole = torch.full((n + (8 << 20),), 0xA5, dtype=torch.uint8, device=DEV)
        whole[:n] = 0
        return whole[:n], whole[n:]


@pytest.mark.parametrize("lens,cands,H,room,first", [
    ([4096], [32], 8, 1024, 0), ([4096], [32], 8, 1024, 600), ([3000], [17], 1, 4000, 1),
    ([2500, 900], [40, 3], 4, 900, 5), ([700, 0, 90], [5, 0, 2], 8, 300, 100)])
@pytest.mark.parametrize("time", [True, False])
def test_padded_candidate_buffers(lens, cands, H, room, first, time):
    c = Served(lens, cands, H, room, first, time)
    lo, hi = c.coff[0], c.coff[-1]
    want = c.call(lo, hi)                       # the users' candidates alone
    ws, behind = c.guarded()
    y = torch.full((room, H * 128), 3.0, dtype=BF16, device=DEV)
    c.call(workspace=ws, y=y)
    assert pa.hstu_attn_check(ws) == 0
    assert torch.equal(y[lo:hi], want)          # the same cut, the same sums
    assert bool((y[:lo] == 3.0).all()) and bool((y[hi:] == 3.0).all())
    assert bool((behind == 0xA5).all())


def test_ranges_past_the_sums_are_reported():
    """A user with more candidates than max_cands puts the next one's past the
    rows of the sums: reported, and neither is written."""
    c = Served([2000, 1500], [20, 20], 4, 3000)
    ok = c.call(0, 40)
    ws, behind = c.guarded()
    y = torch.full((3000, 512), 3.0, dtype=BF16, device=DEV)
    c.call(coff=[0, 2900, 2920], workspace=ws, y=y)
    assert pa.hstu_attn_check(ws) == pa._binding.HSTU_ERR_INVALID_ARG
    assert bool((y == 3.0).all()) and bool((behind == 0xA5).all())
    c.call(workspace=ws, y=y)
    assert pa.hstu_attn_check(ws) == 0
    assert torch.equal(y[:40], ok) and bool((y[40:] == 3.0).all())


def test_padded_buffers_with_device_index_checks():
    """The same under the build that checks every index of the sums."""
    sys.path.insert(0, ROOT)
    from pointwise_attention_b200 import build
    build.build(debug_bounds=True)
    r = subprocess.run(
        [sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider",
         "tests/test_gpu_cand4_buffers.py", "-k", "candidate_buffers or past_the_sums"],
        cwd=ROOT, env=dict(os.environ, HSTU_DEBUG_BOUNDS="1"), capture_output=True, text=True,
        timeout=600)
    tail = "\n".join((r.stdout + r.stderr).splitlines()[-30:])
    assert r.returncode == 0, tail
    assert " passed" in tail and "failed" not in tail, tail
