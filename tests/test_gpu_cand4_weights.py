"""GPU tests of the attention weights of scoring against the 4-bit cache with up
to 16 candidates a user: they enter the sum as two bf16 parts, so that 2^-16 of
a weight is lost, not the 2^-8 of one bf16 number.

The histories are pairs of tokens with opposite values and scores a hundredth
apart: what is left of a pair is the small difference of its weights, and the
LayerNorm scales the rest up, so an error of the weights is as large beside the
result as it is beside that difference.
"""
import pytest
import torch

import pointwise_attention_b200 as pa

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16, F64 = torch.bfloat16, torch.float64
PAIRS, H = 16, 2


def silu(x):
    return x / (1.0 + torch.exp(-x))


class Pairs:
    def __init__(self, cands, time):
        g = torch.Generator().manual_seed(5)
        n, B, C = 2 * PAIRS, len(cands), sum(cands)
        self.cands = cands
        v = torch.randn(B, PAIRS, 1, H, 128, generator=g)
        v = torch.cat([v, -v], 2).reshape(B * n, H, 128).to(BF16).to(DEV)
        k = torch.zeros_like(v)                     # scores are the biases
        self.cache = pa.hstu_kv4_pack(k, v)
        self.v = pa.hstu_kv4_unpack(self.cache)[1].view(B, n, H, 128)
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
        self.off = i32([n * b for b in range(B + 1)])
        self.coff = i32([sum(cands[:b]) for b in range(B + 1)])
        b = 0.5 + 3.5 * torch.rand(H, PAIRS, 1, generator=g)
        d = 0.01 * torch.randn(H, PAIRS, 1, generator=g)
        self.bias = torch.cat([b, b + d], 2).flatten(1).to(DEV)        # of token j
        self.rab_pos = torch.zeros(H, 2 * n + 1, device=DEV)           # L = n + 1
        self.rab_pos[:, n + 1:] = self.bias.flip(1)
        self.q = torch.randn(C, H, 128, generator=g).to(BF16).to(DEV)
        self.k = torch.zeros_like(self.q)
        self.vc = torch.zeros_like(self.q)
        self.u = torch.randn(C, H * 128, generator=g).to(BF16).to(DEV)
        self.time = {}
        if time:      # every candidate and token in one bucket, whose bias all scores get
            self.rt = 0.2
            self.time = dict(timestamps=torch.zeros(B * n, dtype=torch.int64, device=DEV),
                             cand_timestamps=torch.full((C,), 5000, dtype=torch.int64, device=DEV),
                             rab_time=torch.full((H, 128), self.rt, device=DEV))

    def call(self):
        ws = pa.hstu_cand_kv4_workspace(len(self.cands), H, 2 * PAIRS, sum(self.cands),
                                        max(self.cands), DEV)
        y = pa.hstu_cand_kv4_fwd(self.cache, self.off, 2 * PAIRS, self.q, self.k, self.vc, self.u,
                                 self.coff, max(self.cands), rab_pos=self.rab_pos, norm_len=1,
                                 workspace=ws, **self.time)
        assert pa.hstu_attn_check(ws) == 0
        return y.double()

    def reference(self, weights=lambda a: a, eps=1e-5):
        """(y, tolerance) in 64 bits; ``weights`` makes mistakes of them."""
        ys, tols = [], []
        for b, m in enumerate(self.cands):
            x = self.bias.to(F64)
            if self.time:
                x = x + self.time["rab_time"][:, :1].to(F64)
            a, v = silu(x), self.v[b].to(F64).transpose(0, 1)          # [H, n], [H, n, 128]
            o = torch.einsum("hn,hnd->hd", weights(a), v).flatten()
            # a weight: its two parts, the exponential and the quotient, and two
            # roundings of its score; a sum of as many terms in fp32, twice
            da = a.abs() * (2.0 ** -16 + 2.0 ** -20) + 1.1 * x.abs() * 2.0 ** -23
            do = (torch.einsum("hn,hnd->hd", da, v.abs()) +
                  torch.einsum("hn,hnd->hd", a.abs(), v.abs()) * 2 * (2 * PAIRS + 8) * 2.0 ** -24).flatten()
            mean = o.mean()
            r = 1.0 / torch.sqrt(((o - mean) ** 2).mean() + eps)
            xh = (o - mean) * r
            # first order of the LayerNorm, a quarter more for the rest of it
            dx = 1.25 * r * (do + do.mean() + xh.abs() * (xh.abs() * do).mean()) + xh.abs() * 2.0 ** -16
            at = int(self.coff[b])
            gate = silu(self.u[at:at + m].to(F64))
            ys.append(xh * gate)
            tols.append(dx * gate.abs() + (xh * gate).abs() * (2.0 ** -8 + 2.0 ** -16) + 1e-30)
        return torch.cat(ys), torch.cat(tols)


def beyond(y, ref, tol):
    return float(((y - ref).abs() / tol).max())


@pytest.mark.parametrize("time", [False, True])
@pytest.mark.parametrize("cands", [[1], [3, 8, 1], [16, 2]])
def test_weights_keep_both_parts(cands, time):
    c = Pairs(cands, time)
    ref, tol = c.reference()
    y = c.call()
    assert torch.isfinite(y).all()
    assert beyond(y, ref, tol) <= 1.0
    # the test sees one part alone, and parts of neighbouring tokens exchanged
    high = lambda a: a.to(BF16).to(F64)
    assert beyond(c.reference(high)[0], ref, tol) > 2.0
    swapped = lambda a: high(a) + (a - high(a)).view(H, -1, 2).flip(2).flatten(1)
    assert beyond(c.reference(swapped)[0], ref, tol) > 2.0
