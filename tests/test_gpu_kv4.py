"""GPU tests of the 4-bit history cache and of candidate scoring against it.

The cache's contents are compared bit by bit with the definition in 64 bits.
Scoring is compared with the formula in 64 bits over the values that the cache
holds; the tolerance follows the roundings: every attention weight is rounded
to bf16 once (half a step, 2^-8 of its value), the rest is fp32, the output is
rounded to bf16.  With more than 16 candidates a user the weight is
x/2 (1 + tanh(x/2)) with the hardware's tanh, whose documented relative error
is 2^-11: |x|/2 2^-11 more.
"""
import pytest
import torch

import pointwise_attention_b200 as pa

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16 = torch.bfloat16


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rnd(seed, *shape, std=1.0):
    return (std * torch.randn(*shape, generator=gen(seed))).to(BF16).to(DEV)


def groups64(x):
    """Whole numbers and scales of the definition, in 64 bits."""
    g = x.double().unflatten(-1, (4, 32))
    top = g.abs().amax(-1).clamp_min(2.0 ** -100) / 7.0
    e = torch.floor(torch.log2(top)) - 4.0
    s = torch.ceil(top / torch.exp2(e)) * torch.exp2(e)
    return torch.round(g / s[..., None]), s


def codes64(n):
    """Bytes of the cache from whole numbers [.., 4, 32]."""
    c = (n + 8).to(torch.int64).flatten(-2).unflatten(-1, (16, 8))
    word = sum(c[..., i] << (4 * (i // 2) + 16 * (i % 2)) for i in range(8))
    return torch.stack([(word >> (8 * b)) & 255 for b in range(4)], -1).flatten(-2).to(torch.uint8)


@pytest.mark.parametrize("T,H", [(1, 1), (5, 3), (33, 8), (1000, 2), (7, 16)])
def test_pack_and_unpack(T, H):
    k, v = rnd(T, T, H, 128), rnd(T + 1, T, H, 128, std=30.0)
    k[0, 0, :32] = 0.0
    k[T // 2, 0, 40] = 200.0
    v[0, H - 1, 64:96] *= 2.0 ** -120          # below the floor of the scale
    # quotients that are ties: 7 s = 7 * 17, odd multiples of s / 2
    v[T - 1, 0, :32] = 8.5 * torch.arange(-14, 18, device=DEV).clamp(-14, 14).to(BF16)
    cache = pa.hstu_kv4_pack(k, v)
    for x, codes, scales in ((k, cache[0], cache[1]), (v, cache[2], cache[3])):
        n, s = groups64(x)
        assert torch.equal(scales.double(), s)
        assert torch.equal(codes, codes64(n))
    kk, vv = pa.hstu_kv4_unpack(cache)
    for x, got in ((k, kk), (v, vv)):
        n, s = groups64(x)
        assert torch.equal(got.double(), (n * s[..., None]).flatten(-2))
        # half a step of a scale that is at most 17/16 of max / 7
        top = x.double().unflatten(-1, (4, 32)).abs().amax(-1, keepdim=True).clamp_min(2.0 ** -100)
        err = (got.double() - x.double()).abs().unflatten(-1, (4, 32))
        assert bool((err <= top / 7 * 17 / 32).all())


def test_every_maximum():
    """Groups whose largest magnitude runs through all 32640 finite bf16
    numbers: scales and codes are the definition's, ties among them."""
    bits = torch.arange(0x7F80, dtype=torch.int32).to(torch.int16)
    top = bits.view(BF16).to(DEV).view(4080, 2, 4, 1)
    f = torch.cat([torch.tensor([1.0, -0.5, 0.25, -0.125]), 2 * torch.rand(28, generator=gen(1)) - 1])
    x = (top.double() * f.double().to(DEV)).to(BF16).flatten(2)
    cache = pa.hstu_kv4_pack(x, -x)
    n, s = groups64(x)
    assert torch.equal(cache[1].double(), s) and torch.equal(cache[3].double(), s)
    assert torch.equal(cache[0], codes64(n)) and torch.equal(cache[2], codes64(-n))


def test_rows_holes_and_bad_rows():
    R, H = 50, 4
    cache = pa.hstu_kv4_cache(R, H, DEV)
    k, v = rnd(1, 10, H, 128), rnd(2, 10, H, 128)
    rows = torch.tensor([49, 3, -1, 0, 17, 21, 22, 23, -1, 30], dtype=torch.int32, device=DEV)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    pa.hstu_kv4_pack(k, v, cache=cache, rows=rows, workspace=ws)
    assert pa.hstu_attn_check(ws) == 0
    kk, vv = pa.hstu_kv4_unpack(cache)
    want = pa.hstu_kv4_unpack(pa.hstu_kv4_pack(k, v))
    live = rows >= 0
    at = rows[live].long()
    assert torch.equal(kk[at], want[0][live]) and torch.equal(vv[at], want[1][live])
    rest = torch.ones(R, dtype=torch.bool, device=DEV)
    rest[at] = False
    assert bool((kk[rest] == 0).all()) and bool((cache[0][rest] == 0x88).all())
    out = (torch.full((10, H, 128), 5.0, dtype=BF16, device=DEV),
           torch.full((10, H, 128), 5.0, dtype=BF16, device=DEV))
    pa.hstu_kv4_unpack(cache, rows=rows, out=out, workspace=ws)
    assert torch.equal(out[0][live], want[0][live]) and bool((out[1][~live] == 5.0).all())
    assert pa.hstu_attn_check(ws) == 0
    before = [t.clone() for t in cache]
    bad = torch.full((10,), R, dtype=torch.int32, device=DEV)
    bad[4] = -7
    pa.hstu_kv4_pack(k, v, cache=cache, rows=bad, workspace=ws)
    assert pa.hstu_attn_check(ws) == pa._binding.HSTU_ERR_INVALID_ARG
    assert all(torch.equal(a, b) for a, b in zip(before, cache))


def test_keys_off_32_bytes():
    """k, v and the tensors read into on 16 bytes, not 32."""
    T, H = 19, 3
    k, v = rnd(1, T, H, 128), rnd(2, T, H, 128)
    want = pa.hstu_kv4_pack(k, v)
    off = lambda t: torch.cat([t.new_zeros(8), t.flatten()])[8:].view(t.shape)
    got = pa.hstu_kv4_pack(off(k), off(v))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    out = (off(torch.zeros_like(k)), off(torch.zeros_like(v)))
    pa.hstu_kv4_unpack(got, out=out)
    assert all(torch.equal(a, b) for a, b in zip(out, pa.hstu_kv4_unpack(want)))


@pytest.mark.parametrize("T,H", [(4001, 3), (9473, 1), (1700, 8)])
def test_long_calls_are_the_calls_of_their_parts(T, H):
    """Calls that fill the GPU against calls of a few tokens, bit for bit:
    packed in order, packed to rows in another order with holes, read back."""
    k, v = rnd(7, T, H, 128, std=3.0), rnd(8, T, H, 128)
    parts = [pa.hstu_kv4_pack(k[i:i + 500].contiguous(), v[i:i + 500].contiguous())
             for i in range(0, T, 500)]
    want = [torch.cat(t) for t in zip(*parts)]
    got = pa.hstu_kv4_pack(k, v)
    assert all(torch.equal(a, b) for a, b in zip(got, want))

    R = T + 77
    rows = torch.randperm(R, generator=torch.Generator().manual_seed(9))[:T].int().cuda()
    rows[::5] = -1
    live = rows >= 0
    cache = [torch.full((R, *t.shape[1:]), 3, dtype=t.dtype, device="cuda") for t in want]
    expect = [t.clone() for t in cache]
    for e, w in zip(expect, want):
        e[rows[live].long()] = w[live]
    pa.hstu_kv4_pack(k, v, cache=cache, rows=rows)
    assert all(torch.equal(a, b) for a, b in zip(cache, expect))

    out = (torch.full_like(k, 5.0), torch.full_like(v, 5.0))
    pa.hstu_kv4_unpack(cache, rows=rows, out=out)
    whole = pa.hstu_kv4_unpack(want)
    for o, w in zip(out, whole):
        assert torch.equal(o[live], w[live])
        assert bool((o[~live] == 5.0).all())


def test_infinities_and_nan_stay_in_their_group():
    k, v = rnd(1, 4, 2, 128), rnd(2, 4, 2, 128)
    clean = pa.hstu_kv4_unpack(pa.hstu_kv4_pack(k, v))
    k[1, 0, 5], v[2, 1, 127] = float("nan"), float("-inf")
    kk, vv = pa.hstu_kv4_unpack(pa.hstu_kv4_pack(k, v))
    assert torch.isnan(kk[1, 0, :32]).all() and torch.isnan(vv[2, 1, 96:]).all()
    kk[1, 0, :32], vv[2, 1, 96:] = clean[0][1, 0, :32], clean[1][2, 1, 96:]
    assert torch.equal(kk, clean[0]) and torch.equal(vv, clean[1])


# ------------------------------------------------------------------ scoring
class Case:
    """Histories in a cache, candidates and tables."""

    def __init__(self, seed, lens, cands, H, pos=True, time=True, affine=False, norm_len=0,
                 scattered=False, L=None, nb=128, wide=False):
        g = gen(seed)
        self.lens, self.cands, self.H, self.norm_len = lens, cands, H, norm_len
        B = len(lens)
        off = [0]
        coff = [0]
        for n, m in zip(lens, cands):
            off.append(off[-1] + n)
            coff.append(coff[-1] + m)
        self.off, self.coff = off, coff
        T, C = off[-1], coff[-1]
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
        self.offsets, self.cand_offsets = i32(off), i32(coff)
        k, v = rnd(seed, T, H, 128, std=128 ** -0.5), rnd(seed + 1, T, H, 128)
        self.q, self.k = (rnd(seed + s, C, H, 128, std=128 ** -0.5) for s in (2, 3))
        self.v, self.u = rnd(seed + 4, C, H, 128), rnd(seed + 5, C, H * 128)
        self.first_rows = None
        if scattered:       # users in another order, with free rows between them
            first, at = [0] * B, 3
            for b in reversed(range(B)):
                first[b] = at
                at += lens[b] + 5
            self.first_rows = i32(first)
            self.cache = pa.hstu_kv4_cache(at, H, DEV)
            rows = torch.cat([torch.arange(n) + f for n, f in zip(lens, first)] +
                             [torch.zeros(0, dtype=torch.int64)])
            pa.hstu_kv4_pack(k, v, cache=self.cache, rows=rows.to(torch.int32).to(DEV))
        else:
            self.cache = pa.hstu_kv4_pack(k, v)
        self.hist = pa.hstu_kv4_unpack(pa.hstu_kv4_pack(k, v))
        self.L = max(lens + [0]) + 1 if L is None else L
        self.rab_pos = (0.5 * torch.randn(H, 2 * self.L - 1, generator=g)).to(DEV) if pos else None
        self.rab_time = (0.5 * torch.randn(H, nb, generator=g)).to(DEV) if time else None
        self.ts = self.cts = None
        if time:
            gaps = torch.randint(0, 2 ** 29 if wide else 5000, (T,), generator=g)
            self.ts = (1_600_000_000 + torch.cumsum(gaps, 0)).to(DEV)
            cts = []
            for b in range(B):
                last = int(self.ts[off[b + 1] - 1]) if lens[b] else 1_600_000_000
                cts.append(last + torch.randint(-50, 90000, (cands[b],), generator=g))
            self.cts = torch.cat(cts).to(DEV)
        self.ln_weight = (1 + 0.2 * torch.randn(H * 128, generator=g)).to(DEV) if affine else None
        self.ln_bias = (0.2 * torch.randn(H * 128, generator=g)).to(DEV) if affine else None

    def call(self, max_len=None, max_cands=None, **kw):
        return pa.hstu_cand_kv4_fwd(
            self.cache, self.offsets, max(self.lens + [0]) if max_len is None else max_len, self.q,
            self.k, self.v, self.u, self.cand_offsets,
            max(self.cands + [0]) if max_cands is None else max_cands, first_rows=self.first_rows,
            timestamps=self.ts, cand_timestamps=self.cts, rab_pos=self.rab_pos,
            rab_time=self.rab_time, norm_len=self.norm_len, ln_weight=self.ln_weight,
            ln_bias=self.ln_bias, **kw)

    def reference(self, eps=1e-5):
        """(y, tolerance) in 64 bits."""
        H, d = self.H, torch.float64
        thr = torch.from_numpy(pa.hstu_time_bucket_thresholds(
            128 if self.rab_time is None else max(self.rab_time.shape[1], 2))).to(DEV)
        if self.rab_time is not None and self.rab_time.shape[1] == 1:
            thr = thr[:0]
        ys, tols = [], []
        silu = lambda x: x / (1.0 + torch.exp(-x))
        for b in range(len(self.lens)):
            s, e, c0, c1 = self.off[b], self.off[b + 1], self.coff[b], self.coff[b + 1]
            n = e - s
            if c0 == c1:
                continue
            q, k, v = (t[c0:c1].to(d).transpose(0, 1) for t in (self.q, self.k, self.v))
            kh, vh = (t[s:e].to(d).transpose(0, 1) for t in self.hist)
            x = q @ kh.transpose(1, 2)                       # [H, m, n]
            mag = q.abs() @ kh.abs().transpose(1, 2)
            x0 = (q * k).sum(-1)
            if self.rab_pos is not None:
                x = x + self.rab_pos.to(d)[:, None, [self.L - 1 + n - j for j in range(n)]]
                x0 = x0 + self.rab_pos.to(d)[:, self.L - 1:self.L]
            if self.rab_time is not None:
                dt = (self.cts[c0:c1, None] - self.ts[None, s:e]).abs().clamp_min(1)
                x = x + self.rab_time.to(d)[:, torch.searchsorted(thr, dt, right=True)]
                x0 = x0 + self.rab_time.to(d)[:, :1]
            a, a0 = silu(x), silu(x0)
            N = self.norm_len if self.norm_len > 0 else n + 1
            o = (a @ vh + a0[..., None] * v) / N
            # a weight: half a bf16 step of its value, 1.1 times the fp32 error
            # of its score, 2^-20 for the exponential and the quotient; a sum of
            # n terms in fp32
            da = a.abs() * (2.0 ** -8 + 2.0 ** -20) + 1.1 * (mag + x.abs() + 1) * 132 * 2.0 ** -24
            if max(self.cands) > 16:
                da = da + x.abs() * 2.0 ** -12
            do = (da @ vh.abs() + (a.abs() @ vh.abs()) * (n + 8) * 2.0 ** -24 +
                  (a0.abs() + 1)[..., None] * v.abs() * 2.0 ** -16) / N
            o, do = (t.transpose(0, 1).flatten(1) for t in (o, do))
            mean = o.mean(1, keepdim=True)
            r = 1.0 / torch.sqrt(((o - mean) ** 2).mean(1, keepdim=True) + eps)
            xh = (o - mean) * r
            # first order of the LayerNorm, five per cent for the rest of it
            dx = 1.05 * r * (do + do.mean(1, keepdim=True) +
                             xh.abs() * (xh.abs() * do).mean(1, keepdim=True)) + xh.abs() * 2.0 ** -16
            gate = silu(self.u[c0:c1].to(d))
            w = 1.0 if self.ln_weight is None else self.ln_weight.to(d)
            y = xh * w + (0.0 if self.ln_bias is None else self.ln_bias.to(d))
            dx = dx * (w if isinstance(w, float) else w.abs())
            y, tol = y * gate, dx * gate.abs()
            ys.append(y)
            tols.append(tol + y.abs() * (2.0 ** -8 + 2.0 ** -16) + 1e-30)
        return torch.cat(ys), torch.cat(tols)


def check(c, y):
    ref, tol = c.reference()
    assert y.shape == ref.shape and torch.isfinite(y).all()
    err = (y.double() - ref).abs()
    assert bool((err <= tol).all()), "off by %.3e, %.2f times the tolerance" % (
        float(err.max()), float((err / tol).max()))


SCORING = [
    # lengths, candidates, heads
    ((5,), (1,), 1), ((0,), (3,), 2), ((16,), (8,), 1), ((17, 0, 1), (9, 2, 1), 3),
    ((300, 40), (1, 1), 8), ((129, 1000), (16, 3), 4), ((700,), (17,), 16), ((64, 33), (0, 7), 5),
    ((2000, 513, 90), (1, 2, 1), 8), ((31, 32, 33, 0), (40, 130, 1, 5), 2), ((257,), (300,), 9),
    ((1500,), (129,), 4), ((128, 256, 127), (128, 256, 33), 8)]


@pytest.mark.parametrize("pos,time", [(True, True), (True, False), (False, True), (False, False)])
@pytest.mark.parametrize("lens,cands,H", SCORING)
def test_scoring(lens, cands, H, pos, time):
    c = Case(sum(lens) + H, list(lens), list(cands), H, pos=pos, time=time)
    ws = pa.hstu_cand_kv4_workspace(len(lens), H, max(lens), sum(cands), max(cands), DEV)
    y = c.call(workspace=ws)
    assert pa.hstu_attn_check(ws) == 0
    check(c, y)


@pytest.mark.parametrize("kw", [
    dict(affine=True), dict(norm_len=700), dict(scattered=True), dict(L=900), dict(nb=1),
    dict(nb=20), dict(wide=True), dict(scattered=True, time=False)])
@pytest.mark.parametrize("cands", [(1, 2, 0), (30, 200, 7)])
def test_scoring_variants(kw, cands):
    c = Case(3, [400, 61, 150], list(cands), 4, **kw)
    check(c, c.call())
    check(c, c.call(max_len=min(c.L - 1, 777), max_cands=max(cands) + 90))


@pytest.mark.parametrize("B,most,cands", [(700, 20, 2), (300, 70, 1), (600, 40, 20), (120, 300, 200)])
def test_many_users(B, most, cands):
    """More users than a block has threads, than are ranked by length, and than
    there are CTAs (one or two tiles of candidates each); empty histories and
    users without candidates among them."""
    g = gen(B)
    lens = torch.randint(0, most + 1, (B,), generator=g).tolist()
    m = torch.randint(0, cands + 1, (B,), generator=g).tolist()
    m[0] = cands
    c = Case(B, lens, m, 4 if B == 120 else 2, time=B in (300, 120))
    check(c, c.call())


@pytest.mark.parametrize("cands", [(5, 2), (90, 170)])
def test_timestamps_in_any_order(cands):
    """Histories whose timestamps do not ascend, candidates before, among and
    after them: every bucket is looked up by itself."""
    c = Case(21, [333, 260], list(cands), 4)
    for s, e in ((0, 333), (333, 593)):
        c.ts[s:e] = c.ts[s:e][torch.randperm(e - s, generator=gen(2)).to(DEV)]
    c.cts -= torch.randint(0, 2_000_000, (sum(cands),), generator=gen(3)).to(DEV)
    check(c, c.call())


def test_users_share_rows():
    """Two users over the same cache rows score as two copies would."""
    c = Case(8, [200, 200], [3, 5], 4, time=False)
    c.first_rows = torch.zeros(2, dtype=torch.int32, device=DEV)
    c.hist = tuple(torch.cat([t[:200], t[:200]]) for t in c.hist)
    check(c, c.call())


def test_a_candidate_depends_on_itself_alone():
    """Changing one candidate leaves the others bitwise unchanged; two runs are
    bitwise equal; rows past the last candidate stay as they were."""
    for m in (5, 150):
        c = Case(9, [333, 50], [m, 2], 8)
        y = c.call()
        assert torch.equal(y, c.call())
        c.q[1] = -c.q[1]
        y2 = c.call()
        assert not torch.equal(y2[1], y[1])
        y2[1] = y[1]
        assert torch.equal(y, y2)
        off = c.cand_offsets.clone()
        off[-1] -= 1                    # one candidate fewer: its row belongs to nobody
        c.cand_offsets = off
        buf = torch.full_like(y, 3.0)
        c.call(y=buf)
        assert bool((buf[-1] == 3.0).all()) and torch.isfinite(buf).all()


def test_bad_ranges_are_reported_and_nothing_is_written():
    for what in ("offsets", "cands", "rows"):
        c = Case(10, [50, 60], [4, 40], 2, scattered=what == "rows")
        ws = pa.hstu_cand_kv4_workspace(2, 2, 60, 44, 40, DEV)
        ok = c.call(workspace=ws)
        assert pa.hstu_attn_check(ws) == 0
        if what == "offsets":
            c.offsets = torch.tensor([0, 50, 300], dtype=torch.int32, device=DEV)
        elif what == "cands":
            c.cand_offsets = torch.tensor([0, 4, 1000], dtype=torch.int32, device=DEV)
        else:
            c.first_rows = c.first_rows.clone()
            c.first_rows[1] = c.cache[0].shape[0] - 59
        buf = torch.full_like(ok, 2.0)
        c.call(workspace=ws, y=buf)
        assert pa.hstu_attn_check(ws) == pa._binding.HSTU_ERR_INVALID_ARG
        assert torch.equal(buf[:4], ok[:4]) and bool((buf[4:] == 2.0).all()), what


def test_one_workspace_for_calls_of_different_sizes():
    big = Case(11, [900, 300, 20], [140, 3, 260], 8)
    small = Case(12, [40], [1], 8)
    ws = pa.hstu_cand_kv4_workspace(3, 8, 900, 403, 260, DEV)
    ws2 = pa.hstu_cand_kv4_workspace(1, 8, 40, 1, 1, DEV)
    if ws2.numel() > ws.numel():
        ws = ws2
    a, b = big.call(), small.call()
    for _ in range(2):
        assert torch.equal(big.call(workspace=ws), a)
        assert torch.equal(small.call(workspace=ws), b)
    assert pa.hstu_attn_check(ws) == 0


def test_two_graphs_share_a_workspace():
    """Two captured calls over one workspace, replayed in turn on new inputs."""
    cases = [Case(13, [600, 77], [1, 6], 8), Case(14, [400, 200], [130, 40], 8)]
    n = max(pa.hstu_cand_kv4_workspace(2, 8, max(c.lens), sum(c.cands), max(c.cands), DEV).numel()
            for c in cases)
    ws = torch.zeros(n, dtype=torch.uint8, device=DEV)
    graphs = []
    for c in cases:
        out = torch.zeros(sum(c.cands), 1024, dtype=BF16, device=DEV)
        c.call(workspace=ws, y=out)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.call(workspace=ws, y=out)
        graphs.append((g, c, out))
    for _ in range(2):
        for g, c, out in graphs:
            c.u.neg_()
            out.zero_()
            g.replay()
            torch.cuda.synchronize()
            check(c, out)
    assert pa.hstu_attn_check(ws) == 0


def test_two_streams_with_their_own_workspaces():
    cases = [Case(15, [1200] * 3, [1, 2, 3], 8), Case(16, [1000] * 3, [140, 5, 60], 8)]
    want = [c.call() for c in cases]
    torch.cuda.synchronize()
    outs = []
    for c in cases:
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            ws = pa.hstu_cand_kv4_workspace(3, 8, 1200, sum(c.cands), max(c.cands), DEV)
            outs.append([c.call(workspace=ws) for _ in range(4)])
    torch.cuda.synchronize()
    for w, ys in zip(want, outs):
        assert all(torch.equal(w, y) for y in ys)


@pytest.mark.parametrize("H", [3, 8])
@pytest.mark.parametrize("cands", [(2, 1, 3), (60, 20, 130)])
def test_free_rows_may_hold_anything(cands, H):
    """Cache rows between the users' hold NaN scales and any codes."""
    c = Case(23, [45, 130, 1], list(cands), H, scattered=True)
    used = torch.zeros(c.cache[0].shape[0], dtype=torch.bool, device=DEV)
    for first, n in zip(c.first_rows.tolist(), c.lens):
        used[first:first + n] = True
    for t in c.cache:
        t[~used] = float("nan") if t.dtype == BF16 else 255
    check(c, c.call())


@pytest.mark.parametrize("cands", [(2, 1), (60, 20)])
def test_lengths_far_below_the_bound(cands):
    """max_seq_len bounds the histories; here it is a thousand times theirs."""
    c = Case(22, [150, 77], list(cands), 2, pos=False)
    check(c, c.call(max_len=150_000))


def test_extreme_scores():
    """Biases at the type's lowest value give weight 0, also where they cover a
    whole history."""
    c = Case(17, [100, 30], [3, 40], 2, time=False)
    c.rab_pos[0, c.L - 1 + 20:] = torch.finfo(torch.float32).min
    c.rab_pos[1, c.L:] = -1e4
    y = c.call()
    keep = c.rab_pos.clone()
    c.rab_pos = keep.clamp_min(-1e4)        # the same weights: exactly 0 in 64 bits too
    check(c, y)


def test_no_candidates_and_no_histories():
    c = Case(18, [10, 0], [0, 0], 2)
    assert c.call(max_cands=0).shape == (0, 256)
    c = Case(19, [0, 0], [2, 0], 2)
    check(c, c.call())
