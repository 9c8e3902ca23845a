"""Cases, plain forms and 64-bit values of the operators around the attention.

Operators: the root-mean-square norm of a layer's input with the residual's
addition (forward, with an output in the input's type or in 8 bits with a scale
per row, and backward), row quantisation to 8 bits, the UVQK projection of
8-bit rows, the position-bias table made from learned buckets (forward and
backward), keys and values written to a cache of 4-bit values (and read back),
and candidate scoring against histories in such a cache.

``run`` computes an operator in plain torch (32 bits, one rounding at the end)
or, with ``own``, through the library's calls.
"""
import math

import torch

own = False

DEV = "cuda"
E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -100
EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one new event for each of eight users, ahead of a layer: latency
        dict(name="norm_events", op="norm", T=8, E=512, dtype="bf16", res=True, out="y"),
        # the packed tokens of a batch of histories, rows in 8 bits for the
        # projection, residual stream and statistics kept; ragged total
        dict(name="norm_batch_8bit", op="norm", T=131071, E=512, dtype="bf16", res=True, out="q8"),
        # the training workload's tokens, gradient of the residual stream added
        dict(name="norm_grad", op="norm_grad", T=32768, E=512, dtype="bf16", dres=True),
        # a width and a token count that no tile divides, in 32 bits
        dict(name="norm_grad_odd", op="norm_grad", T=4099, E=1001, dtype="f32", dres=False),
        # a layer's UVQK weight laid out for serving
        dict(name="quant_weight", op="quant", T=2048, E=512, dtype="f32"),
        # the projection of a batch of histories at the model card's block
        dict(name="uvqk_batch", op="uvqk", T=131072, E=512, H=4, dqk=128, dv=128, act=1),
        # the projection of a few candidates, more heads: latency
        dict(name="uvqk_events", op="uvqk", T=17, E=512, H=8, dqk=128, dv=128, act=1),
        # the position table of the long workload from 32 buckets a head
        dict(name="rab_table", op="rab", H=8, L=8192, buckets=32, exact=16, far=4096),
        # many heads over histories of a hundred thousand events
        # (the gradient that the attention's backward leaves for the table)
        dict(name="rab_grad_long", op="rab_grad", H=32, L=100003, buckets=64, exact=32, far=65536),
        # the histories of 32 users written to the cache, and read back
        dict(name="cache_histories", op="kv4", T=69637, H=8),
        # one event to score for each of 32 users
        dict(name="cand_events", op="cand4", B=32, H=8, least=256, most=4096, cands=1, pos=True,
             time=True),
        # the candidate-scoring workload: hundreds of candidates for each user
        dict(name="cand_batch", op="cand4", B=32, H=8, least=256, most=4096, cands=512, pos=True,
             time=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_grad", "quant", "uvqk", "uvqk", "rab", "rab_grad", "kv4",
                     "cand4", "cand4"])
    if op in ("norm", "norm_grad", "quant"):
        T = _log_int(rng, 1, 131072)
        E = min(_log_int(rng, 16, 8192), max(16, (1 << 26) // T))
        if rng.random() < 0.6:
            E = max(16, E // 16 * 16)
        dtype = "bf16" if rng.random() < 0.7 and T * E < (1 << 26) else "f32"
        if dtype == "f32":
            T = min(T, max(1, (1 << 25) // E))
        c = dict(op=op, T=T, E=E, dtype=dtype)
        if op == "norm":
            c.update(res=rng.random() < 0.7, out=rng.choice(["y", "q8"]))
        elif op == "norm_grad":
            c.update(dres=rng.random() < 0.7)
        return c
    if op == "uvqk":
        H, dqk, dv = rng.choice([(2, 128, 128), (4, 128, 128), (8, 128, 128), (4, 64, 128)])
        E = 16 * rng.randint(4, 64)
        most = int(131072 * 512 * 2048 / (E * 2 * H * (dqk + dv)))
        return dict(op="uvqk", T=_log_int(rng, 1, min(131072, most)), E=E, H=H, dqk=dqk, dv=dv,
                    act=rng.randint(0, 1))
    if op == "kv4":
        H = rng.choice([1, 2, 4, 8])
        return dict(op="kv4", T=_log_int(rng, 1, 500000 // H), H=H)
    if op == "cand4":
        most = _log_int(rng, 1, 8192)
        H = rng.choice([1, 2, 4, 8, 16])
        cands = _log_int(rng, 1, 300)
        B = _log_int(rng, 1, min(64, max(1, (1 << 28) // (most * H * (cands + 16)))))
        return dict(op="cand4", B=B, H=H, least=rng.choice([0, most // 2]), most=most, cands=cands,
                    pos=rng.random() < 0.7, time=rng.random() < 0.7)
    exact_ = rng.choice([1, 8, 16, 31])
    buckets = exact_ + rng.randint(1, 64)
    return dict(op=op, H=rng.choice([1, 4, 8, 24]), L=_log_int(rng, 1, 120000), buckets=buckets,
                exact=exact_, far=exact_ + _log_int(rng, 2, 65536))


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _rows(g, T, E, dtype):
    """Rows of a residual stream: normal values, a few wide channels, row
    magnitudes that differ by a small factor."""
    wide = 1.0 + 9.0 * (torch.rand(E, generator=g, device=DEV) < 0.02)
    size = torch.exp2(2.0 * torch.rand(T, 1, generator=g, device=DEV) - 1.0)
    return (_randn(g, T, E) * wide * size).to(dtype)


def _thresholds(buckets, exact_, far):
    """thr[k - 1] = the smallest distance of bucket k, from whole numbers."""
    thr = list(range(1, min(exact_, buckets - 1) + 1))
    n = buckets - exact_
    for j in range(1, n):
        bound = exact_ ** (n - j) * far ** j
        lo, hi = exact_, far
        while lo < hi:
            mid = (lo + hi) // 2
            if mid ** n >= bound:
                hi = mid
            else:
                lo = mid + 1
        thr.append(lo)
    return thr[:buckets - 1]


def _to_e4m3(v, scale):
    return (v / scale).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _bf16_scale(top):
    """Scale of a group of 4-bit values -7..7: the smallest number of five
    significant bits that is at least max / 7 (so that value times scale is a
    bf16 number)."""
    # (a quotient of two tensors: torch turns a number into its reciprocal)
    s = (top.clamp_min(AMAX_FLOOR) / torch.full_like(top, 7.0)).view(torch.int32)
    return ((s + 0x7FFFF) & ~0x7FFFF).view(torch.float32)


def _to_kv4(x):
    """[.., 128] -> whole numbers -7..7 as floats [.., 4, 32], scales [.., 4]."""
    g = x.float().unflatten(-1, (4, 32))
    sc = _bf16_scale(g.abs().amax(-1))
    return torch.round(g / sc[..., None]), sc


def _kv4_bytes(n):
    """Values [.., 4, 32] as the cache's bytes [.., 64]: eight values to a
    little-endian word, value 2i in bits 4i.., value 2i + 1 in bits 16 + 4i..,
    each plus 8."""
    c = (n + 8.0).to(torch.uint8).flatten(-2).unflatten(-1, (16, 8))
    lo = c[..., [0, 4, 1, 5]]
    hi = c[..., [2, 6, 3, 7]]
    return (lo | (hi << 4)).flatten(-2)


def _kv4_values(codes):
    """The cache's bytes [.., 64] as whole numbers -7..7 [.., 4, 32], floats."""
    c = codes.unflatten(-1, (16, 4))
    both = torch.stack([c & 15, c >> 4], dim=-1).flatten(-2)   # values 0 2 4 6 1 3 5 7
    return (both[..., [0, 4, 1, 5, 2, 6, 3, 7]].flatten(-2).float() - 8.0).unflatten(-1, (4, 32))


def _prepare_cand4(s, c, g):
    B, H = c["B"], c["H"]
    bf = torch.bfloat16
    draw_ = torch.rand(B, generator=g, device=DEV)
    lens = (c["least"] + draw_ * (c["most"] + 1 - c["least"])).long().clamp_max(c["most"]).tolist()
    # one user's candidates are a few more or fewer than another's, or none
    share = torch.rand(B, generator=g, device=DEV).tolist()
    cands = [c["cands"] if c["cands"] in (1, 512) else int(2 * c["cands"] * x) for x in share]
    cands[0] = max(cands[0], 1)
    off, coff = [0], [0]
    for n, m in zip(lens, cands):
        off.append(off[-1] + n)
        coff.append(coff[-1] + m)
    T, C = off[-1], coff[-1]
    s.update(max_len=max(lens), max_cands=max(cands), lens=lens)
    for n in ("k", "v"):
        std = 1.0 if n == "v" else 128 ** -0.5
        codes, sc = _to_kv4((std * _randn(g, T, H, 128)).to(bf))
        s[n + "_codes"], s[n + "_scales"] = _kv4_bytes(codes), sc.to(bf)
    s["q"] = (128 ** -0.5 * _randn(g, C, H, 128)).to(bf)
    s["k"] = (128 ** -0.5 * _randn(g, C, H, 128)).to(bf)
    s["v"] = _randn(g, C, H, 128).to(bf)
    s["u"] = _randn(g, C, H * 128).to(bf)
    s["offsets"] = torch.tensor(off, dtype=torch.int32, device=DEV)
    s["cand_offsets"] = torch.tensor(coff, dtype=torch.int32, device=DEV)
    # events minutes apart, candidates at request time
    gaps = (1.0 - 300.0 * torch.log1p(-torch.rand(T, generator=g, device=DEV))).long()
    run_ = torch.cumsum(gaps, 0)
    s["ts"] = s["cand_ts"] = s["rab_pos"] = s["rab_time"] = None
    if c["time"]:
        s["ts"] = 1_700_000_000 + run_
        ends = torch.tensor([x - 1 for x in off[1:]], device=DEV).clamp_min(0)
        last = s["ts"][ends] if T else torch.full((B,), 1_700_000_000, device=DEV)
        user = torch.repeat_interleave(torch.arange(B, device=DEV), torch.tensor(cands, device=DEV))
        s["cand_ts"] = last[user] + torch.randint(1, 90000, (C,), generator=g, device=DEV)
        s["rab_time"] = 0.02 * _randn(g, H, 128)
    if c["pos"]:
        s["rab_pos"] = 0.02 * _randn(g, H, 2 * (s["max_len"] + 1) - 1)
    if own:   # the scratch memory that a server keeps
        import pointwise_attention_b200 as pa
        s["workspace"] = pa.hstu_cand_kv4_workspace(B, H, s["max_len"], C, s["max_cands"], DEV)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = dict(case=case)
    if op in ("norm", "norm_grad", "quant"):
        T, E, dt = case["T"], case["E"], DTYPES[case["dtype"]]
        s["x"] = _rows(g, T, E, dt)
        s["w"] = 1.0 + 0.2 * _randn(g, E)
        if op == "norm":
            s["res"] = _rows(g, T, E, dt) if case["res"] else None
        elif op == "norm_grad":
            xf = s["x"].float()
            s["rstd"] = torch.rsqrt(xf.square().mean(1) + EPS)
            s["dy"] = (0.01 * _randn(g, T, E)).to(dt)
            s["dres"] = (0.01 * _randn(g, T, E)).to(dt) if case["dres"] else None
    elif op == "uvqk":
        T, E = case["T"], case["E"]
        N = 2 * case["H"] * (case["dqk"] + case["dv"])
        x, w = _randn(g, T, E), _randn(g, N, E) / math.sqrt(E)
        for n, t in (("x", x), ("w", w)):
            sc = t.abs().amax(1).clamp_min(AMAX_FLOOR) / E4M3_MAX
            s[n + "8"], s[n + "_scale"] = _to_e4m3(t, sc[:, None]), sc
        s["bias"] = 0.1 * _randn(g, N)
        s["status"] = torch.zeros(256, dtype=torch.uint8, device=DEV)
    elif op == "kv4":
        T, H = case["T"], case["H"]
        wide = torch.exp2(3.0 * torch.rand(H, 128, generator=g, device=DEV) - 1.5)
        s["k"] = (128 ** -0.5 * wide * _randn(g, T, H, 128)).to(torch.bfloat16)
        s["v"] = (wide * _randn(g, T, H, 128)).to(torch.bfloat16)
        s["status"] = torch.zeros(256, dtype=torch.uint8, device=DEV)
    elif op == "cand4":
        _prepare_cand4(s, case, g)
    else:
        H, L, B = case["H"], case["L"], case["buckets"]
        s["thr"] = torch.tensor(_thresholds(B, case["exact"], case["far"]), dtype=torch.int32)
        if op == "rab":
            s["table"] = 0.02 * _randn(g, H, B)
        else:
            s["d_rab"] = _randn(g, H, 2 * L - 1)
            s["d_rab"][:, :L - 1] = 0.0   # the attention's gradient of later keys
    return s


# ------------------------------------------------------------------ one pass
def _buckets(L, buckets, exact_, far):
    """Bucket of each distance 0..L-1, logarithms in 64 bits; a distance that
    sits on a border (up to the logarithms' rounding) belongs to the upper
    bucket."""
    d = torch.arange(L, device=DEV, dtype=torch.float64)
    x = torch.log(d.clamp_min(1.0) / exact_) / math.log(far / exact_) * (buckets - exact_)
    b = torch.where(d < exact_, d, exact_ + torch.floor(x + 1e-12))
    return b.clamp_max(buckets - 1).long()


def _cand4(s):
    """Each user's candidates against its history, users padded to the longest."""
    c = s["case"]
    B, H, n, m = c["B"], c["H"], s["max_len"], s["max_cands"]
    off, coff = s["offsets"].long(), s["cand_offsets"].long()
    lens, cands = torch.diff(off), torch.diff(coff)
    at = torch.arange(n, device=DEV)
    live = at < lens[:, None]                                         # [B, n]
    row = torch.where(live, off[:-1, None] + at, 0)
    cat = torch.arange(m, device=DEV)
    clive = cat < cands[:, None]
    crow = torch.where(clive, coff[:-1, None] + cat, 0)               # [B, m]
    dec = lambda w, sc: (_kv4_values(w) * sc.float()[..., None]).flatten(-2)
    q, kc, vc = (s[x].float() for x in ("q", "k", "v"))
    o = torch.zeros(B, m, H, 128, device=DEV)
    if n:
        kh, vh = (dec(s[x + "_codes"], s[x + "_scales"])[row] for x in ("k", "v"))
        x = torch.einsum("bchd,bnhd->bhcn", q[crow], kh)
        if c["pos"]:
            rel = (lens[:, None] - at).clamp_min(0)                   # n_b - j
            x += s["rab_pos"][:, s["max_len"] + rel].transpose(0, 1)[:, :, None]
        if c["time"]:
            dt = (s["cand_ts"][crow][:, :, None] - s["ts"][row][:, None]).abs().clamp_min(1)
            bucket = torch.floor(torch.log(dt.double()) / 0.301).long().clamp_max(127)
            x += s["rab_time"][:, bucket].transpose(0, 1)
        a = torch.where(live[:, None, None], x / (1.0 + torch.exp(-x)), 0.0)
        o = torch.einsum("bhcn,bnhd->bchd", a, vh)
    x = (q * kc).sum(-1)                                              # the candidate itself
    if c["pos"]:
        x += s["rab_pos"][:, s["max_len"]]
    if c["time"]:
        x += s["rab_time"][:, 0]
    user = torch.repeat_interleave(torch.arange(B, device=DEV), cands, output_size=q.shape[0])
    o = o[user, torch.arange(q.shape[0], device=DEV) - coff[user]]
    o = (o + (x / (1.0 + torch.exp(-x)))[..., None] * vc) / (lens[user] + 1).float()[:, None, None]
    o = o.flatten(1)
    d = o - o.mean(1, keepdim=True)
    uf = s["u"].float()
    y = d / torch.sqrt((d * d).mean(1, keepdim=True) + 1e-5) * (uf / (1.0 + torch.exp(-uf)))
    return dict(y=y.to(torch.bfloat16))


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "cand4":
        return _cand4(s)
    if op == "kv4":
        return {n: (v * sc[..., None]).flatten(-2).to(torch.bfloat16)
                for n, (v, sc) in (("k", _to_kv4(s["k"])), ("v", _to_kv4(s["v"])))}
    if op in ("norm", "quant"):
        if op == "norm":
            h = s["x"] if s["res"] is None else (s["x"].float() + s["res"].float()).to(s["x"].dtype)
            hf = h.float()
            rstd = 1.0 / torch.sqrt((hf * hf).mean(1) + EPS)
            v = hf * rstd[:, None] * s["w"]
            out = dict(rstd=rstd)
            if s["res"] is not None:
                out["h"] = h
            if c["out"] == "y":
                out["y"] = v.to(h.dtype)
                return out
        else:
            v, out = s["x"].float(), {}
        scale = v.abs().amax(1).clamp_min(AMAX_FLOOR) / E4M3_MAX
        out.update(q8=_to_e4m3(v, scale[:, None]), scale=scale)
        return out
    if op == "norm_grad":
        hf, r = s["x"].float(), s["rstd"][:, None]
        dyf = s["dy"].float()
        gw = dyf * s["w"]
        m = (gw * hf).mean(1, keepdim=True)
        dx = r * (gw - hf * (r * r * m))
        if s["dres"] is not None:
            dx = dx + s["dres"].float()
        return dict(dx=dx.to(s["x"].dtype), dw=(dyf * hf * r).sum(0))
    if op == "uvqk":
        H, dqk, dv = c["H"], c["dqk"], c["dv"]
        p = s["x8"].float() @ s["w8"].float().t()
        p = p * s["x_scale"][:, None] * s["w_scale"] + s["bias"]
        if c["act"]:
            p = p / (1.0 + torch.exp(-p))
        p = p.to(torch.bfloat16)
        T = c["T"]
        u, v, q, k = torch.split(p, [H * dv, H * dv, H * dqk, H * dqk], dim=1)
        return dict(u=u, v=v.reshape(T, H, dv), q=q.reshape(T, H, dqk), k=k.reshape(T, H, dqk))
    b = _buckets(c["L"], c["buckets"], c["exact"], c["far"])
    if op == "rab":
        t = s["table"][:, b]
        return dict(rab_pos=torch.cat([torch.zeros_like(t[:, 1:]), t], dim=1))
    # a bucket holds neighbouring distances: differences of running sums
    run_ = torch.cumsum(s["d_rab"][:, c["L"] - 1:].double(), dim=1)
    run_ = torch.cat([torch.zeros_like(run_[:, :1]), run_], dim=1)
    ends = torch.searchsorted(b, torch.arange(c["buckets"], device=DEV), right=True)
    at = run_[:, ends]
    return dict(d_table=torch.diff(at, dim=1, prepend=torch.zeros_like(at[:, :1])).float())


def _own(s):
    import pointwise_attention_b200 as pa
    c = s["case"]
    op = c["op"]
    if op == "norm":
        out = pa.hstu_rmsnorm_fwd(s["x"], residual=s["res"], weight=s["w"], eps=EPS,
                                  quant=c["out"] == "q8", save_rstd=True)
        return {k: v for k, v in out.items() if v is not None}
    if op == "quant":
        q8, scale = pa.hstu_quant_rows(s["x"])
        return dict(q8=q8, scale=scale)
    if op == "norm_grad":
        dx, dw = pa.hstu_rmsnorm_bwd(s["dy"], s["x"], s["rstd"], weight=s["w"], d_residual=s["dres"])
        return dict(dx=dx, dw=dw)
    if op == "uvqk":
        return pa.hstu_uvqk_fp8_fwd(s["x8"], s["x_scale"], s["w8"], s["w_scale"], c["H"], c["dqk"],
                                    c["dv"], bias=s["bias"], act=c["act"], workspace=s["status"])
    if op == "kv4":
        cache = pa.hstu_kv4_pack(s["k"], s["v"], workspace=s["status"])
        k, v = pa.hstu_kv4_unpack(cache)
        return dict(k=k, v=v)
    if op == "cand4":
        cache = (s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"])
        return dict(y=pa.hstu_cand_kv4_fwd(
            cache, s["offsets"], s["max_len"], s["q"], s["k"], s["v"], s["u"], s["cand_offsets"],
            s["max_cands"], timestamps=s["ts"], cand_timestamps=s["cand_ts"], rab_pos=s["rab_pos"],
            rab_time=s["rab_time"], workspace=s["workspace"]))
    if op == "rab":
        return dict(rab_pos=pa.hstu_rab_bucket_fwd(s["table"], c["L"], s["thr"]))
    return dict(d_table=pa.hstu_rab_bucket_bwd(s["d_rab"], c["buckets"], s["thr"]))


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ work
def work(case):
    op = case["op"]
    if op in ("norm", "norm_grad", "quant"):
        T, E = case["T"], case["E"]
        n, b = T * E, 2 if case["dtype"] == "bf16" else 4
        if op == "quant":
            return dict(bytes=n * (b + 1) + 4 * T, flops=3 * n)
        if op == "norm":
            rows = (3 if case["res"] else 1) * b + (b if case["out"] == "y" else 1)
            return dict(bytes=n * rows + 4 * T * (1 + (case["out"] == "q8")) + 4 * E, flops=6 * n)
        rows = (4 if case["dres"] else 3) * b
        return dict(bytes=n * rows + 4 * T + 8 * E, flops=10 * n)
    if op == "uvqk":
        T, E, N = case["T"], case["E"], 2 * case["H"] * (case["dqk"] + case["dv"])
        return dict(bytes=T * E + N * E + 4 * T + 8 * N + 2 * T * N, flops=2 * T * E * N)
    if op == "kv4":   # bf16 read, 4-bit values and scales written and read, bf16 written
        return dict(bytes=case["T"] * case["H"] * 2 * (256 + 72 + 72 + 256),
                    flops=case["T"] * case["H"] * 256 * 4)
    if op == "cand4":   # lengths and counts at their means
        B, H, C = case["B"], case["H"], case["B"] * case["cands"]
        T = B * (case["least"] + case["most"]) // 2
        size = T * H * 144 + 5 * C * H * 256
        if case["pos"]:
            size += 4 * H * (case["most"] + 1)
        if case["time"]:
            size += 8 * (T + C) + 512 * H
        return dict(bytes=size, flops=4 * 128 * H * case["cands"] * T)
    H, L, B = case["H"], case["L"], case["buckets"]
    if op == "rab":
        return dict(bytes=4 * H * (2 * L - 1) + 4 * H * B, flops=H * L)
    return dict(bytes=4 * H * L + 4 * H * B, flops=H * L)


# ------------------------------------------------------------------ 64 bits
def _exact_kv4(codes, scales):
    """Values of cache rows, byte by byte: value e of a word's eight sits in
    byte 2 (e % 2) + e // 4, in the upper half where e % 4 >= 2."""
    out = torch.empty(*codes.shape[:-1], 128, dtype=torch.float64, device=DEV)
    for e in range(8):
        byte = codes[..., 2 * (e % 2) + e // 4::4].to(torch.int32)
        n = torch.bitwise_and(byte >> (4 if e % 4 >= 2 else 0), 15) - 8
        out[..., e::8] = n.to(torch.float64)
    return out * scales.to(torch.float64).repeat_interleave(32, dim=-1)


def _exact_cand4(s):
    c = s["case"]
    H, d = c["H"], torch.float64
    off, coff = s["offsets"].tolist(), s["cand_offsets"].tolist()
    rows = []
    for b in range(c["B"]):
        lo, hi, c0, c1 = off[b], off[b + 1], coff[b], coff[b + 1]
        n = hi - lo
        if c0 == c1:
            continue
        kh = _exact_kv4(s["k_codes"][lo:hi], s["k_scales"][lo:hi])
        vh = _exact_kv4(s["v_codes"][lo:hi], s["v_scales"][lo:hi])
        q, k, v = (s[x][c0:c1].to(d) for x in ("q", "k", "v"))
        sc = torch.matmul(q.transpose(0, 1), kh.permute(1, 2, 0))     # [H, m, n]
        me = torch.einsum("chd,chd->hc", q, k)
        if c["pos"]:
            table = s["rab_pos"][:, s["max_len"]:].to(d)              # by distance
            sc = sc + table[:, 1:n + 1].flip(1)[:, None]
            me = me + table[:, :1]
        if c["time"]:
            dt = (s["cand_ts"][c0:c1, None] - s["ts"][None, lo:hi]).abs().to(d)
            k_ = torch.clamp(torch.log(dt.clamp(min=1.0)).div(0.301).floor(), max=127.0).long()
            sc = sc + s["rab_time"].to(d)[:, k_]
            me = me + s["rab_time"][:, :1].to(d)
        o = torch.matmul(torch.nn.functional.silu(sc), vh.transpose(0, 1)).transpose(0, 1)
        o = o + torch.nn.functional.silu(me).t()[:, :, None] * v
        o = (o / (n + 1)).reshape(c1 - c0, H * 128)
        u = s["u"][c0:c1].to(d)
        mean, var = o.mean(1, keepdim=True), o.var(1, correction=0, keepdim=True)
        rows.append((o - mean) / (var + 1e-5).sqrt() * torch.nn.functional.silu(u))
    return dict(y=torch.cat(rows))


def exact(case, seed):
    """The operators' definitions in 64 bits.  What is held in 8 bits has its
    value before the rounding here; what is held in 4 bits is whole numbers
    times a scale, which 64 bits have as they are."""
    s = prepare(case, seed)
    op = case["op"]
    d = lambda t: t.to(torch.float64)
    if op == "cand4":
        return _exact_cand4(s)
    if op == "kv4":
        out = {}
        for n in ("k", "v"):
            g = d(s[n]).reshape(-1, 32)
            top = torch.maximum(g.amax(1), -g.amin(1)).clamp_min(AMAX_FLOOR) / 7.0
            # five significant bits, upwards: mantissa in [16, 32) of whole steps
            step = torch.exp2(torch.floor(torch.log2(top)) - 4.0)
            sc = torch.ceil(d(top.float()) / step) * step
            out[n] = (torch.round(g / sc[:, None]) * sc[:, None]).reshape(s[n].shape)
        return out
    if op == "quant" or op == "norm":
        out = {}
        if op == "quant":
            v = d(s["x"])
        else:
            h = s["x"]
            if s["res"] is not None:
                h = (d(s["x"]) + d(s["res"])).to(s["x"].dtype)   # the stream is kept in its type
                out["h"] = d(h)
            ms = torch.einsum("te,te->t", d(h), d(h)) / case["E"]
            out["rstd"] = (ms + EPS) ** -0.5
            v = torch.einsum("te,t,e->te", d(h), out["rstd"], d(s["w"]))
        if op == "norm" and case["out"] == "y":
            out["y"] = v
        else:
            top = torch.maximum(v.amax(1), -v.amin(1)).clamp_min(AMAX_FLOOR)
            out["scale"] = top / E4M3_MAX
            out["q8"] = v * (E4M3_MAX / top)[:, None]
        return out
    if op == "norm_grad":
        h, dy, r, w = d(s["x"]), d(s["dy"]), d(s["rstd"]), d(s["w"])
        dot = torch.einsum("te,te,e->t", dy, h, w)
        dx = torch.einsum("te,e,t->te", dy, w, r) - h * (dot * r ** 3 / case["E"])[:, None]
        if s["dres"] is not None:
            dx += d(s["dres"])
        return dict(dx=dx, dw=torch.einsum("te,te,t->e", dy, h, r))
    if op == "uvqk":
        T, H, dqk, dv = case["T"], case["H"], case["dqk"], case["dv"]
        x = d(s["x8"]) * d(s["x_scale"])[:, None]
        w = d(s["w8"]) * d(s["w_scale"])[:, None]
        out, at = {}, 0
        for name, width in (("u", dv), ("v", dv), ("q", dqk), ("k", dqk)):
            p = torch.addmm(d(s["bias"][at:at + H * width]), x, w[at:at + H * width].t())
            if case["act"]:
                p *= torch.sigmoid(p)
            out[name] = p if name == "u" else p.reshape(T, H, width)
            at += H * width
        return out
    H, L, B = case["H"], case["L"], case["buckets"]
    edges = [0] + [min(t, L) for t in s["thr"].tolist()] + [L]
    if op == "rab":
        full = torch.zeros(H, 2 * L - 1, dtype=torch.float64, device=DEV)
        for k in range(B):
            full[:, L - 1 + edges[k]:L - 1 + edges[k + 1]] = d(s["table"][:, k:k + 1])
        return dict(rab_pos=full)
    parts = [d(s["d_rab"][:, L - 1 + edges[k]:L - 1 + edges[k + 1]]).sum(1) for k in range(B)]
    return dict(d_table=torch.stack(parts, 1))
