"""GPU tests of calls with ``stream=``: what a call allocates and clears belongs
to that stream, so that neither work ahead on the caller's stream nor what the
caller allocates after the call changes a result."""
import pytest
import torch

import pointwise_attention_b200 as pa

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16
LONG = 100_000_000   # clock cycles, some 50 ms


def rnd(seed, *shape, dtype=BF16, std=1.0):
    return (std * torch.randn(*shape, generator=torch.Generator().manual_seed(seed))).to(dtype).to(DEV)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def norm_forward():
    x, res = rnd(1, 999, 512), rnd(2, 999, 512)
    return lambda **kw: [t for t in pa.hstu_rmsnorm_fwd(x, residual=res, quant=True, save_rstd=True,
                                                        **kw).values() if t is not None]


def norm_backward():
    dy, h = rnd(1, 4000, 512), rnd(2, 4000, 512)
    r = torch.rsqrt(h.float().square().mean(1) + 1e-6)
    return lambda **kw: pa.hstu_rmsnorm_bwd(dy, h, r, **kw)


def quant():
    x = rnd(1, 500, 700, dtype=F32)
    return lambda **kw: pa.hstu_quant_rows(x, **kw)


def uvqk_fp8():
    x, xs = pa.hstu_quant_rows(rnd(1, 1000, 512))
    w, ws = pa.hstu_quant_rows(rnd(2, 2048, 512))
    return lambda **kw: list(pa.hstu_uvqk_fp8_fwd(x, xs, w, ws, 4, 128, 128, act=1, **kw).values())


THR = pa.hstu_pos_bucket_thresholds(32, 16, 500)


def rab_forward():
    t = rnd(1, 8, 32, dtype=F32)
    return lambda **kw: [pa.hstu_rab_bucket_fwd(t, 3000, THR, **kw)]


def rab_backward():
    g = rnd(1, 8, 5999, dtype=F32)
    return lambda **kw: [pa.hstu_rab_bucket_bwd(g, 32, THR, **kw)]


def pack():
    k, v = rnd(1, 700, 4, 128), rnd(2, 700, 4, 128)
    return lambda **kw: pa.hstu_kv4_pack(k, v, **kw)


def unpack_rows():
    cache = pa.hstu_kv4_pack(rnd(1, 700, 4, 128), rnd(2, 700, 4, 128))
    rows = torch.arange(699, -1, -1, dtype=torch.int32, device=DEV)
    rows[::7] = -1     # these read as zeros
    return lambda **kw: pa.hstu_kv4_unpack(cache, rows=rows, **kw)


def scoring(m):
    def make():
        B, n, H = 4, 1500, 8
        cache = pa.hstu_kv4_pack(rnd(1, B * n, H, 128, std=128 ** -0.5), rnd(2, B * n, H, 128))
        off, coff = i32([n * b for b in range(B + 1)]), i32([m * b for b in range(B + 1)])
        q, k = rnd(3, B * m, H, 128, std=128 ** -0.5), rnd(4, B * m, H, 128, std=128 ** -0.5)
        v, u = rnd(5, B * m, H, 128), rnd(6, B * m, H * 128)
        ts = 1_700_000_000 + 300 * torch.arange(B * n, device=DEV)
        cts = ts[-1] + 1000 * torch.arange(B * m, device=DEV)
        rab = rnd(7, H, 128, dtype=F32)
        return lambda **kw: [pa.hstu_cand_kv4_fwd(cache, off, n, q, k, v, u, coff, m, timestamps=ts,
                                                  cand_timestamps=cts, rab_time=rab, **kw)]
    return make


CALLS = dict(norm_forward=norm_forward, norm_backward=norm_backward, quant=quant, uvqk_fp8=uvqk_fp8,
             rab_forward=rab_forward, rab_backward=rab_backward, pack=pack, unpack_rows=unpack_rows,
             scoring_few=scoring(3), scoring_many=scoring(70))


def scribble():
    """Blocks of every size that a call may have let go of, filled."""
    keep = []
    for e in range(9, 27):
        for _ in range(6 if e < 24 else 2):
            keep.append(torch.full((1 << e,), 0x7E, dtype=torch.uint8, device=DEV))
    return keep


def same(got, want):
    assert len(got) == len(want)
    for a, b in zip(got, want):
        assert a.dtype == b.dtype and torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def behind_and_before(call):
    want = [t.clone() for t in call()]
    s, mine = torch.cuda.Stream(), torch.cuda.current_stream()
    # long work ahead on the caller's stream: what the call clears must not
    # wait for it while the kernels do not
    torch.cuda.synchronize()
    torch.cuda._sleep(LONG)
    got = call(stream=s)
    s.synchronize()
    same([t.cpu() for t in got], [t.cpu() for t in want])
    # long work ahead on the given stream: the caller allocates meanwhile
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(LONG)
    got = call(stream=s)
    junk = scribble()
    mine.wait_stream(s)
    same(got, want)
    del junk
    # outputs let go of while the caller's stream still reads them
    torch.cuda.synchronize()
    got = call(stream=s)
    mine.wait_stream(s)
    torch.cuda._sleep(LONG)
    copies = [t.clone() for t in got]
    del got
    with torch.cuda.stream(s):
        junk = scribble()
    torch.cuda.synchronize()
    same(copies, want)


@pytest.mark.parametrize("name", list(CALLS))
def test_temporaries_belong_to_the_given_stream(name):
    behind_and_before(CALLS[name]())


def test_outputs_given():
    """Tensors and workspaces of the caller's own stay the caller's."""
    dy, h = rnd(1, 300, 256), rnd(2, 300, 256)
    r = torch.rsqrt(h.float().square().mean(1) + 1e-6)
    dx, ws = torch.empty_like(dy), torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
    want = pa.hstu_rmsnorm_bwd(dy, h, r)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = pa.hstu_rmsnorm_bwd(dy, h, r, dx=dx, workspace=ws, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert got[0].data_ptr() == dx.data_ptr()
    same(got, want)


def attention():
    """Forward and backward inputs: position and time bias, affine LayerNorm."""
    T, H = 1800, 4
    q, k = rnd(1, T, H, 128, std=128 ** -0.5), rnd(2, T, H, 128, std=128 ** -0.5)
    v, u, dy = rnd(3, T, H, 128), rnd(4, T, H * 128), rnd(5, T, H * 128)
    kw = dict(timestamps=1_700_000_000 + 200 * torch.arange(T, device=DEV),
              rab_pos=rnd(6, H, 1999, dtype=F32), rab_time=rnd(7, H, 128, dtype=F32),
              ln_weight=1 + 0.1 * rnd(8, H * 128, dtype=F32), ln_bias=0.1 * rnd(9, H * 128, dtype=F32))
    return (q, k, v, u, i32([0, 1000, 1800]), 1000), dy, kw


def attn_forward():
    args, _, kws = attention()

    def call(**kw):
        y, saved = pa.hstu_attn_fwd(*args, save_for_backward=True, **kws, **kw)
        return [y, *saved]
    return call


def attn_backward():
    args, dy, kws = attention()
    _, saved = pa.hstu_attn_fwd(*args, save_for_backward=True, **kws)
    # (the tables' gradients are sums by atomics, whose last bits vary)
    return lambda **kw: [pa.hstu_attn_bwd(dy, *args, saved, **kws, **kw)[n]
                         for n in ("dq", "dk", "dv", "du")]


def uvqk():
    x, w = rnd(1, 1000, 512), rnd(2, 2048, 512, std=512 ** -0.5)
    return lambda **kw: list(pa.hstu_uvqk_fwd(x, w, 4, 128, 128, act=1, **kw).values())


def out_projection():
    y, w, x = rnd(1, 1000, 512), rnd(2, 512, 512, std=512 ** -0.5), rnd(3, 1000, 512)

    def call(**kw):
        z, stats = pa.hstu_out_fwd(y, w, x, save_stats=True, **kw)
        return [z, *stats]
    return call


def cand_forward():
    (k, v, _, _, off, n), _, kws = attention()
    kws.pop("ln_weight"), kws.pop("ln_bias")
    q, kc = rnd(11, 300, 4, 128, std=128 ** -0.5), rnd(12, 300, 4, 128, std=128 ** -0.5)
    vc, uc = rnd(13, 300, 4, 128), rnd(14, 300, 512)
    cts = kws["timestamps"][-1] + 500 * torch.arange(300, device=DEV)
    kws["rab_pos"] = rnd(15, 4, 2 * n + 1, dtype=F32)
    coff = i32([0, 140, 300])
    return lambda **kw: [pa.hstu_cand_fwd(k, v, off, n, q, kc, vc, uc, coff, 160,
                                          cand_timestamps=cts, **kws, **kw)]


ATTENTION = dict(attn_forward=attn_forward, attn_backward=attn_backward, uvqk=uvqk,
                 out_projection=out_projection, cand_forward=cand_forward)


@pytest.mark.parametrize("name", list(ATTENTION))
def test_temporaries_of_the_attention_belong_to_the_given_stream(name):
    behind_and_before(ATTENTION[name]())


class Watched:
    """The library, noting where the workspaces of its calls are."""

    def __init__(self, lib):
        self.lib, self.rooms = lib, []

    def __getattr__(self, name):
        f = getattr(self.lib, name)
        if not name.startswith("hstu_") or name.endswith("_size"):
            return f

        def call(*args):      # .., workspace, its bytes, stream
            at = getattr(args[-3], "value", args[-3])
            if at:
                self.rooms.append((int(at), int(args[-2])))
            return f(*args)
        return call


@pytest.mark.parametrize("name", ["norm_backward", "uvqk_fp8", "unpack_rows", "scoring_few",
                                  "scoring_many", "attn_forward", "attn_backward"])
def test_workspaces_are_not_handed_out_early(name, monkeypatch):
    """While the given stream is busy, the caller's allocations take none of the
    memory that the call's workspace has."""
    call = (CALLS.get(name) or ATTENTION[name])()
    call()
    lib = Watched(pa.load_library())
    monkeypatch.setattr(pa._binding, "load_library", lambda: lib)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(LONG)
    got = call(stream=s)
    assert lib.rooms
    at, n = lib.rooms[0]
    mine = [torch.empty(n, dtype=torch.uint8, device=DEV) for _ in range(8)] + scribble()
    for t in mine:
        assert t.data_ptr() + t.numel() <= at or at + n <= t.data_ptr()
    torch.cuda.synchronize()
    del got


def test_nothing_on_a_given_stream():
    """Calls without rows allocate nothing to hand over."""
    s, none = torch.cuda.Stream(), rnd(1, 0, 64)
    assert pa.hstu_rmsnorm_fwd(none, quant=True, stream=s)["q8"].shape == (0, 64)
    assert pa.hstu_quant_rows(none, stream=s)[0].shape == (0, 64)
    dx, dw = pa.hstu_rmsnorm_bwd(none, none, rnd(2, 0, dtype=F32), stream=s)
    s.synchronize()
    assert dx.shape == (0, 64) and bool((dw == 0).all())
    cache = pa.hstu_kv4_pack(none.view(0, 2, 128), none.view(0, 2, 128), stream=s)
    assert pa.hstu_kv4_unpack(cache, stream=s)[0].shape == (0, 2, 128)


def test_a_stream_that_is_captured():
    """A call given the stream of a capture: its outputs and workspace belong to
    the graph, and replays follow the inputs."""
    call = norm_backward()
    want = [t.clone() for t in call()]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        got = call(stream=s)
    junk = scribble()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    same(got, want)
    del junk
