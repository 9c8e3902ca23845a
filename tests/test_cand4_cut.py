"""CPU tests of how scoring against the 4-bit cache is cut: every row that the
sums of an accepted call take lies in the workspace that the size query gives,
whatever the candidate buffer's length, compiled from the kernels' own header."""
import ctypes
import os
import random
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "pointwise_attention_b200", "csrc")

SHIM = r"""
#include "cand4_cut.h"
using namespace hstu;
extern "C" {
// the rows of the sums that a call takes at most
long long rows_taken(int B, int H, int n, int C, int m, int tokens) {
  const Cand4Cut c = cand4_cut(B, H, n, m, tokens);
  if (c.many) return (long long)c.splits * cand4_sum_rows(B, C, m);
  return ((long long)c.ctas + B) * c.parts * m;   // pieces: a CTA's or a user's first
}
int splits(int B, int H, int n, int m) { return cand4_cut(B, H, n, m, 0x7FFFFFFF).splits; }
int sum_rows(int B, int C, int m) { return cand4_sum_rows(B, C, m); }
int in_sums(int c0, int cb, int first, int rows) { return cand4_in_sums(c0, cb, first, rows); }
long long part_rows(int B, int H, int n, int C, int m) { return (long long)cand4_part_rows(B, H, n, C, m); }
}
"""


@pytest.fixture(scope="module")
def cut(tmp_path_factory):
    d = tmp_path_factory.mktemp("cut")
    src, so = str(d / "shim.cpp"), str(d / "shim.so")
    with open(src, "w") as f:
        f.write(SHIM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-Wall", "-Werror", "-I", CSRC,
                    src, "-o", so], check=True)
    lib = ctypes.CDLL(so)
    for n in ("rows_taken", "part_rows"):
        getattr(lib, n).restype = ctypes.c_longlong
    return lib


@pytest.fixture(scope="module")
def size():
    from pointwise_attention_b200 import build
    build.build()
    import pointwise_attention_b200 as pa
    return pa.load_library().hstu_cand_kv4_workspace_size


def sizes(rng):
    B, H, m = int(2 ** rng.uniform(0, 9)), rng.randint(1, 16), int(2 ** rng.uniform(0, 11))
    n = int(2 ** rng.uniform(0, 15))
    # buffers of as many candidates as there may be, fewer, and many more
    C = rng.choice([rng.randint(0, B * m), B * m, B * m + int(2 ** rng.uniform(0, 17))])
    return B, H, n, C, m


def test_the_sums_fit_their_workspace(cut, size):
    rng = random.Random(3)
    for _ in range(20000):
        B, H, n, C, m = sizes(rng)
        tokens = rng.choice([0, rng.randint(0, B * n), B * n, 2 ** 31 - 1])
        rows = cut.rows_taken(B, H, n, C, m, tokens)
        assert rows <= cut.part_rows(B, H, n, C, m), (B, H, n, C, m, tokens)
        assert 256 + rows * H * 512 <= size(B, H, n, C, m), (B, H, n, C, m, tokens)


@pytest.mark.parametrize("B,H,n,C,m", [(1, 8, 4096, 1024, 32), (1, 8, 8192, 4096, 32),
                                       (1, 1, 100_000, 100_000, 17), (2, 16, 65_536, 1 << 20, 300)])
def test_a_buffer_of_a_fixed_size(cut, size, B, H, n, C, m):
    """A server's candidate buffer that a call fills in part."""
    assert cut.splits(B, H, n, m) > 1
    rows = cut.rows_taken(B, H, n, C, m, 2 ** 31 - 1)
    assert rows == cut.splits(B, H, n, m) * B * m       # not C
    assert 256 + rows * H * 512 <= size(B, H, n, C, m)


def test_sizes_grow_with_padded_buffers_too(size):
    """The size of a call is never above that of a call with larger sizes, with
    more candidate rows than the users can have among them."""
    rng = random.Random(4)
    for _ in range(4000):
        B, H, n, C, m = sizes(rng)
        small = [rng.randint(0, B), H, rng.randint(0, n), rng.randint(0, C), rng.randint(0, m)]
        assert size(*small) <= size(B, H, n, C, m), (small, (B, H, n, C, m))


def test_which_candidates_have_rows(cut):
    """Users of offsets that keep to the sizes have rows, wherever the offsets
    begin; a user whose rows would pass the end has none."""
    rng = random.Random(5)
    for _ in range(2000):
        B, m = rng.randint(1, 20), rng.randint(1, 40)
        off = [rng.randint(0, 1000)]
        for _b in range(B):
            off.append(off[-1] + rng.randint(0, m))
        C = off[-1] + rng.randint(0, 5000)
        rows = cut.sum_rows(B, C, m)
        for c0, c1 in zip(off, off[1:]):
            assert cut.in_sums(c0, c1 - c0, off[0], rows)
    assert not cut.in_sums(200, 20, 0, 40) and not cut.in_sums(21, 20, 0, 40)
    assert not cut.in_sums(3, 2, 4, 40) and not cut.in_sums(3, 2, -1, 40)
