"""CPU test: a workspace of the norm's backward serves every smaller call."""
import random

import pytest


@pytest.fixture(scope="module")
def size():
    from pointwise_attention_b200 import build
    build.build()
    import pointwise_attention_b200 as pa
    return pa.load_library().hstu_rmsnorm_bwd_workspace_size


@pytest.mark.parametrize("T", [1, 7, 100, 3000, 5000, 200_000])
def test_sizes_grow_with_rows_and_their_length(size, T):
    rng = random.Random(T)
    for _ in range(20000):
        E = int(2 ** rng.uniform(0, 14))
        n = size(T, E)
        assert n >= 256 and n % 256 == 0
        assert size(rng.randint(0, T), rng.randint(1, E)) <= n, E


def test_either_side_of_every_border(size):
    for e in (32, 64, 128, 256, 512, 1024, 2048, 4096, 8192):
        for T in (1, 40, 1000, 4000, 1 << 20):
            for d in (1, 2, 17, 31):
                assert size(T, e) <= size(T, e + d), (T, e, d)
