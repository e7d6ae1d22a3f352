"""Host side of the attention over the 4-bit cache: which sizes a call takes (CPU only)."""
import random

import pytest


@pytest.fixture(scope="module")
def L():
    from ternary_weight_i2_amd import _binding
    return _binding.load()


def test_workspace_query_refuses_what_the_call_refuses(L):
    w = L.bitnet_attn_kv4_workspace
    assert w(1 << 20, 1 << 20, 16, 16, 64, 64, 0, 0) == -1
    assert "too many" in L.bitnet_last_error().decode()
    assert w(1, 1 << 21, 128, 128, 256, 64, 0, 0) == -1
    # below the stated limit every call is taken, however long its histories: splits are
    # given up first
    assert w(1 << 20, 1, 8, 8, 64, 1 << 30, 0, 0) == 0
    assert w((1 << 20) - 1, 1, 15, 15, 256, 1 << 30, 0, 0) == 0
    rng = random.Random(1)
    for _ in range(3000):
        kv = rng.choice([1, 2, 5, 8, 16, 100])
        heads = kv * rng.choice([1, 2, 4, 8])
        n_seqs, n = (int(2 ** rng.uniform(0, 20.5)) for _ in range(2))
        sizes = (min(n_seqs, 1 << 20), n, heads, kv, rng.choice([64, 128, 256]),
                 64 * int(2 ** rng.uniform(0, 24)), rng.choice([0, 1000]), 4)
        if n * heads // 16 + sizes[0] * kv < 1 << 24:
            assert w(*sizes) >= 0, sizes
