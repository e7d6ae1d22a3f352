"""GPU tests of the attention over the 4-bit cache where memory, masks and values are at
their worst: what no token was written to, rows that are not numbers, values of very
different sizes.  Against tests/layer_oracle.py."""
import numpy as np
import pytest
import torch

import layer_oracle as lo
from test_gpu_layer import BF16, F32, Seqs, bn, check_attn, dev, host  # noqa: F401

pytestmark = pytest.mark.gpu


def seen_only(s, window, sinks):
    """Write the positions that some row of a sequence sees, and no others."""
    for b, t in enumerate(s.kv_len):
        t, n = int(t), int(s.new[b])
        low = max(0, t - n - window + 1)
        at = sorted(set(range(min(sinks, t))) | set(range(low, t)))
        k, v = s.rows(len(at)), s.rows(len(at))
        for i, p in enumerate(at):
            for h in range(s.heads):
                lo.put(s.cache[s.table[b, p // 64], h], p % 64, k[i, h], v[i, h])
    return s


# ---------------------------------------------------------------- memory that was never written

@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("fill", [0xFF, 0xA5, 0x7C])    # NaN; negative steps; infinities
@pytest.mark.parametrize("window,sinks", [(1, 0), (70, 4), (100, 70)])
def test_hidden_places_may_hold_anything(bn, d, dtype, fill, window, sinks):  # noqa: F811
    """In front of the window and behind the sinks no token was written: single tokens, a
    continuation and a prompt that leaves its first page unfinished."""
    s = seen_only(Seqs([300, 77, 170], [1, 5, 40], 2, d, seed=50, fill=fill), window, sinks)
    check_attn(bn, s, 4, dtype, window, sinks)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_hidden_places_of_a_split_history(bn, dtype):  # noqa: F811
    s = seen_only(Seqs([9000, 5000], [1, 2], 1, 128, seed=51, fill=0xFF), 1900, 5)
    check_attn(bn, s, 4, dtype, 1900, 5)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("heads,new,window", [(124, 300, 90), (64, 200, 1990)])
def test_hidden_places_of_many_rows(bn, d, dtype, heads, new, window):  # noqa: F811
    """Prompts, with two tiles to a workgroup and with one."""
    s = seen_only(Seqs([2500, 140], [new, 30], 2, d, seed=52, fill=0xFF), window, 3)
    check_attn(bn, s, heads, dtype, window, 3, sample=500)


# ---------------------------------------------------------------- queries that are no numbers

@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("t", [100, 2000, 9000])       # eight waves, splits, many splits
def test_a_query_that_is_no_number_gives_rows_that_are_none(bn, dtype, t):  # noqa: F811
    """Those rows alone, whatever the launch; a row that sees nothing stays zero."""
    s = Seqs([t, 0, 40], [2, 1, 1], 1, 64, seed=53, fill=0xFF).fill(every=range(t - 90, t))
    s.cache[s.cache == 0xFF] = 0
    q = host(dev(s.rng.standard_normal((4, 4, 64)).astype(np.float32), dtype))
    want, tol = lo.attention(q, s.cache, s.table, s.kv_len, s.q_start, 0.125, half=dtype is BF16)
    bad = np.zeros((4, 4), bool)
    for row, head, ch, x in ((0, 1, 3, np.nan), (1, 0, 63, np.inf), (1, 3, 0, -np.inf), (3, 2, 40, np.nan)):
        q[row, head, ch] = x
        bad[row, head] = True
    q[2, 0, 0] = np.nan                                  # the sequence without any token
    got = host(bn.attn_kv4(dev(q, dtype), *s.dev()))
    assert np.isnan(got[bad]).all()
    assert (got[2] == 0).all()
    assert (np.abs(got - want)[~bad] <= tol[~bad]).all()
