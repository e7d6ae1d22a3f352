"""GPU tests of the attention over the 4-bit cache where memory, masks and values are at
their worst: what no token was written to, rows that are not numbers, values of very
different sizes.  Against tests/layer_oracle.py."""
import numpy as np
import pytest
import torch

import layer_oracle as lo
from attn_forms import FORMS
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


# ---------------------------------------------------------------- values of very different sizes

def unequal(s, size, quiet):
    """Histories whose values at position p are of size[p]; positive queries give the
    positions in `quiet` weights of e^-30."""
    new, s.new = s.new, None
    t = int(s.kv_len.max())
    k = 0.3 * s.rng.standard_normal((t, s.heads, s.d))
    k[quiet[:t]] = -30 / (0.8 * s.d ** 0.5)         # q . k: the mean of |normal| is 0.8
    v = s.rng.standard_normal((t, s.heads, s.d)) * np.broadcast_to(
        np.reshape(size, (len(size), 1, -1))[:t], (t, 1, np.reshape(size, (len(size), -1)).shape[1]))
    for b, n in enumerate(s.kv_len):
        for p in range(int(n)):
            for h in range(s.heads):
                lo.put(s.cache[s.table[b, p // 64], h], p % 64, k[p, h].astype(np.float32),
                       v[p, h].astype(np.float32))
    s.new = new
    return s


def floors(s, b, g, half):
    """What a token's part of a sum may be off by whatever its weight, [held][d]: the two
    fp16 terms (bf16 rows: one) of p and of p * step end at half of 2^-24, where the largest
    weight is 2^12 (2^7) or more.  So
      p * mid            2^-37 |mid| (2^-32)
      p * step * code    2^-37 (2^-32) 8 2^E: steps are divided by a 2^E that is at most 2^10
                         times the token's own, and in a page whose steps span more than
                         that, for which E is chosen anew, 4 times the page's largest."""
    end = 2.0 ** (-32 if half else -37)
    out = []
    held = int(s.kv_len[b])
    for p in range(-(-held // 64)):
        _, (_, step, mid) = lo.record(s.cache[s.table[b, p], g], s.d)
        n = min(64, held - 64 * p)
        step, mid = step[:n], mid[:n]
        some = step[step > 0]
        most = 4 * step.max() if some.size and step.max() >= 2.0 ** 10 * some.min() else np.inf
        out.append(np.repeat(end * (np.abs(mid) + 8 * np.minimum(2.0 ** 10 * step, most)), 64, 1))
    return np.concatenate(out)


def check_positive(bn, s, heads, dtype, sample=None):  # noqa: F811
    """Against the oracle's bound and six standard deviations of the floors."""
    half = dtype is BF16
    q = host(dev(np.abs(s.rng.standard_normal((s.n, heads, s.d))).astype(np.float32), dtype))
    only = None if sample is None else {(int(r), int(h)) for r, h in zip(
        s.rng.integers(0, s.n, sample), s.rng.integers(0, heads, sample))}
    want, tol = lo.attention(q, s.cache, s.table, s.kv_len, s.q_start, s.d ** -0.5, half=half, only=only)
    for b in range(len(s.kv_len)):
        rows, held = lo.rows_of(s.kv_len, s.q_start, b, s.table.shape[1])
        for g in range(s.heads):
            end = np.sqrt(np.cumsum(floors(s, b, g, half) ** 2, 0))
            k = lo.history(s.cache, s.table[b], held, g, s.d)[0]
            for r, pos in rows:
                for h in range(g * heads // s.heads, (g + 1) * heads // s.heads):
                    if not np.isnan(want[r, h, 0]):
                        x = s.d ** -0.5 * (k[:pos + 1] @ q[r, h].astype(np.float64))
                        tol[r, h] += 6 * end[pos] / np.exp(x - x.max()).sum()
    got = host(bn.attn_kv4(dev(q, dtype), *s.dev())).astype(np.float64)
    left = ~np.isnan(want)
    off = np.abs(got - want)[left]
    assert np.isfinite(got).all() and (off <= tol[left]).all(), (off / np.maximum(tol[left], 1e-300)).max()


SIZES = [(5e3, 0.05), (2e4, 0.01), (5e4, 0.1), (3e4, 1.0, 1e-3), (100.0, 1e-4)]


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("place", ["first page", "one in each page", "last token but one"])
def test_large_values_without_weight(bn, d, dtype, sizes, place):  # noqa: F811
    """A token with next to no weight leaves the others their accuracy, however large."""
    t = 200
    size, quiet = np.full(t, sizes[-1]), np.zeros(t, bool)
    for i, x in enumerate(sizes[:-1]):
        at = {"first page": slice(i, 64, len(sizes) - 1), "one in each page": slice(9 + i, t, 64),
              "last token but one": slice(t - 2 - i, t - 1 - i)}[place]
        size[at], quiet[at] = x, True
    check_positive(bn, unequal(Seqs([t, 90], [1, 2], 2, d, seed=54), size, quiet), 8, dtype)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("heads", [124, 250])        # one or two tiles to a workgroup
def test_large_values_without_weight_in_prompts(bn, d, dtype, heads):  # noqa: F811
    t = 300
    size, quiet = np.full(t, 0.01), np.zeros(t, bool)
    size[5::70], quiet[5::70] = 2e4, True
    s = unequal(Seqs([t], [t], 1, d, seed=55), size, quiet)
    if heads == 124:                                 # as of a long history
        s.table = np.concatenate([s.table, np.full((1, 90), -1, np.int32)], 1)
    check_positive(bn, s, heads, dtype, sample=400)


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("ratio", [1e5, 1e-5])
def test_groups_of_very_different_sizes(bn, d, dtype, ratio):  # noqa: F811
    size = np.full((200, d), 0.05 if ratio > 1 else 5e3)
    size[:, 64:128] *= ratio
    s = unequal(Seqs([200, 90], [1, 2], 2, d, seed=56), size, np.zeros(200, bool))
    check_positive(bn, s, 8, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_values_of_nothing(bn, dtype):  # noqa: F811
    """Steps of 0: constant groups, pages of zeros, between others."""
    size = np.full(300, 0.5)
    size[64:128], size[130:300:2] = 0.0, 0.0
    check_positive(bn, unequal(Seqs([300, 100], [1, 3], 2, 128, seed=57), size, np.zeros(300, bool)), 8, dtype)


# ---------------------------------------------------------------- every form of launch

@pytest.mark.parametrize("form,d", [(f, d) for f, x in FORMS.items() for d in x["dims"]])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("window", [False, True])
def test_every_form(bn, form, d, dtype, window):  # noqa: F811
    """With a window and sinks, all that they hide unwritten, and without."""
    f = FORMS[form]
    w, sinks = (f["window"], f["sinks"]) if window else (0, 0)
    s = Seqs(f["kv_len"], f["new"], f["kv_heads"], d, seed=58, fill=0xFF)
    if window:
        seen_only(s, w, sinks)
    else:                                            # zeros where a long history has gaps
        s.fill(every=[p for p in range(9000) if p < 300 or p % 8 == 0])
        s.cache[s.cache == 0xFF] = 0
    check_attn(bn, s, f["heads"], dtype, w, sinks, max_kv=f["max_kv"], sample=500)


# ---------------------------------------------------------------- very many sequences

@pytest.mark.parametrize("n_seqs,empty", [(4096, 0.5), (4097, 0.5), (4097, 0.0), (5000, 0.9), (20000, 0.95)])
def test_thousands_of_sequences(bn, n_seqs, empty):  # noqa: F811
    """Sequences are found 64 at a time: over 4096 takes a further step of the search."""
    rng = np.random.default_rng(n_seqs)
    new = np.where(rng.random(n_seqs) < empty, 0, rng.integers(0, 3, n_seqs))
    new[rng.integers(0, n_seqs, 3)] = 70
    s = Seqs(new, new, 1, 64, seed=59, fill=0xFF)
    k, v = s.rows(s.n), s.rows(s.n)
    c, *rest = s.dev()
    bn.kv4_append(c, *rest, dev(k), dev(v))
    lo.append(s.cache, s.table, s.kv_len, s.q_start, k, v)
    assert np.array_equal(c.cpu().numpy(), s.cache)
    want = lo.read(s.cache, s.table, s.kv_len, s.q_start, s.n, 64)
    for got, x in zip(bn.kv4_read(c, *rest, s.n), want):
        assert np.array_equal(host(got), x)
    check_attn(bn, s, 2, max_kv=128)


# ---------------------------------------------------------------- captured

@pytest.mark.parametrize("dtype", [F32, BF16])
def test_captured_with_pages_of_both_kinds(bn, dtype):  # noqa: F811
    """A captured call, replayed over lengths that bring pages of one visit and of several,
    ends under a window and none, gives the eager call's bits each time."""
    size = np.where(np.arange(400) // 64 % 2, 0.3, 0.01)
    size[30::64] = 2e4
    s = unequal(Seqs([400, 260], [1, 1], 2, 128, seed=61), size, size > 1)
    c, table, kv_len, q_start = s.dev()
    q = dev(np.abs(s.rng.standard_normal((2, 8, 128))).astype(np.float32), dtype)

    def run():
        return [bn.attn_kv4(q, c, table, kv_len, q_start, window=w, sinks=3 if w else 0) for w in (0, 100)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = run()
    for i in range(4):
        kv_len.copy_(dev(np.array([400 - 61 * i, 60 + 50 * i], np.int32)))
        g.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in out]
        for a, b in zip(got, run()):
            assert torch.equal(a, b) and torch.isfinite(a).all()
