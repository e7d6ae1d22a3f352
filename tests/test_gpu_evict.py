"""GPU tests of the attention weights of cached tokens and of the eviction by them, against
tests/step_oracle.py, and of a decode loop with all the operators around it."""
import numpy as np
import pytest
import torch

import layer_oracle as lo
import step_oracle as so
from test_gpu_layer import BF16, F32, Seqs, dev, host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bn():
    import ternary_weight_i2_amd as m
    return m


# ---------------------------------------------------------------- weigh

def check_weigh(bn, s, heads, dtype=F32, decay=1.0, window=0, sinks=0, gain=1.0, rows=None, max_kv=None, q=None):
    n = rows or s.n
    if q is None:
        q = s.rng.standard_normal((n, heads, s.d)) * gain
    q = host(dev(q.astype(np.float32), dtype))
    old = np.exp(s.rng.standard_normal((s.n_pages, s.heads, 64))).astype(np.float32)
    c, *rest = s.dev()
    w = dev(old)
    out = torch.full_like(w, 5.0)
    got = bn.kv4_weigh(w, dev(q, dtype), c, *rest, decay=decay, window=window, sinks=sinks, max_kv=max_kv, out=out)
    assert got is out and torch.equal(w, dev(old))
    want, tol, written = so.weigh(old, q, s.cache, s.table, s.kv_len, s.q_start, s.d ** -0.5, decay, window, sinks)
    g = host(got)
    assert (g[~written] == 5).all()
    assert (np.abs(g - want) <= tol)[written].all()
    bn.kv4_weigh(w, dev(q, dtype), c, *rest, decay=decay, window=window, sinks=sinks, max_kv=max_kv)   # in place
    assert np.array_equal(host(w)[written], g[written]) and np.array_equal(host(w)[~written], old[~written])
    return g, written


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("kv_len,new,heads,kv", [
    ([1], [1], 1, 1), ([64, 65, 3], [1, 1, 1], 6, 2), ([130, 70], [130, 3], 5, 1), ([63, 0, 9], [2, 0, 9], 15, 3),
    ([400, 20], [90, 20], 8, 1)])
def test_weigh_forms(bn, d, dtype, kv_len, new, heads, kv):
    check_weigh(bn, Seqs(kv_len, new, kv, d, fill=0xFF).fill(), heads, dtype, decay=0.75)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("window,sinks", [(1, 0), (16, 0), (64, 4), (100, 70), (3, 1), (10 ** 6, 5)])
def test_weigh_under_a_window(bn, dtype, window, sinks):
    for new in ([1, 1], [70, 33], [300, 2]):
        check_weigh(bn, Seqs([300, 150], new, 2, 64, seed=1).fill(), 4, dtype, window=window, sinks=sinks)


@pytest.mark.parametrize("decay", [0.0, 0.5, 1.0])
def test_weigh_sums_to_the_rows(bn, decay):
    """A row gives 1 in all to the tokens it sees."""
    s = Seqs([700, 90, 64], [40, 1, 64], 2, 128, seed=2).fill()
    g, _ = check_weigh(bn, s, 6, decay=decay)
    if decay == 0:
        for b in range(3):
            t = np.arange(s.kv_len[b])
            for h in range(2):
                total = g[s.table[b, t // 64], h, t % 64].astype(np.float64).sum()
                assert abs(total - 3 * s.new[b]) < 3 * s.new[b] * 1e-5


def test_weigh_many_pages_few_expected_and_many_splits(bn):
    s = Seqs([5000], [1], 1, 64, seed=3).fill(every=set(range(0, 5000, 7)) | set(range(64)))
    s.fill()
    for max_kv in (None, 64, 1000, 5000):
        check_weigh(bn, s, 3, max_kv=max_kv)
        check_weigh(bn, s, 3, BF16, max_kv=max_kv, gain=4)
    s = Seqs([900, 10], [400, 10], 1, 64, seed=4).fill()
    for max_kv in (None, 0, 300):
        check_weigh(bn, s, 2, max_kv=max_kv)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_weigh_rows_in_parts(bn, d, dtype):
    """Prompts of many rows over few pages, whose rows several workgroups share; more pages
    than expected, which one of them then has; windows; an absent page."""
    check_weigh(bn, Seqs([700, 333], [600, 333], 1, d, seed=30, fill=0xFF, gap=[(0, 3)]).fill(), 3, dtype, decay=0.5)
    s = Seqs([640], [500], 2, d, seed=31).fill()
    for max_kv in (None, 70, 0):
        check_weigh(bn, s, 8, dtype, max_kv=max_kv)
    check_weigh(bn, s, 8, dtype, window=100, sinks=3)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("group,new", [(1, [8, 9, 7]), (3, [3, 2, 8]), (7, [1, 2, 3]), (8, [1, 3, 2]), (9, [1, 1, 1])])
def test_weigh_last_tiles_of_few_rows(bn, d, dtype, group, new):
    """Tiles of up to eight rows, alone and behind full ones; whole histories and windows."""
    s = Seqs([330, 64, 129], new, 2, d, seed=32, fill=0xFF).fill()
    check_weigh(bn, s, 2 * group, dtype, decay=0.5)
    check_weigh(bn, s, 2 * group, dtype, window=65, sinks=2)


def test_weigh_few_rows_that_are_no_numbers(bn):
    s = Seqs([200, 70], [1, 2], 1, 128, seed=33, fill=0xFF).fill()
    q = s.rng.standard_normal((3, 8, 128)).astype(np.float32)
    q[0, 2, 5], q[0, 7, 0], q[1], q[2, 0, 3] = np.nan, np.inf, -np.inf, np.nan
    g, written = check_weigh(bn, s, 8, BF16, q=q)
    assert np.isfinite(g[written]).all()


def test_weigh_leaves_what_is_not_its_own(bn):
    """Absent pages, rows in front of the first sequence and behind the last, sequences without
    rows, rows before the first position, unwritten memory."""
    check_weigh(bn, Seqs([300, 64, 200], [3, 0, 200], 2, 64, seed=5, lead=4, gap=[(0, 2), (2, 0)], fill=0xFF).fill(),
                4, rows=4 + 203 + 6)
    s = Seqs([3, 0, 0], [5, 2, 1], 2, 64, seed=6).fill()
    s.kv_len[2] = -7
    check_weigh(bn, s, 4)
    s = Seqs([130, 5], [1, 1], 1, 128, seed=7, gap=[(0, 0), (0, 1), (0, 2)], fill=0xFF)
    s.fill()
    g, written = check_weigh(bn, s, 4)      # the first sequence has no page at all
    assert written.sum() == 5
    # only what a window sees was ever written: NaN pairs everywhere else
    s = Seqs([200], [2], 1, 64, seed=8, fill=0xFF).fill(every=set(range(168, 200)) | {0, 1})
    check_weigh(bn, s, 4, window=20, sinks=2, decay=0.0)


def test_weigh_of_rows_that_are_no_numbers(bn):
    s = Seqs([200, 100], [20, 3], 2, 64, seed=9).fill()
    q = s.rng.standard_normal((23, 4, 64)).astype(np.float32)
    q[0], q[5, 1, 3], q[6, 2, 0], q[21, 3, 63] = np.nan, np.nan, np.inf, -np.inf
    q[7] = 0
    for dtype in (F32, BF16):
        g, written = check_weigh(bn, s, 4, dtype, q=q)
        assert np.isfinite(g[written]).all()


def test_weigh_of_large_and_small_scores(bn):
    for gain in (1e-20, 1e-3, 30.0):
        s = Seqs([260, 70], [33, 1], 1, 128, seed=10).fill()
        check_weigh(bn, s, 4, gain=gain)
        check_weigh(bn, s, 4, BF16, gain=gain)


def test_weigh_without_old_weights_and_given_scratch(bn):
    s = Seqs([100, 70], [1, 9], 2, 64, seed=11).fill()
    c, *rest = s.dev()
    q = dev(s.rng.standard_normal((10, 4, 64)).astype(np.float32))
    w = bn.kv4_weights(c)
    assert w.shape == (s.n_pages, 2, 64)
    w.fill_(float("nan"))
    a = bn.kv4_weigh(w, q, c, *rest, decay=0.0, out=torch.zeros_like(w))
    b = bn.kv4_weigh(None, q, c, *rest, decay=0.0, out=torch.zeros_like(w))
    need = bn.kv4_weigh_workspace(2, 10, 4, 2, 64, 128)
    ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device="cuda")
    d = bn.kv4_weigh(None, q, c, *rest, decay=0.0, max_kv=128, out=torch.zeros_like(w), workspace=ws)
    assert torch.equal(a, b) and torch.equal(a, d) and torch.isfinite(a).all()
    assert (ws[need:] == 0xFF).all()
    with pytest.raises(bn.BitnetError):
        bn.kv4_weigh(None, q, c, *rest, decay=0.5, out=w)
    with pytest.raises(ValueError):
        bn.kv4_weigh(None, q, c, *rest, decay=0.0, out=w, workspace=ws[:need - 1])
    # q as slices of a merged projection
    m = torch.zeros((10, 8, 64), device="cuda")
    m[:, 3:7] = q
    assert torch.equal(a, bn.kv4_weigh(None, m[:, 3:7], c, *rest, decay=0.0, out=torch.zeros_like(w)))


def test_weigh_thousands_of_sequences(bn):
    n = 5000
    s = Seqs([1 + i % 3 for i in range(n)], [i % 2 for i in range(n)], 1, 64, seed=12)
    s.q_start = np.concatenate([[0], np.cumsum(s.new)]).astype(np.int32)
    c, *rest = s.dev()
    k = s.rng.standard_normal((int(s.kv_len.sum()), 1, 64)).astype(np.float32)
    start = dev(np.concatenate([[0], np.cumsum(s.kv_len)]).astype(np.int32))
    bn.kv4_append(c, rest[0], rest[1], start, dev(k), dev(k))
    q = torch.zeros((s.n, 2, 64), device="cuda")     # all scores 0: every token gets 2 / its number
    w = torch.full((s.n_pages, 1, 64), 3.0, device="cuda")
    g = host(bn.kv4_weigh(w, q, c, *rest))
    for b in range(n):
        t, page = int(s.kv_len[b]), s.table[b, 0]
        want = np.full(64, 3.0)
        if s.new[b]:
            want[:t] = 2 / t
            want[:t - 1] += 3
        assert np.allclose(g[page, 0], want, rtol=1e-6)


def test_weigh_captured_and_on_two_streams(bn):
    s = Seqs([300, 100], [1, 1], 2, 64, seed=13).fill()
    c, table, kv_len, q_start = s.dev()
    kv_len.sub_(3)
    q = dev(s.rng.standard_normal((2, 8, 64)).astype(np.float32))
    w = torch.zeros((s.n_pages, 2, 64), device="cuda")
    need = bn.kv4_weigh_workspace(2, 2, 8, 2, 64, 320)
    ws = [torch.empty(need, dtype=torch.uint8, device="cuda") for _ in range(2)]
    call = lambda out, k: bn.kv4_weigh(w, q, c, table, kv_len, q_start, max_kv=320, out=out, workspace=ws[k])  # noqa: E731
    out = torch.zeros_like(w)
    call(out, 0)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(out, 0)
    other = torch.cuda.Stream()
    for _ in range(3):
        out.zero_()
        torch.cuda.synchronize()
        g.replay()
        with torch.cuda.stream(other):
            got = call(torch.zeros_like(w), 1)
        torch.cuda.synchronize()
        assert torch.equal(out, call(torch.zeros_like(w), 1)) and torch.equal(out, got)
        w.copy_(out)
        kv_len.add_(1)


# ---------------------------------------------------------------- evict

def check_evict(bn, s, keep, sinks=0, recent=0, weights=None, drop=(), spare=2, cap=None, seed=0, wide=0):
    """s's sequences onto new pages in front of which and behind which nothing may change."""
    rng = np.random.default_rng(seed)
    B, old_pages = len(s.kv_len), s.n_pages
    pages = -(-keep // 64)
    cache = np.concatenate([s.cache, np.full((B * pages + spare, *s.cache.shape[1:]), 0x3C, np.uint8)])
    w = weights if weights is not None else np.exp(2 * rng.standard_normal((old_pages, s.heads, 64)))
    w = np.concatenate([w, np.full((B * pages + spare, s.heads, 64), 11.0)]).astype(np.float32)
    new_table = np.full((B, cap or pages), -1, np.int32)
    new_table[:, :pages] = old_pages + rng.permutation(B * pages + spare)[:B * pages].reshape(B, pages)
    table = np.where(s.table == s.n_pages, len(cache), s.table).astype(np.int32)   # absent ones stay absent
    for b, p in drop:
        new_table[b, p] = (-1, len(cache))[p % 2]
    if wide:    # a table of more entries than any sequence needs
        table = np.pad(table, ((0, 0), (0, wide - table.shape[1])), constant_values=-1)
        assert bn.kv4_evict_workspace(B, s.heads, wide) > 0
    c, wd = dev(cache), dev(w)
    new_len, index = bn.kv4_evict(c, wd, dev(table), dev(s.kv_len), dev(new_table), keep, sinks=sinks, recent=recent)
    want_len, want_index = so.evict(cache, w, table, s.kv_len, new_table, keep, sinks, recent)
    assert np.array_equal(new_len.cpu().numpy(), want_len)
    assert np.array_equal(index.cpu().numpy(), want_index)
    assert np.array_equal(c.cpu().numpy(), cache)
    assert np.array_equal(host(wd).view(np.uint32), w.view(np.uint32))


def full(kv_len, heads, d, seed=0, **kw):
    """Sequences over a cache of random bytes: only moves are made of them."""
    s = Seqs(kv_len, [0] * len(kv_len), heads, d, seed=seed, **kw)
    s.cache = s.rng.integers(0, 256, s.cache.shape, dtype=np.uint8)
    return s


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("keep,sinks,recent", [(1, 0, 0), (1, 1, 0), (1, 0, 1), (70, 0, 0), (64, 4, 20), (63, 60, 3),
                                               (130, 1, 100), (500, 3, 9)])
def test_evict_forms(bn, d, keep, sinks, recent):
    check_evict(bn, full([200, 64, 1, 0, 129], 2, d), keep, sinks, recent)


@pytest.mark.parametrize("heads", [1, 3, 8])
def test_evict_long_ones(bn, heads):
    """More tokens than the four of every thread, twice over."""
    check_evict(bn, full([9000, 4096, 4097], heads, 64, seed=1), 1500, 4, 200)
    check_evict(bn, full([9000], heads, 64, seed=2), 8999, 0, 0)


@pytest.mark.parametrize("wide", [600, 4096])
def test_evict_by_several_workgroups(bn, wide):
    """Tables for long histories, whatever their sequences' lengths."""
    s = full([9000, 70, 0, 4100, 1], 2, 64, seed=10, gap=[(0, 5), (3, 64)])
    for keep, sinks, recent in ((1500, 4, 200), (1, 0, 0), (8999, 0, 9), (64, 64, 0), (3, 1, 1)):
        check_evict(bn, s, keep, sinks, recent, wide=wide)
    rng = np.random.default_rng(11)
    w = rng.integers(0, 3, (s.n_pages, 2, 64)).astype(np.float32)      # ties across slices
    check_evict(bn, s, 3000, 10, 20, weights=w, wide=wide)
    w[:] = 1
    check_evict(bn, s, 3000, 0, 20, weights=w, wide=wide)
    w = rng.choice([np.nan, np.inf, -np.inf, 0.0, -0.0, 1e-45, -1e-45, 3e38, -3e38], w.shape).astype(np.float32)
    check_evict(bn, s, 3000, 0, 20, weights=w, wide=wide)


def test_evict_of_histories_shorter_than_their_slices(bn):
    """Most workgroups have no token: what they load lies inside a page all the same."""
    for held in (33, 61, 62, 63, 64, 127):
        for heads in (1, 3):
            check_evict(bn, full([held], heads, 64, seed=held), 20, 2, 5, spare=0, wide=600)


def test_evict_scratch(bn):
    """Scratch of any content, and none that is too short."""
    s = full([5000], 1, 64, seed=12)
    cache = np.concatenate([s.cache, np.zeros((4, *s.cache.shape[1:]), np.uint8)])
    w = np.random.default_rng(12).standard_normal((len(cache), 1, 64)).astype(np.float32)
    table = np.pad(s.table, ((0, 0), (0, 600 - s.table.shape[1])), constant_values=-1)
    new_table = s.n_pages + np.arange(4, dtype=np.int32)[None]
    need = bn.kv4_evict_workspace(1, 1, 600)
    ws = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    c, wd = dev(cache), dev(w)
    got = bn.kv4_evict(c, wd, dev(table), dev(s.kv_len), dev(new_table), 200, workspace=ws)
    want = so.evict(cache, w, table, s.kv_len, new_table, 200)
    assert all(np.array_equal(a.cpu().numpy(), b) for a, b in zip(got, want))
    assert np.array_equal(c.cpu().numpy(), cache) and (ws[need:] == 0xFF).all()
    with pytest.raises(ValueError):
        bn.kv4_evict(c, wd, dev(table), dev(s.kv_len), dev(new_table), 200, workspace=ws[:need - 1])


def test_evict_by_weights_of_every_kind(bn):
    s = full([300, 300, 300, 300, 300], 2, 64, seed=3)
    w = np.zeros((s.n_pages, 2, 64), np.float32)
    at = lambda b: s.table[b, :5]  # noqa: E731
    rng = np.random.default_rng(3)
    w[at(0)] = 1.5                                                       # all equal: the first are kept
    w[at(1)] = rng.integers(0, 3, (5, 2, 64))                            # many ties
    w[at(2)] = rng.choice([np.nan, np.inf, -np.inf, 0.0, -0.0, 1e-45, -1e-45, 3e38, -3e38], (5, 2, 64))
    w[at(3)] = -np.exp(rng.standard_normal((5, 2, 64)))
    w[at(4)] = (1 + rng.integers(0, 4, (5, 2, 64)) * 2.0 ** -23)         # differ in the last bits only
    for keep, sinks, recent in ((100, 0, 0), (299, 0, 0), (100, 10, 50), (3, 1, 1)):
        check_evict(bn, s, keep, sinks, recent, weights=w)
    w[:] = np.nan
    check_evict(bn, s, 77, weights=w)
    w[:] = np.linspace(1, 2, w.size).reshape(w.shape)
    check_evict(bn, s, 77, 5, 5, weights=w)
    check_evict(bn, s, 77, 5, 5, weights=w[::-1].copy())


def test_evict_absent_pages(bn):
    """Tokens of absent pages are not there; those that go to absent pages are dropped."""
    s = full([300, 130, 64], 2, 64, seed=4, gap=[(0, 0), (0, 3), (1, 2), (2, 0)])
    for keep, sinks, recent in ((100, 0, 0), (200, 70, 90), (64, 64, 0), (64, 0, 64)):
        check_evict(bn, s, keep, sinks, recent)
        check_evict(bn, s, keep, sinks, recent, drop=[(0, 0), (1, (keep - 1) // 64)])


def test_evict_lengths_beyond_the_table_and_wider_tables(bn):
    s = full([200, 5], 1, 64, seed=5)
    s.kv_len[:] = [10 ** 6, -3]
    s.table[1] = s.table[1, 0]
    check_evict(bn, s, 100, cap=7)
    s = full([128, 128], 1, 64, seed=6)
    check_evict(bn, s, 128)            # nothing to choose
    check_evict(bn, s, 150, 100, 50)


def test_evict_many_sequences(bn):
    n = 700
    check_evict(bn, full([1 + i % 90 for i in range(n)], 1, 64, seed=7), 20, 2, 3)


def test_evict_captured_and_on_another_stream(bn):
    s = full([300, 200], 2, 64, seed=8)
    cache = np.concatenate([s.cache, np.zeros((4, *s.cache.shape[1:]), np.uint8)])
    w = np.random.default_rng(8).standard_normal((len(cache), 2, 64)).astype(np.float32)
    new_table = (s.n_pages + np.arange(4, dtype=np.int32)).reshape(2, 2)
    c, wd, table, kv_len, new = dev(cache), dev(w), dev(s.table), dev(s.kv_len), dev(new_table)
    out = torch.empty(2, dtype=torch.int32, device="cuda"), torch.empty((2, 2, 100), dtype=torch.int32, device="cuda")
    run = lambda: bn.kv4_evict(c, wd, table, kv_len, new, 100, sinks=2, recent=10, out=out)  # noqa: E731
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        run()
    st.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for step in range(3):
        kv_len.sub_(30)
        s.kv_len -= 30
        wd.mul_(-1)
        w *= -1
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        want = so.evict(cache, w, s.table, s.kv_len, new_table, 100, 2, 10)
        assert all(np.array_equal(o.cpu().numpy(), x) for o, x in zip(out, want))
        assert np.array_equal(c.cpu().numpy(), cache) and np.array_equal(host(wd), w)


def test_nothing_to_weigh_or_evict(bn):
    s = full([5], 1, 64)
    c, table, kv_len, q_start = s.dev()
    w = torch.full((s.n_pages, 1, 64), 2.0, device="cuda")
    bn.kv4_weigh(w, torch.empty((0, 2, 64), device="cuda"), c, table, kv_len, q_start)
    new_len, index = bn.kv4_evict(c, w, table[:0], kv_len[:0], table[:0], 9)
    assert new_len.shape == (0,) and index.shape == (0, 1, 9)
    assert (w == 2).all() and np.array_equal(c.cpu().numpy(), s.cache)


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("dtype_head", [F32, BF16])
def test_a_decode_loop(bn, dtype_head):
    """Prompts and then single tokens of two sequences through embedding, attention block (rotary
    positions, weights) and output head of 4-bit weights; evictions on the way.  Every stage is
    what the oracle makes of the stage before."""
    rng = np.random.default_rng(50)
    hidden, d, kvh, heads, vocab, B = 256, 64, 2, 8, 515, 2
    mats = {m: (bn.pack(dev(rng.integers(-1, 2, shape).astype(np.int8))), 0.05)
            for m, shape in (("q", (heads * d, hidden)), ("k", (kvh * d, hidden)), ("v", (kvh * d, hidden)),
                             ("o", (hidden, heads * d)))}
    emb_w = rng.standard_normal((vocab, hidden)).astype(np.float32)
    emb = bn.pack_w4(dev(emb_w), 32)
    emb_v = so.w4_values(*so.w4_quantise(emb_w, 32))
    plan = bn.rotary_plan(48, base=500.0, interleaved=True, magnitude=1.05)
    turns = so.turns_of([500.0 ** (-2 * i / 48) for i in range(24)])
    pages, keep, sinks, recent = 24, 40, 2, 8
    cache = bn.kv4_cache(pages, kvh, d)
    cache.fill_(0xFF)
    weights = bn.kv4_weights(cache).fill_(float("nan"))
    tables = [np.arange(2 * B, dtype=np.int32).reshape(B, 2), 8 + np.arange(2 * B, dtype=np.int32).reshape(B, 2)]
    table, kv_len, offset = tables[0], np.zeros(B, np.int32), np.zeros(B, np.int32)
    h_cache, h_w = cache.cpu().numpy(), host(weights)
    evictions = 0
    for step in range(30):
        new = np.array([50, 33] if step == 0 else [1, 1], np.int32)
        kv_len = kv_len + new
        q_start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        N = int(q_start[-1])
        ids = rng.integers(0, vocab, N).astype(np.int32)
        x = bn.w4_rows(emb, dev(ids))
        assert np.array_equal(host(x), emb_v[ids].astype(np.float32))
        _, _, tokens = bn.block_norm_quant(x)
        rest = dev(table), dev(kv_len), dev(q_start)
        y = bn.attn_block(tokens, *(mats[m] for m in "qkvo"), cache, *rest, rotary=plan, offset=dev(offset),
                          weights=weights, decay=0.9)
        # the stages
        (_, yq), (_, yk), (_, yv) = (bn.gemv_group if N <= 64 else bn.gemm_group)([mats[m] for m in "qkv"], *tokens)
        at = np.zeros(N, np.int64)
        for b in range(B):
            for r, pos in lo.rows_of(kv_len, q_start, b, 2)[0]:
                at[r] = pos + offset[b]
        qh = so.rotate(host(yq).reshape(N, heads, d), turns, at, True, 1.05)
        kh = so.rotate(host(yk).reshape(N, kvh, d), turns, at, True, 1.05)
        lo.append(h_cache, table, kv_len, q_start, kh, host(yv).reshape(N, kvh, d))
        assert np.array_equal(cache.cpu().numpy(), h_cache)
        want, tol, written = so.weigh(h_w, qh, h_cache, table, kv_len, q_start, d ** -0.5, 0.9)
        g = host(weights)
        assert (np.abs(g - want) <= tol)[written].all()
        assert np.array_equal(g[~written].view(np.uint32), h_w[~written].view(np.uint32))
        h_w = g
        a = bn.attn_kv4(dev(qh), cache, *rest)
        want, tol = lo.attention(qh, h_cache, table, kv_len, q_start, d ** -0.5)
        assert (np.abs(host(a) - want) <= tol).all()
        _, _, inner = bn.block_norm_quant(a.view(N, -1))
        y2 = (bn.gemv if N <= 64 else bn.gemm)(*mats["o"], *inner)[1]
        assert torch.equal(y, y2)
        _, v, _ = bn.block_norm_quant(y, x, want_v=True, want_q=False)
        last = v[dev((q_start[1:] - 1).astype(np.int64))].to(dtype_head)
        logits = bn.linear_w4(last, emb)
        want, tol = so.w4_linear(host(last), emb_v, 32, dtype_head is BF16)
        assert (np.abs(host(logits) - want) <= tol).all()
        if kv_len.max() >= 56 or step == 0:
            evictions += 1
            new_table = tables[evictions % 2]
            new_len, index = bn.kv4_evict(cache, weights, rest[0], rest[1], dev(new_table), keep, sinks=sinks,
                                          recent=recent)
            want_len, want_index = so.evict(h_cache, h_w, table, kv_len, new_table, keep, sinks, recent)
            assert np.array_equal(new_len.cpu().numpy(), want_len) and np.array_equal(index.cpu().numpy(), want_index)
            assert np.array_equal(cache.cpu().numpy(), h_cache)
            assert np.array_equal(host(weights).view(np.uint32), h_w.view(np.uint32))
            offset, kv_len, table = offset + kv_len - want_len, want_len, new_table
    assert evictions >= 2 and (offset > 0).any()
