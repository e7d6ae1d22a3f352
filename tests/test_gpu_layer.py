"""GPU tests of what stands between a layer's matmuls: the block boundary, the 4-bit
cache and its attention, against tests/layer_oracle.py."""
import numpy as np
import pytest
import torch

import layer_oracle as lo

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def bn():
    import ternary_weight_i2_amd as m
    return m


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t.to(dtype) if dtype is not None else t


def host(t):
    return t.float().cpu().numpy()


# ---------------------------------------------------------------- the boundary

def check_norm(bn, N, F, b_t=F32, s_t=F32, post=False, gate=None, scale=1.0, res=True, gains=True,
               seed=0, spread=1.0, in_place=False):
    rng = np.random.default_rng([seed, N, F])
    b = host(dev((rng.standard_normal((N, F)) * spread).astype(np.float32), b_t))
    r = host(dev(rng.standard_normal((N, F)).astype(np.float32) * 3, s_t)) if res else None
    pg = (1 + 0.3 * rng.standard_normal(F)).astype(np.float32) if post and gains else None
    gm = (1 + 0.3 * rng.standard_normal(F)).astype(np.float32) if gains else None
    gt = None if gate is None else rng.random((F,) if gate == "channel" else (N, F)).astype(np.float32)
    stream_bf16 = (s_t if res else b_t) is BF16
    h, v, xq, s, xsum = lo.block_norm(b, r, post, pg, gt, scale, gm, 1e-5, stream_bf16)
    d = lambda a, t=None: None if a is None else dev(a, t)  # noqa: E731
    rd = d(r, s_t)
    args = (d(b, b_t), rd, post, d(pg), d(gt), scale, d(gm))
    out = None
    if in_place:
        out = (rd, None, (torch.empty((N, F), dtype=torch.int8, device="cuda"),
                          torch.empty(N, device="cuda"),
                          torch.empty(N, dtype=torch.int32, device="cuda")))
    gh, gv, (gq, gs, gsum) = bn.block_norm_quant(*args, want_v=True, out=out)
    if res:
        assert np.array_equal(host(gh), h)
    else:
        assert gh is None
    assert np.array_equal(host(gs), s)
    assert np.array_equal(gq.cpu().numpy(), xq)
    assert np.array_equal(gsum.cpu().numpy(), xsum)
    if gv is not None:
        assert np.array_equal(host(gv), lo.bf16(v) if stream_bf16 else v)


@pytest.mark.parametrize("N,F", [(1, 128), (3, 256), (1, 2560), (2, 6912), (5, 8192), (2, 8320),
                                 (1, 16384), (2, 16512), (1, 32768), (257, 640)])
def test_boundary_sizes(bn, N, F):
    check_norm(bn, N, F, post=True, gate="token", scale=0.5)


@pytest.mark.parametrize("b_t", [F32, BF16])
@pytest.mark.parametrize("s_t", [F32, BF16])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", [None, "channel", "token"])
def test_boundary_forms(bn, b_t, s_t, post, gate):
    check_norm(bn, 7, 1024, b_t, s_t, post, gate, scale=-0.22, seed=1)


@pytest.mark.parametrize("kw", [dict(res=False), dict(res=False, b_t=BF16, post=True),
                                dict(gains=False, post=True), dict(spread=1e-12, res=False),
                                dict(spread=1e15, post=True), dict(spread=0.0, res=False, post=True),
                                dict(in_place=True, s_t=BF16), dict(in_place=True, post=True)])
def test_boundary_corners(bn, kw):
    check_norm(bn, 4, 2560, seed=2, **kw)


def test_boundary_feeds_the_matmul_and_any_batch_gives_the_same(bn):
    rng = np.random.default_rng(3)
    b, r = (dev(rng.standard_normal((9, 512)).astype(np.float32)) for _ in range(2))
    h, _, (q, s, t) = bn.block_norm_quant(b, r)
    v = bn.block_norm_quant(b, r, want_v=True, want_q=False)[1]
    q2, s2, t2 = bn.quant_act(v)
    assert torch.equal(q, q2) and torch.equal(s, s2) and torch.equal(t, t2)
    for i in range(9):
        _, _, (qi, si, ti) = bn.block_norm_quant(b[i:i + 1], r[i:i + 1])
        assert torch.equal(qi[0], q[i]) and si[0] == s[i] and ti[0] == t[i]


def test_boundary_of_more_tokens_than_a_launch_takes(bn):
    """Over 2^21 tokens are several launches: the last tokens, and those on both sides of the
    cut, as a call of their own gives them."""
    N, F = 2 ** 21 + 5, 128
    g = torch.Generator(device="cuda").manual_seed(4)
    b, r = (torch.randn((N, F), generator=g, device="cuda").to(BF16) for _ in range(2))
    gate = torch.rand((N, F), generator=g, device="cuda")
    h, v, (q, s, t) = bn.block_norm_quant(b, r, gate=gate, want_v=True)
    for first in (0, 2 ** 21 - 4, N - 8):
        c = slice(first, first + 8)
        h1, v1, (q1, s1, t1) = bn.block_norm_quant(b[c], r[c], gate=gate[c], want_v=True)
        for x, y in ((h, h1), (v, v1), (q, q1), (s, s1), (t, t1)):
            assert torch.equal(x[c], y)


# ---------------------------------------------------------------- cache

class Seqs:
    """Sequences of given lengths on shuffled pages, over a cache of one byte value."""

    def __init__(self, kv_len, new, heads, d, seed=0, fill=0xA5, spare=2, lead=0, gap=()):
        rng = np.random.default_rng([seed, heads, d, len(kv_len)])
        self.rng, self.heads, self.d = rng, heads, d
        self.kv_len, self.new = np.array(kv_len, np.int32), np.array(new, np.int32)
        self.q_start = (lead + np.concatenate([[0], np.cumsum(new)])).astype(np.int32)
        need = [max(1, -(-int(t) // 64)) for t in np.maximum(self.kv_len, 0)]
        self.n_pages = sum(need) + spare
        perm = rng.permutation(self.n_pages).astype(np.int32)
        self.table = np.full((len(kv_len), max(need)), -1, np.int32)
        at = 0
        for b, p in enumerate(need):
            self.table[b, :p] = perm[at:at + p]
            at += p
        for b, p in gap:
            self.table[b, p] = (-1, self.n_pages)[p % 2]
        self.cache = np.full((self.n_pages, heads, 72 * d), fill, np.uint8)

    @property
    def n(self):
        return int(self.q_start[-1])

    def fill(self, gain=1.0, every=None):
        """Write each whole history (or its positions in `every`)."""
        for b, t in enumerate(self.kv_len):
            t = int(t)
            k, v = self.rows(t, gain), self.rows(t, gain)
            for p in range(t):
                page = self.table[b, p // 64]
                if 0 <= page < self.n_pages and (every is None or p in every):
                    for h in range(self.heads):
                        lo.put(self.cache[page, h], p % 64, k[p, h], v[p, h])
        return self

    def rows(self, n, gain=1.0):
        x = self.rng.standard_normal((n, self.heads, self.d)) * gain
        return (x * (1 + 6 * (self.rng.random(self.d) < 0.05))).astype(np.float32)

    def dev(self):
        return dev(self.cache), dev(self.table), dev(self.kv_len), dev(self.q_start)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("kv_len,new,heads", [
    ([1], [1], 1), ([64, 65, 3], [1, 1, 1], 5), ([130, 70], [130, 3], 2), ([63, 0, 9], [2, 0, 9], 3)])
def test_append_writes_these_bytes_and_no_others(bn, d, dtype, kv_len, new, heads):
    s = Seqs(kv_len, new, heads, d)
    k, v = (host(dev(s.rows(s.n), dtype)) for _ in range(2))
    c, *rest = s.dev()
    bn.kv4_append(c, *rest, dev(k, dtype), dev(v, dtype))
    lo.append(s.cache, s.table, s.kv_len, s.q_start, k, v)
    assert np.array_equal(c.cpu().numpy(), s.cache)


def test_append_takes_slices_of_a_merged_projection(bn):
    s = Seqs([40, 90], [7, 80], 4, 64, seed=4)
    y = s.rng.standard_normal((s.n, 12 * 64)).astype(np.float32)
    for dtype in (F32, BF16):
        yd = dev(y, dtype)
        rows = yd.view(s.n, 12, 64)
        c, *rest = s.dev()
        bn.kv4_append(c, *rest, rows[:, 4:8], rows[:, 8:])
        want = s.cache.copy()
        yh = host(yd).reshape(s.n, 12, 64)
        lo.append(want, s.table, s.kv_len, s.q_start, yh[:, 4:8], yh[:, 8:])
        assert np.array_equal(c.cpu().numpy(), want)


def test_append_of_special_groups(bn):
    s = Seqs([12], [12], 1, 128, seed=5)
    k = s.rows(12)
    k[0] = 0
    k[1] = 3.25
    k[2] = -70000.0                       # beyond what is held
    k[3, 0, 5], k[3, 0, 6] = np.inf, -np.inf
    k[4, 0, 70] = np.nan
    k[5] = 1e-7 * k[5]                    # steps that fp16 cannot hold
    k[6] = 57344.0 * np.sign(k[6])
    k[7] = 1000 + 1e-3 * k[7]             # a middle far larger than the range
    k[8, 0, :64] = 0.5
    k[9, 0, 0] = 3e38
    k[10] = np.where(np.arange(128) % 2, 6.1e-5, -6.1e-5)
    v = k[::-1].copy()
    c, *rest = s.dev()
    bn.kv4_append(c, *rest, dev(k), dev(v))
    lo.append(s.cache, s.table, s.kv_len, s.q_start, k, v)
    assert np.array_equal(c.cpu().numpy(), s.cache)
    gk, gv = bn.kv4_read(c, *rest, 12)
    assert torch.isfinite(gk).all() and torch.isfinite(gv).all()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_read_gives_back_what_the_codes_stand_for(bn, d, dtype):
    s = Seqs([130, 5, 64], [130, 2, 9], 2, d, seed=6, gap=[(0, 1)]).fill()
    k, v = bn.kv4_read(*s.dev(), s.n, dtype=dtype)
    want = lo.read(s.cache, s.table, s.kv_len, s.q_start, s.n, d)
    for got, w in zip((k, v), want):
        assert np.array_equal(host(got), lo.bf16(w) if dtype is BF16 else w)


def test_round_trip_is_within_half_a_step(bn):
    """A value is off by half a step, and by what fp16 loses of the middle and the step."""
    s = Seqs([200], [200], 3, 128, seed=7)
    k, v = s.rows(200), s.rows(200)
    c, *rest = s.dev()
    bn.kv4_append(c, *rest, dev(k), dev(v))
    for got, x in zip(bn.kv4_read(c, *rest, 200), (k, v)):
        g = x.reshape(200, 3, 2, 64)
        span = (g.max(-1) - g.min(-1))[..., None]
        off = np.abs(host(got).reshape(g.shape) - g)
        top = np.abs(g).max(-1)[..., None]
        assert (off <= span / 15 * (0.5 + 2.0 ** -8) + top * 2.0 ** -10).all()


def test_rows_of_no_sequence_stay_as_they_are(bn):
    s = Seqs([20, 30], [4, 6], 2, 64, seed=8, lead=3).fill()
    n = s.n + 5
    inside = np.zeros(n, bool)
    inside[3:s.n] = True
    k, v = (torch.full((n, 2, 64), 7.0, device="cuda") for _ in range(2))
    bn.kv4_read(*s.dev(), n, out=(k, v))
    q = dev(s.rng.standard_normal((n, 4, 64)).astype(np.float32))
    for max_kv in (None, 64):
        o = torch.full((n, 4, 64), 7.0, device="cuda")
        bn.attn_kv4(q, *s.dev(), out=o, max_kv=max_kv)
        for t in (k, v, o):
            assert (host(t)[~inside] == 7.0).all() and (host(t)[inside] != 7.0).all()
    c, *rest = s.dev()
    rows = dev(s.rng.standard_normal((n, 2, 64)).astype(np.float32))
    bn.kv4_append(c, *rest, rows, rows)
    lo.append(s.cache, s.table, s.kv_len, s.q_start, host(rows), host(rows))
    assert np.array_equal(c.cpu().numpy(), s.cache)


def test_read_one_side_only_and_positions_before_the_first(bn):
    s = Seqs([3], [5], 1, 64, seed=9).fill()
    k = torch.full((5, 1, 64), 7.0, device="cuda")
    bn.kv4_read(*s.dev(), 5, out=(k, None))
    want = lo.read(s.cache, s.table, s.kv_len, s.q_start, 5, 64)[0]
    assert np.array_equal(host(k), want) and (host(k)[:2] == 0).all()
    c, *rest = s.dev()
    rows = s.rows(5)
    bn.kv4_append(c, *rest, dev(rows), dev(rows))
    lo.append(s.cache, s.table, s.kv_len, s.q_start, rows, rows)
    assert np.array_equal(c.cpu().numpy(), s.cache)


# ---------------------------------------------------------------- attention

def check_attn(bn, s, heads, dtype=F32, window=0, sinks=0, scale=None, max_kv=None, gain=1.0,
               sample=None):
    q = host(dev((s.rng.standard_normal((s.n, heads, s.d)) * gain).astype(np.float32), dtype))
    sc = s.d ** -0.5 if scale is None else scale
    only = None if sample is None else {(int(r), int(h)) for r, h in zip(
        s.rng.integers(0, s.n, sample), s.rng.integers(0, heads, sample))}
    want, tol = lo.attention(q, s.cache, s.table, s.kv_len, s.q_start, sc, window, sinks,
                             dtype is BF16, only)
    got = bn.attn_kv4(dev(q, dtype), *s.dev(), scale=scale, window=window, sinks=sinks, max_kv=max_kv)
    got = host(got).astype(np.float64)
    assert np.isfinite(got).all()
    left = ~np.isnan(want)
    assert left.any()
    off = np.abs(got - want)[left]
    assert (off <= tol[left]).all(), (off - tol[left]).max()
    return got


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("t", [1, 2, 63, 64, 65, 257, 700])
def test_one_token(bn, d, dtype, t):
    check_attn(bn, Seqs([t], [1], 2, d, seed=t, fill=0xFF).fill(), 8, dtype)


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (5, 5), (20, 5), (16, 8), (64, 8), (24, 1), (40, 2)])
def test_head_layouts(bn, heads, kv_heads):
    check_attn(bn, Seqs([70, 1, 130], [1, 1, 2], kv_heads, 64, seed=11, fill=0xFF).fill(), heads)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_prompts_from_nothing_and_chunks(bn, d, dtype):
    check_attn(bn, Seqs([150, 31, 1, 200, 0], [150, 31, 1, 37, 0], 2, d, seed=12, fill=0xFF).fill(),
               4, dtype)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("window,sinks", [(0, 0), (90, 3)])
def test_many_rows(bn, d, dtype, window, sinks):
    """Over 32768 (token, head) rows take two fragments of rows to a wave and two tiles to a
    workgroup: ragged sequences whose last tiles are partly or wholly empty."""
    s = Seqs([300, 1, 77, 0, 130, 3], [300, 1, 33, 0, 130, 9], 2, d, seed=30, fill=0xFF,
             gap=[(0, 1)]).fill()
    got = check_attn(bn, s, 72, dtype, window, sinks, sample=1500)
    assert (got[-9:-3] == 0).all()              # more rows than tokens
    one = bn.attn_kv4(dev(np.ones((s.n, 72, d), np.float32), dtype), *s.dev(), window=window, sinks=sinks)
    few = bn.attn_kv4(dev(np.ones((s.n, 2, d), np.float32), dtype), *s.dev(), window=window, sinks=sinks)
    # equal queries give every head of a group the same, whichever way it is taken
    w = host(few)
    assert np.abs(host(one).reshape(s.n, 2, 36, d) - w[:, :, None]).max() <= 2.0 ** (-7 if dtype is BF16 else -16) * np.abs(w).max()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("window,sinks", [(0, 0), (2500, 3)])
def test_many_rows_over_long_histories(bn, d, dtype, window, sinks):
    """Over 16384 rows of long histories (here: what the table could hold) put all waves of a
    workgroup on one tile of two fragments."""
    s = Seqs([300, 1, 77, 0, 130, 2600], [200, 1, 33, 0, 30, 9], 2, d, seed=36, fill=0xFF,
             gap=[(0, 1), (5, 3)])
    s.fill(every=[p for p in range(2600) if p < 400 or p > 2300])
    s.cache[s.cache == 0xFF] = 0
    s.table = np.concatenate([s.table, np.full((6, 80 - s.table.shape[1]), -1, np.int32)], 1)
    check_attn(bn, s, 124, dtype, window, sinks, sample=600)


@pytest.mark.parametrize("n_seqs", [63, 64, 65, 130, 700])
def test_many_sequences(bn, n_seqs):
    """Sequences are found 64 at a time: numbers around 64, and over 64 squared / 64."""
    rng = np.random.default_rng(n_seqs)
    kv_len = rng.integers(0, 70, n_seqs)
    new = np.minimum(rng.integers(0, 4, n_seqs), kv_len)
    s = Seqs(kv_len, new, 1, 64, seed=31, fill=0xFF).fill()
    check_attn(bn, s, 2)
    k, v = s.rows(s.n), s.rows(s.n)
    c, *rest = s.dev()
    bn.kv4_append(c, *rest, dev(k), dev(v))
    lo.append(s.cache, s.table, s.kv_len, s.q_start, k, v)
    assert np.array_equal(c.cpu().numpy(), s.cache)
    want = lo.read(s.cache, s.table, s.kv_len, s.q_start, s.n, 64)
    for got, w in zip(bn.kv4_read(c, *rest, s.n), want):
        assert np.array_equal(host(got), w)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_large_batch_of_single_tokens(bn, dtype):
    """Enough rows for a prompt's kernel, but few to each sequence."""
    rng = np.random.default_rng(34)
    check_attn(bn, Seqs(rng.integers(1, 30, 300), [1] * 300, 2, 64, seed=34, fill=0xFF).fill(), 128,
               dtype, sample=800)


@pytest.mark.parametrize("window,sinks", [(1, 0), (5, 1), (64, 4), (65, 64), (100, 70), (64, 300),
                                          (1000, 4), (130, 0)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_window_and_sinks(bn, window, sinks, dtype):
    check_attn(bn, Seqs([300, 70, 129], [40, 1, 129], 1, 64, seed=13, fill=0xFF).fill(), 3, dtype,
               window, sinks)


def test_window_and_sinks_of_any_size(bn):
    s = Seqs([200, 65], [3, 1], 1, 64, seed=13, fill=0xFF).fill()
    top = 2 ** 31 - 1
    for window, sinks in ((top, 0), (top, top), (64, top), (1, top)):
        check_attn(bn, s, 2, window=window, sinks=sinks)


def test_offsets_beyond_32_bits(bn):
    """A cache of over 4 GiB, its last pages in use."""
    s = Seqs([150, 70], [150, 2], 8, 256, seed=32, spare=0)
    far = 2 ** 32 // (8 * 72 * 256) + 1 - 2
    cache = torch.empty((far + s.n_pages, 8, 72 * 256), dtype=torch.uint8, device="cuda")
    cache[far:] = dev(s.cache)
    rest = [dev(np.where(s.table >= 0, s.table + far, -1)), dev(s.kv_len), dev(s.q_start)]
    k, v = s.rows(s.n), s.rows(s.n)
    bn.kv4_append(cache, *rest, dev(k), dev(v))
    lo.append(s.cache, s.table, s.kv_len, s.q_start, k, v)
    assert torch.equal(cache[far:], dev(s.cache))
    assert torch.equal(bn.kv4_read(cache, *rest, s.n)[0], bn.kv4_read(*s.dev(), s.n)[0])
    q = dev(s.rng.standard_normal((s.n, 8, 256)).astype(np.float32))
    assert torch.equal(bn.attn_kv4(q, cache, *rest), bn.attn_kv4(q, *s.dev()))


def test_workspace_given(bn):
    s = Seqs([3000, 10], [1, 1], 1, 64, seed=33, fill=0xFF).fill(every=range(0, 3000, 7))
    s.cache[s.cache == 0xFF] = 0
    q = dev(s.rng.standard_normal((2, 2, 64)).astype(np.float32))
    need = bn.attn_kv4_workspace(2, 2, 2, 1, 64, 64 * s.table.shape[1])
    assert need > 0
    ws = torch.full((need + 64,), 255, dtype=torch.uint8, device="cuda")
    want = bn.attn_kv4(q, *s.dev())
    assert torch.equal(bn.attn_kv4(q, *s.dev(), workspace=ws[:need]), want)
    assert (ws[need:] == 255).all()
    with pytest.raises(ValueError, match="workspace"):
        bn.attn_kv4(q, *s.dev(), workspace=ws[:need - 1])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rows_that_see_nothing_and_absent_pages(bn, dtype):
    # more rows than tokens, a sequence without any, pages that are not there: the
    # second of three, and the only one of a sequence
    s = Seqs([3, 0, 180, 50], [9, 4, 70, 3], 2, 64, seed=14, fill=0xFF, gap=[(2, 1), (3, 0)]).fill()
    got = check_attn(bn, s, 4, dtype)
    assert (got[:6] == 0).all() and (got[9:13] == 0).all() and (got[-3:] == 0).all()
    check_attn(bn, s, 4, dtype, window=20, sinks=2)


def test_window_pages_may_be_given_back(bn):
    """Pages that lie behind the window and the sinks are never looked at."""
    s = Seqs([500], [3], 1, 64, seed=15, fill=0xFF).fill()
    a = check_attn(bn, s, 2, window=100, sinks=3)
    s.table[0, 1:5] = -1
    s.rng = np.random.default_rng([15, 1, 64, 1])
    s2 = Seqs([500], [3], 1, 64, seed=15, fill=0xFF)
    s2.cache, s2.table = s.cache, s.table
    b = check_attn(bn, s2, 2, window=100, sinks=3)
    assert np.isfinite(a).all() and np.isfinite(b).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("gain", [1e-6, 1e-3, 30.0, 5000.0])
def test_large_and_small_values(bn, dtype, gain):
    """Keys and values of any size that the cache holds; logits are kept in range by q."""
    s = Seqs([200, 90], [1, 3], 2, 64, seed=16, fill=0xFF).fill(gain)
    check_attn(bn, s, 4, dtype, gain=1 / gain)


def test_steps_that_grow_along_the_sequence(bn):
    s = Seqs([320], [2], 1, 128, seed=17, fill=0xFF)
    for p in range(5):
        s.fill(10.0 ** (p - 3), every=range(64 * p, 64 * p + 64))
    check_attn(bn, s, 4, gain=0.1)
    check_attn(bn, s, 4, BF16, gain=0.1)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_peaked_rows(bn, dtype):
    s = Seqs([333], [5], 1, 64, seed=18, fill=0xFF).fill()
    check_attn(bn, s, 2, dtype, scale=4.0)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_any_expected_length_gives_the_same_attention(bn, dtype):
    s = Seqs([1500, 20], [1, 1], 1, 64, seed=19, fill=0xFF).fill()
    s.table = np.concatenate([s.table, np.full((2, 900), -1, np.int32)], 1)
    for max_kv in (0, 64, 1500, None):
        st = s.rng.bit_generator.state
        check_attn(bn, s, 2, dtype, max_kv=max_kv)
        s.rng.bit_generator.state = st


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_one_long_history_among_short_ones(bn, d, dtype):
    """Chunks of pages of several lengths, fours and others, of which only the long history
    fills more than one."""
    rng = np.random.default_rng(35)
    s = Seqs([*rng.integers(1, 65, 20), 1500, *rng.integers(1, 65, 20)], [1] * 41, 2, d, seed=35,
             fill=0xFF).fill()
    s.table = np.concatenate([s.table, np.full((41, 150), -1, np.int32)], 1)
    for pages in (24, 60, 110, 170):
        check_attn(bn, s, 4, dtype, max_kv=64 * pages)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_few_sequences_with_rows_among_many(bn, dtype):
    """A step of a fixed number of sequences, of which most add no token."""
    rng = np.random.default_rng(37)
    new = np.zeros(200, np.int64)
    new[[3, 77, 199]] = 1
    kv_len = rng.integers(0, 100, 200)
    kv_len[[3, 77, 199]] = 1500, 90, 600
    check_attn(bn, Seqs(kv_len, new, 2, 64, seed=37, fill=0xFF).fill(), 8, dtype)


def test_queries_as_slices_and_out_given(bn):
    s = Seqs([100, 50], [3, 2], 2, 64, seed=20, fill=0xFF).fill()
    y = dev(s.rng.standard_normal((5, 8, 64)).astype(np.float32))
    q = y[:, 2:6]
    out = torch.empty((5, 4, 64), device="cuda")
    got = bn.attn_kv4(q, *s.dev(), out=out)
    assert got is out
    assert torch.equal(out, bn.attn_kv4(q.contiguous(), *s.dev()))


def test_same_bits_again(bn):
    s = Seqs([900, 300], [1, 1], 2, 128, seed=21, fill=0xFF).fill()
    args = s.dev()
    q = dev(s.rng.standard_normal((2, 8, 128)).astype(np.float32))
    first = bn.attn_kv4(q, *args)
    for _ in range(5):
        assert torch.equal(first, bn.attn_kv4(q, *args))


# ---------------------------------------------------------------- graphs and streams

def test_a_captured_step_follows_its_lengths(bn):
    """One decode step (boundary, append, attention) captured once and replayed with other
    lengths and tokens, eager work between the replays, each against the eager step."""
    s = Seqs([400, 130], [1, 1], 2, 64, seed=22, fill=0xFF).fill()
    cache, table, kv_len, q_start = s.dev()
    q, k, v = (torch.zeros((2, h, 64), device="cuda") for h in (4, 2, 2))
    b, r = torch.zeros((2, 256), device="cuda"), torch.zeros((2, 256), device="cuda")

    def step():
        bn.kv4_append(cache, table, kv_len, q_start, k, v)
        o = bn.attn_kv4(q, cache, table, kv_len, q_start)
        return o, bn.block_norm_quant(o.view(2, 256), r)[2][0]

    def feed(i):
        g = np.random.default_rng(i)
        for t in (q, k, v, r):
            t.copy_(dev(g.standard_normal(tuple(t.shape)).astype(np.float32)))
        kv_len.copy_(dev(np.array([200 + 61 * i, 90 + 13 * i], np.int32)))

    feed(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, code = step()
    for i in range(4):
        feed(i)
        g.replay()
        torch.cuda.synchronize()
        got, gc = o.clone(), code.clone()
        want, wc = step()
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(gc, wc)


def test_two_streams_at_once(bn):
    s = [Seqs([600 + 100 * i, 80], [1, 1], 2, 128, seed=23 + i, fill=0xFF).fill() for i in range(2)]
    args = [x.dev() for x in s]
    q = [dev(x.rng.standard_normal((2, 8, 128)).astype(np.float32)) for x in s]
    want = [bn.attn_kv4(q[i], *args[i]) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(4):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(bn.attn_kv4(q[i], *args[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(want[i], g) for g in got[i])


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("n_new,quantised", [([1, 1], True), ([1, 1], False), ([40, 30], True),
                                             ([3, 2], False)])
def test_a_layer_step(bn, n_new, quantised):
    """Boundary, attention block, boundary, matmul, as a layer runs them: 2 kv heads and 8
    query heads of 64 channels on ternary weights, histories already in the cache.  The block
    is the chain of its calls bit for bit, and every stage is what the oracle makes of the
    stage before."""
    rng = np.random.default_rng(40 + len(n_new) + n_new[0])
    hidden, d, kvh, heads = 256, 64, 2, 8
    old = [90, 30]
    s = Seqs([a + b for a, b in zip(old, n_new)], n_new, kvh, d, seed=41, fill=0xFF)
    s.kv_len[:] = old
    keep, s.q_start = s.q_start, np.array([0, *np.cumsum(old)], np.int32)
    k0, v0 = s.rows(sum(old)), s.rows(sum(old))
    lo.append(s.cache, s.table, s.kv_len, s.q_start, k0, v0)
    s.kv_len, s.q_start = np.array([a + b for a, b in zip(old, n_new)], np.int32), keep
    N = s.n
    mats = {}
    for name, m, kk in (("q", heads * d, hidden), ("k", kvh * d, hidden), ("v", kvh * d, hidden),
                        ("o", hidden, heads * d), ("up", 512, hidden)):
        w = rng.integers(-1, 2, (m, kk)).astype(np.int8)
        mats[name] = (bn.pack(dev(w)), 0.05)
    b, r = (dev(rng.standard_normal((N, hidden)).astype(np.float32)) for _ in range(2))
    gamma = dev((1 + 0.2 * rng.standard_normal(hidden)).astype(np.float32))
    sub = dev((1 + 0.2 * rng.standard_normal(heads * d)).astype(np.float32))
    turn = lambda q, k: (q * 0.5, k.flip(2))  # noqa: E731  (any map of q and k)

    h, v, tokens = bn.block_norm_quant(b, r, gamma=gamma, want_v=True)
    x = tokens if quantised else v
    c, *rest = s.dev()
    y = bn.attn_block(x, *(mats[m] for m in "qkvo"), c, *rest, gamma=sub, rotary=turn, window=64, sinks=2)
    # the same calls one by one
    c2 = dev(s.cache)
    (_, yq), (_, yk), (_, yv) = (bn.gemv_group if N <= 64 else bn.gemm_group)(
        [mats[m] for m in "qkv"], *tokens)
    qh, kh = turn(yq.view(N, heads, d), yk.view(N, kvh, d))
    bn.kv4_append(c2, *rest, kh, yv.view(N, kvh, d))
    a = bn.attn_kv4(qh, c2, *rest, window=64, sinks=2)
    _, _, inner = bn.block_norm_quant(a.view(N, -1), gamma=sub)
    y2 = (bn.gemv if N <= 64 else bn.gemm)(*mats["o"], *inner)[1]
    assert torch.equal(c, c2) and torch.equal(y, y2)
    # and each against the oracle
    lo.append(s.cache, s.table, s.kv_len, s.q_start, host(kh), host(yv).reshape(N, kvh, d))
    assert np.array_equal(c.cpu().numpy(), s.cache)
    want, tol = lo.attention(host(qh), s.cache, s.table, s.kv_len, s.q_start, d ** -0.5, 64, 2)
    assert (np.abs(host(a) - want) <= tol).all()
    _, _, xq, xs, xsum = lo.block_norm(host(a).reshape(N, -1), gamma=host(sub))
    assert np.array_equal(inner[0].cpu().numpy(), xq) and np.array_equal(host(inner[1]), xs)
    h2, _, t2 = bn.block_norm_quant(y, h, post_norm=True, scale=0.3)
    wh, _, wq, _, wsum = lo.block_norm(host(y), host(h), post=True, scale=0.3)
    assert np.array_equal(host(h2), wh) and np.array_equal(t2[0].cpu().numpy(), wq)
    assert np.array_equal(t2[2].cpu().numpy(), wsum)
    up = (bn.gemv_group if N <= 64 else bn.gemm_group)([mats["up"]], *t2)[0][1]
    assert torch.isfinite(up).all()


def test_nothing_to_do(bn):
    s = Seqs([5], [1], 1, 64, seed=25).fill()
    c, table, kv_len, q_start = s.dev()
    none = torch.empty((0, 2, 64), device="cuda")
    assert bn.attn_kv4(none, c, table, kv_len, q_start).shape == (0, 2, 64)
    bn.kv4_append(c, table, kv_len, q_start, none[:, :1], none[:, :1])
    k, v = bn.kv4_read(c, table, kv_len, q_start, 0)
    assert k.shape == v.shape == (0, 1, 64)
    h, _, (q, _, _) = bn.block_norm_quant(torch.empty((0, 128), device="cuda"),
                                          torch.empty((0, 128), device="cuda"))
    assert h.shape == (0, 128) and q.shape == (0, 128)
    wide, mat = ((bn.pack(torch.ones((m, 128), dtype=torch.int8, device="cuda")), 1.0) for m in (128, 64))
    y = bn.attn_block(torch.empty((0, 128), device="cuda"), wide, mat, mat, wide, c, table, kv_len, q_start)
    assert y.shape == (0, 128)
    assert np.array_equal(c.cpu().numpy(), s.cache)
