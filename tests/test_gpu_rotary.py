"""GPU tests of the rotary positions, alone and with the append to the 4-bit cache, against
tests/step_oracle.py: bit for bit, since the definition says where it rounds."""
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


def freqs(rot, base=10000.0):
    return [base ** (-2 * i / rot) for i in range(rot // 2)]


def plan(bn, rot, interleaved=False, magnitude=1.0, base=10000.0):
    """The package's plan and the oracle's turns, which have to be the same numbers."""
    p = bn.rotary_plan(rot, base=base, interleaved=interleaved, magnitude=magnitude)
    turns = so.turns_of(freqs(rot, base))
    assert np.array_equal(p.turns.cpu().numpy(), turns)
    return p, turns


def same(got, want):
    """Equal bits, but any NaN for a NaN."""
    g, nan = host(got), np.isnan(want)
    assert np.array_equal(np.isnan(g), nan)
    assert np.array_equal(g.view(np.uint32)[~nan], want.view(np.uint32)[~nan])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rot", [(8, 2), (8, 8), (64, 64), (64, 22), (80, 32), (80, 80), (96, 50),
                                     (128, 16), (128, 128), (192, 6), (256, 192), (1024, 1024), (1024, 30)])
def test_rotary_forms(bn, dtype, interleaved, dim, rot):
    rng = np.random.default_rng([dim, rot])
    p, turns = plan(bn, rot, interleaved, 1.1386)
    for n, heads in ((1, 1), (7, 3), (33, 8)):
        x = host(dev(rng.standard_normal((n, heads, dim)).astype(np.float32), dtype))
        at = rng.integers(0, 200000, n).astype(np.int32)
        for inverse in (False, True):
            got = bn.rotary(dev(x, dtype), p, dev(at), inverse=inverse)
            assert got.dtype is dtype
            same(got, so.rotate(x, turns, at, interleaved, 1.1386, inverse, dtype is BF16))


def test_rotary_at_the_ends_of_the_positions(bn):
    """Quarter turns and their neighbours, zero, the largest and the negative positions."""
    rng = np.random.default_rng(1)
    turns = np.array([0, 2 ** 62, -2 ** 63, 2 ** 61, 2 ** 61 - 1, 2 ** 61 + 1, -2 ** 61, 3 * 2 ** 60,
                      1, -1, 2 ** 63 - 1, 2 ** 44 + 12345], np.int64)
    at = np.array([0, 1, 2, 3, 4, 5, -1, -2, 131071, 10 ** 6 + 7, 2 ** 31 - 1, -2 ** 31], np.int32)
    x = rng.standard_normal((len(at), 2, 24)).astype(np.float32)
    for interleaved in (False, True):
        got = bn.rotary(dev(x), bn.Rotary(dev(turns), interleaved), dev(at))
        # a fraction next to a quarter turn has a sine or cosine of 2^-64: either sign of what
        # is left of it is below the other product's last bit
        same(got, so.rotate(x, turns, at, interleaved))


def test_rotary_strides_in_place_and_other_rows(bn):
    rng = np.random.default_rng(2)
    for dtype in (F32, BF16):
        for rot, interleaved in ((32, False), (64, True), (20, False)):
            p, turns = plan(bn, rot, interleaved)
            merged = host(dev(rng.standard_normal((50, 12, 64)).astype(np.float32), dtype))
            at = rng.integers(0, 5000, 50).astype(np.int32)
            want = so.rotate(merged[:, 2:9], turns, at, interleaved, half=dtype is BF16)
            m = dev(merged, dtype)
            same(bn.rotary(m[:, 2:9], p, dev(at)), want)
            same(m, merged)
            assert bn.rotary(m[:, 2:9], p, dev(at), out=m[:, 2:9]).data_ptr() == m[:, 2:9].data_ptr()
            merged[:, 2:9] = want
            same(m, merged)
            back = torch.full((50, 9, 64), 7.0, device="cuda", dtype=dtype)
            bn.rotary(m[:, 2:9], p, dev(at), inverse=True, out=back[:, 1:8])
            same(back[:, 1:8], so.rotate(want, turns, at, interleaved, inverse=True, half=dtype is BF16))
            assert (back[:, 0] == 7).all() and (back[:, 8] == 7).all()


def test_rotary_of_rows_that_are_no_numbers(bn):
    x = np.random.default_rng(3).standard_normal((3, 2, 32)).astype(np.float32)
    x[0, 0, 3], x[1, 1, 20], x[2, 0, 30] = np.nan, np.inf, -np.inf
    p, turns = plan(bn, 16)
    at = np.array([5, 6, 7], np.int32)
    for dtype in (F32, BF16):
        got = host(bn.rotary(dev(x, dtype), p, dev(at)))
        want = so.rotate(host(dev(x, dtype)), turns, at)
        bad = ~np.isfinite(want)
        assert np.array_equal(~np.isfinite(got), bad)
        assert (bad.sum((1, 2)) == [2, 1, 1]).all() and np.isinf(got[1, 1, 20]) and got[2, 0, 30] == -np.inf


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [64, 20])
def test_the_inverse_is_the_gradient(bn, rot, interleaved):
    """<dout, R x> differentiated by x: against the formula in binary64 and, as the map is
    linear, against differences of any size.  With numbers below 8 and factors of at most 1.25
    products are below 10 and sums below 20: four roundings of at most 2^-20 each, 2^-18 (twice
    that for numbers up to 16, which the differences have)."""
    rng = np.random.default_rng(4)
    p, turns = plan(bn, rot, interleaved, 1.25)
    x, dout = (rng.standard_normal((6, 2, 64)).astype(np.float32) for _ in range(2))
    at = rng.integers(0, 100000, 6).astype(np.int32)
    dx = host(bn.rotary(dev(dout), p, dev(at), inverse=True))
    # the formula: each pair's transposed matrix
    frac = (at.astype(np.uint64)[:, None] * turns.view(np.uint64)).astype(np.float64) / 2.0 ** 64
    c, s = 1.25 * np.cos(2 * np.pi * frac)[:, None], 1.25 * np.sin(2 * np.pi * frac)[:, None]
    i = np.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    want = dout.astype(np.float64)
    da, db = want[..., a], want[..., b]
    want[..., a], want[..., b] = da * c + db * s, db * c - da * s
    assert (np.abs(dx - want) <= 2.0 ** -18).all()
    for _ in range(4):    # two rotated rows off by 2^-17, and x + d / 2 by 2^-21 times 2.5
        d = rng.standard_normal(x.shape).astype(np.float32)
        up, down = (host(bn.rotary(dev((x + e * d).astype(np.float32)), p, dev(at))).astype(np.float64)
                    for e in (0.5, -0.5))
        slope = ((up - down) * dout).sum()
        assert abs(slope - (dx.astype(np.float64) * d).sum()) <= np.abs(dout).sum() * 2.0 ** -15 + np.abs(d).sum() * 2.0 ** -18


def run_append(bn, s, heads, rot, dtype, interleaved=False, offset=None, magnitude=1.0, rows=None):
    """The fused call on s's cache -> (q_out, k turned by the oracle, q turned by the oracle)."""
    p, turns = plan(bn, rot, interleaved, magnitude)
    n = rows or s.n
    q = host(dev(s.rng.standard_normal((n, heads, s.d)).astype(np.float32), dtype))
    k, v = (host(dev(s.rng.standard_normal((n, s.heads, s.d)).astype(np.float32), dtype)) for _ in range(2))
    c, *rest = s.dev()
    out = torch.full((n, heads, s.d), 9.0, device="cuda", dtype=dtype)
    off = None if offset is None else dev(np.array(offset, np.int32))
    got = bn.rotary_kv4_append(c, *rest, dev(q, dtype), dev(k, dtype), dev(v, dtype), p, offset=off, out=out)
    at, mine = np.zeros(n, np.int64), np.zeros(n, bool)
    for b in range(len(s.kv_len)):
        for r, pos in lo.rows_of(s.kv_len, s.q_start, b, s.table.shape[1])[0]:
            at[r], mine[r] = pos + (offset[b] if offset else 0), True
    kr = so.rotate(k, turns, at, interleaved, magnitude, half=dtype is BF16)
    qr = so.rotate(q, turns, at, interleaved, magnitude, half=dtype is BF16)
    same(got[dev(mine)], qr[mine])
    assert (host(got)[~mine] == 9).all()
    lo.append(s.cache, s.table, s.kv_len, s.q_start, kr, v)
    assert np.array_equal(c.cpu().numpy(), s.cache)
    # and the chain of the two calls that it stands for
    c2, *rest = s.dev()
    at32 = at.astype(np.int32)
    same(bn.rotary(dev(q, dtype), p, dev(at32))[dev(mine)], qr[mine])
    bn.kv4_append(c2, *rest, bn.rotary(dev(k, dtype), p, dev(at32)), dev(v, dtype))
    assert torch.equal(c, c2)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d,rot,interleaved", [(64, 64, False), (64, 16, True), (64, 38, False), (128, 128, False),
                                               (128, 64, True), (128, 32, False), (256, 256, False),
                                               (256, 130, True), (256, 10, False)])
def test_append_forms(bn, dtype, d, rot, interleaved):
    run_append(bn, Seqs([70, 3, 130], [1, 1, 1], 2, d), 4, rot, dtype, interleaved, magnitude=1.1)
    run_append(bn, Seqs([130, 64, 9], [75, 0, 9], 3, d, seed=1), 3, rot, dtype, interleaved, offset=[0, 5, 99999])


@pytest.mark.parametrize("kv_len,new,heads,kv", [
    ([1], [1], 1, 1), ([5, 0, 2, 64], [2, 0, 2, 1], 6, 1), ([3, 7], [9, 4], 8, 2), ([1000] * 70, [1] * 70, 20, 5),
    ([400, 1, 350], [380, 1, 349], 40, 8)])
def test_append_lengths(bn, kv_len, new, heads, kv):
    """Ragged ones, rows before the first position, lanes spread over workgroups and not."""
    run_append(bn, Seqs(kv_len, new, kv, 64, seed=2), heads, 64, F32)


def test_append_leaves_padding_and_absent_pages_alone(bn):
    s = Seqs([200, 100], [130, 40], 2, 128, seed=3, lead=3, gap=[(0, 1), (1, 0)])
    run_append(bn, s, 4, 128, BF16, rows=s.n + 5)
    run_append(bn, Seqs([0, -5], [3, 2], 2, 64, seed=4), 2, 64, F32)


def test_append_in_place_on_a_merged_projection(bn):
    s = Seqs([40, 90], [7, 80], 2, 64, seed=5)
    y = s.rng.standard_normal((s.n, 12, 64)).astype(np.float32)
    p, turns = plan(bn, 64)
    at = np.concatenate([np.arange(33, 40), np.arange(10, 90)])
    m = dev(y)
    c, *rest = s.dev()
    bn.rotary_kv4_append(c, *rest, m[:, :8], m[:, 8:10], m[:, 10:], p, out=m[:, :8])
    lo.append(s.cache, s.table, s.kv_len, s.q_start, so.rotate(y[:, 8:10], turns, at), y[:, 10:])
    assert np.array_equal(c.cpu().numpy(), s.cache)
    y[:, :8] = so.rotate(y[:, :8], turns, at)
    same(m, y)


def test_append_of_special_rows(bn):
    s = Seqs([12], [12], 1, 64, seed=6)
    p, turns = plan(bn, 32)
    q, k, v = (s.rng.standard_normal((12, 1, 64)).astype(np.float32) for _ in range(3))
    k[0] = 0
    k[1, 0, 3], k[2, 0, 40], k[3] = np.nan, np.inf, -70000.0
    k[4] *= 1e-7
    c, *rest = s.dev()
    bn.rotary_kv4_append(c, *rest, dev(q), dev(k), dev(v), p)
    lo.append(s.cache, s.table, s.kv_len, s.q_start, so.rotate(k, turns, np.arange(12)), v)
    assert np.array_equal(c.cpu().numpy(), s.cache)


def test_append_captured(bn):
    """The lengths, the table and the offsets are read when the graph runs."""
    s = Seqs([20, 70], [1, 1], 2, 64, seed=7)
    s.kv_len[:] = [17, 64]
    p, turns = plan(bn, 64)
    q, k, v = (s.rng.standard_normal((2, h, 64)).astype(np.float32) for h in (4, 2, 2))
    c, table, kv_len, q_start = s.dev()
    off = dev(np.array([0, 0], np.int32))
    qd, kd, vd = dev(q), dev(k), dev(v)
    out = torch.empty_like(qd)
    bn.rotary_kv4_append(c, table, kv_len, q_start, qd, kd, vd, p, offset=off, out=out)
    torch.cuda.synchronize()
    c.copy_(dev(s.cache))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bn.rotary_kv4_append(c, table, kv_len, q_start, qd, kd, vd, p, offset=off, out=out)
    for step in range(3):
        g.replay()
        bn.rotary(qd, p, kv_len)          # eager work between
        torch.cuda.synchronize()
        at = s.kv_len - 1 + np.array([10 * step, 3 * step])
        lo.append(s.cache, s.table, s.kv_len, s.q_start, so.rotate(k, turns, at), v)
        same(out, so.rotate(q, turns, at))
        assert np.array_equal(c.cpu().numpy(), s.cache)
        s.kv_len += 1
        kv_len.add_(1)
        off.add_(dev(np.array([10, 3], np.int32)))


def test_on_another_stream(bn):
    rng = np.random.default_rng(8)
    p, turns = plan(bn, 64)
    x, at = rng.standard_normal((500, 8, 64)).astype(np.float32), np.arange(500, dtype=np.int32)
    xd, ad = dev(x), dev(at)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        got = bn.rotary(xd, p, ad)
        got = bn.rotary(got, p, ad, inverse=True)
    st.synchronize()
    same(got, so.rotate(so.rotate(x, turns, at), turns, at, inverse=True))


def test_scaled_plans(bn):
    """What `factor`, `length` and `freqs` make of the frequencies, in plain arithmetic."""
    f = np.array(freqs(64))
    near = lambda p, w: np.allclose(p.turns.cpu().numpy().view(np.uint64) / 2.0 ** 64 * 2 * np.pi,  # noqa: E731
                                    w, rtol=1e-12, atol=1e-18)
    assert near(bn.rotary_plan(64), f)
    assert near(bn.rotary_plan(64, factor=4.0), f / 4)
    kept = np.clip((2048 * f / (2 * np.pi) - 2) / (16 - 2), 0, 1)
    assert 0 < (kept == 1).sum() and 0 < (kept == 0).sum() and ((kept > 0) & (kept < 1)).any()
    assert near(bn.rotary_plan(64, factor=8.0, length=2048, low=2, high=16), f * kept + f / 8 * (1 - kept))
    assert near(bn.rotary_plan(4, freqs=[0.5, 2 * np.pi + 0.25]), [0.5, 0.25])


def test_attention_block_with_a_plan(bn):
    """attn_block with a Rotary is the chain of its calls, bit for bit."""
    rng = np.random.default_rng(9)
    s = Seqs([90, 30], [3, 2], 2, 64, seed=9, fill=0xFF).fill()
    mats = {m: (bn.pack(dev(rng.integers(-1, 2, shape).astype(np.int8))), 0.05)
            for m, shape in (("q", (512, 256)), ("k", (128, 256)), ("v", (128, 256)), ("o", (256, 512)))}
    x = dev(rng.standard_normal((5, 256)).astype(np.float32))
    p, _ = plan(bn, 32, True)
    off = dev(np.array([7, 1000], np.int32))
    c, *rest = s.dev()
    y = bn.attn_block(x, *(mats[m] for m in "qkvo"), c, *rest, rotary=p, offset=off)
    at = dev(np.array([94, 95, 96, 1028, 1029], np.int32))
    turn = lambda q, k: (bn.rotary(q, p, at), bn.rotary(k, p, at))  # noqa: E731
    c2, *rest = s.dev()
    y2 = bn.attn_block(x, *(mats[m] for m in "qkvo"), c2, *rest, rotary=turn)
    assert torch.equal(y, y2) and torch.equal(c, c2)


def test_nothing_to_turn(bn):
    p, _ = plan(bn, 64)
    none, at = torch.empty((0, 2, 64), device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda")
    assert bn.rotary(none, p, at).shape == (0, 2, 64)
    s = Seqs([5], [1], 1, 64)
    c, *rest = s.dev()
    assert bn.rotary_kv4_append(c, *rest, none, none[:, :1], none[:, :1], p).shape == (0, 2, 64)
    assert np.array_equal(c.cpu().numpy(), s.cache)
