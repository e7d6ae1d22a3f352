"""Host-side refusals of the block boundary, the 4-bit cache and its attention (CPU only:
nothing is launched, fake pointers are never dereferenced), and the oracle's own checks."""
import ctypes

import numpy as np
import pytest
import torch

import layer_oracle as lo

OK, E_NULL, E_SHAPE, E_ALIGN, E_DTYPE, E_VALUE, E_HIP = range(7)
FAKE = 0x10000          # 64 KiB-aligned non-null value, never dereferenced
MIS = 0x10004           # 4- but not 16-byte aligned


@pytest.fixture(scope="module")
def L():
    from ternary_weight_i2_amd import _binding
    return _binding.load()


def test_boundary_validation(L):
    a = dict(b=FAKE, bd=0, post=0, pg=None, gate=None, gs=0, scale=1.0, res=FAKE, h=FAKE, d=1,
             gamma=FAKE, eps=1e-5, N=2, F=256, v=None, xq=FAKE, xs=FAKE, xsum=FAKE, st=None)

    def call(**kw):
        return L.bitnet_block_norm_quant_i8(*dict(a, **kw).values())

    assert call(bd=2) == E_DTYPE and call(d=-1) == E_DTYPE
    assert call(N=-1) == E_SHAPE and call(N=1 << 31) == E_SHAPE
    for F in (0, 100, -128, 32768 + 128):
        assert call(F=F) == E_SHAPE
    for eps in (0.0, -1.0, float("inf"), float("nan")):
        assert call(eps=eps) == E_VALUE
    for scale in (float("inf"), float("-inf"), float("nan")):
        assert call(scale=scale) == E_VALUE
    assert call(gate=FAKE, gs=128) == E_SHAPE and call(gate=FAKE, gs=258) == E_SHAPE
    assert call(gate=FAKE, gs=-256) == E_SHAPE
    assert call(b=None) == E_NULL
    assert call(res=None) == E_NULL                     # h without res
    assert call(pg=FAKE) == E_VALUE                     # a gain without its norm
    for k in ("xq", "xs", "xsum"):
        assert call(**{k: None}) == E_NULL
    assert call(h=None, xq=None, xs=None, xsum=None) == E_NULL
    for k in ("b", "res", "h", "gamma", "v", "xq", "gate"):
        assert call(**{k: MIS}) == E_ALIGN
    assert call(pg=MIS, post=1) == E_ALIGN
    assert call(xs=FAKE + 2) == E_ALIGN and call(xsum=FAKE + 1) == E_ALIGN
    assert call(N=0, b=None, res=None, h=None, xq=None) == OK
    assert L.bitnet_last_error().decode() == ""


def _batch(**kw):
    from ternary_weight_i2_amd import KV4Batch
    a = dict(cache=FAKE, n_pages=4, n_kv_heads=2, head_dim=64, table=FAKE, max_pages=3,
             kv_len=FAKE, q_start=FAKE, n_seqs=2)
    return ctypes.byref(KV4Batch(*dict(a, **kw).values()))


CALLS = {
    "append": lambda L, b, dt=0, N=3, k=FAKE, ks=128, v=FAKE, vs=128:
        L.bitnet_kv4_append(b, k, ks, v, vs, dt, N, None),
    "read": lambda L, b, dt=0, N=3, k=FAKE, v=FAKE: L.bitnet_kv4_read(b, k, v, dt, N, None),
    "attn": lambda L, b, dt=0, N=3, q=FAKE, qs=256, heads=4, scale=0.125, window=0, sinks=0,
        max_kv=64, out=FAKE, ws=None, wb=0:
        L.bitnet_attn_kv4(b, q, qs, dt, N, heads, scale, window, sinks, max_kv, out, ws, wb, None),
}


@pytest.mark.parametrize("name", CALLS)
def test_cache_descriptor_validation(L, name):
    f = CALLS[name]
    assert f(L, None) == E_NULL
    assert f(L, _batch(), dt=2) == E_DTYPE
    assert f(L, _batch(), N=-1) == E_SHAPE and f(L, _batch(), N=(1 << 21) + 1) == E_SHAPE
    for d in (0, 32, 96, 192, 512, -64):
        assert f(L, _batch(head_dim=d)) == E_SHAPE
    assert f(L, _batch(n_kv_heads=0)) == E_SHAPE and f(L, _batch(n_kv_heads=1025)) == E_SHAPE
    assert f(L, _batch(n_pages=0)) == E_SHAPE and f(L, _batch(n_pages=1 << 31)) == E_SHAPE
    assert f(L, _batch(max_pages=0)) == E_SHAPE
    assert f(L, _batch(max_pages=(1 << 24) + 1)) == E_SHAPE
    assert f(L, _batch(n_seqs=-1)) == E_SHAPE and f(L, _batch(n_seqs=(1 << 20) + 1)) == E_SHAPE
    for p in ("cache", "table", "kv_len", "q_start"):
        assert f(L, _batch(**{p: None})) == E_NULL
    assert f(L, _batch(cache=MIS)) == E_ALIGN
    for p in ("table", "kv_len", "q_start"):
        assert f(L, _batch(**{p: FAKE + 2})) == E_ALIGN
    assert f(L, _batch(cache=None, table=None), N=0) == OK
    assert f(L, _batch(cache=None, table=None, n_seqs=0)) == OK
    assert L.bitnet_last_error().decode() == ""


def test_row_array_validation(L):
    f = CALLS["append"]
    for p in ("k", "v"):
        assert f(L, _batch(), **{p: None}) == E_NULL
        assert f(L, _batch(), **{p: MIS}) == E_ALIGN
    for s in ("ks", "vs"):
        for bad in (127, 64, 130, 0, -128, 1 << 41):
            assert f(L, _batch(), **{s: bad}) == E_SHAPE
        assert f(L, _batch(), dt=1, **{s: 132}) == E_SHAPE      # 264 bytes
    f = CALLS["read"]
    assert f(L, _batch(), k=None, v=None) == E_NULL
    assert f(L, _batch(), k=MIS) == E_ALIGN and f(L, _batch(), v=MIS) == E_ALIGN


def test_attention_validation(L):
    f = CALLS["attn"]
    for heads in (0, 3, -2, 1026):
        assert f(L, _batch(), heads=heads) == E_SHAPE
    for scale in (0.0, -1.0, float("inf"), float("nan")):
        assert f(L, _batch(), scale=scale) == E_VALUE
    assert f(L, _batch(), window=-1) == E_SHAPE and f(L, _batch(), sinks=-1) == E_SHAPE
    assert f(L, _batch(), window=1 << 31) == E_SHAPE and f(L, _batch(), sinks=1 << 31) == E_SHAPE
    assert f(L, _batch(), max_kv=-1) == E_SHAPE and f(L, _batch(), max_kv=193) == E_SHAPE
    assert f(L, _batch(), q=None) == E_NULL and f(L, _batch(), out=None) == E_NULL
    assert f(L, _batch(), q=MIS) == E_ALIGN and f(L, _batch(), out=MIS) == E_ALIGN
    assert f(L, _batch(), ws=MIS) == E_ALIGN
    for bad in (255, 258, 0):
        assert f(L, _batch(), qs=bad) == E_SHAPE
    # more workgroups than a launch takes
    assert f(L, _batch(n_kv_heads=16, n_seqs=1 << 20), heads=16, N=1 << 20, qs=1024) == E_SHAPE
    assert "too many" in L.bitnet_last_error().decode()
    # a long history is shared by several workgroups, which takes a workspace
    need = L.bitnet_attn_kv4_workspace(2, 3, 4, 2, 64, 64 * 100, 0, 0)
    assert need > 0
    long = _batch(max_pages=100)
    assert f(L, long, max_kv=6400) == E_NULL
    assert f(L, long, max_kv=6400, ws=FAKE, wb=need - 1) == E_SHAPE


def test_workspace_sizes(L):
    w = L.bitnet_attn_kv4_workspace
    assert w(0, 3, 4, 2, 64, 6400, 0, 0) == 0 and w(2, 0, 4, 2, 64, 6400, 0, 0) == 0
    assert 0 < w(2, 3, 4, 2, 64, 640000, 0, 0)
    assert w(2, 3, 4, 2, 64, 640000, 64, 4) < w(2, 3, 4, 2, 64, 640000, 0, 0)
    for bad in ((-1, 3, 4, 2, 64, 64, 0, 0), (2, -1, 4, 2, 64, 64, 0, 0),
                (2, 3, 5, 2, 64, 64, 0, 0), (2, 3, 4, 0, 64, 64, 0, 0),
                (2, 3, 4, 2, 96, 64, 0, 0), (2, 3, 4, 2, 64, -1, 0, 0),
                (2, 3, 4, 2, 64, (1 << 30) + 1, 0, 0), (2, 3, 4, 2, 64, 64, -1, 0),
                (2, 3, 4, 2, 64, 64, 0, -1), (2, 3, 4, 2, 64, 64, 1 << 31, 0)):
        assert w(*bad) == -1
        assert L.bitnet_last_error()


def test_binding_refuses_before_any_launch():
    import ternary_weight_i2_amd as bn
    z = torch.zeros
    i32 = torch.int32
    cache, table = z((4, 2, 72 * 64), dtype=torch.uint8), z((2, 3), dtype=i32)
    lens, start = z(2, dtype=i32), z(3, dtype=i32)
    k = z((3, 2, 64))

    def refused(what, f, *a, **kw):
        with pytest.raises((ValueError, TypeError), match=what):
            f(*a, **kw)

    refused("GPU", bn.kv4_append, cache, table, lens, start, k, k)       # CPU tensors
    refused("GPU", bn.block_norm_quant, z((2, 128)))
    refused("cache", bn.kv4_append, cache.float(), table, lens, start, k, k)
    refused("table", bn.kv4_append, cache, table[0], lens, start, k, k)
    refused("table", bn.kv4_append, cache, table.long(), lens, start, k, k)
    refused("head_dim", bn.kv4_cache, 4, 2, 96, device="cpu")
    refused("2-D", bn.block_norm_quant, z(128))
    refused("float32 or bfloat16", bn.block_norm_quant, z((2, 128), dtype=torch.float16))


# ---------------------------------------------------------------- the oracle itself

@pytest.mark.parametrize("d", [64, 128, 256])
def test_oracle_record_gives_back_what_was_put(d):
    rng = np.random.default_rng(d)
    rec = np.full(72 * d, 0xFF, np.uint8)
    k, v = rng.standard_normal((2, 64, d)).astype(np.float32)
    for t in rng.permutation(64):
        lo.put(rec, int(t), k[t], v[t])
    for (code, step, mid), x in zip(lo.record(rec, d), (k, v)):
        want = [lo.quantise(x[t]) for t in range(64)]
        assert np.array_equal(code, np.stack([w[0].reshape(-1) for w in want]))
        assert np.array_equal(step, np.stack([w[1] for w in want]).astype(np.float64))
        assert np.array_equal(mid, np.stack([w[2] for w in want]).astype(np.float64))
        assert np.abs(lo.value(code, step, mid) - x).max() < 0.51 * step.max()


def test_oracle_quantiser_by_hand():
    x = np.linspace(-8.0, 7.0, 64, dtype=np.float32)      # step 1, middle 0
    code, step, mid = lo.quantise(x)
    assert step[0] == 1 and mid[0] == 0
    assert np.array_equal(code[0], np.rint(x + 8))
    code, step, mid = lo.quantise(np.full(64, 2.5, np.float32))
    assert step[0] == 0 and mid[0] == 2.5 and (code == 8).all()
    code, step, mid = lo.quantise(np.array([np.nan, np.inf, -np.inf, 1e30] * 16, np.float32))
    assert np.isfinite(step).all() and np.isfinite(mid).all()
    assert float(mid[0]) + 7 * float(step[0]) < 65504


def test_oracle_attention_in_closed_form():
    """Equal keys: the mean of the visible values; a window of one: the row's own value."""
    d = 64
    cache, table = np.zeros((2, 1, 72 * d), np.uint8), np.array([[1, 0]], np.int32)
    kv_len, start = np.array([70], np.int32), np.array([0, 70], np.int32)
    v = np.random.default_rng(0).standard_normal((70, 1, d)).astype(np.float32)
    lo.append(cache, table, kv_len, start, np.ones((70, 1, d), np.float32), v)
    held = lo.read(cache, table, kv_len, start, 70, d)[1]
    q = np.ones((70, 1, d), np.float32)
    out, tol = lo.attention(q, cache, table, kv_len, start, 0.125)
    mean = np.cumsum(held.astype(np.float64), 0) / np.arange(1, 71)[:, None, None]
    assert np.abs(out - mean).max() < 1e-12 and np.isfinite(tol).all()
    out, _ = lo.attention(q, cache, table, kv_len, start, 0.125, window=1)
    assert np.abs(out - held).max() < 1e-6


def test_binding_workspace_size():
    import ternary_weight_i2_amd as bn
    a = bn.attn_kv4_workspace(1, 1, 4, 2, 64, 6400)
    assert a == bn.attn_kv4_workspace(1, 1, 4, 2, 64, 6400) and a % 16 == 0
    with pytest.raises(bn.BitnetError):
        bn.attn_kv4_workspace(1, 1, 3, 2, 64, 6400)
