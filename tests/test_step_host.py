"""Host-side refusals of the operators around a decode step (CPU only: nothing is launched,
fake pointers are never dereferenced)."""
import ctypes

import pytest
import torch

from test_layer_host import FAKE, MIS, OK, E_ALIGN, E_DTYPE, E_NULL, E_SHAPE, E_VALUE, _batch


@pytest.fixture(scope="module")
def L():
    from ternary_weight_i2_amd import _binding
    return _binding.load()


def _plan(**kw):
    from ternary_weight_i2_amd import RotaryPlan
    return ctypes.byref(RotaryPlan(*dict(dict(turns=FAKE, rot=64, inter=0, magnitude=1.0), **kw).values()))


ROTARY = {
    "rotary": lambda L, plan=None, x=FAKE, xs=128, dt=0, N=3, heads=2, dim=64, at=FAKE, out=2 * FAKE, os=128:
        L.bitnet_rotary(plan or _plan(), x, xs, dt, N, heads, dim, at, 0, out, os, None),
    "append": lambda L, plan=None, b=None, x=FAKE, xs=256, dt=0, N=3, heads=4, out=2 * FAKE, os=256, k=FAKE, ks=128,
        v=FAKE, vs=128, off=FAKE:
        L.bitnet_rotary_kv4_append(b or _batch(), plan or _plan(), x, xs, out, os, heads, k, ks, v, vs, dt, N,
                                   off, None),
}


@pytest.mark.parametrize("name", ROTARY)
def test_rotary_validation(L, name):
    f = ROTARY[name]
    assert f(L, dt=2) == E_DTYPE
    assert f(L, N=-1) == E_SHAPE and f(L, N=(1 << 21) + 1) == E_SHAPE
    for rot in (0, -2, 3, 63, 66, 1 << 40):
        assert f(L, plan=_plan(rot=rot)) == E_SHAPE
    for m in (0.0, -1.0, float("inf"), float("nan"), 1e31):
        assert f(L, plan=_plan(magnitude=m)) == E_VALUE
    assert f(L, plan=_plan(turns=None)) == E_NULL and f(L, plan=_plan(turns=MIS)) == E_ALIGN
    assert f(L, x=None) == E_NULL and f(L, out=None) == E_NULL
    assert f(L, x=MIS) == E_ALIGN and f(L, out=MIS) == E_ALIGN
    for s in ("xs", "os"):
        for bad in (127, 0, -256, 1 << 41, 258):
            assert f(L, **{s: bad}) == E_SHAPE
    assert f(L, out=FAKE, os=512) == E_SHAPE        # in place with another stride
    for heads in (0, -1, 1025):
        assert f(L, heads=heads) == E_SHAPE
    assert f(L, N=0, x=None, out=None) == OK and L.bitnet_last_error().decode() == ""


def test_rotary_alone_validation(L):
    f = ROTARY["rotary"]
    for dim in (0, 4, 60, -64, 1032):
        assert f(L, dim=dim, plan=_plan(rot=2)) == E_SHAPE
    assert f(L, at=None) == E_NULL and f(L, at=FAKE + 2) == E_ALIGN
    assert L.bitnet_rotary(None, FAKE, 128, 0, 3, 2, 64, FAKE, 0, FAKE, 128, None) == E_NULL


def test_rotary_append_validation(L):
    f = ROTARY["append"]
    assert L.bitnet_rotary_kv4_append(None, _plan(), FAKE, 256, FAKE, 256, 4, FAKE, 128, FAKE, 128, 0, 3, None,
                                      None) == E_NULL
    assert f(L, b=_batch(head_dim=96)) == E_SHAPE and f(L, b=_batch(table=None)) == E_NULL
    assert f(L, heads=3) == E_SHAPE
    for p in ("k", "v"):
        assert f(L, **{p: None}) == E_NULL and f(L, **{p: MIS}) == E_ALIGN
        assert f(L, **{p + "s": 64}) == E_SHAPE
    assert f(L, off=FAKE + 2) == E_ALIGN


def test_rotary_binding_refuses():
    import ternary_weight_i2_amd as bn
    t = torch.zeros(32, dtype=torch.int64)
    with pytest.raises(TypeError):
        bn.Rotary(t.int())
    with pytest.raises(TypeError):
        bn.Rotary(torch.zeros((2, 4), dtype=torch.int64))
    with pytest.raises(TypeError):
        bn.Rotary(torch.zeros(64, dtype=torch.int64)[::2])
    p, at = bn.Rotary(t), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(AttributeError):
        p.magnitude = 2.0
    x = torch.zeros((3, 2, 64))
    for bad in (dict(x=x[0]), dict(x=x.to(torch.float16)), dict(at=at.long()), dict(at=at[:2]), dict(x=x[:, :, :63]),
                dict(x=x.transpose(0, 1)), dict(out=x[:2]), dict(out=x.bfloat16()), dict()):
        with pytest.raises((ValueError, TypeError)):    # the last: not on a GPU
            bn.rotary(bad.get("x", x), p, bad.get("at", at), out=bad.get("out"))
    for kw in (dict(rot=3), dict(rot=0), dict(rot=4, freqs=[1.0]), dict(rot=4, freqs=[1.0, float("nan")]),
               dict(rot=4, factor=0.0), dict(rot=4, length=-1), dict(rot=4, length=5, low=3, high=3)):
        with pytest.raises(ValueError):
            bn.rotary_plan(**kw, device="cpu")
    c, table = torch.zeros((2, 1, 72 * 64), dtype=torch.uint8), torch.zeros((1, 1), dtype=torch.int32)
    one, start = torch.ones(1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    q, k = torch.zeros((1, 2, 64)), torch.zeros((1, 1, 64))
    for bad in (dict(q=q.bfloat16()), dict(q=q[:0]), dict(v=k.bfloat16()), dict(off=one.long()), dict(out=k), dict()):
        with pytest.raises((ValueError, TypeError)):
            bn.rotary_kv4_append(c, table, one, start, bad.get("q", q), k, bad.get("v", k), p,
                                 offset=bad.get("off"), out=bad.get("out"))
    with pytest.raises((ValueError, TypeError)):        # a slice that no aligned load can take
        bn.rotary(torch.zeros((3, 2, 65))[:, :, 1:], p, at)


# ---------------------------------------------------------------- 4-bit weights

def _mat(**kw):
    from ternary_weight_i2_amd import W4Desc
    return ctypes.byref(W4Desc(*dict(dict(codes=FAKE, steps=FAKE, M=20, K=256, group=64), **kw).values()))


W4 = {
    "pack": lambda L, m=None, dt=0, w=FAKE: L.bitnet_pack_w4(w, dt, m or _mat(), None),
    "codes": lambda L, m=None, w=FAKE, s=FAKE: L.bitnet_pack_w4_codes(w, s, m or _mat(), None),
    "rows": lambda L, m=None, dt=0, ids=FAKE, n=3, out=FAKE: L.bitnet_w4_rows(m or _mat(), ids, n, out, dt, None),
    "linear": lambda L, m=None, dt=0, x=FAKE, N=3, y=FAKE, ws=None, wb=0:
        L.bitnet_linear_w4(x, dt, N, m or _mat(), y, ws, wb, None),
}


@pytest.mark.parametrize("name", W4)
def test_w4_matrix_validation(L, name):
    f = W4[name]
    assert f(L, _mat(M=-1)) == E_SHAPE and f(L, _mat(M=(1 << 24) + 1)) == E_SHAPE
    for k in (0, 64, 100, -128, 32768 + 128):
        assert f(L, _mat(K=k)) == E_SHAPE
    for g in (0, 16, 48, 256, -64):
        assert f(L, _mat(group=g)) == E_SHAPE
    for p in ("codes", "steps"):
        assert f(L, _mat(**{p: None})) == E_NULL and f(L, _mat(**{p: MIS})) == E_ALIGN
    if name != "codes":
        assert f(L, dt=2) == E_DTYPE
    if name != "rows":
        assert f(L, _mat(M=0, codes=None, steps=None)) == OK
    assert {"pack": L.bitnet_pack_w4, "codes": L.bitnet_pack_w4_codes}.get(
        name, lambda *a: E_NULL)(FAKE, 0 if name == "pack" else FAKE, None, None) == E_NULL


def test_w4_operand_validation(L):
    assert W4["pack"](L, w=None) == E_NULL and W4["pack"](L, w=MIS) == E_ALIGN
    assert W4["codes"](L, w=None) == E_NULL and W4["codes"](L, s=None) == E_NULL
    assert W4["codes"](L, w=MIS) == E_ALIGN and W4["codes"](L, s=FAKE + 1) == E_ALIGN
    f = W4["rows"]
    assert f(L, n=-1) == E_SHAPE and f(L, n=(1 << 21) + 1) == E_SHAPE
    assert f(L, out=None) == E_NULL and f(L, out=MIS) == E_ALIGN and f(L, ids=FAKE + 2) == E_ALIGN
    assert f(L, n=0, out=None) == OK
    f = W4["linear"]
    assert f(L, N=-1) == E_SHAPE and f(L, N=(1 << 21) + 1) == E_SHAPE
    assert f(L, x=None) == E_NULL and f(L, y=None) == E_NULL
    assert f(L, x=MIS) == E_ALIGN and f(L, y=FAKE + 2) == E_ALIGN
    assert f(L, N=0, x=None, y=None) == OK and L.bitnet_last_error().decode() == ""
    need = L.bitnet_linear_w4_workspace(20, 20, 8192)
    big = lambda **kw: f(L, _mat(K=8192), N=20, **kw)  # noqa: E731
    assert need >= 2 * 20 * 20 * 4 and big() == E_NULL and big(ws=FAKE, wb=need - 1) == E_SHAPE
    assert f(L, ws=MIS) == E_ALIGN
    assert L.bitnet_linear_w4_workspace(16, 1 << 24, 32768) == 0 == L.bitnet_linear_w4_workspace(0, 5, 128)
    assert L.bitnet_linear_w4_workspace(16, 0, 32768) == 0
    for bad in ((-1, 5, 128), (5, -1, 128), (5, 5, 100), ((1 << 21) + 1, 5, 128), (5, (1 << 24) + 1, 128)):
        assert L.bitnet_linear_w4_workspace(*bad) == -1


def test_w4_binding_refuses():
    import ternary_weight_i2_amd as bn
    m = bn.W4Matrix.empty(20, 256, 64, device="cpu")
    assert m.codes.shape == (2, 2, 64, 16) and m.steps.shape == (2, 2, 16, 2) and (m.rows, m.k, m.group) == (20, 256, 64)
    assert bn.W4Matrix(m.codes, m.steps).rows == 32
    with pytest.raises(AttributeError):
        m.rows = 19
    for rows in (16, 33, 0, -1):
        with pytest.raises(ValueError):
            bn.W4Matrix(m.codes, m.steps, rows)
    for c, s in ((m.codes[:1], m.steps), (m.codes.view(2, 2, 16, 64), m.steps), (m.codes.to(torch.int8), m.steps),
                 (m.codes, m.steps.float()), (m.codes, m.steps[..., :0]), (m.codes, m.steps.view(2, 2, 32, 1)),
                 (m.codes.transpose(0, 1), m.steps)):
        with pytest.raises((TypeError, ValueError)):
            bn.W4Matrix(c, s, 20)
    for k, g in ((100, 64), (256, 16), (256, 256)):
        with pytest.raises(ValueError):
            bn.W4Matrix.empty(4, k, g, device="cpu")
    x = torch.zeros((3, 256))
    for bad in (x[:, :128], x[0], x.half(), torch.zeros((256, 3)).t(), x):    # the last: not on a GPU
        with pytest.raises((TypeError, ValueError)):
            bn.linear_w4(bad, m)
    with pytest.raises(ValueError):
        bn.linear_w4(x, m, out=torch.zeros((3, 21)))
    with pytest.raises(TypeError):
        bn.linear_w4(x, m, out=torch.zeros((3, 20), dtype=torch.bfloat16))
    for w, g in ((x[0], 64), (x.half(), 64), (x, 48), (x.t(), 64), (x[:, :100].contiguous(), 64), (x, 64)):
        with pytest.raises((TypeError, ValueError)):
            bn.pack_w4(w, g)
    with pytest.raises(ValueError):
        bn.pack_w4(x, 64, out=m)
    w, s = torch.zeros((3, 256), dtype=torch.int8), torch.zeros((3, 4), dtype=torch.float16)
    for a, b in ((w.int(), s), (w, s.float()), (w, s[:2]), (w, s[:, :3].contiguous()), (w, s[:, :0])):
        with pytest.raises((TypeError, ValueError)):
            bn.pack_w4_codes(a, b)
    with pytest.raises(TypeError):
        bn.w4_rows(m, torch.zeros(3, dtype=torch.int64))


@pytest.mark.parametrize("name", W4)
def test_w4_steps_in_either_order_validation(L, name):
    """A group may carry the order of the steps; nothing else beside its size is taken."""
    f, none = W4[name], dict(M=0, codes=None, steps=None)
    for g in (32, 64, 128):
        kw = {"rows": dict(n=0, out=None), "linear": dict(N=0, x=None, y=None)}.get(name, {})
        assert f(L, _mat(group=g | 0x1000, **(none if not kw else {})), **kw) == OK
    for g in (0x1000, 0x1000 | 48, 0x1000 | 256, 0x2000 | 64, 0x1800 | 64, (1 << 32) | 64):
        assert f(L, _mat(group=g)) == E_SHAPE


@pytest.mark.parametrize("group", [32, 64, 128])
def test_w4_matrix_takes_steps_in_either_order(group):
    import ternary_weight_i2_amd as bn
    m = bn.W4Matrix.empty(20, 256, group, device="cpu")
    by_group = bn.W4Matrix(m.codes, m.steps.transpose(2, 3).contiguous(), 20)
    for a in (m, by_group):
        assert (a.rows, a.k, a.group) == (20, 256, group)
    assert m._desc.group == group and by_group._desc.group in (group, group | 0x1000)
    assert group == 128 or by_group._desc.group == group | 0x1000
    for shape in ((2, 2, 3, 16), (2, 2, 16, 3), (2, 2, 8, 16), (2, 2, 16, 16), (2, 2, 4, 4), (2, 3, 4, 16), (1, 2, 4, 16)):
        with pytest.raises(TypeError):
            bn.W4Matrix(m.codes, torch.empty(shape, dtype=torch.float16), 20)
    with pytest.raises(ValueError):     # not laid out so
        bn.W4Matrix(m.codes, torch.empty((2, 2, 16, 4), dtype=torch.float16).transpose(2, 3), 20)


# ---------------------------------------------------------------- weights of cached tokens, eviction

def _weigh(L, b=None, q=FAKE, qs=256, dt=0, N=3, heads=4, scale=0.125, window=0, sinks=0, max_kv=64, w=FAKE,
           decay=1.0, out=FAKE, ws=FAKE, wb=1 << 20):
    return L.bitnet_kv4_weigh(b or _batch(), q, qs, dt, N, heads, scale, window, sinks, max_kv, w, decay, out, ws, wb,
                              None)


def test_weigh_validation(L):
    f = _weigh
    assert f(L, _batch(n_kv_heads=0)) == E_SHAPE and f(L, _batch(q_start=None)) == E_NULL
    assert f(L, dt=2) == E_DTYPE and f(L, N=-1) == E_SHAPE
    for heads in (0, 3, -2, 1026):
        assert f(L, heads=heads) == E_SHAPE
    for bad in (0.0, -1.0, float("inf"), float("nan")):
        assert f(L, scale=bad) == E_VALUE
    for bad in (-0.5, float("inf"), float("nan")):
        assert f(L, decay=bad) == E_VALUE
    for k in ("window", "sinks"):
        assert f(L, **{k: -1}) == E_SHAPE and f(L, **{k: 1 << 31}) == E_SHAPE
    assert f(L, max_kv=-1) == E_SHAPE and f(L, max_kv=193) == E_SHAPE
    for p in ("q", "out", "w", "ws"):
        assert f(L, **{p: None}) == E_NULL and f(L, **{p: MIS}) == E_ALIGN
    for bad in (255, 258, 0):
        assert f(L, qs=bad) == E_SHAPE
    need = L.bitnet_kv4_weigh_workspace(2, 3, 4, 2, 64, 64, 0, 0)
    assert need >= 3 * 4 * 8 and f(L, wb=need - 1) == E_SHAPE
    assert f(L, N=0, q=None, ws=None) == OK and f(L, _batch(n_seqs=0), q=None) == OK
    for bad in ((-1, 3, 4, 2, 64, 64, 0, 0), (2, -1, 4, 2, 64, 64, 0, 0), (2, 3, 3, 2, 64, 64, 0, 0),
                (2, 3, 4, 2, 64, -1, 0, 0), (2, 3, 4, 2, 64, (1 << 30) + 1, 0, 0), (2, 3, 4, 2, 64, 64, -1, 0),
                (2, 3, 4, 2, 64, 64, 0, -1), (2, 3, 4, 2, 96, 64, 0, 0)):
        assert L.bitnet_kv4_weigh_workspace(*bad) == -1
    assert L.bitnet_kv4_weigh_workspace(0, 3, 4, 2, 64, 64, 0, 0) == 0


def _evict(L, b=None, w=FAKE, nt=FAKE, cap=3, keep=64, sinks=4, recent=8, nl=FAKE, idx=FAKE, ws=None, wb=0):
    return L.bitnet_kv4_evict(b or _batch(q_start=None), w, nt, cap, keep, sinks, recent, nl, idx, ws, wb, None)


def test_evict_validation(L):
    f = _evict
    assert f(L, _batch(head_dim=80)) == E_SHAPE and f(L, _batch(table=None)) == E_NULL
    assert f(L, _batch(q_start=None, kv_len=FAKE + 2)) == E_ALIGN
    assert f(L, cap=0) == E_SHAPE and f(L, cap=(1 << 24) + 1) == E_SHAPE
    for keep in (0, -1, 193):
        assert f(L, keep=keep) == E_SHAPE
    for sinks, recent in ((-1, 0), (0, -1), (65, 0), (0, 65), (60, 5), (1 << 62, 1 << 62)):
        assert f(L, sinks=sinks, recent=recent) == E_SHAPE
    for p in ("w", "nt", "nl", "idx"):
        assert f(L, **{p: None}) == E_NULL
        assert f(L, **{p: MIS if p == "w" else FAKE + 2}) == E_ALIGN
    assert L.bitnet_kv4_evict(None, FAKE, FAKE, 3, 64, 0, 0, FAKE, FAKE, None, 0, None) == E_NULL
    assert f(L, _batch(n_seqs=0, q_start=None), w=None) == OK
    long = _batch(max_pages=4096)
    need = L.bitnet_kv4_evict_workspace(2, 2, 4096)
    assert need > 0 and f(L, long) == E_NULL and f(L, long, ws=FAKE, wb=need - 1) == E_SHAPE
    assert f(L, ws=MIS) == E_ALIGN
    assert L.bitnet_kv4_evict_workspace(2, 2, 3) == 0 == L.bitnet_kv4_evict_workspace(0, 2, 4096)
    for bad in ((-1, 2, 3), (2, 0, 3), (2, 2, 0), (2, 1025, 3), (2, 2, (1 << 24) + 1)):
        assert L.bitnet_kv4_evict_workspace(*bad) == -1


def test_evict_in_place_is_refused(L):
    """Heads that have not begun still read kv_len, and every page of the table."""
    other = FAKE + 4096
    for nl in (FAKE, FAKE + 4, FAKE - 4):   # two sequences
        assert _evict(L, nt=other, nl=nl) == E_VALUE
    assert _evict(L, nl=other) == E_VALUE


def test_weigh_and_evict_binding_refuses():
    import ternary_weight_i2_amd as bn
    c, table = torch.zeros((2, 1, 72 * 64), dtype=torch.uint8), torch.zeros((1, 1), dtype=torch.int32)
    one, start = torch.ones(1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    q, w = torch.zeros((1, 2, 64)), torch.zeros((2, 1, 64))
    assert bn.kv4_weights(c).shape == (2, 1, 64)
    for bad in (dict(w=w[:1]), dict(w=w.bfloat16()), dict(q=q[0]), dict(q=q.half()), dict(out=w[:1]),
                dict(ws=torch.empty(3, dtype=torch.uint8)), dict()):
        with pytest.raises((ValueError, TypeError)):
            bn.kv4_weigh(bad.get("w", w), bad.get("q", q), c, table, one, start, out=bad.get("out"),
                         workspace=bad.get("ws"))
    for bad in (dict(w=None), dict(w=w[:1]), dict(nt=None), dict(nt=table[0]), dict(nt=table.long()), dict(kv=one.long()),
                dict(nt=torch.zeros((2, 1), dtype=torch.int32)), dict(out=(one, one)), dict()):
        with pytest.raises((ValueError, TypeError)):
            bn.kv4_evict(c, bad.get("w", w), table, bad.get("kv", one), bad.get("nt", table), 5, out=bad.get("out"))
    from ternary_weight_i2_amd import _binding
    for k in (dict(weights=w), dict()):   # an offset is only for a Rotary
        with pytest.raises((ValueError, TypeError)):
            bn.attn_block(torch.zeros((1, 256)), *[(torch.zeros((64, 64), dtype=torch.uint8), 1.0)] * 4, c, table, one,
                          start, offset=one, **k)
    assert _binding.kv4_weigh_workspace(1, 1, 2, 1, 64, 64) > 0
    with pytest.raises(bn.BitnetError):
        _binding.kv4_weigh_workspace(1, 1, 3, 2, 64, 64)
