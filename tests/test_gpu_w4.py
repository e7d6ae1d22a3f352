"""GPU tests of the matrices of 4-bit weights: quantiser and rows bit for bit, products against
binary64 (tests/step_oracle.py) and, where every sum is an integer below 2^24, exactly."""
import numpy as np
import pytest
import torch

import layer_oracle as lo
import step_oracle as so
from test_gpu_layer import BF16, F32, dev, host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bn():
    import ternary_weight_i2_amd as m
    return m


def check_matrix(mat, codes, steps):
    c, s = so.w4_layout(codes, steps)
    assert np.array_equal(mat.codes.cpu().numpy(), c)
    assert np.array_equal(mat.steps.cpu().numpy().view(np.uint16), s.view(np.uint16))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,K", [(1, 128), (16, 256), (17, 640), (50, 1152)])
def test_pack(bn, dtype, group, M, K):
    rng = np.random.default_rng([M, K, group])
    w = host(dev((rng.standard_normal((M, K)) * 0.02 * np.exp(rng.standard_normal((M, 1)))).astype(np.float32), dtype))
    mat = bn.pack_w4(dev(w, dtype), group)
    codes, steps = so.w4_quantise(w, group)
    check_matrix(mat, codes, steps)
    want = so.w4_values(codes, steps).astype(np.float32)    # 11 bits times 4: exact
    assert np.array_equal(host(bn.w4_rows(mat)), want)
    assert np.array_equal(host(bn.w4_rows(mat, dtype=BF16)), lo.bf16(want))
    again = bn.pack_w4_codes(dev(codes), dev(steps))
    assert torch.equal(again.codes, mat.codes) and torch.equal(again.steps, mat.steps)


def test_pack_of_special_groups(bn):
    rng = np.random.default_rng(1)
    w = rng.standard_normal((16, 128)).astype(np.float32)
    w[0] = 0
    w[1] = np.abs(w[1]) + 1
    w[2] = -np.abs(w[2]) - 1
    w[3, 5], w[3, 70], w[3, 100] = np.nan, np.inf, -np.inf
    w[4] *= 1e-8
    w[5] *= 1e-6
    w[6] = 3e38
    w[7] = np.where(np.arange(128) % 2, 7.0, -8.0)
    w[8] = np.arange(128) % 16 - 8
    w[9] = -0.0
    w[10] = 3.5 * (np.arange(128) % 3 - 1)       # ties of the rounding
    for group in (32, 64, 128):
        codes, steps = so.w4_quantise(w, group)
        mat = bn.pack_w4(dev(w), group)
        check_matrix(mat, codes, steps)
        assert torch.isfinite(bn.w4_rows(mat)).all()


def test_given_codes_are_held(bn):
    w = np.arange(-128, 128, dtype=np.int8).reshape(2, 128)
    steps = np.array([[-0.5], [np.inf]], np.float16)
    mat = bn.pack_w4_codes(dev(w), dev(steps))
    check_matrix(mat, np.clip(w, -8, 7), steps)


def test_rows_by_id(bn):
    rng = np.random.default_rng(2)
    w = rng.standard_normal((37, 256)).astype(np.float32)
    mat = bn.pack_w4(dev(w), 32)
    all_rows = host(bn.w4_rows(mat))
    ids = np.array([36, 0, 5, 5, -1, 37, 40, 47, 48, 2 ** 31 - 1, -2 ** 31, 16], np.int32)
    got = host(bn.w4_rows(mat, dev(ids)))
    for i, r in enumerate(ids):
        assert np.array_equal(got[i], all_rows[r] if 0 <= r < 37 else np.zeros(256, np.float32))


SHAPES = [(1, 128), (15, 256), (16, 640), (33, 1024), (100, 2560), (700, 384), (257, 6912), (40, 16384), (20, 32768),
          (4500, 256)]


@pytest.mark.parametrize("M,K", SHAPES)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_products_of_integers_are_exact(bn, dtype, M, K):
    """Channels up to 15 (bf16) or 2^16 + 1 (fp32, which needs both terms), codes times steps of 1
    and 2; a token has few channels that are not zero, so every sum stays below 2^24."""
    rng = np.random.default_rng([M, K])
    group = (32, 64, 128)[K // 128 % 3]
    codes = rng.integers(-8, 8, (M, K)).astype(np.int8)
    steps = rng.choice([1.0, 2.0, -1.0, 0.0], (M, K // group)).astype(np.float16)
    mat = bn.pack_w4_codes(dev(codes), dev(steps))
    top = 15 if dtype is BF16 else 2 ** 16 + 1
    for N in (1, 2, 3, 4, 5, 7, 8, 9, 16, 17, 31, 33, 64, 65, 130):
        x = np.zeros((N, K), np.float32)
        for t in range(N):
            at = rng.permutation(K)[:min(K, 8)]
            x[t, at] = rng.integers(-top, top + 1, len(at))
        y = bn.linear_w4(dev(x, dtype), mat)
        want = x.astype(np.float64) @ so.w4_values(codes, steps).T
        assert np.array_equal(host(y), want.astype(np.float32)), N


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("N,M,K", [(1, 2560, 2560), (1, 33, 128), (3, 70, 1152), (16, 300, 2560), (20, 48, 8192),
                                   (48, 100, 1024), (64, 530, 4096), (200, 90, 640), (1, 9000, 512)])
def test_products(bn, dtype, group, N, M, K):
    rng = np.random.default_rng([N, M, K])
    w = (0.02 * rng.standard_normal((M, K))).astype(np.float32)
    mat = bn.pack_w4(dev(w), group)
    x = rng.standard_normal((N, K)) * (1 + 30 * (rng.random(K) < 0.01)) * np.exp(rng.standard_normal((N, 1)))
    x = host(dev(x.astype(np.float32), dtype))
    y = host(bn.linear_w4(dev(x, dtype), mat))
    want, tol = so.w4_linear(x, so.w4_values(*so.w4_quantise(w, group)), group, dtype is BF16)
    assert (np.abs(y - want) <= tol).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_products_of_values_of_very_different_sizes(bn, dtype):
    """Blocks of 1e-30 next to blocks of 1e30, a token of zeros, a token of subnormals, steps of every size that fp16 has."""
    rng = np.random.default_rng(3)
    M, K = 40, 512
    codes = rng.integers(-8, 8, (M, K)).astype(np.int8)
    steps = np.exp(rng.uniform(np.log(6e-8), np.log(60000), (M, K // 64))).astype(np.float16)
    mat = bn.pack_w4_codes(dev(codes), dev(steps))
    x = rng.standard_normal((6, K)).astype(np.float32)
    x[1] = 0
    x[2] *= np.repeat([1e-30, 1, 1e30, 1e-10], 128).astype(np.float32)
    x[3] *= 1e-39
    x[4] *= 1e33
    x[5, ::2] *= 1e-6
    x = host(dev(x, dtype))
    y = host(bn.linear_w4(dev(x, dtype), mat))
    want, tol = so.w4_linear(x, so.w4_values(codes, steps), 64, dtype is BF16)
    # token 3: below 2^-111 the scale that makes the largest 2^14 is none, 2^126 is; its terms end
    # at 2^-25 of that, and sums of subnormals at 2^-150
    tol[3] += (2.0 ** -151 + 2.0 ** -150) * (np.abs(so.w4_values(codes, steps)).sum(1) + 2 * K)
    # y is fp32: where sum |x weight| reaches 2^127 a partial sum may not fit: most of token 4's rows
    fits = np.abs(x.astype(np.float64)) @ np.abs(so.w4_values(codes, steps)).T < 2.0 ** 127
    assert fits[[0, 1, 2, 3, 5]].all() and fits[4].any()
    assert (np.abs(y - want) <= tol)[fits].all()


def test_a_token_that_is_no_number_spoils_no_other(bn):
    rng = np.random.default_rng(4)
    mat = bn.pack_w4(dev(rng.standard_normal((50, 384)).astype(np.float32)))
    for N in (3, 20, 50):
        x = rng.standard_normal((N, 384)).astype(np.float32)
        clean = bn.linear_w4(dev(x), mat)
        x[1, 7], x[2, 200] = np.nan, np.inf
        got = bn.linear_w4(dev(x), mat)
        keep = [i for i in range(N) if i not in (1, 2)]
        assert torch.equal(got[keep], clean[keep])
        assert not torch.isfinite(got[1:3]).any()


def test_any_batch_gives_close_results_and_the_same_call_the_same_bits(bn):
    rng = np.random.default_rng(5)
    mat = bn.pack_w4(dev((0.02 * rng.standard_normal((640, 2560))).astype(np.float32)))
    x = rng.standard_normal((70, 2560)).astype(np.float32)
    xd = dev(x)
    want, tol = so.w4_linear(x, host(bn.w4_rows(mat)), 64, False)
    for N in (1, 5, 16, 30, 64, 70):
        a, b = bn.linear_w4(xd[:N], mat), bn.linear_w4(xd[:N], mat)
        assert torch.equal(a, b) and (np.abs(host(a) - want[:N]) <= tol[:N]).all()


def test_outputs_and_nothing_around_them(bn):
    rng = np.random.default_rng(6)
    for M, N in ((50, 3), (16, 40)):
        mat = bn.pack_w4(dev(rng.standard_normal((M, 256)).astype(np.float32)))
        x = dev(rng.standard_normal((N, 256)).astype(np.float32))
        buf = torch.full((N * M + 64,), 7.0, device="cuda")
        out = buf[32:32 + N * M].view(N, M)
        assert bn.linear_w4(x, mat, out=out) is out
        assert torch.equal(out, bn.linear_w4(x, mat))
        assert (buf[:32] == 7).all() and (buf[32 + N * M:] == 7).all()


def test_captured_and_on_another_stream(bn):
    rng = np.random.default_rng(7)
    mat = bn.pack_w4(dev(rng.standard_normal((900, 1024)).astype(np.float32)))
    xs = [dev(rng.standard_normal((n, 1024)).astype(np.float32)) for n in (1, 20, 64)]
    want = [bn.linear_w4(x, mat) for x in xs]
    outs = [torch.empty_like(w) for w in want]
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        for x, o in zip(xs, outs):
            bn.linear_w4(x, mat, out=o)
    st.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for x, o in zip(xs, outs):
            bn.linear_w4(x, mat, out=o)
    for _ in range(3):
        for o in outs:
            o.zero_()
        bn.linear_w4(xs[1], mat)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_shares_of_the_channels_and_given_scratch(bn, dtype):
    """Sizes for one share and for many, one tile of rows to a wave and two; scratch of any content."""
    rng = np.random.default_rng(8)
    for N, M, K in ((1, 100, 8192), (16, 3000, 4096), (5, 20000, 256), (3, 12000, 4480), (17, 40, 128), (20, 40, 32768), (64, 300, 12800), (33, 5000, 1408), (64, 4200, 2560), (130, 4100, 4096)):
        codes = rng.integers(-8, 8, (M, K)).astype(np.int8)
        steps = rng.choice([1.0, 2.0, -1.0], (M, K // 64)).astype(np.float16)
        mat = bn.pack_w4_codes(dev(codes), dev(steps))
        x = np.zeros((N, K), np.float32)
        for t in range(N):
            x[t, rng.permutation(K)[:16]] = rng.integers(-15, 16, 16)
        need = bn.linear_w4_workspace(N, M, K)
        ws = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device="cuda")
        y = bn.linear_w4(dev(x, dtype), mat, workspace=ws)
        assert np.array_equal(host(y), (x.astype(np.float64) @ so.w4_values(codes, steps).T).astype(np.float32))
        assert (ws[need:] == 0xFF).all()
        if need:
            with pytest.raises(ValueError):
                bn.linear_w4(dev(x, dtype), mat, workspace=ws[:need - 1])


def test_nothing_to_multiply(bn):
    mat = bn.pack_w4(torch.ones((20, 128), device="cuda"))
    assert bn.linear_w4(torch.empty((0, 128), device="cuda"), mat).shape == (0, 20)
    assert bn.w4_rows(mat, torch.empty(0, dtype=torch.int32, device="cuda")).shape == (0, 128)
    none = bn.pack_w4(torch.empty((0, 128), device="cuda"))
    assert none.rows == 0 and bn.linear_w4(torch.ones((3, 128), device="cuda"), none).shape == (3, 0)
    assert (bn.w4_rows(none, torch.zeros(2, dtype=torch.int32, device="cuda")) == 0).all()


def by_group(bn, mat):
    return bn.W4Matrix(mat.codes, mat.steps.transpose(2, 3).contiguous(), mat.rows)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_steps_that_lie_group_by_group(bn, dtype, group):
    """Packed and read in either order of the steps, a matrix is the same, bit for bit, and so are
    its products, in every form of launch."""
    rng = np.random.default_rng([9, group])
    w = rng.standard_normal((37, 640)).astype(np.float32)
    mat = bn.pack_w4(dev(w, dtype), group)
    other = by_group(bn, mat)
    into = bn.W4Matrix(torch.empty_like(other.codes), torch.empty_like(other.steps), 37)
    assert bn.pack_w4(dev(w, dtype), group, out=into) is into
    assert torch.equal(into.codes, other.codes) and torch.equal(into.steps, other.steps)
    codes, steps = so.w4_quantise(host(dev(w, dtype)), group)
    into.codes.zero_()
    into.steps.zero_()
    bn.pack_w4_codes(dev(codes), dev(steps), out=into)
    assert torch.equal(into.codes, other.codes) and torch.equal(into.steps, other.steps)
    ids = dev(np.array([36, 0, -1, 37, 16, 15], np.int32))
    assert torch.equal(bn.w4_rows(other), bn.w4_rows(mat)) and torch.equal(bn.w4_rows(other, ids), bn.w4_rows(mat, ids))
    for M, K in SHAPES + [(20000, 256), (12000, 4480), (4200, 2560)]:
        codes = rng.integers(-8, 8, (M, K)).astype(np.int8)
        steps = rng.choice([1.0, 2.0, -1.0, 0.5], (M, K // group)).astype(np.float16)
        mat = bn.pack_w4_codes(dev(codes), dev(steps))
        other, v = by_group(bn, mat), so.w4_values(codes, steps)
        for N in (1, 3, 4, 5, 8, 16, 20, 33, 64):
            x = np.zeros((N, K), np.float32)
            for t in range(N):     # every sum is a multiple of 1/2 below 2^22
                x[t, rng.permutation(K)[:8]] = rng.integers(-15, 16, 8)
            y = bn.linear_w4(dev(x, dtype), other)
            assert torch.equal(y, bn.linear_w4(dev(x, dtype), mat)), (M, K, N)
            if N in (1, 5, 20, 64):
                assert np.array_equal(host(y), (x.astype(np.float64) @ v.T).astype(np.float32)), (M, K, N)


@pytest.mark.parametrize("group", [32, 64])
def test_products_of_floats_with_steps_group_by_group(bn, group):
    rng = np.random.default_rng([10, group])
    for N, M, K in ((1, 2560, 2560), (5, 531, 1024), (64, 530, 4096)):
        w = (0.02 * rng.standard_normal((M, K))).astype(np.float32)
        mat = by_group(bn, bn.pack_w4(dev(w), group))
        x = (rng.standard_normal((N, K)) * (1 + 30 * (rng.random(K) < 0.01))).astype(np.float32)
        want, tol = so.w4_linear(x, so.w4_values(*so.w4_quantise(w, group)), group, False)
        assert (np.abs(host(bn.linear_w4(dev(x), mat)) - want) <= tol).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rows_of_steps_that_are_no_numbers(bn, dtype):
    """A NaN of any bits stays one when it is rounded to bf16."""
    codes = np.arange(-8, 8, dtype=np.int8).repeat(8)[None].repeat(6, 0)
    bits = np.array([[0x7FFF], [0xFFFF], [0x7E00], [0x7C01], [0xFDFF], [0x3C00]], np.uint16)
    got = host(bn.w4_rows(bn.pack_w4_codes(dev(codes), dev(bits.view(np.float16))), dtype=dtype))
    assert np.isnan(got[:5]).all() and np.array_equal(got[5], codes[5].astype(np.float32))
