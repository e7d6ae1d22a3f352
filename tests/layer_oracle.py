"""The block boundary, the 4-bit cache and its attention from their definitions
in include/bitnet_i2s.h, in numpy: binary64 throughout, rounded to fewer bits only
where the definition rounds.  Shares no code with the library."""
import numpy as np

F4, F8 = np.float32, np.float64
PAGE, GROUP, TOP = 64, 64, F4(57344)


def bf16(a):
    """fp32 values rounded to bf16 (half to even), as fp32."""
    u = np.ascontiguousarray(a, F4).view(np.uint32).astype(np.uint64)
    u = (u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000
    return u.astype(np.uint32).view(F4)


def times(a, b):
    return (np.asarray(a, F8) * np.asarray(b, F8)).astype(F4)


# ---------------------------------------------------------------- the boundary

def norm_factor(x, eps):
    return (1 / np.sqrt((x.astype(F8) ** 2).sum(1, keepdims=True) / x.shape[1] + F8(F4(eps)))).astype(F4)


def block_norm(b, res=None, post=False, post_gamma=None, gate=None, scale=1.0, gamma=None,
               eps=1e-5, stream_bf16=False):
    """-> (h, v fp32, xq, s, xsum)."""
    t = b.astype(F4)
    if post:
        t = times(t, norm_factor(t, eps))
        if post_gamma is not None:
            t = times(t, post_gamma)
    if gate is not None:
        t = times(t, gate)
    t = times(t, F4(scale))
    h = None
    if res is not None:
        t = (res.astype(F8) + t.astype(F8)).astype(F4)
        h = t = bf16(t) if stream_bf16 else t
    v = times(t, norm_factor(t, eps))
    if gamma is not None:
        v = times(v, gamma)
    s = (127.0 / np.maximum(np.abs(v).max(1), F4(1e-5)).astype(F8)).astype(F4)
    xq = np.clip(np.rint(times(v, s[:, None])), -128, 127).astype(np.int8)
    return h, v, xq, s, xq.astype(np.int32).sum(1, dtype=np.int32)


# ---------------------------------------------------------------- the cache

def quantise(x):
    """x[..., dim] -> codes [..., groups, 64], step and mid [..., groups] (fp16)."""
    x = np.where(np.isnan(x), -TOP, np.clip(x.astype(F4), -TOP, TOP))
    x = x.reshape(*x.shape[:-1], -1, GROUP)
    lo, hi = x.min(-1), x.max(-1)
    mid = (lo + (hi - lo) * F4(8 / 15)).astype(np.float16)
    m = mid.astype(F4)
    step = np.maximum((hi - m) * F4(1 / 7), (m - lo) / F4(8)).astype(np.float16)
    with np.errstate(divide="ignore"):
        inv = np.where(step > 0, F4(1) / step.astype(F4), F4(0))
    code = np.clip(np.rint((x - m[..., None]) * inv[..., None] + F4(8)), 0, 15)
    return code.astype(np.uint8), step, mid


def put(rec, t, key, value):
    """Write one token (key and value rows of dim) into a record's bytes, in place."""
    d = key.size
    g = d // 64
    code, step, mid = quantise(key)
    c = code.reshape(d)
    for ch in range(d):
        j, i, e = ch // 32, ch % 32 // 8, ch % 8
        at = t * d // 2 + (i * (d // 32) + j) * 4 + e // 2
        rec[at] = (rec[at] & (0xF0 if e % 2 == 0 else 0x0F)) | (int(c[ch]) << (4 * (e % 2)))
    pair = np.stack([step, mid], -1).astype("<f2").tobytes()
    rec[64 * d + t * 4 * g:64 * d + (t + 1) * 4 * g] = np.frombuffer(pair, np.uint8)
    code, step, mid = quantise(value)
    c = code.reshape(d)
    for ch in range(d):
        p, i, e = ch // 64, ch % 64 // 4, ch % 4
        at = 32 * d + 2 * ((((t // 4) * 16 + i) * g + p) * 4 + t % 4) + e // 2
        rec[at] = (rec[at] & (0xF0 if e % 2 == 0 else 0x0F)) | (int(c[ch]) << (4 * (e % 2)))
    for p in range(g):
        for kind, x in ((0, step), (1, mid)):
            at = 68 * d + 2 * (((t // 4) * g + p) * 8 + 4 * kind + t % 4)
            rec[at:at + 2] = np.frombuffer(x[p:p + 1].astype("<f2").tobytes(), np.uint8)


def rows_of(kv_len, q_start, b, max_pages):
    """[(row, position)] of sequence b."""
    n = int(q_start[b + 1] - q_start[b])
    held = min(max(int(kv_len[b]), 0), PAGE * max_pages)
    return [(int(q_start[b]) + i, held - n + i) for i in range(n)], held


def append(cache, table, kv_len, q_start, k, v):
    """cache [pages][heads][72 dim] uint8, in place."""
    for b in range(len(kv_len)):
        for r, pos in rows_of(kv_len, q_start, b, table.shape[1])[0]:
            if pos < 0:
                continue
            page = table[b, pos // PAGE]
            if 0 <= page < len(cache):
                for h in range(cache.shape[1]):
                    put(cache[page, h], pos % PAGE, k[r, h], v[r, h])


def record(rec, d):
    """One record -> (codes, step, mid) of keys, and of values: [64][d], [64][g], [64][g]."""
    g = d // 64
    kw = rec[:32 * d].copy().view("<u4").reshape(PAGE, 4, d // 32)
    kc, vc = np.empty((PAGE, d), np.int64), np.empty((PAGE, d), np.int64)
    for j in range(d // 32):
        for i in range(4):
            for e in range(8):
                kc[:, 32 * j + 8 * i + e] = (kw[:, i, j] >> (4 * e)) & 15
    vw = rec[32 * d:64 * d].copy().view("<u2").reshape(16, 16, g, 4)
    for p in range(g):
        for i in range(16):
            for e in range(4):
                vc[:, 64 * p + 4 * i + e] = ((vw[:, i, p] >> (4 * e)) & 15).reshape(-1)
    km = rec[64 * d:68 * d].copy().view("<f2").reshape(PAGE, g, 2).astype(F8)
    vm = rec[68 * d:].copy().view("<f2").reshape(16, g, 2, 4).transpose(0, 3, 1, 2)
    vm = vm.reshape(PAGE, g, 2).astype(F8)
    return (kc, km[..., 0], km[..., 1]), (vc, vm[..., 0], vm[..., 1])


def value(code, step, mid):
    g = step.shape[-1]
    c = code.reshape(*code.shape[:-1], g, GROUP).astype(F8) - 8
    return (mid[..., None] + step[..., None] * c).reshape(code.shape)


def history(cache, table_row, held, head, d):
    """Positions 0 .. held-1 of one sequence and head: keys, values (binary64), whether
    the page is there, and the values' magnitudes |mid| + 8 step that rounding goes by."""
    k, v, there, mag, kmag = [], [], [], [], []
    for p in range(-(-held // PAGE)):
        page = table_row[p]
        if not 0 <= page < len(cache):
            k.append(np.zeros((PAGE, d))); v.append(np.zeros((PAGE, d)))
            mag.append(np.zeros((PAGE, d))); kmag.append(np.zeros((PAGE, d)))
            there.append(np.zeros(PAGE, bool))
            continue
        (kc, ks, km), (vc, vs, vm) = record(cache[page, head], d)
        with np.errstate(invalid="ignore", over="ignore"):
            k.append(value(kc, ks, km)); v.append(value(vc, vs, vm))
            mag.append(np.repeat(np.abs(vm) + 8 * vs, GROUP, 1))
            kmag.append(np.repeat(np.abs(km) + 8 * ks, GROUP, 1))
        there.append(np.ones(PAGE, bool))
    cat = lambda x: np.concatenate(x)[:held] if x else np.zeros((0, d))  # noqa: E731
    return cat(k), cat(v), (np.concatenate(there)[:held] if there else np.zeros(0, bool)), cat(mag), cat(kmag)


def read(cache, table, kv_len, q_start, n, d):
    """-> (k, v) [n][heads][d] fp32, NaN in rows that belong to no sequence."""
    heads = cache.shape[1]
    out = [np.full((n, heads, d), np.nan, F4) for _ in range(2)]
    for b in range(len(kv_len)):
        rows, held = rows_of(kv_len, q_start, b, table.shape[1])
        for h in range(heads):
            k, v = history(cache, table[b], held, h, d)[:2]
            for r, pos in rows:
                out[0][r, h] = k[pos] if pos >= 0 else 0
                out[1][r, h] = v[pos] if pos >= 0 else 0
    return out


def attention(q, cache, table, kv_len, q_start, scale, window=0, sinks=0, half=False, only=None):
    """-> (out binary64 [N][heads][d], bound on what the kernel may be off by); NaN
    in rows of no sequence, and in those that `only` (a set of (row, head)) leaves out.  The bound is six standard deviations of roundings taken as
    independent, each at its largest, and the bf16 result's half step, 2^-8 of it:

    * weight t is off, relatively, by e_t, with e_t^2 the sum of
      - (2^-22 scale |q * mag_t|_2)^2: q is carried in 22 bits (bf16's 8 bits are exact),
        mag = |mid| + 8 step being what a channel's two terms are made of;
      - n (2^-24 scale sum_d |q_d| mag_td)^2: the logit's n = D + 2 D/64 + 4 fp32 sums;
      - (2^-22 + 2^-22 |x_t|)^2: 2^z, its argument, and the constants in it;
      so the result is off by the root of sum_t (p_t e_t (|v_t| + |out|))^2 / den;
    * p step is carried in 22 or, for bf16 calls, 11 bits: the root of
      sum_t (2^-22 or 2^-11 p_t mag_t)^2 / den;
    * T + 64 fp32 sums, numerator and denominator: 2^-24 sqrt(T + 64) sum_t p_t (mag_t + |out|) / den.
    """
    N, heads, d = q.shape
    kvh = cache.shape[1]
    out, tol = np.full(q.shape, np.nan), np.full(q.shape, np.nan)
    u = 2.0 ** -24
    for b in range(len(kv_len)):
        rows, held = rows_of(kv_len, q_start, b, table.shape[1])
        for g in range(kvh):
            k, v, there, mag, kmag = history(cache, table[b], held, g, d)
            for r, pos in rows:
                if only is not None and not any((r, h) in only for h in range(g * heads // kvh, (g + 1) * heads // kvh)):
                    continue
                j = np.arange(held)
                see = there & (j <= pos)
                if window:
                    see &= (j > pos - window) | (j < sinks)
                for h in range(g * heads // kvh, (g + 1) * heads // kvh):
                    if only is not None and (r, h) not in only:
                        continue
                    if not see.any():
                        out[r, h] = 0
                        tol[r, h] = 0
                        continue
                    qr = q[r, h].astype(F8)
                    x = scale * (k[see] @ qr)
                    top = x.max()
                    p = np.exp(x - top)
                    den = p.sum()
                    out[r, h] = (p @ v[see]) / den
                    qa = np.abs(qr)
                    e2 = (4 * u * scale) ** 2 * (kmag[see] ** 2 @ qa ** 2)
                    e2 += (d + 2 * (d // 64) + 4) * (u * scale * (kmag[see] @ qa)) ** 2
                    e2 += (4 * u) ** 2 * (1 + np.abs(x)) ** 2
                    o = np.abs(out[r, h])
                    var = (p * p * e2) @ (np.abs(v[see]) + o) ** 2
                    var += ((2.0 ** -11 if half else 4 * u) * p) ** 2 @ mag[see] ** 2
                    var += (see.sum() + 64) * (u * (p @ (mag[see] + o))) ** 2
                    tol[r, h] = 6 * np.sqrt(var) / den
                    if half:
                        tol[r, h] += 2.0 ** -8 * np.abs(out[r, h])
    return out, tol
