"""The operators around a decode step from their definitions in include/bitnet_i2s.h, in
numpy: rotary positions, 4-bit weights, the weights that attention gave cached tokens,
and eviction by them.  binary64 or more, rounded to fewer bits only where a definition
rounds.  Shares no code with the library."""
import numpy as np

import layer_oracle as lo

F4, F8 = np.float32, np.float64


# ---------------------------------------------------------------- rotary positions

def turns_of(freqs):
    """Radians per position -> 64-bit fractions of a turn, as int64."""
    t = [int(f / (2 * np.pi) * 2.0 ** 64) % 2 ** 64 for f in freqs]
    return np.array([x - 2 ** 64 if x >= 2 ** 63 else x for x in t], np.int64)


def cos_sin(turns, positions, magnitude=1.0, sign=1):
    """[N][rot / 2] fp32 cosines and sines: the fraction of a turn in integers, the functions in
    extended precision (binary64 misses the nearest fp32 number once in 2^28)."""
    pos = np.asarray(positions, np.int64).astype(np.uint64)
    frac = (pos[:, None] * turns.view(np.uint64)).view(np.int64).astype(np.longdouble)
    angle = frac * (2 * np.longdouble("3.14159265358979323846264338327950288") / np.longdouble(2) ** 64)
    return ((magnitude * np.cos(angle)).astype(F4), (sign * magnitude * np.sin(angle)).astype(F4))


def rotate(x, turns, positions, interleaved=False, magnitude=1.0, inverse=False, half=False):
    """x [N][heads][dim] fp32 -> the turned rows (rounded to bf16 if half), fp32."""
    c, s = (a[:, None] for a in cos_sin(turns, positions, magnitude, -1 if inverse else 1))
    r = 2 * len(turns)
    a, b = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2), slice(r // 2, r))
    out = np.array(x, F4)
    with np.errstate(invalid="ignore"):
        p, q = lo.times(x[..., a], c), lo.times(x[..., b], s)
        out[..., a] = (p.astype(F8) - q.astype(F8)).astype(F4)
        p, q = lo.times(x[..., b], c), lo.times(x[..., a], s)
        out[..., b] = (p.astype(F8) + q.astype(F8)).astype(F4)
    return lo.bf16(out) if half else out


# ---------------------------------------------------------------- 4-bit weights

W4_TOP = F4(7 * 65504.0)


def w4_quantise(w, group):
    """w [M][K] -> codes [M][K] in -8..7 and steps [M][K / group] (fp16)."""
    w = np.where(np.isnan(w), F4(0), np.clip(np.asarray(w, F4), -W4_TOP, W4_TOP))
    g = w.reshape(w.shape[0], -1, group)
    # a step of 0 is +0: one of the two ends is
    step = (np.maximum(lo.times(g.max(2), F4(1 / 7)), lo.times(g.min(2), F4(-0.125))) + F4(0)).astype(np.float16)
    with np.errstate(divide="ignore"):
        inv = np.where(step > 0, F4(1) / step.astype(F4), F4(0))
    code = np.clip(np.rint(lo.times(g, inv[..., None])), -8, 7)
    return code.reshape(w.shape).astype(np.int8), step


def w4_layout(codes, steps):
    """codes [M][K] in -8..7, steps [M][K / group] -> the arrays that a matrix consists of."""
    M, K = codes.shape
    tiles, blocks, per = -(-M // 16), K // 128, 128 * steps.shape[1] // K
    c = np.zeros((16 * tiles, K), np.int64)
    c[:M] = codes
    s = np.zeros((16 * tiles, steps.shape[1]), np.float16)
    s[:M] = steps
    out = np.zeros((tiles, blocks, 64, 16), np.uint8)
    for quad in range(4):
        for row in range(16):
            for j in range(4):
                for e in range(8):
                    col = 128 * np.arange(blocks) + 32 * j + 8 * quad + e
                    code = (c[row::16][:, col] + 8).astype(np.uint8)
                    out[:, :, quad * 16 + row, 4 * j + e // 2] |= code << (4 * (e % 2))
    return out, s.reshape(tiles, 16, blocks, per).transpose(0, 2, 1, 3).copy()


def w4_values(codes, steps):
    return (codes.astype(F8).reshape(codes.shape[0], steps.shape[1], -1) * steps.astype(F8)[..., None]).reshape(codes.shape)


def w4_linear(x, w, group, half):
    """y in binary64 and a bound on what the product may be off by:
    * x is carried in two fp16 terms: hi is off by 2^-12 of its value, and what is left by
      2^-12 of that, 2^-24; 2^-23 covers both, and 2^-41 of the block's largest is the
      half step of the smallest fp16 at a largest of 2^15 (bf16: nothing, and 2^-40);
    * step * scale is exact; K + K / group + 16 fp32 roundings of at most 2^-24 of sum |x w|
      each, taken as independent: six standard deviations."""
    a, b = np.asarray(x, F8), np.asarray(w, F8)
    mag = np.abs(a) @ np.abs(b).T
    K = a.shape[1]
    top = np.abs(a.reshape(len(a), -1, 128)).max(2)
    tol = (0 if half else 2.0 ** -23) * mag
    tol += 2.0 ** (-40 if half else -41) * (top @ np.abs(b).reshape(len(b), -1, 128).sum(2).T)
    return a @ b.T, tol + 6 * np.sqrt(K + K // group + 16) * 2.0 ** -24 * mag


# ---------------------------------------------------------------- weights of cached tokens

def weigh(weights, q, cache, table, kv_len, q_start, scale, decay=1.0, window=0, sinks=0):
    """weights [pages][heads][64] -> (the new ones in binary64, what they may be off by, whether
    the call writes them).  What a row's weight p_t may be off by, relatively:
    * e_t, with e_t^2 the sum of (2^-22 scale |q * mag_t|_2)^2 (q in 22 bits, mag = |mid| + 8 step
      being what a channel's two terms are made of), n (2^-24 scale sum |q_d| mag_td)^2 (the logit's
      n = D + 2 D / 64 + 4 fp32 sums) and (2^-22 (1 + |x_t|))^2 (2^z and its argument);
    * and as much as its denominator, sum_s p_s e_s and the sum's own roundings, 2^-22.
    Six standard deviations of these, taken as independent between rows, and of the sums over
    rows, 2^-24 of the result each, of which there are the rows', 20 and the old weight's.  A
    weight below 2^-126 of its row's largest is none of fp32's normal numbers and may be 0."""
    N, heads, d = q.shape
    kvh = cache.shape[1]
    out, tol = np.array(weights, F8), np.zeros(weights.shape)
    written = np.zeros(weights.shape, bool)
    u = 2.0 ** -24
    for b in range(len(kv_len)):
        rows, held = lo.rows_of(kv_len, q_start, b, table.shape[1])
        if not rows:
            continue
        first = held - len(rows)
        j = np.arange(held)
        for g in range(kvh):
            k, _, there, _, kmag = lo.history(cache, table[b], held, g, d)
            got, var = np.zeros(held), np.zeros(held)
            for r, pos in rows:
                see = there & (j <= pos)
                if window:
                    see &= (j > pos - window) | (j < sinks)
                for h in range(g * heads // kvh, (g + 1) * heads // kvh):
                    qr = q[r, h].astype(F8)
                    if not see.any() or not np.isfinite(qr).all():
                        continue
                    x = scale * (k[see] @ qr)
                    p = np.exp(x - x.max())
                    p /= p.sum()
                    qa = np.abs(qr)
                    e = np.sqrt((4 * u * scale) ** 2 * (kmag[see] ** 2 @ qa ** 2)
                                + (d + 2 * (d // 64) + 4) * (u * scale * (kmag[see] @ qa)) ** 2
                                + (4 * u) ** 2 * (1 + np.abs(x)) ** 2)
                    got[see] += p
                    var[see] += (p * (e + p @ e + 4 * u)) ** 2
            at = (table[b, j // 64], g, j % 64)
            at = tuple(np.broadcast_to(a, j.shape)[there] for a in at)
            old = np.where((j < first)[there], decay * np.nan_to_num(weights[at].astype(F8)), 0.0) if decay else 0.0
            new = got[there] + old
            out[at], written[at] = new, True
            n = len(rows) * heads // kvh
            tol[at] = 6 * np.sqrt(var[there] + (n + 21) * (u * np.abs(new)) ** 2) + n * 2.0 ** -126
    return out, tol, written


def token_bytes(d, t):
    """Where a record has token t: the bytes of its key, then of its value, in order."""
    g = d // 64
    key = [t * d // 2 + i for i in range(d // 2)] + [64 * d + t * 4 * g + i for i in range(4 * g)]
    a, e = t // 4, t % 4
    code = [32 * d + 2 * (((a * 16 + i) * g + p) * 4 + e) + s for i in range(16) for p in range(g) for s in range(2)]
    pair = [68 * d + 2 * ((a * g + p) * 8 + 4 * kind + e) + s for p in range(g) for kind in range(2) for s in range(2)]
    return np.array(key + code + pair)


def evict(cache, weights, table, kv_len, new_table, keep, sinks=0, recent=0):
    """In place -> (new_len, index)."""
    pages, heads, d = len(cache), cache.shape[1], cache.shape[2] // 72
    B = len(kv_len)
    new_len, index = np.zeros(B, np.int32), np.full((B, heads, keep), -1, np.int32)
    before, w0 = cache.copy(), weights.copy()
    where = [token_bytes(d, t) for t in range(64)]
    for b in range(B):
        held = min(max(int(kv_len[b]), 0), 64 * table.shape[1])
        t = np.array([i for i in range(held) if 0 <= table[b, i // 64] < pages], np.int64)
        new_len[b] = min(len(t), keep)
        for h in range(heads):
            w = np.array([w0[table[b, i // 64], h, i % 64] for i in t], F8)
            w[np.isnan(w)] = -np.inf
            spared = (t < sinks) | (t >= held - recent)
            order = sorted(range(len(t)), key=lambda i: (not spared[i], -w[i] if not spared[i] else 0, t[i]))
            kept = np.sort(t[order[:new_len[b]]])
            index[b, h, :len(kept)] = kept
            for to, i in enumerate(kept):
                page = new_table[b, to // 64]
                if 0 <= page < pages:
                    cache[page, h, where[to % 64]] = before[table[b, i // 64], h, where[i % 64]]
                    weights[page, h, to % 64] = w0[table[b, i // 64], h, i % 64]
    return new_len, index
