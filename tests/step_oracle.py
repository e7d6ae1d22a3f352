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
