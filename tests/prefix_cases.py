"""Inputs for shared prefixes whose results are known to fp16's last bit: keys and queries that the codes hold exactly, with
scores that depend on one dim, and values of unlike sizes tile by tile.  Test infrastructure only."""
import numpy as np

from oracle import codec, paged as op

KEYS = 128   # of a tile


def tops(climb):
    """Where every tile's largest score lies, in units of log2: climb[t] above the one before."""
    return np.cumsum(np.asarray(climb, float))


def codes_exactly(x):
    """[n][d] values, the first dim of each group its smallest and the second its largest, as codes that stand for them."""
    c, mn, sc = codec.quantize_g64(x.astype(np.float16))
    return c, mn, sc


def rows_of(level, d, step=1.0 / 8):
    """Keys whose dim 2 is level * step and whose other dims are the ends of a range that holds it exactly: the codes are
    0 .. 15 of a power of two."""
    n = len(level)
    k = np.zeros((n, d))
    unit = step * 2.0 ** np.ceil(np.log2(np.maximum(np.abs(level), 1)))   # a code is worth unit / 8
    for g in range(d // 64):
        k[:, 64 * g], k[:, 64 * g + 1] = -unit, unit * 7 / 8
    k[:, 2] = np.round(level * step / (unit / 8)) * (unit / 8)
    return k


def attention(q, k, v, scale):
    """Rows of one head in 64 bits."""
    s = q @ k.T * scale
    p = np.exp(s - s.max(1, keepdims=True))
    return p @ v / p.sum(1, keepdims=True)


def rescaled(q, k, v, scale, fault=None, lift=4.0, most=15.0):
    """The same as a running sum over tiles of 128 keys whose weights are held against the known maximum, which is replaced
    where a weight passes 2^15; weights and values as fp16 and what that leaves.  fault: what is done wrong."""
    if fault == "zeros":
        return np.zeros((len(q), v.shape[1]))
    z = q @ k.T * scale / np.log(2.0)
    half = lambda x: x.astype(np.float16).astype(np.float64)
    vh = half(v)
    vl = half(v - vh)
    rows, d = q.shape[0], v.shape[1]
    hi, lo, low, l = np.zeros((rows, d)), np.zeros((rows, d)), np.zeros((rows, d)), np.zeros((rows, 1))
    neg = lift - z[:, :KEYS].max(1, keepdims=True)
    for t in range(0, len(k), KEYS):
        top = z[:, t:t + KEYS].max(1, keepdims=True)
        new = np.where(top + neg > most, lift - top, neg)
        f = 2.0 ** (new - neg)
        if fault == "rescale lost":
            f = 1.0 + 0 * f
        if fault == "rescale doubled":
            f = f * f
        l *= 1.0 if fault == "normaliser not rescaled" else f
        hi *= f
        lo *= 1.0 if fault == "remainders of weights not rescaled" else f
        low *= 1.0 if fault == "remainders of values not rescaled" else f
        neg = new
        w = 2.0 ** (z[:, t:t + KEYS] + neg)
        wh = half(np.minimum(w, 65504))
        wl = half(w - wh)
        l += w.sum(1, keepdims=True)
        hi += wh @ vh[t:t + KEYS]
        lo += 0.0 if fault == "no remainders of weights" else wl @ vh[t:t + KEYS]
        low += 0.0 if fault == "no remainders of values" else wh @ vl[t:t + KEYS]
    return (hi + lo + low) / l


def climbing(climb, d, rows, seed):
    """Queries, codes of keys and of values of a head: scores climb from tile to tile by climb (log2), and values fall as fast,
    so that every tile within 2^13 of the last counts as much."""
    rng = np.random.default_rng(seed)
    top = tops(climb)
    level = (top[:, None] - rng.integers(0, 3, (len(climb), KEYS))).reshape(-1)
    k = codes_exactly(rows_of(level, d))
    size = np.repeat(2.0 ** np.clip(top[-1] - top, 0, 13), KEYS)
    v = codes_exactly(size[:, None] * rng.normal(size=(len(level), d)))
    # one dim of q, ln 2 a unit of the level: scores are near whole numbers of log2
    q = np.zeros((rows, d))
    q[:, 2] = np.log(2.0) * np.sqrt(d) * 8 * (1 + 0.02 * rng.integers(-1, 2, rows))
    return q.astype(np.float16), k, v


CLIMBS = {   # a weight passes 2^15 where the climb since the last maximum is 12 or more
    "none": [0] * 8,
    "one of 13": [0, 0, 13, 0, 0],
    "of 5 and 8": [0, 5, 0, 8, 0, 0],
    "of 10, which stays": [0, 0, 10, 0, 0],
    "of 40, then of 13": [0, 40, 0, 13, 0, 0],
    "downwards": [0, -6, -3, 0],
}
FAULTS = ("zeros", "rescale lost", "rescale doubled", "normaliser not rescaled", "remainders of weights not rescaled",
          "remainders of values not rescaled", "no remainders of weights", "no remainders of values")
# Elements that are not the nearest fp16: a score's roundings (fp32, of terms up to 2^6: 2^-18), the weight's exponential
# (2^-22) and fp32 sums leave an error of about 2^-17 of the result, in the mean 1 / 100 of a step of fp16 (2^-10 to 2^-11
# of the value), and as large a share of other roundings; a sixteenth is allowed.
MOST = 1.0 / 16
