"""The bounds that the paged attention is held to (oracle/paged.py, attention_bound) are wide enough for the kernels'
arithmetic and too narrow for a mistake of a token."""
import numpy as np
import pytest

from oracle import codec, paged as op

U = op.HALF


def _data(seed, n, d, rows, size=1.0):
    rng = np.random.default_rng(seed)
    k, v = (codec.quantize_g64((size * rng.normal(size=(n, d)) * (0.5 + rng.random(d))).astype(np.float16)) for _ in range(2))
    q = (1.3 * rng.normal(size=(rows, d))).astype(np.float16).astype(np.float64)
    return q, k, v


def _rounded(q, k, v, pos, window, sinks, kind):
    """The kernels' roundings, written out: weights to fp16 (steps), K, V and P to fp16 (chunks), the result to fp16."""
    kk, vv = op.restore(*k), op.restore(*v)
    if kind == "chunk":
        kk, vv = kk.astype(np.float16).astype(np.float64), vv.astype(np.float16).astype(np.float64)
    see = op.visible(pos, len(kk), window, sinks)
    s = np.where(see, q @ kk.T / np.sqrt(q.shape[1]), -np.inf)
    p = np.exp(s - s.max(axis=1, keepdims=True))
    total = p.sum(axis=1, keepdims=True)
    if kind == "chunk":
        o = (p * 16).astype(np.float16).astype(np.float64) @ vv / 16
    else:
        codes = codec.unpack_codes(v[0]).reshape(len(vv), -1, 64).astype(np.float64)
        o = np.zeros((len(q), codes.shape[1], 64))
        for g in range(codes.shape[1]):
            sc, mn = v[2][:, g].astype(np.float64), v[1][:, g].astype(np.float64)
            w = p * sc
            f = 2.0 ** (5 - np.floor(np.log2(w.max(axis=1, keepdims=True))))
            o[:, g] = (w * f).astype(np.float16).astype(np.float64) / f @ (codes[:, g] - 8) + (p @ (mn + 8 * sc))[:, None]
        o = o.reshape(len(q), -1)
    return (o / total).astype(np.float16).astype(np.float64)


@pytest.mark.parametrize("kind", ["step", "chunk"])
@pytest.mark.parametrize("n,d,rows,size", [(300, 128, 4, 1.0), (1000, 64, 8, 1.0), (300, 128, 16, 30.0), (40, 64, 1, 1e-3)])
def test_the_roundings_pass(kind, n, d, rows, size):
    q, k, v = _data(n, n, d, rows, size)
    pos = np.arange(n - rows, n)
    ref, tol = op.attention_bound(q, k, v, pos, 100, 3, kind=kind)
    assert op.off_by_too_much(_rounded(q, k, v, pos, 100, 3, kind), ref, tol, (2 if kind == "step" else 3) * U if size == 1 else None) is None


@pytest.mark.parametrize("kind", ["step", "chunk"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("seed", range(4))
def test_a_mistake_of_a_token_does_not(kind, d, seed):
    n, rows = 300, 4
    q, k, v = _data(seed, n, d, rows)
    pos = np.arange(n - rows, n)
    ref, tol = op.attention_bound(q, k, v, pos, 100, 3, kind=kind)
    limit = (2 if kind == "step" else 3) * U
    kv, vv = op.restore(*k), op.restore(*v)

    def refused(window=100, sinks=3, pos=pos, present=None, k=kv, v=vv):
        got = op.attention(q, k, v, pos, window, sinks, present)[0].astype(np.float16).astype(np.float64)
        return op.off_by_too_much(got, ref, tol, limit) is not None

    assert not refused()
    assert refused(window=99) and refused(window=101)
    assert refused(sinks=0) and refused(sinks=2) and refused(sinks=4)
    assert refused(pos=pos - 1)
    score = (q @ kv[250:296].T).sum(axis=0)                   # tokens that every row sees; the median of them
    for lost in (0, 250, 250 + int(np.argsort(score)[len(score) // 2])):
        there = np.ones(n, bool)
        there[lost] = False
        assert refused(present=there)
    other = vv.copy()
    other[[230, 231]] = vv[[231, 230]]
    assert refused(v=other)
    other = kv.copy()
    other[[230, 231]] = kv[[231, 230]]
    assert refused(k=other)
