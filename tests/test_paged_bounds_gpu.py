"""The paged attention against the oracle in 64 bits with bounds taken over the tokens that each row sees
(oracle/paged.py, attention_bound; tests/test_paged_bounds_cpu.py shows what they refuse), and in the mean: the roundings
are independent, each at most u / sqrt(3) of the row's size (times 8 / 4.3 for the centred codes), u = 2^-11, so the root
mean square error of a step is below 2 u, of a chunk below 3 u."""
import numpy as np
import pytest
import torch

from oracle import codec, paged as op
from test_paged_gpu import CHUNK, STEP, Setup, _attend, _i32, _ids, _q

pytestmark = pytest.mark.gpu
U = op.HALF
KINDS = {"step": 2 * U, "chunk": 3 * U, "f32": None}


@pytest.fixture(scope="module")
def fg():
    import int4_group_quantized_gb300 as fg
    return fg


def _kind(S, n, q_heads):
    """How the library takes a sequence of n rows."""
    return "f32" if S.dtype == torch.float32 else "step" if n * (q_heads // S.heads) <= 16 else "chunk"


def _hold(S, out, cu, q, q_heads, window=0, sinks=0, mean=True, rows_mean=None):
    """Every sequence and K/V head within its bound; `mean` (and rows_mean, a factor, row by row): in the mean as well."""
    r, d = q_heads // S.heads, S.d
    got, q = out.cpu().numpy().astype(np.float64), q.cpu().numpy().astype(np.float64)
    live = np.zeros(len(got), bool)
    live[int(cu[0]):int(cu[-1])] = True
    assert (got[~live] == 7.0).all(), "a row outside the batch was written"
    parts = {}
    for i in range(len(S.lens)):
        a, e, length = int(cu[i]), int(cu[i + 1]), int(S.lens[i])
        if a == e:
            continue
        kind = _kind(S, e - a, q_heads)
        j = np.arange(length)
        col = np.minimum(j // S.ps, S.table.shape[1] - 1)
        page = np.where(j // S.ps < S.table.shape[1], S.table[i, col], -1)
        ok = (page >= 0) & (page < S.pages)
        page = np.where(ok, page, 0)
        pos = np.repeat(np.arange(length - (e - a), length), r)
        for h in range(S.heads):
            k, v = ([x[page, h, j % S.ps] for x in S.arr[w]] for w in "kv")
            sl = np.s_[a:e, h * r * d:(h + 1) * r * d]
            o = got[sl].reshape(-1, d)
            ref, tol = op.attention_bound(q[sl].reshape(-1, d), k, v, pos, window, sinks, ok, kind)
            why = op.off_by_too_much(o, ref, tol)
            assert why is None, f"sequence {i}, head {h}: {why}"
            if rows_mean is not None and KINDS[kind]:
                for x, w in zip(o, ref):
                    why = op.off_by_too_much(x, w, np.inf + 0 * x, rows_mean * KINDS[kind])
                    assert why is None, f"sequence {i}, head {h}, a row: {why}"
            parts.setdefault(kind, []).append((o, ref))
    for kind, p in parts.items():
        if mean and KINDS[kind]:
            o, ref = (np.concatenate([x[n].reshape(-1) for x in p]) for n in (0, 1))
            why = op.off_by_too_much(o, ref, np.full(o.shape, np.inf), KINDS[kind])
            assert why is None, f"{kind}: {why}"


def _run(fg, S, n, q_heads, window=0, sinks=0, q=None, status=None, **kw):
    cu = np.concatenate(([0], np.cumsum(n)))
    q = _q(S, int(cu[-1]), q_heads) if q is None else q
    out = _attend(fg, S, cu, q, q_heads, window, sinks)
    if status is None:
        fg.fg_sync_status()
    else:
        with pytest.raises(fg.FGError) as e:
            fg.fg_sync_status()
        assert e.value.status == status
    _hold(S, out, cu, q, q_heads, window, sinks, **kw)
    return out


@pytest.mark.parametrize("case", STEP + CHUNK, ids=_ids)
@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_every_row_within_its_bound(fg, case, dtype):
    lens, n, qh, h, d, ps, window, sinks = case
    _run(fg, Setup(fg, lens, h, d, ps, dtype, 11), n, qh, window, sinks)


@pytest.mark.parametrize("n", [[1, 2], [7, 5], [40, 90]])
@pytest.mark.parametrize("scale", [1e-6, 1e-3, 30.0])
def test_rows_of_any_size(fg, scale, n):
    _run(fg, Setup(fg, [400, 300], 2, 128, 32, torch.float16, 14, scale=scale), n, 4, mean=scale < 1)


@pytest.mark.parametrize("seqs", [129, 1100])
@pytest.mark.parametrize("most", [1, 59])
@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_many_sequences(fg, seqs, most, dtype):
    rng = np.random.default_rng(seqs)
    lens = rng.integers(1, 60, seqs)
    n = np.minimum(lens, np.where(rng.random(seqs) < 0.3, 0, np.where(rng.random(seqs) < 0.8, 1, rng.integers(1, most + 1, seqs))))
    _run(fg, Setup(fg, lens, 1, 64, 16, dtype, seqs), n, 2)


@pytest.mark.parametrize("n", [[1, 1, 1], [30, 20, 10]])
@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_missing_pages(fg, n, dtype):
    S = Setup(fg, [200, 100, 90], 2, 64, 16, dtype, 17, extra=4)
    S.table[0, 3], S.table[1, 0], S.table[2, 2] = -1, S.pages, 2 ** 30
    S.upload(fg)
    _run(fg, S, n, 4, status=4)


@pytest.mark.parametrize("n", [[1, 1], [30, 40]])
@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_a_table_row_too_short(fg, n, dtype):
    S = Setup(fg, [64, 50], 1, 64, 16, dtype, 51, spare=0)
    S.lens = np.array([90, 50])
    S.upload(fg)
    _run(fg, S, n, 2, status=4)


@pytest.mark.parametrize("n", [6, 40])
@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_more_rows_than_tokens(fg, n, dtype):
    _run(fg, Setup(fg, [4, 30], 1, 64, 16, dtype, 18), [n, 1], 2)


@pytest.mark.parametrize("n", [[1, 1, 1], [4, 3, 8], [20, 150, 33]])
@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_nan_groups_leave_the_other_rows_exact(fg, n, dtype):
    lens = [150, 300, 64]
    S = Setup(fg, lens, 2, 128, 32, dtype, 15)
    for w in "kv":
        for i, length in enumerate(lens):
            last = S.table[i, (length - 1) // 32]
            for x in S.arr[w][1:]:
                x[last, :, (length - 1) % 32 + 1:] = np.nan
        S.arr[w][1][S.refs == 0] = np.inf
        S.arr[w][2][S.refs == 0] = np.nan
    for w, i, h, t, g in (("v", 1, 0, 10, 1), ("v", 1, 1, 295, 0), ("v", 1, 0, 298, 0), ("k", 2, 1, 62, 1), ("k", 0, 0, 20, 0)):
        S.arr[w][2][S.table[i, t // 32], h, t % 32, g] = np.nan
    S.upload(fg)
    _run(fg, S, n, 2, 100, 3)


# ---- values whose sizes differ ------------------------------------------------------

def _towards(S, n, q_heads, spread=0.05):
    """Query rows that all point the same way, per K/V head, and that direction as unit vectors."""
    d, r = S.d, q_heads // S.heads
    u = S.rng.normal(size=(S.heads, d))
    u /= np.linalg.norm(u, axis=1, keepdims=True)
    x = np.repeat(u * np.sqrt(d), r, axis=0)[None] + spread * S.rng.normal(size=(n, q_heads, d))
    return torch.as_tensor(x.reshape(n, -1), device="cuda").to(S.dtype), u


def _put(S, w, i, t, rows):
    """Token t of sequence i becomes `rows` [heads][d]."""
    for a, new in zip(S.arr[w], codec.quantize_g64(np.asarray(rows).astype(np.float16))):
        a[S.table[i, t // S.ps], :, t % S.ps] = new


SHAPES = [(1, 2, 2), (1, 8, 1), (1, 16, 1), (3, 2, 2), (7, 1, 1), (9, 1, 1)]   # rows, query heads, K/V heads: steps


@pytest.mark.parametrize("n,qh,h", SHAPES + [(40, 2, 2)])
@pytest.mark.parametrize("d", [64, 128])
def test_hidden_tokens_do_not_cost_accuracy(fg, n, qh, h, d):
    """Values far larger than the rest, behind the window's edge: rows that do not see them are as exact as without."""
    S = Setup(fg, [1000], h, d, 32, torch.float16, 71)
    S.arr["v"] = list(codec.quantize_g64((0.01 * S.rng.normal(size=(S.pages, h, 32, d))).astype(np.float16)))
    first = 1000 - n - 190 + 1                                 # the first token that any row sees
    for t in (first - 1, first - 3):
        _put(S, "v", 0, t, 6e4 * np.sign(S.rng.normal(size=(h, d))))
    S.upload(fg)
    _run(fg, S, [n], qh, window=190, rows_mean=2)


@pytest.mark.parametrize("n,qh,h", [s for s in SHAPES if s[0] > 1] + [(40, 2, 2)])
def test_a_later_rows_token_does_not_cost_the_earlier_rows(fg, n, qh, h):
    S = Setup(fg, [1000], h, 128, 32, torch.float16, 72)
    S.arr["v"] = list(codec.quantize_g64((0.01 * S.rng.normal(size=(S.pages, h, 32, 128))).astype(np.float16)))
    _put(S, "v", 0, 999, 6e4 * np.sign(S.rng.normal(size=(h, 128))))
    S.upload(fg)
    _run(fg, S, [n], qh, rows_mean=2)


@pytest.mark.parametrize("n,qh,h", SHAPES + [(40, 2, 2)])
@pytest.mark.parametrize("at", [3, 500, 990])
def test_large_values_of_no_weight_do_not_cost_accuracy(fg, n, qh, h, at):
    """A token that all rows see and none weighs (its score 50 below the others'), with values far larger."""
    S = Setup(fg, [1000], h, 128, 32, torch.float16, 73)
    S.arr["v"] = list(codec.quantize_g64((0.01 * S.rng.normal(size=(S.pages, h, 32, 128))).astype(np.float16)))
    q, u = _towards(S, n, qh)
    _put(S, "k", 0, at, -50 * u)
    _put(S, "v", 0, at, 6e4 * np.sign(S.rng.normal(size=(h, 128))))
    S.upload(fg)
    _run(fg, S, [n], qh, q=q, rows_mean=2)


@pytest.mark.parametrize("n,qh,h", SHAPES)
def test_large_values_that_lose_their_weight(fg, n, qh, h):
    """Large values lead until later tokens, whose scores lie 40 above, leave them no weight.  (Steps alone: a chunk rounds
    K, and scores of 50 are then 0.4 * 50 * sqrt(3 / d) u = 3 u off in the mean.)"""
    S = Setup(fg, [1000], h, 128, 32, torch.float16, 74)
    S.arr["v"] = list(codec.quantize_g64((0.01 * S.rng.normal(size=(S.pages, h, 32, 128))).astype(np.float16)))
    q, u = _towards(S, n, qh)
    x = S.rng.normal(size=(1000, h, 128)) * 0.5
    x[200:] += 40 * u
    x[600:] += 10 * u
    for t in range(1000):
        _put(S, "k", 0, t, x[t])
    _put(S, "v", 0, 5, 6e4 * np.sign(S.rng.normal(size=(h, 128))))
    S.upload(fg)
    _run(fg, S, [n], qh, q=q, rows_mean=2)


@pytest.mark.parametrize("n", [[2, 9], [8, 16], [1, 300], [5, 70]])
def test_values_of_two_sizes_in_one_call(fg, n):
    """The same beside sequences of other numbers of rows."""
    S = Setup(fg, [1000, 700], 2, 128, 32, torch.float16, 78)
    S.arr["v"] = list(codec.quantize_g64((0.01 * S.rng.normal(size=(S.pages, 2, 32, 128))).astype(np.float16)))
    q, u = _towards(S, sum(n), 2)
    for i, length in enumerate((1000, 700)):
        for t in (40, length // 2):
            _put(S, "k", i, t, -50 * u)
            _put(S, "v", i, t, 6e4 * np.sign(S.rng.normal(size=(2, 128))))
    S.upload(fg)
    _run(fg, S, n, 2, q=q, rows_mean=2)


@pytest.mark.parametrize("n,qh,h", SHAPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", [1e-4, 2e-6])
def test_small_queries(fg, n, qh, h, d, size):
    """Queries near fp16's smallest numbers against keys near its largest: every bit of q counts."""
    S = Setup(fg, [300], h, d, 32, torch.float16, 76)
    S.arr["k"] = list(codec.quantize_g64((1.3e4 * S.rng.normal(size=(S.pages, h, 32, d))).clip(-6e4, 6e4).astype(np.float16)))
    S.upload(fg)
    q = _q(S, n, qh, size)
    _run(fg, S, [n], qh, q=q, rows_mean=2)


@pytest.mark.parametrize("n,qh,h", SHAPES + [(40, 2, 2), (300, 1, 1)])
def test_many_small_weights_beside_a_large_one(fg, n, qh, h):
    """A first token whose score lies 18 above the others' and whose values are zero: the output is the sum of thousands of
    weights of 2^-26."""
    S = Setup(fg, [4000], h, 128, 64, torch.float16, 75)
    S.arr["v"] = list(codec.quantize_g64((60 * (1 + 0.5 * S.rng.normal(size=(S.pages, h, 64, 128)))).astype(np.float16)))
    S.arr["k"] = list(codec.quantize_g64((0.3 * S.rng.normal(size=(S.pages, h, 64, 128))).astype(np.float16)))
    q, u = _towards(S, n, qh)
    _put(S, "k", 0, 0, 18 * u)
    _put(S, "v", 0, 0, np.zeros((h, 128)))
    S.upload(fg)
    _run(fg, S, [n], qh, q=q, rows_mean=2)


# ---- waits --------------------------------------------------------------------------

def test_a_wait_that_runs_out_is_never_silent(fg):
    """Whatever the limit, a call either reports a wait that ran out or is right."""
    S = Setup(fg, [700, 300], 2, 128, 64, torch.float16, 77)
    cu = np.array([0, 600, 700])
    q = _q(S, 700, 4)
    want = _attend(fg, S, cu, q, 4)
    fg.fg_sync_status()
    seen = set()
    old = fg.fg_set_wait_limit(0)
    try:
        for limit in sorted({int(1.17 ** k) for k in range(75)}):
            fg.fg_set_wait_limit(limit)
            for _ in range(4):
                out = _attend(fg, S, cu, q, 4)
                try:
                    fg.fg_sync_status()
                    assert torch.equal(out, want), f"limit {limit}: wrong, and no status"
                    seen.add(True)
                except fg.FGError as e:
                    assert e.status == 7
                    seen.add(False)
    finally:
        fg.fg_set_wait_limit(old)
    assert torch.equal(_attend(fg, S, cu, q, 4), want)
    fg.fg_sync_status()
    assert seen == {True, False}


# ---- forks --------------------------------------------------------------------------

def test_a_fork_that_cannot_be_made_takes_no_page(fg):
    """A source whose last page is missing is refused; the free pages go to the forks that can be made, lowest first."""
    ps = 16
    table = np.full((9, 2), -1)
    table[0, 0], table[1, 0], table[2, :2] = 5, -1, [1, -1]     # sources: whole; no page; a full page and no second
    lens = np.array([7, 9, 20, 0, 0, 0, 0, 0, 0])
    refs = np.zeros(8, int)
    refs[[5, 1, 0, 2, 7]] = 1                                   # free: 3, 4, 6
    tab = fg.PageTable(_i32(table), _i32(lens), _i32(refs), ps)
    pool = fg.PagePool(8, ps, 1, 64)
    pool.k_codes.copy_(torch.arange(8, device="cuda", dtype=torch.uint8).view(8, 1, 1, 1).expand_as(pool.k_codes))
    fg.fg_pages_fork(tab, fg.PagePools([pool]), _i32([1, 0, 2, 0, 0, 0]), _i32([3, 4, 5, 6, 7, 8]))
    with pytest.raises(fg.FGError) as e:
        fg.fg_sync_status()
    assert e.value.status == 4
    assert tab.table[:, 0].tolist() == [5, -1, 1, -1, 3, -1, 4, 6, -1]
    assert tab.lens.tolist() == [7, 9, 20, 0, 7, 0, 7, 7, 0]
    assert tab.refs.tolist() == [1, 1, 1, 1, 1, 1, 1, 1]
    assert pool.k_codes[:, 0, 0, 0].tolist() == [0, 1, 2, 5, 5, 5, 5, 7]
