"""GPU parity of the paged 4-bit cache (fg_paged_append, fg_paged_attention,
fg_pages_*) against the oracle in 64 bits (oracle/paged.py).

Bounds, with u = 2^-11 (half a step of fp16, relative) and for a row whose
weights are p_j, mag = sum_j p_j |v_j| and work = max_j sum_d |q_d k_jd| /
sqrt(d):
  * rounding the result: u |out| (fp16), 2^-24 |out| (fp32);
  * fp32 sums of n terms and exponentials: (n + d + 16) 2^-23 of mag, and of
    work (scores), which moves each weight by up to twice that (numerator and
    normaliser);
  * steps (at most 16 rows per K/V head): the weight p * scale is rounded to
    fp16 and multiplies c - 8, |c - 8| <= 8: u * 8 * max scale; scores are sums
    of c q in fp32, allowed d 2^-23 * 1039 * sum |q| * scale / sqrt(d), what
    sums of (1024 + c) q would need;
  * chunks of fp16: K and V rounded to fp16 (2 u work on the weights, u mag),
    P rounded to fp16 (u mag, and 2^-25 of the largest weight where P is
    subnormal).
Random rows are also held in the mean: the roundings are independent, each at
most u/sqrt(3) of the row's size (times 8 / 4.3 for the centred codes), so the
root mean square error of a step is below 2 u, of a chunk below 3 u.
"""
import math

import numpy as np
import pytest
import torch

from oracle import codec, paged as op

pytestmark = pytest.mark.gpu
U = 2.0 ** -11


@pytest.fixture(scope="module")
def fg():
    import int4_group_quantized_gb300 as fg
    return fg


def _i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Setup:
    """A pool of random quantized rows and a table with these lengths (its pages in random order)."""

    def __init__(self, fg, lens, heads, d, ps, dtype, seed, extra=2, spare=1, scale=1.0):
        rng = np.random.default_rng(seed)
        self.rng = rng
        lens = np.asarray(lens)
        need = -(-lens // ps)
        pages = int(need.sum()) + extra
        perm = rng.permutation(pages)
        self.table = np.full((len(lens), max(1, int(need.max(initial=0))) + spare), -1)
        self.refs = np.zeros(pages, int)
        at = 0
        for i, n in enumerate(need):
            self.table[i, :n] = perm[at:at + n]
            self.refs[perm[at:at + n]] = 1
            at += n
        self.lens, self.ps, self.heads, self.d, self.dtype, self.pages = lens, ps, heads, d, dtype, pages
        np_dt = np.float16 if dtype == torch.float16 else np.float32
        self.arr = {}
        for w in "kv":
            x = (scale * rng.normal(size=(pages, heads, ps, d)) * (0.5 + rng.random((heads, 1, d)))).astype(np_dt)
            self.arr[w] = list(codec.quantize_g64(x))
        self.upload(fg)

    def upload(self, fg):
        k, v = ([torch.as_tensor(a, device="cuda") for a in self.arr[w]] for w in "kv")
        self.pool = fg.PagePool.of(*k, *v, self.dtype)
        self.tab = fg.PageTable(_i32(self.table), _i32(self.lens), _i32(self.refs), self.ps)

    def rows(self, w, i, h, n):
        """The values of tokens 0..n-1 of sequence i (NaN where the table has no page), and which are present."""
        j = np.arange(n)
        page = np.where(j // self.ps < self.table.shape[1], self.table[i, np.minimum(j // self.ps, self.table.shape[1] - 1)], -1)
        ok = (page >= 0) & (page < self.pages)
        p = np.where(ok, page, 0)
        return op.restore(*(a[p, h, j % self.ps] for a in self.arr[w])), ok, self.arr[w][2][p, h, j % self.ps]


def _expect(S, cu, q, q_heads, window, sinks, step):
    """Reference rows and their elementwise bounds; rows outside every sequence are None."""
    d, r = S.d, q_heads // S.heads
    ref = np.full(q.shape, np.nan)
    tol = np.zeros(q.shape)
    for i in range(len(S.lens)):
        a, e = int(cu[i]), int(cu[i + 1])
        if a == e:
            continue
        length = int(S.lens[i])
        pos = np.repeat(np.arange(length - (e - a), length), r)
        for h in range(S.heads):
            k, ok, ks = S.rows("k", i, h, length)
            v, _, vs = S.rows("v", i, h, length)
            qq = q[a:e].reshape(e - a, q_heads, d)[:, h * r:(h + 1) * r].reshape(-1, d)
            out, mag, work = op.attention(qq, k, v, pos, window, sinks, ok)
            work = work[:, None]
            n = length + d + 16
            t = n * 2.0 ** -23 * (mag + 2 * work * mag)
            if S.dtype == torch.float32:
                t += 2.0 ** -24 * np.abs(out)
            elif step:
                t += U * (np.abs(out) + 8 * np.nanmax(vs[np.isfinite(vs)], initial=0.0))
                smax = np.nanmax(ks[np.isfinite(ks)], initial=0.0)
                t += 2 * mag * d * 2.0 ** -23 * 1039 * np.abs(qq).sum(1, keepdims=True) * smax / math.sqrt(d)
            else:
                vmax = np.abs(v[np.isfinite(v)]).max(initial=0.0)
                t += U * (np.abs(out) + 2 * mag + 2 * work * mag) + length * 2.0 ** -25 * vmax
            shape = (e - a, r, d)
            sl = np.s_[a:e, h * r * d:(h + 1) * r * d]
            ref[sl] = out.reshape(shape).reshape(e - a, -1)
            tol[sl] = t.reshape(shape).reshape(e - a, -1)
    return ref, tol


def _attend(fg, S, cu, q, q_heads, window=0, sinks=0, max_q=None, **kw):
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    n = int(np.diff(cu).max()) if max_q is None else max_q
    fg.fg_paged_attention(S.pool, S.tab, _i32(cu), q, q_heads, out, n, window=window, sinks=sinks, **kw)
    return out


def _q(S, rows, q_heads, scale=1.3):
    x = scale * S.rng.normal(size=(rows, q_heads * S.d))
    return torch.as_tensor(x, device="cuda").to(S.dtype)


def _compare(S, out, ref, tol, cu, rms=None):
    got = out.cpu().numpy().astype(np.float64)
    live = np.zeros(len(got), bool)
    live[int(cu[0]):int(cu[-1])] = True
    assert (got[~live] == 7.0).all(), "a row outside the batch was written"
    g, w, t = got[live], ref[live], tol[live]
    assert np.array_equal(np.isnan(g), np.isnan(w)), "NaN where there should be none, or none where there should be"
    f = ~np.isnan(w)
    err = np.abs(g[f] - w[f])
    worst = (err - t[f]).max(initial=-1.0)
    assert worst <= 0, f"error {err.max():.3g} above its bound by {worst:.3g}"
    if rms is not None and f.any():
        rel = np.sqrt(np.mean(err ** 2)) / np.sqrt(np.mean(w[f] ** 2))
        assert rel <= rms, f"rms error {rel:.3g} > {rms:.3g}"


# (lens, chunk rows, q_heads, heads, d, page_size, window, sinks)
STEP = [
    ([1], [1], 1, 1, 64, 16, 0, 0),                           # one token that sees itself
    ([1, 2, 16, 17, 33], [1, 1, 1, 1, 1], 4, 4, 128, 16, 0, 0),
    ([300, 5, 64, 129], [1, 0, 1, 1], 6, 2, 64, 64, 0, 0),    # three heads to one, a sequence that takes no part
    ([777, 90, 512], [1, 1, 1], 8, 1, 128, 32, 0, 0),
    ([600, 31, 250], [1, 1, 1], 32, 2, 128, 128, 0, 0),       # 16 rows
    ([200, 40], [7, 3], 2, 2, 128, 16, 0, 0),                 # several rows of one head: causal among them
    ([200, 40, 9], [5, 4, 9], 3, 1, 64, 256, 0, 0),           # 9 rows of a head group
    ([500, 33, 100], [1, 1, 1], 4, 4, 128, 16, 64, 4),
    ([500, 333], [2, 3], 4, 2, 64, 32, 1, 0),                 # a window of the token itself
    ([500, 333], [2, 3], 4, 2, 64, 32, 1, 1),
    ([2100], [1], 2, 2, 128, 64, 100, 1900),                  # sinks reach past the window's start
    ([5000, 4321], [1, 2], 4, 2, 128, 64, 0, 0),              # long: split over several workers
    ([40, 40], [1, 1], 5, 5, 64, 16, 1000, 3),                # a window longer than the sequence
]
CHUNK = [
    ([17], [17], 1, 1, 64, 16, 0, 0),
    ([300], [300], 2, 2, 128, 64, 0, 0),                      # a whole prompt
    ([700, 130, 257], [129, 130, 1], 4, 2, 128, 32, 0, 0),    # a step beside chunks
    ([1000, 60, 400], [256, 0, 399], 4, 4, 64, 16, 0, 0),
    ([900], [257], 1, 1, 128, 128, 0, 0),                     # one row past a tile of 256
    ([900, 800], [300, 100], 6, 2, 128, 64, 200, 5),
    ([900, 800], [300, 100], 3, 1, 64, 256, 17, 0),           # tiles that a row's window leaves empty
    ([1300], [64], 8, 1, 128, 64, 300, 130),                  # sinks past one tile
    ([520, 20, 21], [40, 20, 17], 7, 1, 64, 16, 0, 0),        # seven heads to one
    ([3000], [33], 1, 1, 128, 64, 0, 0),                      # few rows: split over the keys
    ([260, 259], [130, 131], 2, 1, 128, 16, 128, 0),
]


def _ids(c):
    return "len%s_q%s_h%d-%d_d%d_p%d_w%d-%d" % ("+".join(map(str, c[0])), "+".join(map(str, c[1])), *c[2:])


def _run_case(fg, case, dtype, step, seed):
    lens, n, qh, h, d, ps, window, sinks = case
    S = Setup(fg, lens, h, d, ps, dtype, seed)
    lead, tail = 2, 3                                         # rows before and behind the batch's own
    cu = lead + np.concatenate(([0], np.cumsum(n)))
    q = _q(S, int(cu[-1]) + tail, qh)
    out = _attend(fg, S, cu, q, qh, window, sinks)
    fg.fg_sync_status()
    ref, tol = _expect(S, cu, q.cpu().numpy().astype(np.float64), qh, window, sinks, step)
    _compare(S, out, ref, tol, cu, None if dtype == torch.float32 else (2 * U if step else 3 * U))


@pytest.mark.parametrize("case", STEP, ids=_ids)
def test_steps_f16(fg, case):
    _run_case(fg, case, torch.float16, True, 11)


@pytest.mark.parametrize("case", CHUNK, ids=_ids)
def test_chunks_f16(fg, case):
    _run_case(fg, case, torch.float16, False, 12)


@pytest.mark.parametrize("case", [STEP[i] for i in (0, 1, 2, 5, 8, 10)] + [CHUNK[i] for i in (0, 2, 5, 6, 8)], ids=_ids)
def test_f32(fg, case):
    _run_case(fg, case, torch.float32, True, 13)


@pytest.mark.parametrize("step", [True, False])
@pytest.mark.parametrize("scale", [1e-6, 30.0])
def test_small_and_large_values(fg, scale, step):
    """Rows of any size: weights are scaled before they are rounded, sharp softmaxes are exact where one token wins."""
    S = Setup(fg, [400, 300], 2, 128, 32, torch.float16, 14, scale=scale)
    n = [1, 2] if step else [40, 90]
    cu = np.concatenate(([0], np.cumsum(n)))
    q = _q(S, int(cu[-1]), 4)
    out = _attend(fg, S, cu, q, 4)
    fg.fg_sync_status()
    ref, tol = _expect(S, cu, q.cpu().numpy().astype(np.float64), 4, 0, 0, step)
    if scale < 1:   # subnormal results: half a step is 2^-25
        tol += 2.0 ** -25 + (0 if step else 3 * 2.0 ** -25)
    _compare(S, out, ref, tol, cu)


@pytest.mark.parametrize("case", [([37, 300, 64], [1, 1, 1], True), ([150, 300, 64], [20, 150, 33], False)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_nan_groups_reach_only_the_rows_that_see_them(fg, case, dtype):
    """NaN and infinite activations restore to NaN groups: future tokens, tokens before the window and slots past the
    end do not touch a row."""
    lens, n, step = case
    S = Setup(fg, lens, 2, 128, 32, dtype, 15)
    for w in "kv":   # every slot past a sequence's end, and free pages
        for i, length in enumerate(lens):
            last = S.table[i, (length - 1) // 32]
            S.arr[w][1][last, :, (length - 1) % 32 + 1:] = np.nan
            S.arr[w][2][last, :, (length - 1) % 32 + 1:] = np.nan
        S.arr[w][1][S.refs == 0] = np.inf
        S.arr[w][2][S.refs == 0] = np.nan
    # a NaN V group of token 10 (behind the window of 100 in sequence 1), a NaN V group of a late token of sequence 1
    S.arr["v"][2][S.table[1, 10 // 32], :, 10 % 32, 1] = np.nan
    S.arr["v"][1][S.table[1, 10 // 32], :, 10 % 32, 1] = np.inf
    late = 290
    S.arr["v"][2][S.table[1, late // 32], 0, late % 32, 0] = np.nan
    S.arr["k"][2][S.table[2, 62 // 32], 1, 62 % 32, 1] = np.nan
    S.upload(fg)
    cu = np.concatenate(([0], np.cumsum(n)))
    q = _q(S, int(cu[-1]), 2)
    out = _attend(fg, S, cu, q, 2, window=100, sinks=3)
    fg.fg_sync_status()
    ref, tol = _expect(S, cu, q.cpu().numpy().astype(np.float64), 2, 100, 3, step)
    assert np.isnan(ref).any() and not np.isnan(ref).all()
    _compare(S, out, ref, tol, cu)


def test_nan_query_stays_in_its_row(fg):
    for n in ([3, 1], [30, 40]):
        S = Setup(fg, [100, 80], 1, 64, 16, torch.float16, 16)
        cu = np.concatenate(([0], np.cumsum(n)))
        q = _q(S, int(cu[-1]), 2)
        clean = _attend(fg, S, cu, q, 2)
        q[1, :64] = float("nan")
        out = _attend(fg, S, cu, q, 2)
        fg.fg_sync_status()
        assert torch.isnan(out[1, :64]).all()
        out[1, :64] = clean[1, :64]
        assert torch.equal(out, clean)


@pytest.mark.parametrize("n", [[1, 1, 1], [30, 20, 10]])
@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_missing_pages_are_not_seen_and_reported(fg, n, dtype):
    S = Setup(fg, [200, 100, 90], 2, 64, 16, dtype, 17, extra=4)
    S.table[0, 3], S.table[1, 0], S.table[2, 2] = -1, S.pages, 2 ** 30
    S.upload(fg)
    cu = np.concatenate(([0], np.cumsum(n)))
    q = _q(S, int(cu[-1]), 4)
    out = _attend(fg, S, cu, q, 4)
    with pytest.raises(fg.FGError) as e:
        fg.fg_sync_status()
    assert e.value.status == 4
    ref, tol = _expect(S, cu, q.cpu().numpy().astype(np.float64), 4, 0, 0, max(n) <= 8)
    _compare(S, out, ref, tol, cu)
    # a row that sees no token at all gives zeros
    S.table[:] = -1
    S.upload(fg)
    out = _attend(fg, S, cu, q, 4)
    with pytest.raises(fg.FGError):
        fg.fg_sync_status()
    assert (out == 0).all()


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_chunk_longer_than_its_sequence(fg, dtype):
    """Rows at negative positions see nothing; the others are as ever."""
    for n in (6, 40):
        S = Setup(fg, [4, 30], 1, 64, 16, dtype, 18)
        cu = np.array([0, n, n + 1])
        q = _q(S, n + 1, 2)
        out = _attend(fg, S, cu, q, 2)
        fg.fg_sync_status()
        assert (out[:n - 4] == 0).all()
        ref, tol = _expect(S, cu, q.cpu().numpy().astype(np.float64), 2, 0, 0, n < 9)
        _compare(S, out, ref, tol, cu)


def test_bad_offsets_are_reported_and_skipped(fg):
    S = Setup(fg, [40, 50, 60], 1, 64, 16, torch.float16, 19)
    q = _q(S, 12, 1)
    good = _attend(fg, S, np.array([0, 1, 2, 3]), q, 1)
    fg.fg_sync_status()
    # sequence 1's rows run backwards, past the batch, or before it
    for cu in ([0, 1, 0, 3], [0, 1, 13, 3], [0, 1, 2 ** 30, 3], [0, 1, -5, 3]):
        out = _attend(fg, S, np.array(cu), q, 1, max_q=12)
        with pytest.raises(fg.FGError) as e:
            fg.fg_sync_status()
        assert e.value.status == 1
        if cu[2] != 0:   # there sequence 2 claims row 0 too
            assert torch.equal(out[0], good[0])
    # a sequence with more rows than max_q says, beside one that keeps to it
    out = _attend(fg, S, np.array([0, 1, 5, 5]), q, 1, max_q=2)
    with pytest.raises(fg.FGError) as e:
        fg.fg_sync_status()
    assert e.value.status == 1
    assert torch.equal(out[0], good[0]) and (out[1:] == 7.0).all()
    # a negative length
    S.lens[0] = -3
    S.upload(fg)
    out = _attend(fg, S, np.array([0, 1, 2, 3]), q, 1)
    with pytest.raises(fg.FGError):
        fg.fg_sync_status()
    assert (out[0] == 7.0).all()


def test_strided_rows(fg):
    """Q as columns of a wider buffer, out into another."""
    for n in ([2, 1], [30, 25]):
        S = Setup(fg, [90, 100], 2, 64, 16, torch.float16, 20)
        cu = np.concatenate(([0], np.cumsum(n)))
        rows = int(cu[-1])
        q = _q(S, rows, 4)
        plain = _attend(fg, S, cu, q, 4)
        wide = torch.zeros((rows, 4 * 64 + 136), dtype=torch.float16, device="cuda")
        wide[:, 72:72 + 256] = q
        dest = torch.full((rows, 512), 7.0, dtype=torch.float16, device="cuda")
        fg.fg_paged_attention(S.pool, S.tab, _i32(cu), wide[:, 72:72 + 256], 4, dest[:, 128:384], max(n))
        fg.fg_sync_status()
        assert torch.equal(dest[:, 128:384], plain)
        assert (dest[:, :128] == 7).all() and (dest[:, 384:] == 7).all()


def test_same_bits_every_time_and_alone(fg):
    """Repeats give the same bits; so do other workspaces' contents."""
    for n in ([1, 1, 1, 1], [100, 1, 37, 260]):
        S = Setup(fg, [3000, 1, 500, 260], 4, 128, 64, torch.float16, 21)
        cu = np.concatenate(([0], np.cumsum(n)))
        q = _q(S, int(cu[-1]), 8)
        ws = fg.workspace(fg.fg_paged_attention_workspace_bytes(S.pool, S.tab, 8, q.shape[0], max(n)))
        first = _attend(fg, S, cu, q, 8, ws=ws)
        for fill in (0, 255):
            ws.fill_(fill)
            assert torch.equal(_attend(fg, S, cu, q, 8, ws=ws), first)
        fg.fg_sync_status()


def test_matches_the_contiguous_decode_attention(fg):
    """One sequence length, one token each: fg_decode_attention on the same rows."""
    b, h, d, length, ps = 3, 4, 128, 210, 32
    S = Setup(fg, [length] * b, h, d, ps, torch.float16, 22)
    kv = fg.KVCache(b, h, d, length, True, torch.float16)
    j = np.arange(length)
    for w in "kv":
        for name, a in zip(("codes", "mins", "scales"), S.arr[w]):
            rows = np.stack([a[S.table[i, j // ps], :, j % ps] for i in range(b)])      # [b][length][h][..]
            getattr(kv, f"{w}_{name}").copy_(torch.as_tensor(rows.transpose(0, 2, 1, 3).copy(), device="cuda"))
    q = _q(S, b, h)
    want = torch.empty_like(q)
    fg.fg_decode_attention(kv, q, length - 1, want)
    got = _attend(fg, S, np.arange(b + 1), q, h)
    fg.fg_sync_status()
    # both round weights and results to fp16 around the same sums; the contiguous kernel keeps 1024 + c in its sums
    err = (got.double() - want.double()).abs().max().item()
    assert err <= 5e-3 * want.double().abs().max().item()


# ---- append ----------------------------------------------------------------------

def _np_rows(t):
    return t.cpu().numpy()


def _append_case(fg, lens, n, heads, d, ps, dtype, restored, seed, poison=True, x=None, wide=0):
    S = Setup(fg, lens, heads, d, ps, dtype, seed)
    if poison:
        for w in "kv":
            S.arr[w][0][:] = 0xA5
            S.arr[w][1][:] = 123.0
            S.arr[w][2][:] = np.nan
        S.upload(fg)
    lead, tail = 1, 2
    cu = lead + np.concatenate(([0], np.cumsum(n)))
    rows = int(cu[-1]) + tail
    if x is None:
        x = {w: S.rng.normal(size=(rows, heads * d)) * 1.3 for w in "kv"}
    t = {}
    for w in "kv":
        buf = torch.zeros((rows, heads * d + wide), dtype=dtype, device="cuda")
        t[w] = buf[:, wide // 2:wide // 2 + heads * d]
        t[w].copy_(torch.as_tensor(x[w], device="cuda"))
    res = {w: torch.full((rows, heads * d), 7.0, dtype=dtype, device="cuda") if restored else None for w in "kv"}
    fg.fg_paged_append(S.pool, S.tab, _i32(cu), t["k"], t["v"], res["k"], res["v"])
    want = {w: [a.copy() for a in S.arr[w]] for w in "kv"}
    rest = {w: np.full((rows, heads * d), 7.0) for w in "kv"}
    missing = False
    for i, length in enumerate(lens):
        for tt in range(int(n[i])):
            pos, row = int(length) - int(n[i]) + tt, int(cu[i]) + tt
            col = pos // ps
            page = S.table[i, col] if pos >= 0 and col < S.table.shape[1] else -1
            if not 0 <= page < S.pages:
                missing = True
                continue
            for w in "kv":
                c, m, s = codec.quantize_g64(_np_rows(t[w])[row].reshape(heads, d))
                for a, new in zip(want[w], (c, m, s)):
                    a[page, :, pos % ps] = new
                rest[w][row] = codec.dequant_g64(c, m, s, _np_rows(t[w]).dtype).reshape(-1)
    return S, want, res, rest, missing


def _same(got, want):
    a, b = np.asarray(got), np.asarray(want)
    if a.dtype.kind == "f":
        return np.array_equal(np.isnan(a), np.isnan(b)) and np.array_equal(a[~np.isnan(a)], b[~np.isnan(b)].astype(a.dtype))
    return np.array_equal(a, b)


def _check_append(fg, S, want, res, rest):
    for w, names in (("k", ("k_codes", "k_mins", "k_scales")), ("v", ("v_codes", "v_mins", "v_scales"))):
        for name, a in zip(names, want[w]):
            assert _same(getattr(S.pool, name).cpu().numpy(), a), name
        if res[w] is not None:
            assert _same(res[w].cpu().numpy(), rest[w].astype(res[w].cpu().numpy().dtype)), w + " restored"


APPEND = [
    ([1], [1], 1, 64, 16, False),
    ([40, 16, 100, 7], [40, 1, 37, 0], 3, 128, 16, True),     # whole prompts, a step, a chunk, none
    ([64, 65, 300], [1, 2, 299], 5, 64, 64, True),
    ([500] * 9, [1] * 9, 2, 128, 256, False),
    ([33, 90], [20, 50], 1, 128, 32, False),
]


@pytest.mark.parametrize("case", APPEND, ids=lambda c: "len%s_n%s_h%d_d%d_p%d_r%d" % ("+".join(map(str, c[0])), "+".join(map(str, c[1])), *c[2:]))
@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_append_is_the_codec_bit_for_bit(fg, case, dtype):
    S, want, res, rest, missing = _append_case(fg, *case[:5], dtype, case[5], 31)
    fg.fg_sync_status()
    assert not missing
    _check_append(fg, S, want, res, rest)


def _special(rows, cols):
    """Groups of special values: NaN, infinities, constants, signed zeros, subnormals, halfway quotients."""
    rng = np.random.default_rng(5)
    x = rng.normal(size=(rows, cols)).astype(np.float32)
    g = x.reshape(-1, 64)
    g[0] = 0.0
    g[1] = -0.0
    g[2, ::2] = -0.0
    g[2, 1::2] = 0.0
    g[3] = 2.5
    g[4, 7] = np.nan
    g[5] = np.nan
    g[6, 3] = np.inf
    g[7, 3] = -np.inf
    g[8, 0], g[8, 1] = np.inf, -np.inf
    g[9] = np.arange(64) % 16 / 2 + 0.25 * (np.arange(64) % 2)     # quotients on the halves
    g[10] = np.linspace(0, 15, 64).round(1)
    g[11] *= 6e-8
    g[12] *= 2e4
    g[13, 0], g[13, 1] = 65504.0, -65504.0
    g[14] = np.arange(64) % 2
    g[15, :] = 1.0
    g[15, 5] = 1.0 + 2 ** -10
    for k in range(16, len(g)):
        if k % 3 == 0:
            g[k] = np.round(g[k] * 7.5) / 7.5
    return x


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_append_special_values(fg, dtype):
    x = {"k": _special(43, 256), "v": _special(43, 256)[::-1].copy()}
    S, want, res, rest, _ = _append_case(fg, [60], [40], 2, 128, 16, dtype, True, 32, x=x)
    fg.fg_sync_status()
    _check_append(fg, S, want, res, rest)


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_append_strided_and_in_place(fg, dtype):
    S, want, res, rest, _ = _append_case(fg, [60, 30], [40, 5], 3, 64, 16, dtype, True, 33, wide=144)
    fg.fg_sync_status()
    _check_append(fg, S, want, res, rest)
    # the restored rows over the rows themselves
    S2 = Setup(fg, [60, 30], 3, 64, 16, dtype, 33)
    rows = torch.as_tensor(S2.rng.normal(size=(45, 192)), device="cuda").to(dtype)
    k, v = rows.clone(), rows.clone() * 2
    cu = _i32([0, 40, 45])
    kr, vr = torch.empty_like(k), torch.empty_like(v)
    fg.fg_paged_append(S2.pool, S2.tab, cu, k, v, kr, vr)
    fg.fg_paged_append(S2.pool, S2.tab, cu, k, v, k, v)
    fg.fg_sync_status()
    assert torch.equal(k, kr) and torch.equal(v, vr)


def test_append_skips_what_has_no_slot(fg):
    S = Setup(fg, [40, 40, 20], 2, 64, 16, torch.float16, 34)
    S.table[0, 1], S.table[1, 2] = -1, S.pages + 5
    S.lens[2] = 3                                             # 5 rows, 3 tokens: two rows stand before the sequence
    S.upload(fg)
    before = [t.clone() for t in (S.pool.k_codes, S.pool.v_mins)]
    cu = np.array([0, 40, 60, 65])
    k = torch.randn((65, 128), device="cuda").half()
    kr, vr = torch.full_like(k, 7.0), torch.full_like(k, 7.0)
    fg.fg_paged_append(S.pool, S.tab, _i32(cu), k, k, kr, vr)
    with pytest.raises(fg.FGError) as e:
        fg.fg_sync_status()
    assert e.value.status in (1, 4)
    skipped = list(range(16, 32)) + list(range(52, 60)) + [60, 61]
    assert (kr[skipped] == 7).all() and (vr[skipped] == 7).all()
    kept = [r for r in range(65) if r not in skipped]
    assert not (kr[kept] == 7).any()
    free = torch.as_tensor(S.refs == 0, device="cuda")
    assert torch.equal(S.pool.k_codes[free], before[0][free]) and torch.equal(S.pool.v_mins[free], before[1][free])
    # offsets that run backwards: those rows are left out, the rest is stored
    with pytest.raises(fg.FGError) as e:
        fg.fg_paged_append(S.pool, S.tab, _i32([0, 4, 2, 9]), k, k)
        fg.fg_sync_status()
    assert e.value.status == 1


# ---- pages -----------------------------------------------------------------------

def _meta(pg, fg):
    return fg.PageTable(_i32(pg.table), _i32(pg.lens), _i32(pg.refs), pg.ps)


def _assert_meta(tab, pg, table=True):
    assert np.array_equal(tab.lens.cpu().numpy(), pg.lens)
    assert np.array_equal(tab.refs.cpu().numpy(), pg.refs)
    if table:
        for i in range(len(pg.lens)):
            n = pg.held(i)
            assert np.array_equal(tab.table[i, :n].cpu().numpy(), pg.table[i, :n]), i


def _pools(fg, layers, pages, ps, heads, d, dtype=torch.float16):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    got = []
    for _ in range(layers):
        p = fg.PagePool(pages, ps, heads, d, dtype)
        for c in (p.k_codes, p.v_codes):
            c.copy_(torch.randint(0, 256, c.shape, generator=gen, device="cuda", dtype=torch.uint8))
        for m in (p.k_mins, p.k_scales, p.v_mins, p.v_scales):
            m.copy_(torch.randn(m.shape, generator=gen, device="cuda"))
        got.append(p)
    return got


ARRAYS = ("k_codes", "v_codes", "k_mins", "k_scales", "v_mins", "v_scales")


@pytest.mark.parametrize("shape", [(9, 60, 7, 16, 1, 64, 1), (23, 300, 11, 32, 3, 128, 2), (70, 5000, 41, 16, 1, 64, 1),
                                   (5, 40, 6, 256, 2, 128, 67)])
def test_runs_of_page_calls_follow_the_oracle(fg, shape):
    """Growth, forks, ends and compactions in turn; tables, counts and every layer's pages, and the pages left alone."""
    seqs, pages, stride, ps, heads, d, layers = shape
    rng = np.random.default_rng(seqs)
    pg = op.Pages(np.full((seqs, stride), -1), np.zeros(seqs, int), np.zeros(pages, int), ps)
    tab = _meta(pg, fg)
    pools = _pools(fg, layers, pages, ps, heads, d)
    mirror = [[getattr(p, a).clone() for a in ARRAYS] for p in pools]
    arr = fg.PagePools(pools)
    for step in range(24):
        what = rng.choice(["grow", "grow", "fork", "free", "compact"])
        moves = []
        pg.full = False
        if what == "grow":
            n = rng.integers(0, 3 * ps, seqs) * (rng.random(seqs) < 0.6)
            n = np.where(pg.lens + n > stride * ps, 0, n)
            base = int(rng.integers(0, 100))
            pg.reserve(n)
            fg.fg_pages_reserve(tab, _i32(base + np.concatenate(([0], np.cumsum(n)))))
        elif what == "fork":
            m = int(rng.integers(1, seqs))
            src, dst = rng.integers(0, seqs, m), rng.integers(0, seqs, m)
            moves = pg.fork(src, dst)
            fg.fg_pages_fork(tab, arr, _i32(src), _i32(dst))
        elif what == "free":
            rows = rng.integers(0, seqs, int(rng.integers(1, max(2, seqs // 2))))
            pg.free(rows)
            fg.fg_pages_free(tab, _i32(rows))
        else:
            moves = pg.compact()
            fg.fg_pages_compact(tab, arr)
        if pg.full:
            with pytest.raises(fg.FGError):
                fg.fg_sync_status()
        else:
            fg.fg_sync_status()
        _assert_meta(tab, pg)
        if moves:
            a, b = (torch.as_tensor([m[k] for m in moves], device="cuda") for k in (0, 1))
            for m in mirror:
                for x in m:
                    x[b] = x[a]
    for p, m in zip(pools, mirror):
        for name, x in zip(ARRAYS, m):
            assert torch.equal(getattr(p, name).view(torch.int32 if x.dtype == torch.float32 else torch.uint8),
                               x.view(torch.int32 if x.dtype == torch.float32 else torch.uint8)), name


def test_reserve_at_the_limits(fg):
    # more pages wanted than there are: rows in order, the rest -1; a row too short
    pg = op.Pages(np.full((3, 3), -1), np.array([0, 16, 0]), np.zeros(6, int), 16)
    pg.table[1, 0], pg.refs[4] = 4, 1
    tab = _meta(pg, fg)
    for n in ([40, 1, 33], [1, 100, 0]):
        pg.full = False
        pg.reserve(n)
        fg.fg_pages_reserve(tab, _i32(np.concatenate(([0], np.cumsum(n)))))
        with pytest.raises(fg.FGError) as e:
            fg.fg_sync_status()
        assert e.value.status == 4 and pg.full
        _assert_meta(tab, pg)
    # offsets that decrease, lengths that would overflow
    pg = op.Pages(np.full((3, 3), -1), np.zeros(3, int), np.zeros(6, int), 16)
    tab = _meta(pg, fg)
    tab.lens[2] = 5
    fg.fg_pages_reserve(tab, _i32([0, 2, 1, 2 ** 31 - 1]))
    with pytest.raises(fg.FGError) as e:
        fg.fg_sync_status()
    assert e.value.status == 1
    assert tab.lens.tolist() == [2, 0, 5] and tab.table[0, 0] == 0 and tab.refs.tolist() == [1, 0, 0, 0, 0, 0]


def test_forks_that_cannot_be_made(fg):
    pg = op.Pages(np.full((6, 3), -1), np.array([20, 32, 0, 0, 0, 0]), np.zeros(5, int), 16)
    pg.table[0, :2], pg.table[1, :2] = [3, 1], [0, 4]
    pg.refs[[3, 1, 0, 4]] = 1
    tab = _meta(pg, fg)
    pools = fg.PagePools(_pools(fg, 1, 5, 16, 1, 64))
    keep = pools.pools[0].k_codes.clone()
    src, dst = [0, 0, 1, 9, 1, -1, 1, 2], [2, 3, 2, 4, 1, 5, 0, 3]
    # 0 -> 2 takes the one free page; 0 -> 3 finds none; 2 is named twice; out of range; onto itself; onto a filled row;
    # an empty source onto a row already named
    moves = pg.fork(src, dst)
    fg.fg_pages_fork(tab, pools, _i32(src), _i32(dst))
    with pytest.raises(fg.FGError):
        fg.fg_sync_status()
    _assert_meta(tab, pg)
    assert moves == [(1, 2)]
    keep[2] = keep[1]
    assert torch.equal(pools.pools[0].k_codes, keep)
    # a full page is only shared, an empty sequence forks into an empty one
    fg.fg_pages_free(tab, _i32([2]))
    fg.fg_pages_fork(tab, pools, _i32([1, 5]), _i32([2, 3]))
    fg.fg_sync_status()
    assert tab.table[2, :2].tolist() == [0, 4] and tab.refs.tolist() == [2, 1, 0, 1, 2]
    assert tab.lens.tolist() == [20, 32, 32, 0, 0, 0]


def test_free_skips_bad_rows(fg):
    pg = op.Pages(np.full((3, 2), -1), np.array([20, 5, 0]), np.zeros(5, int), 16)
    pg.table[0], pg.table[1, 0] = [3, 1], 0
    pg.refs[[3, 1, 0]] = 1
    tab = _meta(pg, fg)
    fg.fg_pages_free(tab, _i32([0, 7, 0, -1, 2]))
    with pytest.raises(fg.FGError) as e:
        fg.fg_sync_status()
    assert e.value.status == 1
    assert tab.lens.tolist() == [0, 5, 0] and tab.refs.tolist() == [1, 0, 0, 0, 0]
    assert tab.table.tolist() == [[-1, -1], [0, -1], [-1, -1]]


# ---- together ----------------------------------------------------------------------

def _serve(fg, dtype, graph, stream=None):
    """Prompts, forks, steps with windows, ends, compaction, more steps, as a server runs them; the same tokens in plain
    rows per sequence on the side.  Returns nothing; asserts along the way."""
    heads, qh, d, ps, seqs, pages, stride = 2, 4, 64, 16, 6, 40, 8
    rng = np.random.default_rng(7)
    np_dt = np.float16 if dtype == torch.float16 else np.float32
    pool = fg.PagePool(pages, ps, heads, d, dtype)
    tab = fg.PageTable.empty(seqs, stride, pages, ps)
    pools = fg.PagePools([pool])
    hist = [{"k": np.zeros((0, heads, d)), "v": np.zeros((0, heads, d))} for _ in range(seqs)]
    ntok = 64
    cu = torch.zeros(seqs + 1, dtype=torch.int32, device="cuda")
    k, v, q, out = (torch.zeros((ntok, (qh if i > 1 else heads) * d), dtype=dtype, device="cuda") for i in range(4))
    pws = fg.workspace(fg.fg_pages_workspace_bytes(tab, 4))
    aws = fg.workspace(fg.fg_paged_attention_workspace_bytes(pool, tab, qh, ntok, ntok))

    def calls():
        fg.fg_pages_reserve(tab, cu, pws)
        fg.fg_paged_append(pool, tab, cu, k, v)
        fg.fg_paged_attention(pool, tab, cu, q, qh, out, ntok, window=50, sinks=2, ws=aws)

    g = None
    if graph:
        calls()                      # nothing in cu: the kernels are loaded
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            calls()

    def step(n):
        n = np.asarray(n)
        c = np.concatenate(([0], np.cumsum(n)))
        x = {w: rng.normal(size=(ntok, heads * d)).astype(np_dt) for w in "kv"}
        xq = rng.normal(size=(ntok, qh * d)).astype(np_dt)
        cu.copy_(torch.as_tensor(c.astype(np.int32)))
        k.copy_(torch.as_tensor(x["k"]))
        v.copy_(torch.as_tensor(x["v"]))
        q.copy_(torch.as_tensor(xq))
        out.fill_(7.0)
        (g.replay if graph else calls)()
        fg.fg_sync_status()
        got = out.cpu().numpy().astype(np.float64)
        assert (got[c[-1]:] == 7).all()
        for i in range(seqs):
            for w in "kv":
                rows = x[w][c[i]:c[i + 1]].reshape(-1, heads, d)
                hist[i][w] = np.concatenate((hist[i][w], op.restore(*codec.quantize_g64(rows))))
            length = len(hist[i]["k"])
            if n[i] == 0:
                continue
            for h in range(heads):
                qq = xq[c[i]:c[i + 1]].astype(np.float64).reshape(-1, qh, d)[:, 2 * h:2 * h + 2].reshape(-1, d)
                ref, mag, work = op.attention(qq, hist[i]["k"][:, h], hist[i]["v"][:, h],
                                              np.repeat(np.arange(length - n[i], length), 2), 50, 2)
                o = got[c[i]:c[i + 1], 2 * h * d:(2 * h + 2) * d].reshape(-1, d)
                u = U if dtype == torch.float16 else 2.0 ** -17
                assert (np.abs(o - ref) <= u * (np.abs(ref) + 4 * mag * (1 + work[:, None]) + 1)).all()

    def fork(a, b):
        fg.fg_pages_fork(tab, pools, _i32([a]), _i32([b]), pws)
        hist[b] = {w: hist[a][w].copy() for w in "kv"}

    def end(i):
        fg.fg_pages_free(tab, _i32([i]))
        hist[i] = {w: hist[i][w][:0] for w in "kv"}

    step([20, 7, 0, 33, 0, 0])
    fork(0, 2)
    step([1, 1, 1, 1, 0, 0])
    step([1, 0, 3, 1, 17, 0])
    end(1)
    fork(3, 5)
    step([1, 0, 1, 1, 1, 1])
    end(0)
    fg.fg_pages_compact(tab, pools, pws)
    step([9, 0, 1, 20, 1, 1])
    step([1, 40, 1, 0, 1, 1])
    fg.fg_pages_compact(tab, pools, pws)
    step([1, 1, 1, 1, 1, 1])
    assert int((tab.refs > 0).sum()) <= pages


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_a_run_of_all_calls(fg, dtype):
    _serve(fg, dtype, False)


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_a_run_captured_and_replayed(fg, dtype):
    _serve(fg, dtype, True)


def test_on_another_stream(fg):
    S = Setup(fg, [300, 100], 2, 128, 64, torch.float16, 40)
    for n in ([1, 1], [60, 100]):
        cu = np.concatenate(([0], np.cumsum(n)))
        q = _q(S, int(cu[-1]), 4)
        want = _attend(fg, S, cu, q, 4)
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        out = torch.zeros_like(q)
        c = _i32(cu)
        st.wait_stream(torch.cuda.current_stream())
        fg.fg_paged_attention(S.pool, S.tab, c, q, 4, out, max(n), stream=st)
        fg.fg_sync_status(st)
        assert torch.equal(out, want)


def test_a_calls_own_workspace_belongs_to_its_stream(fg):
    """A workspace freed by a call on one stream may still be in use there: a call on another stream has other memory."""
    S = Setup(fg, [300], 2, 64, 16, torch.float16, 42)
    side, n = torch.cuda.Stream(), 1 << 20
    here = fg._paged_ws(None, n, S.tab, None)
    at = here.data_ptr()
    del here
    for st in (side, side.cuda_stream):
        there = fg._paged_ws(None, n, S.tab, st)
        assert there.data_ptr() != at
    again = fg._paged_ws(None, n, S.tab, None)
    assert again.data_ptr() == at


def test_python_checks(fg):
    S = Setup(fg, [30], 2, 64, 16, torch.float16, 41)
    q = torch.zeros((1, 128), dtype=torch.float16, device="cuda")
    cu = _i32([0, 1])
    with pytest.raises(ValueError):
        fg.fg_paged_attention(S.pool, S.tab, cu.long(), q, 2, q.clone(), 1)
    with pytest.raises(ValueError):
        fg.fg_paged_attention(S.pool, S.tab, cu, q.float(), 2, q.clone(), 1)
    with pytest.raises(ValueError):
        fg.fg_paged_attention(S.pool, S.tab, _i32([0, 1, 1]), q, 2, q.clone(), 1)
    with pytest.raises(ValueError):
        fg.fg_paged_append(S.pool, S.tab, cu, q, q.cpu())
    with pytest.raises(ValueError):
        fg.PagePool.of(S.pool.k_codes, S.pool.k_mins.half(), S.pool.k_scales, S.pool.v_codes, S.pool.v_mins, S.pool.v_scales)
    with pytest.raises(ValueError):
        fg.PageTable(S.tab.table, S.tab.lens.long(), S.tab.refs, 16)


def test_waits_that_run_out_are_reported(fg):
    """With a wait limit of 0 the chunk kernel gives up at once, reports it, and the next call is right."""
    S = Setup(fg, [500, 300], 2, 128, 64, torch.float16, 42)
    cu = np.array([0, 400, 500])
    q = _q(S, 500, 4)
    want = _attend(fg, S, cu, q, 4)
    fg.fg_sync_status()
    old = fg.fg_set_wait_limit(0)
    try:
        _attend(fg, S, cu, q, 4)
        with pytest.raises(fg.FGError) as e:
            fg.fg_sync_status()
        assert e.value.status == 7
    finally:
        fg.fg_set_wait_limit(old)
    assert torch.equal(_attend(fg, S, cu, q, 4), want)
    fg.fg_sync_status()


@pytest.mark.parametrize("seqs", [129, 300, 1100])
@pytest.mark.parametrize("kind", ["steps", "chunks", "f32"])
def test_many_sequences(fg, seqs, kind):
    """More sequences than a kernel plans for by itself; some take no part."""
    rng = np.random.default_rng(seqs)
    lens = rng.integers(1, 60, seqs)
    n = np.where(rng.random(seqs) < 0.3, 0, 1)
    if kind != "steps":
        n = np.where(rng.random(seqs) < 0.2, rng.integers(1, 60, seqs), n)
    n = np.minimum(n, lens)
    dtype = torch.float32 if kind == "f32" else torch.float16
    S = Setup(fg, lens, 1, 64, 16, dtype, seqs)
    cu = np.concatenate(([0], np.cumsum(n)))
    q = _q(S, int(cu[-1]), 2)
    out = _attend(fg, S, cu, q, 2)
    fg.fg_sync_status()
    ref, tol = _expect(S, cu, q.cpu().numpy().astype(np.float64), 2, 0, 0, True)
    if kind == "chunks":   # the bound of a chunk where a sequence is one, of a step elsewhere: the larger
        tol = np.maximum(tol, _expect(S, cu, q.cpu().numpy().astype(np.float64), 2, 0, 0, False)[1])
    _compare(S, out, ref, tol, cu)


@pytest.mark.parametrize("n", [[1, 1, 1], [1, 13, 40]])
@pytest.mark.parametrize("heads", [(20, 1), (40, 2), (33, 1)])
def test_more_query_heads_than_a_step_takes(fg, n, heads):
    qh, h = heads
    S = Setup(fg, [300, 13, 129], h, 128, 32, torch.float16, 50)
    cu = np.concatenate(([0], np.cumsum(n)))
    q = _q(S, int(cu[-1]), qh)
    out = _attend(fg, S, cu, q, qh, window=90, sinks=2)
    fg.fg_sync_status()
    ref, tol = _expect(S, cu, q.cpu().numpy().astype(np.float64), qh, 90, 2, False)
    _compare(S, out, ref, tol, cu, 3 * U)


@pytest.mark.parametrize("n", [[1, 1], [30, 40]])
@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_a_row_too_short_for_its_length(fg, n, dtype):
    """Tokens past the table row's end are not seen, and reported."""
    S = Setup(fg, [64, 50], 1, 64, 16, dtype, 51, spare=0)
    S.lens = np.array([90, 50])
    S.upload(fg)
    cu = np.concatenate(([0], np.cumsum(n)))
    q = _q(S, int(cu[-1]), 2)
    out = _attend(fg, S, cu, q, 2)
    with pytest.raises(fg.FGError) as e:
        fg.fg_sync_status()
    assert e.value.status == 4
    ref, tol = _expect(S, cu, q.cpu().numpy().astype(np.float64), 2, 0, 0, max(n) == 1)
    _compare(S, out, ref, tol, cu)


def test_two_calls_at_once(fg):
    """Two streams, two workspaces, the same pool."""
    S = Setup(fg, [3000, 900, 1500], 4, 128, 64, torch.float16, 52)
    jobs = []
    for n in ([1, 1, 1], [300, 40, 200], [200, 1, 3]):
        cu = np.concatenate(([0], np.cumsum(n)))
        q = _q(S, int(cu[-1]), 8)
        jobs.append((_i32(cu), q, max(n), _attend(fg, S, cu, q, 8), torch.zeros_like(q), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for cu, q, mq, _, out, st in jobs:
            fg.fg_paged_attention(S.pool, S.tab, cu, q, 8, out, mq, stream=st)
    torch.cuda.synchronize()
    fg.fg_sync_status()
    for *_, want, out, _ in jobs:
        assert torch.equal(out, want)


@pytest.mark.parametrize("seqs,dtype", [(20, torch.float16), (150, torch.float16), (20, torch.float32), (150, torch.float32)])
def test_calls_one_after_another(fg, seqs, dtype):
    """Every call's kernels may be set up while the call before still runs: the results are those of calls that each wait
    for the one before."""
    heads, qh, d, ps, pages, turns = 2, 4, 128, 16, 3000, 5
    rng = np.random.default_rng(54)
    lengths = np.array([0, 1, 1, 2, 20, 70])
    jobs = []
    for _ in range(turns):
        n = lengths[rng.integers(len(lengths), size=seqs)]
        n[seqs - 2:] = 0                                      # forked into and freed
        cu = np.concatenate(([0], np.cumsum(n)))
        x = [torch.as_tensor(rng.normal(size=(int(cu[-1]), w * d)), device="cuda").to(dtype) for w in (heads, heads, qh)]
        jobs.append((_i32(cu), *x, _i32(rng.integers(0, seqs - 2, size=2)), int(n.max())))
    dst = _i32([seqs - 2, seqs - 1])
    most = max(q.shape[0] for *_, q, _, _ in jobs)
    results = []
    for wait in (True, False):
        after = torch.cuda.synchronize if wait else (lambda: None)
        pool, tab = fg.PagePool(pages, ps, heads, d, dtype), fg.PageTable.empty(seqs, 64, pages, ps)
        pools = fg.PagePools([pool])
        ws = fg.workspace(max(fg.fg_pages_workspace_bytes(tab, 2), fg.fg_paged_attention_workspace_bytes(pool, tab, qh, most, 70)))
        outs = []
        torch.cuda.synchronize()
        for cu, k, v, q, src, _ in jobs:
            out = [torch.zeros_like(q) for _ in range(3)]
            kr, vr = torch.zeros_like(k), torch.zeros_like(v)
            for call in (lambda: fg.fg_pages_reserve(tab, cu, ws),
                         lambda: fg.fg_paged_append(pool, tab, cu, k, v, kr, vr),
                         lambda: fg.fg_paged_attention(pool, tab, cu, q, qh, out[0], 70, ws=ws),
                         lambda: fg.fg_paged_attention(pool, tab, cu, out[0], qh, out[1], 70, window=40, sinks=3, ws=ws),
                         lambda: fg.fg_pages_fork(tab, pools, src, dst, ws),
                         lambda: fg.fg_pages_free(tab, src[:1]),
                         lambda: fg.fg_pages_compact(tab, pools, ws),
                         lambda: fg.fg_paged_attention(pool, tab, cu, out[1], qh, out[2], 70, ws=ws),
                         lambda: fg.fg_pages_free(tab, dst)):
                call()
                after()
            outs += out + [kr, vr, tab.table.clone(), tab.lens.clone(), tab.refs.clone()]
        torch.cuda.synchronize()
        fg.fg_sync_status()
        results.append(outs)
    for a, b in zip(*results):
        assert torch.equal(a, b)
    assert all(bool(t.isfinite().all()) for t in results[0])


def test_two_graphs_share_a_workspace(fg):
    S = Setup(fg, [700, 400], 2, 64, 32, torch.float16, 53)
    ws = fg.workspace(fg.fg_paged_attention_workspace_bytes(S.pool, S.tab, 4, 300, 200))
    graphs = []
    for n in ([1, 1], [200, 100]):
        cu = np.concatenate(([0], np.cumsum(n)))
        q = _q(S, int(cu[-1]), 4)
        want, c, out = _attend(fg, S, cu, q, 4, max_q=200), _i32(cu), torch.zeros_like(q)
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            fg.fg_paged_attention(S.pool, S.tab, c, q, 4, out, 200, ws=ws)
        graphs.append((g, out, want, c, q))
    for _ in range(3):
        for g, out, want, _, _ in graphs:
            out.zero_()
            g.replay()
        torch.cuda.synchronize()
        for _, out, want, _, _ in graphs:
            assert torch.equal(out, want)
    fg.fg_sync_status()


def test_offsets_past_32_bits(fg):
    """Pages more than 4 GB into the arrays: appended, copied and attended."""
    heads, d, ps, pages = 8, 128, 256, 36000                  # 4.7 GB of codes each for K and V
    pool = fg.PagePool(pages, ps, heads, d)
    assert pool.k_codes.numel() > 2 ** 32
    tab = fg.PageTable.empty(4, 4, pages, ps)
    tab.refs[:pages - 6] = 1                                  # only the last pages are free
    rng = np.random.default_rng(60)
    n = [300, 0, 40, 0]
    cu = np.concatenate(([0], np.cumsum(n)))
    x = {w: rng.normal(size=(340, heads * d)).astype(np.float16) for w in "kv"}
    fg.fg_pages_reserve(tab, _i32(cu))
    fg.fg_paged_append(pool, tab, _i32(cu), *(torch.as_tensor(x[w], device="cuda") for w in "kv"))
    fg.fg_pages_fork(tab, fg.PagePools([pool]), _i32([0, 2]), _i32([1, 3]))
    fg.fg_sync_status()
    assert tab.table[0, :2].tolist() == [pages - 6, pages - 5] and tab.table[1, 1].item() == pages - 3
    q = torch.as_tensor(rng.normal(size=(42, heads * d)), device="cuda").half()
    for m in ([1, 1, 1, 1], [1, 20, 1, 20]):
        c = np.concatenate(([0], np.cumsum(m)))
        out = torch.zeros_like(q)
        fg.fg_paged_attention(pool, tab, _i32(c), q, heads, out, max(m))
        fg.fg_sync_status()
        for i, (src, length) in enumerate(((0, 300), (0, 300), (2, 40), (2, 40))):
            k, v = (op.restore(*codec.quantize_g64(x[w][cu[src]:cu[src + 1]].reshape(-1, heads, d))) for w in "kv")
            for h in (0, heads - 1):
                qq = q[c[i]:c[i + 1], h * d:(h + 1) * d].double().cpu().numpy()
                ref, mag, work = op.attention(qq, k[:, h], v[:, h], np.arange(length - m[i], length))
                got = out[c[i]:c[i + 1], h * d:(h + 1) * d].double().cpu().numpy()
                assert (np.abs(got - ref) <= U * (np.abs(ref) + 4 * mag * (1 + work[:, None]) + 4)).all()
