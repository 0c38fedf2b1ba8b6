"""GPU parity of shared prefixes: fg_pages_share against the oracle's plain search,
fg_paged_attention_shared against attention in 64 bits."""
import numpy as np
import pytest
import torch

from oracle import paged as op

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fg():
    import int4_group_quantized_gb300 as fg
    return fg


def _i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device="cuda")


FIELDS = ("group", "tokens", "first", "leader", "begin", "rows")


def _forest(rng, seqs, ps, stride, depth, missing=0.0, idle=0.2):
    """Sequences forked from one another at random places, some of them twice over, with pages of their own after that."""
    page, table, lens, n = 0, np.full((seqs, stride), -1), np.zeros(seqs, int), np.zeros(seqs, int)
    order = rng.permutation(seqs)
    for at, i in enumerate(order):
        own = int(rng.integers(1, stride + 1))
        keep = 0
        if at and rng.random() < 0.75:
            src = order[rng.integers(max(0, at - depth), at)]
            keep = int(rng.integers(0, min(own, (lens[src] // ps)) + 1)) if lens[src] >= ps else 0
            table[i, :keep] = table[src, :keep]
        table[i, keep:own] = page + np.arange(own - keep)
        page += own - keep
        lens[i] = min(own * ps, (own - 1) * ps + int(rng.integers(1, ps + 1)))
        n[i] = 0 if rng.random() < idle else min(int(rng.integers(1, 2 * ps)), lens[i]) if rng.random() < 0.4 else 1
    if missing:
        table[(rng.random(table.shape) < missing) & (table >= 0)] = rng.choice([-1, page + 7, -5])
    return table, lens, n, page


@pytest.mark.parametrize("seed", range(12))
def test_share_matches_a_plain_search(fg, seed):
    rng = np.random.default_rng(seed)
    seqs = [1, 2, 5, 31, 33, 64, 100, 129, 300, 40, 40, 1100][seed]
    ps = int(rng.choice([16, 32, 64]))
    table, lens, n, pages = _forest(rng, seqs, ps, int(rng.integers(1, 40)), [1, 3, 1000][seed % 3], 0.01 if seed % 4 == 3 else 0.0)
    cu = np.concatenate(([0], np.cumsum(n)))
    tab = fg.PageTable(_i32(table), _i32(lens), _i32(np.ones(max(pages, 1))), ps)
    share = fg.PageShare.empty(tab, int(cu[-1]))
    for least in (1, ps, ps + 1, 5 * ps, 10 ** 9):
        for t in FIELDS:
            getattr(share, t).fill_(-77)
        fg.fg_pages_share(tab, _i32(cu), share, min_tokens=least)
        fg.fg_sync_status()
        want = op.share(table, lens, cu, max(pages, 1), ps, least)
        for name, w in zip(FIELDS, want):
            assert np.array_equal(getattr(share, name).cpu().numpy(), w), (name, least)
    assert share.group.max() < 0 and (share.rows < 0).all()      # nobody shares 10^9 tokens


def test_share_of_long_prefixes_and_many_rows(fg):
    """Comparing takes many rounds; a shorter common part of more sequences wins or loses by what it saves."""
    ps, stride = 16, 3000
    base = np.arange(stride)
    cuts = [2999, 2998, 1025, 1024, 700, 256, 255, 1, 2999]
    table = np.tile(base, (len(cuts) + 1, 1))
    page = stride
    for i, c in enumerate(cuts):
        table[i + 1, c:] = page + np.arange(stride - c)
        page += stride - c
    lens, n = np.full(len(table), stride * ps), np.full(len(table), 3)
    cu = np.concatenate(([0], np.cumsum(n)))
    tab = fg.PageTable(_i32(table), _i32(lens), _i32(np.ones(page)), ps)
    share = fg.PageShare.empty(tab, int(cu[-1]))
    fg.fg_pages_share(tab, _i32(cu), share, 1)
    fg.fg_sync_status()
    for name, w in zip(FIELDS, op.share(table, lens, cu, page, ps, 1)):
        assert np.array_equal(getattr(share, name).cpu().numpy(), w), name


def test_share_of_offsets_out_of_range(fg):
    """Offsets that run backwards or past the rows: reported, and nothing is written past the arrays."""
    ps = 16
    table = np.tile(np.arange(4), (4, 1))
    tab = fg.PageTable(_i32(table), _i32([60] * 4), _i32(np.ones(4)), ps)
    for cu in ([0, 2, 1, 3, 4], [0, 1, 2, 3, 9], [-1, 1, 2, 3, 4], [0, 4, 0, 4, 4]):
        guard = torch.full((64,), -77, dtype=torch.int32, device="cuda")
        share = fg.PageShare(*[torch.zeros(k, dtype=torch.int32, device="cuda") for k in (4, 4, 4, 4, 5)], guard[16:20])
        fg.fg_pages_share(tab, _i32(cu), share, 1)
        with pytest.raises(fg.FGError, match="FG_ERR_ARG"):
            fg.fg_sync_status()
        assert (guard[:16] == -77).all() and (guard[20:] == -77).all()


# ---- attention ---------------------------------------------------------------------
#
# A row's bound: the prefix is multiplied as chunks are (K, V and the weights rounded to fp16), a sequence's own tokens as
# steps or as chunks; with the row's weights p_j over all of its tokens each part's terms (oracle/paged.py,
# attention_bound) are sums over some of them, so the two kinds' sum bounds both.  The parts are joined in fp32: at most
# 130 parts, a rounding of the sums (2^-24) and of a factor (2^-22 in all) each.

class Forked:
    """Sequences that share leading pages group by group, with rows of their own after that; values, keys and queries of
    unlike sizes."""

    def __init__(self, fg, groups, tails, n, heads, r, d, ps, seed, q_size=1.0, dtype=torch.float16):
        # groups: of each sequence (group or -1); pages of a group: shared[g]
        rng = np.random.default_rng(seed)
        which, shared = groups
        self.which = np.asarray(which)
        lead = np.array([0 if g < 0 else shared[g] for g in which])
        tails, n = np.asarray(tails), np.asarray(n)
        own = -(-tails // ps)
        pages = int(sum(shared) + own.sum()) + 2
        perm = rng.permutation(pages)
        start = np.concatenate(([0], np.cumsum(shared)))
        self.table = np.full((len(which), int((lead + own).max()) + 1), -1)
        at = int(sum(shared))
        for i, g in enumerate(which):
            if g >= 0:
                self.table[i, :lead[i]] = perm[start[g]:start[g + 1]]
            self.table[i, lead[i]:lead[i] + own[i]] = perm[at:at + own[i]]
            at += own[i]
        self.lens, self.n, self.ps, self.heads, self.r, self.d, self.pages, self.dtype = lead * ps + tails, n, ps, heads, r, d, pages, dtype
        self.cu = np.concatenate(([0], np.cumsum(n)))
        np_dt = np.float16 if dtype == torch.float16 else np.float32
        self.arr = {}
        for w in "kv":
            x = rng.normal(size=(pages, heads, ps, d)) * (0.5 + rng.random((heads, 1, d))) * 2.0 ** rng.integers(-2, 2, (pages, heads, ps, 1))
            self.arr[w] = list(op.codec.quantize_g64(x.astype(np_dt)))
        self.q = (q_size * rng.normal(size=(int(self.cu[-1]), heads * r * d))).astype(np_dt)
        self.upload(fg)

    def upload(self, fg):
        k, v = ([torch.as_tensor(a, device="cuda") for a in self.arr[w]] for w in "kv")
        self.pool = fg.PagePool.of(*k, *v, self.dtype)
        self.tab = fg.PageTable(_i32(self.table), _i32(self.lens), _i32(np.ones(self.pages)), self.ps)

    def find(self, fg, least=1):
        s = fg.PageShare.empty(self.tab, int(self.cu[-1]))
        fg.fg_pages_share(self.tab, _i32(self.cu), s, least)
        return s

    def expect(self):
        d, r = self.d, self.r
        ref, tol = np.full(self.q.shape, np.nan), np.zeros(self.q.shape)
        for i, length in enumerate(self.lens):
            a, e = int(self.cu[i]), int(self.cu[i + 1])
            if a == e:
                continue
            pos = np.repeat(np.arange(length - (e - a), length), r)
            j = np.arange(length)
            page = self.table[i, j // self.ps]
            ok = (page >= 0) & (page < self.pages)
            at = np.where(ok, page, 0), j % self.ps
            for h in range(self.heads):
                qq = self.q[a:e].reshape(e - a, -1, d)[:, h * r:(h + 1) * r].reshape(-1, d).astype(np.float64)
                k, v = ([x[at[0], h, at[1]] for x in self.arr[w]] for w in "kv")
                if self.dtype == torch.float32:
                    out, t = op.attention_bound(qq, k, v, pos, present=ok, kind="f32")
                else:
                    out, t = op.attention_bound(qq, k, v, pos, present=ok, kind="step")
                    _, t2 = op.attention_bound(qq, k, v, pos, present=ok, kind="chunk")
                    with np.errstate(all="ignore"):
                        t = t + t2 + 130 * 2.0 ** -22 * np.abs(out)
                sl = np.s_[a:e, h * r * d:(h + 1) * r * d]
                ref[sl], tol[sl] = out.reshape(e - a, -1), t.reshape(e - a, -1)
        return ref, tol


def _run(fg, F, share=None, max_q=None, min_saved=0, **kw):
    out = torch.full(F.q.shape, 7.0, dtype=F.dtype, device="cuda")
    fg.fg_paged_attention_shared(F.pool, F.tab, _i32(F.cu), F.find(fg) if share is None else share, torch.as_tensor(F.q, device="cuda"),
                                 F.heads * F.r, out, int(F.n.max()) if max_q is None else max_q, min_saved, **kw)
    return out


def _hold(got, ref, tol, rms=3 * 2.0 ** -11):
    why = op.off_by_too_much(got.double().cpu().numpy(), ref, tol, rms)
    assert why is None, why


def _sizes(b, lo, hi, seed):
    return np.random.default_rng(seed).integers(lo, hi + 1, b)


SHARED = {   # groups, tails, rows, heads, query heads a head, d, page size
    "two sequences of a page": (([0, 0], [1]), [1, 5], [1, 1], 1, 1, 64, 16),
    "a step": (([0] * 6, [19]), _sizes(6, 1, 60, 1), [1] * 6, 12, 1, 64, 16),
    "a step of wide heads": (([0] * 5 + [-1], [5]), _sizes(6, 1, 60, 2), [1] * 6, 3, 1, 128, 64),
    "130 followers, two units": (([0] * 130, [26]), _sizes(130, 1, 30, 3), [1] * 130, 2, 1, 128, 16),
    "eight query heads, three groups": (([0, 1, 2, -1] * 5, [3, 9, 1]), _sizes(20, 1, 200, 4), [1] * 20, 2, 8, 128, 32),
    "few rows, idle sequences": (([0, 0, 1, 1, 0, -1], [4, 7]), [9, 1, 30, 3, 5, 6], [2, 0, 3, 1, 4, 2], 3, 2, 64, 16),
    "chunks": (([0, 1, 0, 1, -1, 0], [7, 2]), [60, 40, 5, 33, 70, 61], [60, 17, 5, 33, 70, 1], 2, 4, 128, 32),
    "chunks beside steps": (([0] * 8, [10]), [1, 200, 1, 2, 90, 1, 1, 7], [1, 100, 1, 2, 90, 1, 1, 7], 2, 3, 64, 32),
    "a long prefix over many shares": (([0] * 3, [200]), [3, 4, 5], [1] * 3, 1, 1, 64, 32),
    "a long prefix of chunks": (([0] * 3, [33]), [150, 4, 64], [150, 4, 64], 1, 4, 128, 128),
    "tokens that no tile divides": (([0] * 4 + [1] * 4, [9, 17]), _sizes(8, 1, 40, 5), [1] * 8, 2, 2, 128, 16),
    "wide groups": (([0, 0, 0], [8]), [20, 30, 40], [3, 1, 2], 1, 20, 64, 64),
    "300 sequences": (([0] * 120 + [-1] * 30 + [1] * 150, [4, 6]), _sizes(300, 1, 40, 6), [1] * 300, 1, 1, 64, 16),
    "one row a unit more": (([0] * 129, [2]), [3] * 129, [1] * 129, 1, 1, 64, 64),
}


@pytest.mark.parametrize("name", SHARED)
def test_shared_attention(fg, name):
    groups, tails, n, heads, r, d, ps = SHARED[name]
    F = Forked(fg, groups, tails, n, heads, r, d, ps, 11)
    out = _run(fg, F)
    fg.fg_sync_status()
    _hold(out, *F.expect())
    assert torch.equal(_run(fg, F), out)                     # the same bits again


@pytest.mark.parametrize("size", [8.0, 40.0])
def test_large_scores(fg, size):
    """A later tile's scores may lie far above the first ones'."""
    F = Forked(fg, ([0] * 5, [70]), [3, 40, 100, 7, 1], [1, 1, 3, 1, 1], 2, 2, 128, 16, 12, q_size=size)
    out = _run(fg, F)
    fg.fg_sync_status()
    ref, tol = F.expect()
    _hold(out, ref, tol, rms=None)


def test_every_sequence_of_fp32_by_itself(fg):
    F = Forked(fg, ([0, 0, 0, -1], [5]), [20, 30, 40, 7], [3, 1, 20, 7], 2, 2, 64, 16, 13, dtype=torch.float32)
    out = _run(fg, F)
    fg.fg_sync_status()
    _hold(out, *F.expect(), rms=None)


def test_nobody_shares(fg):
    F = Forked(fg, ([-1] * 5, []), [40, 1, 30, 100, 17], [1, 1, 30, 2, 1], 2, 2, 64, 16, 14)
    out, plain = _run(fg, F), torch.full(F.q.shape, 7.0, dtype=torch.float16, device="cuda")
    fg.fg_paged_attention(F.pool, F.tab, _i32(F.cu), torch.as_tensor(F.q, device="cuda"), 4, plain, 30)
    fg.fg_sync_status()
    assert torch.equal(out, plain)                           # the same launches over the same lines
    _hold(out, *F.expect())


def test_what_saves_too_little_is_not_shared(fg):
    """Below min_saved the bits are those of fg_paged_attention; a table row too short for that much is refused sharing on the
    host, a longer one on the device."""
    F = Forked(fg, ([0] * 6 + [1] * 3, [9, 30]), [4, 1, 30, 100, 17, 5, 6, 7, 8], [1, 1, 30, 2, 1, 1, 1, 1, 1], 2, 2, 64, 16, 24)
    plain = torch.full(F.q.shape, 7.0, dtype=torch.float16, device="cuda")
    fg.fg_paged_attention(F.pool, F.tab, _i32(F.cu), torch.as_tensor(F.q, device="cuda"), 4, plain, 30)
    # reads alone less those of the group (72 rows of a K/V head: two units; 6: one), the chunk's four, and the 39 rows' parts
    saved = 2 * 64 * 5 // 4 * (9 * 16 * (5 + 4 - 2) + 30 * 16 * (3 - 1) - 8 * 2 * 39)
    ref = F.expect()
    for least, same in ((saved + 1, True), (saved, False), (1 << 60, True), (-1, True)):
        out = _run(fg, F, min_saved=least)
        fg.fg_sync_status()
        assert torch.equal(out, plain) == same, least
        _hold(out, *ref)


def test_rows_that_reach_into_the_prefix_go_alone(fg):
    """A share made earlier: one sequence's rows now begin before its group's tokens end, another takes no part."""
    F = Forked(fg, ([0] * 5, [6]), [40, 20, 50, 33, 2], [4] * 4 + [2], 2, 2, 64, 16, 15)
    s = F.find(fg)
    F.lens[1] = 6 * 16 + 3                                   # of 4 rows, one stands inside the prefix
    F.upload(fg)
    out = _run(fg, F, s)
    fg.fg_sync_status()
    _hold(out, *F.expect())
    F.lens[1] = 4                                            # all of them, at the beginning
    F.upload(fg)
    out = _run(fg, F, s)
    fg.fg_sync_status()
    _hold(out, *F.expect())


def test_pages_may_be_compacted_and_lengths_grow(fg):
    F = Forked(fg, ([0, 0, 1, 1], [3, 4]), [5, 6, 7, 8], [1] * 4, 2, 1, 64, 16, 16)
    s = F.find(fg)
    perm = np.random.default_rng(17).permutation(F.pages)    # page p is now perm[p]
    F.table = np.where(F.table >= 0, perm[F.table], -1)
    F.arr = {w: [x[np.argsort(perm)] for x in F.arr[w]] for w in "kv"}
    F.lens = F.lens + 3
    F.upload(fg)
    out = _run(fg, F, s)
    fg.fg_sync_status()
    _hold(out, *F.expect())


def test_a_missing_page_of_the_prefix_is_not_seen(fg):
    F = Forked(fg, ([0] * 4, [9]), [5, 6, 7, 80], [1, 1, 1, 70], 2, 2, 64, 16, 18)
    s = F.find(fg)
    F.table[:, 3] = -1
    F.upload(fg)
    out = _run(fg, F, s)
    with pytest.raises(fg.FGError, match="FG_ERR_CAPACITY"):
        fg.fg_sync_status()
    _hold(out, *F.expect())
    F.table[:, :9] = F.pages + 3                             # the whole prefix: rows see their own tokens
    F.upload(fg)
    out = _run(fg, F, s)
    with pytest.raises(fg.FGError, match="FG_ERR_CAPACITY"):
        fg.fg_sync_status()
    _hold(out, *F.expect())


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_what_is_not_finite_reaches_the_group_alone(fg, bad):
    F = Forked(fg, ([0, 0, 1, 1, -1], [10, 9]), [5, 6, 7, 8, 90], [1, 1, 1, 20, 1], 1, 2, 128, 16, 19)
    F.arr["v"][2][F.table[0, 4], 0, 7, 1] = bad              # dims 64 .. 127 of one value of group 0
    F.upload(fg)
    out = _run(fg, F)
    fg.fg_sync_status()
    ref, tol = F.expect()
    assert np.isnan(ref[:2]).sum() == 2 * 2 * 64 and not np.isnan(ref[2:]).any()
    _hold(out, ref, tol)
    F.arr["k"][2][F.table[2, 2], 0, 3, 0] = bad              # a key of group 1's prefix: its rows' scores are NaN
    F.upload(fg)
    got = _run(fg, F).double().cpu().numpy()
    fg.fg_sync_status()
    assert np.isnan(got[2:-1]).all() and not np.isnan(got[-1]).any()


def test_rows_behind_the_last_sequence_stay(fg):
    F = Forked(fg, ([0, 0, 0], [9]), [5, 6, 40], [1, 1, 25], 2, 1, 64, 16, 20)
    wide = torch.randn((F.cu[-1] + 3, 2 * 64 + 24), device="cuda").half()
    wide[:F.cu[-1], :128] = torch.as_tensor(F.q, device="cuda")
    out = torch.full_like(wide, 7.0)
    share = fg.PageShare.empty(F.tab, int(F.cu[-1]) + 3)
    fg.fg_pages_share(F.tab, _i32(F.cu), share, 1)
    fg.fg_paged_attention_shared(F.pool, F.tab, _i32(F.cu), share, wide[:, :128], 2, out[:, :128], 25, 0)
    fg.fg_sync_status()
    _hold(out[:F.cu[-1], :128], *F.expect())
    assert (out[F.cu[-1]:] == 7.0).all() and (out[:, 128:] == 7.0).all()


def test_a_share_of_nonsense_is_not_followed(fg):
    """Numbers out of range are no groups: every sequence goes by itself."""
    F = Forked(fg, ([0] * 4, [9]), [5, 6, 7, 80], [1, 1, 1, 70], 2, 2, 64, 16, 21)
    good = F.find(fg)
    ref = F.expect()
    for field, values in (("group", [10 ** 9, -(10 ** 9), 77]), ("tokens", [17, -16, 10 ** 9, 2 ** 31 - 16]), ("first", [-1, 10 ** 9, 60]),
                          ("leader", [-5, 10 ** 9, 4]), ("begin", [-1, 10 ** 9, -(10 ** 9), 74]), ("rows", [-1, 10 ** 9])):
        for v in values:
            s = fg.PageShare(*[getattr(good, f).clone() for f in FIELDS])
            getattr(s, field).fill_(v)
            out = _run(fg, F, s)
            fg.fg_sync_status()
            _hold(out, *ref)


def test_graphs_streams_and_shared_workspaces(fg):
    """Two captured graphs use one workspace in turn; a call on another stream gives the same bits."""
    A = Forked(fg, ([0] * 5, [20]), [5, 6, 7, 80, 9], [1, 1, 1, 70, 2], 2, 2, 64, 16, 22)
    B = Forked(fg, ([0, 0, 1, 1], [3, 40]), [5, 6, 7, 8], [1] * 4, 3, 1, 128, 32, 23)
    need = max(fg.fg_paged_attention_shared_workspace_bytes(F.pool, F.tab, F.heads * F.r, len(F.q), int(F.n.max())) for F in (A, B))
    ws = fg.workspace(need)
    want, graphs = [], []
    for F in (A, B):
        F.out, F.dev_q, F.dev_cu, F.s = torch.empty(F.q.shape, dtype=torch.float16, device="cuda"), torch.as_tensor(F.q, device="cuda"), _i32(F.cu), F.find(fg)

        def call(F=F, stream=None):
            fg.fg_pages_share(F.tab, F.dev_cu, F.s, 1, ws=ws, stream=stream)
            fg.fg_paged_attention_shared(F.pool, F.tab, F.dev_cu, F.s, F.dev_q, F.heads * F.r, F.out, int(F.n.max()), 0, ws=ws, stream=stream)

        call()
        torch.cuda.synchronize()
        want.append(F.out.clone())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        graphs.append(g)
        F.out.zero_()
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        call(stream=st)
        st.synchronize()
        assert torch.equal(F.out, want[-1])
    for _ in range(5):
        for F in (A, B):
            F.out.zero_()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(F.out, w) for F, w in zip((A, B), want))
    fg.fg_sync_status()


def test_waits_that_run_out(fg):
    """With a limit of 0 every wait gives up at once: the error word says so, and the next call is right."""
    F = Forked(fg, ([0] * 5 + [1] * 40, [40, 12]), [5] * 45, [1] * 5 + [2] * 40, 2, 4, 128, 16, 25)
    want = _run(fg, F)
    fg.fg_sync_status()
    old = fg.fg_set_wait_limit(0)
    try:
        _run(fg, F)
        with pytest.raises(fg.FGError) as e:
            fg.fg_sync_status()
        assert e.value.status == 7
    finally:
        fg.fg_set_wait_limit(old)
    assert torch.equal(_run(fg, F), want)
    fg.fg_sync_status()
    _hold(want, *F.expect())


def test_one_row_listed_twice_and_groups_that_overlap_stay_in_bounds(fg):
    """Lists that contradict themselves: whoever's rows are not where the share says goes by itself."""
    F = Forked(fg, ([0, 0, 0, 1, 1, 1], [6, 8]), [5, 6, 7, 8, 9, 1], [1] * 6, 2, 2, 64, 16, 26)
    good = F.find(fg)
    ref = F.expect()
    s = fg.PageShare(*[getattr(good, f).clone() for f in FIELDS])
    s.rows[1] = s.rows[0]                                    # sequence 1's place names sequence 0's row
    _hold(_run(fg, F, s), *ref)
    s = fg.PageShare(*[getattr(good, f).clone() for f in FIELDS])
    s.begin[1] = 0                                           # group 0 has no rows, group 1 everyone's
    _hold(_run(fg, F, s)[3:], ref[0][3:], ref[1][3:])
    fg.fg_sync_status()


def test_a_gap_between_groups_ends_them(fg):
    """Groups are numbered without gaps: those behind one are not made, and their sequences go by themselves."""
    n = 40
    F = Forked(fg, (np.repeat(np.arange(n), 2), [4] * n), [3] * (2 * n), [1] * (2 * n), 1, 2, 64, 16, 28)
    good, ref = F.find(fg), F.expect()
    assert int(good.leader[n - 1]) == 2 * n - 2
    s = fg.PageShare(*[getattr(good, f).clone() for f in FIELDS])
    s.leader[3] = -1
    _hold(_run(fg, F, s), *ref)
    every = _run(fg, F, good, min_saved=2 ** 63 - 1)         # never worth it
    alone = torch.empty_like(every)
    fg.fg_paged_attention(F.pool, F.tab, _i32(F.cu), torch.as_tensor(F.q, device="cuda"), F.heads * F.r, alone, 1)
    fg.fg_sync_status()
    assert torch.equal(every, alone)


@pytest.mark.parametrize("d", [64, 128])
def test_many_groups_of_both_kinds(fg, d):
    """40 groups, of few rows and of more than 128 in turn, and more sequences than a CTA plans for itself."""
    which = np.concatenate((np.repeat(np.arange(40), 2), np.full(60, -1)))
    few = np.concatenate((np.repeat(np.arange(40) % 3 > 0, 2), np.arange(60) % 2 > 0))
    F = Forked(fg, (which, [3 + g % 7 for g in range(40)]), np.where(few, 9, 50), np.where(few, 1 + np.arange(140) % 3, 41 + np.arange(140) % 9),
               2, 2, d, 16, 30)
    ref = F.expect()
    out = _run(fg, F)
    assert torch.equal(out, _run(fg, F))
    fg.fg_sync_status()
    _hold(out, *ref)
    alone = torch.empty_like(out)
    fg.fg_paged_attention(F.pool, F.tab, _i32(F.cu), torch.as_tensor(F.q, device="cuda"), 4, alone, int(F.n.max()))
    assert torch.equal(_run(fg, F, min_saved=-1), alone)
    fg.fg_sync_status()


@pytest.mark.parametrize("n, pages, shares", [(1, 20, False), (1, 90, True), (7, 10, False), (20, 24, True), (150, 24, False)])
def test_sharing_where_it_saves(fg, n, pages, shares):
    """The library's own bound: 16 sequences over one prefix go by themselves, bit for bit, where that is cheaper."""
    F = Forked(fg, ([0] * 16, [pages]), [n] * 16, [n] * 16, 16, 1, 128, 64, 29)
    alone, both = torch.empty(F.q.shape, dtype=torch.float16, device="cuda"), _run(fg, F)
    fg.fg_paged_attention(F.pool, F.tab, _i32(F.cu), torch.as_tensor(F.q, device="cuda"), 16, alone, n)
    assert not torch.equal(alone, both)
    assert torch.equal(_run(fg, F, min_saved=-1), both if shares else alone)
    token = 16 * 128 * 5 // 4
    rows = 16 * n
    units = (16 if n <= 16 else 16 * 4) - (-(-rows // 64) if rows <= 128 else 4 * -(-rows // 256))
    saved = (units * 64 * pages - 8 * rows) * token
    assert (saved >= 64 << 20) == shares
    if saved > 0:
        assert torch.equal(_run(fg, F, min_saved=saved), both) and torch.equal(_run(fg, F, min_saved=saved + 1), alone)
    else:
        assert torch.equal(_run(fg, F, min_saved=1), alone)
    fg.fg_sync_status()


@pytest.mark.parametrize("captured", [False, True])
def test_a_serving_run(fg, captured):
    """A prompt, its children, and their steps: queries and keys rotated as they are appended, the prompt's pages found and read
    once for all, every step's rows held to attention over what the cache then holds, which is read back besides."""
    heads, r, d, ps, steps = 2, 2, 64, 16, 6
    seqs, pages = 6, 120
    gen = torch.Generator(device="cuda").manual_seed(31)
    pool, tab = fg.PagePool(pages, ps, heads, d), fg.PageTable.empty(seqs, 40, pages, ps)
    pools, rotary = fg.PagePools([pool]), fg.Rotary(d)

    def rows(n):
        return [torch.randn((n, k * d), generator=gen, device="cuda").half() for k in (heads * r, heads, heads)]

    def hold(q, out, cu):
        table, lens = tab.table.cpu().numpy(), tab.lens.cpu().numpy()
        arr = [[t.cpu().numpy() for t in x] for x in ((pool.k_codes, pool.k_mins, pool.k_scales), (pool.v_codes, pool.v_mins, pool.v_scales))]
        for i in range(seqs):
            a, e = int(cu[i]), int(cu[i + 1])
            if a == e:
                continue
            j = np.arange(lens[i])
            pos = np.repeat(np.arange(lens[i] - (e - a), lens[i]), r)
            for h in range(heads):
                qq = q[a:e].double().cpu().numpy().reshape(e - a, -1, d)[:, h * r:(h + 1) * r].reshape(-1, d)
                k, v = ([t[table[i, j // ps], h, j % ps] for t in x] for x in arr)
                ref, t1 = op.attention_bound(qq, k, v, pos, kind="step")
                _, t2 = op.attention_bound(qq, k, v, pos, kind="chunk")
                got = out[a:e].double().cpu().numpy().reshape(e - a, -1, d)[:, h * r:(h + 1) * r].reshape(-1, d)
                assert op.off_by_too_much(got, ref, t1 + t2 + 130 * 2.0 ** -22 * np.abs(ref)) is None

    # the prompt: 100 rows of sequence 0, and another of 37 that shares nothing
    cu = _i32([0, 100, 100, 100, 100, 137, 137])
    fg.fg_pages_reserve(tab, cu)
    q, k, v = rows(137)
    fg.fg_paged_append_rotated(pool, tab, cu, rotary, q, heads * r, None, k, v)
    share = fg.PageShare.empty(tab, 137)
    fg.fg_pages_share(tab, cu, share, 1)
    assert share.group.max() < 0
    out = torch.empty_like(q)
    fg.fg_paged_attention_shared(pool, tab, cu, share, q, heads * r, out, 100, 0)
    fg.fg_sync_status()
    hold(q, out, cu.tolist())
    # three children; then steps of everyone but row 5
    fg.fg_pages_fork(tab, pools, _i32([0, 0, 0]), _i32([1, 2, 3]))
    cu = _i32([0, 1, 2, 3, 4, 5, 5])
    q, k, v = rows(5)
    turned, out = torch.empty_like(q), torch.empty_like(q)
    share = fg.PageShare.empty(tab, 5)
    kr, vr = torch.empty_like(k), torch.empty_like(v)
    back = [torch.empty_like(k), torch.empty_like(v)]

    def step():
        fg.fg_pages_reserve(tab, cu)
        fg.fg_paged_append_rotated(pool, tab, cu, rotary, q, heads * r, turned, k, v, kr, vr)
        fg.fg_pages_share(tab, cu, share, 1)
        fg.fg_paged_attention_shared(pool, tab, cu, share, turned, heads * r, out, 1, 0)
        fg.fg_paged_read(pool, tab, cu, *back)

    graph = None
    for n in range(steps):
        for t, new in zip((q, k, v), rows(5)):
            t.copy_(new)
        if captured and n == 1:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
        if graph is None:
            step()
        else:
            graph.replay()
        fg.fg_sync_status()
        assert tab.lens.tolist() == [101 + n] * 4 + [38 + n, 0]
        assert share.group.tolist() == [0, 0, 0, 0, -1, -1] and share.tokens.tolist()[:4] == [96] * 4
        hold(turned, out, cu.tolist())
        assert torch.equal(back[0], kr) and torch.equal(back[1], vr)


def test_pools_past_32_bits(fg):
    """Codes of K past 4 GB: the last pages hold what a small pool's first ones do."""
    heads, d, ps, big = 8, 128, 256, 34000
    F = Forked(fg, ([0] * 3, [2]), [40, 300, 7], [1, 20, 1], heads, 1, d, ps, 27)
    want = _run(fg, F)
    pool = fg.PagePool(big, ps, heads, d)
    assert pool.k_codes.numel() > 2 ** 32
    for dst, src in zip((pool.k_codes, pool.k_mins, pool.k_scales, pool.v_codes, pool.v_mins, pool.v_scales),
                        (F.pool.k_codes, F.pool.k_mins, F.pool.k_scales, F.pool.v_codes, F.pool.v_mins, F.pool.v_scales)):
        dst[big - F.pages:] = src
    table = np.where(F.table >= 0, F.table + big - F.pages, -1)
    tab = fg.PageTable(_i32(table), _i32(F.lens), torch.ones(big, dtype=torch.int32, device="cuda"), ps)
    small, F.pool, F.tab = (F.pool, F.tab), pool, tab
    assert torch.equal(_run(fg, F), want)
    n = np.array([100, 552, 0])
    cu = _i32(np.concatenate(([0], np.cumsum(n))))
    k, v, k2, v2 = (torch.empty((652, heads * d), dtype=torch.float16, device="cuda") for _ in range(4))
    fg.fg_paged_read(small[0], small[1], cu, k, v)
    fg.fg_paged_read(pool, tab, cu, k2, v2)
    assert torch.equal(k, k2) and torch.equal(v, v2)
    rotary = fg.Rotary(128, "pairs")
    n = np.array([40, 300, 7])                               # rows behind the shared pages: one writer for each
    cu = _i32(np.concatenate(([0], np.cumsum(n))))
    k, v, k2, v2, *new = (torch.randn((347, heads * d), device="cuda").half() for _ in range(6))
    fg.fg_paged_append_rotated(small[0], small[1], cu, rotary, None, 0, None, *new, k, v)
    fg.fg_paged_append_rotated(pool, tab, cu, rotary, None, 0, None, *new, k2, v2)
    fg.fg_sync_status()
    assert torch.equal(k, k2) and torch.equal(v, v2) and torch.equal(pool.k_codes[big - F.pages:], small[0].k_codes)
