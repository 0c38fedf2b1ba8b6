"""Steps over shared prefixes to fp16's last bit: neither keys, values nor weights are rounded to fp16 on the way (one row a
K/V head and sequence goes by itself so as well), so nearly every element is the 64-bit result rounded once.  What the
criterion refuses is in test_paged_prefix_exact_cpu.py."""
import numpy as np
import pytest
import torch

from oracle import paged as op
from prefix_cases import CLIMBS, KEYS, MOST, attention, climbing
from test_paged_share_gpu import Forked, _i32, _run, _sizes

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fg():
    import int4_group_quantized_gb300 as fg
    return fg


def _hold(got, ref, mag):
    """Near the 64-bit result everywhere (scores to 2^-17, and fp32 sums), and the nearest fp16 nearly everywhere."""
    got = got.double().cpu().numpy()
    why = op.off_by_too_much(got, ref, op.HALF * np.abs(ref) + 2.0 ** -25 + 2.0 ** -15 * mag)
    assert why is None, why
    share = op.not_nearest(got, ref)
    assert share <= MOST, share


def _climbing(fg, climb, d, members, r, heads, groups, seed):
    """`groups` prefixes of len(climb) tiles, with `members` sequences each that go on for 1 to 3 tokens of their own."""
    ps, pre = 64, len(climb) * KEYS
    shared = pre // ps
    own = 1 + np.arange(groups * members) % 3
    pages = groups * shared + len(own)
    table = np.full((len(own), shared + 1), -1)
    arr = {w: [np.zeros((pages, heads, ps, d // 2), np.uint8)] + [np.zeros((pages, heads, ps, d // 64), np.float32) for _ in range(2)] for w in "kv"}
    q = np.zeros((len(own), heads * r * d), np.float16)
    ref, mag = np.zeros(q.shape), np.zeros(q.shape)
    for g in range(groups):
        at = np.arange(g * shared, (g + 1) * shared)
        for h in range(heads):
            # the last tile once more: the sequences' own tokens are some of its keys
            qs, *kv = climbing([*climb, 0], d, members * r, seed + 1000 * g + h)
            for w, x in zip("kv", kv):
                for to, a in zip(arr[w], x):
                    to[at, h] = a[:pre].reshape(shared, ps, -1)
            keep = [op.restore(*x) for x in kv]
            for m in range(members):
                i = g * members + m
                page = groups * shared + i
                table[i, :shared], table[i, shared] = at, page
                mine = pre + (7 * m + np.arange(own[i])) % KEYS
                for w, x in zip("kv", kv):
                    for to, a in zip(arr[w], x):
                        to[page, h, :own[i]] = a[mine]
                sl = np.s_[h * r * d:(h + 1) * r * d]
                q[i, sl] = qs[m * r:(m + 1) * r].reshape(-1)
                k, v = (np.concatenate((x[:pre], x[mine])) for x in keep)
                rows = qs[m * r:(m + 1) * r].astype(np.float64)
                ref[i, sl] = attention(rows, k, v, 1 / np.sqrt(d)).reshape(-1)
                mag[i, sl] = attention(rows, k, np.abs(v), 1 / np.sqrt(d)).reshape(-1)
    k, v = ([torch.as_tensor(a, device="cuda") for a in arr[w]] for w in "kv")
    pool = fg.PagePool.of(*k, *v, torch.float16)
    tab = fg.PageTable(_i32(table), _i32(pre + own), _i32(np.ones(pages)), ps)
    return pool, tab, q, ref, mag


@pytest.mark.parametrize("members, r", [(3, 2), (21, 3)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("name", CLIMBS)
def test_scores_that_climb(fg, name, d, members, r):
    """64 heads of three prefixes: a CTA's share of the line holds several tiles, beginning anywhere in a climb."""
    pool, tab, q, ref, mag = _climbing(fg, CLIMBS[name], d, members, r, 64, 3, 5)
    n = len(q)
    cu = _i32(np.arange(n + 1))
    share = fg.PageShare.empty(tab, n)
    fg.fg_pages_share(tab, cu, share, 1)
    assert share.group.tolist() == [i // members for i in range(n)]
    out = torch.empty(q.shape, dtype=torch.float16, device="cuda")
    fg.fg_paged_attention_shared(pool, tab, cu, share, torch.as_tensor(q, device="cuda"), 64 * r, out, 1, 0)
    fg.fg_sync_status()
    _hold(out, ref, mag)


STEPS = {   # groups, tails, rows, heads, query heads a head, d, page size
    "one row": (([0] * 6 + [1] * 3, [60, 31]), _sizes(9, 1, 300, 1), [1] * 9, 4, 1, 64, 16),
    "four query heads": (([0] * 20 + [-1], [20]), _sizes(21, 1, 300, 2), [1] * 21, 2, 4, 128, 64),
    "some rows": (([0, 1] * 4, [40, 26]), _sizes(8, 3, 200, 3), [1, 2, 1, 1, 2, 2, 1, 1], 3, 2, 128, 16),
    "three units": (([0] * 150, [70]), _sizes(150, 1, 20, 4), [1] * 150, 2, 1, 64, 16),
    "eleven tiles a CTA": (([0] * 5, [90]), _sizes(5, 1, 20, 5), [1] * 5, 40, 2, 64, 64),
    "the same of 128": (([0] * 5, [90]), _sizes(5, 1, 20, 6), [1] * 5, 40, 2, 128, 64),
}


@pytest.mark.parametrize("name", STEPS)
def test_steps(fg, name):
    groups, tails, n, heads, r, d, ps = STEPS[name]
    F = Forked(fg, groups, tails, n, heads, r, d, ps, 41)
    out = _run(fg, F)
    fg.fg_sync_status()
    ref, mag = F.expect()[0], np.zeros(F.q.shape)
    for i, length in enumerate(F.lens):
        j = np.arange(length)
        for h in range(heads):
            sl = np.s_[F.cu[i]:F.cu[i + 1], h * r * d:(h + 1) * r * d]
            v = op.restore(*(x[F.table[i, j // ps], h, j % ps] for x in F.arr["v"]))
            mag[sl] = np.abs(v).max()                        # no less than the weighted mean
    _hold(out, ref, mag)


MIXED = {   # groups, tails, rows, heads, query heads a head, d, page size: steps of at most 4 rows a K/V head, and chunks of their group
    "steps first": (([0] * 36, [24]), np.r_[_sizes(30, 1, 60, 1), _sizes(6, 100, 160, 2)], [1] * 30 + [40, 100, 64, 9, 77, 90], 2, 2, 128, 64),
    "in turn": (([0, 1] * 20, [50, 33]), np.resize([7, 9, 90, 130], 40), np.resize([1, 1, 70, 33], 40), 2, 2, 64, 16),
    "one among many": (([0] * 7 + [-1], [30]), [80, 70, 60, 5, 99, 64, 40, 50], [50, 60, 41, 2, 64, 64, 40, 1], 3, 1, 128, 32),
    "few rows of chunks": (([0] * 50, [30]), np.r_[_sizes(49, 1, 60, 3), 70], [1] * 49 + [60], 2, 1, 64, 32),
    "two kinds of groups": (([0] * 20 + [1] * 20 + [2] * 5, [40, 11, 20]), np.r_[np.full(20, 9), _sizes(25, 60, 90, 4)],
                            [1] * 20 + [1, 2] * 5 + [50] * 10 + [55] * 5, 2, 1, 64, 32),
    "more than a CTA plans": (([0, 1, 2] * 60, [40, 3, 20]), np.resize([3, 66, 5, 40], 180), np.resize([1, 50, 2, 40], 180), 1, 2, 64, 16),
}


@pytest.mark.parametrize("name", MIXED)
def test_steps_beside_chunks_of_their_group(fg, name):
    """A step is as exact beside chunks as without them; the chunks keep their bounds."""
    groups, tails, n, heads, r, d, ps = MIXED[name]
    F = Forked(fg, groups, tails, n, heads, r, d, ps, 43)
    out = _run(fg, F)
    assert torch.equal(out, _run(fg, F))
    fg.fg_sync_status()
    ref, tol = F.expect()
    got = out.double().cpu().numpy()
    why = op.off_by_too_much(got, ref, tol, 3 * op.HALF)
    assert why is None, why
    steps = np.repeat(np.asarray(n) * r <= 4, n)
    assert (np.asarray(n) * r <= 16).sum() == (np.asarray(n) * r <= 4).sum() > 0
    share = op.not_nearest(got[steps], ref[steps])
    assert share <= MOST, share


def test_more_sequences_and_groups_than_a_plan_keeps_near(fg):
    """1,060 groups of two: two chunks, two steps, a chunk and a step in turn, past what the plan's shared memory holds."""
    g = 1060
    kind = np.arange(g) % 3
    n = np.stack((np.where(kind == 0, 70, np.where(kind == 1, 1, 131)), np.where(kind == 0, 66, 1)), 1).reshape(-1)
    F = Forked(fg, (np.repeat(np.arange(g), 2), np.ones(g, int)), n + np.arange(2 * g) % 5, n, 1, 1, 64, 16, 44)
    share = F.find(fg)
    assert int(share.group.max()) == g - 1
    out = _run(fg, F, share)
    assert torch.equal(out, _run(fg, F, share))
    fg.fg_sync_status()
    ref, tol = F.expect()
    got = out.double().cpu().numpy()
    why = op.off_by_too_much(got, ref, tol, 3 * op.HALF)
    assert why is None, why
    steps = np.repeat(n == 1, n)
    assert op.not_nearest(got[steps], ref[steps]) <= MOST


@pytest.mark.parametrize("seqs", [1023, 1024, 1025, 1100])
def test_one_group_of_many_sequences(fg, seqs):
    """Steps and chunks of one prefix in turn, around the number of sequences that the plan keeps near."""
    n = np.where(np.arange(seqs) % 7 == 3, 18, 1)
    F = Forked(fg, (np.where(np.arange(seqs) % 11 == 5, -1, 0), [9]), n + np.arange(seqs) % 3, n, 1, 1, 64, 16, 45)
    out = _run(fg, F)
    fg.fg_sync_status()
    ref, tol = F.expect()
    got = out.double().cpu().numpy()
    why = op.off_by_too_much(got, ref, tol, 3 * op.HALF)
    assert why is None, why
    steps = np.repeat(n == 1, n)
    assert op.not_nearest(got[steps], ref[steps]) <= MOST
