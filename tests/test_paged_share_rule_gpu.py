"""When a call shares: what is counted, where a share is older than the batch it is used for.  A call that does not share
gives the bits of fg_paged_attention, one that does gives others."""
import numpy as np
import pytest
import torch

from test_paged_share_gpu import FIELDS, Forked, _hold, _i32, _run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fg():
    import int4_group_quantized_gb300 as fg
    return fg


def _alone(fg, F):
    out = torch.full(F.q.shape, 7.0, dtype=F.dtype, device="cuda")
    fg.fg_paged_attention(F.pool, F.tab, _i32(F.cu), torch.as_tensor(F.q, device="cuda"), F.heads * F.r, out, int(F.n.max()))
    return out


def _decides(fg, F, share, saved):
    """Shares up to `saved` bytes and no further."""
    ref, alone, both = F.expect(), _alone(fg, F), _run(fg, F, share)
    assert not torch.equal(alone, both)
    for least, want in ((1, both), (saved, both), (saved + 1, alone), (2 * saved, alone)):
        got = _run(fg, F, share, min_saved=least)
        assert torch.equal(got, want), least
        _hold(got, *ref)
    fg.fg_sync_status()


def test_sequences_cut_back_save_nothing(fg):
    """Three of six sequences now end inside the prefix: their rows go by themselves, and what they read is not saved."""
    F = Forked(fg, ([0] * 6, [30]), [40, 20, 50, 33, 25, 60], [1] * 6, 2, 2, 128, 16, 51)
    share = F.find(fg)
    assert share.tokens.tolist() == [480] * 6
    F.lens[[1, 3, 4]] = [480, 400, 5]
    F.upload(fg)
    # three read 480 tokens each, the group them once, and six rows of two query heads leave their parts
    _decides(fg, F, share, 2 * 128 * 5 // 4 * (480 * (3 - 1) - 8 * 2 * 6))


def test_groups_behind_a_gap_save_nothing(fg):
    """Groups are looked at 32 at a time up to the first gap: what others would save is not counted."""
    n = 40
    F = Forked(fg, (np.repeat(np.arange(n), 2), [8] * n), [3] * (2 * n), [1] * (2 * n), 1, 2, 64, 16, 52)
    good = F.find(fg)
    share = fg.PageShare(*[getattr(good, f).clone() for f in FIELDS])
    share.leader[3] = -1
    groups = 31                                              # 0 .. 31 but the gap
    _decides(fg, F, share, 64 * 5 // 4 * (groups * (2 - 1) * 128 - 8 * 2 * 2 * groups))


def test_rows_that_the_share_lists_elsewhere_save_nothing(fg):
    """Sequences whose place in the list names other rows go by themselves."""
    F = Forked(fg, ([0] * 8, [25]), [9] * 8, [1] * 8, 2, 1, 64, 16, 53)
    good = F.find(fg)
    share = fg.PageShare(*[getattr(good, f).clone() for f in FIELDS])
    share.rows[5:8] = share.rows[0]
    _decides(fg, F, share, 2 * 64 * 5 // 4 * (400 * (5 - 1) - 8 * 8))


@pytest.mark.parametrize("d", [64, 128])
def test_steps_and_chunks_of_a_group_decide_apart(fg, d):
    """A prefix over two steps and twelve chunks of 20 rows: the chunks save much, the steps little."""
    F = Forked(fg, ([0] * 14, [30]), [9] + [30] * 12 + [12], [1] + [20] * 12 + [1], 2, 1, d, 16, 54)
    share, ref, alone = F.find(fg), F.expect(), _alone(fg, F)
    both = _run(fg, F, share)
    token = 2 * d * 5 // 4
    steps = token * (480 * (2 - 1) - 8 * 2)
    chunks = token * (480 * 4 * (12 - 1) - 8 * 240)          # 240 rows: one unit of 256
    row = torch.as_tensor(np.repeat(F.n == 1, F.n), device="cuda")
    for least, s, c in ((0, both, both), (steps, both, both), (steps + 1, alone, both), (chunks, alone, both), (chunks + 1, alone, alone)):
        out = _run(fg, F, share, min_saved=least)
        fg.fg_sync_status()
        assert torch.equal(out[row], s[row]) and torch.equal(out[~row], c[~row]), least
        _hold(out, *ref)
    assert not torch.equal(alone[row], both[row]) and not torch.equal(alone[~row], both[~row])


BY_ITSELF = {   # 32 heads of 128, one prefix: sequences, rows of each, tokens, and whether sharing is faster (us alone, shared)
    "4 steps over 8,192": (4, 1, 8192, False),               # 44, 55
    "8 steps over 2,048": (8, 1, 2048, False),               # 33, 37
    "16 chunks of 32 over 512": (16, 32, 512, False),        # 78, 107 (they save 126 MB by the count that min_saved has)
    "4 chunks of 128 over 4,096": (4, 128, 4096, False),     # 84, 99 (147 MB)
    "16 steps over 2,048": (16, 1, 2048, True),              # 60, 41
    "16 chunks of 20 over 2,048": (16, 20, 2048, True),      # 150, 122
}


@pytest.mark.parametrize("name", BY_ITSELF)
def test_the_librarys_own_rule(fg, name):
    """Calls that measured slower when they shared go by themselves."""
    b, n, tokens, shares = BY_ITSELF[name]
    F = Forked(fg, ([0] * b, [tokens // 64]), [300] * b, [n] * b, 32, 1, 128, 64, 55)
    share = F.find(fg)
    alone, both = _alone(fg, F), _run(fg, F, share)
    assert not torch.equal(alone, both)
    assert torch.equal(_run(fg, F, share, min_saved=-1), both if shares else alone)
    fg.fg_sync_status()
