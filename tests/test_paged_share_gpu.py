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
