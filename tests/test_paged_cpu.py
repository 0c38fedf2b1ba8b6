"""CPU checks of the paged cache: the entry points refuse bad arguments on the
host before any CUDA call, and the oracle's bookkeeping and attention agree
with independent statements of what they should do."""
import ctypes
import random

import numpy as np
import pytest

from oracle import codec, layer as olayer, paged as op


@pytest.fixture(scope="module")
def fg():
    import __graft_entry__
    __graft_entry__.build()
    import int4_group_quantized_gb300 as fg
    return fg


P = 4096


def _pool(fg, pages=8, ps=16, heads=2, d=64, dtype=0):
    return fg.fg_page_pool(P, P, P, P, P, P, pages, ps, heads, d, dtype)


def _tab(fg, seqs=3, stride=4, pages=8, ps=16):
    return fg.fg_page_table(P, P, P, seqs, stride, pages, ps)


def _br(x):
    return ctypes.byref(x)


def _append(fg, pool, tab, cu=P, k=P, v=P, ld=128, ntok=4, kr=None, vr=None, ldr=128):
    return fg.lib.fg_paged_append(_br(pool), _br(tab), cu, k, v, ld, ntok, kr, vr, ldr, None)


def _attn(fg, pool, tab, cu=P, q=P, ldq=256, qh=4, ntok=4, mq=2, window=0, sinks=0, out=P, ldo=256, ws=P, wsb=1 << 40):
    return fg.lib.fg_paged_attention(_br(pool), _br(tab), cu, q, ldq, qh, ntok, mq, window, sinks, out, ldo, ws, wsb, None)


POOL_ERRORS = [("pages", 0, 1), ("heads", 0, 1), ("page_size", 24, 2), ("page_size", 8, 2), ("page_size", 512, 2),
               ("head_dim", 96, 8), ("head_dim", 256, 8), ("dtype", 5, 1), ("k_codes", 0, 1), ("v_mins", 0, 1),
               ("v_codes", P + 8, 3), ("k_scales", P + 4, 3), ("pages", (1 << 25) + 1, 8), ("pages", 9, 2)]
TAB_ERRORS = [("seqs", -1, 1), ("stride", 0, 1), ("pages", 0, 1), ("page_size", 20, 2), ("table", 0, 1), ("lens", 0, 1),
              ("refs", 0, 1), ("lens", P + 2, 3), ("seqs", (1 << 20) + 1, 8), ("stride", 1 << 27, 8), ("page_size", 32, 2)]


@pytest.mark.parametrize("field,value,status", POOL_ERRORS)
def test_bad_pools_are_refused(fg, field, value, status):
    pool, tab = _pool(fg), _tab(fg)
    setattr(pool, field, value)
    assert _append(fg, pool, tab) == status
    assert _attn(fg, pool, tab) == status
    assert fg.lib.fg_pages_compact(_br(tab), _br(pool), 1, P, 1 << 40, None) == status
    assert fg.lib.fg_pages_fork(_br(tab), _br(pool), 1, P, P, 1, P, 1 << 40, None) == status
    assert fg.lib.fg_paged_attention_workspace_bytes(_br(pool), _br(tab), 4, 4, 2) == 0


@pytest.mark.parametrize("field,value,status", TAB_ERRORS)
def test_bad_tables_are_refused(fg, field, value, status):
    pool, tab = _pool(fg), _tab(fg)
    setattr(tab, field, value)
    assert _append(fg, pool, tab) == status
    assert _attn(fg, pool, tab) == status
    if (field, value) != ("page_size", 32):   # a size of its own, only unlike the pool's
        assert fg.lib.fg_pages_reserve(_br(tab), P, P, 1 << 40, None) == status
        assert fg.lib.fg_pages_free(_br(tab), P, 1, None) == status
        assert fg.lib.fg_pages_workspace_bytes(_br(tab), 0) == 0


def test_null_structures(fg):
    pool, tab = _pool(fg), _tab(fg)
    L = fg.lib
    assert L.fg_paged_append(None, _br(tab), P, P, P, 128, 4, None, None, 0, None) == 1
    assert L.fg_paged_append(_br(pool), None, P, P, P, 128, 4, None, None, 0, None) == 1
    assert L.fg_pages_reserve(None, P, P, 1 << 30, None) == 1
    assert L.fg_pages_compact(_br(tab), None, 2, P, 1 << 30, None) == 1
    assert L.fg_pages_workspace_bytes(None, 0) == 0


def test_append_arguments(fg):
    pool, tab = _pool(fg), _tab(fg)
    assert _append(fg, pool, tab, ntok=-1) == 1
    assert _append(fg, pool, tab, cu=None) == 1
    assert _append(fg, pool, tab, v=None) == 1
    assert _append(fg, pool, tab, kr=P) == 1                  # restored K without V
    assert _append(fg, pool, tab, ld=120) == 2
    assert _append(fg, pool, tab, kr=P, vr=P, ldr=64) == 2
    assert _append(fg, pool, tab, ld=132) == 3
    assert _append(fg, pool, tab, k=P + 8) == 3
    assert _append(fg, pool, tab, kr=P + 8, vr=P) == 3
    assert _append(fg, pool, tab, cu=P + 1) == 3
    assert _append(fg, pool, tab, ntok=(1 << 31) - 1) == 8
    assert _append(fg, pool, tab, ntok=0, cu=None, k=None, v=None) == 0
    empty = _tab(fg, seqs=0)
    assert _append(fg, pool, empty) == 0


def test_attention_arguments(fg):
    pool, tab = _pool(fg), _tab(fg)
    assert _attn(fg, pool, tab, qh=3) == 2                    # no multiple of the K/V heads
    assert _attn(fg, pool, tab, qh=0) == 1
    assert _attn(fg, pool, tab, ntok=-1) == 1
    assert _attn(fg, pool, tab, mq=-1) == 1
    assert _attn(fg, pool, tab, window=-1) == 1
    assert _attn(fg, pool, tab, sinks=-1) == 1
    assert _attn(fg, pool, tab, q=None) == 1
    assert _attn(fg, pool, tab, out=None) == 1
    assert _attn(fg, pool, tab, ldq=248) == 2
    assert _attn(fg, pool, tab, ldo=248) == 2
    assert _attn(fg, pool, tab, ldq=260) == 3
    assert _attn(fg, pool, tab, q=P + 2) == 3
    assert _attn(fg, pool, tab, ws=None) == 5
    need = fg.lib.fg_paged_attention_workspace_bytes(_br(pool), _br(tab), 4, 4, 2)
    assert need > 0 and _attn(fg, pool, tab, wsb=need - 1) == 5
    assert _attn(fg, pool, tab, ws=P + 16) == 3
    assert _attn(fg, pool, tab, ntok=1 << 30) == 8
    assert _attn(fg, pool, tab, ntok=0, q=None, out=None, ws=None, wsb=0) == 0


def test_page_call_arguments(fg):
    pool, tab = _pool(fg), _tab(fg)
    L = fg.lib
    need = L.fg_pages_workspace_bytes(_br(tab), 5)
    assert need > 0
    assert L.fg_pages_workspace_bytes(_br(tab), -1) == 0
    assert L.fg_pages_reserve(_br(tab), None, P, need, None) == 1
    assert L.fg_pages_reserve(_br(tab), P, None, need, None) == 5
    assert L.fg_pages_reserve(_br(tab), P, P, 16, None) == 5
    assert L.fg_pages_reserve(_br(tab), P, P + 8, need, None) == 3
    assert L.fg_pages_free(_br(tab), P, -1, None) == 1
    assert L.fg_pages_free(_br(tab), None, 1, None) == 1
    assert L.fg_pages_free(_br(tab), P + 2, 1, None) == 3
    assert L.fg_pages_free(_br(tab), None, 0, None) == 0
    assert L.fg_pages_fork(_br(tab), _br(pool), 1, P, None, 1, P, need, None) == 1
    assert L.fg_pages_fork(_br(tab), _br(pool), 1, P, P, -1, P, need, None) == 1
    assert L.fg_pages_fork(_br(tab), _br(pool), -1, P, P, 1, P, need, None) == 1
    assert L.fg_pages_fork(_br(tab), _br(pool), 1, P, P, 5, P, need - 1, None) == 5
    assert L.fg_pages_fork(_br(tab), _br(pool), 1, P, P, (1 << 20) + 1, P, 1 << 40, None) == 8
    assert L.fg_pages_fork(_br(tab), _br(pool), 1, None, None, 0, None, 0, None) == 0
    two = (fg.fg_page_pool * 2)(_pool(fg), _pool(fg, heads=3))
    assert L.fg_pages_compact(_br(tab), two, 2, P, need, None) == 2      # layers of unlike geometry
    assert L.fg_pages_compact(_br(tab), _br(pool), 1, P, 100, None) == 5


def test_a_bound_past_32_bits_is_no_bound(fg):
    """max_q times the group must not wrap round: the layout is that of the largest bound, with the chunks' class."""
    pool, tab = _pool(fg), _tab(fg)
    need = fg.lib.fg_paged_attention_workspace_bytes
    small, large = need(_br(pool), _br(tab), 4, 64, 2), need(_br(pool), _br(tab), 4, 64, 1 << 20)
    assert 0 < small < large
    for mq in ((1 << 31) - 1, 1 << 62, (1 << 63) - 1):
        assert need(_br(pool), _br(tab), 4, 64, mq) == large
    for n in (1 << 62, (1 << 63) - 1):
        assert need(_br(pool), _br(tab), 4, n, 2) == 0
        assert _attn(fg, pool, tab, ntok=n) == 8


def test_python_keeps_a_call_on_one_device(fg):
    class At:
        def __init__(self, index):
            self.index, self.device = index, f"device {index}"
    assert fg._beside(At(0), At(0)).index == 0
    for pool, tab in ((At(-1), At(0)), (At(1), At(0)), (At(0), At(1))):
        with pytest.raises(ValueError):
            fg._beside(pool, tab)
    ws = fg.workspace(64, "cpu")
    with pytest.raises(ValueError):
        fg._paged_ws(ws, 64, At(0), None)
    assert fg._beside(fg.PagePools([]), At(0)).index is None      # no pools: the table alone moves
    layers = [At(0), At(1)]
    for p in layers:
        p.struct = _pool(fg)
    with pytest.raises(ValueError):
        fg.PagePools(layers)


def test_python_row_strides(fg):
    import torch
    pool = fg.PagePool(2, 16, 2, 64, device="cpu")
    rows = torch.zeros((3, 136), dtype=torch.float16)
    assert fg._rows(rows[:, :128], pool, 3, 128, "q") == 136
    for stride in (0, 1, 130, 136):                    # a single row has no next one
        assert fg._rows(torch.as_strided(rows, (1, 128), (stride, 1)), pool, 1, 128, "q") == 128
    for bad in (torch.as_strided(rows, (1, 64), (136, 2)), rows[:, :128].float(), rows[:, :64], rows[0, :128]):
        with pytest.raises(ValueError):
            fg._rows(bad, pool, 1 if bad.shape[0] == 1 else 3, bad.shape[-1] if bad.dim() == 2 and bad.shape[0] == 1 else 128, "q")


# ---- the oracle -----------------------------------------------------------------

def _check_invariants(pg, pages):
    """Every page's count is the number of entries that name it."""
    want = np.zeros(pages, int)
    for i in range(len(pg.lens)):
        for j in range(pg.held(i)):
            if pg.table[i, j] >= 0:
                want[pg.table[i, j]] += 1
    assert np.array_equal(want, pg.refs)


@pytest.mark.parametrize("seed", range(6))
def test_oracle_bookkeeping_keeps_every_token(seed):
    """Tokens written by position are found again after any run of operations."""
    rng = random.Random(seed)
    ps, seqs, pages, stride = rng.choice([2, 3, 4]), 7, 40, 9
    pg = op.Pages(np.full((seqs, stride), -1), np.zeros(seqs, int), np.zeros(pages, int), ps)
    data = np.full((pages, ps), -1)
    held = [[] for _ in range(seqs)]
    token = 0
    for _ in range(60):
        what = rng.choice(["grow", "grow", "fork", "free", "compact"])
        if what == "grow":
            n = [rng.randrange(0, 5) if len(held[i]) + 5 <= stride * ps else 0 for i in range(seqs)]
            if sum(n) + sum(map(len, held)) > pages * ps // 2:
                continue
            pg.reserve(n)
            for i, m in enumerate(n):
                for t in range(m):
                    pos = len(held[i])
                    data[pg.table[i, pos // ps], pos % ps] = token
                    held[i].append(token)
                    token += 1
        elif what == "fork":
            a, b = rng.randrange(seqs), rng.randrange(seqs)
            if a == b or held[b] or len(pg.free_pages()) < 1:
                continue
            for x, y in pg.fork([a], [b]):
                data[y] = data[x]
            held[b] = list(held[a])
        elif what == "free":
            i = rng.randrange(seqs)
            pg.free([i, i])
            held[i] = []
        else:
            for x, y in pg.compact():
                data[y] = data[x]
            live = int((pg.refs > 0).sum())
            assert (pg.refs[:live] > 0).all() and (pg.refs[live:] == 0).all()
        _check_invariants(pg, pages)
        for i in range(seqs):
            assert [data[pg.table[i, p // ps], p % ps] for p in range(len(held[i]))] == held[i]
            assert pg.lens[i] == len(held[i])


def test_oracle_attention_agrees_with_the_layer_oracle():
    rng = np.random.default_rng(3)
    q, k, v = rng.normal(size=(5, 64)), rng.normal(size=(40, 64)), rng.normal(size=(40, 64))
    pos = np.arange(35, 40)
    want = olayer.attention(q[None, :, None], k[None, None], v[None, None], pos)[0, :, 0]
    assert np.allclose(op.attention(q, k, v, pos)[0], want, rtol=0, atol=1e-13)
    # a window that covers everything, and sinks that do
    assert np.allclose(op.attention(q, k, v, pos, window=40)[0], want, rtol=0, atol=1e-13)
    assert np.allclose(op.attention(q, k, v, pos, window=1, sinks=40)[0], want, rtol=0, atol=1e-13)
    # a window of one token is that token's value; sinks add the first ones
    assert np.allclose(op.attention(q, k, v, pos, window=1)[0], v[pos], rtol=0, atol=1e-13)
    sel = np.r_[0:2, 36:40]
    w = olayer.attention(q[None, -1:, None], k[None, None, sel], v[None, None, sel], np.array([5]))[0, :, 0]
    assert np.allclose(op.attention(q[-1:], k, v, pos[-1:], window=4, sinks=2)[0], w, rtol=0, atol=1e-13)


def test_oracle_attention_of_rows_that_see_nothing_and_of_nan_groups():
    rng = np.random.default_rng(4)
    q, k, v = rng.normal(size=(3, 128)), rng.normal(size=(6, 128)), rng.normal(size=(6, 128))
    v[4, 64:] = np.nan
    out, _, _ = op.attention(q, k, v, [-1, 3, 5])
    assert (out[0] == 0).all() and np.isfinite(out[1]).all()
    assert np.isfinite(out[2, :64]).all() and np.isnan(out[2, 64:]).all()


def test_oracle_restore_is_the_codec():
    x = np.random.default_rng(5).normal(size=(3, 128)).astype(np.float16)
    c, m, s = codec.quantize_g64(x)
    assert np.array_equal(op.restore(c, m, s).astype(np.float16), codec.dequant_g64(c, m, s, np.float16))
