"""CPU checks of shared prefixes, rotary positions and rows read back: the entry
points refuse bad arguments on the host before any CUDA call, the frequencies
are the formulas', and the oracle agrees with independent statements."""
import ctypes
import math

import numpy as np
import pytest

from oracle import paged as op, rotary as orot


@pytest.fixture(scope="module")
def fg():
    import __graft_entry__
    __graft_entry__.build()
    import int4_group_quantized_gb300 as fg
    return fg


P = 4096


def _br(x):
    return ctypes.byref(x)


def _pool(fg, pages=8, ps=16, heads=2, d=64, dtype=0):
    return fg.fg_page_pool(P, P, P, P, P, P, pages, ps, heads, d, dtype)


def _tab(fg, seqs=3, stride=4, pages=8, ps=16):
    return fg.fg_page_table(P, P, P, seqs, stride, pages, ps)


def _rot(fg, turns=P, rot=64, layout=0, scale=1.0):
    return fg.fg_rotary(turns, rot, layout, scale)


# ---- rotary ------------------------------------------------------------------------

@pytest.mark.parametrize("scaling", ["plain", "linear", "base", "bands", "ramp"])
@pytest.mark.parametrize("rot", [2, 4, 16, 64, 128, 20])
def test_turns_are_the_formulas(fg, scaling, rot):
    if scaling == "base" and rot == 2:
        pytest.skip("refused: see test_turns_arguments")
    for base, factor, context, low, high in ((10000.0, 8.0, 4096.0, 1.0, 4.0), (5e5, 32.0, 8192.0, 1.0, 32.0), (10000.0, 1.0, 100.0, 0.5, 2.0)):
        turns, scale = fg.fg_rotary_turns(rot, fg._SCALINGS[scaling], base, factor, context, low, high)
        theta, want = orot.thetas(rot, scaling, base, factor, context, low, high)
        assert scale == np.float32(want)
        got = turns.numpy().view(np.uint64)
        assert len(got) == rot // 2
        for g, t in zip(got, theta):
            part = t / (2 * math.pi)
            # both from fp64: a dozen roundings of 2^-53, and half a unit of 2^-64.  The oracle's power is exp(y): y, at most
            # ln of the base, is a product of a rounded logarithm and rounded itself, which moves exp(y) by 2 |y| 2^-53
            y = math.log(base) + (math.log(factor) * rot / (rot - 2) if scaling == "base" else 0.0)
            assert abs(int(g) / 2.0 ** 64 - (part - math.floor(part))) <= (16 + 2 * y) * 2.0 ** -53 * part + 2.0 ** -64


def test_turns_arguments(fg):
    t = (ctypes.c_uint64 * 64)()
    s = ctypes.c_float()

    def turns(rot=64, kind=0, base=1e4, factor=2.0, context=100.0, low=1.0, high=2.0, out=t, scale=_br(s)):
        return fg.lib.fg_rotary_turns(rot, kind, base, factor, context, low, high, out, scale)

    assert turns() == 0
    assert turns(out=None) == 1 and turns(scale=None) == 1
    assert turns(kind=5) == 1 and turns(kind=-1) == 1
    assert turns(rot=0) == 2 and turns(rot=7) == 2 and turns(rot=-2) == 2 and turns(rot=65538) == 2
    for base in (1.0, 0.0, -3.0, math.nan, math.inf):
        assert turns(base=base) == 1
    for factor in (0.0, -1.0, math.nan, math.inf):
        assert turns(kind=1, factor=factor) == 1
    assert turns(kind=0, factor=0.0) == 0                     # not read
    assert turns(kind=2, rot=2) == 2
    assert turns(kind=4, factor=0.5) == 1 and turns(kind=3, factor=0.5) == 0
    for kind in (3, 4):
        assert turns(kind=kind, context=0.0) == 1 and turns(kind=kind, low=0.0) == 1 and turns(kind=kind, low=2.0) == 1
        assert turns(kind=kind, high=math.inf) == 1 and turns(kind=kind, low=math.nan) == 1


def test_rotate_arguments(fg):
    def rot(r=_rot(fg), x=P, dt=0, rows=3, ldx=128, heads=2, d=64, pos=P, out=P, ldo=128):
        return fg.lib.fg_rotate(_br(r) if r is not None else None, x, dt, rows, ldx, heads, d, pos, out, ldo, None)

    assert rot(rows=0) == 0 and rot(heads=0) == 0 and rot(rows=0, x=None, out=None, pos=None) == 0
    assert rot(r=None) == 1 and rot(r=_rot(fg, turns=None)) == 1 and rot(r=_rot(fg, layout=2)) == 1
    assert rot(r=_rot(fg, scale=math.inf)) == 1 and rot(r=_rot(fg, scale=math.nan)) == 1
    assert rot(r=_rot(fg, turns=P + 4)) == 3
    for n in (0, 1, 63, 66, -2):
        assert rot(r=_rot(fg, rot=n)) == 2
    assert rot(dt=2) == 1 and rot(rows=-1) == 1 and rot(heads=-1) == 1 and rot(d=-64) == 1
    assert rot(heads=65536) == 8 and rot(d=65538, heads=1) == 8
    assert rot(x=None) == 1 and rot(out=None) == 1 and rot(pos=None) == 1
    assert rot(ldx=127) == 2 and rot(ldo=64, out=1 << 20) == 2
    assert rot(x=P + 1) == 3 and rot(pos=P + 2) == 3 and rot(dt=1, out=P + 2) == 3
    # out: x itself with its stride, columns beside x's in the same rows, or other memory
    assert rot(ldo=256) == 1
    for off in (2, 128, 254, -2):                             # bytes; a row of 2 heads is 256
        assert rot(out=P + off) == 1
    assert rot(x=P, out=P + 256, ldx=192, ldo=192) == 1       # 192 - 128 columns between them


def test_append_rotated_arguments(fg):
    def app(pool=_pool(fg), tab=_tab(fg), cu=P, r=_rot(fg), q=P, ldq=256, qh=4, qo=P, ldqo=256, k=P, v=P, ld=128, ntok=4, kr=None, vr=None, ldr=128):
        return fg.lib.fg_paged_append_rotated(_br(pool) if pool else None, _br(tab), cu, _br(r) if r else None, q, ldq, qh, qo, ldqo, k, v, ld,
                                              ntok, kr, vr, ldr, None)

    assert app(ntok=0) == 0 and app(tab=_tab(fg, seqs=0)) == 0
    assert app(pool=None) == 1 and app(r=None) == 1 and app(r=_rot(fg, turns=None)) == 1
    assert app(pool=_pool(fg, pages=9)) == 2 and app(pool=_pool(fg, d=96)) == 8 and app(pool=_pool(fg, dtype=7)) == 1
    for n in (8, 24, 56, 80):
        assert app(r=_rot(fg, rot=n)) == 2                    # no multiple of 16, or more than the head
    assert app(ntok=-1) == 1 and app(qh=-1) == 1 and app(qh=65536) == 8
    assert app(cu=None) == 1 and app(k=None) == 1 and app(v=None) == 1 and app(qo=None) == 1
    assert app(kr=P) == 1 and app(vr=P) == 1
    assert app(ld=120) == 2 and app(ldq=248) == 2 and app(ldqo=248) == 2 and app(kr=P, vr=P, ldr=64) == 2
    assert app(ld=132) == 3 and app(ldq=260) == 3 and app(q=P + 8) == 3 and app(qo=P + 2) == 3 and app(k=P + 8) == 3 and app(cu=P + 1) == 3
    assert app(ntok=(1 << 31) - 1) == 8
    # rotated queries: q itself with its stride, or memory apart from it
    assert app(ldqo=264) == 1 and app(qo=P + 16) == 1 and app(qo=P + 256) == 1 and app(qo=P + 512, ldq=512, ldqo=264) == 1


def test_read_arguments(fg):
    def read(pool=_pool(fg), tab=_tab(fg), cu=P, start=None, k=P, v=P, ld=128, ntok=4):
        return fg.lib.fg_paged_read(_br(pool) if pool else None, _br(tab), cu, start, k, v, ld, ntok, None)

    assert read(ntok=0) == 0 and read(k=None, v=None) == 0 and read(tab=_tab(fg, seqs=0)) == 0
    assert read(pool=None) == 1 and read(cu=None) == 1 and read(ntok=-1) == 1
    assert read(pool=_pool(fg, ps=32)) == 2 and read(ld=120) == 2
    assert read(ld=132) == 3 and read(k=P + 8) == 3 and read(v=P + 2) == 3 and read(start=P + 2) == 3
    assert read(ntok=(1 << 31) - 1) == 8


# ---- sharing -----------------------------------------------------------------------

def _share(fg, seqs=3, ntok=4, **kw):
    s = fg.fg_page_share(P, P, P, P, P, P, seqs, ntok)
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def test_share_arguments(fg):
    def find(tab=_tab(fg), cu=P, least=1, s=None, ws=P, wsb=1 << 40):
        s = _share(fg) if s is None else s
        return fg.lib.fg_pages_share(_br(tab) if tab else None, cu, least, _br(s) if s else None, ws, wsb, None)

    assert find(tab=None) == 1 and find(s=False) == 1 and find(cu=None) == 1
    assert find(least=0) == 1 and find(least=-5) == 1
    assert find(s=_share(fg, seqs=2)) == 2 and find(s=_share(fg, ntok=-1)) == 1
    for field in ("group", "tokens", "first", "leader", "begin", "rows"):
        assert find(s=_share(fg, **{field: None})) == 1
        assert find(s=_share(fg, **{field: P + 2})) == 3
    assert find(cu=P + 2) == 3 and find(ws=None) == 5 and find(ws=P + 16) == 3
    need = fg.lib.fg_pages_share_workspace_bytes(_br(_tab(fg)))
    assert need > 0 and find(wsb=need - 1) == 5
    assert find(tab=_tab(fg, seqs=20000), s=_share(fg, seqs=20000)) == 8
    assert find(tab=_tab(fg, seqs=0), s=_share(fg, seqs=0), cu=None, ws=None) == 0
    assert fg.lib.fg_pages_share_workspace_bytes(None) == 0


def test_oracle_share_by_hand():
    t = np.array([[5, 6, 7, 8], [5, 6, 9, -1], [5, 6, 7, 1], [2, 3, -1, -1], [2, 3, 4, -1], [5, 6, 7, 8]])
    lens, n = np.array([64, 40, 60, 20, 40, 64]), np.array([1, 2, 1, 1, 0, 1])
    cu = np.concatenate(([0], np.cumsum(n)))
    # 0, 2 and 5 share three pages (6 reads saved), 1 shares two with them (also 6): three it is.  4 takes no part, so 3 is alone
    group, tokens, first, leader, begin, rows = op.share(t, lens, cu, 10, 16, 1)
    assert group.tolist() == [0, -1, 0, -1, -1, 0] and tokens.tolist() == [48, 0, 48, 0, 0, 48]
    assert first.tolist() == [0, 0, 1, 0, 0, 2] and leader.tolist() == [0] + [-1] * 5
    assert begin.tolist() == [0] + [3] * 6 and rows.tolist() == [0, 3, 5, -1, -1, -1]
    assert op.share(t, lens, cu, 10, 16, 49)[0].max() == -1
    # an entry that names no page ends the prefix: with two pages everyone is in
    t[5, 2] = 77
    assert op.share(t, lens, cu, 10, 16, 1)[0].tolist() == [0, 0, 0, -1, -1, 0]


def test_shared_attention_arguments(fg):
    pool, tab = _pool(fg), _tab(fg)

    def attend(pool=pool, tab=tab, cu=P, s=None, q=P, ldq=256, qh=4, ntok=4, mq=2, out=P, ldo=256, ws=P, wsb=1 << 40):
        s = _share(fg) if s is None else s
        return fg.lib.fg_paged_attention_shared(_br(pool), _br(tab), cu, _br(s) if s else None, q, ldq, qh, ntok, mq, 0, out, ldo, ws, wsb, None)

    assert attend(s=False) == 1 and attend(s=_share(fg, seqs=4)) == 2 and attend(s=_share(fg, ntok=5)) == 2
    for field in ("group", "tokens", "first", "leader", "begin", "rows"):
        assert attend(s=_share(fg, **{field: None})) == 1
        assert attend(s=_share(fg, **{field: P + 1})) == 3
    assert attend(qh=3) == 2 and attend(qh=0) == 1 and attend(ntok=-1) == 1 and attend(mq=-1) == 1
    assert attend(cu=None) == 1 and attend(q=None) == 1 and attend(out=None) == 1
    assert attend(ldq=248) == 2 and attend(ldo=248) == 2 and attend(ldq=260) == 3 and attend(q=P + 2) == 3 and attend(cu=P + 1) == 3
    need = fg.lib.fg_paged_attention_shared_workspace_bytes(_br(pool), _br(tab), 4, 4, 2)
    assert need > fg.lib.fg_paged_attention_workspace_bytes(_br(pool), _br(tab), 4, 4, 2)
    assert attend(ws=None) == 5 and attend(wsb=need - 1) == 5 and attend(ws=P + 16) == 3
    assert attend(ntok=0, s=_share(fg, ntok=0)) == 0 and attend(mq=0) == 0
    assert fg.lib.fg_paged_attention_shared_workspace_bytes(_br(_pool(fg, ps=32)), _br(tab), 4, 4, 2) == 0
    f32 = _pool(fg, dtype=1)      # every sequence by itself, in that call's workspace
    assert fg.lib.fg_paged_attention_shared_workspace_bytes(_br(f32), _br(tab), 4, 4, 2) == \
        fg.lib.fg_paged_attention_workspace_bytes(_br(f32), _br(tab), 4, 4, 2)
    assert attend(pool=f32, wsb=16) == 5


def test_python_checks(fg):
    import torch

    i32 = lambda *n: torch.zeros(n, dtype=torch.int32)
    with pytest.raises(ValueError, match="layout"):
        fg.Rotary(64, "sideways", device="cpu")
    with pytest.raises(fg.FGError, match="FG_ERR_SHAPE"):
        fg.Rotary(63, device="cpu")
    rotary = fg.Rotary(64, device="cpu")
    assert rotary.turns.dtype == torch.int64 and rotary.turns.numel() == 32 and rotary.scale == 1.0
    x = torch.zeros((4, 128), dtype=torch.float16)
    with pytest.raises(ValueError, match="heads"):
        fg.fg_rotate(rotary, x, i32(4), 3)
    with pytest.raises(ValueError, match="pos"):
        fg.fg_rotate(rotary, x, i32(3), 2)
    with pytest.raises(ValueError, match="pos"):
        fg.fg_rotate(rotary, x, i32(4).long(), 2)
    with pytest.raises(ValueError, match="out"):
        fg.fg_rotate(rotary, x, i32(4), 2, x.float())
    with pytest.raises(ValueError, match="adjacent"):
        fg.fg_rotate(rotary, torch.zeros((4, 256), dtype=torch.float16)[:, ::2], i32(4), 2)
    with pytest.raises(ValueError, match="no device"):
        fg.fg_rotate(rotary, x, i32(4), 2)
    with pytest.raises(ValueError, match="first"):
        fg.PageShare(i32(3), i32(3), i32(2), i32(3), i32(4), i32(5))
    with pytest.raises(ValueError, match="begin"):
        fg.PageShare(i32(3), i32(3), i32(3), i32(3), i32(3), i32(5))
    with pytest.raises(ValueError, match="rows"):
        fg.PageShare(i32(3), i32(3), i32(3), i32(3), i32(4), torch.zeros(5))
    s = fg.PageShare(i32(3), i32(3), i32(3), i32(3), i32(4), i32(5))
    assert (s.seqs, s.ntok) == (3, 5)
