"""GPU parity of rotary positions (fg_rotate, fg_paged_append_rotated) and of rows
read back (fg_paged_read).

fg_rotate is held to the oracle in 64 bits, whose angles come exactly from the
turns.  An element's bound: cosine and sine rounded to fp32 (2^-24 of the pair's
size each way), two products and a sum rounded (2^-24 each), and half a step of
the result's type: eps/2 relative, half the smallest subnormal.

fg_paged_append_rotated is the same bits as fg_rotate and fg_paged_append, and
fg_paged_read the codec's own restored values, both compared bit for bit.
"""
import numpy as np
import pytest
import torch

from oracle import codec, rotary as orot

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "f32": torch.float32}


@pytest.fixture(scope="module")
def fg():
    import int4_group_quantized_gb300 as fg
    return fg


def _i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _turns(rotary):
    return rotary.turns.cpu().numpy().view(np.uint64)


def _bound(ref, tol, dt):
    eps, tiny = (2.0 ** -11, 2.0 ** -25) if dt == torch.float16 else (2.0 ** -24, 2.0 ** -150)
    return tol + eps * (np.abs(ref) + tol) + tiny


def _check_rotate(got, x, pos, heads, rotary):
    ref, tol = orot.rotate(x.double().cpu().numpy(), pos, heads, rotary.rot, rotary.layout, _turns(rotary), rotary.scale)
    err = np.abs(got.double().cpu().numpy() - ref)
    over = err - _bound(ref, tol, x.dtype)
    assert over.max(initial=-1.0) <= 0, f"off by {err.max()}, {over.max()} above the bound"


SHAPES = [  # rows, heads, head_dim, rot
    (1, 1, 64, 64), (3, 2, 128, 128), (5, 3, 128, 32), (7, 1, 80, 16), (9, 2, 64, 48), (2, 3, 24, 10), (4, 2, 6, 2), (6, 1, 33, 20),
    (17, 5, 256, 256), (1, 64, 128, 128), (130, 12, 64, 64), (33, 1, 96, 96)]


@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("n,heads,d,rot", SHAPES)
def test_rotate(fg, n, heads, d, rot, dt, layout):
    gen = torch.Generator(device="cuda").manual_seed(n * 1000 + d + rot)
    rotary = fg.Rotary(rot, layout)
    x = torch.randn((n, heads * d), generator=gen, device="cuda").to(DT[dt])
    pos = torch.randint(0, 40000, (n,), generator=gen, device="cuda", dtype=torch.int32)
    out = torch.full_like(x, 7.0)
    assert fg.fg_rotate(rotary, x, pos, heads, out) is out
    fg.fg_sync_status()
    _check_rotate(out, x, pos.tolist(), heads, rotary)
    y = x.clone()
    fg.fg_rotate(rotary, y, pos, heads)          # in place: the same bits
    assert torch.equal(y, out)


@pytest.mark.parametrize("layout", ["half", "pairs"])
def test_sums_and_products_are_rounded_one_by_one(fg, layout):
    """fp32 rows moved 16 bytes at a time and two elements at a time are the same bits, those of separate operations on
    cosines and sines rounded to fp32 (which differ from fp64's rounded ones in 3.5e-5 of the angles)."""
    n, d = 400, 128
    rotary = fg.Rotary(d, layout)
    gen = torch.Generator(device="cuda").manual_seed(8)
    wide = torch.randn((n, d + 1), generator=gen, device="cuda")
    pos = torch.randint(0, 5000, (n,), generator=gen, device="cuda", dtype=torch.int32)
    x = wide[:, 1:].contiguous()
    a, b = (fg.fg_rotate(rotary, t, pos, 1, torch.empty_like(x)) for t in (x, wide[:, 1:]))
    assert torch.equal(a, b)
    ang = torch.as_tensor(orot.angles(pos.tolist(), _turns(rotary)), device="cuda")
    c, s = torch.cos(ang).float(), torch.sin(ang).float()
    u, v = (x[:, :64], x[:, 64:]) if layout == "half" else (x[:, 0::2], x[:, 1::2])
    y, z = u * c - v * s, u * s + v * c
    want = torch.cat((y, z), 1) if layout == "half" else torch.stack((y, z), -1).reshape(n, d)
    assert float((a != want).float().mean()) < 1e-3


@pytest.mark.parametrize("dt", ["f16", "f32"])
def test_far_positions_lose_nothing(fg, dt):
    rotary = fg.Rotary(64)
    pos = [0, 1, 2 ** 24 + 1, 2 ** 30, 2 ** 31 - 1, -1, -(2 ** 31)]
    x = torch.randn((len(pos), 64), device="cuda").to(DT[dt])
    out = fg.fg_rotate(rotary, x, _i32(pos), 1, torch.empty_like(x))
    _check_rotate(out, x, pos, 1, rotary)
    assert torch.equal(out[0], x[0])             # position 0 changes nothing


@pytest.mark.parametrize("kind,kw", [("linear", dict(factor=4.0)), ("base", dict(factor=8.0)),
                                     ("bands", dict(factor=8.0, context=4096.0, low=1.0, high=4.0)),
                                     ("ramp", dict(factor=16.0, context=2048.0, low=1.0, high=32.0))])
def test_scaled_rotations(fg, kind, kw):
    for rot in (16, 64, 128):
        rotary = fg.Rotary(rot, "half", kind, **kw)
        x = torch.randn((9, 2 * 128), device="cuda")
        pos = [3, 4095, 4096, 100000, 1, 0, 77, 32767, 12345]
        _check_rotate(fg.fg_rotate(rotary, x, _i32(pos), 2, torch.empty_like(x)), x, pos, 2, rotary)


@pytest.mark.parametrize("off,ld", [(0, 264), (8, 272), (1, 261), (3, 264)])
@pytest.mark.parametrize("dt", ["f16", "f32"])
def test_strides_and_columns_of_wider_rows(fg, dt, off, ld):
    """Rows inside wider ones, aligned and not; what lies around them stays as it is."""
    n, heads, d = 11, 2, 64
    rotary = fg.Rotary(32, "pairs")
    wide = torch.randn((n, ld), device="cuda").to(DT[dt])
    before = wide.clone()
    pos = _i32(np.arange(n) * 37)
    x = wide[:, off:off + heads * d]
    out = torch.empty((n, heads * d), dtype=DT[dt], device="cuda")
    fg.fg_rotate(rotary, x, pos, heads, out)
    _check_rotate(out, x, pos.tolist(), heads, rotary)
    fg.fg_rotate(rotary, x, pos, heads)
    assert torch.equal(wide[:, off:off + heads * d], out)
    wide[:, off:off + heads * d] = before[:, off:off + heads * d]
    assert torch.equal(wide, before)


def test_out_may_be_other_columns_of_the_same_rows(fg):
    rotary = fg.Rotary(64)
    buf = torch.randn((5, 512), device="cuda").half()
    x, y = buf[:, :128], buf[:, 256:384]
    ref = fg.fg_rotate(rotary, x, _i32(range(5)), 2, torch.empty((5, 128), dtype=torch.float16, device="cuda"))
    fg.fg_rotate(rotary, x, _i32(range(5)), 2, y)
    assert torch.equal(y, ref)
    for bad in (buf[:, 64:192], buf[:, 8:136]):
        with pytest.raises(fg.FGError, match="FG_ERR_ARG"):
            fg.fg_rotate(rotary, x, _i32(range(5)), 2, bad)


def test_infinities_and_nan_stay_in_their_pairs(fg):
    rotary = fg.Rotary(64)
    x = torch.randn((3, 128), device="cuda").half()
    x[1, 5], x[1, 70], x[2, 127] = float("inf"), float("nan"), float("nan")
    clean = torch.nan_to_num(x, 0.0, 0.0, 0.0)
    pos = _i32([7, 8, 9])
    a, b = (fg.fg_rotate(rotary, t, pos, 2, torch.empty_like(t)) for t in (x, clean))
    hit = torch.zeros_like(x, dtype=torch.bool)
    hit[1, [5, 37, 70, 102]] = hit[2, [95, 127]] = True
    assert torch.equal(a[~hit], b[~hit]) and not torch.isfinite(a[hit]).any()


@pytest.mark.parametrize("layout", ["half", "pairs"])
def test_gradient_is_the_rotation_back(fg, layout):
    """y = R x is linear: its gradient R^T g, from the formula and from differences, is the rotation by -p."""
    rotary = fg.Rotary(48, layout, "ramp", factor=4.0, context=1024.0)
    gen = torch.Generator(device="cuda").manual_seed(5)
    x, g = (torch.randn((6, 2 * 64), generator=gen, device="cuda") for _ in range(2))
    pos = _i32([0, 1, 5, 100, 999, 20000])
    back = fg.fg_rotate(rotary, g, -pos, 2, torch.empty_like(g))
    _check_rotate(back, g, (-pos).tolist(), 2, rotary)
    ang = orot.angles(pos.tolist(), _turns(rotary))
    for j in (0, 3, 23, 24, 47, 50, 64, 127):    # differences in 64 bits: exact for a linear map, up to rounding
        e = np.zeros((6, 128))
        e[:, j] = 1.0
        col, _ = orot.rotate(e, pos.tolist(), 2, 48, layout, _turns(rotary), rotary.scale)
        want = (g.double().cpu().numpy() * col).sum(1)
        got = back[:, j].double().cpu().numpy()
        assert np.abs(got - want).max() <= 5 * 2.0 ** -24 * 2 * float(g.abs().max()) * rotary.scale
    assert ang.shape == (6, 24)


# ---- pages -----------------------------------------------------------------------------

class Cache:
    """An empty pool, and a table whose sequences have these lengths, in pages at random."""

    def __init__(self, fg, lens, n, heads, d, ps, dt, seed, missing=()):
        rng = np.random.default_rng(seed)
        need = [-(-x // ps) for x in lens]
        pages = sum(need) + 2
        perm = rng.permutation(pages)
        self.table = np.full((len(lens), max(need + [1]) + 1), -1)
        at = 0
        for i, k in enumerate(need):
            self.table[i, :k] = perm[at:at + k]
            at += k
        for i, j in missing:
            self.table[i, j] = -1
        self.lens, self.n, self.ps, self.heads, self.d, self.dt, self.pages = lens, n, ps, heads, d, dt, pages
        self.cu = np.concatenate(([0], np.cumsum(n)))
        self.tab = fg.PageTable(_i32(self.table), _i32(lens), _i32(np.ones(pages)), ps)
        self.pools = [fg.PagePool(pages, ps, heads, d, dt) for _ in range(2)]
        self.ntok = int(self.cu[-1])
        self.pos = np.concatenate([np.arange(x - k, x) for x, k in zip(lens, n)] + [np.zeros(0, int)])

    def arrays(self, which):
        p = self.pools[which]
        return [p.k_codes, p.k_mins, p.k_scales, p.v_codes, p.v_mins, p.v_scales]


def _bits(t):
    return t.view(torch.int16) if t.dtype == torch.float16 else t.view(torch.int32) if t.dtype == torch.float32 else t


def _same(a, b):
    return torch.equal(_bits(a), _bits(b))


ROTATED = [  # lens, rows, heads, group, d, ps, rot
    ([1], [1], 1, 1, 64, 16, 64), ([5, 0, 33], [5, 0, 1], 2, 2, 128, 16, 128), ([100, 17, 64, 300], [1, 1, 1, 1], 12, 1, 64, 16, 32),
    ([70, 300], [70, 113], 3, 3, 128, 64, 48), ([40, 41, 42], [16, 17, 31], 8, 4, 128, 32, 128), ([600], [600], 2, 1, 64, 128, 16)]


@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("lens,n,heads,group,d,ps,rot", ROTATED)
def test_append_rotated_is_rotate_then_append(fg, lens, n, heads, group, d, ps, rot, dt, layout):
    C = Cache(fg, lens, n, heads, d, ps, DT[dt], 3)
    rotary = fg.Rotary(rot, layout)
    gen = torch.Generator(device="cuda").manual_seed(1)

    def rows(h):
        return (1.5 * torch.randn((C.ntok, h * d), generator=gen, device="cuda")).to(DT[dt])

    q, k, v = rows(heads * group), rows(heads), rows(heads)
    q0, k0, v0 = q.clone(), k.clone(), v.clone()
    cu, pos = _i32(C.cu), _i32(C.pos)
    q1 = fg.fg_rotate(rotary, q, pos, heads * group, torch.empty_like(q))
    k1 = fg.fg_rotate(rotary, k, pos, heads, torch.empty_like(k))
    kr, vr, kr2, vr2, q2 = (torch.full_like(t, 3.0) for t in (k, v, k, v, q))
    fg.fg_paged_append(C.pools[0], C.tab, cu, k1, v, kr, vr)
    fg.fg_paged_append_rotated(C.pools[1], C.tab, cu, rotary, q, heads * group, q2, k, v, kr2, vr2)
    fg.fg_sync_status()
    for a, b in zip([q1, kr, vr] + C.arrays(0), [q2, kr2, vr2] + C.arrays(1)):
        assert _same(a, b)
    assert _same(q, q0) and _same(k, k0) and _same(v, v0)
    # without restored rows, and with everything in place
    for p in C.arrays(1):
        p.zero_()
    fg.fg_paged_append_rotated(C.pools[1], C.tab, cu, rotary, None, 0, None, k, v)
    for a, b in zip(C.arrays(0), C.arrays(1)):
        assert _same(a, b)
    fg.fg_paged_append_rotated(C.pools[1], C.tab, cu, rotary, q, heads * group, None, k, v, k, v)
    fg.fg_sync_status()
    for a, b in zip([q1, kr, vr] + C.arrays(0), [q, k, v] + C.arrays(1)):
        assert _same(a, b)


def test_append_rotated_of_wide_rows_and_rows_behind_the_last_sequence(fg):
    C = Cache(fg, [30, 50], [7, 20], 2, 64, 16, torch.float16, 4)
    rotary = fg.Rotary(64)
    extra = 5
    buf = torch.randn((C.ntok + extra, 6 * 64 + 16), device="cuda").half()   # q (2 heads) | k | v side by side
    before = buf.clone()
    q, k, v = buf[:, :128], buf[:, 128:256], buf[:, 256:384]
    cu, pos = _i32(C.cu), _i32(list(C.pos) + [0] * extra)
    k1 = fg.fg_rotate(rotary, k, pos, 2, torch.empty((C.ntok + extra, 128), dtype=torch.float16, device="cuda"))
    q1 = fg.fg_rotate(rotary, q, pos, 2, torch.empty_like(k1))
    fg.fg_paged_append(C.pools[0], C.tab, cu, k1, v.contiguous())
    fg.fg_paged_append_rotated(C.pools[1], C.tab, cu, rotary, q, 2, None, k, v)
    fg.fg_sync_status()
    for a, b in zip(C.arrays(0), C.arrays(1)):
        assert _same(a, b)
    assert _same(q[:C.ntok].contiguous(), q1[:C.ntok]) and _same(buf[C.ntok:], before[C.ntok:]) and _same(buf[:, 128:], before[:, 128:])


def test_append_rotated_reports_and_leaves_out(fg):
    """A missing page: its rows are not stored, their queries are rotated; a row before the first token is left out."""
    C = Cache(fg, [40, 3], [24, 5], 1, 64, 16, torch.float16, 5, missing=[(0, 1)])
    rotary = fg.Rotary(64)
    k, v, q = (torch.randn((C.ntok, 64), device="cuda").half() for _ in range(3))
    kr, vr, qo = (torch.full_like(k, 9.0) for _ in range(3))
    fg.fg_paged_append_rotated(C.pools[0], C.tab, _i32(C.cu), rotary, q, 1, qo, k, v, kr, vr)
    with pytest.raises(fg.FGError, match="FG_ERR_ARG"):
        fg.fg_sync_status()
    gone = torch.tensor([16 <= p < 32 for p in C.pos[:24]] + [True, True, False, False, False])
    assert (kr[gone] == 9.0).all() and (vr[gone] == 9.0).all() and not (kr[~gone] == 9.0).all(1).any()
    want = fg.fg_rotate(rotary, q, _i32(C.pos), 1, torch.empty_like(q))
    assert _same(qo[:24], want[:24]) and _same(qo[26:], want[26:]) and (qo[24:26] == 9.0).all()


@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("lens,n,heads,d,ps", [([1], [1], 1, 64, 16), ([100, 0, 37], [100, 0, 12], 3, 64, 16), ([300, 65, 64, 1], [300, 33, 64, 0], 2, 128, 64),
                                               ([1000], [1000], 5, 128, 256), ([40] * 70, [3] * 70, 2, 64, 32)])
def test_read(fg, lens, n, heads, d, ps, dt):
    C = Cache(fg, lens, n, heads, d, ps, DT[dt], 6)
    rng = np.random.default_rng(7)
    np_dt = np.float16 if dt == "f16" else np.float32
    q = [codec.quantize_g64((rng.normal(size=(C.pages, heads, ps, d)) * 10.0 ** rng.integers(-3, 3, (C.pages, heads, ps, 1))).astype(np_dt))
         for _ in range(2)]
    pool = fg.PagePool.of(*[torch.as_tensor(a, device="cuda") for x in q for a in x], DT[dt])
    wide = torch.full((2, C.ntok + 2, heads * d + 8), 5.0, dtype=DT[dt], device="cuda")
    k, v = wide[0, :, :heads * d], wide[1, :, :heads * d]
    fg.fg_paged_read(pool, C.tab, _i32(C.cu), k, v)
    fg.fg_sync_status()
    ref = [codec.dequant_g64(*x, np_dt) for x in q]
    seq = np.repeat(np.arange(len(lens)), n)

    def want(which, pos):
        page, slot = C.table[seq, pos // ps], pos % ps
        return ref[which][page, :, slot].reshape(len(pos), -1)

    for which, t in enumerate((k, v)):
        assert np.array_equal(t[:C.ntok].cpu().numpy().view(np.uint16 if dt == "f16" else np.uint32),
                              want(which, C.pos).view(np.uint16 if dt == "f16" else np.uint32))
    assert (wide[:, C.ntok:] == 5.0).all() and (wide[:, :, heads * d:] == 5.0).all()
    # from a position on, one of the two
    start = np.array([max(0, (x - m) // 2) for x, m in zip(lens, n)])
    out = torch.full_like(wide, 5.0)[0, :, :heads * d]
    fg.fg_paged_read(pool, C.tab, _i32(C.cu), v=out, start=_i32(start))
    fg.fg_sync_status()
    pos = np.concatenate([np.arange(s, s + m) for s, m in zip(start, n)])
    assert np.array_equal(out[:C.ntok].cpu().numpy(), want(1, pos))


def test_read_leaves_what_is_not_there(fg):
    C = Cache(fg, [40, 20], [10, 10], 1, 64, 16, torch.float16, 8, missing=[(0, 1)])
    pool = C.pools[0]
    pool.k_mins.fill_(1.0)
    k, v = (torch.full((20, 64), 9.0, dtype=torch.float16, device="cuda") for _ in range(2))
    fg.fg_paged_read(pool, C.tab, _i32(C.cu), k, v, start=_i32([10, 0]))      # positions 10 .. 19; the page of 16 .. 31 is missing
    with pytest.raises(fg.FGError, match="FG_ERR_CAPACITY"):
        fg.fg_sync_status()
    assert (k[:6] == 1.0).all() and (k[6:10] == 9.0).all() and (k[10:] == 1.0).all()
    for start in ([35, 0], [-1, 0], [2 ** 31 - 1, 0], [30, 15]):
        k.fill_(9.0)
        fg.fg_paged_read(pool, C.tab, _i32(C.cu), k, start=_i32(start))
        with pytest.raises(fg.FGError, match="FG_ERR_ARG"):
            fg.fg_sync_status()
    assert (k[:2] == 9.0).all()          # 30 and 31: no page
    assert (k[2:10] == 1.0).all() and (k[10:15] == 1.0).all() and (k[15:] == 9.0).all()


def test_calls_on_another_stream_and_in_a_graph(fg):
    C = Cache(fg, [40, 80], [1, 1], 4, 128, 16, torch.float16, 9)
    rotary = fg.Rotary(128)
    q, k, v = (torch.randn((2, 4 * 128), device="cuda").half() for _ in range(3))
    qo, kb, vb = (torch.zeros_like(q) for _ in range(3))
    cu = _i32(C.cu)

    def step():
        fg.fg_paged_append_rotated(C.pools[0], C.tab, cu, rotary, q, 4, qo, k, v)
        fg.fg_paged_read(C.pools[0], C.tab, cu, kb, vb)
        fg.fg_rotate(rotary, qo, _i32_pos, 4)

    _i32_pos = _i32([-39, -79])
    step()
    torch.cuda.synchronize()
    first = [t.clone() for t in (qo, kb, vb)]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        step()
    st.synchronize()
    assert all(_same(a, b) for a, b in zip(first, (qo, kb, vb)))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for scale in (1.0, 0.5):
        q.mul_(scale), k.mul_(scale), v.mul_(scale)
        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in (qo, kb, vb)]
        for t in (qo, kb, vb):
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(_same(a, b) for a, b in zip(want, (qo, kb, vb)))
    # rotated there and back: q again, but for two roundings
    assert float((qo - q).abs().max()) <= 2.0 ** -10 * 2 * float(q.abs().max())
