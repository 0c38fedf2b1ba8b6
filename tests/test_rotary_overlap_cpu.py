"""fg_paged_append_rotated refuses rows that one block writes while another reads them: rotated queries over keys, values or
restored rows, and restored rows over queries.  (What it accepts runs in test_rotary_overlap_gpu.py: pointers here name no
memory.)"""
import ctypes

import pytest

P = 1 << 20
H, QH, D, N = 2, 4, 64, 8
ROW, QROW = H * D, QH * D                                    # elements


@pytest.fixture(scope="module")
def fg():
    import __graft_entry__
    __graft_entry__.build()
    import int4_group_quantized_gb300 as fg
    return fg


def _append(fg, q, qo, k, v, kr=None, vr=None, ldq=QROW, ldqo=QROW, ld=ROW, ldr=ROW, dtype=0):
    pool = fg.fg_page_pool(P, P, P, P, P, P, 8, 16, H, D, dtype)
    tab = fg.fg_page_table(P, P, P, 3, 4, 8, 16)
    rot = fg.fg_rotary(P, 64, 0, 1.0)
    return fg.lib.fg_paged_append_rotated(ctypes.byref(pool), ctypes.byref(tab), P, ctypes.byref(rot), q, ldq, QH, qo, ldqo, k, v, ld, N, kr, vr, ldr, None)


@pytest.mark.parametrize("dtype", [0, 1])
def test_rows_that_overlap_are_refused(fg, dtype):
    e = 2 if dtype == 0 else 4
    q, k, v, kr, vr, qo = (P + i * (1 << 20) for i in range(6))
    far = dict(q=q, qo=qo, k=k, v=v, kr=kr, vr=vr, dtype=dtype)
    for name in ("k", "v", "kr", "vr"):
        for off in (0, 16 * e, (N - 1) * ROW * e, -(N - 1) * QROW * e):
            assert _append(fg, **(far | dict(qo=far[name] + off))) == 1, (name, off)
        assert _append(fg, **(far | dict(qo=far[name], q=far[name]))) == 1, name   # in place
    for name in ("kr", "vr"):
        assert _append(fg, **(far | {name: q})) == 1 and _append(fg, **(far | {name: q + (N - 1) * QROW * e})) == 1, name
    # rows of one buffer, side by side, one column too near
    wide = QROW + 2 * ROW
    near = dict(q=P, ldq=wide, qo=P, ldqo=wide, ld=wide, dtype=dtype)
    assert _append(fg, k=P + (QROW - 8) * e, v=P + (QROW + ROW) * e, **near) == 1
    assert _append(fg, k=P + QROW * e, v=P + (QROW + ROW + 8) * e, **near) == 1   # the last heads' values reach the next row's queries
