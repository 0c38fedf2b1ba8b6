"""fg_paged_append_rotated on rows of one buffer: queries rotated in place beside the keys and values that it reads, restored
rows back over these."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
@pytest.mark.parametrize("n", [1, 3, 700])
def test_rows_of_one_buffer(n, dtype):
    import int4_group_quantized_gb300 as fg
    heads, qh, d, ps = 2, 6, 128, 16
    pages = -(-n // ps)
    gen = torch.Generator(device="cuda").manual_seed(3)
    rows = torch.randn((n, (qh + 2 * heads) * d + 8), generator=gen, device="cuda").to(dtype)
    rotary = fg.Rotary(64, "pairs")
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    got = []
    for apart in (True, False):
        pool = fg.PagePool(pages, ps, heads, d, dtype)
        tab = fg.PageTable(torch.arange(pages, dtype=torch.int32, device="cuda")[None], cu[1:], torch.ones(pages, dtype=torch.int32, device="cuda"), ps)
        x = rows.clone()
        q, k, v = x[:, :qh * d], x[:, qh * d:(qh + heads) * d], x[:, (qh + heads) * d:(qh + 2 * heads) * d]
        if apart:
            q, k, v = (t.contiguous() for t in (q, k, v))
            out, kr, vr = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        else:
            out, kr, vr = q, k, v
        fg.fg_paged_append_rotated(pool, tab, cu, rotary, q, qh, out, k, v, kr, vr)
        fg.fg_sync_status()
        if not apart:
            assert torch.equal(x[:, -8:], rows[:, -8:])
        got.append([t.clone() for t in (out, kr, vr, pool.k_codes, pool.k_mins, pool.k_scales, pool.v_codes, pool.v_mins, pool.v_scales)])
    assert all(torch.equal(a, b) for a, b in zip(*got))


def test_python_refuses_what_overlaps():
    import int4_group_quantized_gb300 as fg
    heads, d, n = 2, 64, 5
    pool, tab = fg.PagePool(2, 16, heads, d), fg.PageTable.empty(1, 2, 2, 16)
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    q, k, v = (torch.zeros((n, heads * d), dtype=torch.float16, device="cuda") for _ in range(3))
    for out in (k, v):
        with pytest.raises(fg.FGError, match="FG_ERR_ARG"):
            fg.fg_paged_append_rotated(pool, tab, cu, fg.Rotary(d), q, heads, out, k, v)
