"""The paged 4-bit KV cache, measured: appending ragged chunks, attention of
chunks over pages (single tokens, windows with sinks, grouped heads), forking
and growing sequences, freeing them and compacting the pool.

`own = False` runs each operator in elementary torch operations, `own = True`
through the library's entry points.  A cache is [pages][heads][page_size]
[head_dim] in groups of 64 (codes two to a byte, a float32 minimum and scale
per group); row i of the page table lists the pages of sequence i.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
DT = {"f16": torch.float16, "f32": torch.float32}


# ---- cases -------------------------------------------------------------------

def listed():
    return [
        # one step of four short sequences at the 125M shape: launch latency counts
        dict(name="attn step small", op="attn", dt="f16", b=4, qh=12, kvh=12, d=64, ps=16, lo=100, hi=300, clo=1, chi=1,
             window=0, sinks=0),
        # one step of a full block at the 6.7B shape, lengths around its 544 tokens
        dict(name="attn step block", op="attn", dt="f16", b=64, qh=32, kvh=32, d=128, ps=64, lo=300, hi=900, clo=1, chi=1,
             window=0, sinks=0),
        # one step over long contexts, eight query heads to a K/V head
        dict(name="attn step long", op="attn", dt="f16", b=8, qh=64, kvh=8, d=128, ps=128, lo=30001, hi=65000, clo=1, chi=1,
             window=0, sinks=0),
        # a chunk of a long prompt over the part that is already cached (6.7B heads)
        dict(name="attn chunk", op="attn", dt="f16", b=1, qh=32, kvh=32, d=128, ps=64, lo=16384, hi=16384, clo=2048, chi=2048,
             window=0, sinks=0),
        # a mixed batch under continuous batching: single tokens beside chunks, a sliding window with four sinks
        dict(name="attn mixed window", op="attn", dt="f16", b=12, qh=32, kvh=8, d=128, ps=32, lo=700, hi=6011, clo=1, chi=601,
             window=1000, sinks=4),
        # fp32 activations (the exactness check of the small shapes)
        dict(name="attn f32", op="attn", dt="f32", b=3, qh=12, kvh=12, d=64, ps=16, lo=300, hi=777, clo=5, chi=67,
             window=0, sinks=0),
        # the new tokens of a decode step
        dict(name="append step", op="append", dt="f16", b=64, kvh=32, d=128, ps=64, lo=300, hi=900, clo=1, chi=1, restored=False),
        # ragged prompts, with the restored rows that a dense prefill attention reads
        dict(name="append prompts", op="append", dt="f16", b=48, kvh=32, d=128, ps=64, lo=300, hi=700, clo=300, chi=700,
             restored=True),
        # parallel sampling: children of a few prompts, then one token of growth
        dict(name="fork small", op="fork", dt="f16", l=2, b=3, n=6, kvh=12, d=64, ps=16, lo=40, hi=200, grow=1, spare=24),
        # the same for a block, over several layers
        dict(name="fork block", op="fork", dt="f16", l=8, b=16, n=48, kvh=32, d=128, ps=64, lo=300, hi=900, grow=1, spare=160),
        # a few sequences end, the pool is compacted
        dict(name="recycle small", op="recycle", dt="f16", l=2, b=8, n=3, kvh=12, d=64, ps=16, lo=40, hi=200),
        # half of a block's sequences end
        dict(name="recycle block", op="recycle", dt="f16", l=4, b=64, n=32, kvh=32, d=128, ps=64, lo=300, hi=900),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "append", "fork", "recycle"])
    d = rng.choice([64, 128])
    ps = rng.choice([16, 32, 64, 128])
    dt = "f16" if rng.random() < 0.85 else "f32"
    if op == "attn":
        kvh = _log(rng, 1, 32)
        r = rng.choice([1, 1, 1, 2, 3, 4, 8])
        step = rng.random() < 0.5
        if dt == "f32":
            b, hi, chi = _log(rng, 1, 6), _log(rng, 64, 900), 1 if step else _log(rng, 2, 90)
        elif step:
            b, chi = _log(rng, 1, 64), 1
            hi = _log(rng, 64, max(65, min(65000, (1 << 22) // (b * kvh))))
        else:
            b, chi = _log(rng, 1, 12), _log(rng, 2, 1500)
            hi = max(chi, _log(rng, 64, 16000))
            while b * chi * hi * kvh * r > 400_000_000:
                b, chi, hi = max(1, b // 2), max(2, chi * 3 // 4), max(65, hi * 3 // 4)
            hi = max(hi, chi)
        win = rng.random() < 0.35
        return dict(op=op, dt=dt, b=b, qh=kvh * r, kvh=kvh, d=d, ps=ps, lo=max(1, hi // rng.choice([1, 2, 3])), hi=hi,
                    clo=max(1, chi // rng.choice([1, 3, 50])), chi=chi,
                    window=_log(rng, 16, 3000) if win else 0, sinks=rng.choice([0, 1, 4, 50]) if win else 0)
    kvh = _log(rng, 1, 32)
    if op == "append":
        b = _log(rng, 1, 64)
        chi = 1 if rng.random() < 0.4 else _log(rng, 2, 600)
        hi = max(chi, _log(rng, 20, 900))
        return dict(op=op, dt=dt, b=b, kvh=kvh, d=d, ps=ps, lo=max(1, hi // 2), hi=hi, clo=max(1, chi // 3), chi=chi,
                    restored=rng.random() < 0.5)
    hi = _log(rng, 20, 900)
    b = _log(rng, 2, 40)
    l = _log(rng, 1, 4)
    if op == "fork":
        n = _log(rng, 1, 40)
        grow = _log(rng, 1, 40)
        return dict(op=op, dt=dt, l=l, b=b, n=n, kvh=kvh, d=d, ps=ps, lo=max(1, hi // 3), hi=hi, grow=grow,
                    spare=2 * n + (b + n) * (grow // ps + 1))
    return dict(op=op, dt=dt, l=l, b=b, n=max(1, b * rng.choice([1, 2, 3]) // 5), kvh=kvh, d=d, ps=ps, lo=max(1, hi // 3), hi=hi)


# ---- inputs ------------------------------------------------------------------

def _spread(b, lo, hi, phase):
    """b sizes between lo and hi, the same for every seed (golden-ratio steps)."""
    f = (np.arange(b) * 0.6180339887498949 + phase) % 1.0
    return np.floor(lo + f * (hi - lo + 0.999)).astype(np.int64)


def _sizes(case):
    """Tokens of each sequence, and of its chunk."""
    lens = _spread(case["b"], case["lo"], case["hi"], 0.37)
    n = np.minimum(lens, _spread(case["b"], case["clo"], case["chi"], 0.83))
    return lens, n


def _up(x, ps):
    return -(-x // ps)


def _ints(x):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=torch.int32, device=DEV)


def _quantize(x):
    """Codes, minima and scales of x [..., d] in groups of 64 (fp32, the literal order of operations)."""
    g = x.float().reshape(x.shape[:-1] + (x.shape[-1] // 64, 64))
    mn = g.amin(-1)
    r = g.amax(-1) - mn
    q = (((g - mn[..., None]) / r[..., None]) * 15.0).round().clamp(0.0, 15.0).nan_to_num(0.0).to(torch.uint8)
    q = q.reshape(x.shape)
    return q[..., 0::2] | (q[..., 1::2] << 4), mn, r / 15.0


def _restore(codes, mn, sc):
    """The values that codes stand for, in 32 bits."""
    q = torch.stack((codes & 15, codes >> 4), -1).reshape(codes.shape[:-1] + (codes.shape[-1] * 2,)).float()
    g = q.reshape(q.shape[:-1] + (q.shape[-1] // 64, 64))
    return (g * sc[..., None] + mn[..., None]).reshape(q.shape)


def _pool(lead, case, gen, dt):
    """Pages of quantized rows: K or V values of about unit size, some dims larger than others."""
    d = case["d"]
    shape = tuple(lead) + (case["kvh"], case["ps"], d)
    size = 0.5 + torch.rand((case["kvh"], 1, d), generator=gen, device=DEV)
    x = (torch.randn(shape, generator=gen, device=DEV, dtype=torch.float16) * size.half()).to(dt)
    return _quantize(x)


def _table(pages, lens, rows, ps, gen, spare):
    """A table of `rows` rows whose first len(lens) hold those lengths, in pages drawn at random."""
    need = _up(lens, ps)
    stride = int(need.max()) + spare
    perm = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
    table = torch.full((rows, stride), -1, dtype=torch.int32, device=DEV)
    start = _ints(np.concatenate(([0], np.cumsum(need)))[:-1]).long()
    col = torch.arange(stride, device=DEV)
    on = col[None] < _ints(need)[:, None]
    at = (start[:, None] + col[None]).clamp(max=pages - 1)
    table[: len(lens)] = torch.where(on, perm[at], table[: len(lens)])
    refs = torch.zeros(pages, dtype=torch.int32, device=DEV)
    refs[perm[: int(need.sum())].long()] = 1
    ln = torch.zeros(rows, dtype=torch.int32, device=DEV)
    ln[: len(lens)] = _ints(lens)
    return table, ln, refs


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    dt, ps, d = DT[case["dt"]], case["ps"], case["d"]
    s = dict(case=case, dt=dt)
    if case["op"] in ("attn", "append"):
        lens, n = _sizes(case)
        pages = int(_up(lens, ps).sum()) + 3
        s["table"], s["lens"], s["refs"] = _table(pages, lens, case["b"], ps, gen, 1)
        cu = np.concatenate(([0], np.cumsum(n)))
        s["cu"], s["ntok"], s["max_q"] = _ints(cu), int(cu[-1]), int(n.max())
        s["max_kv"] = int(lens.max())
        if case["op"] == "attn":
            s["k"], s["v"] = _pool((pages,), case, gen, dt), _pool((pages,), case, gen, dt)
            q = torch.randn((s["ntok"], case["qh"] * d), generator=gen, device=DEV)
            s["q"] = (1.3 * q).to(dt)
            s["out"] = torch.zeros_like(s["q"])
            return s
        shape = (pages, case["kvh"], ps)
        for name in ("k", "v"):
            s[name] = (torch.zeros(shape + (d // 2,), dtype=torch.uint8, device=DEV),
                       torch.zeros(shape + (d // 64,), device=DEV), torch.zeros(shape + (d // 64,), device=DEV))
            x = torch.randn((s["ntok"], case["kvh"] * d), generator=gen, device=DEV)
            s[name + "_new"] = (1.3 * x).to(dt)
            s[name + "_out"] = torch.zeros_like(s[name + "_new"]) if case["restored"] else None
        return s
    lens = _spread(case["b"], case["lo"], case["hi"], 0.37)
    fork = case["op"] == "fork"
    rows = case["b"] + (case["n"] if fork else 0)
    pages = int(_up(lens, ps).sum()) + (case["spare"] if fork else 5)
    table, ln, refs = _table(pages, lens, rows, ps, gen, 1 + (_up(case["grow"], ps) if fork else 0))
    # the bookkeeping lies in one buffer, so that a pass can begin from the same state with one copy
    s["meta0"] = torch.cat((table.reshape(-1), ln, refs))
    s["meta"] = s["meta0"].clone()
    a, b = table.numel(), table.numel() + rows
    s["table"], s["lens"], s["refs"] = s["meta"][:a].view(table.shape), s["meta"][a:b], s["meta"][b:]
    s["k"], s["v"] = _pool((case["l"], pages), case, gen, dt), _pool((case["l"], pages), case, gen, dt)
    if fork:
        s["src"] = torch.randint(case["b"], (case["n"],), generator=gen, device=DEV, dtype=torch.int32)
        s["dst"] = torch.randperm(case["n"], generator=gen, device=DEV).to(torch.int32) + case["b"]
        s["cu"] = torch.arange(rows + 1, device=DEV, dtype=torch.int32) * case["grow"]
    else:
        s["rows"] = torch.randperm(case["b"], generator=gen, device=DEV)[: case["n"]].to(torch.int32)
    return s


# ---- one pass ------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if own:
        return {"attn": _own_attn, "append": _own_append, "fork": _own_fork, "recycle": _own_recycle}[op](s)
    return {"attn": _attn, "append": _append, "fork": _fork, "recycle": _recycle}[op](s)


def _rows_of(s):
    """Sequence and position of every row of the ragged batch."""
    cu = s["cu"].long()
    row = torch.arange(s["ntok"], device=DEV)
    seq = torch.searchsorted(cu, row, right=True) - 1
    return seq, s["lens"].long()[seq] - (cu[seq + 1] - row), row - cu[seq]


def _attn(s):
    c = s["case"]
    b, qh, kvh, d, ps = c["b"], c["qh"], c["kvh"], c["d"], c["ps"]
    r = qh // kvh
    lens = s["lens"].long()
    npage = _up(s["max_kv"], ps)
    pages = s["table"][:, :npage].long().clamp(min=0)

    def cached(x):   # [b][kvh][tokens][d] in 32 bits
        v = _restore(*[t[pages] for t in x])
        return v.permute(0, 2, 1, 3, 4).reshape(b, kvh, npage * ps, d)

    seq, pos, at = _rows_of(s)
    mq = s["max_q"]
    q = torch.zeros((b, mq, qh * d), device=DEV)
    q[seq, at] = s["q"].float()
    q = q.view(b, mq, kvh, r, d).permute(0, 2, 3, 1, 4).reshape(b, kvh, r * mq, d)
    w = torch.matmul(q, cached(s["k"]).transpose(2, 3)).view(b, kvh, r, mq, npage * ps)
    p = (lens - (s["cu"][1:] - s["cu"][:-1]).long())[:, None] + torch.arange(mq, device=DEV)[None]   # [b][mq]
    key = torch.arange(npage * ps, device=DEV)
    see = key <= p[..., None]
    if c["window"]:
        see &= (key > p[..., None] - c["window"]) | (key < c["sinks"])
    w = w.mul_(1.0 / math.sqrt(d)).masked_fill_(~see[:, None, None], float("-inf"))
    w = w.sub_(w.amax(-1, keepdim=True)).exp_()
    w = w.div_(w.sum(-1, keepdim=True)).view(b, kvh, r * mq, npage * ps)
    v = cached(s["v"]).masked_fill_((key >= lens[:, None])[:, None, :, None], 0.0)
    o = torch.matmul(w, v).view(b, kvh, r, mq, d).permute(0, 3, 1, 2, 4).reshape(b, mq, qh * d)
    return o[seq, at].to(s["dt"])


def _append(s):
    c = s["case"]
    seq, pos, _ = _rows_of(s)
    page, slot = s["table"][seq, pos // c["ps"]].long(), pos % c["ps"]
    got = []

    def store(name):
        x = s[name + "_new"].view(s["ntok"], c["kvh"], c["d"])
        new = _quantize(x)
        s[name][0][page, :, slot], s[name][1][page, :, slot], s[name][2][page, :, slot] = new
        got.extend(s[name])
        if c["restored"]:
            got.append(_restore(*new).to(s["dt"]).view(s["ntok"], -1))

    store("k")
    store("v")
    return got


def _free_pages(refs):
    """Page ids with the free ones first, ascending, and how many are free."""
    return torch.argsort((refs != 0).to(torch.int8), stable=True), (refs == 0).sum()


def _copy_pages(s, src, dst):
    def move(x):
        x[:, dst] = x[:, src]

    list(map(move, s["k"] + s["v"]))


def _fork(s):
    c, ps = s["case"], s["case"]["ps"]
    s["meta"].copy_(s["meta0"])
    table, lens, refs = s["table"].clone(), s["lens"].long(), s["refs"].clone()
    src, dst = s["src"].long(), s["dst"].long()
    col = torch.arange(table.shape[1], device=DEV)
    full, part = lens[src] // ps, lens[src] % ps > 0
    order, nfree = _free_pages(refs)
    rank = part.cumsum(0) - 1
    old = table[src, full].long().clamp(min=0)
    fresh = torch.where(part, order[rank.clamp(min=0)], old)
    _copy_pages(s, old[part], fresh[part])
    shared = col[None] < full[:, None]
    refs.index_add_(0, table[src].long().clamp(min=0).reshape(-1), shared.reshape(-1).to(torch.int32))
    refs[fresh[part]] = 1
    table[dst] = torch.where(shared, table[src], torch.where((col[None] == full[:, None]) & part[:, None], fresh[:, None].int(), table[dst]))
    lens = lens.index_copy(0, dst, lens[src])
    # growth
    n = (s["cu"][1:] - s["cu"][:-1]).long()
    have, want = _up(lens, ps), _up(lens + n, ps)
    new = (col[None] >= have[:, None]) & (col[None] < want[:, None])
    order, nfree = _free_pages(refs)
    rank = new.reshape(-1).cumsum(0).view(new.shape) - 1
    page = torch.where(rank < nfree, order[rank.clamp(min=0, max=refs.numel() - 1)], -1)
    table = torch.where(new, page.int(), table)
    refs[page[new & (page >= 0)]] = 1
    return [table, (lens + n).int(), refs, *s["k"], *s["v"]]


def _recycle(s):
    ps = s["case"]["ps"]
    s["meta"].copy_(s["meta0"])
    table, lens, refs, rows = s["table"].clone(), s["lens"].clone(), s["refs"].clone(), s["rows"].long()
    col = torch.arange(table.shape[1], device=DEV)
    held = col[None] < _up(lens[rows].long(), ps)[:, None]
    refs.index_add_(0, table[rows].long().clamp(min=0).reshape(-1), -held.reshape(-1).to(torch.int32))
    table[rows] = torch.where(held, -1, table[rows])
    lens[rows] = 0
    live = refs > 0
    idx = torch.arange(refs.numel(), device=DEV)
    nlive = live.sum()
    src, dst = idx[live & (idx >= nlive)], idx[~live & (idx < nlive)]
    _copy_pages(s, src, dst)
    to = idx.clone()
    to[src] = dst
    held = col[None] < _up(lens.long(), ps)[:, None]
    table = torch.where(held, to[table.long().clamp(min=0)].int(), table)
    new = torch.where(idx < nlive, refs, 0)
    new[dst] = refs[src]
    return [table, lens, new, *s["k"], *s["v"]]


# ---- the same through the library --------------------------------------------------

def _handle(s):
    """What a user's program keeps between calls: the pools' and the table's handles and a workspace."""
    if "handle" not in s:
        import int4_group_quantized_gb300 as fg
        c = s["case"]
        layers = [(s["k"], s["v"])] if c["op"] in ("attn", "append") else [
            ([t[i] for t in s["k"]], [t[i] for t in s["v"]]) for i in range(c["l"])]
        pools = [fg.PagePool.of(k[0], k[1], k[2], v[0], v[1], v[2], s["dt"]) for k, v in layers]
        tab = fg.PageTable(s["table"], s["lens"], s["refs"], c["ps"])
        need = 0
        if c["op"] == "attn":
            need = fg.fg_paged_attention_workspace_bytes(pools[0], tab, c["qh"], s["ntok"], s["max_q"])
        elif c["op"] != "append":
            need = fg.fg_pages_workspace_bytes(tab, c.get("n", 0))
        s["handle"] = fg, pools[0], fg.PagePools(pools), tab, fg.workspace(need)
    return s["handle"]


def _own_attn(s):
    fg, pool, _, tab, ws = _handle(s)
    c = s["case"]
    fg.fg_paged_attention(pool, tab, s["cu"], s["q"], c["qh"], s["out"], s["max_q"], window=c["window"], sinks=c["sinks"], ws=ws)
    return s["out"]


def _own_append(s):
    fg, pool, _, tab, _ = _handle(s)
    fg.fg_paged_append(pool, tab, s["cu"], s["k_new"], s["v_new"], s["k_out"], s["v_out"])
    if s["case"]["restored"]:
        return [*s["k"], s["k_out"], *s["v"], s["v_out"]]
    return [*s["k"], *s["v"]]


def _own_fork(s):
    fg, _, pools, tab, ws = _handle(s)
    s["meta"].copy_(s["meta0"])
    fg.fg_pages_fork(tab, pools, s["src"], s["dst"], ws)
    fg.fg_pages_reserve(tab, s["cu"], ws)
    return [s["table"], s["lens"], s["refs"], *s["k"], *s["v"]]


def _own_recycle(s):
    fg, _, pools, tab, ws = _handle(s)
    s["meta"].copy_(s["meta0"])
    fg.fg_pages_free(tab, s["rows"])
    fg.fg_pages_compact(tab, pools, ws)
    return [s["table"], s["lens"], s["refs"], *s["k"], *s["v"]]


# ---- what a pass cannot do without ----------------------------------------------------

def work(case):
    ps, d, e = case["ps"], case["d"], 2 if case["dt"] == "f16" else 4
    tok = case["kvh"] * d * 0.625   # bytes of one token's K (or V) row
    if case["op"] in ("attn", "append"):
        lens, n = _sizes(case)
        rows = float(n.sum())
        if case["op"] == "append":
            return {"bytes": 2 * rows * (case["kvh"] * d * e * (2 if case["restored"] else 1) + tok),
                    "flops": 10.0 * rows * case["kvh"] * d}
        pairs = keys = 0.0
        w, k = case["window"], case["sinks"]
        for length, m in zip(lens.tolist(), n.tolist()):
            p = np.arange(length - m, length, dtype=np.float64)
            if w:
                recent = np.minimum(p + 1, w)
                pairs += float((recent + np.minimum(k, p + 1 - recent)).sum())
                first = max(0, length - m - w + 1)
                keys += length - first + min(k, first)
            else:
                pairs += float((p + 1).sum())
                keys += length
        return {"bytes": 2 * keys * tok + 2 * rows * case["qh"] * d * e, "flops": 4.0 * d * case["qh"] * pairs}
    lens = _spread(case["b"], case["lo"], case["hi"], 0.37)
    need = _up(lens, ps)
    page = 2 * ps * tok * case["l"]
    if case["op"] == "fork":
        share = float((lens % ps > 0).mean())
        return {"bytes": 2 * case["n"] * share * page + 8.0 * float(need.mean()) * case["n"], "flops": 0.0}
    pages = float(need.sum()) + 5
    live = float(need.sum()) * (1 - case["n"] / case["b"])
    return {"bytes": 2 * live * (1 - live / pages) * page + 8.0 * pages, "flops": 0.0}


# ---- 64 bits -----------------------------------------------------------------------

def exact(case, seed):
    if case["op"] in ("fork", "recycle"):
        return None   # whole pages are copied: nothing is computed
    s = prepare(case, seed)
    d, ps, kvh = case["d"], case["ps"], case["kvh"]
    lens, cu = s["lens"].tolist(), s["cu"].tolist()
    if case["op"] == "append":
        got = []
        for name in ("k", "v"):
            codes, mn, sc = s[name]
            x = s[name + "_new"].double().view(s["ntok"], kvh, d // 64, 64)
            lo, hi = x.min(-1).values, x.max(-1).values
            mins, scales = mn.double(), sc.double()
            for i, length in enumerate(lens):
                n = cu[i + 1] - cu[i]
                p = torch.arange(length - n, length, device=DEV)
                page = s["table"][i, p // ps].long()
                mins[page, :, p % ps] = lo[cu[i]:cu[i + 1]]
                scales[page, :, p % ps] = (hi - lo)[cu[i]:cu[i + 1]] / 15
            got += [None, mins, scales]
            if case["restored"]:
                # the codes are fixed by fp32 operations: those of the row, then their values exactly
                f = s[name + "_new"].float().view(x.shape)
                u = (f - lo.float()[..., None]) / (hi - lo).float()[..., None] * 15
                q = torch.clamp(torch.round(u), 0, 15).double()
                got.append((q * ((hi - lo).float() / 15).double()[..., None] + lo[..., None]).view(s["ntok"], -1))
        return got
    qh = case["qh"]
    r = qh // kvh
    out = torch.zeros((s["ntok"], kvh, r, d), dtype=torch.float64, device=DEV)
    q = s["q"].double().view(s["ntok"], kvh, r, d)

    def rows_of(x, i, h, lo, hi):
        at = torch.arange(lo, hi, device=DEV)
        page = s["table"][i, at // ps].long()
        c, mn, sc = (t[page, h, at % ps] for t in x)
        v = torch.empty((hi - lo, d), dtype=torch.float64, device=DEV)
        v[:, 0::2], v[:, 1::2] = (c & 15).double(), (c >> 4).double()
        return (v.view(-1, d // 64, 64) * sc.double()[..., None] + mn.double()[..., None]).view(-1, d)

    for i, length in enumerate(lens):
        a, e = cu[i], cu[i + 1]
        p = torch.arange(length - (e - a), length, device=DEV)
        for h in range(kvh):
            k, v = rows_of(s["k"], i, h, 0, length), rows_of(s["v"], i, h, 0, length)
            j = torch.arange(length, device=DEV)
            hidden = j[None] > p[:, None]
            if case["window"]:
                hidden |= (j[None] <= p[:, None] - case["window"]) & (j[None] >= case["sinks"])
            x = torch.einsum("trd,jd->trj", q[a:e, h], k) / math.sqrt(d)
            x = torch.softmax(x.masked_fill(hidden[:, None], -math.inf), -1)
            out[a:e, h] = torch.einsum("trj,jd->trd", x, v)
    return out.view(s["ntok"], -1)
