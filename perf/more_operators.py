"""The paged 4-bit KV cache beyond its first operators, measured: finding the
sequences that share leading pages, attention that reads a shared prefix once
for all of them, rotary positions (of rows, and of queries and keys as these
are appended), and reading cached rows back.

`own = False` runs each operator in elementary torch operations, `own = True`
through the library's entry points.  A cache is [pages][heads][page_size]
[head_dim] in groups of 64 (codes two to a byte, a float32 minimum and scale
per group); row i of the page table lists the pages of sequence i, and
sequences that were forked from one another begin with the same pages.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
DT = {"f16": torch.float16, "f32": torch.float32}


# ---- cases -------------------------------------------------------------------
# b sequences; g groups of them share their leading pages (plo .. phi pages a
# group, its members spread over the batch), `lone` share nothing; slo .. shi
# tokens of their own, of which clo .. chi are the call's rows

def listed():
    return [
        # answers sampled from two short prompts, beside other requests: the smallest call, latency counts
        dict(name="share small", op="share", b=12, g=2, lone=4, ps=16, plo=8, phi=12, slo=3, shi=40, clo=1, chi=1),
        # a serving batch after it changed: a few system prompts of thousands of tokens, some requests without one
        dict(name="share batch", op="share", b=256, g=7, lone=31, ps=16, plo=100, phi=1500, slo=20, shi=900, clo=1, chi=1),
        # a step of a few answers to one short prompt (125M heads)
        dict(name="attn small", op="attn", dt="f16", b=6, g=1, lone=0, qh=12, kvh=12, d=64, ps=16, plo=19, phi=19, slo=5, shi=60,
             clo=1, chi=1),
        # a step of a block of 64 (6.7B heads) whose prompts begin alike: 4096 tokens, 100 to 500 of their own
        dict(name="attn block", op="attn", dt="f16", b=64, g=1, lone=0, qh=32, kvh=32, d=128, ps=64, plo=64, phi=64, slo=100, shi=500,
             clo=1, chi=1),
        # questions about a few long documents, eight query heads to a K/V head
        dict(name="attn long", op="attn", dt="f16", b=32, g=3, lone=2, qh=64, kvh=8, d=128, ps=128, plo=101, phi=243, slo=50, shi=1500,
             clo=1, chi=1),
        # the users' turns of two system prompts arrive as ragged chunks, beside requests without one
        dict(name="attn chunks", op="attn", dt="f16", b=20, g=2, lone=3, qh=32, kvh=8, d=128, ps=32, plo=60, phi=130, slo=40, shi=400,
             clo=1, chi=151),
        # queries and keys of a decode step of 64 sequences, half layout
        dict(name="rotate step", op="rotate", dt="f16", n=64, heads=64, d=128, rot=128, layout="half", kind="plain", top=4000),
        # ragged prompts: part of the head, pairs side by side, frequencies stretched for a long context
        dict(name="rotate prompts", op="rotate", dt="f16", n=19999, heads=40, d=128, rot=64, layout="pairs", kind="bands", top=120000),
        # a decode step: queries and keys rotated, keys and values into their pages
        dict(name="rotated step", op="rotated", dt="f16", b=64, qh=32, kvh=32, d=128, rot=128, layout="half", kind="plain", ps=64,
             lo=300, hi=900, clo=1, chi=1),
        # ragged prompts, shared K/V heads, half of the head rotated with stretched positions
        dict(name="rotated prompts", op="rotated", dt="f16", b=48, qh=32, kvh=8, d=128, rot=128, layout="half", kind="ramp", ps=64,
             lo=300, hi=900, clo=300, chi=700),
        # the rows of a few short sequences
        dict(name="read small", op="read", dt="f16", b=4, kvh=12, d=64, ps=16, lo=100, hi=300, clo=100, chi=300),
        # a block's whole caches, to go on in another form or on another machine
        dict(name="read block", op="read", dt="f16", b=64, kvh=32, d=128, ps=64, lo=300, hi=900, clo=300, chi=900),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["share", "attn", "attn", "attn", "rotate", "rotated", "read"])
    d = rng.choice([64, 128])
    ps = rng.choice([16, 32, 64, 128])
    dt = "f16" if rng.random() < 0.85 else "f32"
    if op in ("share", "attn"):
        g = rng.choice([1, 1, 2, 3, 7])
        b = g * 2 + (_log(rng, 6, 200) if op == "share" else _log(rng, 1, 50))
        lone = rng.randrange(3, b - 2 * g + 1) if op == "share" else rng.randrange(0, b - 2 * g + 1) if rng.random() < 0.5 else 0
        step = op == "share" or rng.random() < 0.6
        chi = 1 if step else _log(rng, 2, 150)
        shi = max(chi, _log(rng, 4, 700))
        top = _log(rng, 64, 24000)
        kvh = _log(rng, 1, 32)
        r = rng.choice([1, 1, 1, 2, 3, 4, 8])
        if op == "attn":   # what the plain form holds
            if dt == "f32":
                b, g, lone, top, chi = min(b, 8), 1, 0, min(top, 1500), min(chi, 40)
            while b * chi * kvh * r * (top + shi) > 250_000_000 or b * kvh * (shi + ps) > 600_000 or g * kvh * top > 1_500_000:
                top, chi, shi, kvh = max(64, top * 3 // 4), max(1, chi * 3 // 4), max(4, shi * 3 // 4), max(1, kvh * 7 // 8)
            shi = max(shi, chi)
        phi = max(1, top // ps)
        case = dict(op=op, b=b, g=g, lone=lone, ps=ps, plo=max(1, phi // rng.choice([1, 2, 5])), phi=phi,
                    slo=max(1, shi // rng.choice([1, 3, 20])), shi=shi, clo=max(1, chi // rng.choice([1, 3, 50])), chi=chi)
        return dict(case, dt=dt, qh=kvh * r, kvh=kvh, d=d) if op == "attn" else case
    rot = rng.choice([d, d, d // 2, d // 4])
    layout, kind = rng.choice(["half", "pairs"]), rng.choice(["plain", "linear", "base", "bands", "ramp"])
    if op == "rotate":
        return dict(op=op, dt=dt, n=_log(rng, 1, 9000), heads=_log(rng, 1, 64), d=d, rot=rot, layout=layout, kind=kind,
                    top=_log(rng, 50, 200000))
    b = _log(rng, 1, 48)
    kvh = _log(rng, 1, 32)
    hi = _log(rng, 20, 900)
    if op == "read":
        chi = _log(rng, 1, hi)
        return dict(op=op, dt=dt, b=b, kvh=kvh, d=d, ps=ps, lo=max(1, hi // 3), hi=hi, clo=max(1, chi // 3), chi=chi)
    chi = 1 if rng.random() < 0.4 else _log(rng, 2, 400)
    hi = max(chi, hi)
    return dict(op=op, dt=dt, b=b, qh=kvh * rng.choice([1, 1, 2, 4]), kvh=kvh, d=d, rot=rot, layout=layout, kind=kind, ps=ps,
                lo=max(1, hi // 2), hi=hi, clo=max(1, chi // 3), chi=chi)


# ---- inputs ------------------------------------------------------------------

def _spread(b, lo, hi, phase):
    """b sizes between lo and hi, the same for every seed (golden-ratio steps)."""
    f = (np.arange(b) * 0.6180339887498949 + phase) % 1.0
    return np.floor(lo + f * (hi - lo + 0.999)).astype(np.int64)


def _up(x, ps):
    return -(-x // ps)


def _ints(x):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=torch.int32, device=DEV)


def _before(n):
    """Offsets of parts of these sizes, laid end to end."""
    return np.concatenate(([0], np.cumsum(n)))


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


def _pool(pages, case, gen, dt):
    """Pages of quantized rows: K or V values of about unit size, some dims larger than others."""
    size = 0.5 + torch.rand((case["kvh"], 1, case["d"]), generator=gen, device=DEV)
    x = torch.randn((pages, case["kvh"], case["ps"], case["d"]), generator=gen, device=DEV, dtype=torch.float16)
    return _quantize((x * size.half()).to(dt))


def _empty_pool(pages, case):
    shape = (pages, case["kvh"], case["ps"])
    meta = shape + (case["d"] // 64,)
    return (torch.zeros(shape + (case["d"] // 2,), dtype=torch.uint8, device=DEV), torch.zeros(meta, device=DEV), torch.zeros(meta, device=DEV))


def _family(case):
    """Of every sequence: its group (-1: none), the pages that it shares, its own tokens and rows."""
    b, g = case["b"], case["g"]
    group = np.where(np.arange(b) < b - case["lone"], np.arange(b) % g, -1)
    shared = np.where(group >= 0, _spread(g, case["plo"], case["phi"], 0.61)[np.maximum(group, 0)], 0)
    tail = _spread(b, case["slo"], case["shi"], 0.37)
    n = np.minimum(tail, _spread(b, case["clo"], case["chi"], 0.83))
    return group, shared, tail, n


def _shared_table(case, gen):
    """The page table of forks that have grown since: shared leading pages, then pages of each sequence's own.  For finding
    the groups, the sequences stand in an order drawn from the seed."""
    group, shared, tail, n = _family(case)
    if case["op"] == "share":
        order = torch.randperm(case["b"], generator=gen, device=DEV).cpu().numpy()
        group, shared, tail, n = [x[order] for x in (group, shared, tail, n)]
    ps, g = case["ps"], case["g"]
    mine = _up(tail, ps)
    lead = _spread(g, case["plo"], case["phi"], 0.61)
    pages = int(lead.sum() + mine.sum()) + 3
    perm = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
    col = torch.arange(int((shared + mine).max()) + 1, device=DEV)[None]
    start = _ints(_before(lead)[np.maximum(group, 0)])[:, None]
    own_start = _ints(int(lead.sum()) + _before(mine)[:-1])[:, None]
    sh, all_ = _ints(shared)[:, None], _ints(shared + mine)[:, None]
    at = torch.where(col < sh, start + col, own_start + col - sh).clamp(max=pages - 1).long()
    table = torch.where(col < all_, perm[at], -1).to(torch.int32)
    refs = torch.zeros(pages, dtype=torch.int32, device=DEV)
    refs.index_add_(0, table[table >= 0].long(), torch.ones_like(table[table >= 0]))
    return dict(table=table, refs=refs, lens=_ints(shared * ps + tail), cu=_ints(_before(n)), ntok=int(n.sum()), max_q=int(n.max()),
                pages=pages, own_pages=int(mine.max()), max_tail=int(tail.max()))


def _shares(case):
    """The groups as fg_pages_share writes them: what a serving program keeps while its batch stays the same."""
    group, shared, _, n = _family(case)
    cu, rows, first, begin = _before(n), [], np.zeros(case["b"], np.int64), [0]
    for g in range(case["g"]):
        for i in np.flatnonzero(group == g):
            first[i] = len(rows) - begin[-1]
            rows += range(cu[i], cu[i + 1])
        begin.append(len(rows))
    b = case["b"]
    leader = np.where(np.arange(b) < case["g"], np.arange(b), -1)
    return dict(group=_ints(group), tokens=_ints(shared * case["ps"]), first=_ints(first), leader=_ints(leader),
                begin=_ints(begin + [begin[-1]] * (b - case["g"])), rows=_ints(rows + [-1] * (int(n.sum()) - len(rows))))


def _theta(case):
    """Angle that a position adds to each pair, in 64 bits, and the factor of cosines and sines."""
    rot, base, factor, ctx = case["rot"], 10000.0, 8.0, 4096.0
    i = np.arange(rot // 2, dtype=np.float64)
    if case["kind"] == "base":
        base *= factor ** (rot / (rot - 2))
    f = base ** (-2.0 * i / rot)
    if case["kind"] == "linear":
        f = f / factor
    elif case["kind"] == "bands":   # turns in the first context: many keep their pace, few are stretched, between them a blend
        t = (ctx * f / (2 * math.pi) - 1.0) / (4.0 - 1.0)
        s = np.clip(t, 0.0, 1.0)
        f = (1 - s) * f / factor + s * f
    elif case["kind"] == "ramp":    # the same along the pairs' numbers, and larger scores
        def at(turns):
            return rot * math.log(ctx / (2 * math.pi * turns)) / (2 * math.log(base))
        lo, hi = max(0.0, math.floor(at(32.0))), min(rot - 1.0, math.ceil(at(1.0)))
        s = np.clip((i - lo) / max(hi - lo, 0.001), 0.0, 1.0)
        f = (1 - s) * f + s * f / factor
        return f, float(np.float32(0.1 * math.log(factor) + 1.0))
    return f, 1.0


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    op, d = case["op"], case["d"] if "d" in case else 0
    s = dict(case=case)
    if op in ("share", "attn"):
        s |= _shared_table(case, gen)
        if op == "share":
            return s
        s["dt"] = DT[case["dt"]]
        s["shares"] = _shares(case)
        group, shared, _, _ = _family(case)
        size = np.bincount(group[group >= 0], _family(case)[3][group >= 0], case["g"])
        s["max_rows"], s["max_shared"] = int(size.max()), int(shared.max())
        s["k"], s["v"] = _pool(s["pages"], case, gen, s["dt"]), _pool(s["pages"], case, gen, s["dt"])
        s["q"] = (1.3 * torch.randn((s["ntok"], case["qh"] * d), generator=gen, device=DEV)).to(s["dt"])
        s["out"] = torch.zeros_like(s["q"])
        return s
    dt = s["dt"] = DT[case["dt"]]

    def rows(n, heads):
        return (1.3 * torch.randn((n, heads * d), generator=gen, device=DEV)).to(dt)

    if op in ("rotate", "rotated"):
        f, s["factor"] = _theta(case)
        s["theta"] = torch.as_tensor(f, device=DEV)
    if op == "rotate":
        s["x"] = rows(case["n"], case["heads"])
        s["pos"] = torch.randint(case["top"], (case["n"],), generator=gen, device=DEV, dtype=torch.int32)
        s["out"] = torch.zeros_like(s["x"])
        return s
    ps = case["ps"]
    lens = _spread(case["b"], case["lo"], case["hi"], 0.37)
    n = np.minimum(lens, _spread(case["b"], case["clo"], case["chi"], 0.83))
    need = _up(lens, ps)
    pages = int(need.sum()) + 3
    perm = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
    col = torch.arange(int(need.max()) + 1, device=DEV)[None]
    at = (_ints(_before(need)[:-1])[:, None] + col).clamp(max=pages - 1).long()
    s["table"] = torch.where(col < _ints(need)[:, None], perm[at], -1).to(torch.int32)
    s["refs"] = torch.zeros(pages, dtype=torch.int32, device=DEV)
    s["refs"][perm[: int(need.sum())].long()] = 1
    s["lens"], s["cu"], s["ntok"] = _ints(lens), _ints(_before(n)), int(n.sum())
    if op == "read":
        s["k"], s["v"] = _pool(pages, case, gen, dt), _pool(pages, case, gen, dt)
    else:
        s["k"], s["v"] = _empty_pool(pages, case), _empty_pool(pages, case)
        s["q"], s["k_new"], s["v_new"] = rows(s["ntok"], case["qh"]), rows(s["ntok"], case["kvh"]), rows(s["ntok"], case["kvh"])
        s["q_out"] = torch.zeros_like(s["q"])
    for name in ("k_out", "v_out"):
        s[name] = torch.zeros((s["ntok"], case["kvh"] * d), dtype=dt, device=DEV)
    return s


# ---- one pass ------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if own:
        return {"share": _own_share, "attn": _own_attn, "rotate": _own_rotate, "rotated": _own_rotated, "read": _own_read}[op](s)
    return {"share": _share, "attn": _attn, "rotate": _rotate, "rotated": _rotated, "read": _read}[op](s)


def _rows_of(s):
    """Sequence, position and number of every row of the ragged batch."""
    cu = s["cu"].long()
    row = torch.arange(s["ntok"], device=DEV)
    seq = torch.searchsorted(cu, row, right=True) - 1
    return seq, s["lens"].long()[seq] - (cu[seq + 1] - row), row - cu[seq]


def _share(s):
    table, ps, pages = s["table"], s["case"]["ps"], s["refs"].numel()
    b, stride = table.shape
    n = s["cu"][1:] - s["cu"][:-1]
    idx = torch.arange(b, device=DEV)
    usable = ((s["lens"] - n).clamp(min=0) // ps).clamp(max=stride)
    there = (table >= 0) & (table < pages)
    part = (n > 0) & (usable > 0) & there[:, 0]
    same = part[:, None] & part[None] & (table[:, :1] == table[:, 0][None])
    lead = torch.where(same, idx[None], b).amin(1).clamp(max=b - 1)
    col = torch.arange(stride, device=DEV)[None]
    alike = there & (table == table[lead]) & (col < torch.minimum(usable, usable[lead])[:, None])
    common = alike.to(torch.int32).cumprod(1).sum(1)
    other = part & (lead != idx)
    fit = (other[None] & same & (common[None] >= common[:, None])).sum(1)
    saved = torch.where(other & (common > 0), common * fit, 0)
    best = torch.zeros(b, dtype=torch.int64, device=DEV).scatter_reduce_(0, lead, saved, "amax")
    chosen = torch.where((saved > 0) & (saved == best[lead]), common, 0)
    pick = torch.zeros(b, dtype=torch.int64, device=DEV).scatter_reduce_(0, lead, chosen, "amax")
    member = part & (pick[lead] > 0) & ((common >= pick[lead]) | (lead == idx))
    heads = member & (lead == idx)
    group = torch.where(member, (heads.cumsum(0) - 1)[lead], -1)
    tokens = torch.where(member, pick[lead] * ps, 0)
    mates = member[None] & (group[:, None] == group[None])
    first = (torch.where(mates & (idx[None] < idx[:, None]), n[None], 0)).sum(1) * member
    size = torch.where(member[None] & (group[None] == idx[:, None]), n[None], 0).sum(1)
    begin = torch.cat((torch.zeros(1, dtype=torch.int64, device=DEV), size.cumsum(0)))
    leader = torch.where(heads[None] & (group[None] == idx[:, None]), idx[None], -1).amax(1)
    seq, _, at = _rows_of(s)
    slot = torch.where(member[seq], begin[group[seq].clamp(min=0)] + first[seq] + at, s["ntok"])
    rows = torch.full((s["ntok"] + 1,), -1, dtype=torch.int64, device=DEV).scatter_(0, slot, torch.arange(s["ntok"], device=DEV))
    return [x.int() for x in (group, tokens, first, leader, begin, rows[:-1])]


def _attn(s):
    c, sh = s["case"], s["shares"]
    b, g, qh, kvh, d, ps = c["b"], c["g"], c["qh"], c["kvh"], c["d"], c["ps"]
    r, mr, mq = qh // kvh, s["max_rows"], s["max_q"]
    lens, seq, at = s["lens"].long(), *_rows_of(s)[::2]

    def cached(x, pages):   # [sequences][kvh][tokens][d] in 32 bits
        v = _restore(*[t[pages.clamp(min=0)] for t in x])
        return v.permute(0, 2, 1, 3, 4).reshape(pages.shape[0], kvh, -1, d)

    def part(q, pages, see):   # largest score, sum and weighted values of padded rows [n][m][qh * d]
        n, m = q.shape[:2]
        q = q.view(n, m, kvh, r, d).permute(0, 2, 3, 1, 4).reshape(n, kvh, r * m, d)
        w = torch.matmul(q, cached(s["k"], pages).transpose(2, 3)).view(n, kvh, r, m, -1)
        w = w.mul_(1.0 / math.sqrt(d)).masked_fill_(~see[:, None, None], float("-inf"))
        top = w.amax(-1, keepdim=True).clamp(min=-1e30)
        w = w.sub_(top).exp_()
        v = torch.matmul(w.view(n, kvh, r * m, -1), cached(s["v"], pages)).view(n, kvh, r, m, d)
        return [x.permute(0, 3, 1, 2, 4).reshape(n, m, qh, -1) for x in (top, w.sum(-1, keepdim=True), v)]

    # the groups' prefixes, every row of a group at once
    group = sh["group"].long()[seq]
    row_at = sh["first"].long()[seq] + at
    tokens = sh["tokens"].long()
    lead = sh["leader"][:g].long()
    q = torch.zeros((g + 1, mr, qh * d), device=DEV)
    q[group, row_at.clamp(max=mr - 1)] = s["q"].float()   # rows of no group land in the last, unused one
    key = torch.arange(s["max_shared"] * ps, device=DEV)
    see = (key < tokens[lead][:, None])[:, None].expand(g, mr, -1)
    head = [x[group.clamp(min=0), row_at.clamp(max=mr - 1)] for x in part(q[:g], s["table"][lead, : s["max_shared"]], see)]
    # what the sequences have of their own
    col = tokens[:, None] // ps + torch.arange(s["own_pages"], device=DEV)
    pages = s["table"].long().gather(1, col.clamp(max=s["table"].shape[1] - 1))
    q = torch.zeros((b, mq, qh * d), device=DEV)
    q[seq, at] = s["q"].float()
    p = (lens - (s["cu"][1:] - s["cu"][:-1]).long())[:, None] + torch.arange(mq, device=DEV)[None]
    key = tokens[:, None] + torch.arange(s["own_pages"] * ps, device=DEV)
    see = (key[:, None] <= p[..., None]) & (key < lens[:, None])[:, None]
    tail = [x[seq, at] for x in part(q, pages, see)]
    both = (group >= 0)[:, None, None]
    top = torch.where(both, torch.maximum(head[0], tail[0]), tail[0])
    fh = torch.where(both, (head[0] - top).exp(), 0.0)
    ft = (tail[0] - top).exp()
    o = (fh * head[2] + ft * tail[2]) / (fh * head[1] + ft * tail[1])
    return o.reshape(s["ntok"], -1).to(s["dt"])


def _turned(s, x, pos, heads):
    """Rows of heads, rotated to their positions: angles in 64 bits, products in 32."""
    c, h = s["case"], s["case"]["rot"] // 2
    angle = pos.double()[:, None] * s["theta"]
    cos, sin = [(f(angle) * s["factor"]).float()[:, None] for f in (torch.cos, torch.sin)]
    y = x.float().view(x.shape[0], heads, c["d"]).clone()
    if c["layout"] == "half":
        a, b = y[..., :h].clone(), y[..., h:2 * h].clone()
        y[..., :h], y[..., h:2 * h] = a * cos - b * sin, a * sin + b * cos
    else:
        a, b = y[..., :2 * h:2].clone(), y[..., 1:2 * h:2].clone()
        y[..., :2 * h:2], y[..., 1:2 * h:2] = a * cos - b * sin, a * sin + b * cos
    return y.view(x.shape).to(s["dt"])


def _rotate(s):
    return _turned(s, s["x"], s["pos"], s["case"]["heads"])


def _rotated(s):
    """Returns the rotated queries, and the appended rows as the cache holds them: what their codes stand for."""
    c = s["case"]
    seq, pos, _ = _rows_of(s)
    page, slot = s["table"][seq, pos // c["ps"]].long(), pos % c["ps"]

    def store(name, x):
        new = _quantize(x.view(s["ntok"], c["kvh"], c["d"]))
        s[name][0][page, :, slot], s[name][1][page, :, slot], s[name][2][page, :, slot] = new
        return [s[name][1], s[name][2], _restore(*new).to(s["dt"]).view(s["ntok"], -1)]

    return [_turned(s, s["q"], pos, c["qh"]), *store("k", _turned(s, s["k_new"], pos, c["kvh"])), *store("v", s["v_new"])]


def _read(s):
    seq, pos, _ = _rows_of(s)
    ps = s["case"]["ps"]
    page, slot = s["table"][seq, pos // ps].long(), pos % ps
    return [_restore(*[t[page, :, slot] for t in s[name]]).to(s["dt"]).view(s["ntok"], -1) for name in ("k", "v")]


# ---- the same through the library --------------------------------------------------

def _handle(s):
    """What a user's program keeps between calls: the pool's and the table's handles, a workspace, the groups, the rotation."""
    if "handle" not in s:
        import int4_group_quantized_gb300 as fg
        c, ws, more = s["case"], None, None
        tab = fg.PageTable(s["table"], s["lens"], s["refs"], c["ps"]) if "table" in s else None
        pool = fg.PagePool.of(*s["k"], *s["v"], s["dt"]) if "k" in s else None
        if c["op"] == "share":
            more = fg.PageShare.empty(tab, s["ntok"])
            ws = fg.workspace(fg.fg_pages_share_workspace_bytes(tab))
        elif c["op"] == "attn":
            more = fg.PageShare(**s["shares"])
            ws = fg.workspace(fg.fg_paged_attention_shared_workspace_bytes(pool, tab, c["qh"], s["ntok"], s["max_q"]))
        elif c["op"] in ("rotate", "rotated"):
            more = fg.Rotary(c["rot"], layout=c["layout"], scaling=c["kind"], base=10000.0, factor=8.0, context=4096,
                             low=1.0, high=4.0 if c["kind"] == "bands" else 32.0)
        s["handle"] = fg, pool, tab, ws, more
    return s["handle"]


def _own_share(s):
    fg, _, tab, ws, share = _handle(s)
    fg.fg_pages_share(tab, s["cu"], share, min_tokens=1, ws=ws)
    return [share.group, share.tokens, share.first, share.leader, share.begin, share.rows]


def _own_attn(s):
    fg, pool, tab, ws, share = _handle(s)
    fg.fg_paged_attention_shared(pool, tab, s["cu"], share, s["q"], s["case"]["qh"], s["out"], s["max_q"], ws=ws)
    return s["out"]


def _own_rotate(s):
    fg, _, _, _, rotary = _handle(s)
    fg.fg_rotate(rotary, s["x"], s["pos"], s["case"]["heads"], s["out"])
    return s["out"]


def _own_rotated(s):
    fg, pool, tab, _, rotary = _handle(s)
    fg.fg_paged_append_rotated(pool, tab, s["cu"], rotary, s["q"], s["case"]["qh"], s["q_out"], s["k_new"], s["v_new"], s["k_out"],
                               s["v_out"])
    return [s["q_out"], s["k"][1], s["k"][2], s["k_out"], s["v"][1], s["v"][2], s["v_out"]]


def _own_read(s):
    fg, pool, tab, _, _ = _handle(s)
    fg.fg_paged_read(pool, tab, s["cu"], s["k_out"], s["v_out"])
    return [s["k_out"], s["v_out"]]


# ---- what a pass cannot do without ----------------------------------------------------

def work(case):
    op = case["op"]
    if op == "share":   # the entries that members and leaders have in common, once each, and the lists
        group, shared, _, n = _family(case)
        return {"bytes": 4.0 * float(shared.sum() + 6 * case["b"] + n.sum()), "flops": 0.0}
    d, e = case["d"], 2 if case["dt"] == "f16" else 4
    if op == "rotate":
        size = float(case["n"]) * case["heads"] * d
        return {"bytes": 2 * size * e + 4.0 * case["n"], "flops": 3.0 * size * case["rot"] / d}
    tok = case["kvh"] * d * 0.625   # bytes of one token's K (or V) row
    if op == "attn":
        group, shared, tail, n = _family(case)
        ps = case["ps"]
        keys = float(_spread(case["g"], case["plo"], case["phi"], 0.61).sum()) * ps + float(tail.sum())
        pairs = float((n * (shared * ps + tail) - n * (n - 1) // 2).sum())
        return {"bytes": 2 * keys * tok + 2.0 * float(n.sum()) * case["qh"] * d * e, "flops": 4.0 * d * case["qh"] * pairs}
    lens = _spread(case["b"], case["lo"], case["hi"], 0.37)
    rows = float(np.minimum(lens, _spread(case["b"], case["clo"], case["chi"], 0.83)).sum())
    if op == "read":
        return {"bytes": 2 * rows * (tok + case["kvh"] * d * e), "flops": 4.0 * rows * case["kvh"] * d}
    return {"bytes": 2 * rows * (2 * case["kvh"] * d * e + tok) + 2 * rows * case["qh"] * d * e,
            "flops": rows * d * (20.0 * case["kvh"] + 3.0 * case["qh"] * case["rot"] / d)}


# ---- 64 bits -----------------------------------------------------------------------

def _values(x, page, slot, head):
    """Rows of one head in 64 bits."""
    c, mn, sc = (t[page, head, slot] for t in x)
    v = torch.empty((len(c), 2 * c.shape[1]), dtype=torch.float64, device=DEV)
    v[:, 0::2], v[:, 1::2] = (c & 15).double(), (c >> 4).double()
    return (v.view(len(c), -1, 64) * sc.double()[..., None] + mn.double()[..., None]).view(len(c), -1)


def _spun(case, theta, factor, x, pos, heads):
    """Rotation as a product of complex numbers, in 64 bits."""
    rot, n = case["rot"], x.shape[0]
    z = x.double().view(n, heads, case["d"])
    front = z[..., :rot]
    front = front.view(n, heads, 2, rot // 2).transpose(2, 3) if case["layout"] == "half" else front.view(n, heads, rot // 2, 2)
    front = torch.view_as_complex(front.contiguous()) * torch.polar(torch.full_like(theta, factor)[None], pos.double()[:, None] * theta)[:, None]
    front = torch.view_as_real(front)
    front = front.transpose(2, 3) if case["layout"] == "half" else front
    return torch.cat((front.reshape(n, heads, rot), z[..., rot:]), -1).view(n, -1)


def exact(case, seed):
    op = case["op"]
    if op == "share":
        return None   # whole numbers: nothing is computed
    s = prepare(case, seed)
    dt = s["dt"]
    if op == "rotate":
        return _spun(case, s["theta"], s["factor"], s["x"], s["pos"], case["heads"])
    d, ps, kvh = case["d"], case["ps"], case["kvh"]
    lens, cu = s["lens"].tolist(), s["cu"].tolist()

    def places(i):   # pages and slots of sequence i's tokens
        at = torch.arange(lens[i], device=DEV)
        return s["table"][i, at // ps].long(), at % ps

    if op == "attn":
        r = case["qh"] // kvh
        q = s["q"].double().view(s["ntok"], kvh, r, d)
        out = torch.zeros_like(q)
        for i, length in enumerate(lens):
            a, e = cu[i], cu[i + 1]
            page, slot = places(i)
            p = torch.arange(length - (e - a), length, device=DEV)
            hidden = torch.arange(length, device=DEV)[None] > p[:, None]
            for h in range(kvh):
                x = torch.einsum("trd,jd->trj", q[a:e, h], _values(s["k"], page, slot, h)) / math.sqrt(d)
                x = torch.softmax(x.masked_fill(hidden[:, None], -math.inf), -1)
                out[a:e, h] = torch.einsum("trj,jd->trd", x, _values(s["v"], page, slot, h))
        return out.view(s["ntok"], -1)
    if op == "read":
        got = []
        for name in ("k", "v"):
            y = torch.zeros((s["ntok"], kvh, d), dtype=torch.float64, device=DEV)
            for i in range(case["b"]):
                page, slot = [t[lens[i] - (cu[i + 1] - cu[i]):] for t in places(i)]
                for h in range(kvh):
                    y[cu[i]:cu[i + 1], h] = _values(s[name], page, slot, h)
            got.append(y.view(s["ntok"], -1))
        return got
    pos = torch.cat([torch.arange(lens[i] - (cu[i + 1] - cu[i]), lens[i], device=DEV) for i in range(case["b"])])
    got = [_spun(case, s["theta"], s["factor"], s["q"], pos, case["qh"])]
    # the codes are fixed by the rotated row in the activations' type and fp32 operations: those, then their values exactly
    for name, x in (("k", _spun(case, s["theta"], s["factor"], s["k_new"], pos, kvh)), ("v", s["v_new"])):
        f = x.to(dt).float().view(s["ntok"], kvh, d // 64, 64)
        lo, hi = f.min(-1).values, f.max(-1).values
        code = torch.clamp(torch.round((f - lo[..., None]) / (hi - lo)[..., None] * 15), 0, 15).double()
        mins, scales = s[name][1].double(), s[name][2].double()
        for i in range(case["b"]):
            page, slot = [t[lens[i] - (cu[i + 1] - cu[i]):] for t in places(i)]
            mins[page, :, slot], scales[page, :, slot] = lo[cu[i]:cu[i + 1]].double(), (hi - lo).double()[cu[i]:cu[i + 1]] / 15
        got += [mins, scales, (code * ((hi - lo) / 15).double()[..., None] + lo.double()[..., None]).view(s["ntok"], -1)]
    return got
