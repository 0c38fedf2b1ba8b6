"""Paged 4-bit KV cache, written out plainly in numpy (test oracle).

The notes' cache is one block of sequences that grow together ("背景知识", KV
Concat; "5. 近似方法", KV in 4-bit groups along the hidden dimension); here its
rows lie in pages, so that sequences of different lengths can grow, fork, end
and move.  Readings:
  * pages are handed out lowest number first, sequence by sequence (growth) or
    fork by fork;
  * a fork shares the source's full pages and copies a partly filled last one;
  * compaction with m pages in use moves the pages numbered m and above, in
    ascending order, into the free pages below m, in ascending order;
  * the query at position p sees token j iff j <= p and (no window, or
    j > p - window, or j < sinks); a query that sees nothing gives 0;
  * attention reads fmaf(q, scale, min), in fp64 here.
Test infrastructure only.
"""
from __future__ import annotations

import numpy as np

from . import codec


class Pages:
    """Table, lengths and reference counts, as the device holds them."""

    def __init__(self, table, lens, refs, page_size):
        self.table, self.lens, self.refs = np.array(table), np.array(lens), np.array(refs)
        self.ps = int(page_size)
        self.stride = self.table.shape[1]
        self.full = False   # a page could not be had

    def held(self, i):
        return min(-(-int(self.lens[i]) // self.ps), self.stride)

    def free_pages(self):
        return [int(p) for p in np.flatnonzero(self.refs == 0)]

    def reserve(self, n):
        free = self.free_pages()
        for i, m in enumerate(n):
            have = self.held(i)
            want = -(-(int(self.lens[i]) + int(m)) // self.ps)
            if want > self.stride:
                self.full = True
            for j in range(have, min(want, self.stride)):
                if free:
                    p = free.pop(0)
                    self.refs[p] = 1
                else:
                    p, self.full = -1, True
                self.table[i, j] = p
            self.lens[i] += m

    def fork(self, src, dst):
        """Returns the pages to copy, [(from, to)]."""
        free = self.free_pages()
        lens0 = self.lens.copy()
        taken, moves = set(), []
        for a, b in zip(src, dst):
            a, b = int(a), int(b)
            if not (0 <= a < len(lens0) and 0 <= b < len(lens0)) or a == b or lens0[b] != 0 or b in taken:
                if 0 <= b < len(lens0):
                    taken.add(b)
                self.full = True
                continue
            taken.add(b)
            full, part = divmod(int(lens0[a]), self.ps)
            if part:
                if not free:
                    self.full = True
                    continue
                p = free.pop(0)
                moves.append((int(self.table[a, full]), p))
                self.table[b, full] = p
                self.refs[p] = 1
            for j in range(full):
                self.table[b, j] = self.table[a, j]
                self.refs[self.table[a, j]] += 1
            self.lens[b] = lens0[a]
        return moves

    def free(self, rows):
        for i in rows:
            i = int(i)
            if not 0 <= i < len(self.lens):
                continue
            for j in range(self.held(i)):
                if 0 <= self.table[i, j] < len(self.refs):
                    self.refs[self.table[i, j]] -= 1
                self.table[i, j] = -1
            self.lens[i] = 0

    def compact(self):
        """Returns the pages to move, [(from, to)]."""
        live = int((self.refs > 0).sum())
        src = [p for p in range(live, len(self.refs)) if self.refs[p] > 0]
        dst = [p for p in range(live) if self.refs[p] <= 0]
        to = dict(zip(src, dst))
        for i in range(len(self.lens)):
            for j in range(self.held(i)):
                self.table[i, j] = to.get(int(self.table[i, j]), self.table[i, j])
        for a, b in to.items():
            self.refs[b], self.refs[a] = self.refs[a], 0
        return list(to.items())


def restore(codes, mins, scales):
    """The values that the codes stand for, fp64 (fmaf rounded once to fp32)."""
    return codec.dequant_g64(codes, mins, scales, np.float32).astype(np.float64)


def visible(pos, keys, window, sinks):
    """[rows][keys] truth values."""
    j = np.arange(keys)[None]
    p = np.asarray(pos)[:, None]
    see = j <= p
    if window:
        see &= (j > p - window) | (j < sinks)
    return see


def attention(q, k, v, pos, window=0, sinks=0, present=None):
    """q: [rows][d] at positions pos; k, v: [keys][d], fp64.  Returns the rows'
    output, sum_j p_j |v_j| and max_j sum_d |q_d k_jd| / sqrt(d) (what error
    bounds are made of).  A column group of 64 with NaN values gives NaN to
    the rows that see it and nothing to the others."""
    rows, d = q.shape
    see = visible(pos, k.shape[0], window, sinks)
    if present is not None:
        see &= np.asarray(present)[None]
    with np.errstate(all="ignore"):
        s = np.where(see, q @ np.where(np.isfinite(k), k, 0.0).T / np.sqrt(d), -np.inf)
        bad_k = ~np.isfinite(k).all(axis=1)
        s = np.where(see & bad_k[None], np.nan, s)
        m = np.max(np.where(see, s, -np.inf), axis=1, keepdims=True, initial=-np.inf)
        p = np.where(see, np.exp(s - np.where(np.isneginf(m), 0.0, m)), 0.0)
        total = p.sum(axis=1, keepdims=True)
        p = np.where(total == 0, 0.0, p / np.where(total == 0, 1.0, total))
        fin = np.isfinite(v)
        out = p @ np.where(fin, v, 0.0)
        out = np.where((see.astype(np.float64) @ (~fin).astype(np.float64)) > 0, np.nan, out)
        mag = p @ np.where(fin, np.abs(v), 0.0)
        work = np.where(see, np.abs(q) @ np.abs(np.where(np.isfinite(k), k, 0.0)).T / np.sqrt(d), 0.0)
    return out, mag, work.max(axis=1, initial=0.0)


# ---- how far a kernel's rows may be off ------------------------------------------

HALF = 2.0 ** -11   # half a step of fp16, relative; of its subnormals 2^-25
F32 = 2.0 ** -23    # a truncated fp32 sum, relative


def attention_bound(q, k, v, pos, window=0, sinks=0, present=None, kind="step"):
    """The rows' output (attention above) and what an element of it may be off, for K and V given as (codes, mins,
    scales) of a head's tokens.  Every term is taken over the tokens that a row sees, with their weights p_j:

      * the result's rounding: half a step;
      * sums in fp32: (n + d + 16) steps of what is summed.  A score off by e moves the output by at most
        (exp(2 e) - 1) sum p |v|;
      * step: scores are sums of q c, c <= 15, times the scale, and of the minimum times sum q.  The weight w = p scale
        is rounded to fp16 and multiplies c - 8.  Its power of two keeps the largest w of the row and group at 2^4 or
        more, so a small w is off by 2^-25 / 2^4 of the largest;
      * chunk: K, V and P are rounded to fp16.  The largest P of a row is 2^4 or more, so a small one is off by 2^-25 /
        2^4 of the largest;
      * f32: no rounding but fp32's own."""
    kv, vv = restore(*k), restore(*v)
    out, mag, work = attention(q, kv, vv, pos, window, sinks, present)
    n, d = kv.shape
    groups = d // 64
    see = visible(pos, n, window, sinks)
    if present is not None:
        see &= np.asarray(present)[None]
    with np.errstate(all="ignore"):
        fin = lambda x: np.where(np.isfinite(x), x, 0.0)   # what is not finite gives NaN rows or groups: no bound there
        s = np.where(see, q @ fin(kv).T / np.sqrt(d), -np.inf)
        p = np.exp(s - np.max(s, axis=1, keepdims=True, initial=-1e300))
        p = np.where(see, p, 0.0)
        p /= np.maximum(p.sum(axis=1, keepdims=True), 1e-300)
        qg = np.abs(fin(q)).reshape(len(q), groups, 64).sum(2)
        terms = np.where(see, qg @ (15 * np.abs(fin(k[2])) + np.abs(fin(k[1]))).astype(np.float64).T / np.sqrt(d), 0.0).max(axis=1, initial=0.0)
    wide = lambda x: np.repeat(x, 64, axis=1)              # a value a group, for each of its dims
    vmin, vscale = np.abs(fin(v[1])).astype(np.float64), np.abs(fin(v[2])).astype(np.float64)
    steps = (n + d + 16) * F32
    work, terms = work[:, None], terms[:, None]
    if kind == "f32":
        tol = 2.0 ** -24 * np.abs(out) + steps * mag + np.expm1(2 * steps * work) * mag
    elif kind == "step":
        big = (p[:, :, None] * vscale[None]).max(axis=1, initial=0.0)
        tol = HALF * np.abs(out) + 2.0 ** -25 + steps * wide(p @ (vmin + 15 * vscale)) + np.expm1(2 * (d + 16) * F32 * terms) * mag
        tol = tol + wide(HALF * 8 * (p @ vscale) + n * 2.0 ** -26 * big)
    else:
        tiny = 2.0 ** -25 * np.abs(fin(q)).sum(1, keepdims=True) / np.sqrt(d)     # K's subnormals, in the scores
        tol = HALF * (np.abs(out) + 2 * mag) + 2.0 ** -24 + steps * mag + np.expm1(2 * ((HALF + steps) * work + tiny)) * mag
        tol = tol + n * 2.0 ** -29 * p.max(axis=1, initial=0.0)[:, None] * np.abs(fin(vv)).max(axis=0, initial=0.0)[None]
    return out, tol


def off_by_too_much(got, ref, tol, rms=None):
    """Why `got` is not `ref` within `tol`, and within `rms` in the mean (relative, and half a step of fp16's
    subnormals); None where it is."""
    if not np.array_equal(np.isnan(got), np.isnan(ref)):
        return "NaN where there should be none, or none where there should be"
    f = ~np.isnan(ref)
    err = np.abs(got[f] - ref[f])
    worst = (err - tol[f]).max(initial=-1.0)
    if worst > 0:
        return f"error {err.max():.3g} above its bound by {worst:.3g}"
    if rms is not None and f.any():
        e, w = np.sqrt(np.mean(err ** 2)), np.sqrt(np.mean(ref[f] ** 2))
        if e > rms * w + 2.0 ** -25:
            return f"rms error {e / w:.3g} > {rms:.3g}"
    return None


def not_nearest(got, ref):
    """The share of elements that are not the 64-bit result rounded to fp16: what arithmetic adds to that rounding shows
    here and hardly in a bound (a result off by e steps before it is rounded is another fp16 in a share e of the cases).
    Results of fp16's subnormals, and NaN, are left out."""
    f = np.isfinite(ref) & (np.abs(ref) > 2.0 ** -13)
    want = ref[f].astype(np.float16)
    return float(np.mean(got[f].astype(np.float16) != want)) if f.any() else 0.0


# ---- shared prefixes ---------------------------------------------------------------

def share(table, lens, cu, pages, ps, min_tokens):
    """Groups of sequences that share leading pages: (group, tokens, first, leader, begin, rows), one sequence after another.
    A sequence takes part with the full pages before its rows; its leader is the lowest one with the same first page; a
    group shares the P >= min_tokens / ps that saves the most page reads, the larger of two that save the same."""
    seqs, stride = table.shape
    n = np.diff(cu)

    def usable(i):
        k = 0 if n[i] <= 0 else min(max(int(lens[i]) - int(n[i]), 0) // ps, stride)
        for j in range(k):
            if not 0 <= table[i, j] < pages:
                return j
        return k

    use = [usable(i) for i in range(seqs)]
    group, tokens, first = np.full(seqs, -1), np.zeros(seqs, int), np.zeros(seqs, int)
    leaders, members = [], []
    for lead in range(seqs):
        if use[lead] == 0 or any(use[j] and table[j, 0] == table[lead, 0] for j in range(lead)):
            continue
        common = {}
        for i in range(lead + 1, seqs):
            if use[i] and table[i, 0] == table[lead, 0]:
                c = 0
                while c < min(use[i], use[lead]) and table[i, c] == table[lead, c]:
                    c += 1
                common[i] = c
        best = (0, 0)
        for p in set(common.values()):
            if p * ps >= min_tokens:
                best = max(best, (p * sum(c >= p for c in common.values()), p))
        if best[0]:
            leaders.append(lead)
            members.append([lead] + [i for i, c in common.items() if c >= best[1]])
            for i in members[-1]:
                group[i], tokens[i] = len(leaders) - 1, best[1] * ps
    begin, rows = [0], []
    for m in members:
        for i in m:
            first[i] = len(rows) - begin[-1]
            rows += range(int(cu[i]), int(cu[i + 1]))
        begin.append(len(rows))
    pad = lambda x, k, fill: np.array(list(x) + [fill] * (k - len(x)), dtype=int)
    return group, tokens, first, pad(leaders, seqs, -1), pad(begin, seqs + 1, len(rows)), pad(rows, int(cu[-1]), -1)
