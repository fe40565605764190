"""Plain models of the decode-loop operators: beam selection in 64 bits,
reordering, and a paged cache kept sequence by sequence.  numpy and Python
only; nothing is shared with the GPU path."""
from __future__ import annotations

import numpy as np

HALF_STEP = 2.0 ** -24  # relative, of fp32


def beam_candidates(logits, scores, temperature, finished=None, eos=-1):
    """c[w, v] of one sequence in 64 bits, -inf where there is no candidate."""
    z = np.asarray(logits, dtype=np.float64)
    W, V = z.shape
    c = np.full((W, V), -np.inf)
    for w in range(W):
        s = float(scores[w])
        if s == -np.inf:
            continue
        if finished is not None and finished[w]:
            c[w, eos] = s
            continue
        m = z[w].max()
        if m == -np.inf:
            continue
        with np.errstate(over="ignore"):
            e = np.exp((z[w] - m) / temperature)
            c[w] = s + (z[w] - m) / temperature - np.log(e.sum())
        c[w, z[w] == -np.inf] = -np.inf
    return c


def beam_tolerance(c, V):
    """How far a returned score may be from c.  Rounding to fp32: half a step
    of |c|.  The sum of exponentials, relative: a term exp(-y) is off by the
    rounded scale and the rounded exponent, 2^-24 y each, by its exponential
    (a step, 2^-23) and by three additions in fp32 (2^-24 each); weighted by
    the terms the y average to at most ln V (entropy = ln sum + mean y <= ln V)."""
    return HALF_STEP * np.abs(c) + (2 * np.log(V + 1.0) + 5) * HALF_STEP


def check_beams(c, out_score, out_parent, out_token, M):
    """The returned lists against c[W, V]: the M largest in descending order,
    each at a (beam, token) that has that value, none twice, -inf and -1 past
    the last."""
    W, V = c.shape
    n = min(M, int((c > -np.inf).sum()))
    best = np.sort(c[c > -np.inf].ravel())[::-1][:n]
    assert np.all(out_score[n:] == -np.inf) and np.all(out_parent[n:] == -1) and np.all(out_token[n:] == -1)
    got = out_score[:n].astype(np.float64)
    with np.errstate(over="ignore"):
        best32 = best.astype(np.float32).astype(np.float64)
    fine = np.isfinite(best32)
    assert np.array_equal(got[~fine], best32[~fine])
    assert np.all(np.abs(got[fine] - best[fine]) <= beam_tolerance(best[fine], V)), (got, best)
    assert np.all(out_score[1:n] <= out_score[:max(n - 1, 0)])
    assert np.all((out_parent[:n] >= 0) & (out_parent[:n] < W) & (out_token[:n] >= 0) & (out_token[:n] < V))
    at = c[out_parent[:n], out_token[:n]]
    assert np.all(at > -np.inf)
    assert np.all(np.abs(at[fine] - best[fine]) <= 2 * beam_tolerance(best[fine], V))
    assert len({(p, t) for p, t in zip(out_parent[:n], out_token[:n])}) == n


class CacheModel:
    """A paged cache, one sequence after the other."""

    def __init__(self, seq_len, tables, free, page_size, max_blocks, num_pages):
        self.seq_len, self.tables, self.free = list(seq_len), [list(t) for t in tables], list(free)
        self.page, self.blocks, self.pages = page_size, max_blocks, num_pages

    def _blocks(self, tokens):
        return -(-tokens // self.page)

    def extend(self, counts, max_tokens):
        """(slots, positions, seq_ids, query_start, granted, length error, lack of pages)"""
        slots, positions, ids = [-1] * max_tokens, [0] * max_tokens, [-1] * max_tokens
        start, granted, t = [], [], 0
        bad = lack = stopped = False
        for b, n in enumerate(counts):
            s = self.seq_len[b]
            if s < 0 or n < 0 or s + n > self.blocks * self.page:
                bad, n = True, 0
                s = max(s, 0)
            start.append(min(t, max_tokens))
            room = t + n <= max_tokens
            bad |= not room
            need = self._blocks(s + n) - self._blocks(s)
            fits = room
            if need and room:
                if stopped or need > len(self.free):
                    fits, stopped, lack = False, True, True
                else:
                    at = self._blocks(s)
                    for j in range(need):
                        self.tables[b][at + j] = self.free.pop()
            granted.append(n if fits else 0)
            for i in range(n):
                if t + i < max_tokens:
                    positions[t + i], ids[t + i] = s + i, b
                    if fits:
                        slots[t + i] = self.tables[b][(s + i) // self.page] * self.page + (s + i) % self.page
            t += n
        start.append(min(t, max_tokens))
        return slots, positions, ids, start, granted, bad, lack

    def commit(self, reserved, accepted, extra=1, finished=None):
        bad, back = False, []
        for b, r in enumerate(reserved):
            s, ended = self.seq_len[b], bool(finished is not None and finished[b])
            if s < 0 or r < 0 or s + r > self.blocks * self.page:
                bad = True
                if ended:
                    self.seq_len[b] = 0
                continue
            keep = min(max(accepted[b] + extra, 0), r)
            if ended:
                now = 0
            else:
                bad |= keep != accepted[b] + extra and r > 0
                now = s + keep
            back += self.tables[b][self._blocks(now):self._blocks(s + r)]
            self.seq_len[b] = now
        self.free += back[::-1]
        return bad
