"""CPU oracle of the decoder cache: plain numpy, 64 bits, one row or page at a time.

TEST INFRASTRUCTURE ONLY, as the rest of this package.  Written from the
definitions in include/had.h; it shares no code with the CUDA library.  Pins
are in ``tests/test_cache_host.py``: codes against exact fractions and the
half-step bound, attention against the causal oracle of this package on a
whole sequence and against a dense softmax, the books against hand-worked
tables.
"""
import numpy as np


def bf16_round(x, way):
    """The nearest bf16 value not below (way +1) or not above (way -1) the fp32 array x."""
    x = np.ascontiguousarray(np.asarray(x, np.float32))
    cut = (x.view(np.uint32) & np.uint32(0xFFFF0000)).view(np.float32)
    with np.errstate(over="ignore", invalid="ignore"):
        away = ((cut.view(np.uint32) >> 16) + 1 << 16).astype(np.uint32).view(np.float32)
        # a cut towards zero lies below a positive x and above a negative one
        return np.where(cut == x, cut, np.where((x > 0) == (way > 0), away, cut)).astype(np.float32)


def quantise(v):
    """Codes [.., d], scale [..] and zero point [..] (fp32) of the fp32 rows v."""
    v = np.asarray(v, np.float32)
    with np.errstate(all="ignore"):
        zero = bf16_round(v.min(-1) + np.float32(0), -1)
        scale = bf16_round((v.max(-1) - zero) / np.float32(15), +1)
        fine = np.isfinite(v).all(-1) & np.isfinite(zero) & np.isfinite(np.float32(15) * scale)
        most = 15 * scale.astype(np.float64) + zero                # exact, then rounded once
        fine &= np.isfinite(most.astype(np.float32))
        step = np.where(fine & (scale > 0), scale, np.float32(1))[..., None]
        code = np.clip(np.rint((v - zero[..., None]) / step), 0, 15)
        code = np.where((fine & (scale > 0))[..., None], code, 0)
    nan = np.float32("nan")
    return code.astype(np.int64), np.where(fine, scale, nan), np.where(fine, zero, nan)


def visible(pos, window, sinks):
    """Cached positions that the query at position pos sees, ascending."""
    if pos < 0:
        return np.zeros(0, np.int64)
    j = np.arange(pos + 1)
    return j[(j > pos - window) | (j < sinks)] if window > 0 else j


def attend(sq, sk, codes, scale, zero, N, tau, window, sinks, pos):
    """One row: query signs sq [d] at position pos against key signs sk [L, d] and values
    codes [L, d], scale [L], zero [L]; returns (out [d], kept positions, sum p (|c s| + |z|))."""
    j = visible(pos, window, sinks)
    if j.size == 0:
        return np.zeros(sq.shape[-1]), j, np.zeros(sq.shape[-1])
    s = sk[j].astype(np.int64) @ sq.astype(np.int64)
    kept = np.sort(j[np.lexsort((j, -s))[:N]])
    logit = np.float64(tau) * (sk[kept].astype(np.int64) @ sq.astype(np.int64))
    p = np.exp(logit - logit.max())
    p /= p.sum()
    cs = codes[kept].astype(np.float64) * scale[kept].astype(np.float64)[:, None]
    z = zero[kept].astype(np.float64)[:, None]
    return p @ (cs + z), kept, p @ (np.abs(cs) + np.abs(z))


class Books:
    """The pages' books as Python lists; each method is one operator."""

    def __init__(self, table, lens, refs, page):
        self.table = [list(map(int, r)) for r in table]
        self.lens, self.refs, self.page = list(map(int, lens)), list(map(int, refs)), page

    def arrays(self):
        return np.array(self.table), np.array(self.lens), np.array(self.refs)

    def _drop(self, s, c):
        if self.table[s][c] >= 0:
            self.refs[self.table[s][c]] -= 1
            self.table[s][c] = -1

    def fork(self, src, dst):
        old = [(list(self.table[s]), self.lens[s]) for s in src]
        for (row, n), t in zip(old, dst):
            row = [p if c * self.page < n else -1 for c, p in enumerate(row)]
            for p in row:
                if p >= 0:
                    self.refs[p] += 1
            for c in range(len(row)):
                self._drop(t, c)
            self.table[t], self.lens[t] = row, n

    def reserve(self, grow):
        """(src, dst), or None where the pool has too few free pages."""
        keep = [list(r) for r in self.table], list(self.refs)
        free = iter([p for p, r in enumerate(self.refs) if r == 0])
        before, holders = list(self.refs), list(self.refs)
        src, dst = [-1] * len(grow), [-1] * len(grow)
        try:
            for s, g in enumerate(grow):
                if g <= 0:
                    continue
                n, row = self.lens[s], self.table[s]
                have, want = -(-n // self.page), -(-(n + g) // self.page)
                if n % self.page and holders[row[have - 1]] > 1:
                    src[s], dst[s] = row[have - 1], next(free)
                    holders[src[s]] -= 1
                    self.refs[src[s]] -= 1
                    row[have - 1] = dst[s]
                    self.refs[dst[s]] = 1
                for c in range(have, want):
                    if row[c] >= 0 and before[row[c]] > 1:      # another entry's too
                        self._drop(s, c)
                    if row[c] < 0:
                        row[c] = next(free)
                        self.refs[row[c]] = 1
        except StopIteration:
            self.table, self.refs = keep
            return None
        return src, dst

    def free(self, seqs):
        for s in seqs:
            for c in range(len(self.table[s])):
                self._drop(s, c)
            self.lens[s] = 0

    def evict(self, window, sinks):
        for s, n in enumerate(self.lens):
            for c in range(len(self.table[s])):
                if c * self.page >= sinks and (c + 1) * self.page <= n - window:
                    self._drop(s, c)

    def compact(self):
        """(src, dst, live)."""
        live = sum(r > 0 for r in self.refs)
        hole = [p for p in range(live) if self.refs[p] == 0]
        far = [p for p in range(live, len(self.refs)) if self.refs[p] > 0]
        to = dict(zip(far, hole))
        for a, b in to.items():
            self.refs[b], self.refs[a] = self.refs[a], 0
        self.table = [[to.get(p, p) for p in row] for row in self.table]
        pad = [-1] * (len(self.refs) - len(far))
        return far + pad, hole + pad, live
