"""References of the serving operators' tests: attention of given (row, key) pairs in 64 bits
with the error its rounding steps allow, and the pages of a cache as a program of one request
after the other.

Error of the kernels, from their roundings (half a step each: bf16 2^-8, fp32 2^-24):
- a score is a sum of d products accumulated in fp32 by the matrix unit, which may truncate
  (a whole step, 2^-23, per addition), then scaled: at most (d + 8) 2^-23 * scale *
  sum_c |q_c k_c| off, called ds below;
- a weight p = exp(s - m) is off by ds and by the exponential's error (2^-21 is above the
  special-function unit's and the polynomial's), and is rounded to bf16 for P V: 2^-8;
  the sum keeps the unrounded p;
- so out is off by at most sum_j w_j |v_j| (2^-8 + 2 (exp(ds) - 1) + 2^-20), with fp32
  accumulation of P V within 2^-23 per key (L 2^-23), and bf16 output adds 2^-8 |out|;
- lse = m + log l is off by ds + 2^-20 and its own fp32 steps, 2^-22 (|lse| + 1);
- joining key splits adds a few fp32 steps to both, inside the same terms.
"""
import numpy as np


def attn(q, k, v, see, scale):
    """One sequence: q [S, Hq, d], k and v [L, Hk, d] in 64 bits, see [S, L] truth values.
    Returns out [S, Hq, d], lse [Hq, S] and the allowed errors of both (fp32 output)."""
    S, Hq, d = q.shape
    L, Hk = k.shape[0], k.shape[1]
    g = Hq // Hk
    out = np.zeros((S, Hq, d))
    lse = np.full((Hq, S), -np.inf)
    tol, ltol = np.zeros((S, Hq, d)), np.zeros((Hq, S))
    for h in range(Hq if L else 0):
        kk, vv = k[:, h // g], v[:, h // g]
        x = np.where(see, scale * (q[:, h] @ kk.T), -np.inf)
        ds = (d + 8) * 2.0 ** -23 * abs(scale) * np.where(see, np.abs(q[:, h]) @ np.abs(kk).T, 0).max(1)
        any_ = see.any(1)
        m = np.where(any_, x.max(1), 0.0)
        p = np.where(see, np.exp(x - m[:, None]), 0.0)
        l = p.sum(1)
        w = p / np.where(l > 0, l, 1.0)[:, None]
        vz = np.where(see.any(0)[:, None], vv, 0.0)  # keys that nobody sees may hold anything
        out[:, h] = w @ vz
        tol[:, h] = (w @ np.abs(vz)) * (2.0 ** -8 + 2 * np.expm1(ds) + 2.0 ** -20 + L * 2.0 ** -23)[:, None]
        lse[h] = np.where(any_, m + np.log(np.where(l > 0, l, 1.0)), -np.inf)
        ltol[h] = ds + 2.0 ** -20 + 2.0 ** -22 * (np.abs(np.where(any_, lse[h], 0.0)) + 1)
    return out, lse, tol, ltol


def check(got_out, got_lse, out, lse, tol, ltol, bf16=False, what=""):
    got_out, got_lse = got_out.double().cpu().numpy(), got_lse.double().cpu().numpy()
    assert np.isfinite(got_out).all(), f"{what}: non-finite output"
    empty = np.isneginf(lse)
    assert np.array_equal(empty, np.isneginf(got_lse)), f"{what}: rows without keys differ"
    if bf16:
        tol = tol + 2.0 ** -8 * (np.abs(out) + tol)
    err = np.abs(got_out - out) - tol
    assert err.max(initial=-1) <= 1e-30, f"{what}: out {err.max()} above its tolerance"
    zero = np.where(empty, 0.0, 0.0)
    lerr = np.abs(np.where(empty, zero, got_lse) - np.where(empty, zero, lse)) - ltol
    assert lerr.max(initial=-1) <= 1e-30, f"{what}: lse {lerr.max()} above its tolerance"


def causal(S, L):
    return np.arange(L)[None, :] <= np.arange(S)[:, None] + (L - S)


DONE, NO_PAGES, INVALID, SHARED = 0, 1, 2, 3


class Pages:
    """A cache's pages, kept by the rules of the calls' documentation, one request at a time.
    rows: the pools as an array [layers, num_pages, page_size, x] per tensor (or none)."""

    def __init__(self, S, M, P, ps, pools=()):
        self.S, self.M, self.P, self.ps = S, M, P, ps
        self.table = np.full((S, M), -1, dtype=np.int64)
        self.lens = np.zeros(S, dtype=np.int64)
        self.refs = np.zeros(P, dtype=np.int64)
        self.pools = list(pools)

    def pages(self, n):
        return -(-int(n) // self.ps)

    def give_up(self, s, lo, hi):
        for j in range(lo, hi):
            if 0 <= self.table[s, j] < self.P:
                self.refs[self.table[s, j]] -= 1
            self.table[s, j] = -1

    def take(self, wants):
        """wants: (request, slot, first entry, pages); returns the requests that got theirs."""
        free, used, got = np.flatnonzero(self.refs == 0), 0, set()
        asked = 0
        for i, s, first, need in wants:
            asked += need
            if need and asked > len(free):
                continue
            for j in range(need):
                self.table[s, first + j] = free[used + j]
                self.refs[free[used + j]] = 1
            used += need
            got.add(i)
        return got

    def resize(self, slots, new_lens):
        st, wants, seen = [DONE] * len(slots), [], set()
        act = []
        for i, (s, m) in enumerate(zip(slots, new_lens)):
            if not 0 <= s < self.S or s in seen or not 0 <= m <= self.M * self.ps:
                st[i] = INVALID
            elif m != self.lens[s]:
                stay = min(m, self.lens[s])
                if stay % self.ps and self.refs[self.table[s, stay // self.ps]] > 1:
                    st[i] = SHARED
            seen.add(s)
            if st[i] == DONE:
                act.append(i)
        for i in act:
            self.give_up(slots[i], self.pages(new_lens[i]), self.pages(self.lens[slots[i]]))
        for i in act:
            had = self.pages(self.lens[slots[i]])
            wants.append((i, slots[i], had, max(self.pages(new_lens[i]) - had, 0)))
        got = self.take(wants)
        for i in act:
            if i in got:
                self.lens[slots[i]] = new_lens[i]
            else:
                st[i] = NO_PAGES
        return st

    def fork(self, parents, children):
        st, seen = [DONE] * len(parents), set()
        act = []
        for i, (p, c) in enumerate(zip(parents, children)):
            ok = 0 <= p < self.S and 0 <= c < self.S and c not in seen and (p == c or c not in parents)
            seen.add(c)
            if not ok:
                st[i] = INVALID
            elif p != c:
                act.append(i)
        for i in act:
            self.give_up(children[i], 0, self.pages(self.lens[children[i]]))
        wants = []
        for i in act:
            p, c = parents[i], children[i]
            whole = int(self.lens[p]) // self.ps
            self.table[c, :whole] = self.table[p, :whole]
            self.refs[self.table[p, :whole]] += 1
            wants.append((i, c, whole, self.pages(self.lens[p]) - whole))
        got = self.take(wants)
        for i, c, whole, need in wants:
            p = parents[i]
            if i not in got:
                st[i] = NO_PAGES
                self.give_up(c, 0, whole)
                self.lens[c] = 0
                continue
            self.lens[c] = self.lens[p]
            if need:
                tail = int(self.lens[p]) % self.ps
                for x in self.pools:
                    x[:, self.table[c, whole], :tail] = x[:, self.table[p, whole], :tail]
        return st

    def compact(self, keep, keep_lens, tree_lens):
        S, T = len(keep), len(keep[0])
        st, plan = [DONE] * S, []
        for s in range(S):
            L = int(self.lens[s])
            n = min(max(T if tree_lens is None else int(tree_lens[s]), 0), min(T, L))
            m, base = int(keep_lens[s]), L - n
            path = list(keep[s][:max(m, 0)])
            if not 0 <= m <= n or any(not 0 <= x < n for x in path) or any(a >= b for a, b in zip(path, path[1:])):
                st[s] = INVALID
            elif any(self.refs[self.table[s, j]] > 1 for j in range(base // self.ps, self.pages(base + m))):
                st[s] = SHARED
            else:
                plan.append((s, L, base, path))
        for s, L, base, path in plan:
            at = lambda pos: (self.table[s, pos // self.ps], pos % self.ps)  # noqa: E731
            for x in self.pools:
                rows = [x[:, at(base + i)[0], at(base + i)[1]].copy() for i in path]
                for j, r in enumerate(rows):
                    x[:, at(base + j)[0], at(base + j)[1]] = r
            self.give_up(s, self.pages(base + len(path)), self.pages(L))
            self.lens[s] = base + len(path)
        return st
