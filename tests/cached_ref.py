"""Plain 64-bit forms of the cached-decoding operators, for the GPU parity tests, and a
step-by-step model of the cache's book in Python integers."""
import numpy as np
import torch

BF16_HALF = 2.0 ** -8  # a bf16 rounding, relative to the value


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().double().cpu().numpy()


# ---------------------------------------------------------------- norm + rotation

def norm_rope(x, gamma, eps, positions, inv_freq, pairs):
    """x [M, heads, hd] fp64 -> (y, size): y the result, size what an absolute error scales with
    (the length of each rotated pair)."""
    hd, rot = x.shape[-1], 2 * len(inv_freq)
    if gamma is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * gamma
    y, size = x.copy(), np.abs(x)
    if rot:
        i0, i1 = (np.arange(0, rot, 2), np.arange(1, rot, 2)) if pairs else (np.arange(rot // 2), np.arange(rot // 2, rot))
        # the angle reduced in integers: position * (inv_freq / 2 pi) in units of 2^-80 turn
        turns = [int(np.floor(np.ldexp(f / (2 * np.pi), 80))) for f in inv_freq]
        a = np.array([[((int(p) * t) % (1 << 80)) / 2.0 ** 80 for t in turns] for p in positions]) * 2 * np.pi
        c, s = np.cos(a)[:, None, :], np.sin(a)[:, None, :]
        y[..., i0] = x[..., i0] * c - x[..., i1] * s
        y[..., i1] = x[..., i1] * c + x[..., i0] * s
        size[..., i0] = size[..., i1] = np.hypot(x[..., i0], x[..., i1])
    return y, size


def rope_tol(ref, size):
    """One rounding to bf16; before it the norm (2^-21 of the value: the sum, rsqrt and two
    products) and the rotation: sine and cosine within 2^-20.9 on [-pi, pi], the angle within
    2^-23 (pi times 2^-24, and 2^-32 turn), three fp32 operations. 2^-19 of the pair's length
    is above their sum."""
    return BF16_HALF * np.abs(ref) + 2.0 ** -19 * size + 1e-38


# ---------------------------------------------------------------- attention

def tree_attn(q, k, v, masks, scale):
    """q [T, n_q, hd]; k, v [len, n_kv, hd] with the block's T tokens last; masks: T integers.
    Returns (o, spread [T, n_q, hd] = sum p |v|)."""
    T, n_q, hd = q.shape
    n, n_kv = k.shape[0], k.shape[1]
    base, G = n - T, n_q // n_kv
    o, spread = np.zeros_like(q), np.zeros_like(q)
    for i in range(T):
        see = np.concatenate([np.arange(base), [base + j for j in range(T) if masks[i] >> j & 1]]).astype(int)
        if see.size == 0:
            continue
        for h in range(n_q):
            kk, vv = k[see, h // G], v[see, h // G]
            s = kk @ q[i, h] * scale
            p = np.exp(s - s.max())
            p /= p.sum()
            o[i, h] = p @ vv
            spread[i, h] = p @ np.abs(vv)
    return o, spread


def attn_tol(ref, spread):
    """The weights' rounding to bf16 (2^-8 each, numerator and sum both up to it) and the output's;
    scores in fp32 (hd products: under 2^-15 for the tests' score sizes, twice through the
    softmax)."""
    return (BF16_HALF + 2.0 ** -14) * spread + BF16_HALF * np.abs(ref) + 1e-38


# ---------------------------------------------------------------- log probabilities

def logprobs(x, targets, k):
    """x [M, N] fp64 -> logp, entropy, top_idx, top_logp by the header's definition."""
    M, N = x.shape
    logp = np.zeros(targets.shape)
    ent, idx, tlp = np.zeros(M), np.zeros((M, k), np.int64), np.zeros((M, k))
    for m in range(M):
        r = x[m]
        odd = bool(np.isnan(r).any() or np.isposinf(r).any())
        none = bool(np.isneginf(r).all())
        # NaN below every number, -0 as +0; ties to the lower index
        key = np.where(np.isnan(r), -np.inf, r) + 0.0
        order = np.lexsort((np.arange(N), np.where(np.isnan(r), 1, 0), -key))[:k]
        idx[m] = order
        if odd:
            lp = np.full(N, np.nan)
        elif none:
            lp = np.full(N, -np.inf)
        else:
            z = r - r.max()
            rest = np.sort(np.exp(z))[:-1].sum()  # the largest own 1 left out
            log_total = np.log1p(rest)
            lp = z - log_total
            with np.errstate(invalid="ignore"):
                ent[m] = -np.where(np.isneginf(lp), 0.0, np.exp(lp) * lp).sum()
        if odd:
            ent[m] = np.nan
        tlp[m] = lp[order]
        for i, t in enumerate(targets[m]):
            logp[m, i] = lp[t] if 0 <= t < N else (0.0 if t == -1 else np.nan)
    return logp, ent, idx, tlp


# ---------------------------------------------------------------- the book

class Book:
    """The cache's book and the tokens it stands for, in Python."""

    def __init__(self, n_seqs, n_pages, max_pages, page):
        self.page, self.max_pages = page, max_pages
        self.len, self.refs = [0] * n_seqs, [0] * n_pages
        self.table = [[-1] * max_pages for _ in range(n_seqs)]

    def flat(self):
        return self.len + self.refs + [p for r in self.table for p in r]

    def pages(self, n):
        return -(-n // self.page)

    def free(self):
        return [i for i, r in enumerate(self.refs) if r == 0]

    def slot(self, s, row):
        return self.table[s][row // self.page] * self.page + row % self.page

    def extend(self, seqs, rows):
        """The new rows' slots, or None: nothing done."""
        need = [self.pages(self.len[s] + r) - self.pages(self.len[s]) for s, r in zip(seqs, rows)]
        free = self.free()
        if any(self.pages(self.len[s] + r) > self.max_pages for s, r in zip(seqs, rows)) or sum(need) > len(free):
            return None
        at, slots = 0, []
        for s, r, n in zip(seqs, rows, need):
            first = self.pages(self.len[s])
            for i in range(n):
                self.table[s][first + i] = free[at]
                self.refs[free[at]] = 1
                at += 1
            slots += [self.slot(s, self.len[s] + j) for j in range(r)]
            self.len[s] += r
        return slots

    def fork(self, parent):
        """[(source page, fresh page, rows)], or None: nothing done."""
        free, copies, fresh = self.free(), [], {}
        keeper = {}
        for s, p in enumerate(parent):
            if p >= 0 and (p not in keeper or p == s):
                keeper[p] = s
        for s, p in enumerate(parent):
            if p >= 0 and p != s and self.len[p] % self.page and keeper[p] != s:
                if len(copies) >= len(free):
                    return None
                fresh[s] = free[len(copies)]
                copies.append((self.table[p][self.len[p] // self.page], fresh[s], self.len[p] % self.page))
        old_len, old = list(self.len), [list(r) for r in self.table]
        for s, p in enumerate(parent):
            if p == s:
                continue
            for a in old[s]:
                if a >= 0:
                    self.refs[a] -= 1
            self.len[s] = 0 if p < 0 else old_len[p]
            self.table[s] = [-1] * self.max_pages if p < 0 else list(old[p])
            if s in fresh:
                self.table[s][old_len[p] // self.page] = fresh[s]
            for a in self.table[s]:
                if a >= 0:
                    self.refs[a] += 1
        return copies

    def keep(self, s, rows, kept):
        """[(from row's slot, to row's slot)] of a sequence."""
        base = self.len[s] - rows
        moves = [(self.slot(s, base + k), self.slot(s, base + j)) for j, k in enumerate(kept)]
        for i in range(self.pages(base + len(kept)), self.pages(self.len[s])):
            self.refs[self.table[s][i]] = 0
            self.table[s][i] = -1
        self.len[s] = base + len(kept)
        return moves
