"""Plain 64-bit reference of the 4-bit cache, the attention over it, the token weights and
the eviction, in numpy, from their definitions; no code of the library."""

from __future__ import annotations

import numpy as np

DIM, GROUP = 128, 16


def scale_grid() -> np.ndarray:
    """The scales in ascending order: the fp16 numbers b << 7 up to 896."""
    g = (np.arange(248, dtype=np.uint16) << 7).view(np.float16).astype(np.float64)
    return g[g <= 896.0]


def nearest_even(grid: np.ndarray, x: np.ndarray) -> np.ndarray:
    """Index of the grid point nearest to x, the even index on a tie."""
    hi = np.clip(np.searchsorted(grid, x), 0, len(grid) - 1)
    lo = np.maximum(hi - 1, 0)
    a, b = np.abs(x - grid[lo]), np.abs(grid[hi] - x)
    return np.where(a < b, lo, np.where(b < a, hi, np.where(lo % 2 == 0, lo, hi)))


def quantise(x: np.ndarray):
    """Rows [n, 128] -> nibbles uint8 [n, 128] (q + 8) and scale bytes uint8 [n, 8].  A group
    with an infinity or a NaN: nibbles 8, byte 255."""
    g = x.astype(np.float64).reshape(len(x), -1, GROUP)
    bad = ~np.isfinite(g).all(-1)
    g = np.where(bad[..., None], 0.0, g)
    grid = scale_grid()
    # |x| / 7 against the grid: both sides times 7, which is exact
    byte = nearest_even(grid * 7, np.abs(g).max(-1))
    s = grid[byte][..., None]
    q = np.zeros(g.shape)
    for i in range(1, 8):  # |q| >= i where |x| is above (i - 1/2) s, or on it and i is even
        edge = (i - 0.5) * s
        q += (np.abs(g) > edge) | ((np.abs(g) == edge) & (i % 2 == 0) & (s > 0))
    q = np.where(s > 0, q * np.sign(g), 0.0)
    u = (q + 8).astype(np.uint8).reshape(len(x), DIM)
    return u, np.where(bad, 255, byte).astype(np.uint8)


def pack(ku, ks, vu, vs):
    """The cache rows uint8 [n, 128] and scales uint8 [n, 16]."""
    def half(u):
        return u[:, 0::2] | (u[:, 1::2] << 4)
    return np.concatenate([half(ku), half(vu)], 1), np.concatenate([ks, vs], 1)


def values(codes: np.ndarray, scales: np.ndarray):
    """Keys and values fp64 [n, 128] of cache rows."""
    out = []
    for h in range(2):
        c = codes[:, 64 * h:64 * h + 64]
        u = np.stack([c & 15, c >> 4], -1).reshape(len(c), DIM).astype(np.float64) - 8
        s = (scales[:, 8 * h:8 * h + 8].astype(np.uint16) << 7).view(np.float16)
        with np.errstate(invalid="ignore"):
            out.append(u * np.repeat(s.astype(np.float64), GROUP, 1))
    return out


class Attention:
    """Reference outputs and the sizes their tolerances go by, for every query row.

    out, lse; spread = sum_j softmax_j |v_j|; size = the largest scale * sum_d |q_d k_d|;
    weight[row, entry] = sum over the heads of the entry's softmax (0 where there is none)."""

    def __init__(self, q, k, v, idx, cu_q, cu_k, scale):
        n, heads = q.shape[:2]
        self.out = np.zeros((n, heads, DIM))
        self.spread = np.zeros((n, heads, DIM))
        self.lse = np.full((n, heads), -np.inf)
        self.size = np.zeros((n, heads))
        self.weight = np.zeros(idx.shape)
        self.rows = np.zeros(idx.shape, np.int64)
        for r in range(n):
            s = int(np.searchsorted(cu_q, r, side="right") - 1)
            at = np.flatnonzero(idx[r] >= 0)
            self.rows[r] = cu_k[s] + np.maximum(idx[r], 0)
            if not len(at):
                continue
            kr, qr = k[self.rows[r, at]], q[r].astype(np.float64)
            x = scale * (qr @ kr.T)
            self.size[r] = (abs(scale) * (np.abs(qr) @ np.abs(kr).T)).max(1)
            top = x.max(1, keepdims=True)
            p = np.exp(x - top)
            total = p.sum(1, keepdims=True)
            self.lse[r] = (top + np.log(total))[:, 0]
            p /= total
            self.weight[r, at] = p.sum(0)
            if v is not None:
                vr = v[self.rows[r, at]]
                self.out[r], self.spread[r] = p @ vr, p @ np.abs(vr)

    def totals(self, rows_k):
        """Accumulated weight per cache row, and how many times each row was added to."""
        w, n = np.zeros(rows_k), np.zeros(rows_k)
        np.add.at(w, self.rows.ravel(), self.weight.ravel())
        np.add.at(n, self.rows.ravel(), (self.weight > 0).ravel())
        return w, n

    # Errors.  A score: a sum of 128 exact products in fp32 (127 additions, each at most
    # 2^-23 of the sum of magnitudes, allowing for truncation) and its scaling by an fp32
    # factor (3 roundings), so 2^-16 of `size` covers it; the fast 2^x is off by 2^-22
    # relative and its argument's subtraction by 2^-24 of its magnitude, at most 2 size.
    def score_error(self):
        return self.size * (2.0 ** -16 + 2.0 ** -22) + 2.0 ** -21

    # A softmax weight is then off by twice that relative (numerator and denominator), the
    # sum of up to n terms in fp32 by n 2^-24 more; in the value product weights carry an
    # fp16 rounding (2^-11), or 2^-25 of the reference in its subnormal range for each of n
    # entries; products are exact and their fp32 sums covered by n 2^-23; the output is
    # rounded to bf16 (2^-8).
    def check_out(self, out, vmax):
        n = self.weight.shape[1]
        rel = 2.0 ** -11 + 2 * self.score_error() + n * 2.0 ** -22
        tol = 2.0 ** -8 * np.abs(self.out) + rel[..., None] * self.spread * (1 + 2.0 ** -8) \
            + n * 2.0 ** -24 * vmax
        # n 2^-24 vmax: the subnormal roundings, 2^-25 each, on both sides of bf16's step
        err = np.abs(out - self.out)
        assert np.all(err <= tol), float((err - tol).max())

    def check_lse(self, lse):
        none = np.isinf(self.lse)
        assert np.all(np.isneginf(lse[none]))
        tol = self.score_error() + self.weight.shape[1] * 2.0 ** -24 + \
            2.0 ** -21 * np.abs(np.where(none, 0, self.lse)) + 2.0 ** -20
        err = np.abs(np.where(none, 0, lse) - np.where(none, 0, self.lse))
        assert np.all(err <= tol), float((err - tol).max())

    # lse enters the weight: its error, and the score's, relative; half a unit per addition
    def check_weights(self, w, rows_k):
        ref, n = self.totals(rows_k)
        rel = 2 * float(self.score_error().max()) + self.weight.shape[1] * 2.0 ** -24 + \
            2.0 ** -20 * (1 + np.abs(self.lse[np.isfinite(self.lse)]).max(initial=0))
        err = np.abs(w * 2.0 ** -32 - ref)
        tol = rel * ref + n * 2.0 ** -33
        assert np.all(err <= tol), float((err - tol).max())


def evict_select(weights, length, keep, sink, recent):
    """Positions that stay, ascending."""
    if length <= keep:
        return np.arange(length)
    sink = min(sink, keep)
    recent = min(recent, keep - sink)
    stay = set(range(sink)) | set(range(length - recent, length))
    middle = sorted(range(sink, length - recent), key=lambda i: (-int(weights[i]), i))
    stay |= set(middle[:keep - sink - recent])
    return np.array(sorted(stay), dtype=np.int64)
