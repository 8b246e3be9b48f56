"""The paged cache's operators in 64 bits, for the tests: row by row from their definitions, on
the host (numpy), sharing nothing with the library."""
from __future__ import annotations

import numpy as np

D = 128


def e4m3_values() -> np.ndarray:
    """The value of each of the 256 codes (NaN for 0x7f and 0xff)."""
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = (m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v[c] = np.nan if (c & 0x7f) == 0x7f else (-x if c & 0x80 else x)
    return v


VALUES = e4m3_values()


def quantise_row(x):
    """(codes uint8 [128], scale byte) of one row, by nearest value (ties: the even code)."""
    x = np.asarray(x, dtype=np.float64)
    if not np.all(np.isfinite(x)):
        return np.full(D, 0x7f, np.uint8), 255
    top = np.abs(x).max()
    e = -120
    while e < 119 and top > 448.0 * 2.0 ** e:
        e += 1
    y = np.minimum(np.abs(x) / 2.0 ** e, 448.0)
    grid = VALUES[:127]                                   # 0 .. 448, ascending with the code
    hi = np.searchsorted(grid, y)
    lo = np.maximum(hi - 1, 0)
    dl, dh = y - grid[lo], grid[hi] - y
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    return (code | np.where(np.signbit(x), 0x80, 0)).astype(np.uint8), e + 127


def dequantise(codes, byte):
    """Values [..., 128] of code rows [..., 128] with scale bytes [...]."""
    f = np.where(np.asarray(byte) == 255, np.nan, 2.0 ** (np.asarray(byte, np.float64) - 127))
    return VALUES[codes] * f[..., None]


def bf16_round(x):
    """fp32 values to the nearest bf16 (ties to even), as fp32."""
    u = np.ascontiguousarray(x, np.float32).view(np.uint32)
    r = ((u + 0x7fff + ((u >> 16) & 1)) & np.uint32(0xffff0000)).view(np.float32)
    return np.where(np.isnan(x), np.float32(np.nan), r)


class Cache:
    """Pages as values (float64 [pages, heads, page, 128]) plus tables; positions to slots."""

    def __init__(self, k, v, table, kv_len, q_start, max_q=1 << 30):
        self.k, self.v, self.table = k, v, table
        self.kv_len, self.q_start, self.max_q = kv_len, q_start, max_q
        self.page = k.shape[2]

    def slot(self, s, t):
        """(page, row) of position t of sequence s, or None."""
        if t < 0 or t >= self.table.shape[1] * self.page:
            return None
        p = int(self.table[s, t // self.page])
        return (p, t % self.page) if 0 <= p < self.k.shape[0] else None

    def tokens(self, s):
        n = min(int(self.kv_len[s]), self.table.shape[1] * self.page)
        return [t for t in range(max(n, 0)) if self.slot(s, t) is not None]

    def rows(self, s):
        """(row, position) of the new tokens of sequence s."""
        a, b = int(self.q_start[s]), int(self.q_start[s + 1])
        n = b - a
        return [(a + j, int(self.kv_len[s]) - n + j) for j in range(min(n, self.max_q))]


def attend(cache: Cache, q, group, scale, causal):
    """(out, lse, weight, reach): the attention of every new token in 64 bits; weight is
    sum_t p_t |v_t| (what relative errors of the weights multiply), reach the largest
    scale * sum_i |q_i k_i| of the row. Rows of no sequence stay NaN."""
    total, hq, _ = q.shape
    out = np.full((total, hq, D), np.nan)
    lse = np.full((total, hq), np.nan)
    weight = np.zeros((total, hq, D))
    reach = np.zeros((total, hq))
    for s in range(len(cache.kv_len)):
        toks = cache.tokens(s)
        slots = [cache.slot(s, t) for t in toks]
        toks = np.array(toks, dtype=np.int64)
        pi = np.array([p for p, _ in slots], dtype=np.int64)
        ri = np.array([r for _, r in slots], dtype=np.int64)
        rows = cache.rows(s)
        if not rows:
            continue
        row = np.array([r for r, _ in rows])
        pos = np.array([p for _, p in rows])
        see = toks[None, :] <= pos[:, None] if causal else np.ones((len(rows), len(toks)), bool)
        some = see.any(1)
        for h in range(cache.k.shape[1]):
            K, V = cache.k[pi, h, ri], cache.v[pi, h, ri]
            for g in range(group):
                i = h * group + g
                out[row[~some], i], lse[row[~some], i] = 0.0, -np.inf
                if not some.any():
                    continue
                r, m = row[some], see[some]
                x = np.where(m, q[r, i] @ K.T * scale, -np.inf)
                top = x.max(1, keepdims=True)
                p = np.exp(x - top)
                z = p.sum(1, keepdims=True)
                p /= z
                out[r, i] = p @ V
                lse[r, i] = (top + np.log(z))[:, 0]
                weight[r, i] = p @ np.abs(V)
                reach[r, i] = np.where(m, np.abs(q[r, i]) @ np.abs(K).T * abs(scale), 0).max(1)
    return out, lse, weight, reach


def tolerances(weight, reach, ref, n, out_bits, p_bits):
    """Bounds on out and lse by the roundings made. out_bits, p_bits: half steps of the output's
    type and of the weights' (2^-8: bf16, 2^-24: fp32 and 24-bit weights).
      scores: a dot product of 128 exact products in fp32, each addition off by at most a step
      (2^-23, if the unit truncates) of reach, times scale * log2(e) with two roundings: at most
      (128 + 8) * 2^-23 * reach; they enter the weights relatively, above and below the bar.
      exp2: 2 steps; rescalings to new maxima: one rounding and one exp2 a change, counted with
      the sums; sums of n weights, 16 at a time: n / 16 + 16 steps of at most the total."""
    score = (128 + 8) * 2.0 ** -23 * reach + 4 * 2.0 ** -23
    sums = (n / 16 + 16) * 2.0 ** -23
    rel = 2 * score + 2 * sums
    tol = weight * (rel[..., None] + p_bits) + np.abs(ref) * out_bits + 2.0 ** -126
    return tol, score + sums
