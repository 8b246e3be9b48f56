"""The paged K/V cache on the GPU (include/pariskv_paged.h) against 64-bit references: codes and
scale bytes exactly, read-back exactly, attention within bounds counted from its roundings."""
import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

import paged_reference as ref
from long_context_kv_srht_b200 import pariskv as pk

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
D = 128
SCALE = 1 / np.sqrt(D)


def _dev(a, dtype=None):
    return torch.tensor(np.ascontiguousarray(a), device=DEV, dtype=dtype)


def _bf(a):
    return _dev(ref.bf16_round(np.asarray(a, np.float32))).to(torch.bfloat16)


class Case:
    """A ragged batch with its pages in random order. q, kv: lengths; holes: (s, page) entries
    taken out of the table. Slots that hold no token are NaN (bf16) or NaN rows (8-bit)."""

    def __init__(self, seed, fmt, q, kv, heads=2, group=4, page=16, holes=(), width=None, spare=2,
                 tail=3, amp=1.0):
        rng = np.random.default_rng(seed)
        self.fmt, self.heads, self.group, self.page = fmt, heads, group, page
        self.q_len, self.kv = list(q), np.array(kv, np.int32)
        batch = len(q)
        self.width = width or max(1, max(-(-n // page) for n in kv))
        need = [min(self.width, -(-n // page)) for n in kv]
        self.pages = sum(need) + spare
        order = rng.permutation(self.pages)
        self.table = np.full((batch, self.width), -1, np.int32)
        at = 0
        for s in range(batch):
            self.table[s, :need[s]] = order[at:at + need[s]]
            at += need[s]
        for s, p in holes:
            self.table[s, p] = [-1, self.pages, -(1 << 31), (1 << 31) - 1][(s + p) % 4]
        self.q_start = np.concatenate([[0], np.cumsum(q)]).astype(np.int32)
        self.total = int(self.q_start[-1]) + tail          # rows behind the last sequence
        shape = (self.pages, heads, page, D)
        k = rng.standard_normal(shape).astype(np.float32) * amp
        k[..., rng.integers(0, D, 4)] *= 4
        v = rng.standard_normal(shape).astype(np.float32)
        self.q = ref.bf16_round(rng.standard_normal((self.total, heads * group, D)).astype(np.float32))
        self.live = np.zeros((self.pages, page), bool)
        c = ref.Cache(k, v, self.table, self.kv, self.q_start)
        for s in range(batch):
            for t in c.tokens(s):
                self.live[c.slot(s, t)] = True
        if fmt == "bf16":
            self.k, self.v = ref.bf16_round(k), ref.bf16_round(v)
            for x in (self.k, self.v):
                x[~np.broadcast_to(self.live[:, None], x.shape[:3])] = np.nan
            self.kd, self.vd = _dev(self.k).to(torch.bfloat16), _dev(self.v).to(torch.bfloat16)
            self.ks = self.vs = None
        else:
            (self.kc, self.kb), (self.vc, self.vb) = self._codes(k), self._codes(v)
            dead = ~np.broadcast_to(self.live[:, None], self.kb.shape)
            for codes, byte in ((self.kc, self.kb), (self.vc, self.vb)):
                codes[dead], byte[dead] = 0x7f, 255
            self.k, self.v = ref.dequantise(self.kc, self.kb), ref.dequantise(self.vc, self.vb)
            self.kd, self.vd = (_dev(x).view(torch.float8_e4m3fn) for x in (self.kc, self.vc))
            self.ks, self.vs = _dev(self.kb), _dev(self.vb)
        self.cfg = pk.config(batch=batch, num_kv_heads=heads, group=group, dtype="bf16")
        self.chunk = pk.Chunk(_dev(self.table), _dev(self.kv), _dev(self.q_start), self.total,
                              max(max(q), 1))

    @staticmethod
    def _codes(x):
        flat = [ref.quantise_row(r) for r in x.reshape(-1, D)]
        return (np.stack([c for c, _ in flat]).reshape(x.shape),
                np.array([b for _, b in flat], np.uint8).reshape(x.shape[:3]))

    def pool(self):
        return pk.Pages(self.kd, self.vd, self.ks, self.vs)

    def reference(self, causal, scale=SCALE):
        c = ref.Cache(np.float64(self.k), np.float64(self.v), self.table, self.kv, self.q_start)
        return ref.attend(c, np.float64(self.q), self.group, scale, causal)

    def check(self, out, lse, causal, scale=SCALE):
        o, l, w, reach = self.reference(causal, scale)
        f32 = out.dtype == torch.float32
        longest = max(len(ref.Cache(self.k, self.v, self.table, self.kv, self.q_start).tokens(s))
                      for s in range(len(self.q_len)))
        tol, ltol = ref.tolerances(w, reach, o, longest, 2.0 ** (-24 if f32 else -8),
                                   2.0 ** (-24 if f32 else -8))
        got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
        n = int(self.q_start[-1])
        assert np.isnan(got[n:]).all() and np.isnan(gl[n:]).all(), "rows of no sequence written"
        err = np.abs(got[:n] - o[:n])
        assert (err <= tol[:n]).all(), (err.max(), (err / tol[:n]).max(),
                                        np.argwhere(~(err <= tol[:n]))[:5])
        empty = np.isneginf(l[:n])
        assert (np.isneginf(gl[:n]) == empty).all()
        lerr = np.abs(np.where(empty, 0, gl[:n]) - np.where(empty, 0, l[:n]))
        assert (lerr <= ltol[:n] + 2.0 ** -24 * np.abs(np.where(empty, 0, l[:n]))).all(), lerr.max()


def _attend(c, causal=True, out_dtype=torch.bfloat16, q=None, chunk=None, scale=SCALE, pages=None):
    n, hq = c.total, c.heads * c.group
    out = torch.full((n, hq, D), float("nan"), dtype=out_dtype, device=DEV)
    lse = torch.full((n, hq), float("nan"), device=DEV)
    q = _bf(c.q) if q is None else q
    pk.paged_attend(c.cfg, pages or c.pool(), chunk or c.chunk, q, scale, causal=causal, out=out,
                    lse=lse)
    return out, lse


# ------------------------------------------------------------------------------- write, read
def _fresh(c):
    """An empty pool of c's shape, filled with a pattern."""
    k = torch.full(c.kd.shape, 1.5, device=DEV).to(c.kd.dtype)
    ks = None if c.ks is None else torch.full(c.ks.shape, 77, dtype=torch.uint8, device=DEV)
    return pk.Pages(k, k.clone(), ks, None if ks is None else ks.clone())


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("page,heads,q,kv,holes", [
    (16, 1, [1], [1], ()),
    (16, 2, [3, 0, 40, 1], [3, 17, 60, 33], ((2, 2),)),
    (64, 3, [65, 1, 130], [65, 64, 200], ()),
    (256, 5, [7, 300], [300, 301], ((1, 1),)),
    (32, 8, [10, 4], [6, 4], ()),                     # kv_len < q_len: positions below zero
])
def test_write_matches_definition(fmt, dtype, page, heads, q, kv, holes):
    c = Case(11, fmt, q, kv, heads=heads, group=1, page=page, holes=holes)
    rng = np.random.default_rng(5)
    new = rng.standard_normal((2, c.total, heads, D)).astype(np.float32)
    new *= 10.0 ** rng.integers(-6, 6, (2, c.total, heads, 1))
    new[0, 0, 0] = 0
    if dtype == "bf16":
        new = ref.bf16_round(new)
    c.cfg.dtype = pk.BF16 if dtype == "bf16" else pk.F32
    pages = _fresh(c)
    want = [t.clone().float().cpu().numpy() if t is not None and t.dtype != torch.uint8 else
            None if t is None else t.clone().cpu().numpy() for t in pages.tensors]
    cache = ref.Cache(np.zeros(c.kd.shape), None, c.table, c.kv, c.q_start)
    for s in range(len(q)):
        for row, pos in cache.rows(s):
            at = cache.slot(s, pos) if pos < c.kv[s] else None
            if at is None:
                continue
            for i in range(2):
                for h in range(heads):
                    if fmt == "bf16":
                        want[i][at[0], h, at[1]] = ref.bf16_round(new[i, row, h])
                    else:
                        code, byte = ref.quantise_row(new[i, row, h])
                        want[i][at[0], h, at[1]] = ref.VALUES[code]
                        want[2 + i][at[0], h, at[1]] = byte
    kn, vn = (_bf(x) if dtype == "bf16" else _dev(x) for x in new)
    pk.paged_write(c.cfg, pages, c.chunk, kn, vn)
    assert pk.last_launch_count() == 1
    for t, w in zip(pages.tensors, want):
        if t is not None:
            np.testing.assert_array_equal(t.float().cpu().numpy(), w)


def test_write_strides_special_rows_and_extremes():
    """Rows inside a wider tensor; rows with an infinity or NaN; the largest and least floats."""
    c = Case(3, "e4m3", [8], [8], heads=2, group=1, page=16)
    c.cfg.dtype = pk.F32
    rng = np.random.default_rng(2)
    wide = rng.standard_normal((c.total, 6, D)).astype(np.float32)
    wide[0, 0, 5], wide[1, 0, 7], wide[2, 1, 0] = np.inf, np.nan, -np.inf
    wide[3, 0], wide[3, 1] = 3.4e38, 1e-44
    wide[4, 0, 1:], wide[4, 0, 0] = 0, 448 * 2.0 ** 10
    wide[5, 0, 1:], wide[5, 0, 0] = 0, np.nextafter(np.float32(448 * 2.0 ** 10), np.float32(np.inf))
    wide[6, 0] = np.float32(2.0 ** -126) * np.arange(D)
    t = _dev(wide)
    pages = _fresh(c)
    pk.paged_write(c.cfg, pages, c.chunk, t[:, :2], t[:, 2:4])
    k, v, ks, vs = (x.float().cpu().numpy() for x in pages.tensors)
    for i in range(8):
        p = c.table[0, 0]
        for h in range(2):
            for got, gs, src in ((k, ks, wide[i, h]), (v, vs, wide[i, 2 + h])):
                code, byte = ref.quantise_row(src)
                assert gs[p, h, i] == byte
                np.testing.assert_array_equal(got[p, h, i], ref.VALUES[code])


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("page,kv,first,n,holes", [
    (16, [1], 0, 1, ()), (16, [50, 7, 0, 91], 5, 60, ((0, 1), (3, 5))),
    (128, [300, 129], 127, 200, ()), (256, [513], 250, 263, ((0, 1),)), (32, [40], 100, 8, ())])
def test_read_matches_pages(fmt, dtype, page, kv, first, n, holes):
    c = Case(7, fmt, [1] * len(kv), kv, heads=3, group=1, page=page, holes=holes)
    c.cfg.dtype = pk.BF16 if dtype == "bf16" else pk.F32
    td = torch.bfloat16 if dtype == "bf16" else torch.float32
    shape = (len(kv), 3, n + 5, D)
    K, V = (torch.full(shape, -7.0, dtype=td, device=DEV) for _ in range(2))
    pk.paged_read(c.cfg, c.pool(), c.chunk, first, n, K, V)
    wK, wV = np.full(shape, -7.0), np.full(shape, -7.0)
    cache = ref.Cache(np.float64(c.k), np.float64(c.v), c.table, c.kv, c.q_start)
    for s in range(len(kv)):
        for t in cache.tokens(s):
            if first <= t < first + n:
                p, r = cache.slot(s, t)
                wK[s, :, t - first], wV[s, :, t - first] = cache.k[p, :, r], cache.v[p, :, r]
    np.testing.assert_array_equal(K.float().cpu().numpy(), wK)
    np.testing.assert_array_equal(V.float().cpu().numpy(), wV)
    # slabs on 16 bytes but not on 32
    pad = 16 // K.element_size()
    both = [torch.full((K.numel() + pad,), -7.0, dtype=td, device=DEV)[pad:].view(shape) for _ in range(2)]
    assert all(t.data_ptr() % 32 == 16 for t in both)
    pk.paged_read(c.cfg, c.pool(), c.chunk, first, n, *both)
    assert torch.equal(both[0], K) and torch.equal(both[1], V)
    # one of the two alone, and into pinned host memory
    V2 = torch.full(shape, -7.0, dtype=td).pin_memory()
    pk.paged_read(c.cfg, c.pool(), c.chunk, first, n, V=V2)
    K2 = torch.full(shape, -7.0, dtype=td, device=DEV)
    pk.paged_read(c.cfg, c.pool(), c.chunk, first, n, K=K2)
    torch.cuda.synchronize()
    assert torch.equal(V2, V.cpu()) and torch.equal(K2, K)


# ------------------------------------------------------------------------------------ attend
LENGTHS = [
    ([1], [1]), ([1], [100]), ([1, 1, 1], [64, 65, 700]), ([3, 1, 0, 5], [3, 40, 12, 129]),
    ([17, 1], [17, 300]), ([40, 130], [90, 131]), ([200], [457]),
]


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("causal", [True, False], ids=["causal", "full"])
@pytest.mark.parametrize("q,kv", LENGTHS)
def test_attend_lengths(fmt, out_dtype, causal, q, kv):
    c = Case(sum(kv), fmt, q, kv, heads=2, group=4, page=32)
    out, lse = _attend(c, causal, out_dtype)
    c.check(out, lse, causal)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads,group", [(1, 1), (3, 2), (2, 3), (1, 5), (2, 7), (1, 8), (1, 12),
                                         (1, 16), (2, 40), (1, 128)])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_attend_head_layouts_and_pages(fmt, heads, group, page):
    c = Case(group * 31 + page, fmt, [1, 4, 33], [70, 4, 290], heads=heads, group=group, page=page)
    for out_dtype in (torch.bfloat16, torch.float32):   # (with tiles of 125 rows: group 5, fp32)
        out, lse = _attend(c, out_dtype=out_dtype)
        c.check(out, lse, True)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_attend_holes_empty_rows_and_positions_below_zero(fmt, out_dtype):
    """Pages given back (every kind of id that is none), rows whose whole past is gone, sequences
    shorter than their chunk, and a table too narrow for the length."""
    holes = [(0, p) for p in (0, 1, 2, 5, 9)] + [(1, 0), (2, 0), (2, 1), (2, 2)]
    c = Case(9, fmt, [6, 40, 3, 70, 2], [200, 33, 44, 300, 60], heads=2, group=3, page=16,
             holes=holes, width=16)
    for causal in (True, False):
        out, lse = _attend(c, causal, out_dtype)
        c.check(out, lse, causal)
    assert torch.isneginf(lse[c.q_start[2]:c.q_start[3]]).all()


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("q,kv", [([5], [70]), ([130], [140]), ([300], [300])])
def test_nan_and_inf_reach_only_rows_that_see_them(fmt, q, kv):
    """Tokens of the chunk itself hold NaN or infinity in K and V: earlier rows are exact."""
    c = Case(21, fmt, q, kv, heads=1, group=4, page=16)
    base, blse = _attend(c)
    at = kv[0] - q[0] // 2 - 1                       # a position inside the chunk
    p, r = c.table[0, at // 16], at % 16
    row = at - (kv[0] - q[0])                        # its row
    for which in ("v", "k"):
        x = getattr(c, which + "d").clone()
        sc = None if c.ks is None else (c.ks if which == "k" else c.vs).clone()
        if fmt == "bf16":
            x[p, 0, r, 3], x[p, 0, r, 100] = float("nan"), float("inf")
        else:
            x.view(torch.uint8)[p, 0, r], sc[p, 0, r] = 0x7f, 255
        pages = pk.Pages(x if which == "k" else c.kd, x if which == "v" else c.vd,
                         sc if which == "k" else c.ks, sc if which == "v" else c.vs)
        out, lse = _attend(c, pages=pages)
        n = q[0]
        assert torch.equal(out[:row], base[:row]) and torch.equal(lse[:row], blse[:row])
        seen = out[row:n].float()
        if which == "k":
            assert torch.isnan(seen).all() and not torch.isfinite(lse[row:n]).any()
        else:
            dims = [3, 100] if fmt == "bf16" else list(range(D))
            assert not torch.isfinite(seen[..., dims]).any()
            rest = [d for d in range(D) if d not in dims]
            assert torch.equal(out[row:n][..., rest], base[row:n][..., rest])
            assert torch.equal(lse[:n], blse[:n])


def test_large_scores_and_strided_q_and_interleaved_pool():
    """A saturated softmax, q as a slice of a fused projection, K and V side by side in one pool,
    a table with room behind it, negative and zero scales."""
    c = Case(4, "bf16", [9, 1], [200, 65], heads=2, group=4, page=32, amp=8.0)
    fused = torch.zeros((c.total, c.heads * (c.group + 2), D), dtype=torch.bfloat16, device=DEV)
    fused[:, :c.heads * c.group] = _bf(c.q)
    pool = torch.stack([c.kd, c.vd], 1)
    table = torch.full((2, c.width + 3), -5, dtype=torch.int32, device=DEV)
    table[:, :c.width] = _dev(c.table)
    chunk = pk.Chunk(table[:, :c.width], _dev(c.kv), _dev(c.q_start), c.total, 9)
    pages = pk.Pages(pool[:, 0], pool[:, 1])
    for scale in (3.0, SCALE, 0.0, -0.5):
        out, lse = _attend(c, out_dtype=torch.float32, q=fused[:, :c.heads * c.group], chunk=chunk,
                           scale=scale, pages=pages)
        c.check(out, lse, True, scale)


def test_rows_past_max_q_are_left_and_malformed_starts_stay_inside():
    c = Case(6, "bf16", [40, 2], [90, 2], heads=2, group=4, page=16)
    full, _ = _attend(c)
    short = pk.Chunk(_dev(c.table), _dev(c.kv), _dev(c.q_start), c.total, 7)
    out, lse = _attend(c, chunk=short)
    assert torch.equal(out[:7], full[:7]) and torch.isnan(out[7:40].float()).all()
    assert torch.equal(out[40:42], full[40:42])
    # starts that overlap, run backwards or leave the arrays: nothing outside is touched
    for starts in ([0, 45, 20], [40, 0, 45], [-5, 10, 1000], [30, 1 << 30, (1 << 31) - 1],
                   [-(1 << 31), (1 << 31) - 1, 0]):
        bad = pk.Chunk(_dev(c.table), _dev(c.kv), _dev(np.array(starts, np.int32)), c.total, 45)
        _attend(c, chunk=bad)
        kn = torch.zeros((c.total, 2, D), dtype=torch.bfloat16, device=DEV)
        pk.paged_write(c.cfg, _fresh(c), bad, kn, kn)
    torch.cuda.synchronize()


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("q", [[1, 2], [4, 1], [60, 1]])
@pytest.mark.parametrize("scale", [3.0, SCALE, 0.0, -0.5])
def test_saturated_zero_and_negative_scores(fmt, out_dtype, q, scale):
    """Scores up to hundreds apart and none apart, by every kernel and in every type."""
    c = Case(4, fmt, q, [200, 65], heads=2, group=4, page=32, amp=8.0)
    out, lse = _attend(c, out_dtype=out_dtype, scale=scale)
    c.check(out, lse, True, scale)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("rows", [1, 2, 4, 40])
def test_fp32_output_of_small_scores_and_few_tokens(fmt, rows):
    """Scores near zero, 60 tokens, V of every size and sign: what is left to be off is the weights'
    bits and the sums. In units of 2^-24 of sum p|v|: 48 for truncated sums (4 products of 16 tokens
    and three parts, 2 each: 24; and their alignment as much again), 2 * 20 for sums of 64 weights,
    warps and parts, 8 for exponentials, 4 for the division and the output, and scores off by 136 *
    2^-23 of their reach (below 2^-7), above and below the bar. In all less than half a step of
    weights of 16 bits (2^-17)."""
    c = Case(17, fmt, [rows], [60], heads=2, group=4, page=16)
    c.q = c.q * np.float32(2.0 ** -12)
    out, _ = _attend(c, False, torch.float32)
    o, _, w, reach = c.reference(False)
    assert reach.max() < 2.0 ** -7
    err = np.abs(out.double().cpu().numpy() - o)[:rows]
    tol = (w * (48 + 40 + 8 + 4 + 4 * 136 * reach[..., None]) * 2.0 ** -24)[:rows]
    assert (err <= tol).all(), (err / tol).max()


def _inside(t, margin):
    """A contiguous copy of t in the middle of a larger tensor of the same bytes' pattern 0xa5, and
    that larger tensor's bytes before and behind."""
    n = t.numel() * t.element_size()
    buf = torch.full((n + 2 * margin,), 0xa5, dtype=torch.uint8, device=DEV)
    x = buf[margin:margin + n].view(t.dtype).view(t.shape)
    x.copy_(t)
    return x, (buf[:margin], buf[margin + n:])


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("max_q", [2, 45])
@pytest.mark.parametrize("starts", [[0, 45, 20], [40, 0, 45], [-5, 10, 1000], [30, 1 << 30, (1 << 31) - 1],
                                    [-(1 << 31), (1 << 31) - 1, 0], [45, 45, 45], [3, 9, 4]])
def test_malformed_starts_touch_nothing_else(fmt, max_q, starts):
    """Outputs and pools lie inside larger buffers of a pattern: what no start covers, and all around,
    keeps it. A sequence covers rows [a, a + min(b - a, max_q, total - a)) (none if a < 0), at
    positions from kv_len - (b - a) on."""
    c = Case(6, fmt, [40, 2], [90, 2], heads=2, group=4, page=16)
    chunk = pk.Chunk(_dev(c.table), _dev(c.kv), _dev(np.array(starts, np.int32)), c.total, max_q)
    rows, slots = np.zeros(c.total, bool), np.zeros((c.pages, 16), bool)
    cache = ref.Cache(c.k, c.v, c.table, c.kv, c.q_start)
    for s in range(2):
        a, b = starts[s], starts[s + 1]
        n = 0 if a < 0 else max(0, min(b - a, max_q, c.total - a))
        rows[a:a + n] = True
        for j in range(n):
            pos = int(c.kv[s]) - max(0, b - a) + j
            if pos < c.kv[s] and cache.slot(s, pos) is not None:
                slots[cache.slot(s, pos)] = True
    free, margin = _dev(~rows), 1 << 16
    untouched = lambda around: all((x == 0xa5).all() for x in around)
    for out_dtype in (torch.bfloat16, torch.float32):
        out, around = _inside(torch.full((c.total, 8, D), -7.0, dtype=out_dtype, device=DEV), margin)
        lse, beside = _inside(torch.full((c.total, 8), -7.0, device=DEV), margin)
        pk.paged_attend(c.cfg, c.pool(), chunk, _bf(c.q), SCALE, out=out, lse=lse)
        assert untouched(around) and untouched(beside)
        assert (out[free] == -7).all() and (lse[free] == -7).all()
        assert (lse[~free] != -7).all()                  # and the rows covered are written
    pool, sides = zip(*(_inside(t, margin) for t in _fresh(c).tensors if t is not None))
    before = [t.clone() for t in pool]
    new = torch.ones((c.total, 2, D), dtype=torch.bfloat16, device=DEV)
    pk.paged_write(c.cfg, pk.Pages(*pool), chunk, new, new)
    free = _dev(~slots)
    for t, old, around in zip(pool, before, sides):
        assert untouched(around)
        kept = (t.view(torch.uint8) == old.view(torch.uint8)).reshape(*t.shape[:3], -1).all(-1)
        assert kept.transpose(1, 2)[free].all()
    pk.paged_sync()


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_same_bits_on_every_call_streams_and_graphs(fmt):
    """Twice in a row, on another stream, and from a captured graph that follows new lengths."""
    c = Case(12, fmt, [1, 1, 1], [900, 33, 400], heads=2, group=4, page=16)
    q = _bf(c.q)
    a, al = _attend(c, q=q)
    b, bl = _attend(c, q=q)
    assert torch.equal(a[:3], b[:3]) and torch.equal(al[:3], bl[:3])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b, bl = _attend(c, q=q)
    s.synchronize()
    assert torch.equal(a[:3], b[:3]) and torch.equal(al[:3], bl[:3])
    graphs, outs = [], []
    pages = c.pool()
    kv = c.chunk.tensors[1]
    for _ in range(2):                      # two graphs that live at once
        out, lse = torch.zeros_like(a), torch.zeros_like(al)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pk.paged_attend(c.cfg, pages, c.chunk, q, SCALE, out=out, lse=lse)
        graphs.append(g)
        outs.append((out, lse))
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for out, lse in outs:
        assert torch.equal(out[:3], a[:3]) and torch.equal(lse[:3], al[:3])
    kv.copy_(_dev(np.array([77, 20, 399], np.int32)))
    want, wl = _attend(c, q=q)
    graphs[1].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[1][0][:3], want[:3]) and torch.equal(outs[1][1][:3], wl[:3])


def test_many_sequences():
    """More sequences than the plan takes at once, lengths from zero on."""
    rng = np.random.default_rng(0)
    n = 1500
    q = rng.integers(0, 3, n).tolist()
    kv = [int(a + rng.integers(0, 40)) for a in q]
    c = Case(1, "e4m3", q, kv, heads=1, group=2, page=16)
    out, lse = _attend(c)
    c.check(out, lse, True)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("causal", [True, False], ids=["causal", "full"])
def test_many_tiles_a_cta(fmt, out_dtype, causal):
    """A ragged batch that gives each CTA many tiles one after the other: full ones, ones with few
    rows, ones without a single page, single blocks and long ones, in every order."""
    rng = np.random.default_rng(3)
    q = [int(rng.choice([1, 3, 33, 64, 70, 129])) for _ in range(48)]
    kv = [a + int(rng.choice([0, 5, 130, 700])) for a in q]
    holes = [(s, p) for s in range(0, 48, 5) for p in range((kv[s] + 31) // 32) if s % 10 or p % 3]
    c = Case(5, fmt, q, kv, heads=4, group=4, page=32, holes=holes)
    out, lse = _attend(c, causal, out_dtype)
    pk.paged_sync()
    c.check(out, lse, causal)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("rows", [1, 32])
def test_fp32_sums_do_not_shrink_over_a_long_range(fmt, rows):
    """2.4 million tokens (a few pages again and again), 128 blocks a CTA, V all of one sign and
    scores near zero: what truncating sums would take from the output grows with the range. The
    output is that of the pages once, lse more by ln of how often they come. Bound: at most 48
    truncated steps of 2^-23 in a row (2 blocks of 8 products of three parts), and roundings of
    2^-24: 256 turns' sums of 64 weights each (7 additions deep), 64 folds, 296 parts; exponentials
    2^-22, scores 2 * 136 * 2^-23 of at most 2^-7."""
    sms, page, few = torch.cuda.get_device_properties(0).multi_processor_count, 64, 64
    n = sms * 128 * 128 // (few * page)                  # times that the pages come
    gen = torch.Generator(device=DEV)
    gen.manual_seed(6)
    k = torch.randn((few, 1, page, D), device=DEV, generator=gen)
    v = 1 + 0.1 * torch.randn((few, 1, page, D), device=DEV, generator=gen)
    kind = torch.bfloat16 if fmt == "bf16" else torch.float8_e4m3fn
    k, v = k.to(kind), v.to(kind)
    one = torch.full((few, 1, page), 127, dtype=torch.uint8, device=DEV)
    pages = pk.Pages(k, v, *((one, one.clone()) if fmt == "e4m3" else ()))
    q = (torch.randn((rows, 4, D), device=DEV, generator=gen) * 2.0 ** -12).to(torch.bfloat16)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    table = torch.arange(few, dtype=torch.int32, device=DEV).repeat(n)[None].contiguous()
    chunk = pk.Chunk(table, ints([n * few * page]), ints([0, rows]), rows, rows)
    cfg = pk.config(batch=1, num_kv_heads=1, group=4, dtype="bf16")
    out, lse = pk.paged_attend(cfg, pages, chunk, q, SCALE, causal=False, want_lse=True,
                               out_dtype=torch.float32)
    x = torch.einsum("rhd,td->rht", q.double(), k.double().view(-1, D)) * SCALE
    want = x.softmax(-1) @ v.double().view(-1, D)
    rel = (48 + 2 * 136 * 2.0 ** -7 + 2) * 2.0 ** -23 + (256 + 7 + 64 + 296) * 2.0 ** -24
    assert ((out.double() - want).abs() <= rel * want.abs()).all()
    more = x.logsumexp(-1) + np.log(n)
    assert ((lse.double() - more).abs() <= (256 + 7 + 296 + 4) * 2.0 ** -24 + 2.0 ** -23 * more).all()


@pytest.mark.parametrize("rows", [1, 32])
def test_as_many_tokens_as_a_length_can_say(rows):
    """2^31 - 1 tokens of a few pages again and again, the last block ending 1 short: a row's output
    is that of the pages once, each token with the number of times that the row sees it. Weights
    near 1 are added up 2^18 times in a row at most, each time off by 2^-24 of the sum."""
    page, few, n = 256, 64, (1 << 31) - 1
    gen = torch.Generator(device=DEV)
    gen.manual_seed(8)
    k, v = (torch.randn((few, 1, page, D), device=DEV, generator=gen).to(torch.bfloat16)
            for _ in range(2))
    v[:, :, 200:] += 2
    q = (torch.randn((rows, 4, D), device=DEV, generator=gen) * 2.0 ** -6).to(torch.bfloat16)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    table = torch.arange(few, dtype=torch.int32, device=DEV).repeat((n + 1) // (few * page))[None]
    chunk = pk.Chunk(table.contiguous(), ints([n]), ints([0, rows]), rows, rows)
    cfg = pk.config(batch=1, num_kv_heads=1, group=4, dtype="bf16")
    out, lse = pk.paged_attend(cfg, pk.Pages(k, v), chunk, q, SCALE, want_lse=True,
                               out_dtype=torch.float32)
    pk.paged_sync()
    seen = n - rows + 1 + torch.arange(rows, device=DEV)                     # tokens a row sees
    often = seen[:, None] // (few * page) + \
        (torch.arange(few * page, device=DEV) < seen[:, None] % (few * page))
    x = torch.einsum("rhd,td->rht", q.double(), k.double().view(-1, D)) * SCALE
    x = x + often.double().log()[:, None]
    want, weight = (x.softmax(-1) @ y.double().view(-1, D) for y in (v, v.abs()))
    tol = 2.0 ** 18 * 2.0 ** -24
    assert ((out.double() - want).abs() <= 2 * tol * weight).all()
    assert ((lse.double() - x.logsumexp(-1)).abs() <= tol).all()


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads,n", [(8, 1600), (4, 1984)])
def test_masked_blocks_soon_after_a_cta_begins(fmt, heads, n):
    """Prompts whose ranges begin a few blocks before the end of a tile, so that a block that is
    masked and looked over for its V comes while the first copies are still under way, out of a
    cold L2 as well. Against the formula in 64 bits: one rounding of the output and one of the
    weights to bf16, and the same bits from every call."""
    rng = np.random.default_rng(n)
    page, width = 64, -(-n // 64)
    dt = torch.bfloat16
    k, v = (torch.randn((width, heads, page, D), device=DEV).to(dt) for _ in range(2))
    table = rng.permutation(width).astype(np.int32)
    if fmt == "bf16":
        pages, kf, vf = pk.Pages(k, v), k.double(), v.double()
    else:
        one = torch.full((width, heads, page), 127, dtype=torch.uint8, device=DEV)
        k, v = k.to(torch.float8_e4m3fn), v.to(torch.float8_e4m3fn)
        pages, kf, vf = pk.Pages(k, v, one, one.clone()), k.double(), v.double()
    chunk = pk.Chunk(_dev(table[None]), _dev(np.array([n], np.int32)), _dev(np.array([0, n], np.int32)),
                     n, n)
    cfg = pk.config(batch=1, num_kv_heads=heads, group=4, dtype="bf16")
    q = torch.randn((n, heads * 4, D), device=DEV).to(dt)
    order = torch.tensor(table.astype(np.int64), device=DEV)
    kf, vf = (x[order].permute(1, 0, 2, 3).reshape(heads, width * page, D)[:, :n] for x in (kf, vf))
    late = torch.ones((n, n), dtype=torch.bool, device=DEV).triu(1)
    want, weight = (torch.empty((n, heads * 4, D), dtype=torch.float64, device=DEV) for _ in range(2))
    for h in range(heads * 4):
        p = (q[:, h].double() @ kf[h // 4].T * SCALE).masked_fill(late, -np.inf).softmax(-1)
        want[:, h], weight[:, h] = p @ vf[h // 4], p @ vf[h // 4].abs()
    flush = torch.empty(1 << 28, dtype=torch.uint8, device=DEV)
    first = None
    for i in range(6):
        flush.fill_(i)
        out, _ = pk.paged_attend(cfg, pages, chunk, q, SCALE)
        # (the scores' part of the bound, 2 * 136 * 2^-23 of at most some 30, is below 2^-9)
        tol = 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -9) * weight
        assert ((out.double() - want).abs() <= tol).all()
        assert first is None or torch.equal(out, first)
        first = out


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("q,page", [([3, 2], 16), ([90, 33], 16), ([90, 33], 128)])
def test_long_caches_of_which_little_is_left(fmt, out_dtype, q, page):
    """Caches of some 300 000 tokens with a few pages here and there: first ones, whole stretches
    without any, single pages inside a block of 128 tokens, the last ones."""
    c = Case(13, fmt, q, [40 * page, 40 * page], heads=1, group=4, page=page)
    rng = np.random.default_rng(4)
    n = [300_000 // page, 270_000 // page]
    table = np.full((2, n[0]), -1, np.int32)
    for s in range(2):
        tail = np.arange(n[s] - 9, n[s])
        at = [0, 1, 5] if s == 0 else []
        at = np.concatenate([at, np.sort(rng.choice(np.arange(n[s] // 2, n[s] - 40),
                                                    31 - len(at), replace=False)), tail])
        table[s, at.astype(int)] = c.table[s, :40]
    c.table, c.kv = table, np.array([n[0] * page, n[1] * page], np.int32)
    c.chunk = pk.Chunk(_dev(table), _dev(c.kv), _dev(c.q_start), c.total, max(q))
    for causal in (True, False):
        out, lse = _attend(c, causal, out_dtype)
        c.check(out, lse, causal)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("q", [[2, 1], [140, 1]])
def test_outputs_on_16_bytes_and_two_streams_at_once(fmt, q):
    """Outputs that begin on 16 bytes but not on 32, and calls that overlap on two streams."""
    c = Case(31, fmt, q, [2000, 500], heads=2, group=4, page=64)
    qd, pages, n = _bf(c.q), c.pool(), c.total * 8 * D
    streams = [torch.cuda.Stream() for _ in range(2)]
    for out_dtype in (torch.bfloat16, torch.float32):
        want, wl = _attend(c, True, out_dtype, q=qd)
        pad = 16 // want.element_size()
        outs = []
        for i in range(8):
            buf = torch.full((n + pad,), float("nan"), dtype=out_dtype, device=DEV)
            lse = torch.full((c.total, 8), float("nan"), device=DEV)
            outs.append((buf[pad:].view(c.total, 8, D), lse))
            assert outs[-1][0].data_ptr() % 32 == 16
        torch.cuda.synchronize()
        for i, (out, lse) in enumerate(outs):
            with torch.cuda.stream(streams[i % 2]):
                pk.paged_attend(c.cfg, pages, c.chunk, qd, SCALE, out=out, lse=lse)
        torch.cuda.synchronize()
        rows = int(c.q_start[-1])
        for out, lse in outs:
            assert torch.equal(out[:rows], want[:rows]) and torch.equal(lse[:rows], wl[:rows])
            assert torch.isnan(out[rows:].float()).all()


_FIRST_IN_CAPTURE = """
import torch
from long_context_kv_srht_b200 import pariskv as pk
dev = "cuda:0"
torch.manual_seed(0)
k, v = (torch.randn(9, 2, 64, 128, device=dev).bfloat16() for _ in range(2))
ints = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
table, kv = ints([[3, 1, 4, 0, 5, 8, 2, 6]]), ints([500])
cfg, pages = pk.config(batch=1, num_kv_heads=2, group=4, dtype="bf16"), pk.Pages(k, v)
runs = []
for n in (1, 100):
    chunk = pk.Chunk(table, kv, ints([0, n]), n, n)
    q = torch.randn(n, 8, 128, device=dev).bfloat16()
    out = torch.zeros(n, 8, 128, device=dev).bfloat16()
    runs.append((chunk, q, out))
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    for chunk, q, out in runs:
        pk.paged_attend(cfg, pages, chunk, q, 0.1, out=out)
graph.replay()
torch.cuda.synchronize()
pk.paged_sync()
for chunk, q, out in runs:
    want, _ = pk.paged_attend(cfg, pages, chunk, q, 0.1)
    assert torch.equal(out, want) and out.abs().max() > 0
print("same")
"""


def test_first_call_of_a_process_inside_a_capture():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", _FIRST_IN_CAPTURE], capture_output=True, text=True,
                       timeout=300, cwd=root)
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stderr[-2000:]


def test_refusals_with_device_buffers():
    c = Case(2, "bf16", [2], [20], heads=2, group=4, page=16)
    q, pages = _bf(c.q), c.pool()
    host = torch.zeros((c.total, 2, D), dtype=torch.bfloat16)
    for bad in (host, host.pin_memory()):
        with pytest.raises(pk.PariskvError) as e:
            pk.paged_write(c.cfg, pages, c.chunk, bad, bad)
        assert e.value.status == pk.EINVAL and "device memory" in str(e.value)
    with pytest.raises(pk.PariskvError):
        pk.paged_attend(c.cfg, pages, c.chunk, q, float("nan"))
    f32 = pk.config(batch=1, num_kv_heads=2, group=4, dtype="f32")
    with pytest.raises(pk.PariskvError):
        pk.paged_attend(f32, pages, c.chunk, q, SCALE)
    odd = torch.zeros((c.total, 8, D + 1), dtype=torch.bfloat16, device=DEV)[..., 1:]
    with pytest.raises(pk.PariskvError):
        pk.paged_attend(c.cfg, pages, c.chunk, odd, SCALE)


@pytest.mark.parametrize("kind,status", [("alloc", pk.ENOMEM), ("launch", pk.ECUDA)])
def test_injected_failures_leave_outputs_alone(monkeypatch, kind, status):
    c = Case(2, "bf16", [2], [20], heads=2, group=4, page=16)
    out = torch.full((c.total, 8, D), 5.0, dtype=torch.bfloat16, device=DEV)
    monkeypatch.setenv("PARISKV_FAULT", kind)
    with pytest.raises(pk.PariskvError) as e:
        pk.paged_attend(c.cfg, c.pool(), c.chunk, _bf(c.q), SCALE, out=out)
    assert e.value.status == status
    monkeypatch.delenv("PARISKV_FAULT")
    assert (out == 5.0).all()
    pk.paged_attend(c.cfg, c.pool(), c.chunk, _bf(c.q), SCALE, out=out)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 200])
def test_a_wait_that_runs_out_reaches_the_caller(fmt, n):
    c = Case(8, fmt, [n], [300], heads=2, group=4, page=16)
    pk.paged_sync()
    pk.inject_paged_timeout()
    _attend(c)
    with pytest.raises(pk.PariskvError) as e:
        pk.paged_sync()
    assert e.value.status == pk.ETIMEOUT
    out, lse = _attend(c)                  # reported once; the next call is whole again
    pk.paged_sync()
    c.check(out, lse, True)


def _far_below(fmt, page, n, sinks, tail0, tail1, rng):
    """K and V pages [n / page, 1, page, D] in fmt and as values: tokens `sinks` score 0 for the
    queries of the tests below and have V = 0 in the first half of the elements and -1 in the
    others; the rest have K = (tail0, tail1[t]) in the first two elements, V in [1, 2)."""
    k = rng.integers(-8, 8, (n, D)).astype(np.float32) / 8         # (q is 0 there)
    k[:, 0], k[:, 1] = tail0, tail1
    v = 1 + rng.integers(0, 8, (n, D)).astype(np.float32) / 8
    k[sinks, :2] = 0
    v[sinks, :D // 2], v[sinks, D // 2:] = 0, -1
    kind = torch.bfloat16 if fmt == "bf16" else torch.float8_e4m3fn
    kd, vd = (_dev(x.reshape(-1, 1, page, D)).to(kind) for x in (k, v))
    assert torch.equal(kd.float().cpu().view(-1, D), torch.tensor(k))       # exact in both
    one = torch.full(kd.shape[:3], 127, dtype=torch.uint8, device=DEV)
    return pk.Pages(kd, vd, *((one, one.clone()) if fmt == "e4m3" else ())), k, v


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 2, 4, 40])
@pytest.mark.parametrize("n", [64, 320])
def test_weights_far_below_the_largest_keep_their_bits(fmt, out_dtype, rows, n):
    """A few tokens at score 0 that have V = 0 in half of the elements, and tokens of one score
    each row, down to 2^-30 of them: what is left in those elements is the small weights' alone.
    Scores are exact but for the factor scale * log2(e), so the bounds can be the weights': 24 bits
    (fp32) or 8 bits (bf16, down to 2^-24).
    In units of 2^-24 relative to sum p|v|: scores 3 roundings times their size times ln 2, and one
    of at most 16 where the weight's exponent is put together; two exponentials 4 each; the tensor
    cores' sums truncate, three parts every 16 tokens, for 256 tokens in a row at most (2 each);
    sums of 64 weights, warps and parts: n / 64 + 16, of weights and of O; the division and the
    output 2; the weight itself 1."""
    rng = np.random.default_rng(n + rows)
    pages, k, v = _far_below(fmt, 64, n, [0, 16, 32, 48], -1, -1, rng)
    f32 = out_dtype == torch.float32
    q = np.zeros((rows, 4, D), np.float32)
    q[..., 0] = rng.integers(0, 30 if f32 else 24, (rows, 4))
    q[0, 0, 0] = 0
    q[0, 1:, 0] = [8, 16, 29 if f32 else 23]
    q[..., 1] = rng.integers(0, 64, (rows, 4)) / 64
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    chunk = pk.Chunk(ints([list(range(n // 64))]), ints([n]), ints([0, rows]), rows, rows)
    cfg = pk.config(batch=1, num_kv_heads=1, group=4, dtype="bf16")
    scale = float(np.float32(np.log(2)))
    out, lse = pk.paged_attend(cfg, pages, chunk, _bf(q), scale, causal=False, want_lse=True,
                               out_dtype=out_dtype)
    x = np.float64(q) @ np.float64(k).T * scale
    p = np.exp(x)
    z = p.sum(-1, keepdims=True)
    want, weight = p / z @ v, p / z @ np.abs(v)
    size = np.abs(x).max(-1)[..., None]                      # (ln 2 is in it)
    rel = (3 * size + 16 * np.log(2) + 8 + 6 * min(n, 256) / 16 + 2 * (n / 64 + 16) + 3) * 2.0 ** -24
    tol = weight * rel if f32 else weight * (rel + 2.0 ** -8) + 2.0 ** -8 * np.abs(want)
    err = np.abs(out.double().cpu().numpy() - want)
    assert (err <= tol).all(), (err / tol).max()
    assert (np.abs(lse.double().cpu().numpy() - np.log(z[..., 0])) <= rel[..., 0]).all()


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 4])
def test_a_long_tail_far_below_the_largest_counts(out_dtype, rows):
    """131072 8-bit tokens, all but a few at the start with weights of 2^-26 to 2^-25.2 of theirs,
    in so many sequences that a CTA takes one from its start on: together the tail is 2^-11 of the
    output and more, and all of it where V of the few is 0.
    Bound in fp32: roundings of 2^-24, 2 blocks of 128 tokens a block and lane in the sums of the
    weights and 2 in those of O, 64 more for warps, parts and the rest; scores 3 times their size
    (they matter to the tail alone). In bf16: the output's rounding, and each weight's, 2^-8 of it or
    2^-32 of the largest, which are four."""
    rng = np.random.default_rng(rows)
    page, n, batch, heads = 64, 131072, 40, 8
    few = 4 * page
    pages, k, v = _far_below("e4m3", page, few, [0, 16, 32, 48], -26,
                             rng.integers(0, 8, few) / 8, rng)
    kd, vd, ks, vs = (x.expand(-1, heads, *x.shape[2:]).contiguous() for x in pages.tensors)
    pages = pk.Pages(kd, vd, ks, vs)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    table = [0] + [1 + i % 3 for i in range(n // page - 1)]  # the page of the few, then the others
    often = np.repeat(np.bincount(table), page).astype(np.float64)
    q = np.zeros((rows * batch, 4 * heads, D), np.float32)
    q[..., 0], q[..., 1] = 1, rng.choice([0.5, 0.75, 0.875], q.shape[:2])
    chunk = pk.Chunk(ints([table] * batch), ints([n] * batch),
                     ints([rows * i for i in range(batch + 1)]), rows * batch, rows)
    cfg = pk.config(batch=batch, num_kv_heads=heads, group=4, dtype="bf16")
    scale = float(np.float32(np.log(2)))
    out, _ = pk.paged_attend(cfg, pages, chunk, _bf(q), scale, causal=False, out_dtype=out_dtype)
    x = np.float64(q) @ np.float64(k).T * scale
    p = np.exp(x) * often
    z = p.sum(-1, keepdims=True)
    want, weight, tail = p / z @ v, p / z @ np.abs(v), p / z @ np.where(k[:, :1] == 0, 0, np.abs(v))
    assert (tail > 2.0 ** -11).all()
    tol = weight * (4 * (n / 128) + 64) * 2.0 ** -24 + 2 * tail * 3 * 26 * 2.0 ** -24
    if out_dtype == torch.bfloat16:
        tol += 2.0 ** -8 * (tail + np.abs(want)) + n * 2.0 ** -32 / 4 * np.abs(v).max()
    err = np.abs(out.double().cpu().numpy() - want)
    assert (err <= tol).all(), (err / tol).max()


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("rows", [1, 4, 40])
@pytest.mark.parametrize("high", [64, 128, 256, 1024])
@pytest.mark.parametrize("at", [3, 170, 299])
def test_one_token_far_above_the_rest_is_the_output(fmt, rows, high, at):
    """A token whose score is above all others' by 2^60 and more, scores of 2^10 to 2^14 and V of
    scales 2^-10 to 2^10 (8 bits): fp32 output is that token's V, however coarse the scores are. Its
    weight is the same number in both sums; left are the weight's 24 bits, the division, and at most
    6 steps of the sums it is in, 2^-24 each."""
    rng = np.random.default_rng(at + high)
    n, page = 300, 32
    k, v = rng.standard_normal((2, 320, D)).astype(np.float32)
    q = ref.bf16_round(rng.standard_normal((1, 1, D)).astype(np.float32)) * np.ones((rows, 4, 1), np.float32)
    k[at] = high * np.sign(q[0, 0])
    kd, vd = (_dev(x.reshape(10, 1, page, D)) for x in (k, v))
    if fmt == "bf16":
        pages = pk.Pages(kd.to(torch.bfloat16), vd.to(torch.bfloat16))
        kf, vf = (x.double().cpu().numpy().reshape(-1, D) for x in pages.tensors[:2])
    else:
        kb = np.full(320, 127, np.uint8)
        kb[at] = 127 + 2
        k[at] /= 4
        vb = rng.integers(117, 138, 320).astype(np.uint8)
        codes = [_dev(x.reshape(10, 1, page, D)).to(torch.float8_e4m3fn) for x in (k, v)]
        pages = pk.Pages(*codes, *(_dev(x.reshape(10, 1, page)) for x in (kb, vb)))
        kf, vf = (c.double().cpu().numpy().reshape(-1, D) * 2.0 ** (b.astype(np.float64) - 127)[:, None]
                  for c, b in zip(codes, (kb, vb)))
    x = kf[:n] @ q[0, 0].astype(np.float64) * SCALE / np.log(2)
    assert np.sort(x)[-1] - np.sort(x)[-2] > 60 and x[at] > 2.0 ** 9
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    chunk = pk.Chunk(ints([list(range(10))]), ints([n]), ints([0, rows]), rows, rows)
    cfg = pk.config(batch=1, num_kv_heads=1, group=4, dtype="bf16")
    out, lse = pk.paged_attend(cfg, pages, chunk, _bf(q), SCALE, causal=False, want_lse=True,
                               out_dtype=torch.float32)
    err = np.abs(out.double().cpu().numpy() - vf[at])
    assert (err <= 8 * 2.0 ** -24 * np.abs(vf[at]) + n * 2.0 ** -60 * np.abs(vf[:n]).max()).all(), \
        (err / np.abs(vf[at])).max()
    assert (np.abs(lse.double().cpu().numpy() - x[at] * np.log(2)) <= 2 * 136 * 2.0 ** -23 * x[at]).all()


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 4])
@pytest.mark.parametrize("big", [1 << e for e in range(22, 29)])
def test_maxima_whose_steps_are_as_wide_as_their_growth(out_dtype, rows, big):
    """8-bit pages whose blocks of 128 tokens score `big` and big + 8 (base 2) in turn, V = -1 and 1:
    the second is just not above what a maximum may lag by, where fp32 steps are 1/2 to 32. Scores
    are exact (scale * log2(e) is 1 in fp32) but for big + 8 being rounded to a step."""
    page, n, heads, batch = 128, 20, 8, 8
    scale = np.nextafter(np.float32(np.log(2)), np.float32(0))
    while np.float32(scale * np.float32(1.4426950408889634)) < 1:
        scale = np.nextafter(scale, np.float32(1))
    assert np.float32(scale * np.float32(1.4426950408889634)) == 1
    k, v = np.zeros((2, heads, page, D), np.float32), np.ones((2, heads, page, D), np.float32)
    k[..., 0], k[1, ..., 1] = 256, 2.0 ** -4                       # times 2^4
    v[0] = -1
    kd, vd = (_dev(x).to(torch.float8_e4m3fn) for x in (k, v))
    up = torch.full((2, heads, page), 127 + 4, dtype=torch.uint8, device=DEV)
    pages = pk.Pages(kd, vd, up, torch.full_like(up, 127))
    q = np.zeros((rows * batch, heads * 4, D), np.float32)
    q[..., 0], q[..., 1] = big / 4096, 8
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    chunk = pk.Chunk(ints([[i % 2 for i in range(n)]] * batch), ints([n * page] * batch),
                     ints([rows * i for i in range(batch + 1)]), rows * batch, rows)
    cfg = pk.config(batch=batch, num_kv_heads=heads, group=4, dtype="bf16")
    out, _ = pk.paged_attend(cfg, pages, chunk, _bf(q), float(scale), causal=False,
                             out_dtype=out_dtype)
    grown = np.float64(np.float32(big) + np.float32(8)) - big
    w = 2.0 ** grown
    tol = 2.0 ** -8 if out_dtype == torch.bfloat16 else 2.0 ** -16
    assert ((out.double() - (w - 1) / (w + 1)).abs() <= tol).all()


@pytest.mark.parametrize("n", [1, 200])
def test_of_two_threads_one_gets_the_report(n):
    """Two threads ask at once, on streams of their own, about one wait that ran out: it is reported
    once, and the next one again."""
    c = Case(8, "bf16", [n], [300], heads=2, group=4, page=16)
    streams = [torch.cuda.Stream() for _ in range(2)]
    pk.paged_sync()
    for _ in range(20):
        pk.inject_paged_timeout()
        _attend(c)
        torch.cuda.synchronize()
        gate, told = threading.Barrier(2), [None, None]

        def ask(i):
            torch.cuda.set_device(0)
            gate.wait()
            told[i] = pk.lib.pariskv_paged_sync(streams[i].cuda_stream)

        threads = [threading.Thread(target=ask, args=(i,)) for i in range(2)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        assert sorted(told) == [pk.OK, pk.ETIMEOUT]
    out, lse = _attend(c)
    pk.paged_sync()
    c.check(out, lse, True)


# ------------------------------------------------------------------------------- together
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_prompt_in_chunks_to_the_retrieval_index_and_decode(fmt):
    """As a serving program uses them: two prompts come in by chunks (write, attend), the pages are
    read back into slabs, the index is built from those, and decode steps write, attend over all
    pages, and search and attend sparsely over the slabs."""
    rng = np.random.default_rng(8)
    heads, group, page, n = 2, 4, 16, [700, 333]
    cap, steps = 720, 3
    width = -(-cap // page)
    x = rng.standard_normal((2, 2, heads, cap, D)).astype(np.float32)      # k, v by sequence
    x[0, ..., 5] *= 6
    x = ref.bf16_round(x)
    q = ref.bf16_round(rng.standard_normal((2, cap, heads * group, D)).astype(np.float32))
    dt = torch.bfloat16 if fmt == "bf16" else torch.float8_e4m3fn
    pool = [torch.zeros((2 * width + 1, heads, page, D), device=DEV).to(dt) for _ in range(2)]
    sc = [torch.zeros((2 * width + 1, heads, page), dtype=torch.uint8, device=DEV)
          for _ in range(2)] if fmt == "e4m3" else [None, None]
    pages = pk.Pages(pool[0], pool[1], sc[0], sc[1])
    table = _dev(rng.permutation(2 * width + 1)[:2 * width].reshape(2, width).astype(np.int32))
    cfg = pk.config(batch=2, num_kv_heads=heads, group=group, dtype="bf16", capacity=cap,
                    cand_bp=2000)
    if fmt == "bf16":
        kept = np.float64(x)
    else:
        rows = [ref.quantise_row(r) for r in x.reshape(-1, D)]
        kept = ref.dequantise(np.stack([c for c, _ in rows]),
                              np.array([b for _, b in rows])).reshape(x.shape)

    def step(done, take):
        """Write and attend take[s] new tokens of each sequence after done[s]."""
        starts = np.concatenate([[0], np.cumsum(take)]).astype(np.int32)
        total = int(starts[-1])
        kv = np.array([a + b for a, b in zip(done, take)], np.int32)
        chunk = pk.Chunk(table, _dev(kv), _dev(starts), total, max(take))
        k_new, v_new = (np.concatenate([x[i, s, :, done[s]:kv[s]].transpose(1, 0, 2)
                                        for s in range(2)]) for i in range(2))
        qs = np.concatenate([q[s, done[s]:kv[s]] for s in range(2)])
        pk.paged_write(cfg, pages, chunk, _bf(k_new), _bf(v_new))
        out, lse = pk.paged_attend(cfg, pages, chunk, _bf(qs), SCALE, want_lse=True)
        cache = ref.Cache(kept[0], kept[1], np.arange(2, dtype=np.int32)[:, None], kv, starts)
        cache.k, cache.v, cache.page = kept[0], kept[1], cap          # a sequence is a page here
        o, l, w, reach = ref.attend(cache, np.float64(qs), group, SCALE, True)
        tol, ltol = ref.tolerances(w, reach, o, int(kv.max()), 2.0 ** -8, 2.0 ** -8)
        assert (np.abs(out.double().cpu().numpy() - o) <= tol).all()
        assert (np.abs(lse.double().cpu().numpy() - l) <= ltol + 2.0 ** -24 * np.abs(l)).all()
        return chunk, out

    done = [0, 0]
    for take in ([256, 200], [256, 133], [188, 0]):
        chunk, _ = step(done, take)
        done = [a + b for a, b in zip(done, take)]
    assert done == n
    K, V = (torch.zeros((2, heads, cap, D), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    pk.paged_read(cfg, pages, chunk, 0, cap, K, V)
    for got, want in ((K, kept[0]), (V, kept[1])):
        for s in range(2):
            np.testing.assert_array_equal(got[s, :, :n[s]].double().cpu().numpy(), want[s, :, :n[s]])
            assert (got[s, :, n[s]:] == 0).all()
    # the index of the slabs is the index of the rows themselves
    signs = np.where(rng.integers(0, 2, D) == 1, -1, 1).astype(np.int8)
    m = min(n)
    ix = pk.build_index(cfg, signs, K, n=m)
    direct = pk.build_index(cfg, signs, _bf(kept[0][:, :, :m]))
    for a, b in zip(ix.export_index(), direct.export_index()):
        np.testing.assert_array_equal(a, b)
    for _ in range(steps):
        chunk, out = step(done, [1, 1])
        done = [a + 1 for a in done]
    # all rows retrieved, the sparse attention over the slabs is the paged one over those rows
    top, _ = ix.search(_bf(q[:, n[0]][:, :]).contiguous(), m)
    assert (torch.sort(top, 1).values == torch.arange(m, device=DEV)).all()
    qd = _bf(q[:, n[0]]).contiguous()
    sparse = pk.sparse_attend(cfg, qd, K, V, top, m, SCALE, n=m, out_dtype=torch.float32)
    last = pk.Chunk(table, _dev(np.full(2, m, np.int32)), _dev(np.arange(3, dtype=np.int32)), 2, 1)
    dense = pk.dense_attend(cfg, qd, K, V, SCALE, n=m, out_dtype=torch.float32)
    paged, _ = pk.paged_attend(cfg, pages, last, qd, SCALE, out_dtype=torch.float32)
    # of each of the two that are compared: 16 bits of a weight (half a step: 2^-17), scores off by
    # 136 * 2^-23 of their reach, above and below the bar, sums of m weights, 16 at a time
    reach = SCALE * max(float(np.einsum("hd,td->ht", np.abs(q[s, n[0], 4 * h:4 * h + 4]),
                                        np.abs(kept[0][s, h, :m])).max())
                        for s in range(2) for h in range(heads))
    bound = 2 * (2.0 ** -17 + 2 * 136 * 2.0 ** -23 * reach + 2 * (m / 16 + 16) * 2.0 ** -23)
    bound *= float(V[:, :, :m].abs().max())
    assert (dense - paged).abs().max() <= bound and (sparse - paged).abs().max() <= bound
