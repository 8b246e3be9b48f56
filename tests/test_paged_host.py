"""Refusals of the paged cache's calls that need no GPU, and its 64-bit reference against torch's
own 8-bit type."""
import ctypes

import numpy as np
import pytest
import torch

import paged_reference as ref
from long_context_kv_srht_b200 import pariskv as pk


def _raw(fmt="bf16", **kw):
    p = pk._Pages(4096, 4096, 4096, 4096, 8, 2 * 16 * 128, 2 * 16, 16,
                  pk.PAGES_E4M3 if fmt == "e4m3" else pk.PAGES_BF16)
    c = pk._Chunk(4096, 4096, 4096, 4, 3, 3, 4)
    for k, v in kw.items():
        setattr(p if hasattr(p, k) else c, k, v)
    return p, c


def _calls(cfg, p, c, q_ld=8 * 128, ld=2 * 128, first=0, n=4, ld_tok=4, scale=0.1, out=0):
    cf, pp, cc = (ctypes.byref(x) for x in (cfg, p, c))
    return (pk.lib.pariskv_paged_write(cf, pp, cc, 4096, 4096, ld, ld, None),
            pk.lib.pariskv_paged_read(cf, pp, cc, first, n, 4096, 4096, ld_tok, None),
            pk.lib.pariskv_paged_attend(cf, pp, cc, 4096, q_ld, scale, 1, 4096, out, None, None))


CFG = dict(batch=1, num_kv_heads=2, group=4)


@pytest.mark.parametrize("fmt,bad", [
    ("bf16", dict(format=2)), ("bf16", dict(page_size=8)), ("bf16", dict(page_size=48)),
    ("bf16", dict(page_size=512)), ("bf16", dict(num_pages=0)), ("bf16", dict(num_pages=1 << 31)),
    ("bf16", dict(page_stride=2 * 16 * 128 - 8)), ("bf16", dict(page_stride=2 * 16 * 128 + 4)),
    ("e4m3", dict(page_stride=2 * 16 * 128 + 8)), ("e4m3", dict(scale_stride=16)),
    ("e4m3", dict(scale_stride=40)), ("bf16", dict(table_width=0)),
    ("bf16", dict(table_stride=2)), ("bf16", dict(total_q=-1)), ("bf16", dict(total_q=1 << 31)),
    ("bf16", dict(max_q=-1))])
def test_bad_descriptions_are_refused_by_every_call(fmt, bad):
    p, c = _raw(fmt, **bad)
    assert _calls(pk.config(**CFG), p, c) == (pk.EINVAL,) * 3, bad
    assert pk.last_error()


def test_bad_arguments_are_refused():
    p, c = _raw()
    cfg = pk.config(**CFG)
    lib, b = pk.lib, ctypes.byref
    assert lib.pariskv_paged_write(b(cfg), None, b(c), 1, 1, 256, 256, None) == pk.EINVAL
    assert lib.pariskv_paged_write(b(cfg), b(p), None, 1, 1, 256, 256, None) == pk.EINVAL
    assert lib.pariskv_paged_write(None, b(p), b(c), 1, 1, 256, 256, None) == pk.EINVAL
    for ld in (128, 260):                                    # too short, not whole words
        assert _calls(cfg, p, c, ld=ld)[0] == pk.EINVAL
    for kw in (dict(first=-1), dict(n=-1), dict(ld_tok=3), dict(first=1 << 31)):
        assert _calls(cfg, p, c, **kw)[1] == pk.EINVAL
    assert lib.pariskv_paged_read(b(cfg), b(p), b(c), 0, 4, None, None, 4, None) == pk.EINVAL
    for kw in (dict(q_ld=8 * 128 - 8), dict(q_ld=8 * 128 + 4), dict(scale=float("nan")),
               dict(out=7)):
        assert _calls(cfg, p, c, **kw)[2] == pk.EINVAL
    assert _calls(pk.config(**CFG, dtype="f32"), p, c)[2] == pk.EINVAL
    wide = pk.config(batch=1, num_kv_heads=2, group=129)
    assert _calls(wide, p, c, q_ld=2 * 129 * 128)[2] == pk.EINVAL
    p, c = _raw(total_q=(1 << 31) - 1)
    assert _calls(cfg, p, c)[2] == pk.EINVAL                 # rows past 2^31


def test_binding_refuses_what_does_not_fit():
    bf, e4, u8, i32 = torch.bfloat16, torch.float8_e4m3fn, torch.uint8, torch.int32
    k = torch.zeros(4, 2, 16, 128, dtype=bf)
    s = torch.zeros(4, 2, 16, dtype=u8)
    for args in ((k, k.float()), (k.float(), k.float()), (k, k[:3]), (k[..., :64], k[..., :64]),
                 (k, k, s, s), (k.to(e4), k.to(e4)), (k.to(e4), k.to(e4), s, None),
                 (k.to(e4), k.to(e4), s, s[:, :1]), (k.to(e4), k.to(e4), s.int(), s),
                 (k.transpose(1, 2), k.transpose(1, 2)), (k, torch.zeros(8, 2, 16, 128, dtype=bf)[::2])):
        with pytest.raises(pk.PariskvError) as e:
            pk.Pages(*args)
        assert e.value.status == pk.EINVAL
    pool = torch.zeros(4, 2, 2, 16, 128, dtype=bf)
    assert pk.Pages(pool[:, 0], pool[:, 1]).raw.page_stride == 2 * 2 * 16 * 128
    t, n, q = torch.zeros(2, 3, dtype=i32), torch.zeros(2, dtype=i32), torch.zeros(3, dtype=i32)
    for args in ((t.long(), n, q), (t, n.long(), q), (t, n, q[:2]), (t, n[:1], q), (t[0], n, q),
                 (t.T.contiguous().T, n, q)):
        with pytest.raises(pk.PariskvError):
            pk.Chunk(*args, 4, 2)
    pages, chunk = pk.Pages(k, k), pk.Chunk(t, n, q, 4, 2)
    cfg = pk.config(batch=2, num_kv_heads=2, group=4)
    x = torch.zeros(4, 2, 128, dtype=bf)
    y = torch.zeros(4, 8, 128, dtype=bf)
    slab = torch.zeros(2, 2, 9, 128, dtype=bf)
    for call in (lambda: pk.paged_write(pk.config(batch=1, num_kv_heads=2), pages, chunk, x, x, 0),
                 lambda: pk.paged_write(pk.config(batch=2, num_kv_heads=3), pages, chunk, x, x, 0),
                 lambda: pk.paged_write(cfg, pages, chunk, x.float(), x, 0),
                 lambda: pk.paged_write(cfg, pages, chunk, x[:3], x, 0),
                 lambda: pk.paged_write(cfg, pages, chunk, x, x.transpose(0, 1), 0),
                 lambda: pk.paged_read(cfg, pages, chunk, 0, 10, slab, slab, 0),
                 lambda: pk.paged_read(cfg, pages, chunk, 0, 9, slab.float(), None, 0),
                 lambda: pk.paged_read(cfg, pages, chunk, 0, 3, slab, slab[:, :, :5].contiguous(), 0),
                 lambda: pk.paged_attend(cfg, pages, chunk, x, 1.0, stream=0),
                 lambda: pk.paged_attend(cfg, pages, chunk, y.float(), 1.0, stream=0),
                 lambda: pk.paged_attend(cfg, pages, chunk, y, 1.0, out=y[:2], stream=0),
                 lambda: pk.paged_attend(cfg, pages, chunk, y, 1.0, lse=y, stream=0)):
        with pytest.raises(pk.PariskvError) as e:
            call()
        assert e.value.status == pk.EINVAL


def test_reference_rows_agree_with_the_8_bit_type():
    """The reference's codes are torch's conversion of x / 2^e, and e is the least that fits."""
    rng = np.random.default_rng(0)
    for i in range(300):
        x = (rng.standard_normal(128) * 10.0 ** rng.integers(-30, 30)).astype(np.float32)
        if i % 3 == 0:
            x = ref.bf16_round(x)
        code, byte = ref.quantise_row(x)
        e = byte - 127
        y = torch.tensor(np.float64(x) / 2.0 ** e).float()
        assert np.array_equal(y.to(torch.float8_e4m3fn).view(torch.uint8).numpy(), code)
        top = np.abs(np.float64(x)).max()
        assert top <= 448 * 2.0 ** e and top > 448 * 2.0 ** (e - 1)
        np.testing.assert_allclose(ref.dequantise(code, byte), x, rtol=2.0 ** -4,
                                   atol=2.0 ** (e - 10))


def _ints(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def test_tables_whose_rows_overlap_are_refused():
    """One row expanded over the batch, or rows closer than they are wide: the library would step
    past the tensor's end. Rows further apart are a slice of a wider table."""
    n, q = _ints(4), _ints(5)
    for table in (_ints(1, 3).expand(4, 3), _ints(3).expand(4, 3), _ints(9).as_strided((4, 3), (2, 1))):
        with pytest.raises(pk.PariskvError) as e:
            pk.Chunk(table, n, q, 4, 2)
        assert e.value.status == pk.EINVAL
    assert pk.Chunk(_ints(4, 3), n, q, 4, 2).raw.table_stride == 3
    assert pk.Chunk(_ints(4, 7)[:, :3], n, q, 4, 2).raw.table_stride == 7
    # (one row has no distance to the next)
    assert pk.Chunk(_ints(1, 7)[:, :3], n[:1], q[:2], 4, 2).raw.table_stride in (3, 7)
    assert pk.Chunk(_ints(9).as_strided((1, 3), (1, 1)), n[:1], q[:2], 4, 2).raw.table_stride == 3


def test_counts_that_the_description_cannot_hold_are_refused():
    """max_q and total_q are passed in 32 and 64 bits: 2^32 must not become 0 rows."""
    t, n, q = _ints(2, 3), _ints(2), _ints(3)
    for total, most in ((4, 1 << 31), (4, 1 << 32), (4, (1 << 32) + 1), (4, -1), (1 << 31, 4),
                        ((1 << 64) + 3, 4), (-1, 4)):
        with pytest.raises(pk.PariskvError) as e:
            pk.Chunk(t, n, q, total, most)
        assert e.value.status == pk.EINVAL
    raw = pk.Chunk(t, n, q, (1 << 31) - 1, (1 << 31) - 1).raw
    assert raw.total_q == raw.max_q == (1 << 31) - 1
