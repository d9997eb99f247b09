"""Refusals of the attention calls: nothing here reaches a device. The addresses are of no memory, so a call that is not
refused for its arguments is made only where there is no device to run it."""

import ctypes
import math

import pytest
import torch

import weight_only_bit_qgemv_b200 as woq
from weight_only_bit_qgemv_b200 import _lib

OK = 1 << 20  # an address that no call below dereferences
FAR = 1 << 40


def rows(data=OK, dtype=0, heads=2, row=256, head=128):
    return _lib.WoqRows(data, dtype, heads, row, head)


def kv4(codes=FAR, scales=2 * FAR, pages=4, heads=2, dim=128, page=16):
    return _lib.WoqKv4(codes, scales, pages, heads, dim, page)


BAD_CACHES = [
    (kv4(codes=0), _lib.WOQ_EINVAL), (kv4(scales=0), _lib.WOQ_EINVAL),
    (kv4(page=8), _lib.WOQ_EINVAL), (kv4(page=48), _lib.WOQ_EINVAL), (kv4(page=131072), _lib.WOQ_EINVAL),
    (kv4(dim=96), _lib.WOQ_ESHAPE), (kv4(dim=256), _lib.WOQ_ESHAPE), (kv4(pages=0), _lib.WOQ_ESHAPE),
    (kv4(pages=2**31), _lib.WOQ_ESHAPE), (kv4(heads=0), _lib.WOQ_ESHAPE), (kv4(heads=1025), _lib.WOQ_ESHAPE),
    (kv4(codes=FAR + 32), _lib.WOQ_EALIGN), (kv4(scales=FAR + 2), _lib.WOQ_EALIGN),
]
BAD_ROWS = [
    (rows(data=0), _lib.WOQ_EINVAL), (rows(dtype=3), _lib.WOQ_EINVAL), (rows(dtype=-1), _lib.WOQ_EINVAL),
    (rows(row=0), _lib.WOQ_ESHAPE), (rows(row=-256), _lib.WOQ_ESHAPE), (rows(row=258), _lib.WOQ_ESHAPE),
    (rows(dtype=1, row=260), _lib.WOQ_ESHAPE), (rows(head=64), _lib.WOQ_ESHAPE), (rows(row=2**40), _lib.WOQ_ESHAPE),
    (rows(data=OK + 8), _lib.WOQ_EALIGN),
]


def test_step_refusals():
    L = _lib.lib()

    def both(c=None, k=None, v=None, tokens=4, cu=OK, start=None, batch=1, table=OK, width=1):
        c, k, v = c or kv4(), k or rows(), v or rows(data=FAR)
        a = L.kv4_append(ctypes.byref(c), ctypes.byref(k), ctypes.byref(v), tokens, cu, start, batch, table, width, None)
        b = L.kv4_gather(ctypes.byref(c), cu, start, batch, table, width, tokens, ctypes.byref(k), ctypes.byref(v), None)
        assert a == b
        return a

    for c, want in BAD_CACHES:
        assert both(c=c) == want
    for r, want in BAD_ROWS + [(rows(heads=3), _lib.WOQ_EINVAL)]:
        assert both(k=r) == want and both(v=r) == want
    assert both(tokens=-1) == _lib.WOQ_EINVAL and both(tokens=2**31) == _lib.WOQ_ESHAPE
    assert both(cu=None) == _lib.WOQ_EINVAL and both(table=None) == _lib.WOQ_EINVAL
    assert both(cu=OK + 2) == both(start=OK + 1) == both(table=OK + 2) == _lib.WOQ_EALIGN
    assert both(batch=0) == both(batch=4097) == _lib.WOQ_EINVAL
    assert both(width=0) == both(width=2**31) == _lib.WOQ_ESHAPE
    assert L.kv4_append(None, ctypes.byref(rows()), ctypes.byref(rows()), 1, OK, None, 1, OK, 1, None) == _lib.WOQ_EINVAL
    # what is gathered may not lie on itself
    k, c = rows(), kv4()
    for v in (rows(), rows(data=OK + 512), rows(data=OK + 1024, dtype=1)):
        assert L.kv4_gather(ctypes.byref(c), OK, None, 1, OK, 1, 4, ctypes.byref(k), ctypes.byref(v),
                            None) == _lib.WOQ_EINVAL


def test_attention_refusals():
    L = _lib.lib()

    def call(q=None, c=None, lens=OK, batch=2, table=OK, width=1, scale=0.1, o=None, ws=1 << 21, n=1 << 30):
        q, c, o = q or rows(heads=4, row=512), c or kv4(), o or rows(data=FAR, heads=4, row=512)
        return L.kv4_attn(ctypes.byref(q), ctypes.byref(c), lens, batch, table, width, scale, ctypes.byref(o), ws, n, None)

    for c, want in BAD_CACHES[:9]:
        assert call(c=c) == want
    for r, want in BAD_ROWS:
        r = _lib.WoqRows(r.data, r.dtype, 4, r.row_stride * 2, r.head_stride)
        if r.row_stride != 516 and r.row_stride != 520:
            assert call(q=r) == want and call(o=r) in (want, _lib.WOQ_EINVAL)
    assert call(q=rows(heads=3)) == call(q=rows(heads=0)) == call(q=rows(heads=2 * 65)) == _lib.WOQ_EINVAL
    assert call(o=rows(data=FAR, heads=2)) == _lib.WOQ_EINVAL
    assert call(o=rows(data=FAR, heads=4, row=512, dtype=1)) == _lib.WOQ_EINVAL
    for scale in (0.0, -1.0, math.inf, math.nan):
        assert call(scale=scale) == _lib.WOQ_EINVAL
    assert call(lens=None) == call(table=None) == call(batch=0) == call(batch=4097) == _lib.WOQ_EINVAL
    assert call(lens=OK + 2) == _lib.WOQ_EALIGN and call(width=0) == _lib.WOQ_ESHAPE
    assert call(ws=None) == call(n=64) == _lib.WOQ_EWORKSPACE and call(ws=(1 << 21) + 128) == _lib.WOQ_EALIGN
    # o on q, or one row of it
    assert call(o=rows(heads=4, row=512)) == _lib.WOQ_EINVAL
    assert call(o=rows(data=OK + 4 * 512, heads=4, row=512)) == _lib.WOQ_EINVAL
    # beside it in one array is another matter: refused only for want of a device (with one it would run)
    if not torch.cuda.is_available():
        side = call(q=rows(heads=4, row=1024), o=rows(data=OK + 4 * 512, heads=4, row=1024))
        assert side in (_lib.WOQ_ECUDA, _lib.WOQ_EDEVICE)


def test_prompt_refusals():
    L = _lib.lib()

    def call(q=None, k=None, v=None, o=None, tokens=4, cu=OK, batch=1, dim=128, scale=0.1, ws=1 << 21, n=1 << 30):
        args = [q or rows(heads=4, row=512), k or rows(data=FAR), v or rows(data=2 * FAR),
                o or rows(data=3 * FAR, heads=4, row=512)]
        q, k, v, o = (ctypes.byref(x) for x in args)
        return L.attn_prompt(q, k, v, tokens, cu, batch, dim, scale, o, ws, n, None)

    for r, want in BAD_ROWS:
        assert call(k=r) in (want, _lib.WOQ_EINVAL) and call(v=r) in (want, _lib.WOQ_EINVAL)
    assert call(q=rows(heads=3)) == call(o=rows(heads=2)) == call(v=rows(heads=1)) == _lib.WOQ_EINVAL
    assert call(k=rows(heads=1025, row=1025 * 128), q=rows(heads=1025, row=1025 * 128)) == _lib.WOQ_EINVAL
    for name in ("q", "k", "v", "o"):  # one type for all
        r = rows(data=5 * FAR, dtype=2, heads=4 if name in "qo" else 2, row=512)
        assert call(**{name: r}) == _lib.WOQ_EINVAL
    assert call(dim=96) == call(dim=32) == _lib.WOQ_ESHAPE
    for scale in (0.0, -1.0, math.inf, math.nan):
        assert call(scale=scale) == _lib.WOQ_EINVAL
    assert call(tokens=-1) == call(cu=None) == call(batch=0) == call(batch=2**20 + 1) == _lib.WOQ_EINVAL
    assert call(tokens=2**31) == _lib.WOQ_ESHAPE and call(cu=OK + 2) == _lib.WOQ_EALIGN
    many = rows(data=4 * FAR, heads=32768, row=32768 * 128)
    assert call(q=many, o=rows(data=8 * FAR, heads=32768, row=32768 * 128), tokens=2**25) == _lib.WOQ_ESHAPE
    assert call(ws=None) == call(n=1024) == _lib.WOQ_EWORKSPACE and call(ws=(1 << 21) + 64) == _lib.WOQ_EALIGN
    for name in ("q", "k", "v"):  # the output on an input
        r = rows(data=3 * FAR, heads=4 if name == "q" else 2, row=512)
        assert call(**{name: r}) == _lib.WOQ_EINVAL
    size = L.attn_prompt_workspace_bytes
    assert size(100, 1, 4, 2, 128, _lib.WOQ_BF16) == 0 and size(100, 1, 4, 2, 128, _lib.WOQ_F32) > 100 * 8 * 128 * 4
    for bad in ((-1, 1, 4, 2, 128, 0), (100, 0, 4, 2, 128, 0), (100, 1, 3, 2, 128, 0), (100, 1, 4, 2, 96, 0)):
        assert size(*bad) == 0


def test_workspace_sizes():
    L = _lib.lib()
    size = L.kv4_attn_workspace_bytes
    assert size(ctypes.byref(kv4()), 4, 1) > 0 and size(ctypes.byref(kv4()), 4, 1) % 16 == 0
    assert size(ctypes.byref(kv4()), 4, 4096) > size(ctypes.byref(kv4()), 4, 1)
    for c, h, b in ((kv4(dim=32), 4, 1), (kv4(), 3, 1), (kv4(), 4, 0), (kv4(), 4, 4097), (kv4(), 2 * 65, 1)):
        assert size(ctypes.byref(c), h, b) == 0


def test_binding_refuses_host_tensors_and_wrong_shapes():
    with pytest.raises(ValueError):
        woq.KV4Cache(torch.zeros(1, 1, 2, 16, 64), torch.zeros(1, 1, 16, 2, 4, dtype=torch.float16))
    with pytest.raises(ValueError):
        woq.KV4Cache(torch.zeros(1, 1, 2, 16, 64, dtype=torch.uint8), torch.zeros(1, 1, 16, 2, 2, dtype=torch.float16))
    cache = woq.KV4Cache.empty(1, 1, 128, 16, device="cpu")
    assert (cache.kv_heads, cache.dim, cache.page) == (1, 128, 16) and cache.nbytes == 16 * 144
    x, i = torch.zeros(1, 1, 128), torch.zeros(2, dtype=torch.int32)
    for call in (lambda: woq.kv4_append(cache, x, x, i, i[None]), lambda: woq.kv4_attn(x, cache, i[:1], i[None, :1]),
                 lambda: woq.attn_prompt(x, x, x, i), lambda: woq.attn_prompt_workspace(x[0], x, 1),
                 lambda: woq.kv4_gather(cache, i, i[None], k_out=x, v_out=x), lambda: woq.kv4_gather(cache, i, i[None])):
        with pytest.raises(ValueError):
            call()
    for name in ("attn_prompt", "kv4_append", "kv4_gather", "kv4_attn", "KV4Cache"):
        assert name in woq.__all__


def test_no_rows_and_interleaved_arrays():
    """Empty prompts have no address; arrays that only interleave are not refused. Without a device both end there."""
    L = _lib.lib()
    through = (_lib.WOQ_ECUDA, _lib.WOQ_EDEVICE)
    none = _lib.WOQ_OK if torch.cuda.is_available() else None
    c, r, big = kv4(), rows(data=0), rows(data=0, heads=4, row=512)
    for rc in (L.kv4_append(ctypes.byref(c), ctypes.byref(r), ctypes.byref(r), 0, OK, None, 1, OK, 1, None),
               L.kv4_gather(ctypes.byref(c), OK, None, 1, OK, 1, 0, ctypes.byref(r), ctypes.byref(r), None),
               L.attn_prompt(ctypes.byref(big), ctypes.byref(r), ctypes.byref(r), 0, OK, 1, 128, 0.1, ctypes.byref(big),
                             None, 0, None)):
        assert rc in through or rc == none

    def gather(a, b, tokens=4):
        return L.kv4_gather(ctypes.byref(c), OK, None, 1, OK, 1, tokens, ctypes.byref(a), ctypes.byref(b), None)

    if not torch.cuda.is_available():  # these would run
        size = 4
        for a, b in (
            (rows(row=512, head=256), rows(data=OK + 128 * size, row=512, head=256)),  # [tokens, heads, 2, dim]
            (rows(data=OK + 128 * size, row=512, head=256), rows(row=512, head=256)),
            (rows(row=512), rows(data=OK + 256 * size, row=512)),  # [tokens, 2, heads, dim]
            (rows(row=128, head=1024), rows(data=OK + 512 * size, row=128, head=1024)),  # [heads, 2, tokens, dim]
            (rows(row=256, head=1024), rows(data=OK + 128 * size, row=256, head=1024)),  # [heads, tokens, 2, dim]
        ):
            assert gather(a, b) in through
    for a, b in (
        (rows(row=512, head=256), rows(data=OK + 256 * 4, row=512, head=256)),  # on the other head
        (rows(row=128, head=1024), rows(data=OK + 384 * 4, row=128, head=1024)),  # on the last token
        (rows(row=256, head=1024), rows(data=OK + 256 * 4, row=256, head=1024)),  # on the next token
        (rows(row=768, head=256), rows(data=OK + 64 * 4, row=768, head=256)),  # half a row
    ):
        assert gather(a, b) == gather(b, a) == _lib.WOQ_EINVAL


def test_strides_and_extents_that_nothing_can_hold():
    """Strides of 2^40 bytes, arrays beyond 64 bits of offsets, more rows than a grid has blocks for."""
    L = _lib.lib()

    def gather(a, b, tokens=4, c=None):
        return L.kv4_gather(ctypes.byref(c or kv4()), OK, None, 1, OK, 1, tokens, ctypes.byref(a), ctypes.byref(b), None)

    def prompt(q, tokens=4):
        k, o = rows(heads=1, data=3 * FAR, dtype=q.dtype), rows(heads=1, data=5 * FAR, dtype=q.dtype)
        return L.attn_prompt(ctypes.byref(q), ctypes.byref(k), ctypes.byref(k), tokens, OK, 1, 128, 0.1, ctypes.byref(o),
                             1 << 21, 1 << 62, None)

    for dtype, size in ((0, 4), (1, 2), (2, 2)):
        for stride in (2**40 // size, 2**40 - 16, 2**62):
            assert gather(rows(dtype=dtype, row=stride), rows(data=FAR, dtype=dtype)) == _lib.WOQ_ESHAPE
            assert gather(rows(dtype=dtype, head=stride, row=128), rows(data=FAR, dtype=dtype)) == _lib.WOQ_ESHAPE
            assert prompt(rows(heads=1, dtype=dtype, row=stride)) == _lib.WOQ_ESHAPE
        wide = 2**40 // size - 64
        assert gather(rows(dtype=dtype, row=wide), rows(data=FAR, dtype=dtype), tokens=2**30) == _lib.WOQ_ESHAPE
        assert prompt(rows(heads=1, dtype=dtype, row=wide), tokens=2**30) == _lib.WOQ_ESHAPE
        # appended rows may share elements, so that this many are no more than 32 GB
        k, c = rows(dtype=dtype, heads=1024, row=16 // size, head=128), kv4(heads=1024)
        assert L.kv4_append(ctypes.byref(c), ctypes.byref(k), ctypes.byref(k), 2**31 - 1, OK, None, 1, OK, 1,
                            None) == _lib.WOQ_ESHAPE


def test_written_arrays_whose_rows_share_elements():
    L = _lib.lib()
    through = (_lib.WOQ_ECUDA, _lib.WOQ_EDEVICE)
    big = {"data": 16 * FAR}

    def attn(o, batch=3):
        q, c = rows(heads=o.heads, row=128 * o.heads), kv4(heads=1)
        return L.kv4_attn(ctypes.byref(q), ctypes.byref(c), OK, batch, OK, 1, 0.1, ctypes.byref(o), 1 << 21, 1 << 30, None)

    def prompt(o, tokens=3):
        q, k = rows(heads=o.heads, row=128 * o.heads), rows(heads=1, data=3 * FAR)
        return L.attn_prompt(ctypes.byref(q), ctypes.byref(k), ctypes.byref(k), tokens, OK, 1, 128, 0.1, ctypes.byref(o),
                             1 << 21, 1 << 30, None)

    def gather(o, tokens=3):
        v, c = rows(data=5 * FAR, heads=o.heads, row=128 * o.heads), kv4(heads=o.heads)
        return L.kv4_gather(ctypes.byref(c), OK, None, 1, OK, 1, tokens, ctypes.byref(o), ctypes.byref(v), None)

    def gather_v(o, tokens=3):
        k, c = rows(data=5 * FAR, heads=o.heads, row=128 * o.heads), kv4(heads=o.heads)
        return L.kv4_gather(ctypes.byref(c), OK, None, 1, OK, 1, tokens, ctypes.byref(k), ctypes.byref(o), None)

    for o in (rows(heads=1, row=16, **big), rows(heads=1, row=124, **big), rows(heads=2, row=128, head=128, **big),
              rows(heads=2, row=128, head=256, **big), rows(heads=2, row=192, head=128, **big),
              rows(heads=3, row=256, head=320, **big), rows(heads=4, row=400, head=132, **big)):
        for call in (attn, prompt, gather, gather_v):
            assert call(o) == _lib.WOQ_ESHAPE, (o.heads, o.row_stride, o.head_stride)
    if not torch.cuda.is_available():  # these would run
        for o in (rows(heads=1, row=128, **big), rows(heads=2, row=256, head=128, **big),
                  rows(heads=2, row=128, head=384, **big), rows(heads=2, row=132, head=392, **big),
                  rows(heads=2, row=256, head=640, **big), rows(heads=3, row=384, head=512, **big)):
            for call in (attn, prompt, gather, gather_v):
                assert call(o) in through, (o.heads, o.row_stride, o.head_stride)
        for o in (rows(heads=1, row=16, **big), rows(heads=2, row=16, head=128, **big)):  # a single row
            assert attn(o, 1) in through and prompt(o, 1) in through and gather(o, 1) in through


def test_results_on_the_cache():
    L = _lib.lib()
    c = kv4()  # 4 pages of 16 tokens, 2 heads: 16384 bytes of codes, 2048 of scales
    far = rows(data=8 * FAR)
    for at, on in ((FAR - 4 * 1024, False), (FAR - 4 * 1024 + 16, True), (FAR + 16384 - 16, True), (FAR + 16384, False),
                   (2 * FAR, True), (2 * FAR + 2048, False), (2 * FAR - 4 * 1024, False)):
        r = rows(data=at)  # 4 rows of 2 heads of 128 float32
        q = rows(heads=2, data=9 * FAR)
        calls = [lambda: L.kv4_gather(ctypes.byref(c), OK, None, 1, OK, 1, 4, ctypes.byref(r), ctypes.byref(far), None),
                 lambda: L.kv4_gather(ctypes.byref(c), OK, None, 1, OK, 1, 4, ctypes.byref(far), ctypes.byref(r), None),
                 lambda: L.kv4_attn(ctypes.byref(q), ctypes.byref(c), OK, 4, OK, 1, 0.1, ctypes.byref(r), 1 << 21, 1 << 30,
                                    None)]
        for call in calls:
            if on:
                assert call() == _lib.WOQ_EINVAL
            elif not torch.cuda.is_available():  # it would run
                assert call() in (_lib.WOQ_ECUDA, _lib.WOQ_EDEVICE)


def test_scales_next_to_the_end_of_the_range():
    L = _lib.lib()
    q, k, o, c = rows(heads=2), rows(data=3 * FAR), rows(data=4 * FAR, heads=2), kv4()
    for scale, good in ((2.0**127, True), (1e-44, True), (1.8e38, False), (3.4e38, False)):
        if good and torch.cuda.is_available():  # it would run
            continue
        got = (L.kv4_attn(ctypes.byref(q), ctypes.byref(c), OK, 2, OK, 1, scale, ctypes.byref(o), 1 << 21, 1 << 30, None),
               L.attn_prompt(ctypes.byref(q), ctypes.byref(k), ctypes.byref(k), 4, OK, 1, 128, scale, ctypes.byref(o),
                             1 << 21, 1 << 30, None))
        assert all((x in (_lib.WOQ_ECUDA, _lib.WOQ_EDEVICE)) if good else x == _lib.WOQ_EINVAL for x in got)
