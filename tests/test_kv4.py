"""The 4-bit cache: kv4_append and kv4_gather against the oracle's quantiser, bit for bit, and kv4_attn against
attention in 64 bits over the values that the cache holds."""

import copy

import numpy as np
import pytest
import torch

import weight_only_bit_qgemv_b200 as woq
from weight_only_bit_qgemv_b200 import _lib
from tests import attn_ref as ref

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def packed(rng, tokens, heads, dim, dtype, spare=0):
    """Rows of a fused array [tokens + spare, q | k | v]: k and v are slices with a stride of their own."""
    x = torch.from_numpy(rng.standard_normal((tokens + spare, 3 * heads, dim)).astype(np.float32))
    x = x.to(dtype).cuda()
    return x[:, heads:2 * heads], x[:, 2 * heads:]


def expected(k, v, cu, start, table, pages, heads, dim, page):
    codes = np.zeros((pages, heads, 2, page, dim // 2), np.uint8)
    scales = np.zeros((pages, heads, page, 2, dim // 32), np.float16)
    values = {}
    for b in range(len(cu) - 1):
        for t in range(cu[b], cu[b + 1]):
            at = start[b] + t - cu[b]
            if start[b] < 0 or at // page >= table.shape[1] or not 0 <= table[b, at // page] < pages:
                continue
            for i, x in enumerate((k, v)):
                q, s, val = ref.quantised(x[t].float().cpu().numpy())
                ref.write_pages(q, s, i, codes, scales, table[b, at // page], at % page)
                values[t, i] = val
    return codes, scales, values


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("heads,dim,page,lens,start", [
    (1, 64, 16, [1], [0]),
    (3, 128, 16, [5, 0, 33, 1], [0, 7, 15, 31]),       # odd heads; a sequence without rows; pages that end inside
    (8, 128, 64, [64, 65, 63], [0, 0, 1]),
    (5, 64, 32, [100, 1], [28, 200]),
])
def test_append_is_the_quantiser_bit_for_bit_and_gather_reads_it(dtype, heads, dim, page, lens, start):
    rng = np.random.default_rng(heads * 100 + dim)
    cu = np.concatenate([[2], 2 + np.cumsum(lens)]).astype(int)  # rows 0, 1 belong to no sequence
    tokens = int(cu[-1])
    width = max(-(-(n + s) // page) for n, s in zip(lens, start)) + 1
    pages = len(lens) * width + 3
    table = rng.permutation(pages)[: len(lens) * width].reshape(len(lens), width)
    k, v = packed(rng, tokens, heads, dim, dtype, spare=3)
    cache = woq.KV4Cache.empty(pages, heads, dim, page)
    woq.kv4_append(cache, k, v, ints(cu), ints(table), start=ints(start))
    codes, scales, values = expected(k, v, cu, start, table, pages, heads, dim, page)
    assert np.array_equal(cache.codes.cpu().numpy(), codes)
    assert np.array_equal(cache.scales.cpu().numpy().view(np.uint16), scales.view(np.uint16))
    k2, v2 = (torch.full((tokens + 3, heads, dim), 7.0, device="cuda") for _ in "kv")
    woq.kv4_gather(cache, ints(cu), ints(table), start=ints(start), k_out=k2, v_out=v2)
    for i, out in enumerate((k2, v2)):
        out = out.cpu().numpy()
        for t in range(tokens + 3):
            want = values[t, i] if (t, i) in values else 7.0  # rows outside the sequences stay as they were
            assert np.array_equal(out[t], np.broadcast_to(want, out[t].shape)), (t, i)
    k3, _ = woq.kv4_gather(cache, ints(cu), ints(table), start=ints(start), tokens=tokens, dtype=dtype)
    assert torch.equal(k3[2:], k2[2:tokens].to(dtype)) and not k3[:2].any()


def test_append_rounds_ties_and_extremes_as_the_quantiser():
    """Values on and next to the codes' borders, tiny and huge blocks, zeros."""
    heads, dim, page = 2, 128, 16
    rng = np.random.default_rng(5)
    x = rng.standard_normal((300, heads, dim)).astype(np.float32)
    s = np.float32(np.float16(0.37))
    ties = ((rng.integers(-7, 7, size=(100, heads, dim)) + 0.5) * s).astype(np.float32)
    x[:100] = np.nextafter(ties, rng.choice([-np.inf, 0, np.inf], size=ties.shape).astype(np.float32))
    x[:50] = ties[:50]
    x[:100, :, ::32] = 7 * s
    x[100:150] *= 1e-9
    x[150:170] *= 1e-40
    x[170:190] *= 1e5
    x[190:200] = 0
    x[200] = 65519.0 * 7 / 1.0001
    k = torch.from_numpy(x).cuda()
    cache = woq.KV4Cache.empty(20, heads, dim, page)
    table = np.arange(20)[None]
    woq.kv4_append(cache, k, -k, ints([0, 300]), ints(table))
    codes, scales, _ = expected(k, -k, [0, 300], [0], table, 20, heads, dim, page)
    assert np.array_equal(cache.codes.cpu().numpy(), codes)
    assert np.array_equal(cache.scales.cpu().numpy().view(np.uint16), scales.view(np.uint16))


@pytest.mark.parametrize("kind", ["scales", "codes", "sizes"])
def test_append_next_to_the_borders_of_rounding(kind):
    """Block maxima within 3 ulp of 7 times a binary16 midpoint, values within 4 ulp of a tie, blocks of all sizes."""
    rng = np.random.default_rng(len(kind))
    n, heads, dim, page = 800, 4, 128, 16
    x = rng.uniform(-1, 1, (n, heads, dim)).astype(np.float32)
    if kind == "scales":
        low = rng.integers(1, 0x7B00, (n, heads, dim // 32)).astype(np.uint16).view(np.float16)
        a = (low.astype(np.float64) + np.nextafter(low, np.float16(np.inf)).astype(np.float64)) / 2 * 7
        a = a.astype(np.float32)
        a = (a.view(np.int32) + rng.integers(-3, 4, a.shape).astype(np.int32)).view(np.float32)
        x *= np.repeat(a, 32, -1)
        x[..., ::32] = a
    elif kind == "codes":
        s = rng.integers(1, 0x7000, (n, heads, dim // 32)).astype(np.uint16).view(np.float16).astype(np.float32)
        tie = ((rng.integers(-7, 7, x.shape) + 0.5) * np.repeat(s, 32, -1)).astype(np.float32)
        x = (tie.view(np.int32) + rng.integers(-4, 5, tie.shape).astype(np.int32)).view(np.float32)
        x[..., ::32] = 7 * s
    else:
        x *= np.exp(rng.uniform(-100, 10, (n, heads, 1))).astype(np.float32)
    k = torch.from_numpy(x).cuda()
    cache = woq.KV4Cache.empty(n // page, heads, dim, page)
    table = np.arange(n // page)[None]
    woq.kv4_append(cache, k, -k, ints([0, n]), ints(table))
    codes, scales, _ = expected(k, -k, [0, n], [0], table, n // page, heads, dim, page)
    assert np.array_equal(cache.codes.cpu().numpy(), codes)
    assert np.array_equal(cache.scales.cpu().numpy().view(np.uint16), scales.view(np.uint16))


def test_append_marks_blocks_it_cannot_hold():
    k = torch.randn(16, 1, 64, device="cuda")
    v = torch.randn(16, 1, 64, device="cuda")
    k[3, 0, 5], k[4, 0, 40], v[5, 0, 0], v[6, 0, 63] = float("nan"), float("inf"), 65520.0 * 7, -float("inf")
    cache = woq.KV4Cache.empty(1, 1, 64, 16)
    cu, table = ints([0, 16]), ints([[0]])
    woq.kv4_append(cache, k, v, cu, table)
    ko, vo = woq.kv4_gather(cache, cu, table, tokens=16)
    for out, bad in ((ko, {(3, 0), (4, 1)}), (vo, {(5, 0), (6, 1)})):
        nan = out.isnan().view(16, 2, 32)
        for t in range(16):
            for b in range(2):
                assert nan[t, b].all() if (t, b) in bad else not nan[t, b].any()


def test_append_drops_what_has_no_page_and_touches_nothing_else():
    cache = woq.KV4Cache.empty(4, 2, 128, 16)
    cache.codes.fill_(0x5A)
    cache.scales.fill_(3.0)
    before = cache.codes.clone(), cache.scales.clone()
    k = torch.randn(64, 2, 128, device="cuda")
    table = ints([[-1, 4], [7, -2], [2**31 - 1, -2**31]])
    woq.kv4_append(cache, k, k, ints([0, 20, 40, 64]), table)           # no entry names a page of the pool
    woq.kv4_append(cache, k, k, ints([0, 64]), ints([[0]]), start=ints([16]))   # beyond the table
    woq.kv4_append(cache, k, k, ints([0, 64]), ints([[0]]), start=ints([-3]))
    assert torch.equal(cache.codes, before[0]) and torch.equal(cache.scales, before[1])
    ko, vo = (torch.full((64, 2, 128), 7.0, device="cuda") for _ in "kv")
    woq.kv4_gather(cache, ints([0, 20, 40, 64]), table, k_out=ko, v_out=vo)
    assert not ko.any() and not vo.any()


def random_cache(rng, pages, heads, dim, page):
    """Every code, -8 among them, and scales of all sizes."""
    codes = torch.from_numpy(rng.integers(0, 256, (pages, heads, 2, page, dim // 2), dtype=np.uint8)).cuda()
    scales = torch.from_numpy((rng.standard_normal((pages, heads, page, 2, dim // 32)) * 0.2).astype(np.float16)).cuda()
    return woq.KV4Cache(codes, scales)


def check_attention(cache, q, lens, table, scale=None, **kw):
    out = woq.kv4_attn(q, cache, ints(lens), ints(table), scale=scale, **kw)
    k, v = ref.read_pages(cache.codes, cache.scales)
    scale = cache.dim**-0.5 if scale is None else scale
    for b, n in enumerate(lens):
        at = [(table[b][j // cache.page], j % cache.page) for j in range(max(0, min(n, len(table[b]) * cache.page)))]
        at = [(p, s) for p, s in at if 0 <= p < k.shape[0]]
        kb = np.array([k[p, :, s] for p, s in at]).reshape(-1, cache.kv_heads, cache.dim)
        vb = np.array([v[p, :, s] for p, s in at]).reshape(-1, cache.kv_heads, cache.dim)
        want, size = ref.attend(q[b].double().cpu().numpy(), kb, vb, scale)
        err = np.abs(out[b].double().cpu().numpy() - want)
        assert (err <= ref.tolerance(want, size, q.dtype)).all(), (b, n, err.max())
    assert woq.device_status() == _lib.WOQ_OK
    return out


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("heads,kv,dim,page,lens", [
    (1, 1, 64, 16, [1]),
    (2, 1, 128, 16, [0, 1, 15, 16, 17, 31, 32, 33]),     # around a page, half a unit and a unit
    (16, 8, 128, 64, [1000, 0, 129, 3]),
    (15, 3, 128, 32, [500, 64]),                           # five query heads to a key head
    (9, 1, 64, 64, [300, 7]),                              # nine: two passes, one of a single head
    (64, 1, 128, 16, [257]),
    (12, 12, 64, 128, [4096 + 5, 1]),
])
def test_attention_matches_the_formula(dtype, heads, kv, dim, page, lens):
    rng = np.random.default_rng(heads * 7 + dim + page)
    width = max(1, max(-(-n // page) for n in lens))
    table = rng.permutation(len(lens) * width + 2)[: len(lens) * width].reshape(len(lens), width)
    cache = random_cache(rng, len(lens) * width + 2, kv, dim, page)
    q = torch.from_numpy(rng.standard_normal((len(lens), heads, dim)).astype(np.float32)).to(dtype).cuda()
    check_attention(cache, q, lens, table.tolist())


def test_attention_over_long_and_ragged_contexts():
    """Parts that hold several sequences, and sequences that many parts share."""
    rng = np.random.default_rng(3)
    lens = [70001, 1, 0, 33, 4097, 12345, 2, 600] + [17] * 40
    page, kv, dim = 64, 2, 128
    need = [-(-n // page) for n in lens]
    order = rng.permutation(sum(need))
    table = np.full((len(lens), max(need)), -1)
    for b, n in enumerate(need):
        table[b, :n] = order[sum(need[:b]):sum(need[:b + 1])]
    cache = random_cache(rng, sum(need), kv, dim, page)
    q = torch.from_numpy(rng.standard_normal((len(lens), 4, dim)).astype(np.float32)).cuda()
    ws = woq.kv4_attn_workspace(cache, q)
    first = check_attention(cache, q, lens, table.tolist(), workspace=ws)
    for _ in range(3):  # the same bits, and the workspace left ready
        assert torch.equal(woq.kv4_attn(q, cache, ints(lens), ints(table), workspace=ws), first)


def test_attention_keeps_precision_at_extreme_sizes():
    """Tiny and huge queries and values; one token's scale far above the others', early and late."""
    rng = np.random.default_rng(9)
    page, kv, dim = 16, 1, 128
    table = [list(range(20))]
    for qs, ss in ((1e-20, 1.0), (1e-3, 2.0**-18), (30.0, 1.0), (1e4, 2.0**-14)):
        cache = random_cache(rng, 20, kv, dim, page)
        cache.scales[:, :, :, 1] *= ss
        cache.scales[:, :, :, 0] *= min(1.0, 1.0 / qs)
        q = torch.from_numpy((rng.standard_normal((1, 8, dim)) * qs).astype(np.float32)).cuda()
        check_attention(cache, q, [311], table)
    for at in (0, 150, 310):
        cache = random_cache(rng, 20, kv, dim, page)
        cache.scales[at // page, 0, at % page, 1] = 60000.0
        q = torch.from_numpy(rng.standard_normal((1, 8, dim)).astype(np.float32)).cuda()
        check_attention(cache, q, [311], table)
    # scores far apart: all weight on a few tokens
    cache = random_cache(rng, 20, kv, dim, page)
    q = torch.from_numpy((40 * rng.standard_normal((1, 8, dim))).astype(np.float32)).cuda()
    check_attention(cache, q, [320], table)


def test_attention_ignores_what_is_not_there():
    """NaN and infinities behind the last token, in pages of other sequences, entries outside the pool."""
    rng = np.random.default_rng(11)
    page, kv, dim = 32, 2, 128
    cache = random_cache(rng, 12, kv, dim, page)
    lens, table = [70, 5, 40], [[0, 1, 2], [3, -1, 99], [5, 12, 4]]   # of the third, tokens 32..39 have no page
    cache.scales[2, :, 6:] = float("nan")
    cache.scales[3, :, 5:] = float("inf")
    cache.scales[6:] = float("nan")
    q = torch.from_numpy(rng.standard_normal((3, 4, dim)).astype(np.float32)).cuda()
    check_attention(cache, q, lens, table)
    out = woq.kv4_attn(q, cache, ints([-5, 64, 2**31 - 1]), ints([[0, 1, 2], [12, -1, 0], [12, -1, -7]]))
    assert not out.any()  # no length; no page at all
    cache = random_cache(rng, 12, kv, dim, page)
    check_attention(cache, q, [2**31 - 1, 96, 97], [[0, 1, 2], [3, 4, 5], [6, 7, 8]])  # longer than the table


def test_attention_passes_on_what_is_not_finite():
    rng = np.random.default_rng(12)
    cache = random_cache(rng, 4, 2, 64, 16)
    q = torch.from_numpy(rng.standard_normal((1, 4, 64)).astype(np.float32)).cuda()
    table, lens = ints([[0, 1, 2, 3]]), ints([50])
    clean = woq.kv4_attn(q, cache, lens, table)
    cache.scales[1, 0, 3, 0, 1] = float("nan")  # a key of head 0
    out = woq.kv4_attn(q, cache, lens, table)
    assert out[0, :2].isnan().all() and torch.equal(out[0, 2:], clean[0, 2:])
    cache = random_cache(np.random.default_rng(12), 4, 2, 64, 16)
    cache.scales[2, 1, 0, 1, 0] = float("nan")  # block 0 of a value of head 1
    out = woq.kv4_attn(q, cache, lens, table)
    assert out[0, 2:, :32].isnan().all() and not out[0, 2:, 32:].isnan().any() and not out[0, :2].isnan().any()
    q[0, 1, 7] = float("nan")
    out = woq.kv4_attn(q, cache, lens, table)
    assert out[0, 1].isnan().all() and not out[0, 0].isnan().any()


def test_attention_takes_strides_and_leaves_the_rest():
    rng = np.random.default_rng(13)
    cache = random_cache(rng, 8, 2, 128, 16)
    fused = torch.from_numpy(rng.standard_normal((3, 10, 128)).astype(np.float32)).cuda()
    out = torch.full((3, 9, 128), 7.0, device="cuda")
    lens, table = [40, 16, 1], [[0, 1, 2], [3, 4, 5], [6, 7, 0]]
    check_attention(cache, fused[:, 2:8], lens, table, out=out[:, 1:7])
    assert (out[:, :1] == 7).all() and (out[:, 7:] == 7).all()
    # an output beside the queries in one array
    both = torch.zeros(3, 12, 128, device="cuda")
    both[:, :6] = fused[:, 2:8]
    woq.kv4_attn(both[:, :6], cache, ints(lens), ints(table), out=both[:, 6:])
    assert torch.equal(both[:, 6:], out[:, 1:7])


def test_attention_on_another_stream_and_captured():
    rng = np.random.default_rng(14)
    cache = random_cache(rng, 64, 2, 128, 16)
    q = torch.from_numpy(rng.standard_normal((2, 4, 128)).astype(np.float32)).cuda()
    lens, table = ints([500, 100]), ints(np.arange(64).reshape(2, 32))
    want = woq.kv4_attn(q, cache, lens, table)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = woq.kv4_attn(q, cache, lens, table, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    # one captured step, append and attention, follows the lengths that are on the device
    ws, out = woq.kv4_attn_workspace(cache, q), torch.empty_like(q)
    k, v = (torch.randn(2, 2, 128, device="cuda") for _ in "kv")
    start = lens - 1
    cu = ints([0, 1, 2])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        woq.kv4_append(cache, k, v, cu, table, start=start)
        woq.kv4_attn(q, cache, lens, table, out=out, workspace=ws)
    for n in ((500, 100), (17, 512), (1, 33)):
        lens.copy_(ints(n))
        start.copy_(lens - 1)
        k.normal_()
        graph.replay()
        got = out.clone()
        k2, _ = woq.kv4_gather(cache, cu, table, start=start, tokens=2)
        assert (k2 - k).abs().max() <= k.abs().max() / 7 * 0.501
        check = check_attention(cache, q, list(n), table.tolist())
        assert torch.equal(got, check)


def test_two_workspaces_on_two_streams():
    rng = np.random.default_rng(15)
    cache = random_cache(rng, 256, 2, 128, 64)
    q = torch.from_numpy(rng.standard_normal((4, 4, 128)).astype(np.float32)).cuda()
    lens, table = ints([4096, 4000, 3000, 17]), ints(np.arange(256).reshape(4, 64))
    want = woq.kv4_attn(q, cache, lens, table)
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [woq.kv4_attn_workspace(cache, q) for _ in streams]
    torch.cuda.synchronize()
    outs = [[woq.kv4_attn(q, cache, lens, table, workspace=w, stream=s) for _ in range(10)]
            for s, w in zip(streams, spaces)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for row in outs for o in row)


def test_no_tokens_and_interleaved_results():
    """Calls with no rows, a cache that is copied, and k and v gathered into one array [tokens, heads, 2, dim]."""
    torch.manual_seed(5)
    cache, cu, table = woq.KV4Cache.empty(3, 2, 64, 16), ints([0, 40]), ints([[2, 0, 1]])
    x = torch.randn(40, 2, 64, device="cuda")
    woq.kv4_append(cache, x, -x, cu, table)
    empty = torch.empty(0, 2, 64, device="cuda")
    before = cache.codes.clone()
    woq.kv4_append(cache, empty, empty, ints([0, 0]), table)
    k, v = woq.kv4_gather(cache, ints([0, 0]), table, tokens=0)
    assert k.shape == v.shape == empty.shape and torch.equal(cache.codes, before)
    assert woq.attn_prompt(empty, empty, empty, ints([0, 0])).shape == empty.shape
    k, v = woq.kv4_gather(cache, cu, table, tokens=40)
    both = torch.empty(40, 2, 2, 64, device="cuda")
    woq.kv4_gather(copy.deepcopy(cache), cu, table, k_out=both[:, :, 0], v_out=both[:, :, 1])
    assert torch.equal(both[:, :, 0], k) and torch.equal(both[:, :, 1], v) and torch.equal(v, -k)


@pytest.mark.parametrize("batch,length,kv", [(1, 2000, 8), (8, 300, 8), (32, 260, 8), (70, 200, 8), (3, 9000, 2)])
def test_attention_over_sequences_of_one_length(batch, length, kv):
    """Few and many sequences of one length: parts of a sequence's own, a sequence in each part, and more of both."""
    rng = np.random.default_rng(batch)
    page, dim = 64, 64
    width = -(-length // page)
    table = rng.permutation(batch * width).reshape(batch, width)
    cache = random_cache(rng, batch * width, kv, dim, page)
    q = torch.from_numpy(rng.standard_normal((batch, 2 * kv, dim)).astype(np.float32)).cuda()
    ws = woq.kv4_attn_workspace(cache, q)
    first = check_attention(cache, q, [length] * batch, table.tolist(), workspace=ws)
    for lens in ([length - 31] * batch, [(7 * b) % length for b in range(batch)], [length] + [0] * (batch - 1)):
        out = check_attention(cache, q, lens, table.tolist(), workspace=ws)
        assert torch.equal(woq.kv4_attn(q, cache, ints(lens), ints(table), workspace=ws), out)
    assert torch.equal(woq.kv4_attn(q, cache, ints([length] * batch), ints(table), workspace=ws), first)


def test_one_workspace_serves_calls_of_many_shapes():
    """Sized and zeroed once for the largest call; smaller and larger ones in turn, with sequences that parts share."""
    rng = np.random.default_rng(16)
    caches = {dim: random_cache(rng, 64, 8, dim, 64) for dim in (64, 128)}
    calls = []
    for batch, group, dim in ((8, 2, 128), (16, 2, 128), (3, 16, 128), (16, 16, 64), (8, 2, 64), (3, 2, 64), (16, 16, 128)):
        q = torch.from_numpy(rng.standard_normal((batch, 8 * group, dim)).astype(np.float32)).cuda()
        lens = rng.integers(1, 1024, batch)
        lens[0] = 4000
        calls.append((q, caches[dim], ints(lens), ints(rng.integers(0, 64, (batch, 63)))))
    want = [woq.kv4_attn(*c) for c in calls]
    sizes = [woq.kv4_attn_workspace(c[1], c[0]).nbytes for c in calls]
    ws = torch.zeros(max(sizes), dtype=torch.uint8, device="cuda")
    for i in (0, 1, 2, 3, 4, 5, 6, 0, 6, 5, 3, 1, 2, 4, 0):
        out = torch.full_like(want[i], 7.0)
        assert torch.equal(woq.kv4_attn(*calls[i], out=out, workspace=ws), want[i]), i
    assert woq.device_status() == _lib.WOQ_OK


def check_columns(cache, q, n, table, **kw):
    """One sequence's attention, with a tolerance by column: a token far above the others counts by its weight."""
    out = woq.kv4_attn(q, cache, ints([n]), ints([table]), **kw)
    k, v = ref.read_pages(cache.codes, cache.scales)
    at = [(table[j // cache.page], j % cache.page) for j in range(n)]
    kb, vb = (np.array([x[p, :, s] for p, s in at]) for x in (k, v))
    want, e, col = ref.attend_by_column(q[0].double().cpu().numpy(), kb, vb, cache.dim**-0.5)
    err = np.abs(out[0].double().cpu().numpy() - want)
    assert (err <= ref.tolerance_by_column(want, e, col, q.dtype)).all(), (err.max(), (err / (col + 1e-300)).max())
    assert woq.device_status() == _lib.WOQ_OK


def plain_cache(rng, pages, heads, dim, page):
    """Scales as kv4_append writes them of normal values."""
    cache = random_cache(rng, pages, heads, dim, page)
    s = np.abs(2.0 + 0.4 * rng.standard_normal(tuple(cache.scales.shape))) / 7
    cache.scales.copy_(torch.from_numpy(s.astype(np.float16)))
    return cache


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("score", [0.0, -6.0, -40.0])
@pytest.mark.parametrize("big", [8.0, 1024.0, 60000.0])
@pytest.mark.parametrize("at", [0, 150, 310])
def test_attention_a_value_far_above_the_others(dim, score, big, at):
    """One token's values are far above the others', in all blocks or in one, whatever its weight."""
    rng = np.random.default_rng(at)
    cache = plain_cache(rng, 20, 1, dim, 16)
    q = torch.from_numpy((0.2 + rng.random((1, 8, dim))).astype(np.float32)).cuda()
    # the token's key: codes -1, scales that bring its scores to about `score`
    cache.codes[at // 16, 0, 0, at % 16] = 0xFF
    cache.scales[at // 16, 0, at % 16, 0] = -score / (0.7 * dim**0.5)
    for blocks in (slice(None), slice(1, 2)):
        cache.scales[at // 16, 0, at % 16, 1, blocks] = big
        check_columns(cache, q, 311, list(range(20)))


@pytest.mark.parametrize("dim", [64, 128])
def test_attention_value_blocks_and_tokens_of_different_sizes(dim):
    rng = np.random.default_rng(18)
    nb, table = dim // 32, list(range(20))
    q = torch.from_numpy(rng.standard_normal((1, 8, dim)).astype(np.float32)).cuda()
    every = torch.arange(16, device="cuda")
    for low in (2.0**-8, 2.0**-12, 2.0**-15, 2.0**-20):
        for high in (1.0, 64.0, 30000.0):
            cache = plain_cache(rng, 20, 1, dim, 16)
            cache.scales[..., 1, 0] = low                       # one block of all tokens
            cache.scales[..., 1, nb - 1] = high
            check_columns(cache, q, 320, table)
            cache = plain_cache(rng, 20, 1, dim, 16)
            cache.scales[:, :, every % 3 == 0, 1] = low         # tokens in turn
            cache.scales[:, :, every % 3 == 1, 1] = high
            check_columns(cache, q, 320, table)
            cache.scales[:10, :, :, 1] = low                    # one part of the context, then the other
            cache.scales[10:, :, :, 1] = high
            check_columns(cache, q, 320, table)
            cache.scales[10:, :, 3, 1] = 0                      # and blocks of zeros
            check_columns(cache, q, 320, table)
            cache.scales[:10, :, :, 1] = high
            cache.scales[10:, :, :, 1] = low
            check_columns(cache, q, 320, table)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("gap", [5.0, 12.0, 25.0])
def test_attention_a_token_with_the_weight_and_small_values(dim, gap):
    """The first token has nearly all the weight and tiny values, or none: the others' small weights make the result."""
    rng = np.random.default_rng(19)
    for size in (0.5, 1e-3, 2.0**-22, 0.0):
        cache = plain_cache(rng, 70, 1, dim, 16)
        q = torch.from_numpy((0.2 + rng.random((1, 8, dim))).astype(np.float32)).cuda()
        cache.codes[0, 0, 0, 0] = 0x11
        cache.scales[0, 0, 0, 0] = gap / (0.7 * dim**0.5) + 1
        cache.scales[0, 0, 0, 1] = size
        cache.scales[:, :, :, 0] *= 0.1
        cache.scales[0, 0, 0, 0] *= 10
        check_columns(cache, q, 1111, list(range(70)))


def test_attention_turns_from_values_of_one_size_to_another_and_back():
    """Long stretches of large and of tiny values in turn, between which the scores fall and rise by tens."""
    rng = np.random.default_rng(20)
    cache = plain_cache(rng, 128, 2, 128, 64)
    for i in range(128):
        cache.scales[i, :, :, 1] *= (2.0**-14, 1.0, 2.0**12, 2.0**-8, 2.0**14)[i // 7 % 5]
        cache.scales[i, :, :, 0] *= (1.0, 0.25, 2.0)[i // 11 % 3]
    q = torch.from_numpy((3 * rng.standard_normal((1, 6, 128))).astype(np.float32)).cuda()
    check_columns(cache, q, 8190, list(range(128)))


@pytest.mark.parametrize("size", [2.0**20, 2.0**25, 2.0**27, 2.0**30, -(2.0**25), -(2.0**28), -(2.0**30)])
def test_attention_scores_far_from_zero(size):
    """Scores that are exact whole numbers times `size`: equal ones share the weight, others have none of it."""
    rng = np.random.default_rng(22)
    cache = plain_cache(rng, 20, 1, 64, 16)
    cache.codes[:, :, 0] = 0x11
    cache.scales[:, :, :, 0] = torch.from_numpy(rng.integers(1, 4, (20, 1, 16, 2)).astype(np.float16)).cuda()
    cache.scales[:7, :, :, 0] = 2.0
    cache.scales[:, :, :, 0, 1:] = 0
    q = torch.zeros(1, 2, 64, device="cuda")
    q[0, :, 5] = size
    out = woq.kv4_attn(q, cache, ints([320]), ints([list(range(20))]), scale=1.0)[0].double().cpu().numpy()
    k, v = ref.read_pages(cache.codes, cache.scales)
    x = k[:, 0, :, 5].reshape(-1) * size
    p = np.exp(x - x.max())
    p /= p.sum()
    v = v[:, 0].reshape(-1, 64)
    big = np.repeat(np.abs(v).reshape(-1, 2, 32).max(-1), 32, axis=-1)
    assert (np.abs(out - p @ v) <= ref.tolerance_by_column(p @ v, 0.0, p @ big, q.dtype)).all()


def test_attention_a_wait_that_gives_up_is_reported_and_the_context_survives():
    rng = np.random.default_rng(21)
    cache = random_cache(rng, 64, 2, 128, 64)
    q = torch.from_numpy(rng.standard_normal((2, 4, 128)).astype(np.float32)).cuda()
    lens, table = ints([2048, 1500]), ints(np.arange(64).reshape(2, 32))
    ws = woq.kv4_attn_workspace(cache, q)
    want = woq.kv4_attn(q, cache, lens, table, workspace=ws)
    assert woq.device_status(clear=True) == _lib.WOQ_OK
    L = _lib.lib()
    try:
        L.woq_debug_set_wait_limit(-200000)
        woq.kv4_attn(q, cache, lens, table, workspace=ws)
        assert woq.device_status(clear=True) == _lib.WOQ_ETIMEOUT
    finally:
        L.woq_debug_set_wait_limit(0)
    ws.zero_()
    assert torch.equal(woq.kv4_attn(q, cache, lens, table, workspace=ws), want)
    assert woq.device_status(clear=True) == _lib.WOQ_OK
