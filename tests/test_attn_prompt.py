"""attn_prompt against causal attention in 64 bits."""

import numpy as np
import pytest
import torch

import weight_only_bit_qgemv_b200 as woq
from weight_only_bit_qgemv_b200 import _lib
from tests import attn_ref as ref

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.float16, torch.bfloat16]


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def fused(seed, tokens, heads, kv, dim, dtype):
    """Slices of one projection's rows: queries, keys, values."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(tokens, heads + 2 * kv, dim, generator=g).to(dtype).cuda()
    return x[:, :heads], x[:, heads:heads + kv], x[:, heads + kv:]


def exact(q, k, v, cu, scale):
    """(result, its tolerance) in float64, on the GPU: rows of no sequence are 0 with tolerance 0."""
    dtype, heads, group = q.dtype, q.shape[1], q.shape[1] // k.shape[1]
    q, k, v = (x.double() for x in (q, k, v))
    out, tol = torch.zeros_like(q), torch.zeros_like(q)
    products = 22 if dtype == torch.float32 else 60  # 16-bit operands take part as they are
    weight = 0.0 if dtype == torch.float32 else ref.UNIT[dtype]
    for a, b in zip(cu[:-1], cu[1:]):
        for h in range(heads):
            kh, vh = k[a:b, h // group], v[a:b, h // group]
            for i in range(a, b, 2048):
                j = min(b, i + 2048)
                x = q[i:j, h] @ kh[:j - a].T * scale
                seen = torch.arange(j - a, device="cuda") <= torch.arange(i - a, j - a, device="cuda")[:, None]
                p = torch.softmax(x.masked_fill(~seen, -torch.inf), -1)
                out[i:j, h] = p @ vh[:j - a]
                # ref.tolerance's derivation, with sums over what a row sees: FP32 sums of a score's 2^7 terms add
                # 2^-17 of sum |q k| at most (rounding to nothing, 2^-24 a step), a rounded weight half a step of
                # it on either side of the quotient
                e = (2.0 ** (2 - products) + 2.0**-17) * (q[i:j, h].abs() @ kh[:j - a].abs().T * scale)
                e = e.masked_fill(~seen, 0).amax(-1, keepdim=True)
                tol[i:j, h] = (2 * e + 2.0**-18 + 2 * weight) * (p @ vh[:j - a].abs())
                # weights of up to 2^-25 of the largest are lost in binary16, and its subnormals' steps
                tol[i:j, h] += (2.0**-25 if dtype == torch.float16 else 0.0) * seen.sum(-1, keepdim=True) * vh.abs().max()
    unit = 0.0 if dtype == torch.float32 else ref.UNIT[dtype]
    return out, tol + unit * out.abs() + (6e-8 if dtype == torch.float16 else 0.0)


def check(q, k, v, cu, scale=None, **kw):
    out = woq.attn_prompt(q, k, v, ints(cu), scale=scale, **kw)
    want, tol = exact(q, k, v, cu, q.shape[2] ** -0.5 if scale is None else scale)
    for a, b in zip(cu[:-1], cu[1:]):
        err = (out[a:b].double() - want[a:b]).abs()
        assert (err <= tol[a:b]).all(), ((a, b), err.max().item(), (err - tol[a:b]).max().item())
    assert woq.device_status() == _lib.WOQ_OK
    return out


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("heads,kv,dim,lens", [
    (1, 1, 64, [1]),
    (1, 1, 128, [2]),
    (2, 1, 128, [63, 64, 65, 0, 127, 128, 129]),          # around the tiles of keys and rows
    (4, 4, 64, [255, 256, 257, 0, 0, 1]),
    (6, 2, 128, [700, 3]),
    (16, 8, 128, [137]),
    (5, 1, 64, [383, 385, 511, 513]),
    (8, 1, 128, [1030]),
])
def test_matches_the_formula(dtype, heads, kv, dim, lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    q, k, v = fused(heads + dim + len(lens), cu[-1], heads, kv, dim, dtype)
    check(q, k, v, cu)


@pytest.mark.parametrize("dtype", TYPES)
def test_long_prompts(dtype):
    cu = [0, 4999, 5000, 9201]
    q, k, v = fused(3, cu[-1], 2, 1, 128, dtype)
    check(q, k, v, cu)


def test_many_short_sequences():
    """More sequences than one pass over their ends holds, most of them of a few rows."""
    lens = [(i * 37) % 19 for i in range(200)]
    cu = np.concatenate([[0], np.cumsum(lens)]).tolist()
    q, k, v = fused(4, cu[-1], 2, 2, 64, torch.float32)
    check(q, k, v, cu)


@pytest.mark.parametrize("dtype", TYPES)
def test_rows_outside_the_sequences(dtype):
    """Rows before, behind and between hold NaN: they are not written and have no influence."""
    cu = [5, 5 + 130, 5 + 130 + 20]
    q, k, v = fused(5, 170, 4, 2, 128, dtype)
    for x in (q, k, v):
        x[:5] = float("nan")
        x[155:] = float("inf")
    out = torch.full((170, 4, 128), 7.0, dtype=dtype, device="cuda")
    check(q, k, v, cu, out=out)
    assert (out[:5] == 7).all() and (out[155:] == 7).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("at", [0, 100, 131, 255, 300])
def test_values_that_are_not_finite_enter_only_rows_that_see_them(dtype, at):
    cu = [0, 301, 420]
    q, k, v = fused(6, 420, 4, 2, 64, dtype)
    clean = woq.attn_prompt(q, k, v, ints(cu))
    v2 = v.clone()
    v2[at, 0, 9], v2[at, 1, 3] = float("nan"), float("inf")
    out = woq.attn_prompt(q, k, v2, ints(cu))
    hit = torch.zeros(420, 4, 64, dtype=torch.bool, device="cuda")
    hit[at:301, :2, 9] = True
    hit[at:301, 2:, 3] = True
    assert torch.equal(~out.isfinite(), hit)

    def same():
        # float32: what is not finite has no part in its tile's power of two, so bits below 2^-22 may move
        if dtype != torch.float32:
            return torch.equal(out[~hit], clean[~hit])
        return (out[~hit] - clean[~hit]).abs().max() <= 2.0**-16 * v.abs().max()

    assert same()
    assert out[at, 2, 3] == float("inf")
    # keys and queries: rows that see one are NaN as a whole, the others as they were
    k2 = k.clone()
    k2[at, 0, 1] = float("nan")
    out = woq.attn_prompt(q, k2, v, ints(cu))
    hit[:] = False
    hit[at:301, :2] = True
    assert torch.equal(out.isnan(), hit) and same()
    q2 = q.clone()
    q2[at, 1, 5] = float("nan")
    out = woq.attn_prompt(q2, k, v, ints(cu))
    hit[:] = False
    hit[at, 1] = True
    assert torch.equal(out.isnan(), hit) and same()


@pytest.mark.parametrize("dtype", TYPES)
def test_scores_far_apart_and_sizes_far_from_one(dtype):
    cu = [0, 400, 600]
    q, k, v = fused(7, 600, 4, 2, 128, dtype)
    check(q * 30, k, v, cu)                       # one key has nearly all the weight
    check(q, k, v, cu, scale=1e-4)                # all keys weigh the same
    check(torch.zeros_like(q), k, v, cu)
    if dtype == torch.float32:
        check(q * 1e-18, k * 1e18, v * 1e-25, cu)
        check(q * 1e12, k * 1e-12, v * 1e30, cu)
        grow = torch.logspace(-6, 6, 600, device="cuda")[:, None, None]
        check(q / grow, k, v * grow, cu)          # each tile with powers of two of its own
    if dtype == torch.bfloat16:
        check(q, k, v * 1e30, cu)


@pytest.mark.parametrize("dtype", TYPES)
def test_one_key_far_above_the_others(dtype):
    """Row maxima that rise late: what was summed before is scaled down to nothing."""
    q, k, v = fused(8, 520, 2, 1, 64, dtype)
    k = k.clone()
    k[300] = q[300, :1] * 6
    check(q, k, v, [0, 520])


def test_strides_and_neighbours():
    q, k, v = fused(9, 300, 6, 3, 128, torch.float32)
    wide = torch.full((300, 10, 160), 7.0, device="cuda")
    check(q, k, v, [0, 300], out=wide[:, 2:8, 16:144])
    assert (wide[:, :2] == 7).all() and (wide[:, 8:] == 7).all()
    assert (wide[..., :16] == 7).all() and (wide[..., 144:] == 7).all()
    heads_first = q.transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(woq.attn_prompt(heads_first, k, v, ints([0, 300])), wide[:, 2:8, 16:144])


@pytest.mark.parametrize("dtype", TYPES)
def test_rows_of_heads_stored_head_after_head(dtype):
    q, k, v = fused(13, 300, 4, 2, 64, dtype)
    want = woq.attn_prompt(q, k, v, ints([0, 300]))
    q, k, v = (x.transpose(0, 1).contiguous().transpose(0, 1) for x in (q, k, v))
    out = torch.empty(4, 300, 64, dtype=dtype, device="cuda").transpose(0, 1)
    assert torch.equal(woq.attn_prompt(q, k, v, ints([0, 300]), out=out), want)
    with pytest.raises(woq.WoqError):
        woq.attn_prompt(q[:, :1].expand(-1, 4, -1), k, v, ints([0, 300]))  # a stride of 0


@pytest.mark.parametrize("dtype", TYPES)
def test_same_bits_every_time_captured_and_on_another_stream(dtype):
    cu = ints([0, 700, 900])
    q, k, v = fused(10, 900, 4, 2, 128, dtype)
    want = woq.attn_prompt(q, k, v, cu)
    for _ in range(3):
        assert torch.equal(woq.attn_prompt(q, k, v, cu), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = woq.attn_prompt(q, k, v, cu, stream=side, out=torch.zeros_like(want))
    side.synchronize()
    assert torch.equal(got, want)
    ws, out = woq.attn_prompt_workspace(q, k, 2), torch.zeros_like(want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        woq.attn_prompt(q, k, v, cu, out=out, workspace=ws)
        woq.attn_prompt(q, k, v, cu, out=out, workspace=ws)  # shares the workspace, ordered behind it
    for ends in ([0, 700, 900], [0, 1, 900], [10, 450, 451]):  # other lengths in the same graph
        cu.copy_(ints(ends))
        out.zero_()
        graph.replay()
        assert torch.equal(out, woq.attn_prompt(q, k, v, cu))


def test_more_tokens_than_the_sequences_have_and_ends_out_of_order():
    q, k, v = fused(11, 500, 2, 1, 64, torch.float32)
    out = woq.attn_prompt(q, k, v, ints([0, 0, 0]))
    assert not out.any()
    # ends that are no ends: nothing outside the rows is read or written, and a good sequence is right
    out = torch.full((600, 2, 64), 7.0, device="cuda")
    woq.attn_prompt(q, k, v, ints([0, 100, -5, 2**31 - 1, 50]), out=out[:500])
    assert (out[500:] == 7).all() and woq.device_status() == _lib.WOQ_OK


def test_a_stuck_wait_gives_up_and_the_context_survives():
    q, k, v = fused(12, 300, 2, 1, 128, torch.float32)
    want = woq.attn_prompt(q, k, v, ints([0, 300]))
    L = _lib.lib()
    assert woq.device_status(clear=True) == _lib.WOQ_OK
    try:
        L.woq_debug_set_wait_limit(-200000)
        woq.attn_prompt(q, k, v, ints([0, 300]))
        assert woq.device_status(clear=True) == _lib.WOQ_ETIMEOUT
    finally:
        L.woq_debug_set_wait_limit(0)
    assert torch.equal(woq.attn_prompt(q, k, v, ints([0, 300])), want)
    assert woq.device_status(clear=True) == _lib.WOQ_OK


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128])
def test_many_more_tiles_than_blocks_run_at_once(dtype, dim):
    """A block goes on from tile to tile: sequences of one to a few tiles of rows, some empty, some with values that
    are not finite, and the same bits on every call."""
    lens = [300, 1, 0, 513, 64, 900, 257, 5, 0, 1100, 128, 256, 129, 31] * 3
    cu = np.concatenate([[0], np.cumsum(lens)]).tolist()
    q, k, v = fused(14, cu[-1], 24, 8, dim, dtype)
    out = check(q, k, v, cu)
    for _ in range(3):
        assert torch.equal(woq.attn_prompt(q, k, v, ints(cu)), out)
    v2 = v.clone()
    hit = torch.zeros(out.shape, dtype=torch.bool, device="cuda")
    for i in range(0, len(lens), 3):  # the last value of every third sequence
        if lens[i]:
            v2[cu[i + 1] - 1, 3, 17] = float("inf")
            hit[cu[i + 1] - 1, 9:12, 17] = True
    got = woq.attn_prompt(q, k, v2, ints(cu))
    assert torch.equal(~got.isfinite(), hit)
    if dtype != torch.float32:  # float32: such a value has no part in its tile's power of two
        assert torch.equal(got[~hit], out[~hit])
    assert woq.device_status() == _lib.WOQ_OK


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_thousands_of_sequences(dtype):
    """Tiles are looked up among many sequences: 5000 of one to three rows and every other one empty."""
    lens = [(i % 2) * (1 + i % 3) for i in range(10000)]
    cu = np.concatenate([[0], np.cumsum(lens)]).tolist()
    q, k, v = fused(15, cu[-1], 3, 1, 64, dtype)
    out = woq.attn_prompt(q, k, v, ints(cu))
    seq = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), torch.tensor(lens, device="cuda"))
    x = torch.einsum("ihd,jd->hij", q.double(), k[:, 0].double()) / 8
    row = torch.arange(cu[-1], device="cuda")
    seen = (seq[:, None] == seq) & (row[:, None] >= row)
    for i in range(0, cu[-1], 2000):
        j = min(i + 2000, cu[-1])
        p = torch.softmax(x[:, i:j].masked_fill(~seen[None, i:j], -torch.inf), -1)
        want = torch.einsum("hij,jd->ihd", p, v[:, 0].double())
        # exact()'s tolerance: three keys at most
        size = torch.einsum("hij,jd->ihd", p, v[:, 0].double().abs())
        e = (2.0**-20 if dtype == torch.float32 else 2.0**-58) + 2.0**-17
        e = e * (q[i:j].double().abs().sum(-1) * k.double().abs().max() / 8)[..., None]  # above every sum |q k| scale
        unit = 0.0 if dtype == torch.float32 else ref.UNIT[dtype]
        assert ((out[i:j].double() - want).abs() <= (2 * e + 2.0**-18 + 2 * unit) * size + unit * want.abs()).all()
    assert woq.device_status() == _lib.WOQ_OK


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_thousands_of_empty_sequences(dtype):
    """Many more blocks than tiles: what there is of rows belongs to no sequence, or to the last one."""
    q, k, v = fused(16, 600, 4, 2, 64, dtype)
    out = torch.full((600, 4, 64), 7.0, dtype=dtype, device="cuda")
    woq.attn_prompt(q, k, v, torch.full((20001,), 600, dtype=torch.int32, device="cuda"), out=out)
    assert (out == 7).all()
    cu = torch.zeros(20001, dtype=torch.int32, device="cuda")
    cu[-1] = 600
    assert torch.equal(woq.attn_prompt(q, k, v, cu), woq.attn_prompt(q, k, v, ints([0, 600])))
    assert woq.device_status() == _lib.WOQ_OK


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("size", [2.0**20, 2.0**25, 2.0**27, 2.0**30, -(2.0**25), -(2.0**28), -(2.0**30)])
def test_scores_far_from_zero(dtype, size):
    """Scores that are exact whole numbers times `size`: equal ones share the weight, others have none of it."""
    n, dim = 300, 64
    g = torch.Generator().manual_seed(3)
    a = torch.randint(1, 4, (n,), generator=g).cuda()
    q = torch.zeros(n, 1, dim, device="cuda")
    k = torch.zeros(n, 1, dim, device="cuda")
    half = 2.0 ** round(np.log2(abs(size)) / 2)
    q[:, 0, 3:5], k[:, 0, 3:5] = half, a[:, None] * (size / half / 2)  # two halves: binary16 has no 3 * 2^15
    k[:100, 0, 3:5] = size / half / 2  # the first 100 are all the same
    v = torch.randn(n, 1, dim, generator=g).cuda()
    q, k, v = (x.to(dtype) for x in (q, k, v))
    out = woq.attn_prompt(q, k, v, ints([0, n]), scale=1.0).double()
    x = torch.tril(torch.ones(n, n, dtype=torch.float64, device="cuda")).log() + k[:, 0, 3].double() * 2 * half
    p = torch.softmax(x, -1)
    want, col = p @ v[:, 0].double(), p @ v[:, 0].double().abs()
    # exact()'s tolerance without the scores', which are exact
    unit = 0.0 if dtype == torch.float32 else ref.UNIT[dtype]
    assert ((out[:, 0] - want).abs() <= (2.0**-18 + 2 * unit) * col + unit * want.abs()).all()
    assert woq.device_status() == _lib.WOQ_OK


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("size", [1e6, 1e12, 1e30])
@pytest.mark.parametrize("at", [0, 1, 40, 63, 64, 100])
def test_rows_before_a_far_larger_one_keep_their_precision(dim, size, at):
    """float32: a key's or value's size has no influence on the rows before it, and none on the keys and values beside."""
    cu = [3, 3 + 150, 3 + 150 + 70]
    q, k, v = fused(17, cu[-1], 4, 2, dim, torch.float32)
    v2 = v.clone()
    v2[3 + at] *= size
    check(q, k, v2, cu)
    v2[3 + at, 0] = v[3 + at, 0]
    v2[3 + at, 0, 5] = size
    # the columns beside the large one are bounded by it from that row on, as by one value of 22 bits
    out = woq.attn_prompt(q, k, v2, ints(cu))
    want, tol = exact(q, k, v2, cu, dim**-0.5)
    tol[3 + at:cu[1], :2] += 2.0**-36 * size
    assert ((out.double() - want).abs() <= tol).all()
    k2 = k.clone()
    k2[3 + at] *= size
    if size < 1e30:  # the scores of the rows that see it are beyond 32 bits otherwise
        check(q, k2, v, cu)
        check(q, k2, v2, [3, 3 + at, 3 + at, cu[1], cu[2]][(at == 0):])
    else:
        out = woq.attn_prompt(q, k2, v, ints(cu))
        want, tol = exact(q, k, v, cu, dim**-0.5)
        assert ((out.double() - want).abs() <= tol)[3:3 + at].all()
        assert ((out.double() - want).abs() <= tol)[cu[1]:].all()


@pytest.mark.parametrize("dim", [64, 128])
def test_rows_of_very_different_sizes(dim):
    """float32: every row of a tile has a size of its own, zeros among them; and a large weight on tiny values."""
    cu = [0, 130, 331]
    q, k, v = fused(18, cu[-1], 4, 2, dim, torch.float32)
    g = torch.Generator().manual_seed(1)
    sizes = torch.exp2(torch.randint(-60, 61, (cu[-1], 1, 1), generator=g).float()).cuda()
    check(q, k, v * sizes, cu)
    few = torch.exp2(torch.randint(-30, 1, (cu[-1], 1, 1), generator=g).float()).cuda()
    check(q, k * few, v, cu)
    check(q, k * few, v * sizes, cu)
    v2 = v * sizes
    v2[::7] = 0
    k2 = k * few
    k2[::5] = 0
    check(q, k2, v2, cu)
    k2 = k.clone()
    k2[0], k2[130] = 2.0, 2.0
    q2 = q.abs() + 0.1
    v2 = v.clone()
    v2[0] *= 1e-6
    v2[130] = 0
    check(q2, k2 * 0.3, v2, cu)
    out = woq.attn_prompt(q2, k2 * 0.3, v2 * sizes, ints(cu))
    for _ in range(3):
        assert torch.equal(woq.attn_prompt(q2, k2 * 0.3, v2 * sizes, ints(cu)), out)


@pytest.mark.parametrize("dim", [64, 128])
def test_rows_of_very_different_sizes_that_are_not_finite(dim):
    """float32: infinities and NaN beside finite values of all sizes."""
    cu = [0, 301]
    q, k, v = fused(19, 301, 4, 2, dim, torch.float32)
    g = torch.Generator().manual_seed(2)
    v = v * torch.exp2(torch.randint(-40, 41, (301, 1, 1), generator=g).float()).cuda()
    want, tol = exact(q, k, v, cu, dim**-0.5)
    for at in (0, 100, 255, 300):
        v2 = v.clone()
        v2[at, 0, 9], v2[at, 1, 3] = float("nan"), float("inf")
        out = woq.attn_prompt(q, k, v2, ints(cu))
        hit = torch.zeros(out.shape, dtype=torch.bool, device="cuda")
        hit[at:, :2, 9] = True
        hit[at:, 2:, 3] = True
        assert torch.equal(~out.isfinite(), hit)
        assert ((out.double() - want).abs() <= tol)[~hit].all()


def test_values_next_to_the_end_of_the_range():
    """Finite values of up to 1e37: their weighted means are finite, and so are the sums on the way."""
    for dim in (64, 128):
        q, k, v = fused(20, 40, 2, 1, dim, torch.float32)
        check(q, k, v.clamp(-3, 3) * 3e36, [0, 7, 8, 19, 40])  # a sum of 21 of them fits 32 bits
        # a key in a later tile takes over, just less than 2^8 above the others before it. A sum of weights of at most 1 is
        # 200e36 at most, which 32 bits hold; with the key's weight as 233 instead of 1 it would be 383e36
        for dtype in (torch.float32, torch.bfloat16):
            q = torch.ones(200, 1, dim, dtype=dtype, device="cuda")
            k = torch.zeros(200, 1, dim, dtype=dtype, device="cuda")
            k[150] = 5.45 / dim**0.5
            v = torch.full((200, 1, dim), 1e36, dtype=dtype, device="cuda")
            check(q, k, v, [0, 200])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("value", [float("inf"), -float("inf")])
@pytest.mark.parametrize("at", [0, 100, 200, 300])
def test_infinite_keys_and_queries(dtype, value, at):
    """float32: a row that sees an infinity in a key, or has one, is NaN. 16-bit rows go by the scores: one of -infinity
    weighs nothing, one of +infinity and NaN make the row NaN."""
    cu = [0, 301, 420]
    q, k, v = fused(21, 420, 4, 2, 64, dtype)
    clean, bound = exact(q, k, v, cu, 0.125)
    q2, k2 = q.clone(), k.clone()
    k2[at, 0, 1] = value
    out = woq.attn_prompt(q, k2, v, ints(cu))
    hit = torch.zeros(420, 4, 64, dtype=torch.bool, device="cuda")
    hit[at:301, :2] = True
    if dtype == torch.float32:
        assert torch.equal(out.isnan(), hit)
    else:
        want, tol = exact(q, k2, v, cu, 0.125)
        assert want.isnan().any() and torch.equal(out.isnan(), want.isnan())
        assert at == 300 or want[at + 1:301, :2].isfinite().any()  # the last row has no others behind it
        seen = want.isfinite() & tol.isfinite()  # rows that see it have an infinite bound
        assert ((out.double() - want).abs() <= tol)[seen].all()
        # of those, exact()'s terms with what bounds them: half a step of weight and result, three in all, of at most max |v|,
        # and of the finite scores, whose sum |q k| scale is below 64 here, 2^-16 of that: two half steps of binary16
        want = want[at:301, :2]
        assert ((out[at:301, :2].double() - want).abs() <= 8 * ref.UNIT[dtype] * v.abs().max())[want.isfinite()].all()
    # The other rows are as exact as without it. They need not have the same bits: rows of a warp are scaled down together.
    assert ((out.double() - clean).abs() <= bound)[~hit].all()
    q2[at, 1, 5] = value
    out = woq.attn_prompt(q2, k, v, ints(cu))
    hit[:] = False
    hit[at, 1] = True
    assert torch.equal(out.isnan(), hit) and ((out.double() - clean).abs() <= bound)[~hit].all()


@pytest.mark.parametrize("dtype", TYPES)
def test_ends_out_of_order_leave_the_sequences_beside_them_right(dtype):
    q, k, v = fused(22, 500, 2, 1, 64, dtype)
    out = woq.attn_prompt(q, k, v, ints([-7, 0, 100, 300, 250, 2**31 - 1]))
    want, tol = exact(q, k, v, [0, 100], 0.125)  # rows 250..299 are two sequences', and 300.. see them
    assert ((out.double() - want).abs() <= tol)[:100].all()
    want, tol = exact(q, k, v, [100, 300], 0.125)
    assert ((out.double() - want).abs() <= tol)[100:192].all()  # whole tiles of 64 rows before the shared ones
    assert woq.device_status() == _lib.WOQ_OK


@pytest.mark.parametrize("dim", [64, 128])
def test_tiny_rows_of_very_different_sizes(dim):
    """float32: values of 1e-27 and less in tiles with a power for each row, behind a tile with nearly all the weight."""
    cu = [0, 300]
    q, k, v = fused(23, 300, 4, 2, dim, torch.float32)
    g = torch.Generator().manual_seed(4)
    sizes = torch.exp2(torch.randint(-15, 1, (300, 1, 1), generator=g).float()).cuda() * 1e-27
    q, k2 = q.abs() + 0.1, k * 0.1
    k2[:20] = 2.0 * (dim / 64) ** -0.5  # scores of 16 and more above the others
    v2 = v * sizes
    v2[:20] = v[:20] * 1e-33
    out = woq.attn_prompt(q, k2, v2, ints(cu)).double()
    want, tol = exact(q, k2, v2, cu, dim**-0.5)
    assert ((out - want).abs() <= tol).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("size", [2.0**13, 0.999 * 2.0**15, 1.001 * 2.0**15, 2.0**16, 2.0**18])
def test_equal_scores_about_where_they_count_as_far_from_zero(dtype, sign, size):
    """All products at the upper end of their powers of two: scores of 506 `size` to base 2, all the same."""
    q = torch.full((200, 2, 128), 1.9921875, dtype=dtype, device="cuda")
    k = sign * q[:, :1].contiguous()
    v = torch.randn(200, 1, 128, generator=torch.Generator().manual_seed(5)).to(dtype).cuda()
    out = woq.attn_prompt(q, k, v, ints([0, 70, 200]), scale=size / 1.4426950408889634).double()
    unit = 0.0 if dtype == torch.float32 else ref.UNIT[dtype]
    for a, b in ((0, 70), (70, 200)):
        count = torch.arange(1, b - a + 1, device="cuda", dtype=torch.float64)[:, None]
        want, col = (x.double().cumsum(0) / count for x in (v[a:b, 0], v[a:b, 0].abs()))
        tol = (2.0**-18 + 2 * unit) * col + unit * want.abs()
        assert ((out[a:b] - want[:, None]).abs() <= tol[:, None]).all()
