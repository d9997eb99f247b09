"""What the decoder's attention operators compute and cost: cases, inputs, plain forms and definitions in 64 bits.

Three operators that stand between a decoder layer's packed matrix products:

* ``prompt``: causal attention over whole prompts, packed one after another, with grouped heads;
* ``decode``: one token a sequence attends to a paged cache held in 4 bits;
* ``store``: new keys and values are quantised into that cache and read back from it.

Cache layout: codes ``[pages, kv_heads, 2 (k, v), page, dim / 2]`` bytes and scales ``[pages, kv_heads, page, 2 (k, v),
dim / 32]`` binary16. A row is 32-element blocks of two's-complement nibbles, element 2j in the low half of byte j;
of a key row the 32-bit words are stored transposed from [block, 4] to [4, block], of a value row the 16-bit
halfwords from [block, 8] to [8, block].
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# ---- cases ---------------------------------------------------------------------------------------------------------

def listed():
    return [
        # a short text prompt: latency
        {"name": "prompt_137_f32", "op": "prompt", "type": "f32", "heads": 16, "kv_heads": 8, "dim": 128,
         "batch": 1, "shortest": 137, "longest": 137},
        # one long recording's prompt in the library's own activation type
        {"name": "prompt_4096_f32", "op": "prompt", "type": "f32", "heads": 16, "kv_heads": 8, "dim": 128,
         "batch": 1, "shortest": 4096, "longest": 4096},
        # a batch of requests with prompts of odd lengths, packed
        {"name": "prompt_packed_f32", "op": "prompt", "type": "f32", "heads": 16, "kv_heads": 8, "dim": 128,
         "batch": 24, "shortest": 11, "longest": 2011},
        # the same in 16 bits with eight query heads to a key head
        {"name": "prompt_packed_bf16", "op": "prompt", "type": "bf16", "heads": 32, "kv_heads": 4, "dim": 128,
         "batch": 16, "shortest": 301, "longest": 4003},
        # a very long prompt
        {"name": "prompt_32k_bf16", "op": "prompt", "type": "bf16", "heads": 16, "kv_heads": 8, "dim": 128,
         "batch": 1, "shortest": 32768, "longest": 32768},
        # narrow heads, no sharing, odd lengths
        {"name": "prompt_d64_f16", "op": "prompt", "type": "f16", "heads": 12, "kv_heads": 12, "dim": 64,
         "batch": 3, "shortest": 1, "longest": 5003},
        # one user, a short context: latency
        {"name": "decode_1x1k_f32", "op": "decode", "type": "f32", "heads": 16, "kv_heads": 8, "dim": 128,
         "batch": 1, "shortest": 1000, "longest": 1000, "page": 64},
        # batched serving, contexts of all lengths
        {"name": "decode_64_ragged_f32", "op": "decode", "type": "f32", "heads": 16, "kv_heads": 8, "dim": 128,
         "batch": 64, "shortest": 1, "longest": 8191, "page": 64},
        # a few users with very long contexts
        {"name": "decode_4x128k_f32", "op": "decode", "type": "f32", "heads": 16, "kv_heads": 8, "dim": 128,
         "batch": 4, "shortest": 100003, "longest": 131072, "page": 128},
        # eight query heads to a key head, small pages
        {"name": "decode_16_g8_bf16", "op": "decode", "type": "bf16", "heads": 64, "kv_heads": 8, "dim": 128,
         "batch": 16, "shortest": 2049, "longest": 16001, "page": 16},
        # the cache's side of one decode step
        {"name": "store_step_64_f32", "op": "store", "type": "f32", "heads": 16, "kv_heads": 8, "dim": 128,
         "batch": 64, "shortest": 1, "longest": 1, "page": 64},
        # the cache's side of a long prefill
        {"name": "store_prompts_f32", "op": "store", "type": "f32", "heads": 16, "kv_heads": 8, "dim": 128,
         "batch": 9, "shortest": 511, "longest": 8190, "page": 64},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "decode", "decode", "store"])
    kv = rng.choice([1, 2, 4, 8])
    case = {"op": op, "type": rng.choice(["f32", "f32", "bf16", "f16"]), "heads": kv * rng.choice([1, 2, 4, 5, 8]),
            "kv_heads": kv, "dim": rng.choice([64, 128, 128])}
    if op == "prompt":
        most, batch = 8192 if case["type"] == "f32" else 16384, _log(rng, 1, 32)
        most = min(most, 40000 // batch, math.isqrt(int(4e12 / (2 * case["dim"] * case["heads"] * batch))))
        longest = _log(rng, 1, most)
    elif op == "decode":
        batch = _log(rng, 1, 128)
        longest = _log(rng, 16, min(131072, 400000 // batch))
    else:
        batch = _log(rng, 1, 64)
        longest = _log(rng, 1, min(16384, 40000 // batch))
    case.update(batch=batch, longest=longest, shortest=rng.randint(1, longest))
    if op != "prompt":
        case["page"] = rng.choice([16, 32, 64, 128])
    return case


def _lengths(case):
    """The sequences' lengths: they go by the case alone, so that its work does too."""
    lo, hi, n = case["shortest"], case["longest"], case["batch"]
    if n == 1:
        return [hi]
    mix = [(i * 7919 + 13) % n for i in range(n)] if n % 7919 else list(range(n))
    return [lo + (hi - lo) * m // (n - 1) for m in mix]


def work(case):
    lens = _lengths(case)
    hq, hk, d = case["heads"], case["kv_heads"], case["dim"]
    size, total = torch.empty(0, dtype=DTYPES[case["type"]]).element_size(), sum(lens)
    row = 2 * (d // 2 + d // 16)  # one token's codes and scales of one key head, key and value
    if case["op"] == "prompt":
        return {"bytes": total * (2 * hq + 2 * hk) * d * size, "flops": sum(2 * d * hq * n * (n + 1) for n in lens)}
    if case["op"] == "decode":
        return {"bytes": total * hk * row + 2 * case["batch"] * hq * d * size, "flops": 4 * total * hq * d}
    # rows in, codes and scales out, the same codes and scales in, rows out in 32 bits
    return {"bytes": total * hk * (2 * d * size + 2 * row + 2 * d * 4), "flops": 6 * total * hk * d}


# ---- inputs --------------------------------------------------------------------------------------------------------

def prepare(case, seed):
    if own:
        import weight_only_bit_qgemv_b200 as woq
    g = torch.Generator(device="cuda").manual_seed(seed)
    lens, dt = _lengths(case), DTYPES[case["type"]]
    hq, hk, d, n = case["heads"], case["kv_heads"], case["dim"], case["batch"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    state = {"case": dict(case), "lens": lens, "scale": d ** -0.5}
    ends = [0]
    for x in lens:
        ends.append(ends[-1] + x)
    ints = dict(dtype=torch.int32, device="cuda")
    if case["op"] != "decode":
        # one fused projection's rows: queries, keys, values; some key channels stand out, as they do in earnest
        rows = normal(ends[-1], hq + 2 * hk, d)
        rows[:, :hq] *= 1.5
        rows[:, hq:hq + hk] += 2.0 * normal(hk, d) * (torch.rand(hk, d, generator=g, device="cuda") < 0.05)
        rows = rows.to(dt)
        state.update(q=rows[:, :hq], k=rows[:, hq:hq + hk], v=rows[:, hq + hk:], cu=torch.tensor(ends, **ints))
    if case["op"] == "prompt":
        if own:
            state["out"] = torch.empty(ends[-1], hq, d, dtype=dt, device="cuda")
            state["ws"] = woq.attn_prompt_workspace(state["q"], state["k"], n)
        return state

    page = case["page"]
    # a decode step adds one token behind what is there; a prompt starts an empty sequence
    before = [(i * 1777 + 5) % (4 * page) for i in range(n)] if case["op"] == "store" and case["longest"] == 1 else [0] * n
    width = max(-(-(x + b) // page) for x, b in zip(lens, before))
    need = n * width
    state["table"] = torch.randperm(need, generator=g, device="cuda").to(torch.int32).view(n, width)
    pool = (need, hk, 2, page, d // 2)
    if case["op"] == "store":
        state.update(codes=torch.zeros(pool, dtype=torch.uint8, device="cuda"),
                     scales=torch.zeros(need, hk, page, 2, d // 32, dtype=torch.float16, device="cuda"),
                     start=torch.tensor(before, **ints))
    else:
        # codes as quantised normal values have them, drawn from a table of pairs
        pair = (normal(2, 65536) * 2.9).round().clamp(-7, 7).to(torch.int32) & 15
        pair = (pair[0] | pair[1] << 4).to(torch.uint8)
        state["codes"] = pair[torch.randint(0, 65536, pool, generator=g, device="cuda", dtype=torch.int32)]
        state["scales"] = ((2.0 + 0.4 * normal(need, hk, page, 2, d // 32)).abs() / 7).to(torch.float16)
        state.update(q=(1.5 * normal(n, hq, d)).to(dt), lengths=torch.tensor(lens, **ints))
    if own:
        state["cache"] = woq.KV4Cache(state["codes"], state["scales"])
        if case["op"] == "decode":
            state["out"] = torch.empty(n, hq, d, dtype=dt, device="cuda")
            state["ws"] = woq.kv4_attn_workspace(state["cache"], state["q"])
        else:
            state["rows"] = torch.empty(2, ends[-1], hk, d, device="cuda")
    return state


# ---- the operators -------------------------------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        import weight_only_bit_qgemv_b200 as woq

        if op == "prompt":
            return woq.attn_prompt(state["q"], state["k"], state["v"], state["cu"], scale=state["scale"],
                                   out=state["out"], workspace=state["ws"])
        if op == "decode":
            return woq.kv4_attn(state["q"], state["cache"], state["lengths"], state["table"], scale=state["scale"],
                                out=state["out"], workspace=state["ws"])
        woq.kv4_append(state["cache"], state["k"], state["v"], state["cu"], state["table"], start=state["start"])
        k, v = state["rows"]
        woq.kv4_gather(state["cache"], state["cu"], state["table"], start=state["start"], k_out=k, v_out=v)
        return {"k": k, "v": v}
    return {"prompt": _prompt, "decode": _decode, "store": _store}[op](state)


def _prompt(state):
    """Each sequence by itself, in blocks of rows where all its scores at once would be too many."""
    hq, hk = state["case"]["heads"], state["case"]["kv_heads"]
    q, k, v = (state[n].float().transpose(0, 1) for n in "qkv")
    q = q.unflatten(0, (hk, hq // hk))
    out, at = torch.empty_like(q), 0
    for n in state["lens"]:
        s, at = slice(at, at + n), at + n
        ks, vs = k[:, None, s], v[:, None, s]
        place = torch.arange(n, device="cuda")
        for i in range(0, n, 4096):
            j = min(i + 4096, n)
            x = q[:, :, s][:, :, i:j] @ ks[:, :, :j].transpose(-1, -2) * state["scale"]
            x = x.masked_fill_(place[:j] > place[i:j, None], -torch.inf)
            x = torch.exp(x - x.amax(-1, keepdim=True))
            out[:, :, s][:, :, i:j] = (x @ vs[:, :, :j]) / x.sum(-1, keepdim=True)
    return out.flatten(0, 1).transpose(0, 1).to(state["q"].dtype).contiguous()


def _unpacked(codes, parts, unit):
    """Stored rows of codes [..., dim / 2] as 32-bit numbers [..., dim]."""
    c = codes.unflatten(-1, (parts, -1, unit)).transpose(-3, -2).flatten(-3)
    c = torch.stack((c & 15, c >> 4), -1).flatten(-2).to(torch.int8)
    return (c - 16 * (c > 7)).float()


def _values(codes, scales, parts, unit):
    c = _unpacked(codes, parts, unit).unflatten(-1, (-1, 32))
    return (c * scales.float().unsqueeze(-1)).flatten(-2)


def _decode(state):
    """Every sequence padded to the longest: pages, values, scores, softmax, sum."""
    case, table, page = state["case"], state["table"].long(), state["case"]["page"]
    n, hq, hk, d = case["batch"], case["heads"], case["kv_heads"], case["dim"]
    codes, scales = state["codes"][table], state["scales"][table]  # [n, width, hk, ...]
    codes, scales = codes.transpose(1, 2), scales.transpose(1, 2)
    q = state["q"].float().view(n, hk, hq // hk, d)
    k = _values(codes[:, :, :, 0], scales[:, :, :, :, 0], 4, 4).flatten(2, 3)  # [n, hk, width * page, d]
    x = q @ k.transpose(-1, -2) * state["scale"]
    del k
    place = torch.arange(x.shape[-1], device="cuda")
    x = x.masked_fill_((place >= state["lengths"][:, None])[:, None, None], -torch.inf)
    x = torch.exp(x - x.amax(-1, keepdim=True))
    v = _values(codes[:, :, :, 1], scales[:, :, :, :, 1], 8, 2).flatten(2, 3)
    out = (x @ v) / x.sum(-1, keepdim=True)
    return out.view(n, hq, d).to(state["q"].dtype)


def _half(x):
    """x >= 0 in 64 bits, rounded once to binary16, ties to even."""
    # the power of two that is binary16's spacing at x, from x's exponent bits; the smallest is 2^-24
    quantum = ((x.view(torch.int64) >> 52).clamp_min(1023 - 14) - 10 << 52).view(torch.float64)
    return (torch.round(x / quantum) * quantum).to(torch.float16)


def _store(state):
    page, out = state["case"]["page"], {}
    cu, table = state["cu"].long(), state["table"].long()
    tokens = state["k"].shape[0]
    seq = torch.repeat_interleave(torch.arange(table.shape[0], device="cuda"), cu.diff(), output_size=tokens)
    at = state["start"].long()[seq] + torch.arange(tokens, device="cuda") - cu[seq]
    pages, slots = table[seq, at // page], at % page
    for i, (name, parts, unit) in enumerate((("k", 4, 4), ("v", 8, 2))):
        x = state[name].float().unflatten(-1, (-1, 32))
        a = x.abs().amax(-1).double()
        s = _half(a / torch.full_like(a, 7))
        c = torch.round(x.double() / s.double().unsqueeze(-1)).clamp(-8, 7).nan_to_num(0.0).to(torch.int32) & 15
        c = c.flatten(-2).unflatten(-1, (-1, 2))
        c = (c[..., 0] | c[..., 1] << 4).to(torch.uint8)
        c = c.unflatten(-1, (-1, parts, unit)).transpose(-3, -2).flatten(-3)
        state["codes"][pages, :, i, slots] = c
        state["scales"][pages, :, slots, i] = s
        out[name] = _values(state["codes"][pages, :, i, slots], state["scales"][pages, :, slots, i], parts, unit)
    return out


# ---- the definitions in 64 bits ------------------------------------------------------------------------------------

def _nibbles(rows):
    """Two's-complement nibbles of plain (not transposed) rows of bytes, as 64-bit numbers."""
    both = torch.empty(*rows.shape, 2, dtype=torch.float64, device=rows.device)
    both[..., 0], both[..., 1] = rows % 16, rows // 16
    both = both.reshape(*rows.shape[:-1], -1)
    return torch.where(both >= 8, both - 16, both)


def exact(case, seed):
    s = prepare(case, seed)
    hq, hk, d = case["heads"], case["kv_heads"], case["dim"]
    group, blocks = hq // hk, d // 32
    if case["op"] == "store":
        found = {}
        for name in ("k", "v"):
            x = s[name].to(torch.float64).reshape(-1, hk, blocks, 32)
            # NumPy rounds binary64 to binary16 at once, and divides by 7 as written
            step = (x.abs().max(-1, keepdim=True).values.cpu().numpy() / 7).astype(np.float16)
            step = torch.from_numpy(step).cuda().double()
            code = torch.where(step > 0, x / torch.where(step > 0, step, 1.0), 0.0).round().clamp(-8, 7)
            found[name] = (code * step).reshape(-1, hk, d)
        return found
    if case["op"] == "decode":
        rows = []
        for b, n in enumerate(s["lens"]):
            pages = s["table"][b, : -(-n // case["page"])].long()
            heads = []
            for h in range(hk):
                codes, scales = s["codes"][pages, h], s["scales"][pages, h].double()
                key = codes[:, 0].reshape(-1, 4, blocks, 4).permute(0, 2, 1, 3).reshape(-1, d // 2)[:n]
                val = codes[:, 1].reshape(-1, 8, blocks, 2).permute(0, 2, 1, 3).reshape(-1, d // 2)[:n]
                scales = scales.reshape(-1, 2, blocks)[:n]
                key = _nibbles(key) * scales[:, 0].repeat_interleave(32, -1)
                val = _nibbles(val) * scales[:, 1].repeat_interleave(32, -1)
                p = torch.softmax(torch.einsum("gd,nd->gn", s["q"][b, h * group:(h + 1) * group].double(), key) * s["scale"], -1)
                heads.append(torch.einsum("gn,nd->gd", p, val))
            rows.append(torch.cat(heads))
        return torch.stack(rows)
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    first = 0
    for n in s["lens"]:
        for h in range(hq):
            key, val = (s[x][first:first + n, h // group].double() for x in ("k", "v"))
            for i in range(0, n, 8192):
                j = min(n, i + 8192)
                x = torch.einsum("id,jd->ij", s["q"][first + i:first + j, h].double(), key[:j]) * s["scale"]
                x = x + torch.full_like(x, -torch.inf).triu_(1 + i)
                out[first + i:first + j, h] = torch.softmax(x, -1) @ val[:j]
        first += n
    return out
