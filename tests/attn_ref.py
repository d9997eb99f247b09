"""Attention and the 4-bit cache in 64 bits on the CPU, straight from their definitions."""

import numpy as np
import torch

import oracle

UNIT = {torch.float32: 2.0**-24, torch.float16: 2.0**-11, torch.bfloat16: 2.0**-8}  # half a step, relative


def halfword_places(dim):
    """[2, dim] nibble index within a stored row of element d, for a key row and for a value row."""
    nb = dim // 32
    d = np.arange(dim)
    block, e = d // 32, d % 32
    key = ((e // 8) * nb + block) * 8 + e % 8      # 32-bit words of 8 codes: word t of block b at t * nb + b
    value = ((e // 4) * nb + block) * 4 + e % 4    # 16-bit halfwords of 4 codes: g of block b at g * nb + b
    return np.stack([key, value])


def quantised(x):
    """Rows [..., dim] through the oracle's int4 quantiser: (codes, scales as binary16 bits, values float64)."""
    x = np.asarray(x, dtype=np.float32)
    q, s = oracle.quantise(x.reshape(-1, x.shape[-1]), 4)
    s = np.asarray(s).view(np.uint16)
    values = q.astype(np.float64) * np.repeat(s.view(np.float16).astype(np.float64), 32, axis=1)
    return q.reshape(x.shape), s.reshape(*x.shape[:-1], -1), values.reshape(x.shape)


def read_pages(codes, scales):
    """Pools (torch, any device) -> float64 [2, pages, heads, page, dim]."""
    codes, scales = codes.cpu().numpy(), scales.cpu().numpy().astype(np.float64)
    pages, heads, _, page, half = codes.shape
    nib = np.stack([codes & 15, codes >> 4], -1).reshape(pages, heads, 2, page, 2 * half).astype(np.int64)
    nib = np.where(nib > 7, nib - 16, nib)
    at = halfword_places(2 * half)
    s = np.repeat(scales, 32, axis=-1)
    with np.errstate(invalid="ignore"):  # 0 times an infinite scale
        return np.stack([nib[:, :, i][..., at[i]] * s[:, :, :, i] for i in (0, 1)])


def write_pages(q, s, i, codes, scales, page, slot):
    """Codes q [heads, dim] and scale bits s [heads, dim / 32] of one token into NumPy pools, i = 0 keys, 1 values."""
    dim = q.shape[-1]
    nib = np.zeros((q.shape[0], dim), dtype=np.uint8)
    nib[:, halfword_places(dim)[i]] = (q & 15).astype(np.uint8)
    codes[page, :, i, slot] = nib[:, 0::2] | nib[:, 1::2] << 4
    scales[page, :, slot, i] = s.view(np.float16) if s.dtype == np.uint16 else s


def attend(q, k, v, scale):
    """q [heads, dim] over k, v [tokens, kv_heads, dim] -> [heads, dim], and what bounds its error: per head the
    largest sum_d |q_d k_d| scale of a token, and the largest |v|."""
    heads, kv = q.shape[0], k.shape[1]
    out, size = np.zeros(q.shape), np.zeros((heads, 2))
    for h in range(heads):
        kh, vh = k[:, h * kv // heads], v[:, h * kv // heads]
        if not len(kh):
            continue
        x = kh @ q[h] * scale
        p = np.exp(x - x.max())
        out[h] = p @ vh / p.sum()
        size[h] = (np.abs(kh) @ np.abs(q[h])).max() * scale, np.abs(vh).max()
    return out, size


def tolerance(ref, size, dtype, products=22):
    """Largest error of an attention result whose products keep `products` bits of both factors.

    A score is a sum whose terms are each off by at most 2^(1 - products) of themselves (two factors, half a step
    each), and FP32 sums of up to 2^8 terms that double that at most: E = 2^(2 - products) sum |q k| scale. A weight
    is then off by a factor e^(2 E), its maximum's and the sum's among them; the exponential, the weights' split and
    the values' sum add 2^(3 - products) more. In total (2 E + 2^(3 - products)) max |v|, and a 16-bit result half a
    step of itself."""
    e = 2.0 ** (2 - products) * size[..., :1]
    unit = 0.0 if dtype == torch.float32 else UNIT[dtype]
    return (2 * e + 2.0 ** (3 - products)) * size[..., 1:] + unit * np.abs(ref) + 1e-30


def attend_by_column(q, k, v, scale):
    """attend() for q [heads, dim] over k, v [tokens, kv_heads, dim], and what bounds its error column by column: per head
    the largest sum_d |q_d k_d| scale of a token, and per column sum_j p_j times the largest |v_j| of its 32 columns."""
    out, size = attend(q, k, v, scale)
    heads, kv, dim = q.shape[0], k.shape[1], q.shape[1]
    big = np.repeat(np.abs(v).reshape(*v.shape[:2], dim // 32, 32).max(-1), 32, axis=-1)
    col = np.zeros(q.shape)
    for h in range(heads):
        x = k[:, h * kv // heads] @ q[h] * scale
        p = np.exp(x - x.max())
        col[h] = p @ big[:, h * kv // heads] / p.sum()
    return out, size[:, :1], col


def tolerance_by_column(ref, e, col, dtype):
    """tolerance() with the weighted mean of the values' sizes for the largest of them. Scores as there: E = 2^-20 sum
    |q k| scale, 2 E of every weight. Weights' exponentials and splits and the products with the scales are off by
    2^-22 of each term, three times; the split's last step is 2^-25 of a unit's largest term at most for each of 32
    tokens, 2^-20; FP32 additions of a few units 2^-21: less than 2^-18 of the sum of all terms' sizes."""
    unit = 0.0 if dtype == torch.float32 else UNIT[dtype]
    return (2.0**-19 * e + 2.0**-18) * col + unit * np.abs(ref) + 1e-30
