"""The 8-bit paged cache in float64, plain loops: norms, scales, codes, append, read-back.

Test infrastructure.  A code is an e4m3 number (sign, 4 bits of exponent with a
bias of 7, 3 bits of fraction; all ones is NaN); the entries of a block share a
scale 2^e, kept as the byte e + 127.  Pools of codes are uint8 arrays [n_pages,
page_size, n_heads, D], scales uint8 [n_pages, page_size / block, n_heads].
"""
from __future__ import annotations

import math

import numpy as np

from . import paged

LOW = {"bf16": -100, "fp16": -15}
HIGH = {"bf16": 120, "fp16": 8}


def _value(code):
    if code & 0x7F == 0x7F:
        return math.nan
    exponent, fraction = code >> 3 & 15, code & 7
    x = fraction / 8 * 2.0 ** -6 if exponent == 0 else (1 + fraction / 8) * 2.0 ** (exponent - 7)
    return -x if code & 0x80 else x


VALUES = np.array([_value(c) for c in range(256)])


def encode(x):
    """Codes of the nearest values of e4m3, ties to the even code; |x| up to 240 or NaN."""
    x = np.asarray(x, dtype=np.float64)
    grid = VALUES[:127]
    at = np.clip(np.searchsorted(grid, np.abs(x)), 1, 126)  # grid[at - 1] < |x| <= grid[at]
    below, above = np.abs(x) - grid[at - 1], grid[at] - np.abs(x)
    code = np.where((below < above) | ((below == above) & (at % 2 == 1)), at - 1, at)
    code = np.where(np.isnan(x), 0x7F, code | np.where(np.signbit(x), 0x80, 0))
    return code.astype(np.uint8)


def exponent(x, dtype):
    """A block's exponent for the values x."""
    x = np.abs(x[np.isfinite(x)])
    top = min(x.max(initial=0.0), most(dtype))
    return max(math.frexp(top)[1] - 8, LOW[dtype]) if top > 0 else LOW[dtype]


def most(dtype):
    return 240.0 * 2.0 ** HIGH[dtype]


def quantise(x, e, dtype):
    x = np.where(np.isfinite(x), np.clip(x, -most(dtype), most(dtype)), np.nan)
    return encode(x * 2.0 ** -e)


def values(codes, scales):
    """What whole pools stand for."""
    block = codes.shape[1] // scales.shape[1]
    return VALUES[codes] * 2.0 ** (np.repeat(scales, block, axis=1).astype(np.float64) - 127)[..., None]


def norm(x, weight, eps):
    """x [..., D] with root-mean-square 1, times weight; None: as it is."""
    x = np.asarray(x, dtype=np.float64)
    return x if weight is None else x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight


def append_block(codes, scales, new, behind, dtype):
    """One block of one head: codes [block, D] and its scale byte; `new` [n, D]
    stands behind `behind` older entries.  Returns both, changed."""
    codes, e = codes.copy(), exponent(new, dtype)
    if behind:
        was = int(np.clip(int(scales) - 127, LOW[dtype], HIGH[dtype]))
        if e > was:
            codes[:behind] = encode(VALUES[codes[:behind]] * 2.0 ** (was - e))
        e = max(e, was)
    codes[behind:behind + len(new)] = quantise(new, e, dtype)
    return codes, e + 127


def append8(codes, scales, x, q_indptr, block_table, kv_len, dtype):
    """x [N, heads, D] (float64, normalised and rotated) into one side's pools (copies)."""
    codes, scales = codes.copy(), scales.copy()
    page_size, block = codes.shape[1], codes.shape[1] // scales.shape[1]
    for b in range(len(kv_len)):
        first, end = int(q_indptr[b]), int(q_indptr[b + 1])
        n = first
        while n < end:
            t = paged.entry_of(end - first, int(kv_len[b]), n - first)
            behind = t % block
            count = min(block - behind, end - n)
            page, slot = int(block_table[b, t // page_size]), t % page_size - behind
            for h in range(x.shape[1]):
                got, byte = append_block(codes[page, slot:slot + block, h], scales[page, slot // block, h], x[n:n + count, h],
                                         behind, dtype)
                codes[page, slot:slot + block, h], scales[page, slot // block, h] = got, byte
            n += count
    return codes, scales


def read8(codes, scales, out_indptr, block_table, first):
    """Rows [out_indptr[-1], heads, D] of the entries from first[b] on."""
    v = values(codes, scales)
    page_size = codes.shape[1]
    rows = []
    for b in range(len(first)):
        for i in range(int(out_indptr[b + 1]) - int(out_indptr[b])):
            t = int(first[b]) + i
            rows.append(v[int(block_table[b, t // page_size]), t % page_size])
    return np.array(rows).reshape((-1,) + v.shape[2:])
