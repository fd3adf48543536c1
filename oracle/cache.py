"""Slot maps, quantising writes and attention over a paged MXFP4 cache.

Straight from the definitions, in float64 and Python integers:

  kv_slots    sequence by sequence, token by token;
  quantise    the smallest power-of-two scale of a group under which no element
              exceeds the largest code, then the nearest code (ties to the even
              code) by comparison with every code of the format;
  attention   out = sum_j softmax_j(scale <q, k_j>) v_j over the keys a row
              sees (or the listed ones among them), lse = log sum_j exp(..),
              with an error bound per entry.
"""

import math

import numpy as np

from . import codecs
from .reference import paged_row_ranges

TOP = {"fp8": 448.0, "mxfp8": 448.0, "mxfp4": 6.0}


def kv_slots(context_lens, new_lens, free_blocks, block_table, num_blocks, block_size,
             max_context_len, max_tokens):
    """(slots, token_offsets, blocks_taken, block_table after the step)."""
    table = np.array(block_table, dtype=np.int32)
    slots = [-1] * max_tokens
    offsets, taken, k = [0], 0, 0
    for b, (ctx, new) in enumerate(zip(context_lens, new_lens)):
        ctx = min(max(int(ctx), 0), max_context_len)
        new = min(max(int(new), 0), ctx)
        old = ctx - new
        for j in range(-(-old // block_size), -(-ctx // block_size)):
            table[b, j] = free_blocks[taken] if taken < len(free_blocks) else -1
            taken += 1
        for pos in range(old, ctx):
            block = int(table[b, pos // block_size])
            if k < max_tokens and 0 <= block < num_blocks:
                slots[k] = block * block_size + pos % block_size
            k += 1
        offsets.append(k)
    return (np.array(slots, dtype=np.int64).reshape(max_tokens), np.array(offsets, np.int32),
            np.array([taken], np.int32), table)


def _scale_exponent(amax, top, least):
    if amax == 0:
        return 0
    e = math.ceil(math.log2(amax) - math.log2(top)) - 2
    while amax > math.ldexp(top, e):
        e += 1
    return max(e, least)


def _nearest(table, y):
    """Codes (non-negative ones of `table`) nearest to y >= 0, ties to the even code."""
    order = np.argsort(table, kind="stable")
    values = table[order]
    above = np.clip(np.searchsorted(values, y), 1, len(values) - 1)
    up, down = values[above] - y, y - values[above - 1]
    take_up = (up < down) | ((up == down) & (order[above] % 2 == 0))
    return np.where(take_up, order[above], order[above - 1])


def quantise(fmt, x):
    """(codes, scales, values) of rows x [.., D]: bytes (packed for mxfp4), e8m0
    bytes [.., D/32] or fp32 scales [..], float64 values."""
    x = np.asarray(x, dtype=np.float64)
    d = x.shape[-1]
    size = d if fmt == "fp8" else 32
    groups = x.reshape(-1, size)
    amax = np.abs(groups).max(-1)
    fine = np.isfinite(amax)
    e = np.array([_scale_exponent(a, TOP[fmt], -126 if fmt == "fp8" else -127) if f else 0
                  for a, f in zip(amax.tolist(), fine.tolist())])
    two = np.array([math.ldexp(1.0, int(k)) for k in e])
    y = np.where(fine[:, None], groups / two[:, None], 0.0)
    table = (codecs.E2M1_TABLE[:8] if fmt == "mxfp4" else codecs.E4M3_TABLE[:0x7f])
    code = _nearest(table, np.abs(y))
    values = np.where(fine[:, None], np.copysign(table[code], y) * two[:, None], np.nan)
    code = (code + np.signbit(y) * (8 if fmt == "mxfp4" else 0x80)).astype(np.uint8)
    code = code.reshape(x.shape)
    if fmt == "mxfp4":
        code = code[..., 0::2] | (code[..., 1::2] << 4)
    if fmt == "fp8":
        scales = np.where(fine, two, np.nan).astype(np.float32).reshape(x.shape[:-1])
    else:
        scales = np.where(fine, e + 127, 255).astype(np.uint8).reshape(*x.shape[:-1], d // 32)
    return code, scales, values.reshape(x.shape)


def decode_cache(codes, sf):
    """Values of MXFP4 cache rows; scale bytes over 252 are NaN."""
    sf = np.asarray(sf, dtype=np.uint8)
    return codecs.decode("mxfp4", codes, np.where(sf > 252, 255, sf).astype(np.uint8))


def attention(q, k_pool, k_sf_pool, v_pool, v_sf_pool, context_lens, block_table, next_n,
              max_context_len, scale, half_step, weight_step, indices=None):
    """(out, lse, out_bound, lse_bound) float64.

    q [batch * next_n, Hq, D] as float64.  half_step: the result type's largest
    relative rounding; weight_step: that of the weights p in the second product.

    The bounds.  Products of q and e2m1 elements under a power-of-two scale are
    exact in fp32; a sum of n of them in fp32 is off by at most n 2^-23 of the
    sum of their magnitudes (2^-23: the matrix core may truncate).  So a score
    is off by scale * D 2^-23 sum_d |q_d k_d|, and its scaling and the shift by
    the maximum by 2^-22 (|score| + |maximum|) more: e_j in all, which is the
    relative error of p_j next to the exponential's own 2^-22.  Rescaling the
    running sums with a few exponentials of rounded differences costs the same
    again.  The sums over n keys are made of at most n / 64 + 100 additions in
    a row.  out = sum w_j v_j with w = p / sum p then errs by
    sum_j w_j |v_j| (e_j + max e + weight_step + (n / 64 + 100) 2^-22) and its
    rounding, and lse by max e + (n / 64 + 100) 2^-23 and its own rounding.
    """
    q = np.asarray(q, dtype=np.float64)
    rows, hq, d = q.shape
    bs, hkv = k_pool.shape[1], k_pool.shape[2]
    group = hq // hkv
    _, seen = paged_row_ranges(context_lens, next_n, max_context_len)
    out, lse = np.zeros((rows, hq, d)), np.full((rows, hq), -np.inf)
    out_bound, lse_bound = np.zeros((rows, hq, d)), np.zeros((rows, hq))
    for r in range(rows):
        keys = np.arange(seen[r])
        if indices is not None:
            keys = np.asarray(indices[r], dtype=np.int64)
            keys = keys[(keys >= 0) & (keys < seen[r])]
        n = keys.size
        if n == 0:
            continue
        block = np.clip(np.asarray(block_table)[r // next_n, keys // bs], 0, len(k_pool) - 1)
        at = block, keys % bs
        k = decode_cache(k_pool[at], k_sf_pool[at])
        v = decode_cache(v_pool[at], v_sf_pool[at])
        for h in range(hkv):
            hs = slice(h * group, (h + 1) * group)
            s = (q[r, hs] @ k[:, h].T) * scale
            top = s.max(-1, keepdims=True)
            p = np.exp(s - top)
            total = p.sum(-1, keepdims=True)
            w = p / total
            out[r, hs] = w @ v[:, h]
            lse[r, hs] = (top + np.log(total))[:, 0]
            mags = np.abs(q[r, hs]) @ np.abs(k[:, h]).T
            e = abs(scale) * d * 2.0 ** -23 * mags + 2.0 ** -21 * (
                np.abs(s) + np.abs(s).max(-1, keepdims=True)) + 2.0 ** -20
            chain = (n / 64 + 100)
            worst = e.max(-1, keepdims=True)
            out_bound[r, hs] = ((w * (e + worst + weight_step + chain * 2.0 ** -22)) @ np.abs(v[:, h])
                                * (1 + 2 * half_step) + half_step * np.abs(out[r, hs]) + 2.0 ** -24)
            lse_bound[r, hs] = worst[:, 0] + chain * 2.0 ** -23 + 2.0 ** -22 * np.abs(lse[r, hs])
    return out, lse, out_bound, lse_bound
