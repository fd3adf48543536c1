"""Slot maps, quantising writes and attention over a paged MXFP4 cache.

Straight from the definitions, in float64 and Python integers:

  kv_slots    sequence by sequence, token by token;
  quantise    the smallest power-of-two scale of a group under which no element
              exceeds the largest code, then the nearest code (ties to the even
              code) by comparison with every code of the format;
  gathered    the attention weight that every key has gathered;
  evict       the recent tokens and the heaviest of the others, in free blocks;
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
    _, seen = paged_row_ranges(context_lens, next_n, max_context_len)
    return attend_rows(q, k_pool, k_sf_pool, v_pool, v_sf_pool, block_table,
                       np.arange(len(seen)) // next_n, seen, scale, half_step, weight_step, indices)


def chunk_rows(context_lens, token_offsets, tokens, max_context_len):
    """(sequence, keys seen) of every row of q, -1 and 0 for rows that no sequence has: row t of
    the n of a sequence sees min(ctx - n + 1 + t, max_context_len) keys."""
    sequence, seen = np.full(tokens, -1), np.zeros(tokens, np.int64)
    for b, ctx in enumerate(np.asarray(context_lens, np.int64)):
        lo, hi = int(token_offsets[b]), int(token_offsets[b + 1])
        for r in range(max(lo, 0), min(hi, tokens)):
            sequence[r] = b
            seen[r] = min(max(ctx - (hi - lo) + 1 + r - lo, 0), max(ctx, 0), max_context_len)
    return sequence, seen


def attend_rows(q, k_pool, k_sf_pool, v_pool, v_sf_pool, block_table, sequence, seen, scale,
                half_step, weight_step, indices=None, weight_floor=0.0):
    """attention() for rows of given sequences that see their first `seen` keys.  weight_floor:
    the least rounding of a weight, relative to the row's largest one."""
    q = np.asarray(q, dtype=np.float64)
    rows, hq, d = q.shape
    bs, hkv = k_pool.shape[1], k_pool.shape[2]
    group = hq // hkv
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
        block = np.clip(np.asarray(block_table)[sequence[r], keys // bs], 0, len(k_pool) - 1)
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
            out_bound[r, hs] = ((w * (e + worst + weight_step + chain * 2.0 ** -22)
                                  + weight_floor * w.max(-1, keepdims=True)) @ np.abs(v[:, h])
                                * (1 + 2 * half_step) + half_step * np.abs(out[r, hs]) + 2.0 ** -24)
            lse_bound[r, hs] = worst[:, 0] + chain * 2.0 ** -23 + 2.0 ** -22 * np.abs(lse[r, hs])
    return out, lse, out_bound, lse_bound


def gathered(q, lse, k_pool, k_sf_pool, block_table, sequence, seen, scale, lengths, before=None):
    """(sums, bound) float64 [batch, most]: before + sum exp(scale <q, k> - lse) of the rows that see a
    key, for keys below `lengths`, 0 behind.

    The bound: a score is off by e (see attention), the shift by lse by 2^-22 (|score| + |lse|), which
    with the exponential's own 2^-22 is the relative error of a term; sums of n terms, in parts that are
    added in turn, by at most n 2^-24 + 2^-20 of their sum."""
    q = np.asarray(q, dtype=np.float64)
    hq, d = q.shape[1:]
    bs, hkv = k_pool.shape[1], k_pool.shape[2]
    group = hq // hkv
    lengths = np.asarray(lengths)
    sums = np.zeros((len(lengths), max(int(lengths.max()), 1)))
    error, count = np.zeros_like(sums), np.zeros_like(sums)
    for b, n in enumerate(lengths):
        if before is not None:
            sums[b, :n] = np.asarray(before, np.float64)[b, :n]
        keys = np.arange(n)
        block = np.clip(np.asarray(block_table)[b, keys // bs], 0, len(k_pool) - 1)
        k = decode_cache(k_pool[block, keys % bs], k_sf_pool[block, keys % bs])
        for r in np.flatnonzero(np.asarray(sequence) == b):
            m = int(seen[r])
            for h in range(hq):
                if m == 0 or np.isneginf(lse[r, h]):
                    continue
                kh = k[:m, h // group]
                s = (kh @ q[r, h]) * scale
                p = np.exp(s - float(lse[r, h]))
                e = (abs(scale) * d * 2.0 ** -23 * (np.abs(kh) @ np.abs(q[r, h]))
                     + 2.0 ** -22 * (np.abs(s) + abs(float(lse[r, h]))) + 2.0 ** -22)
                sums[b, :m] += p
                error[b, :m] += p * e
                count[b, :m] += 1
    return sums, error * 1.01 + np.abs(sums) * (count * 2.0 ** -24 + 2.0 ** -20)


def evict(weights, context_lens, block_table, free_blocks, pools, keep, recent, max_context_len):
    """(context_lens, block_table, weights, kept, freed, counts, pools) afterwards."""
    size = pools[0].shape[1]
    table, weights = np.asarray(block_table), np.asarray(weights)
    batch, width = len(table), -(-max_context_len // size)
    num_blocks = len(pools[0])
    new_table = np.full((batch, width), -1, np.int32)
    new_weights = np.zeros((batch, max_context_len), np.float32)
    kept, lens, freed, taken = np.full((batch, keep), -1, np.int32), [], [], 0
    before, pools = pools, [np.array(p) for p in pools]
    for b, ctx in enumerate(context_lens):
        n = min(max(int(ctx), 0), max_context_len)
        old, at, moved = table[b, :-(-n // size)], np.arange(n), False
        if n > keep:
            w = weights[b, :n - recent]
            bits = w.view(np.int32).astype(np.int64)
            order = np.where(bits < 0, -(bits & 0x7fffffff) - 1, bits)     # IEEE total order
            chosen = [j for j in sorted(range(n - recent), key=lambda j: (-order[j], j)) if w[j] != -np.inf]
            at = np.array(sorted(chosen[:keep - recent]) + list(range(n - recent, n)), int)
            want = -(-len(at) // size)
            moved = taken + want <= len(free_blocks)
            if moved:
                mine = np.asarray(free_blocks[taken:taken + want], np.int32)
                for i, j in enumerate(at):
                    src, dst = old[j // size], mine[i // size]
                    if 0 <= src < num_blocks and 0 <= dst < num_blocks:
                        for p, q in zip(before, pools):
                            q[dst, i % size] = p[src, j % size]
                freed += old.tolist()
                old = mine
            else:
                at = np.arange(n)
            taken += want
        new_table[b, :len(old)] = old
        if n <= keep or moved:
            kept[b, :len(at)] = at
        new_weights[b, :len(at)] = weights[b, at]
        lens.append(len(at))
    back = np.full(batch * width, -1, np.int32)
    back[:len(freed)] = freed
    return (np.array(lens, np.int32), new_table, new_weights, kept, back,
            np.array([taken, len(freed)], np.int32), pools)
