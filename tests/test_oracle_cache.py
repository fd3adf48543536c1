"""Pins of the cache oracle (CPU only): slot maps, quantisation, attention."""

import math

import numpy as np
import pytest
import torch

import oracle
from oracle import cache


def test_slots_by_hand():
    # blocks of 4; sequence 0 has 5 tokens in blocks 7, 2 and grows by 4 into a new block;
    # sequence 1 is fresh (6 tokens); sequence 2 does nothing; sequence 3 gets one token in place
    table = np.array([[7, 2, -1], [-1, -1, -1], [5, -1, -1], [3, -1, 9]])
    slots, offsets, taken, after = cache.kv_slots(
        [9, 6, 2, 3], [4, 6, 0, 1], [11, 12, 10, 8], table, 13, 4, 12, 13)
    assert taken.tolist() == [3]
    assert after.tolist() == [[7, 2, 11], [12, 10, -1], [5, -1, -1], [3, -1, 9]]
    assert offsets.tolist() == [0, 4, 10, 10, 11]
    assert slots.tolist() == [9, 10, 11, 44, 48, 49, 50, 51, 40, 41, 14, -1, -1]


def test_slots_free_list_runs_out_and_tokens_past_the_end():
    slots, offsets, taken, after = cache.kv_slots([6, 5], [6, 5], [1, 2], [[-1, -1], [-1, -1]],
                                                  3, 4, 8, 9)
    assert taken.tolist() == [4]
    assert after.tolist() == [[1, 2], [-1, -1]]
    assert offsets.tolist() == [0, 6, 11]
    assert slots.tolist() == [4, 5, 6, 7, 8, 9, -1, -1, -1]


@pytest.mark.parametrize("fmt,top", [("fp8", 448.0), ("mxfp8", 448.0), ("mxfp4", 6.0)])
def test_quantise_is_the_nearest_code_under_the_least_scale(fmt, top):
    rng = np.random.default_rng(3)
    x = rng.normal(size=(40, 64)) * np.exp2(rng.integers(-20, 20, (40, 1)))
    codes, scales, values = cache.quantise(fmt, x)
    held = (oracle.codecs.decode(fmt, codes, scales) if fmt != "fp8"
            else oracle.codecs.decode(fmt, codes) * scales[..., None].astype(np.float64))
    assert np.array_equal(held, values)
    size = 64 if fmt == "fp8" else 32
    s = (scales if fmt == "fp8" else np.exp2(scales.astype(float) - 127)).reshape(-1, 1)
    g, v = x.reshape(-1, size), values.reshape(-1, size)
    amax = np.abs(g).max(-1, keepdims=True)
    assert (amax <= top * s).all() and (amax > top * s / 2).all()
    grid = (oracle.codecs.E2M1_TABLE[:8] if fmt == "mxfp4" else oracle.codecs.E4M3_TABLE[:127])
    best = np.abs(np.abs(g / s)[..., None] - grid).min(-1)
    assert np.array_equal(np.abs(g / s - v / s), best)


def test_quantise_ties_and_edges():
    # scale 1 (the group's 6): every tie goes to the even code
    x = np.zeros((1, 32))
    x[0, :9] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25]
    codes, scales, values = cache.quantise("mxfp4", x)
    assert scales.tolist() == [[127]]
    assert values[0, :9].tolist() == [6, 0, 1, 1, 2, 2, 4, 4, -0.0] and np.signbit(values[0, 8])
    assert codes[0, :5].tolist() == [0x07, 0x22, 0x44, 0x66, 0x08]
    # zeros have scale 1; tiny rows the least scale; an infinity or NaN spoils its group
    assert cache.quantise("mxfp8", np.zeros((1, 32)))[1].tolist() == [[127]]
    assert cache.quantise("fp8", np.zeros((1, 64)))[1].tolist() == [1.0]
    assert cache.quantise("mxfp4", np.full((1, 32), 2.0 ** -149))[1].tolist() == [[0]]
    assert cache.quantise("fp8", np.full((1, 64), 2.0 ** -149))[1].tolist() == [2.0 ** -126]
    for bad in (np.inf, np.nan):
        y = np.ones((1, 64))
        y[0, 40] = bad
        codes, scales, values = cache.quantise("mxfp4", y)
        assert scales[0, 1] == 255 and not codes[0, 16:].any() and np.isnan(values[0, 32:]).all()
        assert np.array_equal(values[0, :32], y[0, :32])
        assert np.isnan(cache.quantise("fp8", y)[1]).all()


@pytest.mark.parametrize("sparse", [False, True])
def test_attention_against_a_direct_softmax(sparse):
    rng = np.random.default_rng(5)
    nb, bs, hkv, d, n = 6, 16, 2, 64, 3
    k, v = (rng.integers(0, 256, (nb, bs, hkv, d // 2), dtype=np.uint8) for _ in range(2))
    ks, vs = (rng.integers(124, 130, (nb, bs, hkv, 2), dtype=np.uint8) for _ in range(2))
    table, ctx = np.array([[4, 1], [0, 3]]), np.array([20, 2])
    q = rng.normal(size=(6, 4, d))
    indices = np.array([[0, 17, 19, -1]] * 3 + [[1, 0, 7, 5]] * 3) if sparse else None
    out, lse, _, _ = cache.attention(q, k, ks, v, vs, ctx, table, n, 24, 0.1, 0, 0, indices)
    K = oracle.codecs.decode("mxfp4", k, ks)
    V = oracle.codecs.decode("mxfp4", v, vs)
    for r in range(6):
        b, t = divmod(r, n)
        keys = [j for j in range(max(0, ctx[b] - n + 1 + t))
                if not sparse or j in indices[r].tolist()]
        for h in range(4):
            if not keys:
                assert not out[r, h].any() and lse[r, h] == -math.inf
                continue
            s = [0.1 * float(q[r, h] @ K[table[b, j // bs], j % bs, h // 2]) for j in keys]
            p = torch.softmax(torch.tensor(s, dtype=torch.float64), 0).numpy()
            ref = sum(pj * V[table[b, j // bs], j % bs, h // 2] for pj, j in zip(p, keys))
            assert np.allclose(out[r, h], ref, rtol=1e-12, atol=1e-12)
            assert np.isclose(lse[r, h], math.log(sum(math.exp(x) for x in s)), rtol=1e-12)
