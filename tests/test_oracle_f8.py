"""Pins of the 8-bit block-scaled cache's oracle (CPU, no library)."""
import math

import numpy as np
import pytest
import torch

from oracle import f8


def test_code_values_are_e4m3():
    want = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn)
    want = want.to(torch.float64).numpy()
    got = f8.code_values()
    assert (np.isnan(got) == np.isnan(want)).all()
    fin = ~np.isnan(want)
    assert (got[fin] == want[fin]).all()
    assert got[0x7e] == 448.0 and got[1] == 2.0 ** -9 and got[8] == 2.0 ** -6


def test_encode_is_the_nearest_code_ties_to_even():
    # every f16 up to 448: ties between neighbours among them
    x = np.arange(65536, dtype=np.uint16).view(np.float16).astype(np.float32)
    x = x[np.isfinite(x) & (np.abs(x) <= 448)]
    x = np.concatenate([x, x * np.float32(2.0 ** -6)])
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert (f8.encode(x) == want).all()


def test_encode_saturates_and_keeps_nan():
    got = f8.encode(np.array([500.0, -1e9, math.inf, -math.inf, math.nan, 0.0, -0.0]))
    assert got.tolist()[:4] == [0x7e, 0xfe, 0x7e, 0xfe]
    assert got[4] in (0x7f, 0xff) and got[5] == 0 and got[6] == 0x80


@pytest.mark.parametrize("amax,want", [(0.0, 0.0), (448.0, 1.0), (448.0001, 2.0), (1.0, 2.0 ** -8),
                                       (1.75, 2.0 ** -8), (1.7500001, 2.0 ** -7),
                                       (1e-45, 2.0 ** -126)])
def test_pow2_scale(amax, want):
    assert f8.pow2_scale(amax) == want


def test_store_grows_the_scale_and_keeps_values():
    rng = np.random.default_rng(3)
    bs, h, d = 16, 2, 64
    pool = rng.integers(0, 127, (3, bs, h, d)).astype(np.uint8)
    scales = np.full((3, h), np.nan, dtype=np.float32)
    table, first = np.array([[2]], dtype=np.int32), rng.normal(size=(5, h, d))
    f8.store(pool, scales, first, table, [5], [0, 5], bs)
    before = f8.values(pool, scales)[2, :5].copy()
    stale = pool[2, 6:].copy()
    err = np.abs(before - first)
    # half a step of 2^-4 relative, or half the least step of the scale
    assert (err <= np.maximum(np.abs(first) / 16, scales[2][None, :, None] * 2.0 ** -10)).all()
    f8.store(pool, scales, 100 * rng.normal(size=(1, h, d)), table, [6], [0, 1], bs)
    after = f8.values(pool, scales)[2, :5]
    least = scales[2][None, :, None] * 2.0 ** -9
    normal = np.abs(after) >= 8 * least
    assert (after[normal] == before[normal]).all()          # exponents only
    assert (np.abs(after - before) <= least / 2).all()
    assert (pool[2, 6:] == stale).all()


def test_attention_matches_sdpa():
    rng = np.random.default_rng(4)
    bs, h, g, d, n_phys = 16, 2, 3, 64, 12
    pools = [rng.integers(0, 256, (n_phys, bs, h, d)).astype(np.uint8) for _ in range(2)]
    for p in pools:
        p[(p & 127) == 127] = 5
    sc = [2.0 ** rng.integers(-9, -6, (n_phys, h)).astype(np.float32) for _ in range(2)]
    ctx, table = [37, 90], rng.permutation(n_phys).reshape(2, 6).astype(np.int32)
    q = rng.normal(size=(7, h * g, d))
    q_start = [0, 5, 7]
    out, lse = f8.attention(q, *pools, *sc, table, ctx, bs, 0.125, q_start=q_start)
    for s in range(2):
        c, n = ctx[s], q_start[s + 1] - q_start[s]
        k, v = (torch.from_numpy(f8.values(p, x)[table[s]].reshape(-1, h, d)[:c])
                for p, x in zip(pools, sc))
        qs = torch.from_numpy(q[q_start[s]:q_start[s + 1]])
        mask = torch.arange(c)[None] <= torch.arange(c - n, c)[:, None]
        for i in range(h * g):
            t = torch.nn.functional.scaled_dot_product_attention(
                qs[None, :, i], k[None, :, i // g], v[None, :, i // g], attn_mask=mask, scale=0.125)
            assert np.abs(t[0].numpy() - out[q_start[s]:q_start[s + 1], i]).max() < 1e-12
            x = (qs[:, i] @ k[:, i // g].T) * 0.125
            x = torch.logsumexp(x.masked_fill(~mask, -math.inf), 1)
            assert np.abs(x.numpy() - lse[q_start[s]:q_start[s + 1], i]).max() < 1e-12


def test_load_reads_what_the_codes_say():
    rng = np.random.default_rng(5)
    pool = rng.integers(0, 127, (4, 16, 1, 64)).astype(np.uint8)
    scales = 2.0 ** rng.integers(-4, 4, (4, 1)).astype(np.float32)
    table = np.array([[3, -1, 0]], dtype=np.int32)
    y = f8.load(pool, scales, table, [40], [0, 40], 16)
    v = f8.values(pool, scales)
    assert (y[:16] == v[3]).all() and (y[16:32] == 0).all() and (y[32:] == v[0, :8]).all()
    y = f8.load(pool, scales, table, [40], [0, 3], 16, pos0=[38])
    assert (y[:2] == v[0, 6:8]).all() and (y[2] == 0).all()
