"""The 8-bit block-scaled cache on the GPU: store, load and decode attention
against the float64 oracle.

Tolerances. Store: bit-exact (every step is exact or one defined rounding).
Load: exact (one float32 product, one rounding to the type). Attention, for
values of about N(0, 1) and |v| <= vmax: with t accurate to d_t = 2^-17
(scores of |t| <= ~10 from products kept to ~2^-22, sums in float32), each
probability is off by d_t relatively, numerator and denominator together by
2 d_t vmax ~ 1e-4 (vmax <= 6), which is TOL["f32"]. 16-bit outputs add half
a step of the type relative to the value and, for the probabilities rounded
to f16, 2^-11 vmax in the worst case of all roundings alike.
"""
import math

import numpy as np
import pytest
import torch

from oracle import f8

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}  # half a step, relative
RUNS = 8


@pytest.fixture(scope="module")
def mt():
    import __graft_entry__
    __graft_entry__.build()
    from paged_kv_cache_gqa_gb300 import mtkv
    return mtkv


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).to("cuda")


def rounded(x, dt):
    """float64 array of the values of `dt` nearest to x."""
    return torch.from_numpy(np.asarray(x, dtype=np.float32)).to(DT[dt]).to(torch.float64).numpy()


class World:
    """A cache with every sequence filled up to its context, on host and device."""

    def __init__(self, mt, seed, ctx, h, d, bs, extra_blocks=3, holes=0.0, max_blocks=None):
        rng = self.rng = np.random.default_rng(seed)
        self.mt, self.ctx = mt, np.array(ctx, dtype=np.int32)
        self.h, self.d, self.bs = h, d, bs
        nb = [-(-int(c) // bs) for c in ctx]
        self.max_blocks = max(max(nb, default=0), 1) if max_blocks is None else max_blocks
        n_phys = self.n_phys = sum(nb) + extra_blocks
        ids = rng.permutation(n_phys)
        self.table = np.full((len(ctx), self.max_blocks), -1, dtype=np.int32)
        # entries past the context are never read: out-of-range ids there
        self.table[:] = 10 ** 8
        k = 0
        for s, n in enumerate(nb):
            self.table[s, :n] = ids[k:k + n]
            k += n
            if holes and n > 1:
                self.table[s, :n - 1][rng.random(n - 1) < holes] = -1
        self.pools = [rng.integers(0, 256, (n_phys, bs, h, d)).astype(np.uint8) for _ in range(2)]
        self.scales = [np.full((n_phys, h), np.nan, dtype=np.float32) for _ in range(2)]
        for s, n in enumerate(nb):
            for b in range(n):
                p = self.table[s, b]
                if p < 0:
                    continue
                rows = min(bs, int(ctx[s]) - b * bs)
                for pool, sc in zip(self.pools, self.scales):
                    x = rng.normal(size=(rows, h, d)) * np.exp(rng.normal(size=(1, h, 1)) * 0.3)
                    for j in range(h):
                        sc[p, j] = f8.pow2_scale(float(np.abs(x[:, j]).max()))
                    pool[p, :rows] = f8.encode(x / sc[p][None, :, None])

    def upload(self):
        self.dp = [dev(p) for p in self.pools]
        self.ds = [dev(s) for s in self.scales]
        self.cache = self.mt.f8_cache(*self.dp, *self.ds, dev(self.table), dev(self.ctx))
        return self.cache

    def q(self, rows, g, dt):
        x = rounded(self.rng.normal(size=(rows, self.h * g, self.d)), dt)
        return x, dev(x).to(DT[dt])


def runs_of(rng, rows, ctx):
    r = np.zeros((rows, RUNS, 2), dtype=np.int32)
    for i in range(rows):
        for k in rng.choice(RUNS, 3, replace=False):
            r[i, k] = rng.integers(-5, ctx[i] + 5), rng.integers(-3, ctx[i] // 2 + 4)
    return r


def compare(got, lse, want, want_lse, dt, vmax=6.0):
    got, lse = got.to(torch.float64).cpu().numpy(), lse.cpu().numpy()
    none = np.isinf(want_lse)
    assert (np.isneginf(lse) == none).all() and (got[none] == 0).all()
    tol = 1e-4 + STEP[dt] * np.abs(want) + (0.0 if dt == "f32" else 2.0 ** -11 * vmax)
    err = np.abs(got - want)
    assert (err <= tol).all(), f"out off by {err.max():.3g}"
    if (~none).any():
        e = np.abs(lse[~none] - want_lse[~none]).max()
        assert e <= 1e-4, f"lse off by {e:.3g}"


# ------------------------------------------------------------------- store

def run_store(w, cache, new, q_start, dt):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    x = [dev(n).to(DT[dt]) for n in new]
    w.mt.mt_kv_store_f8(cache, *x, dev(np.array(q_start, dtype=np.int32)), status=status)
    return w.mt.mt_check_device_status(status)


def check_cache(w):
    for pool, sc, dp, ds in zip(w.pools, w.scales, w.dp, w.ds):
        a, b = ds.cpu().numpy(), sc
        assert ((a == b) | (np.isnan(a) & np.isnan(b))).all()
        a = dp.cpu().numpy()
        nan = ((a & 127) == 127) & ((pool & 127) == 127)
        assert ((a == pool) | nan).all()


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("h,d,bs", [(3, 64, 16), (8, 128, 16), (2, 256, 16), (1, 64, 32),
                                    (5, 128, 32), (4, 256, 32)])
def test_store_is_bit_exact(mt, dt, h, d, bs):
    ctx = [1, 40, 0, 64, 17, 16, 33, 100]
    w = World(mt, 11, ctx, h, d, bs)
    cache = w.upload()
    # one row, all rows, none, a block's edge, across blocks, a whole block
    n = [1, 40, 0, 16, 2, 16, 20, 7]
    q_start = np.concatenate([[0], np.cumsum(n)])
    new = [w.rng.normal(size=(q_start[-1], h, d)) * 3 for _ in range(2)]
    for x in new:
        x[5:9] *= 40.0      # growth in the middle of blocks
        x[-2] = 0.0
    new = [rounded(x, dt) for x in new]
    assert run_store(w, cache, new, q_start, dt) == mt.MT_OK
    for x, pool, sc in zip(new, w.pools, w.scales):
        f8.store(pool, sc, x, w.table, w.ctx, q_start, bs)
    check_cache(w)


def test_store_step_by_step_equals_the_oracle(mt):
    # a sequence grown row by row and in chunks, rows getting larger
    h, d, bs = 2, 128, 16
    w = World(mt, 12, [60, 60], h, d, bs)
    w.upload()
    done = np.array([0, 0])
    while (done < 60).any():
        n = np.minimum(w.rng.integers(0, 7, 2), 60 - done)
        done = done + n
        q_start = np.concatenate([[0], np.cumsum(n)])
        if q_start[-1] == 0:
            continue
        ctx = done.astype(np.int32)
        cache = mt.f8_cache(*w.dp, *w.ds, dev(w.table), dev(ctx))
        new = [rounded(w.rng.normal(size=(q_start[-1], h, d)) * 1.2 ** done.max(), "f32")
               for _ in range(2)]
        assert run_store(w, cache, new, q_start, "f32") == mt.MT_OK
        for x, pool, sc in zip(new, w.pools, w.scales):
            f8.store(pool, sc, x, w.table, ctx, q_start, bs)
    check_cache(w)


@pytest.mark.parametrize("d,bs", [(64, 16), (256, 32)])
def test_store_special_values(mt, d, bs):
    h = 2
    w = World(mt, 13, [20, 3, 2 * bs, 7], h, d, bs)
    w.scales[0][w.table[0, 20 // bs - (20 % bs == 0)]] = np.inf  # kept rows under a bad scale
    w.scales[1][w.table[0, (20 - 1) // bs]] = 0.0
    w.scales[0][w.table[3, 0]] = 0.3                              # not a power of two
    cache = w.upload()
    q_start = [0, 2, 5, 5 + 2 * bs, 6 + 2 * bs]
    new = [w.rng.normal(size=(q_start[-1], h, d)).astype(np.float32) for _ in range(2)]
    new[0][0, 0, :3] = [np.nan, np.inf, -np.inf]
    new[1][1, 1, 5] = -np.inf
    new[0][2:5] = 0.0                       # a block of zeros with an infinity
    new[0][3, 1, 7] = np.inf
    new[1][2:5] = 1e-41                     # subnormal values
    new[0][5:9] *= 1e-30
    new[1][6] *= 1e30
    new[0][-1] *= 1e-3                      # fits under the kept 0.3
    assert run_store(w, cache, new, q_start, "f32") == mt.MT_OK
    for x, pool, sc in zip(new, w.pools, w.scales):
        f8.store(pool, sc, np.asarray(x, dtype=np.float64), w.table, w.ctx, q_start, bs)
    check_cache(w)


def test_store_skips_holes_and_flags_bad_input(mt):
    h, d, bs = 2, 64, 16
    w = World(mt, 14, [40, 40, 40, 40], h, d, bs)
    w.table[0, 1] = -1
    w.table[1, 1] = w.n_phys          # out of range
    w.ctx[2] = 5                      # fewer positions than rows
    cache = w.upload()
    q_start = [0, 30, 60, 70, 90]
    new = [w.rng.normal(size=(90, h, d)).astype(np.float32) for _ in range(2)]
    assert run_store(w, cache, new, q_start, "f32") == mt.MT_ERR_DEVICE_CHECK
    ok = [0, 1, 3]
    for x, pool, sc in zip(new, w.pools, w.scales):
        for s in ok:
            f8.store(pool, sc, x[q_start[s]:q_start[s + 1]], w.table[s:s + 1], w.ctx[s:s + 1],
                     [0, q_start[s + 1] - q_start[s]], bs)
    check_cache(w)
    # rows past the dense array, and a falling q_start
    assert run_store(w, cache, [x[:80] for x in new], [0, 0, 0, 0, 90], "f32") == \
        mt.MT_ERR_DEVICE_CHECK
    assert run_store(w, cache, new, [10, 5, 5, 5, 5], "f32") == mt.MT_ERR_DEVICE_CHECK
    check_cache(w)


@pytest.mark.parametrize("n_seqs", [1, 31, 32, 33, 70, 1100])
def test_store_finds_its_rows_among_any_number_of_sequences(mt, n_seqs):
    rng = np.random.default_rng(15)
    ctx = rng.integers(0, 50, n_seqs)
    n = np.minimum(rng.integers(0, 3, n_seqs) * rng.integers(0, 40, n_seqs), ctx)
    w = World(mt, 16, ctx, 1, 64, 16)
    cache = w.upload()
    q_start = np.concatenate([[0], np.cumsum(n)])
    new = [rounded(rng.normal(size=(q_start[-1], 1, 64)), "f16") for _ in range(2)]
    assert run_store(w, cache, new, q_start, "f16") == mt.MT_OK
    for x, pool, sc in zip(new, w.pools, w.scales):
        f8.store(pool, sc, x, w.table, w.ctx, q_start, 16)
    check_cache(w)


@pytest.mark.parametrize("q_start", [[0, 5, -2 ** 31, 7], [0, 5, 2 ** 31 - 1, 9],
                                     [-2 ** 31, 2 ** 31 - 1, 4, 4]])
def test_row_bounds_at_the_ends_of_the_integers(mt, q_start):
    w = World(mt, 17, [20, 20, 20], 2, 64, 16)
    cache = w.upload()
    new = [w.rng.normal(size=(7, 2, 64)).astype(np.float32) for _ in range(2)]
    assert run_store(w, cache, new, q_start, "f32") == mt.MT_ERR_DEVICE_CHECK
    q, qd = w.q(7, 2, "f32")
    out, _ = run_prefill(w, cache, qd, q_start, "f32", want_status=mt.MT_ERR_DEVICE_CHECK)
    good = 5 if q_start[1] == 5 else 0
    assert out[:good].isfinite().all() and out[good:].isnan().all()


# -------------------------------------------------------------------- load

@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("h,d,bs", [(3, 64, 16), (8, 128, 32), (1, 256, 16), (12, 64, 32)])
def test_load_is_exact(mt, dt, h, d, bs):
    ctx = [1, 70, 0, 33, 16]
    w = World(mt, 21, ctx, h, d, bs, holes=0.3)
    cache = w.upload()
    n = [1, 50, 0, 33, 3]
    q_start = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    for pos0 in (None, np.array([0, 7, 0, 0, 13], dtype=np.int32)):
        y = [torch.full((q_start[-1] + 2, h, d), 77.0, dtype=DT[dt], device="cuda")
             for _ in range(2)]
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        mt.mt_kv_load_f8(cache, *y, dev(q_start), pos0=None if pos0 is None else dev(pos0),
                         status=status)
        assert mt.mt_check_device_status(status) == mt.MT_OK
        for t, pool, sc in zip(y, w.pools, w.scales):
            want = f8.load(pool, sc, w.table, ctx, q_start, bs, pos0)
            want = torch.from_numpy(want).to(DT[dt])
            assert torch.equal(t[:-2].cpu(), want)
            assert (t[-2:] == 77.0).all()   # rows behind the last sequence


def test_load_flags_positions_outside_the_context(mt):
    w = World(mt, 22, [20, 5], 2, 64, 16)
    w.table[0, 0] = w.n_phys + 3
    cache = w.upload()
    for q_start, pos0 in (([0, 4, 4], [18, 0]), ([0, 1, 2], [19, -1]), ([0, 20, 20], None)):
        y = [torch.full((q_start[-1], 2, 64), 7.0, device="cuda") for _ in range(2)]
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        p = None if pos0 is None else dev(np.array(pos0, dtype=np.int32))
        mt.mt_kv_load_f8(cache, *y, dev(np.array(q_start, dtype=np.int32)), pos0=p, status=status)
        assert mt.mt_check_device_status(status) == mt.MT_ERR_DEVICE_CHECK
        for t, pool, sc in zip(y, w.pools, w.scales):
            want = f8.load(pool, sc, w.table, [20, 5], q_start, 16, pos0)
            assert (t.cpu().numpy() == want).all()


# ------------------------------------------------------------------ decode

def run_decode(w, cache, q, dt, ws=None, **kw):
    out = torch.full_like(q, float("nan"))
    lse = torch.full(q.shape[:2], float("nan"), device="cuda")
    args = w.mt.f8_attn_args(cache, q, out, scale=w.d ** -0.5, lse=lse, **kw)
    if ws is None:
        need = w.mt.mt_paged_attn_decode_f8_workspace_bytes(args)
        ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
        ws[:4] = 0
    w.mt.mt_paged_attn_decode_f8(args, ws)
    assert w.mt.mt_check_device_status(ws) == w.mt.MT_OK
    return out, lse


def oracle(w, q, **kw):
    return f8.attention(q, *w.pools, *w.scales, w.table, w.ctx, w.bs, w.d ** -0.5, **kw)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("h,g,d,bs", [(2, 2, 64, 16), (3, 3, 64, 32), (8, 4, 128, 16),
                                      (5, 8, 128, 32), (4, 4, 256, 16), (1, 7, 256, 32),
                                      (11, 1, 64, 16)])
@pytest.mark.parametrize("window", ["none", "spans", "runs"])
def test_decode_matches_the_oracle(mt, dt, h, g, d, bs, window):
    # lengths of zero and one, odd ends, a few CTAs' worth, holes
    ctx = [0, 1, 15, 16, 17, 100, 700, 333]
    w = World(mt, 31, ctx, h, d, bs, holes=0.15)
    cache = w.upload()
    q, qd = w.q(len(ctx), g, dt)
    kw = {}
    if window == "spans":
        sp = np.array([[0, 5], [0, 1], [3, 9], [16, 40], [5, 5], [-9, 50], [33, 690], [332, 999]],
                      dtype=np.int32)
        kw = {"spans": sp}
    elif window == "runs":
        kw = {"kv_map": runs_of(w.rng, len(ctx), ctx)}
    out, lse = run_decode(w, cache, qd, dt, **{k: dev(v) for k, v in kw.items()})
    compare(out, lse, *oracle(w, q, **kw), dt)


@pytest.mark.parametrize("h,g,d", [(8, 4, 128), (1, 8, 64), (3, 2, 256)])
def test_decode_long_context_is_split_and_merged(mt, h, g, d):
    ctx = [9000, 3, 5000]
    w = World(mt, 32, ctx, h, d, 16)
    cache = w.upload()
    q, qd = w.q(3, g, "f32")
    out, lse = run_decode(w, cache, qd, "f32")
    want, want_lse = oracle(w, q)
    compare(out, lse, want, want_lse, "f32")


def test_decode_short_table_takes_one_launch_with_the_same_result(mt):
    # up to 256 positions a table: every (sequence, head group) is one CTA's
    ctx = [0, 1, 200, 256, 100]
    w = World(mt, 33, ctx, 12, 128, 16, holes=0.1, max_blocks=16)
    cache = w.upload()
    q, qd = w.q(5, 2, "f32")
    want = oracle(w, q)
    compare(*run_decode(w, cache, qd, "f32"), *want, "f32")
    w.table = np.concatenate([w.table, np.full((5, 1), -1, dtype=np.int32)], 1)
    compare(*run_decode(w, w.upload(), qd, "f32"), *want, "f32")


@pytest.mark.parametrize("n_seqs", [1, 3, 32, 40, 200, 700])
@pytest.mark.parametrize("h,d", [(1, 64), (11, 64), (8, 128)])
def test_decode_splits_any_number_of_sequences(mt, n_seqs, h, d):
    rng = np.random.default_rng(33)
    ctx = rng.integers(0, 40, n_seqs) * rng.integers(0, 2 + 600 // n_seqs, n_seqs)
    w = World(mt, 34, ctx, h, d, 16, max_blocks=max(17, -(-int(ctx.max()) // 16)))
    cache = w.upload()
    q, qd = w.q(n_seqs, 1, "f16")
    out, lse = run_decode(w, cache, qd, "f16")
    compare(out, lse, *oracle(w, q), "f16")


def test_decode_is_the_same_every_time(mt):
    w = World(mt, 34, [3000, 40, 800], 2, 128, 16)
    cache = w.upload()
    _, qd = w.q(3, 4, "f32")
    a, la = run_decode(w, cache, qd, "f32")
    for _ in range(3):
        b, lb = run_decode(w, cache, qd, "f32")
        assert torch.equal(a, b) and torch.equal(la, lb)


def test_decode_extreme_magnitudes(mt):
    # tiny and huge scales, queries far from 1, logits far apart, one V block
    # much larger than the rest
    h, g, d, bs = 2, 4, 128, 16
    w = World(mt, 35, [500, 64, 200], h, d, bs)
    w.scales[0] *= np.float32(2.0 ** 40)
    w.scales[1] *= np.float32(2.0 ** -60)
    w.scales[1][w.table[0, 3]] *= np.float32(2.0 ** 20)
    cache = w.upload()
    q, _ = w.q(3, g, "f32")
    q = (q * 2.0 ** -40).astype(np.float32).astype(np.float64)
    q[1] *= 30.0
    out, lse = run_decode(w, cache, dev(q).float(), "f32")
    want, want_lse = oracle(w, q)
    unit = np.array([2.0 ** -40, 2.0 ** -60, 2.0 ** -60])[:, None, None]
    # the second sequence's logits reach a few hundred: d_t grows with them
    tol = np.array([1e-4, 3e-3, 1e-4])[:, None, None]
    assert (np.abs(out.cpu().numpy() - want) <= tol * unit * 6).all()
    assert (np.abs(lse.cpu().numpy() - want_lse) <= np.array([1e-4, 3e-3, 1e-4])[:, None]).all()


def test_decode_codes_outside_the_window_have_no_influence(mt):
    # NaN codes and NaN scales wherever nothing may be read
    h, g, d, bs = 3, 2, 64, 16
    w = World(mt, 36, [50, 20], h, d, bs)
    for s, c in enumerate(w.ctx):
        for p in range(int(c)):
            if not (s == 0 and 5 <= p < 44) and not (s == 1 and p >= 18):
                for pool in w.pools:
                    pool[w.table[s, p // bs], p % bs] = 0x7f
    for sc in w.scales:
        sc[w.table[1, 0]] = np.nan
    cache = w.upload()
    q, qd = w.q(2, g, "f32")
    sp = np.array([[5, 44], [18, 20]], dtype=np.int32)
    compare(*run_decode(w, cache, qd, "f32", spans=dev(sp)), *oracle(w, q, spans=sp), "f32")


def test_decode_nan_reaches_only_its_own_rows(mt):
    w = World(mt, 37, [40, 40], 2, 64, 16)
    cache = w.upload()
    q, _ = w.q(2, 2, "f32")
    q[0, 1, 3] = np.nan
    out, lse = run_decode(w, cache, dev(q).float(), "f32")
    assert out[0, 1].isnan().all() and lse[0, 1].isnan()
    want, want_lse = oracle(w, np.nan_to_num(q))
    keep = np.ones((2, 4), dtype=bool)
    keep[0, 1] = False
    assert np.abs(out.cpu().numpy() - want)[keep].max() <= 1e-4
    assert np.abs(lse.cpu().numpy() - want_lse)[keep].max() <= 1e-4


def test_decode_flags_bad_ids_and_lengths(mt):
    w = World(mt, 38, [100, 60], 2, 64, 16)
    good = w.table.copy()
    w.table[0, 2] = w.n_phys
    w.ctx[1] = 1000   # beyond the table
    cache = w.upload()
    q, qd = w.q(2, 2, "f32")
    out, lse = torch.empty_like(qd), torch.empty(2, 4, device="cuda")
    args = mt.f8_attn_args(cache, qd, out, scale=0.125, lse=lse)
    ws = torch.zeros(mt.mt_paged_attn_decode_f8_workspace_bytes(args), dtype=torch.uint8,
                     device="cuda")
    mt.mt_paged_attn_decode_f8(args, ws)
    assert mt.mt_check_device_status(ws) == mt.MT_ERR_DEVICE_CHECK
    w.table = good
    w.table[0, 2] = -1   # the bad block reads as a hole
    want, _ = f8.attention(q, *w.pools, *w.scales, w.table[:1], w.ctx[:1], 16, 0.125,
                           q_start=None)
    assert np.abs(out[0].cpu().numpy() - want[0]).max() <= 1e-4


def test_decode_offsets_beyond_32_bits(mt):
    # a pool of 4.5 GB whose last blocks hold the sequence
    h, d, bs = 8, 256, 32
    n_phys = (9 << 29) // (bs * h * d)
    w = World(mt, 39, [90], h, d, bs, extra_blocks=0)
    pools = [torch.empty(n_phys, bs, h, d, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.empty(n_phys, h, device="cuda") for _ in range(2)]
    for i in range(2):
        pools[i][-w.n_phys:] = dev(w.pools[i])
        scales[i][-w.n_phys:] = dev(w.scales[i])
    table = dev(w.table + np.int32(n_phys - w.n_phys))
    cache = mt.f8_cache(*pools, *scales, table, dev(w.ctx))
    q, qd = w.q(1, 2, "f32")
    compare(*run_decode(w, cache, qd, "f32"), *oracle(w, q), "f32")
    # and rows stored and read back there
    new = [rounded(w.rng.normal(size=(20, h, d)) * 2, "bf16") for _ in range(2)]
    qs = np.array([0, 20], dtype=np.int32)
    mt.mt_kv_store_f8(cache, *[dev(x).bfloat16() for x in new], dev(qs))
    y = [torch.empty(90, h, d, device="cuda") for _ in range(2)]
    mt.mt_kv_load_f8(cache, *y, dev(np.array([0, 90], dtype=np.int32)))
    for i in range(2):
        f8.store(w.pools[i], w.scales[i], new[i], w.table, w.ctx, qs, bs)
        want = f8.load(w.pools[i], w.scales[i], w.table, w.ctx, [0, 90], bs)
        assert (y[i].cpu().numpy() == want).all()


# --------------------------------------------------------- as used together

def test_store_then_decode_then_load(mt):
    # prompts stored at once, steps row by row, every step's attention and at
    # the end the whole cache read back
    h, g, d, bs, dt = 4, 2, 128, 16, "bf16"
    w = World(mt, 41, [60, 30, 16], h, d, bs)
    w.upload()
    table = dev(w.table)
    ctx = torch.tensor([52, 22, 8], dtype=torch.int32, device="cuda")
    cache = mt.f8_cache(*w.dp, *w.ds, table, ctx)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    n = [52, 22, 8]
    for step in range(9):
        q_start = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        new = [rounded(w.rng.normal(size=(q_start[-1], h, d)), dt) for _ in range(2)]
        mt.mt_kv_store_f8(cache, *[dev(x).bfloat16() for x in new], dev(q_start), status=status)
        w.ctx = ctx.cpu().numpy()
        for x, pool, sc in zip(new, w.pools, w.scales):
            f8.store(pool, sc, x, w.table, w.ctx, q_start, bs)
        q, qd = w.q(3, g, dt)
        compare(*run_decode(w, cache, qd, dt), *oracle(w, q), dt)
        if step < 8:
            ctx += 1
        n = [1, 1, 1]
    check_cache(w)
    q_start = np.concatenate([[0], np.cumsum(w.ctx)]).astype(np.int32)
    y = [torch.empty(q_start[-1], h, d, device="cuda") for _ in range(2)]
    mt.mt_kv_load_f8(cache, *y, dev(q_start), status=status)
    for t, pool, sc in zip(y, w.pools, w.scales):
        assert (t.cpu().numpy() == f8.load(pool, sc, w.table, w.ctx, q_start, bs)).all()
    assert mt.mt_check_device_status(status) == mt.MT_OK


def test_copy_on_write_of_a_block(mt):
    # a fork's last block, cells and scales, moved with mt_copy_cells, then
    # both sequences go their own ways
    h, d, bs = 2, 64, 16
    w = World(mt, 42, [24, 24], h, d, bs)
    w.table[1, 0] = w.table[0, 0]
    src, dst = int(w.table[0, 1]), int(w.table[1, 1])
    w.upload()
    mt.mt_copy_cells(w.dp, h * d, w.n_phys * bs, [(src * bs, dst * bs, bs)])
    mt.mt_copy_cells(w.ds, 4 * h, w.n_phys, [(src, dst, 1)])
    for pool, sc in zip(w.pools, w.scales):
        pool[dst], sc[dst] = pool[src], sc[src]
    ctx = np.array([25, 26], dtype=np.int32)
    cache = mt.f8_cache(*w.dp, *w.ds, dev(w.table), dev(ctx))
    new = [rounded(w.rng.normal(size=(3, h, d)) * 5, "f32") for _ in range(2)]
    assert run_store(w, cache, new, [0, 1, 3], "f32") == mt.MT_OK
    for x, pool, sc in zip(new, w.pools, w.scales):
        f8.store(pool, sc, x, w.table, ctx, [0, 1, 3], bs)
    check_cache(w)
    w.ctx = ctx
    q, qd = w.q(2, 2, "f32")
    compare(*run_decode(w, cache, qd, "f32"), *oracle(w, q), "f32")


def test_step_captured_into_a_graph_and_replayed(mt):
    h, g, d, bs = 2, 4, 128, 16
    w = World(mt, 43, [400, 90], h, d, bs)
    w.upload()
    ctx = torch.tensor([395, 80], dtype=torch.int32, device="cuda")
    cache = mt.f8_cache(*w.dp, *w.ds, dev(w.table), ctx)
    new = [torch.empty(2, h, d, device="cuda") for _ in range(2)]
    q = torch.empty(2, h * g, d, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(2, h * g, device="cuda")
    args = mt.f8_attn_args(cache, q, out, scale=d ** -0.5, lse=lse)
    ws = torch.zeros(mt.mt_paged_attn_decode_f8_workspace_bytes(args), dtype=torch.uint8,
                     device="cuda")
    qs = dev(np.array([0, 1, 2], dtype=np.int32))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        mt.mt_paged_attn_decode_f8(args, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mt.mt_kv_store_f8(cache, *new, qs)
        mt.mt_paged_attn_decode_f8(args, ws)
    for step in range(5):
        x = [rounded(w.rng.normal(size=(2, h, d)), "f32") for _ in range(2)]
        for t, v in zip(new, x):
            t.copy_(dev(v))
        qh, qd = w.q(2, g, "f32")
        q.copy_(qd)
        ctx += 1
        graph.replay()
        torch.cuda.synchronize()
        w.ctx = ctx.cpu().numpy()
        for v, pool, sc in zip(x, w.pools, w.scales):
            f8.store(pool, sc, v, w.table, w.ctx, [0, 1, 2], bs)
        compare(out, lse, *oracle(w, qh), "f32")
    check_cache(w)


def test_calls_on_two_streams_at_once(mt):
    w = World(mt, 44, [2500, 30], 2, 128, 16)
    cache = w.upload()
    qs = [w.q(2, 4, "f32") for _ in range(2)]
    sets = []
    for q, qd in qs:
        out, lse = torch.empty_like(qd), torch.empty(2, 8, device="cuda")
        args = mt.f8_attn_args(cache, qd, out, scale=w.d ** -0.5, lse=lse)
        ws = torch.zeros(mt.mt_paged_attn_decode_f8_workspace_bytes(args), dtype=torch.uint8,
                         device="cuda")
        sets.append((args, ws, out, lse, q, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(10):
        for args, ws, _, _, _, st in sets:
            mt.mt_paged_attn_decode_f8(args, ws, stream=st)
    torch.cuda.synchronize()
    for _, _, out, lse, q, _ in sets:
        compare(out, lse, *oracle(w, q), "f32")


# ----------------------------------------------------------------- prefill

def run_prefill(w, cache, q, q_start, dt, want_status=0, **kw):
    out = torch.full_like(q, float("nan"))
    lse = torch.full(q.shape[:2], float("nan"), device="cuda")
    kw = {k: dev(v) for k, v in kw.items()}
    args = w.mt.f8_attn_args(cache, q, out, scale=w.d ** -0.5, lse=lse,
                             q_start=dev(np.array(q_start, dtype=np.int32)), **kw)
    need = w.mt.mt_paged_attn_prefill_f8_workspace_bytes(args)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    ws[:4] = 0
    w.mt.mt_paged_attn_prefill_f8(args, ws)
    assert w.mt.mt_check_device_status(ws) == want_status
    return out, lse


def starts(n):
    return np.concatenate([[0], np.cumsum(n)]).astype(np.int32)


@pytest.mark.parametrize("h,g,d,bs", [(2, 1, 64, 16), (1, 3, 64, 32), (2, 4, 128, 16),
                                      (1, 8, 128, 32), (3, 7, 128, 16)])
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("window", ["none", "spans", "runs"])
def test_prefill_matches_the_oracle(mt, dt, h, g, d, bs, window):
    # no queries, one, all positions, odd ends, more than one tile, holes; an
    # empty sequence between others
    ctx = [1, 60, 0, 300, 129, 200]
    n = [1, 60, 0, 70, 1, 13]
    w = World(mt, 51, ctx, h, d, bs, holes=0.2)
    cache = w.upload()
    qs = starts(n)
    q, qd = w.q(int(qs[-1]), g, dt)
    kw = {}
    if window == "spans":
        sp = np.stack([w.rng.integers(-20, 150, qs[-1]), w.rng.integers(0, 320, qs[-1])], 1)
        kw = {"spans": sp.astype(np.int32)}
    elif window == "runs":
        kw = {"kv_map": runs_of(w.rng, int(qs[-1]), np.repeat(ctx, n))}
    out, lse = run_prefill(w, cache, qd, qs, dt, **kw)
    compare(out, lse, *oracle(w, q, q_start=qs, **kw), dt)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("h,g,d,n", [(1, 4, 128, 5), (2, 2, 64, 200), (8, 1, 128, 40)])
def test_prefill_long_context_is_cut_into_pieces(mt, dt, h, g, d, n):
    ctx = [2500, 40]
    w = World(mt, 52, ctx, h, d, 16, holes=0.02)
    cache = w.upload()
    qs = starts([n, 3])
    q, qd = w.q(int(qs[-1]), g, dt)
    rows = sorted({0, 1, n // 2, n - 1, n, n + 2})
    want, want_lse = oracle(w, q, q_start=qs, rows=rows)
    out, lse = run_prefill(w, cache, qd, qs, dt)
    compare(out[rows], lse[rows], want[rows], want_lse[rows], dt)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("order", [1, -1])
def test_prefill_pieces_of_long_and_short_sequences(mt, dt, order):
    # the long one's pieces set how many every unit is cut into; most pieces of the
    # short ones have no chunk
    ctx = ([6000] + [9 + 11 * s for s in range(9)])[::order]
    w = World(mt, 57, ctx, 8, 64, 16)
    cache = w.upload()
    n = [3] * 10
    q, qd = w.q(30, 1, dt)
    out, lse = run_prefill(w, cache, qd, starts(n), dt)
    want, want_lse = oracle(w, q, q_start=starts(n))
    compare(out, lse, want, want_lse, dt)


@pytest.mark.parametrize("dt", ["f32", "f16"])
@pytest.mark.parametrize("d", [64, 128])
def test_prefill_many_units_a_cta(mt, dt, d):
    # several units for every CTA, of unequal lengths: the hand-over from unit
    # to unit, sampled rows of every sequence
    rng = np.random.default_rng(53)
    ctx = rng.integers(1, 700, 40)
    n = np.minimum(rng.integers(1, 260, 40), ctx)
    w = World(mt, 53, ctx, 8, d, 16)
    cache = w.upload()
    qs = starts(n)
    q, qd = w.q(int(qs[-1]), 4, dt)
    rows = sorted(set((qs[:-1]).tolist() + (qs[1:] - 1).tolist()
                      + rng.integers(0, qs[-1], 30).tolist()))
    want, want_lse = oracle(w, q, q_start=qs, rows=set(rows))
    out, lse = run_prefill(w, cache, qd, qs, dt)
    compare(out[rows], lse[rows], want[rows], want_lse[rows], dt)
    assert torch.isfinite(out.float()).all() and torch.isfinite(lse).all()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("live", [[0], [0, 1, 2, 60, 61, 199], [199], []])
def test_prefill_long_runs_of_rows_that_see_nothing(mt, dt, live):
    # 200 sequences x 8 heads of one query each: a CTA has about ten units, most of
    # them without a position to read
    w = World(mt, 51, [20 + 7 * (s % 30) for s in range(200)], 8, 64, 16)
    cache = w.upload()
    q, qd = w.q(200, 1, dt)
    spans = np.zeros((200, 2), dtype=np.int32)
    spans[live] = 0, 1000
    out, lse = run_prefill(w, cache, qd, starts([1] * 200), dt, spans=spans)
    want, want_lse = oracle(w, q, q_start=starts([1] * 200), spans=spans)
    compare(out, lse, want, want_lse, dt)


def test_prefill_window_far_from_the_start(mt):
    # chunks before every query's window are not needed at all
    ctx, n = [1500, 900], [20, 150]
    w = World(mt, 54, ctx, 2, 128, 16)
    for pool in w.pools:
        for b in range(1500 // 16 - 30):
            pool[w.table[0, b]] = 0x7f      # NaN where no query looks
    cache = w.upload()
    qs = starts(n)
    q, qd = w.q(int(qs[-1]), 2, "bf16")
    pos = np.concatenate([np.arange(1480, 1500), np.arange(750, 900)])
    sp = np.stack([np.maximum(pos - 400, 0), pos + 1], 1).astype(np.int32)
    out, lse = run_prefill(w, cache, qd, qs, "bf16", spans=sp)
    compare(out, lse, *oracle(w, q, q_start=qs, spans=sp), "bf16")


@pytest.mark.parametrize("dt", ["f32", "f16"])
def test_prefill_nan_reaches_only_those_who_see_it(mt, dt):
    ctx = [200]
    w = World(mt, 55, ctx, 2, 64, 16)
    clean = [p.copy() for p in w.pools]
    w.pools[0][w.table[0, 150 // 16], 150 % 16, 0, 5] = 0x7f   # K of position 150, head 0
    w.pools[1][w.table[0, 170 // 16], 170 % 16, 1, 9] = 0xff   # V of position 170, head 1
    # slots past the context hold NaN too
    for p in w.pools:
        p[w.table[0, 199 // 16], 8:] = 0x7f
    cache = w.upload()
    q, qd = w.q(100, 2, dt)
    out, lse = run_prefill(w, cache, qd, [0, 100], dt)
    w.pools = clean
    want, want_lse = oracle(w, q, q_start=[0, 100])
    pos = np.arange(100, 200)
    hit = np.stack([pos >= 150, pos >= 150, pos >= 170, pos >= 170], 1)
    o, ls = out.double().cpu().numpy(), lse.cpu().numpy()
    assert np.isnan(o[hit]).all() and np.isnan(ls[hit]).all()
    tol = 1e-4 + STEP[dt] * np.abs(want[~hit]) + (0 if dt == "f32" else 2.0 ** -11 * 6)
    assert (np.abs(o[~hit] - want[~hit]) <= tol).all()
    assert np.abs(ls[~hit] - want_lse[~hit]).max() <= 1e-4


@pytest.mark.parametrize("dt", ["f32", "f16"])
def test_prefill_extreme_magnitudes(mt, dt):
    # V scales that differ by 2^30 between blocks, rising along the sequence,
    # and one block of zeros; tiny and huge K scales against the queries
    h, g, d, bs = 1, 4, 128, 16
    w = World(mt, 56, [400], h, d, bs)
    w.scales[0] *= np.float32(2.0 ** 12)
    for b in range(25):
        w.scales[1][w.table[0, b]] *= np.float32(2.0 ** (b - 12))
    w.scales[1][w.table[0, 4]] = 0.0
    cache = w.upload()
    q, _ = w.q(33, g, "f32")
    q = rounded(q * 2.0 ** -12, dt)
    out, lse = run_prefill(w, cache, dev(q).to(DT[dt]), [0, 33], dt)
    want, want_lse = oracle(w, q, q_start=[0, 33])
    # errors scale with the largest values around (2^12 times N(0, 1))
    tol = 2.0 ** 12 * (1e-4 + (0 if dt == "f32" else 2.0 ** -11 * 6)) + STEP[dt] * np.abs(want)
    assert (np.abs(out.double().cpu().numpy() - want) <= tol).all()
    assert np.abs(lse.cpu().numpy() - want_lse).max() <= 1e-4


def test_prefill_negative_softmax_scale(mt):
    w = World(mt, 57, [150], 1, 64, 16)
    cache = w.upload()
    q, qd = w.q(20, 2, "f32")
    out, lse = torch.empty_like(qd), torch.empty(20, 2, device="cuda")
    args = mt.f8_attn_args(cache, qd, out, scale=-0.125, lse=lse, q_start=dev(starts([20])))
    ws = torch.zeros(mt.mt_paged_attn_prefill_f8_workspace_bytes(args), dtype=torch.uint8,
                     device="cuda")
    mt.mt_paged_attn_prefill_f8(args, ws)
    want = f8.attention(q, *w.pools, *w.scales, w.table, w.ctx, 16, -0.125, q_start=[0, 20])
    compare(out, lse, *want, "f32")


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_prefill_leaves_other_rows_and_flags_bad_input(mt, dt):
    w = World(mt, 58, [40, 30, 50], 2, 64, 16)
    w.table[2, 1] = w.n_phys + 1
    cache = w.upload()
    # rows behind the last sequence are not written
    q, qd = w.q(30, 2, dt)
    out, lse = run_prefill(w, cache, qd, [3, 13, 13, 23], dt, want_status=mt.MT_ERR_DEVICE_CHECK)
    rest = list(range(3)) + list(range(23, 30))
    assert out[rest].isnan().all() and lse[rest].isnan().all()
    w.table[2, 1] = -1
    want, want_lse = oracle(w, q, q_start=[3, 13, 13, 23], rows=set(range(3, 23)))
    compare(out[3:23], lse[3:23], want[3:23], want_lse[3:23], dt)
    # more queries than positions: those without one see nothing
    out, lse = run_prefill(w, w.upload(), qd, [0, 0, 30, 30], dt)
    w.ctx[1] = 20
    out2, lse2 = run_prefill(w, w.upload(), qd, [0, 0, 30, 30], dt,
                             want_status=mt.MT_ERR_DEVICE_CHECK)
    assert (out2[:10] == 0).all() and lse2[:10].isneginf().all()
    want, want_lse = f8.attention(q[10:], *w.pools, *w.scales, w.table[1:2], w.ctx[1:2], 16,
                                  w.d ** -0.5, q_start=[0, 20])
    compare(out2[10:], lse2[10:], want, want_lse, dt)
    # rows outside the array, a falling q_start
    for bad in ([0, 0, 31, 31], [-2, 5, 5, 5], [9, 4, 4, 4]):
        out, _ = run_prefill(w, cache, qd, bad, dt, want_status=mt.MT_ERR_DEVICE_CHECK)
        assert out.isnan().all()


def test_prefill_chunks_equal_decode_and_one_prefill(mt):
    # a prompt stored and attended in chunks, then a decode step: the same rows
    # as one prefill over the whole, within the rounding of each
    h, g, d, bs, dt = 2, 4, 128, 16, "bf16"
    w = World(mt, 59, [300], h, d, bs)
    w.upload()
    table, ctx = dev(w.table), torch.zeros(1, dtype=torch.int32, device="cuda")
    cache = mt.f8_cache(*w.dp, *w.ds, table, ctx)
    done = 0
    for n in (128, 100, 71, 1):
        done += n
        ctx.fill_(done)
        qs = dev(starts([n]))
        new = [rounded(w.rng.normal(size=(n, h, d)), dt) for _ in range(2)]
        mt.mt_kv_store_f8(cache, *[dev(x).bfloat16() for x in new], qs)
        w.ctx[0] = done
        for x, pool, sc in zip(new, w.pools, w.scales):
            f8.store(pool, sc, x, w.table, w.ctx, [0, n], bs)
        q, qd = w.q(n, g, dt)
        want = oracle(w, q, q_start=[0, n])
        compare(*run_prefill(w, cache, qd, [0, n], dt), *want, dt)
        if n == 1:
            compare(*run_decode(w, cache, qd, dt), *want, dt)
    check_cache(w)


def test_prefill_captured_into_a_graph_and_on_two_streams(mt):
    w = World(mt, 60, [900, 200], 2, 128, 16)
    cache = w.upload()
    qs = starts([40, 100])
    sets = []
    for _ in range(2):
        q, qd = w.q(140, 4, "f16")
        out, lse = torch.empty_like(qd), torch.empty(140, 8, device="cuda")
        args = mt.f8_attn_args(cache, qd, out, scale=w.d ** -0.5, lse=lse, q_start=dev(qs))
        ws = torch.zeros(mt.mt_paged_attn_prefill_f8_workspace_bytes(args), dtype=torch.uint8,
                         device="cuda")
        sets.append((args, ws, out, lse, q, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for args, ws, _, _, _, st in sets:
            mt.mt_paged_attn_prefill_f8(args, ws, stream=st)
    torch.cuda.synchronize()
    for _, _, out, lse, q, _ in sets:
        compare(out, lse, *oracle(w, q, q_start=qs), "f16")
    args, ws, out, lse, q, _ = sets[0]
    first = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mt.mt_paged_attn_prefill_f8(args, ws)
        mt.mt_paged_attn_prefill_f8(sets[1][0], ws)   # the same workspace, in order
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)
        compare(sets[1][2], sets[1][3], *oracle(w, sets[1][4], q_start=qs), "f16")


@pytest.mark.parametrize("max_blocks", [0, 2, 40])
def test_a_cache_without_blocks(mt, max_blocks):
    pool = torch.empty(0, 16, 2, 64, dtype=torch.uint8, device="cuda")
    sc = torch.empty(0, 2, device="cuda")
    ctx = np.array([0, min(max_blocks * 16, 500)], dtype=np.int32)
    table = torch.full((2, max_blocks), -1, dtype=torch.int32, device="cuda")
    cache = mt.f8_cache(pool, pool, sc, sc, table, dev(ctx))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q_start = dev(np.array([0, 0, min(ctx[1], 3)], dtype=np.int32))
    x = [torch.randn(3, 2, 64, device="cuda") for _ in range(2)]
    mt.mt_kv_store_f8(cache, *x, q_start, status=status)
    y = [torch.full((3, 2, 64), 7.0, device="cuda") for _ in range(2)]
    mt.mt_kv_load_f8(cache, *y, q_start, status=status)
    assert mt.mt_check_device_status(status) == mt.MT_OK
    for call, rows, kw in (("decode", 2, {}), ("prefill", 3, {"q_start": q_start})):
        q = torch.randn(rows, 4, 64, device="cuda")
        out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
        args = mt.f8_attn_args(cache, q, out, scale=0.1, lse=lse, **kw)
        size = getattr(mt, f"mt_paged_attn_{call}_f8_workspace_bytes")(args)
        ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
        getattr(mt, f"mt_paged_attn_{call}_f8")(args, ws)
        assert mt.mt_check_device_status(ws) == mt.MT_OK
        n = rows if call == "decode" or max_blocks else 0   # rows that a sequence has
        assert (out[:n] == 0).all() and lse[:n].isneginf().all()
        assert (out[n:] == 7.0).all()
    n = 3 if max_blocks else 0
    for t in y:
        assert (t[:n] == 0).all() and (t[n:] == 7.0).all()
