"""Argument checks of the 8-bit block-scaled cache's entry points: refused on
the host, before any launch (no GPU needed)."""
import ctypes
import os

import pytest
import torch


@pytest.fixture(scope="module")
def mt():
    from paged_kv_cache_gqa_gb300 import mtkv
    if not os.path.exists(mtkv.LIB_PATH):
        from paged_kv_cache_gqa_gb300 import build as b
        try:
            b.build()
        except RuntimeError as e:  # pragma: no cover - no toolkit
            pytest.skip(f"cannot build libmtkv here: {e}")
    mtkv.lib()
    return mtkv


A = 0x10000  # a stand-in address: refused calls never look at it


def cache_of(mt, **kw):
    c = mt.mt_f8_cache()
    base = dict(k_pool=A, v_pool=A, k_scales=A, v_scales=A, block_table=A, context_lens=A,
                n_seqs=2, n_kv_heads=2, head_dim=64, block_size=16, max_blocks=4,
                n_phys_blocks=8)
    for k, v in {**base, **kw}.items():
        setattr(c, k, v)
    return c


BAD_CACHE = [(dict(n_seqs=-1), 1), (dict(n_kv_heads=0), 1), (dict(max_blocks=-1), 1),
             (dict(n_phys_blocks=-1), 1), (dict(head_dim=96), 2), (dict(head_dim=0), 1),
             (dict(block_size=8), 2), (dict(n_kv_heads=257), 2), (dict(k_pool=None), 1),
             (dict(v_scales=None), 1), (dict(block_table=None), 1), (dict(context_lens=None), 1),
             (dict(k_pool=A + 8), 1), (dict(max_blocks=1 << 28), 2),
             (dict(max_blocks=(1 << 27) - 1), 2), (dict(max_blocks=(1 << 26) - 1, block_size=32), 2),
             (dict(n_phys_blocks=1 << 31), 2)]


@pytest.mark.parametrize("bad,status", BAD_CACHE)
def test_bad_caches_are_refused(mt, bad, status):
    c = cache_of(mt, **bad)
    L = mt.lib()
    assert L.mt_kv_store_f8(ctypes.byref(c), 0, A, A, A, 3, None, None) == status
    assert L.mt_kv_load_f8(ctypes.byref(c), 0, A, A, A, None, 3, None, None) == status
    a = attn_of(mt, cache=c)
    assert L.mt_paged_attn_decode_f8(ctypes.byref(a), A, 1 << 40, None) == status
    assert L.mt_paged_attn_decode_f8_workspace_bytes(ctypes.byref(a)) == 0
    assert L.mt_paged_attn_prefill_f8(ctypes.byref(a), A, 1 << 40, None) == status
    assert L.mt_paged_attn_prefill_f8_workspace_bytes(ctypes.byref(a)) == 0
    assert mt.mt_last_error()


@pytest.mark.parametrize("call", ["mt_kv_store_f8", "mt_kv_load_f8"])
def test_bad_rows_are_refused(mt, call):
    def run(dtype=0, k=A, v=A, qs=A, n=3):
        c, f = ctypes.byref(cache_of(mt)), getattr(mt.lib(), call)
        return f(c, dtype, k, v, qs, n, None, None) if call == "mt_kv_store_f8" else \
            f(c, dtype, k, v, qs, None, n, None, None)
    assert run(dtype=3) == mt.MT_ERR_INVALID_ARG and run(dtype=-1) == mt.MT_ERR_INVALID_ARG
    assert run(n=-1) == mt.MT_ERR_INVALID_ARG
    assert run(k=None) == mt.MT_ERR_INVALID_ARG and run(v=None) == mt.MT_ERR_INVALID_ARG
    assert run(qs=None) == mt.MT_ERR_INVALID_ARG
    assert run(k=A + 4) == mt.MT_ERR_INVALID_ARG and run(v=A + 8) == mt.MT_ERR_INVALID_ARG
    assert run(n=0) == mt.MT_OK   # nothing to do, nothing launched


def attn_of(mt, cache=None, **kw):
    a = mt.mt_f8_attn_args()
    a.cache = cache_of(mt) if cache is None else cache
    base = dict(dtype=0, q=A, out=A, lse=A, q_start=None, spans=None, kv_map=None, n_tokens=2,
                n_heads=4, scale=0.125)
    for k, v in {**base, **kw}.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("bad,status", [
    (dict(dtype=5), 1), (dict(n_heads=3), 1), (dict(n_heads=0), 1), (dict(n_heads=18), 2),
    (dict(n_tokens=3), 1), (dict(q_start=A), 1), (dict(spans=A, kv_map=A), 1), (dict(q=None), 1),
    (dict(out=None), 1), (dict(q=A + 4), 1), (dict(out=A + 8), 1)])
def test_bad_decode_arguments_are_refused(mt, bad, status):
    a = attn_of(mt, **bad)
    if bad.get("n_tokens") == 3:
        a.cache.n_seqs = 2
    assert mt.lib().mt_paged_attn_decode_f8(ctypes.byref(a), A, 1 << 40, None) == status
    assert mt.mt_last_error()


@pytest.mark.parametrize("bad,status", [
    (dict(dtype=5), 1), (dict(n_heads=3), 1), (dict(n_heads=0), 1), (dict(n_heads=18), 2),
    (dict(n_tokens=-3), 1), (dict(q_start=None), 1), (dict(spans=A, kv_map=A), 1),
    (dict(q=None), 1), (dict(out=None), 1), (dict(q=A + 4), 1), (dict(out=A + 8), 1),
    (dict(n_tokens=1 << 30), 2)])
def test_bad_prefill_arguments_are_refused(mt, bad, status):
    a = attn_of(mt, **{"n_tokens": 7, "q_start": A, **bad})
    # (a size that only the device count limits is refused after the device query)
    got = mt.lib().mt_paged_attn_prefill_f8(ctypes.byref(a), A, 1 << 40, None)
    assert got == status or (bad.get("n_tokens") == 1 << 30 and got == mt.MT_ERR_CUDA)
    assert mt.mt_last_error()


def test_prefill_refuses_wide_heads(mt):
    a = attn_of(mt, cache=cache_of(mt, head_dim=256), n_tokens=7, q_start=A)
    assert mt.lib().mt_paged_attn_prefill_f8(ctypes.byref(a), A, 1 << 40, None) == \
        mt.MT_ERR_UNSUPPORTED


def test_null_arguments_are_refused(mt):
    L = mt.lib()
    assert L.mt_kv_store_f8(None, 0, A, A, A, 3, None, None) == mt.MT_ERR_INVALID_ARG
    assert L.mt_kv_load_f8(None, 0, A, A, A, None, 3, None, None) == mt.MT_ERR_INVALID_ARG
    assert L.mt_paged_attn_decode_f8(None, A, 1 << 40, None) == mt.MT_ERR_INVALID_ARG
    assert L.mt_paged_attn_prefill_f8(None, A, 1 << 40, None) == mt.MT_ERR_INVALID_ARG


def test_binding_refuses_tensors_of_other_places(mt):
    pool = torch.zeros(2, 16, 1, 64, dtype=torch.uint8)
    sc, tab, ctx = torch.zeros(2, 1), torch.zeros(1, 2, dtype=torch.int32), \
        torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="current CUDA device"):
        mt.f8_cache(pool, pool, sc, sc, tab, ctx)
    with pytest.raises(ValueError, match="shape"):
        mt.f8_cache(pool, pool[:1], sc, sc, tab, ctx)
    with pytest.raises(ValueError, match="scales"):
        mt.f8_cache(pool, pool, sc[:1], sc, tab, ctx)
    with pytest.raises(ValueError, match="context_lens"):
        mt.f8_cache(pool, pool, sc, sc, tab, tab)


class Elsewhere:
    """A tensor's face on a device that is not the current one."""

    def __init__(self, t, index):
        self._t, self.device = t, torch.device("cuda", index)
        self.dtype, self.shape = t.dtype, t.shape

    def get_device(self):
        return self.device.index

    def is_contiguous(self):
        return self._t.is_contiguous()

    def data_ptr(self):
        return A


def test_binding_checks_device_dtype_and_layout(mt, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    t = torch.zeros(4, 6)
    f32 = (torch.float32,)
    assert mt._ptr_here(Elsewhere(t, 0), f32, "x") == A
    with pytest.raises(ValueError, match="current CUDA device"):
        mt._ptr_here(Elsewhere(t, 1), f32, "x")
    with pytest.raises(ValueError, match="dtype"):
        mt._ptr_here(Elsewhere(t.half(), 0), f32, "x")
    with pytest.raises(ValueError, match="contiguous"):
        mt._ptr_here(Elsewhere(t.t(), 0), f32, "x")
    with pytest.raises(ValueError, match="workspace"):
        mt._scratch_here(Elsewhere(t, 1), "workspace", 0)
    with pytest.raises(ValueError, match="contiguous"):
        mt._scratch_here(Elsewhere(t[:, ::2], 0), "workspace", 0)
    c = cache_of(mt)
    assert mt._here(c, "x") == 0
    c._device = 1
    for call in (lambda: mt.mt_kv_store_f8(c, t, t, t), lambda: mt.mt_kv_load_f8(c, t, t, t),
                 lambda: mt.mt_paged_attn_decode_f8(c, t), lambda: mt.mt_paged_attn_prefill_f8(c, t)):
        with pytest.raises(ValueError, match="on device 1"):
            call()
