"""Host-side checks of the calls for long, shared and bounded latent caches,
which answer without a GPU."""
import ctypes

import pytest

import sequence_sharded_mla_gb300 as mla

INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -6


def p(x):
    return None if x is None else ctypes.c_void_p(x)


def evict(data=512, scale=None, dtype=0, pages=4, page=64, bt=512, mp=4, sl=512, B=2, w=1024, ws_=300,
          width=256, keep=512, first=None, recent=0, nbt=512, nmp=2, new=8192, kept=512, mk=128,
          wo=65536, ws=512, wb=256):
    kv = mla.mla_kv_pages(data, scale, dtype, pages, page)
    return mla.lib().mla_cache_evict(ctypes.byref(kv), p(bt), mp, p(sl), B, p(w), ws_, width, p(keep),
                                     p(first), recent, p(nbt), nmp, p(new), p(kept), mk, p(wo), p(ws),
                                     wb, None)


@pytest.mark.parametrize("kw,want", [
    (dict(data=None), INVALID), (dict(data=520), INVALID), (dict(dtype=2), INVALID),
    (dict(dtype=1), INVALID), (dict(scale=512), INVALID), (dict(dtype=1, scale=514), INVALID),
    (dict(pages=0), INVALID), (dict(page=32), UNSUPPORTED), (dict(bt=None), INVALID),
    (dict(bt=514), INVALID), (dict(mp=0), INVALID), (dict(sl=None), INVALID), (dict(sl=513), INVALID),
    (dict(B=0), INVALID), (dict(w=None), INVALID), (dict(w=1026), INVALID), (dict(ws_=255), INVALID),
    (dict(width=0), INVALID), (dict(width=(1 << 30) + 1, ws_=1 << 31), UNSUPPORTED),
    (dict(keep=None), INVALID), (dict(keep=514), INVALID), (dict(first=514), INVALID),
    (dict(recent=-1), INVALID), (dict(nbt=None), INVALID), (dict(nbt=514), INVALID),
    (dict(nmp=0), INVALID), (dict(nmp=1), INVALID), (dict(new=None), INVALID), (dict(new=512), INVALID),
    (dict(new=516), INVALID), (dict(new=514), INVALID), (dict(keep=8196), INVALID),
    (dict(first=8188), INVALID), (dict(kept=None), INVALID),
    (dict(kept=514), INVALID), (dict(mk=0), INVALID), (dict(mk=129), INVALID), (dict(wo=65538), INVALID),
    (dict(wo=1024), INVALID), (dict(wo=512), INVALID), (dict(B=1 << 30, mk=256, nmp=4), INVALID),
    (dict(ws=None), WORKSPACE), (dict(ws=520), WORKSPACE), (dict(wb=255), WORKSPACE),
])
def test_eviction_refusals(kw, want):
    assert evict(**kw) == want


@pytest.mark.parametrize("mk", [(1 << 30) + 1, (1 << 31) - 16384, (1 << 31) - 1])
def test_eviction_refuses_more_positions_than_it_indexes(mk):
    # a position and a cluster's step have to fit 32 bits
    assert evict(B=1, mk=mk, nmp=1 << 25, wo=None) == UNSUPPORTED
    assert evict(B=1, mk=1 << 30, nmp=1 << 25, wo=None, ws=None) == WORKSPACE


@pytest.mark.parametrize("kw", [
    dict(kept=8192), dict(kept=8196), dict(kept=8192 - 1020), dict(kept=65536), dict(kept=65536 + 1020),
    dict(wo=8196), dict(wo=8192 - 1020), dict(kept=512), dict(kept=1024), dict(kept=2000), dict(kept=4096),
    dict(kept=4096 + 4), dict(wo=4100), dict(new=4096 + 28), dict(wo=600), dict(kept=16384 + 12),
    dict(wo=16384), dict(new=16384 + 12), dict(first=900000, kept=900000 + 4), dict(kept=3244),
])
def test_eviction_refuses_outputs_in_other_arrays(kw):
    # block_table 4096 .. 4128, new_block_table 16384 .. 16400, weights 1024 .. 3248,
    # kept and weights_out of 1024 bytes, new_seq_lens 8192 .. 8200
    apart = dict(bt=4096, nbt=16384, sl=512, keep=520, w=1024, new=8192, kept=32768, wo=65536)
    assert evict(**{**apart, **kw}) == INVALID
    # next to each other is apart
    ends = dict(apart, kept=8200, wo=8200 + 1024, new=8192, ws=None)
    assert evict(**ends) == WORKSPACE


def weights(q=512, data=512, scale=None, dtype=0, pages=4, page=64, bt=512, mp=4, sl=512,
            shape=(2, 1, 16, 0, 0.07, None), lse=512, before=None, bs=0, out=65536, os_=256, width=256,
            ws=512, wb=1 << 30):
    kv = mla.mla_kv_pages(data, scale, dtype, pages, page)
    sh = mla.mla_shape(*shape)
    return mla.lib().mla_attention_weights(p(q), ctypes.byref(kv), p(bt), mp, p(sl), ctypes.byref(sh),
                                           p(lse), p(before), bs, p(out), os_, width, p(ws), wb, None)


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), INVALID), (dict(q=520), INVALID), (dict(data=None), INVALID), (dict(data=520), INVALID),
    (dict(dtype=2), INVALID), (dict(dtype=1), INVALID), (dict(scale=512), INVALID),
    (dict(pages=0), INVALID), (dict(pages=(1 << 24) + 1), UNSUPPORTED), (dict(page=32), UNSUPPORTED),
    (dict(bt=None), INVALID), (dict(bt=514), INVALID), (dict(mp=0), INVALID), (dict(sl=None), INVALID),
    (dict(sl=514), INVALID), (dict(lse=None), INVALID), (dict(lse=514), INVALID), (dict(out=None), INVALID),
    (dict(out=514), INVALID), (dict(os_=255), INVALID), (dict(width=0), INVALID),
    (dict(before=514, bs=256), INVALID), (dict(before=1024, bs=255), INVALID),
    (dict(before=65540, bs=256), INVALID), (dict(before=65536, bs=300), INVALID),
    (dict(shape=(0, 1, 16, 0, 0.07, None)), INVALID), (dict(shape=(2, 0, 16, 0, 0.07, None)), INVALID),
    (dict(shape=(2, 1, 16, 2, 0.07, None)), INVALID), (dict(shape=(2, 1, 16, 0, 0.0, None)), INVALID),
    (dict(shape=(2, 1, 16, 0, 0.07, 514)), INVALID), (dict(shape=(2, 1, 24, 0, 0.07, None)), UNSUPPORTED),
    (dict(shape=(1 << 15, 256, 64, 0, 0.07, None)), UNSUPPORTED),
    (dict(width=(1 << 30) + 1, os_=1 << 31), UNSUPPORTED),
    (dict(shape=(1 << 10, 1, 16, 0, 0.07, None), width=1 << 30, os_=1 << 30, mp=1 << 24), UNSUPPORTED),
    (dict(ws=None), WORKSPACE), (dict(ws=520), WORKSPACE), (dict(wb=255), WORKSPACE),
])
def test_weights_refusals(kw, want):
    assert weights(**kw) == want


def test_weights_workspace():
    size = mla.mla_attention_weights_workspace_size
    assert 0 < size(3, 1, 16) <= 1024
    assert size(3, 2, 16, fp8=True) >= 96 * (1152 + 4)
    assert size(0, 1, 16) == 0 and size(1, 0, 16) == 0
