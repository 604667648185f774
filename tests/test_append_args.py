"""Host-side checks of the rotary, append and e4m3 grouped-query calls, which
answer without a GPU, and the rotary frequency tables against closed forms."""
import ctypes
import math

import pytest
import torch

import sequence_sharded_mla_gb300 as mla

FAKE, ODD8, ODD4, ODD2 = (ctypes.c_void_p(x) for x in (512, 520, 516, 514))
INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -6


def tok(batch=2, q_len=1, seq=512, q=None, pos=None):
    return mla.mla_tokens(batch, q_len, seq, q, pos)


def rope(inv=512, rot=64, first=0, inter=0, f=1.0):
    return mla.mla_rope(inv, rot, first, inter, f)


def apply(x=FAKE, xs=1024, out=FAKE, ys=1024, t=None, H=8, D=128, r=None):
    return mla.lib().mla_rope_apply(x, xs, out, ys, ctypes.byref(t or tok()), H, D,
                                    ctypes.byref(r or rope()), None)


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), INVALID), (dict(out=None), INVALID), (dict(x=ODD8), INVALID),
    (dict(xs=1020), INVALID), (dict(xs=1016), INVALID), (dict(ys=1032), INVALID),
    (dict(H=0), INVALID), (dict(H=9), INVALID), (dict(D=0), INVALID),
    (dict(t=tok(batch=0)), INVALID), (dict(t=tok(q_len=0)), INVALID),
    (dict(t=tok(seq=None)), INVALID), (dict(t=tok(q=514)), INVALID), (dict(t=tok(pos=514)), INVALID),
    (dict(t=tok(batch=1 << 20, q_len=1 << 10)), INVALID),
    (dict(r=rope(inv=None)), INVALID), (dict(r=rope(inv=516)), INVALID), (dict(r=rope(rot=0)), INVALID),
    (dict(r=rope(rot=144)), INVALID), (dict(r=rope(first=72)), INVALID), (dict(r=rope(first=-8)), INVALID),
    (dict(r=rope(inter=2)), INVALID), (dict(r=rope(f=math.inf)), INVALID),
    (dict(r=rope(rot=24)), UNSUPPORTED), (dict(r=rope(first=4)), UNSUPPORTED),
    (dict(D=132, xs=1056, ys=1056), UNSUPPORTED), (dict(D=2048, xs=1 << 14, ys=1 << 14), UNSUPPORTED),
])
def test_rotation_refusals(kw, want):
    assert apply(**kw) == want


def latent(x=FAKE, xs=576, data=512, scale=None, dtype=0, pages=4, page=64, bt=FAKE, mp=1, t=None,
           r=None, q=None, qs=0, y=None, ys=0, H=0, shard=0, N=1, ws=FAKE, wb=256):
    kv = mla.mla_kv_pages(data, scale, dtype, pages, page)
    return mla.lib().mla_cache_append(x, xs, ctypes.byref(kv), bt, mp, ctypes.byref(t or tok()),
                                      None if r is None else ctypes.byref(r), q, qs, y, ys, H, shard,
                                      N, ws, wb, None)


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), INVALID), (dict(xs=568), INVALID), (dict(xs=580), INVALID), (dict(x=ODD4), INVALID),
    (dict(data=None), INVALID), (dict(data=520), INVALID), (dict(dtype=2), INVALID),
    (dict(dtype=1), INVALID), (dict(scale=512), INVALID), (dict(dtype=1, scale=514), INVALID),
    (dict(pages=0), INVALID), (dict(page=32), UNSUPPORTED), (dict(bt=None), INVALID),
    (dict(bt=ODD2), INVALID), (dict(mp=0), INVALID), (dict(t=tok(seq=None, pos=512)), INVALID),
    (dict(N=0), INVALID), (dict(N=9), INVALID), (dict(N=2, shard=2), INVALID), (dict(shard=-1), INVALID),
    (dict(r=rope(first=520)), INVALID), (dict(r=rope(rot=72, first=0)), UNSUPPORTED),
    (dict(q=FAKE, qs=576, y=FAKE, ys=576, H=1), INVALID),                 # q without rope
    (dict(r=rope(first=512), q=FAKE, qs=576, y=None, ys=576, H=1), INVALID),
    (dict(r=rope(first=512), q=FAKE, qs=576, y=FAKE, ys=584, H=1), INVALID),
    (dict(r=rope(first=512), q=FAKE, qs=576, y=FAKE, ys=576, H=0), INVALID),
    (dict(ws=None), WORKSPACE), (dict(ws=ODD8), WORKSPACE), (dict(wb=255), WORKSPACE),
])
def test_latent_append_refusals(kw, want):
    assert latent(**kw) == want


def pages(k=512, v=512, ks=512, vs=512, dtype=1, block=64, n=4, page=64, Hkv=2):
    return mla.gqa_block_pages(k, v, ks, vs, dtype, block, n, page, Hkv)


def heads(k=FAKE, ks=256, v=FAKE, vs=256, c=None, wb=256):
    return mla.lib().gqa_cache_append(k, ks, v, vs, ctypes.byref(c or pages()), FAKE, 1,
                                      ctypes.byref(tok()), None, None, 0, None, 0, 0, 0, 1, FAKE, wb,
                                      None)


@pytest.mark.parametrize("kw,want", [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(k=ODD8), INVALID), (dict(ks=248), INVALID),
    (dict(vs=260), INVALID), (dict(c=pages(k=None)), INVALID), (dict(c=pages(v=520)), INVALID),
    (dict(c=pages(ks=None)), INVALID), (dict(c=pages(vs=514)), INVALID), (dict(c=pages(dtype=0)), INVALID),
    (dict(c=pages(dtype=3)), INVALID), (dict(c=pages(block=0)), INVALID), (dict(c=pages(block=48)), INVALID),
    (dict(c=pages(block=128)), INVALID), (dict(c=pages(n=0)), INVALID), (dict(c=pages(Hkv=0)), INVALID),
    (dict(c=pages(page=128)), UNSUPPORTED), (dict(wb=0), WORKSPACE),
])
def test_head_append_refusals(kw, want):
    assert heads(**kw) == want


def attend(q=FAKE, c=None, bt=FAKE, mp=1, sl=FAKE, ql=None, shape=(2, 1, 8, 2, 128, 0, 0.088), shard=-1,
           N=2, layout=0, o=FAKE, l=FAKE, ws=FAKE, wb=1 << 30):
    sh = mla.gqa_shape(*shape)
    return mla.lib().gqa_decode_partial_fp8(q, ctypes.byref(c or pages()), bt, mp, sl, ql,
                                            ctypes.byref(sh), shard, N, layout, o, l, ws, wb, None)


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), INVALID), (dict(bt=None), INVALID), (dict(sl=None), INVALID), (dict(o=None), INVALID),
    (dict(l=None), INVALID), (dict(q=ODD8), INVALID), (dict(o=ODD8), INVALID), (dict(bt=ODD2), INVALID),
    (dict(sl=ODD2), INVALID), (dict(ql=ODD2), INVALID), (dict(mp=0), INVALID), (dict(N=0), INVALID),
    (dict(N=9), INVALID), (dict(shard=2), INVALID), (dict(shard=-2), INVALID), (dict(layout=4), INVALID),
    (dict(layout=-1), INVALID), (dict(layout=2), INVALID), (dict(layout=3), INVALID),
    (dict(N=3), UNSUPPORTED), (dict(c=pages(k=None)), INVALID), (dict(c=pages(k=520)), INVALID),
    (dict(c=pages(vs=None)), INVALID), (dict(c=pages(ks=514)), INVALID), (dict(c=pages(dtype=0)), INVALID),
    (dict(c=pages(block=3)), INVALID), (dict(c=pages(Hkv=4)), INVALID), (dict(c=pages(n=0)), INVALID),
    (dict(c=pages(page=32)), UNSUPPORTED), (dict(c=pages(n=1 << 24)), UNSUPPORTED),
    (dict(shape=(0, 1, 8, 2, 128, 0, 0.1)), INVALID), (dict(shape=(2, 0, 8, 2, 128, 0, 0.1)), INVALID),
    (dict(shape=(2, 1, 8, 2, 128, 2, 0.1)), INVALID), (dict(shape=(2, 1, 8, 2, 128, 0, 0.0)), INVALID),
    (dict(shape=(2, 1, 8, 2, 128, 0, math.nan)), INVALID),
    (dict(shape=(1 << 12, 1 << 8, 64, 2, 128, 0, 0.1)), INVALID),
    (dict(shape=(2, 1, 8, 2, 64, 0, 0.1)), UNSUPPORTED), (dict(shape=(2, 1, 7, 2, 128, 0, 0.1)), UNSUPPORTED),
    (dict(shape=(2, 1, 256, 2, 128, 0, 0.1)), UNSUPPORTED),
    (dict(ws=None), WORKSPACE), (dict(ws=ODD8), WORKSPACE),
])
def test_attention_refusals(kw, want):
    assert attend(**kw) == want


def test_workspace_of_refused_shapes_is_zero():
    size = mla.gqa_fp8_workspace_size
    assert size(2, 1, 7, 2, 1) == 0 and size(2, 1, 8, 2, 9) == 0 and size(2, 1, 8, 2, 2, 2) == 0
    assert size(2, 1, 8, 2, 1, head_dim=64) == 0


# ------------------------------------------------------- frequency tables
def test_plain_and_linear_frequencies():
    inv, f = mla.mla_rope_frequencies(64, 500000.0, device="cpu")
    assert inv.dtype == torch.float64 and f == 1.0
    for i in range(32):
        assert abs(float(inv[i]) / 500000.0 ** (-2 * i / 64) - 1) < 1e-14
    lin, f = mla.mla_rope_frequencies(64, 500000.0, dict(type="linear", factor=4.0), device="cpu")
    assert f == 1.0 and torch.equal(lin, inv / 4.0)


def test_ntk_stretches_the_slowest_pair_by_the_factor():
    inv, _ = mla.mla_rope_frequencies(128, device="cpu")
    ntk, f = mla.mla_rope_frequencies(128, scaling=dict(type="ntk", factor=8.0), device="cpu")
    assert f == 1.0 and float(ntk[0]) == 1.0
    assert abs(float(inv[-1] / ntk[-1]) - 8.0) < 1e-12


def test_yarn_keeps_fast_pairs_and_stretches_slow_ones():
    sc = dict(type="yarn", factor=40.0, original_max_position=4096)
    inv, _ = mla.mla_rope_frequencies(64, device="cpu")
    y, f = mla.mla_rope_frequencies(64, scaling=sc, device="cpu")
    assert abs(f - (0.1 * math.log(40.0) + 1)) < 1e-15
    turns = 4096 * inv / (2 * math.pi)
    low, high = math.floor(64 * math.log(4096 / (32 * 2 * math.pi)) / (2 * math.log(1e4))), math.ceil(
        64 * math.log(4096 / (2 * math.pi)) / (2 * math.log(1e4)))
    assert turns[low] > 32 * 0.75 and turns[high] < 1.0
    assert torch.equal(y[:low + 1], inv[:low + 1])
    assert torch.allclose(y[high:], inv[high:] / 40.0, rtol=1e-15)
    mid = (low + high) // 2
    r = (mid - low) / (high - low)
    assert abs(float(y[mid]) - float(inv[mid]) * (r / 40.0 + 1 - r)) < 1e-15
    assert mla.mla_rope_frequencies(64, scaling=dict(sc, attention_factor=1.0), device="cpu")[1] == 1.0


def test_wavelength_scaling():
    sc = dict(type="wavelength", factor=8.0, original_max_position=8192, low_freq_factor=1.0,
              high_freq_factor=4.0)
    inv, _ = mla.mla_rope_frequencies(128, 500000.0, device="cpu")
    y, f = mla.mla_rope_frequencies(128, 500000.0, sc, device="cpu")
    assert f == 1.0
    for a, b in zip(inv.tolist(), y.tolist()):
        wave = 2 * math.pi / a
        if wave < 8192 / 4.0:
            want = a
        elif wave > 8192 / 1.0:
            want = a / 8.0
        else:
            s = (8192 / wave - 1.0) / 3.0
            want = (1 - s) * a / 8.0 + s * a
        assert abs(b - want) <= 1e-15 * a


@pytest.mark.parametrize("kw", [dict(rot_dim=7), dict(rot_dim=0), dict(rot_dim=64, theta=1.0),
                                dict(rot_dim=64, scaling=dict(type="other", factor=2.0)),
                                dict(rot_dim=64, scaling=dict(type="linear", factor=0.5)),
                                dict(rot_dim=2, scaling=dict(type="ntk", factor=2.0)),
                                dict(rot_dim=64, scaling=dict(type="wavelength", factor=2.0,
                                                              original_max_position=100,
                                                              low_freq_factor=2.0,
                                                              high_freq_factor=2.0))])
def test_bad_frequency_arguments(kw):
    with pytest.raises(ValueError):
        mla.mla_rope_frequencies(device="cpu", **kw)


def test_binding_refuses_wrong_tensors():
    """Type and device errors come before any library call."""
    x = torch.zeros(1, 1, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        mla.Rope(torch.zeros(32, dtype=torch.float64))          # not on a device
    with pytest.raises(ValueError):
        mla.mla_rope_apply(x, None, seq_lens=torch.zeros(1, dtype=torch.int32))
    with pytest.raises(TypeError):
        mla.mla_rope_apply(x.float(), None)
    with pytest.raises(ValueError):
        mla.mla_cache_append(torch.zeros(1, 1, 576, dtype=torch.bfloat16), x, x, x)
    with pytest.raises(ValueError):
        mla.gqa_cache_append(x, x, x, x, x, x)
    with pytest.raises(ValueError):
        mla.gqa_decode_partial_fp8(x, x, x, x, x, x, x, 1)
