"""A NaN in a cache row, as the cache appends keep it, makes the rows that
attend to it NaN in the latent and the bf16 grouped-query attention: never an
output of zeros, which stands for "no token".  Other requests and KV heads are
not touched."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mla():
    import sequence_sharded_mla_gb300 as m
    return m


def latent(lens, H, fp8, seed, bad):
    """q, cache, scales, table, lengths; request 0 has NaN at token `bad`."""
    g = torch.Generator().manual_seed(seed)
    pages = [-(-n // 64) for n in lens]
    bt = torch.zeros(len(lens), max(pages), dtype=torch.int32)
    off = 0
    for b, n in enumerate(pages):
        bt[b, :n] = torch.arange(off, off + n)
        off += n
    q = torch.randn(len(lens), 1, H, 576, generator=g).bfloat16()
    kv = torch.randn(off, 64, 576, generator=g)
    if fp8:
        kv, sc = (kv * 100).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), torch.full((off, 64), 0.01)
        kv[int(bt[0, bad // 64]), bad % 64, 5] = 0x7F
    else:
        kv, sc = kv.bfloat16(), None
        kv[int(bt[0, bad // 64]), bad % 64, 5] = math.nan
    d = lambda t: None if t is None else t.cuda()
    return d(q), d(kv), d(sc), d(bt), torch.tensor(lens, dtype=torch.int32).cuda()


def nan_then_finite(out, lse):
    assert bool(torch.isnan(out[0]).all()) and bool(torch.isnan(lse[0]).all())
    assert bool(torch.isfinite(out[1:]).all()) and bool(torch.isfinite(lse[1:]).all())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens", [[50, 300], [30000, 64]])
@pytest.mark.parametrize("H", [16, 128])
def test_latent_attention(mla, fp8, lens, H):
    q, kv, sc, bt, sl = latent(lens, H, fp8, 140 + H, bad=lens[0] // 2)
    s = (lens[0] // 2) % 2                      # the shard that holds the NaN
    part, lse, ws = mla.mla_decode_partial(q, kv, bt, sl, 2, kv_scale=sc)
    assert mla.mla_get_device_error(ws) == 0
    nan_then_finite(part[s], lse[s])
    assert bool(torch.isfinite(part[1 - s]).all()) and bool(torch.isfinite(lse[1 - s]).all())
    nan_then_finite(*mla.mla_shard_combine(part, lse))
    w_uv = torch.randn(H, 512, 128, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    nan_then_finite(*mla.mla_shard_combine(part, lse, w_uv=w_uv))
    for N in (1, 2):
        for w in (None, w_uv):
            out, l, ws = mla.mla_decode_step(q, kv, bt, sl, N, kv_scale=sc, w_uv=w)
            assert mla.mla_get_device_error(ws) == 0
            nan_then_finite(out, l)


@pytest.mark.parametrize("lens", [[50, 300], [20000, 64]])
@pytest.mark.parametrize("N", [1, 2])
def test_bf16_grouped_query_attention(mla, lens, N):
    g = torch.Generator().manual_seed(150 + N)
    pages = [-(-n // 64) for n in lens]
    bt = torch.zeros(2, max(pages), dtype=torch.int32)
    bt[0, :pages[0]] = torch.arange(pages[0])
    bt[1, :pages[1]] = torch.arange(pages[1]) + pages[0]
    k = torch.randn(sum(pages), 64, 2, 128, generator=g).bfloat16()
    v = torch.randn(sum(pages), 64, 2, 128, generator=g).bfloat16()
    bad = lens[0] // 2
    k[int(bt[0, bad // 64]), bad % 64, 1, 3] = math.nan
    q = torch.randn(2, 1, 8, 128, generator=g).bfloat16()
    part, lse, ws = mla.gqa_decode_partial(q.cuda(), k.cuda(), v.cuda(), bt.cuda(),
                                           torch.tensor(lens, dtype=torch.int32).cuda(), N)
    assert mla.mla_get_device_error(ws) == 0
    out, lse_out = mla.gqa_shard_combine(part, lse)
    for o, l in ((part[bad % N], lse[bad % N]), (out, lse_out)):
        assert bool(torch.isfinite(o[0, :, :4]).all()) and bool(torch.isfinite(l[0, :, :4]).all())
        assert bool(torch.isnan(o[0, :, 4:]).all()) and bool(torch.isnan(l[0, :, 4:]).all())
        assert bool(torch.isfinite(o[1]).all()) and bool(torch.isfinite(l[1]).all())
