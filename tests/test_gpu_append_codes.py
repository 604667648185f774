"""Every byte of an e4m3 K/V cache after an append without rotation, where scales
and codes are exact: new tokens, earlier ones of blocks whose scale is kept or
grows, blocks next to them, slots behind the context and pages of nobody."""
import math

import pytest
import torch

from _block_ref import FP8, PAGE, e4m3, pow2_scale, round_e4m3
from test_gpu_append import bf, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mla():
    import sequence_sharded_mla_gb300 as m
    return m


def codes_of(x):
    """Codes of 64-bit values that e4m3 can hold, NaN among them."""
    return x.float().to(FP8).view(torch.uint8)


def expected(cache, scale, x, bt, lens, q_lens, block, N=1, s_id=0):
    """The cache and scales [P, 64 / block, Hkv] that appending x leaves, by the
    rule: one pass over requests, blocks and heads.  Also which rows may change
    at all, and how many blocks with earlier tokens keep their scale or not."""
    cache, scale, written = cache.clone(), scale.clone(), torch.zeros(cache.shape[:3], dtype=torch.bool)
    seen = dict(kept=0, grown=0, new=0)
    for b, (L, n) in enumerate(zip(lens, q_lens)):
        mine = [p for p in range(L - n, L) if p % N == s_id]     # new tokens of this shard
        if not mine:
            continue
        first, end = mine[0] // N, mine[-1] // N + 1             # their slots
        rows = torch.tensor(mine) - (L - n)
        for blk in range(first // block, (end - 1) // block + 1):
            page, row0 = int(bt[b, blk * block // PAGE]), blk * block % PAGE
            for h in range(cache.shape[2]):
                lo, hi = max(first, blk * block), min(end, (blk + 1) * block)
                new = x[b, rows[lo - first:hi - first], h].double()
                fin = torch.where(torch.isfinite(new), new.abs(), torch.zeros_like(new))
                need = pow2_scale(float(fin.max()))
                s = float(scale[page, row0 // block, h])
                had = lo - blk * block
                if had and not abs(s) < need:
                    seen["kept"] += 1
                else:
                    seen["grown" if had else "new"] += 1
                    written[page, row0:row0 + had, h] = True
                    old = cache[page, row0:row0 + had, h]
                    val = round_e4m3(e4m3(old) * (s / need))
                    cache[page, row0:row0 + had, h] = torch.where(
                        torch.isnan(val), torch.full_like(old, 0x7F), codes_of(val))
                    s = need
                val = round_e4m3((new / s).float().double())
                cache[page, row0 + had:row0 + had + hi - lo, h] = torch.where(
                    torch.isnan(val), torch.full_like(val, 0x7F, dtype=torch.uint8), codes_of(val))
                written[page, row0 + had:row0 + had + hi - lo, h] = True
                scale[page, row0 // block, h] = s
    return cache, scale, written, seen


def same_bits(got, want, what):
    """Equal bytes, zeros and NaN of either sign taken as one."""
    g, w = got.cpu(), want
    nan = (g & 0x7F == 0x7F) & (w & 0x7F == 0x7F)
    zero = (g & 0x7F == 0) & (w & 0x7F == 0)
    bad = (g != w) & ~nan & ~zero
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} codes differ, first at {bad.nonzero()[0].tolist()}"


@pytest.mark.parametrize("block", [64, 32, 16, 4, 1])
@pytest.mark.parametrize("Hkv", [1, 3, 8])
@pytest.mark.parametrize("size", [0.02, 1.0, 60.0])
def test_every_byte(mla, block, Hkv, size):
    """Small new values keep the scales, large ones make them grow."""
    g = torch.Generator().manual_seed(210 + block + Hkv)
    lens, q_lens, q_len = [70, 9, 64, 131, 200], [3, 9, 1, 70, 2], 70
    P = 14
    perm = torch.randperm(P, generator=g).to(torch.int32)
    table, off = torch.full((5, 5), -1, dtype=torch.int32), 0
    for b, L in enumerate(lens):
        n = -(-L // PAGE)
        table[b, :n] = perm[off:off + n]
        off += n
    x = {n: bf((5, q_len, Hkv, 128), 220 + i, size) for i, n in enumerate("kv")}
    x["k"][0, 1, 0, 5], x["v"][3, 60, 0, 9] = math.inf, math.nan
    c = {n: torch.randint(0, 256, (P, PAGE, Hkv, 128), generator=g).to(torch.uint8) for n in "kv"}
    sc = {n: torch.exp2(torch.randint(-12, -3, (P, PAGE // block, Hkv), generator=g).float())
          for n in "kv"}
    d = {n: t.clone().cuda() for n, t in c.items()}
    ds = {n: t.clone().cuda() for n, t in sc.items()}
    _, ws = mla.gqa_cache_append(x["k"].cuda(), x["v"].cuda(), d["k"], d["v"], table.cuda(),
                                 i32(lens).cuda(), k_scale=ds["k"], v_scale=ds["v"],
                                 q_lens=i32(q_lens).cuda())
    assert mla.mla_get_device_error(ws) == 0
    for n in "kv":
        want, want_s, written, seen = expected(c[n], sc[n], x[n], table, lens, q_lens, block)
        assert torch.equal(ds[n].cpu(), want_s)
        same_bits(d[n], want, f"{n} {seen}")
        assert torch.equal(d[n].cpu()[~written], c[n][~written])
        if block > 1 and size != 1.0:
            assert seen["kept" if size < 1.0 else "grown"] > 0


@pytest.mark.parametrize("N", [2, 3, 8])
@pytest.mark.parametrize("block", [64, 8])
def test_every_byte_of_a_slice(mla, N, block):
    """A ragged batch into each rank's interleaved slice; some requests bring it
    no token."""
    g = torch.Generator().manual_seed(240 + N + block)
    lens, q_lens, q_len = [70, 2, 64, 131, 900], [3, 1, 1, 70, 5], 70
    P = 5 * 8
    table = torch.randperm(P, generator=g).to(torch.int32).view(5, 8)
    x = {n: bf((5, q_len, 2, 128), 250 + i, 3.0) for i, n in enumerate("kv")}
    c = {n: torch.randint(0, 256, (P, PAGE, 2, 128), generator=g).to(torch.uint8) for n in "kv"}
    sc = {n: torch.exp2(torch.randint(-12, -3, (P, PAGE // block, 2), generator=g).float())
          for n in "kv"}
    for s in range(N):
        d = {n: t.clone().cuda() for n, t in c.items()}
        ds = {n: t.clone().cuda() for n, t in sc.items()}
        _, ws = mla.gqa_cache_append(x["k"].cuda(), x["v"].cuda(), d["k"], d["v"], table.cuda(),
                                     i32(lens).cuda(), k_scale=ds["k"], v_scale=ds["v"],
                                     q_lens=i32(q_lens).cuda(), shard_id=s, num_shards=N)
        assert mla.mla_get_device_error(ws) == 0
        for n in "kv":
            want, want_s, written, _ = expected(c[n], sc[n], x[n], table, lens, q_lens, block, N, s)
            assert torch.equal(ds[n].cpu(), want_s)
            same_bits(d[n], want, f"{n} of shard {s}")
            assert torch.equal(d[n].cpu()[~written], c[n][~written])
