"""GPU parity of rotary positions and of the cache appends against a 64-bit
reference, and runs of them with the attention that reads the caches."""
import math

import numpy as np
import pytest
import torch

import mla_inputs as mi
import oracle
from _block_ref import (FP8, PAGE, attend, check_attention, e4m3, pow2_scale, round_e4m3, turn,
                        turn_error)
from _helpers import REL_OUT, TOL_LSE, TOL_OUT, check_close

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mla():
    import sequence_sharded_mla_gb300 as m
    return m


def bf(shape, seed, sigma=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * sigma).bfloat16()


def rope_of(mla, rot, first=0, interleaved=False, theta=10000.0, scaling=None):
    inv, f = mla.mla_rope_frequencies(rot, theta, scaling)
    return mla.Rope(inv, first, interleaved, f)


def i32(x):
    return torch.tensor(x, dtype=torch.int32)


def positions_of(lens, q_lens, q_len, b, i):
    n = q_len if q_lens is None else int(q_lens[b])
    return int(lens[b]) - n + i, i < n


def check_rotated(got, x, rope, pos, real, before):
    """Rows [B, q_len, H, D] against turn(): bf16 rounds by 2^-8 of the value
    on top of turn_error."""
    inv = rope.inv_freq.cpu()
    for b in range(x.shape[0]):
        for i in range(x.shape[1]):
            if not real(b, i):
                assert torch.equal(got[b, i], before[b, i])
                continue
            v = x[b, i].double()
            y = turn(v, pos(b, i), inv, rope.first_dim, rope.interleaved, rope.attention_factor)
            e = turn_error(v, rope.first_dim, inv.numel(), rope.interleaved, rope.attention_factor)
            tol = y.abs() * 2.0 ** -8 * (e > 0) + e
            assert bool(((got[b, i].double() - y).abs() <= tol).all())


YARN = dict(type="yarn", factor=40.0, original_max_position=4096)


@pytest.mark.parametrize("D,rot,first", [(576, 64, 512), (128, 128, 0), (128, 32, 0), (128, 96, 16),
                                         (64, 16, 8), (1024, 1024, 0)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("inplace", [False, True])
def test_rotation(mla, D, rot, first, interleaved, inplace):
    lens, q_lens, q_len, H = [131072, 2, 70], [3, 2, 1], 3, 5
    rope = rope_of(mla, rot, first, interleaved, scaling=YARN)
    x = bf((3, q_len, H, D), D + rot)
    dx = x.cuda()
    out = dx if inplace else torch.full_like(dx, 7.0)
    before = out.cpu().clone()
    got = mla.mla_rope_apply(dx, rope, i32(lens).cuda(), i32(q_lens).cuda(), out=out)
    assert got is out
    check_rotated(got.cpu(), x, rope, lambda b, i: lens[b] - q_lens[b] + i,
                  lambda b, i: i < q_lens[b], before)


@pytest.mark.parametrize("positions", [[0], [1], [-5], [2 ** 31 - 1], [-2 ** 31], [1048575]])
def test_far_and_given_positions(mla, positions):
    rope = rope_of(mla, 64)
    x = bf((1, 1, 2, 128), 5)
    got = mla.mla_rope_apply(x.cuda(), rope, positions=i32([positions]).cuda())
    # the 64-bit reference's own angle is off by 2^-53 of itself: 2^-22 rad at 2^31
    v = x[0, 0].double()
    y = turn(v, positions[0], rope.inv_freq.cpu(), 0, False, 1.0)
    e = turn_error(v, 0, 32, False, 1.0) * 2
    assert bool(((got[0, 0].cpu().double() - y).abs() <= y.abs() * 2.0 ** -8 + e).all())


def test_rotating_back_returns_the_input(mla):
    rope = rope_of(mla, 128, 0, True)
    x = bf((2, 4, 3, 128), 6).cuda()
    pos = i32([[5, 1000, 77777, 3], [9, 8, 1, 0]]).cuda()
    y = mla.mla_rope_apply(x, rope, positions=pos)
    back = mla.mla_rope_apply(y, rope, positions=-pos)
    # two roundings to bf16, each 2^-8 of a value of at most |x_a| + |x_b|
    big = x.float().abs().view(2, 4, 3, 64, 2).sum(-1, keepdim=True).expand(-1, -1, -1, -1, 2)
    assert bool(((back.float() - x.float()).abs() <= big.reshape(x.shape) * 2.0 ** -6).all())


def test_rotation_of_a_slice_of_a_fused_projection(mla):
    rope = rope_of(mla, 64, 0, True)
    fused = bf((2, 5, 12 * 128 + 8), 7).cuda()
    keep = fused.cpu().clone()
    x = fused[..., 256:256 + 4 * 128].unflatten(-1, (4, 128))
    lens = i32([5, 900]).cuda()
    want = mla.mla_rope_apply(x.contiguous(), rope, lens)
    assert torch.equal(mla.mla_rope_apply(x, rope, lens), want)
    mla.mla_rope_apply(x, rope, lens, out=x)
    assert torch.equal(x, want)
    rest = fused.cpu()
    rest[..., 256:256 + 512] = keep[..., 256:256 + 512]
    assert torch.equal(rest, keep)


# ------------------------------------------------------------- GQA append
def pool(P, Hkv, block, fp8, seed):
    g = torch.Generator().manual_seed(seed)
    c = {}
    for n in "kv":
        if fp8:
            c[n] = (torch.randn(P, PAGE, Hkv, 128, generator=g) * 110).clamp(-448, 448).to(FP8).view(torch.uint8)
            c[n + "s"] = torch.exp2(torch.randint(-9, -6, (P, PAGE // block, Hkv), generator=g).float())
        else:
            c[n] = (torch.randn(P, PAGE, Hkv, 128, generator=g)).bfloat16()
    return c


def table(lens, N=1, seed=0, spare=2):
    n = [-(-(-(-L // N)) // PAGE) + 1 for L in lens]
    P = sum(n) + spare
    perm = torch.randperm(P, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    bt = torch.full((len(lens), max(n)), -1, dtype=torch.int32)
    off = 0
    for b, k in enumerate(n):
        bt[b, :k] = perm[off:off + k]
        off += k
    return P, bt


def expect_gqa(c, k, v, bt, lens, q_lens, rope, block, fp8, shard=0, N=1, positions=None):
    """The caches after the append in 64 bits (values under the scales for
    e4m3), and the error bound of each value; scales as (low, high)."""
    B, q_len, Hkv, _ = k.shape
    out = {}
    for n, x in (("k", k), ("v", v)):
        val = e4m3(c[n]) if fp8 else c[n].double()
        tol = torch.zeros_like(val)
        sc = c[n + "s"].double().clone() if fp8 else None
        band = (sc.clone(), sc.clone()) if fp8 else None
        for b in range(B):
            rows = {}
            for i in range(q_len):
                p, real = positions_of(lens, q_lens, q_len, b, i)
                if not real or p < 0 or p % N != shard:
                    continue
                y, e = x[b, i].double(), torch.zeros(Hkv, 128, dtype=torch.float64)
                if n == "k" and rope is not None:
                    at = p if positions is None else int(positions[b, i])
                    e = turn_error(y, rope.first_dim, rope.inv_freq.numel(), rope.interleaved,
                                   rope.attention_factor)
                    y = turn(y, at, rope.inv_freq.cpu(), rope.first_dim, rope.interleaved,
                             rope.attention_factor)
                rows[p // N] = (y, e)
            if not fp8:
                for p, (y, e) in rows.items():
                    pg = int(bt[b, p // PAGE])
                    val[pg, p % PAGE] = y
                    tol[pg, p % PAGE] = y.abs() * 2.0 ** -8 + e
                continue
            if not rows:
                continue
            first = min(rows)
            for blk in sorted({p // block for p in rows}):
                pg, sub = int(bt[b, blk * block // PAGE]), (blk * block % PAGE) // block
                here = [p for p in sorted(rows) if p // block == blk]
                had = here[0] > blk * block
                for h in range(Hkv):
                    fin = lambda t: torch.where(torch.isfinite(t), t.abs(), torch.zeros_like(t))
                    a = max(float(fin(rows[p][0][h]).max()) for p in here)
                    slack = max(float(fin(rows[p][1][h]).max()) for p in here)
                    was = float(sc[pg, sub, h])
                    pick = lambda need: was if had and abs(was) >= need else need
                    lo, hi = pick(pow2_scale(max(a - slack, 0.0))), pick(pow2_scale(a + slack))
                    band[0][pg, sub, h], band[1][pg, sub, h] = lo, hi
                    s = hi
                    for p in range(blk * block, here[0]):
                        old = val[pg, p % PAGE, h] * was
                        val[pg, p % PAGE, h] = old
                        # unchanged, or rounded again to a scale that grew; half the smallest
                        # step is 2^-10 of the scale's magnitude
                        if s != was:
                            tol[pg, p % PAGE, h] = torch.maximum(old.abs() * 2.0 ** -4,
                                                                 torch.tensor(2.0 ** -10 * abs(s)))
                            exact = round_e4m3(old / s) * s == old
                            tol[pg, p % PAGE, h][exact] = 0
                    for p in here:
                        y, e = rows[p]
                        val[pg, p % PAGE, h] = torch.where(torch.isfinite(y[h]), y[h],
                                                           torch.full_like(y[h], math.nan))
                        tol[pg, p % PAGE, h] = torch.maximum(y[h].abs() * 2.0 ** -4,
                                                             torch.tensor(2.0 ** -10 * abs(s))) + e[h]
                    done = set(range(blk * block, here[-1] + 1))
                    for p in range(blk * block, (blk + 1) * block):
                        if p not in done:     # behind the context: codes as they were
                            val[pg, p % PAGE, h] = val[pg, p % PAGE, h] * math.nan
                            tol[pg, p % PAGE, h] = -1
        out[n] = (val, tol, band)
    return out


def check_gqa(got, before, want, block, fp8):
    for n in "kv":
        val, tol, band = want[n]
        if not fp8:
            same = tol == 0
            assert torch.equal(got[n][same], before[n][same])
            assert bool(((got[n].double() - val).abs() <= tol).all())
            continue
        sc = got[n + "s"].double()
        assert bool(((sc == band[0]) | (sc == band[1])).all())
        behind = tol < 0
        assert torch.equal(got[n][behind], before[n][behind])
        full = sc.repeat_interleave(block, 1)[..., None]
        g = e4m3(got[n])
        touched = tol > 0
        x, y = (g * full)[touched], val[touched]
        assert torch.equal(torch.isnan(x), torch.isnan(y))
        ok = torch.isnan(y) | ((x - y).abs() <= tol[touched] * (1 + 2.0 ** -20))
        assert bool(ok.all())


def run_gqa(mla, c, k, v, bt, lens, q_lens, rope, fp8, q=None, status=0, **kw):
    d = {n: t.clone().cuda() for n, t in c.items()}
    ql = None if q_lens is None else i32(q_lens).cuda()
    q_out, ws = mla.gqa_cache_append(k.cuda(), v.cuda(), d["k"].view(FP8) if fp8 else d["k"],
                                     d["v"].view(FP8) if fp8 else d["v"], bt.cuda(),
                                     i32(lens).cuda(), rope=rope, q=None if q is None else q.cuda(),
                                     k_scale=d.get("ks"), v_scale=d.get("vs"), q_lens=ql, **kw)
    assert mla.mla_get_device_error(ws) == status
    return {n: t.cpu() for n, t in d.items()}, None if q_out is None else q_out.cpu()


@pytest.mark.parametrize("fp8,block", [(False, 64), (True, 64), (True, 32), (True, 16), (True, 1)])
@pytest.mark.parametrize("q_len,rot,interleaved", [(1, 128, False), (9, 64, True), (75, 96, False)])
def test_gqa_append(mla, fp8, block, q_len, rot, interleaved):
    lens = [q_len, 64 + q_len, 63, 300, 129]
    lens = [max(x, q_len) for x in lens]
    q_lens = [q_len, max(1, q_len // 2), 1, q_len, max(1, q_len - 3)]
    Hkv, H = 3, 6
    P, bt = table(lens, seed=q_len)
    c = pool(P, Hkv, block, fp8, 11)
    k, v, q = bf((5, q_len, Hkv, 128), 12), bf((5, q_len, Hkv, 128), 13, 3.0), bf((5, q_len, H, 128), 14)
    rope = rope_of(mla, rot, 0, interleaved, scaling=YARN)
    got, q_out = run_gqa(mla, c, k, v, bt, lens, q_lens, rope, fp8, q=q,
                         q_out=torch.zeros(q.shape, dtype=torch.bfloat16, device="cuda"))
    check_gqa(got, c, expect_gqa(c, k, v, bt, lens, q_lens, rope, block, fp8), block, fp8)
    check_rotated(q_out, q, rope, lambda b, i: lens[b] - q_lens[b] + i, lambda b, i: i < q_lens[b],
                  torch.zeros_like(q))


def test_untouched_blocks_keep_their_bits(mla):
    lens = [70, 200]
    P, bt = table(lens, seed=1)
    c = pool(P, 2, 16, True, 15)
    k, v = bf((2, 2, 2, 128), 16), bf((2, 2, 2, 128), 17)
    got, _ = run_gqa(mla, c, k, v, bt, lens, None, rope_of(mla, 128), True)
    hit = {(int(bt[b, p // 64]), (p % 64) // 16) for b in range(2) for p in range(lens[b] - 2, lens[b])}
    for pg in range(P):
        for sub in range(4):
            if (pg, sub) not in hit:
                for n in "kv":
                    assert torch.equal(got[n][pg, 16 * sub:16 * sub + 16], c[n][pg, 16 * sub:16 * sub + 16])
                    assert torch.equal(got[n + "s"][pg, sub], c[n + "s"][pg, sub])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("N", [2, 3, 8])
def test_gqa_append_to_interleaved_slices(mla, fp8, N):
    lens, q_lens, q_len = [3, 100, 517], [3, 5, 7], 7
    rope = rope_of(mla, 64, 0, True)
    k, v = bf((3, q_len, 2, 128), 18), bf((3, q_len, 2, 128), 19)
    for s in range(N):
        P, bt = table(lens, N, seed=s)
        c = pool(P, 2, 16, fp8, 20 + s)
        got, _ = run_gqa(mla, c, k, v, bt, lens, q_lens, rope, fp8, shard_id=s, num_shards=N)
        check_gqa(got, c, expect_gqa(c, k, v, bt, lens, q_lens, rope, 16, fp8, s, N), 16, fp8)


def test_given_positions_turn_keys_and_queries(mla):
    lens, q_len = [50, 9], 4
    P, bt = table(lens)
    c = pool(P, 2, 32, True, 21)
    k, v, q = bf((2, q_len, 2, 128), 22), bf((2, q_len, 2, 128), 23), bf((2, q_len, 4, 128), 24)
    pos = i32([[46, 47, 47, 48], [5, 6, 6, 6]])
    rope = rope_of(mla, 128)
    got, q_out = run_gqa(mla, c, k, v, bt, lens, None, rope, True, q=q, positions=pos.cuda())
    check_gqa(got, c, expect_gqa(c, k, v, bt, lens, None, rope, 32, True, positions=pos), 32, True)
    check_rotated(q_out, q, rope, lambda b, i: int(pos[b, i]), lambda b, i: True, q)


def test_scales_grow_and_earlier_tokens_keep_their_values(mla):
    """Tokens of growing size one at a time into one block: with power-of-two
    scales an earlier token's value moves only once it is subnormal."""
    P, bt = table([40])
    c = pool(P, 1, 64, True, 25)
    rope = None
    truth = []
    for t in range(40):
        x = bf((1, 1, 1, 128), 100 + t, 2.0 ** (t / 4.0))
        before = {n: y.clone() for n, y in c.items()}
        c, _ = run_gqa(mla, c, x, x, bt, [t + 1], None, rope, True)
        check_gqa(c, before, expect_gqa(before, x, x, bt, [t + 1], None, rope, 64, True), 64, True)
        truth.append(x[0, 0, 0].double())
        pg = int(bt[0, 0])
        s = float(c["ks"][pg, 0, 0])
        assert s == pow2_scale(max(float(y.abs().max()) for y in truth))
        val = e4m3(c["k"][pg, :t + 1, 0]) * s
        want = torch.stack(truth)
        # one rounding of 2^-4, or half the smallest step of each scale since
        assert bool(((val - want).abs() <= torch.maximum(want.abs() * 2.0 ** -4, torch.tensor(2.0 ** -9 * s))).all())


def test_foreign_scales_are_kept_while_they_are_wide_enough(mla):
    """A block quantised to max / 448, or under a negative scale."""
    P, bt = table([10, 10])
    c = pool(P, 1, 64, True, 26)
    pa, pb = int(bt[0, 0]), int(bt[1, 0])
    for n in "kv":
        c[n + "s"][pa] = 0.0123
        c[n + "s"][pb] = -0.5
    k, v = bf((2, 1, 1, 128), 27, 0.5), bf((2, 1, 1, 128), 28, 20.0)
    got, _ = run_gqa(mla, c, k, v, bt, [10, 10], None, None, True)
    check_gqa(got, c, expect_gqa(c, k, v, bt, [10, 10], None, None, 64, True), 64, True)


def test_nonfinite_values_are_stored_as_nan(mla):
    P, bt = table([5])
    c = pool(P, 1, 64, True, 29)
    x = bf((1, 1, 1, 128), 30)
    x[..., 3], x[..., 4], x[..., 5] = math.inf, -math.inf, math.nan
    got, _ = run_gqa(mla, c, x, x, bt, [5], None, None, True)
    check_gqa(got, c, expect_gqa(c, x, x, bt, [5], None, None, 64, True), 64, True)
    zero = torch.zeros_like(x)
    got, _ = run_gqa(mla, c, zero, zero, bt, [1], None, None, True)
    pg = int(bt[0, 0])
    assert float(got["ks"][pg, 0, 0]) == 2.0 ** -60 and int(got["k"][pg, 0].max()) == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_bad_pages_and_lengths_write_nothing_there(mla, fp8):
    lens = [10, 70, 2]
    P, bt = table(lens)
    c = pool(P, 2, 64, fp8, 31)
    k = bf((3, 1, 2, 128), 32)
    bad = bt.clone()
    bad[1, 1] = P
    got, _ = run_gqa(mla, c, k, k, bad, lens, None, None, fp8, status=-5)
    for n in "kv":
        changed = (got[n] != c[n]).flatten(1).any(1).nonzero().flatten().tolist()
        assert set(changed) <= {int(bt[0, 0]), int(bt[2, 0])}
    # more new tokens than the context has: the ones before its start are dropped
    k3 = bf((3, 4, 2, 128), 33)
    got, _ = run_gqa(mla, c, k3, k3, bt, lens, None, None, fp8, status=-1)
    pg = int(bt[2, 0])
    assert torch.equal(got["k"][pg, 2:], c["k"][pg, 2:])
    assert not torch.equal(got["k"][pg, :2], c["k"][pg, :2])


def test_append_of_slices_of_a_fused_projection(mla):
    B, q_len, H, Hkv = 2, 3, 4, 2
    fused = bf((B, q_len, (H + 2 * Hkv) * 128), 34).cuda()
    q, k, v = fused.split([H * 128, Hkv * 128, Hkv * 128], -1)
    q, k, v = (t.unflatten(-1, (-1, 128)) for t in (q, k, v))
    lens = [30, 90]
    P, bt = table(lens)
    c = pool(P, Hkv, 64, True, 35)
    rope = rope_of(mla, 128)
    got, q_out = run_gqa(mla, c, k.cpu(), v.cpu(), bt, lens, None, rope, True, q=q.cpu())
    d = {n: t.clone().cuda() for n, t in c.items()}
    qo, ws = mla.gqa_cache_append(k, v, d["k"], d["v"], bt.cuda(), i32(lens).cuda(), rope, q=q, q_out=q,
                                  k_scale=d["ks"], v_scale=d["vs"])
    assert mla.mla_get_device_error(ws) == 0
    assert all(torch.equal(d[n].cpu(), got[n]) for n in d)
    assert torch.equal(q.cpu(), q_out)


# -------------------------------------------------------------- MLA append
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("q_len,N,interleaved", [(1, 1, True), (5, 1, False), (70, 3, True)])
def test_latent_append(mla, fp8, q_len, N, interleaved):
    lens, q_lens, H = [q_len, 200, 65 + q_len], [q_len, max(1, q_len - 2), 1], 3
    rope = rope_of(mla, 64, 512, interleaved)
    x, q = bf((3, q_len, 576), 40), bf((3, q_len, H, 576), 41)
    for s in range(N):
        P, bt = table(lens, N, seed=s)
        if fp8:
            kv = torch.randint(0, 120, (P, PAGE, 576), dtype=torch.uint8)
            sc = torch.rand(P, PAGE)
        else:
            kv, sc = bf((P, PAGE, 576), 42), None
        d, ds = kv.clone().cuda(), None if sc is None else sc.clone().cuda()
        dq = q.cuda()
        q_out, ws = mla.mla_cache_append(x.cuda(), d.view(FP8) if fp8 else d, bt.cuda(),
                                         i32(lens).cuda(), rope, q=dq, q_out=dq, kv_scale=ds,
                                         q_lens=i32(q_lens).cuda(), shard_id=s, num_shards=N)
        assert mla.mla_get_device_error(ws) == 0
        check_rotated(q_out.cpu(), q, rope, lambda b, i: lens[b] - q_lens[b] + i,
                      lambda b, i: i < q_lens[b], q)
        want, wsc = kv.clone(), None if sc is None else sc.clone()
        got, gsc = d.cpu(), None if ds is None else ds.cpu()
        for b in range(3):
            for i in range(q_lens[b]):
                p = lens[b] - q_lens[b] + i
                if p % N != s:
                    continue
                pg, r = int(bt[b, p // N // PAGE]), p // N % PAGE
                v = x[b, i].double()
                y = turn(v, p, rope.inv_freq.cpu(), 512, interleaved, 1.0)
                e = turn_error(v, 512, 32, interleaved, 1.0)
                if fp8:
                    a, slack = float(y.abs().max()), float(e.max())
                    g = float(gsc[pg, r])
                    assert g in (pow2_scale(a - slack), pow2_scale(a + slack))
                    tol = torch.maximum(y.abs() * 2.0 ** -4, torch.tensor(2.0 ** -10 * g)) + e
                    assert bool(((e4m3(got[pg, r]) * g - y).abs() <= tol).all())
                    wsc[pg, r] = gsc[pg, r]
                else:
                    assert bool(((got[pg, r].double() - y).abs() <= y.abs() * 2.0 ** -8 * (e > 0) + e).all())
                want[pg, r] = got[pg, r]
        assert torch.equal(got, want)
        assert sc is None or torch.equal(gsc, wsc)


# ---------------------------------------------------------------- together
def test_decode_steps_of_a_gqa_layer(mla):
    """A prompt chunk, then single tokens and a verify step, appended and
    attended to; the attention against the reference over the cache as the
    appends left it, the cache against the true keys and values."""
    H, Hkv, block, B = 8, 2, 16, 2
    steps = [(100, [100, 37]), (1, [1, 1]), (1, [1, 1]), (5, [5, 2]), (1, [1, 1])]
    P, bt = table([200, 200])
    d = {n: t.cuda() for n, t in pool(P, Hkv, block, True, 50).items()}
    rope = rope_of(mla, 64, 0, True)
    lens, keys = [0, 0], [[], []]
    ws_a = torch.zeros(256, dtype=torch.uint8, device="cuda")
    for st, (q_len, q_lens) in enumerate(steps):
        lens = [a + n for a, n in zip(lens, q_lens)]
        k, v = bf((B, q_len, Hkv, 128), 60 + st), bf((B, q_len, Hkv, 128), 70 + st)
        q = bf((B, q_len, H, 128), 80 + st).cuda()
        L, n = i32(lens).cuda(), i32(q_lens).cuda()
        mla.gqa_cache_append(k.cuda(), v.cuda(), d["k"], d["v"], bt.cuda(), L, rope, q=q, q_out=q,
                             k_scale=d["ks"], v_scale=d["vs"], q_lens=n, workspace=ws_a)
        part, lse, ws = mla.gqa_decode_partial_fp8(q, d["k"], d["v"], d["ks"], d["vs"], bt.cuda(), L,
                                                   2, causal=True, q_lens=n)
        out, lse_out = mla.gqa_shard_combine(part, lse)
        assert mla.mla_get_device_error(ws) == 0
        c = {m: t.cpu() for m, t in d.items()}
        check_attention(out, lse_out, attend(q.cpu(), c["k"], c["v"], c["ks"], c["vs"], bt, lens,
                                             q_lens, True, 128 ** -0.5, 1, -1, "interleaved"),
                        out_rel=2.0 ** -8)
        for b in range(B):
            for i in range(q_lens[b]):
                keys[b].append(turn(k[b, i].double(), len(keys[b]), rope.inv_freq.cpu(), 0, True, 1.0))
    assert mla.mla_get_device_error(ws_a) == 0
    for b in range(B):
        want = torch.stack(keys[b])
        p = torch.arange(lens[b])
        pg = bt[b].long()[p // PAGE]
        s = c["ks"].double()[pg, p % PAGE // block][..., None]
        got = e4m3(c["k"])[pg, p % PAGE] * s
        assert bool(((got - want).abs() <= torch.maximum(want.abs() * 2.0 ** -4, 2.0 ** -9 * s) + 1e-5).all())


@pytest.mark.parametrize("kv_dtype", ["bf16", "fp8"])
def test_decode_step_over_an_appended_latent_cache(mla, kv_dtype):
    """Latent rows appended in two chunks without rotation, then the decode
    step: the oracle over the same cache."""
    lens = [130, 64, 7]
    w = mi.build_workload("append", 3, 1, 16, lens, 2, "interleaved", "bf16", False, seed=51, poison=True)
    src = torch.from_numpy(w.kv.view(np.int16)).view(torch.bfloat16)
    rows = torch.zeros(3, max(lens), 576, dtype=torch.bfloat16)
    for b, L in enumerate(lens):
        for p in range(L):
            rows[b, p] = src[int(w.block_table[b, p // PAGE]), p % PAGE]
    bt = torch.from_numpy(w.block_table).cuda()
    if kv_dtype == "fp8":
        kv = torch.full(src.shape, 0x7F, dtype=torch.uint8, device="cuda")
        sc = torch.full(src.shape[:2], math.nan, device="cuda")
    else:
        kv, sc = torch.full(src.shape, math.nan, dtype=torch.bfloat16, device="cuda"), None
    half = [L // 2 for L in lens]
    for done, upto in ((None, half), (half, lens)):
        n = [u - (0 if done is None else done[b]) for b, u in enumerate(upto)]
        ql = max(n)
        x = torch.zeros(3, ql, 576, dtype=torch.bfloat16)
        for b in range(3):
            x[b, :n[b]] = rows[b, upto[b] - n[b]:upto[b]]
        _, ws = mla.mla_cache_append(x.cuda(), kv, bt, i32(upto).cuda(), kv_scale=sc, q_lens=i32(n).cuda())
        assert mla.mla_get_device_error(ws) == 0
    if kv_dtype == "bf16":
        for b, L in enumerate(lens):
            for p in range(L):
                assert torch.equal(kv[int(w.block_table[b, p // PAGE]), p % PAGE].cpu(), rows[b, p])
    else:
        w.kv, w.kv_scale, w.kv_dtype = kv.cpu().numpy(), sc.cpu().numpy(), "fp8"
    q = torch.from_numpy(w.q.view(np.int16)).view(torch.bfloat16).cuda()
    out, lse, ws = mla.mla_decode_step(q, kv, bt, i32(lens).cuda(), 2, kv_scale=sc)
    assert mla.mla_get_device_error(ws) == 0
    o, l = oracle.attend(w, shard=-1)
    check_close(out.float().cpu().numpy().reshape(o.shape), o, TOL_OUT, "out", rel=REL_OUT)
    check_close(lse.cpu().numpy().ravel(), l, TOL_LSE, "lse")


def test_append_and_attention_in_one_graph(mla):
    """Two captured steps over one cache and one workspace each, replayed in
    order, equal the same calls made eagerly."""
    H, Hkv, B, block = 8, 2, 2, 32
    P, bt = table([100, 100])
    start = {n: t.cuda() for n, t in pool(P, Hkv, block, True, 52).items()}
    dbt = bt.cuda()
    lens = i32([50, 33]).cuda()
    k, v, q = bf((B, 1, Hkv, 128), 53).cuda(), bf((B, 1, Hkv, 128), 54).cuda(), bf((B, 1, H, 128), 55).cuda()
    rope = rope_of(mla, 128)
    need = mla.gqa_fp8_workspace_size(B, 1, H, Hkv, 1)

    def step(d, ws, wa):
        qr, _ = mla.gqa_cache_append(k, v, d["k"], d["v"], dbt, lens, rope, q=q, k_scale=d["ks"],
                                     v_scale=d["vs"], workspace=wa)
        part, lse, _ = mla.gqa_decode_partial_fp8(qr, d["k"], d["v"], d["ks"], d["vs"], dbt, lens, 1,
                                                  workspace=ws)
        return mla.gqa_shard_combine(part, lse)

    new = lambda n: torch.zeros(n, dtype=torch.uint8, device="cuda")
    eager, d = [], {n: t.clone() for n, t in start.items()}
    for t in range(4):
        lens.copy_(i32([50 + t, 33 + t]))
        k.copy_(bf((B, 1, Hkv, 128), 90 + t))
        eager.append([x.clone() for x in step(d, new(need), new(256))])
    dg = {n: t.clone() for n, t in start.items()}
    graphs = []
    torch.cuda.synchronize()
    for _ in range(2):
        ws, wa = new(need), new(256)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step(dg, ws, wa)
        graphs.append((g, out, ws, wa))
    for n in dg:
        dg[n].copy_(start[n])
    for t in range(4):
        lens.copy_(i32([50 + t, 33 + t]))
        k.copy_(bf((B, 1, Hkv, 128), 90 + t))
        g, out, ws, wa = graphs[t % 2]
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], eager[t][0]) and torch.equal(out[1], eager[t][1])
    assert all(torch.equal(dg[n], d[n]) for n in d)


@pytest.mark.parametrize("positions", [[3], [-70000], [1000003]])
def test_frequencies_of_every_size(mla, positions):
    """Zero, negative, above a turn per token, far below any angle."""
    w = torch.tensor([0.0, -0.3, 100.0, 2 * math.pi, 1e-300, 1e-12, 7.0, 0.5], dtype=torch.float64)
    rope = mla.Rope(w.cuda(), 8, True, 1.25)
    x = bf((1, 1, 3, 32), 50)
    got = mla.mla_rope_apply(x.cuda(), rope, positions=i32([positions]).cuda())
    v = x[0, 0].double()
    y = turn(v, positions[0], w, 8, True, 1.25)
    # the 64-bit reference's own angle is off by 2^-53 of up to 2^26.6 rad
    e = turn_error(v, 8, 8, True, 1.25) * (1 + 2.0 ** -4)
    assert bool(((got[0, 0].cpu().double() - y).abs() <= y.abs() * 2.0 ** -8 * (e > 0) + e).all())


@pytest.mark.parametrize("Hkv,block", [(1, 64), (5, 32), (9, 16), (9, 2), (3, 8), (2, 4)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_gqa_append_of_part_of_the_head(mla, Hkv, block, interleaved):
    """Heads that do not fill a block's warps, dims 16..111 turned, appends
    that end, start and stay inside blocks of scales."""
    lens, q_lens, q_len = [130, 67, 40, 64, 65], [130, 3, 40, 1, 33], 130
    P, bt = table(lens, seed=Hkv)
    c = pool(P, Hkv, block, True, 51)
    k, v = bf((5, q_len, Hkv, 128), 52), bf((5, q_len, Hkv, 128), 53, 0.01)
    rope = rope_of(mla, 96, 16, interleaved)
    got, _ = run_gqa(mla, c, k, v, bt, lens, q_lens, rope, True)
    check_gqa(got, c, expect_gqa(c, k, v, bt, lens, q_lens, rope, block, True), block, True)


def test_infinities_beside_wide_foreign_scales(mla):
    """An infinity among values under a scale that is kept, and in another
    head's tokens only."""
    P, bt = table([70])
    c = pool(P, 2, 64, True, 54)
    pg = int(bt[0, 1])
    for n in "kv":
        c[n + "s"][pg] = 1000.0
    x = bf((1, 3, 2, 128), 55)
    x[0, 1, 0, 7], x[0, 2, 0, 100], x[0, 0, 0, 8] = math.inf, -math.inf, math.nan
    got, _ = run_gqa(mla, c, x, x, bt, [69], None, None, True)
    check_gqa(got, c, expect_gqa(c, x, x, bt, [69], None, None, 64, True), 64, True)


def test_appends_on_a_given_stream(mla):
    """The workspace and q_out that a call allocates belong to its stream."""
    lens = [30, 90]
    P, bt = table(lens)
    c = pool(P, 2, 32, True, 56)
    k, q = bf((2, 3, 2, 128), 57), bf((2, 3, 4, 128), 58)
    rope = rope_of(mla, 128)
    want, q_want = run_gqa(mla, c, k, k, bt, lens, None, rope, True, q=q)
    d = {n: t.clone().cuda() for n, t in c.items()}
    dk, dq, dbt, dl = k.cuda(), q.cuda(), bt.cuda(), i32(lens).cuda()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    q_out, ws = mla.gqa_cache_append(dk, dk, d["k"], d["v"], dbt, dl, rope, q=dq, k_scale=d["ks"],
                                     v_scale=d["vs"], stream=side)
    q_two = mla.mla_rope_apply(dq, rope, dl, stream=side)
    side.synchronize()
    assert mla.mla_get_device_error(ws) == 0
    assert all(torch.equal(d[n].cpu(), want[n]) for n in d)
    assert torch.equal(q_out.cpu(), q_want) and torch.equal(q_two.cpu(), q_want)


def test_append_binding_refusals(mla):
    P, bt = table([30, 90])
    c = {n: t.cuda() for n, t in pool(P, 2, 32, True, 59).items()}
    k, q = bf((2, 3, 2, 128), 60).cuda(), bf((2, 3, 4, 128), 61).cuda()
    bt, lens, rope = bt.cuda(), i32([30, 90]).cuda(), rope_of(mla, 128)

    def heads(**kw):
        a = dict(k=k, v=k, k_cache=c["k"], v_cache=c["v"], block_table=bt, seq_lens=lens, rope=rope,
                 q=q, k_scale=c["ks"], v_scale=c["vs"])
        return mla.gqa_cache_append(**{**a, **kw})

    for kw in (dict(k=k[..., :64]), dict(v=k[:1]), dict(k=k.float()), dict(k=k.transpose(1, 2)),
               dict(q=q[:, :1]), dict(q=q[..., :64]), dict(q=None, q_out=q), dict(q_out=q[:, :, :2]),
               dict(q_out=q.flatten()[128:].expand(2, 3, 4, -1)), dict(block_table=bt[:1]),
               dict(seq_lens=None), dict(seq_lens=lens.long()), dict(k_scale=None),
               dict(k_scale=c["ks"][:, :1]), dict(v_cache=c["v"][:1]),
               dict(positions=i32([[1, 2, 3]]).cuda()), dict(workspace=torch.zeros(300, device="cuda"))):
        with pytest.raises((TypeError, ValueError)):
            heads(**kw)
    wide = torch.zeros(2, 3, 5, 128, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):            # shifted by one head
        mla.mla_rope_apply(wide[:, :, :4], rope, lens, out=wide[:, :, 1:])
    with pytest.raises(ValueError):
        mla.mla_rope_apply(q, rope)
    with pytest.raises(TypeError):
        mla.mla_rope_apply(q, None, lens)
    with pytest.raises(mla.MLAError):
        heads(rope=None)                       # a query without a rotation
    with pytest.raises(mla.MLAError):
        heads(shard_id=2, num_shards=2)
    with pytest.raises(ValueError):
        mla.Rope(rope.inv_freq[::2])
    with pytest.raises(TypeError):
        mla.Rope(rope.inv_freq.float())


def test_a_graph_with_copies_and_fills_between_the_calls(mla):
    """Launches that may begin early, behind a copy and behind the clearing of
    the workspace that the call allocates."""
    lens, H, Hkv = [30, 90], 4, 2
    P, bt = table([x + 8 for x in lens])
    c = pool(P, Hkv, 32, True, 62)
    steps = [(bf((2, 1, Hkv, 128), 63 + i), bf((2, 1, H, 128), 73 + i)) for i in range(3)]
    rope = rope_of(mla, 128)
    dbt, dl = bt.cuda(), i32(lens).cuda()
    d = {n: t.clone().cuda() for n, t in c.items()}
    k, q, src_k, src_q = (t.clone().cuda() for t in (*steps[0], *steps[0]))

    def step():
        k.copy_(src_k)
        q.copy_(src_q)
        dl.add_(1)
        q_out, ws = mla.gqa_cache_append(k, k, d["k"], d["v"], dbt, dl, rope, q=q, k_scale=d["ks"],
                                         v_scale=d["vs"])
        part, lse, ws2 = mla.gqa_decode_partial_fp8(q_out, d["k"], d["v"], d["ks"], d["vs"], dbt, dl, 2)
        return mla.gqa_shard_combine(part, lse), ws, ws2

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        (out, lse_out), ws, ws2 = step()
    for n, t in c.items():
        d[n].copy_(t)
    dl.copy_(i32(lens))
    for i, (dk, dq) in enumerate(steps):
        src_k.copy_(dk)
        src_q.copy_(dq)
        g.replay()
        torch.cuda.synchronize()
        assert mla.mla_get_device_error(ws) == 0 and mla.mla_get_device_error(ws2) == 0
        now = [x + i + 1 for x in lens]
        before = {n: t.clone() for n, t in c.items()}
        c, q_want = run_gqa(mla, c, dk, dk, bt, now, None, rope, True, q=dq)
        check_gqa(c, before, expect_gqa(before, dk, dk, bt, now, None, rope, 32, True), 32, True)
        assert all(torch.equal(d[n].cpu(), c[n]) for n in c)
        ref = attend(q_want, c["k"], c["v"], c["ks"], c["vs"], bt, now, None, False, 128 ** -0.5, 1, -1,
                     "interleaved")
        check_attention(out, lse_out, ref, out_rel=2.0 ** -8)
