"""GPU parity of grouped-query attention over an e4m3 cache with block scales
against a 64-bit reference: group sizes, blocks, shards and layouts, ragged and
padded batches, causal rows that see nothing, poisoned unused rows, extreme
scales and queries, NaN in seen and unseen places, bad pages, graphs, streams."""
import math

import pytest
import torch

from _block_ref import FP8, PAGE, attend, check_attention, owned

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mla():
    import sequence_sharded_mla_gb300 as m
    return m


def make(lens, H, Hkv, block=64, q_len=1, seed=0, poison=True, q_sigma=1.0, spare=2, N=1, s=0,
         layout="interleaved"):
    """A batch on the CPU.  Slots that hold no token are NaN codes under NaN
    scales, except where a live token shares the block."""
    g = torch.Generator().manual_seed(seed)
    slots = [owned(L, s, N, layout)[1] if layout.endswith("local") else list(range(L)) for L in lens]
    need = [-(-len(x) // PAGE) for x in slots]
    P = sum(need) + spare
    perm = torch.randperm(P, generator=g).to(torch.int32)
    bt = torch.full((len(lens), max(need + [1]) + 1), -1, dtype=torch.int32)
    off = 0
    for b, n in enumerate(need):
        bt[b, :n] = perm[off:off + n]
        off += n
    w = dict(q=(torch.randn(len(lens), q_len, H, 128, generator=g) * q_sigma).bfloat16(), bt=bt,
             lens=torch.tensor(lens, dtype=torch.int32))
    used = torch.zeros(P, PAGE, dtype=torch.bool)
    for b, x in enumerate(slots):
        for p in x:
            used[int(bt[b, p // PAGE]), p % PAGE] = True
    for n in "kv":
        c = (torch.randn(P, PAGE, Hkv, 128, generator=g) * 110).clamp(-448, 448).to(FP8).view(torch.uint8)
        sc = (torch.rand(P, PAGE // block, Hkv, generator=g) + 0.5) / 110
        if poison:
            c[~used] = 0x7F
            sc[~used.view(P, PAGE // block, block).any(-1)] = math.nan
        w[n], w[n + "s"] = c, sc
    return w


def call(mla, w, N=1, layout="interleaved", shard_id=-1, causal=False, q_lens=None, scale=None, **kw):
    d = lambda t: None if t is None else t.cuda()
    part, lse, ws = mla.gqa_decode_partial_fp8(
        d(w["q"]), d(w["k"]).view(FP8), d(w["v"]).view(FP8), d(w["ks"]), d(w["vs"]), d(w["bt"]),
        d(w["lens"]), N, layout, shard_id=shard_id, causal=causal, softmax_scale=scale,
        q_lens=d(q_lens), **kw)
    return part, lse, mla.mla_get_device_error(ws)


def ref(w, N=1, layout="interleaved", s=0, causal=False, q_lens=None, scale=None, rows=None):
    return attend(w["q"], w["k"], w["v"], w["ks"], w["vs"], w["bt"], w["lens"], q_lens, causal,
                  128 ** -0.5 if scale is None else scale, N, s, layout, rows)


def check(mla, w, N=1, layout="interleaved", causal=False, q_lens=None, scale=None, status=0):
    part, lse, st = call(mla, w, N, layout, causal=causal, q_lens=q_lens, scale=scale)
    assert st == status
    for s in range(N):
        check_attention(part[s], lse[s], ref(w, N, layout, s, causal, q_lens, scale))
    out, lse_out = mla.gqa_shard_combine(part, lse)
    check_attention(out, lse_out, ref(w, 1, "interleaved", -1, causal, q_lens, scale),
                    out_rel=2.0 ** -8)


@pytest.mark.parametrize("H,Hkv", [(8, 8), (16, 8), (20, 4), (14, 2), (8, 1), (16, 1), (32, 2),
                                   (24, 1), (48, 1), (64, 1)])
def test_group_sizes(mla, H, Hkv):
    check(mla, make([1, 63, 64, 65, 127, 700], H, Hkv, seed=H + Hkv))


@pytest.mark.parametrize("block", [1, 2, 8, 16, 32, 64])
def test_blocks(mla, block):
    check(mla, make([1, 129, 300], 16, 2, block, seed=30 + block))


@pytest.mark.parametrize("N,layout", [(1, "interleaved"), (2, "interleaved"), (4, "interleaved"),
                                      (8, "interleaved"), (1, "contiguous"), (3, "contiguous"),
                                      (8, "contiguous")])
def test_shards_and_layouts(mla, N, layout):
    check(mla, make([1, 5, 400, 1300], 16, 4, 16, seed=50 + N), N, layout)


@pytest.mark.parametrize("N,layout", [(3, "interleaved_local"), (4, "interleaved_local"),
                                      (5, "contiguous_local"), (2, "contiguous_local")])
def test_local_slices(mla, N, layout):
    for s in range(N):
        w = make([1, 300, 77], 8, 2, 32, q_len=2, seed=60 + s, N=N, s=s, layout=layout)
        part, lse, st = call(mla, w, N, layout, shard_id=s, causal=True)
        assert st == 0
        check_attention(part[0], lse[0], ref(w, N, layout, s, True))


@pytest.mark.parametrize("q_len,H,Hkv", [(3, 16, 4), (9, 64, 8), (5, 14, 2), (9, 32, 2), (2, 64, 1),
                                         (70, 4, 2)])
@pytest.mark.parametrize("layout", ["interleaved", "contiguous"])
def test_causal_verify(mla, q_len, H, Hkv, layout):
    """The second request is shorter than its query tokens: its first rows see
    nothing."""
    check(mla, make([200, max(1, q_len - 2), 131], H, Hkv, seed=q_len + H, q_len=q_len), 2, layout,
          causal=True)


@pytest.mark.parametrize("causal", [False, True])
def test_padded_batch(mla, causal):
    w = make([300, 40, 5, 130], 40, 4, 32, q_len=9, seed=70)
    check(mla, w, 2, causal=causal, q_lens=torch.tensor([9, 1, 5, 4], dtype=torch.int32))


def test_query_counts_out_of_range_are_clamped_and_reported(mla):
    w = make([100, 40], 8, 2, q_len=3, seed=71)
    ql = torch.tensor([7, 0], dtype=torch.int32)
    part, lse, st = call(mla, w, causal=True, q_lens=ql)
    assert st == -1
    check_attention(part[0], lse[0], ref(w, causal=True, q_lens=ql.clamp(0, 3)))


def test_no_tokens(mla):
    w = make([0, 10, 0], 8, 2, seed=72)
    part, lse, st = call(mla, w, 2)
    assert st == 0
    for s in range(2):
        check_attention(part[s], lse[s], ref(w, 2, s=s))


def test_long_contexts_are_split_and_joined(mla):
    lens = [20011, 3, 70001]
    w = make(lens, 8, 2, seed=73)
    part, lse, st = call(mla, w, 2)
    assert st == 0
    for s in range(2):
        check_attention(part[s], lse[s], ref(w, 2, s=s))


def test_scales_of_every_size(mla):
    """Zero, negative, far apart and tiny block scales; one block outweighs the
    rest by 2^40 in V, and the query looks away from it."""
    w = make([640], 8, 2, 16, seed=74, poison=False)
    g = torch.Generator().manual_seed(75)
    for n in ("ks", "vs"):
        e = torch.randint(-12, -4, w[n].shape, generator=g)
        w[n] = torch.exp2(e.float()) * (1 - 2 * torch.randint(0, 2, w[n].shape, generator=g))
    w["vs"][0] = 0.0
    w["vs"][1, 0] = 2.0 ** 40
    w["ks"][1, 0] = 0.0
    w["vs"][2, 1] = 2.0 ** -58
    w["ks"][3, 1] = 2.0 ** -100
    check(mla, w)
    w["vs"][...] = 2.0 ** -40
    check(mla, w)
    w["vs"][...] = 0.0
    check(mla, w)


def test_a_flat_tail_below_one_large_weight(mla):
    """40000 tokens whose weights are 2^-12 of the largest: together they are
    ten times its weight."""
    w = make([40001], 1, 1, seed=76, poison=False)
    w["q"][...] = 0
    w["q"][..., 0] = 1.0
    w["k"][...] = 0
    w["ks"][...] = 1.0
    page, row = int(w["bt"][0, 100]), 7
    w["k"][page, row, 0, 0] = torch.tensor(12 * math.log(2.0)).to(FP8).view(torch.uint8)
    check(mla, w, scale=1.0)


@pytest.mark.parametrize("size", [0.0, 1e-30, 1e-3, 300.0, 1e30])
def test_query_magnitudes(mla, size):
    w = make([150, 64], 8, 2, seed=77)
    w["q"] = (w["q"].float() * size).bfloat16()
    check(mla, w, scale=min(128 ** -0.5, 0.1 / max(size, 1e-30)))


def test_query_rows_of_mixed_magnitude(mla):
    w = make([150], 8, 1, seed=78)
    w["q"] *= torch.exp2(torch.arange(8) * 3.0 - 20)[None, None, :, None].bfloat16()
    check(mla, w)


def test_nonfinite_query_is_reported(mla):
    w = make([100, 80], 8, 2, q_len=2, seed=79)
    w["q"][1, 1, 3, 5] = math.inf
    ql = torch.tensor([2, 1], dtype=torch.int32)
    assert call(mla, w)[2] == -7
    part, lse, st = call(mla, w, q_lens=ql)     # the row is padding
    assert st == 0
    check_attention(part[0], lse[0], ref(w, q_lens=ql))


def test_nan_reaches_the_rows_that_see_it(mla):
    """A NaN key makes its head's rows NaN, a NaN value one dim; a NaN in a
    drafted token reaches only the rows that see the token."""
    w = make([200, 90], 8, 2, q_len=4, seed=80)
    w["k"][w["bt"][0, 1].long(), 10, 1, 7] = 0x7F
    w["v"][w["bt"][1, 0].long(), 30, 0, 9] = 0xFF
    w["v"][w["bt"][1, 1].long(), 90 - 64 - 2, 1, 11] = 0x7F     # token L - 2: rows 2, 3
    w["k"][w["bt"][1, 1].long(), 90 - 64 - 1, 0, 0] = 0x7F      # token L - 1: row 3
    part, lse, st = call(mla, w, causal=True)
    assert st == 0
    check_attention(part[0], lse[0], ref(w, causal=True))


def test_bad_pages_read_as_zeros(mla):
    w = make([300, 70], 8, 2, seed=81)
    w["bt"][0, 2] = w["k"].shape[0] + 5
    w["bt"][1, 1] = -3
    check(mla, w, status=-5)


def test_same_bits_every_time_and_one_error_word_per_call(mla):
    w = make([900, 5000, 17], 32, 4, q_len=3, seed=82)
    a = call(mla, w, 2, causal=True)
    b = call(mla, w, 2, causal=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_graph_replay_and_streams(mla):
    w = make([900, 333], 16, 2, seed=83)
    d = {n: t.cuda() for n, t in w.items()}
    need = mla.gqa_fp8_workspace_size(2, 1, 16, 2, 2)

    def go(stream=None, ws=None):
        return mla.gqa_decode_partial_fp8(d["q"], d["k"], d["v"], d["ks"], d["vs"], d["bt"],
                                          d["lens"], 2, workspace=ws, stream=stream)

    p0, l0, _ = go()
    side = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for k in range(6):
        got.append(go(side[k % 2], torch.empty(need, dtype=torch.uint8, device="cuda")))
    torch.cuda.synchronize()
    for p, l, _ in got:
        assert torch.equal(p, p0) and torch.equal(l, l0)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p, l, _ = go(ws=ws)
    d["lens"].copy_(torch.tensor([20, 64], dtype=torch.int32))
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    w["lens"] = torch.tensor([20, 64], dtype=torch.int32)
    for s in range(2):
        check_attention(p[s], l[s], ref(w, 2, s=s))


def test_more_units_than_a_cta_plans_for_itself(mla):
    """1300 requests: the plan kernel's path, errors included."""
    g = torch.Generator().manual_seed(84)
    lens = torch.randint(0, 150, (1300,), generator=g).tolist()
    w = make(lens, 4, 1, 32, q_len=2, seed=85)
    ql = torch.randint(1, 3, (1300,), generator=g).to(torch.int32)
    part, lse, st = call(mla, w, causal=True, q_lens=ql)
    assert st == 0
    check_attention(part[0], lse[0], ref(w, causal=True, q_lens=ql))
    ql[1299] = 0
    assert call(mla, w, causal=True, q_lens=ql)[2] == -1


def test_wait_budget_runs_out_and_the_next_call_is_clean(mla):
    """The queries of each CTA's first piece are withheld, so the waits for
    them run out after 1 ms: reported, and nothing is left behind."""
    for H in (8, 32, 64):
        w = make([3000, 300], H, 1, seed=86)
        try:
            mla.mla_set_wait_budget_ns(1_000_000)
            mla.mla_set_withhold_query(True)
            assert call(mla, w)[2] == -4
        finally:
            mla.mla_set_withhold_query(False)
            mla.mla_set_wait_budget_ns(0)
        part, lse, st = call(mla, w)
        assert st == 0
        check_attention(part[0], lse[0], ref(w))


@pytest.mark.parametrize("H,N", [(1, 1), (16, 1), (48, 1), (2, 8)])
def test_one_request_over_every_cta(mla, H, N):
    """20000 tokens over one KV head: about 80 pieces to a unit, more than it
    has rows, joined by the blocks of all the CTAs that share it."""
    check(mla, make([20000], H, 1, seed=87 + H), N)


def test_a_long_context_among_short_ones(mla):
    """Units of many pieces, of one and of none side by side."""
    check(mla, make([3, 15000, 0, 700, 129], 12, 2, 32, q_len=4, seed=91), 2, causal=True)


def test_bad_pages_at_eight_shards(mla):
    w = make([300, 70], 8, 2, 32, seed=92)
    w["bt"][0, 2] = w["k"].shape[0]
    w["bt"][1, 0] = -1
    part, lse, st = call(mla, w, 8)
    assert st == -5
    for s in range(8):
        o, l, spread, err = ref(w, 8, s=s)
        # a token of a missing page has V scale 0, which stands as lv = -60 in
        # its weight's exponent s + lv - m (log2 units); here |lv - m| < 64, so
        # lv - m and the exponent are each rounded by up to 2^-19: 2^-18 ln 2
        check_attention(part[s], lse[s], (o, l, spread, err + 2.0 ** -18 * math.log(2.0)))


def test_eight_shards_of_many_rows(mla):
    check(mla, make([400, 7, 1300], 40, 1, 16, seed=93), 8)
    check(mla, make([500, 90], 16, 2, 64, q_len=9, seed=94), 8, causal=True)


def test_context_longer_than_its_table(mla):
    """It is cut at its last page and reported; the others are whole."""
    w = make([200, 300], 8, 2, seed=95)
    w["bt"] = w["bt"][:, :4].contiguous()
    w["lens"] = torch.tensor([200, 2 ** 31 - 1], dtype=torch.int32)
    part, lse, st = call(mla, w)
    assert st == -5
    w["lens"] = torch.tensor([200, 256], dtype=torch.int32)
    check_attention(part[0], lse[0], ref(w))


def test_work_that_passes_31_bits_is_refused(mla):
    w = make([20] * 64, 65, 65, seed=96)      # (an odd number of heads: no teams)
    w["bt"] = torch.zeros(64, 1 << 20, dtype=torch.int32)
    with pytest.raises(mla.MLAError) as e:
        call(mla, w, 2)
    assert e.value.status == -2


def test_memory_of_a_call_on_a_given_stream(mla):
    """Outputs and workspace that a call allocates belong to its stream."""
    w = make([900, 333], 16, 2, seed=97)
    d = {n: t.cuda() for n, t in w.items()}
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    part, lse, ws = mla.gqa_decode_partial_fp8(d["q"], d["k"], d["v"], d["ks"], d["vs"], d["bt"],
                                               d["lens"], 2, stream=side)
    out, lse_out = mla.gqa_shard_combine(part, lse, stream=side)
    assert torch.cuda.current_stream() != side
    side.synchronize()
    assert mla.mla_get_device_error(ws) == 0
    check_attention(out, lse_out, ref(w, 1, "interleaved", -1), out_rel=2.0 ** -8)


def test_two_graphs_with_one_workspace(mla):
    """Replayed in turn, over a workspace of arbitrary bytes."""
    ws = torch.full((mla.gqa_fp8_workspace_size(2, 2, 48, 1, 2),), 0xFF, dtype=torch.uint8,
                    device="cuda")
    runs = []
    for seed, lens in ((98, [3000, 5]), (99, [64, 1700])):
        w = make(lens, 48, 1, q_len=2, seed=seed)
        d = {n: t.cuda() for n, t in w.items()}

        def go():
            return mla.gqa_decode_partial_fp8(d["q"], d["k"], d["v"], d["ks"], d["vs"], d["bt"],
                                              d["lens"], 2, causal=True, workspace=ws)

        go()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            part, lse, _ = go()
        runs.append((w, d, g, part, lse))
    for _ in range(2):
        for w, d, g, part, lse in runs:
            part.fill_(float("nan"))
            g.replay()
    torch.cuda.synchronize()
    for w, d, g, part, lse in runs:
        for s in range(2):
            check_attention(part[s], lse[s], ref(w, 2, s=s, causal=True))


def test_binding_refusals(mla):
    w = {n: t.cuda() for n, t in make([100, 40], 8, 2, seed=100).items()}
    args = lambda **k: [{**w, **k}[n] for n in ("q", "k", "v", "ks", "vs", "bt", "lens")]
    bad = [dict(q=w["q"].float()), dict(k=w["k"][..., :64]), dict(v=w["v"][:1]),
           dict(ks=w["ks"].double()), dict(vs=w["vs"][:, :, :1]), dict(bt=w["bt"].cpu()),
           dict(lens=w["lens"].long()), dict(lens=w["lens"][:1]), dict(bt=w["bt"][:1]),
           dict(q=w["q"].transpose(1, 2)), dict(k=w["k"].view(torch.int8))]
    for k in bad:      # (the transposed q is [2, 8, 1, 128]: one head for two KV heads)
        with pytest.raises((TypeError, ValueError, mla.MLAError)):
            mla.gqa_decode_partial_fp8(*args(**k), 1)
    for k in (dict(out_partial=torch.empty(1, 2, 1, 8, 64, device="cuda")),
              dict(lse_partial=torch.empty(2, 2, 1, 8, device="cuda")),
              dict(workspace=torch.empty(16, device="cuda")), dict(q_lens=w["lens"][:1])):
        with pytest.raises((TypeError, ValueError)):
            mla.gqa_decode_partial_fp8(*args(), 1, **k)
    with pytest.raises(KeyError):
        mla.gqa_decode_partial_fp8(*args(), 1, "diagonal")
    with pytest.raises(mla.MLAError):
        mla.gqa_decode_partial_fp8(*args(), 9)
    with pytest.raises(mla.MLAError):
        mla.gqa_decode_partial_fp8(*args(), 1, workspace=torch.empty(64, dtype=torch.uint8,
                                                                     device="cuda"))
    part, lse, _ = mla.gqa_decode_partial_fp8(*args(), 2)
    for k in (dict(lses=lse[:1]), dict(out=torch.empty(2, 1, 8, 64, dtype=torch.bfloat16, device="cuda")),
              dict(out=torch.empty(2, 1, 8, 128, dtype=torch.bfloat16)),
              dict(lse_out=torch.empty(2, 1, 4, device="cuda"))):
        with pytest.raises(ValueError):
            mla.gqa_shard_combine(part, k.pop("lses", lse), **k)


def test_teams_behind_the_plan_kernel(mla):
    """800 requests over two heads: a plan of 800 units for teams of two."""
    g = torch.Generator().manual_seed(101)
    lens = torch.randint(0, 200, (800,), generator=g).tolist()
    w = make(lens, 6, 2, 16, seed=102)
    part, lse, st = call(mla, w)
    assert st == 0
    check_attention(part[0], lse[0], ref(w))


@pytest.mark.parametrize("Hkv", [1, 2, 3, 4, 6, 8, 12, 16])
def test_teams_of_every_size(mla, Hkv):
    """Split, whole and empty units of 1, 2, 4 and 8 CTAs a team."""
    check(mla, make([2500, 0, 31, 200], 2 * Hkv, Hkv, 32, q_len=2, seed=103 + Hkv), 2, causal=True)
