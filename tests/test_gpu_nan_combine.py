"""A NaN key or value stays NaN through the combine of grouped-query shards, and
reaches no row that does not see it."""
import math

import pytest
import torch

from _block_ref import check_attention
from test_gpu_gqa_fp8 import call, make, ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mla():
    import sequence_sharded_mla_gb300 as m
    return m


@pytest.mark.parametrize("N", [1, 2, 8])
@pytest.mark.parametrize("lens", [[200, 90], [9000, 90]])
def test_nan_codes_reach_the_answer(mla, N, lens):
    """Codes as the append stores infinities and NaN: a key makes its head's
    rows NaN, a value one dim of those that see it."""
    w = make(lens, 8, 2, q_len=4, seed=110 + N)
    w["k"][w["bt"][0, 1].long(), 10, 1, 7] = 0x7F
    w["v"][w["bt"][1, 0].long(), 30, 0, 9] = 0xFF
    w["v"][w["bt"][1, 1].long(), 90 - 64 - 2, 1, 11] = 0x7F     # token L - 2: rows 2, 3
    w["k"][w["bt"][1, 1].long(), 90 - 64 - 1, 0, 0] = 0x7F      # token L - 1: row 3
    part, lse, st = call(mla, w, N, causal=True)
    assert st == 0
    out, lse_out = mla.gqa_shard_combine(part, lse)
    o = ref(w, 1, "interleaved", -1, True)
    assert bool(torch.isnan(o[0]).any()) and bool(torch.isnan(o[1]).any())
    check_attention(out, lse_out, o, out_rel=2.0 ** -8)


@pytest.mark.parametrize("N", [1, 2, 5, 8])
def test_combine_of_missing_finite_and_nan_shards(mla, N):
    """Every row has its own mixture of shards without a token, finite ones and
    NaN ones; a shard without a token counts for nothing."""
    g = torch.Generator().manual_seed(130 + N)
    kind = torch.randint(0, 3, (N, 6, 3, 8), generator=g)
    kind[:, 0] = 0                                   # no shard has a token
    kind[:, 1] = kind[:, 1].clamp(max=1)             # some rows without NaN
    lse = torch.randn(kind.shape, generator=g) * 8
    lse[kind == 0] = -math.inf
    lse[kind == 2] = math.nan
    part = torch.randn(*kind.shape, 128, generator=g)
    part[kind == 2] = math.nan
    part[kind == 0] = 0.0
    out, lse_out = mla.gqa_shard_combine(part.cuda(), lse.cuda())
    nan, none = (kind == 2).any(0), (kind == 0).all(0)
    want_lse = torch.logsumexp(lse.double(), 0)
    p = torch.exp(lse.double() - want_lse)
    want = (p[..., None] * part.double()).nan_to_num(0.0).sum(0)
    g_out, g_lse = out.double().cpu(), lse_out.double().cpu()
    assert torch.equal(torch.isnan(g_out), nan[..., None].expand_as(g_out))
    assert torch.equal(torch.isnan(g_lse), nan) and torch.equal(torch.isneginf(g_lse), none)
    assert bool((g_out[none] == 0).all())
    fine = ~nan & ~none
    # bf16 rounding of the result, and weights of fp32 exponentials of arguments
    # up to 60: 2^-8 of the largest term leaves room for both
    assert bool(((g_out - want).abs()[fine] <= part.abs().nan_to_num(0.0).amax(0)[fine].double() * 2.0 ** -8).all())
    assert bool(((g_lse - want_lse).abs()[fine] <= 2.0 ** -17).all())
