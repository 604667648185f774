"""Accuracy of the e4m3 grouped-query attention against bounds that are tighter
than those of the parity tests: how its weights are held."""
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


@pytest.mark.parametrize("H,Hkv,q_len", [(64, 4, 1), (64, 2, 1), (48, 1, 1), (64, 8, 9)])
def test_weights_are_held_to_eleven_bits(mla, H, Hkv, q_len):
    """Short contexts, where no average over tokens hides a weight's rounding:
    fp16's 2^-11 of each weight, and as much as 2^-14 for the sums and for the
    weights' exponential."""
    w = make([1, 2, 3, 4, 5, 7, 12, 33, 200], H, Hkv, seed=120 + H + q_len, q_len=q_len)
    part, lse, st = call(mla, w)
    assert st == 0
    check_attention(part[0], lse[0], ref(w), P_REL=2.0 ** -11 + 2.0 ** -14)


def wide_block(S, seed):
    """200 tokens in blocks of 16 whose second block's V scale is S times the
    others' and whose V codes there are zero but in dim 0; equal logits."""
    w = make([200], 4, 2, 16, seed=seed, poison=False)
    w["q"][...] = 0
    w["vs"][...] = 2.0 ** -7
    page = int(w["bt"][0, 0])
    w["vs"][page, 1] = 2.0 ** -7 * S
    w["v"][page, 16:32, :, 1:] = 0
    return w


@pytest.mark.parametrize("S", [2.0 ** 4, 2.0 ** 10, 2.0 ** 16, 2.0 ** 20, 2.0 ** 40, 2.0 ** 90])
def test_v_scales_far_apart(mla, S):
    """An error of 2^-11 of every p_t |sv_t| and of 2^-27 of the row's largest,
    times the codes: the other blocks' values live as far as that goes, and the
    lse does not notice."""
    w = wide_block(S, 160)
    part, lse, st = call(mla, w)
    assert st == 0
    o, want, spread, err = ref(w)
    codes = w["v"].view(torch.float8_e4m3fn).double().abs()
    page = w["bt"][0].long()[torch.arange(200) // 64]
    total = codes[page, torch.arange(200) % 64].sum(0).repeat_interleave(2, 0)     # [H, 128]
    lost = total * 2.0 ** -27 * (2.0 ** -7 * S / 200)
    got = part[0, 0, 0].double().cpu()
    assert bool(((got - o[0, 0]).abs() <= spread[0, 0] * (2.0 ** -11 + 2.0 ** -14) + lost).all())
    if S <= 2.0 ** 16:      # in the dims where the wide block has zeros
        assert bool(((got - o[0, 0]).abs() <= spread[0, 0] * 2.0 ** -9)[:, 1:].all())
    assert bool(((lse[0].double().cpu() - want).abs() <= 2.0 ** -18).all())


@pytest.mark.parametrize("scale,status", [(2.0 ** 120, 0), (2.0 ** 121, -7), (-2.0 ** 126, -7),
                                          (3.0e38, -7)])
def test_v_scales_above_the_range_are_reported(mla, scale, status):
    w = make([100], 4, 2, 16, seed=161, poison=False)
    w["vs"][...] = 1.0
    w["vs"][int(w["bt"][0, 0]), 3, 1] = scale
    assert call(mla, w)[2] == status
    w["lens"] = torch.tensor([48], dtype=torch.int32)      # the block is behind the context
    assert call(mla, w)[2] == 0
