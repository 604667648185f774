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
