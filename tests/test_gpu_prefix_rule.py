"""Shared-prefix attention as users get it, with the library's own choice of
what to share, and over the slices of several ranks."""
import math
import random

import pytest
import torch

import sequence_sharded_mla_gb300 as mla

from _helpers import REL_OUT, TOL_LSE, TOL_OUT, check_close
from test_gpu_prefix import Batch, check, i32, in_slice_0

pytestmark = pytest.mark.gpu

PAGE, DEV = 64, "cuda"


@pytest.mark.parametrize("fp8", [False, True])
def test_groups_that_share_beside_groups_that_do_not(fp8):
    rng = random.Random(3)
    sizes, common = [24, 1, 2, 20], [9000, 5000, 100, 4000]
    b = Batch(sizes, common, [rng.randint(1, 300) for _ in range(47)], H=64, fp8=fp8, seed=1)
    _, lse, _ = check(b)
    assert in_slice_0(lse) == [k in (0, 3) for k in b.group]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("causal", [False, True])
def test_verify_steps(causal, fp8):
    rng = random.Random(7)
    new = [rng.randint(1, 5) for _ in range(18)]
    b = Batch([10, 8], [20000, 9000], [5 + rng.randint(0, 500) for _ in range(18)], 5, 64, fp8, causal, q_lens=new,
              seed=3)
    for r, n in enumerate(new):
        b.q[r, n:] = math.nan
    _, lse, _ = check(b)
    assert all(in_slice_0(lse))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("sizes,common,H", [([1], [300], 16), ([2], [2000], 128), ([3, 3], [700, 64], 48),
                                            ([1] * 40, [1000] * 40, 16), ([200], [64], 16)])
def test_batches_that_share_nothing(sizes, common, H, fp8):
    rng = random.Random(H)
    b = Batch(sizes, common, [rng.randint(1, 90) for _ in range(sum(sizes))], H=H, fp8=fp8, seed=5)
    part, lse, _ = check(b)
    assert not any(in_slice_0(lse)) and (part[0] == 0).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("always", [False, True])
def test_slices_of_two_ranks(always, fp8):
    # every rank passes the lengths of its own slice (every other token), with no
    # causal mask, and all four partials meet in the combine
    b = Batch([12, 7], [60000, 700], [1 + 31 * i for i in range(19)], H=64, fp8=fp8, seed=8)
    want = b.expect()
    parts, lses = [], []
    for r in range(2):
        local = Batch([12, 7], [-(-(n - r) // 2) for n in b.common],
                      [-(-(L - r) // 2) - -(-(b.common[k] - r) // 2) for L, k in zip(b.lens, b.group)],
                      H=64, fp8=fp8, causal=False, seed=8)
        for k, L, mine, whole in zip(range(19), local.lens, local.bt, b.bt):
            t = torch.arange(L, device=DEV)
            to = mine[t // PAGE].long() * PAGE + t % PAGE
            at = 2 * t + r
            src = whole[at // PAGE].long() * PAGE + at % PAGE
            local.kv.view(-1, 576)[to] = b.kv.view(-1, 576)[src]
            if fp8:
                local.scale.view(-1)[to] = b.scale.view(-1)[src]
        local.q = b.q
        mla.mla_set_prefix_sharing(always)
        try:
            part, lse, ws = local.call()
        finally:
            mla.mla_set_prefix_sharing(False)
        assert mla.mla_get_device_error(ws) == 0
        assert in_slice_0(lse)[:12] == [True] * 12
        parts.append(part)
        lses.append(lse)
    out, lse = mla.mla_shard_combine(torch.cat(parts), torch.cat(lses))
    check_close(lse.cpu(), want[1].cpu(), TOL_LSE, "lse")
    check_close(out.float().cpu(), want[0].cpu(), TOL_OUT, "out", rel=REL_OUT)
