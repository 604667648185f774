"""Rotation from some columns of a fused tensor into others of the same one."""
import pytest
import torch

from test_gpu_append import bf, i32, rope_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mla():
    import sequence_sharded_mla_gb300 as m
    return m


def columns(t, first, heads, D):
    return t[..., first:first + heads * D].unflatten(-1, (heads, D))


@pytest.mark.parametrize("x0,y0", [(0, 512), (512, 0), (264, 1040), (1040, 8)])
def test_disjoint_columns_of_one_tensor(mla, x0, y0):
    fused = bf((2, 5, 1552), 190).cuda()
    keep = fused.clone()
    x, y = columns(fused, x0, 4, 128), columns(fused, y0, 4, 128)
    lens, rope = i32([5, 900]).cuda(), rope_of(mla, 64, 0, True)
    want = mla.mla_rope_apply(x.contiguous(), rope, lens)
    assert mla.mla_rope_apply(x, rope, lens, out=y) is y
    assert torch.equal(y, want)
    columns(keep, y0, 4, 128).copy_(want)
    assert torch.equal(fused, keep)                       # nothing else moved


def test_columns_of_an_append(mla):
    B, H, Hkv = 3, 4, 2
    fused = bf((B, 1, (2 * H + 2 * Hkv) * 128), 191).cuda()
    q, q_out = columns(fused, 0, H, 128), columns(fused, H * 128, H, 128)
    k, v = columns(fused, 2 * H * 128, Hkv, 128), columns(fused, (2 * H + Hkv) * 128, Hkv, 128)
    lens, rope = i32([5, 64, 1]).cuda(), rope_of(mla, 128)
    bt = torch.arange(3, dtype=torch.int32).view(3, 1).cuda()
    kc, vc = (torch.zeros(3, 64, Hkv, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    want = mla.mla_rope_apply(q.contiguous(), rope, lens)
    before = q.clone()
    got, ws = mla.gqa_cache_append(k, v, kc, vc, bt, lens, rope, q=q, q_out=q_out)
    assert mla.mla_get_device_error(ws) == 0
    assert got is q_out and torch.equal(q_out, want) and torch.equal(q, before)


@pytest.mark.parametrize("x0,y0", [(0, 504), (0, 8), (1040, 600)])
def test_columns_that_meet_are_refused(mla, x0, y0):
    fused = bf((2, 5, 1552), 192).cuda()
    keep = fused.clone()
    lens, rope = i32([5, 900]).cuda(), rope_of(mla, 64, 0, True)
    x, y = columns(fused, x0, 4, 128), columns(fused, y0, 4, 128)
    with pytest.raises(ValueError):
        mla.mla_rope_apply(x, rope, lens, out=y)
    assert torch.equal(fused, keep)


def test_other_overlaps_are_refused(mla):
    flat = bf((8192,), 193).cuda()
    lens, rope = i32([5]).cuda(), rope_of(mla, 64, 0, True)
    x = flat[:1536].view(1, 3, 512).unflatten(-1, (4, 128))
    for y in (flat[512:2048].view(1, 3, 512), flat[:3 * 1032].view(1, 3, 1032)[..., 512:1024],
              flat[1024:1024 + 3 * 520].view(1, 3, 520)[..., :512]):
        with pytest.raises(ValueError):
            mla.mla_rope_apply(x, rope, lens, out=y.unflatten(-1, (4, 128)))
    y = flat[1600:3136].view(1, 3, 512).unflatten(-1, (4, 128))
    mla.mla_rope_apply(x, rope, lens, out=y)
    assert torch.equal(y, mla.mla_rope_apply(x, rope, lens))
    # one row of tokens shifted by a token: the same columns
    wide = bf((1, 4, 1024), 194).cuda()
    with pytest.raises(ValueError):
        mla.mla_rope_apply(columns(wide[:, :3], 0, 4, 128), rope, lens, out=columns(wide[:, 1:], 0, 4, 128))
