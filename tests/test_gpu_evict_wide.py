"""Eviction from weights in wide rows, which clusters of 8 and 16 CTAs select
from: any bit pattern, ties among NaN and zeros, short contexts in wide rows."""
import pytest
import torch

import sequence_sharded_mla_gb300 as mla

pytestmark = pytest.mark.gpu

PAGE, DEV = 64, "cuda"


def order_of(w):
    """Positions by falling weight, NaN first, equal ones (both zeros) in order."""
    bits = (w + 0.0).view(torch.int32).long()
    key = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits)      # the order of the numbers
    key = torch.where(torch.isnan(w), torch.full_like(key, 1 << 40), key)
    return torch.argsort(-key, stable=True)


def weights(kind, B, W, g):
    if kind == "any bits":
        w = torch.randint(-2**31, 2**31 - 1, (B, W), device=DEV, generator=g, dtype=torch.int32).view(torch.float32)
    elif kind == "NaN ties":
        w = torch.rand((B, W), device=DEV, generator=g)
        w = torch.where(torch.rand((B, W), device=DEV, generator=g) < 0.3, torch.full_like(w, float("nan")), w)
        w[:, ::3] = -w[:, ::3]                                    # NaN of either sign
    elif kind == "infinities and zeros":
        v = torch.tensor([float("inf"), -float("inf"), 0.0, -0.0, 1e-45, -1e-45, 3e38], device=DEV)
        w = v[torch.randint(0, 7, (B, W), device=DEV, generator=g)]
    return w


@pytest.mark.parametrize("kind", ["any bits", "NaN ties", "infinities and zeros"])
@pytest.mark.parametrize("W", [65537, 262144, 262145, 400003])
def test_wide_rows(W, kind):
    g = torch.Generator(device=DEV).manual_seed(W)
    w = weights(kind, 4, W, g)
    lens = [W, W // 2 + 5, 777, 8000]
    old = -(-W // PAGE)
    first, recent = [3, 0, 64, 100], 41
    bt = torch.arange(4 * old, dtype=torch.int32, device=DEV).view(4, old)
    # codes and scales are the row's place, in parts
    n = 8 * old * PAGE
    kv = torch.zeros((8 * old, PAGE, 576), dtype=torch.uint8, device=DEV)
    place = torch.arange(n, device=DEV)
    for i in range(4):
        kv.view(-1, 576)[:, 150 * i] = (place >> (8 * i)).to(torch.uint8)
    scale = place.to(torch.int32).view(torch.float32).view(-1, PAGE)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    for share in (0.001, 0.3, 0.97):
        keep = [max(int(L * share), 150) for L in lens]      # both windows, and others
        new, kept, out, _ = mla.mla_cache_evict(kv, bt, i32(lens), w, i32(keep), bt + 4 * old, keep_first=i32(first),
                                                recent=recent, kv_scale=scale, workspace=ws)
        torch.cuda.synchronize()
        assert mla.mla_get_device_error(ws) == 0 and new.tolist() == keep
        for b, (L, k, f) in enumerate(zip(lens, keep, first)):
            mid = order_of(w[b, f:L - recent])[:k - f - recent].sort().values + f
            want = torch.cat((torch.arange(f, device=DEV), mid, torch.arange(L - recent, L, device=DEV)))
            assert torch.equal(kept[b, :k].long(), want) and (kept[b, k:] == -1).all()
            assert torch.equal(out[b, :k].view(torch.int32), w[b, want].view(torch.int32))
            src = b * old * PAGE + want
            rows = slice((4 + b) * old * PAGE, (4 + b) * old * PAGE + k)
            assert torch.equal(scale.view(-1)[rows].view(torch.int32).long(), src)
            for i in range(4):
                assert torch.equal(kv.view(-1, 576)[rows, 150 * i].long(), (src >> (8 * i)) & 255)
