"""The error word of a workspace that serves one call after another."""
import pytest
import torch

from test_gpu_append import bf, i32
from test_gpu_gqa_fp8 import make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mla():
    import sequence_sharded_mla_gb300 as m
    return m


@pytest.mark.parametrize("lens", [[300, 70], [5] * 900])
def test_attention_reports_its_last_call_alone(mla, lens):
    """A clean call over the word that a failed one left, or over any bytes, with
    few units (planned by every CTA) and many (by the plan kernel)."""
    w = {n: t.cuda() for n, t in make(lens, 8, 1, seed=230).items()}
    bad = w["bt"].clone()
    bad[0, 0] = w["k"].shape[0]
    ws = torch.full((mla.gqa_fp8_workspace_size(len(lens), 1, 8, 1, 1),), 0xFF, dtype=torch.uint8,
                    device="cuda")

    def go(bt):
        mla.gqa_decode_partial_fp8(w["q"], w["k"], w["v"], w["ks"], w["vs"], bt, w["lens"], 1,
                                   workspace=ws)

    go(w["bt"])
    assert mla.mla_get_device_error(ws) == 0
    go(bad)
    go(w["bt"])
    assert mla.mla_get_device_error(ws) == 0
    go(w["bt"])
    go(bad)
    assert mla.mla_get_device_error(ws) == -5
    assert mla.mla_get_device_error(ws) == 0          # reading clears it


@pytest.mark.parametrize("kind", ["latent", "bf16", "e4m3"])
def test_appends_keep_their_errors_until_they_are_read(mla, kind):
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    lens = i32([70, 3]).cuda()
    good, bad = i32([[0, 1], [2, -1]]).cuda(), i32([[0, 9], [2, -1]]).cuda()
    x = bf((2, 2, 576), 231).cuda()
    k = bf((2, 2, 2, 128), 232).cuda()
    kv = torch.zeros(4, 64, 576, dtype=torch.bfloat16, device="cuda")
    dt = torch.bfloat16 if kind == "bf16" else torch.uint8
    c = [torch.zeros(4, 64, 2, 128, dtype=dt, device="cuda") for _ in "kv"]
    sc = [torch.zeros(4, 2, 2, device="cuda") if kind == "e4m3" else None for _ in "kv"]

    def go(bt):
        if kind == "latent":
            mla.mla_cache_append(x, kv, bt, lens, workspace=ws)
        else:
            mla.gqa_cache_append(k, k, *c, bt, lens, k_scale=sc[0], v_scale=sc[1], workspace=ws)

    go(good)
    assert mla.mla_get_device_error(ws) == 0
    go(bad)
    go(good)
    assert mla.mla_get_device_error(ws) == -5
    assert mla.mla_get_device_error(ws) == 0
    go(good)
    assert mla.mla_get_device_error(ws) == 0
