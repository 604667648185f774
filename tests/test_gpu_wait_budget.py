"""Device-side waits give up when their budget has run out: not before, and not
much later.  The wait that runs out is one for a query that a testing hook
withholds."""
import pytest
import torch

from test_gpu_gqa_fp8 import make

pytestmark = pytest.mark.gpu


def shortest(call):
    """Device time of the fastest of eight calls, in ms."""
    best = 1e9
    for _ in range(8):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        torch.cuda.synchronize()
        a.record()
        call()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b))
    return best


@pytest.mark.parametrize("kind", ["latent", "grouped"])
@pytest.mark.parametrize("budget_ms", [0.05, 0.5, 2.0])
def test_a_wait_gives_up_at_its_limit(kind, budget_ms):
    import sequence_sharded_mla_gb300 as mla
    w = {n: t.cuda() for n, t in make([500, 300], 8, 1, seed=180).items()}
    q = torch.randn(2, 1, 16, 576, device="cuda").bfloat16()
    kv = torch.randn(16, 64, 576, device="cuda").bfloat16()
    bt = torch.arange(16, dtype=torch.int32, device="cuda").view(2, 8)
    last = []

    def call():
        if kind == "latent":
            r = mla.mla_decode_partial(q, kv, bt, w["lens"], 1)
        else:
            r = mla.gqa_decode_partial_fp8(w["q"], w["k"], w["v"], w["ks"], w["vs"], w["bt"],
                                           w["lens"], 1)
        last.append(r[2])

    call()
    try:
        mla.mla_set_wait_budget_ns(int(budget_ms * 1e6))
        mla.mla_set_withhold_query(True)
        ms = shortest(call)
        assert mla.mla_get_device_error(last[-1]) == -4
    finally:
        mla.mla_set_withhold_query(False)
        mla.mla_set_wait_budget_ns(0)
    # the launches take about 0.05 ms; a sleep in the barrier may take 0.2
    assert budget_ms <= ms < budget_ms + 0.25, f"{ms} ms"
    call()
    assert mla.mla_get_device_error(last[-1]) == 0
