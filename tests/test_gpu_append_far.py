"""Appends at the last positions that a context length can count."""
import pytest
import torch

from test_gpu_append import bf, i32

pytestmark = pytest.mark.gpu
LAST = 2 ** 31 - 1
PAGES = 2 ** 25                    # a table row that reaches them


@pytest.fixture(scope="module")
def mla():
    import sequence_sharded_mla_gb300 as m
    return m


def cache(fp8, block):
    if not fp8:
        return [torch.zeros(2, 64, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in "kv"] + [None, None]
    return ([torch.zeros(2, 64, 2, 128, dtype=torch.uint8, device="cuda") for _ in "kv"] +
            [torch.zeros(2, 64 // block, 2, device="cuda") for _ in "kv"])


@pytest.mark.parametrize("fp8,block", [(True, 64), (True, 16), (True, 1), (False, 64)])
@pytest.mark.parametrize("q_len", [1, 70])
def test_the_last_positions(mla, fp8, block, q_len):
    """They go where the same rows of the table's last pages go from length
    2 x 64 - 1, and are reported where the table is too short."""
    k, v = bf((1, q_len, 2, 128), 200).cuda(), bf((1, q_len, 2, 128), 201).cuda()

    def append(L, bt):
        kc, vc, ks, vs = c = cache(fp8, block)
        _, ws = mla.gqa_cache_append(k, v, kc, vc, bt, i32([L]).cuda(), k_scale=ks, v_scale=vs)
        return c, mla.mla_get_device_error(ws)

    want, st = append(127, i32([[0, 1]]).cuda())
    assert st == 0 and bool(want[0].any())
    bt = torch.full((1, PAGES), -1, dtype=torch.int32, device="cuda")
    bt[0, -2:] = i32([0, 1]).cuda()
    got, st = append(LAST, bt)
    assert st == 0
    for a, b in zip(want, got):
        assert a is None or torch.equal(a, b)
    got, st = append(LAST, i32([[0, 1]]).cuda())
    assert st == -5
    assert all(t is None or not bool(t.any()) for t in got)
