"""Calls of the e4m3 grouped-query chain that a user may make besides a decode
step: a prompt chunk's queries, two host threads, many KV heads."""
import threading

import pytest
import torch

from _block_ref import check_attention
from test_gpu_append import bf, i32
from test_gpu_gqa_fp8 import call, make, ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mla():
    import sequence_sharded_mla_gb300 as m
    return m


@pytest.mark.parametrize("q_len,H,Hkv,N", [(600, 32, 4, 1), (257, 8, 8, 2), (1025, 2, 1, 1)])
def test_prompt_chunk(mla, q_len, H, Hkv, N):
    """Causal, the first request all chunk and the second behind a context; every
    40th query and the ends against the reference."""
    lens = [q_len, q_len + 700]
    w = make(lens, H, Hkv, 32, q_len=q_len, seed=240 + q_len)
    part, lse, st = call(mla, w, N, causal=True)
    assert st == 0
    rows = {(b, i) for b in range(2) for i in [*range(0, q_len, 40), q_len - 1]}
    at = torch.tensor(sorted(rows))
    pick = lambda t: t[at[:, 0], at[:, 1]]
    for s in range(N):
        check_attention(pick(part[s].cpu()), pick(lse[s].cpu()),
                        [pick(t) for t in ref(w, N, "interleaved", s, True, rows=rows)])


def test_many_heads(mla):
    w = make([130, 1], 96, 48, 16, seed=250)
    part, lse, st = call(mla, w, 2)
    assert st == 0
    for s in range(2):
        check_attention(part[s], lse[s], ref(w, 2, s=s))


def test_two_host_threads(mla):
    """Each with its stream, caches and workspaces: append, attend and combine,
    over and over, give the bits of a single thread."""
    work = []
    for seed in (260, 261):
        g = torch.Generator().manual_seed(seed)
        lens = [40 + seed % 7, 700]
        table = torch.arange(2 * 12, dtype=torch.int32).view(2, 12)
        work.append(dict(
            q=bf((2, 1, 16, 128), seed).cuda(), k=bf((2, 1, 2, 128), seed + 1).cuda(),
            v=bf((2, 1, 2, 128), seed + 2).cuda(), lens=i32(lens).cuda(), bt=table.cuda(),
            cache=torch.randint(0, 120, (2, 24, 64, 2, 128), generator=g).to(torch.uint8).cuda(),
            scale=torch.exp2(torch.randint(-9, -5, (2, 24, 2, 2), generator=g).float()).cuda(),
            rope=mla.Rope(mla.mla_rope_frequencies(128)[0])))

    def step(w, stream):
        c, sc = w["cache"].clone(), w["scale"].clone()
        q, aws = mla.gqa_cache_append(w["k"], w["v"], c[0], c[1], w["bt"], w["lens"], w["rope"],
                                      q=w["q"], k_scale=sc[0], v_scale=sc[1], stream=stream)
        part, lse, ws = mla.gqa_decode_partial_fp8(q, c[0], c[1], sc[0], sc[1], w["bt"], w["lens"],
                                                   2, stream=stream)
        return *mla.gqa_shard_combine(part, lse, stream=stream), aws, ws

    want = [step(w, None) for w in work]
    torch.cuda.synchronize()
    got, failed = [[], []], []

    def run(k):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(60):
                    got[k].append(step(work[k], s))
            s.synchronize()
        except BaseException as e:      # a thread's failure is the test's
            failed.append(e)

    threads = [threading.Thread(target=run, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    for k in range(2):
        for out, lse, aws, ws in got[k]:
            assert torch.equal(out, want[k][0]) and torch.equal(lse, want[k][1])
            assert mla.mla_get_device_error(aws) == 0 and mla.mla_get_device_error(ws) == 0
