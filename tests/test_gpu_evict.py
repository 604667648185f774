"""Eviction from latent caches against a plain selection: every byte of the
pool, the positions, weights and lengths, at the budgets, ties and weights
where it can go wrong."""
import math
import random

import numpy as np
import pytest
import torch

import sequence_sharded_mla_gb300 as mla

pytestmark = pytest.mark.gpu

PAGE = 64
DEV = "cuda"


def pages(n):
    return -(-n // PAGE)


def chosen(w, L, keep, first, recent):
    """The kept positions: Python's own sort, NaN above +inf, zeros equal."""
    n = min(L, keep)
    first = min(first, n)
    recent = min(recent, n - first)
    if n == L:
        return list(range(L))

    def rank(t):
        x = float(w[t])
        return (-math.inf, 0) if math.isnan(x) else (-x, 1)

    held = set(range(first)) | set(range(L - recent, L))
    others = sorted((t for t in range(L) if t not in held),
                    key=lambda t: ((0, 0.0) if math.isnan(float(w[t])) else (1, -float(w[t])), t))
    return sorted(held | set(others[:n - first - recent]))


class Pool:
    """A cache with a batch's old and new pages in random places."""

    def __init__(self, lens, keeps, fp8, seed, shared_pages=0):
        rng = random.Random(seed)
        g = torch.Generator(device=DEV).manual_seed(seed)
        need = sum(pages(n) for n in lens) + sum(pages(k) for k in keeps) + 5
        order = list(range(need))
        rng.shuffle(order)
        self.P = need
        mp, nmp = max(max(map(pages, lens)), 1), max(max(map(pages, keeps)), 1)
        self.bt = np.full((len(lens), mp), -7, dtype=np.int32)
        self.nbt = np.full((len(lens), nmp), -9, dtype=np.int32)
        for b, n in enumerate(lens):
            for i in range(pages(n)):
                self.bt[b, i] = order.pop()
        for b, k in enumerate(keeps):
            for i in range(min(pages(k), nmp)):
                self.nbt[b, i] = self.bt[b, i] if i < shared_pages else order.pop()
        self.fp8 = fp8
        if fp8:
            self.kv = torch.randint(0, 256, (need, PAGE, 576), dtype=torch.uint8, device=DEV, generator=g)
            self.scale = torch.rand((need, PAGE), device=DEV, generator=g)
        else:
            self.kv = torch.randint(-32768, 32767, (need, PAGE, 576), dtype=torch.int16, device=DEV,
                                    generator=g).view(torch.bfloat16)
            self.scale = None

    def rows(self):
        return self.kv.view(torch.uint8).reshape(self.P * PAGE, -1)

    def expect(self, kept):
        want, ws = self.rows().clone(), None if self.scale is None else self.scale.clone().view(-1)
        for b, at in enumerate(kept):
            if not at:
                continue
            src = torch.tensor([int(self.bt[b, t // PAGE]) * PAGE + t % PAGE for t in at], device=DEV)
            dst = torch.tensor([int(self.nbt[b, j // PAGE]) * PAGE + j % PAGE for j in range(len(at))],
                               device=DEV)
            want[dst] = self.rows()[src]
            if ws is not None:
                ws[dst] = self.scale.view(-1)[src]
        return want, ws


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def run(pool, lens, weights, keeps, firsts, recent, max_keep=None, **kw):
    width = max_keep or max(max(keeps), 1)
    kept = torch.full((len(lens), width), 12345, dtype=torch.int32, device=DEV)
    out = torch.full((len(lens), width), -77.0, device=DEV)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    r = mla.mla_cache_evict(pool.kv, i32(pool.bt.tolist()), i32(lens), weights, i32(keeps),
                            i32(pool.nbt.tolist()), keep_first=None if firsts is None else i32(firsts),
                            recent=recent, kv_scale=pool.scale, kept=kept, weights_out=out,
                            workspace=ws, **kw)
    assert r[1] is kept and r[2] is out and r[3] is ws
    return r


def check(pool, lens, weights, keeps, firsts, recent, **kw):
    w = weights.cpu()
    kept = [chosen(w[b], L, k, f, recent) for b, (L, k, f) in
            enumerate(zip(lens, keeps, firsts or [0] * len(lens)))]
    want, wscale = pool.expect(kept)
    new, got, out, ws = run(pool, lens, weights, keeps, firsts, recent, **kw)
    torch.cuda.synchronize()
    assert new.tolist() == [len(k) for k in kept]
    for b, k in enumerate(kept):
        assert got[b].tolist() == k + [-1] * (got.shape[1] - len(k)), b
        o = out[b].cpu()
        assert torch.equal(o[:len(k)].view(torch.int32), w[b, k].view(torch.int32))
        assert (o[len(k):] == -77.0).all()
    assert torch.equal(pool.rows(), want)
    if wscale is not None:
        assert torch.equal(pool.scale.view(-1).view(torch.int32), wscale.view(torch.int32))
    assert mla.mla_get_device_error(ws) == 0


def weights_of(kind, B, W, seed):
    g = torch.Generator(device=DEV).manual_seed(seed + 99)
    if kind == "tail":
        w = torch.exp(3 * torch.randn((B, W), device=DEV, generator=g) - 4)
        return torch.where(w < 0.01, torch.zeros_like(w), w)
    if kind == "equal":
        return torch.full((B, W), 0.25, device=DEV)
    if kind == "few":      # a handful of values, both zeros and signs among them
        v = torch.tensor([0.0, -0.0, 1.0, -1.0, 1.0000001, 3e38, 1e-45, -1e-45], device=DEV)
        return v[torch.randint(0, 8, (B, W), device=DEV, generator=g)]
    if kind == "odd":      # every bit pattern: NaN, infinities, subnormals
        return torch.randint(-2**31, 2**31 - 1, (B, W), device=DEV, generator=g,
                             dtype=torch.int32).view(torch.float32)
    if kind == "last":     # the largest are the last ones
        return torch.arange(W, device=DEV, dtype=torch.float32).expand(B, W).contiguous()
    raise KeyError(kind)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kind", ["tail", "equal", "few", "odd", "last"])
def test_kept_tokens_and_every_byte(kind, fp8):
    lens = [777, 64, 65, 1, 130, 500]
    keeps = [400, 63, 64, 1, 200, 0]
    firsts = [64, 0, 1, 5, 3, 4]
    pool = Pool(lens, keeps, fp8, seed=len(kind) + fp8)
    check(pool, lens, weights_of(kind, 6, max(lens), 3), keeps, firsts, 32)


@pytest.mark.parametrize("first,recent", [(0, 0), (0, 300), (300, 0), (250, 250), (499, 1), (1000, 1000)])
def test_windows_that_meet_the_budget(first, recent):
    lens, keeps = [640, 300, 501], [500, 299, 500]
    pool = Pool(lens, keeps, False, seed=first + recent)
    check(pool, lens, weights_of("tail", 3, 640, 5), keeps, [first] * 3, recent)


@pytest.mark.parametrize("kind", ["tail", "equal", "few", "odd", "last"])
def test_long_contexts_take_a_cluster(kind):
    lens, keeps = [20011, 8193, 9000, 3], [10007, 8192, 1, 3]
    pool = Pool(lens, keeps, True, seed=11)
    check(pool, lens, weights_of(kind, 4, max(lens), 7), keeps, [100, 0, 0, 0], 77)


@pytest.mark.parametrize("kind", ["tail", "equal", "few", "last", "comb up", "comb down"])
@pytest.mark.parametrize("L", [524288, 200003])
def test_selection_of_rows_too_long_for_registers(L, kind):
    """Weights whose every eighth group of 32 is nothing like the others among
    them: what a sample of such rows says of them is wrong."""
    if kind.startswith("comb"):
        t = torch.arange(L, device=DEV)
        w = torch.rand((1, L), device=DEV, generator=torch.Generator(device=DEV).manual_seed(5)) + 1
        w[0, ((t % 256) < 32) == (kind == "comb up")] *= 1000
    else:
        w = weights_of(kind, 1, L, 13)
    pages_old, bt = pages(L), torch.arange(pages(L), dtype=torch.int32, device=DEV)[None]
    order = torch.argsort(-w[0], stable=True)
    kv = torch.zeros((2 * pages_old, PAGE, 576), dtype=torch.uint8, device=DEV)
    scale = torch.arange(2 * pages_old * PAGE, device=DEV, dtype=torch.float32).view(-1, PAGE)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    for keep in (1, 1000, L // 4, L // 2 + 1, L - 1):
        new, kept, wk, _ = mla.mla_cache_evict(kv, bt, i32([L]), w, i32([keep]), bt + pages_old, kv_scale=scale,
                                               workspace=ws)
        want = order[:keep].sort().values
        torch.cuda.synchronize()
        assert mla.mla_get_device_error(ws) == 0 and new.tolist() == [keep]
        assert torch.equal(kept[0, :keep].long(), want) and (kept[0, keep:] == -1).all()
        assert torch.equal(wk[0, :keep], w[0, want])
        assert torch.equal(scale.view(-1)[pages_old * PAGE:][:keep].long(), want)


def test_a_long_tie_ends_at_the_right_token():
    # every weight equal: the kept ones are the first of the candidates
    L, keep = 70001, 50021
    pool = Pool([L], [keep], True, seed=2)
    check(pool, [L], weights_of("equal", 1, L, 0), [keep], [17], 1000)


def test_rows_of_a_wider_tensor_as_weights():
    lens, keeps = [200, 150, 99], [100, 100, 50]
    wide = weights_of("tail", 3, 1024, 9)
    pool = Pool(lens, keeps, False, seed=8)
    check(pool, lens, wide[:, 300:500], keeps, None, 8)


def test_shared_leading_pages_stay():
    # three kept pages are the same pages before and after, and not written
    lens, keeps = [700, 650], [400, 500]
    pool = Pool(lens, keeps, True, seed=4, shared_pages=3)
    check(pool, lens, weights_of("tail", 2, 700, 1), keeps, [192, 200], 10)


def test_a_page_that_would_be_overwritten_is_refused():
    # its fourth page keeps its place in the table but not its rows
    lens, keeps = [700], [400]
    pool = Pool(lens, keeps, False, seed=4, shared_pages=4)
    before = pool.rows().clone()
    w = weights_of("last", 1, 700, 1)
    kept = chosen(w[0].cpu(), 700, 400, 192, 10)
    want, _ = pool.expect([kept])
    fourth = int(pool.nbt[0, 3])
    want[fourth * PAGE:(fourth + 1) * PAGE] = before[fourth * PAGE:(fourth + 1) * PAGE]
    new, got, out, ws = run(pool, lens, w, keeps, [192], 10)
    assert mla.mla_get_device_error(ws) == -1
    assert torch.equal(pool.rows(), want) and got[0].tolist() == kept


def test_bad_pages_are_reported_and_their_rows_left():
    lens, keeps = [300, 300], [200, 200]
    pool = Pool(lens, keeps, True, seed=6)
    w = weights_of("tail", 2, 300, 2)
    kept = [chosen(w[b].cpu(), 300, 200, 0, 0) for b in range(2)]
    real = pool.bt.copy()
    before = pool.rows().clone()
    want, _ = pool.expect(kept)
    pool.bt[0, 2] = pool.P            # a source page
    lost = int(pool.nbt[1, 1])
    pool.nbt[1, 1] = -1               # a new page
    dst = [int(pool.nbt[0, j // PAGE]) * PAGE + j % PAGE for j, t in enumerate(kept[0]) if t // PAGE == 2]
    want[dst] = before[dst]
    want[lost * PAGE:(lost + 1) * PAGE] = before[lost * PAGE:(lost + 1) * PAGE]
    _, _, _, ws = run(pool, lens, w, keeps, None, 0)
    assert mla.mla_get_device_error(ws) == -5 and mla.mla_get_device_error(ws) == 0
    assert torch.equal(pool.rows(), want)


def test_lengths_out_of_range_are_clamped_and_reported():
    # a context beyond its weights, one beyond its table, one below 0, a budget
    # beyond kept and one below 0
    pool = Pool([128, 128, 64, 128, 128], [64] * 5, False, seed=3)
    w = weights_of("tail", 5, 256, 4)
    lens = [300, 200, -5, 100, 100]
    keeps = [64, 64, 64, 1000, -3]
    effective = [128, 128, 0, 100, 100]
    kept = [chosen(w[b].cpu(), L, max(0, min(k, 64)), 0, 4) for b, (L, k) in
            enumerate(zip(effective, keeps))]
    want, _ = pool.expect(kept)
    new, got, _, ws = run(pool, lens, w, keeps, None, 4, max_keep=64)
    assert new.tolist() == [len(k) for k in kept] and torch.equal(pool.rows(), want)
    assert mla.mla_get_device_error(ws) == -1


def test_replayed_on_another_stream_with_new_inputs():
    lens, keeps = [777, 300], [400, 150]
    w0 = weights_of("tail", 2, 777, 1)
    pool = Pool(lens, keeps, True, seed=5)
    sl, keep = i32(lens), i32(keeps)
    bt, nbt = i32(pool.bt.tolist()), i32(pool.nbt.tolist())
    kept = torch.zeros((2, 400), dtype=torch.int32, device=DEV)
    out = torch.zeros((2, 400), device=DEV)
    new = torch.zeros(2, dtype=torch.int32, device=DEV)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    s = torch.cuda.Stream()
    call = lambda: mla.mla_cache_evict(pool.kv, bt, sl, w0, keep, nbt, recent=16, kv_scale=pool.scale,
                                       kept=kept, new_seq_lens=new, weights_out=out, workspace=ws)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        call()
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            call()
    torch.cuda.synchronize()
    for seed in (2, 3):
        w0.copy_(weights_of("tail", 2, 777, seed))
        sl.copy_(i32([700 + seed, 200]))
        want_kept = [chosen(w0[b].cpu(), L, k, 0, 16) for b, (L, k) in
                     enumerate(zip([700 + seed, 200], keeps))]
        want, _ = pool.expect(want_kept)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            graph.replay()
        s.synchronize()
        assert [kept[b, :len(k)].tolist() for b, k in enumerate(want_kept)] == want_kept
        assert new.tolist() == [len(k) for k in want_kept] and torch.equal(pool.rows(), want)


def test_refusals_of_the_binding():
    lens, keeps = [200, 100], [100, 50]
    pool = Pool(lens, keeps, True, seed=5)
    w = weights_of("tail", 2, 200, 1)
    args = dict(kv=pool.kv, block_table=i32(pool.bt.tolist()), seq_lens=i32(lens), weights=w,
                keep=i32(keeps), new_block_table=i32(pool.nbt.tolist()), kv_scale=pool.scale)

    def refused(kind, **kw):
        with pytest.raises(kind):
            mla.mla_cache_evict(**{**args, **kw})

    before = pool.rows().clone()
    refused(ValueError, kv_scale=None)
    refused(TypeError, kv=pool.kv.half())
    refused(ValueError, weights=w[:1])
    refused(TypeError, weights=w.double())
    refused(ValueError, weights=w.t().contiguous().t())
    refused(TypeError, keep=i32(keeps).long())
    refused(ValueError, keep=i32(keeps).cpu())
    refused(ValueError, keep_first=i32([1]))
    refused(ValueError, block_table=args["block_table"][:1])
    refused(ValueError, weights_out=torch.zeros((2, 7), device=DEV))
    refused(mla.MLAError, recent=-1)
    refused(mla.MLAError, new_seq_lens=args["seq_lens"])
    refused(mla.MLAError, workspace=torch.zeros(128, dtype=torch.uint8, device=DEV))
    refused(mla.MLAError, kept=torch.zeros((2, 1000), dtype=torch.int32, device=DEV))
    flat = torch.zeros(2 * 200 + 128 * 2, device=DEV)
    refused(mla.MLAError, weights=flat[:400].view(2, 200), weights_out=flat[256:512].view(2, 128))
    torch.cuda.synchronize()
    assert torch.equal(pool.rows(), before)
