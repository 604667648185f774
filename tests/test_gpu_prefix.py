"""Shared-prefix attention and its combine against attention in 64 bits."""
import math
import random

import numpy as np
import pytest
import torch

import sequence_sharded_mla_gb300 as mla

from _helpers import REL_OUT, TOL_LSE, TOL_OUT, check_close

pytestmark = pytest.mark.gpu

PAGE, DEV = 64, "cuda"
SCALE = mla.DEFAULT_SCALE


@pytest.fixture(autouse=True)
def share_whatever_can_be():
    mla.mla_set_prefix_sharing(True)
    yield
    mla.mla_set_prefix_sharing(False)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Batch:
    """Requests in groups: sizes[g] of them behind common[g] tokens, own[b]
    tokens of their own; pages in random places, unused rows NaN."""

    def __init__(self, sizes, common, own, q_len=1, H=16, fp8=False, causal=True, q_lens=None, seed=0,
                 sigma=0.5):
        rng = random.Random(seed)
        g = torch.Generator(device=DEV).manual_seed(seed)
        B = sum(sizes)
        assert len(own) == B
        self.group = [k for k, n in enumerate(sizes) for _ in range(n)]
        self.lens = [common[k] + o for k, o in zip(self.group, own)]
        self.H, self.q_len, self.causal, self.fp8 = H, q_len, causal, fp8
        self.new = q_lens or [q_len] * B
        self.q_lens = None if q_lens is None else i32(q_lens)
        self.common = common
        shared = [n // PAGE for n in common]
        need = [-(-L // PAGE) - shared[k] for L, k in zip(self.lens, self.group)]
        self.P = sum(shared) + sum(need) + 3
        order = list(range(self.P))
        rng.shuffle(order)
        first = [[order.pop() for _ in range(n)] for n in shared]
        self.bt = torch.full((B, max(max(-(-L // PAGE) for L in self.lens), 1)), -1, dtype=torch.int32)
        for b, k in enumerate(self.group):
            row = first[k] + [order.pop() for _ in range(need[b])]
            if row:
                self.bt[b, :len(row)] = torch.tensor(row, dtype=torch.int32)
        self.bt = self.bt.to(DEV)
        self.starts = i32(np.concatenate([[0], np.cumsum(sizes)]).tolist())
        self.prefix = i32(common)
        self.seq = i32(self.lens)
        self.q = (torch.randn((B, q_len, H, 576), device=DEV, generator=g) * sigma).to(torch.bfloat16)
        x = torch.randn((self.P, PAGE, 576), device=DEV, generator=g)
        if fp8:
            self.scale = (torch.rand((self.P, PAGE), device=DEV, generator=g) + 0.5) / 200
            self.kv = (x * 100).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            self.scale = None
            self.kv = (x * sigma).to(torch.bfloat16)
        # rows behind a context
        for b, L in enumerate(self.lens):
            if L % PAGE and L // PAGE >= shared[self.group[b]]:
                page = int(self.bt[b, L // PAGE])
                if fp8:
                    self.kv[page, L % PAGE:] = 0x7F
                    self.scale[page, L % PAGE:] = math.nan
                else:
                    self.kv[page, L % PAGE:] = math.nan

    def expect(self):
        B = len(self.lens)
        out = torch.zeros((B, self.q_len, self.H, 512), dtype=torch.float64, device=DEV)
        lse = torch.full((B, self.q_len, self.H), -math.inf, dtype=torch.float64, device=DEV)
        for b, L in enumerate(self.lens):
            t = torch.arange(L, device=DEV)
            rows = self.bt[b, t // PAGE].long() * PAGE + t % PAGE
            if self.fp8:
                K = self.kv.view(-1, 576)[rows].view(torch.float8_e4m3fn).double()
                K *= self.scale.view(-1)[rows].double()[:, None]
            else:
                K = self.kv.view(-1, 576)[rows].double()
            for i in range(self.new[b]):
                last = L - self.new[b] + i + 1 if self.causal else L
                if last <= 0:
                    continue
                a = torch.einsum("hd,td->ht", self.q[b, i].double(), K[:last]) * SCALE
                lse[b, i] = torch.logsumexp(a, -1)
                out[b, i] = torch.einsum("ht,td->hd", torch.exp(a - lse[b, i][:, None]), K[:last, :512])
        return out, lse

    def call(self, **kw):
        args = dict(group_starts=self.starts, prefix_lens=self.prefix, kv_scale=self.scale,
                    causal=self.causal, q_lens=self.q_lens)
        return mla.mla_prefix_partial(self.q, self.kv, self.bt, self.seq, **{**args, **kw})


def check(batch, error=0, want=None, **kw):
    ref, ref_lse = want or batch.expect()
    part, lse, ws = batch.call(**kw)
    out, lse_out = mla.mla_shard_combine(part, lse)
    torch.cuda.synchronize()
    assert mla.mla_get_device_error(ws) == error
    check_close(lse_out.cpu(), ref_lse.cpu(), TOL_LSE, "lse")
    check_close(out.float().cpu(), ref.cpu(), TOL_OUT, "out", rel=REL_OUT)
    return part, lse, ws


def in_slice_0(lse):
    """Requests whose rows have something in the shared slice."""
    return (~torch.isneginf(lse[0])).flatten(1).any(1).tolist()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("pages", [1, 2, 3, 4, 5, 9])
def test_few_shared_pages(pages, fp8):
    b = Batch([8], [PAGE * pages], [1, 2, 63, 64, 65, 100, 7, 130], H=16, fp8=fp8, seed=pages)
    part, lse, _ = check(b)
    assert all(in_slice_0(lse))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("B,H", [(2, 48), (5, 16), (9, 16), (3, 64), (2, 128), (7, 112), (40, 16)])
def test_rows_of_odd_counts(B, H, fp8):
    rng = random.Random(B * H)
    b = Batch([B], [700], [rng.randint(1, 200) for _ in range(B)], H=H, fp8=fp8, seed=B)
    part, lse, _ = check(b)
    assert all(in_slice_0(lse))


@pytest.mark.parametrize("fp8", [False, True])
def test_groups_of_odd_sizes_and_lengths(fp8):
    sizes = [1, 5, 1, 9, 2, 6]
    common = [500, 1000, 3, 129, 64, 4097]
    rng = random.Random(5)
    own = [rng.randint(1, 300) for _ in range(sum(sizes))]
    b = Batch(sizes, common, own, H=64, fp8=fp8, seed=3)
    part, lse, _ = check(b)
    got = in_slice_0(lse)
    assert got == [k != 2 for k in b.group]    # a prefix below a page


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("q_len", [2, 5, 9])
def test_verify_steps(q_len, causal, fp8):
    own = [q_len, q_len + 1, 64, 65, 100]
    b = Batch([2, 3], [640, 321], own, q_len, 32, fp8, causal, seed=q_len)
    check(b)


@pytest.mark.parametrize("fp8", [False, True])
def test_padded_batches(fp8):
    new = [1, 5, 3, 2, 5, 4]
    b = Batch([4, 2], [450, 1030], [5, 5, 64, 200, 70, 5], 5, 64, fp8, q_lens=new, seed=2)
    for r, n in enumerate(new):
        b.q[r, n:] = math.nan                  # may hold anything
    part, lse, ws = check(b)
    for r, n in enumerate(new):
        assert torch.isneginf(lse[:, r, n:]).all() and (part[:, r, n:] == 0).all()


def test_a_prefix_that_is_nearly_the_whole_context():
    # the step's own tokens lie inside the common ones: shared pages end before
    # the first query that would see only part of one
    b = Batch([4], [256], [3, 0, 1, 2], q_len=3, H=64, seed=1)
    part, lse, _ = check(b)
    b = Batch([4], [256], [0, 0, 0, 0], q_len=1, H=64, causal=False, seed=1)
    part, lse, _ = check(b)
    assert torch.isneginf(lse[1]).all() and (part[1] == 0).all()


def test_prefix_lengths_longer_than_the_contexts_or_negative():
    b = Batch([3, 3], [300, 200], [10, 20, 30, 5, 6, 7], H=64, seed=4)
    b.prefix = i32([310, -100])                # 310: the shortest context
    part, lse, _ = check(b)
    assert in_slice_0(lse) == [True] * 3 + [False] * 3


def test_empty_groups():
    b = Batch([3, 0, 4, 0], [300, 77, 130, 9], [1, 2, 3, 4, 5, 6, 7], H=64, seed=4)
    check(b)


@pytest.mark.parametrize("starts", [[0, 2, 5], [1, 2, 6], [0, 4, 3], [0, 7, 6], [0, -1, 6]])
def test_groups_that_are_no_ranges(starts):
    b = Batch([3, 3], [300, 200], [10, 20, 30, 5, 6, 7], H=64, seed=4)
    part, lse, _ = check(b, error=-1, group_starts=i32(starts))
    assert not any(in_slice_0(lse))


@pytest.mark.parametrize("fp8", [False, True])
def test_long_prefix_split_over_many_pairs(fp8):
    b = Batch([3, 2], [50000, 9001], [500, 64, 1, 30, 1000], H=64, fp8=fp8, seed=6)
    check(b)


@pytest.mark.parametrize("fp8", [False, True])
def test_many_units_of_few_tiles(fp8):
    n = 150
    rng = random.Random(1)
    sizes = [2] * n
    b = Batch(sizes, [64 + 64 * (i % 4) for i in range(n)], [rng.randint(1, 40) for _ in range(2 * n)],
              H=48, fp8=fp8, seed=6)
    check(b)


@pytest.mark.parametrize("fp8", [False, True])
def test_logits_that_grow_along_the_prefix(fp8):
    # the running maximum grows by far more than 2^8 tile after tile
    b = Batch([4], [1600], [40, 3, 70, 1], H=64, fp8=fp8, seed=9)
    pages = b.bt[0, :25].long()
    ramp = torch.linspace(0.05, 6.0, 25, device=DEV)
    if fp8:
        b.scale[pages] *= ramp[:, None]
    else:
        b.kv[pages] = (b.kv[pages].float() * ramp[:, None, None]).to(torch.bfloat16)
    b.q *= 4
    check(b)


def test_scales_of_any_magnitude():
    b = Batch([4], [900], [40, 3, 70, 1], H=64, fp8=True, seed=9)
    live = torch.zeros_like(b.scale, dtype=torch.bool)
    live[b.bt[0, :14].long()] = True
    g = torch.Generator(device=DEV).manual_seed(1)
    e = torch.randint(-40, 3, b.scale.shape, device=DEV, generator=g).float()
    b.scale = torch.where(live, torch.exp2(e) / 200, b.scale)
    b.scale[int(b.bt[0, 3]), 5] = 0
    check(b)


def test_a_nan_key_reaches_the_rows_that_see_it():
    b = Batch([3, 3], [300, 200], [10, 20, 30, 5, 6, 7], H=64, seed=4)
    ref, ref_lse = b.expect()
    b.kv[int(b.bt[0, 1]), 9, 100] = math.nan    # a shared page of group 0
    part, lse, _ = b.call()
    out, lse_out = mla.mla_shard_combine(part, lse)
    torch.cuda.synchronize()
    assert torch.isnan(lse_out[:3]).all() and torch.isnan(out[:3].float()).all()
    check_close(lse_out[3:].cpu(), ref_lse[3:].cpu(), TOL_LSE, "lse")
    check_close(out[3:].float().cpu(), ref[3:].cpu(), TOL_OUT, "out", rel=REL_OUT)


def test_bad_pages_and_long_contexts_are_reported():
    b = Batch([4], [640], [40, 3, 70, 1], H=64, seed=4)
    real = b.bt.clone()
    b.bt[0, 3] = b.P                            # the table row that the prefix is read by
    _, _, ws = b.call()
    assert mla.mla_get_device_error(ws) == -5 and mla.mla_get_device_error(ws) == 0
    b.bt.copy_(real)
    want = b.expect()
    b.bt[1, 3] = -4                             # not read: shared pages come from the first row
    check(b, want=want)
    b.bt.copy_(real)
    b.bt[2, 11] = -1                            # an own page
    _, _, ws = b.call()
    assert mla.mla_get_device_error(ws) == -5
    b.bt.copy_(real)
    b.seq[2] = 64 * b.bt.shape[1] + 1
    _, _, ws = b.call()
    assert mla.mla_get_device_error(ws) == -5


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("share", [True, False])
def test_contexts_longer_than_their_table_are_cut_alike(share, fp8):
    # what a row sees does not hang on what is shared: the context ends at the
    # table's end, and with it the rows of a causal step
    b = Batch([4], [640], [0, 0, 0, 0], q_len=5, H=64, fp8=fp8, seed=4)
    want = b.expect()
    b.prefix = i32([900])
    for seq in ([740] * 4, [645, 640, 1 << 30, 640]):
        b.seq = i32(seq)
        mla.mla_set_prefix_sharing(share)
        _, lse, _ = check(b, error=-5, want=want)
        assert all(in_slice_0(lse)) == share


def test_infinite_query_over_an_e4m3_prefix():
    b = Batch([4], [640], [40, 3, 70, 1], q_len=2, H=64, fp8=True, q_lens=[2, 1, 2, 1], seed=4)
    b.q[1, 1] = math.inf                        # padding
    check(b)
    b.q[2, 1, 7, 33] = math.inf
    _, _, ws = b.call()
    assert mla.mla_get_device_error(ws) == -7


def test_with_the_value_projection():
    b = Batch([5, 3], [700, 300], [10, 20, 30, 40, 50, 60, 70, 80], H=16, seed=14)
    ref, _ = b.expect()
    g = torch.Generator(device=DEV).manual_seed(3)
    w = (torch.randn((16, 512, 128), device=DEV, generator=g) * 0.02).to(torch.bfloat16)
    part, lse, _ = b.call()
    y, _ = mla.mla_shard_combine(part, lse, w_uv=w)
    want = torch.einsum("bihd,hdo->biho", ref, w.double())
    check_close(y.float().cpu(), want.cpu(), TOL_OUT, "y", rel=REL_OUT)


@pytest.mark.parametrize("fp8", [False, True])
def test_same_bits_again_and_in_a_graph_on_another_stream(fp8):
    b = Batch([6, 3], [5000, 700], [10, 20, 30, 40, 50, 60, 70, 80, 90], H=64, fp8=fp8, seed=14)
    shape = (2, 9, 1, 64)
    out = torch.zeros(shape + (512,), device=DEV)
    lse = torch.zeros(shape, device=DEV)
    size = mla.mla_prefix_workspace_size(9, 1, 64, 2, b.bt.shape[1], fp8=fp8)
    ws = torch.full((size,), 0xEE, dtype=torch.uint8, device=DEV)      # anything
    call = lambda: b.call(out_partial=out, lse_partial=lse, workspace=ws)
    call()
    first = out.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            call()
        for _ in range(3):
            out.zero_()
            graph.replay()
        s.synchronize()
    assert torch.equal(out, first) and mla.mla_get_device_error(ws) == 0
    # other lengths, prefixes and queries in the same buffers
    b.q.copy_(b.q.flip(0))
    b.prefix.copy_(i32([2000, 650]))
    b.seq.sub_(3)
    b.lens = [n - 3 for n in b.lens]
    graph.replay()
    torch.cuda.synchronize()
    ref, ref_lse = b.expect()
    o, l = mla.mla_shard_combine(out, lse)
    check_close(l.cpu(), ref_lse.cpu(), TOL_LSE, "lse")
    check_close(o.float().cpu(), ref.cpu(), TOL_OUT, "out", rel=REL_OUT)


def test_outputs_at_16_byte_addresses():
    b = Batch([4], [640], [40, 3, 70, 1], H=64, seed=4)
    flat = torch.zeros(2 * 4 * 64 * 513 + 16, device=DEV)
    out = flat[4:4 + 2 * 4 * 64 * 512].view(2, 4, 1, 64, 512)
    lse = flat[8 + 2 * 4 * 64 * 512:8 + 2 * 4 * 64 * 513].view(2, 4, 1, 64)
    check(b, out_partial=out, lse_partial=lse)


@pytest.mark.parametrize("fp8", [False, True])
def test_waits_that_run_out_are_reported_and_leave_the_gpu_usable(fp8):
    # the query rows that both CTAs of a pair wait for never come
    b = Batch([4], [64 * 40], [40, 3, 70, 1], H=64, fp8=fp8, seed=4)
    want = b.expect()
    try:
        mla.mla_set_wait_budget_ns(2_000_000)
        mla.mla_set_withhold_query(True)
        _, _, ws = b.call()
        got = mla.mla_get_device_error(ws)
    finally:
        mla.mla_set_withhold_query(False)
        mla.mla_set_wait_budget_ns(0)
    assert got == -4
    check(b, want=want)


def test_a_step_with_weights_and_eviction():
    """The calls together: attend behind a shared prefix, weigh the tokens, cut
    the contexts, attend what is left."""
    b = Batch([4], [640], [300, 120, 70, 260], H=64, seed=21)
    part, lse, _ = check(b)
    _, lse_out = mla.mla_shard_combine(part, lse)
    w, ws = mla.mla_attention_weights(b.q, b.kv, b.bt, b.seq, lse_out, causal=True)
    for r, L in enumerate(b.lens):
        assert abs(w[r, :L].double().sum().item() - 64) < 0.2
    keeps = [800, 760, 705, 800]
    free = i32([b.P + k for k in range(4 * 3)]).view(4, 3)
    pool = torch.cat((b.kv, torch.zeros((12, PAGE, 576), dtype=torch.bfloat16, device=DEV)))
    nbt = torch.cat((b.bt[:, :10], free), 1).contiguous()       # the prefix's pages stay
    new, kept, wk, ews = mla.mla_cache_evict(pool, b.bt, b.seq, w, i32(keeps), nbt, keep_first=i32([640] * 4),
                                             recent=16)
    torch.cuda.synchronize()
    assert mla.mla_get_device_error(ews) == 0 and new.tolist() == [800, 760, 705, 800]
    # the new contexts hold the kept rows
    before = [b.kv.view(-1, 576)[b.bt[r, kept[r, :n].long() // 64].long() * 64 + kept[r, :n].long() % 64]
              for r, n in enumerate(keeps)]
    b.kv, b.bt, b.seq, b.lens, b.P = pool, nbt, new, new.tolist(), b.P + 12
    for r, n in enumerate(keeps):
        t = torch.arange(n, device=DEV)
        assert torch.equal(pool.view(-1, 576)[nbt[r, t // 64].long() * 64 + t % 64].view(torch.int16),
                           before[r].view(torch.int16))
    check(b)


@pytest.mark.parametrize("fp8", [False, True])
def test_pages_whose_offsets_pass_32_bits(fp8):
    """The same pages at the end of a pool of more than 4 GB: the same bits."""
    far = (1 << 32) // (PAGE * 576) + 64
    b = Batch([3], [320], [200, 77, 130], H=64, seed=22, fp8=fp8)
    n, w0 = b.P, torch.rand((3, b.bt.shape[1] * PAGE), device=DEV)
    free = i32([b.P + k for k in range(3 * 4)]).view(3, 4)

    def steps(kv, scale, at):
        table = torch.where(b.bt >= 0, b.bt + at, b.bt)
        part, lse, ws = mla.mla_prefix_partial(b.q, kv, table, b.seq, b.starts, b.prefix, kv_scale=scale,
                                               causal=True)
        _, lse_out = mla.mla_shard_combine(part, lse)
        w, wws = mla.mla_attention_weights(b.q, kv, table, b.seq, lse_out, w0, torch.zeros_like(w0),
                                           kv_scale=scale, causal=True)
        new, kept, wk, ews = mla.mla_cache_evict(kv, table, b.seq, w, i32([200, 256, 130]), free + at,
                                                 recent=8, kv_scale=scale,
                                                 weights_out=torch.zeros((3, 256), device=DEV))
        torch.cuda.synchronize()
        assert [mla.mla_get_device_error(x) for x in (ws, wws, ews)] == [0, 0, 0]
        rows = kv[at + n:at + n + 12].reshape(3, -1, 576)
        moved = [rows[r, :k].clone().view(torch.uint8) for r, k in enumerate((200, 256, 130))]
        scales = [] if scale is None else [scale[at + n:at + n + 12].reshape(3, -1)[r, :k].clone()
                                           for r, k in enumerate((200, 256, 130))]
        return [part, lse, w, new, kept, wk] + moved + scales

    kv = torch.zeros((far + n + 12, PAGE, 576), dtype=b.kv.dtype, device=DEV)
    scale = None if b.scale is None else torch.zeros((far + n + 12, PAGE), device=DEV)
    got = []
    for at in (0, far):
        kv[at:at + n] = b.kv
        if fp8:
            scale[at:at + n] = b.scale
        got.append(steps(kv, scale, at))
    for x, y in zip(*got):
        assert torch.equal(x, y)


@pytest.mark.parametrize("fp8", [False, True])
def test_sharing_where_it_takes_less_time(fp8):
    # many rows behind a long prefix share it; a few behind a short one, and a
    # request alone, do not
    mla.mla_set_prefix_sharing(False)
    own = [5 + 7 * i for i in range(33)]
    b = Batch([32, 1], [9000, 3000], own, H=64, fp8=fp8, seed=2)
    _, lse, _ = check(b)
    assert in_slice_0(lse) == [True] * 32 + [False]
    b = Batch([4], [1000], own[:4], H=64, fp8=fp8, seed=2)
    _, lse, _ = check(b)
    assert not any(in_slice_0(lse))


@pytest.mark.parametrize("fp8", [False, True])
def test_few_rows_behind_a_long_prefix_share_it_too(fp8):
    mla.mla_set_prefix_sharing(False)
    b = Batch([4], [40000], [5, 1, 70, 200], H=16, fp8=fp8, seed=2)
    _, lse, _ = check(b)
    assert all(in_slice_0(lse))


@pytest.mark.parametrize("fp8", [False, True])
def test_padded_requests_side_by_side_in_a_tile(fp8):
    # 128-row tiles hold rows of many requests, with gaps of padding between
    rng = random.Random(8)
    new = [rng.randint(1, 4) for _ in range(40)]
    b = Batch([23, 17], [700, 333], [4 + rng.randint(0, 90) for _ in range(40)], 4, 16, fp8, q_lens=new,
              seed=8)
    for r, n in enumerate(new):
        b.q[r, n:] = math.inf
    part, lse, _ = check(b)
    for r, n in enumerate(new):
        assert torch.isneginf(lse[:, r, n:]).all() and (part[:, r, n:] == 0).all()
        assert not torch.isneginf(lse[0, r, :n]).any()


def test_refusals_of_the_binding():
    b = Batch([2, 2], [100, 70], [1, 2, 3, 4], H=16, fp8=True, seed=1)
    with pytest.raises(ValueError):
        b.call(group_starts=b.starts[:2].contiguous())
    with pytest.raises(TypeError):
        b.call(prefix_lens=b.prefix.long())
    with pytest.raises(ValueError):
        b.call(out_partial=torch.zeros((1, 4, 1, 16, 512), device=DEV))
    with pytest.raises(ValueError):
        b.call(kv_scale=None)
    with pytest.raises(mla.MLAError):
        b.call(workspace=torch.zeros(4096, dtype=torch.uint8, device=DEV))
    with pytest.raises(mla.MLAError):                # more groups than requests
        b.call(group_starts=i32([0, 1, 2, 3, 4, 4]), prefix_lens=i32([1, 1, 1, 1, 1]))
