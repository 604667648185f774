"""Attention weights per cached token against the definition in 64 bits."""
import math
import random

import pytest
import torch

import sequence_sharded_mla_gb300 as mla

pytestmark = pytest.mark.gpu

PAGE, DEV = 64, "cuda"
SCALE = mla.DEFAULT_SCALE


class Step:
    """A step over random pages, its exact logits and log-sum-exps."""

    def __init__(self, lens, q_len=1, H=16, fp8=False, causal=True, q_lens=None, seed=0, width=None,
                 sigma=0.5):
        g = torch.Generator(device=DEV).manual_seed(seed)
        rng = random.Random(seed)
        self.lens, self.H, self.q_len, self.causal = lens, H, q_len, causal
        B = len(lens)
        self.new = q_lens or [q_len] * B
        self.q_lens = None if q_lens is None else torch.tensor(q_lens, dtype=torch.int32, device=DEV)
        need = [-(-n // PAGE) for n in lens]
        self.P = sum(need) + 3
        order = list(range(self.P))
        rng.shuffle(order)
        self.bt = torch.full((B, max(max(need), 1)), -1, dtype=torch.int32)
        for b, k in enumerate(need):
            for i in range(k):
                self.bt[b, i] = order.pop()
        self.q = (torch.randn((B, q_len, H, 576), device=DEV, generator=g) * sigma).to(torch.bfloat16)
        x = torch.randn((self.P, PAGE, 576), device=DEV, generator=g)
        if fp8:
            self.scale = torch.exp2(torch.randint(-9, -5, (self.P, PAGE), device=DEV, generator=g).float())
            self.kv = (x * 100).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            self.values = self.kv.view(torch.float8_e4m3fn).double() * self.scale.double()[..., None]
        else:
            self.scale = None
            self.kv = (x * sigma).to(torch.bfloat16)
            self.values = self.kv.double()
        self.seq = torch.tensor(lens, dtype=torch.int32, device=DEV)
        self.bt = self.bt.to(DEV)
        self.width = width or max(lens) + 9
        self.lse = torch.full((B, q_len, H), -math.inf, dtype=torch.float64, device=DEV)
        self.logits = []
        for b, L in enumerate(lens):
            rows = torch.arange(max(L, 0), device=DEV)
            K = self.values.view(-1, 576)[self.bt[b, rows // PAGE].long() * PAGE + rows % PAGE]
            a = torch.einsum("ihd,td->iht", self.q[b].double(), K) * SCALE
            i = torch.arange(q_len, device=DEV)[:, None]
            n = self.new[b]
            see = (rows[None] <= L - n + i) if causal else torch.ones((q_len, L), dtype=torch.bool, device=DEV)
            a.masked_fill_(~(see & (i < n))[:, None, :], -math.inf)
            self.logits.append(a)
            if L > 0:
                self.lse[b] = torch.logsumexp(a, -1)

    def expect(self, before, lse=None):
        """out for t < L, from the fp32 lse that the call gets."""
        l = (self.lse.float() if lse is None else lse).double()
        rows = []
        for b, L in enumerate(self.lens):
            at = torch.where(torch.isneginf(l[b]), torch.full_like(l[b], math.inf), l[b])[..., None]
            w = torch.exp(self.logits[b] - at).sum((0, 1))
            old = max(L - self.new[b], 0)
            if before is not None:
                w[:old] += before[b, :old].double()
            rows.append(w)
        return rows

    def call(self, **kw):
        kw.setdefault("lse", self.lse.float())
        return mla.mla_attention_weights(self.q, self.kv, self.bt, self.seq, kv_scale=self.scale,
                                         causal=self.causal, q_lens=self.q_lens, **kw)


# Error of a weight w = sum of e_k = exp(a_k - lse_k), each e_k <= 1:
#   fp32 accumulation of the logit over 576 products (tensor cores), relative
#   to sum |q||k| scale, about 576 * 0.25 * 0.072 = 10 of these tests' unit:
#     576 roundings of 2^-24 against 10 bounds |da| by 3.5e-4, and the ex2 and
#     log2 conversions (values up to 2^5, 2^-24 each) add below 1e-5;
#   e4m3 caches: the query's terms leave at most 2^-11 of s_r's unit (max|q|
#     is 2^7 of it or more, up to 2^2 here, so 2^-16 a component) against
#     |K| <= 448 2^-6 = 7 with rms 100 2^-7.5: 576 * 2^-16 * 0.55 * 0.072
#     bounds |da| by 3.5e-4 once more (the errors' signs are not all alike).
# So w is within 1e-3 of itself, its sum over rows likewise.
RTOL = 1e-3


def check(step, before=None, out=None, **kw):
    want = step.expect(before, kw.get("lse"))
    if out is None:
        out = torch.full((len(step.lens), step.width), -5.0, device=DEV)
    tail = out.clone()
    got, ws = step.call(weights=before, out=out, **kw)
    assert got is out
    torch.cuda.synchronize()
    assert mla.mla_get_device_error(ws) == 0
    for b, L in enumerate(step.lens):
        err = (got[b, :L].double() - want[b]).abs()
        assert (err <= RTOL * want[b].abs() + 1e-7).all(), (b, L, (err / (want[b].abs() + 1e-7)).max())
        assert torch.equal(got[b, L:], tail[b, L:])
    return got


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("H", [16, 64, 128])
def test_one_token_of_each_request(H, fp8):
    step = Step([1, 63, 64, 65, 127, 128, 129, 700], H=H, fp8=fp8, seed=H + fp8)
    g = check(step)
    # every row's weights sum to one
    for b, L in enumerate(step.lens):
        assert abs(g[b, :L].double().sum().item() - H) < 2e-3 * H


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("q_len,H", [(2, 16), (3, 48), (5, 64), (9, 64), (4, 128)])
@pytest.mark.parametrize("causal", [False, True])
def test_verify_steps_with_earlier_weights(q_len, H, fp8, causal):
    lens = [q_len, 64 + q_len, 128, 500, 129]
    step = Step(lens, q_len, H, fp8, causal, seed=q_len * H)
    check(step, torch.rand((5, step.width), device=DEV))


@pytest.mark.parametrize("fp8", [False, True])
def test_padded_batches(fp8):
    lens, new = [300, 129, 64, 7, 1000], [1, 5, 3, 2, 4]
    step = Step(lens, 5, 64, fp8, q_lens=new, seed=6)
    # a padding row's query may hold anything
    for b, n in enumerate(new):
        step.q[b, n:] = math.nan
    check(step, torch.rand((5, step.width), device=DEV))


def test_context_shorter_than_the_step():
    step = Step([2, 1, 130], 4, 32, seed=3)    # early queries see nothing
    assert torch.isneginf(step.lse[0, 0]).all()
    check(step, torch.rand((3, step.width), device=DEV))


def test_empty_contexts_and_more_units_than_ctas():
    lens = [0, 5] * 200 + [300]
    step = Step(lens, 1, 16, seed=9)
    check(step)


def test_in_place_on_rows_of_a_wider_tensor():
    step = Step([400, 100, 257], 2, 16, seed=4, width=500)
    wide = torch.rand((3, 1024), device=DEV)
    rest = wide.clone()
    view = wide[:, 100:600]
    before = view.clone()
    want = step.expect(before)
    out, _ = step.call(weights=view, out=view)
    torch.cuda.synchronize()
    for b, L in enumerate(step.lens):
        assert ((wide[b, 100:100 + L].double() - want[b]).abs() <= RTOL * want[b] + 1e-7).all()
        rest[b, 100:100 + L] = wide[b, 100:100 + L]
    assert torch.equal(rest, wide)


def test_new_tensor_has_zeros_behind():
    step = Step([70, 20], 1, 16, seed=4)
    out, ws = step.call()
    assert out.shape == (2, 128) and (out[0, 70:] == 0).all() and (out[1, 20:] == 0).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_long_contexts_over_many_ctas(fp8):
    step = Step([70001, 4097, 12], 1, 64, fp8, seed=8)
    check(step, torch.rand((3, step.width), device=DEV))


def test_nan_rows_past_the_context_do_not_matter_and_within_it_are_theirs():
    step = Step([100, 200], 1, 16, seed=2)
    page = int(step.bt[0, 1])
    step.kv[page, 36:] = math.nan              # behind request 0's context
    check(step)
    row = int(step.bt[1, 0])
    step.kv[row, 7, 3] = math.nan              # token 7 of request 1
    out, ws = step.call()
    torch.cuda.synchronize()
    assert torch.isnan(out[1, 7]) and not torch.isnan(out[1, :7]).any() and not torch.isnan(out[1, 8:]).any()
    assert not torch.isnan(out[0]).any()


def test_lse_of_the_step_itself():
    step = Step([900, 130], 2, 32, seed=12)
    o, lse, _ = mla.mla_decode_step(step.q, step.kv, step.bt, step.seq, 2, causal=True)
    # its log-sum-exps are within 1e-3 of exact: every weight within that, too
    got, _ = step.call(lse=lse)
    want = step.expect(None, lse)
    for b, L in enumerate(step.lens):
        assert ((got[b, :L].double() - want[b]).abs() <= RTOL * want[b] + 1e-7).all()
        assert abs(got[b, :L].sum().item() - 2 * 32) < 2e-3 * 64


def test_errors_and_clamps():
    step = Step([300, 200], 2, 16, fp8=True, q_lens=[2, 1], seed=7)
    real = step.bt.clone()
    step.bt[0, 1] = step.P
    out, ws = step.call()
    assert mla.mla_get_device_error(ws) == -5 and mla.mla_get_device_error(ws) == 0
    step.bt.copy_(real)
    step.q_lens[1] = 3
    out, ws = step.call()
    assert mla.mla_get_device_error(ws) == -1
    step.q_lens[1] = 1
    step.q[0, 1, 5, 9] = math.inf
    out, ws = step.call()
    assert mla.mla_get_device_error(ws) == -7
    step.q[0, 1, 5, 9] = 0
    step.q[1, 1] = math.inf                     # padding
    out, ws = step.call()
    assert mla.mla_get_device_error(ws) == 0
    narrow = torch.full((2, 250), -1.0, device=DEV)
    out, ws = step.call(out=narrow)             # request 0 has 300 tokens
    assert mla.mla_get_device_error(ws) == -1


def test_same_bits_again_and_in_a_graph_on_another_stream():
    step = Step([3000, 129, 64], 3, 64, seed=5)
    before = torch.rand((3, step.width), device=DEV)
    out = torch.zeros_like(before)
    lse = step.lse.float()
    ws = torch.zeros(mla.mla_attention_weights_workspace_size(3, 3, 64), dtype=torch.uint8, device=DEV)
    call = lambda: step.call(weights=before, out=out, lse=lse, workspace=ws)
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
    assert torch.equal(out, first)
    step.q.copy_(torch.randn_like(step.q.float()).to(torch.bfloat16) * 0.4)
    graph.replay()
    torch.cuda.synchronize()
    replayed = out.clone()
    call()
    torch.cuda.synchronize()
    assert torch.equal(out, replayed) and not torch.equal(out, first)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("q_len", [1, 9])
def test_waits_that_run_out_are_reported(q_len, fp8):
    step = Step([5000, 70], q_len, 16, fp8, seed=1)
    try:
        mla.mla_set_wait_budget_ns(2_000_000)
        mla.mla_set_withhold_query(True)
        _, ws = step.call()
        got = mla.mla_get_device_error(ws)
    finally:
        mla.mla_set_withhold_query(False)
        mla.mla_set_wait_budget_ns(0)
    assert got == -4
    check(step)


def test_refusals_of_the_binding():
    step = Step([100, 50], 1, 16, fp8=True, seed=1)
    lse = step.lse.float()
    with pytest.raises(ValueError):
        step.call(lse=lse[:1])
    with pytest.raises(TypeError):
        step.call(lse=lse.double())
    with pytest.raises(ValueError):
        step.call(weights=torch.zeros((2, 200), device=DEV), out=torch.zeros((2, 300), device=DEV))
    with pytest.raises(ValueError):
        step.call(out=torch.zeros((1, 300), device=DEV))
    with pytest.raises(ValueError):
        step.call(out=torch.zeros((300, 2), device=DEV).t())
    with pytest.raises(mla.MLAError):
        step.call(workspace=torch.zeros(512, dtype=torch.uint8, device=DEV))
    flat = torch.zeros(1000, device=DEV)
    with pytest.raises(mla.MLAError):
        step.call(weights=flat[:300].view(2, 150), out=flat[100:400].view(2, 150))
