"""e4m3 caches whose attention has a heavy token and a long flat tail: what a
tail weighs in all must not be lost because each of its tokens weighs little."""
import math

import pytest
import torch

import sequence_sharded_mla_gb300 as mla

pytestmark = pytest.mark.gpu

PAGE, DEV, ROPE = 64, "cuda", slice(512, 576)
SCALE = mla.DEFAULT_SCALE
# What the kernels' probabilities may be off by.  Codes are at most VMAX = 80 and
# a tail's scales lie in one binade, (2^-7, 2^-6), so that a tile's weights P' =
# 2^(b - ref) mant (mant >= 1/2) are alike but for mant and the logits' spread.
#   A tile of the tail has its largest b at ref - 2 or above: every P' of it is at
#   least 2^-3 e^-2d (d: the spread of its logits), and a sum of two e4m3 terms is
#   off by at most 2^-9 there, 2^-6 e^2d of itself; 2^-8 from 2^-1 up.  Values are
#   at most 80 / 64, all errors of one sign at worst.
#   In the heavy token's own tile the other 127 are off by 2^-9 each, codes of 80,
#   where the heavy token has b = ref + 5 or above and so, with its exponent of
#   -5, a weight of 2^10 or above in the same units: 127 * 2^-9 * 80 / 2^10.
def tolerance(d, heavy):
    return 2.0 ** -6 * math.exp(2 * d) * 80 / 64 + heavy * 127 * 2.0 ** -9 * 80 / 2 ** 10


class Cache:
    """n tokens of logits near 0 and values near 0.9, in pages of random order;
    `heavy` maps positions to the logits of rows whose values are `value`."""

    def __init__(self, n, heavy, value=0.0, seed=0, spare=2):
        g = torch.Generator(device=DEV).manual_seed(seed)
        pages = -(-n // PAGE)
        P = pages + spare
        self.n = n
        codes = torch.zeros((P * PAGE, 576), device=DEV)
        codes[:, :512] = 64 + 32 * (torch.rand((P * PAGE, 512), device=DEV, generator=g) - 0.5)
        scale = 1 / (66 + 54 * torch.rand(P * PAGE, device=DEV, generator=g))
        order = torch.randperm(P, device=DEV, generator=g)[:pages]
        self.table = order.to(torch.int32)[None].contiguous()
        self.rows = (order[:, None] * PAGE + torch.arange(PAGE, device=DEV)).flatten()[:n]
        self.top = max(abs(x) for x in heavy.values())
        for at, logit in heavy.items():
            r = self.rows[at]
            scale[r] = 1 / 64
            codes[r, :512] = 64 * value
            codes[r, ROPE] = 64 * logit / self.top
        self.kv = codes.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).view(P, PAGE, 576)
        self.scale = scale.view(P, PAGE).contiguous()
        self.g = g

    def query(self, B, q_len, H):
        q = torch.randn((B, q_len, H, 576), device=DEV, generator=self.g) * 0.01
        q[..., ROPE] = self.top / (64 * SCALE)
        return q.to(torch.bfloat16)

    def tokens(self, n=None):
        r = self.rows[:n]
        return self.kv.view(-1, 576)[r].view(torch.float8_e4m3fn).double() * self.scale.view(-1)[r].double()[:, None]


def expect(q, K):
    """Outputs and log-sum-exps of rows [.., 576] over tokens K, in 64 bits."""
    flat = q.double().reshape(-1, 576)
    out, lse = [], []
    for r in flat.split(16):
        a = r @ K.t() * SCALE
        lse.append(torch.logsumexp(a, -1))
        out.append(torch.exp(a - lse[-1][:, None]) @ K[:, :512])
    return torch.cat(out).view(q.shape[:-1] + (512,)), torch.cat(lse).view(q.shape[:-1])


def spread(q, K):
    """Half the range of the logits that are no heavy token's."""
    a = q.double().reshape(-1, 576) @ K[K[:, ROPE].abs().sum(1) == 0].t() * SCALE
    return float((a.amax(1) - a.amin(1)).max()) / 2


def close(out, lse, q, K, heavy=1):
    ref, ref_lse = expect(q, K)
    assert torch.isfinite(out.float()).all()
    d = spread(q, K)
    assert d < 0.1
    err = (out.double() - ref).abs().max().item()
    assert err <= tolerance(d, heavy), f"{err:.4f} > {tolerance(d, heavy):.4f}"
    # sums are of weights that are not rounded
    assert (lse.double() - ref_lse).abs().max().item() <= 1e-3


CASES = [(16384, {0: 11.0}, 0.0), (65536, {0: 11.0}, 0.0), (65536, {0: 11.0}, -1.0), (65536, {0: 8.0}, 0.0),
         (16384, {5000: 11.0}, 0.5), (16384, {16383: 11.0}, 0.0), (65536, {17: 11.5, 30000: 12.0}, 0.0),
         (8192, {0: 8.0, 3000: -40.0}, 0.0), (12800, {0: 12.0, 128: 9.0, 6000: 10.0, 12000: -12.0}, 0.0)]
# rows enough for every SM to walk through whole contexts: a tail in other pieces
# than the heavy token's has a reference of its own
B, Q, H = 10, 8, 128


def some(x):
    """Rows of all requests, query tokens and units."""
    return x[:, ::3, 5::24].contiguous()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def prefix_call(c, q, own):
    """Slice 0 of the batch behind the n tokens, `own` pages of their own."""
    used = set(c.table[0].tolist())
    free = [p for p in range(c.kv.shape[0]) if p not in used]
    table = torch.cat((c.table.expand(q.shape[0], -1), i32(free[:q.shape[0] * own]).view(-1, own)), 1)
    mla.mla_set_prefix_sharing(True)
    try:
        part, lse, ws = mla.mla_prefix_partial(q, c.kv, table.contiguous(), i32([c.n + 40] * q.shape[0]),
                                               i32([0, q.shape[0]]), i32([c.n]), kv_scale=c.scale, causal=True)
    finally:
        mla.mla_set_prefix_sharing(False)
    assert mla.mla_get_device_error(ws) == 0
    return part[0], lse[0]


@pytest.mark.parametrize("n,heavy,value", CASES)
def test_shared_prefix(n, heavy, value):
    c = Cache(n, heavy, value, spare=B + 2, seed=n)
    q = c.query(B, Q, H)
    part, lse = prefix_call(c, q, 1)
    close(some(part), some(lse), some(q), c.tokens(), len(heavy))


def test_shared_prefix_far_below_its_first_token():
    # nothing overflows where the tail is 2^-1400 of the first token, and what
    # weighs nothing adds nothing
    c = Cache(4096, {0: 970.0}, 0.5, spare=B + 2)
    part, lse = prefix_call(c, c.query(B, Q, H), 1)
    assert (part.double() - 0.5).abs().max().item() <= 2.0 ** -8


def decode(c, q, shards=1, layout="interleaved", seq=None, **kw):
    table = c.table.expand(q.shape[0], -1).contiguous()
    seq = i32([c.n] * q.shape[0]) if seq is None else seq
    part, lse, ws = mla.mla_decode_partial(q, c.kv, table, seq, shards, layout, kv_scale=c.scale, **kw)
    out, lse_out = mla.mla_shard_combine(part, lse)
    assert mla.mla_get_device_error(ws) == 0
    return (part[0], lse[0]) if shards == 1 else (out, lse_out)


@pytest.mark.parametrize("n,heavy,value", CASES)
def test_per_request(n, heavy, value):
    c = Cache(n, heavy, value, seed=n)
    q = c.query(B, Q, H)
    part, lse = decode(c, q)
    close(some(part), some(lse), some(q), c.tokens(), len(heavy))


@pytest.mark.parametrize("layout", ["interleaved", "contiguous"])
def test_a_sharded_step(layout):
    # four shards of 40 requests; the combine's output is rounded to bf16
    c = Cache(20000, {0: 11.0, 7000: 10.0}, 0.0, seed=1)
    q = c.query(40, 1, H)
    out, lse, ws = mla.mla_decode_step(q, c.kv, c.table.expand(40, -1).contiguous(), i32([c.n] * 40), 4, layout,
                                       kv_scale=c.scale)
    assert mla.mla_get_device_error(ws) == 0
    q, out, lse = (x[:, :, ::24].contiguous() for x in (q, out, lse))
    close(out, lse, q, c.tokens(), 2)


def test_per_request_far_below_its_first_token():
    c = Cache(4096, {0: 970.0}, 0.5)
    part, lse = decode(c, c.query(B, Q, H))
    assert (part.double() - 0.5).abs().max().item() <= 2.0 ** -8


def test_masks_that_cut_the_tail():
    # each query token of a causal step sees its own share of the tail, which
    # starts inside a tile; the padding rows' requests see nothing
    c = Cache(16389, {0: 11.0}, 0.0, seed=3)
    q = c.query(B, Q, H)
    new = [8, 1, 3, 8, 5, 2, 8, 7, 4, 6]
    part, lse = decode(c, q, causal=True, q_lens=i32(new))
    K = c.tokens()
    for b in (1, 2, 4):
        for i in range(new[b]):
            last = c.n - new[b] + i + 1
            close(part[b, i, 5::24], lse[b, i, 5::24], q[b, i, 5::24], K[:last])
        assert (part[b, new[b]:] == 0).all() and torch.isneginf(lse[b, new[b]:]).all()


def test_logits_of_three_nats_deviation():
    # wide logits without a heavy token: tiles' maxima go up and down by 2^10.
    # Values are independent and of mean 0, so |O| is |v| sqrt(sum p^2), and weights
    # off by 2^-8 of themselves at most turn it by 2^-8 of that; as much again for
    # the smaller ones of every tile.
    g = torch.Generator(device=DEV).manual_seed(5)
    c = Cache(16384, {0: 1.0}, 0.5, seed=5)
    x = torch.randn(c.kv.shape, device=DEV, generator=g) * 100
    c.kv = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    K = c.tokens()
    q = torch.randn((B, Q, H, 576), device=DEV, generator=g)
    q = (q * (3 / (SCALE * K.std() * math.sqrt(576)))).to(torch.bfloat16)
    part, lse = decode(c, q)
    part, lse, q = some(part), some(lse), some(q)
    ref, ref_lse = expect(q, K)
    assert ((part.double() - ref).norm(dim=-1) / ref.norm(dim=-1)).max().item() <= 2.0 ** -7
    assert (lse.double() - ref_lse).abs().max().item() <= 1e-3


def test_a_step_behind_a_shared_prefix_is_the_step_alone():
    # whole contexts, the heavy token in the shared part: both calls' outputs are
    # rounded to bf16 (2^-8 of values of up to 80 / 64) on top
    c = Cache(20032, {100: 10.0}, 0.0, spare=B + 2, seed=6)
    q = c.query(B, Q, H)
    used = set(c.table[0].tolist())
    own = i32([p for p in range(c.kv.shape[0]) if p not in used][:B])
    table = torch.cat((c.table.expand(B, -1), own[:, None]), 1).contiguous()
    seq = i32([c.n + 9 + 5 * b for b in range(B)])
    part, plse, ws = mla.mla_prefix_partial(q, c.kv, table, seq, i32([0, B]), i32([c.n]), kv_scale=c.scale)
    assert mla.mla_get_device_error(ws) == 0 and not torch.isneginf(plse[0]).any()
    both = [mla.mla_shard_combine(part, plse),
            mla.mla_decode_step(q, c.kv, table, seq, 1, kv_scale=c.scale)[:2]]
    for b in (0, 4, 9):
        rows = torch.cat((c.rows, own[b].long() * PAGE + torch.arange(int(seq[b]) - c.n, device=DEV)))
        K = c.kv.view(-1, 576)[rows].view(torch.float8_e4m3fn).double() * c.scale.view(-1)[rows].double()[:, None]
        x = q[b, ::3, 5::24].contiguous()
        ref, ref_lse = expect(x, K)
        for out, lse in both:
            err = (out[b, ::3, 5::24].double() - ref).abs().max().item()
            assert err <= tolerance(spread(x, K), 1) + 2.0 ** -8 * 80 / 64
            assert (lse[b, ::3, 5::24].double() - ref_lse).abs().max().item() <= 1e-3
