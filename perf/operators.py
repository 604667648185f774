"""Measured cases of the rotary, cache-append and 8-bit grouped-query operators.

Three operators that follow one another in a layer's decode step:

  rotate   rotary positions on query heads (whole head or part of it, both
           pair layouts, scaled frequencies)
  append   the new tokens' rotary positions, quantisation and paged write, for
           the latent cache (MLA) and the K/V caches (GQA), the query rotated
           in the same call
  attend   grouped-query attention over an e4m3 cache with a scale for each
           block of tokens and KV head, and the LSE combine of its shards

`run` computes them in elementary torch operations, or with the framework's
calls where `own` is true.
"""
import math
import random

import torch

own = False

PAGE = 64
FP8 = torch.float8_e4m3fn
DEV = "cuda"


# --------------------------------------------------------------------- cases
def listed():
    return [
        # a verify step of 16 requests, 9 tokens each, 64 absorbed latent query
        # heads: the 64 rope dims behind the 512 latent ones
        dict(name="rotate-latent-q9", op="rotate", batch=16, q_len=9, heads=64, dim=576, first=512,
             rot=64, interleaved=True, scaling="yarn", min_len=8000, max_len=8000, mix=1, ragged=False),
        # the query heads of a prompt chunk of odd length near the end of a
        # 128k context
        dict(name="rotate-chunk", op="rotate", batch=1, q_len=8191, heads=64, dim=128, first=0,
             rot=128, interleaved=False, scaling="none", min_len=131072, max_len=131072, mix=2,
             ragged=False),
        # one decode token of each of 32 requests into 4 KV heads, 64 query heads
        dict(name="append-decode-fp8", op="append_gqa", fp8=True, batch=32, q_len=1, heads=64,
             kv_heads=4, block=64, rot=128, interleaved=False, scaling="linear", min_len=500,
             max_len=9000, mix=3, ragged=False),
        # a prompt chunk of two requests into 8 KV heads, no query
        dict(name="append-chunk-fp8", op="append_gqa", fp8=True, batch=2, q_len=4099, heads=0,
             kv_heads=8, block=32, rot=64, interleaved=True, scaling="none", min_len=4099,
             max_len=20000, mix=4, ragged=True),
        # the bf16 caches of a ragged verify step
        dict(name="append-verify-bf16", op="append_gqa", fp8=False, batch=16, q_len=9, heads=64,
             kv_heads=8, block=64, rot=128, interleaved=False, scaling="none", min_len=100,
             max_len=9000, mix=5, ragged=True),
        # one token of each of 64 requests into the fp8 latent cache, 64 heads
        dict(name="append-latent-fp8", op="append_mla", fp8=True, batch=64, q_len=1, heads=64,
             rot=64, interleaved=True, scaling="yarn", min_len=1000, max_len=8000, mix=6,
             ragged=False),
        # a prompt chunk into the bf16 latent cache
        dict(name="append-latent-chunk-bf16", op="append_mla", fp8=False, batch=1, q_len=2053,
             heads=0, rot=64, interleaved=True, scaling="none", min_len=30000, max_len=30000, mix=7,
             ragged=False),
        # one short request: latency
        dict(name="attend-one-short", op="attend", batch=1, q_len=1, heads=16, kv_heads=4, block=64,
             shards=2, layout="interleaved", min_len=1024, max_len=1024, mix=8, ragged=False),
        # a decode batch of 32 requests, 64 heads over 4 KV heads
        dict(name="attend-batch", op="attend", batch=32, q_len=1, heads=64, kv_heads=4, block=64,
             shards=2, layout="interleaved", min_len=4000, max_len=65536, mix=9, ragged=False),
        # a ragged causal verify step of 16 requests
        dict(name="attend-verify-q9", op="attend", batch=16, q_len=9, heads=64, kv_heads=8, block=32,
             shards=2, layout="contiguous", min_len=5000, max_len=8000, mix=10, ragged=True),
        # seven short requests of odd lengths, every query head with its own KV head
        dict(name="attend-ragged-g1", op="attend", batch=7, q_len=1, heads=8, kv_heads=8, block=16,
             shards=1, layout="interleaved", min_len=1, max_len=5000, mix=11, ragged=False),
        # one request of a million tokens over 8 KV heads and 8 shards
        dict(name="attend-long", op="attend", batch=1, q_len=1, heads=64, kv_heads=8, block=64,
             shards=8, layout="interleaved", min_len=1048576, max_len=1048576, mix=12, ragged=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotate", "append_gqa", "append_gqa", "append_mla", "attend", "attend", "attend"])
    lo = _log(rng, 1, 20000)
    hi = min(max(lo, _log(rng, 16, 200000)), 200000)
    c = dict(op=op, min_len=lo, max_len=hi, mix=rng.randrange(1 << 30), ragged=rng.random() < 0.5)
    scaling = rng.choice(["none", "linear", "yarn"])
    if op == "rotate":
        wide = rng.random() < 0.5
        q_len = rng.choice([1, rng.randint(2, 9), _log(rng, 16, 4000)])
        batch = max(1, min(_log(rng, 1, 64), 4000 // q_len))
        c |= dict(batch=batch, q_len=q_len, heads=rng.choice([1, 8, 16, 24, 64]),
                  dim=576 if wide else 128, first=512 if wide else 0,
                  rot=64 if wide else rng.choice([32, 64, 96, 128]),
                  interleaved=rng.random() < 0.5, scaling=scaling)
    elif op == "append_gqa":
        q_len = rng.choice([1, rng.randint(2, 9), _log(rng, 16, 3000)])
        batch = max(1, min(_log(rng, 1, 64), 4000 // q_len))
        kv = rng.choice([1, 2, 4, 8])
        c |= dict(fp8=rng.random() < 0.7, batch=batch, q_len=q_len,
                  heads=rng.choice([0, kv * rng.choice([1, 2, 5, 8])]), kv_heads=kv,
                  block=rng.choice([16, 32, 64]), rot=rng.choice([32, 64, 96, 128]),
                  interleaved=rng.random() < 0.5, scaling=scaling)
        c["max_len"] = min(c["max_len"], 16000)
    elif op == "append_mla":
        q_len = rng.choice([1, rng.randint(2, 9), _log(rng, 16, 1500)])
        batch = max(1, min(_log(rng, 1, 64), 2000 // q_len))
        c |= dict(fp8=rng.random() < 0.6, batch=batch, q_len=q_len,
                  heads=rng.choice([0, 16, 64]), rot=64, interleaved=rng.random() < 0.5,
                  scaling=scaling)
        c["max_len"] = min(c["max_len"], 16000)
    else:
        kv = rng.choice([1, 2, 4, 8])
        group = rng.choice([1, 2, 4, 5, 7, 8, 16])
        q_len = rng.choice([1, 1, rng.randint(2, 9)])
        layout, shards = rng.choice([("interleaved", 1), ("interleaved", 2), ("interleaved", 4),
                                     ("interleaved", 8), ("contiguous", 2), ("contiguous", 3)])
        # at most 3 million padded token-heads
        batch = max(1, min(_log(rng, 1, 64), 3000000 // (hi * kv)))
        c |= dict(batch=batch, q_len=q_len, heads=kv * group, kv_heads=kv,
                  block=rng.choice([16, 32, 64]), shards=shards, layout=layout)
    c["min_len"] = min(c["min_len"], c["max_len"])
    return c


def _lens(c):
    """Context lengths of the batch (the new tokens among them), spread over
    their logarithm, and each request's new tokens."""
    rng = random.Random(c["mix"])
    B, lo, hi = c["batch"], c["min_len"], c["max_len"]
    lens = [hi] + [_log(rng, lo, hi) for _ in range(B - 1)]
    lens = [max(n, c["q_len"]) for n in lens]
    if c["ragged"]:
        q = [rng.randint(1, c["q_len"]) for _ in range(B)]
    else:
        q = [c["q_len"]] * B
    return lens, q


# -------------------------------------------------------------------- inputs
def _inv_freq(c):
    """Radians per token of each rotated pair, float64 [rot / 2], and the
    factor on the rotated values."""
    rot = c["rot"]
    i = torch.arange(0, rot, 2, dtype=torch.float64)
    inv = 10000.0 ** (-i / rot)
    if c["scaling"] == "linear":
        return inv / 8.0, 1.0
    if c["scaling"] == "yarn":
        # between `slow` turns of the original 4096 positions and `fast` of
        # them the stretched frequency blends into the plain one
        factor, orig, fast, slow = 40.0, 4096.0, 32.0, 1.0
        dim_of = lambda turns: rot * math.log(orig / (turns * 2 * math.pi)) / (2 * math.log(10000.0))
        low, high = max(math.floor(dim_of(fast)), 0), min(math.ceil(dim_of(slow)), rot - 1)
        k = torch.arange(rot // 2, dtype=torch.float64)
        ramp = ((k - low) / max(high - low, 1e-3)).clamp(0, 1)
        return inv / factor * ramp + inv * (1 - ramp), 0.1 * math.log(factor) + 1.0
    return inv, 1.0


def _pages(lens, g, spare=3):
    n = [-(-L // PAGE) for L in lens]
    P = sum(n) + spare
    perm = torch.randperm(P, generator=g, device=DEV, dtype=torch.int32)
    bt = torch.full((len(lens), max(n)), -1, dtype=torch.int32, device=DEV)
    off = 0
    for b, k in enumerate(n):
        bt[b, :k] = perm[off:off + k]
        off += k
    return P, bt


def _codes(shape, g):
    return (torch.randn(shape, generator=g, device=DEV) * 110).clamp_(-448, 448).to(FP8)


def _bf16(shape, g, sigma=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * sigma).to(torch.bfloat16)


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV).manual_seed(seed * 1000003 + 17)
    lens, qn = _lens(c)
    B, ql = c["batch"], c["q_len"]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    s = dict(c=c, seq_lens=i32(lens), q_lens=i32(qn) if c["ragged"] else None)
    if "rot" in c:
        inv, s["factor"] = _inv_freq(c)
        s["inv_freq"] = inv.to(DEV)
    if c["op"] == "rotate":
        s["q"] = _bf16((B, ql, c["heads"], c["dim"]), g)
        s["q_out"] = torch.zeros_like(s["q"])
        return s
    P, s["block_table"] = _pages(lens, g)
    if c["op"] == "attend":
        Hkv = c["kv_heads"]
        s["q"] = _bf16((B, ql, c["heads"], 128), g)
        for n in "kv":
            s[n] = _codes((P, PAGE, Hkv, 128), g)
            # scales of blocks whose largest value came near 448
            s[n + "_scale"] = (torch.rand((P, PAGE // c["block"], Hkv), generator=g, device=DEV) + 0.5) / 110
        return s
    # the row a context ends on, and the pages before it, hold earlier tokens
    if c["op"] == "append_gqa":
        Hkv = c["kv_heads"]
        for n in "kv":
            s[n + "_new"] = _bf16((B, ql, Hkv, 128), g)
            if c["fp8"]:
                s[n] = _codes((P, PAGE, Hkv, 128), g)
                e = torch.randint(-9, -5, (P, PAGE // c["block"], Hkv), generator=g, device=DEV)
                s[n + "_scale"] = torch.exp2(e.float())
            else:
                s[n] = _bf16((P, PAGE, Hkv, 128), g)
        width = 128
    else:
        s["latent"] = _bf16((B, ql, 576), g)
        if c["fp8"]:
            s["kv"] = _codes((P, PAGE, 576), g)
            s["kv_scale"] = torch.exp2(torch.randint(-9, -5, (P, PAGE), generator=g, device=DEV).float())
        else:
            s["kv"] = _bf16((P, PAGE, 576), g)
        width = 576
    if c["heads"]:
        s["q"] = _bf16((B, ql, c["heads"], width), g)
        s["q_out"] = torch.zeros_like(s["q"])
    s["workspace"] = torch.zeros(256, dtype=torch.uint8, device=DEV)
    return s


# ---------------------------------------------------------------- plain forms
def _positions(s, ql):
    """[B, q_len] positions of the new tokens and which of them are real."""
    L = s["seq_lens"].long()
    n = s["q_lens"].long() if s["q_lens"] is not None else torch.full_like(L, ql)
    i = torch.arange(ql, device=L.device)
    return (L - n)[:, None] + i, i[None, :] < n[:, None], L, n


def _rotate(x, pos, s, first, interleaved):
    """x fp32 [B, q_len, H, D] with dims first.. rotated by the positions."""
    ang = pos[:, :, None].double() * s["inv_freq"]
    cos = (ang.cos() * s["factor"]).float()[:, :, None, :]
    sin = (ang.sin() * s["factor"]).float()[:, :, None, :]
    rot = 2 * s["inv_freq"].numel()
    r = x[..., first:first + rot]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
    else:
        a, b = r[..., :rot // 2], r[..., rot // 2:]
    ya, yb = a * cos - b * sin, a * sin + b * cos
    y = torch.stack((ya, yb), -1).flatten(-2) if interleaved else torch.cat((ya, yb), -1)
    return torch.cat((x[..., :first], y, x[..., first + rot:]), -1)


def _pow2_scale(amax):
    """Smallest power of two (2^-60 at least) that puts amax within 448."""
    m, e = torch.frexp(amax)
    return torch.exp2(torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-60).float())


def _write(rows, idx, mask, values):
    """rows[idx] = values where mask, on flattened leading dimensions."""
    keep = mask.flatten()
    rows[idx.flatten()[keep]] = values.flatten(0, mask.dim() - 1)[keep]


def _append_blocks(new, cache, scale, s, block):
    """New fp32 tokens [B, q_len, Hkv, 128] into an e4m3 cache with a scale for
    each block of tokens and head; earlier tokens of a block whose scale grows
    are rounded again to it."""
    B, ql, Hkv, D = new.shape
    _, _, L, n = _positions(s, ql)
    start = L - n
    nb = (ql - 1 + block - 1) // block + 1
    blk = (start // block)[:, None] + torch.arange(nb, device=L.device)       # [B, nb]
    pos = blk[:, :, None] * block + torch.arange(block, device=L.device)      # [B, nb, block]
    fresh = (pos >= start[:, None, None]) & (pos < L[:, None, None])
    old = pos < start[:, None, None]
    touched = fresh.any(-1)
    old &= touched[:, :, None]
    b = torch.arange(B, device=L.device)[:, None]
    slot = (blk * block // PAGE).clamp(max=s["block_table"].shape[1] - 1)
    page = s["block_table"][b, slot].long().clamp(min=0)                      # [B, nb]
    row = page[:, :, None] * PAGE + pos % PAGE                                # [B, nb, block]
    x = new[b[:, :, None], (pos - start[:, None, None]).clamp(0, ql - 1)]     # [B, nb, block, Hkv, D]
    amax = (x.abs() * fresh[..., None, None]).amax(dim=(2, 4))                # [B, nb, Hkv]
    sidx = page * (PAGE // block) + (blk % (PAGE // block))
    was = scale.view(-1, Hkv)[sidx]
    need = _pow2_scale(amax)
    had = old.any(-1)[..., None]
    now = torch.where(had & (was >= need), was, need)
    codes = cache.view(torch.uint8).view(-1, Hkv, D)
    earlier = codes[row].view(FP8).float() * (was / now)[:, :, None, :, None]
    y = torch.where(fresh[..., None, None], x / now[:, :, None, :, None], earlier)
    _write(codes, row, fresh | old, y.to(FP8).view(torch.uint8))
    _write(scale.view(-1, Hkv), sidx, touched, now)


def _plain_append(s):
    c = s["c"]
    pos, real, L, n = _positions(s, c["q_len"])
    mla = c["op"] == "append_mla"
    first = 512 if mla else 0
    out = []
    if c["heads"]:
        y = _rotate(s["q"].float(), pos, s, first, c["interleaved"]).to(torch.bfloat16)
        s["q_out"].copy_(torch.where(real[:, :, None, None], y, s["q_out"]))
        out.append(s["q_out"])
    b = torch.arange(c["batch"], device=L.device)[:, None]
    at = (s["block_table"][b, (pos // PAGE).clamp(0, s["block_table"].shape[1] - 1)].long() * PAGE + pos % PAGE)
    if mla:
        x = _rotate(s["latent"].float()[:, :, None, :], pos, s, first, c["interleaved"])[:, :, 0]
        if c["fp8"]:
            sc = _pow2_scale(x.abs().amax(-1))
            _write(s["kv"].view(torch.uint8).view(-1, 576), at, real, (x / sc[..., None]).to(FP8).view(torch.uint8))
            _write(s["kv_scale"].view(-1), at, real, sc)
            return out + [s["kv"], s["kv_scale"]]
        _write(s["kv"].view(-1, 576), at, real, x.to(torch.bfloat16))
        return out + [s["kv"]]
    Hkv = c["kv_heads"]
    k = _rotate(s["k_new"].float(), pos, s, first, c["interleaved"])
    if c["fp8"]:
        _append_blocks(k, s["k"], s["k_scale"], s, c["block"])
        _append_blocks(s["v_new"].float(), s["v"], s["v_scale"], s, c["block"])
        return out + [s["k"], s["k_scale"], s["v"], s["v_scale"]]
    _write(s["k"].view(-1, Hkv, 128), at, real, k.to(torch.bfloat16))
    _write(s["v"].view(-1, Hkv, 128), at, real, s["v_new"])
    return out + [s["k"], s["v"]]


def _gather(codes, scale, bt, n, block):
    """Dequantised fp32 [B, Hkv, n, 128] of the first n tokens of every request."""
    Hkv = codes.shape[2]
    t = torch.arange(n, device=bt.device)
    row = bt[:, t // PAGE].long().clamp(min=0) * PAGE + t % PAGE
    x = codes.view(torch.uint8).view(-1, Hkv, 128)[row].view(FP8).float()
    x *= scale.view(-1, Hkv)[row // block][..., None]
    return x.transpose(1, 2)


def _plain_attend(s):
    c = s["c"]
    B, ql, H, Hkv = c["batch"], c["q_len"], c["heads"], c["kv_heads"]
    G = H // Hkv
    pos, real, L, n = _positions(s, ql)
    top = s["block_table"].shape[1] * PAGE
    K = _gather(s["k"], s["k_scale"], s["block_table"], top, c["block"])
    q = s["q"].float().view(B, ql, Hkv, G, 128).permute(0, 2, 1, 3, 4).reshape(B, Hkv, ql * G, 128)
    a = torch.matmul(q, K.transpose(-1, -2)) * (1 / math.sqrt(128))
    del K
    a = a.view(B, Hkv, ql, G, top)
    t = torch.arange(top, device=L.device)
    seen = (t <= pos[:, :, None]) & real[:, :, None]                 # [B, q_len, top]
    a.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    m = a.amax(-1, keepdim=True).clamp(min=-3e38)
    a.sub_(m).exp_()
    l = a.sum(-1, keepdim=True)
    V = _gather(s["v"], s["v_scale"], s["block_table"], top, c["block"])
    o = torch.matmul(a.view(B, Hkv, ql * G, top), V).view(B, Hkv, ql, G, 128)
    o = o / torch.where(l > 0, l, torch.ones_like(l))
    lse = torch.where(l > 0, m + l.log(), torch.full_like(m, -math.inf))[..., 0]
    out = o.permute(0, 2, 1, 3, 4).reshape(B, ql, H, 128).to(torch.bfloat16)
    return out, lse.permute(0, 2, 1, 3).reshape(B, ql, H)


def run(state):
    s, c = state, state["c"]
    if own:
        import sequence_sharded_mla_gb300 as mla
        if c["op"] == "attend":
            part, lse, s["workspace"] = mla.gqa_decode_partial_fp8(
                s["q"], s["k"], s["v"], s["k_scale"], s["v_scale"], s["block_table"], s["seq_lens"],
                c["shards"], c["layout"], causal=True, q_lens=s["q_lens"],
                workspace=s.get("workspace"))
            return mla.gqa_shard_combine(part, lse)
        rope = mla.Rope(s["inv_freq"], first_dim=512 if c.get("dim", 576 if c["op"] == "append_mla" else 128) == 576 else 0,
                        interleaved=c["interleaved"], attention_factor=s["factor"])
        if c["op"] == "rotate":
            return mla.mla_rope_apply(s["q"], rope, seq_lens=s["seq_lens"], q_lens=s["q_lens"], out=s["q_out"])
        if c["op"] == "append_mla":
            mla.mla_cache_append(s["latent"], s["kv"], s["block_table"], s["seq_lens"], rope=rope,
                                 q=s.get("q"), q_out=s.get("q_out"), kv_scale=s.get("kv_scale"),
                                 q_lens=s["q_lens"], workspace=s["workspace"])
            new = [s["kv"], s["kv_scale"]] if c["fp8"] else [s["kv"]]
        else:
            mla.gqa_cache_append(s["k_new"], s["v_new"], s["k"], s["v"], s["block_table"],
                                 s["seq_lens"], rope=rope, q=s.get("q"), q_out=s.get("q_out"),
                                 k_scale=s.get("k_scale"), v_scale=s.get("v_scale"),
                                 q_lens=s["q_lens"], workspace=s["workspace"])
            new = [s["k"], s["k_scale"], s["v"], s["v_scale"]] if c["fp8"] else [s["k"], s["v"]]
        return ([s["q_out"]] if c["heads"] else []) + new
    if c["op"] == "attend":
        return _plain_attend(s)
    if c["op"] == "rotate":
        pos, real, _, _ = _positions(s, c["q_len"])
        y = _rotate(s["q"].float(), pos, s, c["first"], c["interleaved"]).to(torch.bfloat16)
        s["q_out"].copy_(torch.where(real[:, :, None, None], y, s["q_out"]))
        return s["q_out"]
    return _plain_append(s)


# ---------------------------------------------------------------------- work
def work(case):
    c = case
    lens, qn = _lens(c)
    T = sum(qn)
    if c["op"] == "rotate":
        # every head is read and written whole; a rotated pair costs 6 operations
        n = T * c["heads"]
        return dict(bytes=4 * n * c["dim"], flops=3 * n * c["rot"])
    if c["op"] == "attend":
        Hkv, H = c["kv_heads"], c["heads"]
        rows = c["batch"] * c["q_len"] * H
        tok = sum(lens)
        pairs = sum(sum(L - n + i + 1 for i in range(n)) for L, n in zip(lens, qn))
        scales = sum(-(-L // c["block"]) for L in lens) * Hkv * 2 * 4
        return dict(bytes=tok * Hkv * 256 + scales + rows * (256 + 256 + 4), flops=pairs * H * 4 * 128)
    width = 576 if c["op"] == "append_mla" else 128
    q = T * c["heads"] * width * 4
    if c["op"] == "append_mla":
        new = T * 576 * (2 + (1 if c["fp8"] else 2)) + (T * 4 if c["fp8"] else 0)
        rows = T * (c["heads"] + 1)
    else:
        new = 2 * T * c["kv_heads"] * 128 * (2 + (1 if c["fp8"] else 2))
        if c["fp8"]:
            blocks = sum((L - 1) // c["block"] - (L - n) // c["block"] + 1 for L, n in zip(lens, qn))
            new += 2 * blocks * c["kv_heads"] * 8
        rows = T * (c["heads"] + c["kv_heads"])
    return dict(bytes=q + new, flops=3 * rows * c["rot"])


# -------------------------------------------------------- definition, 64 bits
def _exact_turn(x, p, inv, factor, first, interleaved):
    """One token's rows [.., D] (64 bits) turned by position p, pair by pair."""
    y = x.clone()
    half = inv.numel()
    i = torch.arange(half, device=x.device)
    ia, ib = (first + 2 * i, first + 2 * i + 1) if interleaved else (first + i, first + half + i)
    z = torch.complex(x[..., ia], x[..., ib]) * torch.polar(torch.full_like(inv, factor), p * inv)
    y[..., ia], y[..., ib] = z.real, z.imag
    return y


def _exact_code(x):
    """Nearest e4m3 value (ties to even) of 64-bit values within 448."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(e - 3)
    return torch.round(x / step) * step


def _exact_scale(amax):
    return 2.0 ** max(math.ceil(math.log2(amax / 448.0)), -60) if amax > 0 else 2.0 ** -60


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    lens, qn = _lens(c)
    if c["op"] == "attend":
        if sum(L * n for L, n in zip(lens, qn)) * c["heads"] > 3e8:
            return None
        G, Hkv = c["heads"] // c["kv_heads"], c["kv_heads"]
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
        lse = torch.full(s["q"].shape[:3], -math.inf, dtype=torch.float64, device=DEV)
        for b, (L, n) in enumerate(zip(lens, qn)):
            pages = s["block_table"][b, :-(-L // PAGE)].long()

            def whole(name):
                x = s[name].view(torch.uint8)[pages].view(FP8).double()
                sc = s[name + "_scale"][pages].double().repeat_interleave(c["block"], dim=1)
                return (x * sc[..., None]).flatten(0, 1)[:L].repeat_interleave(G, dim=1)     # [L, H, 128]

            K, V = whole("k"), whole("v")
            for i in range(n):
                last = L - n + i + 1
                a = torch.einsum("hd,thd->ht", s["q"][b, i].double(), K[:last]) / math.sqrt(128.0)
                lse[b, i] = torch.logsumexp(a, -1)
                out[b, i] = torch.einsum("ht,thd->hd", torch.exp(a - lse[b, i][:, None]), V[:last])
        return out, lse
    if sum(qn) > 300:
        return None
    inv, factor = s["inv_freq"], s["factor"]
    dim = c.get("dim", 576 if c["op"] == "append_mla" else 128)
    first = 512 if dim == 576 else 0
    turn = lambda x, p: _exact_turn(x.double(), float(p), inv, factor, first, c["interleaved"])
    out = []
    if "q" in s:
        q = s["q_out"].double()
        for b, (L, n) in enumerate(zip(lens, qn)):
            for i in range(n):
                q[b, i] = turn(s["q"][b, i], L - n + i)
        if c["op"] == "rotate":
            return q
        out.append(q)
    bt = s["block_table"].tolist()
    names = ["kv"] if c["op"] == "append_mla" else ["k", "v"]
    for name in names:
        cache = s[name].double()
        if c["fp8"]:
            scale = s[name + "_scale"].double()
        for b, (L, n) in enumerate(zip(lens, qn)):
            rows = {}
            for i in range(n):
                p = L - n + i
                if name == "kv":
                    rows[p] = turn(s["latent"][b, i], p)
                elif name == "k":
                    rows[p] = turn(s["k_new"][b, i], p)
                else:
                    rows[p] = s["v_new"][b, i].double()
            if not c["fp8"]:
                for p, x in rows.items():
                    cache[bt[b][p // PAGE], p % PAGE] = x
            elif name == "kv":
                for p, x in rows.items():
                    page, r = bt[b][p // PAGE], p % PAGE
                    scale[page, r] = _exact_scale(x.abs().max().item())
                    cache[page, r] = _exact_code(x / scale[page, r])
            else:
                k = c["block"]
                for blk in range((L - n) // k, (L - 1) // k + 1):
                    page, sub = bt[b][blk * k // PAGE], blk % (PAGE // k)
                    here = [p for p in range(blk * k, blk * k + k) if p in rows]
                    was = scale[page, sub].clone()
                    need = torch.stack([rows[p].abs().amax(-1) for p in here]).amax(0)
                    need = torch.tensor([_exact_scale(v) for v in need.tolist()], dtype=torch.float64, device=DEV)
                    keep = was >= need if here[0] > blk * k else torch.zeros_like(was, dtype=torch.bool)
                    now = torch.where(keep, was, need)
                    for p in range(blk * k, here[0]):
                        cache[page, p % PAGE] = _exact_code(cache[page, p % PAGE] * (was / now)[:, None])
                    for p in here:
                        cache[page, p % PAGE] = _exact_code(rows[p] / now[:, None])
                    scale[page, sub] = now
        out += [cache, scale] if c["fp8"] else [cache]
    return out
