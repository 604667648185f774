"""Measured cases of the operators for long, shared and bounded latent caches.

  prefix   latent attention of a batch whose requests share long prefixes, each
           prefix attended once for all the requests that share it, and the LSE
           combine with every request's own tokens
  weights  the attention weight that a step gives to every cached token, summed
           over its query rows and added to what earlier steps gave
  evict    a context cut to a budget: its first and newest tokens and the most
           attended of the others, moved in order to new pages

`run` computes them in elementary torch operations, or with the framework's
calls where `own` is true.
"""
import math
import random

import torch

own = False

PAGE = 64
WIDTH, VALUE = 576, 512
SCALE = 1.0 / math.sqrt(192.0)
FP8 = torch.float8_e4m3fn
DEV = "cuda"


# --------------------------------------------------------------------- cases
def listed():
    return [
        # two requests behind one short system prompt, 16 heads: latency
        dict(name="prefix-two-short", op="prefix", fp8=False, batch=2, groups=1, q_len=1, heads=16,
             prefix_min=1024, prefix_max=1024, own_min=40, own_max=200, mix=1, ragged=False),
        # 32 agents over one 114k-token prefix, up to 6k tokens of their own
        dict(name="prefix-agents-bf16", op="prefix", fp8=False, batch=32, groups=1, q_len=1, heads=64,
             prefix_min=116736, prefix_max=116736, own_min=400, own_max=6144, mix=2, ragged=False),
        # the same batch size over an fp8 cache: nine prefixes of odd lengths,
        # groups of odd sizes (one request among them)
        dict(name="prefix-groups-fp8", op="prefix", fp8=True, batch=37, groups=9, q_len=1, heads=64,
             prefix_min=1500, prefix_max=65000, own_min=1, own_max=3001, mix=3, ragged=False),
        # a ragged causal verify step of 16 requests, three prefixes
        dict(name="prefix-verify-bf16", op="prefix", fp8=False, batch=16, groups=3, q_len=5, heads=64,
             prefix_min=2000, prefix_max=16000, own_min=300, own_max=2500, mix=4, ragged=True),
        # the decode batch whose contexts are to be cut: 32 requests
        dict(name="weights-batch-bf16", op="weights", fp8=False, batch=32, q_len=1, heads=64,
             min_len=4000, max_len=65536, mix=5, ragged=False),
        # a ragged verify step of 16 requests over an fp8 cache
        dict(name="weights-verify-fp8", op="weights", fp8=True, batch=16, q_len=9, heads=64,
             min_len=5000, max_len=8000, mix=6, ragged=True),
        # one short request, 16 heads: latency
        dict(name="weights-one-short", op="weights", fp8=False, batch=1, q_len=1, heads=16,
             min_len=1024, max_len=1024, mix=7, ragged=False),
        # one fp8 request of a million tokens
        dict(name="weights-long-fp8", op="weights", fp8=True, batch=1, q_len=1, heads=64,
             min_len=1048576, max_len=1048576, mix=8, ragged=False),
        # four short requests, a few rows leave each: latency
        dict(name="evict-short", op="evict", fp8=False, batch=4, min_len=300, max_len=777, first=4,
             recent=64, keep_min=0.8, keep_max=1.0, mix=9),
        # a batch cut to about half, 64 first tokens and a recent window kept
        dict(name="evict-batch-bf16", op="evict", fp8=False, batch=16, min_len=4000, max_len=40000,
             first=64, recent=512, keep_min=0.4, keep_max=0.7, mix=10),
        # one fp8 request of a million tokens cut to a quarter, behind a kept
        # prefix
        dict(name="evict-long-fp8", op="evict", fp8=True, batch=1, min_len=1048576, max_len=1048576,
             first=8192, recent=4096, keep_min=0.25, keep_max=0.25, mix=11),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefix", "prefix", "weights", "evict"])
    c = dict(op=op, fp8=rng.random() < 0.5, mix=rng.randrange(1 << 30))
    if op == "prefix":
        heads = rng.choice([16, 32, 64, 64, 128])
        q_len = rng.choice([1, 1, rng.randint(2, 9)])
        hi = _log(rng, 64, 120000)
        lo = _log(rng, min(hi, 40), hi)
        own_hi = _log(rng, 16, 8000)
        # at most 200 million (row, token) pairs, 200 thousand shared tokens and
        # as many own ones
        most = min(48, 200000000 // (heads * q_len * (hi + own_hi)), 200000 // own_hi)
        batch = _log(rng, 1, max(1, most))
        groups = min(batch, _log(rng, 1, 12), max(1, 200000 // hi))
        c |= dict(batch=batch, groups=groups, q_len=q_len, heads=heads,
                  prefix_min=lo, prefix_max=hi, own_min=min(own_hi, _log(rng, 1, 1000)), own_max=own_hi,
                  ragged=rng.random() < 0.5)
    elif op == "weights":
        heads = rng.choice([16, 32, 64, 64, 128])
        q_len = rng.choice([1, 1, rng.randint(2, 9)])
        hi = _log(rng, 16, 200000 if heads * q_len <= 256 else 50000)
        most = min(64, 60000000 // (heads * q_len * hi), 800000 // hi)
        c |= dict(batch=_log(rng, 1, max(1, most)), q_len=q_len, heads=heads,
                  min_len=_log(rng, 1, hi), max_len=hi, ragged=rng.random() < 0.5)
    else:
        hi = _log(rng, 70, 300000 if c["fp8"] else 150000)
        a, b = sorted((rng.uniform(0.05, 1.0), rng.uniform(0.05, 1.0)))
        c |= dict(batch=_log(rng, 1, max(1, min(48, (300000 if c["fp8"] else 150000) // hi))), min_len=_log(rng, 1, hi),
                  max_len=hi, first=rng.choice([0, 4, _log(rng, 1, 2000)]),
                  recent=rng.choice([0, 32, _log(rng, 1, 2000)]), keep_min=a, keep_max=b)
    return c


def _plan(c):
    """What a case's lengths come to: per request its context and new tokens,
    and for `prefix` the first request of every group and its common tokens."""
    rng = random.Random(c["mix"])
    B = c["batch"]
    if c["op"] == "evict":
        lens = [c["max_len"]] + [_log(rng, c["min_len"], c["max_len"]) for _ in range(B - 1)]
        keep = [int(n * rng.uniform(c["keep_min"], c["keep_max"])) for n in lens]
        return lens, keep
    ql = c["q_len"]
    new = [rng.randint(1, ql) if c["ragged"] else ql for _ in range(B)]
    if c["op"] == "weights":
        lens = [c["max_len"]] + [_log(rng, c["min_len"], c["max_len"]) for _ in range(B - 1)]
        return [max(n, ql) for n in lens], new
    starts = [0] + sorted(rng.sample(range(1, B), c["groups"] - 1)) + [B]
    common = [c["prefix_max"]] + [_log(rng, c["prefix_min"], c["prefix_max"]) for _ in range(c["groups"] - 1)]
    group = [g for g in range(c["groups"]) for _ in range(starts[g + 1] - starts[g])]
    lens = [common[g] + max(ql, _log(rng, c["own_min"], c["own_max"])) for g in group]
    return lens, new, starts, common, group


# -------------------------------------------------------------------- inputs
def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _cache(pages, fp8, g):
    """Latent rows of unit size: bf16, or e4m3 codes with each row's scale."""
    if not fp8:
        kv = torch.empty((pages, PAGE, WIDTH), dtype=torch.bfloat16, device=DEV)
        for i in range(0, pages, 2048):
            kv[i:i + 2048] = torch.randn(kv[i:i + 2048].shape, generator=g, device=DEV) * 0.5
        return kv, None
    kv = torch.empty((pages, PAGE, WIDTH), dtype=FP8, device=DEV)
    for i in range(0, pages, 2048):
        kv[i:i + 2048] = (torch.randn(kv[i:i + 2048].shape, generator=g, device=DEV) * 110).clamp_(-448, 448).to(FP8)
    return kv, (torch.rand((pages, PAGE), generator=g, device=DEV) + 0.5) / 220


def _tables(rows, g, spare=3):
    """A block table for rows of page counts, the pages in random order."""
    P = sum(rows) + spare
    perm = torch.randperm(P, generator=g, device=DEV, dtype=torch.int32)
    bt = torch.full((len(rows), max(max(rows), 1)), -1, dtype=torch.int32, device=DEV)
    off = 0
    for b, k in enumerate(rows):
        bt[b, :k] = perm[off:off + k]
        off += k
    return P, bt


def _rows(s, b, n):
    """Places of request b's first n tokens among the cache's rows."""
    t = torch.arange(n, device=DEV)
    return s["block_table"][b, t // PAGE].long() * PAGE + t % PAGE


def _latent(s, rows, dtype):
    x = s["kv"].view(torch.uint8).view(-1, WIDTH)[rows].view(FP8).to(dtype) if s["c"]["fp8"] \
        else s["kv"].view(-1, WIDTH)[rows].to(dtype)
    if s["c"]["fp8"]:
        x *= s["kv_scale"].view(-1)[rows].to(dtype)[:, None]
    return x


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV).manual_seed(seed * 1000003 + 29)
    B = c["batch"]
    pages = lambda n: -(-n // PAGE)
    plan = _plan(c)
    lens = plan[0]
    s = dict(c=c, plan=plan, seq_lens=_i32(lens))
    if c["op"] == "evict":
        lens, keep = plan
        old = [pages(n) for n in lens]
        new = [pages(k) for k in keep]
        P, both = _tables(old + new, g)
        s["block_table"] = both[:B, :max(old)].contiguous()
        s["new_block_table"] = both[B:, :max(max(new), 1)].contiguous()
        s["kv"], s["kv_scale"] = _cache(P, c["fp8"], g)
        s["keep"] = _i32(keep)
        s["keep_first"] = _i32([c["first"]] * B)
        # weights of a long tail, the least attended tokens at zero together
        w = torch.exp(3.0 * torch.randn((B, max(lens)), generator=g, device=DEV) - 4.0)
        s["weights"] = torch.where(w < 1e-3, torch.zeros_like(w), w)
        s["weights_out"] = torch.zeros((B, max(max(keep), 1)), device=DEV)
        s["kept"] = torch.zeros((B, max(max(keep), 1)), dtype=torch.int32, device=DEV)
        return s
    s["q_lens"] = _i32(plan[1]) if c["ragged"] else None
    if c["op"] == "prefix":
        _, _, starts, common, group = plan
        # a group's whole common pages, then each request's own
        shared = [n // PAGE for n in common]
        mine = [pages(L) - shared[k] for L, k in zip(lens, group)]
        P, bt = _tables(shared + mine, g)
        s["block_table"] = torch.full((B, max(pages(L) for L in lens)), -1, dtype=torch.int32, device=DEV)
        for b, k in enumerate(group):
            s["block_table"][b, :shared[k]] = bt[k, :shared[k]]
            s["block_table"][b, shared[k]:shared[k] + mine[b]] = bt[len(shared) + b, :mine[b]]
        s["group_starts"], s["prefix_lens"] = _i32(starts), _i32(common)
    else:
        P, s["block_table"] = _tables([pages(L) for L in lens], g)
    s["kv"], s["kv_scale"] = _cache(P, c["fp8"], g)
    s["q"] = (torch.randn((B, c["q_len"], c["heads"], WIDTH), generator=g, device=DEV) * 0.5).to(torch.bfloat16)
    if c["op"] == "weights":
        # what the step's attention left, and what earlier steps summed up
        s["lse"] = torch.stack([_attend(s, b, False)[1] for b in range(B)])
        s["weights"] = torch.rand((B, max(lens)), generator=g, device=DEV)
        s["out"] = torch.zeros_like(s["weights"])
    return s


# ---------------------------------------------------------------- plain forms
def _seen(c, L, n):
    """[q_len, L]: which tokens query i may see; a padding row sees none."""
    i = torch.arange(c["q_len"], device=DEV)[:, None]
    return (torch.arange(L, device=DEV)[None, :] <= L - n + i) & (i < n)


def _attend(s, b, values=True):
    """One request's outputs and their log-sum-exp."""
    c, L, n = s["c"], s["plan"][0][b], s["plan"][1][b]
    K = _latent(s, _rows(s, b, L), torch.float32)
    a = torch.matmul(s["q"][b].float().view(-1, WIDTH), K.t()).view(c["q_len"], c["heads"], L) * SCALE
    a.masked_fill_(~_seen(c, L, n)[:, None, :], -math.inf)
    m = a.amax(-1, keepdim=True).clamp(min=-3e38)
    a.sub_(m).exp_()
    l = a.sum(-1, keepdim=True)
    lse = torch.where(l > 0, m + l.log(), torch.full_like(m, -math.inf))[..., 0]
    if not values:
        return None, lse
    o = torch.matmul(a.view(-1, L), K[:, :VALUE]).view(c["q_len"], c["heads"], VALUE)
    return (o / torch.where(l > 0, l, torch.ones_like(l))).to(torch.bfloat16), lse


def _weigh(s, b):
    """One request's row of summed weights."""
    c, L, n = s["c"], s["plan"][0][b], s["plan"][1][b]
    K = _latent(s, _rows(s, b, L), torch.float32)
    a = torch.matmul(s["q"][b].float().view(-1, WIDTH), K.t()).view(c["q_len"], c["heads"], L) * SCALE
    seen = _seen(c, L, n)[:, None, :]
    p = torch.where(seen, a - torch.where(seen, s["lse"][b][..., None], torch.zeros_like(a)), torch.full_like(a, -math.inf))
    w = p.exp_().sum(dim=(0, 1))
    old = torch.arange(L, device=DEV) < L - n
    return w + torch.where(old, s["weights"][b, :L], torch.zeros_like(w))


def _cut(s, b):
    """Positions of the tokens that request b keeps, in order."""
    L, keep = s["plan"][0][b], s["plan"][1][b]
    if keep >= L:
        return torch.arange(L, device=DEV)
    first = min(s["c"]["first"], keep)
    recent = min(s["c"]["recent"], keep - first)
    w = s["weights"][b, first:L - recent]
    by_weight = torch.sort(w, descending=True, stable=True).indices[:keep - first - recent]
    return torch.cat((torch.arange(first, device=DEV), torch.sort(by_weight).values + first,
                      torch.arange(L - recent, L, device=DEV)))


def _plain_evict(s):
    B = s["c"]["batch"]
    new_lens = torch.zeros(B, dtype=torch.int32, device=DEV)
    s["kept"].fill_(-1)
    raw = s["kv"].view(torch.uint8) if s["c"]["fp8"] else s["kv"]
    flat = raw.view(-1, raw.shape[-1])
    for b in range(B):
        at = _cut(s, b)
        n = at.numel()
        j = torch.arange(n, device=DEV)
        src = s["block_table"][b, at // PAGE].long() * PAGE + at % PAGE
        dst = s["new_block_table"][b, j // PAGE].long() * PAGE + j % PAGE
        flat[dst] = flat[src]
        if s["c"]["fp8"]:
            s["kv_scale"].view(-1)[dst] = s["kv_scale"].view(-1)[src]
        s["kept"][b, :n] = at.int()
        s["weights_out"][b, :n] = s["weights"][b, at]
        new_lens[b] = n
    return _evicted(s, new_lens)


def _evicted(s, new_lens):
    return [s["kv"]] + ([s["kv_scale"]] if s["c"]["fp8"] else []) + [new_lens, s["kept"], s["weights_out"]]


def run(state):
    s, c = state, state["c"]
    if own:
        import sequence_sharded_mla_gb300 as mla
        if c["op"] == "prefix":
            part, lse, s["workspace"] = mla.mla_prefix_partial(
                s["q"], s["kv"], s["block_table"], s["seq_lens"], s["group_starts"], s["prefix_lens"],
                kv_scale=s["kv_scale"], causal=True, q_lens=s["q_lens"], workspace=s.get("workspace"))
            return mla.mla_shard_combine(part, lse)
        if c["op"] == "weights":
            out, s["workspace"] = mla.mla_attention_weights(
                s["q"], s["kv"], s["block_table"], s["seq_lens"], s["lse"], weights=s["weights"], out=s["out"],
                kv_scale=s["kv_scale"], causal=True, q_lens=s["q_lens"], workspace=s.get("workspace"))
            return out
        new_lens, kept, weights, s["workspace"] = mla.mla_cache_evict(
            s["kv"], s["block_table"], s["seq_lens"], s["weights"], s["keep"], s["new_block_table"],
            keep_first=s["keep_first"], recent=c["recent"], kv_scale=s["kv_scale"], kept=s["kept"],
            weights_out=s["weights_out"], workspace=s.get("workspace"))
        return _evicted(s, new_lens)
    if c["op"] == "prefix":
        both = [_attend(s, b) for b in range(c["batch"])]
        return torch.stack([o for o, _ in both]), torch.stack([l for _, l in both])
    if c["op"] == "weights":
        for b, L in enumerate(s["plan"][0]):
            s["out"][b, :L] = _weigh(s, b)
        return s["out"]
    return _plain_evict(s)


# ---------------------------------------------------------------------- work
def work(case):
    c = case
    plan = _plan(c)
    row = WIDTH + 4 if c["fp8"] else 2 * WIDTH
    if c["op"] == "evict":
        lens, keep = plan
        kept = sum(min(L, k) for L, k in zip(lens, keep))
        # candidates' weights are read; kept rows, weights and positions move
        return dict(bytes=4 * sum(lens) + kept * (2 * row + 8), flops=0)
    lens, new = plan[:2]
    rows = c["batch"] * c["q_len"] * c["heads"]
    pairs = c["heads"] * sum(sum(L - n + i + 1 for i in range(n)) for L, n in zip(lens, new))
    if c["op"] == "weights":
        return dict(bytes=sum(lens) * (row + 8) + rows * (2 * WIDTH + 4), flops=2 * WIDTH * pairs)
    _, _, starts, common, group = plan
    tokens = sum(n // PAGE * PAGE for n in common) + sum(L - common[k] // PAGE * PAGE for L, k in zip(lens, group))
    return dict(bytes=tokens * row + rows * (2 * WIDTH + 2 * VALUE + 4), flops=2 * (WIDTH + VALUE) * pairs)


# -------------------------------------------------------- definition, 64 bits
def exact(case, seed):
    c = case
    s = prepare(case, seed)
    plan = s["plan"]
    B = c["batch"]
    if c["op"] == "evict":
        lens, keep = plan
        kv = s["kv"].double() if s["kv"].numel() < 2e9 else None
        if kv is None:
            return None
        source = kv.clone()
        scale = s["kv_scale"].double() if c["fp8"] else None
        was = scale.clone() if c["fp8"] else None
        bt, nbt = s["block_table"].tolist(), s["new_block_table"].tolist()
        weights = s["weights"].double().cpu()
        kept = torch.full(s["kept"].shape, -1, dtype=torch.int64)
        out = s["weights_out"].double().cpu()
        for b, (L, k) in enumerate(zip(lens, keep)):
            n = min(L, k)
            held = set(range(min(c["first"], n)))
            held |= set(range(L - min(c["recent"], n - len(held)), L)) if n < L else set(range(L))
            row = weights[b].tolist()
            others = sorted((t for t in range(L) if t not in held), key=lambda t: (-row[t], t))
            at = sorted(held | set(others[:n - len(held)]))
            kept[b, :n] = torch.tensor(at, dtype=torch.int64)
            out[b, :n] = weights[b, at]
            if n:
                src = torch.tensor([bt[b][t // PAGE] * PAGE + t % PAGE for t in at], device=DEV)
                dst = torch.tensor([nbt[b][j // PAGE] * PAGE + j % PAGE for j in range(n)], device=DEV)
                kv.view(-1, WIDTH)[dst] = source.view(-1, WIDTH)[src]
                if c["fp8"]:
                    scale.view(-1)[dst] = was.view(-1)[src]
        new = torch.tensor([min(L, k) for L, k in zip(lens, keep)], device=DEV)
        return [kv] + ([scale] if c["fp8"] else []) + [new, kept.to(DEV), out.to(DEV)]
    lens, new = plan[:2]
    if sum(L * n for L, n in zip(lens, new)) * c["heads"] > 2e9:
        return None
    out = torch.zeros((B, c["q_len"], c["heads"], VALUE), dtype=torch.float64, device=DEV)
    lse = torch.full((B, c["q_len"], c["heads"]), -math.inf, dtype=torch.float64, device=DEV)
    total = s["out"].double() if c["op"] == "weights" else None
    for b, (L, n) in enumerate(zip(lens, new)):
        pages = s["block_table"][b, :-(-L // PAGE)].long()
        if c["fp8"]:
            K = s["kv"].view(torch.uint8)[pages].view(FP8).double() * s["kv_scale"][pages].double()[..., None]
        else:
            K = s["kv"][pages].double()
        K = K.flatten(0, 1)[:L]
        if total is not None:
            total[b, :L - n] = s["weights"][b, :L - n].double()
            total[b, L - n:L] = 0
        for i in range(n):
            last = L - n + i + 1
            a = torch.einsum("hd,td->ht", s["q"][b, i].double(), K[:last]) / math.sqrt(192.0)
            if total is not None:
                total[b, :last] += torch.exp(a - s["lse"][b, i].double()[:, None]).sum(0)
                continue
            lse[b, i] = torch.logsumexp(a, -1)
            out[b, i] = torch.einsum("ht,td->hd", torch.exp(a - lse[b, i][:, None]), K[:last, :VALUE])
    return total if c["op"] == "weights" else (out, lse)
