"""64-bit references of the rotary, cache-append and e4m3 block-scale
grouped-query operators, one token and one row at a time, on the CPU."""
import math

import torch

PAGE = 64
FP8 = torch.float8_e4m3fn


def e4m3(codes):
    """Values of e4m3 codes (float8 or uint8 tensor) in 64 bits."""
    return codes.view(torch.uint8).view(FP8).float().double()


def round_e4m3(x):
    """Nearest e4m3 value (ties to even) of |x| <= 448; not finite: NaN."""
    a = x.abs().clamp(min=2.0 ** -6)
    step = torch.exp2(torch.floor(torch.log2(a)) - 3)
    y = torch.round(x / step) * step
    y = y.clamp(-448.0, 448.0)
    return torch.where(torch.isfinite(x), y, torch.full_like(y, math.nan))


def pow2_scale(a):
    """Smallest power of two >= 2^-60 with a <= 448 s."""
    if a == 0:
        return 2.0 ** -60
    e = math.ceil(math.log2(a / 448.0))
    while a > 448.0 * 2.0 ** e:
        e += 1
    while a <= 448.0 * 2.0 ** (e - 1):
        e -= 1
    return 2.0 ** max(e, -60)


def turn(x, p, inv, first, interleaved, factor):
    """One token's rows [.., D] in 64 bits turned by position p."""
    y = x.clone()
    half = inv.numel()
    for i in range(half):
        a, b = (first + 2 * i, first + 2 * i + 1) if interleaved else (first + i, first + half + i)
        ang = math.fmod(p * float(inv[i]), 2 * math.pi)
        c, s = factor * math.cos(ang), factor * math.sin(ang)
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., a] * s + x[..., b] * c
    return y


def turn_error(x, first, half, interleaved, factor):
    """Bound on the fp32 error of turn()'s values [.., D]: the angle is off by
    at most 2^-24 of an eighth of a turn (2^-24.3 rad) and the sine and cosine
    by 2 ulp (2^-23), and two products and their sum round by 2^-24 each:
    below 2^-21 of |x_a| + |x_b|."""
    e = torch.zeros_like(x)
    for i in range(half):
        a, b = (first + 2 * i, first + 2 * i + 1) if interleaved else (first + i, first + half + i)
        m = (x[..., a].abs() + x[..., b].abs()) * abs(factor) * 2.0 ** -21
        e[..., a], e[..., b] = m, m
    return e


def owned(L, s, N, layout):
    """Tokens of an L-token context that shard s of N owns, in order, and the
    cache slot that holds each."""
    if layout.startswith("interleaved"):
        t = list(range(s, L, N))
    else:
        c = -(-L // N)
        t = list(range(s * c, min((s + 1) * c, L)))
    return t, (list(range(len(t))) if layout.endswith("local") else t)


def attend(q, k, v, ks, vs, bt, lens, q_lens, causal, scale, N, s, layout, rows=None):
    """Partial attention of shard s of N (s < 0: the whole context): o [B,
    q_len, H, D], lse, and per output the bounds that its tolerance is made
    of: sum p |V sv| and the error of a logit.  rows: only these (b, i)."""
    B, q_len, H, D = q.shape
    Hkv = k.shape[2]
    G = H // Hkv
    block = PAGE // ks.shape[1]
    o = torch.zeros(B, q_len, H, D, dtype=torch.float64)
    spread = torch.zeros_like(o)
    lse = torch.full((B, q_len, H), -math.inf, dtype=torch.float64)
    err = torch.zeros_like(lse)
    kv, vv = k.view(torch.uint8), v.view(torch.uint8)
    for b in range(B):
        L = int(lens[b])
        n = q_len if q_lens is None else int(q_lens[b])
        toks, slots = owned(L, s, N, layout) if s >= 0 else (list(range(L)),) * 2
        if not toks:
            continue
        toks, slots = torch.tensor(toks), torch.tensor(slots)
        page = bt[b].long()[slots // PAGE]
        good = (page >= 0) & (page < k.shape[0])
        page = page.clamp(0, k.shape[0] - 1)
        r = slots % PAGE
        K = e4m3(kv[page, r]) * ks.double()[page, r // block][..., None]
        V = e4m3(vv[page, r]) * vs.double()[page, r // block][..., None]
        K[~good] = 0
        V[~good] = 0
        K, V = K.repeat_interleave(G, 1), V.repeat_interleave(G, 1)
        for i in range(n):
            if rows is not None and (b, i) not in rows:
                continue
            see = toks <= (L - n + i if causal else L)
            if not see.any():
                continue
            x = q[b, i].double()
            a = torch.einsum("hd,thd->ht", x, K[see]) * scale
            lse[b, i] = torch.logsumexp(a, -1)
            p = torch.exp(a - lse[b, i][:, None])
            o[b, i] = torch.einsum("ht,thd->hd", p, V[see])
            spread[b, i] = torch.einsum("ht,thd->hd", p, V[see].abs())
            size = (torch.einsum("hd,thd->ht", x.abs(), K[see].abs())).amax(-1)
            wide = x.abs().amax(-1) * K[see].abs().sum(-1).amax(0)
            err[b, i] = scale * (size * 2.0 ** -20 + wide * 2.0 ** -18)
    return o, lse, spread, err


def check_attention(got, got_lse, ref, P_REL=2.0 ** -8, out_rel=0.0):
    """got against attend()'s results.  A weight's error is that of its logit
    (err: the query's two e4m3 terms leave 2^-18 of the row's largest value,
    fp32 sums 2^-20 of their terms) and of its rounding to 2^-9 (three e5m2
    terms of a value in 11 bits), with as much again for the sums; out_rel is
    the rounding of the result's type."""
    o, lse, spread, err = ref
    g, gl = got.double().cpu(), got_lse.double().cpu()
    assert torch.equal(torch.isnan(g), torch.isnan(o)), "NaN pattern of the output differs"
    assert torch.equal(torch.isneginf(gl), torch.isneginf(lse)), "-inf pattern of the lse differs"
    assert torch.equal(torch.isnan(gl), torch.isnan(lse)), "NaN pattern of the lse differs"
    tol = spread * (P_REL + 2 * err[..., None]) + o.abs() * out_rel + 1e-30
    bad = torch.nan_to_num((g - o).abs() - tol, nan=-1.0)
    assert float(bad.max()) <= 0, f"output off by {float((g - o).abs().max())}"
    ltol = err + lse.abs() * 2.0 ** -21 + 2.0 ** -20
    fine = torch.isfinite(lse)
    assert bool(((gl - lse).abs()[fine] <= ltol[fine]).all()), (
        f"lse off by {float((gl - lse).abs()[fine].max())}")
