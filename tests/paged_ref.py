"""The paged cache and its attention from their definitions, in 64 bits on the CPU (no code of the package)."""
from __future__ import annotations

import math

import torch

F64 = torch.float64


def quantise(k, v):
    """k, v [T, H, d] -> (negative signs bool, mu fp64 not yet rounded to bf16, exponents, codes), per row."""
    k, v = k.to(F64), v.to(F64)
    mu = k.abs().mean(-1)
    amax = v.abs().amax(-1)
    e = torch.full(amax.shape, -24, dtype=torch.int64)
    for n in range(-24, 9):
        e[amax > 127 * 2.0 ** n] = n + 1
    step = 2.0 ** e.to(F64)
    codes = (v / step[..., None]).round().clamp(-127, 127).to(torch.int64)
    return k < 0, mu, e, codes


def split_block(block, ps, d):
    """The parts of a cache [pages, heads, bytes] on the CPU, cut by hand: codes [P,H,ps,d], pad columns, negative
    signs [P,H,ps,128], mu (fp64), exponents."""
    P, H = block.shape[:2]
    dp = (d + 15) // 16 * 16
    assert block.shape[2] == ps * (dp + 19)
    cut = [block[:, :, ps * a:ps * b] for a, b in ((0, dp), (dp, dp + 16), (dp + 16, dp + 18), (dp + 18, dp + 19))]
    codes = cut[0].reshape(P, H, ps, dp).to(torch.int64)
    codes = torch.where(codes > 127, codes - 256, codes)
    byte = cut[1].reshape(P, H, ps, 16).to(torch.int64)
    neg = ((byte[..., None] >> torch.arange(8)) & 1).reshape(P, H, ps, 128).bool()
    m = cut[2].reshape(P, H, ps, 2).to(torch.int64)
    mu = ((m[..., 0] << 16) | (m[..., 1] << 24)).to(torch.int32).view(torch.float32).to(F64)
    e = cut[3].reshape(P, H, ps).to(torch.int64)
    return codes[..., :d], codes[..., d:], neg, mu, torch.where(e > 127, e - 256, e)


def visible(p, n, causal, window, sinks):
    """Which of the keys 0 .. n - 1 a token at position p sees."""
    j = torch.arange(n)
    see = torch.ones(n, dtype=torch.bool)
    if causal:
        see &= j <= p
        if window:
            see &= (j > p - window) | (j < sinks)
    return see


def attend(q, block, ps, d, table, kv_lens, cu, causal=True, window=0, sinks=0, scale=0.0, eps_out=0.0):
    """(o, lse, tolerance of o, tolerance of lse) for q [T, Hq, d]; rows of no sequence are NaN.

    The tolerances count the kernels' roundings. A weight carries half a step of fp16 (2^-11) and the error of its
    exponent: scores are a few fp32 products of at most max|s|, together within 2^-19 (1 + max|s|). Weights below
    fp16's normal range are off by at most 2^-25 of the largest weight's unit, times a code of at most 127 in the
    largest exponent. The product adds n / 16 partial sums in fp32. The output rounds once.
    With few rows the weights are fixed-point numbers instead, in units of 1 / 65280 of the largest w_j 2^e_j of a
    block: each of the n weights is off by at most half a unit, times a code of at most 127.
    """
    codes, _, neg, mu, ex = split_block(block, ps, d)
    P, Hkv = block.shape[:2]
    T, Hq = q.shape[:2]
    G = Hq // Hkv
    scale = scale or 1.0 / math.sqrt(d)
    o = torch.full((T, Hq, d), math.nan, dtype=F64)
    lse = torch.full((T, Hq), math.nan, dtype=F64)
    to, tl = torch.zeros_like(o), torch.zeros_like(lse)
    q = q.to(F64)
    for b in range(len(kv_lens)):
        n, t0, t1 = int(kv_lens[b]), int(cu[b]), int(cu[b + 1])
        j = torch.arange(n)
        page = table[b].long()[j // ps] if n else torch.empty(0, dtype=torch.long)
        have = (page >= 0) & (page < P)
        pg = page.clamp(0, max(P - 1, 0))
        kh = torch.where(neg[pg, :, j % ps][..., :d], -1.0, 1.0).to(F64) * mu[pg, :, j % ps][..., None]
        e = ex[pg, :, j % ps]
        vh = codes[pg, :, j % ps].to(F64) * (2.0 ** e.to(F64))[..., None]
        for i in range(t1 - t0):
            p = n - (t1 - t0) + i
            see = visible(p, n, causal, window, sinks) & have
            for h in range(Hq):
                x = q[t0 + i, h]
                if not see.any():
                    o[t0 + i, h] = 0.0
                    lse[t0 + i, h] = -math.inf
                    continue
                y = torch.where(x < 0, -1.0, 1.0).to(F64) * x.abs().mean() * scale
                kk, vv = kh[see, h // G], vh[see, h // G]
                s = kk @ y
                w = torch.softmax(s, 0)
                o[t0 + i, h] = w @ vv
                lse[t0 + i, h] = torch.logsumexp(s, 0)
                big, m = float(s.abs().max()), int(see.sum())
                up = 2.0 ** int(e[see, h // G].max())
                A = w @ vv.abs()
                to[t0 + i, h] = A * (2.0 ** -11 + 2.0 ** -18 * (1 + big) + (m / 16) * 2.0 ** -23) \
                    + m * 2.0 ** -25 * 127 * up \
                    + m * 127 * 0.5 / 65280 * float((w * 2.0 ** e[see, h // G].to(F64)).max()) + o[t0 + i, h].abs() * eps_out / 2 * (1 + 2.0 ** -10)
                tl[t0 + i, h] = 2.0 ** -19 * (1 + big) + m * 2.0 ** -26
    return o, lse, to, tl
