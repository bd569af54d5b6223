"""Measured cases of the paged binary KV cache: writing it, reading it back, and attention over it.

A cache row of one token and KV head holds the sign bits of k (128 bits), their scale mu (bf16, the mean
of |k|), the 8-bit codes of v and one power-of-two exponent for them. The plain forms below state each
operator in elementary torch operations.
"""
import math

import torch

own = False


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # one new token of each of 8 sequences enters the cache: latency
        {"name": "write_tokens", "op": "write", "tokens": 8, "kv_heads": 16, "d": 64, "page": 16, "dtype": "bf16"},
        # ragged prompt of odd length, a head size that is no power of two, padded rows (slot -1)
        {"name": "write_odd", "op": "write", "tokens": 1531, "kv_heads": 16, "d": 72, "page": 48, "dtype": "f16"},
        # a long prompt enters the cache
        {"name": "write_prompt", "op": "write", "tokens": 16384, "kv_heads": 8, "d": 128, "page": 64, "dtype": "bf16"},
        # part of a context comes back as 16-bit numbers, for a layer that wants them
        {"name": "read_odd", "op": "read", "tokens": 4099, "kv_heads": 16, "d": 72, "page": 48, "dtype": "f16"},
        # a whole long context comes back
        {"name": "read_context", "op": "read", "tokens": 65536, "kv_heads": 8, "d": 128, "page": 64, "dtype": "bf16"},
        # one token of one sequence, short context: latency
        {"name": "decode_one", "op": "attend", "batch": 1, "q_max": 1, "kv_max": 1024, "heads": 32, "kv_heads": 8,
         "d": 128, "page": 16, "window": 0, "sinks": 0, "dtype": "bf16"},
        # one token of one sequence over a very long context
        {"name": "decode_long", "op": "attend", "batch": 1, "q_max": 1, "kv_max": 131072, "heads": 32, "kv_heads": 4,
         "d": 128, "page": 64, "window": 0, "sinks": 0, "dtype": "bf16"},
        # a served batch of ragged contexts, one token each
        {"name": "decode_batch", "op": "attend", "batch": 128, "q_max": 1, "kv_max": 8192, "heads": 32, "kv_heads": 8,
         "d": 128, "page": 64, "window": 0, "sinks": 0, "dtype": "bf16"},
        # a served batch with a sliding window and sinks, one KV head for each query head
        {"name": "decode_window", "op": "attend", "batch": 32, "q_max": 1, "kv_max": 16384, "heads": 16,
         "kv_heads": 16, "d": 64, "page": 32, "window": 4096, "sinks": 4, "dtype": "f16"},
        # small chunks of several sequences, odd sizes
        {"name": "chunk_odd", "op": "attend", "batch": 5, "q_max": 197, "kv_max": 1000, "heads": 16, "kv_heads": 16,
         "d": 72, "page": 48, "window": 0, "sinks": 0, "dtype": "f16"},
        # a chunk of a long prompt over what the cache holds of it
        {"name": "chunk_long", "op": "attend", "batch": 1, "q_max": 4096, "kv_max": 32768, "heads": 16, "kv_heads": 4,
         "d": 128, "page": 64, "window": 0, "sinks": 0, "dtype": "bf16"},
        # a long prompt with a sliding window and sinks
        {"name": "prompt_window", "op": "attend", "batch": 2, "q_max": 8192, "kv_max": 8192, "heads": 16,
         "kv_heads": 8, "d": 64, "page": 32, "window": 1024, "sinks": 4, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "read", "attend", "attend", "attend", "attend"])
    c = {"op": op, "kv_heads": rng.choice([1, 2, 3, 4, 8, 16]), "d": rng.choice([16, 40, 64, 64, 72, 80, 96, 120, 128, 128]),
         "page": rng.choice([16, 32, 48, 64, 128, 256]), "dtype": rng.choice(["bf16", "f16"])}
    if op != "attend":
        c["tokens"] = _log(rng, 1, 65536 // max(1, c["kv_heads"] // 8))
        return c
    form = rng.choice(["decode", "decode", "few", "chunk", "chunk"])
    c["heads"] = c["kv_heads"] * rng.choice([1, 2, 4, 7, 8])
    if form == "decode":
        c["q_max"] = 1
        c["batch"] = _log(rng, 1, 128)
        c["kv_max"] = _log(rng, 1, min(131072, (1 << 23) // (c["batch"] * c["kv_heads"])))
    elif form == "few":  # the tokens of a draft, verified together
        c["q_max"] = rng.randint(2, 16)
        c["batch"] = _log(rng, 1, 32)
        c["kv_max"] = c["q_max"] + _log(rng, 1, min(65536, (1 << 22) // (c["batch"] * c["kv_heads"])))
    else:
        c["q_max"] = _log(rng, 17, 4096)
        c["batch"] = rng.randint(1, 4)
        c["kv_max"] = c["q_max"] + _log(rng, 1, max(1, min(32768, (1 << 31) // (c["batch"] * c["heads"] * c["q_max"])) - c["q_max"]))
    c["window"] = rng.choice([0, 0, _log(rng, 16, 4096)])
    c["sinks"] = rng.choice([0, 1, 4, 16]) if c["window"] else 0
    return c


# --------------------------------------------------------------------------- inputs
_DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def _dp(d):
    return (d + 15) // 16 * 16


def _block_bytes(c):
    """Bytes of one page of one KV head: codes, sign rows, mu, exponents of `page` tokens."""
    return c["page"] * (_dp(c["d"]) + 16 + 2 + 1)


def _views(data, c):
    """(codes [P,H,ps,dp] int8, sign words [P,H,ps,4] int32, mu [P,H,ps] bf16, exponents [P,H,ps] int8) of a cache."""
    ps, dp = c["page"], _dp(c["d"])
    P, H = data.shape[:2]
    at = [0, ps * dp, ps * (dp + 16), ps * (dp + 18), ps * (dp + 19)]
    part = [data[:, :, at[i]:at[i + 1]] for i in range(4)]
    return (part[0].view(torch.int8).unflatten(2, (ps, dp)), part[1].view(torch.int32).unflatten(2, (ps, 4)),
            part[2].view(torch.bfloat16), part[3].view(torch.int8))


def _lengths(c):
    """Token counts of the sequences: ragged, the first of the full length. (new tokens, context lengths)"""
    b = c["batch"]
    kv = [c["kv_max"]] + [max(1, c["kv_max"] * (b - i) // b - 3 * i) for i in range(1, b)]
    q = [c["q_max"]] + [max(1, c["q_max"] * (b - i) // b) for i in range(1, b)]
    return [min(x, y) for x, y in zip(q, kv)], kv


def _filled_cache(c, pages, gen):
    """A cache in use: signs that agree with a per-head direction three times in four, mu around 0.8, codes of
    normal values, exponents that go with them."""
    dev, H, d, dp, ps = "cuda", c["kv_heads"], c["d"], _dp(c["d"]), c["page"]
    data = torch.zeros((pages, H, _block_bytes(c)), dtype=torch.uint8, device=dev)
    codes, bits, mu, ex = _views(data, c)
    keep = torch.tensor([-1 if d >= 32 * w + 32 else (1 << max(0, d - 32 * w)) - 1 for w in range(4)],
                        dtype=torch.int32, device=dev)
    word = lambda *shape: torch.randint(-2**31, 2**31, shape, dtype=torch.int32, device=dev, generator=gen)
    base = word(1, H, 1, 4)
    bits.copy_((base ^ (word(pages, H, ps, 4) & word(pages, H, ps, 4))) & keep)
    mu.copy_(0.8 * torch.exp(0.25 * torch.randn((pages, H, ps), device=dev, generator=gen)))
    v = torch.randn((pages, H, ps, d), device=dev, dtype=torch.bfloat16, generator=gen)
    codes[..., :d].copy_((v * 30).round().clamp(-127, 127))
    ex.copy_(torch.randint(-6, -3, (pages, H, ps), device=dev, generator=gen))
    return data, base[0, :, 0]


def prepare(case, seed):
    c = case
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    dt = _DT[c["dtype"]]
    H, d = c["kv_heads"], c["d"]
    s = {"case": c}
    if c["op"] != "attend":
        T = c["tokens"]
        pages = -(-T // c["page"]) + 3
        slots = torch.randperm(pages * c["page"], device=dev, generator=gen)[:T]
        if c["op"] == "write":
            # k and v as slices of one fused projection; every 17th token is a row of padding
            kv = torch.randn((T, 2, H, d), device=dev, generator=gen)
            kv[:, 0] += 0.5 * torch.randn((H, d), device=dev, generator=gen)
            kv = kv.to(dt)
            slots[16::17] = -1
            s |= {"k": kv[:, 0], "v": kv[:, 1],
                  "data": torch.zeros((pages, H, _block_bytes(c)), dtype=torch.uint8, device=dev)}
        else:
            s["data"] = _filled_cache(c, pages, gen)[0]
        s["slots"] = slots
        return s
    qn, kn = _lengths(c)
    per = -(-c["kv_max"] // c["page"])
    need = sum(-(-n // c["page"]) for n in kn)
    s["data"], base = _filled_cache(c, need + 2, gen)
    perm = torch.randperm(need + 2, device=dev, generator=gen)[:need].to(torch.int32)
    table = torch.full((c["batch"], per), -1, dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(kn):
        m = -(-n // c["page"])
        table[b, :m] = perm[at:at + m]
        at += m
    T, G = sum(qn), c["heads"] // H
    # queries that lean towards their KV head's direction, so that attention is not flat
    lean = 1.0 - 2.0 * ((base[:, :, None] >> torch.arange(32, device=dev, dtype=torch.int32)) & 1).flatten(1)[:, :d].float()
    q = torch.randn((T, H, G, d), device=dev, generator=gen) + 0.4 * lean[:, None]
    s |= {"q": q.view(T, c["heads"], d).to(dt), "table": table,
          "kv_lens": torch.tensor(kn, dtype=torch.int32, device=dev),
          "cu": torch.tensor([0] + qn, dtype=torch.int32, device=dev).cumsum(0, dtype=torch.int32)}
    return s


# --------------------------------------------------------------------------- plain forms
def _read(s, slots):
    """k^ = mu * sign and v^ = code * 2^e of the rows at `slots` [...]; rows of slot -1 are 0. fp32 [..., H, d]."""
    c = s["case"]
    codes, bits, mu, ex = _views(s["data"], c)
    ok = slots >= 0
    at = slots.clamp(min=0)
    page, off = at // c["page"], at % c["page"]
    w = bits[page, :, off]
    sign = (w[..., None] >> torch.arange(32, device=w.device, dtype=torch.int32)) & 1
    sign = 1.0 - 2.0 * sign.flatten(-2)[..., :c["d"]]
    m = (mu[page, :, off].float() * ok[..., None])[..., None]
    e = (torch.exp2(ex[page, :, off].float()) * ok[..., None])[..., None]
    return sign, m, codes[page, :, off][..., :c["d"]].float() * e


def _write(s):
    """Sign bits, mu, codes and exponents of the new rows, put at their slots (-1: nowhere)."""
    c = s["case"]
    d, dp = c["d"], _dp(c["d"])
    codes, bits, mu, ex = _views(s["data"], c)
    k, v, slots = s["k"].double(), s["v"].float(), s["slots"]
    T, H = k.shape[:2]
    neg = torch.nn.functional.pad((k < 0).to(torch.int64), (0, 128 - d)).view(T, H, 4, 32)
    words = (neg << torch.arange(32, device=k.device)).sum(-1)
    words = torch.where(words >= 2**31, words - 2**32, words).to(torch.int32)
    mean = k.abs().mean(-1).to(torch.bfloat16)
    amax = v.abs().amax(-1)
    mant, ex2 = torch.frexp(amax)
    e = torch.where(mant <= 127.0 / 128.0, ex2 - 7, ex2 - 6)
    e = torch.where(amax == 0, torch.full_like(e, -24), e).clamp(-24, 9)
    code = torch.round(v * torch.exp2(-e.float())[..., None]).clamp(-127, 127).to(torch.int8)
    code = torch.nn.functional.pad(code, (0, dp - d))
    # a padded row writes again what its slot 0 row gets, or what is there: select instead of dropping rows
    ok = slots >= 0
    at = slots.clamp(min=0)
    page, off = at // c["page"], at % c["page"]
    first = torch.argmax((slots == 0).to(torch.int32))  # the row that goes to slot 0, if any
    some = (slots[first] == 0)

    def put(dst, new):
        old = torch.where(some, new[first], dst[0, :, 0])
        shape = (-1,) + (1,) * (new.dim() - 1)
        dst[page, :, off] = torch.where(ok.view(shape), new, old[None])

    put(codes, code)
    put(bits, words)
    put(mu, mean)
    put(ex, e.to(torch.int8))


def _attend(s):
    c = s["case"]
    B, H, d, L, Q = c["batch"], c["kv_heads"], c["d"], c["kv_max"], c["q_max"]
    G = c["heads"] // H
    q, cu, kv = s["q"], s["cu"].long(), s["kv_lens"].long()
    dev, T = q.device, q.shape[0]
    qn = cu[1:] - cu[:-1]
    pos = torch.arange(L, device=dev)
    pages = s["table"].long()[:, pos // c["page"]]  # [B,L]
    slots = torch.where(pages >= 0, pages * c["page"] + pos % c["page"], pages)
    sign, mu, v = _read(s, slots)  # [B,L,H,d]
    i = torch.arange(Q, device=dev)
    qp = q[(cu[:-1, None] + i).clamp(max=T - 1)].float()  # [B,Q,Hq,d]
    qs = torch.where(qp < 0, -1.0, 1.0).view(B, Q, H, G, d).permute(0, 2, 3, 1, 4).reshape(B, H, G * Q, d)
    mq = qp.abs().mean(-1).view(B, Q, H, G).permute(0, 2, 3, 1).reshape(B, H, G * Q, 1)
    x = qs @ sign.permute(0, 2, 3, 1)  # whole numbers
    x = x * (mq / math.sqrt(d)) * mu.permute(0, 2, 3, 1)
    x = x.view(B, H, G, Q, L)
    p = (kv - qn)[:, None, None] + i[:, None]  # position of query i: [B,Q,1]
    see = (pos < kv[:, None, None]) & (pos <= p)
    if c["window"]:
        see &= (pos > p - c["window"]) | (pos < c["sinks"])
    x = x.masked_fill_(~see[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    x = x.sub_(m).exp_()
    l = x.sum(-1, keepdim=True)
    o = (x.view(B, H, G * Q, L) @ v.permute(0, 2, 1, 3)).view(B, H, G, Q, d)
    o = torch.where(l > 0, o / l, 0.0)
    lse = (m + torch.log(l))[..., 0]
    t = torch.arange(T, device=dev)
    b = torch.bucketize(t, cu[1:], right=True)
    o = o.permute(0, 3, 1, 2, 4)[b, t - cu[b]].reshape(T, H * G, d).to(q.dtype)
    return {"o": o, "lse": lse.permute(0, 3, 1, 2)[b, t - cu[b]].reshape(T, H * G)}


def run(state):
    s, c = state, state["case"]
    dt = _DT[c["dtype"]]
    if own:
        import bit_qk_attention_b200 as ba
        cache = ba.KVCache(s["data"], c["page"], c["d"])
        if c["op"] == "attend":
            o, lse = ba.attention_paged(s["q"], cache, s["table"], s["kv_lens"], s["cu"], max_q_len=c["q_max"],
                                        max_kv_len=c["kv_max"], window=c["window"], sinks=c["sinks"], return_lse=True)
            return {"o": o, "lse": lse}
        if c["op"] == "write":
            ba.cache_write(cache, s["k"], s["v"], s["slots"])
        k, v = ba.cache_read(cache, s["slots"], dtype=dt)
        return {"k": k, "v": v}
    if c["op"] == "attend":
        return _attend(s)
    if c["op"] == "write":  # what went in is what comes back out of it
        _write(s)
    sign, mu, v = _read(s, s["slots"])
    return {"k": (sign * mu).to(dt), "v": v.to(dt)}


# --------------------------------------------------------------------------- cost and definition
def work(case):
    c = case
    H, d, dp = c["kv_heads"], c["d"], _dp(c["d"])
    row = dp + 19
    if c["op"] != "attend":
        n = c["tokens"] * H
        io = 2 * n * d * 2
        # a write reads 16-bit rows and writes cache rows; both cases read cache rows and write 16-bit rows
        return {"bytes": (2 if c["op"] == "write" else 1) * (io + n * row) + 8 * c["tokens"], "flops": 0}
    qn, kn = _lengths(c)
    pairs = keys = 0
    for a, n in zip(qn, kn):
        w = c["window"] or n
        first = n - a  # position of the first query
        used = min(n, w + a - 1)
        keys += used + min(c["sinks"], n - used)
        # sum over positions p of min(p + 1, w), and the sinks before the window
        full = max(0, n - max(first, w))
        part = (first + 1 + min(n, w)) * (min(n, w) - first) // 2 if first < min(n, w) else 0
        pairs += full * w + part + sum(min(c["sinks"], p + 1 - w) for p in range(max(first, w), min(n, w + c["sinks"])))
        pairs += c["sinks"] * max(0, n - max(first, w + c["sinks"]))
    io = 2 * sum(qn) * c["heads"] * d * 2 + sum(qn) * c["heads"] * 4
    return {"bytes": keys * H * row + io, "flops": 4 * d * c["heads"] * pairs}


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    H, d, dp, ps = c["kv_heads"], c["d"], _dp(c["d"]), c["page"]
    f64 = torch.float64
    if c["op"] == "write":
        k, v = s["k"].to(f64), s["v"].to(f64)
        live = (s["slots"] >= 0).to(f64)[:, None, None]
        mu = (k.abs().sum(-1, keepdim=True) / d).to(torch.bfloat16).to(f64)
        khat = torch.where(k < 0, -mu, mu)
        amax = v.abs().amax(-1, keepdim=True)
        step = torch.full_like(amax, 2.0 ** -24)
        for n in range(-24, 9):  # the least power of two that holds the largest value
            step = torch.where(amax > 127 * 2.0 ** n, 2.0 ** (n + 1), step)
        vhat = (v / step).round().clamp(-127, 127) * step
        return {"k": khat * live, "v": vhat * live}
    raw = s["data"]
    power = torch.tensor([2.0 ** n for n in range(-128, 128)], dtype=f64, device=raw.device)

    def rows(page, off):
        """k^ and v^ [n, H, d] of the rows (page, off), from the bytes of the cache."""
        blk = raw[page].view(len(page), H, -1)
        n = torch.arange(len(page), device=raw.device)

        def piece(start, width):
            cols = start + off[:, None] * width + torch.arange(width, device=raw.device)
            return blk[n[:, None], :, cols].permute(0, 2, 1)  # [n,H,width]

        byte = piece(ps * dp, 16)
        ch = torch.arange(d, device=raw.device)
        neg = (byte[:, :, ch // 8].to(torch.int32) >> (ch % 8).to(torch.int32)) & 1
        m = piece(ps * (dp + 16), 2).to(torch.int32)
        m = ((m[..., 0] << 16) | (m[..., 1] << 24)).view(torch.float32).to(f64)
        ee = piece(ps * (dp + 18), 1)[..., 0].contiguous().view(torch.int8).long()
        val = piece(0, dp)[..., :d].contiguous().view(torch.int8).to(f64)
        return m[..., None] * (1 - 2 * neg.to(f64)), val * power[ee + 128][..., None]

    if c["op"] == "read":
        k = torch.empty((c["tokens"], H, d), dtype=f64, device=raw.device)
        v = torch.empty_like(k)
        for a in range(0, c["tokens"], 2048):
            sl = s["slots"][a:a + 2048]
            k[a:a + 2048], v[a:a + 2048] = rows(sl // ps, sl % ps)
        return {"k": k, "v": v}
    qn, kn = _lengths(c)
    G = c["heads"] // H
    o = torch.zeros((sum(qn), c["heads"], d), dtype=f64, device=raw.device)
    lse = torch.zeros((sum(qn), c["heads"]), dtype=f64, device=raw.device)
    at = 0
    for b, (a, n) in enumerate(zip(qn, kn)):
        pos = torch.arange(n, device=raw.device)
        parts = [rows(s["table"][b].long()[x // ps], x % ps) for x in pos.split(4096)]
        kk, vv = (torch.cat([x[i] for x in parts]) for i in (0, 1))
        for lo in range(0, a, 1024):
            m = min(1024, a - lo)
            p = n - a + lo + torch.arange(m, device=raw.device)[:, None]
            see = pos <= p
            if c["window"]:
                see = see & ((p - pos < c["window"]) | (pos < c["sinks"]))
            for h in range(c["heads"]):
                x = s["q"][at + lo:at + lo + m, h].to(f64)
                y = torch.where(x < 0, -1.0, 1.0).to(f64) * x.abs().mean(-1, keepdim=True) / math.sqrt(d)
                z = (y @ kk[:, h // G].T).masked_fill(~see, -math.inf)
                lse[at + lo:at + lo + m, h] = torch.logsumexp(z, -1)
                o[at + lo:at + lo + m, h] = torch.softmax(z, -1) @ vv[:, h // G]
        at += a
    return {"o": o, "lse": lse}
