"""Calls of the paged cache that the documentation allows and that are easy to get wrong, on the GPU against the
definition in 64 bits (tests/paged_ref.py) or a closed form."""
import math

import pytest
import torch

import paged_ref
from paged_ref import F64
from test_gpu_paged import DT, _check_rows, _compare, _gen, _problem, _ref, _run, ba  # noqa: F401 (ba: fixture)

pytestmark = pytest.mark.gpu


# ----------------------------------------------------------------------------- unseen rows
@pytest.mark.parametrize("qn", [65, 300])
@pytest.mark.parametrize("ps,n", [(64, 3 * 128 + 32 + 10), (64, 3 * 128 + 96 + 10), (16, 3 * 128 + 10),
                                  (16, 3 * 128 + 64 + 10), (32, 3 * 128 + 32 + 10)])
def test_nan_scales_behind_a_sequence_that_ends_in_its_largest_keys(ba, ps, n, qn):
    """The last keys score far above all before, and the unused rows beside them hold NaN scales: in the same 32 keys,
    with a neighbour of visible keys, or of no page at all."""
    d, g = 128, _gen(ps + n + qn)
    P = -(-n // ps)
    c = ba.KVCache.zeros(P, 1, d, ps)
    c.data.fill_(0xFF)
    k, v = (torch.randn((n, 1, d), generator=g).bfloat16() for _ in range(2))
    q = torch.randn((qn, 2, d), generator=g).bfloat16()
    k[-10:] = q[-1, 0] * 30
    ba.cache_write(c, k.cuda(), v.cuda(), torch.arange(n).cuda())
    prob = (c, q, torch.arange(P, dtype=torch.int32)[None], torch.tensor([n], dtype=torch.int32),
            torch.tensor([0, qn], dtype=torch.int32))
    for causal in (True, False):
        _compare(*_run(ba, prob, causal=causal), _ref(ba, prob, causal=causal), f"causal {causal}")


@pytest.mark.parametrize("qn", [65, 130])
def test_nan_scales_before_a_window_that_begins_with_its_largest_keys(ba, qn):
    """Rows that the window has left behind hold NaN scales, next to the largest keys; the sinks came before them."""
    d, ps, n, lo, sinks = 128, 16, 700, 276, 4
    window = n - qn - lo + 1  # the first new token sees the keys from lo on
    g = _gen(qn)
    P = -(-n // ps)
    c = ba.KVCache.zeros(P, 1, d, ps)
    k, v = (torch.randn((n, 1, d), generator=g).bfloat16() for _ in range(2))
    q = torch.randn((qn, 2, d), generator=g).bfloat16()
    k[lo + 4:lo + 12] = q[0, 0] * 30
    ba.cache_write(c, k.cuda(), v.cuda(), torch.arange(n).cuda())
    j = torch.arange(P * ps)
    gone = ((j >= sinks) & (j < lo)).view(P, 1, ps).cuda()
    c.k_mu[gone] = math.nan
    c.v_exp[gone] = 127
    prob = (c, q, torch.arange(P, dtype=torch.int32)[None], torch.tensor([n], dtype=torch.int32),
            torch.tensor([0, qn], dtype=torch.int32))
    kw = dict(window=window, sinks=sinks)
    _compare(*_run(ba, prob, **kw), _ref(ba, prob, **kw))


# ----------------------------------------------------------------------------- weights far below the largest
@pytest.mark.parametrize("below", [20.5, 25.5])
@pytest.mark.parametrize("qn", [1, 130])
@pytest.mark.parametrize("large_scale", [False, True])
def test_many_small_weights_beside_one_large(ba, large_scale, qn, below):
    """One key holds nearly all of the mass, and its values are 0: o is what the others, each 2^-below of it, add up to.

    With w = 2^-below and n - 1 keys of value 1 beside the large one, o = (n - 1) w / (1 + (n - 1) w). A weight
    of the kernel for many rows is off by at most 2^-11 of itself or 2^-32 of the largest (2^-28 where a key's scale
    would allow scores far above those there are). One of the kernel for
    few rows is off by at most 2^-17 of the largest w 2^e of its 64 keys: beside the large key, whose values of 0 have
    the exponent -24, that is 2^-9.5 of itself for 63 of n keys, else 2^-17. Scores are fp32 numbers up to 26, off
    by at most 2^-19 (1 + 26), and o rounds once to fp32."""
    d, ps, n = 64, 128, 16384
    B = torch.cuda.get_device_properties(0).multi_processor_count  # as many (tile, head)s: none of them is cut
    c = ba.KVCache.zeros(n // ps, 1, d, ps)
    k = torch.ones((n, 1, d), dtype=torch.bfloat16)
    k[1:, :, ::2] = -1.0  # half of the signs differ: score 0
    if large_scale:
        k[5] *= 64.0  # a score of 0 too
    v = torch.ones_like(k)
    v[0] = 0.0
    ba.cache_write(c, k.cuda(), v.cuda(), torch.arange(n).cuda())
    q = torch.ones((B * qn, 1, d), dtype=torch.bfloat16).cuda()
    table = torch.arange(n // ps, dtype=torch.int32)[None].expand(B, -1).cuda()
    kv = torch.full((B,), n, dtype=torch.int32).cuda()
    cu = torch.arange(0, B * qn + 1, qn, dtype=torch.int32).cuda()
    scale = below * math.log(2.0) / d
    o, lse = ba.attention_paged(q, c, table, kv, cu, max_q_len=qn, causal=False, softmax_scale=scale,
                                out_dtype=torch.float32, return_lse=True)
    torch.cuda.synchronize()
    ba.check_device_status()
    mass = (n - 1) * 2.0 ** -below
    want = mass / (1 + mass)
    tol = want * (2.0 ** -11 + 2.0 ** -19 * 27 + 2.0 ** -23) + n * 2.0 ** (-28 if large_scale else -32)
    assert ((o.double() - want).abs() <= tol).all(), (float((o.double() - want).abs().max()), tol)
    want = below * math.log(2.0) + math.log1p(mass)
    assert ((lse.double() - want).abs() <= 2.0 ** -19 * 27 + n * 2.0 ** -26).all()


# ----------------------------------------------------------------------------- sizes
@pytest.mark.parametrize("bound", [None, 128])
def test_a_large_batch_of_short_sequences_with_the_default_bound(ba, bound):
    """65536 new tokens of 512 sequences in one call: the bound of their lengths is the number of all new tokens
    unless the caller gives one."""
    B, each, Hq, Hkv, d, ps = 512, 128, 64, 8, 16, 128
    g = _gen(40)
    c = ba.KVCache.zeros(B, Hkv, d, ps)
    k, v = (torch.randn((B * each, Hkv, d), generator=g).bfloat16() for _ in range(2))
    ba.cache_write(c, k.cuda(), v.cuda(), torch.arange(B * each).cuda())
    q = torch.randn((B * each, Hq, d), generator=g).bfloat16()
    kv = torch.full((B,), each, dtype=torch.int32)
    kv[3], kv[200] = 60, 0  # fewer keys than new tokens
    table = torch.arange(B, dtype=torch.int32)[:, None].contiguous()
    cu = torch.arange(0, B * each + 1, each, dtype=torch.int32)
    o, lse = _run(ba, (c, q, table, kv, cu), max_q_len=bound)
    for b in (0, 3, 200, 511):
        rows = slice(b * each, (b + 1) * each)
        one = ba.KVCache(c.data[b:b + 1], ps, d)
        ref = _ref(ba, (one, q[rows, ::8], torch.zeros((1, 1), dtype=torch.int32), kv[b:b + 1], torch.tensor([0, each])))
        _compare(o[rows, ::8], lse[rows, ::8], ref, f"sequence {b}")
    assert torch.isfinite(o).all()


# ----------------------------------------------------------------------------- errors
def test_an_allocation_that_fails_raises_out_of_memory(ba):
    """Results that do not fit the device: the error that a server catches, and the next call works."""
    c = ba.KVCache.zeros(1, 1, 128, 16)
    T, H = 4_000_000, 128  # 262 GB of fp32 results; q and the lists take next to nothing
    q = torch.zeros((1, 1, 128), dtype=torch.bfloat16, device="cuda").expand(T, H, 128)
    table, kv = torch.zeros((1, 1), dtype=torch.int32, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    with pytest.raises(torch.OutOfMemoryError):
        ba.attention_paged(q, c, table, kv, cu, max_q_len=1, out_dtype=torch.float32)
    slots = torch.zeros(1, dtype=torch.int64, device="cuda").expand(T * H // 16).contiguous()
    big = ba.KVCache(c.data.expand(1, 16, -1).contiguous(), 16, 128)
    with pytest.raises(torch.OutOfMemoryError):
        ba.cache_read(big, slots, torch.float32)
    o = ba.attention_paged(q[:1], c, table, kv, cu, max_q_len=1)
    torch.cuda.synchronize()
    assert not o[0].any()


@pytest.mark.parametrize("qn,kn,kw", [([1], [20000], {}), ([1, 1], [9000, 40], dict(max_q_len=1)), ([60, 200], [9000, 4000], {}),
                                      ([60, 200], [9000, 4000], dict(max_q_len=200, max_kv_len=1 << 40, window=1 << 35, sinks=3)),
                                      ([3], [40], {})])
def test_a_workspace_of_the_bytes_that_the_package_tells(ba, qn, kn, kw):
    """With the bytes of paged_workspace_bytes the call gives what it gives by itself; with 16 fewer it is refused."""
    c, q, table, kv, cu = _problem(ba, qn, kn, 8, 2, 128, 64, "bf16", 50)
    args = (q.cuda(), c, table.cuda(), kv.cuda(), cu.cuda())
    need = ba.paged_workspace_bytes(*args, **kw)
    want = ba.attention_paged(*args, **kw)
    guard = torch.full((need + 256,), 0xAB, dtype=torch.uint8, device="cuda")
    got = ba.attention_paged(*args, workspace=guard[:need], **kw)
    assert torch.equal(got, want) and (guard[need:] == 0xAB).all()
    if need:
        with pytest.raises(ba.BinAttnError) as e:
            ba.attention_paged(*args, workspace=guard[:need - 16], **kw)
        assert e.value.status == 4
    else:
        assert kn == [40]
    with pytest.raises(ValueError):
        ba.paged_workspace_bytes(*args, window=-1)
    torch.cuda.synchronize()


# ----------------------------------------------------------------------------- ends of bf16's range
@pytest.mark.parametrize("d", [1, 5, 32, 72, 128])
def test_write_of_the_largest_numbers(ba, d):
    """The mean of numbers near bf16's largest is one of them, though their sum is beyond fp32; and the mean of the
    least ones does not vanish."""
    ps, top, least = 16, torch.finfo(torch.bfloat16).max, 2.0 ** -133
    g = _gen(d)
    rows = [torch.full((d,), top), -torch.full((d,), top), torch.full((d,), top / 2), torch.full((d,), least),
            torch.full((d,), 3 * least), torch.rand((d,), generator=g) * top,
            torch.full((d,), torch.finfo(torch.bfloat16).smallest_normal)]
    k = torch.stack(rows).bfloat16()[:, None]
    v = torch.randn(k.shape, generator=g).bfloat16()
    c = ba.KVCache.zeros(1, 1, d, ps)
    slots = torch.arange(len(rows))
    ba.cache_write(c, k.cuda(), v.cuda(), slots.cuda())
    _check_rows(c.data.cpu(), ps, d, k, v, slots)
    kk, _ = ba.cache_read(c, slots.cuda(), torch.float32)
    assert torch.isfinite(kk).all()


@pytest.mark.parametrize("qn", [1, 20, 150])
def test_queries_of_the_largest_numbers(ba, qn):
    """mean |q| within fp32 although the sum is not; keys as small make scores of ordinary size."""
    d, ps, n = 64, 16, 300
    g = _gen(qn)
    c = ba.KVCache.zeros(-(-n // ps), 1, d, ps)
    k, v = (torch.randn((n, 1, d), generator=g) for _ in range(2))
    ba.cache_write(c, (k * 2.0 ** -122).bfloat16().cuda(), v.bfloat16().cuda(), torch.arange(n).cuda())
    q = (torch.randn((qn, 2, d), generator=g).sign() * 2.0 ** 123).bfloat16()
    prob = (c, q, torch.arange(c.num_pages, dtype=torch.int32)[None], torch.tensor([n], dtype=torch.int32),
            torch.tensor([0, qn], dtype=torch.int32))
    _compare(*_run(ba, prob), _ref(ba, prob))


@pytest.mark.parametrize("qn", [1, 20, 150])
def test_queries_of_zeros_over_very_large_keys(ba, qn):
    """A row of q that is 0 has scores of 0, however large the keys' scales are."""
    d, ps, n = 64, 16, 300
    g = _gen(qn + 1)
    c = ba.KVCache.zeros(-(-n // ps), 1, d, ps)
    k, v = (torch.randn((n, 1, d), generator=g) for _ in range(2))
    ba.cache_write(c, (k * 2.0 ** 115).bfloat16().cuda(), v.bfloat16().cuda(), torch.arange(n).cuda())
    q = torch.zeros((qn, 2, d), dtype=torch.bfloat16)
    q[::3, 1] = (torch.randn((d,), generator=g) * 2.0 ** -115).bfloat16()  # and one whose scores are ordinary
    prob = (c, q, torch.arange(c.num_pages, dtype=torch.int32)[None], torch.tensor([n], dtype=torch.int32),
            torch.tensor([0, qn], dtype=torch.int32))
    for causal in (True, False):
        _compare(*_run(ba, prob, causal=causal), _ref(ba, prob, causal=causal))


# ----------------------------------------------------------------------------- the roundings of each kernel
def _weighed(prob, scale, few):
    """(o, lse, tolerances) of a causal problem, with the roundings of one kernel and no others.

    A score is a product of five fp32 numbers (mean |q| a sum of at most 9 steps and a quotient, the scale four
    operations more): within 2^-24 (20 |s| + 40) of s + e ln 2, |e| <= 24. exp2 adds 2^-21 at most. Sums of m
    positive numbers take m / 16 + 20 steps of 2^-24 at most. Numerator and softmax sum have both.
    Few rows: a weight w 2^e is off by half of 1 / 65280 of the largest of its 64 keys. Many: by 2^-11 of itself, or
    2^-28 of the row's largest. o rounds once to fp32."""
    c, q, table, kv_lens, cu = prob
    codes, _, neg, mu, ex = paged_ref.split_block(c.data.cpu(), c.page_size, c.d)
    T, Hq, d = q.shape
    G = Hq // c.n_kv_heads
    o, lse = torch.zeros((T, Hq, d), dtype=F64), torch.zeros((T, Hq), dtype=F64)
    to, tl = torch.zeros_like(o), torch.zeros_like(lse)
    for b in range(len(kv_lens)):
        n, t0, t1 = int(kv_lens[b]), int(cu[b]), int(cu[b + 1])
        j = torch.arange(n)
        pg, off = table[b].long()[j // c.page_size], j % c.page_size
        for h in range(Hq):
            k = torch.where(neg[pg, h // G, off][:, :d], -1.0, 1.0).to(F64) * mu[pg, h // G, off][:, None]
            e = 2.0 ** ex[pg, h // G, off].to(F64)
            code = codes[pg, h // G, off].to(F64)
            for i in range(t1 - t0):
                m = n - (t1 - t0) + i + 1
                x = q[t0 + i, h].to(F64)
                s = k[:m] @ (torch.where(x < 0, -1.0, 1.0).to(F64) * x.abs().mean() * scale)
                w, big = torch.softmax(s, 0), float(s.abs().max())
                we = w * e[:m]
                out, A = we @ code[:m], we @ code[:m].abs()
                rel = 2.0 ** -24 * (20 * big + 40) + 2.0 ** -21 + (m / 16 + 20) * 2.0 ** -24
                if few:
                    pad = (-m) % 64
                    top = torch.nn.functional.pad(we, (0, pad)).view(-1, 64).amax(1)
                    size = torch.nn.functional.pad(code[:m].abs(), (0, 0, 0, pad)).view(-1, 64, d).sum(1)
                    off_by = 0.5 / 65280 * (1 + 2.0 ** -10) * (top @ size)
                else:
                    off_by = 2.0 ** -11 * A + 2.0 ** -28 * w.max() * (e[:m, None] * code[:m].abs()).sum(0)
                o[t0 + i, h], lse[t0 + i, h] = out, torch.logsumexp(s, 0)
                to[t0 + i, h] = off_by + 2 * rel * A + out.abs() * 2.0 ** -24
                tl[t0 + i, h] = rel + lse[t0 + i, h].abs() * 2.0 ** -23
    return o, lse, to, tl


@pytest.mark.parametrize("d", [64, 72, 128])
@pytest.mark.parametrize("qn,kn,few", [([1], [1000], True), ([1, 1, 1], [64, 700, 129], True), ([4], [333], True), ([9], [500], True),
                                       ([70], [900], False), ([65, 90], [80, 400], False)])
def test_weights_have_the_bits_that_are_documented(ba, qn, kn, few, d):
    """fp32 results against the roundings of the kernel that makes them: some 2^-17 for few rows, 2^-11 for many."""
    prob = _problem(ba, qn, kn, 4, 2, d, 32, "bf16", 70 + d)
    scale = 0.25 / math.sqrt(d)
    got = _run(ba, prob, dt_out=torch.float32, softmax_scale=scale, max_q_len=max(qn))
    _compare(*got, _weighed(prob, scale, few))


# ----------------------------------------------------------------------------- very large scores
@pytest.mark.parametrize("scale", [1e3, 6e4])
@pytest.mark.parametrize("qn", [1, 20, 150])
def test_scores_up_to_the_limit(ba, qn, scale):
    """Scores of up to 2^24: each row's largest key takes all, though neighbouring fp32 numbers lie 1 apart.

    The keys' scales are 2^(-j / 8) in an order of its own, and all keys have the signs of q but for one channel, so
    that the largest visible score is 2^(1/8) or more above the next. (A bf16 scale is off by 2^-8 of itself.) The weight of
    that key, 1 or near it, may round to fp16."""
    d, ps, n = 128, 16, 400
    g = _gen(qn)
    sign = torch.randn((d,), generator=g).sign()
    k = sign * (2.0 ** (-torch.randperm(n, generator=g) / 8.0))[:, None]
    k[:, 0] *= -1.0
    v = torch.randn((n, 1, d), generator=g).bfloat16()
    c = ba.KVCache.zeros(-(-n // ps), 1, d, ps)
    ba.cache_write(c, k[:, None].bfloat16().cuda(), v.cuda(), torch.arange(n).cuda())
    q = (sign * (1 + torch.rand((qn, 2, 1), generator=g))).bfloat16()
    prob = (c, q, torch.arange(c.num_pages, dtype=torch.int32)[None], torch.tensor([n], dtype=torch.int32),
            torch.tensor([0, qn], dtype=torch.int32))
    mu, vh = c.k_mu[:, 0].flatten()[:n].float().cpu(), ba.cache_read(c, torch.arange(n).cuda(), torch.float32)[1][:, 0].cpu()
    for causal in (True, False):
        o, lse = _run(ba, prob, dt_out=torch.float32, softmax_scale=scale, causal=causal)
        for i in range(qn):
            top = int(mu[:n - qn + i + 1 if causal else n].argmax())
            want = scale * q[i].double().abs().mean(-1) * float(mu[top]) * (d - 2)
            assert ((o[i].cpu() - vh[top]).abs() <= vh[top].abs() * (2.0 ** -11 + 2.0 ** -20)).all(), (causal, i)
            assert ((lse[i].cpu().double() - want).abs() <= want * 2.0 ** -20).all()

