"""The paged cache on the GPU against its definition in 64 bits (tests/paged_ref.py): rows written and read back,
attention over them at the sizes, masks and layouts where it can go wrong, and all of it as a program uses it."""
import math

import pytest
import torch

import paged_ref
from paged_ref import F64

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def ba():
    assert torch.cuda.is_available(), "needs a CUDA device"
    from bit_qk_attention_b200 import build
    build.build()
    import bit_qk_attention_b200 as mod
    mod.lib()
    return mod


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _check_rows(block, ps, d, k, v, slots):
    """The written rows of a cache (on the CPU) against the definition."""
    codes, pad, neg, mu, ex = paged_ref.split_block(block, ps, d)
    want_neg, want_mu, want_e, want_codes = paged_ref.quantise(k, v)
    ok = (slots >= 0) & (slots < block.shape[0] * ps)
    pg, off = slots[ok] // ps, slots[ok] % ps
    assert torch.equal(neg[pg, :, off][..., :d], want_neg[ok]), "signs"
    assert not neg[pg, :, off][..., d:].any(), "bits past d"
    assert torch.equal(ex[pg, :, off], want_e[ok]), "exponents"
    assert torch.equal(codes[pg, :, off], want_codes[ok]), "codes"
    assert not pad[pg, :, off].any(), "codes past d"
    # bf16: half a step is 2^-8 of the value (2^-134 below the normal range); the fp32 sum adds far less than 2^-18
    diff = (mu[pg, :, off] - want_mu[ok]).abs()
    assert (diff <= want_mu[ok] * 2.0 ** -8 * (1 + 2.0 ** -10) + 2.0 ** -134).all(), "mu"


# ----------------------------------------------------------------------------- write
@pytest.mark.parametrize("T,H,d,ps,dt", [
    (1, 1, 128, 16, "bf16"), (1, 1, 1, 16, "f16"), (7, 3, 64, 16, "f16"), (33, 2, 72, 48, "bf16"),
    (40, 5, 17, 32, "f16"), (300, 8, 128, 64, "bf16"), (129, 1, 120, 1024, "f16"), (65, 4, 100, 80, "bf16")])
def test_write(ba, T, H, d, ps, dt):
    g = _gen(T * 131 + d)
    k = (torch.randn((T, H, d), generator=g) + 0.5).to(DT[dt])
    v = (torch.randn((T, H, d), generator=g) * 2.0 ** torch.randint(-9, 5, (T, H, 1), generator=g)).to(DT[dt])
    pages = -(-T // ps) + 2
    slots = torch.randperm(pages * ps, generator=g)[:T]
    slots[2::5] = -1
    slots[4::7] = pages * ps + 3
    c = ba.KVCache.zeros(pages, H, d, ps)
    c.data.fill_(0xA5)
    ba.cache_write(c, k.cuda(), v.cuda(), slots.cuda())
    block = c.data.cpu()
    _check_rows(block, ps, d, k, v, slots)
    # every other row is as it was
    left = torch.ones(pages * ps, dtype=torch.bool)
    left[slots[(slots >= 0) & (slots < pages * ps)]] = False
    raw = torch.cat([block[:, :, a * ps:b * ps].reshape(pages, H, ps, b - a).permute(0, 2, 1, 3).reshape(pages * ps, -1)
                     for a, b in ((0, c.v_codes.shape[3]), (c.v_codes.shape[3], c.v_codes.shape[3] + 16),
                                  (c.v_codes.shape[3] + 16, c.v_codes.shape[3] + 18),
                                  (c.v_codes.shape[3] + 18, c.v_codes.shape[3] + 19))], 1)
    assert (raw[left] == 0xA5).all()


@pytest.mark.parametrize("form", ["fused", "transposed", "one_off", "every_other", "broadcast"])
@pytest.mark.parametrize("d", [64, 40, 9])
def test_write_takes_strided_rows(ba, form, d):
    T, H, ps = 21, 3, 16
    g = _gen(d)
    if form == "fused":
        x = torch.randn((T, 2, H, d), generator=g).bfloat16().cuda()
        k, v = x[:, 0], x[:, 1]
    elif form == "transposed":
        k, v = (torch.randn((H, T, d), generator=g).bfloat16().cuda().transpose(0, 1) for _ in range(2))
    elif form == "one_off":
        x = torch.randn((2 * T * H * d + 1,), generator=g).bfloat16().cuda()[1:].view(2, T, H, d)
        k, v = x[0], x[1]
    elif form == "every_other":
        x = torch.randn((T, H, 2 * d + 1), generator=g).bfloat16().cuda()
        k, v = x[:, :, :d], x[:, :, d + 1:]
    else:
        k, v = (torch.randn((T, 1, d), generator=g).bfloat16().cuda().expand(T, H, d) for _ in range(2))
    slots = torch.randperm(2 * ps, generator=g)[:T]
    c = ba.KVCache.zeros(2, H, d, ps)
    ba.cache_write(c, k, v, slots.cuda())
    _check_rows(c.data.cpu(), ps, d, k.cpu(), v.cpu(), slots)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_write_special_values(ba, dt):
    """Zero rows, signed zeros, subnormals, the largest numbers, exact ties and the ends of the exponents' range."""
    d, ps = 32, 16
    big = torch.finfo(DT[dt]).max
    tiny = torch.finfo(DT[dt]).smallest_normal
    rows = [torch.zeros(d), -torch.zeros(d), torch.full((d,), big), torch.full((d,), -tiny / 4),
            torch.arange(d) - 15.5, (torch.arange(d) - 16) / 2, torch.linspace(-127, 127, d),
            torch.linspace(-127.5, 127.5, d), torch.full((d,), 127.0 * 2 ** 9), torch.full((d,), 128.0 * 2 ** 8),
            torch.full((d,), 2.0 ** -24), torch.full((d,), 2.0 ** -14), torch.arange(d) * 2.0 ** -20,
            torch.tensor([1.0, -1e-3] * (d // 2)), torch.tensor([254.0, 1.0, 3.0, 5.0] * (d // 4))]
    x = torch.stack(rows).to(DT[dt])[:, None]
    T = x.shape[0]
    c = ba.KVCache.zeros(1, 1, d, ps)
    slots = torch.arange(T)
    k = x.flip(0).contiguous()
    # a mean of the largest numbers is finite in bf16, whose range is that of fp32
    k[k.abs() == big] = 1.0
    ba.cache_write(c, k.cuda(), x.cuda(), slots.cuda())
    _check_rows(c.data.cpu(), ps, d, k, x, slots)


def test_a_row_with_inf_or_nan_leaves_the_others(ba):
    d, ps, T = 64, 16, 6
    g = _gen(3)
    k, v = (torch.randn((T, 2, d), generator=g).bfloat16() for _ in range(2))
    kb, vb = k.clone(), v.clone()
    kb[1, 0, 3], vb[1, 0, 5], kb[4, 1, 0], vb[4, 1, 1] = math.nan, math.inf, -math.inf, math.nan
    got = []
    for a, b in ((k, v), (kb, vb)):
        c = ba.KVCache.zeros(1, 2, d, ps)
        ba.cache_write(c, a.cuda(), b.cuda(), torch.arange(T).cuda())
        kk, vv = ba.cache_read(c, torch.arange(T).cuda(), torch.float32)
        got.append((kk.cpu(), vv.cpu()))
    same = torch.ones(T, 2, dtype=torch.bool)
    same[1, 0] = same[4, 1] = False
    for x, y in zip(*got):
        assert torch.equal(x[same], y[same])


# ----------------------------------------------------------------------------- read
@pytest.mark.parametrize("T,H,d,ps", [(1, 1, 128, 16), (37, 3, 72, 48), (50, 2, 9, 32), (200, 4, 64, 64)])
@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
def test_read(ba, T, H, d, ps, dt):
    """What was written comes back as mu * sign and code * 2^e; slots may repeat, those out of range give zeros."""
    g = _gen(T + d)
    pages = -(-T // ps) + 1
    k = torch.randn((T, H, d), generator=g).bfloat16()
    v = (torch.randn((T, H, d), generator=g) * 2.0 ** torch.randint(-20, 12, (T, H, 1), generator=g)).bfloat16()
    at = torch.randperm(pages * ps, generator=g)[:T]
    c = ba.KVCache.zeros(pages, H, d, ps)
    ba.cache_write(c, k.cuda(), v.cuda(), at.cuda())
    pick = torch.randint(0, T, (2 * T + 1,), generator=g)
    slots = at[pick]
    slots[1::4] = -1
    slots[2::9] = pages * ps
    gk, gv = ba.cache_read(c, slots.cuda(), DT[dt])
    assert gk.dtype == gv.dtype == DT[dt] and gk.shape == (2 * T + 1, H, d)
    codes, _, neg, mu, ex = paged_ref.split_block(c.data.cpu(), ps, d)
    live = ((slots >= 0) & (slots < pages * ps))[:, None, None].to(F64)
    s = slots.clamp(0, pages * ps - 1)
    kh = torch.where(neg[s // ps, :, s % ps][..., :d], -1.0, 1.0).to(F64) * mu[s // ps, :, s % ps][..., None] * live
    vh = codes[s // ps, :, s % ps].to(F64) * (2.0 ** ex[s // ps, :, s % ps].to(F64))[..., None] * live
    assert torch.equal(gk.cpu().to(F64), kh.to(DT[dt]).to(F64))  # one rounding, to fp16; exact in bf16 and fp32
    assert torch.equal(gv.cpu().to(F64), vh)                     # exact in every type
    # the quantisation itself: half a step of 2^e for each value, as long as it does not saturate
    v_err = (gv.cpu().to(F64)[live[:, 0, 0] == 1] - v[pick].to(F64)[live[:, 0, 0] == 1]).abs()
    assert (v_err <= 0.5 * (2.0 ** ex[s // ps, :, s % ps].to(F64))[live[:, 0, 0] == 1][..., None]).all()


def test_read_into_given_tensors(ba):
    c = ba.KVCache.zeros(1, 2, 64, 16)
    k = torch.randn((3, 2, 64), generator=_gen(0)).half().cuda()
    slots = torch.tensor([5, 1, 9]).cuda()
    ba.cache_write(c, k, k, slots)
    ko, vo = torch.empty((3, 2, 64), device="cuda"), torch.empty((3, 2, 64), device="cuda")
    a, b = ba.cache_read(c, slots, k_out=ko, v_out=vo)
    assert a is ko and b is vo
    x, y = ba.cache_read(c, slots, torch.float32)
    assert torch.equal(x, ko) and torch.equal(y, vo)


# ----------------------------------------------------------------------------- attention
def _filled(ba, P, H, d, ps, g, lean=0.0):
    """A cache of quantised rows: every slot written, some heads' keys leaning one way."""
    c = ba.KVCache.zeros(P, H, d, ps)
    n = P * ps
    k = torch.randn((n, H, d), generator=g) + lean * torch.randn((1, H, d), generator=g)
    v = torch.randn((n, H, d), generator=g) * 2.0 ** torch.randint(-3, 3, (n, H, 1), generator=g)
    ba.cache_write(c, k.bfloat16().cuda(), v.bfloat16().cuda(), torch.arange(n).cuda())
    return c


def _problem(ba, qn, kn, Hq, Hkv, d, ps, dt, seed, lean=0.5):
    g = _gen(seed)
    need = [-(-n // ps) for n in kn]
    c = _filled(ba, sum(need) + 2, Hkv, d, ps, g, lean)
    perm = torch.randperm(sum(need) + 2, generator=g).to(torch.int32)
    table = torch.full((len(kn), max(need + [1])), -7, dtype=torch.int32)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = perm[at:at + m]
        at += m
    q = (torch.randn((sum(qn), Hq, d), generator=g) + lean * torch.randn((1, Hq, d), generator=g)).to(DT[dt])
    cu = torch.tensor([0] + list(qn)).cumsum(0).to(torch.int32)
    return c, q, table, torch.tensor(kn, dtype=torch.int32), cu


def _compare(got_o, got_lse, ref, what=""):
    o, lse, to, tl = ref
    got_o, got_lse = got_o.cpu().to(F64), got_lse.cpu().to(F64)
    rows = ~torch.isnan(lse)
    assert torch.isfinite(got_o[rows]).all(), what
    bad = (got_o - o).abs()[rows] > to[rows]
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} values, worst {((got_o - o).abs() / to)[rows].max():.3g} x the tolerance"
    empty = torch.isinf(lse) & rows
    assert torch.equal(got_lse[empty], lse[empty]) and not got_o[empty].any()
    full = rows & ~empty
    assert ((got_lse - lse).abs()[full] <= tl[full]).all(), what


def _run(ba, prob, dt_out=None, **kw):
    c, q, table, kv, cu = prob
    o, lse = ba.attention_paged(q.cuda(), c, table.cuda(), kv.cuda(), cu.cuda(), return_lse=True, out_dtype=dt_out, **kw)
    torch.cuda.synchronize()
    ba.check_device_status()
    return o, lse


def _ref(ba, prob, dt_out=None, **kw):
    c, q, table, kv, cu = prob
    kw.pop("max_q_len", None)
    kw.pop("max_kv_len", None)
    if "softmax_scale" in kw:
        kw["scale"] = kw.pop("softmax_scale")
    return paged_ref.attend(q, c.data.cpu(), c.page_size, c.d, table, kv, cu, eps_out=torch.finfo(dt_out or q.dtype).eps, **kw)


# new tokens, context lengths, query heads, KV heads, d, page size, type
SHAPES = [
    ([1], [1], 1, 1, 64, 16, "f16"),
    ([1], [2], 8, 1, 128, 16, "bf16"),
    ([1, 1, 1], [17, 300, 31], 4, 4, 128, 16, "bf16"),
    ([1, 1], [513, 64], 14, 2, 64, 32, "f16"),           # groups of 7
    ([1, 1, 1, 1], [129, 1000, 5, 640], 32, 2, 128, 48, "bf16"),  # groups of 16: pages end inside blocks
    ([1], [700], 24, 1, 72, 80, "f16"),                  # 24 rows: three tiles of 8
    ([2, 5, 1], [40, 200, 77], 8, 2, 128, 64, "bf16"),
    ([3, 0, 4], [3, 50, 130], 6, 3, 40, 16, "f16"),      # a sequence without new tokens
    ([16], [16], 4, 4, 64, 16, "bf16"),                  # all tokens are new
    ([9, 20], [9, 250], 4, 2, 5, 16, "bf16"),
    ([33, 64], [100, 64], 3, 3, 80, 32, "f16"),
    ([130], [333], 2, 1, 128, 128, "bf16"),
    ([70, 3, 129], [70, 400, 129], 4, 1, 64, 64, "f16"),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)).replace(" ", ""))
def test_attention(ba, shape):
    prob = _problem(ba, *shape, seed=len(shape[0]) * 7 + shape[4])
    _compare(*_run(ba, prob, max_q_len=max(shape[0])), _ref(ba, prob), "tight bounds")


@pytest.mark.parametrize("shape", SHAPES[2:12:2], ids=lambda s: "-".join(map(str, s)).replace(" ", ""))
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (100, 40), (33, 1000), (1 << 30, 5)])
def test_window_and_sinks(ba, shape, window, sinks):
    prob = _problem(ba, *shape, seed=window % 97)
    kw = dict(window=window, sinks=sinks)
    _compare(*_run(ba, prob, max_q_len=max(shape[0]), **kw), _ref(ba, prob, **kw), f"window {window}, sinks {sinks}")


@pytest.mark.parametrize("shape", [SHAPES[4], SHAPES[6], SHAPES[11]], ids=lambda s: "-".join(map(str, s)).replace(" ", ""))
def test_without_causal_mask(ba, shape):
    prob = _problem(ba, *shape, seed=5)
    _compare(*_run(ba, prob, causal=False), _ref(ba, prob, causal=False))


@pytest.mark.parametrize("qn", [[1, 1, 1], [2, 4, 40], [40, 5, 64], [70, 5, 150]])
def test_rows_that_see_nothing(ba, qn):
    """More new tokens than the cache holds: the first ones are before the first key. Also an empty cache."""
    kn = [0, 3, 30]
    prob = _problem(ba, qn, kn, 4, 2, 64, 16, "bf16", 2)
    o, lse, to, tl = ref = _ref(ba, prob)
    assert torch.isinf(lse).any()
    _compare(*_run(ba, prob), ref)


@pytest.mark.parametrize("dt_out", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("shape", [SHAPES[4], SHAPES[10]], ids=["decode", "chunk"])
def test_output_types_and_scale(ba, shape, dt_out):
    prob = _problem(ba, *shape, seed=11)
    kw = dict(softmax_scale=0.25, dt_out=DT[dt_out])
    o, lse = _run(ba, prob, **kw)
    assert o.dtype == DT[dt_out]
    _compare(o, lse, _ref(ba, prob, **kw))


@pytest.mark.parametrize("scale,lean", [(4.0, 0.0), (2.0, 2.0)])
@pytest.mark.parametrize("qn", [[1, 1], [40, 100]])
def test_large_scores(ba, scale, lean, qn):
    """Scores of hundreds: most weights are zero, and the running maximum moves far."""
    prob = _problem(ba, qn, [600, 900], 4, 2, 128, 32, "bf16", 3, lean)
    _compare(*_run(ba, prob, softmax_scale=scale), _ref(ba, prob, softmax_scale=scale))


@pytest.mark.parametrize("qn", [[1], [64], [100]])
def test_values_of_very_different_size(ba, qn):
    """One key's values are 2^30 times another's; zero rows have the least exponent and weigh as much as any."""
    d, ps, n = 64, 16, 200
    g = _gen(8)
    k, v = torch.randn((n, 1, d), generator=g), torch.randn((n, 1, d), generator=g)
    v *= 2.0 ** torch.randint(-22, 9, (n, 1, 1), generator=g)
    v[5:60] = 0.0
    c = ba.KVCache.zeros(-(-n // ps), 1, d, ps)
    ba.cache_write(c, k.bfloat16().cuda(), v.bfloat16().cuda(), torch.arange(n).cuda())
    q = torch.randn((qn[0], 2, d), generator=g).bfloat16()
    prob = (c, q, torch.arange(c.num_pages, dtype=torch.int32)[None], torch.tensor([n], dtype=torch.int32),
            torch.tensor([0] + qn, dtype=torch.int32))
    _compare(*_run(ba, prob), _ref(ba, prob))


@pytest.mark.parametrize("qn,causal", [([1, 1], True), ([30, 50], True), ([1, 40], False), ([70, 30], True), ([2, 80], False)])
def test_missing_pages_and_garbage_outside_the_sequences(ba, qn, causal):
    """Tokens on pages outside the cache are not seen; whatever unused rows hold (NaN scales, any exponent) stays out."""
    c, q, table, kv, cu = _problem(ba, qn, [210, 170], 4, 2, 128, 48, "bf16", 4)
    table[0, 1], table[1, 2], table[1, 3] = -1, c.num_pages, 1 << 30
    used = torch.zeros(c.num_pages, c.page_size, dtype=torch.bool)
    for b in range(2):
        for j in range(int(kv[b])):
            pg = int(table[b, j // c.page_size])
            if 0 <= pg < c.num_pages:
                used[pg, j % c.page_size] = True
    free = (~used).cuda()[:, None].expand(-1, 2, -1)
    c.k_mu[free] = math.nan
    c.v_exp[free] = 127
    c.v_codes[free] = -128
    prob = (c, q, table, kv, cu)
    _compare(*_run(ba, prob, causal=causal), _ref(ba, prob, causal=causal))


@pytest.mark.parametrize("qn", [[2, 3], [40, 30], [70, 80]])
def test_rows_of_no_sequence_stay(ba, qn):
    """Rows behind the last sequence, before the first and past max_q_len are left as they were."""
    c, q, table, kv, cu = _problem(ba, qn, [50, 90], 4, 2, 64, 16, "bf16", 6)
    pad = torch.full((7, 4, 64), 3.0, dtype=q.dtype)
    q2 = torch.cat([pad[:2], q, pad])
    cu2 = cu + 2
    out = torch.full_like(q2, 5.0).cuda()
    want = _run(ba, (c, q, table, kv, cu))[0]
    got = ba.attention_paged(q2.cuda(), c, table.cuda(), kv.cuda(), cu2.cuda(), out=out)
    assert got is out
    assert (out[:2] == 5).all() and (out[2 + sum(qn):] == 5).all() and torch.equal(out[2:2 + sum(qn)], want)
    out.fill_(5.0)
    # another bound may choose another kernel, whose roundings are others
    want = _run(ba, (c, q, table, kv, cu), max_q_len=qn[0])[0]
    ba.attention_paged(q2.cuda(), c, table.cuda(), kv.cuda(), cu2.cuda(), max_q_len=qn[0], out=out)
    n = min(qn)
    assert torch.equal(out[2:2 + n], want[:n])
    over = out[2 + qn[0] + qn[0]:2 + sum(qn)]
    assert (over == 5).all()


@pytest.mark.parametrize("qn", [[1, 1, 1], [5, 9, 2], [50, 80, 3]])
def test_strided_queries(ba, qn):
    c, q, table, kv, cu = _problem(ba, qn, [60, 90, 33], 6, 2, 72, 16, "f16", 9)
    want = _run(ba, (c, q, table, kv, cu))[0]
    T = q.shape[0]
    fused = torch.zeros((T, 10, 72), dtype=q.dtype, device="cuda")
    fused[:, 2:8] = q.cuda()
    odd = torch.zeros((T * 6 * 73 + 1,), dtype=q.dtype, device="cuda")[1:].view(T, 6, 73)[..., :72]
    odd.copy_(q.cuda())
    turned = q.cuda().transpose(0, 1).contiguous().transpose(0, 1)
    for x in (fused[:, 2:8], odd, turned):
        got = ba.attention_paged(x, c, table.cuda(), kv.cuda(), cu.cuda())
        assert torch.equal(got, want)
    # a page table that is a slice of a wider one
    wide = torch.full((3, 40), -1, dtype=torch.int32)
    wide[:, 4:4 + table.shape[1]] = table
    got = ba.attention_paged(q.cuda(), c, wide.cuda()[:, 4:4 + table.shape[1]], kv.cuda(), cu.cuda())
    assert torch.equal(got, want)


@pytest.mark.parametrize("kn,Hq,Hkv,d", [([20000], 8, 1, 128), ([9001, 3, 700], 4, 2, 64)])
def test_split_key_axis(ba, kn, Hq, Hkv, d):
    """Long contexts are split over CTAs and joined; short ones beside them are not."""
    prob = _problem(ba, [1] * len(kn), kn, Hq, Hkv, d, 64, "bf16", 12)
    _compare(*_run(ba, prob, max_q_len=1), _ref(ba, prob))
    kw = dict(window=5000, sinks=70)
    _compare(*_run(ba, prob, max_q_len=1, **kw), _ref(ba, prob, **kw))


@pytest.mark.parametrize("qn,kn,Hq,Hkv,d,ps,dt", [([40], [3001], 4, 1, 128, 64, "bf16"),
                                                  ([20, 70], [2500, 400], 8, 2, 64, 32, "f16")])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1500, 200)])
def test_chunks_split_over_the_key_axis(ba, qn, kn, Hq, Hkv, d, ps, dt, window, sinks):
    """Few chunks over long contexts: the key blocks of one tile are cut over many CTAs and joined."""
    prob = _problem(ba, qn, kn, Hq, Hkv, d, ps, dt, 30)
    kw = dict(window=window, sinks=sinks)
    _compare(*_run(ba, prob, max_q_len=max(qn), **kw), _ref(ba, prob, **kw))


@pytest.mark.parametrize("qn,Hq,Hkv,d", [([3, 2], 8, 2, 128), ([4], 8, 2, 64), ([5, 1, 6], 5, 1, 100), ([8, 8], 2, 1, 33),
                                         ([25, 9], 4, 2, 128), ([60, 100], 1, 1, 80)])
@pytest.mark.parametrize("n", [200, 5000])
def test_several_tiles_of_sixteen_rows(ba, qn, Hq, Hkv, d, n):
    prob = _problem(ba, qn, [n - 7 * b for b in range(len(qn))], Hq, Hkv, d, 32, "bf16", 31 + d)
    kw = dict(max_q_len=max(qn))
    _compare(*_run(ba, prob, **kw), _ref(ba, prob, **kw))


@pytest.mark.parametrize("qn", [[1], [20], [70]])
def test_windows_and_sinks_of_any_size(ba, qn):
    """A window or sinks beyond every position hide nothing, also where a sequence starts before its first key."""
    prob = _problem(ba, qn, [33], 4, 2, 64, 16, "bf16", 32)
    want = _run(ba, prob)
    for window, sinks in (((1 << 31) - 1, 0), ((1 << 31) - 1, (1 << 31) - 1), (1 << 40, 3), (1, 1 << 33), (1 << 28, 0)):
        got = _run(ba, prob, window=window, sinks=sinks, max_q_len=1 << 35, max_kv_len=1 << 40)
        _compare(*got, _ref(ba, prob))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("qn", [[1], [40], [80]])
def test_garbage_on_pages_before_the_window(ba, qn):
    """A table may go on naming pages that the window has left behind: their next use does not show."""
    ps, n, window, sinks = 16, 300, 50, 4
    c, q, table, kv, cu = _problem(ba, qn, [n], 4, 2, 128, ps, "bf16", 33)
    first = (n - qn[0] - window + 1) // ps
    for j in range(1, first):
        c.data[int(table[0, j])] = 0x80  # codes of -128, negative scales
        c.v_exp[int(table[0, j])] = 127
    prob = (c, q, table, kv, cu)
    kw = dict(window=window, sinks=sinks)
    _compare(*_run(ba, prob, **kw), _ref(ba, prob, **kw))


@pytest.mark.parametrize("qn", [[1], [60]])
def test_missing_pages_behind_garbage(ba, qn):
    """A whole block without pages after one whose rows before the window hold garbage: none of that is left over."""
    ps, n = 16, 384
    window = n - qn[0] - 100 + 1  # the first key that any row sees is 100
    c, q, table, kv, cu = _problem(ba, qn, [n], 4, 1, 128, ps, "bf16", 35)
    for j in range(100 // ps):
        c.data[int(table[0, j])] = 0x80
        c.v_exp[int(table[0, j])] = 127
    table[0, 128 // ps:256 // ps] = -1
    prob = (c, q, table, kv, cu)
    for _ in range(20):
        got = _run(ba, prob, window=window)
    _compare(*got, _ref(ba, prob, window=window))


@pytest.mark.parametrize("qn", [[1], [40], [80]])
def test_negative_scales_behind_a_sequence_that_ends_in_its_largest_keys(ba, qn):
    """The last, partly filled block has scores far above all before: what lies behind it must not hide that."""
    d, ps, n = 128, 64, 128 * 3 + 10
    g = _gen(34)
    c = ba.KVCache.zeros(8, 1, d, ps)
    c.data.fill_(0xC0)
    k, v = (torch.randn((n, 1, d), generator=g).bfloat16() for _ in range(2))
    q = torch.randn((qn[0], 2, d), generator=g).bfloat16()
    k[-10:] = q[-1, 0] * 30
    ba.cache_write(c, k.cuda(), v.cuda(), torch.arange(n).cuda())
    prob = (c, q, torch.arange(8, dtype=torch.int32)[None], torch.tensor([n], dtype=torch.int32), torch.tensor([0] + qn, dtype=torch.int32))
    for causal in (True, False):
        _compare(*_run(ba, prob, causal=causal), _ref(ba, prob, causal=causal))


def test_results_repeat_bit_for_bit(ba):
    for qn in ([1, 1], [3, 7], [150, 90]):
        prob = _problem(ba, qn, [5000, 3001], 8, 2, 128, 32, "bf16", 13)
        a, b = _run(ba, prob), _run(ba, prob)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_bounds_larger_than_the_lengths(ba):
    """Loose host bounds (a captured step's) give the results of tight ones, within two roundings."""
    prob = _problem(ba, [1, 1], [900, 40], 8, 2, 128, 16, "bf16", 14)
    c, q, table, kv, cu = prob
    wide = torch.full((2, 3000), -1, dtype=torch.int32)
    wide[:, :table.shape[1]] = table
    _compare(*_run(ba, (c, q, wide, kv, cu), max_q_len=1), _ref(ba, prob), "wide table")
    _compare(*_run(ba, (c, q, wide, kv, cu), max_q_len=200), _ref(ba, prob), "wide query bound")


def test_decode_form_without_offsets(ba):
    prob = _problem(ba, [1, 1, 1], [100, 7, 350], 8, 4, 64, 32, "f16", 15)
    c, q, table, kv, cu = prob
    want = _run(ba, prob)[0]
    got = ba.attention_paged(q.cuda(), c, table.cuda(), kv.cuda())
    assert torch.equal(got, want)
    # rows behind the batch stay
    out = torch.full((5, 8, 64), 2.0, dtype=q.dtype, device="cuda")
    ba.attention_paged(torch.cat([q, q[:2]]).cuda(), c, table.cuda(), kv.cuda(), out=out)
    assert torch.equal(out[:3], want) and (out[3:] == 2).all()


def test_offsets_past_32_bits(ba):
    """A cache of more than 4 GiB: pages at both ends of it."""
    H, d, ps = 16, 128, 256
    P = (5 << 30) // (H * ps * 147)
    c = ba.KVCache(torch.empty((P, H, ba.kv_block_bytes(ps, d)), dtype=torch.uint8, device="cuda"), ps, d)
    assert c.data.numel() > 1 << 32
    g = _gen(16)
    n = 300
    k, v = (torch.randn((n, H, d), generator=g).bfloat16() for _ in range(2))
    table = torch.tensor([[P - 1, 0]], dtype=torch.int32)
    j = torch.arange(n)
    slots = table[0].long()[j // ps] * ps + j % ps
    ba.cache_write(c, k.cuda(), v.cuda(), slots.cuda())
    near = ba.KVCache.zeros(2, H, d, ps)
    near.data.copy_(c.data[[P - 1, 0]])
    q = torch.randn((3, H, d), generator=g).bfloat16()
    kv, cu = torch.tensor([n], dtype=torch.int32), torch.tensor([0, 3], dtype=torch.int32)
    ref = _ref(ba, (near, q, torch.tensor([[0, 1]], dtype=torch.int32), kv, cu))
    _compare(*_run(ba, (c, q, table, kv, cu)), ref)
    kk, vv = ba.cache_read(c, slots.cuda())
    k2, v2 = ba.cache_read(near, j.cuda())
    assert torch.equal(kk, k2) and torch.equal(vv, v2)
    del c
    torch.cuda.empty_cache()


# ----------------------------------------------------------------------------- as a program uses it
@pytest.mark.parametrize("window,sinks", [(0, 0), (24, 3)])
def test_prompt_then_tokens(ba, window, sinks):
    """A prompt in two chunks and then single tokens, written and attended step by step, give what one call over the
    whole sequence gives (each within its tolerance of the definition)."""
    Hq, Hkv, d, ps, n = 8, 2, 64, 16, 120
    g = _gen(17)
    q, k, v = (torch.randn((n, h, d), generator=g).bfloat16().cuda() for h in (Hq, Hkv, Hkv))
    c = ba.KVCache.zeros(12, Hkv, d, ps)
    table = torch.randperm(12, generator=g)[:-(-n // ps)].to(torch.int32)[None].cuda()
    slot = lambda a, b: (table[0].long()[torch.arange(a, b, device="cuda") // ps] * ps + torch.arange(a, b, device="cuda") % ps)
    outs = []
    for a, b in [(0, 50), (50, 110)] + [(i, i + 1) for i in range(110, n)]:
        ba.cache_write(c, k[a:b], v[a:b], slot(a, b))
        outs.append(ba.attention_paged(q[a:b], c, table, torch.tensor([b], dtype=torch.int32, device="cuda"),
                                       torch.tensor([0, b - a], dtype=torch.int32, device="cuda"), window=window, sinks=sinks))
    o = torch.cat(outs)
    prob = (c, q.cpu(), table.cpu(), torch.tensor([n], dtype=torch.int32), torch.tensor([0, n], dtype=torch.int32))
    ref = _ref(ba, prob, window=window, sinks=sinks)
    _compare(o, ref[1], ref)
    _compare(*_run(ba, prob, window=window, sinks=sinks), ref)
    # the definition on the rows that came in: the cache's rounding of V is its largest error here
    kk, vv = ba.cache_read(c, slot(0, n), torch.float32)
    assert ((vv - v.float()).abs() <= v.float().abs().amax(-1, keepdim=True) / 127 * 1.0001).all()
    assert torch.equal(kk < 0, k < 0)


def test_captured_step_replayed_with_other_lengths(ba):
    """One decoding step (write, attend) captured in a graph, replayed as the sequences grow and the queries change."""
    B, Hq, Hkv, d, ps = 3, 8, 2, 128, 16
    g = _gen(18)
    c = _filled(ba, 64, Hkv, d, ps, g)
    table = torch.randperm(63, generator=g).to(torch.int32)[:B * 20].view(B, 20)
    q, k, v = (torch.zeros((B, h, d), dtype=torch.bfloat16, device="cuda") for h in (Hq, Hkv, Hkv))
    kv = torch.ones(B, dtype=torch.int32, device="cuda")
    slots = torch.full((B,), -1, dtype=torch.int64, device="cuda")
    dev_table = table.cuda()
    out = torch.zeros_like(q)

    def step():
        ba.cache_write(c, k, v, slots)
        return ba.attention_paged(q, c, dev_table, kv, out=out, return_lse=True)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _, lse = step()
    for lens in ([1, 2, 3], [320, 17, 100], [64, 65, 0]):
        lens = torch.tensor(lens, dtype=torch.int32)
        for t, h in ((q, Hq), (k, Hkv), (v, Hkv)):
            t.copy_(torch.randn((B, h, d), generator=g).bfloat16())
        last = (lens.long() - 1).clamp(min=0)
        at = table.long()[torch.arange(B), last // ps] * ps + last % ps
        slots.copy_(torch.where(lens > 0, at, -1))
        kv.copy_(lens)
        graph.replay()
        torch.cuda.synchronize()
        ba.check_device_status()
        _check_rows(c.data.cpu(), ps, d, k.cpu(), v.cpu(), slots.cpu())
        prob = (c, q.cpu(), table, lens, torch.arange(B + 1, dtype=torch.int32))
        _compare(out, lse, _ref(ba, prob))


def test_two_calls_on_two_streams(ba):
    """Calls that overlap, each with its own workspace, give what they give alone."""
    probs = [_problem(ba, qn, [9000, 4000], 8, 2, 128, 64, "bf16", 19 + i) for i, qn in enumerate(([1, 1], [60, 200]))]
    dev = [tuple(x.cuda() if torch.is_tensor(x) else x for x in p) for p in probs]
    want = [_run(ba, p)[0] for p in probs]
    streams = [torch.cuda.Stream() for _ in probs]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [ba.attention_paged(q, c, table, kv, cu, stream=s) for (c, q, table, kv, cu), s in zip(dev, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_binding_refusals(ba):
    c, q, table, kv, cu = _problem(ba, [1, 1], [20, 20], 4, 2, 64, 16, "bf16", 21)
    q, table, kv, cu = q.cuda(), table.cuda(), kv.cuda(), cu.cuda()
    ok = torch.arange(2).cuda()
    rows = torch.zeros((2, 2, 64), dtype=torch.bfloat16, device="cuda")
    for bad in (rows[:, :1], rows[..., :32], rows.float(), rows.transpose(1, 2).contiguous().transpose(1, 2), rows[0]):
        with pytest.raises(ValueError):
            ba.cache_write(c, bad, bad, ok)
    for k, v, s in ((rows, rows.half(), ok), (rows, rows[:1], ok), (rows, rows, ok.int()), (rows, rows, ok[:1]),
                    (rows.cpu(), rows, ok), (rows, rows, ok.cpu()), (rows, rows, torch.arange(4).cuda()[::2])):
        with pytest.raises(ValueError):
            ba.cache_write(c, k, v, s)
    for kw in (dict(k_out=rows[:1]), dict(v_out=rows.float()), dict(k_out=rows.cpu())):
        with pytest.raises(ValueError):
            ba.cache_read(c, ok, torch.bfloat16, **kw)
    with pytest.raises(TypeError):
        ba.cache_read(c, ok, torch.int8)
    for kw in (dict(q=q.float()), dict(q=q[..., :32]), dict(q=q.cpu()), dict(page_table=table.long()),
               dict(page_table=table[:1]), dict(kv_lens=kv.long()), dict(cu_seqlens_q=cu[:2]), dict(cu_seqlens_q=cu.cpu()),
               dict(out=q[:1]), dict(out=q.float(), out_dtype=torch.bfloat16), dict(workspace=torch.zeros(64, dtype=torch.uint8)),
               dict(workspace=torch.zeros((1 << 20, 2), dtype=torch.uint8, device="cuda")[:, 0])):
        args = dict(q=q, page_table=table, kv_lens=kv, cu_seqlens_q=cu)
        args.update(kw)
        with pytest.raises(ValueError):
            ba.attention_paged(cache=c, **args)
    for kw in (dict(window=-1), dict(sinks=-2), dict(window=3, causal=False), dict(softmax_scale=math.nan)):
        with pytest.raises(ba.BinAttnError) as e:
            ba.attention_paged(q, c, table, kv, cu, **kw)
        assert e.value.status == 1
    with pytest.raises(ba.BinAttnError) as e:
        ba.attention_paged(torch.zeros((2, 3, 64), dtype=torch.bfloat16, device="cuda"), c, table, kv, cu)
    assert e.value.status == 1  # 3 query heads over 2 KV heads
    with pytest.raises(ValueError):
        ba.KVCache(c.data[:, :, :-16].contiguous(), 16, 64).c()
    with pytest.raises(ValueError):
        ba.KVCache(c.data.cpu(), 16, 64).c()
    with pytest.raises(ba.BinAttnError) as e:
        ba.attention_paged(q, c, torch.zeros((2, 5000), dtype=torch.int32, device="cuda"), kv, cu, max_q_len=1,
                           workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 4
    torch.cuda.synchronize()
