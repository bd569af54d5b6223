"""The paged cache without a GPU: sizes, layout of the views, and what the calls refuse before any launch."""
import ctypes

import pytest
import torch

import paged_ref


@pytest.fixture(scope="module")
def ba():
    from bit_qk_attention_b200 import build
    import bit_qk_attention_b200 as mod
    build.build()
    mod.lib()
    return mod


@pytest.mark.parametrize("ps", [16, 48, 1024])
@pytest.mark.parametrize("d", [1, 16, 17, 64, 72, 128])
def test_block_bytes(ba, ps, d):
    dp = (d + 15) // 16 * 16
    assert ba.kv_block_bytes(ps, d) == ps * (dp + 16 + 2 + 1)
    assert ba.kv_block_bytes(ps, d) % 16 == 0


def test_block_bytes_of_unsupported_sizes(ba):
    for ps, d in ((0, 64), (8, 64), (24, 64), (1040, 64), (-16, 64), (16, 0), (16, 129)):
        assert ba.kv_block_bytes(ps, d) == 0
    with pytest.raises(ValueError):
        ba.KVCache.zeros(1, 1, 64, page_size=20, device="cpu")


@pytest.mark.parametrize("ps,d", [(16, 64), (48, 72), (32, 5)])
def test_views_show_the_documented_layout(ba, ps, d):
    c = ba.KVCache.zeros(3, 2, d, ps, device="cpu")
    c.data.copy_(torch.randint(0, 256, c.data.shape, generator=torch.Generator().manual_seed(1)).to(torch.uint8))
    codes, pad, neg, mu, ex = paged_ref.split_block(c.data, ps, d)
    assert torch.equal(c.v_codes.long()[..., :d], codes) and torch.equal(c.v_codes.long()[..., d:], pad)
    bits = (c.k_bits[..., None] >> torch.arange(32, dtype=torch.int32)) & 1
    assert torch.equal(bits.flatten(-2).bool(), neg)
    got = c.k_mu.to(torch.float64)
    assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(mu))
    assert torch.equal(c.v_exp.long(), ex)


no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="fake pointers: host-only")
FAKE = 0x10000


def _cache(ba, **kw):
    f = dict(data=FAKE, num_pages=10, page_size=16, n_kv_heads=2, d=64)
    f.update(kw)
    return ba.CKvCache(*[f[n] for n, _ in ba.CKvCache._fields_])


BAD_CACHES = [({"page_size": 24}, 2), ({"page_size": 0}, 2), ({"page_size": 2048}, 2), ({"d": 0}, 2), ({"d": 129}, 2),
              ({"n_kv_heads": 0}, 2), ({"n_kv_heads": -1}, 1), ({"n_kv_heads": 65536}, 2), ({"num_pages": -1}, 1),
              ({"data": None}, 1), ({"data": FAKE + 8}, 3), ({"num_pages": 1 << 40}, 2)]


@no_gpu
def test_write_refusals(ba):
    L = ba.lib()

    def call(k=FAKE, v=FAKE, dt=1, T=4, slots=FAKE, st=(128, 64, 128, 64), **kw):
        return L.ba_cache_write(k, st[0], st[1], v, st[2], st[3], dt, T, slots, ctypes.byref(_cache(ba, **kw)), None)

    for kw, want in BAD_CACHES:
        assert call(**kw) == want, kw
    assert L.ba_cache_write(FAKE, 1, 1, FAKE, 1, 1, 1, 4, FAKE, None, None) == 1
    assert call(dt=2) == 1 and call(dt=9) == 1 and call(T=-1) == 1
    for i in range(4):
        assert call(st=tuple(-1 if i == k else 64 for k in range(4))) == 1
    assert call(k=None) == 1 and call(v=None) == 1 and call(slots=None) == 1
    assert call(k=FAKE + 1) == 3 and call(v=FAKE + 1) == 3 and call(slots=FAKE + 4) == 3
    assert call(T=1 << 31) == 2
    assert call(T=0, k=None, v=None, slots=None) == 0  # nothing to write
    assert call(num_pages=0, data=None) == 0           # nowhere to write


@no_gpu
def test_read_refusals(ba):
    L = ba.lib()

    def call(k=FAKE, v=FAKE, dt=1, T=4, slots=FAKE, **kw):
        return L.ba_cache_read(ctypes.byref(_cache(ba, **kw)), slots, T, k, v, dt, None)

    for kw, want in BAD_CACHES:
        assert call(**kw) == want, kw
    assert call(dt=3) == 1 and call(T=-1) == 1 and call(slots=None) == 1
    assert call(k=FAKE + 8) == 3 and call(v=FAKE + 8) == 3 and call(slots=FAKE + 4) == 3
    assert call(T=1 << 31) == 2
    assert call(T=0) == 0 and call(k=None, v=None) == 0


def _seqs(ba, **kw):
    f = dict(B=3, T=7, n_heads=4, max_q_len=4, max_kv_len=100, cu_seqlens_q=FAKE, kv_lens=FAKE, page_table=FAKE,
             table_stride=8, max_pages=8, causal=1, window=0, sinks=0)
    f.update(kw)
    return ba.CPagedSeqs(*[f[n] for n, _ in ba.CPagedSeqs._fields_])


BAD_SEQS = [({"B": -1}, 1), ({"T": -1}, 1), ({"n_heads": 0}, 1), ({"n_heads": 3}, 1), ({"max_q_len": -1}, 1),
            ({"max_kv_len": -1}, 1), ({"max_kv_len": (1 << 28) + 1}, 2), ({"max_pages": -1}, 1),
            ({"table_stride": -1}, 1), ({"causal": 2}, 1), ({"window": -1}, 1), ({"sinks": -1}, 1),
            ({"window": 4, "causal": 0}, 1), ({"T": 1 << 40}, 2)]


@no_gpu
def test_attention_refusals(ba):
    L = ba.lib()

    def call(q=FAKE, st=(256, 64), dt=1, scale=0.0, o=FAKE, odt=1, lse=None, ws=FAKE, nws=1 << 40, cache=None, **kw):
        return L.ba_attention_paged(q, st[0], st[1], dt, ctypes.byref(_cache(ba, **(cache or {}))),
                                    ctypes.byref(_seqs(ba, **kw)), scale, o, odt, lse, ws, nws, None)

    for kw, want in BAD_CACHES:
        assert call(cache=kw) == want, kw
    for kw, want in BAD_SEQS:
        assert call(**kw) == want, kw
        assert L.ba_paged_workspace_bytes(ctypes.byref(_cache(ba)), ctypes.byref(_seqs(ba, **kw))) == \
            ctypes.c_size_t(-1).value, kw
    assert L.ba_attention_paged(FAKE, 1, 1, 1, ctypes.byref(_cache(ba)), None, 0.0, FAKE, 1, None, None, 0, None) == 1
    assert call(dt=2) == 1 and call(odt=3) == 1
    assert call(scale=float("nan")) == 1 and call(scale=float("inf")) == 1
    assert call(st=(-1, 64)) == 1 and call(st=(64, -1)) == 1
    assert call(q=None) == 1 and call(o=None) == 1 and call(kv_lens=None) == 1 and call(page_table=None) == 1
    assert call(q=FAKE + 1) == 3 and call(o=FAKE + 8) == 3 and call(lse=FAKE + 2) == 3
    assert call(kv_lens=FAKE + 2) == 3 and call(cu_seqlens_q=FAKE + 2) == 3 and call(page_table=FAKE + 2) == 3
    for kw in ({"B": 0}, {"T": 0}, {"max_q_len": 0}):
        assert call(q=None, o=None, **kw) == 0, kw  # nothing to do
    # a long context is split and wants a workspace
    need = L.ba_paged_workspace_bytes(ctypes.byref(_cache(ba)), ctypes.byref(_seqs(ba, max_kv_len=1 << 20, max_pages=1 << 16)))
    assert 0 < need < 1 << 30
    long = dict(max_kv_len=1 << 20, max_pages=1 << 16)
    assert call(nws=need - 1, **long) == 4 and call(ws=None, **long) == 4 and call(ws=FAKE + 8, **long) == 3


def test_workspace_does_not_grow_past_the_window(ba):
    L = ba.lib()
    one = lambda **kw: L.ba_paged_workspace_bytes(ctypes.byref(_cache(ba)), ctypes.byref(_seqs(ba, B=1, T=1, max_q_len=1, max_pages=1 << 16, **kw)))
    assert one(max_kv_len=1 << 20, window=64) == 0
    assert one(max_kv_len=128) == 0 and one(max_kv_len=0) == 0 and one(max_kv_len=1 << 20) > 0


def test_python_calls_refuse_what_they_cannot_take(ba):
    """Before anything reaches a device: a cache that is not on one, arguments that are no tensors or numbers."""
    c = ba.KVCache.zeros(1, 1, 64, device="cpu")
    rows, idx = torch.zeros(1, 1, 64, dtype=torch.bfloat16), torch.zeros(1, dtype=torch.int64)
    for call in (lambda: ba.cache_write(c, rows, rows, idx), lambda: ba.cache_read(c, idx),
                 lambda: ba.attention_paged(rows, c, idx[None].int(), idx.int())):
        with pytest.raises(ValueError):
            call()
    m = ba._native()
    for args in ((), (c.data,), (c.data, 64, 64, rows, rows, idx, 0, 0)):
        with pytest.raises(TypeError):
            m.write(*args)
    with pytest.raises(TypeError):
        m.write(None, 64, 64, rows, rows, idx, 0)
    with pytest.raises(ValueError):
        m.write(c.data, 64, 64, rows, rows, idx, 0)
    with pytest.raises(ValueError):
        m.read(c.data, 64, 64, idx, None, None, None, 0)
