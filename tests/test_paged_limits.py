"""Sizes that attention over the paged cache takes and refuses, on the host alone."""
import ctypes

import pytest

REFUSED = ctypes.c_size_t(-1).value


@pytest.fixture(scope="module")
def ba():
    from bit_qk_attention_b200 import build
    import bit_qk_attention_b200 as mod
    build.build()
    mod.lib()
    return mod


def _workspace(ba, B, T, heads, kv_heads, max_q_len, max_kv_len, ps=64):
    cache = ba.CKvCache(0x10000, 1 << 20, ps, kv_heads, 128)
    pages = -(-max_kv_len // ps)
    seqs = ba.CPagedSeqs(B, T, heads, max_q_len, max_kv_len, 0x10000, 0x10000, 0x10000, pages, pages, 1, 0, 0)
    return ba.lib().ba_paged_workspace_bytes(ctypes.byref(cache), ctypes.byref(seqs))


@pytest.mark.parametrize("B,T,heads,kv_heads", [(512, 65536, 64, 8), (4096, 131072, 32, 8), (1024, 262144, 16, 16)])
def test_a_ragged_batch_is_taken_without_a_bound_of_its_lengths(ba, B, T, heads, kv_heads):
    """max_q_len = T, the default: what counts are the rows there are, T * heads."""
    loose = _workspace(ba, B, T, heads, kv_heads, T, 8192)
    tight = _workspace(ba, B, T, heads, kv_heads, 4 * T // B, 8192)
    assert loose != REFUSED and tight != REFUSED
    assert loose <= T * heads * 20 + (1 << 30)


def test_sizes_beyond_the_limits_are_refused(ba):
    assert _workspace(ba, 1, (1 << 31) // 32, 32, 8, 1, 64) == REFUSED                  # rows of the call
    assert _workspace(ba, 1 << 20, 1 << 22, 32, 8, 1 << 22, 64) == REFUSED              # tiles
    assert _workspace(ba, 1 << 14, 1 << 20, 32, 8, 1 << 20, 1 << 28) == REFUSED         # key blocks
    assert _workspace(ba, 1 << 14, 1 << 20, 32, 8, 1 << 6, 1 << 20) != REFUSED
