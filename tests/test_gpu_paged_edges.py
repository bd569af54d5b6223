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

