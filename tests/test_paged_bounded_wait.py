"""The bounded waits of the paged cache's attention kernels, made to run out without faulting or hanging the GPU.

In a test-only build of the library (-DBA_TEST_SKIP_ARRIVE, as in test_bounded_wait.py) the first key block never
arrives in full: in the kernel for few rows it waits for bytes that nobody brings, in the one for many rows its
expanded keys are never announced. Every role then reaches its limit of a second or learns of one that did, copies
and products in flight are waited for, and the kernel ends. The host reads the timeout, and the next call is right.
"""
import ctypes

import pytest
import torch

from test_gpu_paged import _compare, _problem, _ref, _run, ba  # noqa: F401 (ba: fixture)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def short_lib(ba):  # noqa: F811
    from bit_qk_attention_b200 import build
    return ba.lib(build.build_variant("skiparrive", ["BA_TEST_SKIP_ARRIVE"]))


@pytest.mark.parametrize("qn,kn", [([1, 1], [700, 90]),       # few rows, joined within a cluster
                                   ([1, 1], [20000, 90]),     # few rows, parts joined by a second kernel
                                   ([100, 3], [333, 40]),     # many rows, one tile per CTA
                                   ([80, 70], [9000, 500])])  # many rows, parts joined by a second kernel
@pytest.mark.parametrize("d", [64, 128])
def test_expired_wait_reports_timeout_and_device_stays_usable(ba, short_lib, d, qn, kn):  # noqa: F811
    prob = c, q, table, kv, cu = _problem(ba, qn, kn, 4, 2, d, 32, "bf16", 60)
    dev = [x.cuda() for x in (q, table, kv, cu)]
    T, H = q.shape[:2]
    need = ba.paged_workspace_bytes(dev[0], c, *dev[1:], max_q_len=max(qn))
    ws = torch.zeros(max(need, 16), dtype=torch.uint8, device="cuda")
    out = torch.zeros(q.shape, dtype=torch.float32, device="cuda")
    seqs = ba.CPagedSeqs(len(qn), T, H, max(qn), max(kn), dev[3].data_ptr(), dev[2].data_ptr(), dev[1].data_ptr(),
                         dev[1].stride(0), dev[1].shape[1], 1, 0, 0)
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    st = short_lib.ba_attention_paged(dev[0].data_ptr(), H * d, d, 1, ctypes.byref(c.c()), ctypes.byref(seqs), 0.0,
                                      out.data_ptr(), 2, None, ws.data_ptr(), ws.numel(), stream)
    assert st == 0, "the launch itself succeeds"
    assert short_lib.ba_check_device_status(stream) == 6, "BA_ERR_TIMEOUT expected"
    assert short_lib.ba_check_device_status(stream) == 0, "the status word is cleared once read"
    torch.cuda.synchronize()  # no CUDA error: the context survived
    _compare(*_run(ba, prob, max_q_len=max(qn)), _ref(ba, prob), "after a timed-out call")
