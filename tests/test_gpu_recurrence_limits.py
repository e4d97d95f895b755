"""The gated linear recurrence at the edges of its contract: calls from several host threads,
waits that run out."""
import ctypes
import threading

import pytest
import torch

import linear_attention_state_zero_b200 as tr

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def rnd(shape, seed, dtype=F32, std=1.0):
    g = torch.Generator()
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype)


def offsets(lengths):
    out = [0]
    for n in lengths:
        out.append(out[-1] + n)
    return out


@pytest.mark.parametrize("backward", [False, True])
def test_host_threads_with_and_without_clusters(cuda_device, backward):
    """Host threads that launch one kernel with and without a cluster, which take different
    amounts of shared memory, at the same time: every launch succeeds, and each result is what
    the call gives alone."""
    calls, want = [], []
    for lengths, C in (([400] * 30, 512), ([4000], 2048)):
        T, N = sum(lengths), len(lengths)
        host, cu = tr.seqlens(offsets(lengths), cuda_device)
        x, g = rnd((T, C), C, BF).to(cuda_device), (rnd((T, C), 2) - 3).to(BF).to(cuda_device)
        y, h = tr.linear_recurrence(x, g, (host, cu), gate_logits=True)
        if backward:
            want.append(tr.linear_recurrence_backward(x, g, y, (host, cu), gate_logits=True)[:2])
        else:
            want.append((y, h))
        for _ in range(2):
            out = [torch.zeros_like(t) for t in want[-1]]
            if backward:
                a = tr.RecurrenceGradArgs(N, C, T, 1, 1, tr.TR_GATE_LOGITS, 0, 0, 0, 0, 0, x.data_ptr(), g.data_ptr(),
                                          y.data_ptr(), cu.data_ptr(), host.data_ptr(), None, None,
                                          out[0].data_ptr(), out[1].data_ptr(), None)
            else:
                a = tr.RecurrenceArgs(N, C, T, 1, 1, tr.TR_GATE_LOGITS, 0, 0, 0, x.data_ptr(), g.data_ptr(),
                                      cu.data_ptr(), host.data_ptr(), None, out[0].data_ptr(), out[1].data_ptr())
            calls.append((a, out, len(want) - 1, (host, cu, x, g, y), torch.cuda.Stream()))
    torch.cuda.synchronize()
    fn = tr.lib.tr_linear_recurrence_backward if backward else tr.lib.tr_linear_recurrence
    status = []

    def loop(a, stream):
        torch.cuda.set_device(cuda_device)
        for _ in range(1500):
            status.append(fn(ctypes.byref(a), stream.cuda_stream))
    threads = [threading.Thread(target=loop, args=(c[0], c[4])) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    tr.check()
    refused, made = sum(map(bool, status)), len(status)
    assert refused == 0 and made == 1500 * len(calls)
    same = [torch.equal(a, b) for _, out, k, _, _ in calls for a, b in zip(out, want[k])]
    assert all(same)


@pytest.mark.parametrize("limit_ns", [50_000_000, 1])
@pytest.mark.parametrize("backward", [False, True])
def test_waits_that_run_out(cuda_device, backward, limit_ns):
    """The last CTA of each cluster sends nothing: the others give up at the limit, however short,
    every CTA leaves, tr_check reports it, and the next calls are what they were."""
    T, C = 4000, 2048
    host, cu = tr.seqlens([0, T], cuda_device)
    x, g = rnd((T, C), 1, BF).to(cuda_device), (rnd((T, C), 2) - 3).to(BF).to(cuda_device)
    y, h = tr.linear_recurrence(x, g, (host, cu), gate_logits=True)
    want = (y, h) + tr.linear_recurrence_backward(x, g, y, (host, cu), gate_logits=True)[:2]
    out = [torch.empty_like(t) for t in want]
    tr.check()
    flags, stream = tr.TR_GATE_LOGITS | tr.TR_SCAN_STALL_TEST, torch.cuda.current_stream().cuda_stream
    try:
        tr.set_wait_limit_ns(limit_ns)
        if backward:
            a = tr.RecurrenceGradArgs(1, C, T, 1, 1, flags, 0, 0, 0, 0, 0, x.data_ptr(), g.data_ptr(), y.data_ptr(),
                                      cu.data_ptr(), host.data_ptr(), None, None, out[2].data_ptr(),
                                      out[3].data_ptr(), None)
            assert tr.lib.tr_linear_recurrence_backward(ctypes.byref(a), stream) == 0
        else:
            a = tr.RecurrenceArgs(1, C, T, 1, 1, flags, 0, 0, 0, x.data_ptr(), g.data_ptr(), cu.data_ptr(),
                                  host.data_ptr(), None, out[0].data_ptr(), out[1].data_ptr())
            assert tr.lib.tr_linear_recurrence(ctypes.byref(a), stream) == 0
        with pytest.raises(tr.TrError) as e:
            tr.check()
        assert e.value.status == 8   # TR_ERR_TIMEOUT
    finally:
        tr.set_wait_limit_ns(0)
    tr.check()                       # the failed check cleared the error word
    y, h = tr.linear_recurrence(x, g, (host, cu), gate_logits=True)
    got = (y, h) + tr.linear_recurrence_backward(x, g, y, (host, cu), gate_logits=True)[:2]
    tr.check()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
