"""The gated linear recurrence at the edges of its contract: calls from several host threads,
waits that run out, gates that let the state grow."""
import ctypes
import threading

import numpy as np
import pytest
import torch

import linear_attention_state_zero_b200 as tr
from gpu_util import f64
from oracle import layer_ops as ref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}


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


KINDS = 8


def growing(lengths, C, seed, flip):
    """Gates, inputs and start values [T, C], [T, C], [N, C] whose products of decays leave fp32's
    range within a few tokens while the values stay inside it, by the channel's number modulo KINDS
    (flip: in the order of the backward pass):
    0  zero start and zero inputs while the gate grows them, then ordinary tokens
    1  1e-30 grown by e^120 and shrunk again, over and over    2  by e^100 in 4 tokens each
    3  by e^40 and e^-40 in turn                               4  ordinary tokens
    5  1e10 shrunk by e^-80 and grown again in 4 tokens        6  by e^30 in 300 tokens each
    7  as 0, by e^25 a token"""
    wave = lambda n, t, g: torch.where(t // n % 2 == 0, g, -g)  # noqa: E731
    g, x = [], []
    for i, n in enumerate(lengths):
        t = torch.arange(n).float()
        calm = t >= 0.7 * n
        noise = -torch.nn.functional.softplus(rnd((n,), seed + i) - 1)
        parts = [torch.where(calm, noise, 1.0), wave(120, t, 1.0), wave(4, t, 25.0), wave(1, t, 40.0), noise,
                 -wave(2, t, 40.0), wave(300, t, 0.1), torch.where(calm, noise, 25.0)]
        gi = torch.stack(parts, 1)[:, torch.arange(C) % KINDS]
        xi = torch.zeros(n, C)
        xi[:, 4::KINDS] = rnd((n, 1), seed + 50 + i)
        for k in (0, 7):
            xi[:, k::KINDS] = torch.where(calm, rnd((n,), seed + 90 + i), 0.0)[:, None]
        g.append(gi.flip(0) if flip else gi)
        x.append(xi.flip(0) if flip else xi)
    start = torch.tensor([0.0, 1e-30, 1e-30, 1.0, 0.5, 1e10, 1.0, 0.0])[torch.arange(C) % KINDS]
    return torch.cat(g), torch.cat(x), start.expand(len(lengths), C).contiguous()


def near(got, want, bound):
    g, off = f64(got), np.abs(f64(got) - want) - (bound + HALF[got.dtype] * (np.abs(want) + bound))
    assert np.isfinite(g).all() and (off <= 0).all(), [(k, off[..., k].max()) for k in range(off.shape[-1])]


# Every kernel, with a cluster and without: four, two and one channels a lane, segments of 4, 8 and 16
# tokens, one and two groups of lanes
GROWTH = [
    ([4000], 2048, BF, BF), ([9000], 256, BF, BF), ([3000], 1026, BF, F32), ([2500], 98, F32, BF),
    ([3000], 301, BF, BF), ([2000], 2022, F32, F32), ([2600], 512, F32, F32),
    ([400] * 30, 512, BF, BF), ([300] * 40, 1024, BF, F32), ([250] * 40, 301, F32, F32),
    ([500] * 30, 1026, F32, BF), ([600] * 20, 4096, BF, BF), ([300, 0, 1, 700], 4096, F32, F32),
    ([900] * 70, 130, BF, BF), ([17, 1, 0, 30, 2], 98, F32, F32),
]


# The bound's c: a token's decay is off by 2^-22 + 2^-23 |gate|, |gate| <= 40 here, and a step rounds by
# 2^-24.  A segment's map takes the sum of the logarithms to base 2, up to 144 here (channel 2), which
# rounds by 2^-24 of it and by 2^-23 of the token's own 36: ln 2 (144 + 72) 2^-24 a token, less than
# twice the token's own.
C_GROW = 2 * (2.0 ** -22 + 40 * 2.0 ** -23 + 2.0 ** -24)


@pytest.mark.parametrize("case", range(len(GROWTH)))
def test_growing_gates(cuda_device, case):
    lengths, C, xd, gd = GROWTH[case]
    cu = offsets(lengths)
    g, x, h0 = growing(lengths, C, case, False)
    g, x = g.to(gd), x.to(xd)
    dev = [t.to(cuda_device) for t in (x, g, h0)]
    y, fin = tr.linear_recurrence(dev[0], dev[1], cu, h0=dev[2])
    again = tr.linear_recurrence(dev[0], dev[1], cu, h0=dev[2])
    h = dev[2].clone()
    place = tr.linear_recurrence(dev[0], dev[1], cu, h0=h, h_final=h)
    tr.check()
    assert torch.equal(y, again[0]) and torch.equal(fin, again[1])
    assert torch.equal(y, place[0]) and torch.equal(fin, h)
    at = sorted({k for c in (0, C // 2, C - KINDS) for k in range(c, c + KINDS)})
    wy, wf, by, bf = ref.recurrence(f64(x[:, at]), f64(g[:, at]), cu, f64(h0[:, at]), False, C_GROW)
    near(y[:, at], wy, by)
    near(fin[:, at], wf, bf)


@pytest.mark.parametrize("case", range(len(GROWTH)))
def test_growing_gates_backward(cuda_device, case):
    lengths, C, xd, gd = GROWTH[case]
    cu, T, N = offsets(lengths), sum(lengths), len(lengths)
    g, dy, dh = growing(lengths, C, case, True)
    g, dy, y, h0 = g.to(gd), dy.to(xd), rnd((T, C), 3, xd), rnd((N, C), 4)
    dev = {k: v.to(cuda_device) for k, v in dict(dy=dy, gate=g, y=y, h0=h0, dh_final=dh).items()}
    grads = tr.linear_recurrence_backward(cu_seqlens=cu, **dev)
    again = tr.linear_recurrence_backward(cu_seqlens=cu, **dev)
    tr.check()
    assert all(torch.equal(a, b) for a, b in zip(grads, again))
    at = sorted({k for c in (0, C // 2, C - KINDS) for k in range(c, c + KINDS)})
    w = ref.recurrence_grad(*(f64(t[:, at]) for t in (dy, g, y)), cu, f64(h0[:, at]), f64(dh[:, at]), False, C_GROW)
    for k in range(3):
        near(grads[k][:, at], w[k], w[3 + k])


@pytest.mark.parametrize("backward", [False, True])
def test_growing_gates_and_waits_that_run_out(cuda_device, backward):
    """Limits that run out anywhere in a call, or nowhere: it ends, an error or none is reported, and
    the next calls are what they were."""
    g, x, h0 = (t.to(cuda_device) for t in growing([4000], 2048, 1, backward))
    x, g = x.to(BF), g.to(BF)
    cu = tr.seqlens([0, 4000], cuda_device)
    call = (lambda: tr.linear_recurrence_backward(x, g, x, cu, dh_final=h0, want_dh0=True)) if backward \
        else (lambda: tr.linear_recurrence(x, g, cu, h0=h0))
    want = call()
    tr.check()
    try:
        for limit in (1, 1000, 5000, 20000, 100000):
            tr.set_wait_limit_ns(limit)
            call()
            try:
                tr.check()
            except tr.TrError as e:
                assert e.status == 8   # TR_ERR_TIMEOUT
    finally:
        tr.set_wait_limit_ns(0)
    got = call()
    tr.check()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("gd", [BF, F32])
def test_gradients_of_gates_that_forget_everything(cuda_device, gd):
    """Gate logits up to where the decay leaves fp32's range, under gradients that make it visible:
    dh0 and dgate take the decay that the forward pass takes, and 0 where that is 0."""
    N, C = 30, 64
    g = torch.linspace(60, 87, N * C).reshape(N, C).to(gd)
    g[-1] = torch.tensor([90.0, 300.0, 1e30, float("inf")]).repeat(C // 4).to(gd)
    dy, h0 = 1e30 * (1 + rnd((N, C), 1).abs()), rnd((N, C), 2)
    cu = list(range(N + 1))
    dev = [t.to(cuda_device) for t in (dy, g, h0)]
    y, a = tr.linear_recurrence(torch.zeros_like(dev[0]), dev[1], cu, h0=torch.ones_like(dev[0]), gate_logits=True)
    dx, dg, dh0 = tr.linear_recurrence_backward(dev[0], dev[1], y, cu, h0=dev[2], gate_logits=True)
    # one product each from the forward pass's decays; 1 - a is 1, and e^gate a has their error twice
    assert torch.equal(dx, dev[0])
    assert (np.abs(f64(dh0) - f64(a) * f64(dy)) <= 2.0 ** -24 * np.abs(f64(dh0))).all()
    want = -f64(dh0) * f64(h0)
    assert (np.abs(f64(dg) - want) <= (2.0 ** -20 + HALF[gd]) * np.abs(want)).all()
    assert (f64(a)[-1] == 0).all() and (f64(dh0)[-1] == 0).all() and (f64(dg)[-1] == 0).all()
    ref_a = 1 / (1 + np.exp(f64(g)[:-1]))
    assert (np.abs(f64(a)[:-1] - ref_a) <= (2.0 ** -21 + 87 * 2.0 ** -23) * ref_a).all()
