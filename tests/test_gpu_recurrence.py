"""The gated linear recurrence on the GPU, forward and backward, against its fp64 definition
with the running error bound of oracle.layer_ops, and with the 8-bit steps around it."""
import numpy as np
import pytest
import torch

import linear_attention_state_zero_b200 as tr
from gpu_util import f64
from oracle import layer_ops as ref
from test_gpu_fp8_steps import check_product, check_quantized

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}


def rnd(shape, seed, dtype=F32, std=1.0):
    g = torch.Generator()
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype)


def offsets(lengths):
    return [0] + np.cumsum(lengths).tolist()


def gates(shape, seed, dtype, logits, shift=3.0):
    g = rnd(shape, seed) - shift
    return (g if logits else -torch.nn.functional.softplus(g)).to(dtype)


def near(got, want, bound):
    g, w = f64(got), np.asarray(want)
    assert g.shape == w.shape
    off = np.abs(g - w) - (bound + HALF[got.dtype] * (np.abs(w) + bound))
    assert np.isfinite(g).all() and (off <= 0).all(), off.max()


def check_forward(x, g, cu, h0, logits, dev, **kw):
    y, fin = tr.linear_recurrence(x.to(dev), g.to(dev), cu, h0=None if h0 is None else h0.to(dev),
                                  gate_logits=logits, **kw)
    wy, wf, by, bf = ref.recurrence(f64(x), f64(g), cu, None if h0 is None else f64(h0), logits)
    if y is not None:
        assert y.dtype == x.dtype
        near(y, wy, by)
    near(fin, wf, bf)
    return y, fin


def check_backward(dy, g, y, cu, h0, dh, logits, dev, **kw):
    to = lambda t: None if t is None else t.to(dev)  # noqa: E731
    np_ = lambda t: None if t is None else f64(t)  # noqa: E731
    dx, dg, dh0 = tr.linear_recurrence_backward(to(dy), to(g), to(y), cu, h0=to(h0), dh_final=to(dh),
                                                gate_logits=logits, want_dh0=True, **kw)
    wx, wg, wh, ex, eg, eh = ref.recurrence_grad(f64(dy), f64(g), f64(y), cu, np_(h0), np_(dh), logits)
    near(dx, wx, ex)
    near(dg, wg, eg)
    near(dh0, wh, eh)
    return dx, dg, dh0


# one token; lengths around a segment (8, 16), a block's round (64, 128) and a cluster's (1024);
# empty sequences first, between and last; many one-token sequences; one channel, odd and even
# widths, widths of one and of several tiles
SHAPES = [
    ([1], 1), ([1], 64), ([0, 1, 0], 33), ([7], 64), ([8, 16, 17], 2), ([15, 0, 0, 1, 64], 130),
    ([128], 65), ([129, 127], 64), ([63, 65, 1, 1, 1, 200], 96), ([1024], 64), ([1025, 5], 7),
    ([2500], 128), ([0, 300, 0, 1, 1500, 0], 100), ([1] * 300, 40), ([3] * 150 + [0] * 40 + [700], 66),
    ([0, 0, 0], 5), ([2048, 16], 2048),
]


@pytest.mark.parametrize("xd,gd", [(BF, BF), (BF, F32), (F32, BF), (F32, F32)])
@pytest.mark.parametrize("case", range(len(SHAPES)))
def test_forward_and_backward(cuda_device, case, xd, gd):
    lengths, C = SHAPES[case]
    logits, states = bool(case % 2), case % 3 != 0
    cu, T, N = offsets(lengths), sum(lengths), len(lengths)
    x, g = rnd((T, C), 1 + case, xd), gates((T, C), 50 + case, gd, logits)
    h0 = rnd((N, C), 90 + case) if states else None
    y, _ = check_forward(x, g, cu, h0, logits, cuda_device)
    dh = rnd((N, C), 95 + case) if states else None
    check_backward(rnd((T, C), 70 + case, xd), g, y.cpu(), cu, h0, dh, logits, cuda_device)


@pytest.mark.parametrize("logits", [False, True])
@pytest.mark.parametrize("shift", [-6.0, 0.0, 9.0])
def test_decay_regimes(cuda_device, shift, logits):
    """Gates that forget at once, half way and hardly at all (a up to 1 - 1e-4 and exactly 1)."""
    cu = offsets([3000, 200])
    x, g = rnd((3200, 64), 1), gates((3200, 64), 2, F32, logits, shift)
    if not logits:
        g[:, 3] = 0.0
        g[100::50, 5] = -float("inf")
    y, _ = check_forward(x, g, cu, None, logits, cuda_device)
    check_backward(rnd((3200, 64), 3), g, y.cpu(), cu, None, None, logits, cuda_device)


def test_gradient_against_differences(cuda_device):
    """The GPU's gradients against central differences of the fp64 forward pass."""
    cu, T, C = offsets([40, 0, 111]), 151, 6
    x, g, h0 = rnd((T, C), 1), gates((T, C), 2, F32, True, 1.0), rnd((3, C), 3)
    dy, dh = rnd((T, C), 4), rnd((3, C), 5)
    y, _ = tr.linear_recurrence(x.to(cuda_device), g.to(cuda_device), cu, h0=h0.to(cuda_device), gate_logits=True)
    grads = tr.linear_recurrence_backward(dy.to(cuda_device), g.to(cuda_device), y, cu, h0=h0.to(cuda_device),
                                          dh_final=dh.to(cuda_device), gate_logits=True)
    ins = [f64(x), f64(g), f64(h0)]
    for k, grad in enumerate(grads):
        for seed in range(4):
            d = np.random.default_rng(seed).standard_normal(ins[k].shape)

            def loss(e):
                a = [v + e * d if i == k else v for i, v in enumerate(ins)]
                out, fin, _, _ = ref.recurrence(a[0], a[1], cu, a[2], True)
                return (out * f64(dy)).sum() + (fin * f64(dh)).sum()
            slope = (loss(1e-5) - loss(-1e-5)) / 2e-5
            # fp32 gradients: 2^-19 of the magnitudes that the sum adds up
            assert abs(slope - (f64(grad) * d).sum()) <= 2.0 ** -19 * np.abs(f64(grad) * d).sum() + 1e-7


def test_strides_odd_offsets_and_no_output(cuda_device):
    """x and the gate as column slices of one wider matrix, outputs as slices of others, at even
    and odd offsets; what lies beside them stays; final states only."""
    cu, T, C, N = offsets([70, 0, 200]), 270, 48, 3
    for at in (0, 1):
        for dt in (BF, F32):
            wide = rnd((T, 140), 5 + at, dt)
            wide[:, 60 + at:60 + at + C] -= 3
            dw = wide.to(cuda_device)
            out = torch.full((T, 80), 7.0, dtype=dt, device=cuda_device)
            x, g = dw[:, at:at + C], dw[:, 60 + at:60 + at + C]
            y, fin = tr.linear_recurrence(x, g, cu, gate_logits=True, y=out[:, 16 + at:16 + at + C])
            wy, wf, by, bf = ref.recurrence(f64(x), f64(g), cu, None, True)
            near(y, wy, by)
            assert (out[:, :16 + at] == 7).all() and (out[:, 16 + at + C:] == 7).all()
            none, fin2 = tr.linear_recurrence(x, g, cu, gate_logits=True, want_y=False)
            assert none is None and torch.equal(fin, fin2)
            dyw = rnd((T, 60), 9, dt).to(cuda_device)
            gw = torch.full((T, 130), 7.0, dtype=dt, device=cuda_device)
            dx, dg, _ = tr.linear_recurrence_backward(
                dyw[:, at:at + C], g, y, cu, gate_logits=True, dx=gw[:, at:at + C], dgate=gw[:, 64 + at:64 + at + C])
            ex = ref.recurrence_grad(f64(dyw[:, at:at + C]), f64(g), f64(y), cu, None, None, True)
            near(dx, ex[0], ex[3])
            near(dg, ex[1], ex[4])
            assert (gw[:, at + C:64 + at] == 7).all() and (gw[:, 64 + at + C:] == 7).all()


def test_sequences_do_not_see_each_other(cuda_device):
    """NaN and infinities in one sequence: the others are bitwise what they are without them,
    forward and backward, and inside the sequence they reach every later (earlier) token."""
    lengths = [40, 300, 0, 17, 1100, 3]
    cu, T, C, N = offsets(lengths), sum(lengths), 34, len(lengths)
    x, g = rnd((T, C), 1).to(cuda_device), gates((T, C), 2, F32, True).to(cuda_device)
    dy, h0 = rnd((T, C), 3).to(cuda_device), rnd((N, C), 4).to(cuda_device)
    y, fin = tr.linear_recurrence(x, g, cu, h0=h0, gate_logits=True)
    back = tr.linear_recurrence_backward(dy, g, y, cu, h0=h0, gate_logits=True)
    bad_x, bad_dy = x.clone(), dy.clone()
    bad_x[100], bad_x[cu[4] + 600, 3] = float("nan"), float("inf")
    bad_dy[100], bad_dy[cu[4] + 600, 3] = float("nan"), float("inf")
    y2, fin2 = tr.linear_recurrence(bad_x, g, cu, h0=h0, gate_logits=True)
    back2 = tr.linear_recurrence_backward(bad_dy, g, y, cu, h0=h0, gate_logits=True)
    touched = torch.zeros((T, C), dtype=torch.bool, device=cuda_device)
    touched[100:cu[2]] = True
    touched[cu[4] + 600:cu[5], 3] = True
    assert not torch.isfinite(y2[touched]).any() and torch.equal(y2[~touched], y[~touched])
    assert torch.isnan(fin2[1]).all() and torch.isinf(fin2[4, 3]) and torch.equal(fin2[5], fin[5])
    touched.zero_()
    touched[cu[1]:101] = True
    touched[cu[4]:cu[4] + 601, 3] = True
    assert not torch.isfinite(back2[0][touched]).any() and torch.equal(back2[0][~touched], back[0][~touched])
    assert torch.equal(back2[2][[0, 2, 3, 5]], back[2][[0, 2, 3, 5]]) and torch.isnan(back2[2][1]).all()


def test_decode_in_place_continues_the_scan(cuda_device):
    """Token by token with the states updated in place is the scan of the whole sequences."""
    N, L, C = 37, 5, 130
    x, g, h0 = rnd((N, L, C), 1), gates((N, L, C), 2, F32, True), rnd((N, C), 3)
    cu = offsets([L] * N)
    want, wf, by, bf = ref.recurrence(f64(x.reshape(-1, C)), f64(g.reshape(-1, C)), cu, f64(h0), True)
    h = h0.to(cuda_device)
    pair = tr.seqlens(offsets([1] * N), cuda_device)
    for t in range(L):
        y, fin = tr.linear_recurrence(x[:, t].to(cuda_device), g[:, t].to(cuda_device), pair, h0=h, h_final=h,
                                      gate_logits=True)
        assert fin is h
        near(y, want.reshape(N, L, C)[:, t], by.reshape(N, L, C)[:, t])
    near(h, wf, bf)


@pytest.mark.parametrize("lengths", [[900], [1, 0, 30, 400, 2], [1] * 50])
def test_states_in_place(cuda_device, lengths):
    cu, T, C, N = offsets(lengths), sum(lengths), 70, len(lengths)
    x, g, h0 = rnd((T, C), 1).to(cuda_device), gates((T, C), 2, F32, False).to(cuda_device), rnd((N, C), 3).to(cuda_device)
    y, fin = tr.linear_recurrence(x, g, cu, h0=h0)
    h = h0.clone()
    y2, _ = tr.linear_recurrence(x, g, cu, h0=h, h_final=h)
    assert torch.equal(y, y2) and torch.equal(h, fin)
    dh = rnd((N, C), 4).to(cuda_device)
    dx, dg, dh0 = tr.linear_recurrence_backward(x, g, y, cu, h0=h0, dh_final=dh)
    d = dh.clone()
    dx2, dg2, _ = tr.linear_recurrence_backward(x, g, y, cu, h0=h0, dh_final=d, dh0=d)
    assert torch.equal(dx, dx2) and torch.equal(dg, dg2) and torch.equal(dh0, d)


@pytest.mark.parametrize("lengths,C", [([20000], 2048), ([5000, 3000, 1, 9000], 512), ([700] * 40, 1024), ([30000], 66)])
def test_large_calls_on_sampled_channels(cuda_device, lengths, C):
    """Sizes that spread over clusters and runs; some channels against fp64, twice bitwise."""
    cu, T, N = offsets(lengths), sum(lengths), len(lengths)
    gen = torch.Generator(device=cuda_device)
    gen.manual_seed(1)
    rn = lambda *s: torch.randn(s, generator=gen, device=cuda_device)  # noqa: E731
    x, g, dy = rn(T, C).to(BF), (rn(T, C) - 3).to(BF), rn(T, C).to(BF)
    h0, dh = rn(N, C), rn(N, C)
    y, fin = tr.linear_recurrence(x, g, cu, h0=h0, gate_logits=True)
    grads = tr.linear_recurrence_backward(dy, g, y, cu, h0=h0, dh_final=dh, gate_logits=True)
    again = tr.linear_recurrence(x, g, cu, h0=h0, gate_logits=True) + tr.linear_recurrence_backward(
        dy, g, y, cu, h0=h0, dh_final=dh, gate_logits=True)
    assert all(torch.equal(a, b) for a, b in zip((y, fin) + grads, again))
    at = [0, 1, C // 2 + 1, C - 1]
    w = ref.recurrence(f64(x[:, at]), f64(g[:, at]), cu, f64(h0[:, at]), True)
    near(y[:, at], w[0], w[2])
    near(fin[:, at], w[1], w[3])
    w = ref.recurrence_grad(f64(dy[:, at]), f64(g[:, at]), f64(y[:, at]), cu, f64(h0[:, at]), f64(dh[:, at]), True)
    for k in range(3):
        near(grads[k][:, at], w[k], w[3 + k])


# the widths of every vector of channels (4, 2 and 1 a lane) and tile; one long sequence, a few and
# many, unbalanced ones, empty ones by the hundred between the others
SPREADS = [
    ([9000], 2048, F32, F32), ([9000], 256, BF, F32), ([6000], 1024, BF, BF), ([5000], 98, F32, BF), ([7000], 301, BF, BF),
    ([3000, 100, 1, 5000], 2022, F32, F32), ([3000, 0, 2500], 1023, F32, BF), ([200] * 70, 512, BF, F32),
    ([0] * 100 + [5] + [0] * 70 + [300] + [1] * 200 + [0] * 40 + [2000] + [0] * 50, 260, BF, BF),
    ([3] * 400 + [1500] + [2] * 300, 129, BF, BF), ([900, 17] * 40, 4096, F32, F32), ([1200] * 8, 1028, BF, BF),
]


@pytest.mark.parametrize("states", [False, True])
@pytest.mark.parametrize("case", range(len(SPREADS)))
def test_spreads_on_sampled_channels(cuda_device, case, states):
    lengths, C, xd, gd = SPREADS[case]
    cu, T, N, logits = offsets(lengths), sum(lengths), len(lengths), (case + states) % 2 == 0
    gen = torch.Generator(device=cuda_device)
    gen.manual_seed(case)
    rn = lambda *s: torch.randn(s, generator=gen, device=cuda_device)  # noqa: E731
    g = rn(T, C) - 3
    x, g, dy = rn(T, C).to(xd), (g if logits else -torch.nn.functional.softplus(g)).to(gd), rn(T, C).to(xd)
    h0, dh = (rn(N, C), rn(N, C)) if states else (None, None)
    y, fin = tr.linear_recurrence(x, g, cu, h0=h0, gate_logits=logits)
    grads = tr.linear_recurrence_backward(dy, g, y, cu, h0=h0, dh_final=dh, gate_logits=logits, want_dh0=True)
    tr.check()
    again = tr.linear_recurrence(x, g, cu, h0=h0, gate_logits=logits) + tr.linear_recurrence_backward(
        dy, g, y, cu, h0=h0, dh_final=dh, gate_logits=logits, want_dh0=True)
    assert all(torch.equal(a, b) for a, b in zip((y, fin) + grads, again))
    at = sorted({0, 1, 2, 3, C // 2, C // 3, C - 2, C - 1})
    part = lambda t: None if t is None else f64(t[:, at])  # noqa: E731
    w = ref.recurrence(part(x), part(g), cu, part(h0), logits)
    near(y[:, at], w[0], w[2])
    near(fin[:, at], w[1], w[3])
    w = ref.recurrence_grad(part(dy), part(g), part(y), cu, part(h0), part(dh), logits)
    for k in range(3):
        near(grads[k][:, at], w[k], w[3 + k])


@pytest.mark.parametrize("xd,gd", [(BF, BF), (BF, F32), (F32, BF), (F32, F32)])
@pytest.mark.parametrize("C,at", [(7, 0), (8, 0), (1028, 0), (1028, 2), (4096, 4), (300, 1)])
def test_single_tokens(cuda_device, C, at, xd, gd):
    """Sequences of one token or none: with and without states, in place, into and from slices."""
    lengths = [1, 0, 1, 1, 0, 0, 1, 1, 1]
    cu, T, N = offsets(lengths), sum(lengths), len(lengths)
    x, g, h0 = rnd((T, C), 1, xd), gates((T, C), 2, gd, True), rnd((N, C), 3)
    xw = torch.zeros((T, C + 12), dtype=xd)
    xw[:, at:at + C] = x
    gw = torch.zeros((T, C + 8), dtype=gd)
    gw[:, at:at + C] = g
    out = torch.full((T, C + 16), 7.0, dtype=xd, device=cuda_device)
    xs, gs = xw.to(cuda_device)[:, at:at + C], gw.to(cuda_device)[:, at:at + C]
    for start in (None, h0):
        wy, wf, by, bf = ref.recurrence(f64(x), f64(g), cu, None if start is None else f64(start), True)
        h = None if start is None else start.to(cuda_device)
        y, fin = tr.linear_recurrence(xs, gs, cu, h0=h, gate_logits=True, y=out[:, at:at + C], h_final=h)
        near(y, wy, by)
        near(fin, wf, bf)
        assert (out[:, :at] == 7).all() and (out[:, at + C:] == 7).all()
        none, fin2 = tr.linear_recurrence(xs, gs, cu, h0=None if start is None else start.to(cuda_device),
                                          gate_logits=True, want_y=False)
        assert none is None and torch.equal(fin, fin2)


def test_infinite_states_stay_in_their_sequence(cuda_device):
    """An infinite final state and gates that forget everything next to it, over several rounds."""
    lengths, C = [1500, 700, 2000], 66
    cu, T = offsets(lengths), sum(lengths)
    x, g = rnd((T, C), 1).to(cuda_device), gates((T, C), 2, F32, True).to(cuda_device)
    y, fin = tr.linear_recurrence(x, g, cu, gate_logits=True)
    h0 = torch.zeros((3, C), device=cuda_device)
    h0[0] = float("inf")
    y2, fin2 = tr.linear_recurrence(x, g, cu, h0=h0, gate_logits=True)
    assert torch.isinf(y2[:1500]).all() and torch.equal(y2[1500:], y[1500:]) and torch.equal(fin2[1:], fin[1:])
    dh = torch.zeros((3, C), device=cuda_device)
    back = tr.linear_recurrence_backward(x, g, y, cu, dh_final=dh, gate_logits=True, want_dh0=True)
    dh[2] = float("inf")
    back2 = tr.linear_recurrence_backward(x, g, y, cu, dh_final=dh, gate_logits=True, want_dh0=True)
    assert torch.isinf(back2[0][2200:]).all()
    assert all(torch.equal(a[:2200], b[:2200]) for a, b in zip(back[:2], back2[:2])) and torch.equal(back[2][:2], back2[2][:2])


def test_offsets_past_32_bits(cuda_device):
    """More than 2^31 elements: the last, short sequence against fp64, forward and backward."""
    lengths, C, gen = [530000, 900], 4096, torch.Generator(device=cuda_device)
    cu, T = offsets(lengths), sum(lengths)
    gen.manual_seed(1)
    x = torch.empty((T, C), dtype=BF, device=cuda_device).normal_(generator=gen)
    g = torch.empty((T, C), dtype=BF, device=cuda_device).normal_(-3, 1, generator=gen)
    y, fin = tr.linear_recurrence(x, g, cu, gate_logits=True)
    dx, dg, _ = tr.linear_recurrence_backward(x, g, y, cu, gate_logits=True)
    tr.check()
    at, n = [0, 1, 2047, C - 1], lengths[1]
    w = ref.recurrence(f64(x[-n:, at]), f64(g[-n:, at]), [0, n], None, True)
    near(y[-n:, at], w[0], w[2])
    near(fin[1:, at], w[1], w[3])
    w = ref.recurrence_grad(f64(x[-n:, at]), f64(g[-n:, at]), f64(y[-n:, at]), [0, n], None, None, True)
    near(dx[-n:, at], w[0], w[3])
    near(dg[-n:, at], w[1], w[4])


def test_two_calls_at_once(cuda_device):
    """Calls on two streams, clusters among them, interleaved: each is what it is alone."""
    sets = []
    for lengths, C in (([9000], 256), ([400] * 30, 512)):
        T = sum(lengths)
        x, g = rnd((T, C), C, BF).to(cuda_device), gates((T, C), 2, BF, True).to(cuda_device)
        sets.append((x, g, tr.seqlens(offsets(lengths), cuda_device)))
    want = [tr.linear_recurrence(x, g, cu, gate_logits=True) for x, g, cu in sets]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for k, (x, g, cu) in enumerate(sets):
            got[k].append(tr.linear_recurrence(x, g, cu, gate_logits=True, stream=streams[k]))
    torch.cuda.synchronize()
    tr.check()
    for k in range(2):
        for y, fin in got[k]:
            assert torch.equal(y, want[k][0]) and torch.equal(fin, want[k][1])


def test_other_stream_and_graph(cuda_device):
    cu = tr.seqlens(offsets([300, 0, 41, 800]), cuda_device)
    x, g = rnd((1141, 96), 1).to(cuda_device), gates((1141, 96), 2, F32, False).to(cuda_device)
    h0 = rnd((4, 96), 3).to(cuda_device)

    def steps(stream=None):
        y, fin = tr.linear_recurrence(x, g, cu, h0=h0, stream=stream)
        return (y, fin) + tr.linear_recurrence_backward(x, g, y, cu, h0=h0, dh_final=fin, stream=stream)
    want = steps()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = steps(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = steps()
    for seed in (5, 6):
        x.copy_(rnd((1141, 96), seed))
        h0.copy_(rnd((4, 96), seed + 10))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(steps(), held))


def test_binding_refusals(cuda_device):
    x = rnd((6, 32), 1).to(cuda_device)
    h = torch.zeros((2, 32), device=cuda_device)
    for err, call in [
        (ValueError, lambda: tr.linear_recurrence(x, x[:5], [0, 6])), (TypeError, lambda: tr.linear_recurrence(x, x.half(), [0, 6])),
        (tr.TrError, lambda: tr.linear_recurrence(x, x, [0, 5])), (tr.TrError, lambda: tr.linear_recurrence(x, x, [0, 4, 3, 6])),
        (ValueError, lambda: tr.linear_recurrence(x, x, [0, 6], h0=h)), (ValueError, lambda: tr.linear_recurrence(x, x, [0, 2, 6], h0=h.bfloat16())),
        (tr.TrError, lambda: tr.linear_recurrence(x, x, [0, 6], y=x)), (ValueError, lambda: tr.linear_recurrence(x, x[:, ::2], [0, 6])),
        (ValueError, lambda: tr.linear_recurrence(x[0], x[0], [0, 6])), (TypeError, lambda: tr.linear_recurrence(x, x, [0, 6], y=x.bfloat16())),
        (TypeError, lambda: tr.linear_recurrence_backward(x, x, x.bfloat16(), [0, 6])),
        (tr.TrError, lambda: tr.linear_recurrence_backward(x, x.clone(), x, [0, 6], dx=x)),
        (ValueError, lambda: tr.linear_recurrence_backward(x, x, x, [0, 6], dh_final=h)),
    ]:
        with pytest.raises(err):
            call()


@pytest.mark.parametrize("lengths,D,C", [([1, 0, 9, 33], 256, 192), ([205, 64], 512, 320)])
def test_layer_of_8_bit_steps(cuda_device, lengths, D, C):
    """A gated linear recurrence layer as it is used: RMSNorm + residual -> 8 bits -> input
    projection (x and gate logits side by side) -> recurrence -> 8 bits -> output projection ->
    the next layer's norm adds it to the stream.  Each step against fp64 from its own inputs."""
    dev, cu, T, N = cuda_device, offsets(lengths), sum(lengths), len(lengths)
    stream, delta = rnd((T, D), 1).to(dev), rnd((T, D), 2, BF).to(dev)
    w_in, s_in = tr.quantize_fp8(rnd((2 * C, D), 3, BF, 0.05).to(dev), block_rows=128)
    w_out, s_out = tr.quantize_fp8(rnd((D, C), 4, BF, 0.05).to(dev), block_rows=128)
    h0, gain = rnd((N, C), 5).to(dev), (1 + rnd((D,), 6, F32, 0.1)).to(dev)
    before = f64(stream)
    q, s, _ = tr.rmsnorm_fp8(delta, gain, residual=stream, residual_out=stream)
    xg = tr.projection_fp8(q, s, w_in, s_in)
    x, g = xg[:, :C], xg[:, C:]
    y, fin = tr.linear_recurrence(x, g, cu, h0=h0, gate_logits=True)
    yq, ys = tr.quantize_fp8(y)
    out = tr.projection_fp8(yq, ys, w_out, s_out)
    mid = f64(stream)
    q2, s2, _ = tr.rmsnorm_fp8(out, gain, residual=stream, residual_out=stream)
    tr.check()
    assert (np.abs(mid - (before + f64(delta))) <= 2.0 ** -23 * np.abs(mid)).all()
    check_quantized(q, s, ref.rmsnorm(f64(delta), before, f64(gain))[0], 1, 2.0 ** -18)
    check_product(xg, q, s, w_in, s_in)
    wy, wf, by, bf = ref.recurrence(f64(x), f64(g), cu, f64(h0), True)
    near(y, wy, by)
    near(fin, wf, bf)
    check_quantized(yq, ys, f64(y), 1, 2.0 ** -23)
    check_product(out, yq, ys, w_out, s_out)
    check_quantized(q2, s2, ref.rmsnorm(f64(out), mid, f64(gain))[0], 1, 2.0 ** -18)
    assert torch.isfinite(stream).all()
