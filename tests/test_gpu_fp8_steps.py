"""The 8-bit projection steps on the GPU against their fp64 definitions.

Bounds are those of the arithmetic, derived in each test; an e4m3 value is off by at most half
a step (2^-4 of the value, 2^-10 of the scale below the normal range), bf16 by 2^-8, fp32 by
2^-24."""
import numpy as np
import pytest
import torch

import linear_attention_state_zero_b200 as tr
from gpu_util import f64
from oracle import layer_ops as ref

pytestmark = pytest.mark.gpu
BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}


def rnd(shape, seed, dtype, std=1.0):
    g = torch.Generator()
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype)


def check_quantized(q, s, v, block_rows, rel):
    """q * s against v in fp64, v itself known to the kernel within `rel`: the scale then is
    within 2 rel, z = v / s within 3 rel (a division and a reciprocal more), and q is half a step
    from that z."""
    q, s = f64(q), f64(s)
    want = ref.block_scales(v, block_rows)
    assert s.shape == want.shape
    assert (np.abs(s - want) <= 2 * rel * want).all()
    full = ref.expand_scales(s, block_rows, *v.shape)
    step = np.maximum(np.abs(v) * 2.0 ** -4, full * 2.0 ** -10)
    assert (np.abs(q * full - v) <= step * (1 + 4 * rel) + 4 * rel * np.abs(v)).all()
    assert np.abs(q).max() <= 448


# D: below, at and beyond a scale block, every number of warps per row, ragged blocks
@pytest.mark.parametrize("rows,D,xd,rd", [
    (1, 16, F32, None), (1, 2048, BF, F32), (3, 144, BF, BF), (7, 1024, F32, F32), (5, 1040, BF, F32),
    (33, 2000, F32, BF), (2, 4096, BF, BF), (9, 5632, BF, None), (3, 8208, F32, F32), (2, 16400, BF, F32),
    (2, 32768, F32, None), (1639, 256, BF, F32),
])
@pytest.mark.parametrize("gain", [False, True])
def test_rmsnorm_fp8(cuda_device, rows, D, xd, rd, gain):
    x, r = rnd((rows, D), D + rows, xd), None
    if rd is not None:
        r = rnd((rows, D), 2, rd, 3.0)
    g = 1 + rnd((D,), 3, F32, 0.1) if gain else None
    dev = lambda t: None if t is None else t.to(cuda_device)  # noqa: E731
    q, s, out = tr.rmsnorm_fp8(dev(x), dev(g), residual=dev(r))
    n, total = ref.rmsnorm(f64(x), None if r is None else f64(r), None if g is None else f64(g))
    # the sum of squares is at most 32 + 10 + 32 additions deep (lane, shuffles, warps), its root
    # halves that, the reciprocal root is good to 2^-22, the sum and two products round once each
    check_quantized(q, s, n, 1, (37 + 4 + 3 + 4) * 2.0 ** -24)
    if r is None:
        assert out is None
    else:
        assert out.dtype == rd
        assert (np.abs(f64(out) - total) <= (HALF[rd] + 2.0 ** -24) * np.abs(total)).all()


def test_rmsnorm_fp8_strides_in_place_and_given_outputs(cuda_device):
    """Rows of a wider matrix, the residual stream updated in place, outputs given; rows and
    columns beside them stay."""
    wide = rnd((6, 704), 5, BF).to(cuda_device)
    stream = rnd((6, 1024), 6, F32).to(cuda_device)
    before = stream.clone()
    x, r = wide[:, 8:520], stream[:, 256:768]
    q = torch.empty((6, 512), dtype=F8, device=cuda_device)
    s = torch.empty((6, 4), device=cuda_device)
    q2, s2, out = tr.rmsnorm_fp8(x, residual=r, residual_out=r, q=q, scale=s)
    assert q2 is q and s2 is s and out is r
    n, total = ref.rmsnorm(f64(x), f64(before[:, 256:768]))
    check_quantized(q, s, n, 1, 2.0 ** -18)
    assert (np.abs(f64(stream[:, 256:768]) - total) <= 2.0 ** -24 * np.abs(total)).all()
    assert torch.equal(stream[:, :256], before[:, :256]) and torch.equal(stream[:, 768:], before[:, 768:])


def test_quantized_special_values(cuda_device):
    """A zero block gets the smallest scale and zeros; a NaN or an infinity stays in its block."""
    x = torch.ones(4, 400)
    x[0, :128] = 0
    x[1, 130] = float("nan")
    x[2, 10] = float("-inf")
    x[3] *= 1e-42
    q, s = (f64(t) for t in tr.quantize_fp8(x.to(cuda_device)))
    assert s[0, 0] == 2.0 ** -126 and (q[0, :128] == 0).all() and (q[0, 128:] == 448).all()
    assert np.isnan(s[1, 1]) and np.isnan(q[1, 128:256]).all() and (q[1, :128] == 448).all()
    assert np.isinf(s[2, 0]) and np.isnan(q[2, 10]) and (q[2, 128:] == 448).all()
    assert (s[3] == 2.0 ** -126).all() and (q[3] == 0).all()
    with np.errstate(invalid="ignore"):
        assert np.isnan((q * ref.expand_scales(s, 1, 4, 400))[2, :128]).any()
    t, ts = (f64(v) for v in tr.quantize_fp8(x.to(cuda_device), block_rows=128))
    assert np.isinf(ts[0, 0]) and np.isnan(ts[0, 1]) and np.isfinite(ts[0, 2:]).all()
    # the norm of a row that holds a NaN is NaN throughout, and the other rows' are not
    qn, sn, _ = tr.rmsnorm_fp8(x.to(cuda_device))
    assert np.isnan(f64(sn)[1]).all() and np.isfinite(f64(sn)[0]).all() and np.isfinite(f64(qn)[3]).all()


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("rows,cols,xd", [(1, 16, F32), (127, 128, BF), (129, 272, F32), (640, 2064, BF),
                                          (300, 1152, F32)])
def test_quantize_fp8(cuda_device, rows, cols, xd, block_rows):
    wide = rnd((rows, cols + 16), rows, xd, 0.02)
    x = wide.to(cuda_device)[:, 8:8 + cols]
    q, s = tr.quantize_fp8(x, block_rows=block_rows)
    check_quantized(q, s, f64(x), block_rows, 2.0 ** -23)


def operand(rows, K, seed, block_rows, device, std=1.0):
    q, s = tr.quantize_fp8(rnd((rows, K), seed, F32, std).to(device), block_rows=block_rows)
    return q, s


def check_product(y, a, sa, w, sw):
    """The tensor core adds a block's 128 products in fp32, each addition off by at most one unit
    in the last place of the running sum of magnitudes (2^-23, truncation allowed for); the
    scales' product and its product with the sum round twice, and the blocks' sums once each."""
    want, mag = ref.projection(f64(a), f64(sa), f64(w), f64(sw))
    kb = sa.shape[1]
    bound = mag * (2.0 ** -16 + (kb + 3) * 2.0 ** -24) + np.abs(want) * HALF[y.dtype]
    assert tuple(y.shape) == want.shape
    assert (np.abs(f64(y) - want) <= bound).all()


# T around the tiles' rows, N around their columns (odd ones too), K around a block
@pytest.mark.parametrize("T,N,K,yd", [
    (1, 1, 16, F32), (1, 128, 128, BF), (2, 100, 144, F32), (8, 6176, 2048, BF), (17, 129, 2000, BF),
    (64, 256, 512, F32), (65, 1001, 1024, BF), (127, 257, 400, F32), (128, 128, 4096, BF),
    (129, 384, 160, F32), (205, 1001, 2000, F32), (257, 2048, 2048, BF), (300, 513, 1152, BF),
    (1639, 1000, 528, BF), (700, 4100, 272, F32),
])
def test_projection_fp8(cuda_device, T, N, K, yd):
    a, sa = operand(T, K, 7 + T, 1, cuda_device)
    w, sw = operand(N, K, 8 + N, 128, cuda_device, 0.02)
    y = tr.projection_fp8(a, sa, w, sw, out_dtype=yd)
    tr.check()
    assert y.dtype == yd
    check_product(y, a, sa, w, sw)
    assert torch.equal(y, tr.projection_fp8(a, sa, w, sw, out_dtype=yd))   # bitwise


# tiles of 256 and of 128 columns, several to a pair of CTAs, K of odd numbers of blocks and of
# several sets of scales; few tokens with K whole and split; rows of y that are and are not
# 16-byte aligned
@pytest.mark.parametrize("T,N,K,yd", [
    (1300, 3000, 640, BF), (1300, 3001, 2208, F32), (1300, 3004, 2208, F32), (2600, 4104, 2176, BF),
    (3300, 5000, 144, F32), (520, 9000, 400, BF), (300, 1200, 1040, F32),
    (2, 9500, 4240, BF), (40, 9700, 160, F32), (33, 500, 4112, BF), (64, 130, 3200, F32), (12, 2500, 384, BF),
])
def test_projection_fp8_tiles(cuda_device, T, N, K, yd):
    a, sa = operand(T, K, 17 + T, 1, cuda_device)
    w, sw = operand(N, K, 18 + N, 128, cuda_device, 0.02)
    y = tr.projection_fp8(a, sa, w, sw, out_dtype=yd)
    tr.check()
    rows = torch.arange(T) if T <= 64 else torch.cat([torch.arange(3), torch.randperm(T)[:60], torch.arange(T - 3, T)])
    check_product(y[rows], a[rows], sa[rows], w, sw)
    assert torch.equal(y, tr.projection_fp8(a, sa, w, sw, out_dtype=yd))


@pytest.mark.parametrize("yd", [BF, F32])
@pytest.mark.parametrize("T,N,at", [(700, 4100, 16), (1500, 2904, 8), (1500, 2904, 9), (60, 300, 8)])
def test_projection_fp8_into_a_slice(cuda_device, T, N, at, yd):
    """y as a slice of a wider matrix, at a 16-byte aligned column and not: rows and columns
    beside it stay as they were."""
    a, sa = operand(T, 384, 3, 1, cuda_device)
    w, sw = operand(N, 384, 4, 128, cuda_device, 0.05)
    out = torch.full((T + 2, N + 24), 7.0, dtype=yd, device=cuda_device)
    y = tr.projection_fp8(a, sa, w, sw, y=out[1:T + 1, at:at + N])
    tr.check()
    check_product(y, a, sa, w, sw)
    keep = torch.ones_like(out, dtype=torch.bool)
    keep[1:T + 1, at:at + N] = False
    assert (out[keep] == 7).all()


@pytest.mark.parametrize("yd", [BF, F32])
@pytest.mark.parametrize("T", [5, 200, 600])
def test_projection_fp8_strided(cuda_device, T, yd):
    """Operands and the output as slices of wider matrices (the output at an odd offset): what
    lies beside the output stays as it was."""
    aw, sa = operand(T, 512, 1, 1, cuda_device)
    ww, sw = operand(300, 512, 2, 128, cuda_device)
    a, w = aw[:, 128:128 + 256], ww[:, 128:128 + 256]
    sa, sw = sa[:, 1:3].contiguous(), sw[:, 1:3].contiguous()
    out = torch.full((T + 2, 333), 7.0, dtype=yd, device=cuda_device)
    y = tr.projection_fp8(a, sa, w, sw, y=out[1:T + 1, 13:313])
    check_product(y, a, sa, w, sw)
    keep = torch.ones_like(out, dtype=torch.bool)
    keep[1:T + 1, 13:313] = False
    assert (out[keep] == 7).all()


@pytest.mark.parametrize("T", [3, 150, 520])
def test_projection_fp8_nan_stays_in_its_row_and_column(cuda_device, T):
    a, sa = operand(T, 384, 3, 1, cuda_device)
    w, sw = operand(260, 384, 4, 128, cuda_device)
    sa[1, 2] = float("nan")
    w.view(torch.uint8)[200, 5] = 0x7f
    y = f64(tr.projection_fp8(a, sa, w, sw, out_dtype=F32))
    bad = np.zeros_like(y, dtype=bool)
    bad[1], bad[:, 200] = True, True
    assert np.isnan(y[bad]).all() and np.isfinite(y[~bad]).all()


def test_offsets_past_32_bits(cuda_device):
    """More than 2^31 elements in and out: the last rows against fp64."""
    T, D, N = 530000, 4096, 4112
    gen = torch.Generator(device=cuda_device)
    gen.manual_seed(1)
    x = torch.empty((T, D), dtype=BF, device=cuda_device).normal_(generator=gen)
    q, s, out = tr.rmsnorm_fp8(x, residual=x)
    n, total = ref.rmsnorm(f64(x[-40:]), f64(x[-40:]))
    check_quantized(q[-40:], s[-40:], n, 1, 2.0 ** -18)
    assert (np.abs(f64(out[-40:]) - total) <= (HALF[BF] + 2.0 ** -24) * np.abs(total)).all()
    check_quantized(*(t[-40:] for t in tr.quantize_fp8(x)), f64(x[-40:]), 1, 2.0 ** -23)
    tq, ts = tr.quantize_fp8(x, block_rows=128)
    last = T // 128 * 128
    check_quantized(tq[last:], ts[last // 128:], f64(x[last:]), 128, 2.0 ** -23)
    w, sw = operand(N, 128, 2, 128, cuda_device)
    a, sa = q[:, :128], s[:, :1].contiguous()
    y = tr.projection_fp8(a, sa, w, sw)
    tr.check()
    check_product(y[-40:], a[-40:], sa[-40:], w, sw)


def test_no_rows(cuda_device):
    x = torch.empty((0, 256), device=cuda_device)
    q, s, out = tr.rmsnorm_fp8(x, residual=x)
    assert q.shape == (0, 256) and s.shape == (0, 2) and out.shape == (0, 256)
    assert tr.quantize_fp8(x, block_rows=128)[1].shape == (0, 2)
    w, sw = operand(64, 256, 1, 128, cuda_device)
    assert tr.projection_fp8(q, s, w, sw).shape == (0, 64)


def test_binding_refusals(cuda_device):
    x = rnd((4, 256), 1, F32).to(cuda_device)
    q, s = tr.quantize_fp8(x)
    w, sw = tr.quantize_fp8(x, block_rows=128)
    for err, call in [
        (ValueError, lambda: tr.rmsnorm_fp8(x, x[0, :128])), (ValueError, lambda: tr.rmsnorm_fp8(x, x[0].bfloat16())),
        (ValueError, lambda: tr.rmsnorm_fp8(x, residual=x[:3])), (ValueError, lambda: tr.rmsnorm_fp8(x, residual_out=x)),
        (TypeError, lambda: tr.rmsnorm_fp8(x.half())), (ValueError, lambda: tr.rmsnorm_fp8(x[0])),
        (tr.TrError, lambda: tr.rmsnorm_fp8(x[:, :100])), (tr.TrError, lambda: tr.rmsnorm_fp8(x[:, 1:241])),
        (ValueError, lambda: tr.quantize_fp8(x, block_rows=64)), (ValueError, lambda: tr.quantize_fp8(x, q=q[:3])),
        (TypeError, lambda: tr.projection_fp8(x, s, w, sw)), (ValueError, lambda: tr.projection_fp8(q, s[:3], w, sw)),
        (ValueError, lambda: tr.projection_fp8(q, s, w, s)), (TypeError, lambda: tr.projection_fp8(q, s, w, sw, out_dtype=torch.half)),
        (ValueError, lambda: tr.projection_fp8(q, s, w[:, :128], sw)),
        (ValueError, lambda: tr.projection_fp8(q, s, w, sw, y=x)),
    ]:
        with pytest.raises(err):
            call()


def test_other_stream_and_graph(cuda_device):
    """The three steps on a stream of their own, and captured once and replayed on new inputs."""
    x, r = rnd((150, 512), 1, BF).to(cuda_device), rnd((150, 512), 2, F32).to(cuda_device)
    w, sw = operand(700, 512, 3, 128, cuda_device, 0.05)

    def steps(stream=None):
        q, s, out = tr.rmsnorm_fp8(x, residual=r, stream=stream)
        return out, tr.projection_fp8(q, s, w, sw, stream=stream)
    want = steps()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = steps(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = steps()
    for seed in (5, 6):
        x.copy_(rnd((150, 512), seed, BF))
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(steps(), held))
