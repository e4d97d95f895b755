"""The 8-bit projection steps and the gated linear recurrence without a GPU: the oracle's own
pins, and the refusals of the C ABI and of the binding (before any device work)."""
import ctypes

import numpy as np
import pytest
import torch

import linear_attention_state_zero_b200 as tr
from oracle import layer_ops as ref

FAKE = 0x10000  # 16-byte aligned, non-NULL; never dereferenced by validation
T, C, N = 9, 64, 2


# ------------------------------------------------------------------ oracle pins

def test_e4m3_matches_torch():
    """Independent conversion: every rounding of torch's float8_e4m3fn, ties included."""
    v = torch.arange(0, 256, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    v = v[torch.isfinite(v)].unique()
    mid = (v[1:] + v[:-1]) / 2
    z = torch.cat([v, mid, mid * (1 + 1e-6), mid * (1 - 1e-6), torch.randn(5000) * 100])
    want = z.clamp(-448, 448).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ref.e4m3(z.double().numpy()), want)
    assert np.isnan(ref.e4m3(np.array([np.nan]))[0]) and ref.e4m3(np.array([1e9]))[0] == 448


def test_quantized_values_are_within_half_a_step():
    v = np.random.default_rng(1).standard_normal((130, 300)) * 3
    for rows in (1, 128):
        q, s = ref.quantize(v, rows)
        assert s.shape == (-(-130 // rows), 3)
        back = q * ref.expand_scales(s, rows, 130, 300)
        full = ref.expand_scales(s, rows, 130, 300)
        assert (np.abs(back - v) <= np.maximum(np.abs(v) * 2.0 ** -4, full * 2.0 ** -10)).all()
        assert np.abs(q).max() == 448


def test_recurrence_closed_forms():
    """Constant gate and input: h = (1 - a^t) / (1 - a); a = 1: a running sum; gate -inf: h = x;
    the logit form of gate g is the exponential form of -softplus(g)."""
    t = np.arange(1, 11)[:, None]
    one = np.ones((10, 1))
    y, fin, _, _ = ref.recurrence(one, np.log(0.5) * one, [0, 10])
    assert np.allclose(y, (1 - 0.5 ** t) / 0.5) and fin[0, 0] == y[-1, 0]
    assert np.allclose(ref.recurrence(one, 0 * one, [0, 10])[0], t)
    assert np.allclose(ref.recurrence(one, -np.inf * one, [0, 10])[0], 1)
    g = np.random.default_rng(2).standard_normal((10, 3))
    x = np.random.default_rng(3).standard_normal((10, 3))
    a = ref.recurrence(x, g, [0, 4, 4, 10], logits=True)[0]
    b = ref.recurrence(x, -np.log1p(np.exp(g)), [0, 4, 4, 10])[0]
    assert np.allclose(a, b)
    assert np.allclose(a[4:], ref.recurrence(x[4:], g[4:], [0, 6], logits=True)[0])


@pytest.mark.parametrize("logits", [False, True])
def test_recurrence_gradient_against_differences(logits):
    r = np.random.default_rng(4)
    cu = [0, 3, 3, 10]
    x, dy, d1 = (r.standard_normal((10, 2)) for _ in range(3))
    g, h0, dh, d2 = -np.abs(r.standard_normal((10, 2))), *(r.standard_normal((3, 2)) for _ in range(3))
    d3 = r.standard_normal((10, 2))

    def loss(e):
        y, fin, _, _ = ref.recurrence(x + e * d1, g + e * d3, cu, h0 + e * d2, logits)
        return (y * dy).sum() + (fin * dh).sum()
    y = ref.recurrence(x, g, cu, h0, logits)[0]
    dx, dg, dh0, *_ = ref.recurrence_grad(dy, g, y, cu, h0, dh, logits)
    slope = (loss(1e-5) - loss(-1e-5)) / 2e-5
    assert abs(slope - ((dx * d1).sum() + (dg * d3).sum() + (dh0 * d2).sum())) < 1e-8


# ------------------------------------------------------------------ refusals of the C ABI

def _norm(**kw):
    a = dict(x=FAKE, xd=1, xs=0, res=FAKE, rd=0, rs=0, gain=FAKE, rows=4, d=256, eps=0.0, q=FAKE,
             scale=FAKE, out=FAKE, os=0)
    a.update(kw)
    return tr.lib.tr_rmsnorm_fp8(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), 1), (dict(d=0), 1), (dict(d=100), 5), (dict(d=32784), 5), (dict(xd=2), 3),
    (dict(rd=9), 3), (dict(x=None), 1), (dict(q=None), 1), (dict(scale=None), 1),
    (dict(res=None), 1), (dict(x=FAKE + 8), 4), (dict(gain=FAKE + 4), 4), (dict(q=FAKE + 1), 4),
    (dict(scale=FAKE + 2), 4), (dict(out=FAKE + 4), 4), (dict(xs=128), 2), (dict(xs=260), 4),
    (dict(rs=258), 4), (dict(os=100), 2), (dict(rows=1 << 31), 5),
])
def test_norm_refusals(kw, status):
    assert _norm(**kw) == status, tr.lib.tr_last_error()
    assert tr.lib.tr_last_error()


def _quant(**kw):
    a = dict(x=FAKE, xd=1, xs=0, rows=4, cols=256, br=1, q=FAKE, scale=FAKE)
    a.update(kw)
    return tr.lib.tr_quantize_fp8(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), 1), (dict(cols=0), 1), (dict(cols=24), 5), (dict(br=64), 5), (dict(xd=5), 3),
    (dict(x=None), 1), (dict(q=FAKE + 8), 4), (dict(xs=255), 2), (dict(xs=257), 4),
    (dict(rows=1 << 30, cols=1 << 20), 5),
])
def test_quantize_refusals(kw, status):
    assert _quant(**kw) == status, tr.lib.tr_last_error()


def _proj(**kw):
    a = dict(a=FAKE, as_=0, sa=FAKE, w=FAKE, ws=0, sw=FAKE, t=4, n=100, k=256, y=FAKE, yd=1, ys=0)
    a.update(kw)
    return tr.lib.tr_projection_fp8(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(t=-1), 1), (dict(n=0), 1), (dict(k=0), 1), (dict(k=200), 5), (dict(yd=3), 3),
    (dict(a=None), 1), (dict(sw=None), 1), (dict(a=FAKE + 8), 4), (dict(w=FAKE + 1), 4),
    (dict(y=FAKE + 1), 4), (dict(sa=FAKE + 2), 4), (dict(as_=128), 2), (dict(ws=264), 4), (dict(ys=99), 2),
    (dict(t=1 << 31), 1), (dict(t=0x7fffffff, n=0x7fffffff), 5),
])
def test_projection_refusals(kw, status):
    assert _proj(**kw) == status, tr.lib.tr_last_error()


@pytest.mark.parametrize("kw", [dict(t=0x7fffffff), dict(n=0x7fffffff), dict(k=0x7ffffff0)])
def test_projection_sizes_that_pass_32_bits_in_whole_tiles(kw):
    assert _proj(**kw) == 5


def test_projection_of_no_token_needs_no_device():
    assert _proj(t=0, a=None, sa=None, y=None) == 0


_CU = (ctypes.c_int32 * (N + 1))(0, 4, T)


def _rec(**kw):
    a = tr.RecurrenceArgs(N, C, T, 1, 1, 0, 0, 0, 0, FAKE, FAKE + 0x1000, FAKE, ctypes.addressof(_CU), FAKE,
                          FAKE + 0x2000, FAKE)
    for k, v in kw.items():
        setattr(a, k, v)
    return tr.lib.tr_linear_recurrence(ctypes.byref(a), None)


@pytest.mark.parametrize("kw,status", [
    (dict(n_seqs=-1), 1), (dict(n_channels=0), 1), (dict(total_tokens=-1), 1), (dict(total_tokens=10), 2),
    (dict(total_tokens=0x7fffffff), 5), (dict(dtype=2), 3), (dict(gate_dtype=-1), 3), (dict(flags=1), 1),
    (dict(x=None), 1), (dict(gate=None), 1), (dict(h_final=None), 1), (dict(cu_seqlens=None), 1),
    (dict(cu_seqlens_host=None), 1), (dict(x=FAKE + 1), 4), (dict(gate=FAKE + 1), 4), (dict(y=FAKE + 3), 4),
    (dict(dtype=0, x=FAKE + 2), 4), (dict(h0=FAKE + 2), 4), (dict(x_stride=63), 2), (dict(gate_stride=1), 2),
    (dict(y_stride=-64), 2), (dict(y=FAKE), 1), (dict(y=FAKE + 0x1000), 1),
])
def test_recurrence_refusals(kw, status):
    assert _rec(**kw) == status, tr.lib.tr_last_error()


def test_recurrence_refuses_bad_offsets():
    for bad in ((1, 4, T), (0, 5, 4), (0, 4, T - 1)):
        cu = (ctypes.c_int32 * 3)(*bad)
        assert _rec(cu_seqlens_host=ctypes.addressof(cu)) == 2
    assert tr.lib.tr_linear_recurrence(None, None) == 1


def _grad(**kw):
    a = tr.RecurrenceGradArgs(N, C, T, 1, 1, 0, 0, 0, 0, 0, 0, FAKE, FAKE + 0x1000, FAKE + 0x2000, FAKE,
                              ctypes.addressof(_CU), None, None, FAKE + 0x3000, FAKE + 0x4000, None)
    for k, v in kw.items():
        setattr(a, k, v)
    return tr.lib.tr_linear_recurrence_backward(ctypes.byref(a), None)


@pytest.mark.parametrize("kw,status", [
    (dict(n_channels=-3), 1), (dict(dtype=7), 3), (dict(flags=2), 1), (dict(dy=None), 1), (dict(y=None), 1),
    (dict(dx=None), 1), (dict(dgate=None), 1), (dict(dx_stride=8), 2), (dict(dgate_stride=8), 2),
    (dict(dx=FAKE), 1), (dict(dgate=FAKE + 0x1000), 1), (dict(dgate=FAKE + 0x2000), 1),
    (dict(dgate=FAKE + 0x3000), 1), (dict(dh0=FAKE + 1), 4), (dict(dh_final=FAKE + 2), 4), (dict(dy=FAKE + 1), 4),
])
def test_recurrence_gradient_refusals(kw, status):
    assert _grad(**kw) == status, tr.lib.tr_last_error()
    assert tr.lib.tr_linear_recurrence_backward(None, None) == 1


def test_argument_structs_match_the_header():
    assert tr.RecurrenceArgs.x_stride.offset == 32 and tr.RecurrenceArgs.x.offset == 56
    assert ctypes.sizeof(tr.RecurrenceArgs) == 56 + 7 * 8
    assert tr.RecurrenceGradArgs.dy_stride.offset == 32 and tr.RecurrenceGradArgs.dy.offset == 72
    assert ctypes.sizeof(tr.RecurrenceGradArgs) == 72 + 10 * 8


# ------------------------------------------------------------------ refusals of the binding

def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 256)
    q = x.to(torch.float8_e4m3fn)
    for call in (lambda: tr.rmsnorm_fp8(x), lambda: tr.quantize_fp8(x),
                 lambda: tr.projection_fp8(q, x[:, :2], q, x[:1, :2]),
                 lambda: tr.linear_recurrence(x, x, [0, 4]),
                 lambda: tr.linear_recurrence_backward(x, x, x, [0, 4])):
        with pytest.raises(ValueError, match="CUDA"):
            call()


@pytest.mark.parametrize("t,err", [
    (torch.zeros(4, 8, dtype=torch.float16), TypeError), (torch.zeros(4, 9), ValueError),
    (torch.zeros(8, 4).t(), ValueError), (torch.zeros(8).expand(4, 8), ValueError),
    (torch.zeros(4, 16)[:, ::2], ValueError),
])
def test_row_layouts_that_are_refused(t, err):
    with pytest.raises(err):
        tr._row_stride("x", t, (4, 8), tr._DTYPES)


def test_row_layouts_that_pass():
    assert tr._row_stride("x", torch.zeros(4, 16)[:, 3:11], (4, 8), tr._DTYPES) == 16
    assert tr._row_stride("x", torch.zeros(8).expand(1, 8), (1, 8), tr._DTYPES) == 0
    assert tr._row_stride("x", torch.zeros(4, 8)[::2], (2, 8), tr._DTYPES) == 16


def test_offsets_that_are_refused():
    host = torch.arange(8, dtype=torch.int32)
    for pair in ((host[::2], host[::2]), (host, host[:4]), (host.view(2, 4), host.view(2, 4))):
        with pytest.raises(ValueError):
            tr._offsets(pair, "cpu")
