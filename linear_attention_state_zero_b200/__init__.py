"""Tail-Replay on B200: zero-initialised tail replay of Gated DeltaNet layers.

Python binding of ``libtr.so`` (declared in ``include/tr.h``).  This module only
marshals arguments: it checks devices, dtypes and strides of torch tensors,
allocates outputs and workspaces with PyTorch, and calls the C ABI.  Every step
of the computation runs in the library's CUDA kernels; there is no CPU path.
Importing fails if the library has not been built
(``python linear_attention_state_zero_b200/_build.py``).
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import Optional, Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libtr.so")

TR_OK = 0
TR_DTYPE_F32, TR_DTYPE_BF16 = 0, 1
TR_NORMALIZE_QK, TR_SKIP_LAST_OUTPUT, TR_SCAN_RECURRENT, TR_SKIP_LAST_FFN = 1, 2, 4, 8
TR_OUTPUT_GATE = 16
TR_SCAN_STALL_TEST = 256
TR_GATE_LOGITS = 512

STATUS_NAMES = {0: "TR_OK", 1: "TR_ERR_INVALID_ARG", 2: "TR_ERR_SHAPE", 3: "TR_ERR_DTYPE",
                4: "TR_ERR_ALIGNMENT", 5: "TR_ERR_UNSUPPORTED", 6: "TR_ERR_WORKSPACE",
                7: "TR_ERR_CUDA", 8: "TR_ERR_TIMEOUT"}

c_i32, c_i64, c_u32, c_f32, c_vp, c_sz = (ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32,
                                          ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t)


class ScanArgs(ctypes.Structure):
    _fields_ = [("n_seqs", c_i32), ("n_heads", c_i32), ("d_k", c_i32), ("d_v", c_i32),
                ("total_tokens", c_i64), ("dtype", c_i32), ("flags", c_u32), ("scale", c_f32),
                ("q_stride", c_i64), ("k_stride", c_i64), ("v_stride", c_i64),
                ("q", c_vp), ("k", c_vp), ("v", c_vp), ("log_alpha", c_vp), ("beta", c_vp),
                ("cu_seqlens", c_vp), ("cu_seqlens_host", c_vp), ("S0", c_vp), ("o", c_vp),
                ("S_final", c_vp)]


class LALayer(ctypes.Structure):
    _fields_ = [("rms_gain", c_vp), ("W_in", c_vp), ("W_o", c_vp), ("ffn_gain", c_vp),
                ("W_gate", c_vp), ("W_up", c_vp), ("W_down", c_vp), ("conv_w", c_vp),
                ("A_log", c_vp), ("dt_bias", c_vp), ("o_norm_gain", c_vp)]


class GroupArgs(ctypes.Structure):
    _fields_ = [("n_seqs", c_i32), ("n_heads", c_i32), ("d_k", c_i32), ("d_v", c_i32),
                ("d_model", c_i32), ("n_layers", c_i32), ("total_tokens", c_i64),
                ("flags", c_u32), ("rms_eps", c_f32), ("norm_eps", c_f32), ("d_ff", c_i32),
                ("h_tail", c_vp), ("cu_seqlens", c_vp), ("cu_seqlens_host", c_vp),
                ("layers", ctypes.POINTER(LALayer)), ("S_hat", c_vp), ("x_out", c_vp),
                ("conv_width", c_i32), ("conv_state", c_vp)]


class RecurrenceArgs(ctypes.Structure):
    _fields_ = [("n_seqs", c_i32), ("n_channels", c_i32), ("total_tokens", c_i64),
                ("dtype", c_i32), ("gate_dtype", c_i32), ("flags", c_u32), ("x_stride", c_i64),
                ("gate_stride", c_i64), ("y_stride", c_i64), ("x", c_vp), ("gate", c_vp),
                ("cu_seqlens", c_vp), ("cu_seqlens_host", c_vp), ("h0", c_vp), ("y", c_vp),
                ("h_final", c_vp)]


class RecurrenceGradArgs(ctypes.Structure):
    _fields_ = [("n_seqs", c_i32), ("n_channels", c_i32), ("total_tokens", c_i64),
                ("dtype", c_i32), ("gate_dtype", c_i32), ("flags", c_u32), ("dy_stride", c_i64),
                ("gate_stride", c_i64), ("y_stride", c_i64), ("dx_stride", c_i64),
                ("dgate_stride", c_i64), ("dy", c_vp), ("gate", c_vp), ("y", c_vp),
                ("cu_seqlens", c_vp), ("cu_seqlens_host", c_vp), ("h0", c_vp),
                ("dh_final", c_vp), ("dx", c_vp), ("dgate", c_vp), ("dh0", c_vp)]


# exported symbol -> (restype, argtypes)
_SIGNATURES = {
    "tr_last_error": (ctypes.c_char_p, []),
    "tr_version": (ctypes.c_char_p, []),
    "tr_tail_len": (c_i64, [c_i64, c_i64, c_i64]),
    "tr_gdn_scan_workspace_size": (c_sz, [ctypes.POINTER(ScanArgs)]),
    "tr_gdn_scan": (ctypes.c_int, [ctypes.POINTER(ScanArgs), c_vp, c_sz, c_vp]),
    "tr_transition_product_workspace_size": (c_sz, [ctypes.POINTER(ScanArgs)]),
    "tr_transition_product": (ctypes.c_int, [ctypes.POINTER(ScanArgs), c_vp, c_vp, c_sz, c_vp]),
    "tr_replay_group_workspace_size": (c_sz, [ctypes.POINTER(GroupArgs)]),
    "tr_replay_group": (ctypes.c_int, [ctypes.POINTER(GroupArgs), c_vp, c_sz, c_vp]),
    "tr_replay_groups_overlapped": (ctypes.c_int, [ctypes.POINTER(GroupArgs), c_i32, c_vp, c_sz,
                                                   c_vp, c_vp, c_sz, c_vp, c_vp]),
    "tr_replay_group_kernel_count": (c_i32, [ctypes.POINTER(GroupArgs)]),
    "tr_replay_group_kernel_names": (ctypes.c_char_p, [ctypes.POINTER(GroupArgs)]),
    "tr_replay_group_profiled": (ctypes.c_int, [ctypes.POINTER(GroupArgs), c_vp, c_sz, c_vp,
                                                ctypes.POINTER(c_vp), c_i32]),
    "tr_replay_groups_workspace_size": (c_sz, [ctypes.POINTER(GroupArgs), c_i32]),
    "tr_replay_groups_lanes_workspace_size": (c_sz, [ctypes.POINTER(GroupArgs), c_i32, c_i32]),
    "tr_replay_groups": (ctypes.c_int, [ctypes.POINTER(GroupArgs), c_i32, c_vp, c_sz, c_vp]),
    "tr_state_error_workspace_size": (c_sz, [c_i64]),
    "tr_state_error": (ctypes.c_int, [c_vp, c_vp, c_i64, c_i32, c_i32, c_vp, c_vp, c_vp, c_sz,
                                      c_vp]),
    "tr_state_error_noalloc": (ctypes.c_int, [c_vp, c_vp, c_i64, c_i32, c_i32, c_vp, c_vp, c_vp]),
    "tr_rmsnorm": (ctypes.c_int, [c_vp, c_i32, c_vp, c_i64, c_i32, c_f32, c_vp, c_vp]),
    "tr_in_projection": (ctypes.c_int, [c_vp, c_vp, c_i64, c_i32, c_i32, c_i32, c_i32, c_u32,
                                        c_f32, c_vp, c_vp, c_vp, c_vp]),
    "tr_out_projection": (ctypes.c_int, [c_vp, c_i64, c_vp, c_vp, c_i32, c_i64, c_i32, c_i32,
                                         c_vp, c_vp]),
    "tr_rmsnorm_fp8": (ctypes.c_int, [c_vp, c_i32, c_i64, c_vp, c_i32, c_i64, c_vp, c_i64, c_i32,
                                      c_f32, c_vp, c_vp, c_vp, c_i64, c_vp]),
    "tr_quantize_fp8": (ctypes.c_int, [c_vp, c_i32, c_i64, c_i64, c_i32, c_i32, c_vp, c_vp, c_vp]),
    "tr_projection_fp8": (ctypes.c_int, [c_vp, c_i64, c_vp, c_vp, c_i64, c_vp, c_i64, c_i32, c_i32,
                                         c_vp, c_i32, c_i64, c_vp]),
    "tr_linear_recurrence": (ctypes.c_int, [ctypes.POINTER(RecurrenceArgs), c_vp]),
    "tr_linear_recurrence_backward": (ctypes.c_int, [ctypes.POINTER(RecurrenceGradArgs), c_vp]),
    "tr_check": (ctypes.c_int, [c_vp]),
    "tr_set_wait_limit_ns": (ctypes.c_int, [ctypes.c_uint64]),
}


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError("libtr.so is not built (%s); run "
                          "`python linear_attention_state_zero_b200/_build.py`" % LIB_PATH)
    lib = ctypes.CDLL(LIB_PATH)
    for name, (res, args) in _SIGNATURES.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    return lib


lib = _load()


class TrError(RuntimeError):
    def __init__(self, status: int, where: str):
        msg = lib.tr_last_error().decode(errors="replace")
        super().__init__("%s: %s (%s)" % (where, STATUS_NAMES.get(status, status), msg))
        self.status = status


def _ok(st: int, where: str) -> None:
    if st != TR_OK:
        raise TrError(st, where)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream, device=None) -> Optional[int]:
    """The raw handle of `stream`, or of the current stream of `device` when None."""
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return stream.cuda_stream


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return TR_DTYPE_BF16
    if t.dtype == torch.float32:
        return TR_DTYPE_F32
    raise TypeError("unsupported dtype %s" % t.dtype)


def _need_cuda(*ts):
    """Every given tensor lives on one CUDA device; returns that device (None if no tensor).

    The library launches on the current device, so each call below runs with this device
    made current (``torch.cuda.device``) and on its current stream unless one is given."""
    dev, index = None, -1
    for t in ts:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("tensors must live on a CUDA device")
        i = t.get_device()
        if dev is None:
            dev, index = t.device, i
        elif i != index:
            raise ValueError("tensors must live on one device (%s and %s)" % (dev, t.device))
    return dev


def _need_layout(name, t, dtype, shape=None):
    """A weight or parameter tensor must be contiguous, of the dtype the kernels read, and
    (where given) of the expected shape; None passes."""
    if t is None:
        return
    if t.dtype != dtype or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %s tensor, got %s" % (name, dtype, t.dtype))
    if shape is not None and t.shape != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))


def seqlens(cu_seqlens, device):
    """cu_seqlens prepared once as (host int32 tensor, device int32 tensor); the calls below
    accept this pair in place of cu_seqlens and then copy nothing."""
    return _seqlens(cu_seqlens, device)


def _seqlens(cu_seqlens, device):
    """(host int32 tensor, device int32 tensor) for a cu_seqlens given either way."""
    if isinstance(cu_seqlens, tuple) and len(cu_seqlens) == 2:
        host, dev = cu_seqlens
        if not isinstance(device, torch.device):
            device = torch.device(device)
        if host.device.type != "cpu" or dev.device != device or \
                host.dtype != torch.int32 or dev.dtype != torch.int32:
            raise ValueError("a (host, device) cu_seqlens pair must hold int32 tensors")
        return host, dev
    cu = torch.as_tensor(cu_seqlens, dtype=torch.int32)
    host = cu.cpu().contiguous()
    dev = cu.to(device).contiguous() if not (cu.is_cuda and cu.is_contiguous()) else cu
    return host, dev


def version() -> str:
    return lib.tr_version().decode()


def tail_len(m: int, r_num: int, r_den: int) -> int:
    """k = ceil(r m) for r = r_num / r_den, exact, clamped to [0, m] (C ABI, host-only)."""
    k = lib.tr_tail_len(int(m), int(r_num), int(r_den))
    if k < 0:
        raise ValueError("bad tail length arguments")
    return int(k)


def gdn_scan(q, k, v, log_alpha, beta, cu_seqlens, *, S0=None, want_o=True, scale=1.0,
             normalize_qk=False, recurrent=False, o=None, S_final=None, stream=None,
             stall_test=False):
    """Eq. (1) scan over a packed batch: returns (o or None, S_final [N, H, d_k, d_v] fp32)."""
    dev_ = _need_cuda(q, k, v, log_alpha, beta, S0, o, S_final)
    T, H, dk = k.shape
    dv = v.shape[2]
    for t in (q, k, v):
        if t is not None and (t.stride(2) != 1 or t.stride(1) != t.shape[2]):
            raise ValueError("q/k/v must be [T, H, d] with contiguous heads")
    la = log_alpha.contiguous()
    be = beta.contiguous()
    host, dev = _seqlens(cu_seqlens, k.device)
    N = host.numel() - 1
    if want_o and o is None:
        o = torch.empty((T, H, dv), dtype=k.dtype, device=k.device)
    if not want_o:
        o = None
    if S_final is None:
        S_final = torch.empty((N, H, dk, dv), dtype=torch.float32, device=k.device)
    flags = (TR_NORMALIZE_QK if normalize_qk else 0) | (TR_SCAN_RECURRENT if recurrent else 0) | \
        (TR_SCAN_STALL_TEST if stall_test else 0)
    a = ScanArgs(N, H, dk, dv, T, _dtype_code(k), flags, float(scale),
                 q.stride(0) if q is not None else 0, k.stride(0), v.stride(0),
                 _ptr(q), _ptr(k), _ptr(v), _ptr(la), _ptr(be),
                 _ptr(dev), host.data_ptr(), _ptr(S0), _ptr(o), _ptr(S_final))
    ws_bytes = lib.tr_gdn_scan_workspace_size(ctypes.byref(a))
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=k.device) if ws_bytes else None
    with torch.cuda.device(dev_):
        _ok(lib.tr_gdn_scan(ctypes.byref(a), _ptr(ws), ws_bytes, _stream(stream, dev_)),
            "tr_gdn_scan")
    return o, S_final


def transition_product(k, log_alpha, beta, cu_seqlens, *, normalize_qk=False, recurrent=False,
                       P=None, stream=None):
    """P = T_t ... T_1 per (sequence, head): [N, H, d_k, d_k] fp32 (M = S^T convention:
    a state M_0 before the sequence becomes P M_0 + the zero-start state after it)."""
    dev_ = _need_cuda(k, log_alpha, beta, P)
    T, H, dk = k.shape
    if k.stride(2) != 1 or k.stride(1) != dk:
        raise ValueError("k must be [T, H, d] with contiguous heads")
    la = log_alpha.contiguous()
    be = beta.contiguous()
    host, dev = _seqlens(cu_seqlens, k.device)
    N = host.numel() - 1
    if P is None:
        P = torch.empty((N, H, dk, dk), dtype=torch.float32, device=k.device)
    flags = (TR_NORMALIZE_QK if normalize_qk else 0) | (TR_SCAN_RECURRENT if recurrent else 0)
    a = ScanArgs(N, H, dk, dk, T, _dtype_code(k), flags, 1.0, 0, k.stride(0), 0,
                 None, _ptr(k), None, _ptr(la), _ptr(be), _ptr(dev), host.data_ptr(), None, None,
                 None)
    ws_bytes = lib.tr_transition_product_workspace_size(ctypes.byref(a))
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=k.device) if ws_bytes else None
    with torch.cuda.device(dev_):
        _ok(lib.tr_transition_product(ctypes.byref(a), _ptr(P), _ptr(ws), ws_bytes,
                                      _stream(stream, dev_)), "tr_transition_product")
    return P


@dataclass
class Layer:
    """One LA layer's weights, device tensors (W_in [2Hd_k + Hd_v + 2H, D], W_o [D, H d_v]),
    and, if the layer has an FFN sublayer, W_gate and W_up [d_ff, D], W_down [D, d_ff]
    (bf16) and ffn_gain [D] fp32 (None: ones).  Optional Gated DeltaNet details (fp32):
    conv_w [2Hd_k + Hd_v, width] (the short convolution), A_log and dt_bias [H] (gate
    parameters), o_norm_gain [d_v] (the output gate's norm; W_in then has the z rows)."""
    W_in: torch.Tensor
    W_o: torch.Tensor
    rms_gain: Optional[torch.Tensor] = None
    W_gate: Optional[torch.Tensor] = None
    W_up: Optional[torch.Tensor] = None
    W_down: Optional[torch.Tensor] = None
    ffn_gain: Optional[torch.Tensor] = None
    conv_w: Optional[torch.Tensor] = None
    A_log: Optional[torch.Tensor] = None
    dt_bias: Optional[torch.Tensor] = None
    o_norm_gain: Optional[torch.Tensor] = None


class GroupReplay:
    """A prepared tr_replay_group call: fixed buffers, so repeated calls cost one C call.

    ``h_tail`` [T, D] bf16 and ``cu_seqlens`` describe the packed tails of the
    group's requests; ``layers`` the group's LA layers (objects with the fields of
    ``Layer``; FFN fields absent or None: no FFN sublayer).  Outputs: ``S_hat``
    [L, N, H, d_k, d_v] fp32 and, unless ``skip_last_output``, ``x_out`` [T, D].
    ``skip_last_ffn`` (default on, the tail-FFN skip) leaves out the last layer's FFN.
    ``output_gate`` turns on the gated output norm (W_in with the z rows); the layers'
    conv_w turn on the short convolution, and ``want_conv_state`` returns its state
    ``conv_state`` [L, N, width - 1, 2Hd_k + Hd_v] bf16.
    """

    def __init__(self, h_tail, cu_seqlens, layers: Sequence, n_heads: int, d_k: int, d_v: int,
                 *, skip_last_output=False, want_x_out=True, rms_eps=0.0, norm_eps=0.0,
                 skip_last_ffn=True, output_gate=False, want_conv_state=False,
                 S_hat=None, x_out=None, workspace=None):
        _need_cuda(h_tail)
        if h_tail.dtype != torch.bfloat16 or not h_tail.is_contiguous():
            raise ValueError("h_tail must be contiguous bf16 [T, D]")
        dev = h_tail.device
        T, D = h_tail.shape
        self.host, self.dev_cu = _seqlens(cu_seqlens, dev)
        N = self.host.numel() - 1
        L = len(layers)
        self.layers = list(layers)
        self._layer_arr = (LALayer * L)()
        d_ff = 0
        conv_width = 0
        n_in = 2 * n_heads * d_k + n_heads * d_v * (2 if output_gate else 1) + 2 * n_heads
        for i, lw in enumerate(self.layers):
            _need_cuda(h_tail, lw.W_in, lw.W_o, lw.rms_gain)
            _need_layout("W_in", lw.W_in, torch.bfloat16, (n_in, D))
            _need_layout("W_o", lw.W_o, torch.bfloat16, (D, n_heads * d_v))
            _need_layout("rms_gain", lw.rms_gain, torch.float32, (D,))
            Wg = getattr(lw, "W_gate", None)
            Wu, Wd, fg = (getattr(lw, n, None) for n in ("W_up", "W_down", "ffn_gain"))
            if Wg is not None:
                _need_cuda(h_tail, Wg, Wu, Wd, fg)
                if d_ff and Wg.shape[0] != d_ff:
                    raise ValueError("all FFN sublayers of a group must have one width")
                d_ff = Wg.shape[0]
                _need_layout("W_gate", Wg, torch.bfloat16, (d_ff, D))
                _need_layout("W_up", Wu, torch.bfloat16, (d_ff, D))
                _need_layout("W_down", Wd, torch.bfloat16, (D, d_ff))
                _need_layout("ffn_gain", fg, torch.float32, (D,))
            cw, al, db, og = (getattr(lw, n, None) for n in ("conv_w", "A_log", "dt_bias",
                                                                 "o_norm_gain"))
            _need_cuda(h_tail, cw, al, db, og)
            _need_layout("conv_w", cw, torch.float32)
            if cw is not None and cw.shape[0] != 2 * n_heads * d_k + n_heads * d_v:
                raise ValueError("conv_w must be [2 H d_k + H d_v, width]")
            _need_layout("A_log", al, torch.float32, (n_heads,))
            _need_layout("dt_bias", db, torch.float32, (n_heads,))
            _need_layout("o_norm_gain", og, torch.float32, (d_v,))
            widths = {cw.shape[1]} if cw is not None else {0}
            if i == 0:
                conv_width = widths.pop()
            elif widths.pop() != conv_width:
                raise ValueError("every layer of a group has the same convolution width")
            self._layer_arr[i] = LALayer(_ptr(lw.rms_gain), _ptr(lw.W_in), _ptr(lw.W_o),
                                         _ptr(fg), _ptr(Wg), _ptr(Wu), _ptr(Wd), _ptr(cw),
                                         _ptr(al), _ptr(db), _ptr(og))
        _need_cuda(h_tail, S_hat, x_out, workspace)
        self.S_hat = S_hat if S_hat is not None else torch.empty(
            (L, N, n_heads, d_k, d_v), dtype=torch.float32, device=dev)
        if skip_last_output:
            want_x_out = False
        self.x_out = None
        if want_x_out:
            self.x_out = x_out if x_out is not None else torch.empty((T, D), dtype=torch.float32,
                                                                     device=dev)
        flags = (TR_SKIP_LAST_OUTPUT if skip_last_output else 0) | \
            (TR_SKIP_LAST_FFN if skip_last_ffn else 0) | (TR_OUTPUT_GATE if output_gate else 0)
        self.conv_state = None
        if want_conv_state and conv_width > 0:
            self.conv_state = torch.empty(
                (L, N, conv_width - 1, (2 * d_k + d_v) * n_heads), dtype=torch.bfloat16,
                device=dev)
        self.h_tail = h_tail
        self.args = GroupArgs(N, n_heads, d_k, d_v, D, L, T, flags, float(rms_eps),
                              float(norm_eps), d_ff, _ptr(h_tail), _ptr(self.dev_cu),
                              self.host.data_ptr(), self._layer_arr, _ptr(self.S_hat),
                              _ptr(self.x_out), conv_width, _ptr(self.conv_state))
        self.ws_bytes = lib.tr_replay_group_workspace_size(ctypes.byref(self.args))
        # allocated at the first run(): a description used only inside GroupsReplay (which
        # has a workspace of its own) never holds one
        self.workspace = workspace

    def _ws(self):
        if self.workspace is None and self.ws_bytes:
            self.workspace = torch.empty(self.ws_bytes, dtype=torch.uint8,
                                         device=self.h_tail.device)
        return self.workspace

    def run(self, stream=None):
        self._ws()
        dev = self.h_tail.device
        with torch.cuda.device(dev):
            _ok(lib.tr_replay_group(ctypes.byref(self.args), _ptr(self.workspace), self.ws_bytes,
                                    _stream(stream, dev)), "tr_replay_group")
        return self.S_hat, self.x_out

    def kernel_count(self) -> int:
        return int(lib.tr_replay_group_kernel_count(ctypes.byref(self.args)))

    def kernel_names(self) -> list:
        """The kernels one run() launches, in order (the events of run_profiled bracket them)."""
        names = lib.tr_replay_group_kernel_names(ctypes.byref(self.args)).decode()
        return names.split(",") if names else []

    def run_profiled(self, event_handles, stream=None):
        """Same as run(), recording the given raw cudaEvent_t handles between kernel launches."""
        arr = (c_vp * len(event_handles))(*event_handles)
        self._ws()
        dev = self.h_tail.device
        with torch.cuda.device(dev):
            _ok(lib.tr_replay_group_profiled(ctypes.byref(self.args), _ptr(self.workspace),
                                             self.ws_bytes, _stream(stream, dev), arr,
                                             len(event_handles)), "tr_replay_group_profiled")
        return self.S_hat, self.x_out


def replay_group(h_tail, cu_seqlens, layers, n_heads, d_k, d_v, **kw):
    """One group's replay: returns (S_hat [L, N, H, d_k, d_v], x_out or None)."""
    stream = kw.pop("stream", None)
    return GroupReplay(h_tail, cu_seqlens, layers, n_heads, d_k, d_v, **kw).run(stream)


class GroupsReplay:
    """A prepared tr_replay_groups call over several GroupReplay descriptions (shared workspace).
    With lanes = 2..4 the workspace holds that many group slices and the groups run on that
    many streams at once (bitwise the same results)."""

    def __init__(self, groups: Sequence[GroupReplay], lanes: int = 1):
        self.groups = list(groups)
        n = len(self.groups)
        if not 1 <= lanes <= 4:
            raise ValueError("lanes must be 1..4")
        self._arr = (GroupArgs * n)()
        for i, g in enumerate(self.groups):
            self._arr[i] = g.args
        self.lanes = lanes
        self.ws_bytes = (lib.tr_replay_groups_workspace_size(self._arr, n) if lanes == 1 else
                         lib.tr_replay_groups_lanes_workspace_size(self._arr, n, lanes))
        dev = self.groups[0].h_tail.device
        for g in self.groups:
            if g.h_tail.device != dev:
                raise ValueError("every group must live on one device")
        self.workspace = torch.empty(self.ws_bytes, dtype=torch.uint8, device=dev) \
            if self.ws_bytes else None

    def run(self, stream=None):
        dev = self.groups[0].h_tail.device
        with torch.cuda.device(dev):
            _ok(lib.tr_replay_groups(self._arr, len(self.groups), _ptr(self.workspace),
                                     self.ws_bytes, _stream(stream, dev)), "tr_replay_groups")
        return [(g.S_hat, g.x_out) for g in self.groups]

    def run_overlapped(self, kv_host, kv_dev, stream=None, copy_stream=None):
        """run() with kv_host (pinned) copied to kv_dev on copy_stream during the replay;
        `stream` waits for the copy before anything enqueued after this call."""
        if copy_stream is None:
            raise ValueError("the KV copy needs a stream of its own (copy_stream)")
        if kv_host.numel() * kv_host.element_size() != kv_dev.numel() * kv_dev.element_size():
            raise ValueError("kv_host and kv_dev differ in size")
        if not kv_host.is_pinned():
            raise ValueError("kv_host must be pinned host memory")
        nbytes = kv_host.numel() * kv_host.element_size()
        dev = self.groups[0].h_tail.device
        if _need_cuda(kv_dev) != dev:
            raise ValueError("kv_dev must live on the groups' device")
        with torch.cuda.device(dev):
            _ok(lib.tr_replay_groups_overlapped(self._arr, len(self.groups),
                                                _ptr(self.workspace), self.ws_bytes,
                                                kv_host.data_ptr(), _ptr(kv_dev), nbytes,
                                                _stream(stream, dev), _stream(copy_stream, dev)),
                "tr_replay_groups_overlapped")
        return [(g.S_hat, g.x_out) for g in self.groups]


def kv_transfer(kv_host, kv_dev, stream=None, copy_stream=None):
    """The FA KV copy of tr_replay_groups_overlapped alone (no groups): kv_host (pinned) to
    kv_dev on copy_stream, after the work already on `stream`, which then waits for it."""
    dev = _need_cuda(kv_dev)
    if copy_stream is None:
        raise ValueError("the KV copy needs a stream of its own (copy_stream)")
    if kv_host.numel() * kv_host.element_size() != kv_dev.numel() * kv_dev.element_size():
        raise ValueError("kv_host and kv_dev differ in size")
    if not kv_host.is_pinned():
        raise ValueError("kv_host must be pinned host memory")
    nbytes = kv_host.numel() * kv_host.element_size()
    with torch.cuda.device(dev):
        _ok(lib.tr_replay_groups_overlapped(None, 0, None, 0, kv_host.data_ptr(), _ptr(kv_dev),
                                            nbytes, _stream(stream, dev),
                                            _stream(copy_stream, dev)),
            "tr_replay_groups_overlapped")


def state_error(S, S_hat, *, per_mat=True, stream=None):
    """(err_per_mat [n_mats] fp64 or None, err_total [1] fp64), device tensors."""
    dev = _need_cuda(S, S_hat)
    if S.shape != S_hat.shape or S.dtype != torch.float32 or S_hat.dtype != torch.float32:
        raise ValueError("S and S_hat must be fp32 tensors of one shape")
    dk, dv = S.shape[-2:]
    S, S_hat = S.contiguous(), S_hat.contiguous()
    n = S.numel() // (dk * dv)
    per = torch.empty(n, dtype=torch.float64, device=dev) if per_mat else None
    tot = torch.empty(1, dtype=torch.float64, device=dev)
    ws_bytes = lib.tr_state_error_workspace_size(n)
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev) if ws_bytes else None
    with torch.cuda.device(dev):
        _ok(lib.tr_state_error(_ptr(S), _ptr(S_hat), n, dk, dv, _ptr(per), _ptr(tot), _ptr(ws),
                               ws_bytes, _stream(stream, dev)), "tr_state_error")
    return per, tot


def state_error_noalloc(S, S_hat, *, per_mat=True, stream=None):
    """Same as state_error, through the entry point that allocates no scratch
    (for callers that cannot allocate device memory at the call; see include/tr.h)."""
    dev = _need_cuda(S, S_hat)
    if S.shape != S_hat.shape or S.dtype != torch.float32 or S_hat.dtype != torch.float32:
        raise ValueError("S and S_hat must be fp32 tensors of one shape")
    dk, dv = S.shape[-2:]
    S, S_hat = S.contiguous(), S_hat.contiguous()
    n = S.numel() // (dk * dv)
    per = torch.empty(n, dtype=torch.float64, device=dev) if per_mat else None
    tot = torch.empty(1, dtype=torch.float64, device=dev)
    # the library's fixed scratch and the kernel belong to the current device: make the
    # tensors' device current for the call
    with torch.cuda.device(dev):
        _ok(lib.tr_state_error_noalloc(_ptr(S), _ptr(S_hat), n, dk, dv, _ptr(per), _ptr(tot),
                                       _stream(stream, dev)), "tr_state_error_noalloc")
    return per, tot


def rmsnorm(x, gain=None, eps=0.0, stream=None):
    dev = _need_cuda(x, gain)
    x = x.contiguous()
    T, D = x.shape
    out = torch.empty((T, D), dtype=torch.bfloat16, device=dev)
    with torch.cuda.device(dev):
        _ok(lib.tr_rmsnorm(_ptr(x), _dtype_code(x), _ptr(gain), T, D, float(eps), _ptr(out),
                           _stream(stream, dev)), "tr_rmsnorm")
    return out


def in_projection(x_hat, W_in, n_heads, d_k, d_v, *, skip_q=False, norm_eps=0.0, stream=None):
    """(qkv [T, 2Hd_k + Hd_v] bf16, log_alpha [T, H], beta [T, H])."""
    dev = _need_cuda(x_hat, W_in)
    T, D = x_hat.shape
    x_hat = x_hat.contiguous()
    W_in = W_in.contiguous()
    qkv = torch.zeros((T, 2 * n_heads * d_k + n_heads * d_v), dtype=torch.bfloat16, device=dev)
    la = torch.empty((T, n_heads), dtype=torch.float32, device=dev)
    be = torch.empty((T, n_heads), dtype=torch.float32, device=dev)
    with torch.cuda.device(dev):
        _ok(lib.tr_in_projection(_ptr(x_hat), _ptr(W_in), T, D, n_heads,
                                 d_k, d_v, TR_SKIP_LAST_OUTPUT if skip_q else 0, float(norm_eps),
                                 _ptr(qkv), _ptr(la), _ptr(be), _stream(stream, dev)),
            "tr_in_projection")
    return qkv, la, be


def out_projection(o, W_o, x_res, stream=None):
    """x_res + o W_o^T in fp32; o [T, H d_v] bf16 (rows may be strided)."""
    dev = _need_cuda(o, W_o, x_res)
    T, hv = o.shape
    D = W_o.shape[0]
    W_o = W_o.contiguous()
    x_res = x_res.contiguous()
    out = torch.empty((T, D), dtype=torch.float32, device=dev)
    with torch.cuda.device(dev):
        _ok(lib.tr_out_projection(_ptr(o), o.stride(0), _ptr(W_o),
                                  _ptr(x_res), _dtype_code(x_res), T, D, hv, _ptr(out),
                                  _stream(stream, dev)), "tr_out_projection")
    return out


# ------------------------------------------------------------ 8-bit projection steps, recurrence

_FP8 = torch.float8_e4m3fn
_DTYPES = {torch.float32: TR_DTYPE_F32, torch.bfloat16: TR_DTYPE_BF16}


def _handle_of_current_stream(index):
    return torch.cuda.current_stream(index).cuda_stream


def _empty_strided(shape, strides, dtype):
    return torch.empty_strided(shape, strides, dtype=dtype, device="cuda")


# What a call of a small operator costs is the host's: 4 us to make a Stream object, 1.7 us for
# each output that torch.empty allocates, 0.8 us by the allocator's direct entry, 2.5 us for the
# launch.  A build of torch that lacks a direct entry (one without CUDA has none) takes the public one.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _handle_of_current_stream)
_device_index = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
try:
    from torch._C._dynamo.guards import _empty_strided_cuda
except ImportError:
    _empty_strided_cuda = _empty_strided


def _matrix_of(rows, cols, dtype):
    """An uninitialised packed matrix on the current device."""
    return _empty_strided_cuda((rows, cols), (cols, 1), dtype)


def _on(stream, dev, fn, *args, **kw):
    """fn(*args, **kw) with the tensors' device current, on its current stream or on `stream`;
    what fn allocates then belongs to the stream that its kernels run on."""
    if stream is None:
        with torch.cuda.device(dev):
            return fn(*args, **kw)
    if getattr(stream, "device", dev) != dev:
        raise ValueError("the stream belongs to %s, the tensors to %s" % (stream.device, dev))
    with torch.cuda.stream(stream):
        return fn(*args, **kw)


def _row_stride(name, t, shape, dtypes):
    """The row stride of a [rows, columns] operand of one of `dtypes` whose rows are contiguous
    and apart (0, packed, for a single row)."""
    if t.dtype not in dtypes:
        raise TypeError("%s: unsupported dtype %s" % (name, t.dtype))
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if t.is_contiguous():
        return 0
    if shape[1] > 1 and t.stride(1) != 1:
        raise ValueError("%s must have contiguous rows" % name)
    if shape[0] <= 1:
        return 0
    if t.stride(0) < shape[1]:
        raise ValueError("%s has overlapping rows (stride %d)" % (name, t.stride(0)))
    return t.stride(0)


def _matrix(name, t):
    if t.dim() != 2:
        raise ValueError("%s must be a matrix, got %d dimensions" % (name, t.dim()))
    return t.shape


def _blocks128(n):
    return (n + 127) // 128


def rmsnorm_fp8(x, gain=None, eps=0.0, *, residual=None, q=None, scale=None, residual_out=None,
                stream=None):
    """RMSNorm of x (+ residual) as an 8-bit activation: (q [T, D] e4m3, scale [T, ceil(D/128)]
    fp32, residual_out = x + residual in the residual's type, or None without a residual).
    residual_out may be the residual itself."""
    T, D = _matrix("x", x)
    dev = _need_cuda(x, gain, residual, q, scale, residual_out)
    if stream is not None or _device_index() != dev.index:
        return _on(stream, dev, rmsnorm_fp8, x, gain, eps, residual=residual, q=q, scale=scale,
                   residual_out=residual_out)
    xs = _row_stride("x", x, (T, D), _DTYPES)
    _need_layout("gain", gain, torch.float32, (D,))
    rs = ro = rd = 0
    if residual is not None:
        rs = _row_stride("residual", residual, (T, D), _DTYPES)
        rd = _DTYPES[residual.dtype]
        if residual_out is None:
            residual_out = _matrix_of(T, D, residual.dtype)
        else:
            ro = _row_stride("residual_out", residual_out, (T, D), (residual.dtype,))
    elif residual_out is not None:
        raise ValueError("residual_out without a residual")
    if q is None:
        q = _matrix_of(T, D, _FP8)
    else:
        _need_layout("q", q, _FP8, (T, D))
    if scale is None:
        scale = _matrix_of(T, _blocks128(D), torch.float32)
    else:
        _need_layout("scale", scale, torch.float32, (T, _blocks128(D)))
    _ok(lib.tr_rmsnorm_fp8(x.data_ptr(), _DTYPES[x.dtype], xs, _ptr(residual), rd, rs, _ptr(gain),
                           T, D, float(eps), q.data_ptr(), scale.data_ptr(), _ptr(residual_out),
                           ro, _raw_stream(dev.index)), "tr_rmsnorm_fp8")
    return q, scale, residual_out


def quantize_fp8(x, *, block_rows=1, q=None, scale=None, stream=None):
    """x [R, C] as an 8-bit operand: (q [R, C] e4m3, scale [ceil(R/block_rows), ceil(C/128)]
    fp32); block_rows 1 for an activation, 128 for a weight."""
    R, C = _matrix("x", x)
    dev = _need_cuda(x, q, scale)
    if stream is not None or _device_index() != dev.index:
        return _on(stream, dev, quantize_fp8, x, block_rows=block_rows, q=q, scale=scale)
    xs = _row_stride("x", x, (R, C), _DTYPES)
    if block_rows not in (1, 128):
        raise ValueError("block_rows must be 1 or 128")
    rb, cb = (R + block_rows - 1) // block_rows, _blocks128(C)
    if q is None:
        q = _matrix_of(R, C, _FP8)
    else:
        _need_layout("q", q, _FP8, (R, C))
    if scale is None:
        scale = _matrix_of(rb, cb, torch.float32)
    else:
        _need_layout("scale", scale, torch.float32, (rb, cb))
    _ok(lib.tr_quantize_fp8(x.data_ptr(), _DTYPES[x.dtype], xs, R, C, block_rows, q.data_ptr(),
                            scale.data_ptr(), _raw_stream(dev.index)), "tr_quantize_fp8")
    return q, scale


def projection_fp8(a, a_scale, w, w_scale, *, out_dtype=torch.bfloat16, y=None, stream=None):
    """y = a w^T [T, N] for an 8-bit activation a [T, K] and weight w [N, K] (e4m3 with the
    scales of quantize_fp8 / rmsnorm_fp8), fp32 sums, in out_dtype (bf16 or fp32; y's if given)."""
    T, K = _matrix("a", a)
    N = _matrix("w", w)[0]
    dev = _need_cuda(a, a_scale, w, w_scale, y)
    if stream is not None or _device_index() != dev.index:
        return _on(stream, dev, projection_fp8, a, a_scale, w, w_scale, out_dtype=out_dtype, y=y)
    as_ = _row_stride("a", a, (T, K), (_FP8,))
    ws = _row_stride("w", w, (N, K), (_FP8,))
    _need_layout("a_scale", a_scale, torch.float32, (T, _blocks128(K)))
    _need_layout("w_scale", w_scale, torch.float32, (_blocks128(N), _blocks128(K)))
    ys = 0
    if y is not None:
        out_dtype = y.dtype
        ys = _row_stride("y", y, (T, N), _DTYPES)
    elif out_dtype not in _DTYPES:
        raise TypeError("unsupported dtype %s" % out_dtype)
    else:
        y = _matrix_of(T, N, out_dtype)
    _ok(lib.tr_projection_fp8(a.data_ptr(), as_, a_scale.data_ptr(), w.data_ptr(), ws,
                              w_scale.data_ptr(), T, N, K, y.data_ptr(), _DTYPES[out_dtype], ys,
                              _raw_stream(dev.index)), "tr_projection_fp8")
    return y


def _offsets(cu_seqlens, device):
    """seqlens() that also refuses a pair the library would read wrongly."""
    host, dev = _seqlens(cu_seqlens, device)
    if host.dim() != 1 or dev.shape != host.shape or host.numel() < 1 or \
            not host.is_contiguous() or not dev.is_contiguous():
        raise ValueError("cu_seqlens must be N + 1 contiguous offsets")
    return host, dev


def linear_recurrence(x, gate, cu_seqlens, *, h0=None, gate_logits=False, want_y=True, y=None,
                      h_final=None, stream=None):
    """h_t = a_t h_{t-1} + x_t per channel over packed sequences: (y [T, C] or None, h_final
    [N, C] fp32).  a = exp(gate), or exp(-softplus(gate)) with gate_logits.  h0 [N, C] fp32
    (None: zero start); h_final may be h0.  For a captured call give cu_seqlens as seqlens().
    The outputs carry no autograd history; linear_recurrence_backward gives the gradients."""
    T, C = _matrix("x", x)
    dev = _need_cuda(x, gate, h0, y, h_final)
    if stream is not None or _device_index() != dev.index:
        return _on(stream, dev, linear_recurrence, x, gate, cu_seqlens, h0=h0,
                   gate_logits=gate_logits, want_y=want_y, y=y, h_final=h_final)
    xs = _row_stride("x", x, (T, C), _DTYPES)
    gs = _row_stride("gate", gate, (T, C), _DTYPES)
    ys = _row_stride("y", y, (T, C), (x.dtype,)) if y is not None else 0
    host, cu = _offsets(cu_seqlens, dev)
    N = host.shape[0] - 1
    _need_layout("h0", h0, torch.float32, (N, C))
    if not want_y:
        y = None
    elif y is None:
        y = _matrix_of(T, C, x.dtype)
    if h_final is None:
        h_final = _matrix_of(N, C, torch.float32)
    else:
        _need_layout("h_final", h_final, torch.float32, (N, C))
    a = RecurrenceArgs(N, C, T, _DTYPES[x.dtype], _DTYPES[gate.dtype],
                       TR_GATE_LOGITS if gate_logits else 0, xs, gs, ys, x.data_ptr(),
                       gate.data_ptr(), cu.data_ptr(), host.data_ptr(), _ptr(h0), _ptr(y),
                       h_final.data_ptr())
    _ok(lib.tr_linear_recurrence(ctypes.byref(a), _raw_stream(dev.index)), "tr_linear_recurrence")
    return y, h_final


def linear_recurrence_backward(dy, gate, y, cu_seqlens, *, h0=None, dh_final=None,
                               gate_logits=False, want_dh0=None, dx=None, dgate=None, dh0=None,
                               stream=None):
    """Gradients of linear_recurrence given dy and dh_final [N, C] fp32 (None: 0): (dx [T, C],
    dgate [T, C], dh0 [N, C] fp32 or None).  y is the forward call's output; dh0 is computed
    where want_dh0 (by default: where there is an h0 or a dh0 to fill) and may be dh_final."""
    T, C = _matrix("dy", dy)
    dev = _need_cuda(dy, gate, y, h0, dh_final, dx, dgate, dh0)
    if stream is not None or _device_index() != dev.index:
        return _on(stream, dev, linear_recurrence_backward, dy, gate, y, cu_seqlens, h0=h0,
                   dh_final=dh_final, gate_logits=gate_logits, want_dh0=want_dh0, dx=dx,
                   dgate=dgate, dh0=dh0)
    ds = _row_stride("dy", dy, (T, C), _DTYPES)
    gs = _row_stride("gate", gate, (T, C), _DTYPES)
    ys = _row_stride("y", y, (T, C), (dy.dtype,))
    dxs = _row_stride("dx", dx, (T, C), (dy.dtype,)) if dx is not None else 0
    dgs = _row_stride("dgate", dgate, (T, C), (gate.dtype,)) if dgate is not None else 0
    if want_dh0 is None:
        want_dh0 = h0 is not None or dh0 is not None
    host, cu = _offsets(cu_seqlens, dev)
    N = host.shape[0] - 1
    for name, t in (("h0", h0), ("dh_final", dh_final), ("dh0", dh0)):
        _need_layout(name, t, torch.float32, (N, C))
    if dx is None:
        dx = _matrix_of(T, C, dy.dtype)
    if dgate is None:
        dgate = _matrix_of(T, C, gate.dtype)
    if not want_dh0:
        dh0 = None
    elif dh0 is None:
        dh0 = _matrix_of(N, C, torch.float32)
    a = RecurrenceGradArgs(N, C, T, _DTYPES[dy.dtype], _DTYPES[gate.dtype],
                           TR_GATE_LOGITS if gate_logits else 0, ds, gs, ys, dxs, dgs,
                           dy.data_ptr(), gate.data_ptr(), y.data_ptr(), cu.data_ptr(),
                           host.data_ptr(), _ptr(h0), _ptr(dh_final), dx.data_ptr(),
                           dgate.data_ptr(), _ptr(dh0))
    _ok(lib.tr_linear_recurrence_backward(ctypes.byref(a), _raw_stream(dev.index)),
        "tr_linear_recurrence_backward")
    return dx, dgate, dh0


def set_wait_limit_ns(ns: int) -> None:
    """Wall-clock limit of the scan kernels' bounded waits for later calls (0: the default 4 s)."""
    _ok(lib.tr_set_wait_limit_ns(int(ns)), "tr_set_wait_limit_ns")


def check(stream=None) -> None:
    """Wait for the stream and raise if a kernel reported a device-side failure."""
    _ok(lib.tr_check(_stream(stream)), "tr_check")
