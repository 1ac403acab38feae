"""ctypes binding of liblmoe.so, the LatentMoE layer's C ABI (include/lmoe.h).

Argument marshalling only: every function takes torch CUDA tensors, checks
shapes and dtypes, and passes `data_ptr()` plus the current CUDA stream to
the C entry point of the same name.  All arithmetic runs in the library's
CUDA kernels.  Importing this module fails loudly when the library has not
been built (there is no fallback path).
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import sys

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
# LMOE_LIBRARY selects another build of the same library (e.g. a trace build)
LIB_PATH = os.environ.get("LMOE_LIBRARY") or os.path.join(_PKG, "liblmoe.so")

_HOW = ("build it with `python -c \"import __graft_entry__ as g; g.build()\"` or "
        "`python top_routing_mxfp4_gb300/build.py`")
if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: {_HOW}")

_lib = ctypes.CDLL(LIB_PATH)

OK = 0
ERR_INVALID_ARG = -1
ERR_UNSUPPORTED = -2
ERR_WORKSPACE = -3
ERR_CUDA = -4
ERR_DEVICE_CHECK = -5
ERR_TIMEOUT = -6
ACT_MXFP8 = 1
ACT_MXFP4 = 2
LAYOUT_CANONICAL = 0
LAYOUT_TC = 1


class Dims(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("d", ctypes.c_int32), ("E", ctypes.c_int32), ("k", ctypes.c_int32),
                ("I", ctypes.c_int32), ("act", ctypes.c_int32)]


class ExpertWeights(ctypes.Structure):
    _fields_ = [("gate_q", ctypes.c_void_p), ("gate_s", ctypes.c_void_p), ("up_q", ctypes.c_void_p),
                ("up_s", ctypes.c_void_p), ("down_q", ctypes.c_void_p), ("down_s", ctypes.c_void_p),
                ("layout", ctypes.c_int32)]


_vp, _i32, _i64, _sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
_DP, _WP = ctypes.POINTER(Dims), ctypes.POINTER(ExpertWeights)


def _sig(name, restype, *argtypes):
    f = getattr(_lib, name)
    f.restype = restype
    f.argtypes = list(argtypes)
    return f


_lib_version = _sig("lmoe_version", ctypes.c_char_p)
_status_string = _sig("lmoe_status_string", ctypes.c_char_p, ctypes.c_int)
_mxfp4_bytes = _sig("lmoe_mxfp4_bytes", _sz, _i64, _i32, _i32, _i32, ctypes.POINTER(_sz))
_quant_mxfp4 = _sig("lmoe_quant_mxfp4", ctypes.c_int, _vp, _i64, _i32, _i32, _vp, _vp, _i32, _vp)
_quant_mxfp8 = _sig("lmoe_quant_mxfp8", ctypes.c_int, _vp, _i64, _i32, _vp, _vp, _vp)
_repack_mxfp4 = _sig("lmoe_repack_mxfp4", ctypes.c_int, _vp, _vp, _i64, _i32, _i32, _vp, _vp, _vp)
_scale_hist = _sig("lmoe_mxfp4_scale_histogram", ctypes.c_int, _vp, _i64, _i32, _i32, _i32, _vp, _vp)
_route = _sig("lmoe_route", ctypes.c_int, _vp, _vp, _vp, _DP, _vp, _vp, _vp, _vp, _sz, _vp)
_router_bytes = _sig("lmoe_router_prepared_bytes", _sz, _i32, _i32)
_prepare_router = _sig("lmoe_prepare_router", ctypes.c_int, _vp, _i32, _i32, _vp, _vp)
_route_ws = _sig("lmoe_route_workspace_size", _sz, _DP)
_topk = _sig("lmoe_topk_from_logits", ctypes.c_int, _vp, _DP, _vp, _vp, _vp)
_perm_ws = _sig("lmoe_permute_workspace_size", _sz, _DP)
_permute = _sig("lmoe_permute", ctypes.c_int, _vp, _DP, _vp, _vp, _vp, _vp, _vp, _sz, _vp)
_permute_noalloc = _sig("lmoe_permute_noalloc", ctypes.c_int, _vp, _DP, _vp, _vp, _vp, _vp, _vp, _vp)
PERMUTE_NOALLOC_MAX_PAIRS = 524288
_ffn_ws = _sig("lmoe_expert_ffn_workspace_size", _sz, _DP)
_ffn = _sig("lmoe_expert_ffn", ctypes.c_int, _vp, _vp, _WP, _vp, _vp, _vp, _DP, _vp, _vp, _sz, _vp)
_combine = _sig("lmoe_combine", ctypes.c_int, _vp, _vp, _DP, _vp, _vp)
_ws_size = _sig("lmoe_workspace_size", _sz, _DP)
_forward = _sig("lmoe_forward", ctypes.c_int, _vp, _vp, _vp, _WP, _DP, _vp, _vp, _vp, _vp, _vp, _sz, _vp)
_linear = _sig("lmoe_linear_bf16", ctypes.c_int, _vp, _vp, _i64, _i32, _i32, _vp, _vp)
_block_ws = _sig("lmoe_block_workspace_size", _sz, _DP, _i32)
_forward_block = _sig("lmoe_forward_block", ctypes.c_int, _vp, _vp, _vp, _vp, _WP, _vp, _DP, _i32, _vp, _vp, _vp, _vp,
                      _vp, _vp, _vp, _sz, _vp)
_last_status = _sig("lmoe_last_device_status", ctypes.c_int, _vp, ctypes.POINTER(_i32))
_clear_status = _sig("lmoe_clear_device_status", ctypes.c_int, _vp, _vp)
_set_events = _sig("lmoe_set_stage_events", ctypes.c_int, ctypes.POINTER(_vp), _i32)
_kernel_count = _sig("lmoe_forward_kernel_count", _i32, _DP)


def _sig_later(name, restype, *argtypes):
    """As _sig; an earlier library chosen by LMOE_LIBRARY may lack the entry point, which a call then says."""
    if hasattr(_lib, name):
        return _sig(name, restype, *argtypes)

    def missing(*_):
        raise RuntimeError(f"{name} is not in {LIB_PATH}")
    return missing


_rms_norm = _sig_later("lmoe_rms_norm", ctypes.c_int, _vp, _i32, _vp, ctypes.c_float, _i64, _i32, _vp, _vp)
_residual_norm = _sig_later("lmoe_residual_norm", ctypes.c_int, _vp, _vp, _i32, _vp, _vp, _i32, ctypes.c_float,
                            ctypes.c_float, _vp, _i64, _i32, _vp, _vp, _vp)
_linear_mx_ws = _sig_later("lmoe_linear_mxfp4_workspace_size", _sz, _i64, _i32, _i32)
_linear_mx = _sig_later("lmoe_linear_mxfp4", ctypes.c_int, _vp, _vp, _vp, _i64, _i32, _i32, _vp, _vp, _sz, _vp)


class Groups(ctypes.Structure):
    _fields_ = [("offsets", ctypes.c_void_p), ("perm", ctypes.c_void_p), ("P", ctypes.c_int64), ("E", ctypes.c_int32),
                ("k", ctypes.c_int32)]


_GP = ctypes.POINTER(Groups)
_grouped_ws = _sig_later("lmoe_grouped_workspace_size", _sz)
_grouped_linear = _sig_later("lmoe_grouped_linear_bf16", ctypes.c_int, _vp, _i64, _vp, _GP, _i32, _vp, _i32, _i32, _i32,
                             _vp, _vp, _sz, _vp)
_grouped_swiglu = _sig_later("lmoe_grouped_swiglu_bf16", ctypes.c_int, _vp, _i64, _vp, _vp, _GP, _i32, _i32, _i32, _vp,
                             _vp, _sz, _vp)
class Projection(ctypes.Structure):
    _fields_ = [("w", ctypes.c_void_p), ("q", ctypes.c_void_p), ("s", ctypes.c_void_p)]


class ResidualBlockStruct(ctypes.Structure):
    _fields_ = [("inp", Projection), ("out", Projection), ("pre_w", ctypes.c_void_p), ("post_w", ctypes.c_void_p),
                ("gate", ctypes.c_void_p), ("gate_kind", ctypes.c_int32), ("scale", ctypes.c_float),
                ("eps", ctypes.c_float), ("next_w", ctypes.c_void_p)]


_res_block_ws = _sig_later("lmoe_residual_block_workspace_size", _sz, _DP, _i32)
_res_block = _sig_later("lmoe_forward_residual_block", ctypes.c_int, _vp, _i32, _vp,
                        ctypes.POINTER(ResidualBlockStruct), _vp, _vp, _WP, _DP, _i32, _vp, _vp, _vp, _sz, _vp)
class LinearAct(ctypes.Structure):
    _fields_ = [("bias", ctypes.c_void_p), ("bias_fmt", ctypes.c_int32), ("fn", ctypes.c_int32),
                ("res", ctypes.c_void_p), ("res_fmt", ctypes.c_int32)]


class BalanceGrad(ctypes.Structure):
    _fields_ = [("dlogits", ctypes.c_void_p), ("coef_balance", ctypes.c_float), ("coef_z", ctypes.c_float),
                ("scale", ctypes.c_void_p), ("topk_w", ctypes.c_void_p), ("dtopk_w", ctypes.c_void_p)]


_linear_act_ws = _sig_later("lmoe_linear_act_workspace_size", _sz, _i64, _i32, _i32)
_linear_act = _sig_later("lmoe_linear_act_bf16", ctypes.c_int, _vp, _vp, ctypes.POINTER(LinearAct), _i64, _i32, _i32, _i32,
                         _vp, _vp, _vp, _sz, _vp)
_linear_act_back_ws = _sig_later("lmoe_linear_act_backward_workspace_size", _sz, _i64, _i32, _i32)
_linear_act_back = _sig_later("lmoe_linear_act_bf16_backward", ctypes.c_int, _vp, _i32, _vp, _vp, _vp, _i32, _i64, _i32,
                              _i32, _vp, _vp, _i32, _vp, _vp, _sz, _vp)
_layer_norm = _sig_later("lmoe_layer_norm", ctypes.c_int, _vp, _i32, _vp, _vp, ctypes.c_float, _i64, _i32, _vp, _vp, _vp,
                         _vp)
_layer_norm_back_ws = _sig_later("lmoe_layer_norm_backward_workspace_size", _sz, _i64, _i32)
_layer_norm_back = _sig_later("lmoe_layer_norm_backward", ctypes.c_int, _vp, _vp, _i32, _vp, _vp, _vp, _vp, _i64, _i32,
                              _vp, _vp, _vp, _vp, _sz, _vp)
_balance_ws = _sig_later("lmoe_balance_loss_workspace_size", _sz, _i64, _i32, _i32)
_balance = _sig_later("lmoe_balance_loss", ctypes.c_int, _vp, _vp, _vp, _i64, _i32, _i32, _vp, _vp, _vp,
                      ctypes.POINTER(BalanceGrad), _vp, _sz, _vp)
FUNCTIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}
BF16, F32 = 0, 1
GATE_NONE, GATE_CHANNEL, GATE_TOKEN, GATE_FULL = 0, 1, 2, 3


class FfnViews(ctypes.Structure):
    _fields_ = [("xq", _i64), ("xs", _i64), ("hq", _i64), ("hs", _i64), ("dst_row", _i64), ("rows", _i64),
                ("tile_tokens", _i32), ("slot_rows", _i32), ("path", _i32), ("code_row", _i64), ("ksplit", _i64)]


_ws_views = _sig("lmoe_forward_workspace_views", ctypes.c_int, _DP, ctypes.POINTER(FfnViews))
_set_hcap = _sig("lmoe_set_h_capture", ctypes.c_int, _vp, _sz)
_set_wait_test = _sig("lmoe_set_wait_test", ctypes.c_int, _i32, _i64)
_set_small = _sig("lmoe_set_small_batch_pairs", ctypes.c_int, _i32)


def set_wait_test(stall_first_fill: bool, wait_limit_cycles: int = 0):
    """Failure-path test hook of the expert GEMMs' bounded waits
    (lmoe_set_wait_test); (False, 0) restores the normal behaviour."""
    _check(_set_wait_test(1 if stall_first_fill else 0, int(wait_limit_cycles)), "lmoe_set_wait_test")
_get_small = _sig("lmoe_small_batch_pairs", _i32)
SMALL_BATCH_PAIRS_DEFAULT = 0


def set_small_batch_pairs(max_pairs: int):
    """Batches of at most this many pairs (T * k, at most 8 tokens) run the
    small-batch path of lmoe_forward; 0 sends every batch to the tensor-core
    path.  Process-wide."""
    _check(_set_small(int(max_pairs)), "lmoe_set_small_batch_pairs")


def small_batch_pairs() -> int:
    return int(_get_small())


def forward_workspace_views(T: int, d: int, E: int, k: int, I: int) -> FfnViews:
    """Byte offsets of the expert GEMMs' MXFP8 operands inside lmoe_forward's
    workspace (diagnostics)."""
    v = FfnViews()
    D = dims(T, d, E, k, I)
    _check(_ws_views(ctypes.byref(D), ctypes.byref(v)), "lmoe_forward_workspace_views")
    return v


def set_h_capture(buf):
    """Diagnostics: a float32 CUDA tensor that later forward calls fill with
    the fp32 h values their gate/up GEMM rounds to MXFP8; None clears it."""
    if buf is None:
        _check(_set_hcap(None, 0), "lmoe_set_h_capture")
        return
    if buf.dtype != torch.float32 or not buf.is_cuda or not buf.is_contiguous():
        raise ValueError("h capture buffer: contiguous CUDA float32 tensor expected")
    _check(_set_hcap(_ptr(buf), buf.numel() * 4), "lmoe_set_h_capture")


def forward_kernel_count(T: int, d: int, E: int, k: int, I: int) -> int:
    D = dims(T, d, E, k, I)
    return int(_kernel_count(ctypes.byref(D)))
NUM_STAGE_EVENTS = 7
STAGES = ("route", "permute", "act_quant", "gate_up", "down", "combine")


def set_stage_events(events):
    """Record these torch.cuda.Event objects at lmoe_forward's stage boundaries
    (start, after route, permute, activation scatter, gate/up GEMM, down GEMM,
    combine); None clears the hook."""
    if events is None:
        _check(_set_events(None, 0), "lmoe_set_stage_events")
        return
    assert len(events) == NUM_STAGE_EVENTS
    arr = (_vp * NUM_STAGE_EVENTS)(*[ctypes.c_void_p(e.cuda_event) for e in events])
    _check(_set_events(arr, NUM_STAGE_EVENTS), "lmoe_set_stage_events")


class LmoeError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {status_string(code)} ({code})")
        self.code = code


def status_string(code: int) -> str:
    return _status_string(code).decode()


def version() -> str:
    return _lib_version().decode()


def _check(code: int, what: str):
    if code != OK:
        raise LmoeError(code, what)


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _need(t, dtype, shape, name):
    if t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name}: expected contiguous CUDA {dtype} {tuple(shape)}, got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")


def dims(T: int, d: int, E: int, k: int, I: int, act: int = ACT_MXFP8) -> Dims:
    return Dims(T, d, E, k, I, act)


def _empty(shape, dtype, device, stream=None):
    """An uninitialised tensor for a call on `stream` (None: the current one): where that is not the stream it is
    allocated on, it is recorded there, so that its memory goes to no other tensor while the call runs."""
    t = torch.empty(shape, dtype=dtype, device=device)
    if stream is not None:
        t.record_stream(stream)
    return t


def workspace(nbytes: int, device, stream=None) -> torch.Tensor:
    # torch's caching allocator returns 512-byte aligned blocks
    return _empty(max(int(nbytes), 256), torch.uint8, device, stream)


def _on(stream):
    """Allocations in the order of a call's stream."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _kept_workspace(ws, nbytes: int, device, stream):
    """The workspace an object keeps between calls: `ws`, or a larger one made in
    the order of the call's stream.  It is recorded on that stream, so that its
    memory, once it is replaced or dropped, goes to no other tensor while the
    stream still works on it."""
    if ws is None or ws.numel() < nbytes:
        with _on(stream):
            ws = workspace(nbytes, device)
    ws.record_stream(torch.cuda.current_stream(ws.device) if stream is None else stream)
    return ws


# ---- load-time conversion ----------------------------------------------------------

def mxfp4_bytes(nmat: int, rows: int, K: int, layout: int):
    sb = _sz()
    qb = _mxfp4_bytes(nmat, rows, K, layout, ctypes.byref(sb))
    if qb == 0 and nmat > 0:
        raise ValueError("bad MXFP4 matrix sizes")
    return int(qb), int(sb.value)


def quant_mxfp4(w: torch.Tensor, layout: int = LAYOUT_TC, q=None, s=None, stream=None):
    """fp32 [nmat, rows, K] (or [rows, K]) -> (codes, scales) as flat uint8 tensors."""
    w3 = w if w.dim() == 3 else w.unsqueeze(0)
    nmat, rows, K = w3.shape
    _need(w3, torch.float32, (nmat, rows, K), "w")
    qb, sb = mxfp4_bytes(nmat, rows, K, layout)
    q = _empty(qb, torch.uint8, w.device, stream) if q is None else q
    s = _empty(sb, torch.uint8, w.device, stream) if s is None else s
    assert q.numel() >= qb and s.numel() >= sb
    _check(_quant_mxfp4(_ptr(w3), nmat, rows, K, _ptr(q), _ptr(s), layout, _stream(stream)), "lmoe_quant_mxfp4")
    return q, s


def repack_mxfp4(q: torch.Tensor, s: torch.Tensor, nmat: int, rows: int, K: int, q_tc=None, s_tc=None, stream=None):
    """Canonical MXFP4 bytes (uint8 codes [nmat*rows*K/2], scales
    [nmat*rows*K/32], flat or shaped) -> the tensor-core layout, as flat uint8
    tensors (byte rearrangement; lmoe_repack_mxfp4)."""
    qb, sb = mxfp4_bytes(nmat, rows, K, LAYOUT_TC)
    _need(q, torch.uint8, q.shape, "q")
    _need(s, torch.uint8, s.shape, "s")
    if q.numel() != nmat * rows * K // 2 or s.numel() != nmat * rows * K // 32:
        raise ValueError("canonical MXFP4 arrays of the wrong size")
    q_tc = _empty(qb, torch.uint8, q.device, stream) if q_tc is None else q_tc
    s_tc = _empty(sb, torch.uint8, q.device, stream) if s_tc is None else s_tc
    if q_tc.numel() < qb or s_tc.numel() < sb:
        raise ValueError("tensor-core layout destination too small")
    _check(_repack_mxfp4(_ptr(q), _ptr(s), nmat, rows, K, _ptr(q_tc), _ptr(s_tc), _stream(stream)),
           "lmoe_repack_mxfp4")
    return q_tc, s_tc


def scale_histogram(s: torch.Tensor, nmat: int, rows: int, K: int, layout: int = LAYOUT_TC, stream=None):
    """Per-matrix counts of each E8M0 scale byte: int32-viewed uint32 [nmat, 256]."""
    _need(s, torch.uint8, s.shape, "s")
    hist = _empty((nmat, 256), torch.int32, s.device, stream)
    _check(_scale_hist(_ptr(s), nmat, rows, K, layout, _ptr(hist), _stream(stream)), "lmoe_mxfp4_scale_histogram")
    return hist


def quant_mxfp8(x: torch.Tensor, stream=None):
    """bf16 [rows, K] -> (e4m3 codes uint8 [rows, K], scales uint8 [rows, K/32])."""
    rows, K = x.shape
    _need(x, torch.bfloat16, (rows, K), "x")
    q = _empty((rows, K), torch.uint8, x.device, stream)
    s = _empty((rows, K // 32), torch.uint8, x.device, stream)
    _check(_quant_mxfp8(_ptr(x), rows, K, _ptr(q), _ptr(s), _stream(stream)), "lmoe_quant_mxfp8")
    return q, s


class ExpertBank:
    """An expert bank in the tensor-core MXFP4 layout, resident on the device.

    Built matrix by matrix from fp32 weights (load-time conversion), so the
    fp32 copy of the whole bank never has to exist on the device."""

    def __init__(self, E: int, d: int, I: int, device):
        self.E, self.d, self.I = E, d, I
        self.device = torch.device(device)
        gqb, gsb = mxfp4_bytes(E, I, d, LAYOUT_TC)
        dqb, dsb = mxfp4_bytes(E, d, I, LAYOUT_TC)
        self.gate_q, self.gate_s = _empty(gqb, torch.uint8, device), _empty(gsb, torch.uint8, device)
        self.up_q, self.up_s = _empty(gqb, torch.uint8, device), _empty(gsb, torch.uint8, device)
        self.down_q, self.down_s = _empty(dqb, torch.uint8, device), _empty(dsb, torch.uint8, device)
        self._struct = None

    @property
    def nbytes(self) -> int:
        return sum(t.numel() for t in (self.gate_q, self.gate_s, self.up_q, self.up_s, self.down_q, self.down_s))

    def load(self, which: str, e0: int, w: torch.Tensor, stream=None):
        """Quantise fp32 weights of experts [e0, e0 + w.shape[0]) into the bank."""
        n = w.shape[0]
        if which in ("gate", "up"):
            rows, K = self.I, self.d
        else:
            rows, K = self.d, self.I
        qb1, sb1 = mxfp4_bytes(1, rows, K, LAYOUT_TC)
        q = getattr(self, which + "_q")[e0 * qb1:(e0 + n) * qb1]
        s = getattr(self, which + "_s")[e0 * sb1:(e0 + n) * sb1]
        quant_mxfp4(w.reshape(n, rows, K), LAYOUT_TC, q, s, stream)

    def load_mxfp4(self, which: str, e0: int, q: torch.Tensor, s: torch.Tensor, stream=None):
        """Copy a checkpoint's canonical MXFP4 matrices of experts [e0, e0 + n)
        into the bank (lmoe_repack_mxfp4).  q, s: uint8 codes [n, rows, K/2]
        and scales [n, rows, K/32] on the device, e.g. a staging buffer the
        caller refills chunk by chunk."""
        rows, K = (self.I, self.d) if which in ("gate", "up") else (self.d, self.I)
        n = q.shape[0]
        qb1, sb1 = mxfp4_bytes(1, rows, K, LAYOUT_TC)
        qd = getattr(self, which + "_q")[e0 * qb1:(e0 + n) * qb1]
        sd = getattr(self, which + "_s")[e0 * sb1:(e0 + n) * sb1]
        repack_mxfp4(q, s, n, rows, K, qd, sd, stream)

    def scale_histograms(self, stream=None):
        """E8M0 scale-byte counts per expert matrix: {gate, up, down}: [E, 256]."""
        return {w: scale_histogram(getattr(self, w + "_s"), self.E, *((self.I, self.d) if w != "down" else
                                                                       (self.d, self.I)), LAYOUT_TC, stream)
                for w in ("gate", "up", "down")}

    def struct(self) -> ExpertWeights:
        if self._struct is None:
            self._struct = ExpertWeights(self.gate_q.data_ptr(), self.gate_s.data_ptr(), self.up_q.data_ptr(),
                                         self.up_s.data_ptr(), self.down_q.data_ptr(), self.down_s.data_ptr(),
                                         LAYOUT_TC)
        return self._struct


# ---- stages ------------------------------------------------------------------------

def prepare_router(Wr, stream=None):
    """fp32 router weights [E, d] -> the three bf16 planes [3, E, d] the router
    GEMM reads (their sum is Wr exactly)."""
    E, d = Wr.shape
    _need(Wr, torch.float32, (E, d), "Wr")
    if int(_router_bytes(E, d)) == 0:
        raise ValueError(f"router weights [{E}, {d}]: d must be a multiple of 64")
    Wr3 = _empty((3, E, d), torch.bfloat16, Wr.device, stream)
    _check(_prepare_router(_ptr(Wr), E, d, _ptr(Wr3), _stream(stream)), "lmoe_prepare_router")
    return Wr3


def route(x, Wr, k: int, bias=None, stream=None, Wr3=None):
    """Router + top-k + softmax.  Wr: fp32 [E, d] (prepared on the fly) or
    Wr3: prepared planes [3, E, d]."""
    T, d = x.shape
    if Wr3 is None:
        Wr3 = prepare_router(Wr, stream)
    E = Wr3.shape[1]
    _need(x, torch.bfloat16, (T, d), "x")
    _need(Wr3, torch.bfloat16, (3, E, d), "Wr3")
    if bias is not None:
        _need(bias, torch.float32, (E,), "bias")
    D = dims(T, d, E, k, 32)
    logits = _empty((T, E), torch.float32, x.device, stream)
    idx = _empty((T, k), torch.int32, x.device, stream)
    w = _empty((T, k), torch.float32, x.device, stream)
    ws = workspace(_route_ws(ctypes.byref(D)), x.device, stream)
    _check(_route(_ptr(x), _ptr(Wr3), _ptr(bias), ctypes.byref(D), _ptr(logits), _ptr(idx), _ptr(w), _ptr(ws),
                  ws.numel(), _stream(stream)), "lmoe_route")
    return logits, idx, w


def topk_from_logits(logits, k: int, stream=None):
    T, E = logits.shape
    _need(logits, torch.float32, (T, E), "logits")
    D = dims(T, 128, E, k, 32)
    idx = _empty((T, k), torch.int32, logits.device, stream)
    w = _empty((T, k), torch.float32, logits.device, stream)
    _check(_topk(_ptr(logits), ctypes.byref(D), _ptr(idx), _ptr(w), _stream(stream)), "lmoe_topk_from_logits")
    return idx, w


def permute_workspace_size(T: int, E: int, k: int) -> int:
    D = dims(T, 128, E, k, 32)
    return int(_perm_ws(ctypes.byref(D)))


def permute(idx, E: int, ws=None, stream=None):
    T, k = idx.shape
    _need(idx, torch.int32, (T, k), "topk_idx")
    D = dims(T, 128, E, k, 32)
    dev = idx.device
    counts = _empty(E, torch.int32, dev, stream)
    offsets = _empty(E + 1, torch.int32, dev, stream)
    perm = _empty(T * k, torch.int32, dev, stream)
    inv = _empty(T * k, torch.int32, dev, stream)
    ws = workspace(_perm_ws(ctypes.byref(D)), dev, stream) if ws is None else ws
    _check(_permute(_ptr(idx), ctypes.byref(D), _ptr(counts), _ptr(offsets), _ptr(perm), _ptr(inv), _ptr(ws),
                    ws.numel(), _stream(stream)), "lmoe_permute")
    return counts, offsets, perm, inv, ws


def permute_noalloc(idx, E: int, out=None, stream=None):
    """lmoe_permute_noalloc: the permute with no workspace (the library's fixed
    device array holds the scratch).  `out` may pass preallocated
    (counts, offsets, perm, inv, device_status) tensors, so the call itself
    allocates nothing."""
    T, k = idx.shape
    _need(idx, torch.int32, (T, k), "topk_idx")
    D = dims(T, 128, E, k, 32)
    dev = idx.device
    if out is None:
        out = tuple(_empty(n, torch.int32, dev, stream) for n in (E, E + 1, T * k, T * k, 1))
    counts, offsets, perm, inv, status = out
    for t, shape, name in ((counts, (E,), "counts"), (offsets, (E + 1,), "offsets"), (perm, (T * k,), "perm"),
                           (inv, (T * k,), "inv"), (status, (1,), "device_status")):
        _need(t, torch.int32, shape, name)
        if t.device != dev:
            raise ValueError(f"{name}: on {t.device}, topk_idx on {dev}")
    _check(_permute_noalloc(_ptr(idx), ctypes.byref(D), _ptr(counts), _ptr(offsets), _ptr(perm), _ptr(inv),
                            _ptr(status), _stream(stream)), "lmoe_permute_noalloc")
    return counts, offsets, perm, inv, status


def expert_ffn(xq, xs, bank: ExpertBank, offsets, perm, topk_w, k: int, ws=None, stream=None):
    T, d = xq.shape
    D = dims(T, d, bank.E, k, bank.I)
    _need(xq, torch.uint8, (T, d), "xq")
    _need(xs, torch.uint8, (T, d // 32), "xs")
    _need(offsets, torch.int32, (bank.E + 1,), "offsets")
    _need(perm, torch.int32, (T * k,), "perm")
    _need(topk_w, torch.float32, (T, k), "topk_w")
    yp = _empty((T * k, d), torch.float32, xq.device, stream)
    ws = workspace(_ffn_ws(ctypes.byref(D)), xq.device, stream) if ws is None else ws
    W = bank.struct()
    _check(_ffn(_ptr(xq), _ptr(xs), ctypes.byref(W), _ptr(offsets), _ptr(perm), _ptr(topk_w), ctypes.byref(D),
                _ptr(yp), _ptr(ws), ws.numel(), _stream(stream)), "lmoe_expert_ffn")
    return yp, ws


def combine(yp, inv, T: int, k: int, stream=None):
    P, d = yp.shape
    _need(yp, torch.float32, (T * k, d), "yp")
    _need(inv, torch.int32, (T * k,), "inv")
    D = dims(T, d, 32, k, 32)
    y = _empty((T, d), torch.bfloat16, yp.device, stream)
    _check(_combine(_ptr(yp), _ptr(inv), ctypes.byref(D), _ptr(y), _stream(stream)), "lmoe_combine")
    return y


# ---- whole layer -------------------------------------------------------------------

def workspace_size(T: int, d: int, E: int, k: int, I: int) -> int:
    D = dims(T, d, E, k, I)
    return int(_ws_size(ctypes.byref(D)))


class Layer:
    """A LatentMoE layer: router weights (fp32, prepared once into the form the
    router GEMM reads), optional logit bias, expert bank."""

    def __init__(self, Wr: torch.Tensor, bank: ExpertBank, k: int = 16, bias=None, act: int = ACT_MXFP8):
        self.Wr, self.bank, self.k, self.bias, self.act = Wr, bank, k, bias, act
        self.Wr3 = prepare_router(Wr)
        self._ws = None

    def workspace(self, T: int, stream=None) -> torch.Tensor:
        """The layer's own workspace, made larger if T tokens need it, for a call on `stream`."""
        self._ws = _kept_workspace(self._ws, workspace_size(T, self.bank.d, self.bank.E, self.k, self.bank.I),
                                   self.Wr.device, stream)
        return self._ws

    def forward(self, x, y=None, topk_idx=None, topk_w=None, logits=None, stream=None):
        T, d = x.shape
        _need(x, torch.bfloat16, (T, d), "x")
        D = dims(T, d, self.bank.E, self.k, self.bank.I, self.act)
        y = _empty((T, d), torch.bfloat16, x.device, stream) if y is None else y
        ws = self.workspace(T, stream)
        W = self.bank.struct()
        _check(_forward(_ptr(x), _ptr(self.Wr3), _ptr(self.bias), ctypes.byref(W), ctypes.byref(D), _ptr(y),
                        _ptr(topk_idx), _ptr(topk_w), _ptr(logits), _ptr(ws), ws.numel(), _stream(stream)),
               "lmoe_forward")
        return y

    def device_status(self) -> int:
        return last_device_status(self._ws)


def linear_bf16(x, W, out=None, stream=None):
    """out = bf16(x W^T): x bf16 [rows, K], W bf16 [N, K]."""
    rows, K = x.shape
    N = W.shape[0]
    _need(x, torch.bfloat16, (rows, K), "x")
    _need(W, torch.bfloat16, (N, K), "W")
    out = _empty((rows, N), torch.bfloat16, x.device, stream) if out is None else out
    _check(_linear(_ptr(x), _ptr(W), rows, K, N, _ptr(out), _stream(stream)), "lmoe_linear_bf16")
    return out


# ---- norms, MXFP4 linear and grouped products around the layer ----------------------------

# These calls run on the device of their first tensor and, by default, on that
# device's current stream; what they allocate is allocated on the call's stream,
# as within torch.cuda.stream(stream).  The short ones are bound in C++ (csrc/bind_torch.cpp).
# It is loaded at the first of them, so that the rest needs only the library.
class _Binding:
    def __getattr__(self, name):
        global _fast
        if name.startswith("_"):
            raise AttributeError(name)
        entries = (_rms_norm, _residual_norm, _linear_mx, _linear_mx_ws, _grouped_linear, _grouped_swiglu, _grouped_ws)
        for f in entries:
            if not hasattr(f, "argtypes"):
                f()  # raises: not in this library
        try:
            from . import _lmoe_torch
        except ImportError as e:
            path = os.path.join(_PKG, "_lmoe_torch.so")
            raise ImportError(f"{path} is missing or does not load ({e}): {_HOW}") from e
        here = f"torch {torch.__version__}, {sys.implementation.cache_tag}"
        if _lmoe_torch.BUILT_FOR != here:
            raise ImportError(f"_lmoe_torch.so was built for {_lmoe_torch.BUILT_FOR}, this is {here}: {_HOW}")
        _lmoe_torch.bind(LmoeError, *(ctypes.cast(f, _vp).value for f in entries))
        _fast = _lmoe_torch
        return getattr(_fast, name)


_fast = _Binding()


def _arg(t, dtype, shape, name, di):
    """Checks one tensor (contiguous, on CUDA device `di`); returns its address."""
    if t.dtype is not dtype or t.shape != shape or di < 0 or t.get_device() != di or not t.is_contiguous():
        raise ValueError(f"{name}: expected contiguous {dtype} {tuple(shape)} on cuda:{di}, got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}, strides {t.stride()}")
    return t.data_ptr()


def _on_device(t, name, di):
    """The address of weights whose type and shape were checked when they were taken in."""
    if t.get_device() != di:
        raise ValueError(f"{name}: on {t.device}, the call's tensors on cuda:{di}")
    return t.data_ptr()


def _make(shape, dtype, x, stream):
    """An uninitialised tensor on x's device, allocated in the order of the call's stream."""
    with _on(stream):
        return torch.empty(shape, dtype=dtype, device=x.device)


def _fmt(t, name):
    if t.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"{name}: expected bfloat16 or float32, got {t.dtype}")
    return BF16 if t.dtype is torch.bfloat16 else F32


def _gate(gate, T, H, di):
    gs = gate.shape
    if gate.dtype is torch.bfloat16:
        return GATE_FULL, _arg(gate, torch.bfloat16, (T, H), "gate", di)
    if gs == (T, 1):
        return GATE_TOKEN, _arg(gate, torch.float32, gs, "gate", di)
    return GATE_CHANNEL, _arg(gate, torch.float32, (1, H) if len(gs) == 2 else (H,), "gate", di)


def rms_norm(x, w, eps: float = 1e-5, out=None, stream=None):
    """The norm before a block: x [T, H] bf16 or fp32, w fp32 [H] -> bf16 [T, H] (lmoe_rms_norm)."""
    return _fast.rms_norm(x, w, eps, out, stream)


def residual_norm(y, res, post_w=None, gate=None, scale: float = 1.0, next_w=None, eps: float = 1e-5, res_out=None,
                  next_out=None, stream=None):
    """After a block (lmoe_residual_norm): res + scale * gate * norm(y; post_w)
    and, with next_w, its norm.  y bf16 [T, H]; res [T, H] bf16 or fp32; gate
    fp32 [H] or [1, H] (per channel), fp32 [T, 1] (per token) or bf16 [T, H].
    Returns (res_out, next_out or None)."""
    return _fast.residual_norm(y, res, post_w, gate, scale, next_w, eps, res_out, next_out, stream)


def linear_mxfp4_workspace_size(rows: int, K: int, N: int) -> int:
    return int(_linear_mx_ws(rows, K, N))


def linear_mxfp4(x, q, s, N: int, out=None, ws=None, stream=None):
    """out = bf16(x W^T): x bf16 [rows, K], W one MXFP4 matrix [N, K] in the
    tensor-core layout (q, s of quant_mxfp4 or repack_mxfp4).  `ws`: a zeroed
    workspace of linear_mxfp4_workspace_size bytes, kept by the caller
    (last_device_status(ws) says what calls with it found); one is made for the
    call without it (last_call_status)."""
    return _fast.linear_mxfp4(x, q, s, N, out, ws, stream)


def grouped_workspace_size() -> int:
    return int(_grouped_ws())


def grouped_linear_bf16(x, W, offsets, perm=None, k: int = 1, gather=None, row_w=None, out=None, ws=None, stream=None):
    """Products grouped by expert (lmoe_grouped_linear_bf16): row q of expert e
    (offsets[e] <= q < offsets[e + 1]) is x[perm[q] // k] (gather, the default
    with perm) or x[q], times W[e]^T, W bf16 [E, N, K].  Without row_w: bf16
    [P, N].  With row_w (fp32, P values in pair order): fp32 [P, N], row q
    times row_w[perm[q]].  `out` may be given in either type; rows in no group
    are not written.  `ws`: a zeroed workspace kept by the caller
    (last_device_status(ws) says whether offsets or rows were bad); one is made
    for the call without it (last_call_status)."""
    return _fast.grouped(x, W, None, offsets, perm, k, gather, row_w, out, ws, stream)


def grouped_swiglu_bf16(x, Wg, Wu, offsets, perm=None, k: int = 1, gather=None, out=None, ws=None, stream=None):
    """bf16 [P, I] rows silu(x Wg[e]^T) * (x Wu[e]^T), both products and the
    gating in one kernel (lmoe_grouped_swiglu_bf16); arguments as for
    grouped_linear_bf16."""
    if Wu is None:
        raise ValueError("Wu: expected a tensor")
    return _fast.grouped(x, Wg, Wu, offsets, perm, k, gather, None, out, ws, stream)


# ---- the layer's dense, trained neighbours: linear with bias, function and residual, layer norm, balance loss ----
#
# As with every call of this module, autograd records nothing: outputs have no graph, also where inputs require a
# gradient.  A torch.autograd.Function that trains makes the forward and the _backward call itself.

class _TrainBinding:
    """The entry points of these calls, handed to the compiled binding at the first of them."""

    def __getattr__(self, name):
        global _train
        if name.startswith("_"):
            raise AttributeError(name)
        entries = (_linear_act, _linear_act_ws, _linear_act_back, _linear_act_back_ws, _layer_norm, _layer_norm_back,
                   _layer_norm_back_ws, _balance, _balance_ws)
        for f in entries:
            if not hasattr(f, "argtypes"):
                f()  # raises: not in this library
        _fast.own_ws  # loads the binding
        _fast.bind_train(*(ctypes.cast(f, _vp).value for f in entries))
        _train = _fast
        return getattr(_train, name)


_train = _TrainBinding()


def _function(act: str) -> int:
    if act not in FUNCTIONS:
        raise ValueError(f"act: expected one of {', '.join(FUNCTIONS)}, got {act!r}")
    return FUNCTIONS[act]


def linear_act_workspace_size(rows: int, K: int, N: int) -> int:
    """Bytes for linear_act_bf16 with up to `rows` rows."""
    return int(_linear_act_ws(rows, K, N))


def linear_act_bf16(x, W, bias=None, act: str = "none", res=None, out=None, pre=None, ws=None, stream=None):
    """out = act(x W^T + bias) + res (lmoe_linear_act_bf16): x bf16 [rows, K], W
    bf16 [N, K], bias fp32 or bf16 [N], act one of FUNCTIONS, res bf16 or fp32
    [rows, N].  Without `out`: of res's type, bf16 without one.  With pre=True, or a
    bf16 tensor [rows, N] to write, returns (out, pre), pre = x W^T + bias as the
    backward call takes it.  `ws`: a zeroed workspace of linear_act_workspace_size
    bytes, kept by the caller (last_device_status(ws) says what calls with it
    found); one is made for the call without it (last_call_status)."""
    return _train.linear_act(x, W, bias, _function(act), res, out, pre, ws, stream)


def linear_act_backward_workspace_size(rows: int, K: int, N: int) -> int:
    """Bytes for linear_act_bf16_backward with up to `rows` rows."""
    return int(_linear_act_back_ws(rows, K, N))


def linear_act_bf16_backward(dout, x, W, act: str = "none", pre=None, want_dx: bool = True, want_dW: bool = True,
                             want_dbias: bool = True, dx=None, dW=None, dbias=None, ws=None, stream=None):
    """The gradients of linear_act_bf16 (lmoe_linear_act_bf16_backward): dout bf16
    or fp32 [rows, N], pre as the forward call gave it (None where act is "none").
    Returns (dx bf16 [rows, K], dW [N, K], dbias fp32 [N]), None for what is not
    wanted; dW is bf16, or of the type of the one given.  The residual's gradient is
    dout.  `ws` as for linear_act_bf16, of linear_act_backward_workspace_size bytes."""
    return _train.linear_act_backward(dout, x, W, _function(act), pre, want_dx, want_dW, want_dbias, dx, dW, dbias, ws,
                                      stream)


def layer_norm(x, w=None, b=None, eps: float = 1e-5, stats: bool = False, out=None, mean=None, rstd=None, stream=None):
    """Layer norm (lmoe_layer_norm): x [T, H] bf16 or fp32, w and b fp32 [H] or None
    -> bf16 [T, H]; with stats (or mean and rstd to write, fp32 [T]) returns (out,
    mean, rstd), the rows' statistics for the backward call."""
    return _train.layer_norm(x, w, b, eps, stats, out, mean, rstd, stream)


def layer_norm_backward_workspace_size(T: int, H: int) -> int:
    return int(_layer_norm_back_ws(T, H))


def layer_norm_backward(dy, x, mean, rstd, w=None, add=None, want_params: bool = True, dx=None, dw=None, db=None, ws=None,
                        stream=None):
    """The gradients of layer_norm (lmoe_layer_norm_backward): dy bf16 [T, H], x,
    mean, rstd as the forward call took and gave them; add (x's type): a gradient
    that is added to dx.  Returns (dx of x's type, dw fp32 [H], db fp32 [H]), without
    want_params (dx, None, None).  `ws`: a workspace of
    layer_norm_backward_workspace_size bytes (its content does not matter)."""
    return _train.layer_norm_backward(dy, x, mean, rstd, w, add, want_params, dx, dw, db, ws, stream)


def balance_loss_workspace_size(T: int, E: int, k: int) -> int:
    return int(_balance_ws(T, E, k))


def balance_loss(logits, topk_idx, mask=None, coef=(0.01, 0.001), grad: bool = False, topk_w=None, dtopk_w=None, scale=None,
                 dlogits=None, ws=None, stream=None):
    """A router's losses and per-expert counts (lmoe_balance_loss): logits fp32
    [T, E] and topk_idx int32 [T, k] as route gives them, mask bool [T] (False: a
    token that does not count).  Returns (loss fp32 [2]: balance and z, counts int32
    [E], probs fp32 [E]), and with grad (or `dlogits` to write) a fourth, dlogits
    fp32 [T, E]: the gradient of coef[0] loss[0] + coef[1] loss[1], times the fp32
    scalar on the device `scale` where given, plus with topk_w and dtopk_w (fp32
    [T, k]) the gradient that comes through the gate weights.  `ws`: a zeroed
    workspace of balance_loss_workspace_size bytes, kept by the caller
    (last_device_status(ws) says whether ids were bad); one is made for the call
    without it (last_call_status)."""
    return _train.balance_loss(logits, topk_idx, mask, coef[0], coef[1], grad, topk_w, dtopk_w, scale, dlogits, ws, stream)


def last_call_status() -> int:
    """The device status (as last_device_status) of the latest linear_mxfp4,
    grouped_linear_bf16, grouped_swiglu_bf16, expert_ffn_bf16, linear_act_bf16,
    linear_act_bf16_backward or balance_loss call, of any thread, that was given no workspace; of its latest replay, if it was
    captured.  The call's workspace is kept for this until the next such call.
    Calls with a workspace of the caller's are asked with last_device_status."""
    ws = _fast.own_ws()
    if ws is None:
        return OK
    with torch.cuda.device(ws.device):
        return last_device_status(ws)


class LinearMxfp4:
    """A linear layer with MXFP4 weights [N, K] in the tensor-core layout: from
    fp32 or bf16 weights (quantised) or from codes and scales."""

    def __init__(self, W=None, q=None, s=None, N: int = 0, K: int = 0):
        if W is not None:
            N, K = W.shape
            q, s = quant_mxfp4(W.float().contiguous())
        self.N, self.K, self.q, self.s = N, K, q, s
        qb, sb = mxfp4_bytes(1, N, K, LAYOUT_TC)
        _need(q, torch.uint8, (qb,), "q")
        _need(s, torch.uint8, (sb,), "s")

    def forward(self, x, out=None, ws=None, stream=None):
        return linear_mxfp4(x, self.q, self.s, self.N, out=out, ws=ws, stream=stream)


class ExpertBankBf16:
    """An unquantised expert bank: gate and up [E, I, d], down [E, d, I], bf16."""

    def __init__(self, gate: torch.Tensor, up: torch.Tensor, down: torch.Tensor):
        E, I, d = gate.shape
        _need(gate, torch.bfloat16, (E, I, d), "gate")
        _need(up, torch.bfloat16, (E, I, d), "up")
        _need(down, torch.bfloat16, (E, d, I), "down")
        self.gate, self.up, self.down, self.E, self.d, self.I = gate, up, down, E, d, I


def expert_ffn_bf16(x, bank: ExpertBankBf16, offsets, perm, topk_w, k: int, ws=None, stream=None):
    """expert_ffn on a bf16 bank: x bf16 [T, d] in token order -> yp fp32
    [T*k, d] in permuted order, as combine takes it (grouped_swiglu_bf16, then
    grouped_linear_bf16 with the gate weights)."""
    if ws is None:  # one for both, so that neither's errors are lost
        with _on(stream):
            ws = torch.zeros(max(grouped_workspace_size(), 256), dtype=torch.uint8, device=x.device)
        _fast.keep_ws(ws)
    h = grouped_swiglu_bf16(x, bank.gate, bank.up, offsets, perm, k, ws=ws, stream=stream)
    return grouped_linear_bf16(h, bank.down, offsets, perm, k, gather=False, row_w=topk_w, ws=ws, stream=stream)


class ResidualBlock:
    """The layer in a residual stream (lmoe_forward_residual_block): norm before
    (pre_w), projection, LatentMoE layer, projection, norm after (post_w), gate
    (fp32 [hidden]), residual scale.  W_in [d, hidden] and W_out [hidden, d]:
    bf16 tensors or LinearMxfp4.  One forward at a time on the object's own
    workspace; forwards that may overlap on the GPU are given one each (`ws`), and
    a forward captured into a graph without one gets its own, which goes back to
    the graph's memory behind it: give `ws` to ask for a captured forward's status."""

    def __init__(self, layer: Layer, W_in, W_out, pre_w=None, post_w=None, gate=None, scale: float = 1.0,
                 eps: float = 1e-5):
        d = layer.bank.d
        hidden = W_in.K if isinstance(W_in, LinearMxfp4) else W_in.shape[1]
        for W, shape, name in ((W_in, (d, hidden), "W_in"), (W_out, (hidden, d), "W_out")):
            if isinstance(W, LinearMxfp4):
                if (W.N, W.K) != shape:
                    raise ValueError(f"{name}: expected {shape}, got {(W.N, W.K)}")
            else:
                _need(W, torch.bfloat16, shape, name)
        self.layer, self.W_in, self.W_out, self.hidden = layer, W_in, W_out, hidden
        self.pre_w, self.post_w, self.gate, self.scale, self.eps = pre_w, post_w, gate, scale, eps
        self._ws = None

    @staticmethod
    def _proj(W, name, di):
        if isinstance(W, LinearMxfp4):
            return Projection(None, _on_device(W.q, name + ".q", di), _on_device(W.s, name + ".s", di))
        return Projection(_on_device(W, name, di), None, None)

    def workspace_size(self, T: int) -> int:
        bank = self.layer.bank
        D = dims(T, bank.d, bank.E, self.layer.k, bank.I, self.layer.act)
        return int(_res_block_ws(ctypes.byref(D), self.hidden))

    def forward(self, res, x_n=None, gate=None, next_w=None, res_out=None, next_out=None, ws=None, stream=None):
        """res [T, hidden] bf16 or fp32 -> (res_out, next_out or None).  x_n: the
        already normalised rows (a previous block's next_out); gate: per call, as
        residual_norm's, instead of the block's; next_w: the next block's pre_w."""
        T, H = res.shape
        di = res.get_device()
        fmt = _fmt(res, "res")
        rp = _arg(res, res.dtype, (T, self.hidden), "res", di)
        vec = lambda t, name: None if t is None else _arg(t, torch.float32, (H,), name, di)
        xp = None if x_n is None else _arg(x_n, torch.bfloat16, (T, H), "x_n", di)
        gate = self.gate if gate is None else gate
        kind, gp = (GATE_NONE, None) if gate is None else _gate(gate, T, H, di)
        if next_w is None and next_out is not None:
            raise ValueError("next_out without next_w")
        B = ResidualBlockStruct(self._proj(self.W_in, "W_in", di), self._proj(self.W_out, "W_out", di),
                                vec(self.pre_w, "pre_w"), vec(self.post_w, "post_w"), gp, kind, self.scale, self.eps,
                                vec(next_w, "next_w"))
        if x_n is None and self.pre_w is None:
            raise ValueError("neither x_n nor pre_w")
        if stream is not None and stream.device.index != di:
            raise ValueError(f"stream on {stream.device}, tensors on cuda:{di}")
        sp = (torch.cuda.current_stream(di) if stream is None else stream).cuda_stream
        res_out = _make((T, H), res.dtype, res, stream) if res_out is None else res_out
        rop = _arg(res_out, res.dtype, (T, H), "res_out", di)
        if next_w is not None and next_out is None:
            next_out = _make((T, H), torch.bfloat16, res, stream)
        nop = None if next_out is None else _arg(next_out, torch.bfloat16, (T, H), "next_out", di)
        layer, bank = self.layer, self.layer.bank
        D = dims(T, bank.d, bank.E, layer.k, bank.I, layer.act)
        router = _arg(layer.Wr3, torch.bfloat16, (3, bank.E, bank.d), "Wr3", di)
        bias = None if layer.bias is None else _arg(layer.bias, torch.float32, (bank.E,), "bias", di)
        W = ExpertWeights(*(_on_device(getattr(bank, name), name, di) for name in
                            ("gate_q", "gate_s", "up_q", "up_s", "down_q", "down_s")), LAYOUT_TC)
        if ws is None:
            need = max(self.workspace_size(T), 256)
            with _on(stream):
                captured = torch.cuda.is_current_stream_capturing()
            if captured:
                ws = _make((need,), torch.uint8, res, stream)
            else:
                ws = self._ws = _kept_workspace(self._ws, need, res.device, stream)
        wsp = _arg(ws, torch.uint8, ws.shape, "ws", di)
        with torch.cuda.device(di):
            _check(_res_block(rp, fmt, xp, ctypes.byref(B), router, bias, ctypes.byref(W), ctypes.byref(D), H, rop,
                              nop, wsp, ws.numel(), sp), "lmoe_forward_residual_block")
        return res_out, next_out

    def device_status(self) -> int:
        """Of the last forward on the object's own workspace (one that was given no `ws` and not captured)."""
        return last_device_status(self._ws)


class Block:
    """hidden -> latent projection, the LatentMoE layer, latent -> hidden."""

    def __init__(self, W_in: torch.Tensor, layer: Layer, W_out: torch.Tensor):
        self.W_in, self.layer, self.W_out = W_in, layer, W_out
        self._ws = None

    def forward(self, x_h, out=None, lat=None, y=None, topk_idx=None, topk_w=None, logits=None, stream=None):
        T, hidden = x_h.shape
        bank, k = self.layer.bank, self.layer.k
        _need(x_h, torch.bfloat16, (T, hidden), "x_h")
        _need(self.W_in, torch.bfloat16, (bank.d, hidden), "W_in")
        _need(self.W_out, torch.bfloat16, (hidden, bank.d), "W_out")
        D = dims(T, bank.d, bank.E, k, bank.I)
        need = int(_block_ws(ctypes.byref(D), hidden))
        self._ws = _kept_workspace(self._ws, need, x_h.device, stream)
        out = _empty((T, hidden), torch.bfloat16, x_h.device, stream) if out is None else out
        W = bank.struct()
        _check(_forward_block(_ptr(x_h), _ptr(self.W_in), _ptr(self.layer.Wr3), _ptr(self.layer.bias), ctypes.byref(W),
                              _ptr(self.W_out), ctypes.byref(D), hidden, _ptr(out), _ptr(lat), _ptr(y), _ptr(topk_idx),
                              _ptr(topk_w), _ptr(logits), _ptr(self._ws), self._ws.numel(), _stream(stream)),
               "lmoe_forward_block")
        return out


def last_device_status(ws) -> int:
    v = _i32()
    _check(_last_status(_ptr(ws), ctypes.byref(v)), "lmoe_last_device_status")
    return int(v.value)
