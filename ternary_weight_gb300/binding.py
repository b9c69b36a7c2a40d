"""ctypes binding of libbitnet_gb300 (the C ABI in include/bitnet.h).

Argument marshalling only: every step of the computation runs in the library's CUDA
kernels. Tensors are torch CUDA tensors (torch supplies device memory and streams); the
functions pass their data pointers and the current stream to the C entry points and raise
``BitnetError`` on a negative status. There is no CPU fallback: if the shared library is
missing or fails to load, ``lib()`` raises.
"""
from __future__ import annotations

import ctypes
import os

from . import _build

BITNET_OK = 0
BITNET_EINVAL = -1
BITNET_EALIGN = -2
BITNET_ECUDA = -3
BITNET_EUNSUPPORTED = -4
BITNET_ETIMEOUT = -5
BITNET_ERANGE = -6

BITNET_F32 = 0
BITNET_BF16 = 1

ALGO = {"auto": 0, "gemv": 1, "gemm": 2, "smallm": 3, "prefill": 4, "pair": 5}

# every entry point of include/bitnet.h with its ctypes signature
_P = ctypes.c_void_p
_I64 = ctypes.c_int64
SIGNATURES = {
    "bitnet_version": ([], ctypes.c_int),
    "bitnet_strerror": ([ctypes.c_int], ctypes.c_char_p),
    "bitnet_pack_i2s": ([_P, _P, _I64, _I64, _P, _P], ctypes.c_int),
    "bitnet_quant_act": ([_P, ctypes.c_int, _I64, _I64, _P, _P, _P, _P], ctypes.c_int),
    "bitnet_i2s_matmul": ([_P, _P, _P, _P, ctypes.c_float, _P, _P, _I64, _I64, _I64, _P], ctypes.c_int),
    "bitnet_i2s_matmul_algo": (
        [_P, _P, _P, _P, ctypes.c_float, _P, _P, _I64, _I64, _I64, ctypes.c_int, _P], ctypes.c_int),
    "bitnet_w2a8_linear_group": (
        [_P, ctypes.c_int, _I64, _I64, ctypes.c_int, _P, _P, _P, _P, _P, _P, _P, _P, _P], ctypes.c_int),
    "bitnet_w2a8_linear_group_ex": (
        [_P, ctypes.c_int, _I64, _I64, ctypes.c_int, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_int, _P, _P, _P],
        ctypes.c_int),
    "bitnet_w2a8_linear": (
        [_P, ctypes.c_int, _I64, _I64, _P, ctypes.c_float, _I64, _P, _P, _P, _P, _P, _P], ctypes.c_int),
    "bitnet_i2s_matmul_workspace_size": ([_I64, _I64, _I64], _I64),
    "bitnet_i2s_matmul_ws": (
        [_P, _P, _P, _P, ctypes.c_float, _P, _P, _I64, _I64, _I64, _P, _I64, _P], ctypes.c_int),
    "bitnet_i2s_matmul_noalloc": ([_P, _P, _P, _P, ctypes.c_float, _P, _P, _I64, _I64, _I64, _P], ctypes.c_int),
    "bitnet_last_device_error": ([], ctypes.c_int),
    "bitnet_selftest_wait_timeout": ([_P, _I64, ctypes.c_int32, _P, _P], ctypes.c_int),
    "bitnet_quant_weight": ([_P, ctypes.c_int, ctypes.c_int, _I64, _I64, _P, _P, _P], ctypes.c_int),
    "bitnet_ffn_act_quant": ([_P, _P, _P, ctypes.c_float, _I64, _I64, _P, _P, _P, _P, _P], ctypes.c_int),
    "bitnet_w2a8_ffn_workspace_size": ([_I64, _I64, _I64], _I64),
    "bitnet_sweep_plan_create": ([_P, ctypes.c_int, ctypes.c_int, _P], ctypes.c_int),
    "bitnet_sweep_plan_run": ([_P, _P], ctypes.c_int),
    "bitnet_sweep_plan_destroy": ([_P], ctypes.c_int),
    "bitnet_kv4_cache_bytes": ([_I64, _I64, _I64], _I64),
    "bitnet_kv4_append": ([_P, _P, _P, _P, ctypes.c_int, _I64, _I64, _P], ctypes.c_int),
    "bitnet_kv4_read": ([_P, _P, _P, _P, ctypes.c_int, _I64, _I64, _P], ctypes.c_int),
    "bitnet_kv4_attention_workspace_size": ([_P, _P, _I64], _I64),
    "bitnet_kv4_attention": (
        [_P, _P, _P, ctypes.c_int, _I64, _I64, ctypes.c_float, _I64, _I64, _P, _I64, _P, _I64, _P], ctypes.c_int),
    "bitnet_kv4_mass_bytes": ([_I64, _I64], _I64),
    "bitnet_kv4_attention_mass_workspace_size": ([_P, _P, _I64, _I64], _I64),
    "bitnet_kv4_attention_mass": (
        [_P, _P, _P, ctypes.c_int, _I64, _I64, ctypes.c_float, _I64, _I64, _I64, ctypes.c_float, _P, _P, _P, _I64, _P],
        ctypes.c_int),
    "bitnet_kv4_evict_workspace_size": ([_P, _P, _I64], _I64),
    "bitnet_kv4_evict": ([_P, _P, _P, _I64, _I64, _I64, _I64, _P, _I64, _P, _P, _I64, _P], ctypes.c_int),
    "bitnet_rope_turns": (
        [_I64, ctypes.c_double, ctypes.c_int, ctypes.c_double, ctypes.c_double, ctypes.c_double, ctypes.c_double, _P, _P],
        ctypes.c_int),
    "bitnet_rope": (
        [_P, _P, _I64, _P, _I64, _I64, _P, _I64, _P, _I64, _I64, _P, _I64, _I64, ctypes.c_int, _P], ctypes.c_int),
    "bitnet_w4_quant_weight": ([_P, ctypes.c_int, _I64, _I64, _I64, _P, _P, _P, _P], ctypes.c_int),
    "bitnet_w4_matmul": ([_P, ctypes.c_int, _I64, _I64, _P, _P, _P, _I64, _I64, _P, _P], ctypes.c_int),
    "bitnet_w2a8_ffn": (
        [_P, ctypes.c_int, _I64, _I64, _I64, _P, ctypes.c_float, _P, ctypes.c_float, _P, ctypes.c_float, _P,
         ctypes.c_float, _P, _P, _P, _P, _P, _P, _P, _I64, _P], ctypes.c_int),
}

_lib = None


class BitnetError(RuntimeError):
    def __init__(self, status: int, where: str):
        msg = lib().bitnet_strerror(status).decode() if _lib is not None else str(status)
        super().__init__("%s failed with status %d: %s" % (where, status, msg))
        self.status = status


def lib_path() -> str:
    return _build.LIB_PATH


def lib():
    """Load the CUDA library (built in-tree by ``_build.build()``); raise if it is absent."""
    global _lib
    if _lib is not None:
        return _lib
    path = lib_path()
    if not os.path.exists(path):
        raise RuntimeError(
            "libbitnet_gb300.so is not built (%s); run ternary_weight_gb300._build.build() "
            "or __graft_entry__.build() first -- there is no CPU fallback" % path)
    l = ctypes.CDLL(path)
    for name, (args, res) in SIGNATURES.items():
        fn = getattr(l, name)
        fn.argtypes = args
        fn.restype = res
    _lib = l
    return l


def _check(status: int, where: str):
    if status != BITNET_OK:
        raise BitnetError(status, where)


def _stream(stream=None):
    import torch

    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _require_cuda(*ts):
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("tensors must be contiguous CUDA tensors")


def pack_i2s(w, out=None, invalid_count=None, stream=None):
    """Ternary int8 weights (N x K, CUDA) -> i2_s packed uint8 (N x K/4)."""
    import torch

    N, K = w.shape
    if out is None:
        out = torch.empty((N, K // 4), dtype=torch.uint8, device=w.device)
    _require_cuda(w, out, invalid_count)
    _check(lib().bitnet_pack_i2s(_ptr(w), _ptr(out), N, K, _ptr(invalid_count), _stream(stream)),
           "bitnet_pack_i2s")
    return out


QUANT_WEIGHT_MODES = {"absmean": 0, "sign": 1}


def quant_weight(w, mode="absmean", out=None, scale=None, stream=None):
    """fp32 or bf16 weights (N x K, CUDA) -> (i2_s packed uint8 N x K/4, fp32 scale tensor of 1)."""
    import torch

    if w.dtype == torch.float32:
        dt = BITNET_F32
    elif w.dtype == torch.bfloat16:
        dt = BITNET_BF16
    else:
        raise ValueError("w must be float32 or bfloat16")
    N, K = w.shape
    out = torch.empty((N, K // 4), dtype=torch.uint8, device=w.device) if out is None else out
    scale = torch.empty(1, dtype=torch.float32, device=w.device) if scale is None else scale
    _require_cuda(w, out, scale)
    _check(lib().bitnet_quant_weight(_ptr(w), dt, QUANT_WEIGHT_MODES[mode], N, K, _ptr(out), _ptr(scale),
                                     _stream(stream)), "bitnet_quant_weight")
    return out, scale


def quant_act(x, xq=None, scale=None, rowsum=None, stream=None):
    """fp32 or bf16 rows (M x K, CUDA) -> (xq int8 M x K, s fp32 M, rowsum int32 M)."""
    import torch

    if x.dtype == torch.float32:
        dt = BITNET_F32
    elif x.dtype == torch.bfloat16:
        dt = BITNET_BF16
    else:
        raise ValueError("x must be float32 or bfloat16")
    M, K = x.shape
    dev = x.device
    xq = torch.empty((M, K), dtype=torch.int8, device=dev) if xq is None else xq
    scale = torch.empty(M, dtype=torch.float32, device=dev) if scale is None else scale
    rowsum = torch.empty(M, dtype=torch.int32, device=dev) if rowsum is None else rowsum
    _require_cuda(x, xq, scale, rowsum)
    _check(lib().bitnet_quant_act(_ptr(x), dt, M, K, _ptr(xq), _ptr(scale), _ptr(rowsum), _stream(stream)),
           "bitnet_quant_act")
    return xq, scale, rowsum


def i2s_matmul(xq, scale, rowsum, wp, w_scale, out=None, acc_out=None, algo="auto", stream=None):
    """W2A8 ternary matmul: returns out (M x N fp32); fills acc_out (M x N int32) if given."""
    import torch

    M, K = xq.shape
    N = wp.shape[0]
    if wp.shape[1] * 4 != K:
        raise ValueError("wp must be N x K/4")
    out = torch.empty((M, N), dtype=torch.float32, device=xq.device) if out is None else out
    _require_cuda(xq, scale, rowsum, wp, out, acc_out)
    _check(lib().bitnet_i2s_matmul_algo(_ptr(xq), _ptr(scale), _ptr(rowsum), _ptr(wp), float(w_scale),
                                        _ptr(out), _ptr(acc_out), M, N, K, ALGO[algo], _stream(stream)),
           "bitnet_i2s_matmul")
    return out


def _act_dtype(x):
    import torch

    if x.dtype == torch.float32:
        return BITNET_F32
    if x.dtype == torch.bfloat16:
        return BITNET_BF16
    raise ValueError("x must be float32 or bfloat16")


def workspace_size(M, N, K) -> int:
    n = lib().bitnet_i2s_matmul_workspace_size(M, N, K)
    if n < 0:
        raise BitnetError(int(n), "bitnet_i2s_matmul_workspace_size")
    return int(n)


def i2s_matmul_ws(xq, scale, rowsum, wp, w_scale, workspace=None, out=None, acc_out=None, stream=None):
    """The prefill path with a device workspace (allocated here from torch if not given)."""
    import torch

    M, K = xq.shape
    N = wp.shape[0]
    if wp.shape[1] * 4 != K:
        raise ValueError("wp must be N x K/4")
    need = workspace_size(M, N, K)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=xq.device)
    out = torch.empty((M, N), dtype=torch.float32, device=xq.device) if out is None else out
    _require_cuda(xq, scale, rowsum, wp, out, acc_out, workspace)
    _check(lib().bitnet_i2s_matmul_ws(_ptr(xq), _ptr(scale), _ptr(rowsum), _ptr(wp), float(w_scale), _ptr(out),
                                      _ptr(acc_out), M, N, K, _ptr(workspace),
                                      workspace.numel() * workspace.element_size(), _stream(stream)),
           "bitnet_i2s_matmul_ws")
    return out


def i2s_matmul_noalloc(xq, scale, rowsum, wp, w_scale, out=None, acc_out=None, stream=None):
    """The prefill matmul without any workspace: for callers that must not allocate device memory.

    The library's own 64 MiB device scratch array stands in for the workspace (problems that
    need more are refused); the output tensor is allocated here only if ``out`` is not given."""
    import torch

    M, K = xq.shape
    N = wp.shape[0]
    if wp.shape[1] * 4 != K:
        raise ValueError("wp must be N x K/4")
    out = torch.empty((M, N), dtype=torch.float32, device=xq.device) if out is None else out
    _require_cuda(xq, scale, rowsum, wp, out, acc_out)
    _check(lib().bitnet_i2s_matmul_noalloc(_ptr(xq), _ptr(scale), _ptr(rowsum), _ptr(wp), float(w_scale), _ptr(out),
                                           _ptr(acc_out), M, N, K, _stream(stream)),
           "bitnet_i2s_matmul_noalloc")
    return out


def linear_group(x, wps, w_scales, outs=None, accs=None, xq=None, scale=None, rowsum=None, prefetch=None,
                 stream=None):
    """Quantise x (M x K fp32/bf16) and multiply it with up to 8 packed projections sharing it.

    One kernel launch when M == 1; xq/scale/rowsum are then optional outputs. ``prefetch`` is
    an optional list of CUDA tensors (e.g. the next group's packed weights) to pull into L2
    while the kernel runs. Returns the list of M x N_l fp32 outputs."""
    import torch

    dt = _act_dtype(x)
    M, K = x.shape
    n = len(wps)
    for w in wps:
        if w.shape[1] * 4 != K:
            raise ValueError("every wp must be N x K/4")
    if outs is None:
        outs = [torch.empty((M, w.shape[0]), dtype=torch.float32, device=x.device) for w in wps]
    _require_cuda(x, xq, scale, rowsum, *wps, *outs, *(accs or []))
    P = ctypes.c_void_p * n
    wp_arr = P(*[w.data_ptr() for w in wps])
    out_arr = P(*[o.data_ptr() for o in outs])
    acc_arr = P(*[(a.data_ptr() if a is not None else None) for a in accs]) if accs is not None else None
    ws_arr = (ctypes.c_float * n)(*[float(v) for v in w_scales])
    n_arr = (ctypes.c_int64 * n)(*[int(w.shape[0]) for w in wps])
    pf = list(prefetch or [])
    pf_ptr = (ctypes.c_void_p * max(1, len(pf)))(*[t.data_ptr() for t in pf])
    pf_bytes = (ctypes.c_int64 * max(1, len(pf)))(*[t.numel() * t.element_size() for t in pf])
    _check(lib().bitnet_w2a8_linear_group_ex(_ptr(x), dt, M, K, n, wp_arr, ws_arr, n_arr, out_arr, acc_arr,
                                             _ptr(xq), _ptr(scale), _ptr(rowsum), len(pf), pf_ptr, pf_bytes,
                                             _stream(stream)),
           "bitnet_w2a8_linear_group")
    return outs


def last_device_error() -> int:
    return lib().bitnet_last_device_error()


def selftest_wait_timeout(src, max_polls, report=None, stream=None):
    """Run the failure-handling self-test: a bounded wait that runs out while a bulk copy of
    ``src`` (a CUDA tensor of 16..16384 bytes) is in flight. Returns the 3-word uint32 report
    (gave up, copy landed, wrapping word sum) as an int32 CUDA tensor."""
    import torch

    report = torch.zeros(3, dtype=torch.int32, device=src.device) if report is None else report
    _require_cuda(src, report)
    _check(lib().bitnet_selftest_wait_timeout(_ptr(src), src.numel() * src.element_size(), int(max_polls),
                                              _ptr(report), _stream(stream)),
           "bitnet_selftest_wait_timeout")
    return report


def linear(x, wp, w_scale, out=None, algo="auto", stream=None):
    """Quantise activation rows and multiply them with packed ternary weights (two launches)."""
    xq, s, rs = quant_act(x, stream=stream)
    return i2s_matmul(xq, s, rs, wp, w_scale, out=out, algo=algo, stream=stream)


def ffn_act_quant(gate, up, gamma, eps, xq=None, scale=None, rowsum=None, inner_out=None, stream=None):
    """FFN inner activation (squared-ReLU gate times up, RMS sub-norm with weight gamma and
    epsilon eps) fused with its per-token quantisation. gate, up: M x F fp32 CUDA tensors;
    gamma: F fp32. Returns (xq int8 M x F, s fp32 M, rowsum int32 M); inner_out (M x F fp32)
    is written when given."""
    import torch

    M, F = gate.shape
    if up.shape != gate.shape or gamma.shape != (F,):
        raise ValueError("gate and up must be M x F, gamma F")
    dev = gate.device
    xq = torch.empty((M, F), dtype=torch.int8, device=dev) if xq is None else xq
    scale = torch.empty(M, dtype=torch.float32, device=dev) if scale is None else scale
    rowsum = torch.empty(M, dtype=torch.int32, device=dev) if rowsum is None else rowsum
    _require_cuda(gate, up, gamma, xq, scale, rowsum, inner_out)
    _check(lib().bitnet_ffn_act_quant(_ptr(gate), _ptr(up), _ptr(gamma), float(eps), M, F, _ptr(xq), _ptr(scale),
                                      _ptr(rowsum), _ptr(inner_out), _stream(stream)),
           "bitnet_ffn_act_quant")
    return xq, scale, rowsum


def ffn_workspace_size(M, K, F) -> int:
    n = lib().bitnet_w2a8_ffn_workspace_size(M, K, F)
    if n < 0:
        raise BitnetError(int(n), "bitnet_w2a8_ffn_workspace_size")
    return int(n)


def w2a8_ffn(x, wp_gate, a_gate, wp_up, a_up, wp_down, a_down, gamma, eps, out=None, gate_out=None, up_out=None,
             xq=None, scale=None, rowsum=None, workspace=None, stream=None):
    """The FFN block: gate/up W2A8 projections of x (M x K fp32/bf16), the squared-ReLU gate
    and RMS sub-norm, then the down W2A8 projection. Returns out (M x K fp32); gate_out and
    up_out (M x F) and, when given, xq/scale/rowsum (the quantised inner rows) are written.
    For M > 1 the workspace buffers are allocated here if not given; ``workspace`` (a uint8
    CUDA tensor of at least ffn_workspace_size bytes) selects the expand-once GEMM path."""
    import torch

    dt = _act_dtype(x)
    M, K = x.shape
    F = wp_gate.shape[0]
    if wp_gate.shape != (F, K // 4) or wp_up.shape != (F, K // 4) or wp_down.shape != (K, F // 4):
        raise ValueError("wp_gate/wp_up must be F x K/4 and wp_down K x F/4")
    dev = x.device
    out = torch.empty((M, K), dtype=torch.float32, device=dev) if out is None else out
    gate_out = torch.empty((M, F), dtype=torch.float32, device=dev) if gate_out is None else gate_out
    up_out = torch.empty((M, F), dtype=torch.float32, device=dev) if up_out is None else up_out
    if M > 1:
        xq = torch.empty((M, max(K, F)), dtype=torch.int8, device=dev) if xq is None else xq
        scale = torch.empty(M, dtype=torch.float32, device=dev) if scale is None else scale
        rowsum = torch.empty(M, dtype=torch.int32, device=dev) if rowsum is None else rowsum
    _require_cuda(x, wp_gate, wp_up, wp_down, gamma, out, gate_out, up_out, xq, scale, rowsum, workspace)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib().bitnet_w2a8_ffn(_ptr(x), dt, M, K, F, _ptr(wp_gate), float(a_gate), _ptr(wp_up), float(a_up),
                                 _ptr(wp_down), float(a_down), _ptr(gamma), float(eps), _ptr(gate_out),
                                 _ptr(up_out), _ptr(out), _ptr(xq), _ptr(scale), _ptr(rowsum), _ptr(workspace),
                                 ws_bytes, _stream(stream)),
           "bitnet_w2a8_ffn")
    return out


class LinearGroupDesc(ctypes.Structure):
    """ctypes mirror of bitnet_linear_group (include/bitnet.h)."""
    _fields_ = [("x", ctypes.c_void_p), ("K", ctypes.c_int64), ("count", ctypes.c_int),
                ("wp", ctypes.c_void_p * 8), ("w_scale", ctypes.c_float * 8), ("N", ctypes.c_int64 * 8),
                ("out", ctypes.c_void_p * 8)]


class SweepPlan:
    """A persistent sweep over independent projection groups (one kernel launch per run).

    ``groups`` is a list of (x, [(wp, w_scale, out), ...]) with x a 1-D fp32 or bf16 CUDA
    tensor of K values, wp an N x K/4 uint8 tensor and out an N-element fp32 tensor. The
    tensors are bound to the plan (it keeps references to them); run() recomputes every
    group's outputs from the current contents of its x."""

    def __init__(self, groups):
        import torch

        if not groups:
            raise ValueError("at least one group")
        dt = None
        descs = (LinearGroupDesc * len(groups))()
        self._keep = []
        for g, (x, projs) in enumerate(groups):
            d = _act_dtype(x.view(1, -1))
            if dt is None:
                dt = d
            elif d != dt:
                raise ValueError("every group's x must have the same dtype")
            if not 1 <= len(projs) <= 8:
                raise ValueError("1..8 projections per group")
            K = x.numel()
            desc = descs[g]
            desc.x, desc.K, desc.count = x.data_ptr(), K, len(projs)
            for l, (wp, w_scale, out) in enumerate(projs):
                if wp.shape[1] * 4 != K or out.numel() != wp.shape[0] or out.dtype != torch.float32:
                    raise ValueError("wp must be N x K/4 and out N fp32")
                desc.wp[l], desc.w_scale[l], desc.N[l], desc.out[l] = wp.data_ptr(), float(w_scale), wp.shape[0], \
                    out.data_ptr()
            _require_cuda(x, *[t for p in projs for t in (p[0], p[2])])
            self._keep.append((x, projs))
        self._handle = ctypes.c_void_p()
        _check(lib().bitnet_sweep_plan_create(ctypes.cast(descs, ctypes.c_void_p), len(groups), dt,
                                              ctypes.byref(self._handle)),
               "bitnet_sweep_plan_create")

    def run(self, stream=None):
        _check(lib().bitnet_sweep_plan_run(self._handle, _stream(stream)), "bitnet_sweep_plan_run")

    def close(self):
        if getattr(self, "_handle", None) and self._handle.value:
            lib().bitnet_sweep_plan_destroy(self._handle)
            self._handle = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


KV4_PAGE = 64


class _KV4CacheDesc(ctypes.Structure):
    """ctypes mirror of bitnet_kv4_cache (include/bitnet.h)."""
    _fields_ = [("pages", ctypes.c_void_p), ("n_pages", ctypes.c_int64), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32)]


class _KV4BatchDesc(ctypes.Structure):
    """ctypes mirror of bitnet_kv4_batch (include/bitnet.h)."""
    _fields_ = [("cu_q", ctypes.c_void_p), ("kv_len", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
                ("batch", ctypes.c_int64), ("max_pages", ctypes.c_int64), ("total_q", ctypes.c_int64),
                ("max_q", ctypes.c_int64), ("max_kv", ctypes.c_int64)]


def kv4_cache_bytes(n_pages, kv_heads, head_dim) -> int:
    n = lib().bitnet_kv4_cache_bytes(n_pages, kv_heads, head_dim)
    if n < 0:
        raise BitnetError(int(n), "bitnet_kv4_cache_bytes")
    return int(n)


class KV4Cache:
    """A pool of pages of the 4-bit key/value cache: n_pages pages of 64 tokens for kv_heads heads
    of head_dim (64 or 128) numbers. ``pages``, a flat uint8 CUDA tensor of kv4_cache_bytes bytes,
    is allocated here (uninitialised; no page needs to be cleared) if not given."""

    def __init__(self, n_pages, kv_heads, head_dim, pages=None, device="cuda"):
        import torch

        need = kv4_cache_bytes(n_pages, kv_heads, head_dim)
        if pages is None:
            pages = torch.empty(need, dtype=torch.uint8, device=device)
        if pages.dtype != torch.uint8 or pages.numel() != need:
            raise ValueError("pages must be %d bytes of uint8" % need)
        _require_cuda(pages)
        self.pages, self.n_pages, self.kv_heads, self.head_dim = pages, n_pages, kv_heads, head_dim
        self.device, self.index = pages.device, pages.get_device()
        self._desc = _KV4CacheDesc(pages.data_ptr(), n_pages, kv_heads, head_dim)
        self._ref = ctypes.c_void_p(ctypes.addressof(self._desc))


class KV4Batch:
    """The sequences of a call: ``cu_q`` (batch + 1), ``kv_len`` (batch) and ``page_table`` (batch x
    max_pages), int32 CUDA tensors that are read when the call runs (so a program may update them
    in place between calls, also between replays of a captured graph), and the sizes that bound
    them: total_q packed rows, at most max_q new and max_kv cached tokens a sequence."""

    def __init__(self, cu_q, kv_len, page_table, total_q, max_q, max_kv=None):
        import torch

        n = kv_len.numel()
        if any(t.dtype != torch.int32 for t in (cu_q, kv_len, page_table)):
            raise ValueError("cu_q, kv_len and page_table must be int32")
        if cu_q.shape != (n + 1,) or kv_len.shape != (n,) or page_table.dim() != 2 or page_table.shape[0] != n:
            raise ValueError("cu_q must have batch + 1 entries, kv_len batch, and page_table batch rows")
        _require_cuda(cu_q, kv_len, page_table)
        self.index = cu_q.get_device()
        if kv_len.get_device() != self.index or page_table.get_device() != self.index:
            raise ValueError("cu_q, kv_len and page_table must be on one device")
        if max_kv is None:
            max_kv = page_table.shape[1] * KV4_PAGE
        self.cu_q, self.kv_len, self.page_table = cu_q, kv_len, page_table
        self.total_q, self.max_q, self.max_kv = int(total_q), int(max_q), int(max_kv)
        self._desc = _KV4BatchDesc(cu_q.data_ptr(), kv_len.data_ptr(), page_table.data_ptr(), n, page_table.shape[1],
                                   self.total_q, self.max_q, self.max_kv)
        self._ref = ctypes.c_void_p(ctypes.addressof(self._desc))
        self._ws = {}  # attention workspace bytes by cache and query heads


# A decode step makes these calls for every layer, and their kernels take a few microseconds: the helpers
# below look everything up once and touch each tensor's properties once.
_kv4_torch = None  # (torch, its dtypes -> BITNET dtypes, torch.bfloat16, stream handle by device index and stream)


def _kv4_setup():
    global _kv4_torch
    import torch

    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if raw is None:
        def raw(index):
            return torch.cuda.current_stream(index).cuda_stream
    current = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device

    def handle(cache, batch, stream):
        """The stream's handle, where the call can run on it: kernels run on the calling thread's current device,
        and would take pointers to another one as they are."""
        index = cache.index
        if batch.index != index:
            raise ValueError("the batch must be on the cache's device")
        if current() != index:
            raise ValueError("the cache's device must be the current one")
        return raw(index) if stream is None else stream.cuda_stream

    _kv4_torch = torch, {torch.float32: BITNET_F32, torch.bfloat16: BITNET_BF16}, torch.bfloat16, handle
    return _kv4_torch


_on_device = None  # (torch, its dtypes -> BITNET dtypes, stream handle by device index and stream)


def _on_device_setup():
    global _on_device
    import torch

    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if raw is None:
        def raw(index):
            return torch.cuda.current_stream(index).cuda_stream
    current = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device

    def handle(index, stream):
        """The stream's handle, where tensors on device `index` can be used on it."""
        if current() != index:
            raise ValueError("the tensors' device must be the current one")
        return raw(index) if stream is None else stream.cuda_stream

    _on_device = torch, {torch.float32: BITNET_F32, torch.bfloat16: BITNET_BF16}, handle
    return _on_device


def _kv4_rows(t, rows, heads, dim, index):
    """Checks a rows x heads x dim tensor on device `index` whose heads lie one after another; its row stride."""
    if t.shape != (rows, heads, dim):
        raise ValueError("expected a %d x %d x %d tensor" % (rows, heads, dim))
    s = t.stride()
    if t.get_device() != index:
        raise ValueError("rows must be CUDA tensors on the cache's device")
    if rows and (s[2] != 1 or (heads > 1 and s[1] != dim)):
        raise ValueError("rows must be CUDA tensors whose heads lie one after another")
    return s[0] if rows > 1 else heads * dim


def _kv4_empty(torch, shape, dtype, device, stream):
    """An output of a call on `stream` belongs to that stream."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def kv4_append(cache, batch, k, v, stream=None):
    """Quantise the batch's keys and values (total_q x kv_heads x head_dim, fp32 or bf16 CUDA; rows may
    be strided, e.g. slices of a fused q/k/v row) to 4 bits and write them to their places."""
    _, dtypes, _, handle = _kv4_torch or _kv4_setup()
    dt = dtypes.get(k.dtype)
    if dt is None or v.dtype != k.dtype:
        raise ValueError("k and v must both be float32 or bfloat16")
    rows, heads, dim = batch.total_q, cache.kv_heads, cache.head_dim
    ks, vs = _kv4_rows(k, rows, heads, dim, cache.index), _kv4_rows(v, rows, heads, dim, cache.index)
    on = handle(cache, batch, stream)
    if rows:
        st = lib().bitnet_kv4_append(cache._ref, batch._ref, k.data_ptr(), v.data_ptr(), dt, ks, vs, on)
        if st:
            raise BitnetError(st, "bitnet_kv4_append")


def kv4_read(cache, batch, dtype=None, k=None, v=None, stream=None):
    """Read the batch's tokens back from the cache as (k, v), each total_q x kv_heads x head_dim of
    ``dtype`` (fp32 or bf16, default bf16; or that of the given k and v, which are written)."""
    torch, dtypes, bf16, handle = _kv4_torch or _kv4_setup()
    rows, heads, dim = batch.total_q, cache.kv_heads, cache.head_dim
    on = handle(cache, batch, stream)
    ks = vs = heads * dim
    if k is None or v is None:
        given = k if k is not None else v
        if dtype is None:
            dtype = bf16 if given is None else given.dtype
    if k is None:
        k = _kv4_empty(torch, (rows, heads, dim), dtype, cache.device, stream)
    else:
        ks = _kv4_rows(k, rows, heads, dim, cache.index)
    if v is None:
        v = _kv4_empty(torch, (rows, heads, dim), dtype, cache.device, stream)
    else:
        vs = _kv4_rows(v, rows, heads, dim, cache.index)
    dt = dtypes.get(k.dtype)
    if dt is None or v.dtype != k.dtype or (dtype is not None and dtype != k.dtype):
        raise ValueError("k and v must both be float32 or bfloat16, as asked for")
    if rows:
        st = lib().bitnet_kv4_read(cache._ref, batch._ref, k.data_ptr(), v.data_ptr(), dt, ks, vs, on)
        if st:
            raise BitnetError(st, "bitnet_kv4_read")
    return k, v


def kv4_attention_workspace_size(cache, batch, q_heads) -> int:
    n = lib().bitnet_kv4_attention_workspace_size(cache._ref, batch._ref, q_heads)
    if n < 0:
        raise BitnetError(int(n), "bitnet_kv4_attention_workspace_size")
    return int(n)


def kv4_attention(cache, batch, q, scale, window=0, sinks=0, out=None, workspace=None, stream=None):
    """Causal attention of the batch's queries (total_q x q_heads x head_dim, fp32 or bf16 CUDA, rows may
    be strided) over the cache: a query at position p sees position j where j <= p and (window == 0
    or j > p - window or j < sinks). Returns total_q x q_heads x head_dim bf16 (``out`` if given).
    ``workspace``: a uint8 CUDA tensor of at least kv4_attention_workspace_size bytes, allocated
    here if not given."""
    torch, dtypes, bf16, handle = _kv4_torch or _kv4_setup()
    dt = dtypes.get(q.dtype)
    if dt is None or q.dim() != 3:
        raise ValueError("q must be total_q x q_heads x head_dim, float32 or bfloat16")
    rows, heads, dim = batch.total_q, q.shape[1], cache.head_dim
    qs = _kv4_rows(q, rows, heads, dim, cache.index)
    on = handle(cache, batch, stream)
    key = (heads, cache.kv_heads, dim)
    need = batch._ws.get(key)
    if need is None:
        need = batch._ws[key] = kv4_attention_workspace_size(cache, batch, heads)
    if out is None:
        out, os_ = _kv4_empty(torch, (rows, heads, dim), bf16, cache.device, stream), heads * dim
    elif out.dtype != bf16:
        raise ValueError("out must be bfloat16")
    else:
        os_ = _kv4_rows(out, rows, heads, dim, cache.index)
    ws_ptr, ws_bytes = None, 0
    if workspace is not None:
        _require_cuda(workspace)
        if workspace.get_device() != cache.index:
            raise ValueError("the workspace must be on the cache's device")
        ws_ptr, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    elif need:
        workspace, ws_bytes = _kv4_empty(torch, need, torch.uint8, cache.device, stream), need
        ws_ptr = workspace.data_ptr()
    if rows:
        st = lib().bitnet_kv4_attention(cache._ref, batch._ref, q.data_ptr(), dt, heads, qs, scale, window, sinks,
                                        out.data_ptr(), os_, ws_ptr, ws_bytes, on)
        if st:
            raise BitnetError(st, "bitnet_kv4_attention")
    return out


def kv4_mass(cache):
    """Room for the attention weight that a cache's tokens gather: fp32, n_pages x kv_heads x 64, zeros."""
    import torch

    return torch.zeros((cache.n_pages, cache.kv_heads, KV4_PAGE), dtype=torch.float32, device=cache.device)


def _kv4_mass_rows(cache, mass):
    if mass.shape != (cache.n_pages, cache.kv_heads, KV4_PAGE) or mass.dtype != _kv4_torch[0].float32:
        raise ValueError("mass must be n_pages x kv_heads x %d float32" % KV4_PAGE)
    if mass.get_device() != cache.index or not mass.is_contiguous():
        raise ValueError("mass must be contiguous, on the cache's device")


def _kv4_workspace(torch, cache, workspace, need, stream):
    """A call's workspace: the given one (checked), or one allocated for the call's stream. (tensor, pointer, bytes)"""
    if workspace is None:
        workspace = _kv4_empty(torch, need, torch.uint8, cache.device, stream) if need else None
        return workspace, workspace.data_ptr() if need else None, need
    _require_cuda(workspace)
    if workspace.get_device() != cache.index:
        raise ValueError("the workspace must be on the cache's device")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def kv4_attention_mass_workspace_size(cache, batch, q_heads, voters=0) -> int:
    n = lib().bitnet_kv4_attention_mass_workspace_size(cache._ref, batch._ref, q_heads, voters)
    if n < 0:
        raise BitnetError(int(n), "bitnet_kv4_attention_mass_workspace_size")
    return int(n)


def kv4_attention_mass(cache, batch, q, scale, mass, decay=1.0, window=0, sinks=0, voters=0, out=None, workspace=None,
                       stream=None):
    """Add the softmax weights of the batch's queries (as in ``kv4_attention``) to the mass of the cached
    tokens that they see: decay * mass + votes for tokens older than the call, the votes alone for the call's
    own. The last ``voters`` rows of each sequence vote (0: all). ``mass`` (see ``kv4_mass``) is updated in
    place, or ``out`` (which keeps what the call does not write) is; returns it. ``workspace``: a uint8 CUDA
    tensor of at least kv4_attention_mass_workspace_size bytes, allocated here if not given."""
    torch, dtypes, _, handle = _kv4_torch or _kv4_setup()
    dt = dtypes.get(q.dtype)
    if dt is None or q.dim() != 3:
        raise ValueError("q must be total_q x q_heads x head_dim, float32 or bfloat16")
    rows, heads = batch.total_q, q.shape[1]
    qs = _kv4_rows(q, rows, heads, cache.head_dim, cache.index)
    on = handle(cache, batch, stream)
    _kv4_mass_rows(cache, mass)
    if out is None:
        out = mass
    else:
        _kv4_mass_rows(cache, out)
    key = (heads, cache.kv_heads, cache.head_dim, voters)
    need = batch._ws.get(key)
    if need is None:
        need = batch._ws[key] = kv4_attention_mass_workspace_size(cache, batch, heads, voters)
    if rows:
        keep, ws, ws_bytes = _kv4_workspace(torch, cache, workspace, need, stream)
        st = lib().bitnet_kv4_attention_mass(cache._ref, batch._ref, q.data_ptr(), dt, heads, qs, scale, window, sinks, voters,
                                             decay, mass.data_ptr(), out.data_ptr(), ws, ws_bytes, on)
        if st:
            raise BitnetError(st, "bitnet_kv4_attention_mass")
    return out


def kv4_evict_workspace_size(cache, batch, budget) -> int:
    n = lib().bitnet_kv4_evict_workspace_size(cache._ref, batch._ref, budget)
    if n < 0:
        raise BitnetError(int(n), "bitnet_kv4_evict_workspace_size")
    return int(n)


def kv4_evict(cache, batch, mass, budget, limit=None, sinks=0, recent=0, into=None, new_len=None, workspace=None,
              stream=None):
    """Cut the batch's sequences of more than ``limit`` cached tokens (default: budget) to ``budget`` in each
    head: the first ``sinks``, the last ``recent``, and the others of the greatest mass. In place, or into the
    pages of the table ``into`` (int32, batch x pages; then all kept tokens are written there, also those of shorter
    sequences). Returns the new lengths, int32: a new tensor, or ``new_len``, which may be the batch's
    kv_len itself. The batch's cu_q and sizes of new tokens are not used."""
    torch, _, _, handle = _kv4_torch or _kv4_setup()
    limit = budget if limit is None else limit
    n = batch.kv_len.numel()
    on = handle(cache, batch, stream)
    _kv4_mass_rows(cache, mass)
    index = cache.index
    for t, shape in ((into, (n, into.shape[-1]) if into is not None else None), (new_len, (n,))):
        if t is not None and (t.dtype != torch.int32 or t.shape != shape or t.get_device() != index or
                              not t.is_contiguous()):
            raise ValueError("into (batch x pages) and new_len (batch) must be contiguous int32 on the cache's device")
    if new_len is None:
        new_len = _kv4_empty(torch, (n,), torch.int32, cache.device, stream)
    key = ("evict", cache.kv_heads, cache.head_dim, budget)
    need = batch._ws.get(key)
    if need is None:
        need = batch._ws[key] = kv4_evict_workspace_size(cache, batch, budget)
    keep, ws, ws_bytes = _kv4_workspace(torch, cache, workspace, need, stream)
    st = lib().bitnet_kv4_evict(cache._ref, batch._ref, mass.data_ptr(), budget, limit, sinks, recent,
                                into.data_ptr() if into is not None else None, into.shape[1] if into is not None else 0,
                                new_len.data_ptr(), ws, ws_bytes, on)
    if st:
        raise BitnetError(st, "bitnet_kv4_evict")
    return new_len


ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "by_parts": 3, "by_wavelength": 4}
_ROPE_ENDS = {"by_parts": (1.0, 32.0), "by_wavelength": (1.0, 4.0)}


class _RopeDesc(ctypes.Structure):
    """ctypes mirror of bitnet_rope_table (include/bitnet.h)."""
    _fields_ = [("turns", ctypes.c_void_p), ("dims", ctypes.c_int32), ("layout", ctypes.c_int32),
                ("magnitude", ctypes.c_float)]


def rope_turns(dims, base=10000.0, scaling="none", factor=1.0, original=0, low=None, high=None):
    """The frequencies of rotary positions as 64-bit fractions of a turn a position (a list of dims / 2
    integers), and the magnitude. ``scaling``: "none", "linear", "ntk", "by_parts" or "by_wavelength", by
    ``factor``; the last two also take the ``original`` context length and the rotations over it, ``low``
    and ``high``, between which they pass over (1 and 32, 1 and 4 if not given)."""
    if scaling not in ROPE_SCALINGS:
        raise ValueError("scaling must be one of %s" % ", ".join(ROPE_SCALINGS))
    ends = _ROPE_ENDS.get(scaling, (0.0, 0.0))
    turns, magnitude = (ctypes.c_uint64 * max(1, int(dims) // 2))(), ctypes.c_float()
    _check(lib().bitnet_rope_turns(int(dims), float(base), ROPE_SCALINGS[scaling], float(factor), float(original),
                                   float(ends[0] if low is None else low), float(ends[1] if high is None else high),
                                   ctypes.cast(turns, ctypes.c_void_p), ctypes.byref(magnitude)), "bitnet_rope_turns")
    return list(turns), magnitude.value


class Rope:
    """A model's rotary positions: the frequencies (see ``rope_turns``) on the device, and the layout of
    the pairs, "half" or "interleaved". ``dims`` (a multiple of 8) is the part of each head that is turned."""

    def __init__(self, dims, base=10000.0, layout="half", scaling="none", factor=1.0, original=0, low=None, high=None,
                 device="cuda"):
        import torch

        if layout not in ROPE_LAYOUTS:
            raise ValueError("layout must be one of %s" % ", ".join(ROPE_LAYOUTS))
        if dims < 8 or dims % 8:
            raise ValueError("dims must be a multiple of 8")
        turns, self.magnitude = rope_turns(dims, base, scaling, factor, original, low, high)
        self.turns = torch.tensor(turns, dtype=torch.int64, device=device)  # all below 2^62
        self.dims, self.layout, self.index = dims, layout, self.turns.get_device()
        self._desc = _RopeDesc(self.turns.data_ptr(), dims, ROPE_LAYOUTS[layout], self.magnitude)
        self._ref = ctypes.c_void_p(ctypes.addressof(self._desc))


def rope(table, positions, q, k=None, q_out=None, k_out=None, stream=None):
    """Turn queries (rows x q_heads x head_dim, fp32 or bf16 CUDA, rows may be strided) and, if given,
    keys (rows x kv_heads x head_dim) by the positions (rows, int32) of their rows, in one launch. Returns
    the turned q, or (q, k): new tensors, or ``q_out`` and ``k_out``, which may be the inputs themselves."""
    torch, dtypes, handle = _on_device or _on_device_setup()
    dtype, shape, index = q.dtype, q.shape, table.index
    dt = dtypes.get(dtype)
    if dt is None or len(shape) != 3:
        raise ValueError("q must be rows x q_heads x head_dim, float32 or bfloat16")
    rows, qh, dim = shape
    if positions.dtype != torch.int32 or positions.shape != (rows,) or positions.get_device() != index or \
            not positions.is_contiguous():
        raise ValueError("positions must be an int32 for each row, contiguous, on the table's device")
    on = handle(index, stream)
    qs = qos = _kv4_rows(q, rows, qh, dim, index)
    if q_out is None:
        q_out, qos = _kv4_empty(torch, shape, dtype, q.device, stream), qh * dim
    elif q_out is not q:
        if q_out.dtype != dtype:
            raise ValueError("an output must have its input's dtype")
        qos = _kv4_rows(q_out, rows, qh, dim, index)
    kh = ks = kos = 0
    k_in = k_to = None
    if k is not None:
        shape = k.shape
        if k.dtype != dtype or len(shape) != 3:
            raise ValueError("k must be rows x kv_heads x head_dim of q's dtype")
        kh = shape[1]
        ks = kos = _kv4_rows(k, rows, kh, dim, index)
        if k_out is None:
            k_out, kos = _kv4_empty(torch, shape, dtype, k.device, stream), kh * dim
        elif k_out is not k:
            if k_out.dtype != dtype:
                raise ValueError("an output must have its input's dtype")
            kos = _kv4_rows(k_out, rows, kh, dim, index)
        k_in, k_to = k.data_ptr(), k_out.data_ptr()
    elif k_out is not None:
        raise ValueError("k_out without k")
    if rows:
        st = lib().bitnet_rope(table._ref, positions.data_ptr(), rows, q.data_ptr(), qh, qs, q_out.data_ptr(), qos, k_in, kh, ks, k_to,
                               kos, dim, dt, on)
        if st:
            raise BitnetError(st, "bitnet_rope")
    return q_out if k is None else (q_out, k_out)


def w4_quant_weight(w, group=128, with_zeros=False, codes=None, scales=None, zeros=None, stream=None):
    """fp32 or bf16 weights (N x K, CUDA) to 4 bits with an fp16 scale, and with ``with_zeros`` a zero point, for
    each ``group`` (32, 64 or 128) along K. Returns (codes uint8 N x K/2, scales fp16 N x K/group, zeros
    uint8 N x K/group or None)."""
    import torch

    dt = _act_dtype(w)
    N, K = w.shape
    if group not in (32, 64, 128) or K % 128:
        raise ValueError("group must be 32, 64 or 128, and K a multiple of 128")
    with_zeros = with_zeros or zeros is not None
    groups = (N, K // group)
    codes = _kv4_empty(torch, (N, K // 2), torch.uint8, w.device, stream) if codes is None else codes
    scales = _kv4_empty(torch, groups, torch.float16, w.device, stream) if scales is None else scales
    if with_zeros and zeros is None:
        zeros = _kv4_empty(torch, groups, torch.uint8, w.device, stream)
    if tuple(scales.shape) != groups:
        raise ValueError("scales must be N x K/group float16")
    on = (_on_device or _on_device_setup())[2](_w4_check(w, codes, scales, zeros, None)[5], stream)
    _check(lib().bitnet_w4_quant_weight(_ptr(w), dt, N, K, group, _ptr(codes), _ptr(scales), _ptr(zeros), on), "bitnet_w4_quant_weight")
    return codes, scales, zeros


def _w4_check(x, codes, scales, zeros, out):
    """Checks of what both calls have; (torch, rows, N, K, group, index)."""
    torch = (_on_device or _on_device_setup())[0]
    (N, half), (n, groups), (M, K) = codes.shape, scales.shape, x.shape
    if codes.dtype != torch.uint8 or scales.dtype != torch.float16 or n != N or groups == 0 or 2 * half % groups:
        raise ValueError("codes must be N x K/2 uint8 and scales N x K/group float16")
    if zeros is not None and (zeros.dtype != torch.uint8 or zeros.shape != (n, groups)):
        raise ValueError("zeros must be uint8 of the scales' shape")
    if K != 2 * half:
        raise ValueError("expected rows of %d numbers" % (2 * half))
    if out is not None and (out.dtype != torch.float32 or out.shape != (M, N)):
        raise ValueError("out must be M x N float32")
    index = x.get_device()
    for t in (x, codes, scales, zeros, out):
        if t is not None and (t.get_device() != index or index < 0 or not t.is_contiguous()):
            raise ValueError("tensors must be contiguous, on one CUDA device")
    return torch, M, N, K, K // groups, index


def w4_matmul(x, codes, scales, zeros=None, out=None, stream=None):
    """x (M x K fp32 or bf16 CUDA) times 4-bit weights with group scales (see ``w4_quant_weight``): M x N fp32."""
    _, dtypes, handle = _on_device or _on_device_setup()
    dt = dtypes.get(x.dtype)
    if dt is None or x.dim() != 2 or codes.dim() != 2 or scales.dim() != 2:
        raise ValueError("x must be M x K float32 or bfloat16, codes N x K/2, scales N x K/group")
    torch, M, N, K, group, index = _w4_check(x, codes, scales, zeros, out)
    on = handle(index, stream)
    if out is None:
        out = _kv4_empty(torch, (M, N), torch.float32, x.device, stream)
    if M:
        st = lib().bitnet_w4_matmul(x.data_ptr(), dt, M, K, codes.data_ptr(), scales.data_ptr(), zeros.data_ptr() if zeros is not None else None,
                                    N, group, out.data_ptr(), on)
        if st:
            raise BitnetError(st, "bitnet_w4_matmul")
    return out
