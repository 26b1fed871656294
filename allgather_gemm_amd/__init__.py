"""Python binding of libaggemm (include/aggemm.h): chunked AllGather fused with a bf16 GEMM, TGATHER,
and a language model's operators around the gathered product (products, norms and updates), on one MI355X.

Argument marshalling only: every step of the path runs in the library's gfx950 kernels.  Tensors
are torch CUDA (HIP) tensors; the library is given their device pointers and the current stream.
Autograd records none of the calls: what they return has no gradient function, whatever its inputs
require; gradients come from the ..._bwd calls (or a torch.autograd.Function of the caller's around
both).
The library must have been built (``python allgather_gemm_amd/build.py`` or
``__graft_entry__.build()``); there is no fallback implementation.
"""
from __future__ import annotations

import ctypes
import functools
import os
import re

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libaggemm.so")
HEADER_PATH = os.path.join(os.path.dirname(_HERE), "include", "aggemm.h")

AG_OK, AG_EINVAL, AG_ENOMEM, AG_EHIP, AG_ETIMEOUT, AG_EUNSUPPORTED = 0, -1, -2, -3, -4, -5
MODE_FUSED, MODE_UNFUSED, MODE_GEMM_ONLY, MODE_PLAIN_GEMM = 0, 1, 2, 3
_MODES = {"fused": MODE_FUSED, "unfused": MODE_UNFUSED, "gemm_only": MODE_GEMM_ONLY,
          "plain_gemm": MODE_PLAIN_GEMM}
PRODUCER_SIDE_STREAM, PRODUCER_IN_KERNEL, PRODUCER_COPY_ENGINE = 0, 1, 2
OUT_BF16, OUT_FP8_E4M3 = 0, 1
IN_BF16, IN_FP8_E4M3 = 0, 1
_OUT = {"bf16": (OUT_BF16, torch.bfloat16), "fp8_e4m3": (OUT_FP8_E4M3, torch.float8_e4m3fn)}
_IN = {"bf16": (IN_BF16, (torch.bfloat16,)), "fp8_e4m3": (IN_FP8_E4M3, (torch.float8_e4m3fn, torch.uint8))}
_PRODUCERS = {"in_kernel": PRODUCER_IN_KERNEL, "side_stream": PRODUCER_SIDE_STREAM,
              "copy_engine": PRODUCER_COPY_ENGINE}

_i32, _i64, _vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p


class AgOptions(ctypes.Structure):
    _fields_ = [("mode", _i32), ("local_rank", _i32), ("a_out", _vp), ("timeout_us", _i64),
                ("reverse_order", _i32), ("skip_producer", _i32), ("producer", _i32),
                ("gemm_events", _vp * 2), ("out_dtype", _i32), ("out_scale", ctypes.c_float),
                ("wait_stats", _vp), ("in_dtype", _i32)]


class AgError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        msg = "%s failed: %s (%d)" % (what, status_str(code), code)
        if code == AG_EHIP:
            msg += ": " + lib().ag_last_error().decode(errors="replace")
        super().__init__(msg)


_lib = None


def lib() -> ctypes.CDLL:
    """Loads libaggemm.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libaggemm.so is not built; run allgather_gemm_amd/build.py")
        L = ctypes.CDLL(LIB_PATH)
        gemm_args = [_vp, _i32, _i64, _i64, _vp, _i64, _vp, _i64, _vp]
        for name in ("ag_gemm", "ag_gemm_unfused"):
            getattr(L, name).argtypes = gemm_args
            getattr(L, name).restype = ctypes.c_int
        L.ag_gemm_ex.argtypes = gemm_args + [ctypes.POINTER(AgOptions)]
        L.ag_gemm_ex.restype = ctypes.c_int
        L.gemm_rs.argtypes = [_vp, _vp, _i32, _i32, _i64, _i64, _i64, _vp, _vp, _vp, _i32, _vp]
        L.gemm_rs.restype = ctypes.c_int
        L.ag_gemm_noalloc.argtypes = [_vp, _i32, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _i32, _vp]
        L.ag_gemm_noalloc.restype = ctypes.c_int
        L.tgather.argtypes = [_vp, _i32, _vp, _i64, _i64, _i64, _i64, _i64, _i64, _i64, _i32, _vp]
        L.tgather.restype = ctypes.c_int
        L.tgather_ex.argtypes = [_vp, _i32, _vp, _i64, _i64, _i64, _i64, _i64, _i64, _i64, _i64,
                                 _i32, _i32, _vp]
        L.tgather_ex.restype = ctypes.c_int
        for name, n in (("gemm_bias_act_workspace", 3), ("gemm_xent_workspace", 3), ("gemm_xent_bwd_workspace", 3)):
            getattr(L, name).argtypes = [_i64] * n
            getattr(L, name).restype = _i64
        L.gemm_bias_act_bwd_workspace.argtypes = [_i64, _i64, _i64, _i32]
        L.gemm_bias_act_bwd_workspace.restype = _i64
        L.gemm_bias_act.argtypes = [_vp] * 4 + [_i64] * 3 + [_i32, _vp, _vp, _vp, _i64, _vp]
        L.gemm_bias_act_bwd.argtypes = [_vp] * 4 + [_i64] * 3 + [_i32] + [_vp] * 4 + [_i64, _vp]
        L.gemm_grouped.argtypes = [_vp] * 3 + [_i32] + [_i64] * 3 + [_vp, _vp]
        L.gemm_grouped_bwd.argtypes = [_vp] * 4 + [_i32] + [_i64] * 3 + [_vp, _vp, _vp]
        L.gemm_xent.argtypes = [_vp] * 3 + [_i64] * 3 + [_vp] * 3 + [_i64, _vp]
        L.gemm_xent_bwd.argtypes = [_vp] * 5 + [_i64] * 3 + [_vp] * 3 + [_i64, _vp]
        L.layer_norm.argtypes = [_vp] * 4 + [_i64] * 2 + [ctypes.c_float] + [_vp] * 5
        L.layer_norm_bwd_workspace.argtypes = [_i64] * 2
        L.layer_norm_bwd_workspace.restype = _i64
        L.layer_norm_bwd.argtypes = [_vp] * 6 + [_i64] * 2 + [_vp] * 4 + [_i64, _vp]
        L.newton_schulz_workspace.argtypes = [_i64] * 3
        L.newton_schulz_workspace.restype = _i64
        L.newton_schulz.argtypes = [_vp, _i32] + [_i64] * 3 + [_vp, _i32, ctypes.c_float, _vp, _vp, _i64, _vp]
        for name in ("gemm_bias_act", "gemm_bias_act_bwd", "gemm_grouped", "gemm_grouped_bwd", "gemm_xent",
                     "gemm_xent_bwd", "layer_norm", "layer_norm_bwd", "newton_schulz"):
            getattr(L, name).restype = ctypes.c_int
        L.ag_check.argtypes = [_vp, ctypes.POINTER(_i64)]
        L.ag_check.restype = ctypes.c_int
        L.ag_status_str.argtypes = [ctypes.c_int]
        L.ag_status_str.restype = ctypes.c_char_p
        L.ag_last_error.argtypes = []
        L.ag_last_error.restype = ctypes.c_char_p
        L.ag_finalize.argtypes = []
        L.ag_finalize.restype = None
        _lib = L
    return _lib


def declared_functions() -> list[str]:
    """Names of the functions include/aggemm.h declares (used to check the exports)."""
    text = open(HEADER_PATH, encoding="utf-8").read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"^\s*(?:const\s+)?\w+\s*\*?\s*(\w+)\s*\(", text, flags=re.M)))


def status_str(code: int) -> str:
    return lib().ag_status_str(code).decode()


def _stream_ptr(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream)


def _ptrs(tensors) -> ctypes.Array:
    return (_vp * len(tensors))(*[t.data_ptr() for t in tensors])


def _check_dev(t: torch.Tensor, name: str):
    if not t.is_cuda:
        raise ValueError("%s must be a device tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def ag_gemm(shards, B: torch.Tensor, comm_block_rows: int, C: torch.Tensor | None = None,
            mode: str = "fused", local_rank: int = 0, a_out: torch.Tensor | None = None,
            timeout_us: int = 0, reverse_order: bool = False, skip_producer: bool = False,
            producer: str = "side_stream", gemm_events=None, stream=None, out_dtype: str = "bf16",
            out_scale: float = 1.0, wait_stats: torch.Tensor | None = None,
            in_dtype: str = "bf16") -> torch.Tensor:
    """C (M, Nc) = concat(shards) @ B^T.  shards: N tensors (H, K); B: (Nc, K), both bf16, or with
    in_dtype="fp8_e4m3" both FP8 E4M3 "fn" (torch.float8_e4m3fn or their uint8 codes; K % 16 == 0),
    when C = out_scale * (A B^T) (out_scale folds the inputs' per-tensor scales).

    mode: "fused" | "unfused" | "gemm_only" | "plain_gemm"; producer (fused only): "side_stream" |
    "in_kernel" | "copy_engine".  out_dtype: "bf16" or "fp8_e4m3" (C = e4m3fn(sum * out_scale), a
    torch.float8_e4m3fn tensor).  gemm_events: optional (start, end) torch.cuda.Event pair that the
    library records around the GEMM kernel's launch.  wait_stats: optional int64 device tensor of 4
    counters the GEMM adds to (flag-wait ticks at 100 MHz summed over workgroups, waits, pieces
    copied while waiting, tiles that skipped their wait).  The call is asynchronous on `stream`; check()
    reports a wait that gave up."""
    shards = list(shards)
    N = len(shards)
    if N == 0:
        raise ValueError("need at least one shard")
    H, K = shards[0].shape
    M = N * H
    Nc = B.shape[0]
    in_code, in_types = _IN[in_dtype]
    for i, s in enumerate(shards):
        _check_dev(s, "shard %d" % i)
        if s.dtype not in in_types or tuple(s.shape) != (H, K):
            raise ValueError("shards must all be (H, K) %s" % in_dtype)
    _check_dev(B, "B")
    if B.dtype not in in_types or B.shape[1] != K:
        raise ValueError("B must be (Nc, K) %s" % in_dtype)
    out_code, out_torch = _OUT[out_dtype]
    if C is None:
        C = torch.empty((M, Nc), dtype=out_torch, device=B.device)
    _check_dev(C, "C")
    if C.dtype != out_torch or tuple(C.shape) != (M, Nc):
        raise ValueError("C must be (M, Nc) %s" % out_torch)
    ev = (_vp * 2)(*(int(e.event_id) for e in gemm_events)) if gemm_events else (_vp * 2)(None, None)
    opt = AgOptions(_MODES[mode], local_rank, a_out.data_ptr() if a_out is not None else None,
                    timeout_us, int(reverse_order), int(skip_producer), _PRODUCERS[producer], ev,
                    out_code, float(out_scale), None, in_code)
    if wait_stats is not None:
        _check_dev(wait_stats, "wait_stats")
        if wait_stats.dtype != torch.int64 or wait_stats.numel() < 4:
            raise ValueError("wait_stats must be an int64 device tensor of 4 counters")
        opt.wait_stats = wait_stats.data_ptr()
    if a_out is not None:
        _check_dev(a_out, "a_out")
        if a_out.dtype not in in_types or tuple(a_out.shape) != (M, K):
            raise ValueError("a_out must be (M, K) %s" % in_dtype)
    rc = lib().ag_gemm_ex(ctypes.cast(_ptrs(shards), _vp), N, M, K, B.data_ptr(), Nc,
                          C.data_ptr(), comm_block_rows, _stream_ptr(stream), ctypes.byref(opt))
    if rc != AG_OK:
        raise AgError(rc, "ag_gemm_ex")
    return C


def ag_gemm_noalloc(shards, B: torch.Tensor, comm_block_rows: int, C: torch.Tensor, a_out: torch.Tensor,
                    local_rank: int = 0, stream=None) -> torch.Tensor:
    """ag_gemm for callers that cannot allocate: C and a_out are the caller's; the library's control
    words are a fixed array per GPU (calls that overlap on one GPU race)."""
    shards = list(shards)
    N = len(shards)
    if N == 0:
        raise ValueError("need at least one shard")
    H, K = shards[0].shape
    M, Nc = N * H, B.shape[0]
    for i, s in enumerate(shards):
        _check_dev(s, "shard %d" % i)
        if s.dtype != torch.bfloat16 or tuple(s.shape) != (H, K):
            raise ValueError("shards must all be (H, K) bfloat16")
    for t, name, shape in ((B, "B", (Nc, K)), (C, "C", (M, Nc)), (a_out, "a_out", (M, K))):
        _check_dev(t, name)
        if t.dtype != torch.bfloat16 or tuple(t.shape) != shape:
            raise ValueError("%s must be %s bfloat16" % (name, shape))
    rc = lib().ag_gemm_noalloc(ctypes.cast(_ptrs(shards), _vp), N, M, K, B.data_ptr(), Nc, C.data_ptr(),
                               comm_block_rows, a_out.data_ptr(), local_rank, _stream_ptr(stream))
    if rc != AG_OK:
        raise AgError(rc, "ag_gemm_noalloc")
    return C


RS_FUSED, RS_UNFUSED = 0, 1


def gemm_rs(A: torch.Tensor, B: torch.Tensor, recv, local_rank: int, P: torch.Tensor | None = None,
            out: torch.Tensor | None = None, fused: bool = True, stream=None):
    """One rank's GEMM + ReduceScatter.  A (M, K), B (Nc, K) bf16: this rank's K slices; recv: N
    tensors (H, Nc) bf16, H = M / N, the other ranks' partials for this rank's rows (recv[local_rank]
    may be None).  Returns (P, out): P (M, Nc) = A B^T, out (H, Nc) = the reduction of this rank's
    row block over the N partials."""
    recv = list(recv)
    N = len(recv)
    M, K = A.shape
    Nc = B.shape[0]
    if N == 0 or M % N != 0:
        raise ValueError("need N >= 1 partials and M % N == 0")
    H = M // N
    for t, name in ((A, "A"), (B, "B")):
        _check_dev(t, name)
        if t.dtype != torch.bfloat16:
            raise ValueError("%s must be bfloat16" % name)
    if B.shape[1] != K:
        raise ValueError("B must be (Nc, K)")
    for j, t in enumerate(recv):
        if j == local_rank:
            continue
        _check_dev(t, "recv[%d]" % j)
        if t.dtype != torch.bfloat16 or tuple(t.shape) != (H, Nc):
            raise ValueError("recv[%d] must be (H, Nc) bfloat16" % j)
    if P is None:
        P = torch.empty((M, Nc), dtype=torch.bfloat16, device=A.device)
    if out is None:
        out = torch.empty((H, Nc), dtype=torch.bfloat16, device=A.device)
    for t, name, shape in ((P, "P", (M, Nc)), (out, "out", (H, Nc))):
        _check_dev(t, name)
        if t.dtype != torch.bfloat16 or tuple(t.shape) != shape:
            raise ValueError("%s must be %s bfloat16" % (name, shape))
    ptrs = (_vp * N)(*[None if j == local_rank or t is None else t.data_ptr() for j, t in enumerate(recv)])
    rc = lib().gemm_rs(A.data_ptr(), B.data_ptr(), N, local_rank, M, Nc, K, ctypes.cast(ptrs, _vp),
                       P.data_ptr(), out.data_ptr(), RS_FUSED if fused else RS_UNFUSED, _stream_ptr(stream))
    if rc != AG_OK:
        raise AgError(rc, "gemm_rs")
    return P, out


def ag_gemm_unfused(shards, B, comm_block_rows, C=None, a_out=None, stream=None):
    return ag_gemm(shards, B, comm_block_rows, C=C, mode="unfused", a_out=a_out, stream=stream)


def _as5d(t: torch.Tensor) -> tuple:
    if t.dim() == 5:
        return tuple(t.shape)
    if t.dim() == 2:
        return (1, 1, 1) + tuple(t.shape)
    if t.dim() == 1:
        return (1, 1, 1, 1, t.shape[0])
    raise ValueError("tgather takes (D0, D1, D2, H, W), (H, W) or (W,) tensors")


def tgather(shards, valid_rows: int, valid_cols: int, dst: torch.Tensor | None = None,
            dst_rows: int | None = None, root: int = 0, stream=None) -> torch.Tensor:
    """dst[d0, d1, d2, r*H + i, j] = shards[r][d0, d1, d2, i, j]; returns dst."""
    shards = list(shards)
    N = len(shards)
    if N == 0:
        raise ValueError("need at least one shard")
    shape = _as5d(shards[0])
    D0, D1, D2, H, W = shape
    dt = shards[0].dtype
    for i, s in enumerate(shards):
        _check_dev(s, "shard %d" % i)
        if _as5d(s) != shape or s.dtype != dt:
            raise ValueError("all shards must share shape and dtype")
    if dst_rows is None:
        dst_rows = N * H
    if dst is None:
        dst = torch.empty((D0, D1, D2, dst_rows, W), dtype=dt, device=shards[0].device)
    _check_dev(dst, "dst")
    if dst.numel() != D0 * D1 * D2 * dst_rows * W or dst.dtype != dt:
        raise ValueError("dst must hold (D0, D1, D2, dst_rows, W) elements of the shards' dtype")
    esz = shards[0].element_size()
    rc = lib().tgather_ex(ctypes.cast(_ptrs(shards), _vp), N, dst.data_ptr(), D0, D1, D2, H, W,
                          dst_rows, valid_rows, valid_cols, esz, root, _stream_ptr(stream))
    if rc != AG_OK:
        raise AgError(rc, "tgather_ex")
    return dst


# ------------------------------------------------------------------------ language-model operators
ACT_NONE, ACT_RELU, ACT_SILU, ACT_GELU, ACT_GELU_TANH = 0, 1, 2, 3, 4
TYPE_BF16, TYPE_F32 = 0, 1
_ACTS = {"none": ACT_NONE, "relu": ACT_RELU, "silu": ACT_SILU, "gelu": ACT_GELU, "gelu_tanh": ACT_GELU_TANH}


def _need(t, name: str, shape: tuple, dtype=torch.bfloat16, device=None):
    """Checks a tensor argument; returns its device pointer (None for an absent one)."""
    if t is None:
        return None
    if t.dtype is dtype and t.shape == shape and t.is_cuda and t.is_contiguous() and (device is None or t.device == device):
        return t.data_ptr()
    if t.dtype != dtype or t.shape != shape:
        raise ValueError("%s must be %s %s, not %s %s" % (name, shape, dtype, tuple(t.shape), t.dtype))
    _check_dev(t, name)
    raise ValueError("%s is on %s, the other operands on %s" % (name, t.device, device))


def _dims(t, name: str, n: int):
    if t.dim() != n:
        raise ValueError("%s must have %d dimensions" % (name, n))
    return t.shape


class _on:
    """The stream a call runs on: outputs and scratch memory are allocated on it, so that they are not
    handed to other work before the call's kernels are done with them."""

    def __init__(self, stream, device):
        self.guard = torch.cuda.device(device)
        self.ctx = None if stream is None else torch.cuda.stream(stream)

    def __enter__(self):
        self.guard.__enter__()
        if self.ctx is not None:
            self.ctx.__enter__()

    def __exit__(self, *exc):
        if self.ctx is not None:
            self.ctx.__exit__(*exc)
        self.guard.__exit__(*exc)


def _elsewhere(stream, device) -> bool:
    """Whether a call needs another stream or device than the current one (it then enters _on and starts over)."""
    return stream is not None or (device.type == "cuda" and device.index != torch._C._cuda_getDevice())


def _stream_of(device) -> int:
    return torch._C._cuda_getCurrentRawStream(device.index)


@functools.lru_cache(maxsize=4096)
def _work_bytes(entry: str, device: int, *extents) -> int:
    return getattr(lib(), entry + "_workspace")(*extents)


def _work(entry: str, device, *extents):
    """(tensor, bytes) of the scratch memory that a call asks for."""
    n = _work_bytes(entry, device.index, *extents)
    return (torch.empty(n, dtype=torch.uint8, device=device) if n else None), n


def _done(rc: int, entry: str):
    if rc != AG_OK:
        raise AgError(rc, entry)


def _p(t):
    return None if t is None else t.data_ptr()


def _written(t):
    """A tensor of the caller's that a call has written counts as changed in place: autograd then refuses to use it
    where it was saved before."""
    if t is not None:
        torch.autograd.graph.increment_version(t)


def gemm_bias_act(A: torch.Tensor, B: torch.Tensor, bias: torch.Tensor | None = None, act: str = "none",
                  residual: torch.Tensor | None = None, C: torch.Tensor | None = None,
                  pre: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """C (M, Nc) = act(A @ B^T + bias) + residual, all bf16, sums in fp32.  A (M, K), B (Nc, K), bias (Nc),
    residual (M, Nc); act: "none" | "relu" | "silu" | "gelu" (erf) | "gelu_tanh".  pre: optional (M, Nc)
    output that receives A @ B^T + bias, which gemm_bias_act_bwd needs.  residual may be C itself.  C and pre, where
    given, are written in place; the result has no gradient function."""
    M, K = _dims(A, "A", 2)
    Nc = _dims(B, "B", 2)[0]
    dev = A.device
    if _elsewhere(stream, dev):
        with _on(stream, dev):
            return gemm_bias_act(A, B, bias, act, residual, C, pre)
    a, b = _need(A, "A", (M, K)), _need(B, "B", (Nc, K), device=dev)
    bi, r = _need(bias, "bias", (Nc,), device=dev), _need(residual, "residual", (M, Nc), device=dev)
    pr = _need(pre, "pre", (M, Nc), device=dev)
    out = A.new_empty((M, Nc)) if C is None else C
    c = _need(out, "C", (M, Nc), device=dev)
    w, n = _work("gemm_bias_act", dev, M, Nc, K)
    _done(lib().gemm_bias_act(a, b, bi, r, M, Nc, K, _ACTS[act], c, pr, _p(w), n, _stream_of(dev)), "gemm_bias_act")
    _written(C)
    _written(pre)
    return out


def gemm_bias_act_bwd(dC: torch.Tensor, A: torch.Tensor, B: torch.Tensor, act: str = "none",
                      pre: torch.Tensor | None = None, need_dA: bool = True, need_dB: bool = True,
                      need_dbias: bool = True, stream=None):
    """Gradients of gemm_bias_act: (dA (M, K), dB (Nc, K), dbias (Nc)) for dC (M, Nc), None where not
    needed.  pre: what gemm_bias_act stored (act "none" needs none).  The residual's gradient is dC."""
    M, K = _dims(A, "A", 2)
    Nc = _dims(B, "B", 2)[0]
    dev = A.device
    if _elsewhere(stream, dev):
        with _on(stream, dev):
            return gemm_bias_act_bwd(dC, A, B, act, pre, need_dA, need_dB, need_dbias)
    d, a = _need(dC, "dC", (M, Nc), device=dev), _need(A, "A", (M, K))
    b, pr = _need(B, "B", (Nc, K), device=dev), _need(pre, "pre", (M, Nc), device=dev)
    code = _ACTS[act]
    if code != ACT_NONE and pre is None:
        raise ValueError("act %r needs pre" % act)
    dA = torch.empty_like(A) if need_dA else None
    dB = torch.empty_like(B) if need_dB else None
    dbias = A.new_empty((Nc,)) if need_dbias else None
    w, n = _work("gemm_bias_act_bwd", dev, M, Nc, K, code)
    _done(lib().gemm_bias_act_bwd(d, a, b, pr, M, Nc, K, code, _p(dA), _p(dB), _p(dbias), _p(w), n, _stream_of(dev)),
          "gemm_bias_act_bwd")
    return dA, dB, dbias


def gemm_grouped(A: torch.Tensor, B: torch.Tensor, ends: torch.Tensor, C: torch.Tensor | None = None,
                 stream=None) -> torch.Tensor:
    """Rows [ends[e-1], ends[e]) of C (M, Nc) = the same rows of A (M, K) @ B[e]^T, B (E, Nc, K), all bf16;
    rows past ends[-1] are zero.  ends: (E,) int32 on the device, the running sums of the experts' row
    counts; it is not read on the host.  C, where given, is written in place; the result has no gradient function."""
    M, K = _dims(A, "A", 2)
    E, Nc, _ = _dims(B, "B", 3)
    dev = A.device
    if _elsewhere(stream, dev):
        with _on(stream, dev):
            return gemm_grouped(A, B, ends, C)
    a, b = _need(A, "A", (M, K)), _need(B, "B", (E, Nc, K), device=dev)
    en = _need(ends, "ends", (E,), torch.int32, dev)
    out = A.new_empty((M, Nc)) if C is None else C
    c = _need(out, "C", (M, Nc), device=dev)
    _done(lib().gemm_grouped(a, b, en, E, M, Nc, K, c, _stream_of(dev)), "gemm_grouped")
    _written(C)
    return out


def gemm_grouped_bwd(dC: torch.Tensor, A: torch.Tensor, B: torch.Tensor, ends: torch.Tensor, need_dA: bool = True,
                     need_dB: bool = True, stream=None):
    """Gradients of gemm_grouped: (dA (M, K), dB (E, Nc, K)) for dC (M, Nc), None where not needed."""
    M, K = _dims(A, "A", 2)
    E, Nc, _ = _dims(B, "B", 3)
    dev = A.device
    if _elsewhere(stream, dev):
        with _on(stream, dev):
            return gemm_grouped_bwd(dC, A, B, ends, need_dA, need_dB)
    d, a = _need(dC, "dC", (M, Nc), device=dev), _need(A, "A", (M, K))
    b, en = _need(B, "B", (E, Nc, K), device=dev), _need(ends, "ends", (E,), torch.int32, dev)
    dA = torch.empty_like(A) if need_dA else None
    dB = torch.empty_like(B) if need_dB else None
    _done(lib().gemm_grouped_bwd(d, a, b, en, E, M, Nc, K, _p(dA), _p(dB), _stream_of(dev)), "gemm_grouped_bwd")
    return dA, dB


def gemm_xent(A: torch.Tensor, B: torch.Tensor, targets: torch.Tensor, stream=None):
    """Cross entropy of the logits A @ B^T, which are never stored: (loss, lse), both (T,) fp32, for A (T, K),
    B (V, K) bf16 and targets (T,) int64.  A target outside [0, V) marks a row without one: loss 0, no
    gradient.  The results have no gradient function."""
    T, K = _dims(A, "A", 2)
    V = _dims(B, "B", 2)[0]
    dev = A.device
    if _elsewhere(stream, dev):
        with _on(stream, dev):
            return gemm_xent(A, B, targets)
    a, b = _need(A, "A", (T, K)), _need(B, "B", (V, K), device=dev)
    y = _need(targets, "targets", (T,), torch.int64, dev)
    loss = torch.empty((T,), dtype=torch.float32, device=dev)
    lse = torch.empty((T,), dtype=torch.float32, device=dev)
    w, n = _work("gemm_xent", dev, T, V, K)
    _done(lib().gemm_xent(a, b, y, T, V, K, loss.data_ptr(), lse.data_ptr(), _p(w), n, _stream_of(dev)), "gemm_xent")
    return loss, lse


def gemm_xent_bwd(dloss: torch.Tensor, A: torch.Tensor, B: torch.Tensor, targets: torch.Tensor, lse: torch.Tensor,
                  need_dA: bool = True, need_dB: bool = True, work_bytes: int | None = None, stream=None):
    """Gradients of gemm_xent: (dA (T, K), dB (V, K)) for dloss (T,) fp32 and gemm_xent's lse, None where not
    needed.  work_bytes: scratch memory to use, where the default (d logits in pieces of up to 512 MiB) is
    too much; fewer bytes make more, narrower pieces of the vocabulary."""
    T, K = _dims(A, "A", 2)
    V = _dims(B, "B", 2)[0]
    dev = A.device
    if _elsewhere(stream, dev):
        with _on(stream, dev):
            return gemm_xent_bwd(dloss, A, B, targets, lse, need_dA, need_dB, work_bytes)
    a, b = _need(A, "A", (T, K)), _need(B, "B", (V, K), device=dev)
    y, g = _need(targets, "targets", (T,), torch.int64, dev), _need(dloss, "dloss", (T,), torch.float32, dev)
    ls = _need(lse, "lse", (T,), torch.float32, dev)
    dA = torch.empty_like(A) if need_dA else None
    dB = torch.empty_like(B) if need_dB else None
    if work_bytes is None:
        w, n = _work("gemm_xent_bwd", dev, T, V, K)
    else:
        n = work_bytes
        w = torch.empty(n, dtype=torch.uint8, device=dev)
    _done(lib().gemm_xent_bwd(g, a, b, y, ls, T, V, K, _p(dA), _p(dB), _p(w), n, _stream_of(dev)), "gemm_xent_bwd")
    return dA, dB


def layer_norm(x: torch.Tensor, weight: torch.Tensor | None = None, bias: torch.Tensor | None = None, eps: float = 1e-5,
               residual: torch.Tensor | None = None, y: torch.Tensor | None = None, h: torch.Tensor | None = None,
               mean: torch.Tensor | None = None, rstd: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y (rows, width) = (s - mean) rstd weight + bias over each row of s = x, or of x + residual rounded to bf16.  x, residual
    (rows, width), weight, bias (width) bf16.  Optional outputs, which layer_norm_bwd needs: h (rows, width) bf16 receives
    the sum (it may be x or residual itself; without a residual s is x), mean and rstd (rows,) fp32 the statistics.  y, h, mean
    and rstd, where given, are written in place; the result has no gradient function."""
    rows, width = _dims(x, "x", 2)
    dev = x.device
    if _elsewhere(stream, dev):
        with _on(stream, dev):
            return layer_norm(x, weight, bias, eps, residual, y, h, mean, rstd)
    if h is not None and residual is None:
        raise ValueError("h receives x + residual: without a residual there is nothing to keep")
    shape, col, row = x.shape, (width,), (rows,)
    xp, rp = _need(x, "x", shape), _need(residual, "residual", shape, device=dev)
    wp, bp = _need(weight, "weight", col, device=dev), _need(bias, "bias", col, device=dev)
    hp = None if h is None else _need(h, "h", shape, device=dev)
    mp = None if mean is None else _need(mean, "mean", row, torch.float32, dev)
    sp = None if rstd is None else _need(rstd, "rstd", row, torch.float32, dev)
    out = torch.empty_like(x) if y is None else y
    yp = out.data_ptr() if y is None else _need(y, "y", shape, device=dev)
    _done(lib().layer_norm(xp, rp, wp, bp, rows, width, eps, yp, hp, mp, sp, _stream_of(dev)), "layer_norm")
    for t in (y, h, mean, rstd):
        if t is not None:
            _written(t)
    return out


def layer_norm_bwd(dy: torch.Tensor, h: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                   weight: torch.Tensor | None = None, dh: torch.Tensor | None = None, need_dx: bool = True,
                   need_dweight: bool = True, need_dbias: bool = True, stream=None):
    """Gradients of layer_norm: (dx (rows, width), dweight (width), dbias (width)) for dy (rows, width), None where not needed.
    h: what was normalised (layer_norm's h, or its x without a residual), mean and rstd as it wrote them.  dx is the gradient
    of x and of residual; dh, the gradient that reaches h on its other way, is added to it."""
    rows, width = _dims(h, "h", 2)
    dev = h.device
    if _elsewhere(stream, dev):
        with _on(stream, dev):
            return layer_norm_bwd(dy, h, mean, rstd, weight, dh, need_dx, need_dweight, need_dbias)
    dyp, hp = _need(dy, "dy", (rows, width), device=dev), _need(h, "h", (rows, width))
    mp, sp = _need(mean, "mean", (rows,), torch.float32, dev), _need(rstd, "rstd", (rows,), torch.float32, dev)
    wp, dhp = _need(weight, "weight", (width,), device=dev), _need(dh, "dh", (rows, width), device=dev)
    dx = torch.empty_like(h) if need_dx else None
    dweight = h.new_empty((width,)) if need_dweight else None
    dbias = h.new_empty((width,)) if need_dbias else None
    w, n = _work("layer_norm_bwd", dev, rows, width) if need_dweight or need_dbias else (None, 0)
    _done(lib().layer_norm_bwd(dyp, hp, mp, sp, wp, dhp, rows, width, _p(dx), _p(dweight), _p(dbias), _p(w), n,
                               _stream_of(dev)), "layer_norm_bwd")
    return dx, dweight, dbias


# (a, b, c) of five steps that take singular values from about 0.003 of a matrix's norm on to between 0.7 and 1.2
NEWTON_SCHULZ = ((3.4445, -4.7750, 2.0315),) * 5


@functools.lru_cache(maxsize=256)
def _steps(coefficients: tuple):
    return (ctypes.c_float * (3 * len(coefficients)))(*[x for abc in coefficients for x in abc])


def newton_schulz(G: torch.Tensor, coefficients=NEWTON_SCHULZ, eps: float = 1e-7, out: torch.Tensor | None = None,
                  stream=None) -> torch.Tensor:
    """G (R, C) or each matrix of G (E, R, C), bf16 or fp32, made nearly orthogonal: X = G / (|G| + eps), then for each step's
    (a, b, c) X = a X + (b A + c A A) X with A = X X^T (from the right where R > C).  out: bf16, G's shape; it may be G
    itself where that is bf16.  Written in place where given; the result has no gradient function.  Coefficients under which
    X could leave fp16's range are refused (aggemm.h has the bounds)."""
    if G.dim() not in (2, 3):
        raise ValueError("G must have 2 or 3 dimensions")
    if G.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("G must be bfloat16 or float32, not %s" % G.dtype)
    dev = G.device
    if _elsewhere(stream, dev):
        with _on(stream, dev):
            return newton_schulz(G, coefficients, eps, out)
    coefficients = tuple(tuple(float(x) for x in abc) for abc in coefficients)
    if not coefficients or any(len(abc) != 3 for abc in coefficients):
        raise ValueError("coefficients must be (a, b, c) for each of at least one step")
    E, R, C = (1,) * (3 - G.dim()) + tuple(G.shape)
    g = _need(G, "G", G.shape, G.dtype)
    res = torch.empty(G.shape, dtype=torch.bfloat16, device=dev) if out is None else out
    o = _need(res, "out", G.shape, device=dev)
    w, n = _work("newton_schulz", dev, E, R, C)
    _done(lib().newton_schulz(g, TYPE_F32 if G.dtype == torch.float32 else TYPE_BF16, E, R, C, _steps(coefficients),
                              len(coefficients), eps, o, _p(w), n, _stream_of(dev)), "newton_schulz")
    _written(out)
    return res


def check(stream=None) -> tuple[int, list[int]]:
    """Waits for the stream and returns (status, [code, chunk, tile, epoch]) of the device status
    word (the first wait that gave up since the last check, and its call's flag epoch)."""
    info = (_i64 * 4)()
    rc = lib().ag_check(_stream_ptr(stream), info)
    return rc, [int(x) for x in info]


def finalize():
    lib().ag_finalize()
