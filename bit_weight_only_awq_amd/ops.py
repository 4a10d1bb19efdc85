"""Thin torch-facing binding of libawq4.so: argument marshalling only.

Every step of the computation runs in the library's HIP kernels; this module
only checks tensor placement/dtypes, allocates outputs and the per-device
workspace through torch, and passes raw pointers and the current stream.
"""
from __future__ import annotations

import ctypes
import threading

import torch

from . import _lib as L

_F16 = {torch.float16: L.AWQ_DTYPE_F16, torch.bfloat16: L.AWQ_DTYPE_BF16}


def _ptr(t: torch.Tensor | None):
    return None if t is None else t.data_ptr()


def _stream(dev: torch.device):
    return torch.cuda.current_stream(dev).cuda_stream


# The raw handle of a device's current stream: the call behind
# torch.cuda.current_stream(dev).cuda_stream without building the Stream object
# (0.1 us against 1.8; a small kernel takes 3).
_raw_stream = torch._C._cuda_getCurrentRawStream


def _need_cuda(*ts):
    for t in ts:
        if t is not None:
            if not t.is_cuda:
                raise ValueError("all tensors must be on a CUDA (HIP) device")
            if not t.is_contiguous():
                raise ValueError("all tensors must be contiguous")


# ----------------------------------------------------------------------------- workspace

def _zeros(index: int, nbytes: int) -> torch.Tensor:
    """Zero bytes on device `index`, filled on its current stream."""
    return torch.zeros(nbytes, dtype=torch.uint8, device=torch.device("cuda", index))


def _capture_id(stream: int) -> int:
    """Number of the graph capture that `stream` is recording, 0 if none."""
    number = ctypes.c_uint64()
    L.check("awq_stream_capture_id", L.lib().awq_stream_capture_id(stream, ctypes.byref(number)))
    return number.value


class Workspace:
    """One zero-initialised workspace per (device, stream), grown on demand and
    shared by every call ordered on that stream (the library leaves its
    counters zero after each call).  Calls on different streams may overlap in
    time, so each stream gets its own buffer, zero-filled on that stream.  A
    buffer that has been replaced by a larger one is kept, since a graph
    captured earlier may hold its address (sizes at least double, so the kept
    ones together are smaller than the current one).

    A call that is being recorded into a graph takes the stream's buffer where
    it is large enough.  Where it is not, the capture gets one of its own, from
    the graph's memory and with its zero-fill recorded: that one is zero in
    replays of this graph only, so no eager call and no other capture takes
    it."""

    def __init__(self):
        self._bufs: dict[tuple[int, int], torch.Tensor] = {}
        self._kept: list[torch.Tensor] = []
        self._recorded: dict[tuple[int, int], tuple[int, torch.Tensor]] = {}  # (capture, its buffer)
        self._lock = threading.Lock()

    def get(self, device: torch.device, nbytes: int) -> torch.Tensor | None:
        if nbytes == 0:
            return None
        idx = device.index if device.index is not None else torch.cuda.current_device()
        return self._buffer(idx, _raw_stream(idx), nbytes)

    def of_stream(self, index: int, stream: int, nbytes: int):
        """(pointer, bytes) of the workspace of `stream`, the current stream of device `index`, at least nbytes."""
        buf = self._bufs.get((index, stream))
        if buf is None or buf.numel() < nbytes:
            buf = self._buffer(index, stream, nbytes)
        return buf.data_ptr(), buf.numel()

    def _buffer(self, index: int, stream: int, nbytes: int) -> torch.Tensor:
        key = (index, stream)
        with self._lock:
            buf = self._bufs.get(key)
            if buf is not None and buf.numel() >= nbytes:
                return buf
            capture = _capture_id(stream)
            if capture:
                number, buf = self._recorded.get(key, (0, None))
                if number != capture:
                    buf = None
                elif buf.numel() >= nbytes:
                    return buf
            elif buf is not None:
                self._kept.append(buf)
            buf = _zeros(index, max(nbytes, 2 * (buf.numel() if buf is not None else 0), 1 << 20))
            if capture:
                self._recorded[key] = (capture, buf)
            else:
                self._bufs[key] = buf
            return buf


WORKSPACE = Workspace()


def workspace_bytes(op: int, M: int, N: int, K: int, group_size: int, split_k: int = 0,
                    device: torch.device | None = None) -> int:
    """Workspace bytes of a call on `device` (the current device if None)."""
    if device is None:
        return int(L.lib().awq_workspace_bytes(op, M, N, K, group_size, split_k))
    with torch.cuda.device(device):
        return int(L.lib().awq_workspace_bytes(op, M, N, K, group_size, split_k))


def plan_info(op: int, M: int, N: int, K: int, group_size: int, split_k: int = 0, cu_count: int = 0) -> dict:
    """How the library would launch a call (awq_plan_info); cu_count 0 = the current device."""
    info = L.PlanInfo()
    L.check("awq_plan_info", L.lib().awq_plan_info(op, M, N, K, group_size, split_k, cu_count,
                                                   ctypes.byref(info)))
    return {f: getattr(info, f) for f, _ in L.PlanInfo._fields_}


# ----------------------------------------------------------------------------- packing

def pack(vals: torch.Tensor, layout: str = "n8", clamp_count: torch.Tensor | None = None) -> torch.Tensor:
    """Pack 4-bit values: layout "n8" (AWQ, uint8 [rows, cols] -> int32 [rows, cols/8]),
    "v2" (the newer AWQ packing, identity order, int32 [rows, ceil(cols/8)])
    or "k8" (W4A8, int8 [K, N] -> int32 [K/8, N])."""
    _need_cuda(vals, clamp_count)
    rows, cols = vals.shape
    if layout == "v2":
        out = torch.empty(rows, (cols + 7) // 8, dtype=torch.int32, device=vals.device)
        lay = L.AWQ_LAYOUT_V2
    elif layout == "n8":
        out = torch.empty(rows, cols // 8, dtype=torch.int32, device=vals.device)
        lay = L.AWQ_LAYOUT_N8
    else:
        out = torch.empty(rows // 8, cols, dtype=torch.int32, device=vals.device)
        lay = L.W4A8_LAYOUT_K8
    L.check("awq_pack", L.lib().awq_pack(_ptr(vals), _ptr(out), rows, cols, lay, _ptr(clamp_count),
                                         _stream(vals.device)))
    return out


def unpack(packed: torch.Tensor, layout: str = "n8", cols: int | None = None) -> torch.Tensor:
    """Inverse of pack; layout "v2" takes the number of values per row (default: all 8 per word)."""
    _need_cuda(packed)
    if layout == "v2":
        rows = packed.shape[0]
        cols = packed.shape[1] * 8 if cols is None else cols
        out = torch.empty(rows, cols, dtype=torch.uint8, device=packed.device)
        lay = L.AWQ_LAYOUT_V2
    elif layout == "n8":
        rows, cols = packed.shape[0], packed.shape[1] * 8
        out = torch.empty(rows, cols, dtype=torch.uint8, device=packed.device)
        lay = L.AWQ_LAYOUT_N8
    else:
        rows, cols = packed.shape[0] * 8, packed.shape[1]
        out = torch.empty(rows, cols, dtype=torch.int8, device=packed.device)
        lay = L.W4A8_LAYOUT_K8
    L.check("awq_unpack", L.lib().awq_unpack(_ptr(packed), _ptr(out), rows, cols, lay, _stream(packed.device)))
    return out


def repack_v2(qweight_v2: torch.Tensor, qzeros_v2: torch.Tensor | None, group_size: int = 128):
    """Weights in the newer AWQ packing -> (qweight, qzeros) in the format the
    GEMM / GEMV calls take (awq_repack_v2); scales are shared by both formats."""
    _need_cuda(qweight_v2, qzeros_v2)
    K, N = qweight_v2.shape[0], qweight_v2.shape[1] * 8
    qweight = torch.empty_like(qweight_v2)
    qzeros = None if qzeros_v2 is None else torch.empty(K // group_size, N // 8, dtype=torch.int32,
                                                        device=qweight_v2.device)
    L.check("awq_repack_v2", L.lib().awq_repack_v2(_ptr(qweight_v2), _ptr(qzeros_v2), _ptr(qweight), _ptr(qzeros),
                                                   N, K, group_size, _stream(qweight_v2.device)))
    return qweight, qzeros


# ----------------------------------------------------------------------------- W4A16

def _w4a16(fn_name: str, op: int, x, qweight, scales, qzeros, group_size, split_k, out):
    _need_cuda(x, qweight, scales, qzeros, out)
    if x.dtype not in _F16:
        raise ValueError("x must be fp16 or bf16")
    if scales.dtype != x.dtype:
        raise ValueError("scales must have the activation dtype")
    M, K = x.shape
    N = qweight.shape[1] * 8
    if out is None:
        out = torch.empty(M, N, dtype=x.dtype, device=x.device)
    need = workspace_bytes(op, M, N, K, group_size, split_k, x.device)
    ws = WORKSPACE.get(x.device, need)
    fn = getattr(L.lib(), fn_name)
    L.check(fn_name, fn(_ptr(x), _ptr(qweight), _ptr(scales), _ptr(qzeros), _ptr(out), M, N, K, group_size,
                        _F16[x.dtype], split_k, _ptr(ws), 0 if ws is None else ws.numel(), _stream(x.device)))
    return out


def gemm_w4a16(x, qweight, scales, qzeros, group_size: int = 128, split_k: int = 0, out=None):
    """Y = X . dequant(qweight, qzeros, scales) (prefill path, any M)."""
    return _w4a16("awq_gemm_w4a16", L.AWQ_OP_GEMM_W4A16, x, qweight, scales, qzeros, group_size, split_k, out)


def gemv_w4a16(x, qweight, scales, qzeros, group_size: int = 128, split_k: int = 0, out=None):
    """Decode path, M <= 8."""
    return _w4a16("awq_gemv_w4a16", L.AWQ_OP_GEMV_W4A16, x, qweight, scales, qzeros, group_size, split_k, out)


def linear_w4a16(x, qweight, scales, qzeros, group_size: int = 128, out=None):
    """The AWQ linear-layer dispatch: more than 8 rows -> GEMM, else GEMV."""
    if x.shape[0] > 8:
        return gemm_w4a16(x, qweight, scales, qzeros, group_size, out=out)
    return gemv_w4a16(x, qweight, scales, qzeros, group_size, out=out)


def dequant_w4a16(qweight, scales, qzeros, group_size: int = 128, out=None):
    """Dense W = (q - z) * s, [K, N] in the scales' dtype (one rounding per
    element): the weight operand of a dense vendor GEMM, for comparison."""
    _need_cuda(qweight, scales, qzeros, out)
    if scales.dtype not in _F16:
        raise ValueError("scales must be fp16 or bf16")
    K, N = qweight.shape[0], qweight.shape[1] * 8
    if out is None:
        out = torch.empty(K, N, dtype=scales.dtype, device=qweight.device)
    L.check("awq_dequant_w4a16", L.lib().awq_dequant_w4a16(_ptr(qweight), _ptr(scales), _ptr(qzeros), _ptr(out), N,
                                                           K, group_size, _F16[scales.dtype],
                                                           _stream(qweight.device)))
    return out


# ----------------------------------------------------------------------------- W4A8

def quant_act(x: torch.Tensor, a8: torch.Tensor | None = None, s1: torch.Tensor | None = None):
    """Per-token int8 quantisation of fp16 or bf16 activations -> (a8 int8 [M,K], s1 fp32 [M])."""
    _need_cuda(x, a8, s1)
    if x.dtype not in _F16:
        raise ValueError("W4A8 activations must be fp16 or bf16")
    M, K = x.shape
    if a8 is None:
        a8 = torch.empty(M, K, dtype=torch.int8, device=x.device)
    if s1 is None:
        s1 = torch.empty(M, dtype=torch.float32, device=x.device)
    L.check("w4a8_quant_act", L.lib().w4a8_quant_act(_ptr(x), _ptr(a8), _ptr(s1), M, K, _F16[x.dtype],
                                                     _stream(x.device)))
    return a8, s1


def w4a8_gemm(a8, b, s1, s2, s3=None, group_size: int = -1, want_acc: bool = False, out=None):
    """y = act(acc * s1 * s2), acc = a8 . w8 (exact int32), in the dtype of s2
    (fp16 or bf16; s3 and y share it). Returns y or (y, acc)."""
    _need_cuda(a8, b, s1, s2, s3, out)
    if s2.dtype not in _F16 or (s3 is not None and s3.dtype != s2.dtype):
        raise ValueError("W4A8 scales must be fp16 or bf16, s2 and s3 alike")
    M, K = a8.shape
    N = b.shape[1]
    if out is None:
        out = torch.empty(M, N, dtype=s2.dtype, device=a8.device)
    acc = torch.empty(M, N, dtype=torch.int32, device=a8.device) if want_acc else None
    need = workspace_bytes(L.AWQ_OP_W4A8_GEMM, M, N, K, group_size, 0, a8.device)
    ws = WORKSPACE.get(a8.device, need)
    L.check("w4a8_gemm", L.lib().w4a8_gemm(_ptr(a8), _ptr(b), _ptr(s1), _ptr(s2), _ptr(s3), _ptr(out), _ptr(acc),
                                           M, N, K, group_size, _F16[s2.dtype], _ptr(ws),
                                           0 if ws is None else ws.numel(), _stream(a8.device)))
    return (out, acc) if want_acc else out


def linear_w4a8(x, b, s2, s3=None, group_size: int = -1, want_acc: bool = False, out=None, a8=None, s1=None):
    """The whole W4A8 layer in one call (w4a8_linear): per-token quantisation of
    x, then the W4A8 GEMM, fused into one kernel for small batches.  Returns y,
    or (y, s1, acc) with want_acc.  `a8` is scratch for the two-step path."""
    _need_cuda(x, b, s2, s3, out, a8, s1)
    if x.dtype not in _F16 or s2.dtype != x.dtype or (s3 is not None and s3.dtype != x.dtype):
        raise ValueError("W4A8 activations and scales must be fp16 or bf16, all of one type")
    M, K = x.shape
    N = b.shape[1]
    if a8 is None:
        a8 = torch.empty(M, K, dtype=torch.int8, device=x.device)
    if s1 is None:
        s1 = torch.empty(M, dtype=torch.float32, device=x.device)
    if out is None:
        out = torch.empty(M, N, dtype=x.dtype, device=x.device)
    acc = torch.empty(M, N, dtype=torch.int32, device=x.device) if want_acc else None
    need = workspace_bytes(L.AWQ_OP_W4A8_GEMM, M, N, K, group_size, 0, x.device)
    ws = WORKSPACE.get(x.device, need)
    L.check("w4a8_linear", L.lib().w4a8_linear(_ptr(x), _ptr(a8), _ptr(s1), _ptr(b), _ptr(s2), _ptr(s3), _ptr(out),
                                               _ptr(acc), M, N, K, group_size, _F16[x.dtype], _ptr(ws),
                                               0 if ws is None else ws.numel(), _stream(x.device)))
    return (out, s1, acc) if want_acc else out


# ----------------------------------------------------------------------------- INT4-FP8 W4A8

def quant_act_fp8(x: torch.Tensor, a=None, s1=None, asum=None):
    """Per-token E4M3 quantisation -> (codes uint8 [M,K], s1 fp32 [M], asum fp32 [M])."""
    _need_cuda(x, a, s1, asum)
    if x.dtype not in _F16:
        raise ValueError("activations must be fp16 or bf16")
    M, K = x.shape
    a = torch.empty(M, K, dtype=torch.uint8, device=x.device) if a is None else a
    s1 = torch.empty(M, dtype=torch.float32, device=x.device) if s1 is None else s1
    asum = torch.empty(M, dtype=torch.float32, device=x.device) if asum is None else asum
    L.check("w4a8_fp8_quant_act", L.lib().w4a8_fp8_quant_act(_ptr(x), _ptr(a), _ptr(s1), _ptr(asum), M, K,
                                                             _F16[x.dtype], _stream(x.device)))
    return a, s1, asum


def w4a8_fp8_gemm(a, b, s1, asum, s2, want_acc: bool = False, out=None):
    """y = act(acc * s1 * s2), acc = sum_k e4m3(a) q (fp32 on the fp8 matrix
    cores), in the dtype of s2.  Returns y or (y, acc)."""
    _need_cuda(a, b, s1, asum, s2, out)
    if s2.dtype not in _F16:
        raise ValueError("s2 must be fp16 or bf16")
    M, K = a.shape
    N = b.shape[1]
    if out is None:
        out = torch.empty(M, N, dtype=s2.dtype, device=a.device)
    acc = torch.empty(M, N, dtype=torch.float32, device=a.device) if want_acc else None
    need = workspace_bytes(L.AWQ_OP_W4A8_FP8_GEMM, M, N, K, -1, 0, a.device)
    ws = WORKSPACE.get(a.device, need)
    L.check("w4a8_fp8_gemm", L.lib().w4a8_fp8_gemm(_ptr(a), _ptr(b), _ptr(s1), _ptr(asum), _ptr(s2), _ptr(out),
                                                   _ptr(acc), M, N, K, _F16[s2.dtype], _ptr(ws),
                                                   0 if ws is None else ws.numel(), _stream(a.device)))
    return (out, acc) if want_acc else out


def linear_w4a8_fp8(x, b, s2, want_acc: bool = False, out=None, a=None, s1=None, asum=None):
    """The whole INT4-FP8 layer in one call (w4a8_fp8_linear): per-token E4M3
    quantisation of x, then the GEMM, one kernel for a single token.  Returns
    y, or (y, s1, acc) with want_acc.  `a` and `asum` are scratch for the
    two-step path."""
    _need_cuda(x, b, s2, out, a, s1, asum)
    if x.dtype not in _F16 or s2.dtype != x.dtype:
        raise ValueError("activations and s2 must be fp16 or bf16, of one type")
    M, K = x.shape
    N = b.shape[1]
    a = torch.empty(M, K, dtype=torch.uint8, device=x.device) if a is None else a
    s1 = torch.empty(M, dtype=torch.float32, device=x.device) if s1 is None else s1
    asum = torch.empty(M, dtype=torch.float32, device=x.device) if asum is None else asum
    if out is None:
        out = torch.empty(M, N, dtype=x.dtype, device=x.device)
    acc = torch.empty(M, N, dtype=torch.float32, device=x.device) if want_acc else None
    need = workspace_bytes(L.AWQ_OP_W4A8_FP8_GEMM, M, N, K, -1, 0, x.device)
    ws = WORKSPACE.get(x.device, need)
    L.check("w4a8_fp8_linear", L.lib().w4a8_fp8_linear(_ptr(x), _ptr(a), _ptr(s1), _ptr(asum), _ptr(b), _ptr(s2),
                                                       _ptr(out), _ptr(acc), M, N, K, _F16[x.dtype], _ptr(ws),
                                                       0 if ws is None else ws.numel(), _stream(x.device)))
    return (out, s1, acc) if want_acc else out


# ----------------------------------------------------------------------------- RMS norm

def _tensor(t, shape, dtype, index, what):
    """Refuse a tensor that is not contiguous, of this shape and type, on device `index`."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{what} must be {tuple(shape)}, {dtype}, contiguous, on CUDA (HIP) device {index}")


def _rmsnorm(fn, x, weight, eps, residual, residual_out, y, codes):
    """Checks and call of the norm entry points; codes: their code, scale and sum tensors."""
    if not x.is_cuda:
        raise ValueError("all tensors must be on a CUDA (HIP) device")
    dt, dev, shape = x.dtype, x.get_device(), x.shape
    if dt not in _F16 or len(shape) != 2 or not x.is_contiguous():
        raise ValueError("x must be contiguous fp16 or bf16, [rows, columns]")
    _tensor(weight, shape[1:], dt, dev, "weight")
    if residual is not None:
        _tensor(residual, shape, dt, dev, "residual")
        if residual_out is None:
            residual_out = torch.empty_like(x)
        elif residual_out is not residual:
            _tensor(residual_out, shape, dt, dev, "residual_out")
    elif residual_out is not None:
        raise ValueError("residual_out without a residual")
    if y is not None and y is not x:
        _tensor(y, shape, dt, dev, "y")
    status = getattr(L.lib(), fn)(
        x.data_ptr(), None if residual is None else residual.data_ptr(), weight.data_ptr(),
        None if residual is None else residual_out.data_ptr(), None if y is None else y.data_ptr(),
        *[None if c is None else c.data_ptr() for c in codes], shape[0], shape[1], eps, _F16[dt], _raw_stream(dev))
    if status:
        L.check(fn, status)
    return residual_out


def _codes(x, given, fp8: bool):
    """The code, scale (and sum) tensors of x's rows: those given, checked, or new ones."""
    shape, dtype, out = x.shape, torch.uint8 if fp8 else torch.int8, []
    for t in given:
        if t is None:
            t = torch.empty(shape, dtype=dtype, device=x.device)
        else:
            _tensor(t, shape, dtype, x.get_device(), "codes, scales and sums")
        out.append(t)
        shape, dtype = shape[:1], torch.float32
    return out


def rmsnorm(x, weight, eps: float = 1e-6, residual=None, residual_out=None, out=None):
    """y = norm(x + residual) * weight in x's type, for the W4A16 layers.
    Returns y, or (y, x + residual) with a residual (residual_out may be the
    residual itself, out may be x)."""
    out = torch.empty_like(x) if out is None else out
    residual_out = _rmsnorm("w4a8_rmsnorm_quant", x, weight, eps, residual, residual_out, out, (None, None))
    return out if residual is None else (out, residual_out)


def rmsnorm_quant(x, weight, eps: float = 1e-6, residual=None, residual_out=None, y=None, a8=None, s1=None):
    """norm(x + residual) * weight as int8 codes with one scale per token, the
    input of w4a8_gemm: (a8, s1, x + residual or None).  The norm itself is
    written to y where given."""
    a8, s1 = _codes(x, (a8, s1), False)
    residual_out = _rmsnorm("w4a8_rmsnorm_quant", x, weight, eps, residual, residual_out, y, (a8, s1))
    return a8, s1, residual_out


def rmsnorm_quant_fp8(x, weight, eps: float = 1e-6, residual=None, residual_out=None, y=None, a=None, s1=None,
                      asum=None):
    """The same as E4M3 codes, the input of w4a8_fp8_gemm: (codes uint8, s1,
    asum, x + residual or None)."""
    a, s1, asum = _codes(x, (a, s1, asum), True)
    residual_out = _rmsnorm("w4a8_fp8_rmsnorm_quant", x, weight, eps, residual, residual_out, y, (a, s1, asum))
    return a, s1, asum, residual_out


# ----------------------------------------------------------------------------- attention over a 4-bit cache

def kv4_cache(num_pages: int, kv_heads: int, head_dim: int, page_size: int, device=None) -> torch.Tensor:
    """A zeroed paged key/value cache in 4 bits (layout: awq4.h), int32
    [num_pages, kv_heads, words of a page and head]."""
    words = int(L.lib().awq_kv4_head_words(head_dim, page_size))
    if words == 0:
        raise ValueError("head_dim must be 64 or 128, page_size a power of two from 16 to 1024")
    return torch.zeros(num_pages, kv_heads, words, dtype=torch.int32, device="cuda" if device is None else device)


def _kv4_page_size(cache, head_dim: int) -> int:
    if cache.dim() != 3 or cache.dtype != torch.int32:
        raise ValueError("cache must be int32 [num_pages, kv_heads, words]")
    page = cache.shape[2] // (head_dim // 4 + 2)
    if page * (head_dim // 4 + 2) != cache.shape[2]:
        raise ValueError("the cache's words do not fit this head dimension")
    return page


def rope_table(positions: int, rot: int, base: float = 10000.0, scale: float = 1.0, device=None) -> torch.Tensor:
    """fp32 [positions, rot]: the cosines, then the sines, of p / scale *
    base^(-2i / rot) (scale > 1 stretches the positions for longer contexts),
    from angles in 64 bits."""
    inv = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    ang = (torch.arange(positions, dtype=torch.float64) / scale)[:, None] * inv
    return torch.cat((ang.cos(), ang.sin()), 1).float().to("cuda" if device is None else device)


def _heads(t, shape, dtype, index, what):
    """Elements from one token to the next of [T, H, D] with dense heads."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != index:
        raise ValueError(f"{what} must be {tuple(shape)}, {dtype}, on CUDA (HIP) device {index}")
    T, H, D = shape
    step, head, one = t.stride()
    if (one != 1 and D > 1) or (head != D and H > 1):
        raise ValueError(f"{what} must have dense heads")
    return step if T > 1 else H * D  # (a single token's stride says nothing)


def kv4_append(q, k, v, rope, positions, slots, cache, interleaved: bool = False, out=None):
    """Rotary positions on q and k [T, H, D] (rope: fp32 [max_pos, rot], None =
    no rotation), k and v quantised to 4 bits into the cache's slots; returns
    the rotated q (None for q = None).  q, k and v may be views of one fused
    QKV tensor."""
    if not k.is_cuda:
        raise ValueError("all tensors must be on a CUDA (HIP) device")
    dt, dev, shape = k.dtype, k.get_device(), k.shape
    if dt not in _F16 or len(shape) != 3:
        raise ValueError("k must be fp16 or bf16 [tokens, heads, head_dim]")
    T, hkv, D = shape
    k_step, v_step = _heads(k, shape, dt, dev, "k"), _heads(v, shape, dt, dev, "v")
    hq = q_step = rot = max_pos = 0
    q_ptr = out_ptr = rope_ptr = pos_ptr = None
    if q is not None:
        hq = q.shape[1]
        q_shape = torch.Size((T, hq, D))
        q_step = _heads(q, q_shape, dt, dev, "q")
        if out is None:
            out = torch.empty(q_shape, dtype=dt, device=k.device)
        else:
            _tensor(out, q_shape, dt, dev, "out")
        q_ptr, out_ptr = q.data_ptr(), out.data_ptr()
    if rope is not None:
        _tensor(rope, rope.shape, torch.float32, dev, "rope")
        if positions is None or rope.dim() != 2:
            raise ValueError("rope must be [max_pos, rot] and come with positions")
        _tensor(positions, shape[:1], torch.int32, dev, "positions")
        max_pos, rot = rope.shape
        rope_ptr, pos_ptr = rope.data_ptr(), positions.data_ptr()
    _tensor(slots, shape[:1], torch.int64, dev, "slots")
    _tensor(cache, cache.shape, torch.int32, dev, "cache")
    page = _kv4_page_size(cache, D)
    if cache.shape[1] != hkv:
        raise ValueError("the cache has another number of key/value heads")
    status = L.lib().awq_kv4_append(q_ptr, k.data_ptr(), v.data_ptr(), q_step, k_step, v_step, rope_ptr, pos_ptr,
                                    slots.data_ptr(), out_ptr, cache.data_ptr(), T, hq, hkv, D, page, cache.shape[0],
                                    rot, max_pos, int(interleaved), _F16[dt], _raw_stream(dev))
    if status:
        L.check("awq_kv4_append", status)
    return out


def kv4_attention(q, cache, tables, lens, scale: float | None = None, cu_q=None, max_q: int | None = None,
                  max_kv: int | None = None, window: int = 0, out=None):
    """Causal attention of q [total_q, Hq, D] over the paged 4-bit cache.
    tables int32 [B, pages of a sequence], lens int32 [B] (tokens with the new
    ones); cu_q int32 [B + 1] where sequences have more than one new token, and
    max_q, the most that one has (default: all rows of q, which is right but
    launches more than a tight bound; rows past a sequence's first max_q are not
    written); max_kv: the longest sequence (default: what the tables can hold);
    scale: default 1 / sqrt(D)."""
    if not q.is_cuda:
        raise ValueError("all tensors must be on a CUDA (HIP) device")
    dt, dev, shape = q.dtype, q.get_device(), q.shape
    if dt not in _F16 or len(shape) != 3 or not q.is_contiguous():
        raise ValueError("q must be contiguous fp16 or bf16 [tokens, heads, head_dim]")
    total, hq, D = shape
    B = lens.shape[0]
    _tensor(lens, lens.shape[:1], torch.int32, dev, "lens")
    _tensor(tables, torch.Size((B, tables.shape[-1])), torch.int32, dev, "tables")
    if cu_q is not None:
        _tensor(cu_q, torch.Size((B + 1,)), torch.int32, dev, "cu_q")
    _tensor(cache, cache.shape, torch.int32, dev, "cache")
    page = _kv4_page_size(cache, D)
    if out is None:
        out = torch.empty_like(q)
    elif out is not q:
        _tensor(out, shape, dt, dev, "out")
    if max_q is None:
        max_q = 1 if cu_q is None else max(total, 1)
    pages, hkv, _ = cache.shape
    width = tables.shape[1]
    if max_kv is None:
        max_kv = width * page
    lib = L.lib()
    if torch._C._cuda_getDevice() == dev:
        need = lib.awq_kv4_attention_workspace_bytes(B, max_q, hq, hkv, D, max_kv)
    else:
        with torch.cuda.device(dev):
            need = lib.awq_kv4_attention_workspace_bytes(B, max_q, hq, hkv, D, max_kv)
    stream = _raw_stream(dev)
    ws, ws_bytes = WORKSPACE.of_stream(dev, stream, need) if need else (None, 0)
    status = lib.awq_kv4_attention(q.data_ptr(), cache.data_ptr(), tables.data_ptr(), lens.data_ptr(),
                                   None if cu_q is None else cu_q.data_ptr(), out.data_ptr(), B, total, max_q, max_kv,
                                   hq, hkv, D, page, pages, width, D ** -0.5 if scale is None else scale, window,
                                   _F16[dt], ws, ws_bytes, stream)
    if status:
        L.check("awq_kv4_attention", status)
    return out


# ----------------------------------------------------------------------------- measurement helper

STREAM_SINK_WORDS = 8192


def stream_read(src: torch.Tensor, sink: torch.Tensor | None = None) -> torch.Tensor:
    """Read every byte of `src` once on the GPU (bandwidth probe; not part of the
    method).  Returns the int32 sink of per-wave checksums."""
    _need_cuda(src, sink)
    nbytes = src.numel() * src.element_size()
    if sink is None:
        sink = torch.empty(STREAM_SINK_WORDS, dtype=torch.int32, device=src.device)
    if not src.is_contiguous() or sink.numel() < STREAM_SINK_WORDS or sink.dtype != torch.int32:
        raise ValueError("stream_read needs a contiguous source and an int32 sink of STREAM_SINK_WORDS words")
    L.check("awq_stream_read", L.lib().awq_stream_read(_ptr(src), nbytes, _ptr(sink), _stream(src.device)))
    return sink
