"""Thin ctypes binding of libgq (``include/gq.h``, ``include/gq_kv.h``), same names as the C ABI.

The functions here only marshal arguments: they check the dtype, shape,
contiguity and device of every torch tensor they pass (inputs and
caller-supplied outputs alike, all before the first library call), allocate
missing outputs and workspaces with torch (device memory plumbing), and pass
raw pointers plus the current HIP stream to the library.  Every step of the
computation runs in the library's kernels; there is no fallback path.  A
missing ``libgq.so`` raises immediately.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgq.so")

GQ_OK, GQ_ERR_INVALID_ARG, GQ_ERR_UNSUPPORTED, GQ_ERR_MISALIGNED, GQ_ERR_HIP = range(5)
GQ_F32, GQ_F16, GQ_BF16 = 0, 1, 2

# Every entry point declared in include/gq.h.
EXPORTS = (
    "gq_status_str", "gq_version", "gq_packed_sizes", "gq_quantize_groups", "gq_pack_int4",
    "gq_dequantize", "gq_w4a16_gemv", "gq_w4a16_gemv_workspace_size", "gq_w4a16_gemv_ws",
    "gq_w4a16_gemm", "gq_w4a16_gemm_workspace_size", "gq_w4a16_gemm_ws", "gq_w4a16_gemm_noalloc",
    "gq_q4k_quantize", "gq_q4k_gemv", "gq_ingest_group_major",
    "gq_w4a16_gemv_f16", "gq_w4a16_gemv_f16_ws", "gq_w4a16_gemm_f16", "gq_w4a16_gemm_f16_ws",
)
# the 4-bit key/value cache and its attention (include/gq_kv.h)
KV_EXPORTS = ("gq_kv4_cache_bytes", "gq_kv4_write", "gq_kv4_read",
              "gq_kv4_attention_workspace_size", "gq_kv4_attention")
# comparators and probes (include/gq_bench.h)
BENCH_EXPORTS = ("gq_bf16_gemv", "gq_stream_read", "gq_probe_mfma_valu", "gq_probe_lds_read")


class GqQParams(ctypes.Structure):
    _fields_ = [("bits", ctypes.c_int32), ("group_size", ctypes.c_int32),
                ("symmetric", ctypes.c_int32)]


class GqKv4Layout(ctypes.Structure):
    _fields_ = [("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("group_size", ctypes.c_int32),
                ("symmetric", ctypes.c_int32)]


class GqKv4AttentionArgs(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("q_token_stride", ctypes.c_int64),
                ("q_head_stride", ctypes.c_int64), ("q_tokens", ctypes.c_int64),
                ("q_heads", ctypes.c_int32), ("dtype", ctypes.c_int),
                ("cache", ctypes.c_void_p), ("n_pages", ctypes.c_int64), ("layout", GqKv4Layout),
                ("page_table", ctypes.c_void_p), ("batch", ctypes.c_int64),
                ("table_pages", ctypes.c_int64), ("kv_lens", ctypes.c_void_p),
                ("q_starts", ctypes.c_void_p), ("max_q_len", ctypes.c_int64),
                ("max_kv_len", ctypes.c_int64), ("causal", ctypes.c_int32),
                ("window", ctypes.c_int32), ("scale", ctypes.c_float), ("out", ctypes.c_void_p),
                ("lse", ctypes.c_void_p)]


class GqError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {lib().gq_status_str(status).decode()}")


_lib = None


def lib() -> ctypes.CDLL:
    """Load libgq.so (built in-tree); raise if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is not built; run `python -m w4a16_dequant_gemm_group_amd.build`")
    L = ctypes.CDLL(LIB_PATH)
    p, i64, i32, c = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_int
    sz = ctypes.c_size_t
    Q = GqQParams
    L.gq_status_str.restype = ctypes.c_char_p
    L.gq_status_str.argtypes = [c]
    L.gq_version.restype = i32
    L.gq_version.argtypes = []
    mm = [p, i64, i64, p, p, p, i64, Q, p, p]              # x M K qweight scales zeros N p y stream
    mm_ws = [p, i64, i64, p, p, p, i64, Q, p, p, sz, p]    # ... y workspace bytes stream
    sig = {
        "gq_packed_sizes": [i64, i64, Q, ctypes.POINTER(i64), ctypes.POINTER(i64), ctypes.POINTER(i64)],
        "gq_quantize_groups": [p, c, i64, i64, Q, p, p, p, p],
        "gq_pack_int4": [p, i64, i64, i32, p, p],
        "gq_dequantize": [p, p, p, i64, i64, Q, p, c, p],
        "gq_w4a16_gemv": mm,
        "gq_w4a16_gemv_workspace_size": [i64, i64, i64, Q, ctypes.POINTER(sz)],
        "gq_w4a16_gemv_ws": mm_ws,
        "gq_w4a16_gemm": mm,
        "gq_w4a16_gemm_workspace_size": [i64, i64, i64, Q, ctypes.POINTER(sz)],
        "gq_w4a16_gemm_ws": mm_ws,
        "gq_w4a16_gemm_noalloc": mm,
        "gq_q4k_quantize": [p, c, i64, i64, p, p],
        "gq_q4k_gemv": [p, i64, i64, p, i64, p, p],
        "gq_bf16_gemv": [p, i64, i64, p, i64, p, p],
        "gq_ingest_group_major": [p, p, i64, i64, i64, p, p, p],
        "gq_w4a16_gemv_f16": mm,
        "gq_w4a16_gemv_f16_ws": mm_ws,
        "gq_w4a16_gemm_f16": mm,
        "gq_w4a16_gemm_f16_ws": mm_ws,
        "gq_kv4_cache_bytes": [i64, GqKv4Layout, ctypes.POINTER(sz)],
        "gq_kv4_write": [p, i64, i64, p, i64, i64, c, i64, p, p, i64, GqKv4Layout, p],
        "gq_kv4_read": [p, i64, GqKv4Layout, p, i64, p, p, c, p],
        "gq_kv4_attention_workspace_size": [ctypes.POINTER(GqKv4AttentionArgs), ctypes.POINTER(sz)],
        "gq_kv4_attention": [ctypes.POINTER(GqKv4AttentionArgs), p, sz, p],
        "gq_stream_read": [p, i64, p, p],
        "gq_probe_mfma_valu": [i32, i32, i32, p, p, p],
        "gq_probe_lds_read": [i32, i32, i32, p, p, p],
    }
    for name, args in sig.items():
        f = getattr(L, name)
        f.argtypes = args
        f.restype = c
    _lib = L
    return L


def _ok(status: int, where: str) -> None:
    if status != GQ_OK:
        raise GqError(status, where)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


# The current stream's handle without a Stream object around it, a third of a small
# call's host time.  Not part of torch's public interface: where a torch lacks it, the
# public way is taken.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> int:
    """Handle of a stream (default: the current device's current one)."""
    if stream is None:
        if _raw_stream is None:
            return torch.cuda.current_stream().cuda_stream
        return _raw_stream(torch.cuda.current_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _need(t, name: str, dtypes, shape=None):
    """Type, dtype, shape and contiguity of a tensor the library will touch."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype} not in {dtypes}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _on_device(dev, **tensors) -> None:
    """Every given tensor is a GPU tensor on `dev` (checked after all shapes)."""
    index = None if dev is None else dev.index
    for name, t in tensors.items():
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError(f"{name} must be a GPU tensor")
        if index is not None and t.get_device() != index:
            raise ValueError(f"{name} is on {t.device}, expected {dev}")


def _groups(K: int, group_size: int) -> int:
    if group_size <= 0 or K % group_size != 0:
        raise ValueError(f"group_size {group_size} must be positive and divide K={K}")
    return K // group_size


_DT = {torch.float32: GQ_F32, torch.float16: GQ_F16, torch.bfloat16: GQ_BF16}


def qparams(bits: int = 4, group_size: int = 128, symmetric: bool = False) -> GqQParams:
    return GqQParams(int(bits), int(group_size), int(bool(symmetric)))


def gq_version() -> int:
    return int(lib().gq_version())


def gq_packed_sizes(N: int, K: int, bits: int = 4, group_size: int = 128, symmetric: bool = False):
    """(qweight_bytes, scale_bytes, zero_bytes) of an [N, K] weight."""
    q, s, z = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
    _ok(lib().gq_packed_sizes(N, K, qparams(bits, group_size, symmetric),
                              ctypes.byref(q), ctypes.byref(s), ctypes.byref(z)), "gq_packed_sizes")
    return q.value, s.value, z.value


def gq_quantize_groups(w: torch.Tensor, bits: int = 4, group_size: int = 128,
                       symmetric: bool = False, codes=None, scales=None, zeros=None, stream=None):
    """w [N, K] (bf16/fp16/fp32) -> (codes u8/i8 [N,K], scales fp16 [N,K/G], zeros fp16 or None)."""
    _need(w, "w", tuple(_DT))
    if w.dim() != 2:
        raise ValueError(f"w must be 2-D, got {tuple(w.shape)}")
    N, K = w.shape
    ng = _groups(K, group_size)
    cdt = torch.int8 if symmetric else torch.uint8
    if codes is not None:
        _need(codes, "codes", (cdt,), (N, K))
    if scales is not None:
        _need(scales, "scales", (torch.float16,), (N, ng))
    if zeros is not None:
        if symmetric:
            raise ValueError("zeros must be None for symmetric quantization")
        _need(zeros, "zeros", (torch.float16,), (N, ng))
    _on_device(None, w=w)
    dev = w.device
    _on_device(dev, codes=codes, scales=scales, zeros=zeros)
    if codes is None:
        codes = torch.empty((N, K), dtype=cdt, device=dev)
    if scales is None:
        scales = torch.empty((N, ng), dtype=torch.float16, device=dev)
    if zeros is None and not symmetric:
        zeros = torch.empty((N, ng), dtype=torch.float16, device=dev)
    _ok(lib().gq_quantize_groups(_ptr(w), _DT[w.dtype], N, K, qparams(bits, group_size, symmetric),
                                 _ptr(codes), _ptr(scales), _ptr(zeros), _stream(stream)),
        "gq_quantize_groups")
    return codes, scales, zeros


def gq_pack_int4(codes: torch.Tensor, symmetric: bool = False, qweight=None, stream=None):
    """codes [N, K] -> qweight uint8 [N, K/2] (low nibble = even k)."""
    _need(codes, "codes", (torch.uint8, torch.int8))
    if codes.dim() != 2 or codes.shape[1] % 2:
        raise ValueError(f"codes must be [N, K] with K even, got {tuple(codes.shape)}")
    N, K = codes.shape
    if qweight is not None:
        _need(qweight, "qweight", (torch.uint8,), (N, K // 2))
    _on_device(None, codes=codes)
    _on_device(codes.device, qweight=qweight)
    if qweight is None:
        qweight = torch.empty((N, K // 2), dtype=torch.uint8, device=codes.device)
    _ok(lib().gq_pack_int4(_ptr(codes), N, K, int(bool(symmetric)), _ptr(qweight), _stream(stream)),
        "gq_pack_int4")
    return qweight


def _weights(qweight, scales, zeros, group_size: int, symmetric: bool):
    """Check the packed weight bundle; returns (N, K, n_groups)."""
    _need(qweight, "qweight", (torch.uint8,))
    if qweight.dim() != 2:
        raise ValueError(f"qweight must be [N, K/2], got {tuple(qweight.shape)}")
    N, K = qweight.shape[0], qweight.shape[1] * 2
    ng = _groups(K, group_size)
    _need(scales, "scales", (torch.float16,), (N, ng))
    if symmetric:
        if zeros is not None:
            raise ValueError("zeros must be None for symmetric weights")
    else:
        if zeros is None:
            raise ValueError("asymmetric weights need zeros")
        _need(zeros, "zeros", (torch.float16,), (N, ng))
    return N, K, ng


def gq_dequantize(qweight: torch.Tensor, scales: torch.Tensor, zeros: Optional[torch.Tensor],
                  group_size: int = 128, symmetric: bool = False, out_dtype=torch.float32,
                  out=None, stream=None):
    """Packed INT4 -> W^ [N, K] in out_dtype (fp32 exact; bf16/fp16 nearest-even)."""
    N, K, _ = _weights(qweight, scales, zeros, group_size, symmetric)
    if out is not None:
        _need(out, "out", tuple(_DT), (N, K))
    _on_device(None, qweight=qweight)
    _on_device(qweight.device, scales=scales, zeros=zeros, out=out)
    if out is None:
        if out_dtype not in _DT:
            raise TypeError(f"out_dtype {out_dtype} not in {tuple(_DT)}")
        out = torch.empty((N, K), dtype=out_dtype, device=qweight.device)
    _ok(lib().gq_dequantize(_ptr(qweight), _ptr(scales), _ptr(zeros), N, K,
                            qparams(4, group_size, symmetric), _ptr(out), _DT[out.dtype],
                            _stream(stream)), "gq_dequantize")
    return out


def gq_w4a16_gemv_workspace_size(M: int, K: int, N: int, group_size: int = 128,
                                 symmetric: bool = False) -> int:
    """Bytes of scratch gq_w4a16_gemv_ws / gq_w4a16_gemv_f16_ws can use (0: none)."""
    b = ctypes.c_size_t()
    _ok(lib().gq_w4a16_gemv_workspace_size(M, K, N, qparams(4, group_size, symmetric),
                                           ctypes.byref(b)), "gq_w4a16_gemv_workspace_size")
    return int(b.value)


def gq_w4a16_gemm_workspace_size(M: int, K: int, N: int, group_size: int = 128,
                                 symmetric: bool = False) -> int:
    """Bytes of scratch gq_w4a16_gemm_ws / gq_w4a16_gemm_f16_ws can use (0: none).
    The size depends on the current device's compute-unit count."""
    b = ctypes.c_size_t()
    _ok(lib().gq_w4a16_gemm_workspace_size(M, K, N, qparams(4, group_size, symmetric),
                                           ctypes.byref(b)), "gq_w4a16_gemm_workspace_size")
    return int(b.value)


# workspace sizes of the shapes seen so far, per device: the query is a host
# call into the library, repeated for every matmul otherwise
_ws_sizes = {}


def _workspace_size(gemv: bool, dev, M, K, N, group_size, symmetric) -> int:
    key = (gemv, dev, M, K, N, group_size, bool(symmetric))
    n = _ws_sizes.get(key)
    if n is None:
        size = gq_w4a16_gemv_workspace_size if gemv else gq_w4a16_gemm_workspace_size
        n = _ws_sizes[key] = size(M, K, N, group_size, symmetric)
    return n


def _matmul(name, x, qweight, scales, zeros, group_size, symmetric, y, stream, workspace,
            xdtype, gemv):
    """Shared marshalling of the four fused matmuls.  A workspace the call can use
    comes from `workspace` (a uint8 GPU tensor of at least the queried size) or
    is allocated with torch on the call's stream, so the caching allocator hands
    that memory to other work only after the call's kernels (and, under stream
    capture, from the graph's own pool)."""
    _need(x, "x", (xdtype,))
    if x.dim() != 2:
        raise ValueError(f"x must be [M, K], got {tuple(x.shape)}")
    M, K = x.shape
    _need(qweight, "qweight", (torch.uint8,))
    if qweight.dim() != 2 or qweight.shape[1] * 2 != K:
        raise ValueError(f"qweight {tuple(qweight.shape)} does not match K={K}")
    N, _, _ = _weights(qweight, scales, zeros, group_size, symmetric)
    if gemv and M > 16:
        raise ValueError(f"the GEMV takes M <= 16, got M={M}")
    if y is not None:
        _need(y, "y", (xdtype,), (M, N))
    if workspace is not None:
        _need(workspace, "workspace", (torch.uint8,))
    _on_device(None, x=x)
    _on_device(x.device, qweight=qweight, scales=scales, zeros=zeros, y=y, workspace=workspace)
    need = _workspace_size(gemv, x.device, M, K, N, group_size, symmetric) if M > 0 and N > 0 else 0
    if workspace is not None and workspace.numel() < need:
        raise ValueError(f"workspace has {workspace.numel()} bytes, the call needs {need}")
    if y is None:
        y = torch.empty((M, N), dtype=xdtype, device=x.device)
    if need > 0 and workspace is None:
        if stream is not None and not hasattr(stream, "cuda_stream"):
            raise ValueError("with a raw stream handle the caller passes the workspace "
                             f"({need} bytes) that the call needs")
        if stream is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
        else:
            with torch.cuda.stream(stream):
                workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    fn = getattr(lib(), name + "_ws")
    _ok(fn(_ptr(x), M, K, _ptr(qweight), _ptr(scales), _ptr(zeros), N,
           qparams(4, group_size, symmetric), _ptr(y), _ptr(workspace),
           0 if workspace is None else workspace.numel(), _stream(stream)), name + "_ws")
    return y


def gq_w4a16_gemv(x, qweight, scales, zeros, group_size: int = 128, symmetric: bool = False,
                  y=None, stream=None, workspace=None):
    """Fused W4A16 GEMV, x bf16 [M<=16, K] -> y bf16 [M, N] (through gq_w4a16_gemv_ws)."""
    return _matmul("gq_w4a16_gemv", x, qweight, scales, zeros, group_size, symmetric, y, stream,
                   workspace, torch.bfloat16, True)


def gq_w4a16_gemm(x, qweight, scales, zeros, group_size: int = 128, symmetric: bool = False,
                  y=None, stream=None, workspace=None):
    """Fused W4A16 GEMM (bf16 MFMA), x bf16 [M, K] -> y bf16 [M, N] (through gq_w4a16_gemm_ws)."""
    return _matmul("gq_w4a16_gemm", x, qweight, scales, zeros, group_size, symmetric, y, stream,
                   workspace, torch.bfloat16, False)


def gq_w4a16_gemv_f16(x, qweight, scales, zeros, group_size: int = 128, symmetric: bool = False,
                      y=None, stream=None, workspace=None):
    """Fused W4A16 GEMV with fp16 activations, x fp16 [M<=16, K] -> y fp16 [M, N]."""
    return _matmul("gq_w4a16_gemv_f16", x, qweight, scales, zeros, group_size, symmetric, y, stream,
                   workspace, torch.float16, True)


def gq_w4a16_gemm_f16(x, qweight, scales, zeros, group_size: int = 128, symmetric: bool = False,
                      y=None, stream=None, workspace=None):
    """Fused W4A16 GEMM with fp16 activations (fp16 MFMA), x fp16 [M, K] -> y fp16 [M, N]."""
    return _matmul("gq_w4a16_gemm_f16", x, qweight, scales, zeros, group_size, symmetric, y, stream,
                   workspace, torch.float16, False)


def gq_w4a16_plain(name: str, x, qweight, scales, zeros, group_size: int = 128,
                   symmetric: bool = False, y=None, stream=None):
    """One of the entry points without a workspace (gq_w4a16_gemv, gq_w4a16_gemm
    or their _f16 forms), called as it is; for tests of those entry points."""
    xdtype = torch.float16 if name.endswith("_f16") else torch.bfloat16
    _need(x, "x", (xdtype,))
    M, K = x.shape
    N, Kw, _ = _weights(qweight, scales, zeros, group_size, symmetric)
    if Kw != K:
        raise ValueError(f"qweight {tuple(qweight.shape)} does not match K={K}")
    if y is not None:
        _need(y, "y", (xdtype,), (M, N))
    _on_device(None, x=x)
    _on_device(x.device, qweight=qweight, scales=scales, zeros=zeros, y=y)
    if y is None:
        y = torch.empty((M, N), dtype=xdtype, device=x.device)
    _ok(getattr(lib(), name)(_ptr(x), M, K, _ptr(qweight), _ptr(scales), _ptr(zeros), N,
                             qparams(4, group_size, symmetric), _ptr(y), _stream(stream)), name)
    return y


def gq_w4a16_gemm_noalloc(x, qweight, scales, zeros, group_size: int = 128, symmetric: bool = False,
                          y=None, stream=None):
    """gq_w4a16_gemm with its split scratch in the library's fixed device array
    (no allocation by the call; calls that overlap on one GPU race)."""
    return gq_w4a16_plain("gq_w4a16_gemm_noalloc", x, qweight, scales, zeros, group_size, symmetric,
                          y, stream)


def gq_q4k_quantize(w: torch.Tensor, blocks=None, stream=None):
    """w [N, K] (K % 256 == 0) -> blocks uint8 [N, K/256, 144]."""
    _need(w, "w", tuple(_DT))
    if w.dim() != 2 or w.shape[1] % 256:
        raise ValueError(f"w must be [N, K] with K % 256 == 0, got {tuple(w.shape)}")
    N, K = w.shape
    if blocks is not None:
        _need(blocks, "blocks", (torch.uint8,), (N, K // 256, 144))
    _on_device(None, w=w)
    _on_device(w.device, blocks=blocks)
    if blocks is None:
        blocks = torch.empty((N, K // 256, 144), dtype=torch.uint8, device=w.device)
    _ok(lib().gq_q4k_quantize(_ptr(w), _DT[w.dtype], N, K, _ptr(blocks), _stream(stream)),
        "gq_q4k_quantize")
    return blocks


def gq_q4k_gemv(x: torch.Tensor, blocks: torch.Tensor, y=None, stream=None):
    """Fused GEMV over super-block weights, x bf16 [M<=16, K] -> y bf16 [M, N]."""
    _need(x, "x", (torch.bfloat16,))
    if x.dim() != 2:
        raise ValueError(f"x must be [M, K], got {tuple(x.shape)}")
    M, K = x.shape
    if K % 256:
        raise ValueError(f"K={K} must be a multiple of 256")
    _need(blocks, "blocks", (torch.uint8,))
    if blocks.dim() != 3 or blocks.shape[1] * 256 != K or blocks.shape[2] != 144:
        raise ValueError(f"blocks has shape {tuple(blocks.shape)}, expected (N, {K // 256}, 144)")
    N = blocks.shape[0]
    if y is not None:
        _need(y, "y", (torch.bfloat16,), (M, N))
    _on_device(None, x=x)
    _on_device(x.device, blocks=blocks, y=y)
    if y is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    _ok(lib().gq_q4k_gemv(_ptr(x), M, K, _ptr(blocks), N, _ptr(y), _stream(stream)), "gq_q4k_gemv")
    return y


def gq_bf16_gemv(x: torch.Tensor, w: torch.Tensor, y=None, stream=None):
    """Plain bf16 GEMV (the 16-bit comparator), x bf16 [M<=4, K], w bf16 [N, K] -> y bf16 [M, N]."""
    _need(x, "x", (torch.bfloat16,))
    M, K = x.shape
    _need(w, "w", (torch.bfloat16,))
    if w.dim() != 2 or w.shape[1] != K:
        raise ValueError(f"w is {tuple(w.shape)}, expected [N, {K}]")
    N = w.shape[0]
    if y is not None:
        _need(y, "y", (torch.bfloat16,), (M, N))
    _on_device(None, x=x)
    _on_device(x.device, w=w, y=y)
    if y is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    _ok(lib().gq_bf16_gemv(_ptr(x), M, K, _ptr(w), N, _ptr(y), _stream(stream)), "gq_bf16_gemv")
    return y


def gq_stream_read(buf: torch.Tensor, sink: torch.Tensor, stream=None) -> None:
    """Read every byte of the contiguous GPU tensor buf once (bandwidth probe);
    sink is a GPU int32/uint32 tensor of at least one element that the kernel may write."""
    if not isinstance(buf, torch.Tensor) or not buf.is_contiguous():
        raise ValueError("buf must be a contiguous tensor")
    _need(sink, "sink", (torch.int32, torch.uint32))
    if sink.numel() < 1:
        raise ValueError("sink needs at least one element")
    _on_device(None, buf=buf)
    _on_device(buf.device, sink=sink)
    nbytes = buf.numel() * buf.element_size()
    _ok(lib().gq_stream_read(_ptr(buf), nbytes, _ptr(sink), _stream(stream)), "gq_stream_read")


def gq_probe_mfma_valu(valu: int, iters: int, grid: int, stream=None) -> torch.Tensor:
    """Per-wave loop cycles [grid * 8] (int64, on the current device) of the
    matrix-core / vector-ALU issue probe (include/gq_bench.h)."""
    dev = torch.device("cuda", torch.cuda.current_device())
    cycles = torch.zeros(grid * 8, dtype=torch.int64, device=dev)
    sink = torch.zeros(1, dtype=torch.float32, device=dev)
    _ok(lib().gq_probe_mfma_valu(valu, iters, grid, _ptr(cycles), _ptr(sink), _stream(stream)),
        "gq_probe_mfma_valu")
    return cycles


def gq_probe_lds_read(waves: int, iters: int, grid: int, stream=None) -> torch.Tensor:
    """Per-wave loop cycles [grid * waves] (int64, on the current device) of the
    LDS read probe (include/gq_bench.h)."""
    dev = torch.device("cuda", torch.cuda.current_device())
    cycles = torch.zeros(grid * waves, dtype=torch.int64, device=dev)
    sink = torch.zeros(1, dtype=torch.float32, device=dev)
    _ok(lib().gq_probe_lds_read(waves, iters, grid, _ptr(cycles), _ptr(sink), _stream(stream)),
        "gq_probe_lds_read")
    return cycles


def gq_ingest_group_major(codes: torch.Tensor, scales: torch.Tensor, qweight=None, scales_out=None,
                          stream=None):
    """Group-major codes int8 [n_groups, group, N] + scales fp16 [n_groups, N] ->
    (qweight uint8 [N, K/2], scales fp16 [N, n_groups]), symmetric, K = n_groups * group."""
    _need(codes, "codes", (torch.int8,))
    if codes.dim() != 3:
        raise ValueError(f"codes must be [n_groups, group, N], got {tuple(codes.shape)}")
    ng, g, N = codes.shape
    _need(scales, "scales", (torch.float16,), (ng, N))
    if qweight is not None:
        _need(qweight, "qweight", (torch.uint8,), (N, ng * g // 2))
    if scales_out is not None:
        _need(scales_out, "scales_out", (torch.float16,), (N, ng))
    _on_device(None, codes=codes)
    _on_device(codes.device, scales=scales, qweight=qweight, scales_out=scales_out)
    if qweight is None:
        qweight = torch.empty((N, ng * g // 2), dtype=torch.uint8, device=codes.device)
    if scales_out is None:
        scales_out = torch.empty((N, ng), dtype=torch.float16, device=codes.device)
    _ok(lib().gq_ingest_group_major(_ptr(codes), _ptr(scales), ng, g, N, _ptr(qweight),
                                    _ptr(scales_out), _stream(stream)), "gq_ingest_group_major")
    return qweight, scales_out


# ---------------------------------------------------------------------------
# The 4-bit key/value cache (include/gq_kv.h)
# ---------------------------------------------------------------------------

_KV_DIMS = (64, 96, 128, 256)


def _kv4_block_bytes(head_dim: int, group_size: int, symmetric: bool) -> int:
    """Bytes of 16 tokens of one head: keys and values, codes and parameters."""
    return 2 * (8 * head_dim + 16 * (head_dim // group_size) * (2 if symmetric else 4))


def _kv4_shape(head_dim: int, group_size: int) -> None:
    if head_dim not in _KV_DIMS:
        raise ValueError(f"head_dim {head_dim} not in {_KV_DIMS}")
    if group_size < 32 or group_size % 32 or head_dim % group_size:
        raise ValueError(f"group_size {group_size} must be a multiple of 32 that divides "
                         f"head_dim={head_dim}")


def gq_kv4_empty(n_pages: int, kv_heads: int, head_dim: int, page_size: int = 64,
                 group_size: int = 128, symmetric: bool = False, device="cuda") -> torch.Tensor:
    """A cache of n_pages pages of page_size tokens: uint8 [n_pages, kv_heads,
    page_size / 16, bytes of 16 tokens], uninitialised.  The shape carries what
    the other calls need; the bytes are the library's own (gq_kv4_write and
    gq_kv4_read are the way in and out)."""
    _kv4_shape(head_dim, group_size)
    if page_size < 16 or page_size > 1024 or page_size & (page_size - 1):
        raise ValueError(f"page_size {page_size} must be a power of two in 16..1024")
    if n_pages < 1 or kv_heads < 1:
        raise ValueError("n_pages and kv_heads must be positive")
    return torch.empty((n_pages, kv_heads, page_size // 16,
                        _kv4_block_bytes(head_dim, group_size, symmetric)),
                       dtype=torch.uint8, device=device)


# layouts of the cache shapes seen so far (checked once each)
_kv4_layouts = {}


def _kv4_cache(cache, head_dim: int, group_size: int, symmetric: bool):
    """Check a cache against head_dim and the quantisation; its layout."""
    _need(cache, "cache", (torch.uint8,))
    key = (cache.shape, head_dim, group_size, bool(symmetric))
    lay = _kv4_layouts.get(key)
    if lay is None:
        lay = _kv4_layouts[key] = _kv4_layout(cache, head_dim, group_size, symmetric)
    return lay


def _kv4_layout(cache, head_dim: int, group_size: int, symmetric: bool):
    _kv4_shape(head_dim, group_size)
    blk = _kv4_block_bytes(head_dim, group_size, symmetric)
    if cache.dim() != 4 or cache.shape[3] != blk:
        raise ValueError(f"cache has shape {tuple(cache.shape)}, expected (n_pages, kv_heads, "
                         f"page_size / 16, {blk}) for head_dim {head_dim}, group_size {group_size}, "
                         f"symmetric {bool(symmetric)}")
    return GqKv4Layout(cache.shape[1], head_dim, cache.shape[2] * 16, group_size, int(bool(symmetric)))


def _rows16(t, name: str, dtypes, heads=None, dim=None):
    """A [tokens, heads, dim] tensor whose rows of `dim` are contiguous and
    16-byte aligned (a slice of a projection's output); its two strides."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype} not in {dtypes}")
    shape = t.shape
    if len(shape) != 3 or (heads is not None and shape[1] != heads) or \
            (dim is not None and shape[2] != dim):
        raise ValueError(f"{name} has shape {tuple(shape)}, expected (tokens, "
                         f"{'heads' if heads is None else heads}, {'dim' if dim is None else dim})")
    # the stride of a dimension of one element is never walked
    ts, hs, ds = t.stride()
    ts = ts if shape[0] > 1 else 0
    hs = hs if shape[1] > 1 else 0
    if (shape[2] > 1 and ds != 1) or ts % 8 or hs % 8:
        raise ValueError(f"{name}: strides {t.stride()}; the last must be 1, the others multiples of 8")
    return ts, hs


def _slots(slots, tokens: int) -> None:
    _need(slots, "slots", (torch.int64,), (tokens,))


def gq_kv4_write(k: torch.Tensor, v: torch.Tensor, cache: torch.Tensor, slots: torch.Tensor,
                 group_size: int = 128, symmetric: bool = False, stream=None) -> None:
    """Quantise k, v [tokens, kv_heads, head_dim] (bf16 or fp16; views with
    contiguous rows are taken as they are) into the cache at the given slots
    (int64; page * page_size + place, out of range: skipped)."""
    kts, khs = _rows16(k, "k", (torch.bfloat16, torch.float16))
    T, H, D = k.shape
    vts, vhs = _rows16(v, "v", (k.dtype,), H, D)
    if v.shape[0] != T:
        raise ValueError(f"v has {v.shape[0]} tokens, k has {T}")
    lay = _kv4_cache(cache, D, group_size, symmetric)
    if lay.kv_heads != H:
        raise ValueError(f"cache has {lay.kv_heads} heads, k has {H}")
    _slots(slots, T)
    _on_device(None, k=k)
    _on_device(k.device, v=v, cache=cache, slots=slots)
    _ok(lib().gq_kv4_write(_ptr(k), kts, khs, _ptr(v), vts, vhs, _DT[k.dtype], T, _ptr(slots),
                           _ptr(cache), cache.shape[0], lay, _stream(stream)), "gq_kv4_write")


def gq_kv4_read(cache: torch.Tensor, slots: torch.Tensor, head_dim: int, group_size: int = 128,
                symmetric: bool = False, out_dtype=torch.bfloat16, k=None, v=None, stream=None):
    """(k, v) [tokens, kv_heads, head_dim] in out_dtype: the values that the cache
    stands for at the given slots (fp32 exact; a slot out of range: zeros)."""
    lay = _kv4_cache(cache, head_dim, group_size, symmetric)
    if not isinstance(slots, torch.Tensor) or slots.dim() != 1:
        raise ValueError("slots must be a 1-D tensor")
    _slots(slots, slots.shape[0])
    shape = (slots.shape[0], lay.kv_heads, head_dim)
    if out_dtype not in _DT:
        raise TypeError(f"out_dtype {out_dtype} not in {tuple(_DT)}")
    for name, t in (("k", k), ("v", v)):
        if t is not None:
            _need(t, name, (out_dtype,), shape)
    _on_device(None, cache=cache)
    _on_device(cache.device, slots=slots, k=k, v=v)
    if k is None:
        k = torch.empty(shape, dtype=out_dtype, device=cache.device)
    if v is None:
        v = torch.empty_like(k)
    _ok(lib().gq_kv4_read(_ptr(cache), cache.shape[0], lay, _ptr(slots), slots.shape[0], _ptr(k),
                          _ptr(v), _DT[out_dtype], _stream(stream)), "gq_kv4_read")
    return k, v


def gq_kv4_attention_workspace_size(batch: int, q_heads: int, kv_heads: int, head_dim: int,
                                    max_q_len: int, max_kv_len: int) -> int:
    """Bytes of scratch gq_kv4_attention can use (0: none).  Depends on the
    current device's compute-unit count."""
    a = GqKv4AttentionArgs()
    a.layout = GqKv4Layout(kv_heads, head_dim, 16, head_dim, 0)
    a.q_heads, a.batch, a.q_tokens, a.n_pages = q_heads, batch, max(batch, 1), 1
    a.max_q_len, a.max_kv_len, a.scale, a.dtype = max_q_len, max_kv_len, 1.0, GQ_BF16
    b = ctypes.c_size_t()
    _ok(lib().gq_kv4_attention_workspace_size(ctypes.byref(a), ctypes.byref(b)),
        "gq_kv4_attention_workspace_size")
    return int(b.value)


def gq_kv4_attention(q: torch.Tensor, cache: torch.Tensor, page_table: torch.Tensor,
                     kv_lens: torch.Tensor, group_size: int = 128, symmetric: bool = False,
                     q_starts: Optional[torch.Tensor] = None, max_q_len: Optional[int] = None,
                     max_kv_len: Optional[int] = None, causal: bool = True, window: int = 0,
                     scale: Optional[float] = None, return_lse: bool = False, out=None, lse=None,
                     stream=None, workspace=None):
    """Attention of q [tokens, q_heads, head_dim] (bf16 or fp16) over the cache.

    Sequence b owns the query rows q_starts[b] .. q_starts[b + 1] - 1 (row b
    where q_starts is None), its keys are the first kv_lens[b] tokens of its row
    of page_table [batch, pages] (all int32, on the GPU).  Its last query stands
    at the last key; with `causal` a query sees the keys up to its own position,
    with `window` > 0 only the last `window` of them.  A query without keys gives
    zeros and lse = -inf.  max_q_len and max_kv_len bound the lengths for the
    choice of kernels (default: 1 or the number of tokens, and the whole table);
    scale defaults to 1 / sqrt(head_dim).  Returns out, or (out, lse) with the
    natural-log sums [tokens, q_heads] in fp32."""
    qts, qhs = _rows16(q, "q", (torch.bfloat16, torch.float16))
    T, HQ, D = q.shape
    lay = _kv4_cache(cache, D, group_size, symmetric)
    if HQ % lay.kv_heads:
        raise ValueError(f"{HQ} query heads are not a multiple of {lay.kv_heads} key/value heads")
    _need(page_table, "page_table", (torch.int32,))
    if page_table.dim() != 2:
        raise ValueError(f"page_table must be [batch, pages], got {tuple(page_table.shape)}")
    nb = page_table.shape[0]
    _need(kv_lens, "kv_lens", (torch.int32,), (nb,))
    if q_starts is not None:
        _need(q_starts, "q_starts", (torch.int32,), (nb + 1,))
    elif T != nb:
        raise ValueError(f"q has {T} tokens for {nb} sequences; more than one each needs q_starts")
    if out is not None:
        _need(out, "out", (q.dtype,), (T, HQ, D))
    if lse is not None:
        _need(lse, "lse", (torch.float32,), (T, HQ))
    if workspace is not None:
        _need(workspace, "workspace", (torch.uint8,))
    if max_q_len is None:
        max_q_len = 1 if q_starts is None else T
    if max_kv_len is None:
        max_kv_len = page_table.shape[1] * lay.page_size
    _on_device(None, q=q)
    _on_device(q.device, cache=cache, page_table=page_table, kv_lens=kv_lens, q_starts=q_starts,
               out=out, lse=lse, workspace=workspace)
    if out is None:
        out = q.new_empty((T, HQ, D))
    if lse is None and return_lse:
        lse = torch.empty((T, HQ), dtype=torch.float32, device=q.device)
    a = GqKv4AttentionArgs(
        q.data_ptr(), qts, qhs, T, HQ, _DT[q.dtype], cache.data_ptr(), cache.shape[0], lay,
        page_table.data_ptr(), nb, page_table.shape[1], kv_lens.data_ptr(),
        None if q_starts is None else q_starts.data_ptr(), int(max_q_len), int(max_kv_len),
        int(bool(causal)), int(window), D ** -0.5 if scale is None else float(scale), out.data_ptr(),
        None if lse is None else lse.data_ptr())
    ref = ctypes.byref(a)
    size = ctypes.c_size_t()
    L = lib()
    _ok(L.gq_kv4_attention_workspace_size(ref, ctypes.byref(size)), "gq_kv4_attention_workspace_size")
    need = size.value
    if workspace is not None and workspace.numel() < need:
        raise ValueError(f"workspace has {workspace.numel()} bytes, the call needs {need}")
    if need > 0 and workspace is None:
        if stream is not None and not hasattr(stream, "cuda_stream"):
            raise ValueError("with a raw stream handle the caller passes the workspace "
                             f"({need} bytes) that the call needs")
        if stream is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        else:
            with torch.cuda.stream(stream):
                workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    _ok(L.gq_kv4_attention(ref, _ptr(workspace), 0 if workspace is None else workspace.numel(),
                           _stream(stream)), "gq_kv4_attention")
    return (out, lse) if return_lse else out
