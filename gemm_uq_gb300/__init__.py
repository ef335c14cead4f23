"""Python binding of the uq C-ABI library (include/uq.h): argument marshalling only.

Every function here forwards torch tensors' device pointers, sizes and the current CUDA
stream to the same-named ``extern "C"`` entry point of ``libuq.so`` and raises
``UqError`` on a non-OK status.  With ``stream=`` a call runs on that stream, and its result comes
from that stream's memory pool.  No step of the computation runs in Python or in
PyTorch: if the library is missing, importing the ops raises instead of falling back.
"""
from __future__ import annotations

import ctypes
import os

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libuq.so")

FORMATS = {"INT4_SYM": 0, "INT4_ASYM": 1, "INT8_SYM": 2, "INT2_ASYM": 3, "NF4": 4, "K4": 5}
BITS = {"INT4_SYM": 4, "INT4_ASYM": 4, "INT8_SYM": 8, "INT2_ASYM": 2, "NF4": 4, "K4": 4}

# every entry point declared in include/uq.h: name -> (restype, argtypes)
_P, _I, _SZ = ctypes.c_void_p, ctypes.c_int, ctypes.POINTER(ctypes.c_size_t)
_L, _F = ctypes.c_longlong, ctypes.c_float
SIGNATURES = {
    "uq_status_string": (ctypes.c_char_p, [_I]),
    "uq_last_error": (ctypes.c_char_p, []),
    "uq_packed_size": (_I, [_I, _I, _I, _I, _SZ, _SZ, _SZ]),
    "uq_pack_layout": (_I, [_P, _P, _I, _I, _I, _I, _P]),
    "uq_pack_kmeta": (_I, [_P, _P, _P, _P, _P, _I, _I, _P]),
    "uq_gemm": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P]),
    "uq_unpack_codes": (_I, [_P, _P, _I, _I, _I, _I, _P]),
    "uq_dequant": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _P]),
    "uq_quantize": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _P]),
    "uq_quantize_k4": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _P]),
    "uq_pack_zeros": (_I, [_P, _P, _I, _I, _P]),
    "uq_device_fault": (_I, [ctypes.POINTER(ctypes.c_uint)]),
    "uq_gemm_noalloc": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P]),
    "uq_gemm_noalloc_scratch": (_I, [_I, _I, _I, _I, _I, _SZ, _SZ]),
    "uq_set_launch_overlap": (_I, [_I]),
    "uq_set_gemm_path": (_I, [_I]),
    "uq_gemm_kernel_count": (_I, [_I, _I, _I, _I, _I, ctypes.POINTER(_I)]),
    "uq_gemm_gated": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P]),
    "uq_gemm_gated_kernel_count": (_I, [_I, _I, _I, _I, _I, ctypes.POINTER(_I)]),
    "uq_pack_gguf": (_I, [_P, _I, _P, _P, _I, _I, _P]),
    "uq_gemm_w4a8": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P]),
    "uq_gemm_w4a8_kernel_count": (_I, [_I, _I, _I, _I, _I, ctypes.POINTER(_I)]),
    "uq_rope_table": (_I, [_P, _I, _I, ctypes.c_double, _P]),
    "uq_rmsnorm_rope": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, ctypes.c_float, _P]),
    "uq_mx_scales_size": (_I, [_I, _I, _I, _I, _SZ]),
    "uq_pack_mx_scales": (_I, [_P, _P, _I, _I, _I, _I, _P]),
    "uq_quantize_mx": (_I, [_P, _I, _L, _P, _P, _I, _I, _I, _F, _P, _I, _P, _I, _P]),
    "uq_dequant_mx": (_I, [_P, _P, _P, _I, _I, _I, _I, _F, _P, _I, _P]),
    "uq_gemm_mx": (_I, [_P, _I, _L, _P, _F, _P, _P, _P, _I, _I, _I, _I, _I, _F, _P]),
    "uq_gemm_mx_grouped": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P]),
    "uq_moe_sort": (_I, [_P, _I, _I, _I, _P, _P, _P, _P]),
    "uq_moe_gather": (_I, [_P, _I, _P, _P, _I, _P, _I, _I, _I, _P]),
    "uq_moe_gather_grad": (_I, [_P, _I, _P, _P, _I, _I, _I, _P]),
    "uq_moe_combine": (_I, [_P, _I, _P, _P, _P, _I, _I, _I, _P]),
    "uq_moe_combine_grad": (_I, [_P, _P, _I, _P, _P, _P, _I, _P, _P, _I, _I, _I, _P]),
}

_lib = None


class UqError(RuntimeError):
    def __init__(self, status: int, where: str, msg: str):
        super().__init__(f"{where}: status {status} ({msg})")
        self.status = status


def lib() -> ctypes.CDLL:
    """The loaded libuq.so (raises if it has not been built: there is no fallback)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with `python -m gemm_uq_gb300.build` "
                              "(the quantized GEMV has no non-CUDA implementation)")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _check(status: int, where: str):
    if status != 0:
        L = lib()
        raise UqError(status, where, f"{L.uq_status_string(status).decode()}: {L.uq_last_error().decode()}")


def _ptr(t):
    if t is None:
        return None
    assert t.is_cuda and t.is_contiguous(), "tensors passed to uq must be contiguous CUDA tensors"
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _empty(shape, dtype: torch.dtype, device, stream=None) -> torch.Tensor:
    """A result's memory, from the pool of the stream that writes it: memory of the current stream's pool may still
    be in use by work queued there, and may be given out again there while the given stream writes it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def packed_size(N: int, K: int, group: int, fmt: str):
    """(wq_bytes, scales_bytes, zeros_bytes) -- host only."""
    a, b, c = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib().uq_packed_size(N, K, group, FORMATS[fmt], ctypes.byref(a), ctypes.byref(b), ctypes.byref(c)),
           "uq_packed_size")
    return a.value, b.value, c.value


def pack_layout(codes: torch.Tensor, group: int, fmt: str, stream=None) -> torch.Tensor:
    """int8 codes [N][K] (device) -> packed uint8 plane (synchronizes the stream)."""
    N, K = codes.shape
    wq_bytes, _, _ = packed_size(N, K, group, fmt)
    wq = _empty(max(wq_bytes, 16), torch.uint8, codes.device, stream)
    _check(lib().uq_pack_layout(_ptr(codes), _ptr(wq), N, K, group, FORMATS[fmt], _stream(stream)),
           "uq_pack_layout")
    return wq


GGUF_TYPES = {"Q4_0": (0, "INT4_SYM"), "Q8_0": (1, "INT8_SYM")}


def pack_gguf(blocks: torch.Tensor, qtype: str, N: int, K: int, stream=None):
    """uq_pack_gguf: GGUF Q4_0 / Q8_0 block bytes (device uint8) -> (wq, scales) of INT4_SYM / INT8_SYM, group 32."""
    t, fmt = GGUF_TYPES[qtype]
    wq_bytes, sc_bytes, _ = packed_size(N, K, 32, fmt)
    wq = _empty(max(wq_bytes, 16), torch.uint8, blocks.device, stream)
    scales = _empty((N, K // 32), torch.int16, blocks.device, stream)
    assert blocks.is_cuda and blocks.is_contiguous()
    _check(lib().uq_pack_gguf(ctypes.c_void_p(blocks.data_ptr()), t, _ptr(wq), _ptr(scales), N, K, _stream(stream)),
           "uq_pack_gguf")
    return wq, scales


def pack_kmeta(d, dmin, sc, m, stream=None) -> torch.Tensor:
    """K4 fp16 d, dmin [N][S] (as int16/uint16/float16 tensors), uint8 sc, m [N][S][8] -> records [N][S][16]."""
    N, S = d.shape
    meta = _empty((N, S, 16), torch.uint8, d.device, stream)
    _check(lib().uq_pack_kmeta(_ptr(d), _ptr(dmin), _ptr(sc), _ptr(m), _ptr(meta), N, S * 256, _stream(stream)),
           "uq_pack_kmeta")
    return meta


def pack_zeros(z: torch.Tensor, stream=None) -> torch.Tensor:
    """INT4_ASYM zeros, one per byte [N][G] -> two per byte [N][ceil(G/2)]."""
    N, G = z.shape
    out = _empty((N, (G + 1) // 2), torch.uint8, z.device, stream)
    _check(lib().uq_pack_zeros(_ptr(z), _ptr(out), N, G, _stream(stream)), "uq_pack_zeros")
    return out


def gemm(x: torch.Tensor, wq: torch.Tensor, scales: torch.Tensor, zc, N: int, group: int, fmt: str,
         y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y = x . W_hat^T (bf16 [M][N]) with W_hat dequantized on the fly."""
    M, K = x.shape
    assert x.dtype == torch.bfloat16
    if y is None:
        y = _empty((M, N), torch.bfloat16, x.device, stream)
    _check(lib().uq_gemm(_ptr(x), _ptr(wq), _ptr(scales), _ptr(zc), _ptr(y), M, N, K, group, FORMATS[fmt],
                         _stream(stream)), "uq_gemm")
    return y


def gemm_gated(x: torch.Tensor, gate: tuple, up: tuple, N: int, group: int, fmt: str,
               h: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """h = silu(x . W_gate_hat^T) * (x . W_up_hat^T) (bf16 [M][N]); gate and up are (wq, scales, zc)."""
    M, K = x.shape
    assert x.dtype == torch.bfloat16
    if h is None:
        h = _empty((M, N), torch.bfloat16, x.device, stream)
    (wg, sg, zg), (wu, su, zu) = gate, up
    _check(lib().uq_gemm_gated(_ptr(x), _ptr(wg), _ptr(sg), _ptr(zg), _ptr(wu), _ptr(su), _ptr(zu), _ptr(h),
                               M, N, K, group, FORMATS[fmt], _stream(stream)), "uq_gemm_gated")
    return h


def gemm_gated_ptrs(x_ptr: int, gate: tuple, up: tuple, h_ptr: int, M: int, N: int, K: int, group: int, fmt: str,
                    stream_handle: int) -> None:
    """Raw-pointer form of uq_gemm_gated; gate and up are (wq_ptr, scales_ptr, zc_ptr or 0)."""
    P = ctypes.c_void_p
    _check(lib().uq_gemm_gated(P(x_ptr), P(gate[0]), P(gate[1]), P(gate[2]) if gate[2] else None, P(up[0]),
                               P(up[1]), P(up[2]) if up[2] else None, P(h_ptr), M, N, K, group, FORMATS[fmt],
                               P(stream_handle)), "uq_gemm_gated")


def gemm_gated_kernel_count(M: int, N: int, K: int, group: int, fmt: str) -> int:
    v = ctypes.c_int(0)
    _check(lib().uq_gemm_gated_kernel_count(M, N, K, group, FORMATS[fmt], ctypes.byref(v)),
           "uq_gemm_gated_kernel_count")
    return v.value


def rope_table(max_pos: int, head_dim: int, base: float, device=None, stream=None) -> torch.Tensor:
    """uq_rope_table: fp32 [max_pos][head_dim/2][2] (cos, sin) on the device."""
    t = _empty((max_pos, head_dim // 2, 2), torch.float32, device or "cuda", stream)
    _check(lib().uq_rope_table(_ptr(t), max_pos, head_dim, float(base), _stream(stream)), "uq_rope_table")
    return t


def rmsnorm_rope(x: torch.Tensor, gamma: torch.Tensor, pos: torch.Tensor, table: torch.Tensor, head_dim: int,
                 eps: float, y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """uq_rmsnorm_rope: y = RoPE(RMSNorm(x) * gamma, pos) (bf16 [M][D]); y may be x."""
    M, D = x.shape
    assert x.dtype == torch.bfloat16 and gamma.dtype == torch.bfloat16 and pos.dtype == torch.int32
    if y is None:
        y = _empty(x.shape, x.dtype, x.device, stream)
    _check(lib().uq_rmsnorm_rope(_ptr(x), _ptr(gamma), _ptr(pos), _ptr(table), _ptr(y), M, D, head_dim,
                                 table.shape[0], float(eps), _stream(stream)), "uq_rmsnorm_rope")
    return y


def gemm_w4a8(x: torch.Tensor, wq: torch.Tensor, scales: torch.Tensor, zc, N: int, group: int, fmt: str,
              y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """uq_gemm_w4a8: y with x quantized per row to int8 and integer dot products (bf16 [M][N])."""
    M, K = x.shape
    assert x.dtype == torch.bfloat16
    if y is None:
        y = _empty((M, N), torch.bfloat16, x.device, stream)
    _check(lib().uq_gemm_w4a8(_ptr(x), _ptr(wq), _ptr(scales), _ptr(zc), _ptr(y), M, N, K, group, FORMATS[fmt],
                              _stream(stream)), "uq_gemm_w4a8")
    return y


def gemm_w4a8_ptrs(x_ptr: int, wq_ptr: int, scales_ptr: int, zc_ptr, y_ptr: int, M: int, N: int, K: int, group: int,
                   fmt: str, stream_handle: int) -> None:
    P = ctypes.c_void_p
    _check(lib().uq_gemm_w4a8(P(x_ptr), P(wq_ptr), P(scales_ptr), P(zc_ptr) if zc_ptr else None, P(y_ptr), M, N, K,
                              group, FORMATS[fmt], P(stream_handle)), "uq_gemm_w4a8")


def gemm_w4a8_kernel_count(M: int, N: int, K: int, group: int, fmt: str) -> int:
    v = ctypes.c_int(0)
    _check(lib().uq_gemm_w4a8_kernel_count(M, N, K, group, FORMATS[fmt], ctypes.byref(v)), "uq_gemm_w4a8_kernel_count")
    return v.value


def gemm_noalloc(x: torch.Tensor, wq: torch.Tensor, scales: torch.Tensor, zc, N: int, group: int, fmt: str,
                 y: torch.Tensor, stream=None) -> torch.Tensor:
    """uq_gemm_noalloc: the GEMV with the library's static scratch (y must be given: nothing is allocated)."""
    M, K = x.shape
    _check(lib().uq_gemm_noalloc(_ptr(x), _ptr(wq), _ptr(scales), _ptr(zc), _ptr(y), M, N, K, group, FORMATS[fmt],
                                 _stream(stream)), "uq_gemm_noalloc")
    return y


def gemm_noalloc_scratch(M: int, N: int, K: int, group: int, fmt: str):
    """uq_gemm_noalloc_scratch: (ticket_bytes, partial_bytes) of the static scratch the call would use
    (host only; 0, 0 when every worker owns whole row blocks)."""
    t, p = ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib().uq_gemm_noalloc_scratch(M, N, K, group, FORMATS[fmt], ctypes.byref(t), ctypes.byref(p)),
           "uq_gemm_noalloc_scratch")
    return t.value, p.value


def gemm_ptrs(x_ptr: int, wq_ptr: int, scales_ptr: int, zc_ptr, y_ptr: int, M: int, N: int, K: int, group: int,
              fmt: str, stream_handle: int) -> None:
    """Raw-pointer form of uq_gemm (for graph capture loops that pre-compute pointers)."""
    _check(lib().uq_gemm(ctypes.c_void_p(x_ptr), ctypes.c_void_p(wq_ptr), ctypes.c_void_p(scales_ptr),
                         ctypes.c_void_p(zc_ptr) if zc_ptr else None, ctypes.c_void_p(y_ptr), M, N, K, group,
                         FORMATS[fmt], ctypes.c_void_p(stream_handle)), "uq_gemm")


def unpack_codes(wq: torch.Tensor, N: int, K: int, group: int, fmt: str, stream=None) -> torch.Tensor:
    codes = _empty((N, K), torch.int8, wq.device, stream)
    _check(lib().uq_unpack_codes(_ptr(wq), _ptr(codes), N, K, group, FORMATS[fmt], _stream(stream)),
           "uq_unpack_codes")
    return codes


def dequant(wq: torch.Tensor, scales: torch.Tensor, zc, N: int, K: int, group: int, fmt: str,
            stream=None) -> torch.Tensor:
    w = _empty((N, K), torch.float32, wq.device, stream)
    _check(lib().uq_dequant(_ptr(wq), _ptr(scales), _ptr(zc), _ptr(w), N, K, group, FORMATS[fmt],
                            _stream(stream)), "uq_dequant")
    return w


def quantize(w: torch.Tensor, group: int, fmt: str, codebook: torch.Tensor | None = None, stream=None):
    """GPU quantizer for the flat formats: returns (codes int8 [N][K], scales fp16 bits [N][G], zeros)."""
    N, K = w.shape
    G = K // group if group else 0
    codes = _empty((N, K), torch.int8, w.device, stream)
    scales = _empty((N, G), torch.int16, w.device, stream)
    zeros = None
    if fmt == "INT4_ASYM":
        zeros = _empty((N, G), torch.uint8, w.device, stream)
    elif fmt == "INT2_ASYM":
        zeros = _empty((N, G), torch.int16, w.device, stream)
    _check(lib().uq_quantize(_ptr(w), _ptr(codes), _ptr(scales), _ptr(zeros), _ptr(codebook), N, K, group,
                             FORMATS[fmt], _stream(stream)), "uq_quantize")
    return codes, scales, zeros


def quantize_k4(w: torch.Tensor, stream=None):
    """GPU K4 quantizer: returns (codes, d, dmin, sc, m)."""
    N, K = w.shape
    S = K // 256
    dev = w.device
    codes = _empty((N, K), torch.int8, dev, stream)
    d = _empty((N, S), torch.int16, dev, stream)
    dmin = _empty((N, S), torch.int16, dev, stream)
    sc = _empty((N, S, 8), torch.uint8, dev, stream)
    m = _empty((N, S, 8), torch.uint8, dev, stream)
    _check(lib().uq_quantize_k4(_ptr(w), _ptr(codes), _ptr(d), _ptr(dmin), _ptr(sc), _ptr(m), N, K,
                                _stream(stream)), "uq_quantize_k4")
    return codes, d, dmin, sc, m


def set_launch_overlap(enable: bool) -> None:
    """uq_set_launch_overlap: let GEMV, GEMM and microscaled launches prefetch their (constant) weights early."""
    _check(lib().uq_set_launch_overlap(1 if enable else 0), "uq_set_launch_overlap")


GEMM_PATHS = {"auto": 0, "tensor_cores": 1, "mma": 2}


def set_gemm_path(path: str) -> None:
    """uq_set_gemm_path: "auto" (default), "tensor_cores" (the tcgen05 kernel for every block of 16..64
    rows it supports) or "mma" (the mma.sync GEMM for every block of 9..64 rows of a 4-bit / 2-bit format)."""
    _check(lib().uq_set_gemm_path(GEMM_PATHS[path]), "uq_set_gemm_path")


def gemm_kernel_count(M: int, N: int, K: int, group: int, fmt: str) -> int:
    """uq_gemm_kernel_count: kernels one gemm() call of this shape launches on the current device."""
    v = ctypes.c_int(0)
    _check(lib().uq_gemm_kernel_count(M, N, K, group, FORMATS[fmt], ctypes.byref(v)), "uq_gemm_kernel_count")
    return v.value


def device_fault() -> int:
    v = ctypes.c_uint(0)
    _check(lib().uq_device_fault(ctypes.byref(v)), "uq_device_fault")
    return v.value


# ---- microscaled 4-bit operands: a pair (codes uint8 [..., rows, K/2], scales uint8 tiles) -------------------------
# These calls are issued once or more per layer and token, so their marshalling is kept short: plain integers for
# pointers and handles.

MX_FORMATS = {"MXFP4": 0, "NVFP4": 1}
MX_BLOCK = {"MXFP4": 32, "NVFP4": 16}
DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


def _at(t: torch.Tensor, dev: int) -> int:
    assert t.get_device() == dev and t.is_contiguous(), "tensors passed to uq must be contiguous and on one CUDA device"
    return t.data_ptr()


def _at_opt(t, dev: int):
    return None if t is None else _at(t, dev)


def _operand(q: tuple, dev: int, scale_bytes: int):
    """Pointers of a microscaled operand's codes and scales."""
    codes, scales = q
    assert codes.dtype == torch.uint8 and scales.dtype == torch.uint8, "codes and scales are uint8"
    assert scales.numel() >= scale_bytes, "fewer scale tiles than the operand has"
    return _at(codes, dev), _at(scales, dev)


def _handle(stream, dev: int) -> int:
    """The stream's handle (the current one's without building a Stream object); the tensors' device must be current."""
    assert torch._C._cuda_getDevice() == dev, "tensors passed to uq must be on the current CUDA device"
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(dev)


def mx_scales_size(rows: int, K: int, fmt: str, segments: int = 0) -> int:
    """uq_mx_scales_size: bytes of an operand's scale tiles (host only)."""
    v = ctypes.c_size_t()
    _check(lib().uq_mx_scales_size(rows, K, MX_FORMATS[fmt], segments, ctypes.byref(v)), "uq_mx_scales_size")
    return v.value


def _scale_bytes(rows: int, K: int, fmt: str, segments: int = 0) -> int:
    row_tiles = rows // 128 + segments if segments else (rows + 127) // 128
    return row_tiles * (-(-K // (4 * MX_BLOCK[fmt]))) * 512


def pack_mx_scales(scales: torch.Tensor, fmt: str, stream=None) -> torch.Tensor:
    """uq_pack_mx_scales: scale bytes [rows][K/block] or [experts][rows][K/block] -> tiles (of each expert)."""
    experts = scales.shape[0] if scales.dim() == 3 else 1
    rows, K = scales.shape[-2], scales.shape[-1] * MX_BLOCK[fmt]
    assert scales.dtype == torch.uint8
    dev = scales.get_device()
    tiles = _empty((experts, mx_scales_size(rows, K, fmt)), torch.uint8, scales.device, stream)
    _check(lib().uq_pack_mx_scales(_at(scales, dev), tiles.data_ptr(), experts, rows, K, MX_FORMATS[fmt],
                                   _handle(stream, dev)),
           "uq_pack_mx_scales")
    return tiles if scales.dim() == 3 else tiles[0]


def _row_stride(x: torch.Tensor, T: int, K: int) -> int:
    """Row stride of a [T][K] tensor whose rows are dense."""
    ld, one = x.stride()
    assert x.is_cuda and (one == 1 or K <= 1), "x must be a CUDA matrix of dense rows"
    return ld if T > 1 else K


def quantize_mx(x: torch.Tensor, fmt: str, tscale: float = 1.0, offsets: torch.Tensor | None = None,
                pos: torch.Tensor | None = None, stream=None):
    """uq_quantize_mx: rows [T][K] (bf16, fp16 or fp32; rows may be strided) -> (codes, scales).

    ``offsets`` (int32 [experts + 1]): the rows are sorted by expert; with ``pos`` (int32 [T][k]) they are gathered by
    expert on the way, as moe_gather would, and the operand has T*k rows."""
    T, K = x.shape
    rows, topk, segments, off, at, dev = T, 0, 0, None, None, x.get_device()
    if offsets is not None:
        assert offsets.dtype == torch.int32
        segments, off = offsets.numel() - 1, _at(offsets, dev)
    if pos is not None:
        assert pos.dtype == torch.int32 and pos.shape[0] == T
        topk, at = pos.shape[1], _at(pos, dev)
        rows = T * topk
    codes = _empty((rows, K // 2), torch.uint8, x.device, stream)
    scales = _empty(_scale_bytes(rows, K, fmt, segments), torch.uint8, x.device, stream)
    _check(lib().uq_quantize_mx(x.data_ptr(), DTYPES[x.dtype], _row_stride(x, T, K), codes.data_ptr(), scales.data_ptr(),
                                T, K, MX_FORMATS[fmt], tscale, off, segments, at, topk, _handle(stream, dev)),
           "uq_quantize_mx")
    return codes, scales


def dequant_mx(q: tuple, fmt: str, tscale: float = 1.0, offsets: torch.Tensor | None = None,
               dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """uq_dequant_mx: the values (codes, scales) stand for, [rows][K] of ``dtype``."""
    (rows, half), dev = q[0].shape, q[0].get_device()
    segments, off = 0, None
    if offsets is not None:
        assert offsets.dtype == torch.int32
        segments, off = offsets.numel() - 1, _at(offsets, dev)
    codes, scales = _operand(q, dev, _scale_bytes(rows, half * 2, fmt, segments))
    out = _empty((rows, half * 2), dtype, q[0].device, stream)
    _check(lib().uq_dequant_mx(codes, scales, out.data_ptr(), DTYPES[dtype], rows, half * 2, MX_FORMATS[fmt],
                               tscale, off, segments, _handle(stream, dev)), "uq_dequant_mx")
    return out


def gemm_mx(x, w: tuple, fmt: str, tscale: float = 1.0, alpha: float = 1.0, dtype: torch.dtype | None = None,
            y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """uq_gemm_mx: y = alpha * x^ . w^T (``[M][N]``), both operands microscaled.

    ``x``: a matrix (bf16, fp16 or fp32), quantized in the call with ``tscale``, or a pair (codes, scales) of
    quantize_mx.  ``w``: (codes [N][K/2], scales).  The result has ``dtype`` (default: x's, bf16 for a pair)."""
    (N, half), dev = w[0].shape, w[0].get_device()
    K = half * 2
    wcodes, wscales = _operand(w, dev, _scale_bytes(N, K, fmt))
    if isinstance(x, torch.Tensor):
        M, xk = x.shape
        assert x.get_device() == dev, "x and w are on different devices"
        xtype, xptr, xsc, ld = DTYPES[x.dtype], x.data_ptr(), None, _row_stride(x, M, K)
        if dtype is None:
            dtype = x.dtype
    else:
        M, xk = x[0].shape[0], x[0].shape[1] * 2
        xptr, xsc = _operand(x, dev, _scale_bytes(M, K, fmt))
        xtype, ld = 0, 0
    assert xk == K, "x and w have different K"
    if y is None:
        y = _empty((M, N), dtype or torch.bfloat16, w[0].device, stream)
    assert y.shape == (M, N)
    _check(lib().uq_gemm_mx(xptr, xtype, ld, xsc, tscale, wcodes, wscales, _at(y, dev), DTYPES[y.dtype], M, N, K,
                            MX_FORMATS[fmt], alpha, _handle(stream, dev)), "uq_gemm_mx")
    return y


def gemm_mx_grouped(x: tuple, w: tuple, offsets: torch.Tensor, fmt: str, up: tuple | None = None,
                    alpha: torch.Tensor | None = None, alpha_up: torch.Tensor | None = None,
                    dtype: torch.dtype = torch.bfloat16, y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """uq_gemm_mx_grouped: rows sorted by expert times each expert's weight, ``[rows][N]``.

    ``x``: (codes, scales) of quantize_mx with these ``offsets``; ``w`` (and ``up``: silu(x w^T) * (x up^T)): codes
    [experts][N][K/2] and the experts' scale tiles; ``alpha``, ``alpha_up``: fp32 [experts]."""
    (E, N, half), dev = w[0].shape, w[0].get_device()
    K, R = half * 2, x[0].shape[0]
    assert x[0].shape[1] == half, "x and w have different K"
    assert offsets.dtype == torch.int32 and offsets.numel() == E + 1
    wbytes = E * _scale_bytes(N, K, fmt)
    xcodes, xscales = _operand(x, dev, _scale_bytes(R, K, fmt, E))
    wcodes, wscales = _operand(w, dev, wbytes)
    uc = us = None
    if up is not None:
        assert up[0].shape == w[0].shape
        uc, us = _operand(up, dev, wbytes)
    for v in (alpha, alpha_up):
        assert v is None or (v.dtype == torch.float32 and v.numel() == E)
    if y is None:
        y = _empty((R, N), dtype, w[0].device, stream)
    assert y.shape == (R, N)
    _check(lib().uq_gemm_mx_grouped(xcodes, xscales, wcodes, wscales, uc, us, _at(offsets, dev),
                                    _at_opt(alpha, dev), _at_opt(alpha_up, dev), _at(y, dev), DTYPES[y.dtype], R, E, N,
                                    K, MX_FORMATS[fmt], _handle(stream, dev)), "uq_gemm_mx_grouped")
    return y


# ---- expert routing ------------------------------------------------------------------------------------------------
# Plain calls, unknown to autograd: the gradient of moe_gather is moe_gather_grad, that of moe_combine is
# moe_combine_grad, and a caller that trains with them wraps them in a torch.autograd.Function.

def moe_sort(ids: torch.Tensor, experts: int, stream=None):
    """uq_moe_sort: int32 expert ids [T][k] -> (order int32 [T*k], pos int32 [T][k], offsets int32 [experts + 1])."""
    T, k = ids.shape
    assert ids.dtype == torch.int32
    dev = ids.get_device()
    order = _empty(T * k, torch.int32, ids.device, stream)
    pos = _empty((T, k), torch.int32, ids.device, stream)
    offsets = _empty(max(experts, 0) + 1, torch.int32, ids.device, stream)
    _check(lib().uq_moe_sort(_at(ids, dev), T, k, experts, order.data_ptr(), pos.data_ptr(), offsets.data_ptr(),
                             _handle(stream, dev)), "uq_moe_sort")
    return order, pos, offsets


def moe_gather(x: torch.Tensor, pos: torch.Tensor, offsets: torch.Tensor, stream=None) -> torch.Tensor:
    """uq_moe_gather: xs[pos[t][j]] = x[t], [T*k][H]; rows past offsets[-1] are zero."""
    (T, H), (rows, k) = x.shape, pos.shape
    assert pos.dtype == torch.int32 and offsets.dtype == torch.int32 and rows == T
    dev, xs = x.get_device(), _empty((T * k, H), x.dtype, x.device, stream)
    _check(lib().uq_moe_gather(_at(x, dev), DTYPES[x.dtype], _at(pos, dev), _at(offsets, dev), offsets.numel() - 1,
                               xs.data_ptr(), T, k, H, _handle(stream, dev)), "uq_moe_gather")
    return xs


def moe_gather_grad(dxs: torch.Tensor, pos: torch.Tensor, stream=None) -> torch.Tensor:
    """uq_moe_gather_grad: dx[t] = sum_j dxs[pos[t][j]], [T][H]."""
    (T, k), (R, H) = pos.shape, dxs.shape
    assert pos.dtype == torch.int32 and R == T * k
    dev, dx = dxs.get_device(), _empty((T, H), dxs.dtype, dxs.device, stream)
    _check(lib().uq_moe_gather_grad(_at(dxs, dev), DTYPES[dxs.dtype], _at(pos, dev), dx.data_ptr(), T, k, H,
                                    _handle(stream, dev)), "uq_moe_gather_grad")
    return dx


def moe_combine(ys: torch.Tensor, pos: torch.Tensor, weights: torch.Tensor, stream=None) -> torch.Tensor:
    """uq_moe_combine: y[t] = sum_j weights[t][j] * ys[pos[t][j]], [T][H]; weights fp32 [T][k]."""
    (T, k), (R, H) = pos.shape, ys.shape
    assert pos.dtype == torch.int32 and weights.dtype == torch.float32
    assert R == T * k and weights.shape == pos.shape
    dev, y = ys.get_device(), _empty((T, H), ys.dtype, ys.device, stream)
    _check(lib().uq_moe_combine(_at(ys, dev), DTYPES[ys.dtype], _at(pos, dev), _at(weights, dev), y.data_ptr(), T, k, H,
                                _handle(stream, dev)), "uq_moe_combine")
    return y


def moe_combine_grad(dy: torch.Tensor, ys: torch.Tensor, pos: torch.Tensor, weights: torch.Tensor,
                     offsets: torch.Tensor, stream=None):
    """uq_moe_combine_grad: (dys [T*k][H], dweights fp32 [T][k]) of moe_combine for the output gradient dy [T][H]."""
    (T, k), (R, H) = pos.shape, ys.shape
    assert pos.dtype == torch.int32 and offsets.dtype == torch.int32 and weights.dtype == torch.float32
    assert dy.dtype == ys.dtype and dy.shape == (T, H) and R == T * k and weights.shape == pos.shape
    dev, dys = ys.get_device(), _empty(ys.shape, ys.dtype, ys.device, stream)
    dw = _empty((T, k), torch.float32, ys.device, stream)
    _check(lib().uq_moe_combine_grad(_at(dy, dev), _at(ys, dev), DTYPES[ys.dtype], _at(pos, dev), _at(weights, dev),
                                     _at(offsets, dev), offsets.numel() - 1, dys.data_ptr(), dw.data_ptr(), T, k, H,
                                     _handle(stream, dev)), "uq_moe_combine_grad")
    return dys, dw
