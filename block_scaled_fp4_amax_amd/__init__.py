"""block_scaled_fp4_amax_amd -- block-scaled FP4 (E2M1) quantization and the
W4A4 block-scaled GEMM on AMD MI355X (gfx950).

The compute lives in ``libfp4.so`` (hand-written HIP kernels behind the C ABI
of ``include/fp4.h``). This module only marshals arguments:

* ``fp4_quantize``, ``fp4_quantize_noalloc``, ``fp4_dequantize``,
  ``fp4_gemm``, ``fp4_gemm_grouped``, ``fp4_gemm_quantize_output``,
  ``fp4_kv_append``, ``fp4_kv_read``, ``fp4_kv_attention``,
  ``fp4_kv_attention_workspace``, ``fp4_quantize_workspace``,
  ``fp4_status_str`` -- the C entry points with
  the same names and argument order (integers for device pointers);
* ``quantize``, ``dequantize``, ``gemm``, ``gemm_grouped``,
  ``gemm_quantize_output``, and ``KVCache`` with ``kv_append``, ``kv_read``,
  ``kv_attention`` -- conveniences over torch device
  tensors that allocate outputs with torch, pass the current HIP stream (or
  allocate and launch on the one whose handle is given as ``stream``; inputs
  have to be ready there) and raise ``Fp4Error`` on a non-OK status.

There is no fallback: if ``libfp4.so`` is missing or a call fails, an error is
raised.
"""
from __future__ import annotations

import ctypes
import struct
from ctypes import c_float, c_int32, c_int64, c_size_t, c_uint32, c_uint64, c_void_p, c_char_p
from dataclasses import dataclass
from pathlib import Path
from typing import Optional

LIB_PATH = Path(__file__).resolve().with_name("libfp4.so")

# fp4_status
FP4_OK = 0
FP4_ERR_INVALID = -1
FP4_ERR_UNSUPPORTED = -2
FP4_ERR_ALIGN = -3
FP4_ERR_DEVICE = -4
FP4_ERR_WORKSPACE = -5
FP4_ERR_HIP = -6
FP4_ERR_SCRATCH = -7
FP4_NOALLOC_SCRATCH_BYTES = 262144
# fp4_format / fp4_dtype
FP4_MXFP4 = 0
FP4_NVFP4 = 1
FP4_F32 = 0
FP4_BF16 = 1
# flags
FP4_FOUR_OVER_SIX = 1
FP4_BLOCK2D = 2
FP4_TRANSPOSE = 4
FP4_STOCHASTIC = 8
FP4_HADAMARD = 16
FP4_SCALE_SEARCH = 32
FP4_TENSOR_SCALE = 64
# fp4_kv_append_args.flags, fp4_kv_attention_args.flags
FP4_KV_INTERLEAVED = 256
FP4_KV_CAUSAL = 1

EXPORTED_SYMBOLS = ("fp4_quantize_workspace", "fp4_quantize", "fp4_quantize_noalloc", "fp4_dequantize", "fp4_gemm",
                    "fp4_gemm_grouped", "fp4_gemm_quantize_output", "fp4_kv_append", "fp4_kv_read",
                    "fp4_kv_attention_workspace", "fp4_kv_attention", "fp4_status_str")


class fp4_quant_opts(ctypes.Structure):
    _fields_ = [
        ("size", c_uint32),
        ("format", c_int32),
        ("flags", c_uint32),
        ("rht_signs", c_uint32),
        ("seed", c_uint64),
        ("offset", c_uint64),
        ("amax_in", c_void_p),
    ]


class fp4_kv_cache(ctypes.Structure):
    _fields_ = [
        ("size", c_uint32),
        ("format", c_int32),
        ("num_pages", c_int64),
        ("page_size", c_int32),
        ("kv_heads", c_int32),
        ("head_dim", c_int32),
        ("reserved", c_int32),
        ("k_codes", c_void_p),
        ("k_scales", c_void_p),
        ("v_codes", c_void_p),
        ("v_scales", c_void_p),
        ("codes_page_stride", c_int64),
        ("scales_page_stride", c_int64),
        ("k_tensor_scale", c_void_p),
        ("v_tensor_scale", c_void_p),
    ]


class fp4_kv_append_args(ctypes.Structure):
    _fields_ = [
        ("size", c_uint32),
        ("dtype", c_int32),
        ("flags", c_uint32),
        ("q_heads", c_int32),
        ("tokens", c_int64),
        ("k", c_void_p),
        ("v", c_void_p),
        ("q", c_void_p),
        ("q_out", c_void_p),
        ("k_token_stride", c_int64),
        ("k_head_stride", c_int64),
        ("v_token_stride", c_int64),
        ("v_head_stride", c_int64),
        ("q_token_stride", c_int64),
        ("q_head_stride", c_int64),
        ("q_out_token_stride", c_int64),
        ("q_out_head_stride", c_int64),
        ("slots", c_void_p),
        ("positions", c_void_p),
        ("cos_table", c_void_p),
        ("sin_table", c_void_p),
        ("max_position", c_int64),
        ("rotary", c_int32),
        ("reserved", c_int32),
    ]


class fp4_kv_attention_args(ctypes.Structure):
    _fields_ = [
        ("size", c_uint32),
        ("dtype", c_int32),
        ("flags", c_uint32),
        ("q_heads", c_int32),
        ("batch", c_int64),
        ("tokens", c_int64),
        ("q_offsets", c_void_p),
        ("kv_lens", c_void_p),
        ("block_table", c_void_p),
        ("table_stride", c_int64),
        ("table_width", c_int64),
        ("max_kv_len", c_int64),
        ("q", c_void_p),
        ("out", c_void_p),
        ("lse", c_void_p),
        ("q_token_stride", c_int64),
        ("q_head_stride", c_int64),
        ("out_token_stride", c_int64),
        ("out_head_stride", c_int64),
        ("scale", c_float),
        ("softcap", c_float),
        ("window", c_int64),
    ]


_APPEND_SIZE = ctypes.sizeof(fp4_kv_append_args)
_ATTENTION_SIZE = ctypes.sizeof(fp4_kv_attention_args)


def _packer(args):
    """The bytes of a structure's fields (null pointers are 0): a third of the
    time of making the ctypes structure."""
    codes = {c_int32: "i", c_uint32: "I", c_int64: "q", c_void_p: "Q", c_float: "f"}
    packed = struct.Struct("@" + "".join(codes[t] for _, t in args._fields_))
    assert packed.size == ctypes.sizeof(args)

    def pack(*values):
        try:
            return packed.pack(*values)
        except (struct.error, OverflowError) as e:
            raise ValueError(f"{args.__name__}: {e}") from None
    return pack


_pack_append = _packer(fp4_kv_append_args)
_pack_attention = _packer(fp4_kv_attention_args)


class Fp4Error(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {fp4_status_str(status)} ({status})")
        self.status = status


_lib: Optional[ctypes.CDLL] = None


def lib() -> ctypes.CDLL:
    """Load libfp4.so (once). Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not LIB_PATH.exists():
            raise RuntimeError(
                f"{LIB_PATH} is not built; run `python -m block_scaled_fp4_amax_amd.build` "
                "(or __graft_entry__.build())")
        L = ctypes.CDLL(str(LIB_PATH))
        L.fp4_quantize_workspace.restype = c_size_t
        L.fp4_quantize_workspace.argtypes = [c_int64, c_int64, c_int64, ctypes.POINTER(fp4_quant_opts)]
        L.fp4_quantize.restype = c_int32
        L.fp4_quantize.argtypes = [
            c_void_p, c_int32, c_int64, c_int64, c_int64, c_int64, c_int64, ctypes.POINTER(fp4_quant_opts),
            c_void_p, c_int64, c_int64, c_void_p, c_int64, c_int64, c_void_p, c_void_p, c_size_t, c_void_p]
        L.fp4_quantize_noalloc.restype = c_int32
        L.fp4_quantize_noalloc.argtypes = [
            c_void_p, c_int32, c_int64, c_int64, c_int64, c_int64, c_int64, ctypes.POINTER(fp4_quant_opts),
            c_void_p, c_int64, c_int64, c_void_p, c_int64, c_int64, c_void_p, c_void_p]
        L.fp4_dequantize.restype = c_int32
        L.fp4_dequantize.argtypes = [
            c_int32, c_int64, c_int64, c_int64, c_void_p, c_int64, c_int64, c_void_p, c_int64, c_int64,
            c_void_p, c_void_p, c_int32, c_int64, c_int64, c_void_p]
        L.fp4_gemm.restype = c_int32
        L.fp4_gemm.argtypes = [
            c_int32, c_int64, c_int64, c_int64, c_int64,
            c_void_p, c_int64, c_int64, c_void_p, c_int64, c_int64, c_void_p,
            c_void_p, c_int64, c_int64, c_void_p, c_int64, c_int64, c_void_p,
            c_void_p, c_int32, c_int64, c_int64, c_void_p]
        L.fp4_gemm_grouped.restype = c_int32
        L.fp4_gemm_grouped.argtypes = [
            c_int32, c_int64, c_void_p, c_int64, c_int64, c_int64,
            c_void_p, c_int64, c_void_p, c_int64, c_void_p,
            c_void_p, c_int64, c_int64, c_void_p, c_int64, c_int64, c_void_p,
            c_void_p, c_int32, c_int64, c_void_p]
        L.fp4_gemm_quantize_output.restype = c_int32
        L.fp4_gemm_quantize_output.argtypes = [
            c_int32, c_int64, c_int64, c_int64, c_int64,
            c_void_p, c_int64, c_int64, c_void_p, c_int64, c_int64, c_void_p,
            c_void_p, c_int64, c_int64, c_void_p, c_int64, c_int64, c_void_p,
            ctypes.POINTER(fp4_quant_opts), c_void_p, c_int64, c_int64, c_void_p, c_int64, c_int64, c_void_p,
            c_void_p]
        L.fp4_kv_append.restype = c_int32
        L.fp4_kv_append.argtypes = [ctypes.POINTER(fp4_kv_cache), c_void_p, c_void_p]
        L.fp4_kv_read.restype = c_int32
        L.fp4_kv_read.argtypes = [ctypes.POINTER(fp4_kv_cache), c_int64, c_void_p, c_void_p, c_void_p, c_int32,
                                  c_void_p]
        L.fp4_kv_attention_workspace.restype = c_size_t
        L.fp4_kv_attention_workspace.argtypes = [ctypes.POINTER(fp4_kv_cache), c_void_p]
        L.fp4_kv_attention.restype = c_int32
        L.fp4_kv_attention.argtypes = [ctypes.POINTER(fp4_kv_cache), c_void_p, c_void_p, c_size_t, c_void_p]
        L.fp4_status_str.restype = c_char_p
        L.fp4_status_str.argtypes = [c_int32]
        _lib = L
    return _lib


def make_opts(fmt: int, flags: int = 0, rht_signs: int = 0, seed: int = 0, offset: int = 0,
              amax_in: int = 0) -> fp4_quant_opts:
    o = fp4_quant_opts()
    o.size = ctypes.sizeof(fp4_quant_opts)
    o.format = fmt
    o.flags = flags
    o.rht_signs = rht_signs
    o.seed = seed
    o.offset = offset
    o.amax_in = amax_in or None
    return o


# ---------------------------------------------------------------------------
# raw C entry points (same names, same argument order)
# ---------------------------------------------------------------------------
def fp4_status_str(status: int) -> str:
    return lib().fp4_status_str(status).decode()


def fp4_quantize_workspace(batch, rows, cols, opts: fp4_quant_opts) -> int:
    return lib().fp4_quantize_workspace(batch, rows, cols, ctypes.byref(opts))


def fp4_quantize(x, x_dtype, batch, rows, cols, ld_x, batch_stride_x, opts: fp4_quant_opts, codes, ld_codes,
                 batch_stride_codes, scales, ld_scales, batch_stride_scales, tensor_scale, workspace,
                 workspace_bytes, stream) -> int:
    return lib().fp4_quantize(x, x_dtype, batch, rows, cols, ld_x, batch_stride_x, ctypes.byref(opts), codes,
                              ld_codes, batch_stride_codes, scales, ld_scales, batch_stride_scales, tensor_scale,
                              workspace, workspace_bytes, stream)


def fp4_quantize_noalloc(x, x_dtype, batch, rows, cols, ld_x, batch_stride_x, opts: fp4_quant_opts, codes, ld_codes,
                         batch_stride_codes, scales, ld_scales, batch_stride_scales, tensor_scale, stream) -> int:
    return lib().fp4_quantize_noalloc(x, x_dtype, batch, rows, cols, ld_x, batch_stride_x, ctypes.byref(opts), codes,
                                      ld_codes, batch_stride_codes, scales, ld_scales, batch_stride_scales,
                                      tensor_scale, stream)


def fp4_dequantize(fmt, batch, rows, cols, codes, ld_codes, batch_stride_codes, scales, ld_scales,
                   batch_stride_scales, tensor_scale, y, y_dtype, ld_y, batch_stride_y, stream) -> int:
    return lib().fp4_dequantize(fmt, batch, rows, cols, codes, ld_codes, batch_stride_codes, scales, ld_scales,
                                batch_stride_scales, tensor_scale, y, y_dtype, ld_y, batch_stride_y, stream)


def fp4_gemm(fmt, groups, M, N, K, a_codes, lda, a_group_stride, a_scales, lda_scales, a_scales_group_stride,
             a_tensor_scale, b_codes, ldb, b_group_stride, b_scales, ldb_scales, b_scales_group_stride,
             b_tensor_scale, c, c_dtype, ldc, c_group_stride, stream) -> int:
    return lib().fp4_gemm(fmt, groups, M, N, K, a_codes, lda, a_group_stride, a_scales, lda_scales,
                          a_scales_group_stride, a_tensor_scale, b_codes, ldb, b_group_stride, b_scales, ldb_scales,
                          b_scales_group_stride, b_tensor_scale, c, c_dtype, ldc, c_group_stride, stream)


def fp4_gemm_quantize_output(fmt, groups, M, N, K, a_codes, lda, a_group_stride, a_scales, lda_scales,
                             a_scales_group_stride, a_tensor_scale, b_codes, ldb, b_group_stride, b_scales, ldb_scales,
                             b_scales_group_stride, b_tensor_scale, out_opts: fp4_quant_opts, out_codes, ld_out_codes,
                             out_codes_group_stride, out_scales, ld_out_scales, out_scales_group_stride,
                             out_tensor_scale, stream) -> int:
    return lib().fp4_gemm_quantize_output(fmt, groups, M, N, K, a_codes, lda, a_group_stride, a_scales, lda_scales,
                                          a_scales_group_stride, a_tensor_scale, b_codes, ldb, b_group_stride,
                                          b_scales, ldb_scales, b_scales_group_stride, b_tensor_scale,
                                          ctypes.byref(out_opts), out_codes, ld_out_codes, out_codes_group_stride,
                                          out_scales, ld_out_scales, out_scales_group_stride, out_tensor_scale,
                                          stream)


def fp4_gemm_grouped(fmt, groups, group_offsets, M, N, K, a_codes, lda, a_scales, lda_scales, a_tensor_scale,
                     b_codes, ldb, b_group_stride, b_scales, ldb_scales, b_scales_group_stride, b_tensor_scale, c,
                     c_dtype, ldc, stream) -> int:
    return lib().fp4_gemm_grouped(fmt, groups, group_offsets, M, N, K, a_codes, lda, a_scales, lda_scales,
                                  a_tensor_scale, b_codes, ldb, b_group_stride, b_scales, ldb_scales,
                                  b_scales_group_stride, b_tensor_scale, c, c_dtype, ldc, stream)


def fp4_kv_append(cache: fp4_kv_cache, args: fp4_kv_append_args, stream) -> int:
    return lib().fp4_kv_append(ctypes.byref(cache), ctypes.byref(args), stream)


def fp4_kv_read(cache: fp4_kv_cache, tokens, slots, k_out, v_out, y_dtype, stream) -> int:
    return lib().fp4_kv_read(ctypes.byref(cache), tokens, slots, k_out, v_out, y_dtype, stream)


def fp4_kv_attention_workspace(cache: fp4_kv_cache, args: fp4_kv_attention_args) -> int:
    return lib().fp4_kv_attention_workspace(ctypes.byref(cache), ctypes.byref(args))


def fp4_kv_attention(cache: fp4_kv_cache, args: fp4_kv_attention_args, workspace, workspace_bytes, stream) -> int:
    return lib().fp4_kv_attention(ctypes.byref(cache), ctypes.byref(args), workspace, workspace_bytes, stream)


# ---------------------------------------------------------------------------
# torch conveniences (allocation + current stream only)
# ---------------------------------------------------------------------------
def scale_pitch(n_blocks: int) -> int:
    """Scale-row pitch in bytes that fp4_gemm accepts: rounded up to 16."""
    return (n_blocks + 15) // 16 * 16


def code_pitch(n_bytes: int) -> int:
    """Code-row pitch in bytes: rounded up to 128 (one cache line), so that
    every row starts on a line and no store of a row shares a line with the
    next row (rows of 1440 bytes otherwise straddle lines)."""
    return (n_bytes + 127) // 128 * 128


@dataclass
class Quantized:
    """Packed FP4 tensor as written by fp4_quantize. Shapes carry an optional
    leading batch dimension: codes [.., R, C/2], scales [.., R, C/blk],
    tensor_scale [batch] (NVFP4) or None. `codes` and `scales` may be views
    whose row pitch (stride(-2)) exceeds C/2 or C/blk: quantize() pads code
    rows to code_pitch() and scale rows to scale_pitch()."""
    fmt: int
    codes: "torch.Tensor"
    scales: "torch.Tensor"
    tensor_scale: Optional["torch.Tensor"]

    @property
    def block(self) -> int:
        return 16 if self.fmt == FP4_NVFP4 else 32

    @property
    def shape(self):
        return (*self.codes.shape[:-1], self.codes.shape[-1] * 2)


def _fmt(fmt) -> int:
    if isinstance(fmt, str):
        return {"mxfp4": FP4_MXFP4, "nvfp4": FP4_NVFP4}[fmt.lower()]
    return int(fmt)


def _stream():
    import torch
    return torch.cuda.current_stream().cuda_stream


def _on_stream(call, device, stream, given, *args, **kw):
    """The call again, with `stream` current: copies, outputs and workspace are
    then that stream's own, and nothing queued on another still uses their
    memory. The outputs it makes (not `given`) may be used on the caller's
    stream too, and are not reused before that has passed their last use."""
    import torch
    caller = torch.cuda.current_stream(device)
    with torch.cuda.stream(torch.cuda.ExternalStream(stream, device=device)):
        result = call(*args, **kw)
    made = (result.codes, result.scales, result.tensor_scale) if isinstance(result, Quantized) else result
    for t in made if isinstance(made, tuple) else (made,):
        if t is not None and t is not given:
            t.record_stream(caller)
    return result


def _elsewhere(stream) -> bool:
    return stream is not None and stream != _stream()


def _check(status: int, where: str):
    if status != FP4_OK:
        raise Fp4Error(status, where)


def quantize(x, fmt="nvfp4", *, four_over_six=False, block2d=False, transpose=False, stochastic=False,
             hadamard=False, scale_search=False, tensor_scale=False, rht_signs=0, seed=0, offset=0, amax=None,
             stream=None) -> Quantized:
    """Quantize a [rows, cols] or [batch, rows, cols] bf16/fp32 device tensor
    (tensor_scale: the NVFP4 whole-tensor mode, FP4_TENSOR_SCALE)."""
    import torch
    if _elsewhere(stream):
        return _on_stream(quantize, x.device, stream, None, x, fmt, four_over_six=four_over_six, block2d=block2d,
                          transpose=transpose, stochastic=stochastic, hadamard=hadamard, scale_search=scale_search,
                          tensor_scale=tensor_scale, rht_signs=rht_signs, seed=seed, offset=offset, amax=amax)
    fmt = _fmt(fmt)
    squeeze = x.dim() == 2
    x3 = x.unsqueeze(0) if squeeze else x
    if x3.dim() != 3:
        raise ValueError("quantize expects a 2-D or 3-D tensor")
    x3 = x3.contiguous()
    batch, rows, cols = x3.shape
    dt = {torch.bfloat16: FP4_BF16, torch.float32: FP4_F32}[x3.dtype]
    flags = ((FP4_FOUR_OVER_SIX if four_over_six else 0) | (FP4_BLOCK2D if block2d else 0)
             | (FP4_TRANSPOSE if transpose else 0) | (FP4_STOCHASTIC if stochastic else 0)
             | (FP4_HADAMARD if hadamard else 0) | (FP4_SCALE_SEARCH if scale_search else 0)
             | (FP4_TENSOR_SCALE if tensor_scale else 0))
    amax_t = None
    if amax is not None:
        amax_t = torch.as_tensor(amax, dtype=torch.float32, device=x3.device).reshape(-1).contiguous()
    opts = make_opts(fmt, flags, rht_signs, seed, offset, amax_t.data_ptr() if amax_t is not None else 0)
    R, C = (cols, rows) if transpose else (rows, cols)
    blk = 16 if fmt == FP4_NVFP4 else 32
    dev = x3.device
    ldc = code_pitch(C // 2)
    codes = torch.empty((batch, R, ldc), dtype=torch.uint8, device=dev)[:, :, : C // 2]
    lds = scale_pitch(C // blk)
    scales_buf = torch.empty((batch, R, lds), dtype=torch.uint8, device=dev)
    scales = scales_buf[:, :, : C // blk]
    ts = torch.empty((batch,), dtype=torch.float32, device=dev) if fmt == FP4_NVFP4 else None
    ws_bytes = fp4_quantize_workspace(batch, rows, cols, opts)
    ws = torch.empty((max(ws_bytes, 1),), dtype=torch.uint8, device=dev) if ws_bytes else None
    st = fp4_quantize(x3.data_ptr(), dt, batch, rows, cols, cols, rows * cols, opts, codes.data_ptr(), ldc,
                      R * ldc, scales_buf.data_ptr(), lds, R * lds,
                      ts.data_ptr() if ts is not None else None, ws.data_ptr() if ws is not None else None,
                      ws_bytes, _stream())
    _check(st, "fp4_quantize")
    if squeeze:
        codes, scales = codes[0], scales[0]
    return Quantized(fmt, codes, scales, ts)


def _check_scales(scales):
    """Scales are passed by base pointer and row / batch pitch: the last dim
    must be dense."""
    if scales.stride(-1) != 1:
        raise ValueError("scale rows must be contiguous")


def _check_codes(codes):
    """Codes likewise: dense rows, any row / batch pitch."""
    if codes.stride(-1) != 1:
        raise ValueError("code rows must be contiguous")


def dequantize(q: Quantized, dtype=None, stream=None):
    import torch
    if _elsewhere(stream):
        return _on_stream(dequantize, q.codes.device, stream, None, q, dtype)
    dtype = dtype or torch.float32
    codes = q.codes if q.codes.dim() == 3 else q.codes.unsqueeze(0)
    scales = q.scales if q.scales.dim() == 3 else q.scales.unsqueeze(0)
    batch, rows, half = codes.shape
    cols = half * 2
    y = torch.empty((batch, rows, cols), dtype=dtype, device=codes.device)
    dt = {torch.bfloat16: FP4_BF16, torch.float32: FP4_F32}[dtype]
    _check_scales(scales)
    _check_codes(codes)
    st = fp4_dequantize(q.fmt, batch, rows, cols, codes.data_ptr(), codes.stride(1), codes.stride(0),
                        scales.data_ptr(),
                        scales.stride(1), scales.stride(0),
                        q.tensor_scale.data_ptr() if q.tensor_scale is not None else None, y.data_ptr(), dt, cols,
                        rows * cols, _stream())
    _check(st, "fp4_dequantize")
    return y if q.codes.dim() == 3 else y[0]


def gemm(a: Quantized, b: Quantized, out_dtype=None, stream=None):
    """C[g] = deq(A[g]) @ deq(B[g])^T with A [.., M, K] and B [.., N, K]."""
    import torch
    if _elsewhere(stream):
        return _on_stream(gemm, a.codes.device, stream, None, a, b, out_dtype)
    out_dtype = out_dtype or torch.float32
    if a.fmt != b.fmt:
        raise ValueError("operands must share a format")
    ac = a.codes if a.codes.dim() == 3 else a.codes.unsqueeze(0)
    asc = a.scales if a.scales.dim() == 3 else a.scales.unsqueeze(0)
    bc = b.codes if b.codes.dim() == 3 else b.codes.unsqueeze(0)
    bsc = b.scales if b.scales.dim() == 3 else b.scales.unsqueeze(0)
    G, M, half = ac.shape
    Gb, N, halfb = bc.shape
    if G != Gb or half != halfb:
        raise ValueError("operand shapes do not match")
    K = half * 2
    c = torch.empty((G, M, N), dtype=out_dtype, device=ac.device)
    ct = {torch.bfloat16: FP4_BF16, torch.float32: FP4_F32}[out_dtype]
    _check_scales(asc)
    _check_scales(bsc)
    _check_codes(ac)
    _check_codes(bc)
    st = fp4_gemm(a.fmt, G, M, N, K, ac.data_ptr(), ac.stride(1), ac.stride(0), asc.data_ptr(), asc.stride(1),
                  asc.stride(0), a.tensor_scale.data_ptr() if a.tensor_scale is not None else None,
                  bc.data_ptr(), bc.stride(1), bc.stride(0), bsc.data_ptr(), bsc.stride(1), bsc.stride(0),
                  b.tensor_scale.data_ptr() if b.tensor_scale is not None else None, c.data_ptr(), ct, N, M * N,
                  _stream())
    _check(st, "fp4_gemm")
    return c if a.codes.dim() == 3 else c[0]


def gemm_quantize_output(a: Quantized, b: Quantized, fmt="nvfp4", *, four_over_six=False, stochastic=False,
                         hadamard=False, scale_search=False, rht_signs=0, seed=0, offset=0, amax=None,
                         stream=None) -> Quantized:
    """deq(A[g]) @ deq(B[g])^T quantized along its rows in the GEMM's epilogue
    (format `fmt`, options as for quantize); NVFP4 needs `amax`, the tensor
    amax per group that S_t derives from."""
    import torch
    if _elsewhere(stream):
        return _on_stream(gemm_quantize_output, a.codes.device, stream, None, a, b, fmt, four_over_six=four_over_six,
                          stochastic=stochastic, hadamard=hadamard, scale_search=scale_search, rht_signs=rht_signs,
                          seed=seed, offset=offset, amax=amax)
    if a.fmt != b.fmt:
        raise ValueError("operands must share a format")
    ac = a.codes if a.codes.dim() == 3 else a.codes.unsqueeze(0)
    asc = a.scales if a.scales.dim() == 3 else a.scales.unsqueeze(0)
    bc = b.codes if b.codes.dim() == 3 else b.codes.unsqueeze(0)
    bsc = b.scales if b.scales.dim() == 3 else b.scales.unsqueeze(0)
    G, M, half = ac.shape
    Gb, N, halfb = bc.shape
    if G != Gb or half != halfb:
        raise ValueError("operand shapes do not match")
    qfmt = _fmt(fmt)
    flags = ((FP4_FOUR_OVER_SIX if four_over_six else 0) | (FP4_STOCHASTIC if stochastic else 0)
             | (FP4_HADAMARD if hadamard else 0) | (FP4_SCALE_SEARCH if scale_search else 0))
    amax_t = None
    if amax is not None:
        amax_t = torch.as_tensor(amax, dtype=torch.float32, device=ac.device).reshape(-1).contiguous()
    opts = make_opts(qfmt, flags, rht_signs, seed, offset, amax_t.data_ptr() if amax_t is not None else 0)
    blk = 16 if qfmt == FP4_NVFP4 else 32
    dev = ac.device
    ldq = code_pitch(N // 2)
    codes = torch.empty((G, M, ldq), dtype=torch.uint8, device=dev)[:, :, : N // 2]
    lds = scale_pitch(N // blk)
    scales_buf = torch.empty((G, M, lds), dtype=torch.uint8, device=dev)
    ts = torch.empty((G,), dtype=torch.float32, device=dev) if qfmt == FP4_NVFP4 else None
    _check_scales(asc)
    _check_scales(bsc)
    _check_codes(ac)
    _check_codes(bc)
    st = fp4_gemm_quantize_output(a.fmt, G, M, N, half * 2, ac.data_ptr(), ac.stride(1), ac.stride(0),
                                  asc.data_ptr(), asc.stride(1), asc.stride(0),
                                  a.tensor_scale.data_ptr() if a.tensor_scale is not None else None,
                                  bc.data_ptr(), bc.stride(1), bc.stride(0), bsc.data_ptr(), bsc.stride(1),
                                  bsc.stride(0), b.tensor_scale.data_ptr() if b.tensor_scale is not None else None,
                                  opts, codes.data_ptr(), ldq, M * ldq, scales_buf.data_ptr(), lds, M * lds,
                                  ts.data_ptr() if ts is not None else None, _stream())
    _check(st, "fp4_gemm_quantize_output")
    scales = scales_buf[:, :, : N // blk]
    if a.codes.dim() == 2:
        codes, scales = codes[0], scales[0]
    return Quantized(qfmt, codes, scales, ts)


def gemm_grouped(a: Quantized, b: Quantized, offsets, out_dtype=None, stream=None):
    """Mixture-of-experts grouped GEMM: rows offsets[g]:offsets[g + 1] of
    A [M, K] times B[g] [N, K]^T, into C [M, N]. `offsets` is a device int32
    tensor of groups + 1 entries (e.g. a router's cumulative counts)."""
    import torch
    if _elsewhere(stream):
        return _on_stream(gemm_grouped, a.codes.device, stream, None, a, b, offsets, out_dtype)
    out_dtype = out_dtype or torch.float32
    if a.fmt != b.fmt:
        raise ValueError("operands must share a format")
    if a.codes.dim() != 2:
        raise ValueError("A must be one [M, K] matrix")
    bc = b.codes if b.codes.dim() == 3 else b.codes.unsqueeze(0)
    bsc = b.scales if b.scales.dim() == 3 else b.scales.unsqueeze(0)
    G, N, half = bc.shape
    M, halfa = a.codes.shape
    if half != halfa:
        raise ValueError("operand shapes do not match")
    if offsets.dtype != torch.int32 or offsets.dim() != 1 or offsets.numel() != G + 1 or not offsets.is_cuda:
        raise ValueError("offsets must be a device int32 vector of groups + 1 entries")
    offsets = offsets.contiguous()
    c = torch.empty((M, N), dtype=out_dtype, device=a.codes.device)
    ct = {torch.bfloat16: FP4_BF16, torch.float32: FP4_F32}[out_dtype]
    _check_scales(a.scales.unsqueeze(0))
    _check_scales(bsc)
    _check_codes(a.codes)
    _check_codes(bc)
    st = fp4_gemm_grouped(a.fmt, G, offsets.data_ptr(), M, N, half * 2, a.codes.data_ptr(), a.codes.stride(0),
                          a.scales.data_ptr(), a.scales.stride(0),
                          a.tensor_scale.data_ptr() if a.tensor_scale is not None else None,
                          bc.data_ptr(), bc.stride(1), bc.stride(0), bsc.data_ptr(), bsc.stride(1), bsc.stride(0),
                          b.tensor_scale.data_ptr() if b.tensor_scale is not None else None, c.data_ptr(), ct, N,
                          _stream())
    _check(st, "fp4_gemm_grouped")
    return c


# ---------------------------------------------------------------------------
# the paged 4-bit key-value cache
# ---------------------------------------------------------------------------
class KVCache:
    """A paged key-value cache in FP4: the handle of its buffers, made once
    and used by every call on them.

    k_codes, v_codes [pages, kv_heads, page_size, head_dim / 2] and k_scales,
    v_scales [pages, kv_heads, page_size, head_dim / block] are uint8 device
    tensors whose pages are dense (keys and values may be halves of one
    buffer); NVFP4 has fp32 device vectors [kv_heads] of tensor scales. The
    handle keeps references to them, and their addresses."""

    def __init__(self, fmt, k_codes, k_scales, v_codes, v_scales, k_tensor_scale=None, v_tensor_scale=None):
        import torch
        self.fmt = _fmt(fmt)
        blk = 16 if self.fmt == FP4_NVFP4 else 32
        if k_codes.dim() != 4:
            raise ValueError("cache buffers are [pages, kv_heads, page_size, bytes]")
        pages, heads, page_size, half = k_codes.shape
        self.num_pages, self.kv_heads, self.page_size, self.head_dim = pages, heads, page_size, 2 * half
        self.device, self.index = k_codes.device, k_codes.get_device()
        for t, width in ((k_codes, half), (v_codes, half), (k_scales, 2 * half // blk), (v_scales, 2 * half // blk)):
            if t.dtype != torch.uint8 or t.device != self.device or not t.is_cuda:
                raise ValueError("cache buffers must be uint8 tensors on one GPU")
            if tuple(t.shape) != (pages, heads, page_size, width):
                raise ValueError(f"cache buffer of shape {tuple(t.shape)}, expected {(pages, heads, page_size, width)}")
            # (a single kv head, or a row of one scale, may have any stride)
            if pages and any(n > 1 and have != want for n, have, want in
                             zip(t.shape[1:], t.stride()[1:], (page_size * width, width, 1))):
                raise ValueError("the pages of a cache buffer must be dense")
        for a, b in ((k_codes, v_codes), (k_scales, v_scales)):
            if pages > 1 and a.stride(0) != b.stride(0):
                raise ValueError("keys and values must have the same page stride")
        if self.fmt == FP4_NVFP4:
            for t in (k_tensor_scale, v_tensor_scale):
                if (t is None or t.dtype != torch.float32 or t.device != self.device or tuple(t.shape) != (heads,)
                        or not t.is_contiguous()):
                    raise ValueError("NVFP4 needs fp32 tensor scales [kv_heads] on the cache's GPU")
        self.k_codes, self.k_scales, self.v_codes, self.v_scales = k_codes, k_scales, v_codes, v_scales
        self.k_tensor_scale, self.v_tensor_scale = k_tensor_scale, v_tensor_scale
        nv = self.fmt == FP4_NVFP4
        self.handle = fp4_kv_cache(
            ctypes.sizeof(fp4_kv_cache), self.fmt, pages, page_size, heads, self.head_dim, 0, k_codes.data_ptr(),
            k_scales.data_ptr(), v_codes.data_ptr(), v_scales.data_ptr(),
            k_codes.stride(0) if pages > 1 else heads * page_size * half,
            k_scales.stride(0) if pages > 1 else heads * page_size * (2 * half // blk),
            k_tensor_scale.data_ptr() if nv else None, v_tensor_scale.data_ptr() if nv else None)
        self._ref = ctypes.byref(self.handle)

    @classmethod
    def empty(cls, fmt, num_pages, page_size, kv_heads, head_dim, *, k_amax=None, v_amax=None, four_over_six=False,
              device="cuda"):
        """A cache of zeros. NVFP4: k_amax and v_amax are the largest
        magnitudes expected of rotated keys and of values (a number, or one
        per kv head), from which the tensor scales derive as in quantize()."""
        import torch
        fmt = _fmt(fmt)
        blk = 16 if fmt == FP4_NVFP4 else 32
        shape = (num_pages, kv_heads, page_size)
        bufs = [torch.zeros(*shape, w, dtype=torch.uint8, device=device)
                for w in (head_dim // 2, head_dim // blk, head_dim // 2, head_dim // blk)]
        scales = [None, None]
        if fmt == FP4_NVFP4:
            if k_amax is None or v_amax is None:
                raise ValueError("NVFP4 needs k_amax and v_amax")
            # a quotient of tensors is correctly rounded, as fp4_quantize's is (one by a number need not be)
            div = torch.tensor(1792.0 if four_over_six else 2688.0, dtype=torch.float32, device=device)
            scales = [(torch.as_tensor(a, dtype=torch.float32, device=device).expand(kv_heads)
                       / div.expand(kv_heads)).contiguous() for a in (k_amax, v_amax)]
        return cls(fmt, *bufs, *scales)


# A decode step calls these functions for every layer, and a launch costs less
# host time than careless Python: the checks below are written to be cheap.
def _kv_dtype(t, what):
    import torch
    d = t.dtype
    if d is torch.bfloat16:
        return FP4_BF16
    if d is torch.float32:
        return FP4_F32
    raise ValueError(f"{what} must be bfloat16 or float32")


def _kv_rows(t, cache, what):
    """Check a [tokens, heads, head_dim] operand (rows dense, any strides);
    returns its shape and strides."""
    shape, strides = t.shape, t.stride()
    if len(shape) != 3 or shape[2] != cache.head_dim:
        raise ValueError(f"{what} must be [tokens, heads, head_dim]")
    if strides[2] != 1:
        raise ValueError(f"{what} rows must be contiguous")
    if t.get_device() != cache.index:
        raise ValueError(f"{what} must be on the cache's GPU")
    return shape, strides


def _kv_vector(t, cache, n, dtype, what):
    """Check a contiguous device vector of n elements; returns its address."""
    if t.dtype is not dtype or t.dim() != 1 or t.numel() != n or t.get_device() != cache.index or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {dtype} vector of {n} elements on the cache's GPU")
    return t.data_ptr()


def _kv_stream(cache):
    """torch's current stream on the cache's GPU."""
    import torch
    # the handle torch.cuda.current_stream() wraps, without making the object
    return torch._C._cuda_getCurrentRawStream(cache.index)


def _on_cache_gpu(call, cache, *args, **kw):
    """The call again, with the cache's GPU current (outputs and the launch)."""
    import torch
    with torch.cuda.device(cache.index):
        return call(*args, **kw)


def kv_append(cache: KVCache, k, v, slots, *, q=None, positions=None, cos=None, sin=None, interleaved=False,
              four_over_six=False, q_out=None, stream=None):
    """Rotate, quantize and store the keys and values [tokens, kv_heads,
    head_dim] (bf16 or fp32, any token and head strides) of a step's tokens at
    their `slots` (int64 [tokens]: page * page_size + row, -1 for padding),
    and rotate the step's queries [tokens, heads, head_dim]; returns those
    (q_out if given, else a new tensor; None without q).

    cos, sin: fp32 [positions, rotary / 2] tables, rotary being the number of
    leading elements of a row that are rotated, in pairs (i, i + rotary / 2),
    or (2i, 2i + 1) if `interleaved`; positions: int64 [tokens]. Without
    tables nothing is rotated."""
    import torch
    if torch._C._cuda_getDevice() != cache.index:
        return _on_cache_gpu(kv_append, cache, cache, k, v, slots, q=q, positions=positions, cos=cos, sin=sin,
                             interleaved=interleaved, four_over_six=four_over_six, q_out=q_out, stream=stream)
    if stream is not None and stream != _kv_stream(cache):
        return _on_stream(kv_append, cache.device, stream, q_out, cache, k, v, slots, q=q, positions=positions, cos=cos,
                          sin=sin, interleaved=interleaved, four_over_six=four_over_six, q_out=q_out)
    (tokens, kh, _), ks = _kv_rows(k, cache, "k")
    vshape, vs = _kv_rows(v, cache, "v")
    dt = _kv_dtype(k, "k")
    if v.dtype is not k.dtype or kh != cache.kv_heads or vshape != k.shape:
        raise ValueError("k and v must be [tokens, kv_heads, head_dim] of one dtype")
    at_slots = _kv_vector(slots, cache, tokens, torch.int64, "slots")
    rotary = max_position = heads = 0
    at_pos = at_cos = at_sin = at_q = at_out = q0 = q1 = o0 = o1 = 0
    if cos is not None:
        if sin is None or positions is None:
            raise ValueError("rotation needs cos, sin and positions")
        max_position, half = cos.shape
        for t in (cos, sin):
            if (t.dtype is not torch.float32 or t.shape != cos.shape or t.get_device() != cache.index
                    or not t.is_contiguous()):
                raise ValueError("cos and sin must be contiguous float32 tensors of one shape on the cache's GPU")
        at_pos = _kv_vector(positions, cache, tokens, torch.int64, "positions")
        rotary = 2 * half
        at_cos, at_sin = cos.data_ptr(), sin.data_ptr()
    elif sin is not None:
        raise ValueError("rotation needs cos, sin and positions")
    if q is not None:
        qshape, (q0, q1, _) = _kv_rows(q, cache, "q")
        heads = qshape[1]
        if q.dtype is not k.dtype or qshape[0] != tokens:
            raise ValueError("q, k and v must have one dtype and as many tokens")
        if q_out is None:
            q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
            o0, o1 = heads * cache.head_dim, cache.head_dim
        else:
            oshape, (o0, o1, _) = _kv_rows(q_out, cache, "q_out")
            if q_out.dtype is not q.dtype or oshape != qshape:
                raise ValueError("q_out must be like q")
        at_q, at_out = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out without q")
    args = _pack_append(
        _APPEND_SIZE, dt,
        (FP4_FOUR_OVER_SIX if four_over_six else 0) | (FP4_KV_INTERLEAVED if interleaved else 0), heads, tokens,
        k.data_ptr(), v.data_ptr(), at_q, at_out, ks[0], ks[1], vs[0], vs[1], q0, q1, o0, o1, at_slots, at_pos,
        at_cos, at_sin, max_position, rotary, 0)
    st = lib().fp4_kv_append(cache._ref, args, _kv_stream(cache))
    if st != FP4_OK:
        raise Fp4Error(st, "fp4_kv_append")
    return q_out


def kv_read(cache: KVCache, slots, dtype=None, stream=None):
    """The keys and values of the given slots (int64 [tokens]) as plain
    numbers: two [tokens, kv_heads, head_dim] tensors of `dtype` (bf16 unless
    given, or fp32). A slot outside the cache reads as zeros."""
    import torch
    if torch._C._cuda_getDevice() != cache.index:
        return _on_cache_gpu(kv_read, cache, cache, slots, dtype, stream)
    if stream is not None and stream != _kv_stream(cache):
        return _on_stream(kv_read, cache.device, stream, None, cache, slots, dtype)
    tokens = slots.numel()
    at_slots = _kv_vector(slots, cache, tokens, torch.int64, "slots")
    k = slots.new_empty((tokens, cache.kv_heads, cache.head_dim), dtype=dtype or torch.bfloat16)
    dt = _kv_dtype(k, "dtype")
    v = torch.empty_like(k)
    st = lib().fp4_kv_read(cache._ref, tokens, at_slots, k.data_ptr(), v.data_ptr(), dt, _kv_stream(cache))
    if st != FP4_OK:
        raise Fp4Error(st, "fp4_kv_read")
    return k, v


def kv_attention(q, cache: KVCache, block_table, kv_lens, *, q_offsets=None, max_kv_len=None, causal=True, window=0,
                 softcap=0.0, scale=None, return_lse=False, out=None, stream=None):
    """Softmax attention of queries [tokens, heads, head_dim] (bf16 or fp32)
    over the cached rows of their sequences; heads is a multiple of the
    cache's kv_heads, consecutive heads share a kv head.

    block_table int32 [batch, width]: the pages of each sequence in order;
    kv_lens int32 [batch]: its cached rows. q_offsets int32 [batch + 1]: the
    queries of sequence b are rows q_offsets[b]:q_offsets[b + 1]; without it
    every sequence has one. All three are read on the device; max_kv_len
    (default: all the table can hold) bounds kv_lens on the host.

    causal: a sequence's queries are its last tokens, each sees the rows up to
    its own, and with window > 0 only the last `window` of them; otherwise
    every query sees every row. softcap > 0: scores become
    softcap * tanh(score / softcap). scale: default head_dim ** -0.5.
    Returns out (like q), or (out, lse) with fp32 lse [tokens, heads], the
    logarithm of each row's sum of exponentials; rows that see nothing are 0
    and -inf."""
    import torch
    if torch._C._cuda_getDevice() != cache.index:
        return _on_cache_gpu(kv_attention, cache, q, cache, block_table, kv_lens, q_offsets=q_offsets,
                             max_kv_len=max_kv_len, causal=causal, window=window, softcap=softcap, scale=scale,
                             return_lse=return_lse, out=out, stream=stream)
    if stream is not None and stream != _kv_stream(cache):
        return _on_stream(kv_attention, cache.device, stream, out, q, cache, block_table, kv_lens,
                          q_offsets=q_offsets, max_kv_len=max_kv_len, causal=causal, window=window, softcap=softcap, scale=scale,
                          return_lse=return_lse, out=out)
    qshape, (q0, q1, _) = _kv_rows(q, cache, "q")
    dt = _kv_dtype(q, "q")
    tokens, heads, dim = qshape
    if block_table.dim() != 2 or block_table.dtype is not torch.int32 or block_table.get_device() != cache.index:
        raise ValueError("block_table must be an int32 [batch, width] tensor on the cache's GPU")
    batch, width = block_table.shape
    t0, t1 = block_table.stride()
    if width > 1 and t1 != 1:
        raise ValueError("block_table rows must be contiguous")
    at_lens = _kv_vector(kv_lens, cache, batch, torch.int32, "kv_lens")
    at_offs = at_lse = 0
    if q_offsets is not None:
        at_offs = _kv_vector(q_offsets, cache, batch + 1, torch.int32, "q_offsets")
    lse = at_ws = None
    if out is None:
        # (empty_like costs half of empty)
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
        o0, o1 = heads * dim, dim
    else:
        oshape, (o0, o1, _) = _kv_rows(out, cache, "out")
        if out.dtype is not q.dtype or oshape != qshape:
            raise ValueError("out must be like q")
    if return_lse:
        lse = q.new_empty((tokens, heads), dtype=torch.float32)
        at_lse = lse.data_ptr()
    capacity = width * cache.page_size
    args = _pack_attention(
        _ATTENTION_SIZE, dt, FP4_KV_CAUSAL if causal else 0, heads, batch, tokens, at_offs, at_lens,
        block_table.data_ptr(), t0 if batch > 1 else width, width,
        capacity if max_kv_len is None or max_kv_len > capacity else max_kv_len, q.data_ptr(), out.data_ptr(), at_lse,
        q0, q1, o0, o1, dim ** -0.5 if scale is None else scale, softcap, window)
    L = lib()
    need = L.fp4_kv_attention_workspace(cache._ref, args)
    if need:
        ws = q.new_empty((need,), dtype=torch.uint8)
        at_ws = ws.data_ptr()
    st = L.fp4_kv_attention(cache._ref, args, at_ws, need, _kv_stream(cache))
    if st != FP4_OK:
        raise Fp4Error(st, "fp4_kv_attention")
    return (out, lse) if return_lse else out
