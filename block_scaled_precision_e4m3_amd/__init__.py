"""Block-scaled FP8 GEMM with a fused global-amax epilogue on MI355X (gfx950).

Thin Python binding over the C ABI of ``libmxgemm.so`` (declared in
``include/mxgemm.h``).  Every step of the computation runs in the library's
HIP kernels; this module only marshals arguments (PyTorch supplies device
memory and streams).  It fails loudly when the library has not been built.

Low-level functions carry the C names and arguments:
``mxgemm_amax``, ``mxgemm_amax_ex``, ``mxgemm_amax_reset``,
``mxgemm_check_support``, ``mxgemm_sf_bytes``, ``mxgemm_launch_config``,
``mxgemm_strerror``.  Buffers may be torch tensors (their data pointer is
passed) or integer device addresses.

``gemm_amax`` mirrors the page's high-level wrapper ("GEMM + Amax (SM100)",
section "High-level wrapper"): it takes A (M, K, L) / B (N, K, L) k-major
tensors (or (L, M, K)-contiguous storage viewed that way), SF tensors in the
logical atom view or the physical shape, allocates C (M, N, L) n-major and
Amax (1, 1, 1) when not given, and returns (c, amax).
"""

import ctypes
import os

_PKG_DIR = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG_DIR, "libmxgemm.so")

MXG_FMT_E4M3 = 0
MXG_FMT_E5M2 = 1
MXG_FMT_E2M1 = 2
MXG_FLAG_AMAX_ACCUMULATE = 1
MXG_FLAG_FP8_MFMA = 2
MXG_FLAG_TILE_128 = 4
MXG_FLAG_TILE_256 = 8
MXG_FLAG_C_BF16 = 32
MXG_FLAG_C_F16 = 64
MXG_FLAG_C_MMAJOR = 128
MXG_FLAG_A_MMAJOR = 256
MXG_FLAG_B_NMAJOR = 512

MXG_DT_F32 = 0
MXG_DT_BF16 = 1
MXG_DT_F16 = 2
MXG_QUANT_SQUARE = 1
MXG_QUANT_POW2 = 2
MXG_B128_B_ROWS = 1
MXG_B128_ACCUMULATE = 2
MXG_ROPE_HALF = 0
MXG_ROPE_INTERLEAVED = 1
MXG_ROPE_INTERLEAVED_TO_HALF = 2
MXG_ROPE_TRANSPOSE = 1
MXG_ROPE_POS64 = 2
MXG_TRUSTED_POINTERS = 1073741824

MXG_OK = 0
MXG_ERR_NULL = -1
MXG_ERR_SHAPE = -2
MXG_ERR_ALIGN = -3
MXG_ERR_SFVEC = -4
MXG_ERR_FMT = -5
MXG_ERR_DEVICE = -6
MXG_ERR_LAUNCH = -7
MXG_ERR_FLAGS = -8
MXG_ERR_SCRATCH = -9
MXGEMM_NOALLOC_SCRATCH_BYTES = 8 << 20  # fixed per-device scratch of the _noalloc entry

EXPORTED = ("mxgemm_amax", "mxgemm_amax_ex", "mxgemm_amax_reset", "mxgemm_check_support",
            "mxgemm_sf_bytes", "mxgemm_launch_config", "mxgemm_strerror", "mxgemm_mx_quantize",
            "mxgemm_sf_rowwise_to_atoms", "mxgemm_plan_init", "mxgemm_plan_execute", "mxgemm_codes_to_kmajor",
            "mxgemm_proj_rope_mxfp8", "mxgemm_gemm_rope_mxfp8", "mxgemm_projection_workspace_bytes",
            "mxgemm_projection_mxfp8", "mxgemm_projection_mxfp8_noalloc", "mxgemm_block128_quantize", "mxgemm_block128",
            "mxgemm_block128_workspace_bytes", "mxgemm_rope", "mxgemm_qk_norm_rope", "mxgemm_qk_norm_rope_backward",
            "mxgemm_qk_norm_rope_backward_workspace_bytes")


class MxgemmError(Exception):
    def __init__(self, status, msg):
        super().__init__(f"mxgemm status {status}: {msg}")
        self.status = status


class MxgemmValueError(MxgemmError, ValueError):
    pass


class MxgemmRuntimeError(MxgemmError, RuntimeError):
    pass


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it first with "
            "`python -m block_scaled_precision_e4m3_amd._build` (hipcc, gfx950)")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i64, ci, cu = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_uint
    gemm_args = [vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, ci, ci, ci]
    lib.mxgemm_amax.argtypes = gemm_args + [vp]
    lib.mxgemm_amax.restype = ci
    lib.mxgemm_amax_ex.argtypes = gemm_args + [cu, vp]
    lib.mxgemm_amax_ex.restype = ci
    lib.mxgemm_amax_reset.argtypes = [vp, vp]
    lib.mxgemm_amax_reset.restype = ci
    lib.mxgemm_check_support.argtypes = [i64, i64, i64, i64, ci, ci, ci]
    lib.mxgemm_check_support.restype = ci
    lib.mxgemm_sf_bytes.argtypes = [i64, i64, i64, ci]
    lib.mxgemm_sf_bytes.restype = ctypes.c_size_t
    lib.mxgemm_launch_config.argtypes = [i64, i64, i64, i64, ci, ctypes.POINTER(ci), ctypes.POINTER(ci),
                                         ctypes.POINTER(i64)]
    lib.mxgemm_launch_config.restype = ci
    lib.mxgemm_strerror.argtypes = [ci]
    lib.mxgemm_strerror.restype = ctypes.c_char_p
    lib.mxgemm_mx_quantize.argtypes = [vp, vp, vp, i64, i64, i64, ci, ci, vp]
    lib.mxgemm_mx_quantize.restype = ci
    lib.mxgemm_sf_rowwise_to_atoms.argtypes = [vp, vp, i64, i64, i64, ci, vp]
    lib.mxgemm_sf_rowwise_to_atoms.restype = ci
    lib.mxgemm_plan_init.argtypes = [vp, i64, i64, i64, i64, ci, ci, ci, cu]
    lib.mxgemm_plan_init.restype = ci
    lib.mxgemm_plan_execute.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp]
    lib.mxgemm_plan_execute.restype = ci
    lib.mxgemm_codes_to_kmajor.argtypes = [vp, vp, i64, i64, i64, vp]
    lib.mxgemm_codes_to_kmajor.restype = ci
    lib.mxgemm_proj_rope_mxfp8.argtypes = [vp] * 7 + [i64] * 4 + [vp]
    lib.mxgemm_proj_rope_mxfp8.restype = ci
    lib.mxgemm_gemm_rope_mxfp8.argtypes = [vp] * 10 + [i64] * 5 + [ci, ci, ci, vp]
    lib.mxgemm_gemm_rope_mxfp8.restype = ci
    lib.mxgemm_projection_workspace_bytes.argtypes = [i64] * 4
    lib.mxgemm_projection_workspace_bytes.restype = ctypes.c_size_t
    lib.mxgemm_projection_mxfp8.argtypes = [vp] * 10 + [i64] * 5 + [vp, ctypes.c_size_t, vp]
    lib.mxgemm_projection_mxfp8.restype = ci
    lib.mxgemm_projection_mxfp8_noalloc.argtypes = [vp] * 10 + [i64] * 5 + [vp]
    lib.mxgemm_projection_mxfp8_noalloc.restype = ci
    cz, cf, strides = ctypes.c_size_t, ctypes.c_float, ctypes.POINTER(i64)
    lib.mxgemm_block128_quantize.argtypes = [vp, i64, vp, vp, vp, vp, i64, i64, i64, ci, ci, cu, vp]
    lib.mxgemm_block128_quantize.restype = ci
    lib.mxgemm_block128.argtypes = [vp] * 5 + [i64] * 5 + [ci, ci, ci, cu, vp, cz, vp]
    lib.mxgemm_block128.restype = ci
    lib.mxgemm_block128_workspace_bytes.argtypes = [i64] * 4 + [ci]
    lib.mxgemm_block128_workspace_bytes.restype = cz
    lib.mxgemm_rope.argtypes = [vp] * 5 + [strides] + [i64] * 6 + [ci, ci, cu, vp]
    lib.mxgemm_rope.restype = ci
    lib.mxgemm_qk_norm_rope.argtypes = [vp] * 9 + [strides] + [i64] * 7 + [cf, ci, ci, ci, cu, vp]
    lib.mxgemm_qk_norm_rope.restype = ci
    lib.mxgemm_qk_norm_rope_backward.argtypes = [vp] * 13 + [strides] + [i64] * 7 + [cf, ci, ci, ci, cu, vp, cz, vp]
    lib.mxgemm_qk_norm_rope_backward.restype = ci
    lib.mxgemm_qk_norm_rope_backward_workspace_bytes.argtypes = [i64, i64]
    lib.mxgemm_qk_norm_rope_backward_workspace_bytes.restype = cz
    return lib


_lib = _load()


def _raise(status):
    msg = _lib.mxgemm_strerror(status).decode()
    if status in (MXG_ERR_DEVICE, MXG_ERR_LAUNCH):
        raise MxgemmRuntimeError(status, msg)
    raise MxgemmValueError(status, msg)


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


_raw_stream = _current_device = None  # the cheap current stream and device of torch, once its GPU side is up


def _stream(stream):
    global _raw_stream
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(_current_device())
        import torch
        handle = torch.cuda.current_stream().cuda_stream  # initialises the GPU, or says why it cannot
        _bind_stream(torch)
        return handle
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _bind_stream(torch):
    """The cheap way to the current stream (0.1 us a call instead of 2.7) where this torch has it."""
    global _raw_stream, _current_device
    if hasattr(torch._C, "_cuda_getCurrentRawStream") and hasattr(torch._C, "_cuda_getDevice"):
        _current_device = torch._C._cuda_getDevice
        _raw_stream = torch._C._cuda_getCurrentRawStream


def _new(make, stream, device, scratch=False):
    """make(), a new tensor, for a call on `stream`.  Its memory (and a fill of it) belongs to that stream: memory that
    Python has freed on the current stream may still be in use there by work that is queued, and only what is queued
    after that work may write it.  The caller may use the tensor on the current stream, so that one is waited for, too,
    before its memory is handed out again; a scratch tensor only ever meets `stream`."""
    if stream is None:
        return make()
    import torch
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device) if stream else torch.cuda.default_stream(device)
    here = torch.cuda.current_stream(device)
    if stream == here:
        return make()
    with torch.cuda.stream(stream):
        t = make()
    if not scratch:
        t.record_stream(here)
    return t


def mxgemm_strerror(status):
    return _lib.mxgemm_strerror(int(status)).decode()


def mxgemm_check_support(M, N, K, L, sf_vec_size, a_fmt, b_fmt):
    """Status code (0 = supported) for these sizes and formats; host-only."""
    return _lib.mxgemm_check_support(M, N, K, L, sf_vec_size, a_fmt, b_fmt)


def mxgemm_sf_bytes(MN, K, L, sf_vec_size):
    return _lib.mxgemm_sf_bytes(MN, K, L, sf_vec_size)


def mxgemm_launch_config(M, N, K, L, sf_vec_size, with_grid=True):
    """(tile_m, tile_n, grid) the library would use; grid is None unless with_grid (queries the device)."""
    tm, tn, g = ctypes.c_int(), ctypes.c_int(), ctypes.c_int64()
    st = _lib.mxgemm_launch_config(M, N, K, L, sf_vec_size, ctypes.byref(tm), ctypes.byref(tn),
                                   ctypes.byref(g) if with_grid else None)
    if st != MXG_OK:
        _raise(st)
    return tm.value, tn.value, (g.value if with_grid else None)


def mxgemm_amax_ex(A, B, SFA, SFB, C, Amax, M, N, K, L, sf_vec_size, a_fmt, b_fmt, flags=0, stream=None):
    """C-ABI mxgemm_amax_ex on torch tensors or raw device addresses; raises on a nonzero status."""
    st = _lib.mxgemm_amax_ex(_ptr(A), _ptr(B), _ptr(SFA), _ptr(SFB), _ptr(C), _ptr(Amax),
                             M, N, K, L, sf_vec_size, a_fmt, b_fmt, flags, _stream(stream))
    if st != MXG_OK:
        _raise(st)


def mxgemm_amax(A, B, SFA, SFB, C, Amax, M, N, K, L, sf_vec_size, a_fmt, b_fmt, stream=None):
    """C-ABI mxgemm_amax on torch tensors or raw device addresses; raises on a nonzero status."""
    st = _lib.mxgemm_amax(_ptr(A), _ptr(B), _ptr(SFA), _ptr(SFB), _ptr(C), _ptr(Amax),
                          M, N, K, L, sf_vec_size, a_fmt, b_fmt, _stream(stream))
    if st != MXG_OK:
        _raise(st)


def mxgemm_amax_reset(Amax, stream=None):
    st = _lib.mxgemm_amax_reset(_ptr(Amax), _stream(stream))
    if st != MXG_OK:
        _raise(st)


# --- high-level wrapper ---------------------------------------------------------

def _fmt_of(t):
    import torch
    if t.dtype == torch.float8_e4m3fn:
        return MXG_FMT_E4M3
    if t.dtype == torch.float8_e5m2:
        return MXG_FMT_E5M2
    raise MxgemmValueError(MXG_ERR_FMT, f"A/B dtype must be float8_e4m3fn or float8_e5m2, got {t.dtype}")


def _as_lrk(t, name):
    """Return (storage tensor, rows, K, L, m_major) from a (rows, K, L) view or 2-D.

    k-major views (strides (K, 1, rows*K)) come back as (L, rows, K) storage; m-major ones
    (strides (1, rows, rows*K), the pages' m-major A / n-major B) as (L, K, rows) storage with
    m_major True, which the GEMM reads as it is (MXG_FLAG_A_MMAJOR / MXG_FLAG_B_NMAJOR)."""
    import torch
    if t.dim() == 2:
        t = t.unsqueeze(2)
    if t.dim() != 3:
        raise MxgemmValueError(MXG_ERR_SHAPE, f"{name} must be (rows, K) or (rows, K, L)")
    rows, k, l = t.shape
    base = t.permute(2, 0, 1)
    if base.is_contiguous():
        return base, rows, k, l, False
    mmajor = t.permute(2, 1, 0)
    if mmajor.is_contiguous() and t.dtype in (torch.float8_e4m3fn, torch.float8_e5m2):
        return mmajor, rows, k, l, True
    raise MxgemmValueError(MXG_ERR_ALIGN, f"{name} must be k-major (strides (K, 1, rows*K)) or, for FP8 codes, "
                                          f"m-major (strides (1, rows, rows*K)), batch outermost")


def _workspace_bytes(t):
    """The bytes of a given workspace: those that its memory has, which an expanded tensor's element count is not."""
    if not t.is_contiguous():
        raise MxgemmValueError(MXG_ERR_ALIGN, "workspace must be contiguous")
    return t.numel() * t.element_size()


def proj_rope_mxfp8(y, cos, sin, num_heads, head_dim=192, qk_rope=64, stream=None, out=None):
    """C-ABI mxgemm_proj_rope_mxfp8 on torch tensors: y (tokens, num_heads * head_dim) float32, cos / sin
    (tokens, qk_rope) bfloat16.  Returns (out_fp8_row, out_scales_row, out_fp8_col, out_scales_col) as the
    projection page's wrapper does: codes (tokens, H, D) float8_e4m3fn, scales uint8 (tokens, H, D/32) and
    (tokens/32, H, D); `out` may hold those four tensors preallocated."""
    import torch
    tokens = y.shape[0]
    out = _proj_outputs(tokens, num_heads, head_dim, y.device, out, stream)
    for t, name in ((y, "y"), (cos, "cos"), (sin, "sin")):
        if not t.is_contiguous():
            raise MxgemmValueError(MXG_ERR_ALIGN, f"{name} must be contiguous")
    if y.dtype != torch.float32 or cos.dtype != torch.bfloat16 or sin.dtype != torch.bfloat16:
        raise MxgemmValueError(MXG_ERR_FMT, "y must be float32, cos and sin bfloat16")
    st = _lib.mxgemm_proj_rope_mxfp8(_ptr(y), _ptr(cos), _ptr(sin), _ptr(out[0]), _ptr(out[1]), _ptr(out[2]),
                                     _ptr(out[3]), tokens, num_heads, head_dim, qk_rope, _stream(stream))
    if st != MXG_OK:
        _raise(st)
    return out


def _proj_outputs(tokens, num_heads, head_dim, dev, out, stream):
    import torch
    if out is None:
        out = tuple(_new(lambda: torch.empty((rows, num_heads, cols), dtype=dtype, device=dev), stream, dev)
                    for rows, cols, dtype in ((tokens, head_dim, torch.float8_e4m3fn), (tokens, head_dim // 32, torch.uint8),
                                              (tokens, head_dim, torch.float8_e4m3fn), (tokens // 32, head_dim, torch.uint8)))
    for t, name in zip(out, ("row", "row scales", "col", "col scales")):
        if not t.is_contiguous():
            raise MxgemmValueError(MXG_ERR_ALIGN, f"{name} must be contiguous")
    return out


def gemm_rope_mxfp8(A, B, SFA, SFB, cos, sin, tokens, num_heads, head_dim, qk_rope, K, sf_vec_size=32,
                    a_fmt=MXG_FMT_E4M3, b_fmt=MXG_FMT_E4M3, stream=None, out=None):
    """C-ABI mxgemm_gemm_rope_mxfp8: the projection GEMM with RoPE and dual-direction MXFP8 fused into its
    epilogue, on k-major codes A (tokens, K) / B (num_heads * head_dim, K) and atom-layout scales.  Returns
    (out_fp8_row, out_scales_row, out_fp8_col, out_scales_col) shaped as proj_rope_mxfp8's."""
    out = _proj_outputs(tokens, num_heads, head_dim, A.device, out, stream)
    st = _lib.mxgemm_gemm_rope_mxfp8(_ptr(A), _ptr(B), _ptr(SFA), _ptr(SFB), _ptr(cos), _ptr(sin), _ptr(out[0]),
                                     _ptr(out[1]), _ptr(out[2]), _ptr(out[3]), tokens, num_heads, head_dim, qk_rope,
                                     K, sf_vec_size, a_fmt, b_fmt, _stream(stream))
    if st != MXG_OK:
        _raise(st)
    return out


def projection_mxfp8(x, w, x_scale, w_scale, cos, sin, num_heads, head_dim=192, qk_rope=64, workspace=None,
                     stream=None, out=None):
    """C-ABI mxgemm_projection_mxfp8, the projection page's MXFP8-input path: x (tokens, K) and w
    (num_heads * head_dim, K) E4M3 codes, row-wise E8M0 scales x_scale (tokens, ceil(K/32)) and w_scale
    (num_heads * head_dim, ceil(K/32)), bf16 cos / sin (tokens, qk_rope).  Allocates the workspace when
    not given.  Returns the four outputs as proj_rope_mxfp8 does."""
    import torch
    tokens, k = x.shape
    need = _lib.mxgemm_projection_workspace_bytes(tokens, num_heads, head_dim, k)
    if workspace is None:
        workspace = _new(lambda: torch.empty(need, dtype=torch.uint8, device=x.device), stream, x.device, True)
    out = _proj_outputs(tokens, num_heads, head_dim, x.device, out, stream)
    st = _lib.mxgemm_projection_mxfp8(_ptr(x), _ptr(w), _ptr(x_scale), _ptr(w_scale), _ptr(cos), _ptr(sin),
                                      _ptr(out[0]), _ptr(out[1]), _ptr(out[2]), _ptr(out[3]), tokens, num_heads,
                                      head_dim, qk_rope, k, _ptr(workspace), _workspace_bytes(workspace),
                                      _stream(stream))
    if st != MXG_OK:
        _raise(st)
    return out


def projection_mxfp8_noalloc(x, w, x_scale, w_scale, cos, sin, num_heads, head_dim=192, qk_rope=64,
                             stream=None, out=None):
    """C-ABI mxgemm_projection_mxfp8_noalloc: projection_mxfp8 with the workspace taken from the library's
    fixed per-device scratch array (nothing is allocated; `out` must then be given by a caller that cannot
    allocate either).  Calls that overlap on one device race."""
    tokens, k = x.shape
    out = _proj_outputs(tokens, num_heads, head_dim, x.device, out, stream)
    st = _lib.mxgemm_projection_mxfp8_noalloc(_ptr(x), _ptr(w), _ptr(x_scale), _ptr(w_scale), _ptr(cos),
                                              _ptr(sin), _ptr(out[0]), _ptr(out[1]), _ptr(out[2]), _ptr(out[3]),
                                              tokens, num_heads, head_dim, qk_rope, k, _stream(stream))
    if st != MXG_OK:
        _raise(st)
    return out


def codes_to_kmajor(src, dst, MN, K, L, stream=None):
    """C-ABI mxgemm_codes_to_kmajor: (L, K, MN) codes into (L, MN, K); raises on a nonzero status."""
    st = _lib.mxgemm_codes_to_kmajor(_ptr(src), _ptr(dst), MN, K, L, _stream(stream))
    if st != MXG_OK:
        _raise(st)


def _sf_phys(t, mn, k, l, sf):
    """Accept the logical SF view (32, 4, MNb, 4, Kg, L) or the physical (L, MNb, Kg, 32, 4, 4) / flat bytes."""
    import torch
    mnb, kg = -(-mn // 128), -(-k // (4 * sf))
    logical = (32, 4, mnb, 4, kg, l)
    if tuple(t.shape) == logical and t.dim() == 6:
        t = t.permute(5, 2, 4, 0, 1, 3)
    if not t.is_contiguous():
        raise MxgemmValueError(MXG_ERR_ALIGN, "SF tensor must be the physical buffer or its logical view")
    if t.dtype != torch.uint8:
        t = t.view(torch.uint8)
    if t.numel() != 512 * l * mnb * kg:
        raise MxgemmValueError(MXG_ERR_SHAPE, f"SF tensor has {t.numel()} bytes, expected {512 * l * mnb * kg}")
    return t


def gemm_amax(a, b, sfa, sfb, c=None, amax=None, sf_vec_size=32, stream=None, accumulate=False, fp8_mfma=False,
              c_dtype=None, c_major="n"):
    """(c, amax) = block-scaled GEMM + amax of torch FP8 tensors; see the module docstring.

    C is float32 by default; c_dtype (or a preallocated c) of torch.bfloat16 / torch.float16
    stores the accumulators rounded to nearest even (amax still from the float32 values).
    c_major: "n" (C strides (N, 1, M*N), the default) or "m" (strides (1, M, M*N), float32),
    as the pages' wrapper argument of that name."""
    import torch
    a_base, m, k, l, a_mm = _as_lrk(a, "A")
    b_base, n, kb, lb, b_mm = _as_lrk(b, "B")
    if kb != k or lb != l:
        raise MxgemmValueError(MXG_ERR_SHAPE, "A and B disagree on K or L")
    fa, fb = _fmt_of(a), _fmt_of(b)
    sfa_p = _sf_phys(sfa, m, k, l, sf_vec_size)
    sfb_p = _sf_phys(sfb, n, k, l, sf_vec_size)
    if c_major not in ("n", "m"):
        raise MxgemmValueError(MXG_ERR_FLAGS, f"c_major must be 'n' or 'm', got {c_major!r}")
    if c_major == "m":
        if c is None:
            c = _new(lambda: torch.empty((l, n, m), dtype=c_dtype or torch.float32, device=a.device), stream,
                     a.device).permute(2, 1, 0)
        c_base = c.permute(2, 1, 0) if c.dim() == 3 else c.t().unsqueeze(0)
        c_flag = MXG_FLAG_C_MMAJOR if c.dtype == torch.float32 else None
        if c_flag is None or not c_base.is_contiguous():
            raise MxgemmValueError(MXG_ERR_ALIGN, "m-major C must be float32 (M, N, L) with strides (1, M, M*N)")
    else:
        if c is None:
            c = _new(lambda: torch.empty((l, m, n), dtype=c_dtype or torch.float32, device=a.device), stream,
                     a.device).permute(1, 2, 0)
        c_base = c.permute(2, 0, 1) if c.dim() == 3 else c.unsqueeze(0)
        c_flag = {torch.float32: 0, torch.bfloat16: MXG_FLAG_C_BF16, torch.float16: MXG_FLAG_C_F16}.get(c.dtype)
        if c_flag is None or not c_base.is_contiguous():
            raise MxgemmValueError(MXG_ERR_ALIGN, "C must be float32, bfloat16 or float16, n-major (M, N, L) with "
                                                  "strides (N, 1, M*N)")
    if amax is None:
        amax = _new(lambda: torch.zeros((1, 1, 1), dtype=torch.float32, device=a.device), stream, a.device)
    flags = (MXG_FLAG_AMAX_ACCUMULATE if accumulate else 0) | (MXG_FLAG_FP8_MFMA if fp8_mfma else 0) | c_flag | \
        (MXG_FLAG_A_MMAJOR if a_mm else 0) | (MXG_FLAG_B_NMAJOR if b_mm else 0)
    mxgemm_amax_ex(a_base, b_base, sfa_p, sfb_p, c_base, amax, m, n, k, l, sf_vec_size, fa, fb, flags, stream)
    return c, amax


def mxgemm_mx_quantize(X, Q, SF, MN, K, L, sf_vec_size, fmt, stream=None):
    """C-ABI mxgemm_mx_quantize on torch tensors or raw device addresses; raises on a nonzero status."""
    st = _lib.mxgemm_mx_quantize(_ptr(X), _ptr(Q), _ptr(SF), MN, K, L, sf_vec_size, fmt, _stream(stream))
    if st != MXG_OK:
        _raise(st)


class Plan:
    """A validated, configured GEMM + amax launch (C-ABI mxgemm_plan): the pages' class API
    (check_support -> compile -> execute), with the per-call host work reduced to pointer checks.

    plan = Plan(M, N, K, L, sf_vec_size, a_fmt, b_fmt, flags); plan(A, B, SFA, SFB, C, Amax, stream)
    """

    class _C(ctypes.Structure):
        _fields_ = [("opaque", ctypes.c_uint64 * 32)]

    def __init__(self, M, N, K, L, sf_vec_size, a_fmt, b_fmt, flags=0):
        self._plan = Plan._C()
        self._ref = ctypes.byref(self._plan)
        st = _lib.mxgemm_plan_init(self._ref, M, N, K, L, sf_vec_size, a_fmt, b_fmt, flags)
        if st != MXG_OK:
            _raise(st)

    def __call__(self, A, B, SFA, SFB, C, Amax, stream=None):
        st = _lib.mxgemm_plan_execute(self._ref, _ptr(A), _ptr(B), _ptr(SFA), _ptr(SFB), _ptr(C), _ptr(Amax),
                                      _stream(stream))
        if st != MXG_OK:
            _raise(st)


def mxgemm_sf_rowwise_to_atoms(rowwise, SF, MN, K, L, sf_vec_size, stream=None):
    """C-ABI mxgemm_sf_rowwise_to_atoms on torch tensors or raw device addresses; raises on a nonzero status."""
    st = _lib.mxgemm_sf_rowwise_to_atoms(_ptr(rowwise), _ptr(SF), MN, K, L, sf_vec_size, _stream(stream))
    if st != MXG_OK:
        _raise(st)


def sf_from_rowwise(rowwise, k, sf_vec_size=32, sf=None, stream=None):
    """Atom-layout scales (L, ceil(MN/128), ceil(K/(4 sf)), 32, 4, 4) uint8 from a contiguous row-wise
    uint8 CUDA tensor (MN, ceil(K/sf)) or (L, MN, ceil(K/sf)) of E8M0 bytes (e.g. the pages' x_scale)."""
    import torch
    if rowwise.element_size() != 1 or not rowwise.is_contiguous() or rowwise.dim() not in (2, 3):
        raise MxgemmValueError(MXG_ERR_SHAPE, "row-wise scales must be a contiguous one-byte (MN, Kb) or "
                                              "(L, MN, Kb) tensor")
    l, mn, kb = (1,) + tuple(rowwise.shape) if rowwise.dim() == 2 else tuple(rowwise.shape)
    if kb != -(-k // sf_vec_size):
        raise MxgemmValueError(MXG_ERR_SHAPE, f"row-wise scales have {kb} blocks per row, K={k} needs "
                                              f"{-(-k // sf_vec_size)}")
    shape = (l, -(-mn // 128), -(-k // (4 * sf_vec_size)), 32, 4, 4)
    if sf is None:
        sf = _new(lambda: torch.empty(shape, dtype=torch.uint8, device=rowwise.device), stream, rowwise.device)
    if sf.numel() != 512 * shape[0] * shape[1] * shape[2] or not sf.is_contiguous():
        raise MxgemmValueError(MXG_ERR_SHAPE, "sf must be a contiguous buffer of the atom layout's size")
    mxgemm_sf_rowwise_to_atoms(rowwise, sf, mn, k, l, sf_vec_size, stream)
    return sf


def mx_quantize(x, sf_vec_size=32, fmt=MXG_FMT_E4M3, q=None, sf=None, stream=None):
    """MX-quantise a contiguous float32 CUDA tensor x of shape (MN, K) or (L, MN, K).

    Returns (q, sf): q uint8 codes of x's shape (view it as torch.float8_e4m3fn /
    float8_e5m2 for gemm_amax) and sf, the physical atom-layout scale buffer
    (L, ceil(MN/128), ceil(K/(4 sf)), 32, 4, 4) uint8, which gemm_amax accepts
    as SFA / SFB.  Preallocated q / sf are used when given.
    """
    import torch
    if x.dtype != torch.float32 or not x.is_contiguous() or x.dim() not in (2, 3):
        raise MxgemmValueError(MXG_ERR_ALIGN, "x must be a contiguous float32 (MN, K) or (L, MN, K) tensor")
    l, mn, k = (1,) + tuple(x.shape) if x.dim() == 2 else tuple(x.shape)
    shape = (l, -(-mn // 128), -(-k // (4 * sf_vec_size)), 32, 4, 4)
    if q is None:
        q = _new(lambda: torch.empty(x.shape, dtype=torch.uint8, device=x.device), stream, x.device)
    if sf is None:
        sf = _new(lambda: torch.empty(shape, dtype=torch.uint8, device=x.device), stream, x.device)
    if q.numel() != x.numel() or not q.is_contiguous() or q.element_size() != 1:
        raise MxgemmValueError(MXG_ERR_SHAPE, "q must be a contiguous one-byte tensor with x's element count")
    if sf.numel() != 512 * shape[0] * shape[1] * shape[2] or not sf.is_contiguous():
        raise MxgemmValueError(MXG_ERR_SHAPE, f"sf must be a contiguous buffer of {512 * shape[0] * shape[1] * shape[2]} bytes")
    mxgemm_mx_quantize(x, q, sf, mn, k, l, sf_vec_size, fmt, stream)
    return q, sf


# --- block-128 quantisation and product, rotary positions, per-head norm -----------

_ROPE_LAYOUTS = {"half": MXG_ROPE_HALF, "interleaved": MXG_ROPE_INTERLEAVED,
                 "interleaved_to_half": MXG_ROPE_INTERLEAVED_TO_HALF}


class _Torch:
    """What the wrappers below need of torch, bound on first use."""

    def __init__(self):
        import torch
        try:
            from . import _bind
        except ImportError as e:  # a library built without torch at hand: every call goes through the checks below
            _bind = None
            if os.path.exists(os.path.join(_PKG_DIR, "_bind.so")):
                import warnings
                warnings.warn(f"_bind.so does not load, calls take more host time: {e}", RuntimeWarning, stacklevel=3)
        else:
            _bind.on_status(_raise)
        self.torch, self.fast = torch, _bind
        self.empty = torch.empty_strided
        self.f32, self.bf16, self.u8 = torch.float32, torch.bfloat16, torch.uint8
        self.i32, self.i64 = torch.int32, torch.int64
        self.dt = {torch.float32: MXG_DT_F32, torch.bfloat16: MXG_DT_BF16, torch.float16: MXG_DT_F16}
        self.fmt = {torch.float8_e4m3fn: MXG_FMT_E4M3, torch.float8_e5m2: MXG_FMT_E5M2}
        self.code = {MXG_FMT_E4M3: torch.float8_e4m3fn, MXG_FMT_E5M2: torch.float8_e5m2}
        self.rope, self.norm = _differentiable(torch)


_env = None


def _torch():
    global _env
    if _env is None:
        _env = _Torch()
    return _env


def _refuse(status, msg):
    raise MxgemmValueError(status, msg)


def _here(dev, *tensors):
    """The device check of the C entry points, for tensors that know their device: all on the current one, which
    lets the call say MXG_TRUSTED_POINTERS."""
    for t in tensors:
        if t is not None and t.get_device() != dev:
            _raise(MXG_ERR_DEVICE)
    if dev < 0 or dev != (_current_device or _env.torch.cuda.current_device)():
        _raise(MXG_ERR_DEVICE)


def _empty(e, shape, dtype, device, stream, scratch=False):
    """A new contiguous tensor for a kernel on `stream`."""
    n = len(shape)
    if n == 2:
        strides = (shape[1] or 1, 1)
    elif n == 3:
        b, c = shape[1] or 1, shape[2] or 1
        strides = (b * c, c, 1)
    else:
        strides = (1,)
    return _new(lambda: e.empty(shape, strides, dtype=dtype, device=device), stream, device, scratch)


def _changed(e, *tensors):
    """Tensors of the caller's that a call has written: autograd must not take them for what they were."""
    for t in tensors:
        if t is not None and not t.is_inference():
            e.torch.autograd.graph.increment_version(t)


def _history(e, out, *tensors):
    """Whether a call's result needs a history; one that goes into `out` cannot have any."""
    if not e.torch.is_grad_enabled() or not any(t is not None and t.requires_grad for t in (*tensors, *(out or ()))):
        return False
    if out is not None:
        _refuse(MXG_ERR_FLAGS, "out has no gradient: call without out, or under torch.no_grad()")
    return True


def _differentiable(torch):
    """The differentiable forms of rope and qk_norm_rope."""
    def features(g):
        # an expanded gradient (of a sum) has no features side by side
        return g if g.shape[2] <= 1 or g.stride(2) == 1 else g.contiguous()

    class Rope(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, cos, sin, positions, layout, rot_offset, transpose, stream):
            ctx.save_for_backward(cos, sin, positions)
            ctx.how = layout, rot_offset, transpose
            return rope(x, cos, sin, positions, layout, rot_offset, transpose, stream=stream)

        @staticmethod
        def backward(ctx, g):
            layout, rot_offset, transpose = ctx.how
            return rope(features(g), *ctx.saved_tensors, layout, rot_offset, not transpose), *(None,) * 7

    class Norm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, q_weight, k_weight, cos, sin, positions, eps, layout, rot_offset, stream):
            ctx.save_for_backward(q, k, q_weight, k_weight, cos, sin, positions)
            ctx.how = eps, layout, rot_offset
            return qk_norm_rope(q, k, q_weight, k_weight, cos, sin, positions, eps, layout, rot_offset, stream=stream)

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, gq, gk):
            q, k, q_weight, k_weight = ctx.saved_tensors[:4]
            gk = None if k is None else features(gk)
            dq, dk, dwq, dwk = qk_norm_rope_backward(features(gq), gk, *ctx.saved_tensors, *ctx.how)
            return dq, dk, dwq.to(q_weight.dtype), None if dwk is None else dwk.to(k_weight.dtype), *(None,) * 7
    return Rope, Norm


def _expect(t, shape, dtype, name):
    """Checks of a contiguous operand or output given by the caller."""
    if t.shape != shape:
        _refuse(MXG_ERR_SHAPE, f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        _refuse(MXG_ERR_FMT, f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        _refuse(MXG_ERR_ALIGN, f"{name} must be contiguous")


def _matrix_rows(t, name):
    """(leading dimensions, L, rows, columns, row stride) of a (rows, columns) or (L, rows, columns) tensor whose
    columns are contiguous and whose rows are evenly spaced, over batches too."""
    sh, st = t.shape, t.stride()
    if len(sh) == 2:
        m, k = sh
        ld = st[0] if m > 1 else k
        ok = True
        l, lead = 1, ()
    else:
        l, m, k = sh
        lead = (l,)
        ld = st[1] if m > 1 else (st[0] if l > 1 else k)
        ok = l <= 1 or m * k == 0 or st[0] == m * ld
    if not ok or ld < k or (k > 1 and st[-1] != 1):
        _refuse(MXG_ERR_ALIGN, f"{name} must have contiguous rows, evenly spaced over rows and batches")
    return lead, l, m, k, ld


def block128_quantize(x, fmt=MXG_FMT_E4M3, rows=True, cols=False, square=False, pow2=False, out=None, stream=None):
    """C-ABI mxgemm_block128_quantize: 8-bit codes of x with one float32 scale per block of 128.

    x is (M, K) or (L, M, K) float32, bfloat16 or float16, K contiguous (rows may be further apart).  Returns
    (q, s, qt, st), None for what is not asked for, with a leading L where x has one:

    rows: q (M, K16) codes in blocks of 1 x 128, K16 = K rounded up to 16 (codes past K zero), s (ceil(K/128), M);
    cols: qt (K, M16) codes of the transpose in blocks of 128 along M, st (ceil(M/128), K): the operand of a
    product over M (a weight gradient);
    square: blocks of 128 x 128, s (ceil(M/128), ceil(K/128)) and st its transpose (a weight, for the forward
    product and the input gradient).

    pow2: scales are powers of two.  out: those four tensors preallocated (None where not wanted).

    Codes and scales have no gradient; a layer that trains through them defines its own (examples/attention_input.py)."""
    e = _env or _torch()
    if out is None and stream is None and e.fast is not None:
        done = e.fast.quantize(x, fmt, rows, cols, square, pow2)
        if done is not None:
            return done
    dt = e.dt.get(x.dtype)
    if dt is None:
        _refuse(MXG_ERR_FMT, "x must be float32, bfloat16 or float16")
    if x.dim() not in (2, 3):
        _refuse(MXG_ERR_SHAPE, "x must be (M, K) or (L, M, K)")
    f8 = e.code.get(fmt)
    if f8 is None:
        _refuse(MXG_ERR_FMT, "fmt must be MXG_FMT_E4M3 or MXG_FMT_E5M2")
    if not rows and not cols:
        _refuse(MXG_ERR_NULL, "neither rows nor cols asked for")
    lead, l, m, k, ldx = _matrix_rows(x, "x")
    kb, mb = -(-k // 128), -(-m // 128)
    q = s = qt = st = None
    if out is not None:
        q, s, qt, st = out
        for t, want, name in ((q, rows, "q"), (s, rows, "s"), (qt, cols, "qt"), (st, cols, "st")):
            if (t is not None) != bool(want):
                _refuse(MXG_ERR_NULL, f"{name} given but not asked for, or the reverse")
    dev = x.get_device()
    _here(dev, q, s, qt, st) if out is not None or dev < 0 else _here(dev)
    if rows:
        qs, ss = lead + (m, -(-k // 16) * 16), lead + ((mb, kb) if square else (kb, m))
        if q is None:
            q, s = _empty(e, qs, f8, x.device, stream), _empty(e, ss, e.f32, x.device, stream)
        else:
            _expect(q, qs, f8, "q")
            _expect(s, ss, e.f32, "s")
    if cols:
        qs, ss = lead + (k, -(-m // 16) * 16), lead + ((kb, mb) if square else (mb, k))
        if qt is None:
            qt, st = _empty(e, qs, f8, x.device, stream), _empty(e, ss, e.f32, x.device, stream)
        else:
            _expect(qt, qs, f8, "qt")
            _expect(st, ss, e.f32, "st")
    status = _lib.mxgemm_block128_quantize(_ptr(x), ldx, _ptr(q), _ptr(s), _ptr(qt), _ptr(st), m, k, l, dt, fmt,
                                           (MXG_QUANT_SQUARE if square else 0) | (MXG_QUANT_POW2 if pow2 else 0)
                                           | MXG_TRUSTED_POINTERS, _stream(stream))
    if status != MXG_OK:
        _raise(status)
    if out is not None:
        _changed(e, q, s, qt, st)
    return q, s, qt, st


def block128_gemm(a, sa, b, sb, b_block=128, c_dtype=None, c=None, accumulate=False, workspace=None, stream=None):
    """C-ABI mxgemm_block128: c (M, N) = a b^T of block-128 quantised operands, as block128_quantize makes them.

    a (M, K) codes with sa (ceil(K/128), M), b (N, K) codes with sb (ceil(N/128), ceil(K/128)) for b_block=128 or
    (ceil(K/128), N) for b_block=1; K a multiple of 16; all with a leading L or none; E4M3 or E5M2 each.  c_dtype:
    float32, bfloat16 (the default) or float16.  c: the output, whose rows may be further apart than N; accumulate
    adds to a float32 c.

    A float32 c is exact up to float32 rounding.  A 16-bit c is made on the 8-bit matrix cores, which drop a little inside
    groups of 8 K elements (include/mxgemm.h): far less than c's own rounding on ordinary data, but more where large terms
    cancel; take a float32 c and round it where that matters.

    The product has no history for autograd: codes have no gradient (see block128_quantize)."""
    e = _env or _torch()
    if stream is None and workspace is None and e.fast is not None:
        done = e.fast.gemm(a, sa, b, sb, b_block, c_dtype, c, accumulate)
        if done is not None:
            return done
    fa, fb = e.fmt.get(a.dtype), e.fmt.get(b.dtype)
    if fa is None or fb is None:
        _refuse(MXG_ERR_FMT, "a and b must be float8_e4m3fn or float8_e5m2")
    sh, bh = a.shape, b.shape
    if len(sh) == 2 and len(bh) == 2:
        (m, k), n, l, lead = sh, bh[0], 1, ()
    elif len(sh) == 3 and len(bh) == 3 and sh[0] == bh[0]:
        (l, m, k), n = sh, bh[1]
        lead = (l,)
    else:
        _refuse(MXG_ERR_SHAPE, "a and b must be (M, K) and (N, K), or (L, M, K) and (L, N, K)")
    if bh[-1] != k:
        _refuse(MXG_ERR_SHAPE, f"a and b disagree on K: {k} and {bh[-1]}")
    if b_block not in (1, 128):
        _refuse(MXG_ERR_SHAPE, "b_block must be 1 or 128")
    if sa is None or sb is None:
        _refuse(MXG_ERR_NULL, "sa and sb must be given")
    kb = -(-k // 128)
    _expect(sa, lead + (kb, m), e.f32, "sa")
    _expect(sb, lead + ((kb, n) if b_block == 1 else (-(-n // 128), kb)), e.f32, "sb")
    if not a.is_contiguous() or not b.is_contiguous():
        _refuse(MXG_ERR_ALIGN, "a and b must be contiguous")
    if c is not None:
        _history(e, (c,))
        if c.shape != lead + (m, n):
            _refuse(MXG_ERR_SHAPE, f"c must have shape {lead + (m, n)}, got {tuple(c.shape)}")
        if c_dtype is not None and c.dtype != c_dtype:
            _refuse(MXG_ERR_FMT, f"c must be {c_dtype}, got {c.dtype}")
        c_dtype, ldc = c.dtype, _matrix_rows(c, "c")[4]
    elif accumulate:
        _refuse(MXG_ERR_NULL, "accumulate needs c")
    else:
        ldc = n
        if c_dtype is None:
            c_dtype = e.bf16
    ct = e.dt.get(c_dtype)
    if ct is None:
        _refuse(MXG_ERR_FMT, "c must be float32, bfloat16 or float16")
    given = 0 if workspace is None else _workspace_bytes(workspace)
    _here(a.get_device(), sa, b, sb, c, workspace)
    own = c is None
    if own:
        c = _empty(e, lead + (m, n), c_dtype, a.device, stream)
    need = _lib.mxgemm_block128_workspace_bytes(m, n, k, l, ct)
    if need and workspace is None:
        workspace, given = _empty(e, (need,), e.u8, a.device, stream, True), need
    st = _lib.mxgemm_block128(a.data_ptr(), sa.data_ptr(), b.data_ptr(), sb.data_ptr(), c.data_ptr(), ldc, m, n, k, l,
                              fa, fb, ct, (MXG_B128_B_ROWS if b_block == 1 else 0)
                              | (MXG_B128_ACCUMULATE if accumulate else 0) | MXG_TRUSTED_POINTERS, _ptr(workspace), given,
                              _stream(stream))
    if st != MXG_OK:
        _raise(st)
    if not own:
        _changed(e, c)
    return c


def rope_table(length, rot, base=10000.0, scaling="none", factor=1.0, original_length=4096, beta_fast=32.0,
               beta_slow=1.0, device="cuda"):
    """(cos, sin) float32 tables (length, rot/2) for rope and qk_norm_rope, computed on the host in float64.

    Pair i turns by position * base^(-2i/rot).  scaling stretches that for contexts `factor` times longer than the
    original_length the weights were trained on:

    "linear": every frequency divided by factor;
    "ntk": base raised so that the slowest pair is stretched by factor and the fastest kept;
    "yarn": pairs that turn more than beta_fast times within original_length are kept, those below beta_slow
    turns are divided by factor, a linear ramp over the pair index in between (from the pair index of beta_fast turns,
    rounded down and not below 0, to that of beta_slow turns, rounded up and not above rot - 1), and cos and sin are
    multiplied by 0.1 ln(factor) + 1 (Peng et al., "YaRN: Efficient Context Window Extension of Large Language Models",
    2023)."""
    import numpy as np
    import torch
    if length < 0 or rot < 0 or rot % 2:
        raise MxgemmValueError(MXG_ERR_SHAPE, "length must not be negative and rot must be even")
    if scaling not in ("none", "linear", "ntk", "yarn") or factor <= 0:
        raise MxgemmValueError(MXG_ERR_FMT, "scaling must be none, linear, ntk or yarn, and factor positive")
    i = np.arange(rot // 2, dtype=np.float64)
    m = 1.0
    if scaling == "ntk" and rot > 2:
        base = base * factor ** (rot / (rot - 2.0))
    freq = base ** (-2.0 * i / max(rot, 1))
    if scaling == "linear":
        freq = freq / factor
    elif scaling == "yarn":
        # the (fractional) pair that turns a number of times within the original length
        def pair(turns):
            return rot * np.log(original_length / (turns * 2 * np.pi)) / (2 * np.log(base))
        # its ends may lie past the last pair, which is then stretched by a part of factor only
        lo, hi = max(np.floor(pair(beta_fast)), 0.0), min(np.ceil(pair(beta_slow)), rot - 1.0)
        ramp = np.clip((i - lo) / max(hi - lo, 1e-3), 0.0, 1.0)
        freq = freq * (1 - ramp) + freq / factor * ramp
        m = 0.1 * np.log(factor) + 1.0 if factor > 1 else 1.0
    angle = np.arange(length, dtype=np.float64)[:, None] * freq[None, :]
    return (torch.from_numpy((m * np.cos(angle)).astype(np.float32)).to(device),
            torch.from_numpy((m * np.sin(angle)).astype(np.float32)).to(device))


def _rotary(e, cos, sin, positions, tokens, layout):
    """(rot, table rows, layout number, flags) of the rotary arguments."""
    lay = _ROPE_LAYOUTS.get(layout)
    if lay is None:
        _refuse(MXG_ERR_FMT, f"layout must be one of {sorted(_ROPE_LAYOUTS)}")
    if cos is None or sin is None:
        if cos is not None or sin is not None or positions is not None:
            _refuse(MXG_ERR_NULL, "cos and sin come together, and positions with them")
        return 0, 0, lay, MXG_TRUSTED_POINTERS
    table = cos.shape
    if len(table) != 2 or sin.shape != table:
        _refuse(MXG_ERR_SHAPE, "cos and sin must be (table rows, rot / 2)")
    if cos.dtype != e.f32 or sin.dtype != e.f32:
        _refuse(MXG_ERR_FMT, "cos and sin must be float32")
    if not cos.is_contiguous() or not sin.is_contiguous():
        _refuse(MXG_ERR_ALIGN, "cos and sin must be contiguous")
    flags = MXG_TRUSTED_POINTERS
    if positions is not None:
        if positions.shape != (tokens,):
            _refuse(MXG_ERR_SHAPE, "positions must have one entry per token")
        if positions.dtype == e.i64:
            flags |= MXG_ROPE_POS64
        elif positions.dtype != e.i32:
            _refuse(MXG_ERR_FMT, "positions must be int32 or int64")
        if not positions.is_contiguous():
            _refuse(MXG_ERR_ALIGN, "positions must be contiguous")
    return 2 * table[1], table[0], lay, flags


def _heads_of(x, name):
    """Shape and strides of a (T, heads, D) tensor with contiguous features."""
    sh, st = x.shape, x.stride()
    if len(sh) != 3:
        _refuse(MXG_ERR_SHAPE, f"{name} must be (tokens, heads, features)")
    if st[2] != 1 and sh[2] > 1:
        _refuse(MXG_ERR_ALIGN, f"{name} must have contiguous features")
    return sh, st


def _like(t, x, shape, name):
    """Strides of a tensor that must have a (T, heads, D) shape and x's dtype."""
    sh, st = _heads_of(t, name)
    if sh != shape:
        _refuse(MXG_ERR_SHAPE, f"{name} must have shape {tuple(shape)}, got {tuple(sh)}")
    if t.dtype != x.dtype:
        _refuse(MXG_ERR_FMT, f"{name} must be {x.dtype}, got {t.dtype}")
    return st


def _keys(k, q):
    """(shape, strides, heads) of the keys that go with q; k may be None."""
    if k is None:
        return None, (0, 0), 0
    sh, st = _heads_of(k, "k")
    if sh[0] != q.shape[0] or sh[2] != q.shape[2]:
        _refuse(MXG_ERR_SHAPE, "q and k must have the same tokens and features")
    if k.dtype != q.dtype:
        _refuse(MXG_ERR_FMT, f"k must be {q.dtype}, got {k.dtype}")
    return sh, st, sh[1]


def _pair(e, out, q, k, kh, names, stream):
    """Outputs for q and k, new or given: (for q, for k, strides of each)."""
    if out is None:
        yq = _empty(e, q.shape, q.dtype, q.device, stream)
        yk = None if k is None else _empty(e, kh, k.dtype, k.device, stream)
        return yq, yk, yq.stride(), (0, 0) if yk is None else yk.stride()
    yq, yk = out
    if yq is None or (yk is None) != (k is None):
        _refuse(MXG_ERR_NULL, "outputs must be given for q, and for k where there is one")
    return yq, yk, _like(yq, q, q.shape, names[0]), (0, 0) if yk is None else _like(yk, k, kh, names[1])


_Strides4, _Strides8, _Strides12 = ctypes.c_int64 * 4, ctypes.c_int64 * 8, ctypes.c_int64 * 12


def rope(x, cos, sin, positions=None, layout="half", rot_offset=0, transpose=False, out=None, stream=None):
    """C-ABI mxgemm_rope: rotary positions on the heads of x (T, H, D), features contiguous (a view of a wider
    projection output will do), float32, bfloat16 or float16.

    cos, sin: float32 tables (rows, rot / 2) (see rope_table); the features [rot_offset, rot_offset + rot) of every
    head rotate and the others are copied.  positions: (T) int32 or int64 table rows, None for 0, 1, ...; a token
    whose position lies outside the tables gets NaN there.  layout: "half" (pairs i, i + rot/2), "interleaved"
    (pairs 2i, 2i + 1) or "interleaved_to_half" (the latter in, the former out).  transpose: the transposed map, which takes
    the output's gradient to the input's.  out: the result, which may be x; a new tensor by default.

    Differentiable in x (not in the tables) unless out is given."""
    e = _env or _torch()
    if stream is None and e.fast is not None:
        done = e.fast.rope(x, cos, sin, positions, layout, rot_offset, transpose, out)
        if done is not None:
            return done
    if _history(e, out if out is None else (out,), x):
        return e.rope.apply(x, cos, sin, positions, layout, rot_offset, transpose, stream)
    dt = e.dt.get(x.dtype)
    if dt is None:
        _refuse(MXG_ERR_FMT, "x must be float32, bfloat16 or float16")
    sh, xs = _heads_of(x, "x")
    t, h, d = sh
    rot, rows, lay, flags = _rotary(e, cos, sin, positions, t, layout)
    if out is not None:
        os_ = _like(out, x, sh, "out")
    _here(x.get_device(), cos, sin, positions, out)
    own = out is None
    if own:
        out = _empty(e, sh, x.dtype, x.device, stream)
        os_ = out.stride()
    st = _lib.mxgemm_rope(x.data_ptr(), out.data_ptr(), _ptr(cos), _ptr(sin), _ptr(positions),
                          _Strides4(xs[0], xs[1], os_[0], os_[1]), t, h, d, rot, rot_offset, rows, lay, dt,
                          flags | (MXG_ROPE_TRANSPOSE if transpose else 0), _stream(stream))
    if st != MXG_OK:
        _raise(st)
    if not own:
        _changed(e, out)
    return out


def _weights(e, q_weight, k_weight, q, k):
    """MXG_DT_* of the norm weights."""
    if q_weight is None or (k is not None and k_weight is None):
        _refuse(MXG_ERR_NULL, "q_weight must be given, and k_weight with k")
    d, w_dtype = q.shape[2], q_weight.dtype
    if w_dtype not in (q.dtype, e.f32) or (k is not None and k_weight.dtype != w_dtype):
        _refuse(MXG_ERR_FMT, "weights must both be float32 or of the dtype of q and k")
    for w in (q_weight,) if k is None else (q_weight, k_weight):
        if w.shape != (d,):
            _refuse(MXG_ERR_SHAPE, f"weights must have {d} elements")
        if not w.is_contiguous():
            _refuse(MXG_ERR_ALIGN, "weights must be contiguous")
    return e.dt[w_dtype]


def qk_norm_rope(q, k, q_weight, k_weight, cos=None, sin=None, positions=None, eps=1e-6, layout="half", rot_offset=0,
                 out=None, stream=None):
    """C-ABI mxgemm_qk_norm_rope: each head of q (T, Hq, D) and k (T, Hk, D) divided by its root mean square,
    multiplied with its weight (D) and rotated, in one launch.  Returns (q_out, k_out); out: that pair, which may be
    (q, k).  k and k_weight may be None.  cos, sin None: no rotation.  The other arguments are rope's.

    Differentiable once, in q, k and the weights, by qk_norm_rope_backward, unless out is given."""
    e = _env or _torch()
    if out is None and stream is None and e.fast is not None:
        done = e.fast.qk_norm_rope(q, k, q_weight, k_weight, cos, sin, positions, layout, rot_offset, eps)
        if done is not None:
            return done
    if _history(e, out, q, k, q_weight, k_weight):
        return e.norm.apply(q, k, q_weight, k_weight, cos, sin, positions, eps, layout, rot_offset, stream)
    dt = e.dt.get(q.dtype)
    if dt is None:
        _refuse(MXG_ERR_FMT, "q must be float32, bfloat16 or float16")
    (t, hq, d), qs = _heads_of(q, "q")
    kh, ks, hk = _keys(k, q)
    wdt = _weights(e, q_weight, k_weight, q, k)
    rot, rows, lay, flags = _rotary(e, cos, sin, positions, t, layout)
    dev = q.get_device()
    _here(dev, k, q_weight, k_weight, cos, sin, positions)
    yq, yk, yqs, yks = _pair(e, out, q, k, kh, ("q_out", "k_out"), stream)
    if out is not None:
        _here(dev, yq, yk)
    st = _lib.mxgemm_qk_norm_rope(q.data_ptr(), _ptr(k), yq.data_ptr(), _ptr(yk), q_weight.data_ptr(), _ptr(k_weight),
                                  _ptr(cos), _ptr(sin), _ptr(positions),
                                  _Strides8(qs[0], qs[1], ks[0], ks[1], yqs[0], yqs[1], yks[0], yks[1]), t, hq, hk, d,
                                  rot, rot_offset, rows, eps, lay, dt, wdt, flags, _stream(stream))
    if st != MXG_OK:
        _raise(st)
    if out is not None:
        _changed(e, yq, yk)
    return yq, yk


def qk_norm_rope_backward(dq, dk, q, k, q_weight, k_weight, cos=None, sin=None, positions=None, eps=1e-6,
                          layout="half", rot_offset=0, out=None, workspace=None, stream=None):
    """C-ABI mxgemm_qk_norm_rope_backward: from the gradients dq, dk of qk_norm_rope's outputs and its inputs,
    (dq_in, dk_in, dq_weight, dk_weight), the weight gradients float32 (None for a missing k).  out: the first two,
    which may be (dq, dk) or (q, k)."""
    e = _env or _torch()
    if out is None and stream is None and workspace is None and e.fast is not None:
        done = e.fast.qk_norm_rope_backward(dq, dk, q, k, q_weight, k_weight, cos, sin, positions, layout, rot_offset, eps)
        if done is not None:
            return done
    dt = e.dt.get(q.dtype)
    if dt is None:
        _refuse(MXG_ERR_FMT, "q must be float32, bfloat16 or float16")
    qh, qs = _heads_of(q, "q")
    t, hq, d = qh
    kh, ks, hk = _keys(k, q)
    gqs = _like(dq, q, qh, "dq")
    if (dk is None) != (k is None):
        _refuse(MXG_ERR_NULL, "dk must be given with k")
    gks = (0, 0) if dk is None else _like(dk, k, kh, "dk")
    wdt = _weights(e, q_weight, k_weight, q, k)
    rot, rows, lay, flags = _rotary(e, cos, sin, positions, t, layout)
    dev = q.get_device()
    given = 0 if workspace is None else _workspace_bytes(workspace)
    _here(dev, k, dq, dk, q_weight, k_weight, cos, sin, positions, workspace)
    xq, xk, xqs, xks = _pair(e, out, q, k, kh, ("dq_in", "dk_in"), stream)
    if out is not None:
        _here(dev, xq, xk)
    dwq = _empty(e, (d,), e.f32, q.device, stream)
    dwk = None if k is None else _empty(e, (d,), e.f32, q.device, stream)
    if workspace is None:
        given = _lib.mxgemm_qk_norm_rope_backward_workspace_bytes(t, d)
        workspace = _empty(e, (given,), e.u8, q.device, stream, True)
    st = _lib.mxgemm_qk_norm_rope_backward(
        dq.data_ptr(), _ptr(dk), q.data_ptr(), _ptr(k), xq.data_ptr(), _ptr(xk), dwq.data_ptr(), _ptr(dwk),
        q_weight.data_ptr(), _ptr(k_weight), _ptr(cos), _ptr(sin), _ptr(positions),
        _Strides12(gqs[0], gqs[1], gks[0], gks[1], qs[0], qs[1], ks[0], ks[1], xqs[0], xqs[1], xks[0], xks[1]), t, hq, hk,
        d, rot, rot_offset, rows, eps, lay, dt, wdt, flags, workspace.data_ptr(), given, _stream(stream))
    if st != MXG_OK:
        _raise(st)
    if out is not None:
        _changed(e, xq, xk)
    return xq, xk, dwq, dwk


__all__ = [
    "mxgemm_amax", "mxgemm_amax_ex", "mxgemm_amax_reset", "mxgemm_check_support", "mxgemm_sf_bytes",
    "mxgemm_launch_config", "mxgemm_strerror", "gemm_amax", "LIB_PATH", "EXPORTED",
    "mxgemm_mx_quantize", "mx_quantize", "mxgemm_sf_rowwise_to_atoms", "sf_from_rowwise", "Plan",
    "MXG_FMT_E4M3", "MXG_FMT_E5M2", "MXG_FMT_E2M1", "MXG_FLAG_AMAX_ACCUMULATE", "MXG_FLAG_FP8_MFMA", "MXG_FLAG_TILE_128",
    "MXG_FLAG_TILE_256", "MXG_FLAG_C_BF16", "MXG_FLAG_C_F16", "MXG_FLAG_C_MMAJOR", "MXG_FLAG_A_MMAJOR",
    "MXG_FLAG_B_NMAJOR", "codes_to_kmajor",
    "proj_rope_mxfp8", "gemm_rope_mxfp8", "projection_mxfp8", "projection_mxfp8_noalloc", "MxgemmError",
    "MxgemmValueError",
    "MxgemmRuntimeError",
    "block128_quantize", "block128_gemm", "rope_table", "rope", "qk_norm_rope", "qk_norm_rope_backward",
    "MXG_DT_F32", "MXG_DT_BF16", "MXG_DT_F16", "MXG_QUANT_SQUARE", "MXG_QUANT_POW2", "MXG_B128_B_ROWS",
    "MXG_B128_ACCUMULATE", "MXG_ROPE_HALF", "MXG_ROPE_INTERLEAVED", "MXG_ROPE_INTERLEAVED_TO_HALF",
    "MXG_ROPE_TRANSPOSE", "MXG_ROPE_POS64", "MXG_TRUSTED_POINTERS",
]
