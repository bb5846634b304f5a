"""Thin ctypes binding over libtb.so (the C ABI declared in include/tb.h).

Argument marshalling only: tensors are device buffers (torch is used for
device memory and streams), every step of the computation runs in the HIP
kernels behind the C ABI.  There is no fallback: if the library is missing or
a call fails, these functions raise.

Dtypes on the Python side (bit patterns are what matter):
  activations x      torch.bfloat16 (or int16/uint16 bit views)  [rows, K]
  act8 operand       torch.uint8, flat, exactly tb_act8_bytes(B, K) bytes
  weights W          torch.float32 [N, K]
  codes              torch.int32 (uint32 bit patterns): dense [N/16, K/128, 128],
                     2:4 sign plane [N/16, G4, 64, 2] (G4 = ceil(K/512))
  meta               torch.int32, 2:4 only: [N/16, G4, 64, 4]
  scales             torch.float16 (fp16 bit patterns), tile-major: [N/16, K/128, 16]
                     (two-plane [N/16, 2K/128, 16]; 2:4 [N/16, G4, 4, 4, 4])
"""

import ctypes
import os

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libtb.so")

TB_F32, TB_BF16, TB_ACT8, TB_FP8 = 0, 1, 2, 3
TB_FMT_DENSE, TB_FMT_24, TB_FMT_DENSE_MINERR, TB_FMT_DENSE_RESID = 0, 1, 2, 3
TB_EFLAG_NONFINITE, TB_EFLAG_SCALE_OVF = 1, 2
TB_GEMV_MAX_BATCH = 16
TB_MAX_SEGMENTS = 8
TB_NORM_MAX_C = 32768
TB_MAX_DRAFT = 64
TB_NOALLOC_SCRATCH_BYTES = 4 << 20

_lib = None

_i64 = ctypes.c_int64
_vp = ctypes.c_void_p
_int = ctypes.c_int

class FwhtSegment(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("y", ctypes.c_void_p), ("rows", ctypes.c_int64), ("K", ctypes.c_int64),
                ("x_dtype", ctypes.c_int), ("y_dtype", ctypes.c_int), ("x_parts", ctypes.c_int),
                ("reserved", ctypes.c_int)]


class Gemv24Segment(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("meta", ctypes.c_void_p), ("signs", ctypes.c_void_p),
                ("scales", ctypes.c_void_p), ("y", ctypes.c_void_p), ("B", ctypes.c_int64), ("N", ctypes.c_int64),
                ("K", ctypes.c_int64)]


class GemmSegment(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("y", ctypes.c_void_p), ("M", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
                ("y_dtype", ctypes.c_int), ("reserved", ctypes.c_int)]


class GemvSegment(ctypes.Structure):
    _fields_ = [("act", ctypes.c_void_p), ("B", ctypes.c_int64), ("codes", ctypes.c_void_p),
                ("scales", ctypes.c_void_p), ("N", ctypes.c_int64), ("K", ctypes.c_int64), ("y", ctypes.c_void_p),
                ("planes", ctypes.c_int64), ("parts", ctypes.c_int64)]


class BlockNormArgs(ctypes.Structure):
    _fields_ = [("y", _vp), ("resid", _vp), ("w_post", _vp), ("w_pre", _vp), ("gate", _vp), ("h", _vp), ("z", _vp),
                ("rows", _i64), ("C", _i64), ("rows_per_gate", _i64), ("parts", _int), ("y_dtype", _int),
                ("h_dtype", _int), ("w_dtype", _int), ("gate_dtype", _int), ("z_dtype", _int), ("rotate_in", _int),
                ("rotate_out", _int), ("alpha", ctypes.c_float), ("eps", ctypes.c_float)]


class PagedCache(ctypes.Structure):
    _fields_ = [("k_cache", _vp), ("v_cache", _vp), ("k_scale", _vp), ("v_scale", _vp), ("block_table", _vp),
                ("cu_q", _vp), ("kv_len", _vp), ("n_pages", _i64), ("table_stride", _i64), ("table_width", _i64),
                ("B", _i64), ("total_q", _i64), ("max_q", _i64), ("cache_dtype", _int), ("page", _int),
                ("heads_kv", _int), ("head_dim", _int)]


class PagedAttentionArgs(ctypes.Structure):
    _fields_ = [("cache", PagedCache), ("q", _vp), ("out", _vp), ("lse", _vp), ("workspace", _vp),
                ("workspace_bytes", ctypes.c_size_t), ("q_stride", _i64), ("max_kv", _i64), ("window", _i64),
                ("heads_q", _int), ("out_dtype", _int), ("scale", ctypes.c_float), ("reserved", _int)]


class VerifyDraftArgs(ctypes.Structure):
    _fields_ = [("p", _vp), ("q", _vp), ("drafts", _vp), ("u", _vp), ("u_next", _vp), ("cu_draft", _vp),
                ("accepted", _vp), ("tokens", _vp), ("workspace", _vp), ("workspace_bytes", ctypes.c_size_t),
                ("B", _i64), ("total", _i64), ("vocab", _i64), ("p_stride", _i64), ("q_stride", _i64),
                ("max_draft", _int), ("p_dtype", _int), ("q_dtype", _int), ("reserved", _int)]


SIGNATURES = {
    "tb_status_string": (ctypes.c_char_p, [_int]),
    "tb_version": (_int, []),
    "tb_packed_bytes": (_int, [_int, _i64, _i64, ctypes.POINTER(ctypes.c_size_t),
                               ctypes.POINTER(ctypes.c_size_t), ctypes.POINTER(ctypes.c_size_t)]),
    "tb_fwht128": (_int, [_vp, _int, _vp, _int, _i64, _i64, _vp]),
    "tb_fwht128_multi": (_int, [ctypes.POINTER(FwhtSegment), _int, _vp]),
    "tb_ternary_gemv_multi": (_int, [ctypes.POINTER(GemvSegment), _int, _vp]),
    "tb_quantize_pack": (_int, [_vp, _i64, _i64, _int, _vp, _vp, _vp, _vp, _vp]),
    "tb_ternary_gemv": (_int, [_vp, _int, _i64, _vp, _vp, _i64, _i64, _vp, _vp, ctypes.c_size_t, _vp]),
    "tb_ternary_gemv_noalloc": (_int, [_vp, _i64, _vp, _vp, _i64, _i64, _vp, _vp]),
    "tb_ternary_gemv_resid": (_int, [_vp, _int, _i64, _vp, _vp, _i64, _i64, _vp, _vp, ctypes.c_size_t, _vp]),
    "tb_act8_bytes": (ctypes.c_size_t, [_i64, _i64]),
    "tb_act8_prep": (_int, [_vp, _i64, _i64, _vp, _vp]),
    "tb_ternary24_gemv": (_int, [_vp, _i64, _vp, _vp, _vp, _i64, _i64, _vp, _vp]),
    "tb_ternary24_gemv_multi": (_int, [ctypes.POINTER(Gemv24Segment), _int, _vp]),
    "tb_ternary_gemm": (_int, [_vp, _i64, _vp, _vp, _i64, _i64, _vp, _int, _vp]),
    "tb_ternary_gemm_multi": (_int, [ctypes.POINTER(GemmSegment), _int, _vp]),
    "tb_ternary_gemm_splitk_workspace": (ctypes.c_size_t, [_i64, _i64, _i64]),
    "tb_ternary_gemm_splitk": (_int, [_vp, _i64, _vp, _vp, _i64, _i64, _vp, _int, _vp, ctypes.c_size_t, _vp]),
    "tb_ternary_gemm_rotated": (_int, [_vp, _i64, _vp, _vp, _i64, _i64, _vp, _int, _vp, ctypes.c_size_t, _vp]),
    "tb_block_norm": (_int, [ctypes.POINTER(BlockNormArgs), _vp]),
    "tb_paged_append": (_int, [ctypes.POINTER(PagedCache), _vp, _i64, _vp, _i64, _vp]),
    "tb_paged_attention_workspace": (ctypes.c_size_t, [ctypes.POINTER(PagedAttentionArgs)]),
    "tb_paged_attention": (_int, [ctypes.POINTER(PagedAttentionArgs), _vp]),
    "tb_verify_draft_workspace": (ctypes.c_size_t, [_i64, _i64]),
    "tb_verify_draft": (_int, [ctypes.POINTER(VerifyDraftArgs), _vp]),
}


class TBError(RuntimeError):
    def __init__(self, code, where):
        self.code = code
        super().__init__(f"{where}: {status_string(code)}")


def lib():
    """Load libtb.so once; raise if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built; run `python -m ternary_weights_hadamard_amd.build`")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _lib = handle
    return _lib


def status_string(code):
    return lib().tb_status_string(int(code)).decode()


def _check(code, where):
    if code != 0:
        raise TBError(code, where)


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


# the current stream's handle without a Stream object (2.7 us a call on the host)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_raw_device = getattr(torch._C, "_cuda_getDevice", None)


def _stream(stream):
    if stream is None:
        if _raw_stream is not None and _raw_device is not None:
            return ctypes.c_void_p(_raw_stream(_raw_device()))
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dt(t):
    if t.dtype == torch.float32:
        return TB_F32
    if t.dtype == torch.uint8:
        return TB_ACT8
    if t.dtype in (torch.bfloat16, torch.int16, torch.uint16):
        return TB_BF16
    raise TypeError(f"unsupported activation dtype {t.dtype}")


def _dev(*ts):
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("buffers must be contiguous device tensors")


def tb_packed_bytes(fmt, n, k):
    c, m, s = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib().tb_packed_bytes(int(fmt), int(n), int(k), ctypes.byref(c), ctypes.byref(m), ctypes.byref(s)),
           "tb_packed_bytes")
    return c.value, m.value, s.value


def tb_act8_bytes(b, k):
    return int(lib().tb_act8_bytes(int(b), int(k)))


def tb_fwht128(x, y=None, out_dtype=None, stream=None):
    """y[r, 128b + i] = sum_j H[i, j] / sqrt(128) * x[r, 128b + j]; y may be x.
    out_dtype torch.uint8 (or a uint8 y) writes the act8 GEMV operand instead."""
    _dev(x)
    rows = x.numel() // x.shape[-1] if x.numel() else 0
    if y is None:
        if out_dtype == torch.uint8:
            y = torch.empty(tb_act8_bytes(rows, x.shape[-1]), dtype=torch.uint8, device=x.device)
        else:
            y = torch.empty(x.shape, dtype=out_dtype or x.dtype, device=x.device)
    _dev(y)
    _check(lib().tb_fwht128(_p(x), _dt(x), _p(y), _dt(y), rows, x.shape[-1], _stream(stream)), "tb_fwht128")
    return y


def tb_fwht128_multi(pairs, stream=None):
    """One launch rotating several arrays: pairs = [(x, y), ...] or
    [(x, y, x_parts), ...], each with its own dtypes (a uint8 y means the act8
    operand).  With x_parts > 1, x is [x_parts, rows, K] fp32 partial results
    added in order before the transform (y is [rows, K])."""
    if not pairs:
        return
    for p in pairs:
        _dev(p[0], p[1])
    arr = (FwhtSegment * len(pairs))()
    for c, p in enumerate(pairs):
        x, y = p[0], p[1]
        parts = int(p[2]) if len(p) > 2 else 1
        if parts > 1:
            if x.dim() < 2 or x.shape[0] != parts:
                raise ValueError(f"tb_fwht128_multi: x_parts={parts} needs x of shape [{parts}, rows, K], "
                                 f"got {tuple(x.shape)}")
            inner = x[0]
        else:
            inner = x
        rows = inner.numel() // inner.shape[-1] if inner.numel() else 0
        arr[c] = FwhtSegment(x.data_ptr(), y.data_ptr(), rows, x.shape[-1], _dt(x), _dt(y), parts, 0)
    _check(lib().tb_fwht128_multi(arr, len(pairs), _stream(stream)), "tb_fwht128_multi")


def tb_quantize_pack(w, fmt=TB_FMT_DENSE, codes=None, meta=None, scales=None, err_flag=None, stream=None):
    """Quantise fp32 W [N, K]; returns (codes, meta, scales).  For TB_FMT_24 `codes` is the sign plane;
    for TB_FMT_DENSE_RESID codes and scales hold both planes, groups interleaved."""
    _dev(w)
    n, k = w.shape
    dev = w.device
    planes = 2 if fmt == TB_FMT_DENSE_RESID else 1
    g4 = -(-k // 512)  # 2:4 blocks of four groups per tile
    if codes is None:
        shape = (n // 16, planes * k // 128, 128) if fmt != TB_FMT_24 else (n // 16, g4, 64, 2)
        codes = torch.empty(shape, dtype=torch.int32, device=dev)
    if meta is None and fmt == TB_FMT_24:
        meta = torch.empty((n // 16, g4, 64, 4), dtype=torch.int32, device=dev)
    if scales is None:
        shape = (n // 16, planes * k // 128, 16) if fmt != TB_FMT_24 else (n // 16, g4, 4, 4, 4)
        scales = torch.empty(shape, dtype=torch.float16, device=dev)
    _dev(codes, meta, scales, err_flag)
    _check(lib().tb_quantize_pack(_p(w), n, k, int(fmt), _p(codes), _p(meta), _p(scales), _p(err_flag),
                                  _stream(stream)), "tb_quantize_pack")
    return codes, meta, scales


def tb_act8_prep(x, act=None, stream=None):
    """Encode bf16 activations x [B, K] as the act8 operand of tb_ternary_gemv."""
    _dev(x)
    b, k = x.shape
    if act is None:
        act = torch.empty(max(tb_act8_bytes(b, k), 1), dtype=torch.uint8, device=x.device)
    _dev(act)
    _check(lib().tb_act8_prep(_p(x), b, k, _p(act), _stream(stream)), "tb_act8_prep")
    return act


def _act8_operand(act, batch, k, where):
    """Check that `act` is the act8 operand of exactly `batch` rows of length k
    (its scale part starts at byte 4 * batch * k, so the size must match)."""
    if batch is None:
        raise ValueError(f"{where}: an act8 operand needs its batch")
    if batch == 0:
        return  # a no-op call reads nothing
    if act.dtype != torch.uint8 or act.numel() != tb_act8_bytes(batch, k):
        raise ValueError(f"{where}: act8 operand of {batch} rows x {k} must be a uint8 buffer of "
                         f"{tb_act8_bytes(batch, k)} bytes (got {act.dtype}, {act.numel()} elements)")


def _dense_n(scales):
    """Output rows of dense-format scales [N/16, G, 16]."""
    if scales.dim() != 3 or scales.shape[2] != 16:
        raise ValueError(f"dense scales must be [N/16, G, 16] (got {tuple(scales.shape)})")
    return scales.shape[0] * 16


def _gemv(fn, where, x, codes, scales, k, batch, y, workspace, stream):
    _dev(x, codes, scales)
    n = _dense_n(scales)
    if x.dtype == torch.uint8:
        _act8_operand(x, batch, k, where)
        b, dt, wbytes = int(batch), TB_ACT8, 0
    else:
        if x.dtype not in (torch.bfloat16, torch.int16, torch.uint16) or x.dim() != 2 or x.shape[1] != k:
            raise ValueError(f"{where}: x must be bf16 [B, {k}] (got {x.dtype} {tuple(x.shape)})")
        b, dt = x.shape[0], TB_BF16
        if batch is not None and int(batch) != b:
            raise ValueError(f"{where}: batch {batch} but x has {b} rows")
        if workspace is None:
            workspace = torch.empty(max(tb_act8_bytes(b, k), 16), dtype=torch.uint8, device=x.device)
        wbytes = workspace.numel() * workspace.element_size()
    if y is None:
        y = torch.empty((b, n), dtype=torch.float32, device=x.device)
    _dev(y, workspace)
    _check(fn(_p(x), dt, b, _p(codes), _p(scales), n, k, _p(y), _p(workspace) if dt == TB_BF16 else None,
              wbytes, _stream(stream)), where)
    return y


def tb_ternary_gemv(x, codes, scales, batch=None, y=None, workspace=None, stream=None):
    """y[b, n] (fp32) = sum_g scale[n, g] * sum_k t[n, k] x[b, k].  x is either
    the rotated activations as bf16 [B, K] (encoded into `workspace`, a uint8
    device tensor of at least tb_act8_bytes(B, K) bytes, allocated here when
    None) or their act8 operand (uint8, exactly tb_act8_bytes(batch, K) bytes,
    `batch` given)."""
    return _gemv(lib().tb_ternary_gemv, "tb_ternary_gemv", x, codes, scales, scales.shape[1] * 128, batch, y,
                 workspace, stream)


def tb_ternary_gemv_noalloc(x, codes, scales, y, stream=None):
    """tb_ternary_gemv of bf16 x [B, K] into the caller's fp32 y [B, N] with the
    library's own device array for the encoded activations: nothing is
    allocated (the caller passes y).  Calls that may overlap on one GPU race."""
    _dev(x, codes, scales, y)
    n, k = _dense_n(scales), scales.shape[1] * 128
    if x.dtype not in (torch.bfloat16, torch.int16, torch.uint16) or x.dim() != 2 or x.shape[1] != k:
        raise ValueError(f"tb_ternary_gemv_noalloc: x must be bf16 [B, {k}] (got {x.dtype} {tuple(x.shape)})")
    if y.dtype != torch.float32 or tuple(y.shape) != (x.shape[0], n):
        raise ValueError(f"tb_ternary_gemv_noalloc: y must be float32 [{x.shape[0]}, {n}]")
    _check(lib().tb_ternary_gemv_noalloc(_p(x), x.shape[0], _p(codes), _p(scales), n, k, _p(y), _stream(stream)),
           "tb_ternary_gemv_noalloc")
    return y


def tb_ternary_gemv_resid(x, codes, scales, batch=None, y=None, workspace=None, stream=None):
    """tb_ternary_gemv over two-plane weights (TB_FMT_DENSE_RESID): codes
    [N/16, 2K/128, 128], scales [N, 2K/128], groups of the planes interleaved."""
    return _gemv(lib().tb_ternary_gemv_resid, "tb_ternary_gemv_resid", x, codes, scales, scales.shape[1] // 2 * 128,
                 batch, y, workspace, stream)


def tb_ternary_gemv_multi(segments, stream=None):
    """One launch of several GEMVs: segments = [(act, codes, scales, batch, y[, planes[, parts]]), ...];
    planes is 1 (default) or 2 for two-plane weights; parts > 1 (batch 1) splits K over that many
    workgroups per tile and y receives the parts, [parts, batch, N], whose sum is the product."""
    if not segments:
        return
    arr = (GemvSegment * len(segments))()
    for c, seg in enumerate(segments):
        act, codes, scales, batch, y = seg[:5]
        planes = int(seg[5]) if len(seg) > 5 else 1
        parts = int(seg[6]) if len(seg) > 6 else 1
        _dev(act, codes, scales, y)
        n, g = _dense_n(scales), scales.shape[1]
        k = g // max(planes, 1) * 128
        _act8_operand(act, int(batch), k, "tb_ternary_gemv_multi")
        if y.numel() < max(parts, 1) * int(batch) * n:
            raise ValueError(f"tb_ternary_gemv_multi: y holds {y.numel()} floats, needs {max(parts, 1)} x {batch} x {n}")
        arr[c] = GemvSegment(act.data_ptr(), int(batch), codes.data_ptr(), scales.data_ptr(), n, k, y.data_ptr(),
                             planes, parts)
    _check(lib().tb_ternary_gemv_multi(arr, len(segments), _stream(stream)), "tb_ternary_gemv_multi")


def _planes24(x, meta, signs, scales, where):
    """(B, N, K) of a 2:4 product, its planes checked against x."""
    b, k = x.shape
    n = meta.shape[0] * 16
    g4 = -(-k // 512)
    if tuple(meta.shape) != (n // 16, g4, 64, 4) or tuple(signs.shape) != (n // 16, g4, 64, 2) \
            or scales.numel() != n * g4 * 4:
        raise ValueError(f"{where}: 2:4 planes {tuple(meta.shape)}, {tuple(signs.shape)} do not match K = {k}")
    return b, n, k


def tb_ternary24_gemv(x, meta, signs, scales, y=None, stream=None):
    """x bf16 [B, K]; meta [N/16, G4, 64, 4], signs [N/16, G4, 64, 2], scales
    [N/16, G4, 4, 4, 4] (the stored 2:4 format, G4 = ceil(K/512))."""
    _dev(x, meta, signs, scales)
    b, n, k = _planes24(x, meta, signs, scales, "tb_ternary24_gemv")
    if y is None:
        y = torch.empty((b, n), dtype=torch.float32, device=x.device)
    _dev(y)
    _check(lib().tb_ternary24_gemv(_p(x), b, _p(meta), _p(signs), _p(scales), n, k, _p(y), _stream(stream)),
           "tb_ternary24_gemv")
    return y


def tb_ternary24_gemv_multi(segments, stream=None):
    """One launch of several 2:4 GEMVs: segments = [(x, meta, signs, scales, y), ...]
    with the shapes of tb_ternary24_gemv; y fp32 [B, N] each."""
    if not segments:
        return
    arr = (Gemv24Segment * len(segments))()
    for c, (x, meta, signs, scales, y) in enumerate(segments):
        _dev(x, meta, signs, scales, y)
        b, n, k = _planes24(x, meta, signs, scales, "tb_ternary24_gemv_multi")
        if y.numel() < b * n:
            raise ValueError(f"tb_ternary24_gemv_multi: y holds {y.numel()} floats, needs {b} x {n}")
        arr[c] = Gemv24Segment(x.data_ptr(), meta.data_ptr(), signs.data_ptr(), scales.data_ptr(), y.data_ptr(),
                               b, n, k)
    _check(lib().tb_ternary24_gemv_multi(arr, len(segments), _stream(stream)), "tb_ternary24_gemv_multi")


def tb_ternary_gemm(x, codes, scales, y=None, out_dtype=torch.bfloat16, stream=None):
    """Y[m, n] = sum_g scale[n, g] * sum_k t[n, k] x[m, k]; x bf16 [M, K], Y bf16 or fp32."""
    _dev(x, codes, scales)
    m, k = x.shape
    n = _dense_n(scales)
    if y is None:
        y = torch.empty((m, n), dtype=out_dtype, device=x.device)
    _dev(y)
    _check(lib().tb_ternary_gemm(_p(x), m, _p(codes), _p(scales), n, k, _p(y), _dt(y), _stream(stream)),
           "tb_ternary_gemm")
    return y


def tb_ternary_gemm_multi(segments, stream=None):
    """Several GEMMs: segments = [(x, codes, scales, y), ...], x bf16 [M, K], y bf16 or fp32 [M, N];
    one launch when every M <= 16, else one launch per product."""
    if not segments:
        return
    arr = (GemmSegment * len(segments))()
    for c, (x, codes, scales, y) in enumerate(segments):
        _dev(x, codes, scales, y)
        m, k = x.shape
        n = _dense_n(scales)
        if y.numel() < m * n:
            raise ValueError(f"tb_ternary_gemm_multi: y holds {y.numel()} elements, needs {m} x {n}")
        arr[c] = GemmSegment(x.data_ptr(), codes.data_ptr(), scales.data_ptr(), y.data_ptr(), m, n, k, _dt(y), 0)
    _check(lib().tb_ternary_gemm_multi(arr, len(segments), _stream(stream)), "tb_ternary_gemm_multi")


def tb_ternary_gemm_splitk_workspace(m, n, k):
    return int(lib().tb_ternary_gemm_splitk_workspace(int(m), int(n), int(k)))


def tb_ternary_gemm_splitk(x, codes, scales, y=None, out_dtype=torch.bfloat16, workspace=None, stream=None):
    """tb_ternary_gemm with K split across workgroups for few activation rows;
    `workspace` is a device tensor of at least tb_ternary_gemm_splitk_workspace
    bytes (allocated here when None)."""
    _dev(x, codes, scales)
    m, k = x.shape
    n = _dense_n(scales)
    if y is None:
        y = torch.empty((m, n), dtype=out_dtype, device=x.device)
    if workspace is None:
        nbytes = tb_ternary_gemm_splitk_workspace(m, n, k)
        workspace = torch.empty(max(nbytes // 4, 4), dtype=torch.float32, device=x.device)
    _dev(y, workspace)
    _check(lib().tb_ternary_gemm_splitk(_p(x), m, _p(codes), _p(scales), n, k, _p(y), _dt(y), _p(workspace),
                                        workspace.numel() * workspace.element_size(), _stream(stream)),
           "tb_ternary_gemm_splitk")
    return y


def tb_ternary_gemm_rotated(x, codes, scales, y=None, out_dtype=torch.bfloat16, workspace=None, stream=None):
    """The GEMM with its output rotated back along N (y = R_N y') in the same
    launch; `workspace` (a device tensor, or None for one pass over K) as in
    tb_ternary_gemm_splitk."""
    _dev(x, codes, scales)
    m, k = x.shape
    n = _dense_n(scales)
    if y is None:
        y = torch.empty((m, n), dtype=out_dtype, device=x.device)
    _dev(y, workspace)
    wbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib().tb_ternary_gemm_rotated(_p(x), m, _p(codes), _p(scales), n, k, _p(y), _dt(y), _p(workspace),
                                         wbytes, _stream(stream)), "tb_ternary_gemm_rotated")
    return y


# ------------------------------------------------------- serving operators

_FLOATS = {torch.float32: TB_F32, torch.bfloat16: TB_BF16}


def _empty(shape, dtype, device, stream):
    """A new tensor for a call on `stream`: allocated for that stream, so that its
    memory is neither still in use elsewhere nor given away before the call is done."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _float_dt(t, what):
    d = _FLOATS.get(t.dtype)
    if d is None:
        raise TypeError(f"{what} must be float32 or bfloat16 (got {t.dtype})")
    return d


def _addr(t):
    return None if t is None else t.data_ptr()


def _same_device(first, *ts):
    index = first.get_device()
    for t in ts:
        if t is not None and t.get_device() != index:
            raise ValueError(f"every tensor must be on {first.device} (got one on {t.device})")


def tb_block_norm(y, resid=None, w_post=None, w_pre=None, gate=None, rows_per_gate=1, alpha=1.0, eps=1e-6, y_parts=1,
                  rotate_in=False, rotate_out=False, h=None, z=None, h_dtype=None, z_dtype=torch.bfloat16,
                  with_h=True, stream=None):
    """The boundary of a block: u = the sum of y's parts (rotated back if
    rotate_in), normed with w_post if given; h = resid + alpha * gate * u; z =
    norm of h with w_pre (rotated if rotate_out).  Returns (h, z).
    y [rows, C] fp32 or bf16 ([y_parts, rows, C] fp32 with y_parts > 1), or None
    (h = resid, not returned: only the norm).  resid [rows, C] or None.  w_post,
    w_pre [C] of one dtype; without w_pre there is no z.  gate [gates, C]: row r
    takes gate row r // rows_per_gate.  h (resid itself for in place) and z are
    made when not given; z_dtype torch.uint8 writes the act8 operand."""
    _dev(y, resid, w_post, w_pre, gate, h, z)
    first = resid if y is None else y
    if not (first is not None):
        raise ValueError("tb_block_norm: y or resid must be given")
    parts = int(y_parts)
    if y is not None and parts > 1:
        if not (y.dim() == 3 and y.shape[0] == parts):
            raise ValueError(f"tb_block_norm: y_parts={parts} needs y [{parts}, rows, C]")
    else:
        if not (first.dim() == 2):
            raise ValueError("tb_block_norm: y must be [rows, C]")
    rows, ch = first.shape[-2], first.shape[-1]
    dev = first.device
    _same_device(first, y, resid, w_post, w_pre, gate, h, z)
    if not (resid is None or resid.shape == (rows, ch)):
        raise ValueError(f"tb_block_norm: resid must be [{rows}, {ch}]")
    for w in (w_post, w_pre):
        if not (w is None or w.shape == (ch,)):
            raise ValueError(f"tb_block_norm: w_post and w_pre must be [{ch}]")
    if not (w_post is None or w_pre is None or w_post.dtype == w_pre.dtype):
        raise ValueError("tb_block_norm: w_post and w_pre differ in dtype")
    if gate is not None:
        rows_per_gate = int(rows_per_gate)
        if rows_per_gate < 1:
            raise ValueError("tb_block_norm: rows_per_gate must be at least 1")
        if not (gate.dim() == 2 and gate.shape[1] == ch and gate.shape[0] * rows_per_gate >= rows):
            raise ValueError(f"tb_block_norm: gate must be [{-(-rows // rows_per_gate)}, {ch}] at rows_per_gate {rows_per_gate}")
    if y is None or not with_h:
        if h is not None:
            raise ValueError("tb_block_norm: no h without y or with with_h=False")
    elif h is None:
        h = _empty((rows, ch), resid.dtype if resid is not None else h_dtype or y.dtype, dev, stream)
    if not (h is None or h.shape == (rows, ch)):
        raise ValueError(f"tb_block_norm: h must be [{rows}, {ch}]")
    if not (h is None or resid is None or h.dtype == resid.dtype):
        raise ValueError("tb_block_norm: h and resid differ in dtype")
    if w_pre is None:
        if z is not None:
            raise ValueError("tb_block_norm: z needs w_pre")
    elif z is None:
        if z_dtype == torch.uint8:
            z = _empty(tb_act8_bytes(rows, ch), torch.uint8, dev, stream)
        else:
            z = _empty((rows, ch), z_dtype, dev, stream)
    elif z.dtype == torch.uint8:
        if not (z.numel() == tb_act8_bytes(rows, ch)):
            raise ValueError(f"tb_block_norm: z must hold {tb_act8_bytes(rows, ch)} bytes")
    else:
        if not (z.shape == (rows, ch)):
            raise ValueError(f"tb_block_norm: z must be [{rows}, {ch}]")
    w = w_post if w_post is not None else w_pre
    zd = TB_F32 if z is None else TB_ACT8 if z.dtype == torch.uint8 else _float_dt(z, "tb_block_norm: z")
    s = resid if resid is not None else h
    args = BlockNormArgs(
        _addr(y), _addr(resid), _addr(w_post), _addr(w_pre), _addr(gate), _addr(h), _addr(z), rows, ch, rows_per_gate,
        parts, TB_F32 if y is None else _float_dt(y, "tb_block_norm: y"),
        TB_F32 if s is None else _float_dt(s, "tb_block_norm: resid and h"),
        TB_F32 if w is None else _float_dt(w, "tb_block_norm: w_post and w_pre"),
        TB_F32 if gate is None else _float_dt(gate, "tb_block_norm: gate"), zd, int(rotate_in), int(rotate_out),
        alpha, eps)
    _check(lib().tb_block_norm(args, _stream(stream)), "tb_block_norm")
    return h, z


def _token_rows(t, heads, d, where):
    """Elements between tokens of a [tokens, heads, d] tensor whose tokens are
    contiguous inside (a slice of a fused projection's output)."""
    if t.dtype != torch.bfloat16 or t.dim() != 3 or t.shape[1] != heads or t.shape[2] != d:
        raise ValueError(f"{where} must be bfloat16 [tokens, {heads}, {d}] (got {t.dtype} {tuple(t.shape)})")
    if not t.is_cuda or t.stride(2) != 1 or (heads > 1 and t.stride(1) != d):
        raise ValueError(f"{where}: a token's heads must be contiguous on the device")
    return t.stride(0) if t.shape[0] > 1 else heads * d  # of one token it says nothing


def _paged_cache(where, tokens, k_cache, v_cache, block_table, cu_q, kv_len, max_q, k_scale, v_scale):
    _dev(k_cache, v_cache, cu_q, kv_len, k_scale, v_scale)
    if k_cache.dim() != 4 or v_cache.dim() != 4 or k_cache.dtype != v_cache.dtype:
        raise ValueError(f"{where}: k_cache must be [pages, heads, page, d], v_cache [pages, heads, d, page], one dtype")
    pages, heads, page, d = k_cache.shape
    if v_cache.shape != (pages, heads, d, page):
        raise ValueError(f"{where}: v_cache must be [{pages}, {heads}, {d}, {page}] (got {tuple(v_cache.shape)})")
    if k_cache.dtype == torch.bfloat16:
        kind = TB_BF16
    elif k_cache.dtype == torch.float8_e4m3fn:
        kind = TB_FP8
    else:
        raise TypeError(f"{where}: the cache must be bfloat16 or float8_e4m3fn (got {k_cache.dtype})")
    b = kv_len.shape[0]
    if not (cu_q.dtype == kv_len.dtype == block_table.dtype == torch.int32):
        raise TypeError(f"{where}: block_table, cu_q and kv_len must be int32")
    if kv_len.dim() != 1 or cu_q.shape != (b + 1,) or block_table.dim() != 2 or block_table.shape[0] != b:
        raise ValueError(f"{where}: kv_len must be [B], cu_q [B + 1], block_table [B, entries]")
    if not block_table.is_cuda or (block_table.shape[1] > 1 and block_table.stride(1) != 1):
        raise ValueError(f"{where}: a sequence's block_table entries must be contiguous on the device")
    for sc in (k_scale, v_scale):
        if sc is not None and (sc.dtype != torch.float32 or sc.shape != (heads,) or kind != TB_FP8):
            raise ValueError(f"{where}: k_scale and v_scale must be float32 [{heads}], of an 8-bit cache")
    _same_device(tokens, k_cache, v_cache, block_table, cu_q, kv_len, k_scale, v_scale)
    width = block_table.shape[1]
    stride = block_table.stride(0) if b > 1 else width
    return PagedCache(k_cache.data_ptr(), v_cache.data_ptr(), _addr(k_scale), _addr(v_scale), block_table.data_ptr(),
                      cu_q.data_ptr(), kv_len.data_ptr(), pages, stride, width, b, tokens.shape[0], max_q, kind, page,
                      heads, d)


def tb_paged_append(k, v, k_cache, v_cache, block_table, cu_q, kv_len, max_q, k_scale=None, v_scale=None, stream=None):
    """Write the new tokens' keys and values (bf16 [tokens, heads, d], slices of
    a fused projection allowed) into the pages of their positions: sequence b's
    tokens are rows cu_q[b]..cu_q[b + 1] - 1 and its last positions below
    kv_len[b].  k_cache [pages, heads, page, d], v_cache [pages, heads, d, page],
    bf16 or float8_e4m3fn (codes of x / scale[head]); max_q is at least every
    sequence's new tokens."""
    cache = _paged_cache("tb_paged_append", k, k_cache, v_cache, block_table, cu_q, kv_len, int(max_q), k_scale, v_scale)
    _same_device(k, v)
    ks = _token_rows(k, cache.heads_kv, cache.head_dim, "tb_paged_append: k")
    vs = _token_rows(v, cache.heads_kv, cache.head_dim, "tb_paged_append: v")
    if not (v.shape[0] == k.shape[0]):
        raise ValueError("tb_paged_append: k and v differ in tokens")
    _check(lib().tb_paged_append(cache, k.data_ptr(), ks, v.data_ptr(), vs, _stream(stream)), "tb_paged_append")


def _attention_args(q, k_cache, v_cache, block_table, cu_q, kv_len, max_q, max_kv, scale, window, k_scale, v_scale,
                    out_dt):
    where = "tb_paged_attention"
    cache = _paged_cache(where, q, k_cache, v_cache, block_table, cu_q, kv_len, int(max_q), k_scale, v_scale)
    heads = q.shape[1] if q.dim() == 3 else 0
    stride = _token_rows(q, heads, cache.head_dim, where + ": q")
    if scale is None:
        scale = cache.head_dim ** -0.5
    return PagedAttentionArgs(cache, q.data_ptr(), None, None, None, 0, stride, int(max_kv), int(window), heads, out_dt,
                              scale, 0)


def tb_paged_attention_workspace(q, k_cache, v_cache, block_table, cu_q, kv_len, max_q, max_kv, window=0):
    """Bytes of the workspace tb_paged_attention splits the positions into."""
    args = _attention_args(q, k_cache, v_cache, block_table, cu_q, kv_len, max_q, max_kv, None, window, None, None,
                           TB_BF16)
    return int(lib().tb_paged_attention_workspace(args))


def tb_paged_attention(q, k_cache, v_cache, block_table, cu_q, kv_len, max_q, max_kv, scale=None, window=0,
                       k_scale=None, v_scale=None, out=None, out_dtype=torch.bfloat16, lse=None, with_lse=False,
                       workspace=None, stream=None):
    """Attention of each sequence's new tokens q (bf16 [tokens, heads, d]) over
    its cached positions, causal, the last `window` of them only if window > 0;
    the cache as in tb_paged_append, which comes first.  max_kv is the most
    positions a sequence is likely to hold (it only decides the split).  scale
    defaults to 1 / sqrt(d).  Softmax weights are rounded for the product with the
    values, to 8 bits in chunks of more than 16 rows (tokens * shared heads) of a
    bf16 cache: see include/tb.h.  Returns out [tokens, heads, d], and (out, lse) if
    `lse` (fp32 [tokens, heads]) is given or with_lse; rows that see nothing
    are 0 (lse -inf).  `workspace`: a device tensor of
    tb_paged_attention_workspace bytes, allocated here when None."""
    if out is not None:
        _dev(out)
        out_dt = _float_dt(out, "tb_paged_attention: out")
        if not (out.shape == q.shape):
            raise ValueError(f"tb_paged_attention: out must be {tuple(q.shape)}")
    else:
        out = _empty(q.shape, out_dtype, q.device, stream)
        out_dt = _float_dt(out, "tb_paged_attention: out")
    args = _attention_args(q, k_cache, v_cache, block_table, cu_q, kv_len, max_q, max_kv, scale, window, k_scale,
                           v_scale, out_dt)
    if lse is not None:
        _dev(lse)
        if not (lse.dtype == torch.float32 and lse.shape == q.shape[:2]):
            raise ValueError(f"tb_paged_attention: lse must be float32 {tuple(q.shape[:2])}")
    elif with_lse:
        lse = _empty(q.shape[:2], torch.float32, q.device, stream)
    L = lib()
    if workspace is None:
        nbytes = L.tb_paged_attention_workspace(args)
        if nbytes:
            workspace = _empty(nbytes, torch.uint8, q.device, stream)
    else:
        _dev(workspace)
    _same_device(q, out, lse, workspace)
    args.out, args.lse = out.data_ptr(), _addr(lse)
    if workspace is not None:
        args.workspace, args.workspace_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    _check(L.tb_paged_attention(args, _stream(stream)), "tb_paged_attention")
    return out if lse is None else (out, lse)


def tb_verify_draft_workspace(batch, vocab):
    return int(lib().tb_verify_draft_workspace(int(batch), int(vocab)))


def _prob_rows(t, what):
    if not t.is_cuda or t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{what} must be [rows, vocab] on the device, a row contiguous")
    return t.stride(0) if t.shape[0] > 1 else max(t.stride(0), t.shape[1])


def tb_verify_draft(p, q, drafts, u, u_next, cu_draft, max_draft, accepted=None, tokens=None, workspace=None,
                    stream=None):
    """Verify drafted tokens: sequence b's drafts are rows cu_draft[b].. of
    drafts (int32), u (fp32) and q (the drafter's probabilities [total, vocab],
    or None for a certain drafter), its T + 1 target rows start at row
    cu_draft[b] + b of p [total + B, vocab].  Draft j is kept while u * q < p;
    then one token is drawn with u_next [B] from max(p - q, 0), or from p after
    the last.  Returns (accepted int32 [B], tokens int32 [B, max_draft + 1]:
    the kept tokens, the drawn one, then -1)."""
    where = "tb_verify_draft"
    _dev(drafts, u, u_next, cu_draft, accepted, tokens, workspace)
    b, total = u_next.shape[0], drafts.shape[0]
    max_draft = int(max_draft)
    ps = _prob_rows(p, where + ": p")
    vocab = p.shape[1]
    if not (p.shape[0] == total + b):
        raise ValueError(f"{where}: p must have {total + b} rows (drafts + sequences)")
    qs = 0
    if q is not None:
        qs = _prob_rows(q, where + ": q")
        if not (q.shape == (total, vocab)):
            raise ValueError(f"{where}: q must be [{total}, {vocab}]")
    if not (drafts.dtype == cu_draft.dtype == torch.int32):
        raise ValueError(f"{where}: drafts and cu_draft must be int32")
    if not (u.dtype == u_next.dtype == torch.float32):
        raise ValueError(f"{where}: u and u_next must be float32")
    if not (drafts.dim() == 1 and u.shape == drafts.shape and u_next.dim() == 1 and cu_draft.shape == (b + 1,)):
        raise ValueError(f"{where}: drafts and u must be [total], u_next [B], cu_draft [B + 1]")
    dev = p.device
    if accepted is None:
        accepted = _empty(b, torch.int32, dev, stream)
    if tokens is None:
        tokens = _empty((b, max(max_draft, 0) + 1), torch.int32, dev, stream)
    if not (accepted.dtype == tokens.dtype == torch.int32 and accepted.shape == (b,) and tokens.shape == (b, max_draft + 1)):
        raise ValueError(f"{where}: accepted must be int32 [{b}], tokens int32 [{b}, {max_draft + 1}]")
    L = lib()
    if workspace is None:
        nbytes = L.tb_verify_draft_workspace(b, vocab)
        if nbytes:
            workspace = _empty(nbytes, torch.uint8, dev, stream)
    _same_device(p, q, drafts, u, u_next, cu_draft, accepted, tokens, workspace)
    args = VerifyDraftArgs(p.data_ptr(), _addr(q), drafts.data_ptr(), u.data_ptr(), u_next.data_ptr(),
                           cu_draft.data_ptr(), accepted.data_ptr(), tokens.data_ptr(), _addr(workspace),
                           0 if workspace is None else workspace.numel() * workspace.element_size(), b, total, vocab,
                           ps, qs, max_draft, _float_dt(p, where + ": p"), TB_F32 if q is None else _float_dt(q, where + ": q"), 0)
    _check(L.tb_verify_draft(args, _stream(stream)), where)
    return accepted, tokens
