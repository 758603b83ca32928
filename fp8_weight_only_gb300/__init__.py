"""fp8_weight_only_gb300 -- Python binding of libfp8w (include/fp8w.h).

Argument marshalling only: every step of the layer runs in the library's
CUDA kernels.  PyTorch supplies device memory and the current stream.  There
is no CPU fallback: if libfp8w.so is missing or a call fails, an exception is
raised.

    codes, scales = quantize(w)                 # w: [N, K] fp32 CUDA tensor
    y = linear(x, codes, scales, bias)          # x: [M, K] bf16/fp16 CUDA tensor
    codes, e8 = quantize_mx(w)                  # one E8M0 scale byte per 32 along K
    y = linear(x, codes, e8, bias)              # bf16 x for M > 1
    qx, sx = quantize_act(x)                    # W8A8: per-token e4m3 activations
    y = linear_w8a8(qx, sx, codes, scales, bias, out_dtype=torch.bfloat16)
    cache = KVCache(k_pages, v_pages)           # paged keys and values: bf16/fp16, or e4m3 codes with scales
    q = rope_append(q, k, v, slots, cache, positions, Rope(table))
    o = paged_attention(q, cache, block_table, lens)
"""
import ctypes
import os

from .fp8w_file import Fp8wFileError, load as load_fp8w, save as save_fp8w  # noqa: F401  (the .fp8w file)

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libfp8w.so")

FP8W_BF16 = 1
FP8W_F16 = 2
FP8W_F32 = 3
FP8W_E4M3 = 4
KERNEL_AUTO, KERNEL_GEMV, KERNEL_SKINNY, KERNEL_PREFILL = 0, 1, 2, 3

SYMBOLS = ("fp8w_quantize", "fp8w_linear", "fp8w_linear_ex",
           "fp8w_status_string", "fp8w_last_cuda_error", "fp8w_device_error", "fp8w_abi_version",
           "fp8w_linear_noalloc", "fp8w_dequantize", "fp8w_quantize_grouped", "fp8w_linear_grouped",
           "fp8w_quantize_mx", "fp8w_linear_mx", "fp8w_quantize_ex", "fp8w_dequantize_grouped",
           "fp8w_dequantize_mx", "fp8w_quantize_act", "fp8w_linear_w8a8", "fp8w_rope", "fp8w_rope_append",
           "fp8w_paged_attention")
ABI_VERSION = 13
FLAG_WEIGHTS_READY = 1


class Fp8wError(RuntimeError):
    def __init__(self, status, msg):
        super().__init__(msg)
        self.status = status


class LinearConfig(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_int), ("cluster", ctypes.c_int), ("tiles", ctypes.c_int),
                ("flags", ctypes.c_int), ("reserved", ctypes.c_int * 4)]


class RopeSpec(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("max_pos", ctypes.c_int64), ("rot_dim", ctypes.c_int),
                ("interleaved", ctypes.c_int), ("axes", ctypes.c_int), ("sections", ctypes.c_int * 4)]


class KVCacheSpec(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scales", ctypes.c_void_p),
                ("v_scales", ctypes.c_void_p), ("num_pages", ctypes.c_int64), ("page_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64), ("dtype", ctypes.c_int),
                ("kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int), ("page_size", ctypes.c_int)]


_lib = None


def lib():
    """The loaded libfp8w (ctypes.CDLL); raises if it was never built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise Fp8wError(-1, "libfp8w.so is not built (run __graft_entry__.build() or "
                                "python fp8_weight_only_gb300/build.py)")
        L = ctypes.CDLL(LIB_PATH)
        c, P = ctypes, ctypes.c_void_p
        L.fp8w_quantize.restype = c.c_int
        L.fp8w_quantize.argtypes = [P, c.c_int64, c.c_int64, P, P, P]
        L.fp8w_quantize_grouped.restype = c.c_int
        L.fp8w_quantize_grouped.argtypes = [P, c.c_int64, c.c_int64, c.c_int, P, P, P]
        L.fp8w_linear_grouped.restype = c.c_int
        L.fp8w_linear_grouped.argtypes = [P, c.c_int, c.c_int64, c.c_int64, P, P, c.c_int, P, c.c_int64, P, P]
        L.fp8w_quantize_ex.restype = c.c_int
        L.fp8w_quantize_ex.argtypes = [P, c.c_int, c.c_int64, c.c_int64, P, P, P]
        L.fp8w_quantize_mx.restype = c.c_int
        L.fp8w_quantize_mx.argtypes = [P, c.c_int64, c.c_int64, P, P, P]
        L.fp8w_linear_mx.restype = c.c_int
        L.fp8w_linear_mx.argtypes = [P, c.c_int, c.c_int64, c.c_int64, P, P, P, c.c_int64, P, P]
        L.fp8w_dequantize_grouped.restype = c.c_int
        L.fp8w_dequantize_grouped.argtypes = [P, P, c.c_int, c.c_int64, c.c_int64, c.c_int, P, P]
        L.fp8w_dequantize_mx.restype = c.c_int
        L.fp8w_dequantize_mx.argtypes = [P, P, c.c_int64, c.c_int64, c.c_int, P, P]
        L.fp8w_dequantize.restype = c.c_int
        L.fp8w_dequantize.argtypes = [P, P, c.c_int64, c.c_int64, c.c_int, P, P]
        L.fp8w_linear.restype = c.c_int
        L.fp8w_linear.argtypes = [P, c.c_int, c.c_int64, c.c_int64, P, P, P, c.c_int64, P, P]
        L.fp8w_linear_ex.restype = c.c_int
        L.fp8w_linear_ex.argtypes = [P, c.c_int, c.c_int64, c.c_int64, P, P, P, c.c_int64, P,
                                     c.POINTER(LinearConfig), P]
        L.fp8w_linear_noalloc.restype = c.c_int
        L.fp8w_linear_noalloc.argtypes = [P, c.c_int, c.c_int64, c.c_int64, P, P, P, c.c_int64, P, P]
        L.fp8w_quantize_act.restype = c.c_int
        L.fp8w_quantize_act.argtypes = [P, c.c_int, c.c_int64, c.c_int64, P, P, P]
        L.fp8w_linear_w8a8.restype = c.c_int
        L.fp8w_linear_w8a8.argtypes = [P, P, c.c_int64, c.c_int64, P, P, P, c.c_int64, P, c.c_int, c.c_int, P]
        RS, KC = c.POINTER(RopeSpec), c.POINTER(KVCacheSpec)
        L.fp8w_rope.restype = c.c_int
        L.fp8w_rope.argtypes = [P, c.c_int, c.c_int64, c.c_int, c.c_int, c.c_int64, P, RS, P, c.c_int64, P]
        L.fp8w_rope_append.restype = c.c_int
        L.fp8w_rope_append.argtypes = [P, P, P, c.c_int, c.c_int64, c.c_int, c.c_int64, c.c_int64, c.c_int64, P, RS,
                                       P, KC, P, c.c_int64, P]
        L.fp8w_paged_attention.restype = c.c_int
        L.fp8w_paged_attention.argtypes = [P, c.c_int, c.c_int64, c.c_int, c.c_int64, KC, P, c.c_int64, P, P,
                                           c.c_int64, c.c_float, c.c_int64, c.c_int64, c.c_int64, P, c.c_int64, P]
        L.fp8w_status_string.restype = c.c_char_p
        L.fp8w_status_string.argtypes = [c.c_int]
        L.fp8w_last_cuda_error.restype = c.c_char_p
        L.fp8w_last_cuda_error.argtypes = []
        L.fp8w_device_error.restype = c.c_int
        L.fp8w_device_error.argtypes = []
        L.fp8w_abi_version.restype = c.c_int
        L.fp8w_abi_version.argtypes = []
        _lib = L
    return _lib


def _check(status):
    if status != 0:
        L = lib()
        msg = L.fp8w_status_string(status).decode()
        if status == 5:
            msg += ": " + L.fp8w_last_cuda_error().decode()
        raise Fp8wError(status, msg)


def _stream(t):
    import torch
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _act(dtype):
    import torch
    if dtype == torch.bfloat16:
        return FP8W_BF16
    if dtype == torch.float16:
        return FP8W_F16
    raise TypeError("activations must be bfloat16 or float16, got %s" % dtype)


def quantize(w, codes=None, scales=None, group=None):
    """W[N, K] (CUDA, contiguous; fp32, or bf16/fp16 widened exactly) ->
    (codes uint8 [N, K], scales fp32 [N]), or with group (32, 64 or 128; fp32
    weights) scales fp32 [N, K / group], one per run of `group` weights of a row."""
    import torch
    wdt = {torch.float32: FP8W_F32, torch.bfloat16: FP8W_BF16, torch.float16: FP8W_F16}.get(w.dtype)
    if wdt is None or not w.is_cuda or w.dim() != 2 or not w.is_contiguous():
        raise TypeError("w must be a contiguous 2-D float32, bfloat16 or float16 CUDA tensor")
    if wdt != FP8W_F32 and group is not None:
        raise TypeError("per-group quantisation takes float32 weights")
    n, k = w.shape
    if codes is None:
        codes = torch.empty((n, k), dtype=torch.uint8, device=w.device)
    if scales is None:
        shape = (n,) if group is None else (n, k // group)
        scales = torch.empty(shape, dtype=torch.float32, device=w.device)
    if group is None:
        _check(lib().fp8w_quantize_ex(_ptr(w), wdt, n, k, _ptr(codes), _ptr(scales), _stream(w)))
    else:
        _check(lib().fp8w_quantize_grouped(_ptr(w), n, k, int(group), _ptr(codes), _ptr(scales), _stream(w)))
    return codes, scales


def quantize_mx(w, codes=None, scales=None):
    """W[N, K] fp32 (CUDA, contiguous, K % 32 == 0) -> (codes uint8 [N, K],
    scales uint8 [N, K / 32]): the MX-style form, one E8M0 byte (2^(b - 127))
    per 32 weights along K."""
    import torch
    if w.dtype != torch.float32 or not w.is_cuda or w.dim() != 2 or not w.is_contiguous():
        raise TypeError("w must be a contiguous 2-D float32 CUDA tensor")
    n, k = w.shape
    if codes is None:
        codes = torch.empty((n, k), dtype=torch.uint8, device=w.device)
    if scales is None:
        scales = torch.empty((n, k // 32), dtype=torch.uint8, device=w.device)
    _check(lib().fp8w_quantize_mx(_ptr(w), n, k, _ptr(codes), _ptr(scales), _stream(w)))
    return codes, scales


def dequantize(codes, scales, dtype=None, out=None):
    """W'[N, K] = e4m3(codes) * scales[:, None], rounded once to `dtype`
    (torch.float32, bfloat16 or float16; default bfloat16).  scales may also
    be per-group fp32 [N, K / group] or E8M0 uint8 [N, K / 32]."""
    import torch
    if dtype is None:
        dtype = out.dtype if out is not None else torch.bfloat16
    kind = {torch.float32: FP8W_F32, torch.bfloat16: FP8W_BF16, torch.float16: FP8W_F16}.get(dtype)
    if kind is None:
        raise TypeError("dequantize: dtype must be float32, bfloat16 or float16, got %s" % dtype)
    mx = scales.dim() == 2 and scales.dtype == torch.uint8
    for name, t, dt in (("codes", codes, torch.uint8), ("scales", scales, torch.uint8 if mx else torch.float32)):
        if t.dtype != dt or not t.is_cuda or not t.is_contiguous():
            raise TypeError("%s must be a contiguous %s CUDA tensor" % (name, dt))
    n, k = codes.shape
    if out is None:
        out = torch.empty((n, k), dtype=dtype, device=codes.device)
    elif out.shape != (n, k) or out.dtype != dtype or not out.is_contiguous():
        raise ValueError("out must be a contiguous [N, K] tensor of the requested dtype")
    if scales.dim() == 2:
        if scales.shape[0] != n or scales.shape[1] == 0 or k % scales.shape[1] or (mx and scales.shape[1] * 32 != k):
            raise ValueError("shape mismatch for per-group scales")
        if mx:
            _check(lib().fp8w_dequantize_mx(_ptr(codes), _ptr(scales), n, k, kind, _ptr(out), _stream(codes)))
        else:
            _check(lib().fp8w_dequantize_grouped(_ptr(codes), _ptr(scales), k // scales.shape[1], n, k, kind,
                                                 _ptr(out), _stream(codes)))
        return out
    _check(lib().fp8w_dequantize(_ptr(codes), _ptr(scales), n, k, kind, _ptr(out), _stream(codes)))
    return out


def linear(x, codes, scales, bias=None, out=None, kernel=KERNEL_AUTO, cluster=0, tiles=0,
           weights_ready=False):
    """y[M, N] = round(scale[n] * sum_k x[m, k] * e4m3(codes[n, k]) + bias[n]).

    kernel, and for the tensor-core kernel cluster (CTAs per thread-block
    cluster) with tiles (128-channel tiles a cluster shares), override the
    automatic launch choice, for tests and tuning (0, 0 = from the shape).
    weights_ready: every write to codes and scales has completed before this
    call (FP8W_FLAG_WEIGHTS_READY): the kernels stream the codes without
    waiting for the preceding kernel in the stream.  Per-row scales only."""
    import torch
    if x.dim() != 2 or not x.is_cuda or not x.is_contiguous():
        raise TypeError("x must be a contiguous 2-D CUDA tensor")
    # E8M0 scale bytes [N, K / 32] (the MX-style form) or fp32 scales
    mx = scales.dim() == 2 and scales.dtype == torch.uint8
    for name, t, dt in (("codes", codes, torch.uint8), ("scales", scales, torch.uint8 if mx else torch.float32),
                        ("bias", bias, torch.float32)):
        if t is not None and (t.dtype != dt or not t.is_cuda or not t.is_contiguous()):
            raise TypeError("%s must be a contiguous %s CUDA tensor" % (name, dt))
    m, k = x.shape
    n = codes.shape[0]
    if scales.dim() == 2:
        # per-group scales [N, K / group] (fp32), or E8M0 bytes [N, K / 32]
        if codes.dim() != 2 or codes.shape[1] != k or scales.shape[0] != n or k % scales.shape[1] or \
                (mx and scales.shape[1] * 32 != k) or (bias is not None and bias.numel() != n):
            raise ValueError("shape mismatch for per-group scales")
        if out is None:
            out = torch.empty((m, n), dtype=x.dtype, device=x.device)
        elif out.shape != (m, n) or out.dtype != x.dtype or not out.is_contiguous():
            raise ValueError("out must be a contiguous [M, N] tensor of x's dtype")
        if mx:
            _check(lib().fp8w_linear_mx(_ptr(x), _act(x.dtype), m, k, _ptr(codes), _ptr(scales), _ptr(bias), n,
                                        _ptr(out), _stream(x)))
        else:
            _check(lib().fp8w_linear_grouped(_ptr(x), _act(x.dtype), m, k, _ptr(codes), _ptr(scales),
                                             k // scales.shape[1], _ptr(bias), n, _ptr(out), _stream(x)))
        return out
    if codes.dim() != 2 or codes.shape[1] != k or scales.numel() != n or \
            (bias is not None and bias.numel() != n):
        raise ValueError("shape mismatch: x %s, codes %s, scales %s, bias %s" % (
            tuple(x.shape), tuple(codes.shape), tuple(scales.shape),
            None if bias is None else tuple(bias.shape)))
    if out is None:
        out = torch.empty((m, n), dtype=x.dtype, device=x.device)
    elif out.shape != (m, n) or out.dtype != x.dtype or not out.is_contiguous():
        raise ValueError("out must be a contiguous [M, N] tensor of x's dtype")
    act = _act(x.dtype)
    L = lib()
    stream = _stream(x)
    if kernel == KERNEL_AUTO and cluster == 0 and not weights_ready:
        st = L.fp8w_linear(_ptr(x), act, m, k, _ptr(codes), _ptr(scales), _ptr(bias), n, _ptr(out), stream)
    else:
        cfg = LinearConfig(kernel, cluster, tiles, FLAG_WEIGHTS_READY if weights_ready else 0)
        st = L.fp8w_linear_ex(_ptr(x), act, m, k, _ptr(codes), _ptr(scales), _ptr(bias), n,
                              _ptr(out), ctypes.byref(cfg), stream)
    _check(st)
    return out


def quantize_act(x, codes=None, scales=None):
    """W8A8 activation quantisation: x[M, K] bf16/fp16 (CUDA, contiguous) ->
    (codes uint8 [M, K], scales fp32 [M]), the per-row rule on every token."""
    import torch
    if x.dim() != 2 or not x.is_cuda or not x.is_contiguous():
        raise TypeError("x must be a contiguous 2-D CUDA tensor")
    m, k = x.shape
    if codes is None:
        codes = torch.empty((m, k), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty((m,), dtype=torch.float32, device=x.device)
    _check(lib().fp8w_quantize_act(_ptr(x), _act(x.dtype), m, k, _ptr(codes), _ptr(scales), _stream(x)))
    return codes, scales


def linear_w8a8(x_codes, x_scales, codes, scales, bias=None, out=None, out_dtype=None, weights_ready=False):
    """W8A8: y[M, N] = round(x_scales[m] * scales[n] * sum_k e4m3(x_codes[m, k]) e4m3(codes[n, k]) + bias[n]),
    out_dtype torch.bfloat16 (default) or torch.float16."""
    import torch
    for name, t, dt in (("x_codes", x_codes, torch.uint8), ("x_scales", x_scales, torch.float32),
                        ("codes", codes, torch.uint8), ("scales", scales, torch.float32),
                        ("bias", bias, torch.float32)):
        if t is not None and (t.dtype != dt or not t.is_cuda or not t.is_contiguous()):
            raise TypeError("%s must be a contiguous %s CUDA tensor" % (name, dt))
    m, k = x_codes.shape
    n = codes.shape[0]
    if codes.dim() != 2 or codes.shape[1] != k or x_scales.numel() != m or scales.numel() != n or \
            (bias is not None and bias.numel() != n):
        raise ValueError("shape mismatch for W8A8")
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else torch.bfloat16
    if out is None:
        out = torch.empty((m, n), dtype=out_dtype, device=codes.device)
    elif out.shape != (m, n) or out.dtype != out_dtype or not out.is_contiguous():
        raise ValueError("out must be a contiguous [M, N] tensor of out_dtype")
    _check(lib().fp8w_linear_w8a8(_ptr(x_codes), _ptr(x_scales), m, k, _ptr(codes), _ptr(scales), _ptr(bias), n,
                                  _ptr(out), _act(out_dtype), FLAG_WEIGHTS_READY if weights_ready else 0,
                                  _stream(codes)))
    return out


class Rope:
    """Rotary positions for rope and rope_append: table fp32 [max_pos, rot_dim]
    (CUDA, contiguous), each row the cosines of rot_dim / 2 angles and then
    their sines.  Pair i of a head is values (i, i + rot_dim / 2), or
    (2 i, 2 i + 1) with interleaved.  sections: pairs that turn by each axis'
    position (several axes: time, height and width, say); None: one axis."""

    def __init__(self, table, interleaved=False, sections=None):
        import torch
        if table.dtype != torch.float32 or not table.is_cuda or table.dim() != 2 or not table.is_contiguous():
            raise TypeError("table must be a contiguous 2-D float32 CUDA tensor")
        sections = [table.shape[1] // 2] if sections is None else [int(s) for s in sections]
        if not 1 <= len(sections) <= 4:
            raise ValueError("1 to 4 sections, got %d" % len(sections))
        self.table = table
        self.index = table.get_device()
        self.axes = len(sections)
        self.spec = RopeSpec(table.data_ptr(), table.shape[0], table.shape[1], 1 if interleaved else 0, self.axes,
                             (ctypes.c_int * 4)(*sections))
        self._ref = ctypes.byref(self.spec)


class KVCache:
    """A paged cache over the caller's tensors k and v, [num_pages, kv_heads,
    page_size, head_dim] in any memory order whose head_dim values are
    contiguous (a [num_pages, page_size, kv_heads, head_dim] tensor's
    transpose(1, 2), say; both the same strides): bfloat16 or float16, or
    uint8 e4m3 codes with k_scales, v_scales fp32 [num_pages, kv_heads,
    page_size].  It keeps references to the tensors and nothing else."""

    def __init__(self, k, v, k_scales=None, v_scales=None):
        import torch
        dtype = {torch.bfloat16: FP8W_BF16, torch.float16: FP8W_F16, torch.uint8: FP8W_E4M3}.get(k.dtype)
        if dtype is None or v.dtype != k.dtype or not k.is_cuda or v.device != k.device or k.dim() != 4:
            raise TypeError("k and v must be 4-D CUDA tensors, both bfloat16, float16 or uint8 (e4m3 codes)")
        if v.shape != k.shape or v.stride() != k.stride() or k.stride(3) != 1:
            raise ValueError("k and v must have the same shape and strides, head_dim contiguous")
        pages, heads, page, dim = k.shape
        for name, t in (("k_scales", k_scales), ("v_scales", v_scales)):
            if (t is None) != (dtype != FP8W_E4M3):
                raise ValueError("%s comes with e4m3 codes, and only with them" % name)
            if t is not None and (t.dtype != torch.float32 or t.device != k.device or not t.is_contiguous() or
                                  t.shape != (pages, heads, page)):
                raise TypeError("%s must be a contiguous float32 [num_pages, kv_heads, page_size] CUDA tensor" % name)
        self.k, self.v, self.k_scales, self.v_scales = k, v, k_scales, v_scales
        self.device, self.dtype, self.kv_heads, self.page_size, self.head_dim = k.device, k.dtype, heads, page, dim
        self.index = k.get_device()
        self.spec = KVCacheSpec(k.data_ptr(), v.data_ptr(), None if k_scales is None else k_scales.data_ptr(),
                                None if v_scales is None else v_scales.data_ptr(), pages, k.stride(0), k.stride(1),
                                k.stride(2), dtype, heads, dim, page)
        self._ref = ctypes.byref(self.spec)


# The calls below run once a layer and token, where a few microseconds of the
# host count: they read each attribute once and compare in place; _refuse finds
# out what was wrong.

_torch = _stream_of = _empty_like = _dense = _int32 = _int64 = None
_ACT = {}


def _load_torch():
    global _torch, _stream_of, _empty_like, _dense, _int32, _int64
    import torch
    _ACT.update({torch.bfloat16: FP8W_BF16, torch.float16: FP8W_F16})
    # the stream's handle without a Stream object around it, where torch has it
    _stream_of = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
        (lambda index: torch.cuda.current_stream(index).cuda_stream)
    _empty_like, _dense, _int32, _int64 = torch.empty_like, torch.contiguous_format, torch.int32, torch.int64
    lib()
    _torch = torch


def _refuse(name, x, index, dtype=None, shape=None, dense=False):
    """Raises for what is wrong with an operand; returns the token stride of
    rows [tokens, heads, head_dim] that are right after all (a stride of a
    dimension of one)."""
    if x.get_device() != index or index < 0:
        raise TypeError("%s must be a CUDA tensor on the operands' device" % name)
    if (x.dtype not in _ACT) if dtype is None else x.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, "bfloat16 or float16" if dtype is None else dtype, x.dtype))
    if (x.dim() != 3) if shape is None else x.shape != shape:
        raise ValueError("%s must have shape %s, got %s" %
                         (name, "[tokens, heads, head_dim]" if shape is None else tuple(shape), tuple(x.shape)))
    if dense:
        raise TypeError("%s must be contiguous" % name)
    tokens, h, d = x.shape
    s0, s1, s2 = x.stride()
    if (s2 != 1 and d > 1) or (s1 != d and h > 1):
        raise ValueError("%s: the heads of a token must be side by side, got shape %s with strides %s" %
                         (name, tuple(x.shape), x.stride()))
    return s0 if tokens > 1 or s0 >= h * d else h * d


def _rows(name, x, index, dtype, shape):
    """The token stride of an operand that has to have this type and shape."""
    s = x.stride()
    if x.shape != shape or x.dtype is not dtype or x.get_device() != index or s[-1] != 1 or s[-2] != shape[2] or \
            s[0] < shape[1] * shape[2]:
        return _refuse(name, x, index, dtype, shape)
    return s[0]


def _index(name, t, dtype, shape, index):
    if t.dtype is not dtype or t.shape != shape or t.get_device() != index or not t.is_contiguous():
        _refuse(name, t, index, dtype, shape, True)
    return t.data_ptr()


def rope(x, positions, rope, out=None):
    """x[tokens, heads, head_dim] bf16/fp16 with every head rotated by its
    token's positions: int32 [tokens], or [axes, tokens] for a Rope with
    sections.  x may be a view of a fused projection's rows; out may be x."""
    if _torch is None:
        _load_torch()
    dev, dtype, shape, s = x.get_device(), x.dtype, x.shape, x.stride()
    act = _ACT.get(dtype)
    if act is None or dev < 0 or len(shape) != 3:
        _refuse("x", x, dev)
    tokens, heads, dim = shape
    xs = s[0] if s[2] == 1 and s[1] == dim and s[0] >= heads * dim else _refuse("x", x, dev)
    if out is None:
        out, os_ = _empty_like(x, memory_format=_dense), heads * dim
    else:
        os_ = _rows("out", out, dev, dtype, shape)
    if rope.index != dev:
        raise TypeError("the rope's table must be on the operands' device")
    axes = rope.axes
    pos = _index("positions", positions, _int32, (tokens,) if axes == 1 and positions.dim() == 1 else (axes, tokens), dev)
    st = _lib.fp8w_rope(x.data_ptr(), act, tokens, heads, dim, xs, pos, rope._ref, out.data_ptr(), os_, _stream_of(dev))
    if st:
        _check(st)
    return out


def rope_append(q, k, v, slots, cache, positions=None, rope=None, out=None):
    """One launch for a block's new tokens: q[tokens, q_heads, head_dim]
    rotated (returned; q None: returns None), k rotated and v as it is
    [tokens, kv_heads, head_dim] put to slots int64 [tokens] of the cache
    (page * page_size + offset; negative: a padded token).  rope None: no
    rotation."""
    if _torch is None:
        _load_torch()
    dev, dim, dtype = cache.index, cache.head_dim, k.dtype
    act = _ACT.get(dtype)
    if act is None or k.dim() != 3:
        _refuse("k", k, dev)
    tokens = k.shape[0]
    shape = (tokens, cache.kv_heads, dim)
    ks, vs = _rows("k", k, dev, dtype, shape), _rows("v", v, dev, dtype, shape)
    pos = spec = qp = op = None
    qs = os_ = heads = 0
    if (rope is None) != (positions is None):
        raise ValueError("positions and rope come together")
    if rope is not None:
        if rope.index != dev:
            raise TypeError("the rope's table must be on the operands' device")
        axes, spec = rope.axes, rope._ref
        pos = _index("positions", positions, _int32, (tokens,) if axes == 1 and positions.dim() == 1 else (axes, tokens), dev)
    if q is not None:
        if q.dim() != 3:
            _refuse("q", q, dev)
        heads = q.shape[1]
        shape = (tokens, heads, dim)
        qs, qp = _rows("q", q, dev, dtype, shape), q.data_ptr()
        if out is None:
            out, os_ = _empty_like(q, memory_format=_dense), heads * dim
        else:
            os_ = _rows("out", out, dev, dtype, shape)
        op = out.data_ptr()
    st = _lib.fp8w_rope_append(qp, k.data_ptr(), v.data_ptr(), act, tokens, heads, qs, ks, vs, pos, spec,
                               _index("slots", slots, _int64, (tokens,), dev), cache._ref, op, os_, _stream_of(dev))
    if st:
        _check(st)
    return None if q is None else out


def paged_attention(q, cache, block_table, lens, starts=None, scale=None, window=0, max_new=0, max_len=0, out=None):
    """Causal attention of each sequence's new tokens q[tokens, q_heads,
    head_dim] over its lens[s] tokens in the cache (the new ones appended
    before).  block_table int32 [seqs, width], lens int32 [seqs]; starts int32
    [seqs + 1]: first token of each sequence (None: one token each).  scale
    defaults to head_dim ** -0.5.  window: positions a token sees (0: all).
    max_new: a bound on a sequence's new tokens, max_len: about the longest of
    lens, where the caller knows them on the host (0: not known)."""
    if _torch is None:
        _load_torch()
    dev, dim, dtype = cache.index, cache.head_dim, q.dtype
    act = _ACT.get(dtype)
    if act is None or q.dim() != 3 or block_table.dim() != 2:
        _refuse("q", q, dev)
        raise ValueError("block_table must have two dimensions")
    tokens, heads, d = q.shape
    seqs, width = pages = block_table.shape
    shape = (tokens, heads, dim)
    qs = _rows("q", q, dev, dtype, shape)
    if out is None:
        out, os_ = _empty_like(q, memory_format=_dense), heads * dim
    else:
        os_ = _rows("out", out, dev, dtype, shape)
    st = _lib.fp8w_paged_attention(
        q.data_ptr(), act, tokens, heads, qs, cache._ref, _index("block_table", block_table, _int32, pages, dev), width,
        _index("lens", lens, _int32, (seqs,), dev), None if starts is None else _index("starts", starts, _int32, (seqs + 1,), dev),
        seqs, dim ** -0.5 if scale is None else scale, window, max_new, max_len, out.data_ptr(), os_, _stream_of(dev))
    if st:
        _check(st)
    return out


def device_error():
    """Nonzero if a kernel gave up a bounded wait, or met an index out of its
    range, since the last call (syncs)."""
    return lib().fp8w_device_error()
