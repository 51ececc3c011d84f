"""ctypes binding of libwq.so: the C entry points under the same names.

Argument marshalling only: each function checks that tensors are CUDA,
contiguous and of the expected dtype, passes raw pointers and the current
torch CUDA stream, and raises on a non-OK status. Every step of the product
runs in the library's CUDA kernels; there is no CPU or library fallback, and
importing this module fails loudly when libwq.so is missing.
"""

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libwq.so")

WQ_OK = 0
WQ_ERR_INVALID_ARG = 1
WQ_ERR_UNSUPPORTED = 2
WQ_ERR_ALIGNMENT = 3
WQ_ERR_CUDA = 4
WQ_ERR_TIMEOUT = 5
WQ_ERR_WORKSPACE = 6

WQ_FMT_INT4_ASYM = 0
WQ_FMT_NF4 = 1
WQ_BF16 = 0
WQ_FP16 = 1
WQ_FP32 = 2
WQ_OP_GEMV = 0
WQ_OP_GEMM = 1
WQ_OP_MSD_GEMM = 2
WQ_OP_MX_GEMV = 3
WQ_OP_MX_GEMM = 4

# every symbol include/wq.h declares
EXPORTED = [
    "wq_status_string", "wq_version", "wq_nf4_codebook", "wq_packed_sizes",
    "wq_quantize_pack", "wq_unpack", "wq_nf4_dequant", "wq_int4_dequant",
    "wq_w4a16_gemv", "wq_w4a16_gemm", "wq_msd_decompose", "wq_msd_gemm",
    "wq_workspace_bytes", "wq_device_error", "wq_msd_gemm_noalloc",
    "wq_residual", "wq_select_salient", "wq_w4a16_gemv_corrected", "wq_w4a16_gemv_salient",
    "wq_test_set_wait", "wq_mx_quantize", "wq_mx_decompose", "wq_mx_gemv", "wq_msd_gemm_nf4",
    "wq_msd_decode_attention", "wq_msd_decode_attention_workspace",
    "wq_test_set_attention_split", "wq_kv_block_values", "wq_kv_append", "wq_kv_read",
    "wq_prefix_attention", "wq_prefix_attention_workspace", "wq_mx_quantize_planes", "wq_mx_gemm",
    "wq_test_set_prefix_path",
]

_DTYPES = {torch.bfloat16: WQ_BF16, torch.float16: WQ_FP16, torch.float32: WQ_FP32}


class WqError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__("%s: %s (status %d)" % (where, status_string(status), status))


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError("libwq.so not built at %s; run "
                          "`python -m bit_weight_quantized_weights_b200.build_lib`" % LIB_PATH)
    lib = ctypes.CDLL(LIB_PATH)
    P, I64, I32, SZ, U32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t, \
        ctypes.c_uint32
    sig = {
        "wq_status_string": ([ctypes.c_int], ctypes.c_char_p),
        "wq_version": ([], ctypes.c_char_p),
        "wq_nf4_codebook": ([ctypes.POINTER(ctypes.c_float)], ctypes.c_int),
        "wq_packed_sizes": ([ctypes.c_int, I64, I64, I32, ctypes.POINTER(SZ),
                             ctypes.POINTER(SZ), ctypes.POINTER(SZ)], ctypes.c_int),
        "wq_quantize_pack": ([ctypes.c_int, P, I64, I64, I32, P, P, P, P], ctypes.c_int),
        "wq_unpack": ([ctypes.c_int, P, I64, I64, P, P], ctypes.c_int),
        "wq_nf4_dequant": ([P, P, I64, I32, P, ctypes.c_int, P], ctypes.c_int),
        "wq_int4_dequant": ([P, P, P, I64, I64, I32, P, ctypes.c_int, P], ctypes.c_int),
        "wq_w4a16_gemv": ([P, I64, I64, I64, ctypes.c_int, I32, P, P, P, P, P, SZ, P],
                          ctypes.c_int),
        "wq_w4a16_gemm": ([P, I64, I64, I64, ctypes.c_int, I32, P, P, P, P, P, SZ, P],
                          ctypes.c_int),
        "wq_msd_decompose": ([P, I64, I64, I32, P, P, P], ctypes.c_int),
        "wq_msd_gemm": ([P, I64, I64, I64, I32, I32, P, P, P, P, P, SZ, P], ctypes.c_int),
        "wq_workspace_bytes": ([ctypes.c_int, I64, I64, I64, I32, I32, ctypes.POINTER(SZ)],
                               ctypes.c_int),
        "wq_device_error": ([P, ctypes.c_int, ctypes.POINTER(U32)], ctypes.c_int),
        "wq_test_set_wait": ([ctypes.c_uint64, ctypes.c_int], ctypes.c_int),
        "wq_mx_quantize": ([P, I64, I64, P, P, P], ctypes.c_int),
        "wq_mx_decompose": ([P, I64, I64, I32, P, P, P], ctypes.c_int),
        "wq_mx_gemv": ([P, I64, I64, I64, I32, P, P, P, P, SZ, P], ctypes.c_int),
        "wq_msd_gemm_nf4": ([P, I64, I64, I64, I32, P, P, P, P, SZ, P], ctypes.c_int),
        "wq_msd_decode_attention": ([P, I64, I64, I64, I64, I32, I32, P, P, P, P, P, P, P, P, SZ,
                                     P], ctypes.c_int),
        "wq_msd_decode_attention_workspace": ([I64, I64, I64, I64, I32, I32, ctypes.POINTER(SZ)],
                                              ctypes.c_int),
        "wq_test_set_attention_split": ([I32], ctypes.c_int),
        "wq_test_set_prefix_path": ([I32], ctypes.c_int),
        "wq_kv_block_values": ([P, I64, I64, I32, P, P], ctypes.c_int),
        "wq_kv_append": ([P, P, ctypes.c_int, I64, I64, I32, ctypes.POINTER(I64),
                          ctypes.POINTER(I64), I64, P, P, I64, P, P, P, P, P, P, P], ctypes.c_int),
        "wq_kv_read": ([P, P, P, P, P, P, I64, I64, I32, I64, P, P, I64, P, P, ctypes.c_int,
                        ctypes.POINTER(I64), ctypes.POINTER(I64), P], ctypes.c_int),
        "wq_prefix_attention": ([P, ctypes.c_int, I64, I64, I64, I64, I32, I64, I64, P, P, P, P, P,
                                 P, I64, P, P, P, P, P, P, P, P, P, SZ, P], ctypes.c_int),
        "wq_prefix_attention_workspace": ([I64, I64, I64, I32, I64, I64, ctypes.POINTER(SZ)],
                                          ctypes.c_int),
        "wq_mx_quantize_planes": ([P, ctypes.c_int, I64, I64, I64, I32, P, P, P], ctypes.c_int),
        "wq_mx_gemm": ([P, P, I64, I64, I64, I32, P, P, P, P, SZ, P], ctypes.c_int),
        "wq_msd_gemm_noalloc": ([P, I64, I64, I64, I32, I32, P, P, P, P, P], ctypes.c_int),
        "wq_residual": ([ctypes.c_int, P, I64, I64, I32, P, P, P, P, P], ctypes.c_int),
        "wq_select_salient": ([P, I64, I64, I32, P, P], ctypes.c_int),
        "wq_w4a16_gemv_corrected": ([P, I64, I64, I64, ctypes.c_int, I32, P, P, P, P, P, I32, P,
                                     P], ctypes.c_int),
        "wq_w4a16_gemv_salient": ([P, I64, I64, I64, ctypes.c_int, I32, P, P, P, P, I32, P, P,
                                   P], ctypes.c_int),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    return lib


lib = _load()


def status_string(status):
    return lib.wq_status_string(int(status)).decode()


def version():
    return lib.wq_version().decode()


def _check(status, where):
    if status != WQ_OK:
        raise WqError(status, where)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _on(stream, wrapper, *args):
    """A call that is given a stream: made with it as the current one, so that what the
    wrapper allocates comes from that stream's pool. Memory of another pool may still
    be in use on the stream it belongs to, and a workspace that the wrapper drops would
    go back there while the call runs. The results are marked as used on the caller's
    current stream too."""
    with torch.cuda.stream(stream):
        out = wrapper(*args)
    for t in out if isinstance(out, tuple) else (out,):
        if t is not None:
            t.record_stream(torch.cuda.current_stream(t.device))
    return out


# The current device and a device's current stream, as integers: a call of a few
# microseconds on the GPU is launched from here, and the Stream objects of
# torch.cuda.current_stream() cost as much as the launch.
_current_device = torch.cuda.current_device
_BF16, _F16, _I32, _U8 = torch.bfloat16, torch.float16, torch.int32, torch.uint8
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # (None without CUDA)


def _cuda(t, dtype, name):
    if t is None:
        return
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if dtype is not None and t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


# ---------------------------------------------------------------------------
# host-only queries
# ---------------------------------------------------------------------------

def wq_nf4_codebook():
    """The 16 NF4 code values the kernels use (host computation)."""
    buf = (ctypes.c_float * 16)()
    _check(lib.wq_nf4_codebook(buf), "wq_nf4_codebook")
    return [float(v) for v in buf]


def wq_packed_sizes(fmt, n, k, group):
    a, b, c = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib.wq_packed_sizes(fmt, n, k, group, ctypes.byref(a), ctypes.byref(b),
                               ctypes.byref(c)), "wq_packed_sizes")
    return a.value, b.value, c.value


def wq_workspace_bytes(op, m, n, k, group, n_components=2):
    out = ctypes.c_size_t()
    _check(lib.wq_workspace_bytes(op, m, n, k, group, n_components, ctypes.byref(out)),
           "wq_workspace_bytes")
    return out.value


# ---------------------------------------------------------------------------
# device entry points
# ---------------------------------------------------------------------------

def alloc_packed(fmt, n, k, group, device="cuda"):
    """Allocate (qweight, scales, zeros) tensors of the canonical packed layout."""
    qb, sb, zb = wq_packed_sizes(fmt, n, k, group)
    if fmt == WQ_FMT_INT4_ASYM:
        qw = torch.empty(n, k // 8, dtype=torch.int32, device=device)
        sc = torch.empty(n, k // group, dtype=torch.float16, device=device)
        zr = torch.empty(n, k // group, dtype=torch.float16, device=device)
    else:
        qw = torch.empty(n * k // 2, dtype=torch.uint8, device=device)
        sc = torch.empty(n * k // 64, dtype=torch.float32, device=device)
        zr = None
    assert qw.numel() * qw.element_size() == qb and sc.numel() * sc.element_size() == sb
    return qw, sc, zr


def wq_quantize_pack(fmt, w, group, qweight=None, scales=None, zeros=None, stream=None):
    """Quantize fp32 W [N, K] on the GPU; returns (qweight, scales, zeros)."""
    if stream is not None:
        return _on(stream, wq_quantize_pack, fmt, w, group, qweight, scales, zeros)
    _cuda(w, torch.float32, "W")
    n, k = w.shape
    if qweight is None:
        qweight, scales, zeros = alloc_packed(fmt, n, k, group, w.device)
    _check(lib.wq_quantize_pack(fmt, _ptr(w), n, k, group, _ptr(qweight), _ptr(scales),
                                _ptr(zeros), _stream()), "wq_quantize_pack")
    return qweight, scales, zeros


def wq_unpack(fmt, qweight, n, k, out=None, stream=None):
    if stream is not None:
        return _on(stream, wq_unpack, fmt, qweight, n, k, out)
    _cuda(qweight, None, "qweight")
    if out is None:
        out = torch.empty(n * k, dtype=torch.uint8, device=qweight.device)
    _check(lib.wq_unpack(fmt, _ptr(qweight), n, k, _ptr(out), _stream()), "wq_unpack")
    return out


def wq_nf4_dequant(codes, absmax, numel, out=None, out_dtype=torch.bfloat16, stream=None):
    if stream is not None:
        return _on(stream, wq_nf4_dequant, codes, absmax, numel, out, out_dtype)
    _cuda(codes, torch.uint8, "codes")
    _cuda(absmax, torch.float32, "absmax")
    if out is None:
        out = torch.empty(numel, dtype=out_dtype, device=codes.device)
    dt = WQ_BF16 if out.dtype == torch.bfloat16 else WQ_FP16
    _check(lib.wq_nf4_dequant(_ptr(codes), _ptr(absmax), numel, 64, _ptr(out), dt,
                              _stream()), "wq_nf4_dequant")
    return out


def wq_int4_dequant(qweight, scales, zeros, n, k, group, out=None, out_dtype=torch.bfloat16,
                    stream=None):
    if stream is not None:
        return _on(stream, wq_int4_dequant, qweight, scales, zeros, n, k, group, out, out_dtype)
    _cuda(qweight, torch.int32, "qweight")
    _cuda(scales, torch.float16, "scales")
    _cuda(zeros, torch.float16, "zeros")
    if out is None:
        out = torch.empty(n, k, dtype=out_dtype, device=qweight.device)
    dt = WQ_BF16 if out.dtype == torch.bfloat16 else WQ_FP16
    _check(lib.wq_int4_dequant(_ptr(qweight), _ptr(scales), _ptr(zeros), n, k, group, _ptr(out),
                               dt, _stream()), "wq_int4_dequant")
    return out


def _product(fn, name, x, n, fmt, group, qweight, scales, zeros, out, workspace):
    _cuda(x, torch.bfloat16, "x")
    m, k = x.shape
    if out is None:
        out = torch.empty(m, n, dtype=torch.bfloat16, device=x.device)
    _cuda(out, torch.bfloat16, "y")
    ws = _ptr(workspace)
    wsb = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(fn(_ptr(x), m, n, k, fmt, group, _ptr(qweight), _ptr(scales), _ptr(zeros), _ptr(out),
              ws, wsb, _stream()), name)
    return out


def wq_w4a16_gemv(x, n, fmt, group, qweight, scales, zeros, out=None, stream=None):
    """Decode GEMV: x bf16 [M<=16, K] -> y bf16 [M, N]."""
    if stream is not None:
        return _on(stream, wq_w4a16_gemv, x, n, fmt, group, qweight, scales, zeros, out)
    return _product(lib.wq_w4a16_gemv, "wq_w4a16_gemv", x, n, fmt, group, qweight, scales, zeros,
                    out, None)


def wq_residual(fmt, w, group, qweight, scales, zeros, out=None, stream=None):
    """R^T = fp16(W - dequant(W_q)) as fp16 [K, N] from fp32 W [N, K]."""
    if stream is not None:
        return _on(stream, wq_residual, fmt, w, group, qweight, scales, zeros, out)
    _cuda(w, torch.float32, "W")
    n, k = w.shape
    if out is None:
        out = torch.empty(k, n, dtype=torch.float16, device=w.device)
    _cuda(out, torch.float16, "residual_t")
    _check(lib.wq_residual(fmt, _ptr(w), n, k, group, _ptr(qweight), _ptr(scales), _ptr(zeros),
                           _ptr(out), _stream()), "wq_residual")
    return out


def wq_select_salient(x, k, out=None, stream=None):
    """The k salient channels of bf16 x [M, K] as int32 [k], increasing."""
    if stream is not None:
        return _on(stream, wq_select_salient, x, k, out)
    _cuda(x, torch.bfloat16, "x")
    m, kk = x.shape
    if out is None:
        out = torch.empty(max(k, 0), dtype=torch.int32, device=x.device)
    _cuda(out, torch.int32, "idx")
    _check(lib.wq_select_salient(_ptr(x), m, kk, k, _ptr(out), _stream()),
           "wq_select_salient")
    return out


def wq_w4a16_gemv_corrected(x, n, fmt, group, qweight, scales, zeros, residual_t, idx, out=None,
                            stream=None):
    """Decode GEMV plus the residuals of the channels idx (int32 [k])."""
    if stream is not None:
        return _on(stream, wq_w4a16_gemv_corrected, x, n, fmt, group, qweight, scales, zeros,
                   residual_t, idx, out)
    _cuda(x, torch.bfloat16, "x")
    m, k = x.shape
    if out is None:
        out = torch.empty(m, n, dtype=torch.bfloat16, device=x.device)
    _cuda(out, torch.bfloat16, "y")
    nsel = 0 if idx is None else idx.numel()
    _check(lib.wq_w4a16_gemv_corrected(_ptr(x), m, n, k, fmt, group, _ptr(qweight), _ptr(scales),
                                       _ptr(zeros), _ptr(residual_t), _ptr(idx), nsel, _ptr(out),
                                       _stream()), "wq_w4a16_gemv_corrected")
    return out


def wq_w4a16_gemv_salient(x, n, fmt, group, qweight, scales, zeros, residual_t, nsel, idx=None,
                          out=None, stream=None):
    """One corrected decode step: select the nsel salient channels into idx
    (int32 scratch, allocated if None), then the corrected GEMV, launched to
    overlap the selection. Returns y."""
    if stream is not None:
        return _on(stream, wq_w4a16_gemv_salient, x, n, fmt, group, qweight, scales, zeros,
                   residual_t, nsel, idx, out)
    _cuda(x, torch.bfloat16, "x")
    m, k = x.shape
    if out is None:
        out = torch.empty(m, n, dtype=torch.bfloat16, device=x.device)
    _cuda(out, torch.bfloat16, "y")
    if idx is None:
        idx = torch.empty(max(nsel, 1), dtype=torch.int32, device=x.device)
    _cuda(idx, torch.int32, "idx")
    _check(lib.wq_w4a16_gemv_salient(_ptr(x), m, n, k, fmt, group, _ptr(qweight), _ptr(scales),
                                     _ptr(zeros), _ptr(residual_t), nsel, _ptr(idx), _ptr(out),
                                     _stream()), "wq_w4a16_gemv_salient")
    return out


def gemm_workspace(m, n, k, group, device="cuda"):
    nbytes = wq_workspace_bytes(WQ_OP_GEMM, m, n, k, group)
    return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device)


def wq_w4a16_gemm(x, n, fmt, group, qweight, scales, zeros, workspace=None, out=None,
                  stream=None):
    """Prefill GEMM with fused dequantization on tcgen05: y bf16 [M, N]."""
    if stream is not None:
        return _on(stream, wq_w4a16_gemm, x, n, fmt, group, qweight, scales, zeros, workspace, out)
    _cuda(x, torch.bfloat16, "x")
    if workspace is None:
        workspace = gemm_workspace(x.shape[0], n, x.shape[1], group, x.device)
    return _product(lib.wq_w4a16_gemm, "wq_w4a16_gemm", x, n, fmt, group, qweight, scales, zeros,
                    out, workspace)


def wq_msd_decompose(x, n_components=2, digits=None, comp_scales=None, stream=None):
    """Digit planes int8 [C, M, K] and scales fp32 [C, M] of bf16 x [M, K]."""
    if stream is not None:
        return _on(stream, wq_msd_decompose, x, n_components, digits, comp_scales)
    _cuda(x, torch.bfloat16, "x")
    m, k = x.shape
    if digits is None:
        digits = torch.empty(n_components, m, k, dtype=torch.int8, device=x.device)
        comp_scales = torch.empty(n_components, m, dtype=torch.float32, device=x.device)
    _check(lib.wq_msd_decompose(_ptr(x), m, k, n_components, _ptr(digits), _ptr(comp_scales),
                                _stream()), "wq_msd_decompose")
    return digits, comp_scales


def msd_workspace(m, n, k, group, n_components=2, device="cuda"):
    nbytes = wq_workspace_bytes(WQ_OP_MSD_GEMM, m, n, k, group, n_components)
    return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device)


def wq_msd_gemm(x, n, n_components, group, qweight, scales, zeros, workspace=None, out=None,
                stream=None):
    """Multi-Scale Dequant GEMM: y bf16 [M, N] from int8 digit planes of x."""
    if stream is not None:
        return _on(stream, wq_msd_gemm, x, n, n_components, group, qweight, scales, zeros,
                   workspace, out)
    _cuda(x, torch.bfloat16, "x")
    m, k = x.shape
    if workspace is None:
        workspace = msd_workspace(m, n, k, group, n_components, x.device)
    if out is None:
        out = torch.empty(m, n, dtype=torch.bfloat16, device=x.device)
    _check(lib.wq_msd_gemm(_ptr(x), m, n, k, n_components, group, _ptr(qweight), _ptr(scales),
                           _ptr(zeros), _ptr(out), _ptr(workspace),
                           workspace.numel() * workspace.element_size(), _stream()),
           "wq_msd_gemm")
    return out


def wq_msd_gemm_noalloc(x, n, n_components, group, qweight, scales, zeros, out=None,
                        stream=None):
    """wq_msd_gemm without a workspace: the library's fixed device scratch array
    is used, so the call allocates nothing (problem size limited to 8 MiB of
    scratch; calls overlapping on the GPU race on it)."""
    if stream is not None:
        return _on(stream, wq_msd_gemm_noalloc, x, n, n_components, group, qweight, scales, zeros,
                   out)
    _cuda(x, torch.bfloat16, "x")
    m, k = x.shape
    if out is None:
        out = torch.empty(m, n, dtype=torch.bfloat16, device=x.device)
    _check(lib.wq_msd_gemm_noalloc(_ptr(x), m, n, k, n_components, group, _ptr(qweight),
                                   _ptr(scales), _ptr(zeros), _ptr(out), _stream()),
           "wq_msd_gemm_noalloc")
    return out


def wq_device_error(clear=True, stream=None):
    """Synchronise and read the sticky device error word: (status, detail)."""
    d = ctypes.c_uint32()
    st = lib.wq_device_error(_stream(stream), 1 if clear else 0, ctypes.byref(d))
    return st, d.value


def wq_test_set_wait(limit_ns=0, stall=0):
    """Test hook of the bounded device waits (see include/wq.h): the wait
    limit in ns (0 = the default 2 s) and whether the loader withholds the
    first k-tile of the tensor-core kernels."""
    _check(lib.wq_test_set_wait(int(limit_ns), int(stall)), "wq_test_set_wait")


def wq_mx_quantize(w, codes=None, scales=None, stream=None):
    """MXFP4 weights: w fp32 [N, K] -> (codes uint8 [N, K/2], scale bytes uint8 [N, K/32])."""
    if stream is not None:
        return _on(stream, wq_mx_quantize, w, codes, scales)
    _cuda(w, torch.float32, "w")
    n, k = w.shape
    if codes is None:
        codes = torch.empty(n, k // 2, dtype=torch.uint8, device=w.device)
    if scales is None:
        scales = torch.empty(n, k // 32, dtype=torch.uint8, device=w.device)
    _check(lib.wq_mx_quantize(_ptr(w), n, k, _ptr(codes), _ptr(scales), _stream()),
           "wq_mx_quantize")
    return codes, scales


def wq_mx_decompose(x, n_passes=2, planes=None, scales=None, stream=None):
    """x bf16 [M, K] -> (planes uint8 [P, M, K] E4M3 bytes, scale bytes uint8 [P, M, K/32])."""
    if stream is not None:
        return _on(stream, wq_mx_decompose, x, n_passes, planes, scales)
    _cuda(x, torch.bfloat16, "x")
    m, k = x.shape
    if planes is None:
        planes = torch.empty(n_passes, m, k, dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty(n_passes, m, k // 32, dtype=torch.uint8, device=x.device)
    _check(lib.wq_mx_decompose(_ptr(x), m, k, n_passes, _ptr(planes), _ptr(scales),
                               _stream()), "wq_mx_decompose")
    return planes, scales


def mx_workspace(m, n, k, n_passes=2, device="cuda"):
    nbytes = wq_workspace_bytes(WQ_OP_MX_GEMV, m, n, k, 0, n_passes)
    return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device)


def wq_mx_gemv(x, n, n_passes, codes, scales, workspace=None, out=None, stream=None):
    """y bf16 [M, N] = x_hat . w_hat^T (MXFP4 weights; two MXFP4 passes or one MXFP8 pass)."""
    if stream is not None:
        return _on(stream, wq_mx_gemv, x, n, n_passes, codes, scales, workspace, out)
    _cuda(x, torch.bfloat16, "x")
    m, k = x.shape
    if workspace is None:
        workspace = mx_workspace(m, n, k, n_passes, x.device)
    if out is None:
        out = torch.empty(m, n, dtype=torch.bfloat16, device=x.device)
    _check(lib.wq_mx_gemv(_ptr(x), m, n, k, n_passes, _ptr(codes), _ptr(scales), _ptr(out),
                          _ptr(workspace), workspace.numel(), _stream()), "wq_mx_gemv")
    return out


def wq_mx_quantize_planes(x, n_planes=2, planes=None, scales=None, stream=None):
    """MXFP4 activations kept in 4 bits: x [M, K] (bf16, fp16 or fp32; rows may
    be strided) -> (planes uint8 [P, M, K/2], scale bytes uint8 [P, M, K/32])."""
    if stream is not None:
        return _on(stream, wq_mx_quantize_planes, x, n_planes, planes, scales)
    dev = _current_device()
    dt = _DTYPES.get(x.dtype)
    if dt is None or x.dim() != 2:
        raise ValueError("x must be a 2-D bfloat16, float16 or float32 tensor")
    m, k = x.shape
    ldx, inner = x.stride()
    if inner != 1 and k > 1:
        raise ValueError("the rows of x must be contiguous")
    if planes is None:
        planes = x.new_empty((n_planes, m, k // 2), dtype=torch.uint8)
    elif planes.dtype is not torch.uint8 or planes.shape != (n_planes, m, k // 2) or \
            not planes.is_contiguous():
        raise ValueError("planes must be uint8 [%d, %d, %d]" % (n_planes, m, k // 2))
    if scales is None:
        scales = planes.new_empty((n_planes, m, k // 32))
    elif scales.dtype is not torch.uint8 or scales.shape != (n_planes, m, k // 32) or \
            not scales.is_contiguous():
        raise ValueError("scales must be uint8 [%d, %d, %d]" % (n_planes, m, k // 32))
    if x.get_device() != dev or planes.get_device() != dev or scales.get_device() != dev:
        _on_device(dev, x, planes, scales)
    status = lib.wq_mx_quantize_planes(
        x.data_ptr(), dt, ldx if m > 1 else k, m, k, n_planes, planes.data_ptr(),
        scales.data_ptr(), _raw_stream(dev))
    if status:
        raise WqError(status, "wq_mx_quantize_planes")
    return planes, scales


def mx_gemm_workspace(m, n, k, n_planes=2, device="cuda"):
    nbytes = wq_workspace_bytes(WQ_OP_MX_GEMM, m, n, k, 0, n_planes)
    return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device)


def wq_mx_gemm(planes, plane_scales, n, codes, scales, workspace=None, out=None, stream=None):
    """y bf16 [M, N] = (sum of the MXFP4 planes) . w_hat^T for any M, on the FP4
    tensor cores: planes and plane_scales as wq_mx_quantize_planes returns
    them, codes and scales as wq_mx_quantize packs the weights [N, K]."""
    if stream is not None:
        return _on(stream, wq_mx_gemm, planes, plane_scales, n, codes, scales, workspace, out)
    dev = _current_device()
    if planes.dtype is not _U8 or plane_scales.dtype is not _U8 or codes.dtype is not _U8 or \
            scales.dtype is not _U8 or not planes.is_contiguous() or \
            not plane_scales.is_contiguous() or not codes.is_contiguous() or \
            not scales.is_contiguous():
        raise ValueError("planes, codes and their scales must be uint8 and contiguous")
    if planes.dim() != 3:
        raise ValueError("planes must be [P, M, K/2]")
    p, m, kh = planes.shape
    k = 2 * kh
    if plane_scales.shape != (p, m, k // 32) or codes.shape != (n, kh) or \
            scales.shape != (n, k // 32):
        raise ValueError("scales or weights do not match planes %s and N = %d"
                         % (tuple(planes.shape), n))
    if workspace is None:
        workspace = mx_gemm_workspace(m, n, k, p, planes.device)
    if out is None:
        out = planes.new_empty((m, n), dtype=torch.bfloat16)
    elif out.dtype is not torch.bfloat16 or out.shape != (m, n) or not out.is_contiguous():
        raise ValueError("y must be bfloat16 [%d, %d], contiguous" % (m, n))
    if planes.get_device() != dev or plane_scales.get_device() != dev or \
            codes.get_device() != dev or scales.get_device() != dev or \
            workspace.get_device() != dev or out.get_device() != dev:
        _on_device(dev, planes, plane_scales, codes, scales, workspace, out)
    status = lib.wq_mx_gemm(
        planes.data_ptr(), plane_scales.data_ptr(), m, n, k, p, codes.data_ptr(),
        scales.data_ptr(), out.data_ptr(), workspace.data_ptr(),
        workspace.nbytes, _raw_stream(dev))
    if status:
        raise WqError(status, "wq_mx_gemm")
    return out


def wq_msd_gemm_nf4(x, n, n_components, codes, absmax, workspace=None, out=None, stream=None):
    """Decode MSD product with NF4 weights (integer codebook digits); M <= 16."""
    if stream is not None:
        return _on(stream, wq_msd_gemm_nf4, x, n, n_components, codes, absmax, workspace, out)
    _cuda(x, torch.bfloat16, "x")
    m, k = x.shape
    if workspace is None:
        workspace = msd_workspace(m, n, k, 64, n_components, x.device)
    if out is None:
        out = torch.empty(m, n, dtype=torch.bfloat16, device=x.device)
    _check(lib.wq_msd_gemm_nf4(_ptr(x), m, n, k, n_components, _ptr(codes), _ptr(absmax),
                               _ptr(out), _ptr(workspace), workspace.numel(), _stream()),
           "wq_msd_gemm_nf4")
    return out


def kv_quantize_keys(k, stream=None):
    """INT4-quantize a key cache fp32 [B, Hkv, L, D] on the GPU, one group per
    (sequence, head, token) row: returns (codes int32 [B, Hkv, L, D/8], scales
    fp16 [B, Hkv, L], zeros fp16 [B, Hkv, L])."""
    if stream is not None:
        return _on(stream, kv_quantize_keys, k)
    _cuda(k, torch.float32, "k")
    b, hkv, length, d = k.shape
    qw, sc, zr = wq_quantize_pack(WQ_FMT_INT4_ASYM, k.reshape(-1, d), d)
    return (qw.view(b, hkv, length, d // 8), sc.view(b, hkv, length), zr.view(b, hkv, length))


def wq_kv_block_values(codes, rows, length, d, out=None, stream=None):
    """V codes from the token layout (int32 [rows * L, D/8]) to blocks of 8
    tokens: int32 [rows, ceil(L/8), D]."""
    if stream is not None:
        return _on(stream, wq_kv_block_values, codes, rows, length, d, out)
    _cuda(codes, torch.int32, "codes")
    nblk = (length + 7) // 8
    if out is None:
        out = torch.empty(rows, nblk, d, dtype=torch.int32, device=codes.device)
    _check(lib.wq_kv_block_values(_ptr(codes), rows, length, d, _ptr(out), _stream()),
           "wq_kv_block_values")
    return out


def kv_quantize_values(v, stream=None):
    """INT4-quantize a value cache fp32 [B, Hkv, L, D] on the GPU, one group per
    (sequence, head, token) row: returns (codes int32 [B, Hkv, ceil(L/8), D] in
    blocks of 8 tokens, scales fp16 [B, Hkv, L], zeros fp16 [B, Hkv, L])."""
    if stream is not None:
        return _on(stream, kv_quantize_values, v)
    _cuda(v, torch.float32, "v")
    b, hkv, length, d = v.shape
    qw, sc, zr = wq_quantize_pack(WQ_FMT_INT4_ASYM, v.reshape(-1, d), d)
    blocked = wq_kv_block_values(qw, b * hkv, length, d)
    return (blocked.view(b, hkv, (length + 7) // 8, d), sc.view(b, hkv, length),
            zr.view(b, hkv, length))


def _on_device(dev, *tensors):
    """The library launches on the current device: tensors of another are refused."""
    for t in tensors:
        if t.get_device() != dev:
            raise ValueError("tensor on %s, but the current device is cuda:%d" % (t.device, dev))


def _kv_cache(k_cache, v_cache, dev):
    """Check the two parts of an INT4 cache against each other: (B, Hkv, capacity, D)."""
    kq, ks, kz = k_cache
    vq, vs, vz = v_cache
    shape = ks.shape
    if kq.dtype is _I32 and vq.dtype is _I32 and ks.dtype is _F16 and kz.dtype is _F16 and \
            vs.dtype is _F16 and vz.dtype is _F16 and kq.is_contiguous() and \
            vq.is_contiguous() and ks.is_contiguous() and kz.is_contiguous() and \
            vs.is_contiguous() and vz.is_contiguous() and kz.shape == shape and \
            vs.shape == shape and vz.shape == shape and kq.get_device() == dev and \
            vq.get_device() == dev and ks.get_device() == dev and kz.get_device() == dev and \
            vs.get_device() == dev and vz.get_device() == dev and len(shape) == 3:
        b, hkv, cap = shape
        d = vq.shape[-1]
        if kq.shape == (b, hkv, cap, d // 8) and vq.shape == (b, hkv, (cap + 7) // 8, d):
            return b, hkv, cap, d
    # something is wrong: say what
    for t, dt, name in ((kq, torch.int32, "k_codes"), (ks, torch.float16, "k_scales"),
                        (kz, torch.float16, "k_zeros"), (vq, torch.int32, "v_codes"),
                        (vs, torch.float16, "v_scales"), (vz, torch.float16, "v_zeros")):
        _cuda(t, dt, name)
    _on_device(dev, *k_cache, *v_cache)
    raise ValueError("KV cache shapes do not match: codes %s and %s, scales and zeros %s %s %s %s"
                     % tuple(tuple(t.shape) for t in (kq, vq, ks, kz, vs, vz)))


def kv_cache_alloc(b, hkv, capacity, d=128, device="cuda"):
    """An empty INT4 cache with room for `capacity` tokens a sequence: (k_cache,
    v_cache), each (codes, scales, zeros) as kv_quantize_keys and
    kv_quantize_values return them, zero-filled."""
    def part(*codes):
        return (torch.zeros(b, hkv, *codes, dtype=torch.int32, device=device),
                torch.zeros(b, hkv, capacity, dtype=torch.float16, device=device),
                torch.zeros(b, hkv, capacity, dtype=torch.float16, device=device))
    return part(capacity, d // 8), part((capacity + 7) // 8, d)


_Strides = ctypes.c_int64 * 2


def _kv_rows(k, v, cache, starts, offsets, dev):
    """Check packed rows [T, Hkv, D] against a cache: (T, dtype, strides of k and v)."""
    b, hkv, _, d = cache
    shape, kind = k.shape, k.dtype
    dt = _DTYPES.get(kind)
    if dt is None or v.dtype is not kind:
        raise ValueError("k and v must both be bfloat16, float16 or float32")
    t = shape[0] if len(shape) == 3 else -1
    if shape != (t, hkv, d) or v.shape != shape:
        raise ValueError("k and v must be [T, %d, %d], got %s and %s"
                         % (hkv, d, tuple(shape), tuple(v.shape)))
    k0, k1, k2 = k.stride()
    v0, v1, v2 = v.stride()
    if k2 != 1 or v2 != 1:
        raise ValueError("the last dimension of k and v must be contiguous")
    if starts.dtype is not _I32 or offsets.dtype is not _I32 or \
            starts.shape != (b,) or offsets.shape != (b + 1,) or \
            not starts.is_contiguous() or not offsets.is_contiguous():
        raise ValueError("starts must be int32 [%d] and offsets int32 [%d], contiguous" % (b, b + 1))
    if k.get_device() != dev or v.get_device() != dev or starts.get_device() != dev or \
            offsets.get_device() != dev:
        _on_device(dev, k, v, starts, offsets)
    if t == 1:  # the stride of one element means nothing
        k0 = v0 = 0
    if hkv == 1:
        k1 = v1 = 0
    return t, dt, _Strides(k0, k1), _Strides(v0, v1)


def wq_kv_append(k, v, k_cache, v_cache, starts, offsets, stream=None):
    """Quantize new tokens into an INT4 cache: rows k and v [T, Hkv, D] (bf16,
    fp16 or fp32; any strides with a contiguous last dimension that keep rows
    16-byte aligned), sequence b's being offsets[b] .. offsets[b + 1] - 1
    (int32 [B + 1]), written from cache position starts[b] (int32 [B]) on.
    k_cache and v_cache (kv_cache_alloc) are updated in place."""
    if stream is not None:
        return _on(stream, wq_kv_append, k, v, k_cache, v_cache, starts, offsets)
    dev = _current_device()
    b, hkv, cap, d = cache = _kv_cache(k_cache, v_cache, dev)
    t, dt, ks, vs = _kv_rows(k, v, cache, starts, offsets, dev)
    kq, kscale, kzero = k_cache
    vq, vscale, vzero = v_cache
    status = lib.wq_kv_append(
        k.data_ptr(), v.data_ptr(), dt, t, hkv, d, ks, vs, b, starts.data_ptr(),
        offsets.data_ptr(), cap, kq.data_ptr(), kscale.data_ptr(), kzero.data_ptr(),
        vq.data_ptr(), vscale.data_ptr(), vzero.data_ptr(),
        _raw_stream(dev))
    if status:
        raise WqError(status, "wq_kv_append")


def wq_kv_read(k_cache, v_cache, starts, offsets, total, dtype=torch.bfloat16, k_out=None,
               v_out=None, stream=None):
    """Rows of an INT4 cache read back: (k, v) [total, Hkv, D] of dtype bf16,
    fp16 or fp32 (k_out's and v_out's where they are given), token t of sequence
    b (offsets[b] <= t < offsets[b + 1]) from cache position starts[b] + t -
    offsets[b]. Rows behind offsets[B] of a given k_out and v_out stay as they
    were."""
    if stream is not None:
        return _on(stream, wq_kv_read, k_cache, v_cache, starts, offsets, total, dtype, k_out,
                   v_out)
    dev = _current_device()
    b, hkv, cap, d = cache = _kv_cache(k_cache, v_cache, dev)
    if k_out is None:
        k_out = k_cache[1].new_empty((total, hkv, d), dtype=dtype)
    if v_out is None:
        v_out = torch.empty_like(k_out) if k_out.is_contiguous() else \
            k_out.new_empty((total, hkv, d))
    t, dt, ks, vs = _kv_rows(k_out, v_out, cache, starts, offsets, dev)
    if t != total:
        raise ValueError("k_out and v_out must have %d rows" % total)
    kq, kscale, kzero = k_cache
    vq, vscale, vzero = v_cache
    status = lib.wq_kv_read(
        kq.data_ptr(), kscale.data_ptr(), kzero.data_ptr(), vq.data_ptr(), vscale.data_ptr(),
        vzero.data_ptr(), b, hkv, d, cap, starts.data_ptr(), offsets.data_ptr(), t,
        k_out.data_ptr(), v_out.data_ptr(), dt, ks, vs,
        _raw_stream(dev))
    if status:
        raise WqError(status, "wq_kv_read")
    return k_out, v_out


def prefix_attention_workspace(b, hq, hkv, prefix_len, capacity, d=128, device="cuda"):
    size = ctypes.c_size_t(0)
    _check(lib.wq_prefix_attention_workspace(b, hq, hkv, d, prefix_len, capacity,
                                             ctypes.byref(size)),
           "wq_prefix_attention_workspace")
    return torch.empty(max(int(size.value), 1), dtype=torch.uint8, device=device)


def wq_prefix_attention(q, prefix_k, prefix_v, k_cache, v_cache, lengths, prefix_len=None,
                        workspace=None, out=None, stream=None):
    """Decode attention over INT4 caches of a batch that shares a prefix: q
    bf16 or fp16 [B, Hq, D] (contiguous heads, any stride between sequences);
    prefix_k and prefix_v a cache of one sequence ([1, Hkv, ...]), of which the
    first prefix_len tokens (default: all) are attended by every sequence;
    k_cache and v_cache a cache of B sequences, of which sequence b attends the
    first lengths[b] (int32 [B]) tokens. Returns out [B, Hq, D] of q's type.
    prefix_k = prefix_v = None: no prefix."""
    if stream is not None:
        return _on(stream, wq_prefix_attention, q, prefix_k, prefix_v, k_cache, v_cache, lengths,
                   prefix_len, workspace, out)
    dev = _current_device()
    b, hkv, cap, d = _kv_cache(k_cache, v_cache, dev)
    shape, kind = q.shape, q.dtype
    if kind is not _BF16 and kind is not _F16:
        raise ValueError("q must be bfloat16 or float16, got %s" % kind)
    hq = shape[1] if len(shape) == 3 else 0
    if shape != (b, hq, d):
        raise ValueError("q must be [%d, Hq, %d], got %s" % (b, d, tuple(shape)))
    q0, q1, q2 = q.stride()
    if q2 != 1 or (hq > 1 and q1 != d):
        raise ValueError("the heads of q must be contiguous")
    if lengths.dtype is not _I32 or lengths.shape != (b,) or not lengths.is_contiguous():
        raise ValueError("lengths must be int32 [%d], contiguous" % b)
    if prefix_k is None and prefix_v is None:
        if prefix_len:
            raise ValueError("prefix_len is %d, but there is no prefix cache" % prefix_len)
        pre = (None,) * 6
        pcap, prefix_len = 0, 0
    else:
        one, ph, pcap, pd = _kv_cache(prefix_k, prefix_v, dev)
        if one != 1 or ph != hkv or pd != d:
            raise ValueError("the prefix cache must be [1, %d, capacity, ...] with D = %d" % (hkv, d))
        if prefix_len is None:
            prefix_len = pcap
        kq, kscale, kzero = prefix_k
        vq, vscale, vzero = prefix_v
        pre = (kq.data_ptr(), kscale.data_ptr(), kzero.data_ptr(), vq.data_ptr(),
               vscale.data_ptr(), vzero.data_ptr())
    if workspace is None:
        workspace = prefix_attention_workspace(b, hq, hkv, prefix_len, cap, d, q.device)
    if out is None:
        out = torch.empty_like(q) if q.is_contiguous() else q.new_empty(shape)
    elif out.dtype is not kind or out.shape != shape or not out.is_contiguous():
        raise ValueError("out must have q's type and shape, contiguous")
    if q.get_device() != dev or lengths.get_device() != dev or \
            workspace.get_device() != dev or out.get_device() != dev:
        _on_device(dev, q, lengths, workspace, out)
    kq, kscale, kzero = k_cache
    vq, vscale, vzero = v_cache
    status = lib.wq_prefix_attention(
        q.data_ptr(), _DTYPES[kind], q0 if b > 1 else hq * d, b, hq, hkv, d, prefix_len, pcap,
        *pre, cap, kq.data_ptr(), kscale.data_ptr(), kzero.data_ptr(), vq.data_ptr(),
        vscale.data_ptr(), vzero.data_ptr(), lengths.data_ptr(), out.data_ptr(),
        workspace.data_ptr(), workspace.nbytes,
        _raw_stream(dev))
    if status:
        raise WqError(status, "wq_prefix_attention")
    return out


def attention_workspace(b, hq, hkv, length, d, n_components, device):
    size = ctypes.c_size_t(0)
    _check(lib.wq_msd_decode_attention_workspace(b, hq, hkv, length, d, n_components,
                                                 ctypes.byref(size)),
           "wq_msd_decode_attention_workspace")
    return torch.empty(max(int(size.value), 1), dtype=torch.uint8, device=device)


def wq_msd_decode_attention(q, k_cache, v_cache, n_components=2, workspace=None, out=None,
                            stream=None):
    """MSD decode attention: q bf16 [B, Hq, D]; k_cache and v_cache = (codes,
    scales, zeros) as kv_quantize_keys and kv_quantize_values return them.
    Returns out bf16 [B, Hq, D]."""
    if stream is not None:
        return _on(stream, wq_msd_decode_attention, q, k_cache, v_cache, n_components, workspace,
                   out)
    _cuda(q, torch.bfloat16, "q")
    b, hq, d = q.shape
    kq, ks, kz = k_cache
    vq, vs, vz = v_cache
    hkv, length = ks.shape[1], ks.shape[2]
    for t, dt, name in ((kq, torch.int32, "k_codes"), (ks, torch.float16, "k_scales"),
                        (kz, torch.float16, "k_zeros"), (vq, torch.int32, "v_codes"),
                        (vs, torch.float16, "v_scales"), (vz, torch.float16, "v_zeros")):
        _cuda(t, dt, name)
    if tuple(kq.shape) != (b, hkv, length, d // 8) or \
            tuple(vq.shape) != (b, hkv, (length + 7) // 8, d) or \
            tuple(vs.shape) != tuple(ks.shape) or tuple(kz.shape) != tuple(ks.shape) or \
            tuple(vz.shape) != tuple(ks.shape) or ks.shape[0] != b:
        raise ValueError("KV cache shapes do not match q")
    if workspace is None:
        workspace = attention_workspace(b, hq, hkv, length, d, n_components, q.device)
    if out is None:
        out = torch.empty(b, hq, d, dtype=torch.bfloat16, device=q.device)
    _check(lib.wq_msd_decode_attention(_ptr(q), b, hq, hkv, length, d, n_components, _ptr(kq),
                                       _ptr(ks), _ptr(kz), _ptr(vq), _ptr(vs), _ptr(vz), _ptr(out),
                                       _ptr(workspace), workspace.numel(), _stream()),
           "wq_msd_decode_attention")
    return out


def wq_test_set_attention_split(chunks_per_cta=0):
    """Fix the attention kernel's chunks per CTA (0: chosen per launch)."""
    _check(lib.wq_test_set_attention_split(chunks_per_cta), "wq_test_set_attention_split")


def wq_test_set_prefix_path(path=0):
    """Fix the kernel that takes the prefix (0: chosen per call, 1: mma.sync, 2: tcgen05)."""
    _check(lib.wq_test_set_prefix_path(path), "wq_test_set_prefix_path")
