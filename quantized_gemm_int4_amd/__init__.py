"""Python binding of the MI355X low-bit GEMM library (libhm.so).

Thin argument marshalling only: every function takes torch tensors (device
memory), passes their data pointers, sizes and the current HIP stream to the C
entry point of the same name, and raises HmError on a non-zero status.  All
work runs in the library's HIP kernels.  Importing this package fails loudly if
libhm.so has not been built (python quantized_gemm_int4_amd/build.py).

The C functions are declared and documented in include/hm.h.
"""
import contextlib
import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libhm.so")

HM_ABI_VERSION = 2
HM_W_INT4_SYM, HM_W_UINT4_ZP, HM_W_MXFP4, HM_W_MXINT4, HM_W_UINT3_ZP, HM_W_UINT2_ZP, HM_W_INT8_SYM = range(7)
HM_A_BF16, HM_A_FP8_ROWSCALE, HM_A_MXFP4 = 0, 1, 2
WFMT = {"int4_sym": HM_W_INT4_SYM, "uint4_zp": HM_W_UINT4_ZP, "mxfp4": HM_W_MXFP4, "mxint4": HM_W_MXINT4,
        "uint3_zp": HM_W_UINT3_ZP, "uint2_zp": HM_W_UINT2_ZP, "int8_sym": HM_W_INT8_SYM}
CODE_BITS = {HM_W_UINT3_ZP: 3, HM_W_UINT2_ZP: 2, HM_W_INT8_SYM: 8}     # other formats: 4
STATUS = {0: "HM_OK", 1: "HM_ERR_NULL", 2: "HM_ERR_SHAPE", 3: "HM_ERR_ALIGN",
          4: "HM_ERR_UNSUPPORTED", 5: "HM_ERR_WORKSPACE", 6: "HM_ERR_HIP", 7: "HM_ERR_ABI", 8: "HM_ERR_TUNING"}
HM_INT8_GEMM, HM_INT8_GATED, HM_INT8_GATED_GRAD, HM_INT8_GRAD = range(4)
HM_PATH_STREAM, HM_PATH_MID, HM_PATH_BIG, HM_PATH_TILE = 1, 2, 3, 4


class HmError(RuntimeError):
    def __init__(self, fn, code):
        self.code = code
        super().__init__(f"{fn} failed: {STATUS.get(code, code)} ({lib.hm_status_string(code).decode()})")


class hm_wdesc(ctypes.Structure):
    _fields_ = [("abi", ctypes.c_int32), ("wfmt", ctypes.c_int32), ("group", ctypes.c_int32),
                ("num_experts", ctypes.c_int32), ("n", ctypes.c_int64), ("k", ctypes.c_int64)]


class hm_tuning(ctypes.Structure):
    _fields_ = [("abi", ctypes.c_int32), ("path", ctypes.c_int32), ("stream_ks", ctypes.c_int32),
                ("stream_nbw", ctypes.c_int32), ("stream_splits", ctypes.c_int32), ("stream_waves", ctypes.c_int32),
                ("moe_stream_rows", ctypes.c_int32), ("moe_stream_max", ctypes.c_int32),
                ("moe_stream_nbw", ctypes.c_int32), ("moe_stream_ks", ctypes.c_int32),
                ("moe_stream_lds_kb", ctypes.c_int32), ("moe_big_min", ctypes.c_int32),
                ("moe_tile", ctypes.c_int32)]


class hm_lora_desc(ctypes.Structure):
    _fields_ = [("abi", ctypes.c_int32), ("rank", ctypes.c_int32), ("num_adapters", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("n", ctypes.c_int64), ("k", ctypes.c_int64)]


TUNING_FIELDS = tuple(f for f, _ in hm_tuning._fields_ if f != "abi")


def make_tuning(**fields):
    """Explicit choices of one call (hm_tuning); unnamed fields keep the default."""
    t = hm_tuning(HM_ABI_VERSION)
    for k, v in fields.items():
        if k not in TUNING_FIELDS:
            raise ValueError(f"unknown tuning field {k}")
        setattr(t, k, int(v))
    return t


def _tune(t):
    if t is None:
        return None
    if isinstance(t, dict):
        t = make_tuning(**t)
    return ctypes.byref(t)


def wdesc(wfmt, n, k, num_experts=1):
    """Layer description; wfmt is an HM_W_* value or 'int4_sym' / 'uint4_zp' / 'mxfp4'."""
    f = WFMT.get(wfmt, wfmt)
    return hm_wdesc(HM_ABI_VERSION, int(f), 32 if f in (HM_W_MXFP4, HM_W_MXINT4) else 128, int(num_experts),
                    int(n), int(k))


def lora_desc(n, k, rank, num_adapters):
    """Low-rank adapters beside an n x k layer (hm_lora_desc)."""
    return hm_lora_desc(HM_ABI_VERSION, int(rank), int(num_adapters), 0, int(n), int(k))


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python quantized_gemm_int4_amd/build.py` (needs hipcc)")
    L = ctypes.CDLL(LIB_PATH)
    P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    D = ctypes.POINTER(hm_wdesc)
    T = ctypes.POINTER(hm_tuning)
    LD = ctypes.POINTER(hm_lora_desc)
    sig = {
        "hm_transform_size": [D, ctypes.POINTER(SZ)],
        "hm_transform": [D, P, P, P, P, SZ, P],
        "hm_transform_gated": [D, P, P, P, P, SZ, P],
        "hm_dequant": [D, P, SZ, I32, P, P],
        "hm_quant_fp8_rows": [P, I64, I64, P, P, P],
        "hm_quant_mxfp4_rows": [P, I64, I64, P, P, P],
        "hm_gemm_workspace_size": [D, I32, I64, T, ctypes.POINTER(SZ)],
        "hm_gemm": [D, P, I32, P, P, I64, P, P, SZ, T, P],
        "hm_gemm_plan": [D, I32, I64, T, ctypes.c_char_p, SZ],
        "hm_moe_sort_workspace_size": [I64, I32, I32, ctypes.POINTER(SZ)],
        "hm_moe_sort": [P, I64, I32, I32, P, P, P, P, SZ, P],
        "hm_moe_gemm_workspace_size": [D, I32, I64, I32, T, ctypes.POINTER(SZ)],
        "hm_moe_gemm": [D, P, I32, P, P, I32, I64, I32, P, P, P, P, SZ, T, P],
        "hm_moe_gemm_gated": [D, P, I32, P, P, I32, I64, I32, P, P, P, P, SZ, T, P],
        "hm_moe_gemm_plan": [D, I32, I64, I32, I32, T, ctypes.c_char_p, SZ],
        "hm_moe_gemm_gated_plan": [D, I32, I64, I32, I32, T, ctypes.c_char_p, SZ],
        "hm_silu_mul": [P, I64, I64, P, P],
        "hm_silu_mul_fp8": [P, I64, I64, P, P, P],
        "hm_moe_combine": [P, P, I64, I32, I64, P, P],
        "hm_read_probe": [P, I64, I32, I32, P, P],
        "hm_moe_dispatch_workspace_size": [I64, I32, I32, ctypes.POINTER(SZ)],
        "hm_moe_dispatch": [P, P, I64, I32, I32, I64, P, P, P, P, P, P, SZ, P],
        "hm_moe_dispatch_grad": [P, P, I64, I32, I64, P, P],
        "hm_moe_collect": [P, P, P, I64, I32, I64, P, P],
        "hm_moe_collect_grad": [P, P, P, P, I64, I32, I64, P, P, P],
        "hm_lora_workspace_size": [LD, I64, ctypes.POINTER(SZ)],
        "hm_lora": [LD, P, P, P, P, P, I64, P, P, P, P, SZ, P],
        "hm_lora_grad_workspace_size": [LD, I64, ctypes.POINTER(SZ)],
        "hm_lora_grad": [LD, P, P, P, P, P, P, P, I64, P, P, P, P, P, SZ, P],
        "hm_quant_int8_rows": [P, I64, I64, P, P, P],
        "hm_gemm_int8_workspace_size": [I64, I64, I64, ctypes.POINTER(SZ)],
        "hm_gemm_int8": [P, P, P, P, I64, I64, I64, P, P, SZ, P],
        "hm_gemm_int8_gated_workspace_size": [I64, I64, I64, ctypes.POINTER(SZ)],
        "hm_gemm_int8_gated": [P, P, P, P, I64, I64, I64, P, P, SZ, P],
        "hm_gemm_int8_gated_grad_workspace_size": [I64, I64, I64, ctypes.POINTER(SZ)],
        "hm_gemm_int8_gated_grad": [P, P, P, P, P, I64, I64, I64, P, P, SZ, P],
        "hm_gemm_int8_grad_workspace_size": [I64, I64, I64, ctypes.POINTER(SZ)],
        "hm_gemm_int8_plan": [I32, I64, I64, I64, ctypes.c_char_p, SZ],
        "hm_gemm_int8_grad": [P, P, P, P, P, I64, I64, I64, P, P, P, SZ, P],
        "hm_moe_gemm_static": [D, P, I32, P, P, I32, I64, I32, P, P, P, T, P],
    }
    for name, args in sig.items():
        f = getattr(L, name)
        f.argtypes = args
        f.restype = ctypes.c_int
    L.hm_moe_gemm_static_max_workspace.argtypes = []
    L.hm_moe_gemm_static_max_workspace.restype = ctypes.c_size_t
    L.hm_status_string.argtypes = [ctypes.c_int]
    L.hm_status_string.restype = ctypes.c_char_p
    return L


lib = _load()


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    if stream is not None:
        return ctypes.c_void_p(stream.cuda_stream)
    # the handle alone: building torch's Stream object takes 2.7 us of a call's 3 us launch
    return ctypes.c_void_p(torch._C._cuda_getCurrentRawStream(torch.cuda.current_device()))


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)    # of a device index (torch without a GPU backend: none)


def _ok(fn, code):
    if code != 0:
        raise HmError(fn, code)


def _need(t, dtype, numel, name):
    if t is None:
        return
    if not t.is_cuda or not t.is_contiguous() or t.dtype != dtype or t.numel() < numel:
        raise ValueError(f"{name}: need a contiguous CUDA {dtype} tensor with >= {numel} elements")


# --------------------------------------------------------------------- weights

def hm_transform_size(desc):
    out = ctypes.c_size_t()
    _ok("hm_transform_size", lib.hm_transform_size(ctypes.byref(desc), ctypes.byref(out)))
    return out.value


def hm_transform(desc, codes, scales, zeros=None, w_dev=None, stream=None, gated=False):
    """codes uint8 [E,N,K/2]; scales int16/uint16 bits [E,N,K/128] (INT4) or uint8
    [E,N,K/32] (MXFP4); zeros uint8 [E,N,K/128] (UINT4_ZP).  Returns w_dev (uint8).
    gated: a gate_up weight (gate rows, then up rows) into the gated layout
    of hm_moe_gemm_gated (hm_transform_gated)."""
    nbytes = hm_transform_size(desc)
    if w_dev is None:
        w_dev = torch.empty(nbytes, dtype=torch.uint8, device=codes.device)
    E, n, k = desc.num_experts, desc.n, desc.k
    _need(codes, torch.uint8, E * n * k * CODE_BITS.get(desc.wfmt, 4) // 8, "codes")
    _need(w_dev, torch.uint8, nbytes, "w_dev")
    fn = "hm_transform_gated" if gated else "hm_transform"
    _ok(fn, getattr(lib, fn)(ctypes.byref(desc), _ptr(codes), _ptr(scales), _ptr(zeros),
                             _ptr(w_dev), w_dev.numel(), _stream(stream)))
    return w_dev


def hm_dequant(desc, w_dev, expert=0, out=None, stream=None):
    if out is None:
        out = torch.empty(desc.n, desc.k, dtype=torch.float32, device=w_dev.device)
    _need(out, torch.float32, desc.n * desc.k, "out")
    _ok("hm_dequant", lib.hm_dequant(ctypes.byref(desc), _ptr(w_dev), w_dev.numel(), int(expert),
                                     _ptr(out), _stream(stream)))
    return out


# ------------------------------------------------------------------ activations

def hm_quant_fp8_rows(x, x8=None, row_scale=None, stream=None):
    """x bf16 [m,k] -> (E4M3 bytes uint8 [m,k], fp32 row scales [m])."""
    m, k = x.shape
    _need(x, torch.bfloat16, m * k, "x")
    if x8 is None:
        x8 = torch.empty(m, k, dtype=torch.uint8, device=x.device)
    if row_scale is None:
        row_scale = torch.empty(m, dtype=torch.float32, device=x.device)
    _ok("hm_quant_fp8_rows", lib.hm_quant_fp8_rows(_ptr(x), m, k, _ptr(x8), _ptr(row_scale),
                                                   _stream(stream)))
    return x8, row_scale


def hm_quant_mxfp4_rows(x, codes=None, scales=None, stream=None):
    """x bf16 [m,k] -> (E2M1 codes uint8 [m,k/2], E8M0 scales uint8 [m,k/32])."""
    m, k = x.shape
    _need(x, torch.bfloat16, m * k, "x")
    if codes is None:
        codes = torch.empty(m, k // 2, dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty(m, k // 32, dtype=torch.uint8, device=x.device)
    _ok("hm_quant_mxfp4_rows", lib.hm_quant_mxfp4_rows(_ptr(x), m, k, _ptr(codes), _ptr(scales),
                                                       _stream(stream)))
    return codes, scales


# -------------------------------------------------------------------- dense GEMM

def _afmt(x, x_scales=None):
    """Activation format from the tensors: bf16 rows, E4M3 bytes with fp32
    row scales, or E2M1 codes with E8M0 scale bytes (uint8 x_scales)."""
    if x.dtype != torch.uint8:
        return HM_A_BF16
    return HM_A_MXFP4 if x_scales is not None and x_scales.dtype == torch.uint8 else HM_A_FP8_ROWSCALE


def hm_gemm_workspace_size(desc, afmt, m, tuning=None):
    out = ctypes.c_size_t()
    _ok("hm_gemm_workspace_size", lib.hm_gemm_workspace_size(ctypes.byref(desc), int(afmt), int(m),
                                                             _tune(tuning), ctypes.byref(out)))
    return out.value


def hm_gemm_plan(desc, afmt, m, tuning=None):
    buf = ctypes.create_string_buffer(256)
    _ok("hm_gemm_plan", lib.hm_gemm_plan(ctypes.byref(desc), int(afmt), int(m), _tune(tuning), buf, 256))
    return buf.value.decode()


def hm_gemm(desc, w_dev, x, x_scales=None, y=None, ws=None, afmt=None, tuning=None, stream=None):
    """y[m,n] = x_hat . w_hat^T in bf16.  x: bf16 [m,k] (W4A16, any weight
    format) or uint8 E4M3 [m,k] with fp32 x_scales [m] (W4A8-MXFP4).
    tuning: None (default choice), an hm_tuning, or a dict of its fields."""
    afmt = _afmt(x, x_scales) if afmt is None else afmt
    m = x.shape[0]
    if y is None:
        y = torch.empty(m, desc.n, dtype=torch.bfloat16, device=x.device)
    _need(y, torch.bfloat16, m * desc.n, "y")
    if isinstance(tuning, dict):
        tuning = make_tuning(**tuning)
    if ws is None:
        # a caller-provided workspace is passed through as is (the library checks its size)
        need = hm_gemm_workspace_size(desc, afmt, m, tuning)
        if need:
            ws = torch.empty(need, dtype=torch.uint8, device=x.device)
    _ok("hm_gemm", lib.hm_gemm(ctypes.byref(desc), _ptr(w_dev), int(afmt), _ptr(x), _ptr(x_scales),
                               m, _ptr(y), _ptr(ws), ws.numel() if ws is not None else 0,
                               _tune(tuning), _stream(stream)))
    return y


# -------------------------------------------------------------------------- MoE

def hm_moe_sort_workspace_size(t, topk, num_experts):
    out = ctypes.c_size_t()
    _ok("hm_moe_sort_workspace_size", lib.hm_moe_sort_workspace_size(int(t), int(topk),
                                                                     int(num_experts), ctypes.byref(out)))
    return out.value


def hm_moe_sort(topk_ids, num_experts, counts=None, offsets=None, sorted_pairs=None, ws=None, stream=None):
    """topk_ids int32 [t, topk] -> (counts [E], offsets [E+1], sorted_pairs [t*topk]).
    ws: a uint8 buffer of hm_moe_sort_workspace_size bytes (allocated here
    when None and needed)."""
    t, topk = topk_ids.shape
    dev = topk_ids.device
    _need(topk_ids, torch.int32, t * topk, "topk_ids")
    counts = torch.empty(num_experts, dtype=torch.int32, device=dev) if counts is None else counts
    offsets = torch.empty(num_experts + 1, dtype=torch.int32, device=dev) if offsets is None else offsets
    sorted_pairs = (torch.empty(t * topk, dtype=torch.int32, device=dev)
                    if sorted_pairs is None else sorted_pairs)
    need = hm_moe_sort_workspace_size(t, topk, num_experts)
    if ws is None and need:
        ws = torch.empty(need, dtype=torch.uint8, device=dev)
    wsp, wsb = (None, 0) if ws is None else (_ptr(ws), ws.numel() * ws.element_size())
    _ok("hm_moe_sort", lib.hm_moe_sort(_ptr(topk_ids), t, topk, int(num_experts), _ptr(counts),
                                       _ptr(offsets), _ptr(sorted_pairs), wsp, wsb, _stream(stream)))
    return counts, offsets, sorted_pairs


def hm_moe_gemm_workspace_size(desc, afmt, t, topk, tuning=None):
    out = ctypes.c_size_t()
    _ok("hm_moe_gemm_workspace_size", lib.hm_moe_gemm_workspace_size(ctypes.byref(desc), int(afmt), int(t),
                                                                     int(topk), _tune(tuning), ctypes.byref(out)))
    return out.value


def hm_moe_gemm_plan(desc, afmt, t, topk, a_rows_are_pairs, tuning=None, gated=False):
    buf = ctypes.create_string_buffer(512)
    fn = "hm_moe_gemm_gated_plan" if gated else "hm_moe_gemm_plan"
    _ok(fn, getattr(lib, fn)(ctypes.byref(desc), int(afmt), int(t), int(topk),
                             int(a_rows_are_pairs), _tune(tuning), buf, 512))
    return buf.value.decode()


def hm_moe_gemm(desc, w_dev, a, offsets, sorted_pairs, t, topk, a_rows_are_pairs, a_scales=None,
                y=None, ws=None, afmt=None, tuning=None, stream=None, gated=False):
    """Grouped GEMM; returns y bf16 [t*topk, n] in pair order.  a: bf16 rows,
    or E4M3 bytes with fp32 a_scales (MXFP4 weights only).  tuning: None, an
    hm_tuning, or a dict of its fields.  gated: hm_moe_gemm_gated on weights
    from hm_transform(..., gated=True); returns h bf16 [t*topk, n/2]."""
    afmt = _afmt(a, a_scales) if afmt is None else afmt
    P = t * topk
    ncols = desc.n // 2 if gated else desc.n
    if y is None:
        y = torch.empty(P, ncols, dtype=torch.bfloat16, device=a.device)
    _need(y, torch.bfloat16, P * ncols, "y")
    if isinstance(tuning, dict):
        tuning = make_tuning(**tuning)
    if ws is None:
        need = hm_moe_gemm_workspace_size(desc, afmt, t, topk, tuning)
        ws = torch.empty(max(need, 256), dtype=torch.uint8, device=a.device)
    fn = "hm_moe_gemm_gated" if gated else "hm_moe_gemm"
    _ok(fn, getattr(lib, fn)(ctypes.byref(desc), _ptr(w_dev), int(afmt), _ptr(a),
                             _ptr(a_scales), int(a_rows_are_pairs), int(t), int(topk),
                             _ptr(offsets), _ptr(sorted_pairs), _ptr(y), _ptr(ws),
                             ws.numel(), _tune(tuning), _stream(stream)))
    return y


def hm_moe_gemm_static(desc, w_dev, a, offsets, sorted_pairs, t, topk, a_rows_are_pairs, a_scales=None,
                       y=None, afmt=None, tuning=None, stream=None):
    """hm_moe_gemm with the library's static work-list array instead of a
    workspace (no device allocation in the call; calls on one GPU must not
    overlap).  y may be passed in so that nothing is allocated here either."""
    afmt = _afmt(a, a_scales) if afmt is None else afmt
    P = t * topk
    if y is None:
        y = torch.empty(P, desc.n, dtype=torch.bfloat16, device=a.device)
    _need(y, torch.bfloat16, P * desc.n, "y")
    _ok("hm_moe_gemm_static", lib.hm_moe_gemm_static(ctypes.byref(desc), _ptr(w_dev), int(afmt), _ptr(a),
                                                     _ptr(a_scales), int(a_rows_are_pairs), int(t), int(topk),
                                                     _ptr(offsets), _ptr(sorted_pairs), _ptr(y), _tune(tuning),
                                                     _stream(stream)))
    return y


def hm_moe_gemm_static_max_workspace():
    return lib.hm_moe_gemm_static_max_workspace()


# --------------------------------------------------------------- MoE block steps

def hm_silu_mul(gu, h=None, stream=None):
    """gu bf16 [rows, 2d] (gate | up) -> h bf16 [rows, d] = silu(gate) * up."""
    rows, two_d = gu.shape
    if two_d % 2:
        raise ValueError("gu: the last dimension must be even (gate | up)")
    d = two_d // 2
    _need(gu, torch.bfloat16, rows * two_d, "gu")
    if h is None:
        h = torch.empty(rows, d, dtype=torch.bfloat16, device=gu.device)
    _need(h, torch.bfloat16, rows * d, "h")
    _ok("hm_silu_mul", lib.hm_silu_mul(_ptr(gu), rows, d, _ptr(h), _stream(stream)))
    return h


def hm_silu_mul_fp8(gu, h8=None, h_scales=None, stream=None):
    """gu bf16 [rows, 2d] -> (E4M3 bytes [rows, d], fp32 row scales [rows]) of
    silu(gate) * up, in one pass."""
    rows, two_d = gu.shape
    d = two_d // 2
    _need(gu, torch.bfloat16, rows * two_d, "gu")
    if h8 is None:
        h8 = torch.empty(rows, d, dtype=torch.uint8, device=gu.device)
    if h_scales is None:
        h_scales = torch.empty(rows, dtype=torch.float32, device=gu.device)
    _ok("hm_silu_mul_fp8", lib.hm_silu_mul_fp8(_ptr(gu), rows, d, _ptr(h8), _ptr(h_scales), _stream(stream)))
    return h8, h_scales


def hm_moe_combine(y, weights, topk, out=None, stream=None):
    """y bf16 [t*topk, n] (pair order), weights fp32 [t, topk] -> out bf16 [t, n]."""
    t = weights.shape[0]
    n = y.shape[1]
    _need(y, torch.bfloat16, t * topk * n, "y")
    _need(weights, torch.float32, t * topk, "weights")
    if out is None:
        out = torch.empty(t, n, dtype=torch.bfloat16, device=y.device)
    _need(out, torch.bfloat16, t * n, "out")
    _ok("hm_moe_combine", lib.hm_moe_combine(_ptr(y), _ptr(weights), t, int(topk), n, _ptr(out),
                                             _stream(stream)))
    return out


# ------------------------------------------------------ MoE rows in expert order
#
# The calls below run on the device of their first tensor and on `stream` (the
# current stream of that device when None); buffers they allocate belong to
# that stream.  Every tensor must be contiguous, of the named shape, and on that device.

@contextlib.contextmanager
def _other(dev, stream):
    with torch.cuda.device(dev), torch.cuda.stream(stream):
        yield


def _elsewhere(t, stream):
    """None where t's device is the current one and `stream` None; else a
    context that makes t's device and `stream` the current ones."""
    if not t.is_cuda:
        raise ValueError("need CUDA tensors")
    if stream is None:
        return None if t.get_device() == torch._C._cuda_getDevice() else _other(t.device, None)
    if stream.device != t.device:
        raise ValueError("stream: of another device than the tensors")
    return _other(t.device, stream)


def _arg(t, dtype, shape, name, dev):
    """The address of a checked tensor on the device of index dev."""
    if t.get_device() != dev or t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name}: need a contiguous {dtype} tensor of shape {shape} on cuda:{dev}")
    return t.data_ptr()


def _dims(t, name):
    if t.dim() != 2:
        raise ValueError(f"{name}: need a 2-dimensional tensor")
    return t.shape


def _new(dtype, shape, dev):
    return torch.empty(shape, dtype=dtype, device=torch.device("cuda", dev))


def _ws(ws, size, args, dev):
    """(pointer, bytes) of a workspace: the caller's as it is (the library
    checks its size), or one of size(*args) bytes allocated here when that is
    not 0.  Also the tensor, which must live until the launch."""
    if ws is None:
        need = size(*args)
        if need == 0:
            return None, 0, None
        ws = _new(torch.uint8, (need,), dev)
    elif ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError(f"ws: need a contiguous tensor on cuda:{dev}")
    return ws.data_ptr(), ws.numel() * ws.element_size(), ws


def hm_moe_dispatch_workspace_size(t, topk, num_experts):
    out = ctypes.c_size_t()
    _ok("hm_moe_dispatch_workspace_size",
        lib.hm_moe_dispatch_workspace_size(int(t), int(topk), int(num_experts), ctypes.byref(out)))
    return out.value


def hm_moe_dispatch(x, topk_ids, num_experts, xs=None, counts=None, offsets=None, sorted_pairs=None, positions=None,
                    ws=None, stream=None):
    """Token rows in expert order: x bf16 [t, n], topk_ids int32 [t, topk] ->
    (xs bf16 [t*topk, n], counts [E], offsets [E+1], sorted_pairs [t*topk],
    positions [t, topk]).  Rows of xs and entries of sorted_pairs from
    offsets[E] on (as many as ids lie outside [0, E)) are left as they were:
    uninitialised when allocated here.  No tokens: counts and offsets are 0
    (the C entry point, a no-op then, leaves them)."""
    ctx = _elsewhere(x, stream)
    if ctx is not None:
        with ctx:
            return hm_moe_dispatch(x, topk_ids, num_experts, xs, counts, offsets, sorted_pairs, positions, ws)
    (t, n), (_, topk), dev = _dims(x, "x"), _dims(topk_ids, "topk_ids"), x.get_device()
    bf, i32 = torch.bfloat16, torch.int32
    E = int(num_experts)
    xs = _new(bf, (t * topk, n), dev) if xs is None else xs
    counts = _new(i32, (E,), dev) if counts is None else counts
    offsets = _new(i32, (E + 1,), dev) if offsets is None else offsets
    sorted_pairs = _new(i32, (t * topk,), dev) if sorted_pairs is None else sorted_pairs
    positions = _new(i32, (t, topk), dev) if positions is None else positions
    wsp, wsb, ws = _ws(ws, hm_moe_dispatch_workspace_size, (t, topk, E), dev)
    code = lib.hm_moe_dispatch(_arg(x, bf, (t, n), "x", dev), _arg(topk_ids, i32, (t, topk), "topk_ids", dev), t, topk,
                               E, n, _arg(xs, bf, (t * topk, n), "xs", dev), _arg(counts, i32, (E,), "counts", dev),
                               _arg(offsets, i32, (E + 1,), "offsets", dev),
                               _arg(sorted_pairs, i32, (t * topk,), "sorted_pairs", dev),
                               _arg(positions, i32, (t, topk), "positions", dev), wsp, wsb, _stream())
    _ok("hm_moe_dispatch", code)
    if t == 0:
        counts.zero_()
        offsets.zero_()
    return xs, counts, offsets, sorted_pairs, positions


def hm_moe_dispatch_grad(dxs, positions, dx=None, stream=None):
    """dxs bf16 [t*topk, n], positions int32 [t, topk] -> dx bf16 [t, n]: each
    token's sum over its routed rows."""
    ctx = _elsewhere(dxs, stream)
    if ctx is not None:
        with ctx:
            return hm_moe_dispatch_grad(dxs, positions, dx)
    (t, topk), (_, n), dev, bf = _dims(positions, "positions"), _dims(dxs, "dxs"), dxs.get_device(), torch.bfloat16
    dx = _new(bf, (t, n), dev) if dx is None else dx
    code = lib.hm_moe_dispatch_grad(_arg(dxs, bf, (t * topk, n), "dxs", dev),
                                    _arg(positions, torch.int32, (t, topk), "positions", dev), t, topk, n,
                                    _arg(dx, bf, (t, n), "dx", dev), _stream())
    _ok("hm_moe_dispatch_grad", code)
    return dx


def hm_moe_collect(ys, weights, positions, out=None, stream=None):
    """ys bf16 [t*topk, n] in expert order, weights fp32 [t, topk], positions
    int32 [t, topk] -> out bf16 [t, n]: each token's weighted sum."""
    ctx = _elsewhere(ys, stream)
    if ctx is not None:
        with ctx:
            return hm_moe_collect(ys, weights, positions, out)
    (t, topk), (_, n), dev, bf = _dims(positions, "positions"), _dims(ys, "ys"), ys.get_device(), torch.bfloat16
    out = _new(bf, (t, n), dev) if out is None else out
    code = lib.hm_moe_collect(_arg(ys, bf, (t * topk, n), "ys", dev),
                              _arg(weights, torch.float32, (t, topk), "weights", dev),
                              _arg(positions, torch.int32, (t, topk), "positions", dev), t, topk, n,
                              _arg(out, bf, (t, n), "out", dev), _stream())
    _ok("hm_moe_collect", code)
    return out


def hm_moe_collect_grad(dout, ys, weights, positions, dys=None, dweights=None, stream=None):
    """Gradient of hm_moe_collect: dout bf16 [t, n] -> (dys bf16 [t*topk, n],
    dweights fp32 [t, topk]).  Rows of dys that no position names are left as
    they were (zeros when allocated here).  dys may be ys.  With positions 0, 1,
    2, ... it is the gradient of hm_moe_combine."""
    ctx = _elsewhere(dout, stream)
    if ctx is not None:
        with ctx:
            return hm_moe_collect_grad(dout, ys, weights, positions, dys, dweights)
    (t, topk), (_, n), dev = _dims(positions, "positions"), _dims(dout, "dout"), dout.get_device()
    bf, f32 = torch.bfloat16, torch.float32
    if dys is None:
        dys = torch.zeros(t * topk, n, dtype=bf, device=dout.device)
    dweights = _new(f32, (t, topk), dev) if dweights is None else dweights
    code = lib.hm_moe_collect_grad(_arg(dout, bf, (t, n), "dout", dev), _arg(ys, bf, (t * topk, n), "ys", dev),
                                   _arg(weights, f32, (t, topk), "weights", dev),
                                   _arg(positions, torch.int32, (t, topk), "positions", dev), t, topk, n,
                                   _arg(dys, bf, (t * topk, n), "dys", dev),
                                   _arg(dweights, f32, (t, topk), "dweights", dev), _stream())
    _ok("hm_moe_collect_grad", code)
    return dys, dweights


# ------------------------------------------------------------ low-rank adapters

def _lora_ws_size(fn, desc, m):
    out = ctypes.c_size_t()
    _ok(fn, getattr(lib, fn)(ctypes.byref(desc), int(m), ctypes.byref(out)))
    return out.value


def hm_lora_workspace_size(desc, m):
    return _lora_ws_size("hm_lora_workspace_size", desc, m)


def hm_lora_grad_workspace_size(desc, m):
    return _lora_ws_size("hm_lora_grad_workspace_size", desc, m)


def hm_lora(desc, x, adapter_ids, a, b, scales, base=None, y=None, h=None, ws=None, stream=None):
    """Adapters beside a shared projection: x bf16 [m, k], adapter_ids int32
    [m], a bf16 [L, rank, k], b bf16 [L, n, rank], scales fp32 [L] -> y bf16
    [m, n] = base + scale * B (A x) per row; base bf16 [m, n] (hm_gemm's
    output) or None for zeros, and may be y (in place).  h: an fp32 [m, rank]
    tensor to keep scale * A x in for hm_lora_grad."""
    ctx = _elsewhere(x, stream)
    if ctx is not None:
        with ctx:
            return hm_lora(desc, x, adapter_ids, a, b, scales, base, y, h, ws)
    (m, _), dev, bf, f32 = _dims(x, "x"), x.get_device(), torch.bfloat16, torch.float32
    n, k, rank, L = desc.n, desc.k, desc.rank, desc.num_adapters
    y = _new(bf, (m, n), dev) if y is None else y
    wsp, wsb, ws = _ws(ws, hm_lora_workspace_size, (desc, m), dev)
    code = lib.hm_lora(ctypes.byref(desc), _arg(x, bf, (m, k), "x", dev),
                       _arg(adapter_ids, torch.int32, (m,), "adapter_ids", dev), _arg(a, bf, (L, rank, k), "a", dev),
                       _arg(b, bf, (L, n, rank), "b", dev), _arg(scales, f32, (L,), "scales", dev), m,
                       None if base is None else _arg(base, bf, (m, n), "base", dev), _arg(y, bf, (m, n), "y", dev),
                       None if h is None else _arg(h, f32, (m, rank), "h", dev), wsp, wsb, _stream())
    _ok("hm_lora", code)
    return y


def hm_lora_grad(desc, dy, x, h, adapter_ids, a, b, scales, dx_base=None, dx=None, da=None, db=None, need_dx=True,
                 ws=None, stream=None):
    """Gradient of hm_lora: dy bf16 [m, n], x bf16 [m, k], h fp32 [m, rank] ->
    (dx bf16 [m, k] or None, da bf16 [L, rank, k], db bf16 [L, n, rank]).
    dx_base bf16 [m, k]: the gradient through the shared projection, added to
    dx (may be dx); need_dx=False leaves dx out."""
    ctx = _elsewhere(x, stream)
    if ctx is not None:
        with ctx:
            return hm_lora_grad(desc, dy, x, h, adapter_ids, a, b, scales, dx_base, dx, da, db, need_dx, ws)
    if not need_dx and (dx is not None or dx_base is not None):
        raise ValueError("need_dx=False takes neither dx nor dx_base")
    (m, _), dev, bf, f32 = _dims(x, "x"), x.get_device(), torch.bfloat16, torch.float32
    n, k, rank, L = desc.n, desc.k, desc.rank, desc.num_adapters
    if need_dx and dx is None:
        dx = _new(bf, (m, k), dev)
    da = _new(bf, (L, rank, k), dev) if da is None else da
    db = _new(bf, (L, n, rank), dev) if db is None else db
    wsp, wsb, ws = _ws(ws, hm_lora_grad_workspace_size, (desc, m), dev)
    code = lib.hm_lora_grad(ctypes.byref(desc), _arg(dy, bf, (m, n), "dy", dev), _arg(x, bf, (m, k), "x", dev),
                            _arg(h, f32, (m, rank), "h", dev), _arg(adapter_ids, torch.int32, (m,), "adapter_ids", dev),
                            _arg(a, bf, (L, rank, k), "a", dev), _arg(b, bf, (L, n, rank), "b", dev),
                            _arg(scales, f32, (L,), "scales", dev), m,
                            None if dx_base is None else _arg(dx_base, bf, (m, k), "dx_base", dev),
                            None if dx is None else _arg(dx, bf, (m, k), "dx", dev),
                            _arg(da, bf, (L, rank, k), "da", dev), _arg(db, bf, (L, n, rank), "db", dev), wsp, wsb,
                            _stream())
    _ok("hm_lora_grad", code)
    return dx, da, db


# -------------------------------------------------------- 8-bit integer layers

def hm_quant_int8_rows(x, x8=None, row_scale=None, stream=None):
    """x bf16 [m, k] -> (int8 codes [m, k], fp32 row scales [m]): activations of
    the calls below, and their weights (bf16 rows of W)."""
    ctx = _elsewhere(x, stream)
    if ctx is not None:
        with ctx:
            return hm_quant_int8_rows(x, x8, row_scale)
    (m, k), dev = _dims(x, "x"), x.get_device()
    x8 = _new(torch.int8, (m, k), dev) if x8 is None else x8
    row_scale = _new(torch.float32, (m,), dev) if row_scale is None else row_scale
    code = lib.hm_quant_int8_rows(_arg(x, torch.bfloat16, (m, k), "x", dev), m, k, _arg(x8, torch.int8, (m, k), "x8", dev),
                                  _arg(row_scale, torch.float32, (m,), "row_scale", dev), _raw_stream(dev))
    _ok("hm_quant_int8_rows", code)
    return x8, row_scale


def _int8_ws_size(fn, m, n, k):
    out = ctypes.c_size_t()
    _ok(fn, getattr(lib, fn)(int(m), int(n), int(k), ctypes.byref(out)))
    return out.value


def hm_gemm_int8_workspace_size(m, n, k):
    return _int8_ws_size("hm_gemm_int8_workspace_size", m, n, k)


def hm_gemm_int8_gated_workspace_size(m, n, k):
    return _int8_ws_size("hm_gemm_int8_gated_workspace_size", m, n, k)


def hm_gemm_int8_gated_grad_workspace_size(m, n, k):
    return _int8_ws_size("hm_gemm_int8_gated_grad_workspace_size", m, n, k)


def hm_gemm_int8_grad_workspace_size(m, n, k):
    return _int8_ws_size("hm_gemm_int8_grad_workspace_size", m, n, k)


def hm_gemm_int8_plan(op, m, n, k):
    """What the call (an HM_INT8_* value) runs for these sizes, as a text."""
    buf = ctypes.create_string_buffer(256)
    _ok("hm_gemm_int8_plan", lib.hm_gemm_int8_plan(int(op), int(m), int(n), int(k), buf, 256))
    return buf.value.decode()


def _int8_args(x8, x_scales, w8, w_scales, m, n, k, dev):
    return (_arg(x8, torch.int8, (m, k), "x8", dev), _arg(x_scales, torch.float32, (m,), "x_scales", dev),
            _arg(w8, torch.int8, (n, k), "w8", dev), _arg(w_scales, torch.float32, (n,), "w_scales", dev))


def hm_gemm_int8(x8, x_scales, w8, w_scales, y=None, ws=None, stream=None):
    """x8 int8 [m, k] with fp32 x_scales [m], w8 int8 [n, k] with fp32 w_scales
    [n] -> y bf16 [m, n], the product of the values the codes stand for."""
    ctx = _elsewhere(x8, stream)
    if ctx is not None:
        with ctx:
            return hm_gemm_int8(x8, x_scales, w8, w_scales, y, ws)
    (m, k), (n, _), dev = _dims(x8, "x8"), _dims(w8, "w8"), x8.get_device()
    y = _new(torch.bfloat16, (m, n), dev) if y is None else y
    wsp, wsb, ws = _ws(ws, hm_gemm_int8_workspace_size, (m, n, k), dev)
    code = lib.hm_gemm_int8(*_int8_args(x8, x_scales, w8, w_scales, m, n, k, dev), m, n, k,
                            _arg(y, torch.bfloat16, (m, n), "y", dev), wsp, wsb, _raw_stream(dev))
    _ok("hm_gemm_int8", code)
    return y


def hm_gemm_int8_gated(x8, x_scales, w8, w_scales, h=None, ws=None, stream=None):
    """hm_gemm_int8 of a gate_up weight (w8 int8 [2d, k], gate rows, then up
    rows) with the gated activation: h bf16 [m, d] = silu(gate) * up."""
    ctx = _elsewhere(x8, stream)
    if ctx is not None:
        with ctx:
            return hm_gemm_int8_gated(x8, x_scales, w8, w_scales, h, ws)
    (m, k), (n, _), dev = _dims(x8, "x8"), _dims(w8, "w8"), x8.get_device()
    h = _new(torch.bfloat16, (m, n // 2), dev) if h is None else h
    wsp, wsb, ws = _ws(ws, hm_gemm_int8_gated_workspace_size, (m, n, k), dev)
    code = lib.hm_gemm_int8_gated(*_int8_args(x8, x_scales, w8, w_scales, m, n, k, dev), m, n, k,
                                  _arg(h, torch.bfloat16, (m, n // 2), "h", dev), wsp, wsb, _raw_stream(dev))
    _ok("hm_gemm_int8_gated", code)
    return h


def hm_gemm_int8_gated_grad(dh, x8, x_scales, w8, w_scales, dgu=None, ws=None, stream=None):
    """Gradient of hm_gemm_int8_gated to its gate and up products, which are
    computed again from the 8-bit rows: dh bf16 [m, d] -> dgu bf16 [m, 2d]."""
    ctx = _elsewhere(x8, stream)
    if ctx is not None:
        with ctx:
            return hm_gemm_int8_gated_grad(dh, x8, x_scales, w8, w_scales, dgu, ws)
    (m, k), (n, _), dev = _dims(x8, "x8"), _dims(w8, "w8"), x8.get_device()
    dgu = _new(torch.bfloat16, (m, n), dev) if dgu is None else dgu
    wsp, wsb, ws = _ws(ws, hm_gemm_int8_gated_grad_workspace_size, (m, n, k), dev)
    code = lib.hm_gemm_int8_gated_grad(_arg(dh, torch.bfloat16, (m, n // 2), "dh", dev),
                                       *_int8_args(x8, x_scales, w8, w_scales, m, n, k, dev), m, n, k,
                                       _arg(dgu, torch.bfloat16, (m, n), "dgu", dev), wsp, wsb, _raw_stream(dev))
    _ok("hm_gemm_int8_gated_grad", code)
    return dgu


def hm_gemm_int8_grad(dy, x8, x_scales, w8, w_scales, dx=None, dw=None, need_dx=True, need_dw=True, ws=None, stream=None):
    """Gradient of hm_gemm_int8 to its rows and weights: dy bf16 [m, n] -> (dx
    bf16 [m, k] or None, dw bf16 [n, k] or None); need_dx=False, need_dw=False leave
    one out."""
    ctx = _elsewhere(x8, stream)
    if ctx is not None:
        with ctx:
            return hm_gemm_int8_grad(dy, x8, x_scales, w8, w_scales, dx, dw, need_dx, need_dw, ws)
    if (not need_dx and dx is not None) or (not need_dw and dw is not None):
        raise ValueError("need_dx=False takes no dx, need_dw=False no dw")
    (m, k), (n, _), dev, bf = _dims(x8, "x8"), _dims(w8, "w8"), x8.get_device(), torch.bfloat16
    dx = _new(bf, (m, k), dev) if need_dx and dx is None else dx
    dw = _new(bf, (n, k), dev) if need_dw and dw is None else dw
    wsp, wsb, ws = _ws(ws, hm_gemm_int8_grad_workspace_size, (m, n, k), dev)
    code = lib.hm_gemm_int8_grad(_arg(dy, bf, (m, n), "dy", dev), *_int8_args(x8, x_scales, w8, w_scales, m, n, k, dev), m, n, k,
                                 # (a dx of no rows has no address, but NULL would say that it is not wanted: any aligned one)
                                 None if dx is None else _arg(dx, bf, (m, k), "dx", dev) or 16,
                                 None if dw is None else _arg(dw, bf, (n, k), "dw", dev), wsp, wsb, _raw_stream(dev))
    _ok("hm_gemm_int8_grad", code)
    return dx, dw


# ----------------------------------------------------------------- measurement

def hm_read_probe(buf, blocks=2048, unroll=4, out=None, stream=None):
    """Plain-read reference over a device buffer (any dtype, byte size a
    multiple of 16); returns the per-block words."""
    nbytes = buf.numel() * buf.element_size()
    if out is None:
        out = torch.empty(blocks, dtype=torch.int32, device=buf.device)
    _ok("hm_read_probe", lib.hm_read_probe(_ptr(buf), nbytes, int(blocks), int(unroll), _ptr(out),
                                           _stream(stream)))
    return out
