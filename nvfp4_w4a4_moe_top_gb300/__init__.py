"""Python binding of libmoe_nvfp4.so: the native NVFP4 W4A4 MoE expert
forward on one GB300 (sm_103a).

Argument marshalling only: every function passes torch tensors as device
pointers, the current CUDA stream, and raises ``MoeError`` on a negative
return code.  Every step of the computation runs in the library's CUDA
kernels; there is no CPU path.  The library must have been built
(``nvfp4_w4a4_moe_top_gb300.build.build()``); importing a missing library
raises.

Tensor conventions (see include/moe_nvfp4.h): bf16 data may be passed as
torch.bfloat16 or 16-bit integer tensors; all tensors are contiguous, on the
current CUDA device, 16-byte aligned.
"""
from __future__ import annotations

import ctypes
import os
import re

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libmoe_nvfp4.so")
HEADER = os.path.join(os.path.dirname(_HERE), "include", "moe_nvfp4.h")
LEARNER_HEADER = os.path.join(os.path.dirname(_HERE), "include", "moe_learner.h")
TOKENS_HEADER = os.path.join(os.path.dirname(_HERE), "include", "moe_tokens.h")

MOE_OK, MOE_ERR_POINTER, MOE_ERR_SHAPE, MOE_ERR_WORKSPACE, MOE_ERR_CUDA, MOE_ERR_DEVICE = 0, -1, -2, -3, -4, -5
STATUS_NONFINITE_X, STATUS_NONFINITE_LOGITS, STATUS_NONFINITE_WEIGHT = 0x1, 0x2, 0x4
STATUS_BAD_ROUTING, STATUS_TIMEOUT, STATUS_BAD_TOKEN, STATUS_BAD_SAMPLING = 0x8, 0x10, 0x20, 0x40
LOGPROBS_MAX_TOP, DISTILL_MAX_K, DISTILL_MAX_V = 32, 256, 1 << 20
EMBED_MAX_V, EMBED_MAX_D, SAMPLE_MAX_V = 1 << 24, 16384, 1 << 20

WS_FIELDS = ["topk_ids", "topk_w", "token_slot_row", "counts", "offsets", "row_to_token",
             "amax_tok", "x_codes", "x_sf", "x_g", "h_codes", "h_sf", "h_g", "slots",
             "chunk_hist", "fc1_staging"]


class MoeError(RuntimeError):
    def __init__(self, fn, code):
        self.code = code
        super().__init__("%s failed: %d (%s)" % (fn, code, status_string(code)))


P, I32, I64, SZ, F32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
_SIGS = {
    "moe_abi_version": (I32, []),
    "moe_status_string": (ctypes.c_char_p, [I32]),
    "moe_m_cap": (I64, [I32, I32, I32]),
    "nvfp4_sf_bytes": (SZ, [I64, I32]),
    "moe_permute_workspace_bytes": (SZ, [I32, I32]),
    "nvfp4_fc1_workspace_bytes": (SZ, [I32]),
    "moe_expert_forward_workspace_bytes": (SZ, [I32, I32, I32, I32, I32]),
    "moe_expert_forward_workspace_layout": (I32, [I32, I32, I32, I32, I32, P]),
    "moe_nvfp4_quantize_weights": (I32, [P, I32, I32, I32, P, P, P, P, P]),
    "moe_nvfp4_quantize_weights_per_expert": (I32, [P, I32, I32, I32, P, P, P, P, P, P]),
    "moe_permute_amax": (I32, [P, P, P, P, I32, I32, I32, I32, P, P, P, P, P, P, P, P, P, SZ, P, P]),
    "moe_permute_amax_noalloc": (I32, [P, P, P, P, I32, I32, I32, I32, P, P, P, P, P, P, P, P, P, P]),
    "nvfp4_quantize_rows": (I32, [P, I32, I32, P, P, I32, P, P, P, P, P]),
    "nvfp4_grouped_gemm_fc1_swiglu": (I32, [P, P, P, P, I32, I64, I32, I32, P, P, P, P, P, P, P, P, P, SZ, P, P]),
    "nvfp4_grouped_gemm_fc2_unpermute": (I32, [P, P, P, P, I32, I64, I32, I32, P, P, P, P, P, P, I32, I32, P, P, P, P, P]),
    "moe_expert_forward": (I32, [P, P, I32, I32, I32, I32, I32, P, P, P, P, P, P, P, P, SZ, P, P]),
    "moe_pipeline_device_bytes": (SZ, [I32, I32, I32, I32, I32, I32]),
    "moe_pipeline_create": (I32, [I32, I32, I32, I32, I32, I32, P, SZ, P]),
    "moe_pipeline_submit": (I32, [P, P, P, P, P, P, P, P, P, P, P]),
    "moe_pipeline_synchronize": (I32, [P]),
    "moe_pipeline_destroy": (I32, [P]),
    "moe_expert_forward_timed": (I32, [P, P, I32, I32, I32, I32, I32, P, P, P, P, P, P, P, P, SZ, P, P, P]),
    "moe_expert_forward_gather": (I32, [P, P, I32, I32, I32, I32, I32, P, P, P, P, P, P, P, P, SZ, P, P]),
    "moe_expert_forward_train": (I32, [P, P, I32, I32, I32, I32, I32, P, P, P, P, P, P, P, P, SZ, P, P, P, P]),
    "moe_expert_backward_workspace_bytes": (SZ, [I32, I32, I32, I32, I32]),
    "moe_expert_backward": (I32, [P, P, I32, I32, I32, I32, I32] + [P] * 21 + [SZ, P, P]),
    "moe_mx8_sf_bytes": (SZ, [I64, I32]),
    "moe_add_rmsnorm": (I32, [P, I64, P, I64, P, F32, I32, I32, P, P, P, P, P, P, P]),
    "moe_add_rmsnorm_backward_workspace_bytes": (SZ, [I32, I32]),
    "moe_add_rmsnorm_backward": (I32, [P, P, P, P, P, I32, I32, P, P, P, SZ, P, P]),
    "moe_token_logprobs": (I32, [P, I32, I64, I32, I32, P, F32, I32] + [P] * 7),
    "moe_token_logprobs_backward": (I32, [P, I32, I64, I32, I32, P, F32, P, P, P, P, P, I64, P, P]),
    "moe_distill_topk": (I32, [P, I32, I64, I32, I32, P, P, P, I32, F32, P, P, P, P]),
    "moe_distill_topk_backward": (I32, [P, I32, I64, I32, I32, P, P, P, I32, F32, P, P, P, I64, P, P]),
    "moe_distill_topk_train": (I32, [P, I32, I64, I32, I32, P, P, P, I32, F32, P, P, P, I64, P, P]),
    "moe_embed_tokens": (I32, [P, P, I32, I64, I32, I32, I32, F32, P, I64, P, P]),
    "moe_embed_tokens_backward_workspace_bytes": (SZ, [I32, I32, I32]),
    "moe_embed_tokens_backward": (I32, [P, I64, P, I32, I32, I32, F32, I32, P, P, SZ, P, P]),
    "moe_sample_tokens": (I32, [P, I32, I64, I32, I32] + [P] * 10),
}

_lib = None


def lib():
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError("libmoe_nvfp4.so is not built: run nvfp4_w4a4_moe_top_gb300.build.build()")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(L, name)
            f.restype, f.argtypes = res, args
        _lib = L
    return _lib


def header_functions(header=HEADER):
    """Names of the functions a header declares (include/moe_nvfp4.h unless
    another is given)."""
    src = open(header).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    return sorted(set(re.findall(r"\b([a-z][a-z0-9_]*)\s*\(", src)) - {"defined"})


# --------------------------------------------------------------------------
def status_string(code):
    return lib().moe_status_string(int(code)).decode()


def abi_version():
    return lib().moe_abi_version()


def m_cap(T, E, k):
    return int(lib().moe_m_cap(T, E, k))


def sf_bytes(rows, K):
    return int(lib().nvfp4_sf_bytes(rows, K))


def permute_workspace_bytes(T, E):
    return int(lib().moe_permute_workspace_bytes(T, E))


def fc1_workspace_bytes(d_ff):
    return int(lib().nvfp4_fc1_workspace_bytes(d_ff))


def forward_workspace_bytes(T, E, k, d, d_ff):
    return int(lib().moe_expert_forward_workspace_bytes(T, E, k, d, d_ff))


def forward_workspace_layout(T, E, k, d, d_ff):
    arr = (ctypes.c_size_t * 16)()
    _check("moe_expert_forward_workspace_layout",
           lib().moe_expert_forward_workspace_layout(T, E, k, d, d_ff, ctypes.cast(arr, P)))
    return dict(zip(WS_FIELDS, list(arr)))


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _s(stream):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _check(fn, rc):
    if rc != MOE_OK:
        raise MoeError(fn, rc)


# --------------------------------------------------------------------------
# entry points (same names and argument order as the C functions)
# --------------------------------------------------------------------------
def moe_nvfp4_quantize_weights(W, codes, sf, g, status=None, stream=None):
    E, N, K = W.shape
    _check("moe_nvfp4_quantize_weights",
           lib().moe_nvfp4_quantize_weights(_p(W), E, N, K, _p(codes), _p(sf), _p(g), _p(status), _s(stream)))


def moe_nvfp4_quantize_weights_per_expert(W, codes, sf, g, amax_e, status=None, stream=None):
    E, N, K = W.shape
    _check("moe_nvfp4_quantize_weights_per_expert", lib().moe_nvfp4_quantize_weights_per_expert(
        _p(W), E, N, K, _p(codes), _p(sf), _p(g), _p(amax_e), _p(status), _s(stream)))


def moe_permute_amax(logits, ext_ids, ext_w, x, T, E, k, d, topk_ids, topk_w, counts, offsets,
                     row_to_token, token_slot_row, amax_tok, amax_row, ws, status=None, stream=None):
    _check("moe_permute_amax", lib().moe_permute_amax(
        _p(logits), _p(ext_ids), _p(ext_w), _p(x), T, E, k, d, _p(topk_ids), _p(topk_w), _p(counts),
        _p(offsets), _p(row_to_token), _p(token_slot_row), _p(amax_tok), _p(amax_row), _p(ws),
        0 if ws is None else ws.numel() * ws.element_size(), _p(status), _s(stream)))


def moe_permute_amax_noalloc(logits, ext_ids, ext_w, x, T, E, k, d, topk_ids, topk_w, counts, offsets,
                             row_to_token, token_slot_row, amax_tok, amax_row, status=None, stream=None):
    """moe_permute_amax with the library's own fixed scratch array instead of
    a workspace: for callers that cannot allocate device memory.  Calls that
    overlap on the GPU race on that array; see include/moe_nvfp4.h."""
    _check("moe_permute_amax_noalloc", lib().moe_permute_amax_noalloc(
        _p(logits), _p(ext_ids), _p(ext_w), _p(x), T, E, k, d, _p(topk_ids), _p(topk_w), _p(counts),
        _p(offsets), _p(row_to_token), _p(token_slot_row), _p(amax_tok), _p(amax_row), _p(status),
        _s(stream)))


def nvfp4_quantize_rows(src, K, row_map, amax, dst_rows, codes, sf, g, status=None, stream=None):
    src_rows = src.numel() // K
    _check("nvfp4_quantize_rows", lib().nvfp4_quantize_rows(
        _p(src), src_rows, K, _p(row_map), _p(amax), dst_rows, _p(codes), _p(sf), _p(g), _p(status),
        _s(stream)))


def nvfp4_grouped_gemm_fc1_swiglu(a_codes, a_sf, a_g, offsets, E, M_cap, d, d_ff, w1_codes, w1_sf, w1_g,
                                  h_codes, h_sf, h_g, dbg_u_f32, dbg_h, ws, status=None, stream=None):
    _check("nvfp4_grouped_gemm_fc1_swiglu", lib().nvfp4_grouped_gemm_fc1_swiglu(
        _p(a_codes), _p(a_sf), _p(a_g), _p(offsets), E, M_cap, d, d_ff, _p(w1_codes), _p(w1_sf), _p(w1_g),
        _p(h_codes), _p(h_sf), _p(h_g), _p(dbg_u_f32), _p(dbg_h), _p(ws),
        ws.numel() * ws.element_size(), _p(status), _s(stream)))


def nvfp4_grouped_gemm_fc2_unpermute(h_codes, h_sf, h_g, offsets, E, M_cap, d_ff, d, w2_codes, w2_sf, w2_g,
                                     row_to_token, token_slot_row, topk_w, T, k, slots, out, dbg_y_f32,
                                     status=None, stream=None):
    """slots: the z rows, bf16 [M_cap][d] (the kernel stores whole 128-row
    tiles there)."""
    if T > 0 and slots.numel() * slots.element_size() < M_cap * d * 2:
        raise ValueError("slots must hold M_cap x d bf16 values")
    _check("nvfp4_grouped_gemm_fc2_unpermute", lib().nvfp4_grouped_gemm_fc2_unpermute(
        _p(h_codes), _p(h_sf), _p(h_g), _p(offsets), E, M_cap, d_ff, d, _p(w2_codes), _p(w2_sf), _p(w2_g),
        _p(row_to_token), _p(token_slot_row), _p(topk_w), T, k, _p(slots), _p(out), _p(dbg_y_f32),
        _p(status), _s(stream)))


def moe_expert_forward(x, logits, T, E, k, d, d_ff, w1_codes, w1_sf, w1_g, w2_codes, w2_sf, w2_g, out, ws,
                       status=None, stream=None):
    _check("moe_expert_forward", lib().moe_expert_forward(
        _p(x), _p(logits), T, E, k, d, d_ff, _p(w1_codes), _p(w1_sf), _p(w1_g), _p(w2_codes), _p(w2_sf),
        _p(w2_g), _p(out), _p(ws), 0 if ws is None else ws.numel() * ws.element_size(), _p(status),
        _s(stream)))


def moe_expert_forward_timed(x, logits, T, E, k, d, d_ff, w1_codes, w1_sf, w1_g, w2_codes, w2_sf, w2_g, out, ws,
                             status=None, stream=None, events=None):
    """moe_expert_forward recording the eight torch.cuda.Event objects in
    `events` (timing enabled) around its seven launches on the stream."""
    import torch
    if events is None or len(events) != 8:
        raise ValueError("events: eight torch.cuda.Event objects")
    s = torch.cuda.current_stream() if stream is None else stream
    for e in events:  # the handle exists once the event has been recorded
        if e.cuda_event == 0:
            e.record(s)
    arr = (ctypes.c_void_p * 8)(*[e.cuda_event for e in events])
    _check("moe_expert_forward_timed", lib().moe_expert_forward_timed(
        _p(x), _p(logits), T, E, k, d, d_ff, _p(w1_codes), _p(w1_sf), _p(w1_g), _p(w2_codes), _p(w2_sf),
        _p(w2_g), _p(out), _p(ws), 0 if ws is None else ws.numel() * ws.element_size(), _p(status),
        _s(stream), ctypes.cast(arr, P)))


def moe_expert_forward_gather(x, logits, T, E, k, d, d_ff, w1_codes, w1_sf, w1_g, w2_codes, w2_sf, w2_g, out, ws,
                              status=None, stream=None):
    """moe_expert_forward with gather-on-load FC1 (codes quantised once per
    token, fetched by row_to_token with TMA tile::gather4)."""
    _check("moe_expert_forward_gather", lib().moe_expert_forward_gather(
        _p(x), _p(logits), T, E, k, d, d_ff, _p(w1_codes), _p(w1_sf), _p(w1_g), _p(w2_codes), _p(w2_sf),
        _p(w2_g), _p(out), _p(ws), 0 if ws is None else ws.numel() * ws.element_size(), _p(status),
        _s(stream)))


def moe_expert_forward_train(x, logits, T, E, k, d, d_ff, w1_codes, w1_sf, w1_g, w2_codes, w2_sf, w2_g, out, ws,
                             save_u, save_h, status=None, stream=None):
    _check("moe_expert_forward_train", lib().moe_expert_forward_train(
        _p(x), _p(logits), T, E, k, d, d_ff, _p(w1_codes), _p(w1_sf), _p(w1_g), _p(w2_codes), _p(w2_sf),
        _p(w2_g), _p(out), _p(ws), 0 if ws is None else ws.numel() * ws.element_size(), _p(save_u), _p(save_h),
        _p(status), _s(stream)))


def moe_expert_backward(dY, x, T, E, k, d, d_ff, W1, W2, w2_codes, w2_sf, w2_g, topk_ids, topk_w, offsets,
                        row_to_token, token_slot_row, u, h, h_codes, h_sf, h_g, dx, dW1, dW2, dlogits, dw, ws,
                        status=None, stream=None):
    _check("moe_expert_backward", lib().moe_expert_backward(
        _p(dY), _p(x), T, E, k, d, d_ff, _p(W1), _p(W2), _p(w2_codes), _p(w2_sf), _p(w2_g), _p(topk_ids),
        _p(topk_w), _p(offsets), _p(row_to_token), _p(token_slot_row), _p(u), _p(h), _p(h_codes), _p(h_sf),
        _p(h_g), _p(dx), _p(dW1), _p(dW2), _p(dlogits), _p(dw), _p(ws),
        0 if ws is None else ws.numel() * ws.element_size(), _p(status), _s(stream)))


def backward_workspace_bytes(T, E, k, d, d_ff):
    return int(lib().moe_expert_backward_workspace_bytes(T, E, k, d, d_ff))


# --------------------------------------------------------------------------
# learner operators (include/moe_learner.h): sizes and strides come from the
# tensors, whose types, sizes and devices are checked here
# --------------------------------------------------------------------------
def _place(t):
    """Where a tensor is, for a message."""
    dev = t.get_device()
    return "the host" if dev < 0 else "device %d" % dev


def _here(t, what):
    """Index of the current device, on which a call's first tensor has to be
    (and all others: the launch and its stream are that device's)."""
    dev = t.get_device()
    if dev < 0 or dev != _types.device():
        raise ValueError("%s: a tensor on the current CUDA device expected, got one on %s" % (what, _place(t)))
    return dev


def _ints(shape, what):
    """Refuses rows and columns beyond the library's int, which would be passed
    modulo 2^32."""
    if shape[0] > 0x7FFFFFFF or shape[1] > 0x7FFFFFFF:
        raise ValueError("%s: at most 2^31 - 1 rows and columns expected, got %s" % (what, tuple(shape)))


def _tensor(t, dtypes, shape, what, dev):
    """Pointer of a contiguous tensor on device `dev` of one of `dtypes` and of
    `shape` (None: an optional argument left out)."""
    if t is None:
        return None
    if t.dtype not in dtypes or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        raise ValueError("%s: a contiguous CUDA tensor %s of %s on device %d expected, got %s of %s on %s"
                         % (what, tuple(shape), " or ".join(map(str, dtypes)), dev, tuple(t.shape), t.dtype, _place(t)))
    return t.data_ptr()


def _rows(t, dtypes, shape, what, dev):
    """Pointer, row stride and shape of a 2-D tensor on device `dev` whose rows
    are contiguous."""
    own, st = t.shape, t.stride()
    if len(own) != 2 or (shape is not None and own != shape) or t.dtype not in dtypes or t.get_device() != dev or \
            (st[1] != 1 and own[1] > 1):
        raise ValueError("%s: a 2-D CUDA tensor%s of %s with contiguous rows on device %d expected, got %s of %s on "
                         "%s, strides %s" % (what, "" if shape is None else " %s" % (tuple(shape),),
                                             " or ".join(map(str, dtypes)), dev, tuple(own), t.dtype, _place(t), st))
    _ints(own, what)
    return t.data_ptr(), (st[0] if own[0] > 1 else own[1]), own


class _Types:
    """The element types of the learner operators' tensors, once torch is
    imported."""
    ready = False

    def load(self):
        import torch
        self.b16 = (torch.bfloat16, torch.int16, torch.uint16)
        self.f32 = (torch.float32,)
        self.i32 = (torch.int32,)
        self.status = (torch.int32, torch.uint32)
        self.logits = self.b16 + self.f32
        self.codes = (torch.uint8, torch.float8_e4m3fn)
        self.scales = (torch.uint8, torch.float8_e8m0fnu)
        self.same = {t: self.b16 for t in self.b16} | {torch.float32: self.f32}
        # handle of the current stream; torch.cuda.current_stream() builds an
        # object first, which takes as long as the launch
        self.raw_stream, self.device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
        self.ready = True


_types = _Types()


def _dt():
    if not _types.ready:
        _types.load()
    return _types


def _status(t, dev):
    """Pointer of a status word, an int on device `dev`."""
    if t is None:
        return None
    if t.dtype not in _types.status or t.get_device() != dev or t.numel() < 1:
        raise ValueError("status: a 32-bit integer on device %d expected, got %s of %s on %s"
                         % (dev, tuple(t.shape), t.dtype, _place(t)))
    return t.data_ptr()


def _workspace(t, dev):
    """Pointer and bytes of a workspace, contiguous memory on device `dev` of
    any type."""
    if t is None:
        return None, 0
    if t.get_device() != dev or not t.is_contiguous():
        raise ValueError("ws: a contiguous CUDA tensor on device %d expected, got %s on %s, strides %s"
                         % (dev, tuple(t.shape), _place(t), t.stride()))
    return t.data_ptr(), t.numel() * t.element_size()


def _stream(stream, dev):
    return _types.raw_stream(dev) if stream is None else stream.cuda_stream


def mx8_sf_bytes(rows, d):
    return int(lib().moe_mx8_sf_bytes(rows, d))


def add_rmsnorm_backward_workspace_bytes(T, d):
    return int(lib().moe_add_rmsnorm_backward_workspace_bytes(T, d))


def moe_add_rmsnorm(x, res, w, eps, h, y, y8=None, y8_sf=None, rstd=None, status=None, stream=None):
    """Residual add + RMS norm: h = x + res, y = h / rms(h) * w in BF16 and,
    with y8 and y8_sf, in E4M3 with a power-of-two scale per 32 values.  x and
    res [T][d] may have strided rows."""
    ty = _dt()
    b16 = ty.b16
    dev = _here(x, "x")
    px, ldx, shape = _rows(x, b16, None, "x", dev)
    T, d = shape
    pr, ldr, _ = (None, d, None) if res is None else _rows(res, b16, shape, "res", dev)
    if y8_sf is not None and (not y8_sf.is_contiguous() or y8_sf.dtype not in ty.scales or y8_sf.get_device() != dev
                              or y8_sf.numel() < (T + 127) // 128 * (d // 128) * 512):
        raise ValueError("y8_sf: at least %d contiguous scale bytes on device %d expected" % (mx8_sf_bytes(T, d), dev))
    _check("moe_add_rmsnorm", lib().moe_add_rmsnorm(
        px, ldx, pr, ldr, _tensor(w, b16, (d,), "w", dev), eps, T, d, _tensor(h, b16, shape, "h", dev),
        _tensor(y, b16, shape, "y", dev), _tensor(y8, ty.codes, shape, "y8", dev),
        None if y8_sf is None else y8_sf.data_ptr(), _tensor(rstd, ty.f32, (T,), "rstd", dev), _status(status, dev),
        _stream(stream, dev)))


def moe_add_rmsnorm_backward(dy, dh, h, rstd, w, dx, dw, ws, status=None, stream=None):
    """Gradients of moe_add_rmsnorm; dh (the gradient of h) and dw may be
    None."""
    ty = _dt()
    b16 = ty.b16
    shape = dy.shape
    if dy.dim() != 2:
        raise ValueError("dy: a 2-D tensor expected, got %s" % (tuple(shape),))
    _ints(shape, "dy")
    T, d = shape
    dev = _here(dy, "dy")
    pws, ws_bytes = _workspace(ws, dev)
    _check("moe_add_rmsnorm_backward", lib().moe_add_rmsnorm_backward(
        _tensor(dy, b16, shape, "dy", dev), _tensor(dh, b16, shape, "dh", dev), _tensor(h, b16, shape, "h", dev),
        _tensor(rstd, ty.f32, (T,), "rstd", dev), _tensor(w, b16, (d,), "w", dev), T, d,
        _tensor(dx, b16, shape, "dx", dev), _tensor(dw, ty.f32, (d,), "dw", dev), pws, ws_bytes,
        _status(status, dev), _stream(stream, dev)))


def moe_token_logprobs(logits, targets, inv_temperature, n_top, logprob, entropy, stats, top_ids=None,
                       top_logprob=None, status=None, stream=None):
    """Log-probabilities of the targets, entropy, softmax statistics and the
    n_top most likely ids of each row of logits [T][V] (strided rows
    allowed).  Outputs that are None are left out."""
    ty = _dt()
    f32 = ty.f32
    dev = _here(logits, "logits")
    pl, ld, shape = _rows(logits, ty.logits, None, "logits", dev)
    T, V = shape
    _check("moe_token_logprobs", lib().moe_token_logprobs(
        pl, 1 if logits.dtype in f32 else 0, ld, T, V, _tensor(targets, ty.i32, (T,), "targets", dev), inv_temperature,
        n_top, _tensor(logprob, f32, (T,), "logprob", dev), _tensor(entropy, f32, (T,), "entropy", dev),
        _tensor(stats, f32, (T, 2), "stats", dev), _tensor(top_ids, ty.i32, (T, n_top), "top_ids", dev),
        _tensor(top_logprob, f32, (T, n_top), "top_logprob", dev), _status(status, dev), _stream(stream, dev)))


def moe_token_logprobs_backward(logits, targets, inv_temperature, stats, entropy, g_logprob, g_entropy, dlogits,
                                status=None, stream=None):
    """Gradient of moe_token_logprobs with respect to the logits; dlogits may
    be the logits themselves."""
    ty = _dt()
    f32 = ty.f32
    dev = _here(logits, "logits")
    pl, ld, shape = _rows(logits, ty.logits, None, "logits", dev)
    T, V = shape
    pd, ldd, _ = _rows(dlogits, ty.same[logits.dtype], logits.shape, "dlogits", dev)
    _check("moe_token_logprobs_backward", lib().moe_token_logprobs_backward(
        pl, 1 if logits.dtype in f32 else 0, ld, T, V, _tensor(targets, ty.i32, (T,), "targets", dev), inv_temperature,
        _tensor(stats, f32, (T, 2), "stats", dev), _tensor(entropy, f32, (T,), "entropy", dev),
        _tensor(g_logprob, f32, (T,), "g_logprob", dev), _tensor(g_entropy, f32, (T,), "g_entropy", dev), pd, ldd,
        _status(status, dev), _stream(stream, dev)))


def _distill_args(ty, dev, logits, teacher_ids, teacher_logits, teacher_lse, inv_temperature):
    pl, ld, shape = _rows(logits, ty.logits, None, "logits", dev)
    T, V = shape
    if teacher_ids.dim() != 2:
        raise ValueError("teacher_ids: a 2-D tensor expected, got %s" % (tuple(teacher_ids.shape),))
    _ints(teacher_ids.shape, "teacher_ids")
    K = teacher_ids.shape[1]
    return (pl, 1 if logits.dtype in ty.f32 else 0, ld, T, V,
            _tensor(teacher_ids, ty.i32, (T, K), "teacher_ids", dev),
            _tensor(teacher_logits, ty.f32, (T, K), "teacher_logits", dev),
            _tensor(teacher_lse, ty.f32, (T,), "teacher_lse", dev), K, inv_temperature)


def moe_distill_topk(logits, teacher_ids, teacher_logits, teacher_lse, inv_temperature, loss, stats, status=None,
                     stream=None):
    """KL divergence of the rows of logits [T][V] from a teacher's top
    logits [T][K] (teacher_lse [T]: with the teacher's remaining mass as one
    outcome; None: over the listed ids)."""
    ty = _dt()
    T = logits.shape[0]
    dev = _here(logits, "logits")
    a = _distill_args(ty, dev, logits, teacher_ids, teacher_logits, teacher_lse, inv_temperature)
    _check("moe_distill_topk", lib().moe_distill_topk(
        *a, _tensor(loss, ty.f32, (T,), "loss", dev), _tensor(stats, ty.f32, (T, 4), "stats", dev),
        _status(status, dev), _stream(stream, dev)))


def moe_distill_topk_backward(logits, teacher_ids, teacher_logits, teacher_lse, inv_temperature, stats, g, dlogits,
                              status=None, stream=None):
    """Gradient of moe_distill_topk from its stats; dlogits may be the logits
    themselves."""
    ty = _dt()
    T = logits.shape[0]
    dev = _here(logits, "logits")
    a = _distill_args(ty, dev, logits, teacher_ids, teacher_logits, teacher_lse, inv_temperature)
    pd, ldd, _ = _rows(dlogits, ty.same[logits.dtype], logits.shape, "dlogits", dev)
    _check("moe_distill_topk_backward", lib().moe_distill_topk_backward(
        *a, _tensor(stats, ty.f32, (T, 4), "stats", dev), _tensor(g, ty.f32, (T,), "g", dev), pd, ldd,
        _status(status, dev), _stream(stream, dev)))


def moe_distill_topk_train(logits, teacher_ids, teacher_logits, teacher_lse, inv_temperature, g, loss, dlogits,
                           status=None, stream=None):
    """moe_distill_topk and its gradient in one call, each row's gradient
    weighted by g."""
    ty = _dt()
    T = logits.shape[0]
    dev = _here(logits, "logits")
    a = _distill_args(ty, dev, logits, teacher_ids, teacher_logits, teacher_lse, inv_temperature)
    pd, ldd, _ = _rows(dlogits, ty.same[logits.dtype], logits.shape, "dlogits", dev)
    _check("moe_distill_topk_train", lib().moe_distill_topk_train(
        *a, _tensor(g, ty.f32, (T,), "g", dev), _tensor(loss, ty.f32, (T,), "loss", dev), pd, ldd, _status(status, dev),
        _stream(stream, dev)))


# --------------------------------------------------------------------------
# the operators at the token ends (include/moe_tokens.h)
# --------------------------------------------------------------------------
def _ids(t, dtypes, what, dev):
    """Pointer and length of a vector of token ids on device `dev`."""
    if t.dim() != 1 or t.shape[0] > 0x7FFFFFFF:
        raise ValueError("%s: a vector of at most 2^31 - 1 ids expected, got %s" % (what, tuple(t.shape)))
    return _tensor(t, dtypes, t.shape, what, dev), t.shape[0]


def moe_embed_tokens(ids, table, scale, out, status=None, stream=None):
    """out[t] = scale * table[ids[t]] in BF16, zeros for a negative id.  The rows
    of table [V][d] (BF16 or FP32) and out [T][d] may be strided."""
    ty = _dt()
    dev = _here(ids, "ids")
    pi, T = _ids(ids, ty.i32, "ids", dev)
    pt, ldt, (V, d) = _rows(table, ty.logits, None, "table", dev)
    po, ldo, shape = _rows(out, ty.b16, None, "out", dev)
    if shape[0] != T or shape[1] != d:
        raise ValueError("out: %s expected, got %s" % ((T, d), tuple(shape)))
    _check("moe_embed_tokens", lib().moe_embed_tokens(
        pi, pt, 1 if table.dtype in ty.f32 else 0, ldt, T, V, d, scale, po, ldo, _status(status, dev),
        _stream(stream, dev)))


def embed_tokens_backward_workspace_bytes(T, V, d):
    return int(lib().moe_embed_tokens_backward_workspace_bytes(T, V, d))


def moe_embed_tokens_backward(dy, ids, scale, dtable, ws, accumulate=False, status=None, stream=None):
    """Gradient of moe_embed_tokens with respect to the table, dtable [V][d] in
    FP32: all rows written, or, with accumulate, the named rows added to.  The
    rows of dy [T][d] may be strided."""
    ty = _dt()
    dev = _here(dy, "dy")
    py, ldy, (T, d) = _rows(dy, ty.b16, None, "dy", dev)
    if dtable.dim() != 2:
        raise ValueError("dtable: a 2-D tensor expected, got %s" % (tuple(dtable.shape),))
    _ints(dtable.shape, "dtable")
    V = dtable.shape[0]
    pws, ws_bytes = _workspace(ws, dev)
    _check("moe_embed_tokens_backward", lib().moe_embed_tokens_backward(
        py, ldy, _tensor(ids, ty.i32, (T,), "ids", dev), T, V, d, scale, 1 if accumulate else 0,
        _tensor(dtable, ty.f32, (V, d), "dtable", dev), pws, ws_bytes, _status(status, dev), _stream(stream, dev)))


def moe_sample_tokens(logits, u, tokens, inv_temperature=None, top_k=None, top_p=None, min_p=None, logprob=None,
                      kept_logprob=None, status=None, stream=None):
    """A token of each row of logits [T][V] (strided rows allowed), drawn with
    the random number u[t] in [0, 1) and the row's own temperature and filters
    (vectors [T]; None: off); its log-probability under the whole row and under
    what the filters kept."""
    ty = _dt()
    f32 = ty.f32
    dev = _here(logits, "logits")
    pl, ld, (T, V) = _rows(logits, ty.logits, None, "logits", dev)
    row = (T,)
    if u is None or tokens is None:
        raise ValueError("u and tokens are needed")
    _check("moe_sample_tokens", lib().moe_sample_tokens(
        pl, 1 if logits.dtype in f32 else 0, ld, T, V, _tensor(inv_temperature, f32, row, "inv_temperature", dev),
        _tensor(top_k, ty.i32, row, "top_k", dev), _tensor(top_p, f32, row, "top_p", dev),
        _tensor(min_p, f32, row, "min_p", dev), _tensor(u, f32, row, "u", dev), _tensor(tokens, ty.i32, row, "tokens", dev),
        _tensor(logprob, f32, row, "logprob", dev), _tensor(kept_logprob, f32, row, "kept_logprob", dev),
        _status(status, dev), _stream(stream, dev)))


class Pipeline:
    """moe_pipeline_*: the forward on host-resident batches, with the copies
    of neighbouring steps overlapping the forward (three streams, `depth`
    slots).  Host tensors should be pinned."""

    def __init__(self, T, E, k, d, d_ff, depth=2, device="cuda"):
        import torch
        n = int(lib().moe_pipeline_device_bytes(T, E, k, d, d_ff, depth))
        if n == 0:
            raise MoeError("moe_pipeline_device_bytes", MOE_ERR_SHAPE)
        self.buf = torch.empty(n + 1024, dtype=torch.uint8, device=device)
        off = (-self.buf.data_ptr()) % 1024
        self._h = ctypes.c_void_p()
        _check("moe_pipeline_create", lib().moe_pipeline_create(
            T, E, k, d, d_ff, depth, ctypes.c_void_p(self.buf.data_ptr() + off), n, ctypes.byref(self._h)))

    def submit(self, x_host, logits_host, out_host, w1q, w2q, status=None):
        _check("moe_pipeline_submit", lib().moe_pipeline_submit(
            self._h, _p(x_host), _p(logits_host), _p(out_host), _p(w1q["codes"]), _p(w1q["sf"]), _p(w1q["g"]),
            _p(w2q["codes"]), _p(w2q["sf"]), _p(w2q["g"]), _p(status)))

    def synchronize(self):
        _check("moe_pipeline_synchronize", lib().moe_pipeline_synchronize(self._h))

    def close(self):
        if self._h:
            rc = lib().moe_pipeline_destroy(self._h)
            self._h = ctypes.c_void_p()
            _check("moe_pipeline_destroy", rc)


# --------------------------------------------------------------------------
# device-memory helpers (torch allocations of the buffers the calls expect)
# --------------------------------------------------------------------------
def empty_quantized(rows, K, device="cuda"):
    import torch
    return dict(codes=torch.empty((rows, K // 2), dtype=torch.uint8, device=device),
                sf=torch.empty(max(sf_bytes(rows, K), 16), dtype=torch.uint8, device=device),
                g=torch.empty(rows, dtype=torch.float32, device=device))


def quantize_weights(W):
    """Quantise expert weights W [E][N][K] (bf16) on the GPU; returns a dict
    with codes [E][N][K/2], sf (flat) and g [E][N]."""
    E, N, K = W.shape
    q = empty_quantized(E * N, K, W.device)
    moe_nvfp4_quantize_weights(W, q["codes"], q["sf"], q["g"])
    q["codes"] = q["codes"].view(E, N, K // 2)
    q["g"] = q["g"].view(E, N)
    return q


def quantize_weights_per_expert(W):
    """quantize_weights with one outer scale per expert tensor; the dict also
    holds amax_e [E] = max |W_e|."""
    import torch
    E, N, K = W.shape
    q = empty_quantized(E * N, K, W.device)
    q["amax_e"] = torch.empty(E, dtype=torch.float32, device=W.device)
    moe_nvfp4_quantize_weights_per_expert(W, q["codes"], q["sf"], q["g"], q["amax_e"])
    q["codes"] = q["codes"].view(E, N, K // 2)
    q["g"] = q["g"].view(E, N)
    return q


def forward_workspace(T, E, k, d, d_ff, device="cuda"):
    import torch
    n = forward_workspace_bytes(T, E, k, d, d_ff)
    if n == 0:
        raise MoeError("moe_expert_forward_workspace_bytes", MOE_ERR_SHAPE)
    return torch.empty(n, dtype=torch.uint8, device=device)


def forward_views(ws, T, E, k, d, d_ff):
    """Typed views of the intermediates that moe_expert_forward leaves in ws."""
    import torch
    lay = forward_workspace_layout(T, E, k, d, d_ff)
    mc = m_cap(T, E, k)

    def v(name, dtype, shape, nbytes=None):
        o = lay[name]
        esz = torch.empty((), dtype=dtype).element_size()
        n = 1
        for s in shape:
            n *= s
        return ws[o:o + n * esz].view(dtype).view(*shape)

    return dict(
        topk_ids=v("topk_ids", torch.int32, (T, k)), topk_w=v("topk_w", torch.float32, (T, k)),
        token_slot_row=v("token_slot_row", torch.int32, (T, k)), counts=v("counts", torch.int32, (E,)),
        offsets=v("offsets", torch.int32, (E + 1,)), row_to_token=v("row_to_token", torch.int32, (mc,)),
        amax_tok=v("amax_tok", torch.float32, (T,)), x_codes=v("x_codes", torch.uint8, (mc, d // 2)),
        x_sf=v("x_sf", torch.uint8, (sf_bytes(mc, d),)), x_g=v("x_g", torch.float32, (mc,)),
        h_codes=v("h_codes", torch.uint8, (mc, d_ff // 2)), h_sf=v("h_sf", torch.uint8, (sf_bytes(mc, d_ff),)),
        h_g=v("h_g", torch.float32, (mc,)), slots=v("slots", torch.int16, (mc, d)), m_cap=mc)
