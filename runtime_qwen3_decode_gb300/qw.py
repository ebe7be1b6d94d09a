"""ctypes binding of libqw.so (include/qw.h): argument marshalling only.

Every step of the decoder runs in the library's CUDA kernels; PyTorch provides the
device memory (weights, workspace) and the stream.  Importing this module does not
need a GPU; creating a model does, and there is no fallback: if the library is not
built or the device cannot run it, the call raises.
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libqw.so")

OK = 0
INVALID_ARGUMENT = 1
INVALID_HANDLE = 4
ALIGNMENT = 7
INTEGER_OVERFLOW = 8
OUT_OF_MEMORY = 9
UNSUPPORTED_QUANTIZATION = 12
UNSUPPORTED_SHAPE = 13
CONTEXT_EXCEEDED = 14
NUMERICAL_FAILURE = 18
INTERNAL_INVARIANT = 20
CUDA_ERROR = 21

W_BF16 = 0
W_INT8_G32 = 1
W_Q8Q8 = 2
KV_F32 = 0
KV_BF16 = 1
KV_INT8_G32 = 2
DEBUG_HIDDEN = 1
DEBUG_PREFILL_BY_TOKEN = 2
DEBUG_TRACE = 4
DEBUG_ONE_GROUP = 8
DEBUG_WITHHOLD = 16
QUERY_DECODE_CTAS = 1
QUERY_TRACE_LEN = 2
QUERY_WORKSPACE_BYTES = 3
QUERY_DECODE_GROUPS = 4
QUERY_GROUP0_CTAS = 5
QUERY_RT_NEAR_NS = 6
QUERY_RT_FAR_NS = 7
QUERY_XREGION_OFFSET = 8
MATRICES = ("q", "k", "v", "o", "gate", "up", "down")

# every symbol include/qw.h declares
EXPORTS = ("qw_workspace_bytes", "qw_model_create", "qw_prefill", "qw_decode_step", "qw_generate", "qw_logits",
           "qw_kv_reset", "qw_kv_length", "qw_sync", "qw_model_destroy", "qw_kv_import", "qw_kv_export",
           "qw_set_debug", "qw_debug_hidden", "qw_status_string", "qw_abi_version", "qw_debug_trace", "qw_query",
           "qw_decode_step_noalloc", "qw_debug_gemm_f16", "qw_sample_scratch_bytes", "qw_sample_logits",
           "qw_sampler_seed", "qw_sampler_state", "qw_sample", "qw_batch_workspace_bytes", "qw_batch_create",
           "qw_batch_destroy", "qw_batch_reset", "qw_batch_length", "qw_batch_prefill", "qw_batch_step",
           "qw_batch_logits", "qw_batch_debug_hidden", "qw_batch_sync", "qw_checkpoint_open",
           "qw_checkpoint_close", "qw_checkpoint_last_error", "qw_checkpoint_count", "qw_checkpoint_tensor",
           "qw_checkpoint_check", "qw_checkpoint_upload_bytes", "qw_checkpoint_upload", "qw_kv_append", "qw_kv_read",
           "qw_tree_attention_scratch_bytes", "qw_tree_attention", "qw_prefix_attention_scratch_bytes",
           "qw_prefix_attention", "qw_process_logits", "qw_sample_rows", "qw_batch_workspace_bytes_kv",
           "qw_batch_create_kv", "qw_batch_tree_step", "qw_batch_tree_accept", "qw_batch_fork", "qw_batch_sample")
DT_BF16, DT_F16, DT_F32, DT_I8, DT_Q8_0 = 0, 1, 2, 3, 4
BATCH_MAX = 8
TREE_NODES_MAX = 64


class CheckpointReport(ctypes.Structure):
    _fields_ = [("n_tensors", ctypes.c_int32), ("n_expected", ctypes.c_int32), ("n_found", ctypes.c_int32),
                ("n_missing", ctypes.c_int32), ("n_misshaped", ctypes.c_int32), ("n_unexpected", ctypes.c_int32),
                ("n_bad_dtype", ctypes.c_int32), ("lm_head_copy", ctypes.c_int32), ("stored_params", ctypes.c_int64),
                ("logical_params", ctypes.c_int64), ("embedding_params", ctypes.c_int64),
                ("first_problem", ctypes.c_char * 256)]


class QwError(RuntimeError):
    def __init__(self, code: int, what: str):
        msg = _lib().qw_status_string(code).decode() if _LIB is not None else str(code)
        super().__init__(f"{what}: {msg} (status {code})")
        self.code = code


class Config(ctypes.Structure):
    _fields_ = [("n_layers", ctypes.c_int32), ("hidden", ctypes.c_int32), ("n_heads", ctypes.c_int32),
                ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("intermediate", ctypes.c_int32),
                ("vocab", ctypes.c_int32), ("rms_eps", ctypes.c_float), ("rope_theta", ctypes.c_double),
                ("max_ctx", ctypes.c_int32), ("weight_format", ctypes.c_int32), ("kv_format", ctypes.c_int32)]


class LayerWeights(ctypes.Structure):
    _fields_ = [("input_norm", ctypes.c_void_p), ("q_norm", ctypes.c_void_p), ("k_norm", ctypes.c_void_p),
                ("post_norm", ctypes.c_void_p), ("w", ctypes.c_void_p * 7), ("s", ctypes.c_void_p * 7)]


class Sampling(ctypes.Structure):
    _fields_ = [("temperature", ctypes.c_float), ("top_k", ctypes.c_int32), ("top_p", ctypes.c_float),
                ("repetition_penalty", ctypes.c_float)]


SAMPLE_MAX_TOP_K = 64


class KvViewStruct(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("format", ctypes.c_int32), ("n_seq", ctypes.c_int32),
                ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("max_ctx", ctypes.c_int32),
                ("seq_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64), ("pos_stride", ctypes.c_int64),
                ("scale_seq_stride", ctypes.c_int64), ("scale_head_stride", ctypes.c_int64),
                ("scale_pos_stride", ctypes.c_int64)]


class KvRowsStruct(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("n_max", ctypes.c_int32),
                ("seq_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64), ("row_stride", ctypes.c_int64)]


class TreeAttentionArgs(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("out", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("n_max", ctypes.c_int32),
                ("n_heads", ctypes.c_int32), ("max_len", ctypes.c_int32), ("scale", ctypes.c_float),
                ("q_seq_stride", ctypes.c_int64), ("q_node_stride", ctypes.c_int64), ("q_head_stride", ctypes.c_int64),
                ("out_seq_stride", ctypes.c_int64), ("out_node_stride", ctypes.c_int64),
                ("out_head_stride", ctypes.c_int64), ("mask", ctypes.c_void_p), ("len", ctypes.c_void_p),
                ("count", ctypes.c_void_p)]


class ProcessLogitsArgs(ctypes.Structure):
    _fields_ = [("logits", ctypes.c_void_p), ("out", ctypes.c_void_p), ("dtype", ctypes.c_int32),
                ("n_rows", ctypes.c_int32), ("vocab", ctypes.c_int32), ("row_stride", ctypes.c_int64),
                ("out_row_stride", ctypes.c_int64), ("penalties", ctypes.c_void_p), ("history", ctypes.c_void_p),
                ("history_range", ctypes.c_void_p), ("n_history", ctypes.c_int32), ("path", ctypes.c_void_p),
                ("path_len", ctypes.c_int32), ("bias_ids", ctypes.c_void_p), ("bias", ctypes.c_void_p),
                ("bias_range", ctypes.c_void_p), ("n_bias", ctypes.c_int32), ("mask", ctypes.c_void_p),
                ("mask_index", ctypes.c_void_p), ("n_masks", ctypes.c_int32)]


class SampleRowsArgs(ctypes.Structure):
    _fields_ = [("logits", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("n_rows", ctypes.c_int32),
                ("vocab", ctypes.c_int32), ("row_stride", ctypes.c_int64), ("u", ctypes.c_void_p),
                ("temperature", ctypes.c_void_p), ("top_k", ctypes.c_void_p), ("top_p", ctypes.c_void_p),
                ("min_p", ctypes.c_void_p), ("tokens", ctypes.c_void_p), ("probs", ctypes.c_void_p),
                ("kept", ctypes.c_void_p)]


class Weights(ctypes.Structure):
    _fields_ = [("embed", ctypes.c_void_p), ("final_norm", ctypes.c_void_p), ("lm_head", ctypes.c_void_p),
                ("layers", ctypes.POINTER(LayerWeights))]


_LIB = None
_LOCK = threading.Lock()


def _lib():
    global _LIB
    if _LIB is not None:
        return _LIB
    with _LOCK:
        if _LIB is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"libqw.so is not built ({LIB_PATH}); run __graft_entry__.build()")
            L = ctypes.CDLL(LIB_PATH)
            vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
            i32p = ctypes.POINTER(ctypes.c_int32)
            L.qw_workspace_bytes.argtypes = [ctypes.POINTER(Config)]
            L.qw_workspace_bytes.restype = ctypes.c_size_t
            L.qw_model_create.argtypes = [ctypes.POINTER(Config), ctypes.POINTER(Weights), vp, ctypes.c_size_t, vp,
                                          ctypes.POINTER(vp)]
            L.qw_prefill.argtypes = [vp, i32p, i32, i32p]
            L.qw_decode_step.argtypes = [vp, i32, i32p]
            L.qw_generate.argtypes = [vp, i32, i32, vp]
            L.qw_logits.argtypes = [vp, vp, i64]
            L.qw_kv_reset.argtypes = [vp]
            L.qw_kv_length.argtypes = [vp, i32p]
            L.qw_sync.argtypes = [vp]
            L.qw_model_destroy.argtypes = [vp]
            L.qw_model_destroy.restype = None
            L.qw_kv_import.argtypes = [vp, vp, vp, i32]
            L.qw_kv_export.argtypes = [vp, vp, vp, i32]
            L.qw_set_debug.argtypes = [vp, i32]
            L.qw_debug_hidden.argtypes = [vp, vp, i64]
            L.qw_debug_trace.argtypes = [vp, vp, i64]
            L.qw_query.argtypes = [vp, i32, ctypes.POINTER(ctypes.c_int64)]
            L.qw_decode_step_noalloc.argtypes = [ctypes.POINTER(Config), ctypes.POINTER(Weights), vp, vp, i32, i32, vp,
                                                 vp, vp, i32]
            L.qw_debug_gemm_f16.argtypes = [vp, vp, vp, i32, i32, i32, i32, vp]
            L.qw_sample_scratch_bytes.argtypes = [i32]
            L.qw_sample_scratch_bytes.restype = ctypes.c_size_t
            L.qw_sample_logits.argtypes = [vp, i32, vp, i32, ctypes.POINTER(Sampling), vp, vp, vp, ctypes.c_size_t, vp]
            L.qw_sampler_seed.argtypes = [vp, ctypes.c_uint64, ctypes.c_uint64]
            L.qw_sampler_state.argtypes = [vp, vp]
            L.qw_sample.argtypes = [vp, ctypes.POINTER(Sampling), vp, i32, vp]
            L.qw_batch_workspace_bytes.argtypes = [vp, i32, i32]
            L.qw_batch_workspace_bytes.restype = ctypes.c_size_t
            L.qw_batch_create.argtypes = [vp, i32, i32, vp, ctypes.c_size_t, ctypes.POINTER(ctypes.c_void_p)]
            L.qw_batch_destroy.argtypes = [vp]
            L.qw_batch_destroy.restype = None
            L.qw_batch_reset.argtypes = [vp, i32]
            L.qw_batch_length.argtypes = [vp, i32, i32p]
            L.qw_batch_prefill.argtypes = [vp, i32, i32p, i32, i32p]
            L.qw_batch_step.argtypes = [vp, i32, i32p, i32p]
            L.qw_batch_logits.argtypes = [vp, vp, i64]
            L.qw_batch_debug_hidden.argtypes = [vp, vp, i64]
            L.qw_batch_sync.argtypes = [vp]
            L.qw_batch_workspace_bytes_kv.argtypes = [vp, i32, i32, i32]
            L.qw_batch_workspace_bytes_kv.restype = ctypes.c_size_t
            L.qw_batch_create_kv.argtypes = [vp, i32, i32, i32, vp, ctypes.c_size_t, ctypes.POINTER(ctypes.c_void_p)]
            L.qw_batch_tree_step.argtypes = [vp, i32, i32, i32p, i32p, i32p]
            L.qw_batch_tree_accept.argtypes = [vp, i32, i32, i32p]
            L.qw_batch_fork.argtypes = [vp, i32, i32, i32]
            L.qw_batch_sample.argtypes = [vp, i32, vp, vp, vp, vp, vp, i32p]
            u64 = ctypes.c_uint64
            L.qw_checkpoint_open.argtypes = [vp, u64, u64, ctypes.POINTER(ctypes.c_void_p)]
            L.qw_checkpoint_close.argtypes = [vp]
            L.qw_checkpoint_close.restype = None
            L.qw_checkpoint_last_error.argtypes = []
            L.qw_checkpoint_last_error.restype = ctypes.c_char_p
            L.qw_checkpoint_count.argtypes = [vp]
            L.qw_checkpoint_count.restype = i32
            L.qw_checkpoint_tensor.argtypes = [vp, i32, ctypes.c_char_p, i32, i32p, i32p,
                                               ctypes.POINTER(ctypes.c_int64), ctypes.POINTER(u64),
                                               ctypes.POINTER(u64)]
            L.qw_checkpoint_check.argtypes = [vp, ctypes.POINTER(Config), ctypes.POINTER(CheckpointReport)]
            L.qw_checkpoint_upload_bytes.argtypes = [vp, ctypes.POINTER(Config)]
            L.qw_checkpoint_upload_bytes.restype = ctypes.c_size_t
            L.qw_checkpoint_upload.argtypes = [vp, ctypes.POINTER(Config), vp, ctypes.c_size_t,
                                               ctypes.POINTER(LayerWeights), ctypes.POINTER(Weights), vp]
            L.qw_kv_append.argtypes = [vp, vp, vp, vp, vp]
            L.qw_kv_read.argtypes = [vp, vp, vp, vp, vp]
            L.qw_tree_attention_scratch_bytes.argtypes = [vp, i32, i32, i32]
            L.qw_tree_attention_scratch_bytes.restype = ctypes.c_size_t
            L.qw_tree_attention.argtypes = [vp, vp, vp, ctypes.c_size_t, vp]
            L.qw_prefix_attention_scratch_bytes.argtypes = [vp, vp, i32, i32, i32, i32]
            L.qw_prefix_attention_scratch_bytes.restype = ctypes.c_size_t
            L.qw_prefix_attention.argtypes = [vp, vp, vp, vp, i32, vp, ctypes.c_size_t, vp]
            L.qw_process_logits.argtypes = [vp, vp]
            L.qw_sample_rows.argtypes = [vp, vp]
            L.qw_status_string.argtypes = [ctypes.c_int]
            L.qw_status_string.restype = ctypes.c_char_p
            L.qw_abi_version.argtypes = []
            L.qw_abi_version.restype = i32
            _LIB = L
    return _LIB


def lib():
    return _lib()


def _check(rc: int, what: str):
    if rc != OK:
        raise QwError(rc, what)


def make_config(dims, max_ctx: int | None = None) -> Config:
    """dims: any object with the Qwen3 dimension attributes (n_layers, hidden, ...)."""
    fmt = {"bf16": W_BF16, "int8_g32": W_INT8_G32}.get(getattr(dims, "weight_format", "bf16"), -1)
    if getattr(dims, "act_format", "f32") == "q8":
        fmt = W_Q8Q8 if fmt == W_INT8_G32 else -1
    kvf = {"f32": KV_F32, "bf16": KV_BF16}.get(getattr(dims, "kv_format", "f32"), -1)
    return Config(dims.n_layers, dims.hidden, dims.n_heads, dims.n_kv_heads, dims.head_dim, dims.intermediate,
                  dims.vocab, dims.rms_eps, dims.rope_theta, int(max_ctx or dims.max_ctx), fmt, kvf)


def workspace_bytes(cfg: Config) -> int:
    return int(_lib().qw_workspace_bytes(ctypes.byref(cfg)))


def weights_to_device(host_weights: dict, int8: bool, device="cuda"):
    """Copy a {embed, final_norm, layers[...]} dict of numpy arrays to device tensors.

    bf16 tensors travel as int16 bit patterns (the library reads raw bytes).  For the
    int8 format, each matrix m comes as "<m>_q8" (int8) and "<m>_s" (fp16 bits).
    """
    import torch

    def dev(a):
        a = np.ascontiguousarray(a)
        if a.dtype == np.uint16:
            a = a.view(np.int16)
        return torch.from_numpy(a).to(device)

    out = {"embed": dev(host_weights["embed"]), "final_norm": dev(host_weights["final_norm"]), "layers": []}
    for lw in host_weights["layers"]:
        d = {k: dev(lw[k]) for k in ("input_norm", "q_norm", "k_norm", "post_norm")}
        for m in MATRICES:
            if int8:
                d[m + "_q8"] = dev(lw[m + "_q8"])
                d[m + "_s"] = dev(lw[m + "_s"])
            else:
                d[m] = dev(lw[m])
        out["layers"].append(d)
    return out


def weight_table(dev_weights: dict, int8: bool):
    """(Weights struct, layer array) for device weights from ``weights_to_device``; keep both alive."""
    n = len(dev_weights["layers"])
    layers = (LayerWeights * n)()
    for l, lw in enumerate(dev_weights["layers"]):
        L = layers[l]
        L.input_norm = lw["input_norm"].data_ptr()
        L.q_norm = lw["q_norm"].data_ptr()
        L.k_norm = lw["k_norm"].data_ptr()
        L.post_norm = lw["post_norm"].data_ptr()
        for j, m in enumerate(MATRICES):
            if int8:
                L.w[j] = lw[m + "_q8"].data_ptr()
                L.s[j] = lw[m + "_s"].data_ptr()
            else:
                L.w[j] = lw[m].data_ptr()
    w = Weights(dev_weights["embed"].data_ptr(), dev_weights["final_norm"].data_ptr(), None, layers)
    return w, layers


def decode_step_noalloc(cfg: Config, dev_weights: dict, k_cache, v_cache, pos: int, token: int, logits_out,
                        next_token_out, stream=None, wait: bool = True):
    """qw_decode_step_noalloc: one step over caller-owned K/V planes; no device allocation.

    The library cannot see the sizes of the caller's buffers, so they are checked here:
    CUDA, contiguous, K/V planes of the cache element type cfg.kv_format names holding
    n_layers * n_kv_heads * max_ctx * head_dim elements each, f32 logits of at least
    vocab elements, an int32 slot for the pick.
    """
    import torch
    kv_dtype = torch.float32 if cfg.kv_format == KV_F32 else torch.bfloat16
    plane = cfg.n_layers * cfg.n_kv_heads * cfg.max_ctx * cfg.head_dim
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        if not (t.is_cuda and t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
        if t.dtype != kv_dtype:
            raise ValueError(f"{name} must be {kv_dtype} for this kv_format")
        if t.numel() < plane:
            raise ValueError(f"{name} holds {t.numel()} elements, the config needs {plane}")
    if not (logits_out.is_cuda and logits_out.is_contiguous()) or logits_out.dtype != torch.float32 \
            or logits_out.numel() < cfg.vocab:
        raise ValueError("logits_out must be a contiguous CUDA float32 tensor of at least vocab elements")
    if not next_token_out.is_cuda or next_token_out.dtype != torch.int32 or next_token_out.numel() < 1:
        raise ValueError("next_token_out must be a CUDA int32 tensor")
    w, layers = weight_table(dev_weights, cfg.weight_format != W_BF16)
    st = stream if stream is not None else torch.cuda.current_stream()
    _check(_lib().qw_decode_step_noalloc(ctypes.byref(cfg), ctypes.byref(w), k_cache.data_ptr(), v_cache.data_ptr(),
                                         int(pos), int(token), logits_out.data_ptr(), next_token_out.data_ptr(),
                                         st.cuda_stream, 1 if wait else 0), "qw_decode_step_noalloc")


def debug_gemm_f16(a, b, c, bn: int = 256, stream=None):
    """qw_debug_gemm_f16: c[M,N] = a[M,K] @ b[N,K]^T on the prefill's tensor-core GEMM (fp16 in, f32 out)."""
    import torch
    st = stream if stream is not None else torch.cuda.current_stream()
    M, K = a.shape
    N = b.shape[0]
    _check(_lib().qw_debug_gemm_f16(a.data_ptr(), b.data_ptr(), c.data_ptr(), int(M), int(N), int(K), int(bn),
                                    st.cuda_stream), "qw_debug_gemm_f16")


def sample_logits(logits, params: Sampling, rng, token_out, history=None, scratch=None, stream=None):
    """qw_sample_logits on device tensors: logits f32 [V], rng uint64 [2] (int64 tensor),
    token_out int32 [1], history int32 [n] or None."""
    import torch
    V = logits.numel()
    need = _lib().qw_sample_scratch_bytes(V)
    if scratch is None:
        scratch = torch.empty(need, dtype=torch.uint8, device="cuda")
    st = stream if stream is not None else torch.cuda.current_stream()
    n = 0 if history is None else history.numel()
    _check(_lib().qw_sample_logits(logits.data_ptr(), V, history.data_ptr() if n else None, n, ctypes.byref(params),
                                   rng.data_ptr(), token_out.data_ptr(), scratch.data_ptr(), scratch.numel(),
                                   st.cuda_stream), "qw_sample_logits")


# ------------------------------------------------------- operators on caller-owned tensors
#
# These calls sit in a step's inner loop, where their own time counts beside a few microseconds of
# kernel: arguments go into one packed struct (the C layout of the ctypes classes above), and the
# checks use the tensors' cheap accessors.

_KV_ROWS = struct.Struct("@PPiiqqq")
_TREE_ARGS = struct.Struct("@PPiiiif4xqqqqqqPPP")
_LOGITS_ARGS = struct.Struct("@PPiii4xqqPPPi4xPi4xPPPi4xPPi4x")
_SAMPLE_ARGS = struct.Struct("@PiiiqPPPPPPPP")
_T = None  # torch, once one of these operators is used
_DTYPES = {}


def _use_torch():
    global _T
    if _T is None:
        import torch
        _DTYPES.update({torch.float32: DT_F32, torch.bfloat16: DT_BF16, torch.float16: DT_F16})
        _T = torch


def _dtype_code(t, what):
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{what} must be float32, float16 or bfloat16")
    return code


def _on(dev, stream, what, call, *args):
    """call(*args, cuda_stream) with device `dev` current; stream None = that device's current stream."""
    st = _T._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream
    if _T._C._cuda_getDevice() == dev:
        rc = call(*args, st)
    else:
        with _T.cuda.device(dev):
            rc = call(*args, st)
    if rc != OK:
        raise QwError(rc, what)


def _want(t, what, dev, dtype, shape):
    """Address of a contiguous tensor of this type and shape on device dev; 0 for None."""
    if t is None:
        return 0
    if t.get_device() != dev or t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {dtype} tensor of shape {tuple(shape)} on cuda:{dev}")
    return t.data_ptr()


class KvView:
    """A K/V cache in the caller's tensors, for kv_append, kv_read and tree_attention.

    k, v: [n_seq, n_kv_heads, max_ctx, head_dim], float32, bfloat16, or int8 codes with
    k_scale, v_scale: float16 [n_seq, n_kv_heads, max_ctx, head_dim / 32].  Any strides with
    a contiguous last dimension (a layer of a larger cache, a transposed layout); k and v
    share theirs, and so do the scales.  The view keeps the tensors alive."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        _use_torch()
        torch = _T
        if not k.is_cuda:
            raise ValueError("the cache must be CUDA tensors")
        if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype or k.device != v.device or k.stride() != v.stride():
            raise ValueError("k and v must be [n_seq, n_kv_heads, max_ctx, head_dim] alike in type, strides and device")
        if k.stride(3) != 1:
            raise ValueError("the last dimension must be contiguous")
        fmt = {torch.float32: KV_F32, torch.bfloat16: KV_BF16, torch.int8: KV_INT8_G32}.get(k.dtype)
        if fmt is None:
            raise ValueError("the cache must be float32, bfloat16 or int8")
        s = KvViewStruct(k.data_ptr(), v.data_ptr(), None, None, fmt, k.shape[0], k.shape[1], k.shape[3], k.shape[2],
                         k.stride(0), k.stride(1), k.stride(2), 0, 0, 0)
        if fmt == KV_INT8_G32:
            if k_scale is None or v_scale is None:
                raise ValueError("an int8 cache needs k_scale and v_scale")
            want = (*k.shape[:3], k.shape[3] // 32)
            for t in (k_scale, v_scale):
                if t.dtype != torch.float16 or t.shape != want or t.device != k.device or t.stride(3) != 1 \
                        or t.stride() != k_scale.stride():
                    raise ValueError(f"the scales must be float16 {want} tensors with the same strides, beside the codes")
            s.k_scale, s.v_scale = k_scale.data_ptr(), v_scale.data_ptr()
            s.scale_seq_stride, s.scale_head_stride, s.scale_pos_stride = k_scale.stride()[:3]
        elif k_scale is not None or v_scale is not None:
            raise ValueError("only an int8 cache has scales")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.n_seq, self.n_kv_heads, self.max_ctx, self.head_dim = k.shape
        self.device = k.device
        self._dev = k.get_device()
        self.struct = s
        self._ref = ctypes.byref(s)
        self._per_seq = (self.n_seq,)


def _kv_rows(view, k, v, what):
    shape, stride, dev = k.shape, k.stride(), view._dev
    if len(shape) != 4 or shape != v.shape or k.dtype is not v.dtype or stride != v.stride() or stride[3] != 1 \
            or k.get_device() != dev or v.get_device() != dev:
        raise ValueError(f"{what} must be two tensors [n_seq, n_kv_heads, n, head_dim] alike, beside the cache, "
                         "with a contiguous last dimension")
    if shape[0] != view.n_seq or shape[1] != view.n_kv_heads or shape[3] != view.head_dim:
        raise ValueError(f"{what} do not match the cache's sequences, heads or head_dim")
    return _KV_ROWS.pack(k.data_ptr(), v.data_ptr(), _dtype_code(k, what), shape[2], stride[0], stride[1], stride[2])


def kv_append(view: KvView, k, v, start, count=None, stream=None):
    """qw_kv_append: rows k, v [n_seq, n_kv_heads, n, head_dim] (any strides with a contiguous last
    dimension) into positions start[b] .. start[b] + count[b] - 1 of the cache; start, count: int32
    [n_seq] on the device (count None: all n)."""
    i32 = _T.int32
    _on(view._dev, stream, "qw_kv_append", _lib().qw_kv_append, view._ref, _kv_rows(view, k, v, "the rows"),
        _want(start, "start", view._dev, i32, view._per_seq), _want(count, "count", view._dev, i32, view._per_seq))


def kv_read(view: KvView, k_out, v_out, start, count=None, stream=None):
    """qw_kv_read: positions start[b] .. start[b] + count[b] - 1 of the cache into k_out, v_out."""
    i32 = _T.int32
    _on(view._dev, stream, "qw_kv_read", _lib().qw_kv_read, view._ref, _kv_rows(view, k_out, v_out, "the rows"),
        _want(start, "start", view._dev, i32, view._per_seq), _want(count, "count", view._dev, i32, view._per_seq))


def tree_mask(parents) -> np.ndarray:
    """uint64 masks of a drafted tree: parents[i] < i is node i's parent node, -1 for a child of the
    last cached token; bit j of the result's entry i is set when node i sees node j (itself and its
    ancestors)."""
    parents = [int(p) for p in parents]
    if len(parents) > TREE_NODES_MAX:
        raise ValueError(f"a tree has at most {TREE_NODES_MAX} nodes")
    out = []
    for i, p in enumerate(parents):
        if not -1 <= p < i:
            raise ValueError(f"node {i}: parent {p} is not an earlier node")
        out.append((1 << i) | (out[p] if p >= 0 else 0))
    return np.array(out, dtype=np.uint64)


def tree_attention_scratch(view: KvView, n_max: int, n_heads: int, max_len: int | None = None):
    """Workspace of tree_attention calls with these sizes, max_len or less (None: the cache's length),
    one call at a time."""
    n = _lib().qw_tree_attention_scratch_bytes(view._ref, n_max, n_heads, view.max_ctx if max_len is None else max_len)
    if n == 0 and n_max:
        raise QwError(UNSUPPORTED_SHAPE, "qw_tree_attention_scratch_bytes")
    return _T.empty(max(n, 256), dtype=_T.uint8, device=view.device)


def tree_attention(view: KvView, q, mask, lens, out=None, counts=None, max_len=None, scale=None, scratch=None,
                   stream=None):
    """qw_tree_attention: q [n_seq, n, n_heads, head_dim] (float32, float16 or bfloat16, any strides with a
    contiguous last dimension), mask int64 [n_seq, n] (the bits of tree_mask), lens and counts int32
    [n_seq] on the device.  Node i of sequence b attends to cached positions [0, lens[b]) and to the
    drafted rows lens[b] + j that mask[b, i] names.  max_len: about the longest lens (None: the cache's
    length); scale None: 1 / sqrt(head_dim).  Returns out (rows i >= counts[b] as they were)."""
    dev, n, heads = _check_q(view, q)
    if max_len is None:
        max_len = view.max_ctx
    if out is None or scratch is None:
        with _T.cuda.stream(stream):  # what is allocated here belongs to the stream that uses it
            if out is None:
                out = _T.zeros_like(q, memory_format=_T.contiguous_format)
            if scratch is None:
                scratch = tree_attention_scratch(view, n, heads, max_len)
    args = _attention_args(view, q, out, scratch, max_len, scale, _want(mask, "mask", dev, _T.int64, q.shape[:2]), lens, counts)
    _on(dev, stream, "qw_tree_attention", _lib().qw_tree_attention, view._ref, args, scratch.data_ptr(), scratch.nbytes)
    return out


def _check_q(view, q):
    shape, dev = q.shape, view._dev
    if len(shape) != 4 or shape[0] != view.n_seq or shape[3] != view.head_dim or q.stride(3) != 1 or q.get_device() != dev:
        raise ValueError("q must be [n_seq, n, n_heads, head_dim] beside the cache, with a contiguous last dimension")
    return dev, shape[1], shape[2]


def _attention_args(view, q, out, scratch, max_len, scale, mask, lens, counts):
    """The packed qw_tree_attention_args."""
    dev, shape, stride, ostride = view._dev, q.shape, q.stride(), out.stride()
    if out.shape != shape or out.dtype is not q.dtype or out.get_device() != dev or ostride[3] != 1:
        raise ValueError("out must be like q, with a contiguous last dimension")
    if scratch.get_device() != dev or not scratch.is_contiguous():
        raise ValueError("scratch must be contiguous, beside the cache")
    i32 = _T.int32
    return _TREE_ARGS.pack(q.data_ptr(), out.data_ptr(), _dtype_code(q, "q"), shape[1], shape[2], max_len,
                           view.head_dim ** -0.5 if scale is None else scale, stride[0], stride[1], stride[2],
                           ostride[0], ostride[1], ostride[2], mask, _want(lens, "lens", dev, i32, view._per_seq),
                           _want(counts, "counts", dev, i32, view._per_seq))


def prefix_attention_scratch(prefix: KvView, view: KvView, n_max: int, n_heads: int, max_len: int | None = None,
                             max_prefix: int | None = None):
    """Workspace of prefix_attention calls with these sizes (None: the caches' lengths), one call at a time."""
    n = _lib().qw_prefix_attention_scratch_bytes(prefix._ref, view._ref, n_max, n_heads,
                                                 view.max_ctx if max_len is None else max_len,
                                                 prefix.max_ctx if max_prefix is None else max_prefix)
    if n == 0 and n_max:
        raise QwError(UNSUPPORTED_SHAPE, "qw_prefix_attention_scratch_bytes")
    return _T.empty(max(n, 256), dtype=_T.uint8, device=view.device)


def prefix_attention(prefix: KvView, view: KvView, q, lens, prefix_len, mask=None, out=None, counts=None, max_len=None,
                     max_prefix=None, scale=None, scratch=None, stream=None):
    """qw_prefix_attention: tree_attention for sequences that all see the first prefix_len (int32 [1] on the
    device) positions of `prefix`, a view of one sequence, before their own positions in `view`.  mask int64
    [n_seq, n], or None: every row sees itself and the drafted rows before it.  max_len, max_prefix: about the
    longest lens and the prefix's length (None: the caches' lengths).  Returns out."""
    dev, n, heads = _check_q(view, q)
    if prefix._dev != dev:
        raise ValueError("the prefix must be beside the cache")
    if prefix_len is None:
        raise ValueError("prefix_len must be given")
    if max_len is None:
        max_len = view.max_ctx
    if max_prefix is None:
        max_prefix = prefix.max_ctx
    if out is None or scratch is None:
        with _T.cuda.stream(stream):  # what is allocated here belongs to the stream that uses it
            if out is None:
                out = _T.zeros_like(q, memory_format=_T.contiguous_format)
            if scratch is None:
                scratch = prefix_attention_scratch(prefix, view, n, heads, max_len, max_prefix)
    args = _attention_args(view, q, out, scratch, max_len, scale, _want(mask, "mask", dev, _T.int64, q.shape[:2]), lens, counts)
    _on(dev, stream, "qw_prefix_attention", _lib().qw_prefix_attention, prefix._ref, view._ref, args,
        _want(prefix_len, "prefix_len", dev, _T.int32, (1,)), max_prefix, scratch.data_ptr(), scratch.nbytes)
    return out


def process_logits(logits, out=None, *, history=None, history_range=None, path=None, penalties=None, bias_ids=None,
                   bias=None, bias_range=None, mask=None, mask_index=None, stream=None):
    """qw_process_logits: repetition, presence and frequency penalties, biases and grammar masks on
    logits [n_rows, vocab] (contiguous rows); out None works in place.  penalties float32 [n_rows, 3];
    history int32 [n], history_range int32 [n_rows, 2], path int32 [n_rows, p]; bias_ids int32 [m],
    bias float32 [m], bias_range int32 [n_rows, 2]; mask int32 [n_masks, ceil(vocab / 32)],
    mask_index int32 [n_rows].  Returns out."""
    _use_torch()
    shape, stride, dev = logits.shape, logits.stride(), logits.get_device()
    if len(shape) != 2 or dev < 0 or (shape[1] > 1 and stride[1] != 1):
        raise ValueError("logits must be CUDA [n_rows, vocab] with contiguous rows")
    if out is None:
        out, ostride = logits, stride
    else:
        ostride = out.stride()
        if out.shape != shape or out.dtype is not logits.dtype or out.get_device() != dev \
                or (shape[1] > 1 and ostride[1] != 1):
            raise ValueError("out must be like logits, with contiguous rows")
    R, V = shape
    i32, f32 = _T.int32, _T.float32
    if (history is None) != (history_range is None):
        raise ValueError("history and history_range go together")
    if not (bias_ids is None) == (bias is None) == (bias_range is None):
        raise ValueError("bias_ids, bias and bias_range go together")
    if mask_index is not None and mask is None:
        raise ValueError("mask_index needs mask")
    if mask is not None and mask.shape[0] == 0:
        raise ValueError("mask must hold a mask")
    n_hist = 0 if history is None else history.numel()
    n_path = 0 if path is None else path.shape[-1]
    n_bias = 0 if bias is None else bias.numel()
    n_masks = 0 if mask is None else mask.shape[0]
    args = _LOGITS_ARGS.pack(
        logits.data_ptr(), out.data_ptr(), _dtype_code(logits, "logits"), R, V, stride[0], ostride[0],
        _want(penalties, "penalties", dev, f32, (R, 3)), _want(history, "history", dev, i32, (n_hist,)),
        _want(history_range, "history_range", dev, i32, (R, 2)), n_hist, _want(path, "path", dev, i32, (R, n_path)), n_path,
        _want(bias_ids, "bias_ids", dev, i32, (n_bias,)), _want(bias, "bias", dev, f32, (n_bias,)),
        _want(bias_range, "bias_range", dev, i32, (R, 2)), n_bias,
        _want(mask, "mask", dev, i32, (n_masks, (V + 31) // 32)), _want(mask_index, "mask_index", dev, i32, (R,)), n_masks)
    _on(dev, stream, "qw_process_logits", _lib().qw_process_logits, args)
    return out


def sample_rows(logits, u, temperature=None, top_k=None, top_p=None, min_p=None, tokens=None, probs=None, kept=None,
                stream=None):
    """qw_sample_rows: the next token of every row of logits [n_rows, vocab] (float32, float16 or bfloat16, contiguous
    rows), drawn with the given random numbers u float32 [n_rows] of [0, 1).  temperature, top_p, min_p
    float32 [n_rows], top_k int32 [n_rows], on the device; None: 1, 1, 0, 0 (all tokens).  tokens int32
    [n_rows] (None: a new tensor) receives the picks, probs float32 and kept int32 [n_rows], if given, each
    one's probability among the kept tokens and their number.  Returns tokens."""
    _use_torch()
    shape, stride, dev = logits.shape, logits.stride(), logits.get_device()
    if len(shape) != 2 or dev < 0 or (shape[1] > 1 and stride[1] != 1):
        raise ValueError("logits must be CUDA [n_rows, vocab] with contiguous rows")
    if u is None:
        raise ValueError("u must be given")
    i32, f32, per_row = _T.int32, _T.float32, (shape[0],)
    if tokens is None:
        with _T.cuda.stream(stream):  # what is allocated here belongs to the stream that uses it
            tokens = _T.empty(per_row, dtype=i32, device=logits.device)
    args = _SAMPLE_ARGS.pack(
        logits.data_ptr(), _dtype_code(logits, "logits"), shape[0], shape[1], stride[0], _want(u, "u", dev, f32, per_row),
        _want(temperature, "temperature", dev, f32, per_row), _want(top_k, "top_k", dev, i32, per_row),
        _want(top_p, "top_p", dev, f32, per_row), _want(min_p, "min_p", dev, f32, per_row),
        _want(tokens, "tokens", dev, i32, per_row), _want(probs, "probs", dev, f32, per_row),
        _want(kept, "kept", dev, i32, per_row))
    _on(dev, stream, "qw_sample_rows", _lib().qw_sample_rows, args)
    return tokens


class Model:
    """One decoder instance on the current CUDA device and stream."""

    def __init__(self, dims, dev_weights: dict | None, max_ctx: int | None = None, stream=None, table=None):
        """dev_weights: device tensors from weights_to_device; or table = (keep-alive object,
        Weights, layer array) as Checkpoint.upload returns it."""
        import torch

        self.dims = dims
        self.cfg = make_config(dims, max_ctx)
        self.int8 = self.cfg.weight_format in (W_INT8_G32, W_Q8Q8)
        nbytes = workspace_bytes(self.cfg)
        if nbytes == 0:
            raise QwError(UNSUPPORTED_SHAPE, "workspace_bytes")
        self._w = dev_weights if table is None else table
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
        self.stream = stream if stream is not None else torch.cuda.current_stream()
        if table is not None:
            self._layers = table[2]
            h = ctypes.c_void_p()
            _check(_lib().qw_model_create(ctypes.byref(self.cfg), ctypes.byref(table[1]), self.workspace.data_ptr(),
                                          nbytes, self.stream.cuda_stream, ctypes.byref(h)), "qw_model_create")
            self._h = h
            return
        layers = (LayerWeights * self.cfg.n_layers)()
        for l, lw in enumerate(dev_weights["layers"]):
            L = layers[l]
            L.input_norm = lw["input_norm"].data_ptr()
            L.q_norm = lw["q_norm"].data_ptr()
            L.k_norm = lw["k_norm"].data_ptr()
            L.post_norm = lw["post_norm"].data_ptr()
            for j, m in enumerate(MATRICES):
                if self.int8:
                    L.w[j] = lw[m + "_q8"].data_ptr()
                    L.s[j] = lw[m + "_s"].data_ptr()
                else:
                    L.w[j] = lw[m].data_ptr()
        self._layers = layers
        w = Weights(dev_weights["embed"].data_ptr(), dev_weights["final_norm"].data_ptr(), None, layers)
        h = ctypes.c_void_p()
        _check(_lib().qw_model_create(ctypes.byref(self.cfg), ctypes.byref(w), self.workspace.data_ptr(), nbytes,
                                      self.stream.cuda_stream, ctypes.byref(h)), "qw_model_create")
        self._h = h

    # ---------------------------------------------------------------- lifecycle
    def close(self):
        if getattr(self, "_h", None):
            _lib().qw_model_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @property
    def handle(self):
        return self._h

    # ------------------------------------------------------------------- calls
    def prefill(self, tokens, want_token: bool = True):
        t = np.ascontiguousarray(tokens, dtype=np.int32)
        out = ctypes.c_int32(-1)
        _check(_lib().qw_prefill(self._h, t.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)), t.size,
                                 ctypes.byref(out) if want_token else None), "qw_prefill")
        return int(out.value) if want_token else None

    def decode_step(self, token: int = -1, want_token: bool = True):
        out = ctypes.c_int32(-1)
        _check(_lib().qw_decode_step(self._h, int(token), ctypes.byref(out) if want_token else None),
               "qw_decode_step")
        return int(out.value) if want_token else None

    def generate(self, n: int, token: int = -1, tokens_out=None):
        """Greedy n steps with no host sync; tokens_out: device int32 tensor [n] or None."""
        _check(_lib().qw_generate(self._h, int(token), int(n),
                                  tokens_out.data_ptr() if tokens_out is not None else None), "qw_generate")

    def logits(self, out=None):
        import torch
        if out is None:
            out = torch.empty(self.cfg.vocab, dtype=torch.float32, device="cuda")
        _check(_lib().qw_logits(self._h, out.data_ptr(), out.numel()), "qw_logits")
        return out

    def sync(self):
        _check(_lib().qw_sync(self._h), "qw_sync")

    def kv_reset(self):
        _check(_lib().qw_kv_reset(self._h), "qw_kv_reset")

    @property
    def kv_length(self) -> int:
        n = ctypes.c_int32(-1)
        _check(_lib().qw_kv_length(self._h, ctypes.byref(n)), "qw_kv_length")
        return int(n.value)

    def kv_import(self, k, v, n_pos: int):
        _check(_lib().qw_kv_import(self._h, k.data_ptr(), v.data_ptr(), int(n_pos)), "qw_kv_import")

    def kv_export(self, n_pos: int):
        import torch
        c = self.cfg
        shape = (c.n_layers, c.n_kv_heads, n_pos, c.head_dim)
        dt = torch.float32 if c.kv_format == KV_F32 else torch.bfloat16
        k = torch.empty(shape, dtype=dt, device="cuda")
        v = torch.empty(shape, dtype=dt, device="cuda")
        _check(_lib().qw_kv_export(self._h, k.data_ptr(), v.data_ptr(), int(n_pos)), "qw_kv_export")
        return k, v

    def sampler_seed(self, seed: int, stream: int):
        _check(_lib().qw_sampler_seed(self._h, ctypes.c_uint64(seed), ctypes.c_uint64(stream)), "qw_sampler_seed")

    def sampler_state(self):
        out = (ctypes.c_uint64 * 2)()
        _check(_lib().qw_sampler_state(self._h, out), "qw_sampler_state")
        return int(out[0]), int(out[1])

    def sample(self, params: Sampling, history=None, want_token: bool = True):
        """qw_sample: next token from the last position's logits; history: device int32 tensor or None."""
        out = ctypes.c_int32(-1)
        n = 0 if history is None else history.numel()
        _check(_lib().qw_sample(self._h, ctypes.byref(params), history.data_ptr() if n else None, n,
                                ctypes.byref(out) if want_token else None), "qw_sample")
        return int(out.value) if want_token else None

    def set_debug(self, flags: int):
        _check(_lib().qw_set_debug(self._h, int(flags)), "qw_set_debug")

    def query(self, what: int) -> int:
        v = ctypes.c_int64(-1)
        _check(_lib().qw_query(self._h, int(what), ctypes.byref(v)), "qw_query")
        return int(v.value)

    def debug_trace(self):
        """[phase, cta, 16] uint64 ns timeline of the last decode step (needs DEBUG_TRACE)."""
        import torch
        n = self.query(QUERY_TRACE_LEN)
        ncta = self.query(QUERY_DECODE_CTAS)
        out = torch.zeros(n, dtype=torch.int64, device="cuda")
        _check(_lib().qw_debug_trace(self._h, out.data_ptr(), n), "qw_debug_trace")
        return out.view(-1, ncta, 16)

    def debug_hidden(self):
        import torch
        c = self.cfg
        out = torch.empty((c.n_layers + 1, c.hidden), dtype=torch.float32, device="cuda")
        _check(_lib().qw_debug_hidden(self._h, out.data_ptr(), out.numel()), "qw_debug_hidden")
        return out


class Batch:
    """Up to BATCH_MAX sequences of one Model decoded together (qw_batch_*), each with its own
    K/V cache and length; workspace from torch on the model's device.  kv_format: KV_INT8_G32
    for 8-bit caches, None for the model's format."""

    def __init__(self, model: "Model", max_batch: int, max_ctx: int, kv_format: int | None = None):
        import torch

        self.model = model
        self.max_batch = max_batch
        self.max_ctx = max_ctx
        self.kv_format = model.cfg.kv_format if kv_format is None else kv_format
        n = _lib().qw_batch_workspace_bytes_kv(model._h, max_batch, max_ctx, self.kv_format)
        if n == 0:
            raise QwError(INVALID_ARGUMENT, "qw_batch_workspace_bytes_kv")
        self.workspace = torch.empty(n, dtype=torch.uint8, device="cuda")
        h = ctypes.c_void_p()
        _check(_lib().qw_batch_create_kv(model._h, max_batch, max_ctx, self.kv_format, self.workspace.data_ptr(), n,
                                         ctypes.byref(h)), "qw_batch_create_kv")
        self._h = h
        self.last_n = 0

    def close(self):
        if getattr(self, "_h", None):
            _lib().qw_batch_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def reset(self, seq: int = -1):
        _check(_lib().qw_batch_reset(self._h, seq), "qw_batch_reset")

    def length(self, seq: int) -> int:
        out = ctypes.c_int32()
        _check(_lib().qw_batch_length(self._h, seq, ctypes.byref(out)), "qw_batch_length")
        return out.value

    def prefill(self, seq: int, tokens, want_token: bool = True):
        t = (ctypes.c_int32 * len(tokens))(*[int(x) for x in tokens])
        out = ctypes.c_int32(-1)
        _check(_lib().qw_batch_prefill(self._h, seq, t, len(tokens), ctypes.byref(out) if want_token else None),
               "qw_batch_prefill")
        return out.value if want_token else None

    def step(self, n_seq: int, tokens=None, want_tokens: bool = True):
        """One step of sequences 0..n_seq-1; tokens None (or -1 entries) = each one's last pick."""
        t = None if tokens is None else (ctypes.c_int32 * n_seq)(*[int(x) for x in tokens])
        out = (ctypes.c_int32 * n_seq)()
        _check(_lib().qw_batch_step(self._h, n_seq, t, out if want_tokens else None), "qw_batch_step")
        self.last_n = n_seq
        return list(out) if want_tokens else None

    def tree_step(self, seq: int, tokens, parents, want_picks: bool = True):
        """qw_batch_tree_step: drafted tokens of sequence seq in one step (parents[i] < i, -1 = a continuation
        of the cache; tokens[0] = -1: its last pick); the nodes' greedy picks, or None."""
        n = len(tokens)
        if len(parents) != n:
            raise ValueError("tokens and parents must have the same length")
        t = (ctypes.c_int32 * n)(*[int(x) for x in tokens])
        p = (ctypes.c_int32 * n)(*[int(x) for x in parents])
        out = (ctypes.c_int32 * n)()
        _check(_lib().qw_batch_tree_step(self._h, seq, n, t, p, out if want_picks else None), "qw_batch_tree_step")
        self.last_n = n
        return list(out) if want_picks else None

    def tree_accept(self, seq: int, nodes):
        """qw_batch_tree_accept: keep the path `nodes` of the sequence's last tree step."""
        n = len(nodes)
        _check(_lib().qw_batch_tree_accept(self._h, seq, n, (ctypes.c_int32 * n)(*[int(x) for x in nodes]) if n else None),
               "qw_batch_tree_accept")

    def fork(self, src: int, dst: int, n: int | None = None):
        """qw_batch_fork: sequence dst becomes a continuation of the first n positions of src (None: all of them)."""
        _check(_lib().qw_batch_fork(self._h, src, dst, self.length(src) if n is None else n), "qw_batch_fork")

    def sample(self, n_seq: int, u, temperature=None, top_k=None, top_p=None, min_p=None, want_tokens: bool = True):
        """qw_batch_sample: the next tokens of sequences 0..n_seq-1 drawn with the random numbers u (float32 [n_seq] on
        the device, as are the settings; None: sample_rows' defaults), in the place of their greedy picks."""
        _use_torch()
        dev, shape = self.workspace.get_device(), (n_seq,)
        if u is None:
            raise ValueError("u must be given")
        args = [_want(t, name, dev, dt, shape) for t, name, dt in
                ((u, "u", _T.float32), (temperature, "temperature", _T.float32), (top_k, "top_k", _T.int32),
                 (top_p, "top_p", _T.float32), (min_p, "min_p", _T.float32))]
        out = (ctypes.c_int32 * n_seq)()
        _check(_lib().qw_batch_sample(self._h, n_seq, *args, out if want_tokens else None), "qw_batch_sample")
        return list(out) if want_tokens else None

    def logits(self):
        import torch

        V = self.model.cfg.vocab
        out = torch.empty((self.last_n, V), dtype=torch.float32, device="cuda")
        _check(_lib().qw_batch_logits(self._h, out.data_ptr(), out.numel()), "qw_batch_logits")
        return out

    def debug_hidden(self):
        import torch

        c = self.model.cfg
        out = torch.empty((c.n_layers + 1, self.last_n, c.hidden), dtype=torch.float32, device="cuda")
        _check(_lib().qw_batch_debug_hidden(self._h, out.data_ptr(), out.numel()), "qw_batch_debug_hidden")
        return out

    def sync(self):
        _check(_lib().qw_batch_sync(self._h), "qw_batch_sync")


class Checkpoint:
    """A safetensors / SLM2 checkpoint held in host memory (qw_checkpoint_*): `data` is the file's
    bytes (or only its prefix and header, with file_size the whole file's size)."""

    def __init__(self, data, file_size: int | None = None):
        self._buf = bytes(data) if not isinstance(data, (bytes, bytearray)) else data
        self._c = ctypes.create_string_buffer(bytes(self._buf), len(self._buf))
        size = len(self._buf) if file_size is None else file_size
        h = ctypes.c_void_p()
        rc = _lib().qw_checkpoint_open(ctypes.cast(self._c, ctypes.c_void_p), len(self._buf), size, ctypes.byref(h))
        if rc != OK:
            raise QwError(rc, "qw_checkpoint_open: " + _lib().qw_checkpoint_last_error().decode())
        self._h = h

    def close(self):
        if getattr(self, "_h", None):
            _lib().qw_checkpoint_close(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def tensors(self):
        """[(name, dtype, shape, begin, end)] sorted by begin."""
        out = []
        for i in range(_lib().qw_checkpoint_count(self._h)):
            name = ctypes.create_string_buffer(512)
            dt, rk = ctypes.c_int32(), ctypes.c_int32()
            dims = (ctypes.c_int64 * 4)()
            b, e = ctypes.c_uint64(), ctypes.c_uint64()
            _check(_lib().qw_checkpoint_tensor(self._h, i, name, 512, ctypes.byref(dt), ctypes.byref(rk), dims,
                                               ctypes.byref(b), ctypes.byref(e)), "qw_checkpoint_tensor")
            out.append((name.value.decode(), dt.value, tuple(dims[:rk.value]), b.value, e.value))
        return out

    def check(self, cfg: Config):
        """(status, CheckpointReport): status OK when the file matches cfg's tensor set."""
        rep = CheckpointReport()
        rc = _lib().qw_checkpoint_check(self._h, ctypes.byref(cfg), ctypes.byref(rep))
        return rc, rep

    def upload(self, cfg: Config):
        """Device copy of the weights in the layout qw_model_create takes: (workspace tensor, Weights, layers)."""
        import torch

        n = _lib().qw_checkpoint_upload_bytes(self._h, ctypes.byref(cfg))
        if n == 0:
            raise QwError(INVALID_ARGUMENT, "qw_checkpoint_upload_bytes")
        buf = torch.empty(n, dtype=torch.uint8, device="cuda")
        layers = (LayerWeights * cfg.n_layers)()
        table = Weights()
        rc = _lib().qw_checkpoint_upload(self._h, ctypes.byref(cfg), buf.data_ptr(), n, layers, ctypes.byref(table),
                                         torch.cuda.current_stream().cuda_stream)
        if rc != OK:
            raise QwError(rc, "qw_checkpoint_upload: " + _lib().qw_checkpoint_last_error().decode())
        return buf, table, layers
