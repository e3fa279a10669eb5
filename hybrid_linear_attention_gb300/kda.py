"""Python binding of libkda.so (include/kda.h), argument marshalling only.

Each function has the name of the C entry point it calls, takes torch CUDA tensors (or None
for a NULL pointer), checks dtypes/devices/contiguity, passes raw pointers and the current
(or given) CUDA stream, and raises KdaError on a non-OK status.  All arithmetic runs in the
library's CUDA kernels; there is no fallback.  If libkda.so has not been built, loading it
raises immediately.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libkda.so")

KDA_OK, KDA_ERR_INVALID_ARG, KDA_ERR_UNSUPPORTED, KDA_ERR_CUDA, KDA_ERR_WORKSPACE, \
    KDA_ERR_TIMEOUT, KDA_ERR_BAD_INDEX, KDA_ERR_BAD_SEQLENS, KDA_ERR_NO_PAGES = \
    0, -1, -2, -3, -4, -5, -6, -7, -8
KDA_F32, KDA_BF16 = 0, 1

_TORCH_OF = {KDA_F32: torch.float32, KDA_BF16: torch.bfloat16}

EXPORTS = (
    "kda_params_default", "kda_status_string", "kda_state_bytes", "kda_prefill_workspace_size",
    "kda_prologue", "kda_prefill", "kda_prefill_fp8", "kda_prefill_checkpointed",
    "kda_conv_tail_checkpoints", "kda_prefill_host_workspace_size", "kda_prefill_host",
    "kda_prefill_host_plan",
    "kda_decode_step", "kda_conv_state_update", "kda_decode_step_fused",
    "kda_decode_step_fused_fp8", "kda_decode_multi", "kda_state_accept",
    "kda_check_device_error", "kda_launch_count", "kda_trace_ranges", "kda_wait_probe",
    "mla_decode_workspace_size", "mla_set_split_override", "mla_decode_latent",
    "mla_decode_latent_noalloc", "mla_decode",
    "kda_tree_verify", "kda_tree_accept", "mla_tree_mask", "mla_tree_workspace_size",
    "mla_tree_latent", "mla_tree_decode", "mla_cache_append", "mla_cache_accept",
    "mla_pages_copy", "mla_pages_workspace_size", "mla_pages_free", "mla_pages_fork",
    "mla_pages_reserve",
    "mla_tree_latent_lse", "mla_tree_decode_lse", "mla_cache_weights", "mla_weights_accept",
    "mla_cache_evict",
    "mla_pages_trim", "mla_block_keys", "mla_block_scores_workspace_size", "mla_block_scores",
    "mla_block_select", "mla_sparse_workspace_size", "mla_sparse_latent", "mla_sparse_decode",
)


class KdaError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} ({status})")


PREFILL_FORMS = {"auto": 0, "fused": 1, "pair": 2}


class KdaParams(ctypes.Structure):
    _fields_ = [
        ("H", ctypes.c_int), ("d_k", ctypes.c_int), ("d_v", ctypes.c_int),
        ("scale", ctypes.c_float), ("l2_eps", ctypes.c_float), ("norm_eps", ctypes.c_float),
        ("g_min", ctypes.c_float), ("qk_l2norm", ctypes.c_int),
        ("io_dtype", ctypes.c_int), ("state_dtype", ctypes.c_int),
        ("prefill_form", ctypes.c_int),
    ]

    @property
    def io_torch(self):
        return _TORCH_OF[self.io_dtype]

    @property
    def state_torch(self):
        return _TORCH_OF[self.state_dtype]


_lock = threading.Lock()
_lib = None
_vp, _i32, _i64, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
_P = ctypes.POINTER(KdaParams)


def load():
    """Loads libkda.so (built by hybrid_linear_attention_gb300.build.build())."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "hybrid_linear_attention_gb300.build.build() (nvcc, sm_103a)")
        lib = ctypes.CDLL(LIB_PATH)
        sig = {
            "kda_params_default": (None, [_P]),
            "kda_status_string": (ctypes.c_char_p, [_i32]),
            "kda_state_bytes": (_sz, [_P]),
            "kda_prefill_workspace_size": (_sz, [_P, _i32, _i64]),
            "kda_prologue": (_i32, [_P, _vp, _vp, _vp, _vp, _i32, _i64, _i32, _vp, _vp,
                                    _vp, _vp, _vp, _vp, _vp, _vp]),
            "kda_prefill": (_i32, [_P, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i64, _vp, _vp,
                                   _vp, _vp, _vp, _sz, _vp]),
            "kda_prefill_fp8": (_i32, [_P, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i64, _vp,
                                       _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
            "kda_prefill_checkpointed": (_i32, [_P, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32,
                                                _i64, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp,
                                                _vp, _sz, _vp]),
            "kda_conv_tail_checkpoints": (_i32, [_P, _vp, _vp, _vp, _i32, _i64, _vp, _vp, _i32,
                                                 _vp, _vp]),
            "kda_prefill_host_workspace_size": (_sz, [_P, _i32, _i64, _i32]),
            "kda_prefill_host": (_i32, [_P, _vp, _vp, _vp, _vp, _i32, _i64, _vp, _vp, _vp, _vp,
                                        _vp, _vp, _vp, _vp, _sz, _i64, _vp]),
            "kda_prefill_host_plan": (_i64, [_vp, _i32, _i64, _i64, _vp, _i64]),
            "kda_decode_step": (_i32, [_P, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _i32, _vp,
                                       _vp, _vp, _vp]),
            "kda_conv_state_update": (_i32, [_P, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _vp,
                                             _vp]),
            "kda_decode_step_fused": (_i32, [_P, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _i32,
                                             _vp, _vp, _vp, _vp]),
            "kda_decode_step_fused_fp8": (_i32, [_P, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp,
                                                 _i32, _vp, _vp, _vp, _vp, _vp]),
            "kda_decode_multi": (_i32, [_P, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32,
                                        _vp, _vp, _vp, _vp, _i32, _vp]),
            "kda_state_accept": (_i32, [_P, _vp, _i32, _i32, _vp, _vp, _i32, _vp, _vp]),
            "kda_check_device_error": (_i32, [_vp]),
            "kda_launch_count": (ctypes.c_uint64, []),
            "kda_trace_ranges": (_i32, [ctypes.POINTER(ctypes.c_char_p), _i32]),
            "kda_wait_probe": (_i32, [_i64, _vp]),
            "mla_decode_workspace_size": (_sz, [_i32, _i64]),
            "mla_set_split_override": (_i32, [_i32]),
            "mla_decode_latent": (_i32, [_vp, _vp, _i64, _vp, _i32, ctypes.c_float, _vp, _vp,
                                         _sz, _vp]),
            "mla_decode_latent_noalloc": (_i32, [_vp, _vp, _i64, _vp, _i32, ctypes.c_float, _vp,
                                                 _vp]),
            "mla_decode": (_i32, [_vp, _vp, _vp, _vp, _vp, _i64, _vp, _i32, _vp, ctypes.c_float,
                                  _vp, _vp, _vp, _vp, _sz, _vp]),
        }
        tree = [_P, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _vp, _vp, _i32, _i64]
        paged = [_vp, _i32, _i32, _vp, _i32, _vp]  # pool .. lengths of one layer
        layers = [_vp, _i32, _i32, _i32, _vp, _i32, _vp]  # the same of all layers
        sig.update({
            "kda_tree_verify": (_i32, tree + [_i32, _vp, _vp, _vp, _vp]),
            "kda_tree_accept": (_i32, tree + [_vp, _vp]),
            "mla_tree_mask": (_i32, [_vp, _vp, _i32, _i64, _vp, _vp]),
            "mla_tree_workspace_size": (_sz, [_i32, _i64, _i32]),
            "mla_tree_latent": (_i32, [_vp, _i32] + paged + [_vp, _i32, _i64, _vp, ctypes.c_float,
                                                             _vp, _i32, _vp, _sz, _vp]),
            "mla_tree_decode": (_i32, [_vp] * 4 + paged + [_vp, _i32, _i64, _vp, _vp,
                                                           ctypes.c_float, _vp, _vp, _vp, _vp, _sz,
                                                           _vp]),
            "mla_cache_append": (_i32, layers + [_vp, _i32, _i64, _vp, _vp]),
            "mla_cache_accept": (_i32, layers + [_vp, _i32, _i64, _vp, _vp, _vp, _vp]),
            "mla_pages_copy": (_i32, [_vp, _i32, _i32, _i32, _vp, _vp, _i32, _vp]),
            "mla_pages_workspace_size": (_sz, [_i32]),
            "mla_pages_free": (_i32, [_i32, _vp, _vp, _i32, _vp, _vp, _i32, _vp, _i32, _vp]),
            "mla_pages_fork": (_i32, [_vp, _i32, _i32, _i32, _vp, _vp, _i32, _vp, _vp, _i32, _vp,
                                      _vp, _i32, _vp, _sz, _vp]),
            "mla_pages_reserve": (_i32, [_i32, _i32, _vp, _vp, _i32, _vp, _vp, _i32, _vp, _vp,
                                         _i32, _vp, _sz, _vp]),
        })
        f32 = ctypes.c_float
        choice = [_i32, _i32, _i32, _vp, _i64, _vp, _i32, _vp]  # blocks .. sel_lengths
        sig.update({
            "mla_tree_latent_lse": (_i32, [_vp, _i32] + paged + [_vp, _i32, _i64, _vp, f32, _vp,
                                                                 _i32, _vp, _vp, _sz, _vp]),
            "mla_tree_decode_lse": (_i32, [_vp] * 4 + paged + [_vp, _i32, _i64, _vp, _vp, f32] +
                                    [_vp] * 5 + [_sz, _vp]),
            "mla_cache_weights": (_i32, [_vp, _i32] + paged + [_vp, _i32, _i64, _vp, _vp, _vp,
                                                               f32, _vp, _i64, _vp]),
            "mla_weights_accept": (_i32, [_vp, _i64, _vp, _vp, _i32, _i64, _vp, _vp, _vp]),
            "mla_cache_evict": (_i32, layers + [_vp, _i32, _vp, _i64, _i32, _i32, _i32, _vp, _vp,
                                                _vp, _vp]),
            "mla_pages_trim": (_i32, [_i32, _i32, _vp, _vp, _i32, _vp, _vp, _i32, _vp, _i32, _vp]),
            "mla_block_keys": (_i32, [_vp, _i32, _i32, _i32, _vp, _i32, _vp, _vp, _i32, _vp, _vp]),
            "mla_block_scores_workspace_size": (_sz, [_i64, _i32, _i32]),
            "mla_block_scores": (_i32, [_vp, _i32] + paged + [_vp, _i32, _i64, f32, _vp, _i64, _vp,
                                                              _sz, _vp]),
            "mla_block_select": (_i32, [_vp, _i64, _i32, _vp, _i32, _vp, _vp, _i32, _i64, _i32,
                                        _i32, _i32, _vp, _i32, _vp, _vp]),
            "mla_sparse_workspace_size": (_sz, [_i32, _i64, _i32, _i32]),
            "mla_sparse_latent": (_i32, [_vp, _i32, _vp] + paged + [_vp, _i32, _i64, _vp, f32] +
                                  choice + [_vp, _i32, _vp, _sz, _vp]),
            "mla_sparse_decode": (_i32, [_vp] * 5 + paged + [_vp, _i32, _i64, _vp, _vp, f32] +
                                  choice + [_vp, _vp, _vp, _vp, _sz, _vp]),
        })
        for name, (res, args) in sig.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
        return lib


def status_string(status):
    try:
        return load().kda_status_string(int(status)).decode()
    except Exception:  # the library itself failed to load
        return f"status {status}"


def _check(status, where):
    if status != KDA_OK:
        raise KdaError(status, where)


def params(H=64, d=128, *, scale=1.0, l2_eps=1e-6, norm_eps=1e-6, g_min=-5.0, qk_l2norm=True,
           io_dtype=torch.bfloat16, state_dtype=torch.float32, prefill_form="auto"):
    """Builds a kda_params struct (defaults: the pages' configuration).  prefill_form:
    "auto", "fused" or "pair" (the tensor-core prefill's kernel form)."""
    code = {torch.float32: KDA_F32, torch.bfloat16: KDA_BF16}
    return KdaParams(H=H, d_k=d, d_v=d, scale=scale, l2_eps=l2_eps, norm_eps=norm_eps,
                     g_min=g_min, qk_l2norm=1 if qk_l2norm else 0,
                     io_dtype=code[io_dtype], state_dtype=code[state_dtype],
                     prefill_form=PREFILL_FORMS[prefill_form])


def kda_params_default():
    p = KdaParams()
    load().kda_params_default(ctypes.byref(p))
    return p


_Tensor = torch.Tensor


def _ptr(t, dtype=None, name="tensor"):
    if t is None:
        return None
    if (isinstance(t, _Tensor) and t.is_cuda and t.is_contiguous()
            and (dtype is None or t.dtype == dtype)):
        return t.data_ptr()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch tensor or None")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor (device pointer)")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    return t.data_ptr()


def _hptr(t, dtype=None, name="tensor"):
    """Host pointer of a CPU tensor (page-locked memory lets the library overlap its copies)."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch tensor or None")
    if t.is_cuda:
        raise ValueError(f"{name}: must be a host (CPU) tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    return t.data_ptr()


# the current stream's handle without a Stream object (which costs more than a launch)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    if stream is None and _raw_stream is not None:
        return _raw_stream(torch.cuda.current_device())
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream if hasattr(s, "cuda_stream") else int(s)


def kda_state_bytes(p):
    return int(load().kda_state_bytes(ctypes.byref(p)))


def kda_prefill_workspace_size(p, n_seqs, total_tokens):
    return int(load().kda_prefill_workspace_size(ctypes.byref(p), int(n_seqs), int(total_tokens)))


def kda_launch_count():
    return int(load().kda_launch_count())


def kda_wait_probe(probes, stream=None):
    _check(load().kda_wait_probe(int(probes), _stream(stream)), "kda_wait_probe")


def kda_check_device_error(stream=None):
    _check(load().kda_check_device_error(_stream(stream)), "kda_check_device_error")


def kda_prologue(p, x_raw, conv_w, conv_state, cu_seqlens, q, k, v, *, l2norm_qk=False,
                 beta_logit=None, g_raw=None, beta=None, g=None, stream=None):
    io = p.io_torch
    st = load().kda_prologue(
        ctypes.byref(p), _ptr(x_raw, io, "x_raw"), _ptr(conv_w, io, "conv_w"),
        _ptr(conv_state, io, "conv_state"), _ptr(cu_seqlens, torch.int32, "cu_seqlens"),
        cu_seqlens.numel() - 1, x_raw.shape[0], 1 if l2norm_qk else 0,
        _ptr(beta_logit, torch.float32, "beta_logit"), _ptr(g_raw, torch.float32, "g_raw"),
        _ptr(q, io, "q"), _ptr(k, io, "k"), _ptr(v, io, "v"),
        _ptr(beta, torch.float32, "beta"), _ptr(g, torch.float32, "g"), _stream(stream))
    _check(st, "kda_prologue")


def kda_prefill(p, q, k, v, g, beta, cu_seqlens, out, *, init_state=None, final_state=None,
                gate_logit=None, norm_w=None, workspace=None, stream=None):
    io, sd = p.io_torch, p.state_torch
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = load().kda_prefill(
        ctypes.byref(p), _ptr(q, io, "q"), _ptr(k, io, "k"), _ptr(v, io, "v"),
        _ptr(g, torch.float32, "g"), _ptr(beta, torch.float32, "beta"),
        _ptr(init_state, sd, "init_state"), _ptr(cu_seqlens, torch.int32, "cu_seqlens"),
        cu_seqlens.numel() - 1, q.shape[0], _ptr(gate_logit, io, "gate_logit"),
        _ptr(norm_w, torch.float32, "norm_w"), _ptr(out, io, "out"),
        _ptr(final_state, sd, "final_state"), _ptr(workspace, None, "workspace"), ws_bytes,
        _stream(stream))
    _check(st, "kda_prefill")


def kda_prefill_host_workspace_size(p, n_seqs, segment_tokens, with_gate=False):
    return int(load().kda_prefill_host_workspace_size(ctypes.byref(p), int(n_seqs),
                                                       int(segment_tokens), 1 if with_gate else 0))


def kda_prefill_host_plan(cu_seqlens, segment_tokens):
    """Row boundaries of the segments kda_prefill_host cuts a batch into (cu_seqlens: a CPU
    int32 tensor); a list [0, b_1, ..., total_tokens]."""
    cu = cu_seqlens.to(torch.int32).contiguous()
    n, T = cu.numel() - 1, int(cu[-1])
    k = load().kda_prefill_host_plan(_hptr(cu, torch.int32, "cu_seqlens"), n, T,
                                     int(segment_tokens), None, 0)
    if k < 0:
        raise KdaError(KDA_ERR_INVALID_ARG, "kda_prefill_host_plan")
    bounds = (ctypes.c_int64 * (k + 1))()
    load().kda_prefill_host_plan(_hptr(cu, torch.int32, "cu_seqlens"), n, T,
                                 int(segment_tokens), bounds, k)
    return [int(b) for b in bounds] if k > 0 else [0]


def kda_prefill_host(p, x_raw, conv_w, conv_state, cu_seqlens, beta_logit, g_raw, out, *,
                     workspace, segment_tokens=512, init_state=None, final_state=None,
                     gate_logit=None, norm_w=None, stream=None):
    """Prologue + prefill of a packed batch in host memory, streamed through the GPU in
    segments: x_raw, conv_state (in/out or None), cu_seqlens (int32), beta_logit, g_raw,
    init_state, gate_logit, out and final_state are CPU tensors (pinned for overlap); conv_w,
    norm_w and the uint8 workspace are CUDA tensors.  The outputs are in host memory once
    `stream` (default: the current stream) has been synchronised."""
    io = p.io_torch
    st = load().kda_prefill_host(
        ctypes.byref(p), _hptr(x_raw, io, "x_raw"), _ptr(conv_w, io, "conv_w"),
        _hptr(conv_state, io, "conv_state"), _hptr(cu_seqlens, torch.int32, "cu_seqlens"),
        cu_seqlens.numel() - 1, x_raw.shape[0], _hptr(beta_logit, torch.float32, "beta_logit"),
        _hptr(g_raw, torch.float32, "g_raw"), _hptr(init_state, torch.float32, "init_state"),
        _hptr(gate_logit, io, "gate_logit"), _ptr(norm_w, torch.float32, "norm_w"),
        _hptr(out, io, "out"), _hptr(final_state, torch.float32, "final_state"),
        *_ws(workspace), int(segment_tokens), _stream(stream))
    _check(st, "kda_prefill_host")


def kda_prefill_fp8(p, q, k, v, g, beta, cu_seqlens, out_q, out_scale, *, init_state=None,
                    final_state=None, gate_logit=None, norm_w=None, workspace=None, stream=None):
    """out_q [T, H, d] uint8 E4M3 codes, out_scale [T, H] fp32 (one group per token, head)."""
    io, sd = p.io_torch, p.state_torch
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = load().kda_prefill_fp8(
        ctypes.byref(p), _ptr(q, io, "q"), _ptr(k, io, "k"), _ptr(v, io, "v"),
        _ptr(g, torch.float32, "g"), _ptr(beta, torch.float32, "beta"),
        _ptr(init_state, sd, "init_state"), _ptr(cu_seqlens, torch.int32, "cu_seqlens"),
        cu_seqlens.numel() - 1, q.shape[0], _ptr(gate_logit, io, "gate_logit"),
        _ptr(norm_w, torch.float32, "norm_w"), _ptr(out_q, torch.uint8, "out_q"),
        _ptr(out_scale, torch.float32, "out_scale"), _ptr(final_state, sd, "final_state"),
        _ptr(workspace, None, "workspace"), ws_bytes, _stream(stream))
    _check(st, "kda_prefill_fp8")


def kda_prefill_checkpointed(p, q, k, v, g, beta, cu_seqlens, out, ckpt_cu, ckpt_pos,
                             ckpt_states, *, init_state=None, final_state=None, gate_logit=None,
                             norm_w=None, workspace=None, stream=None):
    io, sd = p.io_torch, p.state_torch
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = load().kda_prefill_checkpointed(
        ctypes.byref(p), _ptr(q, io, "q"), _ptr(k, io, "k"), _ptr(v, io, "v"),
        _ptr(g, torch.float32, "g"), _ptr(beta, torch.float32, "beta"),
        _ptr(init_state, sd, "init_state"), _ptr(cu_seqlens, torch.int32, "cu_seqlens"),
        cu_seqlens.numel() - 1, q.shape[0], _ptr(gate_logit, io, "gate_logit"),
        _ptr(norm_w, torch.float32, "norm_w"), _ptr(out, io, "out"),
        _ptr(final_state, sd, "final_state"), _ptr(ckpt_cu, torch.int32, "ckpt_cu"),
        _ptr(ckpt_pos, torch.int32, "ckpt_pos"), ckpt_pos.numel(),
        _ptr(ckpt_states, sd, "ckpt_states"), _ptr(workspace, None, "workspace"), ws_bytes,
        _stream(stream))
    _check(st, "kda_prefill_checkpointed")


def kda_conv_tail_checkpoints(p, x_raw, conv_state, cu_seqlens, ckpt_cu, ckpt_pos, conv_ckpt, *,
                              stream=None):
    io = p.io_torch
    st = load().kda_conv_tail_checkpoints(
        ctypes.byref(p), _ptr(x_raw, io, "x_raw"), _ptr(conv_state, io, "conv_state"),
        _ptr(cu_seqlens, torch.int32, "cu_seqlens"), cu_seqlens.numel() - 1, x_raw.shape[0],
        _ptr(ckpt_cu, torch.int32, "ckpt_cu"), _ptr(ckpt_pos, torch.int32, "ckpt_pos"),
        ckpt_pos.numel(), _ptr(conv_ckpt, io, "conv_ckpt"), _stream(stream))
    _check(st, "kda_conv_tail_checkpoints")


def kda_decode_step(p, q, k, v, g, beta, state, out, *, slot_idx=None, gate_logit=None,
                    norm_w=None, stream=None):
    io, sd = p.io_torch, p.state_torch
    st = load().kda_decode_step(
        ctypes.byref(p), _ptr(q, io, "q"), _ptr(k, io, "k"), _ptr(v, io, "v"),
        _ptr(g, torch.float32, "g"), _ptr(beta, torch.float32, "beta"),
        _ptr(state, sd, "state"), state.shape[0], _ptr(slot_idx, torch.int32, "slot_idx"),
        q.shape[0], _ptr(gate_logit, io, "gate_logit"), _ptr(norm_w, torch.float32, "norm_w"),
        _ptr(out, io, "out"), _stream(stream))
    _check(st, "kda_decode_step")


def kda_decode_step_fused(p, x_raw, conv_w, conv_state, g, beta, state, out, *, slot_idx=None,
                          gate_logit=None, norm_w=None, stream=None):
    io, sd = p.io_torch, p.state_torch
    st = load().kda_decode_step_fused(
        ctypes.byref(p), _ptr(x_raw, io, "x_raw"), _ptr(conv_w, io, "conv_w"),
        _ptr(conv_state, io, "conv_state"), _ptr(g, torch.float32, "g"),
        _ptr(beta, torch.float32, "beta"), _ptr(state, sd, "state"), state.shape[0],
        _ptr(slot_idx, torch.int32, "slot_idx"), x_raw.shape[0],
        _ptr(gate_logit, io, "gate_logit"), _ptr(norm_w, torch.float32, "norm_w"),
        _ptr(out, io, "out"), _stream(stream))
    _check(st, "kda_decode_step_fused")


def kda_decode_step_fused_fp8(p, x_raw, conv_w, conv_state, g, beta, state, out_q, out_scale, *,
                              slot_idx=None, gate_logit=None, norm_w=None, stream=None):
    """out_q [n_seqs, H, d] uint8 E4M3 codes, out_scale [n_seqs, H] fp32."""
    io, sd = p.io_torch, p.state_torch
    st = load().kda_decode_step_fused_fp8(
        ctypes.byref(p), _ptr(x_raw, io, "x_raw"), _ptr(conv_w, io, "conv_w"),
        _ptr(conv_state, io, "conv_state"), _ptr(g, torch.float32, "g"),
        _ptr(beta, torch.float32, "beta"), _ptr(state, sd, "state"), state.shape[0],
        _ptr(slot_idx, torch.int32, "slot_idx"), x_raw.shape[0],
        _ptr(gate_logit, io, "gate_logit"), _ptr(norm_w, torch.float32, "norm_w"),
        _ptr(out_q, torch.uint8, "out_q"), _ptr(out_scale, torch.float32, "out_scale"),
        _stream(stream))
    _check(st, "kda_decode_step_fused_fp8")


def kda_decode_multi(p, q, k, v, g, beta, state, out, K, *, slot_idx=None, gate_logit=None,
                     norm_w=None, step_states=None, commit_final=False, stream=None):
    """K tokens per sequence: q, k, v, g, beta, out, gate_logit have n_seqs * K rows."""
    io, sd = p.io_torch, p.state_torch
    if q.shape[0] % K:
        raise ValueError("rows must be n_seqs * K")
    st = load().kda_decode_multi(
        ctypes.byref(p), _ptr(q, io, "q"), _ptr(k, io, "k"), _ptr(v, io, "v"),
        _ptr(g, torch.float32, "g"), _ptr(beta, torch.float32, "beta"),
        _ptr(state, sd, "state"), state.shape[0], _ptr(slot_idx, torch.int32, "slot_idx"),
        q.shape[0] // K, K, _ptr(gate_logit, io, "gate_logit"),
        _ptr(norm_w, torch.float32, "norm_w"), _ptr(out, io, "out"),
        _ptr(step_states, sd, "step_states"), 1 if commit_final else 0, _stream(stream))
    _check(st, "kda_decode_multi")


def kda_state_accept(p, step_states, accept_len, state, K, *, slot_idx=None, stream=None):
    sd = p.state_torch
    st = load().kda_state_accept(
        ctypes.byref(p), _ptr(step_states, sd, "step_states"), accept_len.shape[0], K,
        _ptr(accept_len, torch.int32, "accept_len"), _ptr(state, sd, "state"), state.shape[0],
        _ptr(slot_idx, torch.int32, "slot_idx"), _stream(stream))
    _check(st, "kda_state_accept")


def kda_conv_state_update(p, x_new, conv_w, conv_state, y, *, slot_idx=None, stream=None):
    io = p.io_torch
    st = load().kda_conv_state_update(
        ctypes.byref(p), _ptr(x_new, io, "x_new"), _ptr(conv_w, io, "conv_w"),
        _ptr(conv_state, io, "conv_state"), conv_state.shape[0],
        _ptr(slot_idx, torch.int32, "slot_idx"), x_new.shape[0], x_new.shape[1],
        _ptr(y, io, "y"), _stream(stream))
    _check(st, "kda_conv_state_update")


# ---- absorbed gated-MLA decode (mla.h) -----------------------------------------------------

MLA_SCALE = 192 ** -0.5


def kda_trace_ranges():
    """Names of the NVTX ranges the library opens around its calls."""
    lib = load()
    n = lib.kda_trace_ranges(None, 0)
    arr = (ctypes.c_char_p * n)()
    lib.kda_trace_ranges(arr, n)
    return [x.decode() for x in arr]


def mla_decode_workspace_size(n_seqs, cache_len):
    return int(load().mla_decode_workspace_size(int(n_seqs), int(cache_len)))


def mla_set_split_override(n_split):
    """Tuning and testing only: force the MLA split count (0 = the automatic rule)."""
    _check(load().mla_set_split_override(int(n_split)), "mla_set_split_override")


class mla_split:
    """Context manager: the MLA split count forced to n inside the block."""

    def __init__(self, n):
        self.n = n

    def __enter__(self):
        mla_set_split_override(self.n)

    def __exit__(self, *exc):
        mla_set_split_override(0)


def _ws(workspace):
    return (_ptr(workspace, None, "workspace"),
            workspace.numel() * workspace.element_size() if workspace is not None else 0)


def mla_decode_latent(q_cat, cache, lengths, z, *, scale=MLA_SCALE, workspace=None, stream=None):
    """q_cat [B,64,576] bf16, cache [B,L,576] bf16, lengths [B] int32, z [B,64,512] fp32."""
    st = load().mla_decode_latent(
        _ptr(q_cat, torch.bfloat16, "q_cat"), _ptr(cache, torch.bfloat16, "cache"),
        cache.shape[1], _ptr(lengths, torch.int32, "lengths"), q_cat.shape[0], float(scale),
        _ptr(z, torch.float32, "z"), *_ws(workspace), _stream(stream))
    _check(st, "mla_decode_latent")


def mla_decode_latent_noalloc(q_cat, cache, lengths, z, *, scale=MLA_SCALE, stream=None):
    """mla_decode_latent with its split scratch in the library's fixed device buffer."""
    st = load().mla_decode_latent_noalloc(
        _ptr(q_cat, torch.bfloat16, "q_cat"), _ptr(cache, torch.bfloat16, "cache"),
        cache.shape[1], _ptr(lengths, torch.int32, "lengths"), q_cat.shape[0], float(scale),
        _ptr(z, torch.float32, "z"), _stream(stream))
    _check(st, "mla_decode_latent_noalloc")


def mla_decode(q_nope, q_rope, w_uk, w_uv, cache, lengths, gate_logit, q_cat, z, out, *,
               scale=MLA_SCALE, workspace=None, stream=None):
    """One absorbed gated-MLA decode step; q_cat and z are caller-owned intermediates."""
    bf = torch.bfloat16
    st = load().mla_decode(
        _ptr(q_nope, bf, "q_nope"), _ptr(q_rope, bf, "q_rope"), _ptr(w_uk, bf, "w_uk"),
        _ptr(w_uv, bf, "w_uv"), _ptr(cache, bf, "cache"), cache.shape[1],
        _ptr(lengths, torch.int32, "lengths"), q_nope.shape[0], _ptr(gate_logit, bf, "gate_logit"),
        float(scale), _ptr(q_cat, bf, "q_cat"), _ptr(z, torch.float32, "z"), _ptr(out, bf, "out"),
        *_ws(workspace), _stream(stream))
    _check(st, "mla_decode")


# ---- verifying a tree of drafted tokens -------------------------------------------------------

_get_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _device():
    try:
        return _get_device()
    except RuntimeError:  # no device: no tensor is on it
        return -2


def _here(t, dtype, name, dev):
    """_ptr, of tensors on device `dev`, the current one, only: the launch goes to its stream."""
    if t is None:
        return None
    try:
        if t.get_device() == dev and t.dtype is dtype and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    p = _ptr(t, dtype, name)
    if t.get_device() != dev:
        raise ValueError(f"{name}: on {t.device}, but the current device is cuda:{dev}")
    return p


def _here_stream(stream, dev):
    return _raw_stream(dev) if stream is None and _raw_stream is not None else _stream(stream)


def _here_ws(t, dev):
    return (None, 0) if t is None else (_here(t, t.dtype, "workspace", dev), t.nbytes)


def _shape(t, shape, name):
    if t is not None and t.shape != shape:
        raise ValueError(f"{name}: expected shape {list(shape)}, got {list(t.shape)}")


def _tree_args(p, x_raw, conv_w, conv_state, g, beta, state, cu_nodes, parent, slot_idx,
               dev):
    io, i32, f32 = p.io_torch, torch.int32, torch.float32
    total, H, d, n = parent.shape[0], p.H, p.d_k, cu_nodes.numel() - 1
    _shape(x_raw, (total, 3 * H * d), "x_raw")
    _shape(conv_w, (3 * H * d, 4), "conv_w")
    _shape(conv_state, (state.shape[0], 3, 3 * H * d), "conv_state")
    _shape(g, (total, H, d), "g")
    _shape(beta, (total, H), "beta")
    _shape(state, (state.shape[0], H, d, d), "state")
    _shape(slot_idx, (n,), "slot_idx")
    return [ctypes.byref(p), _here(x_raw, io, "x_raw", dev), _here(conv_w, io, "conv_w", dev),
            _here(conv_state, io, "conv_state", dev), _here(g, f32, "g", dev),
            _here(beta, f32, "beta", dev), _here(state, p.state_torch, "state", dev),
            state.shape[0], _here(slot_idx, i32, "slot_idx", dev),
            _here(cu_nodes, i32, "cu_nodes", dev), _here(parent, i32, "parent", dev), n, total]


def kda_tree_verify(p, x_raw, conv_w, conv_state, g, beta, state, cu_nodes, parent, out, *,
                    max_nodes=64, slot_idx=None, gate_logit=None, norm_w=None, stream=None):
    """Outputs of every node of the drafted trees: x_raw [nodes, 3*H*d], g [nodes, H, d], beta
    [nodes, H], parent [nodes] and out [nodes, H, d] packed by cu_nodes [n_seqs + 1]; the pool
    state and the conv tails are only read.  max_nodes: the most nodes of any sequence; name it where
    the trees are small (trees of 8 nodes run four times as fast with 8 as with 64)."""
    dev = _device()
    io = p.io_torch
    args = _tree_args(p, x_raw, conv_w, conv_state, g, beta, state, cu_nodes, parent, slot_idx,
                      dev)
    _shape(out, g.shape, "out")
    _shape(gate_logit, g.shape, "gate_logit")
    _shape(norm_w, (p.d_k,), "norm_w")
    st = load().kda_tree_verify(*args, int(max_nodes), _here(gate_logit, io, "gate_logit", dev),
                                _here(norm_w, torch.float32, "norm_w", dev),
                                _here(out, io, "out", dev), _here_stream(stream, dev))
    _check(st, "kda_tree_verify")


def kda_tree_accept(p, x_raw, conv_w, conv_state, g, beta, state, cu_nodes, parent, accept_node, *,
                    slot_idx=None, stream=None):
    """The path to accept_node [n_seqs] (-1: none) replayed into the pool state and conv tail."""
    dev = _device()
    args = _tree_args(p, x_raw, conv_w, conv_state, g, beta, state, cu_nodes, parent, slot_idx,
                      dev)
    _shape(accept_node, (cu_nodes.numel() - 1,), "accept_node")
    st = load().kda_tree_accept(*args, _here(accept_node, torch.int32, "accept_node", dev),
                                _here_stream(stream, dev))
    _check(st, "kda_tree_accept")


def mla_tree_mask(parent, cu_nodes, mask, *, stream=None):
    """mask [nodes] int64: bit j = the node itself or its ancestor j, from parent [nodes]."""
    dev = _device()
    _shape(mask, parent.shape, "mask")
    st = load().mla_tree_mask(_here(parent, torch.int32, "parent", dev),
                              _here(cu_nodes, torch.int32, "cu_nodes", dev), cu_nodes.numel() - 1,
                              parent.shape[0], _here(mask, torch.int64, "mask", dev),
                              _here_stream(stream, dev))
    _check(st, "mla_tree_mask")


def mla_tree_workspace_size(n_seqs, total_nodes, H=64):
    return int(load().mla_tree_workspace_size(int(n_seqs), int(total_nodes), int(H)))


def _paged(pool, page_table, lengths, n_seqs, dev):
    """pool .. lengths of one layer ([n_pages, page_size, 576])."""
    shape = pool.shape
    if len(shape) != 3 or shape[2] != 576:
        raise ValueError("pool: expected [n_pages, page_size, 576]")
    rows, max_pages = page_table.shape
    if rows < n_seqs or lengths.shape[0] < n_seqs:
        raise ValueError("page_table, lengths: fewer rows than sequences")
    return [_here(pool, torch.bfloat16, "pool", dev), shape[0], shape[1],
            _here(page_table, torch.int32, "page_table", dev), max_pages,
            _here(lengths, torch.int32, "lengths", dev)]


def _paged_layers(pool, page_table, lengths, n_seqs, dev):
    """pool .. lengths of all layers ([n_layers, n_pages, page_size, 576])."""
    shape = pool.shape
    if len(shape) != 4 or shape[3] != 576:
        raise ValueError("pool: expected [n_layers, n_pages, page_size, 576]")
    rows, max_pages = page_table.shape
    if rows < n_seqs or lengths.shape[0] < n_seqs:
        raise ValueError("page_table, lengths: fewer rows than sequences")
    return [_here(pool, torch.bfloat16, "pool", dev), shape[0], shape[1], shape[2],
            _here(page_table, torch.int32, "page_table", dev), max_pages,
            _here(lengths, torch.int32, "lengths", dev)]


_DTYPE = {torch.float32: KDA_F32, torch.bfloat16: KDA_BF16}


def mla_tree_latent(q_cat, pool, page_table, lengths, cu_nodes, z, *, mask=None, scale=MLA_SCALE,
                    workspace=None, stream=None):
    """q_cat [nodes, H, 576] bf16, pool [n_pages, page_size, 576] bf16, page_table [n_seqs,
    max_pages], lengths [n_seqs], cu_nodes [n_seqs + 1], z [nodes, H, 512] fp32 or bf16, mask
    [nodes] int64 (None: a chain), workspace of mla_tree_workspace_size bytes."""
    dev = _device()
    total, H, n = q_cat.shape[0], q_cat.shape[1], cu_nodes.numel() - 1
    _shape(q_cat, (total, H, 576), "q_cat")
    _shape(z, (total, H, 512), "z")
    _shape(mask, (total,), "mask")
    if z.dtype not in _DTYPE:
        raise TypeError(f"z: expected float32 or bfloat16, got {z.dtype}")
    cache = _paged(pool, page_table, lengths, n, dev)
    st = load().mla_tree_latent(
        _here(q_cat, torch.bfloat16, "q_cat", dev), H, *cache,
        _here(cu_nodes, torch.int32, "cu_nodes", dev), n, total,
        _here(mask, torch.int64, "mask", dev), float(scale), _here(z, z.dtype, "z", dev),
        _DTYPE[z.dtype], *_here_ws(workspace, dev), _here_stream(stream, dev))
    _check(st, "mla_tree_latent")


def mla_tree_decode(q_nope, q_rope, w_uk, w_uv, pool, page_table, lengths, cu_nodes, gate_logit,
                    q_cat, z, out, *, mask=None, scale=MLA_SCALE, workspace=None, stream=None):
    """One absorbed gated-MLA step for the nodes of drafted trees; q_cat and z are caller-owned
    intermediates."""
    dev = _device()
    bf = torch.bfloat16
    total, n = q_nope.shape[0], cu_nodes.numel() - 1
    for t, tail, name in ((q_nope, (64, 128), "q_nope"), (q_rope, (64, 64), "q_rope"),
                          (gate_logit, (64,), "gate_logit"), (q_cat, (64, 576), "q_cat"),
                          (z, (64, 512), "z"), (out, (64, 128), "out")):
        _shape(t, (total,) + tail, name)
    _shape(w_uk, (64, 128, 512), "w_uk")
    _shape(w_uv, (64, 128, 512), "w_uv")
    _shape(mask, (total,), "mask")
    st = load().mla_tree_decode(
        _here(q_nope, bf, "q_nope", dev), _here(q_rope, bf, "q_rope", dev),
        _here(w_uk, bf, "w_uk", dev), _here(w_uv, bf, "w_uv", dev),
        *_paged(pool, page_table, lengths, n, dev), _here(cu_nodes, torch.int32, "cu_nodes", dev),
        n, total, _here(mask, torch.int64, "mask", dev), _here(gate_logit, bf, "gate_logit", dev),
        float(scale), _here(q_cat, bf, "q_cat", dev), _here(z, torch.float32, "z", dev),
        _here(out, bf, "out", dev), *_here_ws(workspace, dev), _here_stream(stream, dev))
    _check(st, "mla_tree_decode")


def mla_cache_append(pool, page_table, lengths, cu_rows, rows, *, stream=None):
    """rows [n_layers, total, 576] written behind each sequence in pool [n_layers, n_pages,
    page_size, 576]; lengths stay."""
    dev = _device()
    n = cu_rows.numel() - 1
    _shape(rows, (pool.shape[0], rows.shape[1], 576), "rows")
    st = load().mla_cache_append(
        *_paged_layers(pool, page_table, lengths, n, dev),
        _here(cu_rows, torch.int32, "cu_rows", dev), n, rows.shape[1],
        _here(rows, torch.bfloat16, "rows", dev), _here_stream(stream, dev))
    _check(st, "mla_cache_append")


def mla_cache_accept(pool, page_table, lengths, cu_nodes, parent, accept_node, new_lengths, *,
                     stream=None):
    """The accepted paths' rows compacted; new_lengths [n_seqs] may be lengths."""
    dev = _device()
    n, i32 = cu_nodes.numel() - 1, torch.int32
    _shape(accept_node, (n,), "accept_node")
    if new_lengths.shape[0] < n:
        raise ValueError("new_lengths: fewer rows than sequences")
    st = load().mla_cache_accept(
        *_paged_layers(pool, page_table, lengths, n, dev), _here(cu_nodes, i32, "cu_nodes", dev),
        n, parent.shape[0], _here(parent, i32, "parent", dev),
        _here(accept_node, i32, "accept_node", dev),
        _here(new_lengths, i32, "new_lengths", dev), _here_stream(stream, dev))
    _check(st, "mla_cache_accept")


def mla_pages_copy(pool, src, dst, *, stream=None):
    """Pages src[i] copied to dst[i] in every layer of pool [n_layers, n_pages, page_size, 576]."""
    dev = _device()
    _shape(pool, (pool.shape[0], pool.shape[1], pool.shape[2], 576), "pool")
    _shape(dst, src.shape, "dst")
    st = load().mla_pages_copy(_here(pool, torch.bfloat16, "pool", dev), *pool.shape[:3],
                               _here(src, torch.int32, "src", dev),
                               _here(dst, torch.int32, "dst", dev), src.numel(), _here_stream(stream, dev))
    _check(st, "mla_pages_copy")


def mla_pages_workspace_size(n):
    return int(load().mla_pages_workspace_size(int(n)))


def _book(refcount, page_table, held, lengths, dev):
    i32 = torch.int32
    n_slots, max_pages = page_table.shape
    if held.shape != (n_slots,) or lengths.shape != (n_slots,):
        raise ValueError(f"held, lengths: expected shape [{n_slots}]")
    return (_here(refcount, i32, "refcount", dev), _here(page_table, i32, "page_table", dev),
            max_pages, _here(held, i32, "held", dev), _here(lengths, i32, "lengths", dev), n_slots)


def mla_pages_free(refcount, page_table, held, lengths, slots, *, stream=None):
    """All pages of the sequences in slots released."""
    dev = _device()
    st = load().mla_pages_free(refcount.numel(), *_book(refcount, page_table, held, lengths, dev),
                               _here(slots, torch.int32, "slots", dev), slots.numel(),
                               _here_stream(stream, dev))
    _check(st, "mla_pages_free")


def mla_pages_fork(pool, refcount, page_table, held, lengths, src, dst, *, workspace=None,
                   stream=None):
    """Sequences dst become copies of src: full pages shared, a partly filled last one copied."""
    dev = _device()
    i32 = torch.int32
    _shape(pool, (pool.shape[0], refcount.numel(), pool.shape[2], 576), "pool")
    _shape(dst, src.shape, "dst")
    st = load().mla_pages_fork(
        _here(pool, torch.bfloat16, "pool", dev), *pool.shape[:3],
        *_book(refcount, page_table, held, lengths, dev), _here(src, i32, "src", dev),
        _here(dst, i32, "dst", dev), src.numel(), *_here_ws(workspace, dev),
        _here_stream(stream, dev))
    _check(st, "mla_pages_fork")


def mla_pages_reserve(page_size, refcount, page_table, held, lengths, slots, extra, *,
                      workspace=None, stream=None):
    """The pages that sequences `slots` lack for lengths + extra positions."""
    dev = _device()
    i32 = torch.int32
    _shape(extra, slots.shape, "extra")
    st = load().mla_pages_reserve(
        refcount.numel(), int(page_size), *_book(refcount, page_table, held, lengths, dev),
        _here(slots, i32, "slots", dev), _here(extra, i32, "extra", dev), slots.numel(),
        *_here_ws(workspace, dev), _here_stream(stream, dev))
    _check(st, "mla_pages_reserve")


# ---- long contexts: eviction by accumulated attention ------------------------------------------


def mla_tree_latent_lse(q_cat, pool, page_table, lengths, cu_nodes, z, lse, *, mask=None,
                        scale=MLA_SCALE, workspace=None, stream=None):
    """mla_tree_latent that also writes lse [nodes, H] fp32, each row's log of the sum of exp(score)."""
    dev = _device()
    total, H, n = q_cat.shape[0], q_cat.shape[1], cu_nodes.numel() - 1
    _shape(q_cat, (total, H, 576), "q_cat")
    _shape(z, (total, H, 512), "z")
    _shape(lse, (total, H), "lse")
    _shape(mask, (total,), "mask")
    if z.dtype not in _DTYPE:
        raise TypeError(f"z: expected float32 or bfloat16, got {z.dtype}")
    st = load().mla_tree_latent_lse(
        _here(q_cat, torch.bfloat16, "q_cat", dev), H, *_paged(pool, page_table, lengths, n, dev),
        _here(cu_nodes, torch.int32, "cu_nodes", dev), n, total,
        _here(mask, torch.int64, "mask", dev), float(scale), _here(z, z.dtype, "z", dev),
        _DTYPE[z.dtype], _here(lse, torch.float32, "lse", dev), *_here_ws(workspace, dev),
        _here_stream(stream, dev))
    _check(st, "mla_tree_latent_lse")


def _decode_shapes(q_nope, q_rope, w_uk, w_uv, gate_logit, q_cat, z, out, mask):
    total = q_nope.shape[0]
    for t, tail, name in ((q_nope, (64, 128), "q_nope"), (q_rope, (64, 64), "q_rope"),
                          (gate_logit, (64,), "gate_logit"), (q_cat, (64, 576), "q_cat"),
                          (z, (64, 512), "z"), (out, (64, 128), "out")):
        _shape(t, (total,) + tail, name)
    _shape(w_uk, (64, 128, 512), "w_uk")
    _shape(w_uv, (64, 128, 512), "w_uv")
    _shape(mask, (total,), "mask")
    return total


def mla_tree_decode_lse(q_nope, q_rope, w_uk, w_uv, pool, page_table, lengths, cu_nodes, gate_logit,
                        q_cat, z, out, lse, *, mask=None, scale=MLA_SCALE, workspace=None,
                        stream=None):
    """mla_tree_decode that also writes lse [nodes, 64] fp32."""
    dev = _device()
    bf, n = torch.bfloat16, cu_nodes.numel() - 1
    total = _decode_shapes(q_nope, q_rope, w_uk, w_uv, gate_logit, q_cat, z, out, mask)
    _shape(lse, (total, 64), "lse")
    st = load().mla_tree_decode_lse(
        _here(q_nope, bf, "q_nope", dev), _here(q_rope, bf, "q_rope", dev),
        _here(w_uk, bf, "w_uk", dev), _here(w_uv, bf, "w_uv", dev),
        *_paged(pool, page_table, lengths, n, dev), _here(cu_nodes, torch.int32, "cu_nodes", dev),
        n, total, _here(mask, torch.int64, "mask", dev), _here(gate_logit, bf, "gate_logit", dev),
        float(scale), _here(q_cat, bf, "q_cat", dev), _here(z, torch.float32, "z", dev),
        _here(out, bf, "out", dev), _here(lse, torch.float32, "lse", dev),
        *_here_ws(workspace, dev), _here_stream(stream, dev))
    _check(st, "mla_tree_decode_lse")


def mla_cache_weights(q_cat, pool, page_table, lengths, cu_nodes, lse, weights, *, mask=None,
                      node_weight=None, scale=MLA_SCALE, stream=None):
    """weights [n_seqs, positions] fp32 += the attention that each cached position gets from the rows
    q_cat [nodes, H, 576], whose lse [nodes, H] mla_tree_latent_lse wrote; node_weight [nodes] fp32
    (None: ones; 0: a node that does not count)."""
    dev = _device()
    f32, i32 = torch.float32, torch.int32
    total, H, n = q_cat.shape[0], q_cat.shape[1], cu_nodes.numel() - 1
    _shape(q_cat, (total, H, 576), "q_cat")
    _shape(lse, (total, H), "lse")
    _shape(mask, (total,), "mask")
    _shape(node_weight, (total,), "node_weight")
    if len(weights.shape) != 2 or weights.shape[0] < n:
        raise ValueError("weights: expected [n_seqs, positions]")
    st = load().mla_cache_weights(
        _here(q_cat, torch.bfloat16, "q_cat", dev), H, *_paged(pool, page_table, lengths, n, dev),
        _here(cu_nodes, i32, "cu_nodes", dev), n, total, _here(mask, torch.int64, "mask", dev),
        _here(node_weight, f32, "node_weight", dev), _here(lse, f32, "lse", dev), float(scale),
        _here(weights, f32, "weights", dev), weights.shape[1], _here_stream(stream, dev))
    _check(st, "mla_cache_weights")


def mla_weights_accept(weights, lengths, cu_nodes, parent, accept_node, *, stream=None):
    """The weights of accepted paths moved as mla_cache_accept moves their rows (lengths as before it);
    those of the other drafted positions become 0."""
    dev = _device()
    n, i32 = cu_nodes.numel() - 1, torch.int32
    _shape(accept_node, (n,), "accept_node")
    if len(weights.shape) != 2 or weights.shape[0] < n or lengths.shape[0] < n:
        raise ValueError("weights, lengths: fewer rows than sequences")
    st = load().mla_weights_accept(
        _here(weights, torch.float32, "weights", dev), weights.shape[1],
        _here(lengths, i32, "lengths", dev), _here(cu_nodes, i32, "cu_nodes", dev), n,
        parent.shape[0], _here(parent, i32, "parent", dev),
        _here(accept_node, i32, "accept_node", dev), _here_stream(stream, dev))
    _check(st, "mla_weights_accept")


def mla_cache_evict(pool, page_table, lengths, weights, kept, new_lengths, new_weights=None, *,
                    first=0, recent=0, refcount=None, stream=None):
    """Sequences cut to kept.shape[1] positions: the first, the recent and the heaviest others stay;
    pool [n_layers, n_pages, page_size, 576] compacted, kept [n_seqs, budget], new_lengths (may be
    lengths), new_weights like weights [n_seqs, positions] (may be weights)."""
    dev = _device()
    f32, i32 = torch.float32, torch.int32
    n = kept.shape[0]
    if len(kept.shape) != 2 or len(weights.shape) != 2 or weights.shape[0] < n:
        raise ValueError("kept, weights: expected [n_seqs, budget] and [n_seqs, positions]")
    if new_lengths.shape[0] < n:
        raise ValueError("new_lengths: fewer rows than sequences")
    _shape(new_weights, weights.shape, "new_weights")
    _shape(refcount, (pool.shape[1],), "refcount")
    st = load().mla_cache_evict(
        *_paged_layers(pool, page_table, lengths, n, dev), _here(refcount, i32, "refcount", dev), n,
        _here(weights, f32, "weights", dev), weights.shape[1], kept.shape[1], int(first),
        int(recent), _here(kept, i32, "kept", dev), _here(new_lengths, i32, "new_lengths", dev),
        _here(new_weights, f32, "new_weights", dev), _here_stream(stream, dev))
    _check(st, "mla_cache_evict")


def mla_pages_trim(page_size, refcount, page_table, held, lengths, slots, *, stream=None):
    """The pages of sequences `slots` behind their lengths released."""
    dev = _device()
    st = load().mla_pages_trim(
        refcount.numel(), int(page_size), *_book(refcount, page_table, held, lengths, dev),
        _here(slots, torch.int32, "slots", dev), slots.numel(), _here_stream(stream, dev))
    _check(st, "mla_pages_trim")


# ---- long contexts: attention over chosen blocks -------------------------------------------------


def mla_block_keys(pool, page_table, from_lengths, lengths, keys, *, stream=None):
    """keys [n_layers, n_pages, 576]: the mean rows of the pages of pool [n_layers, n_pages,
    page_size, 576] that filled up while from_lengths [n_seqs] grew to lengths."""
    dev = _device()
    n = from_lengths.shape[0]
    _shape(keys, (pool.shape[0], pool.shape[1], 576), "keys")
    layers = _paged_layers(pool, page_table, lengths, n, dev)
    st = load().mla_block_keys(
        *layers[:-1], _here(from_lengths, torch.int32, "from_lengths", dev), layers[-1], n,
        _here(keys, torch.bfloat16, "keys", dev), _here_stream(stream, dev))
    _check(st, "mla_block_keys")


def mla_block_scores_workspace_size(total_nodes, H, max_pages):
    return int(load().mla_block_scores_workspace_size(int(total_nodes), int(H), int(max_pages)))


def _block_keys(keys, n_pages, dev):
    _shape(keys, (n_pages, 576), "keys")
    return _here(keys, torch.bfloat16, "keys", dev)


def _scores(scores, n, dev):
    if len(scores.shape) != 2 or scores.shape[0] < n:
        raise ValueError("scores: expected [n_seqs, blocks]")
    return _here(scores, torch.float32, "scores", dev), scores.shape[1]


def _selection(sel_table, sel_lengths, n, dev):
    if len(sel_table.shape) != 2 or sel_table.shape[0] < n or sel_lengths.shape[0] < n:
        raise ValueError("sel_table, sel_lengths: fewer rows than sequences")
    return (_here(sel_table, torch.int32, "sel_table", dev), sel_table.shape[1],
            _here(sel_lengths, torch.int32, "sel_lengths", dev))


def _tables(page_table, lengths, n, dev):
    rows, max_pages = page_table.shape
    if rows < n or lengths.shape[0] < n:
        raise ValueError("page_table, lengths: fewer rows than sequences")
    return (_here(page_table, torch.int32, "page_table", dev), max_pages,
            _here(lengths, torch.int32, "lengths", dev))


def mla_block_scores(q_cat, keys, page_size, page_table, lengths, cu_nodes, scores, *,
                     scale=MLA_SCALE, workspace=None, stream=None):
    """scores [n_seqs, blocks] fp32 of each sequence's full pages, by keys [n_pages, 576] (a layer's):
    every row's softmax over the pages, summed over the rows q_cat [nodes, H, 576]."""
    dev = _device()
    total, H, n = q_cat.shape[0], q_cat.shape[1], cu_nodes.numel() - 1
    _shape(q_cat, (total, H, 576), "q_cat")
    st = load().mla_block_scores(
        _here(q_cat, torch.bfloat16, "q_cat", dev), H, _block_keys(keys, keys.shape[0], dev),
        keys.shape[0], int(page_size), *_tables(page_table, lengths, n, dev),
        _here(cu_nodes, torch.int32, "cu_nodes", dev), n, total, float(scale),
        *_scores(scores, n, dev), *_here_ws(workspace, dev), _here_stream(stream, dev))
    _check(st, "mla_block_scores")


def mla_block_select(scores, page_size, page_table, lengths, cu_nodes, sel_table, sel_lengths, *,
                     blocks, total_nodes, first=0, recent=0, stream=None):
    """sel_table [n_seqs, sel_pages], sel_lengths [n_seqs]: the page table and lengths of the `blocks`
    full pages of the largest scores (the first and the recent always) and of what is behind them.
    total_nodes: rows of the step's queries."""
    dev = _device()
    n = cu_nodes.numel() - 1
    st = load().mla_block_select(
        *_scores(scores, n, dev), int(page_size), *_tables(page_table, lengths, n, dev),
        _here(cu_nodes, torch.int32, "cu_nodes", dev), n, int(total_nodes), int(blocks), int(first),
        int(recent), *_selection(sel_table, sel_lengths, n, dev), _here_stream(stream, dev))
    _check(st, "mla_block_select")


def mla_sparse_workspace_size(n_seqs, total_nodes, H, max_pages):
    return int(load().mla_sparse_workspace_size(int(n_seqs), int(total_nodes), int(H),
                                                int(max_pages)))


def mla_sparse_latent(q_cat, pool, keys, page_table, lengths, cu_nodes, scores, sel_table,
                      sel_lengths, z, *, blocks, first=0, recent=0, mask=None, scale=MLA_SCALE,
                      workspace=None, stream=None):
    """mla_block_scores, mla_block_select and mla_tree_latent over the chosen pages.  Without nodes nothing
    is written, the selection neither."""
    dev = _device()
    total, H, n = q_cat.shape[0], q_cat.shape[1], cu_nodes.numel() - 1
    _shape(q_cat, (total, H, 576), "q_cat")
    _shape(z, (total, H, 512), "z")
    _shape(mask, (total,), "mask")
    if z.dtype not in _DTYPE:
        raise TypeError(f"z: expected float32 or bfloat16, got {z.dtype}")
    cache = _paged(pool, page_table, lengths, n, dev)
    st = load().mla_sparse_latent(
        _here(q_cat, torch.bfloat16, "q_cat", dev), H, cache[0],
        _block_keys(keys, pool.shape[0], dev), *cache[1:],
        _here(cu_nodes, torch.int32, "cu_nodes", dev), n, total,
        _here(mask, torch.int64, "mask", dev), float(scale), int(blocks), int(first), int(recent),
        *_scores(scores, n, dev), *_selection(sel_table, sel_lengths, n, dev),
        _here(z, z.dtype, "z", dev), _DTYPE[z.dtype], *_here_ws(workspace, dev),
        _here_stream(stream, dev))
    _check(st, "mla_sparse_latent")


def mla_sparse_decode(q_nope, q_rope, w_uk, w_uv, pool, keys, page_table, lengths, cu_nodes,
                      gate_logit, scores, sel_table, sel_lengths, q_cat, z, out, *, blocks, first=0,
                      recent=0, mask=None, scale=MLA_SCALE, workspace=None, stream=None):
    """mla_tree_decode over the pages that mla_block_scores and mla_block_select choose."""
    dev = _device()
    bf, n = torch.bfloat16, cu_nodes.numel() - 1
    total = _decode_shapes(q_nope, q_rope, w_uk, w_uv, gate_logit, q_cat, z, out, mask)
    cache = _paged(pool, page_table, lengths, n, dev)
    st = load().mla_sparse_decode(
        _here(q_nope, bf, "q_nope", dev), _here(q_rope, bf, "q_rope", dev),
        _here(w_uk, bf, "w_uk", dev), _here(w_uv, bf, "w_uv", dev), cache[0],
        _block_keys(keys, pool.shape[0], dev), *cache[1:],
        _here(cu_nodes, torch.int32, "cu_nodes", dev), n, total,
        _here(mask, torch.int64, "mask", dev), _here(gate_logit, bf, "gate_logit", dev),
        float(scale), int(blocks), int(first), int(recent), *_scores(scores, n, dev),
        *_selection(sel_table, sel_lengths, n, dev), _here(q_cat, bf, "q_cat", dev),
        _here(z, torch.float32, "z", dev), _here(out, bf, "out", dev), *_here_ws(workspace, dev),
        _here_stream(stream, dev))
    _check(st, "mla_sparse_decode")
