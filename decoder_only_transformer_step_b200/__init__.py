"""Python binding of libgpt2.so: one GPT-2 pretraining step on one B200.

Argument marshalling only.  Every step of the path runs in the library's
CUDA kernels; PyTorch provides device memory and streams.  The library is
loaded on first use; a RuntimeError is raised if it has not been built (``python -m decoder_only_transformer_step_b200.build_lib``):
there is no CPU fallback.

Functions named like the C entry points take torch tensors (device memory)
and ints/floats; ``GPT2`` bundles the buffers a context needs.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgpt2.so")

GPT2_OK = 0
ERRORS = {
    -1: "GPT2_ERR_INVALID_ARG", -2: "GPT2_ERR_UNSUPPORTED_SHAPE", -3: "GPT2_ERR_CUDA",
    -4: "GPT2_ERR_BAD_STATE", -5: "GPT2_ERR_TOKEN_RANGE", -6: "GPT2_ERR_NONFINITE",
    -7: "GPT2_ERR_TIMEOUT", -8: "GPT2_ERR_WORKSPACE", -9: "GPT2_ERR_TOO_LARGE",
    -10: "GPT2_ERR_POSITION_RANGE",
}
ERRORS_BY_NAME = {v: k for k, v in ERRORS.items()}


class Gpt2Error(RuntimeError):
    def __init__(self, code: int, where: str):
        super().__init__(f"{where}: {ERRORS.get(code, code)} ({_lib().gpt2_strerror(code).decode()})")
        self.code = code


class gpt2_config(ctypes.Structure):
    _fields_ = [("n_layer", ctypes.c_int), ("d_model", ctypes.c_int), ("n_head", ctypes.c_int),
                ("n_ctx", ctypes.c_int), ("vocab_real", ctypes.c_int), ("vocab_padded", ctypes.c_int),
                ("max_batch", ctypes.c_int), ("mode", ctypes.c_int)]


class gpt2_buffers(ctypes.Structure):
    _fields_ = [("master", ctypes.c_void_p), ("shadow", ctypes.c_void_p), ("grad", ctypes.c_void_p),
                ("m", ctypes.c_void_p), ("v", ctypes.c_void_p), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_size_t)]


class gpt2_decode_opts(ctypes.Structure):
    _fields_ = [("q4", ctypes.c_void_p), ("q4_bytes", ctypes.c_size_t), ("q4_group", ctypes.c_int),
                ("prefix", ctypes.c_void_p), ("prefix_bytes", ctypes.c_size_t), ("prefix_cap", ctypes.c_int),
                ("prefix_len", ctypes.c_int), ("scratch", ctypes.c_void_p), ("scratch_bytes", ctypes.c_size_t)]


class gpt2_logit_rules(ctypes.Structure):
    _fields_ = [("history", ctypes.c_void_p), ("history_len", ctypes.c_void_p), ("gen_start", ctypes.c_void_p),
                ("repetition", ctypes.c_void_p), ("presence", ctypes.c_void_p), ("frequency", ctypes.c_void_p),
                ("bias_ids", ctypes.c_void_p), ("bias_values", ctypes.c_void_p), ("allowed", ctypes.c_void_p),
                ("history_ld", ctypes.c_int), ("n_bias", ctypes.c_int), ("allowed_ld", ctypes.c_int),
                ("append", ctypes.c_int)]


EXPORTS = [
    "gpt2_param_count", "gpt2_workspace_bytes", "gpt2_tensor_info", "gpt2_create", "gpt2_destroy",
    "gpt2_init_params", "gpt2_refresh_shadow", "gpt2_forward_loss", "gpt2_backward",
    "gpt2_adamw_step", "gpt2_adamw_step_clip", "gpt2_adamw_step_range", "gpt2_grad_norm", "gpt2_zero_grad", "gpt2_get_status", "gpt2_step_host", "gpt2_strerror",
    "gpt2_kernel_launches",
    "gpt2_kv_cache_bytes", "gpt2_prefill", "gpt2_decode_step", "gpt2_greedy_next",
    "gpt2_op_gemm_bf16", "gpt2_op_attention_fwd_bf16", "gpt2_op_attention_bwd_bf16",
    "gpt2_op_attention_bwd_bf16_noalloc",
    "gpt2_op_layernorm_fwd_bf16", "gpt2_op_layernorm_bwd_scratch_floats", "gpt2_op_layernorm_bwd_bf16",
    "gpt2_op_colsum_scratch_floats", "gpt2_op_colsum_bf16",
    "gpt2_op_lm_head_ce_scratch_bytes", "gpt2_op_lm_head_ce_fwd_bf16", "gpt2_op_lm_head_ce_bwd_bf16",
    "gpt2_set_wait_timeout_ns", "gpt2_op_gemm_bf16_status", "gpt2_backward_bucketed",
    "gpt2_op_linear_bf16", "gpt2_graph_capture", "gpt2_graph_step", "gpt2_graph_release",
    "gpt2_q4_bytes", "gpt2_q4_pack", "gpt2_decode_scratch_bytes", "gpt2_decode_step_ex", "gpt2_rules_next",
    "gpt2_op_q4_packed_bytes", "gpt2_op_q4_scale_count", "gpt2_op_q4_quantize", "gpt2_op_q4_dequantize",
    "gpt2_op_gemv_q4", "gpt2_op_prefix_attention_scratch_bytes", "gpt2_op_prefix_attention_bf16",
    "gpt2_op_logit_rules",
]

_LIB = None


def _lib():
    global _LIB
    if _LIB is not None:
        return _LIB
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                           "`python -m decoder_only_transformer_step_b200.build_lib`")
    L = ctypes.CDLL(LIB_PATH)
    P, I, F, S, U64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.c_uint64
    cfgp = ctypes.POINTER(gpt2_config)
    sig = {
        "gpt2_param_count": (S, [cfgp]),
        "gpt2_workspace_bytes": (S, [cfgp, I]),
        "gpt2_tensor_info": (I, [cfgp, I, ctypes.POINTER(ctypes.c_char_p), ctypes.POINTER(S),
                                 ctypes.POINTER(S), ctypes.POINTER(S)]),
        "gpt2_create": (I, [cfgp, ctypes.POINTER(gpt2_buffers), ctypes.POINTER(P)]),
        "gpt2_destroy": (I, [P]),
        "gpt2_init_params": (I, [P, U64, P]),
        "gpt2_refresh_shadow": (I, [P, P]),
        "gpt2_forward_loss": (I, [P, P, P, I, P, P]),
        "gpt2_backward": (I, [P, F, I, P]),
        "gpt2_adamw_step": (I, [P, F, F, F, F, F, I, P]),
        "gpt2_adamw_step_clip": (I, [P, F, F, F, F, F, I, F, P]),
        "gpt2_adamw_step_range": (I, [P, F, F, F, F, F, I, S, S, P]),
        "gpt2_grad_norm": (I, [P, P, P]),
        "gpt2_zero_grad": (I, [P, P]),
        "gpt2_get_status": (I, [P, P]),
        "gpt2_step_host": (I, [P, P, P, I, P, F, F, F, F, F, I, P]),
        "gpt2_strerror": (ctypes.c_char_p, [I]),
        "gpt2_kernel_launches": (ctypes.c_uint64, []),
        "gpt2_kv_cache_bytes": (S, [cfgp, I, I]),
        "gpt2_prefill": (I, [P, P, S, I, I, P, P, P, P]),
        "gpt2_decode_step": (I, [P, P, S, I, I, P, P, P, P]),
        "gpt2_greedy_next": (I, [P, P, I, P, P, P]),
        "gpt2_op_gemm_bf16": (I, [P, I, I, P, I, I, P, I, I, I, I, I, F, F, P, S, I, I, P]),
        "gpt2_op_attention_fwd_bf16": (I, [P, P, P, I, I, I, I, P]),
        "gpt2_op_attention_bwd_bf16": (I, [P, P, P, P, P, P, I, I, I, I, P]),
        "gpt2_op_attention_bwd_bf16_noalloc": (I, [P, P, P, P, P, I, I, I, I, P]),
        "gpt2_op_layernorm_fwd_bf16": (I, [P, P, P, P, P, P, I, I, P]),
        "gpt2_op_layernorm_bwd_scratch_floats": (S, [I, I]),
        "gpt2_op_layernorm_bwd_bf16": (I, [P, P, P, P, P, P, I, P, P, S, I, I, P]),
        "gpt2_op_colsum_scratch_floats": (S, [I, I]),
        "gpt2_op_colsum_bf16": (I, [P, I, I, P, P, S, P]),
        "gpt2_op_lm_head_ce_scratch_bytes": (S, [I, I]),
        "gpt2_op_lm_head_ce_fwd_bf16": (I, [P, P, P, I, I, I, I, P, P, P, S, P]),
        "gpt2_op_lm_head_ce_bwd_bf16": (I, [P, P, I, I, I, F, P, P, I, P, S, P]),
        "gpt2_set_wait_timeout_ns": (I, [U64]),
        "gpt2_backward_bucketed": (I, [P, F, I, P, I, P]),
        "gpt2_op_gemm_bf16_status": (I, [P, I, I, P, I, I, P, I, I, I, I, I, F, F, P, S, I, I, P, P]),
        "gpt2_op_linear_bf16": (I, [P, P, P, P, P, P, I, I, I, I, P]),
        "gpt2_graph_capture": (I, [P, I, F, I, P, P]),
        "gpt2_graph_step": (I, [P, P, P, P]),
        "gpt2_graph_release": (I, [P]),
        "gpt2_q4_bytes": (S, [cfgp, I]),
        "gpt2_q4_pack": (I, [P, P, S, I, P]),
        "gpt2_decode_scratch_bytes": (S, [cfgp, I, I, I]),
        "gpt2_decode_step_ex": (I, [P, P, S, I, I, P, P, ctypes.POINTER(gpt2_decode_opts), P, P]),
        "gpt2_rules_next": (I, [P, P, I, ctypes.POINTER(gpt2_logit_rules), P, P, P]),
        "gpt2_op_q4_packed_bytes": (S, [I, I]),
        "gpt2_op_q4_scale_count": (S, [I, I, I]),
        "gpt2_op_q4_quantize": (I, [P, I, I, I, I, I, P, P, P]),
        "gpt2_op_q4_dequantize": (I, [P, P, I, I, I, P, I, I, P]),
        "gpt2_op_gemv_q4": (I, [P, I, P, P, P, P, I, I, I, I, I, I, P]),
        "gpt2_op_prefix_attention_scratch_bytes": (S, [I, I, I, I, I, I]),
        "gpt2_op_prefix_attention_bf16": (I, [P, I, P, P, I, I, P, P, P, I, P, I, P, P, S, I, I, I, I, P]),
        "gpt2_op_logit_rules": (I, [P, I, P, I, I, I, ctypes.POINTER(gpt2_logit_rules), P, P, P]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    _LIB = L
    return L


def _check(rc: int, where: str):
    if rc != GPT2_OK:
        raise Gpt2Error(rc, where)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


# --------------------------------------------------------------- C names ---

def make_config(n_layer, d_model, n_head, n_ctx, vocab_real, vocab_padded, max_batch, mode=0):
    return gpt2_config(n_layer, d_model, n_head, n_ctx, vocab_real, vocab_padded, max_batch, mode)


def gpt2_param_count(cfg: gpt2_config) -> int:
    return int(_lib().gpt2_param_count(ctypes.byref(cfg)))


def gpt2_workspace_bytes(cfg: gpt2_config, batch: int) -> int:
    return int(_lib().gpt2_workspace_bytes(ctypes.byref(cfg), batch))


def gpt2_tensor_info(cfg: gpt2_config, index: int):
    """(name, offset, rows, cols) or None past the last tensor."""
    name = ctypes.c_char_p()
    off, r, c = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    rc = _lib().gpt2_tensor_info(ctypes.byref(cfg), index, ctypes.byref(name), ctypes.byref(off),
                                 ctypes.byref(r), ctypes.byref(c))
    if rc != GPT2_OK:
        return None
    return name.value.decode(), off.value, r.value, c.value


def gpt2_tensors(cfg: gpt2_config):
    out, i = [], 0
    while True:
        t = gpt2_tensor_info(cfg, i)
        if t is None:
            return out
        out.append(t)
        i += 1


def gpt2_create(cfg, master, shadow, grad, m, v, workspace):
    bufs = gpt2_buffers(master.data_ptr(), shadow.data_ptr() if shadow is not None else None,
                        grad.data_ptr(), m.data_ptr(), v.data_ptr(), workspace.data_ptr(),
                        workspace.numel() * workspace.element_size())
    ctx = ctypes.c_void_p()
    _check(_lib().gpt2_create(ctypes.byref(cfg), ctypes.byref(bufs), ctypes.byref(ctx)), "gpt2_create")
    ctx.vocab_padded = cfg.vocab_padded  # (for the extent of logits, below)
    return ctx


def gpt2_destroy(ctx):
    _check(_lib().gpt2_destroy(ctx), "gpt2_destroy")


def gpt2_init_params(ctx, seed: int, stream=None):
    _check(_lib().gpt2_init_params(ctx, seed, _stream(stream)), "gpt2_init_params")


def gpt2_refresh_shadow(ctx, stream=None):
    _check(_lib().gpt2_refresh_shadow(ctx, _stream(stream)), "gpt2_refresh_shadow")


def gpt2_forward_loss(ctx, tokens, targets, batch: int, loss_dev, stream=None):
    _check(_lib().gpt2_forward_loss(ctx, _ptr(tokens), _ptr(targets), batch, _ptr(loss_dev),
                                    _stream(stream)), "gpt2_forward_loss")


def gpt2_backward(ctx, grad_scale: float = 1.0, accumulate: int = 0, stream=None):
    _check(_lib().gpt2_backward(ctx, grad_scale, accumulate, _stream(stream)), "gpt2_backward")


def gpt2_backward_bucketed(ctx, grad_scale, accumulate, events, stream=None):
    """events: torch.cuda.Event objects (already created, e.g. recorded once),
    n_layer + 2 of them."""
    arr = (ctypes.c_void_p * len(events))(*[ctypes.c_void_p(e.cuda_event) for e in events])
    _check(_lib().gpt2_backward_bucketed(ctx, grad_scale, accumulate, arr, len(events), _stream(stream)),
           "gpt2_backward_bucketed")


def gpt2_graph_capture(ctx, batch, grad_scale, accumulate, loss_dev, stream):
    """Records forward + loss + backward into the context's graph; `stream` is
    a torch.cuda.Stream the caller created (not the default stream)."""
    _check(_lib().gpt2_graph_capture(ctx, batch, grad_scale, accumulate, _ptr(loss_dev), _stream(stream)),
           "gpt2_graph_capture")


def gpt2_graph_step(ctx, tokens, targets, stream=None):
    _check(_lib().gpt2_graph_step(ctx, _ptr(tokens), _ptr(targets), _stream(stream)), "gpt2_graph_step")


def gpt2_graph_release(ctx):
    _check(_lib().gpt2_graph_release(ctx), "gpt2_graph_release")


def gpt2_adamw_step(ctx, lr, beta1, beta2, eps, weight_decay, step, stream=None):
    _check(_lib().gpt2_adamw_step(ctx, lr, beta1, beta2, eps, weight_decay, step, _stream(stream)),
           "gpt2_adamw_step")


def gpt2_adamw_step_clip(ctx, lr, beta1, beta2, eps, weight_decay, step, max_norm, stream=None):
    _check(_lib().gpt2_adamw_step_clip(ctx, lr, beta1, beta2, eps, weight_decay, step, max_norm,
                                       _stream(stream)), "gpt2_adamw_step_clip")


def gpt2_adamw_step_range(ctx, lr, beta1, beta2, eps, weight_decay, step, offset, count, stream=None):
    _check(_lib().gpt2_adamw_step_range(ctx, lr, beta1, beta2, eps, weight_decay, step, offset, count,
                                        _stream(stream)), "gpt2_adamw_step_range")


def gpt2_grad_norm(ctx, norm_dev=None, stream=None):
    _check(_lib().gpt2_grad_norm(ctx, _ptr(norm_dev), _stream(stream)), "gpt2_grad_norm")


def gpt2_zero_grad(ctx, stream=None):
    _check(_lib().gpt2_zero_grad(ctx, _stream(stream)), "gpt2_zero_grad")


def gpt2_get_status(ctx, stream=None) -> int:
    return int(_lib().gpt2_get_status(ctx, _stream(stream)))


def gpt2_step_host(ctx, tokens_host, targets_host, batch, loss_host, lr, beta1, beta2, eps,
                   weight_decay, step, stream=None):
    """tokens_host/targets_host/loss_host: CPU (ideally pinned) torch tensors."""
    _check(_lib().gpt2_step_host(ctx, _ptr(tokens_host), _ptr(targets_host), batch, _ptr(loss_host),
                                 lr, beta1, beta2, eps, weight_decay, step, _stream(stream)),
           "gpt2_step_host")


def gpt2_kernel_launches() -> int:
    return int(_lib().gpt2_kernel_launches())


def gpt2_kv_cache_bytes(cfg: gpt2_config, batch: int, max_len: int) -> int:
    return int(_lib().gpt2_kv_cache_bytes(ctypes.byref(cfg), batch, max_len))


def _nbytes(t):
    return t.numel() * t.element_size()


def gpt2_prefill(ctx, cache, batch, max_len, tokens, prompt_len, logits, stream=None):
    """cache: a device tensor of at least gpt2_kv_cache_bytes(cfg, batch, max_len) bytes."""
    _check(_lib().gpt2_prefill(ctx, _ptr(cache), _nbytes(cache), batch, max_len, _ptr(tokens), _ptr(prompt_len),
                               _ptr(logits), _stream(stream)), "gpt2_prefill")


def gpt2_decode_step(ctx, cache, batch, max_len, tokens, pos, logits, stream=None):
    """cache: a device tensor of at least gpt2_kv_cache_bytes(cfg, batch, max_len) bytes."""
    _check(_lib().gpt2_decode_step(ctx, _ptr(cache), _nbytes(cache), batch, max_len, _ptr(tokens), _ptr(pos),
                                   _ptr(logits), _stream(stream)), "gpt2_decode_step")


def gpt2_greedy_next(ctx, logits, batch, next_tokens, pos=None, stream=None):
    _check(_lib().gpt2_greedy_next(ctx, _ptr(logits), batch, _ptr(next_tokens), _ptr(pos), _stream(stream)),
           "gpt2_greedy_next")


def gpt2_op_gemm_bf16(A, a_mn_major, lda, B, b_mn_major, ldb, C, c_fp32, ldc, M, N, K,
                      alpha=1.0, beta=0.0, workspace=None, bn=0, splits=0, stream=None):
    wsb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib().gpt2_op_gemm_bf16(_ptr(A), a_mn_major, lda, _ptr(B), b_mn_major, ldb, _ptr(C), c_fp32,
                                    ldc, M, N, K, alpha, beta, _ptr(workspace), wsb, bn, splits,
                                    _stream(stream)), "gpt2_op_gemm_bf16")


def gpt2_op_attention_fwd_bf16(qkv, o, lse, B, T, H, hd, stream=None):
    _check(_lib().gpt2_op_attention_fwd_bf16(_ptr(qkv), _ptr(o), _ptr(lse), B, T, H, hd,
                                             _stream(stream)), "gpt2_op_attention_fwd_bf16")


def gpt2_op_attention_bwd_bf16(qkv, o, lse, dout, dqkv, scratch, B, T, H, hd, stream=None):
    _check(_lib().gpt2_op_attention_bwd_bf16(_ptr(qkv), _ptr(o), _ptr(lse), _ptr(dout), _ptr(dqkv),
                                             _ptr(scratch), B, T, H, hd, _stream(stream)),
           "gpt2_op_attention_bwd_bf16")


def gpt2_op_attention_bwd_bf16_noalloc(qkv, o, lse, dout, dqkv, B, T, H, hd, stream=None):
    """Allocation-free attention backward: scratch lives in the library (see
    include/gpt2.h); for callers that cannot allocate device memory."""
    _check(_lib().gpt2_op_attention_bwd_bf16_noalloc(_ptr(qkv), _ptr(o), _ptr(lse), _ptr(dout), _ptr(dqkv),
                                                     B, T, H, hd, _stream(stream)),
           "gpt2_op_attention_bwd_bf16_noalloc")


def gpt2_op_layernorm_fwd_bf16(x, gamma, beta, y, mean, rstd, M, d, stream=None):
    _check(_lib().gpt2_op_layernorm_fwd_bf16(_ptr(x), _ptr(gamma), _ptr(beta), _ptr(y), _ptr(mean), _ptr(rstd),
                                             M, d, _stream(stream)), "gpt2_op_layernorm_fwd_bf16")


def gpt2_op_linear_bf16(x, w, bias, resid, out, out2, M, N, K, act, stream=None):
    """act 0: out = x w^T + bias; 1: + resid; 2: out = GELU(u), out2 = GELU'(u)."""
    _check(_lib().gpt2_op_linear_bf16(_ptr(x), _ptr(w), _ptr(bias), _ptr(resid), _ptr(out), _ptr(out2), M, N, K,
                                      act, _stream(stream)), "gpt2_op_linear_bf16")


def gpt2_op_layernorm_bwd_scratch_floats(M, d) -> int:
    return int(_lib().gpt2_op_layernorm_bwd_scratch_floats(M, d))


def gpt2_op_layernorm_bwd_bf16(dy, x, mean, rstd, gamma, dx, accumulate, dgamma_dbeta, scratch, M, d, stream=None):
    _check(_lib().gpt2_op_layernorm_bwd_bf16(_ptr(dy), _ptr(x), _ptr(mean), _ptr(rstd), _ptr(gamma), _ptr(dx),
                                             accumulate, _ptr(dgamma_dbeta), _ptr(scratch), scratch.numel(), M, d,
                                             _stream(stream)), "gpt2_op_layernorm_bwd_bf16")


def gpt2_op_colsum_scratch_floats(M, N) -> int:
    return int(_lib().gpt2_op_colsum_scratch_floats(M, N))


def gpt2_op_colsum_bf16(x, M, N, out, scratch, stream=None):
    _check(_lib().gpt2_op_colsum_bf16(_ptr(x), M, N, _ptr(out), _ptr(scratch), scratch.numel(), _stream(stream)),
           "gpt2_op_colsum_bf16")


def gpt2_op_lm_head_ce_scratch_bytes(M, V) -> int:
    return int(_lib().gpt2_op_lm_head_ce_scratch_bytes(M, V))


def gpt2_op_lm_head_ce_fwd_bf16(x, w, targets, M, V, d, vocab_real, loss, loss_rows, scratch, stream=None):
    _check(_lib().gpt2_op_lm_head_ce_fwd_bf16(_ptr(x), _ptr(w), _ptr(targets), M, V, d, vocab_real, _ptr(loss),
                                              _ptr(loss_rows), _ptr(scratch), scratch.numel() * scratch.element_size(),
                                              _stream(stream)), "gpt2_op_lm_head_ce_fwd_bf16")


def gpt2_op_lm_head_ce_bwd_bf16(x, w, M, V, d, grad_scale, dx, dw, accumulate, scratch, stream=None):
    _check(_lib().gpt2_op_lm_head_ce_bwd_bf16(_ptr(x), _ptr(w), M, V, d, grad_scale, _ptr(dx), _ptr(dw), accumulate,
                                              _ptr(scratch), scratch.numel() * scratch.element_size(),
                                              _stream(stream)), "gpt2_op_lm_head_ce_bwd_bf16")


def gpt2_set_wait_timeout_ns(ns: int):
    _check(_lib().gpt2_set_wait_timeout_ns(ns), "gpt2_set_wait_timeout_ns")


def gpt2_op_gemm_bf16_status(A, a_mn, lda, B, b_mn, ldb, C, c_fp32, ldc, M, N, K, alpha=1.0, beta=0.0,
                             workspace=None, bn=0, splits=0, status=None, stream=None):
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib().gpt2_op_gemm_bf16_status(_ptr(A), a_mn, lda, _ptr(B), b_mn, ldb, _ptr(C), c_fp32, ldc, M, N, K,
                                           alpha, beta, _ptr(workspace), ws_bytes, bn, splits, _ptr(status),
                                           _stream(stream)), "gpt2_op_gemm_bf16_status")


# ---- 4-bit weights, shared prefixes, rules on logits ------------------------
# These calls know every buffer's extent, so they check it here: a buffer that
# is too short, of another type or on another device is GPT2_ERR_INVALID_ARG
# instead of a read out of range, and so is a view whose elements do not lie
# where the call looks for them (a transposed weight).  A decode step makes several of them in a few
# microseconds of device time, so the checks are kept to what they need.

_T = None  # what these calls use of torch and of the library, looked up once


class _Torch:
    def __init__(self):
        import torch
        self.bf16, self.f32, self.u8, self.i32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32
        self.words = (torch.int32, torch.uint32)
        # (the bare handle of the current stream, without a Stream object around it, where this torch has it)
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        self.stream_of = raw if raw is not None else lambda dev: torch.cuda.current_stream(dev).cuda_stream
        self.current_device, self.available = torch.cuda.current_device, torch.cuda.is_available
        lib = _lib()
        self.quantize, self.dequantize = lib.gpt2_op_q4_quantize, lib.gpt2_op_q4_dequantize
        self.gemv, self.prefix, self.rules = (lib.gpt2_op_gemv_q4, lib.gpt2_op_prefix_attention_bf16,
                                              lib.gpt2_op_logit_rules)


def _torch():
    global _T
    if _T is None:
        _T = _Torch()
    return _T


def _buf(where, name, t, dtype, dev, need, pitch=None):
    """Address of a buffer on device `dev` of at least `need` elements (of a
    strided view: the memory from its first to its last one, which an expanded
    tensor has less of than elements); None for None where none are needed.
    pitch: how far apart the call's rows lie, which a view has to share (0: the
    call has no pitch, and a view has to be contiguous)."""
    if t is None:
        if need <= 0:
            return None
        raise Gpt2Error(-1, f"{where}: {name} is missing")
    whole = t.is_contiguous()
    if t.dtype is dtype and t.get_device() == dev and (t.numel() if whole else _span(t)) >= need:
        if whole or pitch is None or (t.stride(0) == pitch and t[0].is_contiguous()):
            return t.data_ptr()
        raise Gpt2Error(-1, f"{where}: {name} is a view with strides {t.stride()}, the call reads " +
                        (f"rows {pitch} apart" if pitch else "its elements one behind the other"))
    if t.dtype is not dtype:
        raise Gpt2Error(-1, f"{where}: {name} is {t.dtype}, not {dtype}")
    if t.get_device() != dev:
        raise Gpt2Error(-1, f"{where}: {name} is on {t.device}, not on the current CUDA device")
    raise Gpt2Error(-1, f"{where}: {name} holds {_span(t)} elements, {need} are needed")


def _span(t):
    return 1 + sum((n - 1) * st for n, st in zip(t.shape, t.stride())) if t.numel() else 0


def _scratch(where, t, u8, dev):
    """(address, bytes) of a scratch buffer."""
    n = 1 if t is None else t.numel()
    return _buf(where, "scratch", t, u8, dev, n), n


def _where(stream, T):
    """(device index, stream handle) a call runs on: the current device, whose
    kernels and limits the library takes, and the given or its current stream."""
    try:
        dev = T.current_device()
    except Exception:
        if T.available():
            raise
        return 0, None  # no GPU: every buffer is on another device
    if stream is None:
        return dev, T.stream_of(dev)
    if stream.device_index != dev:
        raise Gpt2Error(-1, f"the stream is on CUDA device {stream.device_index}, the current device is {dev}")
    return dev, stream.cuda_stream


def _extent(rows, ld, cols):
    """Elements from the first of a [rows, cols] matrix of pitch ld to its last."""
    return (rows - 1) * ld + cols if rows > 0 and cols > 0 else 0


def gpt2_op_q4_packed_bytes(N, K) -> int:
    return int(_lib().gpt2_op_q4_packed_bytes(N, K))


def gpt2_op_q4_scale_count(N, K, group) -> int:
    return int(_lib().gpt2_op_q4_scale_count(N, K, group))


def gpt2_op_q4_quantize(w, w_fp32, ldw, N, K, group, packed, scales, stream=None):
    """w [N, ldw] bf16 (or fp32 with w_fp32) -> packed uint8 [N, K/2], scales bf16 [K/group, N up to a multiple of 8]."""
    T, f = _T or _torch(), "gpt2_op_q4_quantize"
    dev, st = _where(stream, T)
    rc = T.quantize(_buf(f, "w", w, T.f32 if w_fp32 else T.bf16, dev, _extent(N, ldw, K), ldw), w_fp32, ldw, N, K, group,
                    _buf(f, "packed", packed, T.u8, dev, N * K // 2, 0),
                    _buf(f, "scales", scales, T.bf16, dev, K // group * ((N + 7) // 8 * 8) if group > 0 else 0, 0), st)
    if rc:
        raise Gpt2Error(rc, f)


def gpt2_op_q4_dequantize(packed, scales, N, K, group, out, out_fp32, ldo, stream=None):
    T, f = _T or _torch(), "gpt2_op_q4_dequantize"
    dev, st = _where(stream, T)
    rc = T.dequantize(_buf(f, "packed", packed, T.u8, dev, N * K // 2, 0),
                      _buf(f, "scales", scales, T.bf16, dev, K // group * ((N + 7) // 8 * 8) if group > 0 else 0, 0), N, K,
                      group, _buf(f, "out", out, T.f32 if out_fp32 else T.bf16, dev, _extent(N, ldo, K), ldo), out_fp32, ldo, st)
    if rc:
        raise Gpt2Error(rc, f)


def gpt2_op_gemv_q4(x, ldx, packed, scales, bias, out, out_fp32, ldo, rows, N, K, group, stream=None):
    """out [rows, ldo] = x [rows, ldx] W^T (+ bias) with W's 4-bit form; rows 1..16."""
    T, f = _T or _torch(), "gpt2_op_gemv_q4"
    dev, st = _where(stream, T)
    rc = T.gemv(_buf(f, "x", x, T.bf16, dev, _extent(rows, ldx, K), ldx), ldx, _buf(f, "packed", packed, T.u8, dev, N * K // 2, 0),
                _buf(f, "scales", scales, T.bf16, dev, K // group * ((N + 7) // 8 * 8) if group > 0 else 0, 0),
                None if bias is None else _buf(f, "bias", bias, T.bf16, dev, N, 0),
                _buf(f, "out", out, T.f32 if out_fp32 else T.bf16, dev, _extent(rows, ldo, N), ldo), out_fp32, ldo, rows, N, K,
                group, st)
    if rc:
        raise Gpt2Error(rc, f)


def gpt2_op_prefix_attention_scratch_bytes(B, Hq, Hkv, hd, prefix_len, max_len) -> int:
    return int(_lib().gpt2_op_prefix_attention_scratch_bytes(B, Hq, Hkv, hd, prefix_len, max_len))


def gpt2_op_prefix_attention_bf16(q, ldq, pk, pv, prefix_len, prefix_cap, k, v, len, max_len, o, ldo, lse, scratch, B, Hq,
                                  Hkv, hd, stream=None):
    """One token per row over the shared prefix pk, pv [Hkv, prefix_cap, hd] and the rows' own k, v
    [B, Hkv, max_len, hd], of which the first prefix_len and len[b] positions count."""
    T, f = _T or _torch(), "gpt2_op_prefix_attention_bf16"
    dev, st = _where(stream, T)
    np = _extent(Hkv, prefix_cap * hd, prefix_len * hd)
    no = B * Hkv * max_len * hd
    bf = T.bf16
    rc = T.prefix(_buf(f, "q", q, bf, dev, _extent(B, ldq, Hq * hd), ldq), ldq, _buf(f, "pk", pk, bf, dev, np, prefix_cap * hd),
                  _buf(f, "pv", pv, bf, dev, np, prefix_cap * hd), prefix_len, prefix_cap, _buf(f, "k", k, bf, dev, no, 0),
                  _buf(f, "v", v, bf, dev, no, 0), _buf(f, "len", len, T.i32, dev, B if max_len > 0 else 0, 0), max_len,
                  _buf(f, "o", o, bf, dev, _extent(B, ldo, Hq * hd), ldo), ldo,
                  None if lse is None else _buf(f, "lse", lse, T.f32, dev, B * Hq, 0),
                  *_scratch(f, scratch, T.u8, dev), B, Hq, Hkv, hd, st)
    if rc:
        raise Gpt2Error(rc, f)


class LogitRules:
    """Rules on the logits of a batch (see gpt2_logit_rules): device tensors,
    None where a rule is not asked for.  history int32 [rows, capacity] with
    history_len int32 [rows] and, where the history starts with a prompt,
    gen_start int32 [rows]; repetition, presence, frequency fp32 [rows];
    bias_ids int32 and bias_values fp32 [rows, n]; allowed int32 or uint32
    [rows, words], bit v % 32 of word v // 32 set where id v may be chosen;
    append: the chosen id is added to the history where there is room.  The tensors stay the
    caller's and are read at every call, so they can be changed in between."""

    def __init__(self, history=None, history_len=None, gen_start=None, repetition=None, presence=None, frequency=None,
                 bias_ids=None, bias_values=None, allowed=None, append=False):
        T, f = _T or _torch(), "LogitRules"
        per_row = dict(history_len=history_len, gen_start=gen_start, repetition=repetition, presence=presence,
                       frequency=frequency)
        tables = dict(history=history, bias_ids=bias_ids, bias_values=bias_values, allowed=allowed)
        rows = {t.shape[0] for t in (*per_row.values(), *tables.values()) if t is not None}
        for name, t in (*per_row.items(), *tables.items()):
            if t is not None and (t.dim() != (1 if name in per_row else 2) or not t.is_contiguous()):
                raise Gpt2Error(-1, f"{f}: {name} has shape {tuple(t.shape)} or is not contiguous")
        if len(rows) > 1:
            raise Gpt2Error(-1, f"{f}: the rules are for {sorted(rows)} rows")
        if (bias_ids is None) != (bias_values is None) or (bias_ids is not None and bias_ids.shape != bias_values.shape):
            raise Gpt2Error(-1, f"{f}: bias_ids and bias_values belong together")
        if history is not None and history_len is None:
            raise Gpt2Error(-1, f"{f}: a history needs history_len")
        if allowed is not None and allowed.shape[1] == 0:  # (its address is NULL: everything would be allowed)
            raise Gpt2Error(-1, f"{f}: allowed has no words")
        self.rows = rows.pop() if rows else None
        self.tensors = {**per_row, **tables}
        width = {n: 0 if t is None else t.shape[1] for n, t in tables.items()}
        dev = next((t.get_device() for t in self.tensors.values() if t is not None), 0)
        if dev < 0:
            raise Gpt2Error(-1, f"{f}: the rules are not on a CUDA device")

        def at(name, dtype):
            a = _buf(f, name, self.tensors[name], dtype, dev, 0)
            return a if width.get(name, 1) else None  # (a table of no columns is none)
        words = T.words[0] if allowed is None or allowed.dtype is T.words[0] else T.words[1]
        self.device = dev
        self.c = gpt2_logit_rules(
            at("history", T.i32), at("history_len", T.i32), at("gen_start", T.i32), at("repetition", T.f32),
            at("presence", T.f32), at("frequency", T.f32), at("bias_ids", T.i32), at("bias_values", T.f32),
            at("allowed", words), width["history"], width["bias_ids"], width["allowed"],
            int(append and (history is None or width["history"] > 0)))
        self._ref = ctypes.byref(self.c)


def _rules(where, rules, rows, dev):
    if rules.rows is not None and (rules.rows != rows or rules.device != dev):
        raise Gpt2Error(-1, f"{where}: rules for {rules.rows} rows on device {rules.device}, logits of {rows} on {dev}")
    return rules._ref


def gpt2_op_logit_rules(logits, ld, out, ldo, rows, vocab, rules, next_tokens=None, pos=None, stream=None):
    """out [rows, ldo] = logits [rows, ld] under `rules` (a LogitRules); next_tokens: the greedy choice."""
    T, f = _T or _torch(), "gpt2_op_logit_rules"
    dev, st = _where(stream, T)
    rc = T.rules(_buf(f, "logits", logits, T.f32, dev, _extent(rows, ld, vocab), ld), ld,
                 _buf(f, "out", out, T.f32, dev, _extent(rows, ldo, vocab), ldo), ldo, rows, vocab, _rules(f, rules, rows, dev),
                 None if next_tokens is None else _buf(f, "next_tokens", next_tokens, T.i32, dev, rows, 0),
                 None if pos is None else _buf(f, "pos", pos, T.i32, dev, rows, 0), st)
    if rc:
        raise Gpt2Error(rc, f)


def gpt2_rules_next(ctx, logits, batch, rules, next_tokens, pos=None, stream=None):
    """gpt2_greedy_next under `rules` (a LogitRules); logits are rewritten in place."""
    T, f = _T or _torch(), "gpt2_rules_next"
    dev, st = _where(stream, T)
    _check(_lib().gpt2_rules_next(ctx, _logits(f, ctx, logits, batch, T, dev), batch, _rules(f, rules, batch, dev),
                                  _buf(f, "next_tokens", next_tokens, T.i32, dev, batch, 0),
                                  None if pos is None else _buf(f, "pos", pos, T.i32, dev, batch, 0), st), f)


def _logits(where, ctx, logits, batch, T, dev):
    """Address of a batch's logits, [batch, vocab_padded] of the context's model."""
    return _buf(where, "logits", logits, T.f32, dev, batch * getattr(ctx, "vocab_padded", 1), 0)


def gpt2_q4_bytes(cfg: gpt2_config, group: int) -> int:
    return int(_lib().gpt2_q4_bytes(ctypes.byref(cfg), group))


def gpt2_q4_pack(ctx, q4, group, stream=None):
    """q4: a device uint8 tensor of at least gpt2_q4_bytes(cfg, group) bytes."""
    T, f = _T or _torch(), "gpt2_q4_pack"
    dev, st = _where(stream, T)
    _check(_lib().gpt2_q4_pack(ctx, _buf(f, "q4", q4, T.u8, dev, 1, 0), _nbytes(q4), group, st), f)


def gpt2_decode_scratch_bytes(cfg: gpt2_config, batch: int, max_len: int, prefix_len: int) -> int:
    return int(_lib().gpt2_decode_scratch_bytes(ctypes.byref(cfg), batch, max_len, prefix_len))


def gpt2_decode_step_ex(ctx, cache, batch, max_len, tokens, pos, opts, logits, stream=None):
    """gpt2_decode_step with a gpt2_decode_opts (or None), whose addresses and sizes the caller vouches for."""
    T, f = _T or _torch(), "gpt2_decode_step_ex"
    dev, st = _where(stream, T)
    _check(_lib().gpt2_decode_step_ex(ctx, _buf(f, "cache", cache, T.u8, dev, 1, 0), _nbytes(cache), batch, max_len,
                                      _buf(f, "tokens", tokens, T.i32, dev, batch, 0),
                                      _buf(f, "pos", pos, T.i32, dev, batch, 0),
                                      None if opts is None else ctypes.byref(opts),
                                      _logits(f, ctx, logits, batch, T, dev), st), f)


# ------------------------------------------------------------ convenience ---

@dataclass(frozen=True)
class ModelConfig:
    n_layer: int
    d_model: int
    n_head: int
    n_ctx: int
    vocab_real: int
    vocab_padded: int
    max_batch: int
    mode: int = 0  # 0 bf16 tensor cores, 1 fp32 correctness mode, 2 bf16 bitwise repeatable

    def c(self) -> gpt2_config:
        return make_config(self.n_layer, self.d_model, self.n_head, self.n_ctx, self.vocab_real,
                           self.vocab_padded, self.max_batch, self.mode)


GPT2_124M = ModelConfig(12, 768, 12, 1024, 50257, 50304, 16)
GPT2_350M = ModelConfig(24, 1024, 16, 1024, 50257, 50304, 16)
GPT2_1558M = ModelConfig(48, 1600, 25, 1024, 50257, 50304, 8)
GPT2_124M_T4096 = ModelConfig(12, 768, 12, 4096, 50257, 50304, 4)
GPT2_TINY = ModelConfig(2, 64, 4, 64, 512, 512, 4, mode=1)


class GPT2:
    """A context plus the torch-owned device buffers it runs on."""

    def __init__(self, mc: ModelConfig, device="cuda"):
        import torch
        self.mc = mc
        self.cfg = mc.c()
        n = gpt2_param_count(self.cfg)
        if n == 0:
            raise ValueError(f"invalid config {mc}")
        self.n_params = n
        f32 = dict(dtype=torch.float32, device=device)
        self.master = torch.zeros(n, **f32)
        self.grad = torch.zeros(n, **f32)
        self.m = torch.zeros(n, **f32)
        self.v = torch.zeros(n, **f32)
        self.shadow = torch.zeros(n, dtype=torch.bfloat16, device=device)
        wsb = gpt2_workspace_bytes(self.cfg, mc.max_batch)
        self.workspace = torch.empty(wsb, dtype=torch.uint8, device=device)
        self.loss = torch.zeros(1, **f32)
        self.ctx = gpt2_create(self.cfg, self.master, self.shadow, self.grad, self.m, self.v, self.workspace)
        self.layout = gpt2_tensors(self.cfg)

    def close(self):
        if self.ctx is not None:
            gpt2_destroy(self.ctx)
            self.ctx = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def view(self, flat, name):
        """View of one named tensor inside a flat buffer (master, grad, m, v)."""
        for nm, off, r, c in self.layout:
            if nm == name:
                t = flat[off:off + r * c]
                return t.view(r, c) if c > 1 else t
        raise KeyError(name)

    def init_params(self, seed=0):
        gpt2_init_params(self.ctx, seed)

    def refresh_shadow(self):
        gpt2_refresh_shadow(self.ctx)

    def forward_loss(self, tokens, targets):
        gpt2_forward_loss(self.ctx, tokens, targets, tokens.shape[0], self.loss)
        return self.loss

    def backward(self, grad_scale=1.0, accumulate=0):
        gpt2_backward(self.ctx, grad_scale, accumulate)

    def graph_capture(self, batch, grad_scale=1.0, accumulate=0, stream=None):
        """Record forward + loss + backward of one micro-batch into the
        context's CUDA graph (after at least one eager step).  The capture runs
        on a side stream of its own unless one is given."""
        import torch
        s = stream if stream is not None else torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        gpt2_graph_capture(self.ctx, batch, grad_scale, accumulate, self.loss, s)
        torch.cuda.current_stream().wait_stream(s)

    def graph_step(self, tokens, targets):
        """One captured micro-step on the current stream: the ids are copied in,
        then the graph runs (as forward_loss + backward)."""
        gpt2_graph_step(self.ctx, tokens, targets)

    def backward_bucketed(self, events, grad_scale=1.0, accumulate=0):
        """The backward recording events[i] when bucket i's gradients are
        final (see gpt2_backward_bucketed; n_layer + 2 events)."""
        gpt2_backward_bucketed(self.ctx, grad_scale, accumulate, events)

    def adamw_step(self, step, lr=6e-4, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, max_norm=0.0):
        """AdamW over the flat buffer; max_norm > 0 clips the gradient to that
        global norm first (on the device)."""
        if max_norm > 0.0:
            gpt2_adamw_step_clip(self.ctx, lr, beta1, beta2, eps, weight_decay, step, max_norm)
        else:
            gpt2_adamw_step(self.ctx, lr, beta1, beta2, eps, weight_decay, step)

    def adamw_step_range(self, step, offset, count, lr=6e-4, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1):
        """AdamW on elements [offset, offset + count) only (one shard of the
        optimizer state)."""
        gpt2_adamw_step_range(self.ctx, lr, beta1, beta2, eps, weight_decay, step, offset, count)

    def grad_norm(self):
        """Global L2 norm of the gradient buffer as a device fp32 scalar tensor."""
        import torch
        out = torch.empty(1, dtype=torch.float32, device=self.grad.device)
        gpt2_grad_norm(self.ctx, out)
        return out

    def zero_grad(self):
        gpt2_zero_grad(self.ctx)

    def status(self) -> int:
        return gpt2_get_status(self.ctx)

    def step_host(self, tokens_host, targets_host, loss_host, step, lr=6e-4, beta1=0.9, beta2=0.95,
                  eps=1e-8, weight_decay=0.1):
        gpt2_step_host(self.ctx, tokens_host, targets_host, tokens_host.shape[0], loss_host, lr, beta1,
                       beta2, eps, weight_decay, step)


class Q4Weights:
    """4-bit weights of one GPT2 context for decoding, in groups of ``group``
    inputs (modes 0 and 2).  ``pack()`` quantises the context's current master
    weights; call it again after they change."""

    def __init__(self, model: "GPT2", group: int = 64):
        import torch
        nbytes = gpt2_q4_bytes(model.cfg, group)
        if nbytes == 0:
            raise ValueError(f"no 4-bit form with group={group} for {model.mc}")
        self.model, self.group = model, group
        self.buf = torch.empty(nbytes, dtype=torch.uint8, device=model.master.device)
        self.pack()

    def pack(self):
        gpt2_q4_pack(self.model.ctx, self.buf, self.group)


class KVCache:
    """Key/value cache of one GPT2 context for ``batch`` sequences of up to
    ``max_len`` positions, with the device-side token, position and logits
    buffers a decode loop runs on (so the loop can be captured in a CUDA
    graph).

    ``q4``: a Q4Weights whose weights the steps read.  ``prefill`` has no 4-bit
    form and computes the prompt with the model's own weights, so that keys,
    values and the first choice are those of the unrounded model; a prompt fed
    by ``step`` sees the 4-bit weights throughout.  ``prefix``: a KVCache of
    one sequence, already filled, whose first ``prefix_len`` positions precede
    every row's own (``prefix_len + max_len <= n_ctx``); the rows' own tokens,
    prompts included, are then fed by ``step``, with ``pos += 1`` after each
    but the last, which ``greedy_advance`` follows."""

    def __init__(self, model: "GPT2", batch: int, max_len: int, prefix: "KVCache" = None, prefix_len: int = 0,
                 q4: Q4Weights = None):
        import torch
        nbytes = gpt2_kv_cache_bytes(model.cfg, batch, max_len)
        if nbytes == 0:
            raise ValueError(f"invalid cache size batch={batch} max_len={max_len}")
        if q4 is not None and q4.model is not model:
            raise ValueError("q4 holds the weights of another model")
        if prefix is not None and (prefix.model is not model or prefix.batch != 1 or prefix.opts_prefix):
            raise ValueError("a prefix is a KVCache of the same model with one row and no prefix of its own")
        if prefix is None and prefix_len or not 0 <= prefix_len <= (prefix.max_len if prefix is not None else 0) or \
                prefix_len + max_len > model.mc.n_ctx:
            raise ValueError(f"invalid prefix_len {prefix_len}")
        dev = model.master.device
        self.model, self.batch, self.max_len = model, batch, max_len
        self.buf = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        self.tokens = torch.zeros(batch, dtype=torch.int32, device=dev)
        self.pos = torch.zeros(batch, dtype=torch.int32, device=dev)
        self.logits = torch.zeros(batch, model.cfg.vocab_padded, dtype=torch.float32, device=dev)
        self.prefix, self.q4, self.opts = prefix, q4, None
        self.opts_prefix = prefix is not None and prefix_len > 0
        if q4 is not None or self.opts_prefix:
            self.opts = gpt2_decode_opts()
            if q4 is not None:
                self.opts.q4, self.opts.q4_bytes, self.opts.q4_group = q4.buf.data_ptr(), _nbytes(q4.buf), q4.group
            if self.opts_prefix:
                n = gpt2_decode_scratch_bytes(model.cfg, batch, max_len, prefix_len)
                self.scratch = torch.empty(n, dtype=torch.uint8, device=dev)
                self.opts.prefix, self.opts.prefix_bytes = prefix.buf.data_ptr(), _nbytes(prefix.buf)
                self.opts.prefix_cap, self.opts.prefix_len = prefix.max_len, prefix_len
                self.opts.scratch, self.opts.scratch_bytes = self.scratch.data_ptr(), n

    def prefill(self, tokens, prompt_len):
        """tokens: int32 [batch, n_ctx] (device); prompt_len: int32 [batch]
        (device).  Leaves the logits after each prompt in self.logits, the
        greedy next id in self.tokens and self.pos = prompt_len.  Reads the
        model's own weights, with q4 too."""
        if self.opts_prefix:
            raise ValueError("rows behind a prefix are fed by step(): prefill would not see the prefix")
        gpt2_prefill(self.model.ctx, self.buf, self.batch, self.max_len, tokens, prompt_len, self.logits)
        self.pos.copy_(prompt_len)
        gpt2_greedy_next(self.model.ctx, self.logits, self.batch, self.tokens)
        return self.logits

    def step(self, tokens=None, pos=None):
        """One decode step on self.tokens / self.pos (or the given device
        tensors); returns the logits [batch, vocab_padded].  self.pos stays."""
        tokens, pos = self.tokens if tokens is None else tokens, self.pos if pos is None else pos
        if self.opts is None:
            gpt2_decode_step(self.model.ctx, self.buf, self.batch, self.max_len, tokens, pos, self.logits)
        else:
            gpt2_decode_step_ex(self.model.ctx, self.buf, self.batch, self.max_len, tokens, pos, self.opts, self.logits)
        return self.logits

    def greedy_advance(self, rules: LogitRules = None):
        """self.tokens = greedy choice from self.logits (under `rules`, which
        rewrite self.logits); self.pos += 1."""
        if rules is None:
            gpt2_greedy_next(self.model.ctx, self.logits, self.batch, self.tokens, self.pos)
        else:
            gpt2_rules_next(self.model.ctx, self.logits, self.batch, rules, self.tokens, self.pos)
