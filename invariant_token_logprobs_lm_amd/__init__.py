"""Python binding of libitl.so: the invariant token-logprob library (MI355X).

Thin ctypes marshalling over the C ABI declared in include/itl.h: every
function checks tensor dtypes, devices and contiguity, allocates outputs and
workspace with torch (PyTorch supplies device memory and the current stream
only) and calls the library; every step of the computation runs in the
library's HIP kernels. There is no fallback: if libitl.so is missing, importing
this package fails.

Entry points (same names as the C ABI without the ``itl_`` prefix):

* ``lmhead_logprob(H, W, tokens) -> (logprob, lse)``
* ``group_advantage(rewards, group_offsets) -> advantages``
* ``reinforce_zero_loss(logprob, rollout_logprob, advantages, resp_offsets) -> (resp_loss, loss, coef)``
* ``reinforce_zero_backward(H, W, tokens, lse, coef) -> (dH, dW)``
* ``mismatch_stats(logprob, rollout_logprob, same_weights_logprob=None) -> stats``
* ``quantize_rows_fp8(X) -> (Xq, scale)``,
  ``lmhead_logprob_fp8(Hq, h_scale, Wq, w_scale, tokens) -> (logprob, lse)``
* ``quantize_rows_mxfp4(X) -> (Xq4, scale_codes)``,
  ``lmhead_logprob_mxfp4(Hq, h_scale, Wq4, w_scale_codes, tokens) -> (logprob, lse)``
* ``residual_norm(x, y, w_pre) -> (h, u, rstd_pre, rstd_post)``,
  ``residual_norm_fp8(x, y, w_pre) -> (h, Uq, u_scale, rstd_pre, rstd_post)``,
  ``residual_norm_backward(du, dh, h, y, w_pre, rstd_pre) -> (dx, dy, dw_pre, dw_post, dgate)``
* ``cross_entropy(H, W, targets) -> (loss, token_loss, lse)``,
  ``cross_entropy_grad(H, W, targets) -> (loss, token_loss, lse, dH, dW)``
* ``adamw_plan(params, grads, lr=...) -> plan``, ``adamw_step(plan) -> grad_norm``
* ``check_inputs(tokens, vocab, resp_offsets=None)``, ``build_info()``
"""

import ctypes
import operator
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libitl.so")

ITL_OK = 0
ITL_BF16 = 0
ITL_F32 = 1

_c_void_p = ctypes.c_void_p
_i64 = ctypes.c_int64
_i32 = ctypes.c_int32
_size = ctypes.c_size_t


_f32 = ctypes.c_float
_f64 = ctypes.c_double


class _AdamWTensor(ctypes.Structure):
    """itl_adamw_tensor."""

    _fields_ = [("param", _c_void_p), ("grad", _c_void_p), ("n", _i64), ("param_dtype", _i32), ("grad_dtype", _i32),
                ("weight_decay", _f32)]


class ItlError(RuntimeError):
    """A non-OK status from the library."""

    def __init__(self, status, message):
        super().__init__(message)
        self.status = status


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is not built; run `python -m invariant_token_logprobs_lm_amd.build` "
            "(there is no fallback implementation)"
        )
    lib = ctypes.CDLL(LIB_PATH)
    sig = {
        "itl_lmhead_logprob_workspace_bytes": (_size, [_i64, _i64]),
        "itl_lmhead_logprob": (ctypes.c_int, [_c_void_p, _c_void_p, ctypes.c_int, _i64, _i64, _i64, _c_void_p,
                                              _c_void_p, _c_void_p, _c_void_p, _size, _c_void_p]),
        "itl_lmhead_logprob_noalloc": (ctypes.c_int, [_c_void_p, _c_void_p, ctypes.c_int, _i64, _i64, _i64,
                                                      _c_void_p, _c_void_p, _c_void_p, _c_void_p]),
        "itl_lmhead_logprob_keep_logits": (ctypes.c_int, [_c_void_p, _c_void_p, ctypes.c_int, _i64, _i64, _i64,
                                                          _c_void_p, _c_void_p, _c_void_p, _c_void_p, _i64,
                                                          _c_void_p, _size, _c_void_p]),
        "itl_group_advantage": (ctypes.c_int, [_c_void_p, _c_void_p, _i32, _i32, _c_void_p, _c_void_p]),
        "itl_reinforce_zero_loss_workspace_bytes": (_size, [_i64, _i32]),
        "itl_reinforce_zero_loss": (ctypes.c_int, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _i32, _i64,
                                                   _c_void_p, _c_void_p, _c_void_p, _c_void_p, _size, _c_void_p]),
        "itl_reinforce_zero_backward_workspace_bytes": (_size, [_i64, _i64, _i64, ctypes.c_int]),
        "itl_reinforce_zero_backward": (ctypes.c_int, [_c_void_p, _c_void_p, ctypes.c_int, _i64, _i64, _i64,
                                                       _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                                       _c_void_p, _size, _c_void_p]),
        "itl_reinforce_zero_backward_from_logits": (ctypes.c_int, [_c_void_p, _c_void_p, ctypes.c_int, _i64, _i64,
                                                                   _i64, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                                                   _i64, _c_void_p, _c_void_p, _c_void_p, _size,
                                                                   _c_void_p]),
        "itl_quantize_rows_fp8": (ctypes.c_int, [_c_void_p, ctypes.c_int, _i64, _i64, _c_void_p, _c_void_p,
                                                 _c_void_p]),
        "itl_lmhead_logprob_fp8": (ctypes.c_int, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _i64, _i64, _i64,
                                                  _c_void_p, _c_void_p, _c_void_p, _c_void_p, _size, _c_void_p]),
        "itl_quantize_rows_mxfp4": (ctypes.c_int, [_c_void_p, ctypes.c_int, _i64, _i64, _c_void_p, _c_void_p,
                                                   _c_void_p]),
        "itl_lmhead_logprob_mxfp4": (ctypes.c_int, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _i64, _i64, _i64,
                                                    _c_void_p, _c_void_p, _c_void_p, _c_void_p, _size, _c_void_p]),
        "itl_residual_norm": (ctypes.c_int, [_c_void_p, _c_void_p, _c_void_p, _i64, _c_void_p, _c_void_p, ctypes.c_int,
                                             _i64, _i64, _f32, _f32, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                             _c_void_p]),
        "itl_residual_norm_fp8": (ctypes.c_int, [_c_void_p, _c_void_p, _c_void_p, _i64, _c_void_p, _c_void_p,
                                                 ctypes.c_int, _i64, _i64, _f32, _f32, _c_void_p, _c_void_p, _c_void_p,
                                                 _c_void_p, _c_void_p, _c_void_p]),
        "itl_residual_norm_backward_workspace_bytes": (_size, [_i64, _i64]),
        "itl_residual_norm_backward": (ctypes.c_int, [_c_void_p, ctypes.c_int, _c_void_p, _c_void_p, _c_void_p,
                                                      _c_void_p, _i64, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                                      ctypes.c_int, _i64, _i64, _f32, _c_void_p, _c_void_p, _c_void_p,
                                                      _c_void_p, _c_void_p, _c_void_p, _size, _c_void_p]),
        "itl_cross_entropy_workspace_bytes": (_size, [_i64, _i64, _i64, ctypes.c_int, _i32, ctypes.c_int]),
        "itl_cross_entropy": (ctypes.c_int, [_c_void_p, _c_void_p, ctypes.c_int, _i64, _i64, _i64, _c_void_p, _f32,
                                             _f32, _i32, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _size,
                                             _c_void_p]),
        "itl_cross_entropy_grad": (ctypes.c_int, [_c_void_p, _c_void_p, ctypes.c_int, _i64, _i64, _i64, _c_void_p,
                                                  _f32, _f32, _i32, _f32, ctypes.c_int, _c_void_p, _c_void_p,
                                                  _c_void_p, _c_void_p, _c_void_p, _c_void_p, _size, _c_void_p]),
        "itl_adamw_plan_sizes": (ctypes.c_int, [ctypes.POINTER(_AdamWTensor), _i32, ctypes.POINTER(_i64),
                                                ctypes.POINTER(_i64)]),
        "itl_adamw_plan": (ctypes.c_int, [ctypes.POINTER(_AdamWTensor), _i32, _c_void_p, _size]),
        "itl_adamw_step_workspace_bytes": (_size, []),
        "itl_adamw_step": (ctypes.c_int, [_c_void_p, _size, _i32, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                          _c_void_p, _c_void_p, _c_void_p, _f64, _f64, _f64, _f32, _c_void_p,
                                          _c_void_p, _size, _c_void_p]),
        "itl_mismatch_stats_workspace_bytes": (_size, [_i64]),
        "itl_mismatch_stats": (ctypes.c_int, [_c_void_p, _c_void_p, _c_void_p, _i64, _c_void_p, _c_void_p, _size,
                                              _c_void_p]),
        "itl_check_inputs": (ctypes.c_int, [_c_void_p, _i64, _i64, _c_void_p, _i32, _c_void_p]),
        "itl_status_string": (ctypes.c_char_p, [ctypes.c_int]),
        "itl_last_error": (ctypes.c_char_p, []),
        "itl_build_info": (ctypes.c_char_p, []),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


lib = _load()

EXPORTS = (
    "itl_lmhead_logprob_workspace_bytes",
    "itl_lmhead_logprob",
    "itl_lmhead_logprob_noalloc",
    "itl_lmhead_logprob_keep_logits",
    "itl_group_advantage",
    "itl_reinforce_zero_loss_workspace_bytes",
    "itl_reinforce_zero_loss",
    "itl_reinforce_zero_backward_workspace_bytes",
    "itl_reinforce_zero_backward",
    "itl_reinforce_zero_backward_from_logits",
    "itl_quantize_rows_fp8",
    "itl_lmhead_logprob_fp8",
    "itl_quantize_rows_mxfp4",
    "itl_lmhead_logprob_mxfp4",
    "itl_residual_norm",
    "itl_residual_norm_fp8",
    "itl_residual_norm_backward_workspace_bytes",
    "itl_residual_norm_backward",
    "itl_cross_entropy_workspace_bytes",
    "itl_cross_entropy",
    "itl_cross_entropy_grad",
    "itl_adamw_plan_sizes",
    "itl_adamw_plan",
    "itl_adamw_step_workspace_bytes",
    "itl_adamw_step",
    "itl_mismatch_stats_workspace_bytes",
    "itl_mismatch_stats",
    "itl_check_inputs",
    "itl_status_string",
    "itl_last_error",
    "itl_build_info",
)


def build_info():
    return lib.itl_build_info().decode()


def _check(status):
    if status != ITL_OK:
        msg = lib.itl_status_string(status).decode()
        detail = lib.itl_last_error().decode()
        raise ItlError(status, f"{msg}: {detail}" if detail else msg)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream_handle(index):
    return torch.cuda.current_stream(index).cuda_stream


# The current stream's handle by device index, without the Stream object that
# torch.cuda.current_stream builds (0.1 us against 1.9 us of a small call's 16),
# where torch has the query: it is private to its GPU builds.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _stream_handle)


def _stream(device):
    return _raw_stream(device.index)


def _need(t, name, dtypes, device=None, ndim=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} has dtype {t.dtype}; expected one of {dtypes}")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on a HIP device, got {t.device}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions, got {t.dim()}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


_HEAD_DTYPES = {torch.bfloat16: ITL_BF16, torch.float32: ITL_F32}


def lmhead_workspace_bytes(n_tok, vocab):
    return int(lib.itl_lmhead_logprob_workspace_bytes(n_tok, vocab))


def lmhead_logprob(H, W, tokens, *, logprob=None, lse=None, workspace=None, want_lse=True):
    """Sampled-token logprob and log-normaliser of every row of H.

    H [n_tok, d] and W [vocab, d] (bf16 or fp32, same dtype), tokens int32
    [n_tok]. Returns (logprob fp32 [n_tok], lse fp32 [n_tok] or None).
    """
    _need(H, "H", tuple(_HEAD_DTYPES), ndim=2)
    _need(W, "W", (H.dtype,), device=H.device, ndim=2)
    _need(tokens, "tokens", (torch.int32,), device=H.device, ndim=1)
    n_tok, d = H.shape
    vocab = W.shape[0]
    if W.shape[1] != d or tokens.shape[0] != n_tok:
        raise ValueError(f"shape mismatch: H {tuple(H.shape)}, W {tuple(W.shape)}, tokens {tuple(tokens.shape)}")
    if logprob is None:
        logprob = torch.empty(n_tok, dtype=torch.float32, device=H.device)
    if lse is None and want_lse:
        lse = torch.empty(n_tok, dtype=torch.float32, device=H.device)
    for name, t in (("logprob", logprob), ("lse", lse)):
        if t is not None:
            _need(t, name, (torch.float32,), device=H.device, ndim=1)
            if t.shape[0] != n_tok:
                raise ValueError(f"{name} must have {n_tok} elements")
    need = lmhead_workspace_bytes(n_tok, vocab)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=H.device)
    _need(workspace, "workspace", (torch.uint8,), device=H.device)
    _check(lib.itl_lmhead_logprob(_ptr(H), _ptr(W), _HEAD_DTYPES[H.dtype], n_tok, d, vocab, _ptr(tokens),
                                  _ptr(logprob), _ptr(lse), _ptr(workspace), workspace.numel(),
                                  _stream(H.device)))
    return logprob, lse


def lmhead_logprob_noalloc(H, W, tokens, *, logprob=None, lse=None, want_lse=True):
    """lmhead_logprob without a workspace (the library's static per-GPU
    scratch; at most 16,368 tokens for large vocabularies). Same bits."""
    _need(H, "H", tuple(_HEAD_DTYPES), ndim=2)
    _need(W, "W", (H.dtype,), device=H.device, ndim=2)
    _need(tokens, "tokens", (torch.int32,), device=H.device, ndim=1)
    n_tok, d = H.shape
    vocab = W.shape[0]
    if W.shape[1] != d or tokens.shape[0] != n_tok:
        raise ValueError(f"shape mismatch: H {tuple(H.shape)}, W {tuple(W.shape)}, tokens {tuple(tokens.shape)}")
    if logprob is None:
        logprob = torch.empty(n_tok, dtype=torch.float32, device=H.device)
    if lse is None and want_lse:
        lse = torch.empty(n_tok, dtype=torch.float32, device=H.device)
    for name, t in (("logprob", logprob), ("lse", lse)):
        if t is not None:
            _need(t, name, (torch.float32,), device=H.device, ndim=1)
            if t.shape[0] != n_tok:
                raise ValueError(f"{name} must have {n_tok} elements")
    _check(lib.itl_lmhead_logprob_noalloc(_ptr(H), _ptr(W), _HEAD_DTYPES[H.dtype], n_tok, d, vocab, _ptr(tokens),
                                          _ptr(logprob), _ptr(lse), _stream(H.device)))
    return logprob, lse


def lmhead_logprob_keep_logits(H, W, tokens, *, logits=None, logprob=None, lse=None, workspace=None):
    """lmhead_logprob (same bits) that also returns the logits z [n_tok, ld]
    fp32 (ld = vocab rounded up to a multiple of 4 when allocated here; a
    caller's buffer may have any ld >= vocab that is a multiple of 4).
    Returns (logprob, lse, logits)."""
    _need(H, "H", tuple(_HEAD_DTYPES), ndim=2)
    _need(W, "W", (H.dtype,), device=H.device, ndim=2)
    _need(tokens, "tokens", (torch.int32,), device=H.device, ndim=1)
    n_tok, d = H.shape
    vocab = W.shape[0]
    if W.shape[1] != d or tokens.shape[0] != n_tok:
        raise ValueError(f"shape mismatch: H {tuple(H.shape)}, W {tuple(W.shape)}, tokens {tuple(tokens.shape)}")
    if logits is None:
        logits = torch.empty((n_tok, (vocab + 3) // 4 * 4), dtype=torch.float32, device=H.device)
    _need(logits, "logits", (torch.float32,), device=H.device, ndim=2)
    if logits.shape[0] != n_tok:
        raise ValueError(f"logits must have {n_tok} rows")
    if logprob is None:
        logprob = torch.empty(n_tok, dtype=torch.float32, device=H.device)
    if lse is None:
        lse = torch.empty(n_tok, dtype=torch.float32, device=H.device)
    for name, t in (("logprob", logprob), ("lse", lse)):
        _need(t, name, (torch.float32,), device=H.device, ndim=1)
        if t.shape[0] != n_tok:
            raise ValueError(f"{name} must have {n_tok} elements")
    need = lmhead_workspace_bytes(n_tok, vocab)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=H.device)
    _need(workspace, "workspace", (torch.uint8,), device=H.device)
    _check(lib.itl_lmhead_logprob_keep_logits(_ptr(H), _ptr(W), _HEAD_DTYPES[H.dtype], n_tok, d, vocab, _ptr(tokens),
                                              _ptr(logprob), _ptr(lse), _ptr(logits), logits.shape[1],
                                              _ptr(workspace), workspace.numel(), _stream(H.device)))
    return logprob, lse, logits


def group_advantage(rewards, group_offsets, *, advantages=None):
    """advantages[i] = rewards[i] - mean reward of i's group (fp32)."""
    _need(rewards, "rewards", (torch.float32,), ndim=1)
    _need(group_offsets, "group_offsets", (torch.int32,), device=rewards.device, ndim=1)
    n_resp = rewards.shape[0]
    n_groups = group_offsets.shape[0] - 1
    if n_groups < 0:
        raise ValueError("group_offsets needs at least one element")
    if advantages is None:
        advantages = torch.empty_like(rewards)
    _need(advantages, "advantages", (torch.float32,), device=rewards.device, ndim=1)
    _check(lib.itl_group_advantage(_ptr(rewards), _ptr(group_offsets), n_groups, n_resp, _ptr(advantages),
                                   _stream(rewards.device)))
    return advantages


def loss_workspace_bytes(n_tok, n_resp):
    return int(lib.itl_reinforce_zero_loss_workspace_bytes(n_tok, n_resp))


def reinforce_zero_loss(logprob, rollout_logprob, advantages, resp_offsets, *, want_coef=True, workspace=None):
    """(resp_loss fp32 [N], loss fp32 [1], coef fp32 [n_tok] or None)."""
    _need(logprob, "logprob", (torch.float32,), ndim=1)
    dev = logprob.device
    _need(rollout_logprob, "rollout_logprob", (torch.float32,), device=dev, ndim=1)
    _need(advantages, "advantages", (torch.float32,), device=dev, ndim=1)
    _need(resp_offsets, "resp_offsets", (torch.int64,), device=dev, ndim=1)
    n_tok = logprob.shape[0]
    n_resp = advantages.shape[0]
    if rollout_logprob.shape[0] != n_tok or resp_offsets.shape[0] != n_resp + 1:
        raise ValueError("shape mismatch between logprobs, advantages and resp_offsets")
    resp_loss = torch.empty(n_resp, dtype=torch.float32, device=dev)
    loss = torch.empty(1, dtype=torch.float32, device=dev)
    coef = torch.empty(n_tok, dtype=torch.float32, device=dev) if want_coef else None
    need = loss_workspace_bytes(n_tok, n_resp)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    _need(workspace, "workspace", (torch.uint8,), device=dev)
    _check(lib.itl_reinforce_zero_loss(_ptr(logprob), _ptr(rollout_logprob), _ptr(advantages), _ptr(resp_offsets),
                                       n_resp, n_tok, _ptr(resp_loss), _ptr(loss), _ptr(coef), _ptr(workspace),
                                       workspace.numel(), _stream(dev)))
    return resp_loss, loss, coef


def backward_workspace_bytes(n_tok, d, vocab, dtype=torch.bfloat16):
    return int(lib.itl_reinforce_zero_backward_workspace_bytes(n_tok, d, vocab, _HEAD_DTYPES[dtype]))


def reinforce_zero_backward(H, W, tokens, lse, coef, *, dH=None, dW=None, workspace=None):
    """(dH fp32 [n_tok, d], dW fp32 [vocab, d]) of the REINFORCE Zero loss."""
    _need(H, "H", tuple(_HEAD_DTYPES), ndim=2)
    dev = H.device
    _need(W, "W", (H.dtype,), device=dev, ndim=2)
    _need(tokens, "tokens", (torch.int32,), device=dev, ndim=1)
    _need(lse, "lse", (torch.float32,), device=dev, ndim=1)
    _need(coef, "coef", (torch.float32,), device=dev, ndim=1)
    n_tok, d = H.shape
    vocab = W.shape[0]
    if W.shape[1] != d or tokens.shape[0] != n_tok or lse.shape[0] != n_tok or coef.shape[0] != n_tok:
        raise ValueError("shape mismatch between H, W, tokens, lse and coef")
    if dH is None:
        dH = torch.empty((n_tok, d), dtype=torch.float32, device=dev)
    if dW is None:
        dW = torch.empty((vocab, d), dtype=torch.float32, device=dev)
    _need(dH, "dH", (torch.float32,), device=dev, ndim=2)
    _need(dW, "dW", (torch.float32,), device=dev, ndim=2)
    need = backward_workspace_bytes(n_tok, d, vocab, H.dtype)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    _need(workspace, "workspace", (torch.uint8,), device=dev)
    _check(lib.itl_reinforce_zero_backward(_ptr(H), _ptr(W), _HEAD_DTYPES[H.dtype], n_tok, d, vocab, _ptr(tokens),
                                           _ptr(lse), _ptr(coef), _ptr(dH), _ptr(dW), _ptr(workspace),
                                           workspace.numel(), _stream(dev)))
    return dH, dW


def reinforce_zero_backward_from_logits(H, W, tokens, lse, coef, logits, *, dH=None, dW=None, workspace=None):
    """reinforce_zero_backward (same bits) with the dlogits formed from the
    logits kept by lmhead_logprob_keep_logits ([n_tok, ld] fp32)."""
    _need(H, "H", tuple(_HEAD_DTYPES), ndim=2)
    dev = H.device
    _need(W, "W", (H.dtype,), device=dev, ndim=2)
    _need(tokens, "tokens", (torch.int32,), device=dev, ndim=1)
    _need(lse, "lse", (torch.float32,), device=dev, ndim=1)
    _need(coef, "coef", (torch.float32,), device=dev, ndim=1)
    _need(logits, "logits", (torch.float32,), device=dev, ndim=2)
    n_tok, d = H.shape
    vocab = W.shape[0]
    if (W.shape[1] != d or tokens.shape[0] != n_tok or lse.shape[0] != n_tok or coef.shape[0] != n_tok
            or logits.shape[0] != n_tok):
        raise ValueError("shape mismatch between H, W, tokens, lse, coef and logits")
    if dH is None:
        dH = torch.empty((n_tok, d), dtype=torch.float32, device=dev)
    if dW is None:
        dW = torch.empty((vocab, d), dtype=torch.float32, device=dev)
    _need(dH, "dH", (torch.float32,), device=dev, ndim=2)
    _need(dW, "dW", (torch.float32,), device=dev, ndim=2)
    need = backward_workspace_bytes(n_tok, d, vocab, H.dtype)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    _need(workspace, "workspace", (torch.uint8,), device=dev)
    _check(lib.itl_reinforce_zero_backward_from_logits(_ptr(H), _ptr(W), _HEAD_DTYPES[H.dtype], n_tok, d, vocab,
                                                       _ptr(tokens), _ptr(lse), _ptr(coef), _ptr(logits),
                                                       logits.shape[1], _ptr(dH), _ptr(dW), _ptr(workspace),
                                                       workspace.numel(), _stream(dev)))
    return dH, dW


def quantize_rows_fp8(X, *, Xq=None, scale=None):
    """Per-row E4M3 codes (uint8 [n, d]) and fp32 scales [n] of a bf16 or
    fp32 matrix [n, d] (d a multiple of 128)."""
    _need(X, "X", tuple(_HEAD_DTYPES), ndim=2)
    n, d = X.shape
    if Xq is None:
        Xq = torch.empty((n, d), dtype=torch.uint8, device=X.device)
    if scale is None:
        scale = torch.empty(n, dtype=torch.float32, device=X.device)
    _need(Xq, "Xq", (torch.uint8,), device=X.device, ndim=2)
    _need(scale, "scale", (torch.float32,), device=X.device, ndim=1)
    if tuple(Xq.shape) != (n, d) or scale.shape[0] != n:
        raise ValueError("Xq must be [n, d] and scale [n]")
    _check(lib.itl_quantize_rows_fp8(_ptr(X), _HEAD_DTYPES[X.dtype], n, d, _ptr(Xq), _ptr(scale), _stream(X.device)))
    return Xq, scale


def lmhead_logprob_fp8(Hq, h_scale, Wq, w_scale, tokens, *, logprob=None, lse=None, workspace=None, want_lse=True):
    """Sampled-token logprob and lse from an E4M3 head with per-row scales
    (as written by quantize_rows_fp8)."""
    _need(Hq, "Hq", (torch.uint8,), ndim=2)
    dev = Hq.device
    _need(h_scale, "h_scale", (torch.float32,), device=dev, ndim=1)
    _need(Wq, "Wq", (torch.uint8,), device=dev, ndim=2)
    _need(w_scale, "w_scale", (torch.float32,), device=dev, ndim=1)
    _need(tokens, "tokens", (torch.int32,), device=dev, ndim=1)
    n_tok, d = Hq.shape
    vocab = Wq.shape[0]
    if Wq.shape[1] != d or h_scale.shape[0] != n_tok or w_scale.shape[0] != vocab or tokens.shape[0] != n_tok:
        raise ValueError("shape mismatch between Hq, h_scale, Wq, w_scale and tokens")
    if logprob is None:
        logprob = torch.empty(n_tok, dtype=torch.float32, device=dev)
    if lse is None and want_lse:
        lse = torch.empty(n_tok, dtype=torch.float32, device=dev)
    need = lmhead_workspace_bytes(n_tok, vocab)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    _need(workspace, "workspace", (torch.uint8,), device=dev)
    _check(lib.itl_lmhead_logprob_fp8(_ptr(Hq), _ptr(h_scale), _ptr(Wq), _ptr(w_scale), n_tok, d, vocab,
                                      _ptr(tokens), _ptr(logprob), _ptr(lse), _ptr(workspace), workspace.numel(),
                                      _stream(dev)))
    return logprob, lse


def quantize_rows_mxfp4(X, *, Xq=None, scale_codes=None):
    """MXFP4 of a bf16 or fp32 matrix [n, d] (d a multiple of 128): packed
    E2M1 codes uint8 [n, d / 2] and E8M0 scale codes uint8 [n, d / 32]."""
    _need(X, "X", tuple(_HEAD_DTYPES), ndim=2)
    n, d = X.shape
    if Xq is None:
        Xq = torch.empty((n, d // 2), dtype=torch.uint8, device=X.device)
    if scale_codes is None:
        scale_codes = torch.empty((n, d // 32), dtype=torch.uint8, device=X.device)
    _need(Xq, "Xq", (torch.uint8,), device=X.device, ndim=2)
    _need(scale_codes, "scale_codes", (torch.uint8,), device=X.device, ndim=2)
    if tuple(Xq.shape) != (n, d // 2) or tuple(scale_codes.shape) != (n, d // 32):
        raise ValueError("Xq must be [n, d/2] and scale_codes [n, d/32]")
    _check(lib.itl_quantize_rows_mxfp4(_ptr(X), _HEAD_DTYPES[X.dtype], n, d, _ptr(Xq), _ptr(scale_codes),
                                       _stream(X.device)))
    return Xq, scale_codes


def lmhead_logprob_mxfp4(Hq, h_scale, Wq4, w_scale_codes, tokens, *, logprob=None, lse=None, workspace=None,
                         want_lse=True):
    """Sampled-token logprob and lse from an MXFP4 head against E4M3 token
    rows (quantize_rows_mxfp4 / quantize_rows_fp8)."""
    _need(Hq, "Hq", (torch.uint8,), ndim=2)
    dev = Hq.device
    _need(h_scale, "h_scale", (torch.float32,), device=dev, ndim=1)
    _need(Wq4, "Wq4", (torch.uint8,), device=dev, ndim=2)
    _need(w_scale_codes, "w_scale_codes", (torch.uint8,), device=dev, ndim=2)
    _need(tokens, "tokens", (torch.int32,), device=dev, ndim=1)
    n_tok, d = Hq.shape
    vocab = Wq4.shape[0]
    if (Wq4.shape[1] * 2 != d or tuple(w_scale_codes.shape) != (vocab, d // 32) or h_scale.shape[0] != n_tok
            or tokens.shape[0] != n_tok):
        raise ValueError("shape mismatch between Hq, h_scale, Wq4, w_scale_codes and tokens")
    if logprob is None:
        logprob = torch.empty(n_tok, dtype=torch.float32, device=dev)
    if lse is None and want_lse:
        lse = torch.empty(n_tok, dtype=torch.float32, device=dev)
    need = lmhead_workspace_bytes(n_tok, vocab)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    _need(workspace, "workspace", (torch.uint8,), device=dev)
    _check(lib.itl_lmhead_logprob_mxfp4(_ptr(Hq), _ptr(h_scale), _ptr(Wq4), _ptr(w_scale_codes), n_tok, d, vocab,
                                        _ptr(tokens), _ptr(logprob), _ptr(lse), _ptr(workspace), workspace.numel(),
                                        _stream(dev)))
    return logprob, lse


def _new(shape, dtype, like, name, given):
    """`given`, checked, or a new tensor of that shape and dtype on like's device."""
    if given is None:
        if like.dtype == dtype and like.shape == shape:
            return torch.empty_like(like)
        return torch.empty(shape, dtype=dtype, device=like.device)
    _need(given, name, (dtype,), device=like.device, ndim=len(shape))
    if tuple(given.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(given.shape)}")
    return given


def _workspace(given, need, device):
    if given is None:  # (sizes the library refuses have no workspace: it says why)
        return torch.empty(max(need, 1) if need < 1 << 62 else 1, dtype=torch.uint8, device=device)
    _need(given, "workspace", (torch.uint8,), device=device)
    return given


def _launch(device, call, *args):
    """call(*args, the current stream of `device`), with `device` the current one."""
    if torch.cuda.current_device() == device.index:
        return _check(call(*args, _raw_stream(device.index)))
    with torch.cuda.device(device):
        return _check(call(*args, _raw_stream(device.index)))


def _norm_operands(x, y, w_pre, w_post, gate, first):
    """Checks what the norms' forward and backward share; (rows, d, gate stride)."""
    _need(x, first, tuple(_HEAD_DTYPES), ndim=2)
    n, d = x.shape
    if d == 0:
        raise ValueError(f"{first} must have at least one column")
    if y is not None:
        _need(y, "y", (x.dtype,), device=x.device, ndim=2)
        if y.shape != x.shape:
            raise ValueError(f"y must have {first}'s shape {tuple(x.shape)}, got {tuple(y.shape)}")
    elif w_post is not None or gate is not None:
        raise ValueError("w_post and gate need y")
    for name, w in (("w_pre", w_pre), ("w_post", w_post)):
        if w is None and name == "w_post":
            continue
        _need(w, name, (x.dtype,), device=x.device, ndim=1)
        if w.shape[0] != d:
            raise ValueError(f"{name} must have {d} elements")
    if gate is None:
        return n, d, 0
    _need(gate, "gate", (x.dtype,), device=x.device)
    if tuple(gate.shape) not in ((d,), (n, d)):
        raise ValueError(f"gate must have shape ({d},) or ({n}, {d}), got {tuple(gate.shape)}")
    return n, d, 0 if gate.dim() == 1 else d


def _stream_rows(x, y, h, n, d):
    """residual_norm's h: x itself without y."""
    if y is None:
        if h is not None and h is not x:
            raise ValueError("h needs y")
        return x
    return _new((n, d), x.dtype, x, "h", h)


def residual_norm(x, y, w_pre, *, w_post=None, gate=None, scale=1.0, eps=1e-6, h=None, u=None):
    """h = x + scale * gate * p and u = rmsnorm(h) * w_pre, where p = y, or
    rmsnorm(y) * w_post with w_post given.

    x, y [n, d] (bf16 or fp32; y None: h is x), w_pre, w_post [d], gate [d] or
    [n, d], all of one dtype. Returns (h, u, rstd_pre fp32 [n], rstd_post fp32
    [n] or None).
    """
    n, d, stride = _norm_operands(x, y, w_pre, w_post, gate, "x")
    h = _stream_rows(x, y, h, n, d)
    u = _new((n, d), x.dtype, x, "u", u)
    rstd_pre = torch.empty(n, dtype=torch.float32, device=x.device)
    rstd_post = None if w_post is None else torch.empty(n, dtype=torch.float32, device=x.device)
    _launch(x.device, lib.itl_residual_norm, _ptr(x), _ptr(y), _ptr(gate), stride, _ptr(w_post), _ptr(w_pre),
            _HEAD_DTYPES[x.dtype], n, d, scale, eps, _ptr(h), _ptr(u), _ptr(rstd_pre), _ptr(rstd_post))
    return h, u, rstd_pre, rstd_post


def residual_norm_fp8(x, y, w_pre, *, w_post=None, gate=None, scale=1.0, eps=1e-6, h=None, Uq=None, u_scale=None):
    """residual_norm with u as E4M3 codes (uint8 [n, d]) and a scale per row
    (fp32 [n]), as lmhead_logprob_fp8 takes them; d a multiple of 128. Returns
    (h, Uq, u_scale, rstd_pre, rstd_post)."""
    n, d, stride = _norm_operands(x, y, w_pre, w_post, gate, "x")
    h = _stream_rows(x, y, h, n, d)
    Uq = _new((n, d), torch.uint8, x, "Uq", Uq)
    u_scale = _new((n,), torch.float32, x, "u_scale", u_scale)
    rstd_pre = torch.empty(n, dtype=torch.float32, device=x.device)
    rstd_post = None if w_post is None else torch.empty(n, dtype=torch.float32, device=x.device)
    _launch(x.device, lib.itl_residual_norm_fp8, _ptr(x), _ptr(y), _ptr(gate), stride, _ptr(w_post), _ptr(w_pre),
            _HEAD_DTYPES[x.dtype], n, d, scale, eps, _ptr(h), _ptr(Uq), _ptr(u_scale), _ptr(rstd_pre),
            _ptr(rstd_post))
    return h, Uq, u_scale, rstd_pre, rstd_post


def residual_norm_backward_workspace_bytes(n_rows, d):
    return int(lib.itl_residual_norm_backward_workspace_bytes(n_rows, d))


def residual_norm_backward(du, dh, h, y, w_pre, rstd_pre, *, w_post=None, rstd_post=None, gate=None, scale=1.0,
                           dx=None, dy=None, dw_pre=None, dw_post=None, dgate=None, workspace=None):
    """Gradients of residual_norm: du [n, d] (h's dtype or fp32) and dh [n, d]
    (h's dtype, or None) are those of u and h. Returns (dx, dy, dw_pre fp32
    [d], dw_post fp32 [d], dgate: fp32 [d] for a shared gate, else like gate);
    dy, dw_post, dgate are None where y, w_post, gate are. Each may be given as
    a tensor to write into (the gradients that an adamw_plan holds). dx is the
    gradient of the residual stream x (all of h's)."""
    n, d, stride = _norm_operands(h, y, w_pre, w_post, gate, "h")
    dev = h.device
    _need(du, "du", (h.dtype, torch.float32), device=dev, ndim=2)
    if dh is not None:
        _need(dh, "dh", (h.dtype,), device=dev, ndim=2)
    for name, t in (("du", du), ("dh", dh)):
        if t is not None and t.shape != h.shape:
            raise ValueError(f"{name} must have shape {tuple(h.shape)}, got {tuple(t.shape)}")
    if w_post is not None and rstd_post is None:
        raise ValueError("w_post needs rstd_post")
    for name, t in (("rstd_pre", rstd_pre), ("rstd_post", rstd_post if w_post is not None else rstd_pre)):
        _need(t, name, (torch.float32,), device=dev, ndim=1)
        if t.shape[0] != n:
            raise ValueError(f"{name} must have {n} elements")
    if dy is not None and y is None:
        raise ValueError("dy needs y")
    if dw_post is not None and w_post is None:
        raise ValueError("dw_post needs w_post")
    if dgate is not None and gate is None:
        raise ValueError("dgate needs gate")
    dx = _new((n, d), h.dtype, h, "dx", dx)
    dy = None if y is None else _new((n, d), h.dtype, h, "dy", dy)
    dw_pre = _new((d,), torch.float32, h, "dw_pre", dw_pre)
    dw_post = None if w_post is None else _new((d,), torch.float32, h, "dw_post", dw_post)
    if gate is None:
        dgate = None
    else:
        dgate = _new((d,), torch.float32, h, "dgate", dgate) if stride == 0 else _new((n, d), h.dtype, h, "dgate", dgate)
    workspace = _workspace(workspace, residual_norm_backward_workspace_bytes(n, d), dev)
    _launch(dev, lib.itl_residual_norm_backward, _ptr(du), _HEAD_DTYPES[du.dtype], _ptr(dh), _ptr(h), _ptr(y),
            _ptr(gate), stride, _ptr(w_post), _ptr(w_pre), _ptr(rstd_pre),
            _ptr(rstd_post if w_post is not None else None), _HEAD_DTYPES[h.dtype], n, d, scale, _ptr(dx), _ptr(dy),
            _ptr(dgate), _ptr(dw_pre), _ptr(dw_post), _ptr(workspace), workspace.numel())
    return dx, dy, dw_pre, dw_post, dgate


_REDUCTIONS = {"sum": 0, "mean": 1}


def cross_entropy_workspace_bytes(n_tok, d, vocab, dtype=torch.bfloat16, grad_dtype=None):
    """Workspace of cross_entropy (grad_dtype None) or cross_entropy_grad."""
    grad = grad_dtype is not None
    return int(lib.itl_cross_entropy_workspace_bytes(n_tok, d, vocab, _HEAD_DTYPES[dtype], int(grad),
                                                     _HEAD_DTYPES[grad_dtype if grad else dtype]))


def _cross_entropy_operands(H, W, targets, reduction):
    _need(H, "H", tuple(_HEAD_DTYPES), ndim=2)
    _need(W, "W", (H.dtype,), device=H.device, ndim=2)
    _need(targets, "targets", (torch.int32,), device=H.device, ndim=1)
    if W.shape[1] != H.shape[1] or targets.shape[0] != H.shape[0]:
        raise ValueError(f"shape mismatch: H {tuple(H.shape)}, W {tuple(W.shape)}, targets {tuple(targets.shape)}")
    if reduction not in _REDUCTIONS:
        raise ValueError(f"reduction must be one of {tuple(_REDUCTIONS)}, got {reduction!r}")
    return H.shape[0], H.shape[1], W.shape[0]


def _loss_outputs(H, n):
    f = dict(dtype=torch.float32, device=H.device)
    return torch.empty(1, **f), torch.empty(n, **f), torch.empty(n, **f)


def cross_entropy(H, W, targets, *, label_smoothing=0.0, z_weight=0.0, reduction="mean", workspace=None):
    """Cross entropy of the head's softmax over the tokens that count.

    H [n, d], W [vocab, d] (bf16 or fp32), targets int32 [n]; a target outside
    [0, vocab), such as -100, does not count. Returns (loss fp32 [1],
    token_loss fp32 [n], lse fp32 [n]).
    """
    n, d, vocab = _cross_entropy_operands(H, W, targets, reduction)
    loss, token_loss, lse = _loss_outputs(H, n)
    workspace = _workspace(workspace, cross_entropy_workspace_bytes(n, d, vocab, H.dtype), H.device)
    _launch(H.device, lib.itl_cross_entropy, _ptr(H), _ptr(W), _HEAD_DTYPES[H.dtype], n, d, vocab, _ptr(targets),
            label_smoothing, z_weight, _REDUCTIONS[reduction], _ptr(loss), _ptr(token_loss), _ptr(lse),
            _ptr(workspace), workspace.numel())
    return loss, token_loss, lse


def cross_entropy_grad(H, W, targets, *, label_smoothing=0.0, z_weight=0.0, reduction="mean", grad_scale=1.0,
                       grad_dtype=torch.float32, dH=None, dW=None, workspace=None):
    """cross_entropy and the gradient of grad_scale * loss in one call.
    Returns (loss, token_loss, lse, dH [n, d], dW [vocab, d]); the gradients
    are of grad_dtype (fp32 or H's)."""
    n, d, vocab = _cross_entropy_operands(H, W, targets, reduction)
    if grad_dtype not in (H.dtype, torch.float32):
        raise ValueError(f"grad_dtype must be {H.dtype} or torch.float32, got {grad_dtype}")
    loss, token_loss, lse = _loss_outputs(H, n)
    dH = _new((n, d), grad_dtype, H, "dH", dH)
    dW = _new((vocab, d), grad_dtype, H, "dW", dW)
    workspace = _workspace(workspace, cross_entropy_workspace_bytes(n, d, vocab, H.dtype, grad_dtype), H.device)
    _launch(H.device, lib.itl_cross_entropy_grad, _ptr(H), _ptr(W), _HEAD_DTYPES[H.dtype], n, d, vocab,
            _ptr(targets), label_smoothing, z_weight, _REDUCTIONS[reduction], grad_scale, _HEAD_DTYPES[grad_dtype],
            _ptr(loss), _ptr(token_loss), _ptr(lse), _ptr(dH), _ptr(dW), _ptr(workspace), workspace.numel())
    return loss, token_loss, lse, dH, dW


class AdamWPlan:
    """Weights, gradients and AdamW states of one optimizer, laid out for
    adamw_step (made by adamw_plan).

    The states are flat: tensor i's begin at offsets[i] (multiples of 256).
    exp_avg, exp_avg_sq: fp32, or uint8 E4M3 codes of m and sqrt(v) with
    exp_avg_scale, exp_avg_sq_scale (fp32, one per 256). master: fp32 weights
    of the bf16 tensors, or None. step (int64 [1]) and lr (fp32 [1]) are device
    tensors: a captured step sees what they hold when it is replayed.

    The step uses the addresses that the tensors had when the plan was made. So
    plan.lr = x and plan.step = n write into the tensors that the plan holds,
    everything else is fixed (its tensors may be written in place), a plan is
    not copied or pickled (save its tensors), and a step whose tensors lie
    elsewhere by then (``.data`` assigned, storage resized) is refused; a
    replayed one cannot look.
    """

    __slots__ = ("params", "grads", "offsets", "state_bits", "exp_avg", "exp_avg_sq", "exp_avg_scale",
                 "exp_avg_sq_scale", "master", "lr", "step", "device", "_table", "_workspace", "_args", "_tensors",
                 "_addresses")

    def __setattr__(self, name, value):
        try:
            held = getattr(self, name)
        except AttributeError:  # being made
            return object.__setattr__(self, name, value)
        if value is held:  # (plan.lr *= 0.5)
            return
        if name not in ("lr", "step"):
            raise AttributeError(f"{name} of an AdamWPlan is fixed: write into its tensors, or make another plan")
        if isinstance(value, torch.Tensor) and value.numel() != 1:
            raise ValueError(f"{name} must have 1 element, got {value.numel()}")
        with torch.no_grad():
            if isinstance(value, torch.Tensor):
                held.copy_(value.reshape(1))
            else:
                held.fill_(float(value) if name == "lr" else operator.index(value))

    def __delattr__(self, name):
        raise AttributeError(f"{name} of an AdamWPlan is fixed")

    def __reduce_ex__(self, protocol):
        raise TypeError("an AdamWPlan holds device addresses: save its tensors and make another plan from them")

    def _named(self):
        """(name, tensor) of everything whose address a step uses."""
        for name in ("params", "grads"):
            yield from ((f"{name}[{i}]", t) for i, t in enumerate(getattr(self, name)))
        for name in ("exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale", "master", "lr", "step", "_table",
                     "_workspace"):
            if getattr(self, name) is not None:
                yield name, getattr(self, name)


def _refuse_shared(plan):
    """What a step writes (all but gradients and rate) may share memory with nothing else."""
    spans = sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size(), name) for name, t in plan._named() if t.numel())
    any_end = written_end = 0, None
    for start, end, name in spans:
        written = not name.startswith("grads") and name != "lr"
        last = any_end if written else written_end
        if start < last[0]:
            raise ValueError(f"{last[1]} and {name} share memory")
        any_end = max(any_end, (end, name))
        if written:
            written_end = max(written_end, (end, name))


def adamw_plan(params, grads, *, lr, weight_decay=0.0, state_bits=32, step=None, master=None, exp_avg=None,
               exp_avg_sq=None, exp_avg_scale=None, exp_avg_sq_scale=None):
    """Lay out an AdamW step over many tensors (any mix of bf16 and fp32).

    params and grads: lists of contiguous tensors of equal sizes, kept by the
    plan and used where they lie: the gradients of every step are written into
    them. Nothing that a step writes may share memory with another tensor of the
    plan. lr: a float or a device tensor fp32 [1]; weight_decay: a float or one
    per tensor. States start as zeros (step 0) unless given, as from a
    checkpoint; master: fp32 flat weights, True (from the params; the default
    where any is bf16) or False for none.
    """
    params, grads = list(params), list(grads)
    if not params or len(params) != len(grads):
        raise ValueError(f"params and grads must be equally many and at least one, got {len(params)} and {len(grads)}")
    decays = list(weight_decay) if isinstance(weight_decay, (list, tuple)) else [weight_decay] * len(params)
    if len(decays) != len(params):
        raise ValueError(f"weight_decay must be a number or {len(params)} of them")
    if state_bits not in (8, 32):
        raise ValueError(f"state_bits must be 8 or 32, got {state_bits}")
    table = (_AdamWTensor * len(params))()
    dev, offsets, total = None, [], 0
    for i, (p, g, wd) in enumerate(zip(params, grads, decays)):
        _need(p, f"params[{i}]", tuple(_HEAD_DTYPES), device=dev)
        dev = p.device
        _need(g, f"grads[{i}]", tuple(_HEAD_DTYPES), device=dev)
        if p.numel() != g.numel():
            raise ValueError(f"grads[{i}] has {g.numel()} elements, params[{i}] {p.numel()}")
        table[i] = _AdamWTensor(p.data_ptr(), g.data_ptr(), p.numel(), _HEAD_DTYPES[p.dtype], _HEAD_DTYPES[g.dtype], wd)
        offsets.append(total)
        total += -(-p.numel() // 256) * 256
    nbytes, elements = _i64(), _i64()
    _check(lib.itl_adamw_plan_sizes(table, len(params), ctypes.byref(nbytes), ctypes.byref(elements)))
    host = torch.empty(max(nbytes.value, 1), dtype=torch.uint8)
    _check(lib.itl_adamw_plan(table, len(params), _ptr(host), nbytes.value))

    plan = AdamWPlan()
    plan.params, plan.grads, plan.offsets = tuple(params), tuple(grads), tuple(offsets)
    plan.state_bits, plan.device = state_bits, dev

    def state(name, given, dtype, n):
        if given is None:
            return torch.zeros(n, dtype=dtype, device=dev)
        _need(given, name, (dtype,), device=dev, ndim=1)
        if given.shape[0] != n:
            raise ValueError(f"{name} must have {n} elements, got {given.shape[0]}")
        return given

    code = torch.float32 if state_bits == 32 else torch.uint8
    plan.exp_avg = state("exp_avg", exp_avg, code, total)
    plan.exp_avg_sq = state("exp_avg_sq", exp_avg_sq, code, total)
    if state_bits == 8:
        plan.exp_avg_scale = state("exp_avg_scale", exp_avg_scale, torch.float32, total // 256)
        plan.exp_avg_sq_scale = state("exp_avg_sq_scale", exp_avg_sq_scale, torch.float32, total // 256)
    elif exp_avg_scale is not None or exp_avg_sq_scale is not None:
        raise ValueError("scales belong to 8-bit states")
    else:
        plan.exp_avg_scale = plan.exp_avg_sq_scale = None
    if master is None:
        master = any(p.dtype == torch.bfloat16 for p in params)
    if master is True:
        plan.master = torch.zeros(total, dtype=torch.float32, device=dev)
        for p, o in zip(params, offsets):
            if p.dtype == torch.bfloat16:
                plan.master[o:o + p.numel()].copy_(p.detach().reshape(-1))
    else:
        plan.master = None if master is False else state("master", master, torch.float32, total)
    plan.step = state("step", step, torch.int64, 1)
    if not isinstance(lr, torch.Tensor):  # (the default dtype may be another)
        lr = torch.full((1,), float(lr), dtype=torch.float32, device=dev)
    plan.lr = state("lr", lr, torch.float32, 1)
    plan._table = host[:nbytes.value].to(dev)
    plan._workspace = torch.empty(int(lib.itl_adamw_step_workspace_bytes()), dtype=torch.uint8, device=dev)
    plan._args = (_ptr(plan._table), nbytes.value, state_bits, _ptr(plan.exp_avg), _ptr(plan.exp_avg_sq),
                  _ptr(plan.exp_avg_scale), _ptr(plan.exp_avg_sq_scale), _ptr(plan.master), _ptr(plan.lr),
                  _ptr(plan.step))
    _refuse_shared(plan)
    plan._tensors = [t for _, t in plan._named()]
    plan._addresses = [*map(torch.Tensor.data_ptr, plan._tensors)]
    return plan


def adamw_step(plan, *, betas=(0.9, 0.999), eps=1e-8, max_norm=None, grad_norm=None):
    """One AdamW step over a plan's tensors, in place. max_norm clips the
    gradients' norm over all tensors; the norm (fp32 [1]) is returned where it
    is computed (max_norm or grad_norm, a tensor for it, given), else None. A
    norm that is not finite skips the step."""
    if not isinstance(plan, AdamWPlan):
        raise TypeError("plan must come from adamw_plan")
    if [*map(torch.Tensor.data_ptr, plan._tensors)] != plan._addresses:
        moved = [name for (name, t), at in zip(plan._named(), plan._addresses) if t.data_ptr() != at]
        raise ValueError(f"{', '.join(moved)} moved since the plan was made: make another plan")
    if grad_norm is not None:
        _need(grad_norm, "grad_norm", (torch.float32,), device=plan.device, ndim=1)
        if grad_norm.shape[0] != 1:
            raise ValueError("grad_norm must have 1 element")
    elif max_norm is not None:
        grad_norm = torch.empty(1, dtype=torch.float32, device=plan.device)
    _launch(plan.device, lib.itl_adamw_step, *plan._args, betas[0], betas[1], eps,
            float("inf") if max_norm is None else max_norm, _ptr(grad_norm), _ptr(plan._workspace),
            plan._workspace.numel())
    # graphs that saved the weights before the step must not go backward with the new ones
    torch.autograd.graph.increment_version(plan.params)
    return grad_norm


# Field order of itl_mismatch_stats' output (the itl_stat enum of include/itl.h).
STAT_FIELDS = (
    "n_tok",
    "kl_k1",
    "kl_k2",
    "kl_k3",
    "weight_mean",
    "weight_max",
    "weight_min",
    "deviation_max",
    "deviation_median",
    "deviation_peak_over_median",
    "lag_abs_mean",
    "lag_abs_max",
    "lag_kl_k3",
    "kernel_abs_mean",
    "kernel_abs_max",
    "kernel_kl_k3",
    "kernel_nonzero",
)


def mismatch_stats_workspace_bytes(n_tok):
    return int(lib.itl_mismatch_stats_workspace_bytes(n_tok))


def mismatch_stats(logprob, rollout_logprob, same_weights_logprob=None, *, stats=None, workspace=None):
    """Mismatch diagnostics of one batch: fp64 device tensor [len(STAT_FIELDS)]
    in STAT_FIELDS order (use ``stats_dict`` to read it on the host)."""
    _need(logprob, "logprob", (torch.float32,), ndim=1)
    dev = logprob.device
    _need(rollout_logprob, "rollout_logprob", (torch.float32,), device=dev, ndim=1)
    n_tok = logprob.shape[0]
    if rollout_logprob.shape[0] != n_tok:
        raise ValueError("logprob and rollout_logprob differ in length")
    if same_weights_logprob is not None:
        _need(same_weights_logprob, "same_weights_logprob", (torch.float32,), device=dev, ndim=1)
        if same_weights_logprob.shape[0] != n_tok:
            raise ValueError("same_weights_logprob differs in length")
    if stats is None:
        stats = torch.empty(len(STAT_FIELDS), dtype=torch.float64, device=dev)
    _need(stats, "stats", (torch.float64,), device=dev, ndim=1)
    if stats.shape[0] < len(STAT_FIELDS):
        raise ValueError(f"stats needs {len(STAT_FIELDS)} elements")
    need = mismatch_stats_workspace_bytes(n_tok)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    _need(workspace, "workspace", (torch.uint8,), device=dev)
    _check(lib.itl_mismatch_stats(_ptr(logprob), _ptr(rollout_logprob), _ptr(same_weights_logprob), n_tok,
                                  _ptr(stats), _ptr(workspace), workspace.numel(), _stream(dev)))
    return stats


def stats_dict(stats):
    """Host dict of a mismatch_stats result (synchronises on the copy)."""
    vals = stats.cpu().tolist()
    return {k: vals[i] for i, k in enumerate(STAT_FIELDS)}


def check_inputs(tokens, vocab, resp_offsets=None):
    """Validate device-resident token ids and offsets (synchronises)."""
    _need(tokens, "tokens", (torch.int32,), ndim=1)
    n_resp = 0
    if resp_offsets is not None:
        _need(resp_offsets, "resp_offsets", (torch.int64,), device=tokens.device, ndim=1)
        n_resp = resp_offsets.shape[0] - 1
    _check(lib.itl_check_inputs(_ptr(tokens), tokens.shape[0], vocab, _ptr(resp_offsets), n_resp,
                                _stream(tokens.device)))
