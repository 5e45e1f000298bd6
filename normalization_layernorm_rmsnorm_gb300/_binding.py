"""ctypes binding of libnorm's C ABI (include/libnorm.h).

Argument marshalling only: every function takes torch tensors (device memory
allocated by the caller), derives the sizes and the dtype code from them, and
calls the C entry point of the same name on the current torch CUDA stream (or
the stream given).  Every step of the computation runs in libnorm's kernels.
A non-OK status raises NrmError.  There is no fallback: if libnorm.so is not
built the first call raises.
"""
from __future__ import annotations

import ctypes
import functools
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_build", "libnorm.so")

NRM_OK, NRM_ERR_INVALID_ARG, NRM_ERR_UNSUPPORTED, NRM_ERR_WORKSPACE, NRM_ERR_CUDA, NRM_ERR_TIMEOUT = range(6)
NRM_F32, NRM_F16, NRM_BF16 = 0, 1, 2
NRM_ACT_NONE, NRM_ACT_RELU, NRM_ACT_GELU, NRM_ACT_SILU, NRM_ACT_MISH = 0, 1, 2, 3, 4
NRM_ACT_LEAKY_RELU, NRM_ACT_ELU, NRM_ACT_SIGMOID, NRM_ACT_CELU, NRM_ACT_SELU = 5, 6, 7, 8, 9
NRM_ACT_RELU6, NRM_ACT_HARDTANH = 10, 11
NRM_OP_LAYERNORM_BWD, NRM_OP_RMSNORM_BWD, NRM_OP_LAYERNORM_CF_BWD, NRM_OP_QK_NORM_BWD = 1, 2, 3, 4
NRM_PAIRS_HALF, NRM_PAIRS_ADJACENT = 0, 1
NRM_CACHE_E4M3, NRM_CACHE_INT8, NRM_CACHE_INT4 = 0, 1, 2

ACTS = {"none": NRM_ACT_NONE, "relu": NRM_ACT_RELU, "gelu": NRM_ACT_GELU, "silu": NRM_ACT_SILU,
        "mish": NRM_ACT_MISH, "leaky_relu": NRM_ACT_LEAKY_RELU, "elu": NRM_ACT_ELU,
        "sigmoid": NRM_ACT_SIGMOID, "celu": NRM_ACT_CELU, "selu": NRM_ACT_SELU,
        "relu6": NRM_ACT_RELU6, "hardtanh": NRM_ACT_HARDTANH}

# Every symbol the header declares (checked by the CPU tests).
EXPORTS = ("nrm_layernorm_fwd", "nrm_layernorm_bwd", "nrm_layernorm_bwd_noalloc",
           "nrm_layernorm_cf_fwd", "nrm_layernorm_cf_bwd",
           "nrm_rmsnorm_fwd", "nrm_rmsnorm_bwd", "nrm_layernorm_fwd_ex", "nrm_layernorm_bwd_ex",
           "nrm_rmsnorm_fwd_ex", "nrm_rmsnorm_bwd_ex",
           "nrm_batchnorm_fwd", "nrm_batchnorm_bwd", "nrm_act_dropout_fwd", "nrm_act_dropout_bwd",
           "nrm_qk_norm_rope_fwd", "nrm_qk_norm_rope_bwd", "nrm_rope_fwd", "nrm_rope_bwd",
           "nrm_kv_cache_write", "nrm_kv_cache_read", "nrm_qk_norm_rope_cache",
           "nrm_kv_cache_attention", "nrm_kv_attention_workspace_bytes", "nrm_kv_cache_evict",
           "nrm_block_norm_fwd", "nrm_block_norm_bwd", "nrm_block_norm_workspace_bytes",
           "nrm_workspace_bytes",
           "nrm_batchnorm_workspace_bytes",
           "nrm_act_mask_words", "nrm_sync_status", "nrm_status_str",
           "nrm_last_error_message", "nrm_version", "nrm_test_expire_peer_waits")


class NrmError(RuntimeError):
    def __init__(self, status: int, func: str, message: str):
        self.status = status
        super().__init__(f"{func}: status {status}: {message}")


_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_F = ctypes.c_float
_I = ctypes.c_int
_lib = None


class _Heads(ctypes.Structure):
    _fields_ = [("data", _P), ("heads", _I64), ("token_stride", _I64), ("head_stride", _I64)]


class _Rope(ctypes.Structure):
    _fields_ = [("pos", _P), ("pos_stride", _I64), ("inv_freq", _P), ("axis", ctypes.c_char_p), ("rot", ctypes.c_int32),
                ("axes", ctypes.c_int32), ("pairs", _I)]


class _Cache(ctypes.Structure):
    _fields_ = [("k_codes", _P), ("k_scales", _P), ("v_codes", _P), ("v_scales", _P)] + [
        (n, _I64) for n in ("pages", "page_size", "heads", "d", "group", "page_stride", "slot_stride", "head_stride",
                            "scale_page_stride", "scale_slot_stride", "scale_head_stride")] + [("kind", _I)]


class _Pages(ctypes.Structure):
    _fields_ = [("table", _P), ("lengths", _P), ("sequences", _I64), ("width", _I64), ("stride", _I64)]


class _Weights(ctypes.Structure):
    _fields_ = [("data", _P), ("capacity", _I64), ("sequence_stride", _I64), ("head_stride", _I64)]


_HP, _RP, _CP, _PP, _WP = (ctypes.POINTER(t) for t in (_Heads, _Rope, _Cache, _Pages, _Weights))


def load(path: str | None = None):
    """Loads libnorm.so (once) and declares the C signatures."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise ImportError(f"libnorm is not built ({p} is missing); run "
                          "`python -m normalization_layernorm_rmsnorm_gb300.build`")
    lib = ctypes.CDLL(p)
    sig = {
        "nrm_layernorm_fwd": [_P, _P, _P, _P, _P, _P, _I64, _I64, _F, _I, _P],
        "nrm_layernorm_bwd": [_P, _P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I, _P, ctypes.c_size_t, _P],
        "nrm_layernorm_bwd_noalloc": [_P, _P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I, _P],
        "nrm_layernorm_cf_fwd": [_P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _F, _I, _P],
        "nrm_layernorm_cf_bwd": [_P, _P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I, _P, ctypes.c_size_t,
                                 _P],
        "nrm_rmsnorm_fwd": [_P, _P, _P, _P, _P, _I64, _I64, _F, _I, _P],
        "nrm_layernorm_fwd_ex": [_P, _P, _P, _P, _P, _P, _I64, _I64, _F, _I, _I, _P],
        "nrm_layernorm_bwd_ex": [_P, _P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I, _I, _P, ctypes.c_size_t, _P],
        "nrm_rmsnorm_fwd_ex": [_P, _P, _P, _P, _P, _I64, _I64, _F, _I, _I, _P],
        "nrm_rmsnorm_bwd_ex": [_P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I, _I, _P, ctypes.c_size_t, _P],
        "nrm_rmsnorm_bwd": [_P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I, _P, ctypes.c_size_t, _P],
        "nrm_batchnorm_fwd": [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _F, _F, _I,
                              _I, _F, _I, _P, ctypes.c_size_t, _P],
        "nrm_batchnorm_bwd": [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I,
                              _I, _F, _I, _P, ctypes.c_size_t, _P],
        "nrm_act_dropout_fwd": [_P, _P, _I64, _I, _F, _F, ctypes.c_uint32, _I, _P],
        "nrm_act_dropout_bwd": [_P, _P, _P, _I64, _I, _F, _F, ctypes.c_uint32, _I, _P],
        "nrm_qk_norm_rope_fwd": [_HP, _HP, _P, _P, _RP, _HP, _HP, _P, _P, _I64, _I64, _F, _I, _P],
        "nrm_qk_norm_rope_bwd": [_HP, _HP, _HP, _HP, _P, _P, _P, _P, _RP, _HP, _HP, _P, _P, _I64, _I64, _I, _P,
                                 ctypes.c_size_t, _P],
        "nrm_rope_fwd": [_HP, _HP, _RP, _HP, _HP, _I64, _I64, _I, _P],
        "nrm_rope_bwd": [_HP, _HP, _RP, _HP, _HP, _I64, _I64, _I, _P],
        "nrm_kv_cache_write": [_HP, _HP, _CP, _P, _I64, _I, _P],
        "nrm_kv_cache_read": [_CP, _P, _HP, _HP, _I64, _I, _P],
        "nrm_qk_norm_rope_cache": [_HP, _HP, _HP, _P, _P, _RP, _HP, _HP, _CP, _P, _I64, _I64, _F, _I, _I, _P],
        "nrm_kv_cache_attention": [_HP, _CP, _PP, _HP, _F, _I64, _P, _WP, _I, _P, ctypes.c_size_t, _P],
        "nrm_kv_attention_workspace_bytes": [_I64, _I64, _CP, _I64],
        "nrm_kv_cache_evict": [_CP, _PP, _WP, _P, _I64, _I64, _P, _WP, _P, _I64, _I64, _I64, _P],
        "nrm_block_norm_fwd": [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _F, _F, _I, _I, _P],
        "nrm_block_norm_bwd": [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _F, _I, _I, _P,
                               ctypes.c_size_t, _P],
        "nrm_block_norm_workspace_bytes": [_I64, _I64, _I64, _I],
        "nrm_workspace_bytes": [_I, _I64, _I64, _I],
        "nrm_batchnorm_workspace_bytes": [_I64, _I64, _I64, _I],
        "nrm_act_mask_words": [_I64, _I64, _I64],
        "nrm_sync_status": [_P],
        "nrm_status_str": [_I],
        "nrm_last_error_message": [],
        "nrm_version": [],
        "nrm_test_expire_peer_waits": [ctypes.c_uint64],
    }
    for name, args in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = _I
    lib.nrm_workspace_bytes.restype = ctypes.c_size_t
    lib.nrm_kv_attention_workspace_bytes.restype = ctypes.c_size_t
    lib.nrm_block_norm_workspace_bytes.restype = ctypes.c_size_t
    lib.nrm_batchnorm_workspace_bytes.restype = ctypes.c_size_t
    lib.nrm_act_mask_words.restype = ctypes.c_int64
    lib.nrm_status_str.restype = ctypes.c_char_p
    lib.nrm_last_error_message.restype = ctypes.c_char_p
    if path is None:
        _lib = lib
    return lib


# ---------------------------------------------------------------------------
# marshalling helpers
# ---------------------------------------------------------------------------

def _dtype_code(t) -> int:
    import torch
    codes = {torch.float32: NRM_F32, torch.float16: NRM_F16, torch.bfloat16: NRM_BF16}
    if t.dtype not in codes:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return codes[t.dtype]


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _check(status: int, func: str):
    if status != NRM_OK:
        msg = load().nrm_last_error_message().decode()
        raise NrmError(status, func, msg)


def _act(act) -> int:
    return ACTS[act] if isinstance(act, str) else int(act)


def _rows_cols(x):
    cols = x.shape[-1] if x.dim() > 0 else 1
    rows = x.numel() // cols if cols else 0
    return rows, cols


# ---------------------------------------------------------------------------
# entry points (same names as the C ABI)
# ---------------------------------------------------------------------------

def nrm_layernorm_fwd(x, w, b, y, mean, rstd, eps, stream=None):
    rows, cols = _rows_cols(x)
    _check(load().nrm_layernorm_fwd(_ptr(x), _ptr(w), _ptr(b), _ptr(y), _ptr(mean), _ptr(rstd),
                                    rows, cols, eps, _dtype_code(x), _stream(stream)),
           "nrm_layernorm_fwd")


def nrm_layernorm_bwd(dy, x, w, mean, rstd, dx, dw, db, workspace, stream=None):
    rows, cols = _rows_cols(x)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().nrm_layernorm_bwd(_ptr(dy), _ptr(x), _ptr(w), _ptr(mean), _ptr(rstd), _ptr(dx),
                                    _ptr(dw), _ptr(db), rows, cols, _dtype_code(x), _ptr(workspace),
                                    ws_bytes, _stream(stream)),
           "nrm_layernorm_bwd")


def nrm_layernorm_cf_fwd(x, w, b, y, mean, rstd, eps, stream=None):
    """LayerNorm over the channels of x[n, c, *spatial]; mean, rstd hold n * prod(spatial)
    floats (or are None)."""
    n, c, l = _ncl(x)
    _check(load().nrm_layernorm_cf_fwd(_ptr(x), _ptr(w), _ptr(b), _ptr(y), _ptr(mean), _ptr(rstd),
                                       n, c, l, eps, _dtype_code(x), _stream(stream)),
           "nrm_layernorm_cf_fwd")


def nrm_layernorm_cf_bwd(dy, x, w, mean, rstd, dx, dw, db, workspace, stream=None):
    n, c, l = _ncl(x)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().nrm_layernorm_cf_bwd(_ptr(dy), _ptr(x), _ptr(w), _ptr(mean), _ptr(rstd), _ptr(dx),
                                       _ptr(dw), _ptr(db), n, c, l, _dtype_code(x), _ptr(workspace),
                                       ws_bytes, _stream(stream)),
           "nrm_layernorm_cf_bwd")


def nrm_layernorm_bwd_noalloc(dy, x, w, mean, rstd, dx, dw, db, stream=None):
    """LayerNorm backward for callers that cannot allocate: no workspace; the
    library's static device scratch holds the dw/db partial rows."""
    rows, cols = _rows_cols(x)
    _check(load().nrm_layernorm_bwd_noalloc(_ptr(dy), _ptr(x), _ptr(w), _ptr(mean), _ptr(rstd),
                                            _ptr(dx), _ptr(dw), _ptr(db), rows, cols,
                                            _dtype_code(x), _stream(stream)),
           "nrm_layernorm_bwd_noalloc")


def nrm_rmsnorm_fwd(x, w, y, rstd, eps, stream=None, b=None):
    """RMSNorm of the rows of x; b is the optional bias."""
    rows, cols = _rows_cols(x)
    _check(load().nrm_rmsnorm_fwd(_ptr(x), _ptr(w), _ptr(b), _ptr(y), _ptr(rstd), rows, cols, eps,
                                  _dtype_code(x), _stream(stream)),
           "nrm_rmsnorm_fwd")


def nrm_layernorm_fwd_ex(x, w, b, y, mean, rstd, eps, stream=None):
    """LayerNorm with y in its own dtype (x's, or float32 for a 16-bit x)."""
    rows, cols = _rows_cols(x)
    _check(load().nrm_layernorm_fwd_ex(_ptr(x), _ptr(w), _ptr(b), _ptr(y), _ptr(mean), _ptr(rstd), rows,
                                       cols, eps, _dtype_code(x), _dtype_code(y), _stream(stream)),
           "nrm_layernorm_fwd_ex")


def nrm_layernorm_bwd_ex(dy, x, w, mean, rstd, dx, dw, db, workspace, stream=None):
    """LayerNorm backward with dy in its own dtype (the forward's y dtype)."""
    rows, cols = _rows_cols(x)
    _check(load().nrm_layernorm_bwd_ex(_ptr(dy), _ptr(x), _ptr(w), _ptr(mean), _ptr(rstd), _ptr(dx),
                                       _ptr(dw), _ptr(db), rows, cols, _dtype_code(x), _dtype_code(dy),
                                       _ptr(workspace), _ws(workspace), _stream(stream)),
           "nrm_layernorm_bwd_ex")


def nrm_rmsnorm_fwd_ex(x, w, y, rstd, eps, stream=None, b=None):
    """RMSNorm with y in its own dtype (x's, or float32 for a 16-bit x)."""
    rows, cols = _rows_cols(x)
    _check(load().nrm_rmsnorm_fwd_ex(_ptr(x), _ptr(w), _ptr(b), _ptr(y), _ptr(rstd), rows, cols, eps,
                                     _dtype_code(x), _dtype_code(y), _stream(stream)),
           "nrm_rmsnorm_fwd_ex")


def nrm_rmsnorm_bwd_ex(dy, x, w, rstd, dx, dw, workspace, stream=None, db=None):
    """RMSNorm backward with dy in its own dtype (the forward's y dtype)."""
    rows, cols = _rows_cols(x)
    _check(load().nrm_rmsnorm_bwd_ex(_ptr(dy), _ptr(x), _ptr(w), _ptr(rstd), _ptr(dx), _ptr(dw), _ptr(db),
                                     rows, cols, _dtype_code(x), _dtype_code(dy), _ptr(workspace),
                                     _ws(workspace), _stream(stream)),
           "nrm_rmsnorm_bwd_ex")


def nrm_rmsnorm_bwd(dy, x, w, rstd, dx, dw, workspace, stream=None, db=None):
    """RMSNorm backward; db receives the bias gradient when given."""
    rows, cols = _rows_cols(x)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().nrm_rmsnorm_bwd(_ptr(dy), _ptr(x), _ptr(w), _ptr(rstd), _ptr(dx), _ptr(dw), _ptr(db),
                                  rows, cols, _dtype_code(x), _ptr(workspace), ws_bytes,
                                  _stream(stream)),
           "nrm_rmsnorm_bwd")


def _ncl(x):
    if x.dim() < 2:
        raise ValueError("input needs at least [n, c] (NCHW-like, channels second)")
    n, c = x.shape[0], x.shape[1]
    l = 1
    for s in x.shape[2:]:
        l *= s
    return n, c, l


def _ws(workspace):
    return 0 if workspace is None else workspace.numel() * workspace.element_size()


def nrm_batchnorm_fwd(x, residual, w, b, y, running_mean, running_var, save_mean, save_rstd,
                      act_mask, eps, momentum, training, act, workspace, stream=None, act_param=0.0):
    n, c, l = _ncl(x)
    _check(load().nrm_batchnorm_fwd(_ptr(x), _ptr(residual), _ptr(w), _ptr(b), _ptr(y),
                                    _ptr(running_mean), _ptr(running_var), _ptr(save_mean),
                                    _ptr(save_rstd), _ptr(act_mask), n, c, l, eps, momentum,
                                    int(bool(training)), _act(act), float(act_param), _dtype_code(x),
                                    _ptr(workspace), _ws(workspace), _stream(stream)),
           "nrm_batchnorm_fwd")


def nrm_batchnorm_bwd(dy, x, residual, w, b, save_mean, save_rstd, act_mask, dx, dres, dw, db,
                      training, act, workspace, stream=None, act_param=0.0):
    n, c, l = _ncl(x)
    _check(load().nrm_batchnorm_bwd(_ptr(dy), _ptr(x), _ptr(residual), _ptr(w), _ptr(b),
                                    _ptr(save_mean), _ptr(save_rstd), _ptr(act_mask), _ptr(dx),
                                    _ptr(dres), _ptr(dw), _ptr(db), n, c, l,
                                    int(bool(training)), _act(act), float(act_param), _dtype_code(x),
                                    _ptr(workspace), _ws(workspace), _stream(stream)),
           "nrm_batchnorm_bwd")


def nrm_batchnorm_workspace_bytes(n: int, c: int, l: int, dtype_code: int) -> int:
    return int(load().nrm_batchnorm_workspace_bytes(n, c, l, dtype_code))


def batchnorm_workspace(x):
    """A device workspace large enough for BatchNorm calls on x ([n, c, ...])."""
    import torch
    n, c, l = _ncl(x)
    nbytes = nrm_batchnorm_workspace_bytes(n, c, l, _dtype_code(x))
    return torch.empty(max(nbytes, 16), dtype=torch.uint8, device=x.device)


def nrm_workspace_bytes(op: int, rows: int, cols: int, dtype_code: int) -> int:
    return int(load().nrm_workspace_bytes(op, rows, cols, dtype_code))


def nrm_act_dropout_fwd(x, y, act, drop_p, seed, stream=None, act_param=0.0):
    """y = act(x) / (1 - drop_p) where kept, else 0 (mask rebuilt from seed and offset)."""
    _check(load().nrm_act_dropout_fwd(_ptr(x), _ptr(y), x.numel(), _act(act), float(act_param), float(drop_p),
                                      int(seed) & 0xFFFFFFFF, _dtype_code(x), _stream(stream)),
           "nrm_act_dropout_fwd")


def nrm_act_dropout_bwd(dy, x, dx, act, drop_p, seed, stream=None, act_param=0.0):
    """dx = dy / (1 - drop_p) * act'(x) where kept, else 0."""
    _check(load().nrm_act_dropout_bwd(_ptr(dy), _ptr(x), _ptr(dx), x.numel(), _act(act), float(act_param),
                                      float(drop_p),
                                      int(seed) & 0xFFFFFFFF, _dtype_code(x), _stream(stream)),
           "nrm_act_dropout_bwd")


# ---------------------------------------------------------------------------
# attention heads: norms with position rotation, quantised key/value cache
# ---------------------------------------------------------------------------
# Views are [tokens, heads, d] or [batch, tokens, heads, d] tensors with
# contiguous rows and any other strides that one token stride describes.  Their
# marshalling is compiled (csrc/heads_binding.cpp): from Python it took longer
# than the kernels of small calls.

@functools.lru_cache(maxsize=None)
def _heads():
    """The compiled marshalling of this section's calls."""
    import importlib.machinery
    import importlib.util

    from .build import heads_path
    load()
    path = heads_path()  # (imports torch, whose libraries the module uses)
    if not os.path.exists(path):
        raise ImportError(f"libnorm's calls on heads are not built for this PyTorch and Python ({path} is missing); "
                          "run `python -m normalization_layernorm_rmsnorm_gb300.build`")
    loader = importlib.machinery.ExtensionFileLoader("_heads", path)
    module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_heads", loader))
    loader.exec_module(module)
    module.set_error(NrmError)
    return module


def rope_axis(sections, interleaved=False) -> bytes:
    """The axis of each pair for nrm_*rope*: sections[a] pairs for axis a, one
    section after another, or taken in turn while they last (interleaved)."""
    if not interleaved:
        return b"".join(bytes([a]) * n for a, n in enumerate(sections))
    left, out = list(sections), bytearray()
    while any(left):
        for a, n in enumerate(left):
            if n > 0:
                out.append(a)
                left[a] -= 1
    return bytes(out)


def qk_norm_workspace(q):
    """A device workspace for nrm_qk_norm_rope_bwd on heads like q's."""
    import torch
    d = q.shape[-1]
    nbytes = nrm_workspace_bytes(NRM_OP_QK_NORM_BWD, q.numel() // max(d, 1), d, _dtype_code(q))
    return torch.empty(max(nbytes, 16), dtype=torch.uint8, device=q.device)


def nrm_qk_norm_rope_fwd(q, k, wq, wk, pos, inv_freq, q_out, k_out, rstd_q, rstd_k, eps, stream=None, axis=None,
                         pairs="half"):
    """RMSNorm of every head of q and k and the rotation by position, in one pass.

    q, k: [tokens, heads, d] views (k may be None); q_out, k_out may be q, k.
    pos: int64 [tokens], or [axes, tokens] with `axis`, the axis of each pair
    (rope_axis).  inv_freq: float32 [rot / 2] (None: no rotation).  pairs:
    "half" turns elements (p, p + rot/2) together, "pair" (2p, 2p + 1)."""
    _heads().qk_norm_rope_fwd(q, k, wq, wk, pos, inv_freq, q_out, k_out, rstd_q, rstd_k, eps, stream, axis, pairs)


def nrm_qk_norm_rope_bwd(dq_out, dk_out, q, k, wq, wk, rstd_q, rstd_k, pos, inv_freq, dq, dk, dwq, dwk, workspace,
                         stream=None, axis=None, pairs="half"):
    """Backward of nrm_qk_norm_rope_fwd: dq, dk (views like q, k) and the weights'
    gradients dwq, dwk (each may be None; workspace from qk_norm_workspace)."""
    _heads().qk_norm_rope_bwd(dq_out, dk_out, q, k, wq, wk, rstd_q, rstd_k, pos, inv_freq, dq, dk, dwq, dwk, workspace,
                              stream, axis, pairs)


def nrm_rope_fwd(q, k, pos, inv_freq, q_out, k_out, stream=None, axis=None, pairs="half"):
    """The rotation by position alone (arguments as nrm_qk_norm_rope_fwd); q_out, k_out may be q, k."""
    _heads().rope_fwd(q, k, pos, inv_freq, q_out, k_out, stream, axis, pairs)


def nrm_rope_bwd(dq_out, dk_out, pos, inv_freq, dq, dk, stream=None, axis=None, pairs="half"):
    """Backward of nrm_rope_fwd: the turn the other way; dq, dk may be dq_out, dk_out."""
    _heads().rope_bwd(dq_out, dk_out, pos, inv_freq, dq, dk, stream, axis, pairs)


class KvCache:
    """A paged, quantised key/value cache (kv_cache): the tensors and their C description.

    Its attributes cannot be set: the description holds the tensors' addresses, and a
    tensor that was replaced here could be freed under it."""

    __slots__ = ("k_codes", "k_scales", "v_codes", "v_scales", "heads", "d", "slots", "held", "address",
                 "_c")

    def __setattr__(self, name, value):
        raise AttributeError(f"{name} of a cache cannot be set: make a new one (kv_cache)")

    def __delattr__(self, name):
        raise AttributeError(f"{name} of a cache cannot be deleted")

    def __copy__(self):
        return self

    def __init__(self, k_codes, k_scales, v_codes, v_scales):
        import torch
        codes, scales = (k_codes, k_scales) if k_codes is not None else (v_codes, v_scales)
        if codes is None or scales is None:
            raise ValueError("a cache needs codes and scales")
        kinds = {torch.float8_e4m3fn: NRM_CACHE_E4M3, torch.int8: NRM_CACHE_INT8, torch.uint8: NRM_CACHE_INT4}
        if codes.dtype not in kinds:
            raise TypeError(f"codes are float8_e4m3fn, int8, or uint8 (two 4-bit values), got {codes.dtype}")
        kind = kinds[codes.dtype]
        if codes.dim() != 4 or scales.dim() != 4 or scales.dtype != torch.float32:
            raise ValueError("codes are [pages, page, heads, d], scales float32 [pages, page, heads, d / group]")
        pages, page, heads, d = codes.shape
        if kind == NRM_CACHE_INT4:
            d *= 2
        if scales.shape[:3] != codes.shape[:3] or scales.shape[3] < 1 or d % scales.shape[3]:
            raise ValueError(f"scales {tuple(scales.shape)} do not go with codes {tuple(codes.shape)}")
        for t, like in ((k_codes, codes), (v_codes, codes), (k_scales, scales), (v_scales, scales)):
            if t is None:
                continue
            if t.shape != like.shape or t.dtype != like.dtype or t.stride() != like.stride():
                raise ValueError("keys and values must have one shape, dtype and strides")
            if t.shape[3] > 1 and t.stride(3) != 1:
                raise ValueError("the rows of codes and scales must be contiguous")
        if (k_codes is None) != (k_scales is None) or (v_codes is None) != (v_scales is None):
            raise ValueError("codes and scales come together")
        dev = torch.cuda.current_device() if torch.cuda.is_available() else None
        for t in (k_codes, k_scales, v_codes, v_scales):
            if t is not None and (not t.is_cuda or t.get_device() != dev):
                raise ValueError(f"tensors must be on the current CUDA device, got {t.device}")
        c = _Cache(_ptr(k_codes), _ptr(k_scales), _ptr(v_codes), _ptr(v_scales), pages, page, heads, d,
                   d // scales.shape[3], *codes.stride()[:3], *scales.stride()[:3], kind)
        for name, value in (("k_codes", k_codes), ("k_scales", k_scales), ("v_codes", v_codes), ("v_scales", v_scales),
                            ("heads", heads), ("d", d), ("slots", pages * page), ("held", codes),
                            ("address", ctypes.addressof(c)), ("_c", c)):
            object.__setattr__(self, name, value)


def kv_cache(k_codes, k_scales, v_codes=None, v_scales=None) -> KvCache:
    """Describes the caller's cache tensors for the cache calls.

    codes: [pages, page, heads, d] float8_e4m3fn or int8, or uint8
    [pages, page, heads, d / 2] (two 4-bit values a byte); scales: float32
    [pages, page, heads, d / group]; any strides but contiguous rows, the same
    for keys and values.  The handle keeps the tensors alive; make a new one
    when they are replaced."""
    return KvCache(k_codes, k_scales, v_codes, v_scales)


def nrm_kv_cache_write(k, v, cache, slots, stream=None):
    """Quantises row t of k and v ([tokens, heads, d]; either may be None) into
    slot slots[t] of the cache; -1 skips a token."""
    _heads().kv_cache_write(cache.address, cache.held, slots, k, v, stream)


def nrm_kv_cache_read(cache, slots, k_out, v_out, stream=None):
    """The values of slot slots[t] as row t of k_out and v_out (either may be
    None); rows of slot -1 are left as they were."""
    _heads().kv_cache_read(cache.address, cache.held, slots, k_out, v_out, stream)


def nrm_qk_norm_rope_cache(q, k, v, wq, wk, pos, inv_freq, q_out, k_out, cache, slots, eps, stream=None, axis=None,
                           pairs="half", norm=True):
    """The step of a served model in one launch: nrm_qk_norm_rope_fwd (nrm_rope_fwd
    with norm=False) of q and k, and the key and v quantised into the cache.
    k_out may be None when only the cache is wanted."""
    _heads().qk_norm_rope_cache(q, k, v, wq, wk, pos, inv_freq, q_out, k_out, cache.address, cache.held, slots, eps,
                                stream, axis, pairs, norm)


# ---------------------------------------------------------------------------
# whole cached sequences: attention of a new token, eviction by weight
# ---------------------------------------------------------------------------

def kv_attention_workspace(q, cache, table, weights=False):
    """A device workspace for nrm_kv_cache_attention on queries like q ([sequences,
    heads, d]) with page tables like table; weights: for calls with weights."""
    import torch
    positions = table.shape[1] * (cache.slots // cache.held.shape[0]) if weights else 0
    nbytes = int(load().nrm_kv_attention_workspace_bytes(table.shape[0], q.shape[-2], ctypes.byref(cache._c), positions))
    return torch.empty(max(nbytes, 16), dtype=torch.uint8, device=q.device)


def nrm_kv_cache_attention(q, cache, table, lengths, out, scale, workspace, stream=None, window=0, lse=None, weights=None):
    """Attention of one new token of each sequence over the cache, straight from its codes.

    q, out: [sequences, heads, d] views, heads a multiple of the cache's.  table:
    int64 [sequences, pages], the pages of each sequence in order; lengths: int64
    [sequences], its written positions (the new token's own among them, once it
    is written).  window: the last positions that count (0: all).  lse: float32
    [sequences, heads] receives log sum exp.  weights: float32 [sequences,
    cache.heads, positions]; each position's attention weight, summed over the
    heads that share it, is added to it (what nrm_kv_cache_evict goes by)."""
    _heads().kv_cache_attention(q, cache.address, cache.held, table, lengths, out, scale, workspace, stream, window, lse,
                                weights)


def nrm_kv_cache_evict(cache, table, lengths, weights, new_table, new_lengths, new_weights, kept, stream=None, first=0,
                       recent=0):
    """Shortens sequences to keep = kept.shape[2] positions by weight, head by head:
    the first `first`, the last `recent` and the largest weights between them
    stay, in order, and their rows are copied to the pages of new_table.

    kept: int64 [sequences, cache.heads, keep] receives the positions that stay
    (-1 behind the last); new_lengths: int64 [sequences]; new_weights: float32
    [sequences, cache.heads, >= keep] or None.  The pages of new_table must not be
    among those that are read."""
    _heads().kv_cache_evict(cache.address, cache.held, table, lengths, weights, new_table, new_lengths, new_weights, kept,
                            stream, first, recent)


# ---------------------------------------------------------------------------
# between two blocks of a residual stream
# ---------------------------------------------------------------------------

def block_norm_workspace(x, gate=None):
    """A device workspace for nrm_block_norm_bwd on rows like x's."""
    import torch
    rows, cols = _rows_cols(x)
    gates = 0 if gate is None or cols == 0 else gate.numel() // cols
    nbytes = int(load().nrm_block_norm_workspace_bytes(rows, cols, gates, _dtype_code(x)))
    return torch.empty(max(nbytes, 16), dtype=torch.uint8, device=x.device)


def nrm_block_norm_fwd(x, f, gate, w_post, w_pre, y, h, rstd_post, rstd_pre, alpha, eps, stream=None, post=True):
    """The RMSNorm after a block, gate, residual scale and add, and the RMSNorm
    before the next block: y = x + alpha * gate * norm(f) * w_post (the norm is
    left out with post=False), h = norm(y) * w_pre.

    x, f, y, h: [..., cols], contiguous; h may be None; y may be x, h may be f.
    gate: None, [cols], or [gates, cols], each row for rows / gates rows of x.
    Weights and statistics (float32, one a row) may be None."""
    _heads().block_norm_fwd(x, f, gate, w_post, w_pre, y, h, rstd_post, rstd_pre, alpha, eps, stream, post)


def nrm_block_norm_bwd(dh, dy, f, y, gate, w_post, w_pre, rstd_post, rstd_pre, dx, df, dgate, dw_post, dw_pre, workspace,
                       alpha, stream=None, post=True):
    """Backward of nrm_block_norm_fwd: dx, df and the gradients of gate and weights
    (each may be None; workspace from block_norm_workspace).  dh is None where the
    forward had no h, dy (the stream's own gradient) where there is none."""
    _heads().block_norm_bwd(dh, dy, f, y, gate, w_post, w_pre, rstd_post, rstd_pre, dx, df, dgate, dw_post, dw_pre,
                            workspace, alpha, stream, post)


def nrm_act_mask_words(n: int, c: int, l: int) -> int:
    return int(load().nrm_act_mask_words(n, c, l))


def nrm_sync_status(stream=None):
    _check(load().nrm_sync_status(_stream(stream)), "nrm_sync_status")


def nrm_status_str(status: int) -> str:
    return load().nrm_status_str(status).decode()


def nrm_version() -> int:
    return int(load().nrm_version())


def nrm_last_error_message() -> str:
    return load().nrm_last_error_message().decode()


def nrm_test_expire_peer_waits(limit_ns: int):
    """Test hook: the next training BatchNorm call on this thread whose kernel
    waits for the other CTAs of a channel waits for one CTA too many and gives
    up after limit_ns (its outputs are then undefined; nrm_sync_status reports
    NRM_ERR_TIMEOUT)."""
    _check(load().nrm_test_expire_peer_waits(int(limit_ns)), "nrm_test_expire_peer_waits")
