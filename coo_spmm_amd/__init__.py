"""coo_spmm_amd -- MI355X (gfx950) truly sparse COO layer.

A thin ctypes binding of ``libsnack.so`` (the C ABI declared in
``include/snack.h``).  Every function below only marshals arguments: tensors
become device pointers, the current torch stream becomes the hipStream_t, and a
non-OK status becomes ``SnackError``.  All computation runs in the library's
HIP kernels; there is no CPU fallback -- importing this package fails loudly
when the library has not been built.

PyTorch is used only for device memory and streams.
"""
from __future__ import annotations

import ctypes
import functools
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsnack.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with `python -m coo_spmm_amd.build` "
                      "(or __graft_entry__.build()); there is no fallback path")

# torch ships its own HIP runtime; loading it before the library makes both use
# that one runtime instance (loaded the other way round, the library's HIP
# calls find no device in a process where torch then initialises the GPU)
import torch  # noqa: E402,F401

_lib = ctypes.CDLL(LIB_PATH)

P = ctypes.c_void_p
i32, i64, u64, f32, f64 = ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64, ctypes.c_float, ctypes.c_double
ST = ctypes.c_int

_SIGS = {
    "snack_status_string": ([ST], ctypes.c_char_p),
    "snack_layer_create": ([i32, i32, i64, P, P, P, u64, P, ctypes.POINTER(P)], ST),
    "snack_layer_destroy": ([P], ST),
    "snack_layer_reserve": ([P, i32], ST),
    "snack_forward": ([P, P, P, i32, P], ST),
    "snack_forward_noalloc": ([P, P, P, i32, P], ST),
    "snack_forward_infer": ([P, P, P, i32, i32, i32, P], ST),
    "snack_forward_chain": ([ctypes.POINTER(P), i32, ctypes.POINTER(i32), P, ctypes.POINTER(P), i32, i32, P], ST),
    "snack_backward": ([P, P, P, P, P, i32, P], ST),
    "snack_backward_sgd": ([P, P, P, P, P, f32, i32, P], ST),
    "snack_train_step_mse": ([P, P, P, P, P, P, P, f32, f32, i32, P], ST),
    "snack_prune_regrow": ([P, i64, P], ST),
    "snack_prune_regrow_grad": ([P, i64, P, P, i32, P], ST),
    "snack_prune_regrow_rows": ([P, i64, i64, i32, P, P, i32, P], ST),
    "snack_layer_shape": ([P, ctypes.POINTER(i32), ctypes.POINTER(i32)], ST),
    "snack_layer_nnz": ([P, ctypes.POINTER(i64)], ST),
    "snack_layer_device_bytes": ([P, ctypes.POINTER(i64)], ST),
    "snack_layer_values": ([P, ctypes.POINTER(P)], ST),
    "snack_layer_values_updated": ([P], ST),
    "snack_layer_export": ([P, P, P, P, P], ST),
    "snack_layer_export_index": ([P, P, P, P, P, P, P], ST),
    "snack_layer_get_epoch": ([P, ctypes.POINTER(u64)], ST),
    "snack_layer_set_epoch": ([P, u64], ST),
    "snack_sgd_step": ([P, P, f32, P], ST),
    "snack_mse_grad": ([P, P, P, i64, f32, P], ST),
    "snack_gelu_fwd": ([P, P, i64, P], ST),
    "snack_gelu_bwd": ([P, P, P, i64, P], ST),
    "snack_ckpt_pack": ([P, i64, i64, i32, P, P, P], ST),
    "snack_ckpt_unpack": ([P, P, i64, i64, i32, P, i32, P], ST),
    "snack_rmsnorm_fwd": ([P, P, i32, P, f32, i64, i64, P, P, P, i32, P, P, P], ST),
    "snack_rmsnorm_bwd_work": ([i64, i64, ctypes.POINTER(i64)], ST),
    "snack_rmsnorm_bwd": ([P, P, i32, P, P, P, P, i64, i64, P, P, P, i64, P], ST),
    "snack_gelu_ckpt_fwd": ([P, i64, i64, i32, P, P, P, P, P, P], ST),
    "snack_gelu_ckpt_bwd": ([P, P, P, i64, i64, i32, P, P], ST),
    "snack_backward_ckpt": ([P, P, P, i32, P, P, P, i32, P], ST),
    "snack_rope_table": ([i32, i32, f64, f64, f64, f64, f64, f64, P, P], ST),
    "snack_qk_rope_fwd": ([P, i64, i64, i32, P, i64, i64, i32, i32, i64, i32, P, P, P, P, f32, P, P, i32, P], ST),
    "snack_qk_rope_bwd_work": ([i64, i32, i32, i32, ctypes.POINTER(i64)], ST),
    "snack_qk_rope_bwd": ([P, i64, i64, i32, P, i64, i64, i32, i32, i64, i32, P, P, P, P, f32, P, i64, i64, P, i64, i64,
                           i32, P, P, P, P, P, i64, P], ST),
    "snack_cache_bytes": ([P, ctypes.POINTER(i64)], ST),
    "snack_cache_slots": ([P, P, i32, P, P, i32, i64, P, P, P], ST),
    "snack_cache_write": ([P, P, i64, i64, P, i64, i64, i32, i64, P, P], ST),
    "snack_cache_write_rope": ([P, P, i64, i64, i32, P, i64, i64, P, i64, i64, i32, i64, P, P, P, P, P, f32, P, i32, P],
                               ST),
    "snack_cache_read": ([P, P, i64, P, P, i32, P], ST),
    "snack_cache_attend_work": ([P, i32, i64, i32, ctypes.POINTER(i64)], ST),
    "snack_cache_attend": ([P, P, i64, i64, i32, i32, i64, P, i32, P, P, i32, f32, i32, P, P, i64, P], ST),
    "snack_profile_enable": ([ctypes.c_int], ST),
    "snack_profile_reset": ([], ST),
    "snack_profile_name": ([ctypes.c_int], ctypes.c_char_p),
    "snack_profile_read": ([ctypes.c_int, ctypes.POINTER(i64), ctypes.POINTER(f64)], ST),
    "snack_profile_set_tag": ([i64], ST),
    "snack_profile_read_tag": ([ctypes.c_int, i64, ctypes.POINTER(i64), ctypes.POINTER(f64)], ST),
}
for _name, (_args, _res) in _SIGS.items():
    _fn = getattr(_lib, _name)
    _fn.argtypes = _args
    _fn.restype = _res

EXPORTED = tuple(_SIGS)

OK, ERR_INVALID_ARG, ERR_INDEX_RANGE, ERR_DUPLICATE, ERR_ALLOC, ERR_HIP, ERR_UNSUPPORTED, ERR_WORKSPACE = range(8)


class SnackError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {snack_status_string(code)} (status {code})")


def snack_status_string(code: int) -> str:
    return _lib.snack_status_string(code).decode()


def _check(code: int, where: str):
    if code != OK:
        raise SnackError(code, where)


def _ptr(t):
    if t is None:
        return None
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch tensor")
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError("tensors passed to the library must be contiguous device tensors")
    return t.data_ptr()


def _spread(t):
    """Address, elements from token to token and from head to head of [tokens, heads, features]."""
    if t is None:
        return None, 0, 0
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch tensor")
    if not t.is_cuda or t.dim() != 3 or (t.stride(2) != 1 and t.shape[2] != 1):
        raise ValueError("heads must be [tokens, heads, features] on the GPU, their features contiguous")
    return t.data_ptr(), t.stride(0), t.stride(1)


def _stream(stream=None):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _need(t, dtype, shape, name):
    import torch
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


# ---------------------------------------------------------------------------
# Functions with the C names (argument marshalling only)
# ---------------------------------------------------------------------------

def snack_layer_create(M, K, rows, cols, vals, seed=0, stream=None):
    """rows/cols int32 [nnz], vals float32 [nnz] or None: device tensors.  Returns the handle (int)."""
    import torch
    nnz = rows.numel()
    _need(rows, torch.int32, (nnz,), "rows")
    _need(cols, torch.int32, (nnz,), "cols")
    if vals is not None:
        _need(vals, torch.float32, (nnz,), "vals")
    h = P()
    _check(_lib.snack_layer_create(M, K, nnz, _ptr(rows), _ptr(cols), _ptr(vals), seed & (2**64 - 1),
                                   _stream(stream), ctypes.byref(h)), "snack_layer_create")
    return h.value


def snack_layer_destroy(h):
    _check(_lib.snack_layer_destroy(h), "snack_layer_destroy")


def snack_layer_reserve(h, max_batch):
    _check(_lib.snack_layer_reserve(h, max_batch), "snack_layer_reserve")


def snack_forward(h, X, Y, stream=None):
    B = X.shape[0]
    _check(_lib.snack_forward(h, _ptr(X), _ptr(Y), B, _stream(stream)), "snack_forward")


def snack_forward_noalloc(h, X, Y, stream=None):
    B = X.shape[0]
    _check(_lib.snack_forward_noalloc(h, _ptr(X), _ptr(Y), B, _stream(stream)), "snack_forward_noalloc")


ACT_NONE, ACT_GELU = 0, 1
REGROW_RANDOM, REGROW_GRADIENT = 0, 1


def snack_forward_infer(h, X, Y, act=ACT_NONE, bf16_values=False, stream=None):
    B = X.shape[0]
    _check(_lib.snack_forward_infer(h, _ptr(X), _ptr(Y), B, int(act), 1 if bf16_values else 0, _stream(stream)),
           "snack_forward_infer")


def snack_forward_chain(handles, acts, X, Ys, bf16_values=False, stream=None):
    """handles: layer handles; acts: activation codes; Ys: output tensors, one per layer."""
    n = len(handles)
    if len(acts) != n or len(Ys) != n:
        raise ValueError("one activation and one output per layer")
    hs = (P * n)(*handles)
    ac = (i32 * n)(*[int(a) for a in acts])
    ys = (P * n)(*[_ptr(y) for y in Ys])
    _check(_lib.snack_forward_chain(hs, n, ac, _ptr(X), ys, X.shape[0], 1 if bf16_values else 0, _stream(stream)),
           "snack_forward_chain")


def snack_backward(h, X, dY, dX=None, dW=None, stream=None):
    B = dY.shape[0]
    _check(_lib.snack_backward(h, _ptr(X), _ptr(dY), _ptr(dX), _ptr(dW), B, _stream(stream)), "snack_backward")


def snack_backward_sgd(h, X, dY, dX, dW, lr, stream=None):
    B = dY.shape[0]
    _check(_lib.snack_backward_sgd(h, _ptr(X), _ptr(dY), _ptr(dX), _ptr(dW), float(lr), B, _stream(stream)),
           "snack_backward_sgd")


def snack_train_step_mse(h, X, T, Y, dY, dX, dW, scale, lr, stream=None):
    B = X.shape[0]
    _check(_lib.snack_train_step_mse(h, _ptr(X), _ptr(T), _ptr(Y), _ptr(dY), _ptr(dX), _ptr(dW), float(scale),
                                     float(lr), B, _stream(stream)), "snack_train_step_mse")


def snack_prune_regrow(h, n_drop, stream=None):
    _check(_lib.snack_prune_regrow(h, int(n_drop), _stream(stream)), "snack_prune_regrow")


def snack_prune_regrow_grad(h, n_drop, X, dY, stream=None):
    """X [B, K], dY [B, M]: the batch whose dense weight gradient picks the grown cells."""
    B = X.shape[0]
    if dY.shape[0] != B:
        raise ValueError("X and dY must have the same batch")
    _check(_lib.snack_prune_regrow_grad(h, int(n_drop), _ptr(X), _ptr(dY), B, _stream(stream)),
           "snack_prune_regrow_grad")


def snack_prune_regrow_rows(h, drop_num, drop_den, mode, X=None, dY=None, stream=None):
    """Row-local drop / regrow: each row drops floor(n_i * drop_num / drop_den) of its smallest |w| and
    regrows as many inside itself, at random (REGROW_RANDOM) or at the largest |dY^T X| (REGROW_GRADIENT,
    X [B, K], dY [B, M])."""
    B = 0
    if X is not None or dY is not None:
        if X is None or dY is None or dY.shape[0] != X.shape[0]:
            raise ValueError("X and dY must both be given, with the same batch")
        B = X.shape[0]
    _check(_lib.snack_prune_regrow_rows(h, int(drop_num), int(drop_den), int(mode), _ptr(X), _ptr(dY), B,
                                        _stream(stream)), "snack_prune_regrow_rows")


def snack_layer_shape(h):
    m, k = i32(), i32()
    _check(_lib.snack_layer_shape(h, ctypes.byref(m), ctypes.byref(k)), "snack_layer_shape")
    return m.value, k.value


def snack_layer_nnz(h):
    n = i64()
    _check(_lib.snack_layer_nnz(h, ctypes.byref(n)), "snack_layer_nnz")
    return n.value


def snack_layer_device_bytes(h):
    n = i64()
    _check(_lib.snack_layer_device_bytes(h, ctypes.byref(n)), "snack_layer_device_bytes")
    return n.value


def snack_layer_values(h):
    p = P()
    _check(_lib.snack_layer_values(h, ctypes.byref(p)), "snack_layer_values")
    return p.value


def snack_layer_values_updated(h):
    _check(_lib.snack_layer_values_updated(h), "snack_layer_values_updated")


def snack_layer_export(h, rows, cols, vals, stream=None):
    _check(_lib.snack_layer_export(h, _ptr(rows), _ptr(cols), _ptr(vals), _stream(stream)), "snack_layer_export")


def snack_layer_export_index(h, row_ptr, perm, rows_t, col_ptr, vals_t=None, stream=None):
    _check(_lib.snack_layer_export_index(h, _ptr(row_ptr), _ptr(perm), _ptr(rows_t), _ptr(col_ptr), _ptr(vals_t),
                                         _stream(stream)), "snack_layer_export_index")


def snack_layer_get_epoch(h):
    e = u64()
    _check(_lib.snack_layer_get_epoch(h, ctypes.byref(e)), "snack_layer_get_epoch")
    return e.value


def snack_layer_set_epoch(h, epoch):
    _check(_lib.snack_layer_set_epoch(h, epoch), "snack_layer_set_epoch")


def snack_sgd_step(h, dW, lr, stream=None):
    _check(_lib.snack_sgd_step(h, _ptr(dW), float(lr), _stream(stream)), "snack_sgd_step")


def snack_mse_grad(Y, T, dY, scale, stream=None):
    _check(_lib.snack_mse_grad(_ptr(Y), _ptr(T), _ptr(dY), Y.numel(), float(scale), _stream(stream)),
           "snack_mse_grad")


def snack_gelu_fwd(X, Y, stream=None):
    _check(_lib.snack_gelu_fwd(_ptr(X), _ptr(Y), X.numel(), _stream(stream)), "snack_gelu_fwd")


def snack_gelu_bwd(X, dY, dX, stream=None):
    _check(_lib.snack_gelu_bwd(_ptr(X), _ptr(dY), _ptr(dX), X.numel(), _stream(stream)), "snack_gelu_bwd")


F32, BF16, INT8, E4M3 = 0, 1, 2, 3


def snack_ckpt_pack(X, fmt, Q, S, stream=None):
    rows, n = X.shape
    _check(_lib.snack_ckpt_pack(_ptr(X), rows, n, fmt, _ptr(Q), _ptr(S), _stream(stream)), "snack_ckpt_pack")


def snack_ckpt_unpack(Q, S, fmt, Y, y_fmt, stream=None):
    rows, n = Y.shape
    _check(_lib.snack_ckpt_unpack(_ptr(Q), _ptr(S), rows, n, fmt, _ptr(Y), y_fmt, _stream(stream)),
           "snack_ckpt_unpack")


def snack_rmsnorm_fwd(X, R, h_fmt, gain, eps, H, Y, rstd, q_fmt=F32, Q=None, S=None, stream=None):
    rows, n = X.shape
    _check(_lib.snack_rmsnorm_fwd(_ptr(X), _ptr(R), h_fmt, _ptr(gain), eps, rows, n, _ptr(H), _ptr(Y), _ptr(rstd),
                                  q_fmt, _ptr(Q), _ptr(S), _stream(stream)), "snack_rmsnorm_fwd")


@functools.lru_cache(maxsize=256)   # a function of the shape alone
def snack_rmsnorm_bwd_work(rows, n):
    b = i64()
    _check(_lib.snack_rmsnorm_bwd_work(rows, n, ctypes.byref(b)), "snack_rmsnorm_bwd_work")
    return b.value


def snack_rmsnorm_bwd(H, HS, h_fmt, gain, rstd, dY, dR, dX, dgain, work, stream=None):
    """work: a device tensor of at least snack_rmsnorm_bwd_work bytes, or None."""
    rows, n = dY.shape
    nbytes = 0 if work is None else work.numel() * work.element_size()
    _check(_lib.snack_rmsnorm_bwd(_ptr(H), _ptr(HS), h_fmt, _ptr(gain), _ptr(rstd), _ptr(dY), _ptr(dR), rows, n,
                                  _ptr(dX), _ptr(dgain), _ptr(work), nbytes, _stream(stream)), "snack_rmsnorm_bwd")


def snack_gelu_ckpt_fwd(X, fmt, Y, QX=None, SX=None, QY=None, SY=None, stream=None):
    rows, n = X.shape
    _check(_lib.snack_gelu_ckpt_fwd(_ptr(X), rows, n, fmt, _ptr(Y), _ptr(QX), _ptr(SX), _ptr(QY), _ptr(SY),
                                    _stream(stream)), "snack_gelu_ckpt_fwd")


def snack_gelu_ckpt_bwd(QX, SX, fmt, dY, dX, stream=None):
    rows, n = dY.shape
    _check(_lib.snack_gelu_ckpt_bwd(_ptr(QX), _ptr(SX), _ptr(dY), rows, n, fmt, _ptr(dX), _stream(stream)),
           "snack_gelu_ckpt_bwd")


def snack_backward_ckpt(h, Q, S, fmt, dY, dX=None, dW=None, stream=None):
    B = dY.shape[0]
    _check(_lib.snack_backward_ckpt(h, _ptr(Q), _ptr(S), fmt, _ptr(dY), _ptr(dX), _ptr(dW), B, _stream(stream)),
           "snack_backward_ckpt")


E2M1 = 4                      # 4-bit numbers, of a cache only
ROPE_HALF, ROPE_PAIRS = 0, 1


class _Rope(ctypes.Structure):
    _fields_ = [("table", P), ("positions", i32), ("rot", i32), ("layout", i32)]


class _Cache(ctypes.Structure):
    _fields_ = [("data", P), ("pages", i64), ("page_tokens", i32), ("heads", i32), ("head_dim", i32), ("fmt", i32)]


def snack_rope_table(positions, rot, base, factor, trained, low, high, amplitude, table, stream=None):
    """table: float32 [positions, rot], written."""
    _need(table, torch.float32, (positions, rot), "table")
    _check(_lib.snack_rope_table(positions, rot, base, factor, trained, low, high, amplitude, _ptr(table),
                                 _stream(stream)), "snack_rope_table")


def snack_qk_rope_fwd(q, k, x_fmt, pos, rope, q_gain, k_gain, eps, Yq, Yk, y_fmt, stream=None):
    """q, k: [tokens, heads, features] device tensors, each row of features contiguous (k may be None); rope: the
    address of a snack_rope, or None."""
    t, hq, d = q.shape
    _check(_lib.snack_qk_rope_fwd(*_spread(q), hq, *_spread(k), 0 if k is None else k.shape[1], x_fmt, t, d, _ptr(pos),
                                  rope, _ptr(q_gain), _ptr(k_gain), eps, _ptr(Yq), _ptr(Yk), y_fmt, _stream(stream)),
           "snack_qk_rope_fwd")


@functools.lru_cache(maxsize=256)   # a function of the shape alone
def snack_qk_rope_bwd_work(tokens, q_heads, k_heads, head_dim):
    b = i64()
    _check(_lib.snack_qk_rope_bwd_work(tokens, q_heads, k_heads, head_dim, ctypes.byref(b)), "snack_qk_rope_bwd_work")
    return b.value


def snack_qk_rope_bwd(q, k, x_fmt, pos, rope, q_gain, k_gain, eps, dYq, dYk, y_fmt, dXq, dXk, dq_gain, dk_gain, work,
                      stream=None):
    """work: a device tensor of at least snack_qk_rope_bwd_work bytes, or None."""
    t, hq, d = dYq.shape
    nbytes = 0 if work is None else work.numel() * work.element_size()
    _check(_lib.snack_qk_rope_bwd(*_spread(q), hq, *_spread(k), 0 if dYk is None else dYk.shape[1], x_fmt, t, d,
                                  _ptr(pos), rope, _ptr(q_gain), _ptr(k_gain), eps, *_spread(dYq), *_spread(dYk), y_fmt,
                                  _ptr(dXq), _ptr(dXk), _ptr(dq_gain), _ptr(dk_gain), _ptr(work), nbytes,
                                  _stream(stream)), "snack_qk_rope_bwd")


def snack_cache_bytes(cache):
    """cache: the address of a snack_cache (here and below)."""
    b = i64()
    _check(_lib.snack_cache_bytes(cache, ctypes.byref(b)), "snack_cache_bytes")
    return b.value


def snack_cache_slots(cache, table, lens, starts, pos, slot, stream=None):
    _check(_lib.snack_cache_slots(cache, _ptr(table), table.shape[1], _ptr(lens), _ptr(starts), table.shape[0],
                                  pos.numel(), _ptr(pos), _ptr(slot), _stream(stream)), "snack_cache_slots")


def snack_cache_write(cache, k, v, x_fmt, slot, stream=None):
    _check(_lib.snack_cache_write(cache, *_spread(k), *_spread(v), x_fmt, slot.numel(), _ptr(slot), _stream(stream)),
           "snack_cache_write")


def snack_cache_write_rope(cache, q, k, v, x_fmt, pos, slot, rope, q_gain, k_gain, eps, Yq, y_fmt, stream=None):
    _check(_lib.snack_cache_write_rope(cache, *_spread(q), q.shape[1], *_spread(k), *_spread(v), x_fmt, slot.numel(),
                                       _ptr(pos), _ptr(slot), rope, _ptr(q_gain), _ptr(k_gain), eps, _ptr(Yq), y_fmt,
                                       _stream(stream)), "snack_cache_write_rope")


def snack_cache_read(cache, slot, K, V, y_fmt, stream=None):
    _check(_lib.snack_cache_read(cache, _ptr(slot), slot.numel(), _ptr(K), _ptr(V), y_fmt, _stream(stream)),
           "snack_cache_read")


def snack_cache_attend_work(cache, q_heads, tokens, sequences):
    b = i64()
    _check(_lib.snack_cache_attend_work(cache, q_heads, tokens, sequences, ctypes.byref(b)), "snack_cache_attend_work")
    return b.value


def snack_cache_attend(cache, q, q_fmt, table, lens, starts, scale, causal, out, work, stream=None):
    _check(_lib.snack_cache_attend(cache, *_spread(q), q.shape[1], q_fmt, q.shape[0], _ptr(table), table.shape[1],
                                   _ptr(lens), _ptr(starts), table.shape[0], scale, 1 if causal else 0, _ptr(out),
                                   _ptr(work), work.numel() * work.element_size(), _stream(stream)),
           "snack_cache_attend")


def snack_profile_enable(on=True):
    _check(_lib.snack_profile_enable(1 if on else 0), "snack_profile_enable")


def snack_profile_reset():
    _check(_lib.snack_profile_reset(), "snack_profile_reset")


def snack_profile_name(k):
    n = _lib.snack_profile_name(k)
    return None if n is None else n.decode()


def snack_profile_read(k):
    n, ms = i64(), f64()
    _check(_lib.snack_profile_read(k, ctypes.byref(n), ctypes.byref(ms)), "snack_profile_read")
    return n.value, ms.value


def snack_profile_set_tag(tag):
    _check(_lib.snack_profile_set_tag(int(tag)), "snack_profile_set_tag")


def snack_profile_read_tag(k, tag):
    n, ms = i64(), f64()
    _check(_lib.snack_profile_read_tag(k, int(tag), ctypes.byref(n), ctypes.byref(ms)), "snack_profile_read_tag")
    return n.value, ms.value


def profile_class_ids():
    """{kernel class name: id}."""
    out, k = {}, 0
    while True:
        name = snack_profile_name(k)
        if name is None:
            return out
        out[name] = k
        k += 1


def profile_snapshot():
    """{kernel class name: (launches, total ms)} for every class."""
    out, k = {}, 0
    while True:
        name = snack_profile_name(k)
        if name is None:
            return out
        out[name] = snack_profile_read(k)
        k += 1


# ---------------------------------------------------------------------------
# Activation checkpoints, the norm and the GELU (tensors made by the call)
# ---------------------------------------------------------------------------

# These calls are a few microseconds of GPU work at the smallest sizes, so the host side is kept short: one check of
# each tensor, one allocation for a checkpoint, and no stream object.  With `stream`, the call and the tensors it
# makes are that stream's.

_HIDDEN = {torch.float32: F32, torch.bfloat16: BF16}
_BLOCK = 32   # features of a row that share one exponent byte
_FLOAT, _BYTE = torch.float32, torch.uint8
_raw_stream = torch._C._cuda_getCurrentRawStream


def _arg(t, shape, name, dev, dtype=_FLOAT):
    """The address of t, a contiguous tensor of this dtype and shape on GPU `dev`."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the same GPU as the other tensors")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _rows(t, name, dtype=_FLOAT):
    """rows, features, address and GPU of t, a contiguous [rows, features] tensor on the current GPU."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    shape = t.shape
    if len(shape) != 2 or shape[1] < 1:
        raise ValueError(f"{name} must be [rows, features], got {tuple(shape)}")
    dev = t.get_device()
    if dev < 0 or dev != torch._C._cuda_getDevice():
        raise ValueError(f"{name} must be on the current GPU")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return shape[0], shape[1], t.data_ptr(), dev


class Ckpt:
    """An activation [rows, n] kept in 8 bits: codes q [rows, 32 ceil(n / 32)] and one exponent byte for every
    32 features of a row, s [rows, ceil(n / 32)] (uint8 device tensors); a code c stands for c * 2^(s - 127), c a
    signed integer (INT8) or an e4m3 number (E4M3).  33/32 bytes a value."""

    __slots__ = ("rows", "n", "fmt", "_q", "_s", "_buf")

    def __init__(self, q, s, fmt, n):
        if fmt != INT8 and fmt != E4M3:
            raise ValueError("a checkpoint's format is INT8 or E4M3")
        if n < 1:
            raise ValueError("a checkpoint has at least one feature")
        nb = -(-n // _BLOCK)
        rows, width, _, dev = _rows(q, "q", _BYTE)
        if width != _BLOCK * nb:
            raise ValueError(f"q must have {_BLOCK * nb} bytes a row, got {width}")
        _arg(s, (rows, nb), "s", dev, _BYTE)
        self.rows, self.n, self.fmt, self._q, self._s, self._buf = rows, n, fmt, q, s, None

    @classmethod
    def _room(cls, like, rows, n, fmt):
        """Room for a checkpoint beside `like`: codes and exponent bytes in one allocation."""
        if fmt != INT8 and fmt != E4M3:
            raise ValueError("a checkpoint's format is INT8 or E4M3")
        ck = cls.__new__(cls)
        ck.rows, ck.n, ck.fmt, ck._q, ck._s = rows, n, fmt, None, None
        ck._buf = like.new_empty(rows * -(-n // _BLOCK) * (_BLOCK + 1), dtype=_BYTE)
        return ck

    def _ptrs(self):
        if self._buf is None:
            return self._q.data_ptr(), self._s.data_ptr()
        p = self._buf.data_ptr()
        return p, p + self.rows * -(-self.n // _BLOCK) * _BLOCK

    def _dev(self):
        """Its GPU, which has to be the current one."""
        dev = (self._q if self._buf is None else self._buf).get_device()
        if dev != torch._C._cuda_getDevice():
            raise ValueError("the checkpoint must be on the current GPU")
        return dev

    @property
    def q(self):
        if self._q is None:
            nb = -(-self.n // _BLOCK)
            self._q = self._buf[: self.rows * nb * _BLOCK].view(self.rows, nb * _BLOCK)
        return self._q

    @property
    def s(self):
        if self._s is None:
            nb = -(-self.n // _BLOCK)
            self._s = self._buf[self.rows * nb * _BLOCK:].view(self.rows, nb)
        return self._s

    @property
    def nbytes(self):
        return self.rows * -(-self.n // _BLOCK) * (_BLOCK + 1)

    @classmethod
    def pack(cls, x, fmt, stream=None):
        """The checkpoint of x, float32 [rows, n]."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return cls.pack(x, fmt)
        rows, n, px, dev = _rows(x, "x")
        ck = cls._room(x, rows, n, fmt)
        q, s = ck._ptrs()
        _check(_lib.snack_ckpt_pack(px, rows, n, fmt, q, s, _raw_stream(dev)), "snack_ckpt_pack")
        return ck

    def unpack(self, dtype=torch.float32, stream=None):
        """The values it stands for, in float32 or bfloat16."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.unpack(dtype)
        y_fmt = _HIDDEN.get(dtype)
        if y_fmt is None:
            raise TypeError("a checkpoint is read as float32 or bfloat16")
        dev = self._dev()
        own = self._q if self._buf is None else self._buf
        y = own.new_empty((self.rows, self.n), dtype=dtype)
        q, s = self._ptrs()
        _check(_lib.snack_ckpt_unpack(q, s, self.rows, self.n, self.fmt, y.data_ptr(), y_fmt,
                                      _raw_stream(dev)), "snack_ckpt_unpack")
        return y


def rmsnorm_fwd(x, gain, eps, residual=None, q_format=None, want_y=True, stream=None):
    """h = x + residual, y = h / sqrt(mean(h^2) + eps) * gain over the rows of x, float32 [rows, n].

    residual: float32 or bfloat16 [rows, n]; h has its type (None: h is x itself).  q_format: INT8 or E4M3 also
    leaves y's checkpoint; with want_y=False only that.  Returns (h, y, rstd, checkpoint), None where there is none."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return rmsnorm_fwd(x, gain, eps, residual, q_format, want_y)
    rows, n, px, dev = _rows(x, "x")
    pg = _arg(gain, (n,), "gain", dev)
    if not want_y and q_format is None:
        raise ValueError("neither y nor its checkpoint is wanted")
    h_fmt, h, pr, ph = F32, x, None, None
    if residual is not None:
        h_fmt = _HIDDEN.get(getattr(residual, "dtype", None))
        if h_fmt is None:
            raise TypeError("residual must be a float32 or bfloat16 tensor")
        pr = _arg(residual, x.shape, "residual", dev, residual.dtype)
        h = torch.empty_like(residual)
        ph = h.data_ptr()
    y = torch.empty_like(x) if want_y else None
    rstd = x.new_empty(rows)
    ck, q, s = None, None, None
    if q_format is not None:
        ck = Ckpt._room(x, rows, n, q_format)
        q, s = ck._ptrs()
    _check(_lib.snack_rmsnorm_fwd(px, pr, h_fmt, pg, eps, rows, n, ph, y.data_ptr() if want_y else None,
                                  rstd.data_ptr(), F32 if ck is None else q_format, q, s, _raw_stream(dev)),
           "snack_rmsnorm_fwd")
    return h, y, rstd, ck


def rmsnorm_bwd(h, gain, rstd, dY, dR=None, want_dgain=True, stream=None):
    """The gradient of rmsnorm_fwd: h as float32 or bfloat16 [rows, n] or as a Ckpt, rstd the forward's, dY float32,
    dR the gradient that reaches h along the residual stream (None: none).  Returns (dX, dgain): dX is the gradient
    of both x and residual, dgain None where it is not wanted."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return rmsnorm_bwd(h, gain, rstd, dY, dR, want_dgain)
    rows, n, pd, dev = _rows(dY, "dY")
    if isinstance(h, Ckpt):
        if h.rows != rows or h.n != n:
            raise ValueError(f"h must have shape {(rows, n)}, got {(h.rows, h.n)}")
        if h._dev() != dev:
            raise ValueError("h must be on the same GPU as the other tensors")
        fmt = h.fmt
        ph, ps = h._ptrs()
    else:
        fmt = _HIDDEN.get(getattr(h, "dtype", None))
        if fmt is None:
            raise TypeError("h must be a float32 or bfloat16 tensor or a Ckpt")
        ph, ps = _arg(h, dY.shape, "h", dev, h.dtype), None
    pg, pt = _arg(gain, (n,), "gain", dev), _arg(rstd, (rows,), "rstd", dev)
    pr = None if dR is None else _arg(dR, dY.shape, "dR", dev)
    dX = torch.empty_like(dY)
    dgain = torch.empty_like(gain) if want_dgain else None
    nbytes = snack_rmsnorm_bwd_work(rows, n)
    work = dY.new_empty(nbytes, dtype=_BYTE)
    _check(_lib.snack_rmsnorm_bwd(ph, ps, fmt, pg, pt, pd, pr, rows, n, dX.data_ptr(),
                                  dgain.data_ptr() if want_dgain else None, work.data_ptr(), nbytes,
                                  _raw_stream(dev)), "snack_rmsnorm_bwd")
    return dX, dgain


def gelu_ckpt_fwd(x, fmt, want_y=True, stream=None):
    """Exact GELU of x, float32 [rows, n].  Returns (y, checkpoint of x, checkpoint of y)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return gelu_ckpt_fwd(x, fmt, want_y)
    rows, n, px, dev = _rows(x, "x")
    y = torch.empty_like(x) if want_y else None
    cx, cy = Ckpt._room(x, rows, n, fmt), Ckpt._room(x, rows, n, fmt)
    qx, sx = cx._ptrs()
    qy, sy = cy._ptrs()
    _check(_lib.snack_gelu_ckpt_fwd(px, rows, n, fmt, y.data_ptr() if want_y else None, qx, sx, qy, sy,
                                    _raw_stream(dev)), "snack_gelu_ckpt_fwd")
    return y, cx, cy


def gelu_ckpt_bwd(ck, dY, stream=None):
    """dY (Phi(x) + x phi(x)) with x read from its checkpoint; dY float32 [rows, n]."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return gelu_ckpt_bwd(ck, dY)
    dev = ck._dev()
    pd = _arg(dY, (ck.rows, ck.n), "dY", dev)
    dX = torch.empty_like(dY)
    q, s = ck._ptrs()
    _check(_lib.snack_gelu_ckpt_bwd(q, s, pd, ck.rows, ck.n, ck.fmt, dX.data_ptr(), _raw_stream(dev)),
           "snack_gelu_ckpt_bwd")
    return dX


# ---------------------------------------------------------------------------
# The attention half of a block: norms and rotation of queries and keys, the cache, the attention over it
# ---------------------------------------------------------------------------

def _heads(t, name, dev=None, dtype=None, shape=None):
    """Address, token stride and head stride of t, [tokens, heads, features] on the current GPU (or on GPU `dev`), each
    row of features contiguous."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype not in _HIDDEN or (dtype is not None and t.dtype is not dtype):
        raise TypeError(f"{name} must be {dtype if dtype is not None else 'float32 or bfloat16'}, got {t.dtype}")
    if shape is None:
        if t.dim() != 3 or not 1 <= t.shape[2] <= 256 or t.shape[1] < 1:
            raise ValueError(f"{name} must be [tokens, heads, features] of at most 256 features, got {tuple(t.shape)}")
    elif t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    on = t.get_device()
    if dev is None:
        if on < 0 or on != torch._C._cuda_getDevice():
            raise ValueError(f"{name} must be on the current GPU")
    elif on != dev:
        raise ValueError(f"{name} must be on the same GPU as the other tensors")
    row, head, one = t.stride()
    if one != 1 and t.shape[2] != 1:
        raise ValueError(f"{name} must have contiguous features")
    return t.data_ptr(), row, head


class RopeTable:
    """The table of rotary positions: float32 [positions, rot], for every position the cosines of rot / 2 angles, then
    their sines; the first rot features of a head are rotated.  layout: ROPE_HALF (feature i turns with i + rot / 2) or
    ROPE_PAIRS (feature 2 i with 2 i + 1)."""

    __slots__ = ("table", "layout", "_c", "_ref")

    def __init__(self, table, layout=ROPE_HALF):
        positions, rot, p, _ = _rows(table, "table")
        if rot % 2 or rot > 256:
            raise ValueError("an even number of features, at most 256, is rotated")
        if positions < 1 or layout not in (ROPE_HALF, ROPE_PAIRS):
            raise ValueError("a table has a position at least, and the layout ROPE_HALF or ROPE_PAIRS")
        self.table, self.layout = table, layout
        self._c = _Rope(p, positions, rot, layout)
        self._ref = ctypes.addressof(self._c)

    @classmethod
    def make(cls, positions, rot, base=10000.0, layout=ROPE_HALF, factor=1.0, trained=0.0, low=1.0, high=32.0,
             amplitude=1.0, stream=None):
        """cos and sin of p f_i, f_i = base^(-2 i / rot), times amplitude, on the current GPU.  For contexts `factor`
        times as long as the trained one: every f_i / factor, or with `trained` (its tokens) only those of pairs that
        make at most `low` turns in it; of at least `high` turns f_i stays, in between it is interpolated."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return cls.make(positions, rot, base, layout, factor, trained, low, high, amplitude)
        if positions < 1 or rot < 2:
            raise ValueError("a table has a position and a pair at least")
        table = torch.empty((positions, rot), dtype=_FLOAT, device=torch.cuda.current_device())
        rope = cls(table, layout)
        _check(_lib.snack_rope_table(positions, rot, base, factor, trained, low, high, amplitude, table.data_ptr(),
                                     _raw_stream(table.get_device())), "snack_rope_table")
        return rope

    @property
    def positions(self):
        return self._c.positions

    @property
    def rot(self):
        return self._c.rot

    def _on(self, dev):
        if self.table.get_device() != dev:
            raise ValueError("the rotation's table must be on the same GPU as the other tensors")
        return self._ref


def _qk_args(pos, rope, q_gain, k_gain, tokens, d, dev):
    """Addresses of what norm and rotation take beside the heads."""
    if rope is None and q_gain is None and k_gain is None:
        raise ValueError("neither a rotation nor a gain is given")
    pp = pr = None
    if rope is not None:
        if rope.rot > d:
            raise ValueError(f"the rotation is of {rope.rot} features, a head has {d}")
        pr = rope._on(dev)
        pp = _arg(pos, (tokens,), "pos", dev, torch.int32)
    gq = None if q_gain is None else _arg(q_gain, (d,), "q_gain", dev)
    gk = None if k_gain is None else _arg(k_gain, (d,), "k_gain", dev)
    return pp, pr, gq, gk


def qk_rope_fwd(q, k, pos=None, rope=None, q_gain=None, k_gain=None, eps=1e-6, dtype=None, stream=None):
    """Norms of queries and keys for each head, y = x / sqrt(mean(x^2) + eps) * gain, then the rotation of y by the
    tokens' positions pos (int32 [tokens]).

    q, k: float32 or bfloat16 [tokens, heads, features], as they lie in the projections' output (each head's features
    contiguous); k may be None.  rope: a RopeTable, None for none; q_gain, k_gain: float32 [features], None: those heads
    are not normed.  Returns (q', k') in dtype (None: q's)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return qk_rope_fwd(q, k, pos, rope, q_gain, k_gain, eps, dtype)
    aq = _heads(q, "q")
    t, hq, d = q.shape
    dev = q.get_device()
    y_fmt = _HIDDEN.get(q.dtype if dtype is None else dtype)
    if y_fmt is None:
        raise TypeError("queries and keys are written as float32 or bfloat16")
    pp, pr, gq, gk = _qk_args(pos, rope, q_gain, k_gain, t, d, dev)
    yq = torch.empty((t, hq, d), dtype=q.dtype if dtype is None else dtype, device=q.device)
    ak, hk, yk, pk = (None, 0, 0), 0, None, None
    if k is not None:
        hk = k.shape[1] if k.dim() == 3 else 1
        ak = _heads(k, "k", dev, q.dtype, (t, hk, d))
        if hk < 1:
            raise ValueError("k must have a head at least")
        yk = torch.empty((t, hk, d), dtype=yq.dtype, device=q.device)
        pk = yk.data_ptr()
    _check(_lib.snack_qk_rope_fwd(*aq, hq, *ak, hk, _HIDDEN[q.dtype], t, d, pp, pr, gq, gk, eps, yq.data_ptr(), pk,
                                  y_fmt, _raw_stream(dev)), "snack_qk_rope_fwd")
    return yq, yk


def qk_rope_bwd(q, k, pos, dq, dk, rope=None, q_gain=None, k_gain=None, eps=1e-6, stream=None):
    """The gradient of qk_rope_fwd from those of its outputs, dq and dk (float32 or bfloat16, each head's features
    contiguous; k and dk None for none).  Returns (gradient of q, of k, of q_gain, of k_gain), None where there is no
    such input."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return qk_rope_bwd(q, k, pos, dq, dk, rope, q_gain, k_gain, eps)
    aq = _heads(q, "q")
    t, hq, d = q.shape
    dev = q.get_device()
    adq = _heads(dq, "dq", dev, None, (t, hq, d))
    pp, pr, gq, gk = _qk_args(pos, rope, q_gain, k_gain, t, d, dev)
    dxq = torch.empty((t, hq, d), dtype=q.dtype, device=q.device)
    ak = adk = (None, 0, 0)
    hk, dxk, pk = 0, None, None
    if (k is None) != (dk is None):
        raise ValueError("k and dk must both be given, or neither")
    if k is not None:
        hk = k.shape[1] if k.dim() == 3 else 1
        ak = _heads(k, "k", dev, q.dtype, (t, hk, d))
        adk = _heads(dk, "dk", dev, dq.dtype, (t, hk, d))
        if hk < 1:
            raise ValueError("k must have a head at least")
        dxk = torch.empty((t, hk, d), dtype=q.dtype, device=q.device)
        pk = dxk.data_ptr()
    elif k_gain is not None:
        raise ValueError("k_gain is given without k")
    dgq = None if q_gain is None else torch.empty_like(q_gain)
    dgk = None if k_gain is None else torch.empty_like(k_gain)
    work, nbytes, pw = None, 0, None
    if dgq is not None or dgk is not None:
        nbytes = snack_qk_rope_bwd_work(t, hq, hk, d)
        work = q.new_empty(nbytes, dtype=_BYTE)
        pw = work.data_ptr()
    _check(_lib.snack_qk_rope_bwd(*aq, hq, *ak, hk, _HIDDEN[q.dtype], t, d, pp, pr, gq, gk, eps, *adq, *adk,
                                  _HIDDEN[dq.dtype], dxq.data_ptr(), pk, None if dgq is None else dgq.data_ptr(),
                                  None if dgk is None else dgk.data_ptr(), pw, nbytes, _raw_stream(dev)),
           "snack_qk_rope_bwd")
    return dxq, dxk, dgq, dgk


class KVCache:
    """Keys and values of attention heads kept in 8 bits (INT8, E4M3) or 4 (E2M1), with an exponent byte for every 32
    features of a token's head, in pages of `page` tokens (a multiple of 32).

    A token's place is its slot, page * tokens of a page + offset; which pages are a sequence's says a page table, int32
    [sequences, width]; lens, int32 [sequences], are the sequences' tokens in the cache with those of the call.  A call's
    tokens are the newest of every sequence, one sequence after the other: starts, int32 [sequences + 1], says where each
    begins (None: equally many of every sequence).  data: uint8 of KVCache.nbytes_of(...) bytes, or None (allocated; not
    cleared: what no token was written to may hold anything)."""

    __slots__ = ("data", "_c", "_ref", "_dev", "_work")

    def __init__(self, pages, heads, head_dim, fmt, page=64, data=None):
        self._c = _Cache(None, pages, page, heads, head_dim, fmt)
        self._ref = ctypes.addressof(self._c)
        nbytes = snack_cache_bytes(self._ref)
        if data is None:
            data = torch.empty(nbytes, dtype=_BYTE, device=torch.cuda.current_device())
        elif not isinstance(data, torch.Tensor) or data.get_device() < 0:
            raise TypeError("data must be a tensor on the GPU")
        self._dev = data.get_device()
        self._c.data = _arg(data, (nbytes,), "data", self._dev, _BYTE)
        self.data, self._work = data, {}
        self._on()

    @staticmethod
    def nbytes_of(pages, heads, head_dim, fmt, page=64):
        c = _Cache(None, pages, page, heads, head_dim, fmt)
        return snack_cache_bytes(ctypes.addressof(c))

    pages = property(lambda self: self._c.pages)
    page = property(lambda self: self._c.page_tokens)
    heads = property(lambda self: self._c.heads)
    head_dim = property(lambda self: self._c.head_dim)
    fmt = property(lambda self: self._c.fmt)
    nbytes = property(lambda self: self.data.numel())

    def _on(self):
        if self._dev != torch._C._cuda_getDevice():
            raise ValueError("the cache must be on the current GPU")
        return self._dev

    def _sequences(self, table, lens, starts, dev):
        if not isinstance(table, torch.Tensor) or table.dim() != 2 or table.shape[1] < 1:
            raise ValueError("table must be [sequences, pages]")
        n, width = table.shape
        return (_arg(table, table.shape, "table", dev, torch.int32), width, _arg(lens, (n,), "lens", dev, torch.int32),
                None if starts is None else _arg(starts, (n + 1,), "starts", dev, torch.int32), n)

    def slots(self, table, lens, tokens, starts=None, stream=None):
        """(pos, slot): position (int32) and place in the cache (int64) of a call's tokens; slot -1 where there is none.
        The same for every block of a model."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.slots(table, lens, tokens, starts)
        dev = self._on()
        pt, width, pl, ps, n = self._sequences(table, lens, starts, dev)
        if starts is None and (n == 0 or tokens % n):
            raise ValueError("without starts the tokens must divide among the sequences")
        pos = torch.empty(tokens, dtype=torch.int32, device=table.device)
        slot = torch.empty(tokens, dtype=torch.int64, device=table.device)
        _check(_lib.snack_cache_slots(self._ref, pt, width, pl, ps, n, tokens, pos.data_ptr(), slot.data_ptr(),
                                      _raw_stream(dev)), "snack_cache_slots")
        return pos, slot

    def write(self, k, v, slot, stream=None):
        """Keep keys and values, float32 or bfloat16 [tokens, heads, features], at distinct slots (int64 [tokens]; those
        outside the cache are not written)."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.write(k, v, slot)
        dev = self._on()
        t = slot.shape[0] if isinstance(slot, torch.Tensor) and slot.dim() else 0
        ps = _arg(slot, (t,), "slot", dev, torch.int64)
        shape = (t, self._c.heads, self._c.head_dim)
        ak = _heads(k, "k", dev, None, shape)
        av = _heads(v, "v", dev, k.dtype, shape)
        _check(_lib.snack_cache_write(self._ref, *ak, *av, _HIDDEN[k.dtype], t, ps, _raw_stream(dev)),
               "snack_cache_write")

    def write_rope(self, q, k, v, pos, slot, rope=None, q_gain=None, k_gain=None, eps=1e-6, dtype=None, stream=None):
        """qk_rope_fwd whose keys go into the cache, the values with them, in one launch.  Returns q'."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.write_rope(q, k, v, pos, slot, rope, q_gain, k_gain, eps, dtype)
        dev = self._on()
        aq = _heads(q, "q", dev)
        t, hq, d = q.shape
        if d != self._c.head_dim:
            raise ValueError(f"a head of the cache has {self._c.head_dim} features, got {d}")
        shape = (t, self._c.heads, d)
        ak, av = _heads(k, "k", dev, q.dtype, shape), _heads(v, "v", dev, q.dtype, shape)
        y_fmt = _HIDDEN.get(q.dtype if dtype is None else dtype)
        if y_fmt is None:
            raise TypeError("queries are written as float32 or bfloat16")
        pp, pr, gq, gk = _qk_args(pos, rope, q_gain, k_gain, t, d, dev)
        ps = _arg(slot, (t,), "slot", dev, torch.int64)
        yq = torch.empty((t, hq, d), dtype=q.dtype if dtype is None else dtype, device=q.device)
        _check(_lib.snack_cache_write_rope(self._ref, *aq, hq, *ak, *av, _HIDDEN[q.dtype], t, pp, ps, pr, gq, gk, eps,
                                           yq.data_ptr(), y_fmt, _raw_stream(dev)), "snack_cache_write_rope")
        return yq

    def read(self, slot, dtype=torch.float32, stream=None):
        """(keys, values) that the cache stands for at slots (int64 [tokens]), [tokens, heads, features] in float32 or
        bfloat16; zeros at a negative slot, NaN past the cache."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.read(slot, dtype)
        dev = self._on()
        y_fmt = _HIDDEN.get(dtype)
        if y_fmt is None:
            raise TypeError("a cache is read as float32 or bfloat16")
        t = slot.shape[0] if isinstance(slot, torch.Tensor) and slot.dim() else 0
        ps = _arg(slot, (t,), "slot", dev, torch.int64)
        shape = (t, self._c.heads, self._c.head_dim)
        k = torch.empty(shape, dtype=dtype, device=slot.device)
        v = torch.empty(shape, dtype=dtype, device=slot.device)
        _check(_lib.snack_cache_read(self._ref, ps, t, k.data_ptr(), v.data_ptr(), y_fmt, _raw_stream(dev)),
               "snack_cache_read")
        return k, v

    def attend(self, q, table, lens, starts=None, scale=None, causal=True, out=None, stream=None):
        """softmax(scale q . k) v over the tokens of each query's sequence, those up to its own with `causal` (else all:
        an encoder's states).  q: float32 or bfloat16 [tokens, query heads, features], each head's features contiguous,
        query heads a multiple of the cache's; scale: 1 / sqrt(features) if None.  Returns out (contiguous, of q's type
        and shape, apart from q); a query that sees no token gets 0, rows of no sequence are not written."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.attend(q, table, lens, starts, scale, causal, out)
        dev = self._on()
        aq = _heads(q, "q", dev)
        t, hq, d = q.shape
        if d != self._c.head_dim or hq % self._c.heads:
            raise ValueError(f"q must have heads of {self._c.head_dim} features, a multiple of {self._c.heads} of them")
        pt, width, pl, ps, n = self._sequences(table, lens, starts, dev)
        if starts is None and (n == 0 or t % n):
            raise ValueError("without starts the tokens must divide among the sequences")
        if out is None:
            out = torch.empty((t, hq, d), dtype=q.dtype, device=q.device)
        po = _arg(out, (t, hq, d), "out", dev, q.dtype)
        key = (hq, t, n)
        nbytes = self._work.get(key)
        if nbytes is None:
            if len(self._work) >= 256:
                self._work.clear()
            nbytes = self._work[key] = snack_cache_attend_work(self._ref, hq, t, n)
        work = q.new_empty(nbytes, dtype=_BYTE)
        _check(_lib.snack_cache_attend(self._ref, *aq, hq, _HIDDEN[q.dtype], t, pt, width, pl, ps, n,
                                       d ** -0.5 if scale is None else scale, 1 if causal else 0, po, work.data_ptr(),
                                       nbytes, _raw_stream(dev)), "snack_cache_attend")
        return out


# ---------------------------------------------------------------------------
# Convenience object over the same calls
# ---------------------------------------------------------------------------

class SnackLayer:
    """Owns one layer handle.  Tensors are torch device tensors."""

    def __init__(self, M, K, rows, cols, vals=None, seed=0, stream=None, max_batch=None):
        """max_batch: also reserve the workspace for batches up to it (create covers up to 64)."""
        self.M, self.K = int(M), int(K)
        self.h = snack_layer_create(self.M, self.K, rows, cols, vals, seed, stream)
        self.nnz = snack_layer_nnz(self.h)
        if max_batch is not None:
            snack_layer_reserve(self.h, int(max_batch))

    def close(self):
        if getattr(self, "h", None):
            snack_layer_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def forward(self, X, Y=None, stream=None):
        import torch
        if Y is None:
            Y = torch.empty((X.shape[0], self.M), dtype=torch.float32, device=X.device)
        snack_forward(self.h, X, Y, stream)
        return Y

    def backward(self, X, dY, want_dx=True, want_dw=True, dX=None, dW=None, stream=None):
        import torch
        if want_dx and dX is None:
            dX = torch.empty((dY.shape[0], self.K), dtype=torch.float32, device=dY.device)
        if want_dw and dW is None:
            dW = torch.empty((self.nnz,), dtype=torch.float32, device=dY.device)
        snack_backward(self.h, X, dY, dX if want_dx else None, dW if want_dw else None, stream)
        return (dX if want_dx else None), (dW if want_dw else None)

    def backward_ckpt(self, ck, dY, want_dx=True, want_dw=True, dX=None, dW=None, stream=None):
        """backward() with its input read from a checkpoint (Ckpt of [B, K]); returns (dX, dW)."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.backward_ckpt(ck, dY, want_dx, want_dw, dX, dW)
        rows, dev = ck.rows, ck._dev()
        if ck.n != self.K:
            raise ValueError(f"the checkpoint must have {self.K} features, got {ck.n}")
        pd = _arg(dY, (rows, self.M), "dY", dev)
        px = pw = None
        if want_dx:
            if dX is None:
                dX = dY.new_empty((rows, self.K))
            px = _arg(dX, (rows, self.K), "dX", dev)
        if want_dw:
            if dW is None:
                dW = dY.new_empty(self.nnz)
            pw = _arg(dW, (self.nnz,), "dW", dev) or None
        q, s = ck._ptrs()
        _check(_lib.snack_backward_ckpt(self.h, q, s, ck.fmt, pd, px, pw, rows, _raw_stream(dev)),
               "snack_backward_ckpt")
        return (dX if want_dx else None), (dW if want_dw else None)

    def backward_sgd(self, X, dY, lr, want_dx=True, dX=None, dW=None, stream=None):
        import torch
        if want_dx and dX is None:
            dX = torch.empty((dY.shape[0], self.K), dtype=torch.float32, device=dY.device)
        if dW is None:
            dW = torch.empty((self.nnz,), dtype=torch.float32, device=dY.device)
        snack_backward_sgd(self.h, X, dY, dX if want_dx else None, dW, lr, stream)
        return (dX if want_dx else None), dW

    def train_step_mse(self, X, T, lr, want_dx=True, scale=None, out=None, stream=None):
        """Forward, MSE gradient (scale defaults to the mean's 2 / (B * M)), backward and SGD step in one
        call; returns (Y, dY, dX, dW).  `out` may supply that tuple of preallocated tensors."""
        import torch
        B = X.shape[0]
        if scale is None:
            scale = 2.0 / (B * self.M)
        if out is None:
            dev = X.device
            out = (torch.empty((B, self.M), dtype=torch.float32, device=dev),
                   torch.empty((B, self.M), dtype=torch.float32, device=dev),
                   torch.empty((B, self.K), dtype=torch.float32, device=dev) if want_dx else None,
                   torch.empty((self.nnz,), dtype=torch.float32, device=dev))
        Y, dY, dX, dW = out
        snack_train_step_mse(self.h, X, T, Y, dY, dX if want_dx else None, dW, scale, lr, stream)
        return Y, dY, (dX if want_dx else None), dW

    def prune_regrow(self, n_drop, stream=None):
        snack_prune_regrow(self.h, n_drop, stream)

    def prune_regrow_grad(self, n_drop, X, dY, stream=None):
        snack_prune_regrow_grad(self.h, n_drop, X, dY, stream)

    def prune_regrow_rows(self, drop_num, drop_den, mode=REGROW_RANDOM, X=None, dY=None, stream=None):
        snack_prune_regrow_rows(self.h, drop_num, drop_den, mode, X, dY, stream)

    def sgd_step(self, dW, lr, stream=None):
        snack_sgd_step(self.h, dW, lr, stream)

    def export(self, device="cuda", stream=None):
        import torch
        r = torch.empty(self.nnz, dtype=torch.int32, device=device)
        c = torch.empty(self.nnz, dtype=torch.int32, device=device)
        v = torch.empty(self.nnz, dtype=torch.float32, device=device)
        snack_layer_export(self.h, r, c, v, stream)
        return r, c, v

    def export_index(self, device="cuda", stream=None, with_values=False):
        import torch
        rp = torch.empty(self.M + 1, dtype=torch.int32, device=device)
        pm = torch.empty(self.nnz, dtype=torch.int32, device=device)
        rt = torch.empty(self.nnz, dtype=torch.int32, device=device)
        cp = torch.empty(self.K + 1, dtype=torch.int32, device=device)
        vt = torch.empty(self.nnz, dtype=torch.float32, device=device)
        ok = self.nnz > 0
        snack_layer_export_index(self.h, rp, pm if ok else None, rt if ok else None, cp,
                                 vt if (ok and with_values) else None, stream)
        if with_values:
            return rp, pm, rt, cp, vt
        return rp, pm, rt, cp

    def values_ptr(self):
        return snack_layer_values(self.h)

    @property
    def epoch(self):
        return snack_layer_get_epoch(self.h)

    @epoch.setter
    def epoch(self, e):
        snack_layer_set_epoch(self.h, e)

    def device_bytes(self):
        return snack_layer_device_bytes(self.h)

    def reserve(self, max_batch):
        snack_layer_reserve(self.h, max_batch)
