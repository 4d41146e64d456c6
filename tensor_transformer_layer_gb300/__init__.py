"""Python binding of libmptp (the C-ABI library in ``_lib/libmptp.so``).

Argument marshalling only: every function below checks the torch tensors'
dtype, shape, device and contiguity, takes their device pointers and the
current CUDA stream, and calls the C entry point of the same name. All compute
runs in the library's CUDA kernels. There is no fallback: if the library is
missing or fails to load, calls raise. The calls of a decoding step go through
an extension first (``_lib/_mptp_bind.so``) that marshals ordinary arguments
faster and leaves the others to the checks here.

Shapes (row-major, contiguous):
  mp_mlp_fwd(X[T,h], A[h,f], B[f,h], Z[T,h], Y[T,f], U_save[T,f] | None, t)
  mp_mlp_bwd(X, A, B, U[T,f], Y[T,f], dZ[T,h], dX[T,h], dA[h,f], dB[f,h], dU_ws[T,f], t)
  mp_mlp_fwd_shards / mp_mlp_bwd_shards: the same with shard_begin, shard_count
  mp_mlp_fwd_fused / mp_mlp_bwd_fused: the same, one launch per direction, with a zeroed
      uint8 workspace of mp_mlp_fused_workspace_bytes(T, h, f, t) bytes
  mp_vocab_ce(X[T,h], E[v_pad,h], target[T] int32, loss[T] fp32, workspace uint8, v_valid, t)
  mp_rope_axes(x[T,heads,d], y[T,heads,d], pos[axes,T] int32, sections)
  mp_attn_varlen_fwd(Q[Tq,heads,d], K[Tk,kv,d], V[Tk,kv,d], O[Tq,heads,d], LSE[heads,Tq] fp32, cu_q, cu_k int32)
  mp_attn_varlen_bwd(Q, K, V, O, LSE, dO, dQ, dK, dV, delta_ws[heads,Tq] fp32, cu_q, cu_k)
      (these three take rows of any pitch, e.g. parts of a packed projection)
  mp_qk_norm_rope(x[T,heads,d], y[T,heads,d], wq[d], wk[d], pos[axes,T] int32, q_heads, sections)
  mp_qk_norm_rope_bwd(x, dy, dx, wq, wk, dwq[d] fp32, dwk[d] fp32, pos, workspace, q_heads, sections)
  mp_kv_cache_write(K[T,kv,d], V[T,kv,d], kc[pages,kv,page,d] e4m3, vc, ks[pages,kv] fp32, vs,
                    page_table[nseq,max_pages] int32, cu[nseq+1] int32, start[nseq] int32, max_n)
  mp_kv_cache_read(kc, vc, ks, vs, K, V, page_table, cu, start, max_n)
  mp_attn_cache_fwd(Q[Tq,heads,d], kc, vc, ks, vs, O[Tq,heads,d], LSE[heads,Tq] fp32, page_table, cu_q[nseq+1],
                    lens[nseq] int32, workspace, max_q, causal)
      (the pools may be views of one pool, e.g. pool[:, 0] and pool[:, 1])
  mp_glu_fwd(X[T,h], W[h,2f], Wd[f,h], Z[T,h], Y[T,f], GU_save[T,2f] | None, t, act)
  mp_glu_bwd(X, W, Wd, GU, Y, dZ[T,h], dX[T,h], dW[h,2f], dWd[f,h], dGU_ws[T,2f], t, act)
"""
from __future__ import annotations

import ctypes
import functools
import importlib.util
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_lib", "libmptp.so")
BIND_PATH = os.path.join(_PKG, "_lib", "_mptp_bind.so")

MP_OK = 0
MP_DEV_TIMEOUT = 0x1
MP_DEV_TARGET_RANGE = 0x2
MP_DEV_SEQ_RANGE = 0x4
MP_DEV_PAGE_RANGE = 0x8
STATUS_NAMES = {
    0: "MP_OK", 1: "MP_ERR_INVALID_ARG", 2: "MP_ERR_UNSUPPORTED_SHAPE", 3: "MP_ERR_MISALIGNED",
    4: "MP_ERR_NO_DEVICE", 5: "MP_ERR_CUDA", 6: "MP_ERR_TIMEOUT", 7: "MP_ERR_TARGET_RANGE",
    8: "MP_ERR_WORKSPACE", 9: "MP_ERR_SEQ_RANGE", 10: "MP_ERR_PAGE_RANGE",
}
# Every symbol include/mptp.h declares.
EXPORTS = ("mp_mlp_fwd", "mp_mlp_bwd", "mp_mlp_fwd_shards", "mp_mlp_bwd_shards", "mp_mlp_fused_workspace_bytes",
           "mp_mlp_fwd_fused", "mp_mlp_bwd_fused", "mp_vocab_ce_workspace_bytes", "mp_vocab_ce", "mp_vocab_ce_partials",
           "mp_vocab_ce_combine", "mp_status_string", "mp_status_from_device", "mp_version",
           "mp_vocab_ce_noalloc", "mp_vocab_ce_bwd_workspace_bytes", "mp_vocab_ce_bwd_workspace_bytes_one_pass",
           "mp_vocab_ce_bwd", "mp_vocab_ce_lse", "mp_vocab_ce_bwd_lse", "mp_vocab_embed",
           "mp_attn_fwd", "mp_glu_fwd", "mp_glu_bwd", "mp_rope_axes",
           "mp_attn_varlen_fwd", "mp_attn_varlen_bwd", "mp_qk_norm_rope", "mp_qk_norm_rope_bwd_workspace_bytes",
           "mp_qk_norm_rope_bwd", "mp_kv_cache_write", "mp_kv_cache_read", "mp_attn_cache_workspace_bytes",
           "mp_attn_cache_fwd")


class MptpError(RuntimeError):
    def __init__(self, fn: str, code: int):
        self.code = int(code)
        super().__init__(f"{fn}: {status_string(code)}")


_lib = None
_P = ctypes.c_void_p
_I = ctypes.c_int
_L = ctypes.c_longlong


def lib() -> ctypes.CDLL:
    """Load (once) and return the C library. Raises OSError if it is not built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise OSError(f"libmptp.so is not built ({LIB_PATH}); run "
                          "`python -m tensor_transformer_layer_gb300.build`")
        L = ctypes.CDLL(LIB_PATH)
        L.mp_mlp_fwd.argtypes = [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P, _P]
        L.mp_mlp_fwd.restype = _I
        L.mp_mlp_bwd.argtypes = [_P] * 10 + [_I, _I, _I, _I, _P, _P]
        L.mp_mlp_bwd.restype = _I
        L.mp_mlp_fwd_shards.argtypes = [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P]
        L.mp_mlp_fwd_shards.restype = _I
        L.mp_mlp_bwd_shards.argtypes = [_P] * 10 + [_I, _I, _I, _I, _I, _I, _P, _P]
        L.mp_mlp_bwd_shards.restype = _I
        L.mp_mlp_fused_workspace_bytes.argtypes = [_I, _I, _I, _I]
        L.mp_mlp_fused_workspace_bytes.restype = ctypes.c_size_t
        L.mp_mlp_fwd_fused.argtypes = [_P] * 6 + [_I] * 6 + [_P, ctypes.c_size_t, _P, _P]
        L.mp_mlp_fwd_fused.restype = _I
        L.mp_mlp_bwd_fused.argtypes = [_P] * 10 + [_I] * 6 + [_P, ctypes.c_size_t, _P, _P]
        L.mp_mlp_bwd_fused.restype = _I
        L.mp_vocab_ce_workspace_bytes.argtypes = [_I, _I, _I]
        L.mp_vocab_ce_workspace_bytes.restype = ctypes.c_size_t
        L.mp_vocab_ce.argtypes = [_P, _P, _P, _P, _P, ctypes.c_size_t, _I, _I, _I, _I, _I, _P, _P]
        L.mp_vocab_ce.restype = _I
        L.mp_vocab_ce_partials.argtypes = [_P, _P, _P, _P, ctypes.c_size_t, _I, _I, _I, _I, _I, _P, _P]
        L.mp_vocab_ce_partials.restype = _I
        L.mp_vocab_ce_combine.argtypes = [_P, ctypes.c_size_t, _P, _P, _I, _I, _I, _I, _P, _P]
        L.mp_vocab_ce_combine.restype = _I
        L.mp_vocab_ce_bwd_workspace_bytes.argtypes = [_I, _I, _I, _I]
        L.mp_vocab_ce_bwd_workspace_bytes.restype = ctypes.c_size_t
        L.mp_vocab_ce_bwd_workspace_bytes_one_pass.argtypes = [_I, _I, _I, _I]
        L.mp_vocab_ce_bwd_workspace_bytes_one_pass.restype = ctypes.c_size_t
        L.mp_vocab_ce_bwd.argtypes = [_P] * 7 + [_P, ctypes.c_size_t, _I, _I, _I, _I, _I, _P, _P]
        L.mp_vocab_ce_bwd.restype = _I
        L.mp_vocab_ce_lse.argtypes = [_P, _P, _P, _P, _P, _P, ctypes.c_size_t, _I, _I, _I, _I, _I, _P, _P]
        L.mp_vocab_ce_lse.restype = _I
        L.mp_vocab_ce_bwd_lse.argtypes = [_P] * 7 + [_P, ctypes.c_size_t, _I, _I, _I, _I, _I, _P, _P]
        L.mp_vocab_ce_bwd_lse.restype = _I
        L.mp_attn_fwd.argtypes = [_P] * 6 + [_I, _I, _I, _I, _I, _P, _P]
        L.mp_attn_fwd.restype = _I
        L.mp_glu_fwd.argtypes = [_P] * 6 + [_I] * 5 + [_P, _P]
        L.mp_glu_fwd.restype = _I
        L.mp_glu_bwd.argtypes = [_P] * 10 + [_I] * 5 + [_P, _P]
        L.mp_glu_bwd.restype = _I
        L.mp_rope_axes.argtypes = [_P, _P, _P, _I, _I, _I, _L, _L, _I, _P, ctypes.c_double, ctypes.c_uint32, _P]
        L.mp_rope_axes.restype = _I
        _F = ctypes.c_float
        L.mp_attn_varlen_fwd.argtypes = [_P] * 7 + [_I] * 8 + [_L] * 4 + [_I, _F, _P, _P]
        L.mp_attn_varlen_fwd.restype = _I
        L.mp_attn_varlen_bwd.argtypes = [_P] * 12 + [_I] * 8 + [_L] * 8 + [_I, _F, _P, _P]
        L.mp_attn_varlen_bwd.restype = _I
        L.mp_qk_norm_rope.argtypes = [_P] * 5 + [_I] * 4 + [_L] * 2 + [_I, _P, ctypes.c_double, _F, ctypes.c_uint32, _P]
        L.mp_qk_norm_rope.restype = _I
        L.mp_qk_norm_rope_bwd_workspace_bytes.argtypes = [_I] * 3
        L.mp_qk_norm_rope_bwd_workspace_bytes.restype = ctypes.c_size_t
        L.mp_qk_norm_rope_bwd.argtypes = ([_P] * 9 + [ctypes.c_size_t] + [_I] * 4 + [_L] * 3 +
                                          [_I, _P, ctypes.c_double, _F, ctypes.c_uint32, _P])
        L.mp_qk_norm_rope_bwd.restype = _I
        L.mp_kv_cache_write.argtypes = [_P] * 9 + [_I] * 8 + [_L] * 6 + [_P, _P]
        L.mp_kv_cache_write.restype = _I
        L.mp_kv_cache_read.argtypes = [_P] * 9 + [_I] * 8 + [_L] * 6 + [_P, _P]
        L.mp_kv_cache_read.restype = _I
        L.mp_attn_cache_workspace_bytes.argtypes = [_I] * 4
        L.mp_attn_cache_workspace_bytes.restype = ctypes.c_size_t
        L.mp_attn_cache_fwd.argtypes = [_P] * 11 + [ctypes.c_size_t] + [_I] * 9 + [_L] * 6 + [_I, _F, _P, _P]
        L.mp_attn_cache_fwd.restype = _I
        L.mp_vocab_embed.argtypes = [_P, _P, _P, _I, _I, _I, _I, _I, _P, _P]
        L.mp_vocab_embed.restype = _I
        L.mp_vocab_ce_noalloc.argtypes = [_P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P]
        L.mp_vocab_ce_noalloc.restype = _I
        L.mp_status_string.argtypes = [_I]
        L.mp_status_string.restype = ctypes.c_char_p
        L.mp_status_from_device.argtypes = [ctypes.c_uint32]
        L.mp_status_from_device.restype = _I
        L.mp_version.argtypes = []
        L.mp_version.restype = _I
        _lib = L
    return _lib


_bind = None


def _fast():
    """The extension that marshals a decoding step's calls; its functions return None for what they leave to the checks here."""
    global _bind
    if _bind is None:
        lib()
        if not os.path.exists(BIND_PATH):
            raise OSError(f"_mptp_bind.so is not built ({BIND_PATH}); run `python -m tensor_transformer_layer_gb300.build`")
        from . import build
        if build.bind_built_for() != build.bind_for():  # it holds the layout of another torch's classes
            raise OSError(f"_mptp_bind.so was built for {build.bind_built_for()}, installed is {build.bind_for()}; run "
                          "`python -m tensor_transformer_layer_gb300.build`")
        spec = importlib.util.spec_from_file_location("_mptp_bind", BIND_PATH)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        _bind = module
    return _bind


def _current_device():
    return torch._C._cuda_getDevice()


def _here(**tensors):
    """Refuses tensors of another GPU than the current one, where a kernel would take their addresses for its own."""
    for name, t in tensors.items():
        if isinstance(t, torch.Tensor) and t.is_cuda and t.get_device() != _current_device():
            raise ValueError(f"{name} lies on cuda:{t.get_device()}, the current device is cuda:{_current_device()}")


def _handle(stream):
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else stream


def status_string(code: int) -> str:
    try:
        return lib().mp_status_string(int(code)).decode()
    except OSError:
        return STATUS_NAMES.get(int(code), f"status {code}")


def _ptr(x, name, dtype=torch.bfloat16, shape=None, allow_none=False):
    # What a right call passes, in as few steps as it takes; everything else is told apart below.
    if type(x) is torch.Tensor and x.dtype is dtype and (shape is None or x.shape == shape) and x.is_cuda and \
            x.is_contiguous():
        return x.data_ptr() or None
    if x is None:
        if allow_none:
            return None
        raise ValueError(f"{name} is required")
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if x.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {x.dtype}")
    if shape is not None and tuple(x.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(x.shape)}")
    if not x.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if x.numel() > 0 and not x.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return x.data_ptr() or None


def _stream(stream):
    if stream is None:
        # torch.cuda.current_stream().cuda_stream, without building the Stream object (0.2 against 2.9 us)
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _status_ptr(d_status):
    if d_status is None:
        return None
    return _ptr(d_status, "d_status", dtype=torch.int32, shape=(1,))


def _check(fn, code):
    if code != MP_OK:
        raise MptpError(fn, code)


def mp_mlp_fwd(X, A, B, Z, Y, U_save=None, *, t: int, d_status=None, stream=None) -> None:
    """Forward of the sharded MLP: Y = GeLU(X A) (U_save = X A), Z = sum_i Y_i B_i."""
    T, h = X.shape
    f = A.shape[1]
    code = lib().mp_mlp_fwd(
        _ptr(X, "X", shape=(T, h)), _ptr(A, "A", shape=(h, f)), _ptr(B, "B", shape=(f, h)),
        _ptr(Z, "Z", shape=(T, h)), _ptr(Y, "Y", shape=(T, f)),
        _ptr(U_save, "U_save", shape=(T, f), allow_none=True),
        T, h, f, int(t), _status_ptr(d_status), _stream(stream))
    _check("mp_mlp_fwd", code)


def mp_mlp_bwd(X, A, B, U, Y, dZ, dX, dA, dB, dU_ws, *, t: int, d_status=None, stream=None) -> None:
    """Backward of the sharded MLP: dX (shard sum fused), dA, dB; dU_ws holds dU."""
    T, h = X.shape
    f = A.shape[1]
    code = lib().mp_mlp_bwd(
        _ptr(X, "X", shape=(T, h)), _ptr(A, "A", shape=(h, f)), _ptr(B, "B", shape=(f, h)),
        _ptr(U, "U", shape=(T, f)), _ptr(Y, "Y", shape=(T, f)), _ptr(dZ, "dZ", shape=(T, h)),
        _ptr(dX, "dX", shape=(T, h)), _ptr(dA, "dA", shape=(h, f)), _ptr(dB, "dB", shape=(f, h)),
        _ptr(dU_ws, "dU_ws", shape=(T, f)), T, h, f, int(t), _status_ptr(d_status), _stream(stream))
    _check("mp_mlp_bwd", code)


def mp_mlp_fwd_shards(X, A, B, Z, Y, U_save=None, *, t: int, shard_begin: int, shard_count: int, d_status=None,
                      stream=None) -> None:
    """Forward of shards [shard_begin, shard_begin + shard_count): their columns of Y (and
    U_save) and their partial output Z = sum over the range of Y_i B_i."""
    T, h = X.shape
    f = A.shape[1]
    code = lib().mp_mlp_fwd_shards(
        _ptr(X, "X", shape=(T, h)), _ptr(A, "A", shape=(h, f)), _ptr(B, "B", shape=(f, h)),
        _ptr(Z, "Z", shape=(T, h)), _ptr(Y, "Y", shape=(T, f)),
        _ptr(U_save, "U_save", shape=(T, f), allow_none=True),
        T, h, f, int(t), int(shard_begin), int(shard_count), _status_ptr(d_status), _stream(stream))
    _check("mp_mlp_fwd_shards", code)


def mp_mlp_bwd_shards(X, A, B, U, Y, dZ, dX, dA, dB, dU_ws, *, t: int, shard_begin: int, shard_count: int,
                      d_status=None, stream=None) -> None:
    """Backward of shards [shard_begin, shard_begin + shard_count): their part of dX, their
    columns of dA and dU_ws, their rows of dB."""
    T, h = X.shape
    f = A.shape[1]
    code = lib().mp_mlp_bwd_shards(
        _ptr(X, "X", shape=(T, h)), _ptr(A, "A", shape=(h, f)), _ptr(B, "B", shape=(f, h)),
        _ptr(U, "U", shape=(T, f)), _ptr(Y, "Y", shape=(T, f)), _ptr(dZ, "dZ", shape=(T, h)),
        _ptr(dX, "dX", shape=(T, h)), _ptr(dA, "dA", shape=(h, f)), _ptr(dB, "dB", shape=(f, h)),
        _ptr(dU_ws, "dU_ws", shape=(T, f)), T, h, f, int(t), int(shard_begin), int(shard_count),
        _status_ptr(d_status), _stream(stream))
    _check("mp_mlp_bwd_shards", code)


def mp_mlp_fused_workspace_bytes(T: int, h: int, f: int, t: int) -> int:
    return int(lib().mp_mlp_fused_workspace_bytes(int(T), int(h), int(f), int(t)))


def mp_mlp_fused_workspace(T: int, h: int, f: int, t: int, device="cuda") -> torch.Tensor:
    """A zero-filled workspace for mp_mlp_fwd_fused / mp_mlp_bwd_fused (every call leaves it zero)."""
    return torch.zeros(mp_mlp_fused_workspace_bytes(T, h, f, t), dtype=torch.uint8, device=device)


def mp_mlp_fwd_fused(X, A, B, Z, Y, U_save=None, *, t: int, workspace, shard_begin: int = 0,
                     shard_count: int | None = None, d_status=None, stream=None) -> None:
    """mp_mlp_fwd_shards in one launch (both GEMMs of the forward); equal outputs bit for bit."""
    T, h = X.shape
    f = A.shape[1]
    n = int(t) - int(shard_begin) if shard_count is None else int(shard_count)
    wp, wb = _ws(workspace)
    code = lib().mp_mlp_fwd_fused(
        _ptr(X, "X", shape=(T, h)), _ptr(A, "A", shape=(h, f)), _ptr(B, "B", shape=(f, h)),
        _ptr(Z, "Z", shape=(T, h)), _ptr(Y, "Y", shape=(T, f)),
        _ptr(U_save, "U_save", shape=(T, f), allow_none=True),
        T, h, f, int(t), int(shard_begin), n, wp, wb, _status_ptr(d_status), _stream(stream))
    _check("mp_mlp_fwd_fused", code)


def mp_mlp_bwd_fused(X, A, B, U, Y, dZ, dX, dA, dB, dU_ws, *, t: int, workspace, shard_begin: int = 0,
                     shard_count: int | None = None, d_status=None, stream=None) -> None:
    """mp_mlp_bwd_shards in one launch (dU, dX, dA, dB); equal outputs bit for bit."""
    T, h = X.shape
    f = A.shape[1]
    n = int(t) - int(shard_begin) if shard_count is None else int(shard_count)
    wp, wb = _ws(workspace)
    code = lib().mp_mlp_bwd_fused(
        _ptr(X, "X", shape=(T, h)), _ptr(A, "A", shape=(h, f)), _ptr(B, "B", shape=(f, h)),
        _ptr(U, "U", shape=(T, f)), _ptr(Y, "Y", shape=(T, f)), _ptr(dZ, "dZ", shape=(T, h)),
        _ptr(dX, "dX", shape=(T, h)), _ptr(dA, "dA", shape=(h, f)), _ptr(dB, "dB", shape=(f, h)),
        _ptr(dU_ws, "dU_ws", shape=(T, f)), T, h, f, int(t), int(shard_begin), n, wp, wb,
        _status_ptr(d_status), _stream(stream))
    _check("mp_mlp_bwd_fused", code)


def mp_vocab_ce_workspace_bytes(T: int, v_pad: int, t: int) -> int:
    return int(lib().mp_vocab_ce_workspace_bytes(int(T), int(v_pad), int(t)))


def _ws(workspace):
    if not isinstance(workspace, torch.Tensor) or not workspace.is_contiguous():
        raise TypeError("workspace must be a contiguous torch.Tensor")
    return workspace.data_ptr() or None, workspace.numel() * workspace.element_size()


def _cuda_ws(workspace):
    if type(workspace) is torch.Tensor and workspace.is_cuda and workspace.is_contiguous():
        return workspace.data_ptr() or None, workspace.nbytes
    if isinstance(workspace, torch.Tensor) and workspace.numel() > 0 and not workspace.is_cuda:
        raise ValueError("workspace must be a CUDA tensor")
    return _ws(workspace)


def mp_vocab_ce(X, E, target, loss, workspace, *, v_valid: int, t: int, d_status=None, stream=None) -> None:
    """Fused vocab-parallel logits + cross-entropy: loss[T] fp32."""
    T, h = X.shape
    v_pad = E.shape[0]
    wp, wb = _ws(workspace)
    code = lib().mp_vocab_ce(
        _ptr(X, "X", shape=(T, h)), _ptr(E, "E", shape=(v_pad, h)),
        _ptr(target, "target", dtype=torch.int32, shape=(T,)), _ptr(loss, "loss", dtype=torch.float32, shape=(T,)),
        wp, wb, T, h, v_pad, int(v_valid), int(t), _status_ptr(d_status), _stream(stream))
    _check("mp_vocab_ce", code)


def mp_vocab_ce_lse(X, E, target, loss, lse, workspace, *, v_valid: int, t: int, d_status=None, stream=None) -> None:
    """mp_vocab_ce that also writes the per-token log-sum-exp lse[T] fp32 (NaN for invalid targets)."""
    T, h = X.shape
    v_pad = E.shape[0]
    wp, wb = _ws(workspace)
    code = lib().mp_vocab_ce_lse(
        _ptr(X, "X", shape=(T, h)), _ptr(E, "E", shape=(v_pad, h)),
        _ptr(target, "target", dtype=torch.int32, shape=(T,)), _ptr(loss, "loss", dtype=torch.float32, shape=(T,)),
        _ptr(lse, "lse", dtype=torch.float32, shape=(T,)), wp, wb, T, h, v_pad, int(v_valid), int(t),
        _status_ptr(d_status), _stream(stream))
    _check("mp_vocab_ce_lse", code)


def mp_vocab_ce_partials(X, E, target, workspace, *, v_valid: int, t: int, d_status=None, stream=None) -> None:
    T, h = X.shape
    v_pad = E.shape[0]
    wp, wb = _ws(workspace)
    code = lib().mp_vocab_ce_partials(
        _ptr(X, "X", shape=(T, h)), _ptr(E, "E", shape=(v_pad, h)),
        _ptr(target, "target", dtype=torch.int32, shape=(T,)), wp, wb, T, h, v_pad, int(v_valid), int(t),
        _status_ptr(d_status), _stream(stream))
    _check("mp_vocab_ce_partials", code)


def mp_vocab_ce_combine(workspace, target, loss, *, v_pad: int, v_valid: int, t: int, d_status=None,
                        stream=None) -> None:
    T = target.shape[0]
    wp, wb = _ws(workspace)
    code = lib().mp_vocab_ce_combine(
        wp, wb, _ptr(target, "target", dtype=torch.int32, shape=(T,)),
        _ptr(loss, "loss", dtype=torch.float32, shape=(T,)), T, int(v_pad), int(v_valid), int(t),
        _status_ptr(d_status), _stream(stream))
    _check("mp_vocab_ce_combine", code)


def mp_vocab_ce_noalloc(X, E, target, loss, *, v_valid: int, t: int, d_status=None, stream=None) -> None:
    """mp_vocab_ce without a workspace argument, for callers that cannot allocate
    device memory: the library's fixed 4 MiB static device array holds the
    triples. Calls that overlap on the GPU race on that array."""
    T, h = X.shape
    v_pad = E.shape[0]
    code = lib().mp_vocab_ce_noalloc(
        _ptr(X, "X", shape=(T, h)), _ptr(E, "E", shape=(v_pad, h)),
        _ptr(target, "target", dtype=torch.int32, shape=(T,)), _ptr(loss, "loss", dtype=torch.float32, shape=(T,)),
        T, h, v_pad, int(v_valid), int(t), _status_ptr(d_status), _stream(stream))
    _check("mp_vocab_ce_noalloc", code)


def mp_vocab_ce_bwd_workspace_bytes(T: int, h: int, v_pad: int, t: int) -> int:
    return int(lib().mp_vocab_ce_bwd_workspace_bytes(int(T), int(h), int(v_pad), int(t)))


def mp_vocab_ce_bwd_workspace_bytes_one_pass(T: int, h: int, v_pad: int, t: int) -> int:
    return int(lib().mp_vocab_ce_bwd_workspace_bytes_one_pass(int(T), int(h), int(v_pad), int(t)))


def mp_vocab_ce_bwd(X, E, target, loss, dloss, dX, dE, workspace, *, v_valid: int, t: int, d_status=None,
                    stream=None) -> None:
    """Backward of the fused vocab-parallel cross-entropy: dX [T,h], dE [v_pad,h] (bf16)."""
    T, h = X.shape
    v_pad = E.shape[0]
    wp, wb = _ws(workspace)
    code = lib().mp_vocab_ce_bwd(
        _ptr(X, "X", shape=(T, h)), _ptr(E, "E", shape=(v_pad, h)),
        _ptr(target, "target", dtype=torch.int32, shape=(T,)), _ptr(loss, "loss", dtype=torch.float32, shape=(T,)),
        _ptr(dloss, "dloss", dtype=torch.float32, shape=(T,)), _ptr(dX, "dX", shape=(T, h)),
        _ptr(dE, "dE", shape=(v_pad, h)), wp, wb, T, h, v_pad, int(v_valid), int(t), _status_ptr(d_status),
        _stream(stream))
    _check("mp_vocab_ce_bwd", code)


def mp_vocab_ce_bwd_lse(X, E, target, lse, dloss, dX, dE, workspace, *, v_valid: int, t: int, d_status=None,
                        stream=None) -> None:
    """Backward of the fused cross-entropy from the forward's exported log-sum-exp."""
    T, h = X.shape
    v_pad = E.shape[0]
    wp, wb = _ws(workspace)
    code = lib().mp_vocab_ce_bwd_lse(
        _ptr(X, "X", shape=(T, h)), _ptr(E, "E", shape=(v_pad, h)),
        _ptr(target, "target", dtype=torch.int32, shape=(T,)), _ptr(lse, "lse", dtype=torch.float32, shape=(T,)),
        _ptr(dloss, "dloss", dtype=torch.float32, shape=(T,)), _ptr(dX, "dX", shape=(T, h)),
        _ptr(dE, "dE", shape=(v_pad, h)), wp, wb, T, h, v_pad, int(v_valid), int(t), _status_ptr(d_status),
        _stream(stream))
    _check("mp_vocab_ce_bwd_lse", code)


def mp_vocab_embed(ids, E, out, *, v_valid: int, t: int, d_status=None, stream=None) -> None:
    """Vocab-parallel embedding lookup: out[r] = E[ids[r]] (zeros for ids outside [0, v_valid))."""
    T = ids.shape[0]
    v_pad, h = E.shape
    code = lib().mp_vocab_embed(
        _ptr(ids, "ids", dtype=torch.int32, shape=(T,)), _ptr(E, "E", shape=(v_pad, h)),
        _ptr(out, "out", shape=(T, h)), T, h, v_pad, int(v_valid), int(t), _status_ptr(d_status), _stream(stream))
    _check("mp_vocab_embed", code)


def mp_attn_fwd(X, Wqkv, Wo, out, QKV, O, *, b: int, s: int, heads: int, t: int, d_status=None,
                stream=None) -> None:
    """Head-parallel causal self-attention block: QKV = X Wqkv, per-head attention O, out = O Wo."""
    T, h = X.shape
    if T != b * s:
        raise ValueError("X must have b * s rows")
    code = lib().mp_attn_fwd(
        _ptr(X, "X", shape=(T, h)), _ptr(Wqkv, "Wqkv", shape=(h, 3 * h)), _ptr(Wo, "Wo", shape=(h, h)),
        _ptr(out, "out", shape=(T, h)), _ptr(QKV, "QKV", shape=(T, 3 * h)), _ptr(O, "O", shape=(T, h)),
        int(b), int(s), h, int(heads), int(t), _status_ptr(d_status), _stream(stream))
    _check("mp_attn_fwd", code)


def _i32(x, name):
    """x as an int that a C int holds: ctypes would keep the low 32 bits of a larger one."""
    x = int(x)
    if not -0x80000000 <= x <= 0x7fffffff:
        raise ValueError(f"{name} must fit in 32 bits, got {x}")
    return x


ACTS = {"silu": 0, "gelu": 1}


def _act(act):
    if act not in ACTS:
        raise ValueError(f"act must be one of {sorted(ACTS)}, got {act!r}")
    return ACTS[act]


def mp_glu_fwd(X, W, Wd, Z, Y, GU_save=None, *, t: int, act: str = "silu", d_status=None, stream=None) -> None:
    """Gated feed-forward block: [G | U] = X W, Y = act(G) * U, Z = Y Wd; W [h, 2f], act "silu" or "gelu"."""
    t = _i32(t, "t")
    T, h = X.shape
    f = Wd.shape[0]
    code = lib().mp_glu_fwd(
        _ptr(X, "X", shape=(T, h)), _ptr(W, "W", shape=(h, 2 * f)), _ptr(Wd, "Wd", shape=(f, h)),
        _ptr(Z, "Z", shape=(T, h)), _ptr(Y, "Y", shape=(T, f)),
        _ptr(GU_save, "GU_save", shape=(T, 2 * f), allow_none=True), T, h, f, t, _act(act),
        _status_ptr(d_status), _stream(stream))
    _check("mp_glu_fwd", code)


def mp_glu_bwd(X, W, Wd, GU, Y, dZ, dX, dW, dWd, dGU_ws, *, t: int, act: str = "silu", d_status=None,
               stream=None) -> None:
    """Backward of mp_glu_fwd from its GU_save and Y: dX [T,h], dW [h,2f], dWd [f,h]; dGU_ws [T,2f] workspace."""
    t = _i32(t, "t")
    T, h = X.shape
    f = Wd.shape[0]
    code = lib().mp_glu_bwd(
        _ptr(X, "X", shape=(T, h)), _ptr(W, "W", shape=(h, 2 * f)), _ptr(Wd, "Wd", shape=(f, h)),
        _ptr(GU, "GU", shape=(T, 2 * f)), _ptr(Y, "Y", shape=(T, f)), _ptr(dZ, "dZ", shape=(T, h)),
        _ptr(dX, "dX", shape=(T, h)), _ptr(dW, "dW", shape=(h, 2 * f)), _ptr(dWd, "dWd", shape=(f, h)),
        _ptr(dGU_ws, "dGU_ws", shape=(T, 2 * f)), T, h, f, t, _act(act), _status_ptr(d_status), _stream(stream))
    _check("mp_glu_bwd", code)


def _heads_view(x, name, shape=None):
    """Pointer and row pitch of a bf16 [tokens, heads, d] tensor whose heads are packed in each row (a view of
    some heads of a wider row is fine)."""
    # What a right call passes, in as few steps as it takes; everything else is told apart below.
    if type(x) is torch.Tensor and x.dtype is torch.bfloat16 and x.shape == shape and x.is_cuda:
        T, heads, d = shape
        pitch, step, unit = x.stride()
        if unit == 1 and step == d and T > 1 and pitch >= heads * d > 0:
            return x.data_ptr(), pitch
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if x.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be {torch.bfloat16}, got {x.dtype}")
    size = x.shape
    if len(size) != 3 or (shape is not None and size != shape):
        want = "[tokens, heads, d]" if shape is None else tuple(shape)
        raise ValueError(f"{name} must have shape {want}, got {tuple(size)}")
    T, heads, d = size
    row = heads * d
    if T == 0 or row == 0:
        return None, row
    pitch, step, unit = x.stride()
    if (d > 1 and unit != 1) or (heads > 1 and step != d):
        raise ValueError(f"{name}: each token's heads must be contiguous (strides (any, d, 1))")
    if not x.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if T == 1:
        pitch = row
    elif pitch < row:
        raise ValueError(f"{name}: rows overlap (pitch {pitch} < {row})")
    return x.data_ptr(), pitch


@functools.lru_cache(maxsize=64)
def _int_array(values):
    """Length and C array of a tuple of ints (read only)."""
    return len(values), (_I * max(len(values), 1))(*(_i32(v, "sections") for v in values))


def mp_rope_axes(x, y, pos, *, sections, base: float = 10000.0, interleaved: bool = False, per_axis: bool = False,
                 inverse: bool = False, stream=None) -> None:
    """Rotary positions with up to four axes: y = x with each head's pairs rotated by pos[axis] * frequency.
    x, y [T, heads, d] (rows may be strided; y may be x), pos [axes, T] int32, sections: pairs of each axis.
    inverse rotates back (the gradient)."""
    size = tuple(x.shape)
    px, ldx = _heads_view(x, "x", size if len(size) == 3 else None)
    py, ldy = _heads_view(y, "y", size)
    T, heads, d = size
    axes, sec = _int_array(tuple(sections))
    flags = (1 if interleaved else 0) | (2 if per_axis else 0) | (4 if inverse else 0)
    code = lib().mp_rope_axes(px, py, _ptr(pos, "pos", torch.int32, (axes, T)), T, heads, d, ldx, ldy, axes, sec,
                              float(base), flags, _stream(stream))
    _check("mp_rope_axes", code)


def _packed_shapes(Q, K, cu_q, cu_k):
    if not isinstance(Q, torch.Tensor) or not isinstance(K, torch.Tensor):
        raise ValueError("Q and K must be [tokens, heads, d] tensors")
    qs, ks = tuple(Q.shape), tuple(K.shape)
    if len(qs) != 3 or len(ks) != 3:
        raise ValueError("Q and K must be [tokens, heads, d] tensors")
    if qs[2] != ks[2]:
        raise ValueError(f"Q and K must have the same head width, got {qs[2]} and {ks[2]}")
    nseq = cu_q.shape[0] - 1
    if nseq < 0:
        raise ValueError("cu_q must have at least one entry")
    return (nseq, qs, ks, _ptr(cu_q, "cu_q", torch.int32, (nseq + 1,)), _ptr(cu_k, "cu_k", torch.int32, (nseq + 1,)))


def mp_attn_varlen_fwd(Q, K, V, O, LSE, cu_q, cu_k, *, max_q: int, max_k: int, causal: bool, scale: float | None = None,
                       d_status=None, stream=None) -> None:
    """Attention over packed sequences: O [Tq, heads, d] and LSE [heads, Tq] fp32 from Q [Tq, heads, d], K, V
    [Tk, kv_heads, d] (rows may be strided). cu_q, cu_k [nseq + 1] int32: sequence i owns rows cu[i] .. cu[i+1]-1;
    max_q, max_k: at least the longest. causal: the last query sees the last key. scale: 1 / sqrt(d) by default."""
    max_q, max_k = _i32(max_q, "max_q"), _i32(max_k, "max_k")
    nseq, qs, ks, pcq, pck = _packed_shapes(Q, K, cu_q, cu_k)
    (Tq, heads, d), (Tk, kv, _) = qs, ks
    (pq, ldq), (pk, ldk) = _heads_view(Q, "Q", qs), _heads_view(K, "K", ks)
    (pv, ldv), (po, ldo) = _heads_view(V, "V", ks), _heads_view(O, "O", qs)
    code = lib().mp_attn_varlen_fwd(
        pq, pk, pv, po, _ptr(LSE, "LSE", torch.float32, (heads, Tq)), pcq, pck, nseq, Tq, Tk, max_q,
        max_k, heads, kv, d, ldq, ldk, ldv, ldo, 1 if causal else 0, d ** -0.5 if scale is None else float(scale),
        _status_ptr(d_status), _stream(stream))
    _check("mp_attn_varlen_fwd", code)


def mp_attn_varlen_bwd(Q, K, V, O, LSE, dO, dQ, dK, dV, delta_ws, cu_q, cu_k, *, max_q: int, max_k: int, causal: bool,
                       scale: float | None = None, d_status=None, stream=None) -> None:
    """Backward of mp_attn_varlen_fwd from its O and LSE: dQ, dK, dV (rows may be strided, e.g. the parts of a
    packed projection's gradient); delta_ws [heads, Tq] fp32 workspace."""
    max_q, max_k = _i32(max_q, "max_q"), _i32(max_k, "max_k")
    nseq, qs, ks, pcq, pck = _packed_shapes(Q, K, cu_q, cu_k)
    (Tq, heads, d), (Tk, kv, _) = qs, ks
    (pq, ldq), (pk, ldk), (pv, ldv) = _heads_view(Q, "Q", qs), _heads_view(K, "K", ks), _heads_view(V, "V", ks)
    (po, ldo), (pdo, lddo) = _heads_view(O, "O", qs), _heads_view(dO, "dO", qs)
    (pdq, lddq), (pdk, lddk), (pdv, lddv) = (_heads_view(dQ, "dQ", qs), _heads_view(dK, "dK", ks),
                                             _heads_view(dV, "dV", ks))
    f32 = torch.float32, (heads, Tq)
    code = lib().mp_attn_varlen_bwd(
        pq, pk, pv, po, _ptr(LSE, "LSE", *f32), pdo, pdq, pdk, pdv, _ptr(delta_ws, "delta_ws", *f32), pcq, pck, nseq,
        Tq, Tk, max_q, max_k, heads, kv, d, ldq, ldk, ldv, ldo, lddo, lddq, lddk, lddv, 1 if causal else 0,
        d ** -0.5 if scale is None else float(scale), _status_ptr(d_status), _stream(stream))
    _check("mp_attn_varlen_bwd", code)


def _weight(w, name, d, needed):
    return _ptr(w, name, shape=(d,), allow_none=not needed)


def _norm_heads(x, q_heads):
    if not isinstance(x, torch.Tensor) or x.dim() != 3:
        raise ValueError("x must be a [tokens, heads, d] tensor")
    return tuple(x.shape), _i32(q_heads, "q_heads")


def mp_qk_norm_rope(x, y, wq, wk, pos, *, q_heads: int, sections, base: float = 10000.0, eps: float = 1e-6,
                    interleaved: bool = False, per_axis: bool = False, stream=None) -> None:
    """Norm of each query and key head with the rotation of mp_rope_axes in one pass: y = R(w x / sqrt(mean(x^2) + eps)),
    w = wq for the first q_heads heads, wk for the others. x, y [T, heads, d] (rows may be strided; y may be x), wq, wk [d],
    pos [axes, T] int32."""
    flags = (1 if interleaved else 0) | (2 if per_axis else 0)
    code = (_bind or _fast()).qk_norm_rope(x, y, wq, wk, pos, q_heads, sections, base, eps, flags, _handle(stream))
    if code is not None:
        return _check("mp_qk_norm_rope", code)
    _here(x=x, y=y, wq=wq, wk=wk, pos=pos)
    size, nq = _norm_heads(x, q_heads)
    T, heads, d = size
    (px, ldx), (py, ldy) = _heads_view(x, "x", size), _heads_view(y, "y", size)
    axes, sec = _int_array(tuple(sections))
    code = lib().mp_qk_norm_rope(px, py, _weight(wq, "wq", d, nq > 0), _weight(wk, "wk", d, nq < heads),
                                 _ptr(pos, "pos", torch.int32, (axes, T)), T, heads, nq, d, ldx, ldy, axes, sec,
                                 float(base), float(eps), flags, _stream(stream))
    _check("mp_qk_norm_rope", code)


def mp_qk_norm_rope_bwd_workspace_bytes(T: int, heads: int, d: int) -> int:
    return int(lib().mp_qk_norm_rope_bwd_workspace_bytes(_i32(T, "T"), _i32(heads, "heads"), _i32(d, "d")))


def mp_qk_norm_rope_bwd(x, dy, dx, wq, wk, dwq, dwk, pos, workspace, *, q_heads: int, sections, base: float = 10000.0,
                        eps: float = 1e-6, interleaved: bool = False, per_axis: bool = False, stream=None) -> None:
    """Backward of mp_qk_norm_rope from its x: dx [T, heads, d] (rows may be strided; may be dy or x), dwq, dwk [d] fp32;
    workspace: mp_qk_norm_rope_bwd_workspace_bytes(T, heads, d) bytes."""
    flags = (1 if interleaved else 0) | (2 if per_axis else 0)
    code = (_bind or _fast()).qk_norm_rope_bwd(x, dy, dx, wq, wk, dwq, dwk, pos, workspace, q_heads, sections, base, eps,
                                               flags, _handle(stream))
    if code is not None:
        return _check("mp_qk_norm_rope_bwd", code)
    _here(x=x, dy=dy, dx=dx, wq=wq, wk=wk, dwq=dwq, dwk=dwk, pos=pos, workspace=workspace)
    size, nq = _norm_heads(x, q_heads)
    T, heads, d = size
    (px, ldx), (pg, ldg), (pd, ldd) = (_heads_view(x, "x", size), _heads_view(dy, "dy", size),
                                       _heads_view(dx, "dx", size))
    axes, sec = _int_array(tuple(sections))
    wp, wb = _cuda_ws(workspace)
    code = lib().mp_qk_norm_rope_bwd(
        px, pg, pd, _weight(wq, "wq", d, nq > 0), _weight(wk, "wk", d, nq < heads),
        _ptr(dwq, "dwq", torch.float32, (d,), nq == 0), _ptr(dwk, "dwk", torch.float32, (d,), nq == heads),
        _ptr(pos, "pos", torch.int32, (axes, T)), wp, wb, T, heads, nq, d, ldx, ldg, ldd, axes, sec, float(base),
        float(eps), flags, _stream(stream))
    _check("mp_qk_norm_rope_bwd", code)


def _page_view(t, name, dtype, size, inner):
    """Pointer and page pitch of a tensor [pages, ...] of this size whose pages are contiguous (strides `inner`)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != size:
        raise ValueError(f"{name} must have shape {tuple(size)}, got {tuple(t.shape)}")
    if size[0] > 0 and not t[0].is_contiguous():
        raise ValueError(f"{name}: what a page holds must be contiguous")
    if t.numel() > 0 and not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.data_ptr() or None, t.stride(0) if size[0] > 1 else size[1] * inner[0]


_F8, _F32 = torch.float8_e4m3fn, torch.float32


def _pool(kc, vc, ks, vs, page_table, nseq):
    """Pointers and pitches of a cache's pool (codes [pages, kv_heads, page, d] e4m3, scales [pages, kv_heads] fp32), the
    pointer of its table [nseq, max_pages] int32, and (pages, max_pages, page, kv_heads, d)."""
    if not isinstance(kc, torch.Tensor) or kc.dim() != 4:
        raise ValueError("kc must be a [pages, kv_heads, page, d] tensor")
    size = kc.shape
    pages, kv, page, d = size
    run = page * d
    psk, ldsk = _page_view(ks, "ks", _F32, (pages, kv), [1])
    psv, ldsv = _page_view(vs, "vs", _F32, (pages, kv), [1])
    pk, ldk = _page_view(kc, "kc", _F8, size, [run, d, 1])
    pv, ldv = _page_view(vc, "vc", _F8, size, [run, d, 1])
    pt = _page_table(page_table, nseq)
    return (pk, pv, psk, psv), (ldk, ldv, ldsk, ldsv), pt, (pages, page_table.shape[1], page, kv, d)


def _page_table(page_table, nseq):
    pt = _ptr(page_table, "page_table", torch.int32)
    if page_table.dim() != 2 or page_table.shape[0] != nseq:
        raise ValueError(f"page_table must have shape [{nseq}, max_pages], got {tuple(page_table.shape)}")
    return pt


def _sequences(cu, name):
    if not isinstance(cu, torch.Tensor) or cu.dim() != 1 or cu.shape[0] < 1:
        raise ValueError(f"{name} must be a tensor with at least one entry")
    return cu.shape[0] - 1, _ptr(cu, name, torch.int32)


def _kv_rows(K, V, kc, vc, ks, vs, page_table, cu, max_n):
    nseq, pcu = _sequences(cu, "cu")
    pool, pitches, pt, (pages, max_pages, page, kv, d) = _pool(kc, vc, ks, vs, page_table, nseq)
    if not isinstance(K, torch.Tensor) or K.dim() != 3:
        raise ValueError("K must be a [tokens, kv_heads, d] tensor")
    T = K.shape[0]
    size = T, kv, d
    pk, ldk = _heads_view(K, "K", size)
    pv, ldv = _heads_view(V, "V", size)
    return pk, pv, pool, pt, pcu, nseq, (nseq, T, _i32(max_n, "max_n"), kv, d, page, pages, max_pages, ldk, ldv, *pitches)


def mp_kv_cache_write(K, V, kc, vc, ks, vs, page_table, cu, start, *, max_n: int, d_status=None, stream=None) -> None:
    """New keys and values into an e4m3 cache: rows cu[i] .. cu[i+1]-1 of K, V [T, kv_heads, d] (rows may be strided)
    become positions start[i] ... of sequence i, in page page_table[i, position // page]. kc, vc [pages, kv_heads, page, d],
    ks, vs [pages, kv_heads] (pages may be strided). max_n: at least the longest sequence's rows."""
    code = (_bind or _fast()).kv_cache_write(K, V, kc, vc, ks, vs, page_table, cu, start, max_n, d_status, _handle(stream))
    if code is not None:
        return _check("mp_kv_cache_write", code)
    _here(K=K, V=V, kc=kc, vc=vc, ks=ks, vs=vs, page_table=page_table, cu=cu, start=start, d_status=d_status)
    pk, pv, pool, pt, pcu, nseq, sizes = _kv_rows(K, V, kc, vc, ks, vs, page_table, cu, max_n)
    code = lib().mp_kv_cache_write(pk, pv, *pool, pt, pcu, _ptr(start, "start", torch.int32, (nseq,)), *sizes,
                                   _status_ptr(d_status), _stream(stream))
    _check("mp_kv_cache_write", code)


def mp_kv_cache_read(kc, vc, ks, vs, K, V, page_table, cu, start=None, *, max_n: int, d_status=None,
                     stream=None) -> None:
    """Cached rows back to bf16: the arguments of mp_kv_cache_write, K and V written. start None: from position 0."""
    code = (_bind or _fast()).kv_cache_read(K, V, kc, vc, ks, vs, page_table, cu, start, max_n, d_status, _handle(stream))
    if code is not None:
        return _check("mp_kv_cache_read", code)
    _here(K=K, V=V, kc=kc, vc=vc, ks=ks, vs=vs, page_table=page_table, cu=cu, start=start, d_status=d_status)
    pk, pv, pool, pt, pcu, nseq, sizes = _kv_rows(K, V, kc, vc, ks, vs, page_table, cu, max_n)
    code = lib().mp_kv_cache_read(*pool, pk, pv, pt, pcu, _ptr(start, "start", torch.int32, (nseq,), True), *sizes,
                                  _status_ptr(d_status), _stream(stream))
    _check("mp_kv_cache_read", code)


def mp_attn_cache_workspace_bytes(heads: int, kv_heads: int, d: int, max_q: int) -> int:
    return int(lib().mp_attn_cache_workspace_bytes(_i32(heads, "heads"), _i32(kv_heads, "kv_heads"), _i32(d, "d"),
                                                   _i32(max_q, "max_q")))


def mp_attn_cache_fwd(Q, kc, vc, ks, vs, O, LSE, page_table, cu_q, lens, workspace, *, max_q: int, causal: bool = True,
                      scale: float | None = None, d_status=None, stream=None) -> None:
    """Attention of the last tokens of each sequence over its e4m3 cache (mp_kv_cache_write): O [Tq, heads, d] and LSE
    [heads, Tq] fp32 from Q [Tq, heads, d] (rows may be strided). cu_q [nseq + 1]: sequence i's queries; lens [nseq]: its
    cached tokens, the queries' own among them. causal: the last query sees the last token. scale: 1 / sqrt(d) by default."""
    code = (_bind or _fast()).attn_cache_fwd(Q, kc, vc, ks, vs, O, LSE, page_table, cu_q, lens, workspace, max_q,
                                             1 if causal else 0, scale, d_status, _handle(stream))
    if code is not None:
        return _check("mp_attn_cache_fwd", code)
    _here(Q=Q, kc=kc, vc=vc, ks=ks, vs=vs, O=O, LSE=LSE, page_table=page_table, cu_q=cu_q, lens=lens, workspace=workspace,
          d_status=d_status)
    if not isinstance(Q, torch.Tensor) or Q.dim() != 3:
        raise ValueError("Q must be a [tokens, heads, d] tensor")
    nseq, pcu = _sequences(cu_q, "cu_q")
    pool, pitches, pt, (pages, max_pages, page, kv, d) = _pool(kc, vc, ks, vs, page_table, nseq)
    T, heads, _ = Q.shape
    size = T, heads, d
    pq, ldq = _heads_view(Q, "Q", size)
    po, ldo = _heads_view(O, "O", size)
    wp, wb = _cuda_ws(workspace)
    code = lib().mp_attn_cache_fwd(
        pq, *pool, po, _ptr(LSE, "LSE", torch.float32, (heads, T)), pt, pcu, _ptr(lens, "lens", torch.int32, (nseq,)), wp,
        wb, nseq, T, _i32(max_q, "max_q"), heads, kv, d, page, pages, max_pages, ldq, ldo, *pitches, 1 if causal else 0,
        d ** -0.5 if scale is None else float(scale), _status_ptr(d_status), _stream(stream))
    _check("mp_attn_cache_fwd", code)


def mp_status_from_device(bits: int) -> int:
    return int(lib().mp_status_from_device(ctypes.c_uint32(int(bits) & 0xFFFFFFFF)))


def mp_version() -> int:
    return int(lib().mp_version())
