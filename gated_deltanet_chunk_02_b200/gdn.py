"""Thin ctypes binding of libgdn (the C ABI declared in include/gdn.h).

Argument marshalling only: every step of the path runs in the library's CUDA
kernels.  Tensors are torch CUDA tensors (PyTorch supplies device memory and
streams); each function passes their data pointers, the shape and the current
(or given) CUDA stream to the C entry point of the same name and raises
``GdnError`` on a nonzero return.  There is no fallback: if libgdn.so is
missing or does not load, every call raises.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgdn.so")

GDN_F32, GDN_BF16 = 0, 1
GDN_PREC_F32, GDN_PREC_F16 = 0, 1
GDN_OK, GDN_ERR_ARG, GDN_ERR_ALIGN, GDN_ERR_UNSUPPORTED, GDN_ERR_CUDA, GDN_ERR_TIMEOUT = \
    0, -1, -2, -3, -4, -5

EXPORTS = [
    "gdn_build_A", "gdn_invert_neumann", "gdn_invert_newton", "gdn_invert_blocked",
    "gdn_invert_fwdsub", "gdn_wy",
    "gdn_invert_neumann_i8", "gdn_invert_neumann_i8_residual", "gdn_invert_neumann_i16",
    "gdn_invert_neumann_i16_residual",
    "gdn_chunk_wy_fused", "gdn_chunk_wy_fused_raw", "gdn_forward",
    "gdn_forward_workspace_bytes", "gdn_forward_static", "gdn_decode", "gdn_get_status",
    "gdn_last_error", "gdn_launch_count", "gdn_debug_arm_wait_expiry", "gdn_forward_raw",
    "gdn_forward_raw_workspace_bytes",
    "gdn_rotary_frequencies", "gdn_rotary", "gdn_linear_forward",
    "gdn_linear_forward_workspace_bytes", "gdn_linear_backward",
    "gdn_linear_backward_workspace_bytes", "gdn_linear_decode", "gdn_block_norm",
    "gdn_block_norm_backward", "gdn_block_norm_backward_workspace_bytes",
    "gdn_debug_arm_linear_expiry",
]
GDN_ACT = {"sigmoid": 0, "silu": 1}
GDN_ROTARY = {"plain": 0, "linear": 1, "ntk": 2, "yarn": 3}


class GdnShape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int64), ("H", ctypes.c_int64), ("T", ctypes.c_int64),
                ("k", ctypes.c_int32), ("d", ctypes.c_int32)]


class GdnStrides(ctypes.Structure):
    _fields_ = [("b", ctypes.c_int64), ("h", ctypes.c_int64), ("t", ctypes.c_int64)]


class GdnLinearShape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int64), ("Hk", ctypes.c_int64), ("Hv", ctypes.c_int64),
                ("T", ctypes.c_int64), ("nseq", ctypes.c_int64), ("d", ctypes.c_int32)]


class GdnError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"libgdn error {code}: {msg}")
        self.code = code


_lib = None
_P = ctypes.c_void_p
_I = ctypes.c_int
_I64 = ctypes.c_int64


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libgdn.so (once) and declare the C signatures."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise GdnError(GDN_ERR_UNSUPPORTED,
                       f"{path} is missing: build it with "
                       "`python -m gated_deltanet_chunk_02_b200.build`")
    lib = ctypes.CDLL(path)
    S = GdnShape
    X, L = GdnStrides, GdnLinearShape
    F = ctypes.c_float
    sig = {
        "gdn_build_A": [_P, _P, _P, _P, S, _I, _P],
        "gdn_invert_neumann": [_P, _P, S, _I, _I, _I, _I, _P],
        "gdn_invert_newton": [_P, _P, S, _I, _I, _I, _P],
        "gdn_invert_blocked": [_P, _P, S, _P],
        "gdn_invert_fwdsub": [_P, _P, S, _P],
        "gdn_wy": [_P, _P, _P, _P, _P, _P, _P, S, _I, _P],
        "gdn_invert_neumann_i8": [_P, _P, _I, _I, _P, _P, _P, S, _P],
        "gdn_invert_neumann_i16": [_P, _P, _I, _I, _P, _P, _P, S, _P],
        "gdn_invert_neumann_i8_residual": [_P, _P, _I, _I, _I, S, _P],
        "gdn_invert_neumann_i16_residual": [_P, _P, _I, _I, _I, S, _P],
        "gdn_chunk_wy_fused": [_P, _P, _P, _P, _I, _I, _I, _I, _P, _P, _P, S, _I, _P],
        "gdn_chunk_wy_fused_raw": [_P, _P, _P, _P, _I, _I, _I, _I, _P, _P, _P, _P, _P, S, _I,
                                   _P],
        "gdn_forward": [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P, _P, _P, _I64, S, _I, _P],
        "gdn_forward_workspace_bytes": [S, _I],
        "gdn_forward_raw": [_P, _P, _P, _P, _P, _P, _I, _I, _I, _P, _P, _P, _I64, S, _I, _P],
        "gdn_forward_raw_workspace_bytes": [S, _I],
        "gdn_forward_static": [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P, _P, S, _I, _P],
        "gdn_decode": [_P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, ctypes.c_int32, _I,
                       _P],
        "gdn_rotary_frequencies": [_P, _P, _I, ctypes.c_double, _I, ctypes.c_double, _I64],
        "gdn_rotary": [_P, X, _P, X, _P, X, _P, X, _P, _P, F, _I, _I, _I, _I64, _I64, _I64, _I64,
                       ctypes.c_int32, _I, _P],
        "gdn_linear_forward": [_P, _P, _P, _P, _P, _P, F, _P, _P, _P, _I64, L, _I, _P],
        "gdn_linear_forward_workspace_bytes": [L, _I],
        "gdn_linear_backward": [_P, _P, _P, _P, _P, _P, _P, _P, F, _P, _P, _P, _P, _P, _I64, L, _I,
                                _P],
        "gdn_linear_backward_workspace_bytes": [L, _I],
        "gdn_linear_decode": [_P, _P, _P, _P, _P, _P, _I64, F, _P, _I64, _I64, _I64, _I64,
                              ctypes.c_int32, _I, _P],
        "gdn_block_norm": [_P, X, _P, _P, _P, _P, F, F, _I, _P, _P, _I64, _I64, _I64, _I64, _I,
                           _P],
        "gdn_block_norm_backward": [_P, X, _P, _P, _P, _P, _P, _P, F, F, _I, _P, X, _P, _P, _P, _P,
                                    _P, _I64, _I64, _I64, _I64, _I64, _I, _P],
        "gdn_block_norm_backward_workspace_bytes": [_I64, _I64, _I64, _I64],
        "gdn_get_status": [_P],
        "gdn_debug_arm_wait_expiry": [_I, _I, ctypes.c_double],
        "gdn_debug_arm_linear_expiry": [_I, _I, ctypes.c_double],
        "gdn_last_error": [],
        "gdn_launch_count": [],
    }
    for name, args in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = _I
    lib.gdn_forward_workspace_bytes.restype = _I64
    lib.gdn_forward_raw_workspace_bytes.restype = _I64
    for name in ("gdn_linear_forward_workspace_bytes", "gdn_linear_backward_workspace_bytes",
                 "gdn_block_norm_backward_workspace_bytes"):
        getattr(lib, name).restype = _I64
    lib.gdn_launch_count.restype = _I64
    lib.gdn_last_error.restype = ctypes.c_char_p
    _lib = lib
    return lib


def _check(rc: int) -> None:
    if rc != GDN_OK:
        raise GdnError(rc, (load().gdn_last_error() or b"").decode())


def _ptr(t):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch tensor")
    if t.numel() and not t.is_cuda:
        raise ValueError("libgdn takes CUDA tensors")
    if not t.is_contiguous():
        raise ValueError("libgdn takes contiguous tensors")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _dtype(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return GDN_BF16
    if t.dtype == torch.float32:
        return GDN_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def shape(B: int, H: int, T: int, k: int, d: int = 128) -> GdnShape:
    return GdnShape(B, H, T, k, d)


def shape_of(x: torch.Tensor, k: int) -> GdnShape:
    """Shape struct of a ``[B, H, T, d]`` tensor with chunk size ``k``."""
    B, H, T, d = x.shape
    return GdnShape(B, H, T, k, d)


def shape_of_chunks(A: torch.Tensor, d: int = 128) -> GdnShape:
    """Shape struct of a ``[B, H, T/k, k, k]`` tensor (A or T)."""
    B, H, n, k, _ = A.shape
    return GdnShape(B, H, n * k, k, d)


def gdn_build_A(K, beta, g, A, k, stream=None):
    """A = -b_i (k_i . k_j) e^(g_i - g_j) below the diagonal of every chunk: K
    ``[B, H, T, d]`` (bf16 or float32), beta, g ``[B, H, T]`` float32 -> A
    ``[B, H, T/k, k, k]`` float32."""
    _check(load().gdn_build_A(_ptr(K), _ptr(beta), _ptr(g), _ptr(A), shape_of(K, k), _dtype(K),
                              _stream(stream)))


def gdn_invert_neumann(A, T, N, mask, S, prec=GDN_PREC_F32, stream=None):
    """T = truncated series of order N (band mask if ``mask``) corrected by S
    residual powers; A, T ``[B, H, T/k, k, k]`` float32; ``prec`` selects the
    fp16-operand tensor-core chain or the float32 CUDA-core one."""
    _check(load().gdn_invert_neumann(_ptr(A), _ptr(T), shape_of_chunks(A), N, int(mask), S, prec,
                                     _stream(stream)))


def gdn_invert_newton(A, T, N, mask, M, stream=None):
    """The series of order N, then M sequential corrections T <- T + T(I - (I - A)T)."""
    _check(load().gdn_invert_newton(_ptr(A), _ptr(T), shape_of_chunks(A), N, int(mask), M,
                                    _stream(stream)))


def gdn_invert_blocked(A, T, stream=None):
    """Exact T by 2 x 2 block decomposition on the tensor cores (k <= 64)."""
    _check(load().gdn_invert_blocked(_ptr(A), _ptr(T), shape_of_chunks(A), _stream(stream)))


def gdn_invert_fwdsub(A, T, stream=None):
    """Exact T by forward substitution (float32)."""
    _check(load().gdn_invert_fwdsub(_ptr(A), _ptr(T), shape_of_chunks(A), _stream(stream)))


def gdn_wy(T, K, V, beta, g, W, U, stream=None):
    """W = T diag(beta) K (W_g = T diag(beta e^g) K when ``g`` is given) and
    U = T diag(beta) V; W, U ``[B, H, T, d]`` in the dtype of K."""
    k = T.shape[-1]
    _check(load().gdn_wy(_ptr(T), _ptr(K), _ptr(V), _ptr(beta), _ptr(g), _ptr(W), _ptr(U),
                         shape_of(K, k), _dtype(K), _stream(stream)))


def gdn_invert_neumann_i8(A, T, N, mask, q=None, acc=None, scale=None, stream=None):
    """INT8 series (bit-exact scheme of gdn.h); optional dumps: codes ``q``
    int8 ``[nc, N, k, k]``, accumulators ``acc`` int32, scales float32 ``[nc, N]``."""
    _check(load().gdn_invert_neumann_i8(_ptr(A), _ptr(T), N, int(mask), _ptr(q), _ptr(acc),
                                        _ptr(scale), shape_of_chunks(A), _stream(stream)))


def gdn_invert_neumann_i8_residual(A, T, N, mask, S, stream=None):
    """INT8 series followed by S residual powers, every product in int8 codes."""
    _check(load().gdn_invert_neumann_i8_residual(_ptr(A), _ptr(T), N, int(mask), S,
                                                 shape_of_chunks(A), _stream(stream)))


def gdn_invert_neumann_i16(A, T, N, mask, q=None, acc=None, scale=None, stream=None):
    """INT16 series (int64 accumulators, binary64 scales); optional dumps: codes
    int16, accumulators int64, scales float64."""
    _check(load().gdn_invert_neumann_i16(_ptr(A), _ptr(T), N, int(mask), _ptr(q), _ptr(acc),
                                         _ptr(scale), shape_of_chunks(A), _stream(stream)))


def gdn_invert_neumann_i16_residual(A, T, N, mask, S, stream=None):
    """INT16 series followed by S residual powers, every product in int16 codes."""
    _check(load().gdn_invert_neumann_i16_residual(_ptr(A), _ptr(T), N, int(mask), S,
                                                  shape_of_chunks(A), _stream(stream)))


def gdn_chunk_wy_fused(K, V, beta, g, N, mask, S, gated, W, U, T=None, k=64, stream=None):
    """A, the series + mask + residual and W, U in one kernel; T is written
    only when a ``T`` tensor is given."""
    _check(load().gdn_chunk_wy_fused(_ptr(K), _ptr(V), _ptr(beta), _ptr(g), N, int(mask), S,
                                     int(gated), _ptr(W), _ptr(U), _ptr(T), shape_of(K, k),
                                     _dtype(K), _stream(stream)))


def gdn_chunk_wy_fused_raw(K_raw, V, beta, loggate, N, mask, S, gated, W, U, T=None,
                           K_out=None, g_out=None, k=64, stream=None):
    """The fused step from raw keys (normalised in the kernel) and per-token
    log-gates (summed chunk-locally in the kernel)."""
    _check(load().gdn_chunk_wy_fused_raw(_ptr(K_raw), _ptr(V), _ptr(beta), _ptr(loggate), N,
                                         int(mask), S, int(gated), _ptr(W), _ptr(U), _ptr(T),
                                         _ptr(K_out), _ptr(g_out), shape_of(K_raw, k),
                                         _dtype(K_raw), _stream(stream)))


def gdn_forward_workspace_bytes(K, k):
    """Scratch bytes ``gdn_forward`` needs for K's shape and dtype."""
    return int(load().gdn_forward_workspace_bytes(shape_of(K, k), _dtype(K)))


def gdn_forward(Q, K, V, beta, g, S0, N, mask, S, exact, O, S_final, workspace, k=64,
                stream=None):
    """Chunk-wise forward: O ``[B, H, T, d]`` and the final state ``S_final``
    ``[B, H, d, d]`` float32 from the start state ``S0`` (None = zero);
    ``exact`` inverts by forward substitution instead of the series."""
    ws = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().gdn_forward(_ptr(Q), _ptr(K), _ptr(V), _ptr(beta), _ptr(g), _ptr(S0), N,
                              int(mask), S, int(exact), _ptr(O), _ptr(S_final), _ptr(workspace),
                              ws, shape_of(K, k), _dtype(K), _stream(stream)))


def gdn_forward_raw_workspace_bytes(K, k):
    """Scratch bytes ``gdn_forward_raw`` needs for K's shape (bf16)."""
    return int(load().gdn_forward_raw_workspace_bytes(shape_of(K, k), _dtype(K)))


def gdn_forward_raw(Q_raw, K_raw, V, beta, loggate, S0, N, mask, S, O, S_final, workspace, k=64,
                    stream=None):
    """Chunk-wise forward from un-normalised query and key rows and per-token
    log-gates (normalised and summed in the kernels); O and the final state as
    in ``gdn_forward``."""
    ws = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().gdn_forward_raw(_ptr(Q_raw), _ptr(K_raw), _ptr(V), _ptr(beta), _ptr(loggate),
                                  _ptr(S0), N, int(mask), S, _ptr(O), _ptr(S_final),
                                  _ptr(workspace), ws, shape_of(K_raw, k), _dtype(K_raw),
                                  _stream(stream)))


def gdn_forward_static(Q, K, V, beta, g, S0, N, mask, S, exact, O, S_final, k=64, stream=None):
    """gdn_forward with the library's own fixed scratch array (no workspace, no
    allocation); see include/gdn.h for its size limit and sharing rules."""
    _check(load().gdn_forward_static(_ptr(Q), _ptr(K), _ptr(V), _ptr(beta), _ptr(g), _ptr(S0), N,
                                     int(mask), S, int(exact), _ptr(O), _ptr(S_final),
                                     shape_of(K, k), _dtype(K), _stream(stream)))


def gdn_decode(Q, K, V, beta, loggate, S, O, stream=None):
    """Decode n tokens: Q, K ``[B, Hk, n, d]``, V, O ``[B, Hv, n, d]``, beta,
    loggate ``[B, Hv, n]``, state S ``[B, Hv, d, d]`` (float32, in place)."""
    B, Hk, n, d = K.shape
    Hv = V.shape[1]
    _check(load().gdn_decode(_ptr(Q), _ptr(K), _ptr(V), _ptr(beta), _ptr(loggate), _ptr(S),
                             _ptr(O), B, Hk, Hv, n, d, _dtype(K), _stream(stream)))


class _Call:
    """Checks of one call's tensors: shapes, types, one CUDA device (made
    current for the launch) and the stream on it.  Kept short: a call on a few
    rows costs the host more than the GPU."""
    __slots__ = ("index", "stream")

    def __init__(self, stream, first):
        if not isinstance(first, torch.Tensor):
            raise TypeError("expected a torch tensor")
        self.index, self.stream = first.get_device(), stream

    def check(self, t, name, shape=None, dtype=None, strided=False):
        """The data pointer of ``t`` (None passes as NULL)."""
        if t is None:
            return None
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name}: expected a torch tensor")
        if shape is not None and t.shape != shape:
            raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
        if dtype is not None and t.dtype != dtype:
            raise TypeError(f"{name}: {t.dtype}, expected {dtype}")
        index = t.get_device()
        if index < 0:
            raise ValueError(f"{name}: libgdn takes CUDA tensors")
        if index != self.index:
            raise ValueError(f"{name} is on cuda:{index}, expected cuda:{self.index}")
        if strided:
            if t.stride(-1) != 1 and t.shape[-1] > 1 and t.numel():
                raise ValueError(f"{name}: the last dimension is not contiguous")
        elif not t.is_contiguous():
            raise ValueError(f"{name}: libgdn takes contiguous tensors")
        return t.data_ptr()

    def run(self, name, *args):
        """The C call on the tensors' device and its current (or the given) stream."""
        f, index = getattr(_lib or load(), name), self.index
        if self.stream is None:
            stream = torch._C._cuda_getCurrentRawStream(index)
        elif self.stream.device.index != index:
            raise ValueError(f"the stream is on {self.stream.device}, the tensors on cuda:{index}")
        else:
            stream = self.stream.cuda_stream
        if torch.cuda.current_device() == index:
            rc = f(*args, stream)
        else:
            with torch.cuda.device(index):
                rc = f(*args, stream)
        if rc != GDN_OK:
            _check(rc)


def _strides(t, b, h, tok):
    """Element strides of the named dimensions (0 where nothing is walked)."""
    n, st = t.shape, t.stride()
    return GdnStrides(st[b] if n[b] > 1 else 0, st[h] if n[h] > 1 else 0,
                      st[tok] if n[tok] > 1 else 0)


def _apart(outs, ins):
    """Outputs share no memory with inputs or one another (contiguous tensors)."""
    spans = [(t.data_ptr(), t.nbytes, True, n) for n, t in outs if t is not None]
    spans += [(t.data_ptr(), t.nbytes, False, n) for n, t in ins if t is not None]
    spans.sort()
    end_out, end_all, last_out, last = 0, 0, "", ""
    for at, size, out, name in spans:
        if not size:
            continue
        if at < (end_all if out else end_out):
            raise ValueError(f"{name} shares memory with {last if out else last_out}")
        if out and at + size > end_out:
            end_out, last_out = at + size, name
        if at + size > end_all:
            end_all, last = at + size, name


def gdn_rotary_frequencies(rot, base=10000.0, scaling="plain", factor=1.0, original_length=0):
    """Frequencies of ``rot / 2`` rotated pairs (CPU float32 tensor) and the
    factor on sines and cosines; ``scaling``: plain, linear, ntk or yarn."""
    inv = torch.empty(max(0, rot // 2), dtype=torch.float32)
    m = ctypes.c_float()
    _check(load().gdn_rotary_frequencies(inv.data_ptr(), ctypes.byref(m), rot,
                                         float(base), GDN_ROTARY[scaling], float(factor),
                                         int(original_length)))
    return inv, m.value


def gdn_rotary(Q, K, positions, inv_freq, Q_out, K_out, mscale=1.0, interleaved=False,
               inverse=False, stream=None):
    """Rotary positions on the first ``2 * len(inv_freq)`` columns of Q
    ``[B, Hq, T, d]`` and K ``[B, Hk, T, d]`` (either may be None; views of any
    strides with contiguous rows) at ``positions`` int64 ``[B, T]``; outputs may
    be the inputs.  ``inverse`` turns back: the gradient."""
    given = Q if Q is not None else K
    c = _Call(stream, given)
    B, _, T, d = given.shape
    ptr, strides, heads = [], [], []
    for x, y, name in ((Q, Q_out, "Q"), (K, K_out, "K")):
        if x is None:
            ptr += [None, None]
            strides += [GdnStrides(), GdnStrides()]
            heads.append(0)
            continue
        if y is None:
            raise TypeError(f"{name}_out: expected a torch tensor")
        H = x.shape[1]
        ptr += [c.check(x, name, (B, H, T, d), given.dtype, strided=True),
                c.check(y, name + "_out", (B, H, T, d), given.dtype, strided=True)]
        strides += [_strides(x, 0, 1, 2), _strides(y, 0, 1, 2)]
        heads.append(H)
    c.run("gdn_rotary", ptr[0], strides[0], ptr[1], strides[1], ptr[2], strides[2], ptr[3],
          strides[3], c.check(positions, "positions", (B, T), torch.int64),
          c.check(inv_freq, "inv_freq", (inv_freq.numel(),), torch.float32), mscale,
          2 * inv_freq.numel(), int(interleaved), int(inverse), B, heads[0], heads[1], T, d,
          _dtype(given))


def _linear_shape(K, V, cu_seqlens):
    B, Hk, T, d = K.shape
    return GdnLinearShape(B, Hk, V.shape[1], T,
                          0 if cu_seqlens is None else cu_seqlens.numel() - 1, d)


def _workspace(fn, *args):
    n = int(fn(*args))
    if n < 0:
        raise GdnError(GDN_ERR_ARG, gdn_last_error())
    return n


def gdn_linear_forward_workspace_bytes(K, V, cu_seqlens=None):
    """Scratch bytes ``gdn_linear_forward`` needs for these shapes and dtype."""
    with torch.cuda.device(K.device):
        return _workspace(load().gdn_linear_forward_workspace_bytes,
                          _linear_shape(K, V, cu_seqlens), _dtype(K))


def gdn_linear_backward_workspace_bytes(K, V, cu_seqlens=None):
    """Scratch bytes ``gdn_linear_backward`` needs for these shapes and dtype."""
    with torch.cuda.device(K.device):
        return _workspace(load().gdn_linear_backward_workspace_bytes,
                          _linear_shape(K, V, cu_seqlens), _dtype(K))


def _linear_inputs(c, Q, K, V, loggate, cu_seqlens):
    """Checked pointers of Q, K, V, loggate, cu_seqlens and the shapes of a
    tensor over value heads and of the states."""
    B, Hk, T, d = K.shape
    Hv = V.shape[1]
    n = B
    if cu_seqlens is not None:
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
            raise ValueError("cu_seqlens: expected [nseq + 1] bounds")
        n = cu_seqlens.numel() - 1
    rows, states = (B, Hv, T, d), (n, Hv, d, d)
    return ([c.check(Q, "Q", K.shape, K.dtype), c.check(K, "K"), c.check(V, "V", rows, K.dtype),
             c.check(loggate, "loggate", (Hv,), torch.float32),
             c.check(cu_seqlens, "cu_seqlens", None, torch.int32)], rows, states)


def gdn_linear_forward(Q, K, V, loggate, S0, O, S_final, workspace, scale=1.0, cu_seqlens=None,
                       stream=None):
    """Linear attention with a decay per head, o_t = scale S_t q_t with S_t =
    e^loggate S_{t-1} + v_t k_t^T: Q, K ``[B, Hk, T, d]``, V, O ``[B, Hv, T, d]``,
    loggate float32 ``[Hv]``, S0 (or None) and S_final (or None) float32
    ``[n, Hv, d, d]``; n = B, or with ``cu_seqlens`` (int32 ``[n + 1]``, B = 1)
    the number of packed sequences."""
    _apart([("O", O), ("S_final", S_final), ("workspace", workspace)],
           [("Q", Q), ("K", K), ("V", V), ("S0", S0), ("loggate", loggate),
            ("cu_seqlens", cu_seqlens)])
    c = _Call(stream, K)
    (q, k, v, lg, cu), rows, states = _linear_inputs(c, Q, K, V, loggate, cu_seqlens)
    ws = 0 if workspace is None else workspace.numel() * workspace.element_size()
    c.run("gdn_linear_forward", q, k, v, lg, c.check(S0, "S0", states, torch.float32), cu, scale,
          c.check(O, "O", rows, K.dtype), c.check(S_final, "S_final", states, torch.float32),
          c.check(workspace, "workspace"), ws, _linear_shape(K, V, cu_seqlens), _dtype(K))


def gdn_linear_backward(Q, K, V, loggate, S0, dO, dS_final, dQ, dK, dV, dS0, workspace, scale=1.0,
                        cu_seqlens=None, stream=None):
    """Gradients of ``gdn_linear_forward`` for dO and dS_final (or None): dQ, dK
    (summed over the value heads that share them), dV, and dS0 (or None)."""
    _apart([("dQ", dQ), ("dK", dK), ("dV", dV), ("dS0", dS0), ("workspace", workspace)],
           [("Q", Q), ("K", K), ("V", V), ("S0", S0), ("dO", dO), ("dS_final", dS_final),
            ("loggate", loggate), ("cu_seqlens", cu_seqlens)])
    c = _Call(stream, K)
    (q, k, v, lg, cu), rows, states = _linear_inputs(c, Q, K, V, loggate, cu_seqlens)
    ws = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lambda t, name: c.check(t, name, states, torch.float32)
    c.run("gdn_linear_backward", q, k, v, lg, st(S0, "S0"), c.check(dO, "dO", rows, K.dtype),
          st(dS_final, "dS_final"), cu, scale, c.check(dQ, "dQ", K.shape, K.dtype),
          c.check(dK, "dK", K.shape, K.dtype), c.check(dV, "dV", rows, K.dtype), st(dS0, "dS0"),
          c.check(workspace, "workspace"), ws, _linear_shape(K, V, cu_seqlens), _dtype(K))


def gdn_linear_decode(Q, K, V, loggate, S, O, slots=None, scale=1.0, stream=None):
    """n tokens of the same recurrence: Q, K ``[B, Hk, n, d]``, V, O
    ``[B, Hv, n, d]``, loggate float32 ``[Hv]``; states S float32 ``[slots, Hv, d, d]``
    in place, row b using ``S[slots[b]]`` (int32 ``[B]``; negative: the row is left
    out), or ``S[b]`` without slots."""
    c = _Call(stream, K)
    B, Hk, n, d = K.shape
    Hv = V.shape[1]
    _apart([("O", O), ("S", S)], [("Q", Q), ("K", K), ("V", V), ("loggate", loggate),
                                  ("slots", slots)])
    c.run("gdn_linear_decode", c.check(Q, "Q", K.shape, K.dtype), c.check(K, "K"),
          c.check(V, "V", (B, Hv, n, d), K.dtype),
          c.check(loggate, "loggate", (Hv,), torch.float32),
          c.check(S, "S", (S.shape[0], Hv, d, d), torch.float32),
          c.check(slots, "slots", (B,), torch.int32), S.shape[0], scale,
          c.check(O, "O", (B, Hv, n, d), K.dtype), B, Hk, Hv, n, d, _dtype(K))


def gdn_block_norm(Y, Z, w_post, R, w_pre, X, N, scale=1.0, eps=1e-6, act="silu", stream=None):
    """x = R + scale act(Z) w_post norm(Y) and N = w_pre norm(x): Y ``[B, T, H, d]``
    (a view of any strides with contiguous channels, normalised over d), the
    others ``[B, T, H * d]``, weights float32 ``[H * d]``.  w_post, Z, R, and
    w_pre with N may be None (left out); X may be R, or None."""
    c = _Call(stream, Y)
    B, T, H, d = Y.shape
    wide = lambda t, name: c.check(t, name, (B, T, H * d), Y.dtype)
    weight = lambda t, name: c.check(t, name, (H * d,), torch.float32)
    c.run("gdn_block_norm", c.check(Y, "Y", strided=True), _strides(Y, 0, 2, 1), wide(Z, "Z"),
          weight(w_post, "w_post"), wide(R, "R"), weight(w_pre, "w_pre"), scale, eps, GDN_ACT[act],
          wide(X, "X"), wide(N, "N"), B, T, H, d, _dtype(Y))


def gdn_block_norm_backward_workspace_bytes(Y):
    """Scratch bytes ``gdn_block_norm_backward`` needs for Y ``[B, T, H, d]``."""
    B, T, H, d = Y.shape
    with torch.cuda.device(Y.device):
        n = int(load().gdn_block_norm_backward_workspace_bytes(B, T, H, d))
    if n < 0:
        raise GdnError(GDN_ERR_UNSUPPORTED, f"rows of {H} x {d} channels are not served")
    return n


def gdn_block_norm_backward(Y, Z, w_post, R, w_pre, dX, dN, dY, dZ, dR, dw_post, dw_pre, workspace,
                            scale=1.0, eps=1e-6, act="silu", stream=None):
    """Gradients of ``gdn_block_norm`` for dX and dN; each of Z, w_post and
    w_pre (with dN) goes together with its gradient; dR may be None or dX."""
    c = _Call(stream, Y)
    B, T, H, d = Y.shape
    wide = lambda t, name: c.check(t, name, (B, T, H * d), Y.dtype)
    weight = lambda t, name: c.check(t, name, (H * d,), torch.float32)
    ws = 0 if workspace is None else workspace.numel() * workspace.element_size()
    c.run("gdn_block_norm_backward", c.check(Y, "Y", strided=True), _strides(Y, 0, 2, 1),
          wide(Z, "Z"), weight(w_post, "w_post"), wide(R, "R"), weight(w_pre, "w_pre"),
          wide(dX, "dX"), wide(dN, "dN"), scale, eps, GDN_ACT[act],
          c.check(dY, "dY", (B, T, H, d), Y.dtype, strided=True), _strides(dY, 0, 2, 1),
          wide(dZ, "dZ"), wide(dR, "dR"), weight(dw_post, "dw_post"), weight(dw_pre, "dw_pre"),
          c.check(workspace, "workspace"), ws, B, T, H, d, _dtype(Y))


def gdn_get_status(stream=None) -> int:
    """Synchronise the stream; return (and clear) the device status code."""
    return int(load().gdn_get_status(_stream(stream)))


def gdn_debug_arm_wait_expiry(tile: int, which: str, timeout_ms: float) -> None:
    """Tests only: the next fused call on this thread leaves tile ``tile``'s
    ``which`` load ("K" or "V") unissued and bounds its waits by
    ``timeout_ms`` (the wait runs out, the status word reports
    GDN_ERR_TIMEOUT)."""
    _check(load().gdn_debug_arm_wait_expiry(int(tile), {"K": 0, "V": 1}[which], float(timeout_ms)))


def gdn_debug_arm_linear_expiry(block: int, kernel: str, timeout_ms: float) -> None:
    """Tests only: the same for linear attention on bf16 data; block ``block`` of
    the next launch of its ``"outputs"`` or ``"states"`` kernel waits for a tile
    that never comes."""
    _check(load().gdn_debug_arm_linear_expiry(int(block), {"outputs": 0, "states": 1}[kernel],
                                              float(timeout_ms)))


def gdn_last_error() -> str:
    return (load().gdn_last_error() or b"").decode()


def gdn_launch_count() -> int:
    return int(load().gdn_launch_count())
