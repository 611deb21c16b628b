"""Thin ctypes binding of librehyat.so (C ABI in include/rehyat.h).

Argument marshalling only: tensors are checked for device/dtype/shape/contiguity, outputs and
workspaces are allocated with torch on the tensors' device, and every computation runs in the
library's CUDA kernels.  There is no CPU fallback: without the built library every call raises.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
import struct

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_lib", "librehyat.so")

REHYAT_F32 = 0
REHYAT_BF16 = 1
PHI_POLY = 0   # softplus parts raised to powers 1..P
PHI_ELU1 = 1   # elu(u) + 1

STATUS = {0: "OK", -1: "ERR_ARG", -2: "ERR_SHAPE", -3: "ERR_DTYPE", -4: "ERR_WORKSPACE",
          -5: "ERR_CUDA", -6: "ERR_TIMEOUT", -7: "ERR_ALIGN", -8: "ERR_BOUNDS"}

EXPORTED = ["rehyat_last_error", "rehyat_version", "rehyat_featmap",
            "rehyat_forward_workspace_size", "rehyat_forward", "rehyat_forward_states",
            "rehyat_forward_phiq", "rehyat_forward_attend", "rehyat_chunk_workspace_size",
            "rehyat_chunk_forward", "rehyat_chunk_forward_sched", "rehyat_chunk_carry_workspace_size",
            "rehyat_chunk_forward_carry", "rehyat_chunk_forward_static", "rehyat_chunk_states",
            "rehyat_forward_train", "rehyat_backward_workspace_size", "rehyat_backward",
            "rehyat_gemm_bf16", "rehyat_segment_workspace_size", "rehyat_segment_states",
            "rehyat_segment_attend", "rehyat_selftest_wait_timeout", "rehyat_selftest_bounds",
            "rehyat_sync_status", "rehyat_debug_bounds", "rehyat_rotary",
            "rehyat_decay_workspace_size", "rehyat_decay_forward", "rehyat_decay_backward",
            "rehyat_decay_step"]


class RehyatError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS.get(status, status)}: {message}")
        self.status = status


class Dims(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("H", ctypes.c_int), ("D", ctypes.c_int), ("F", ctypes.c_int),
                ("G", ctypes.c_int), ("P", ctypes.c_int), ("phi", ctypes.c_int)]


# Argument blocks of the sequence operators (rehyat_*_args in include/rehyat.h).  A tensor of rows is
# four 64-bit values: pointer and the strides of sequence, head and row.
_ROTARY = struct.Struct("12i 7q 16q f4x")
_DECAY_FORWARD = struct.Struct("6i 16q 6q f4x")
_DECAY_BACKWARD = struct.Struct("6i 28q 7q f4x")
_DECAY_STEP = struct.Struct("6i 16q 3q f4x")


_lib = None


def lib_path() -> str:
    return _LIB_PATH


def use_library(path: str) -> ctypes.CDLL:
    """Make every later call go through the library at `path` (for example the debug-bounds
    build, build.build(debug_bounds=True)); returns it loaded."""
    global _lib, _LIB_PATH
    _lib, _LIB_PATH = None, path
    decay_workspace_size.cache_clear()
    return load()


def load() -> ctypes.CDLL:
    """Load librehyat.so (built in-tree by the package build step) and declare its signatures."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise RuntimeError(f"librehyat.so is not built ({_LIB_PATH}); run the package build "
                           "step (hybrid_softmax_linear_chunked_b200.build.build()) first")
    L = ctypes.CDLL(_LIB_PATH)
    c_int, c_void_p, c_size_t = ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t
    P = c_void_p
    L.rehyat_last_error.restype = ctypes.c_char_p
    L.rehyat_last_error.argtypes = []
    L.rehyat_version.restype = c_int
    L.rehyat_featmap.argtypes = [Dims, c_int, c_int, P, P, P, P, P]
    L.rehyat_forward_workspace_size.argtypes = [Dims, c_int, c_int, c_int, c_int, c_int,
                                                ctypes.POINTER(c_size_t)]
    L.rehyat_forward.argtypes = [Dims, c_int, c_int, c_int, c_int, c_int, P, P, P, P, P, P, P, P,
                                 P, c_size_t, P]
    L.rehyat_forward_states.argtypes = [Dims, c_int, c_int, c_int, c_int, c_int, P, P, P, P, P,
                                        c_size_t, P]
    L.rehyat_forward_phiq.argtypes = [Dims, c_int, c_int, c_int, c_int, c_int, P, P, P, P,
                                      c_size_t, P]
    L.rehyat_forward_attend.argtypes = [Dims, c_int, c_int, c_int, c_int, c_int, P, P, P, P, P,
                                        c_size_t, P]
    L.rehyat_chunk_workspace_size.argtypes = [Dims, c_int, c_int, c_int, c_int,
                                              ctypes.POINTER(c_size_t)]
    L.rehyat_segment_workspace_size.argtypes = [Dims, c_int, c_int, c_int, c_int, c_int, c_int,
                                                c_int, ctypes.POINTER(c_size_t)]
    L.rehyat_segment_states.argtypes = [Dims, c_int, c_int, c_int, c_int, c_int, c_int, c_int,
                                        P, P, P, P, P, P, P, c_size_t, P]
    L.rehyat_segment_attend.argtypes = [Dims, c_int, c_int, c_int, c_int, c_int, c_int, c_int,
                                        P, P, P, P, P, c_int, P, P, P, P, c_size_t, P]
    L.rehyat_chunk_forward.argtypes = [Dims, c_int, c_int, c_int, c_int, c_int, P, P, P, P, P, P,
                                       P, P, P, P, P, c_size_t, P]
    L.rehyat_chunk_forward_sched.argtypes = [Dims, c_int, c_int, c_int, c_int, c_int, c_int, P, P,
                                             P, P, P, P, P, P, P, P, P, c_size_t, P]
    L.rehyat_chunk_carry_workspace_size.argtypes = [Dims, c_int, c_int, c_int, c_int, c_int,
                                                    ctypes.POINTER(c_size_t)]
    L.rehyat_chunk_forward_carry.argtypes = [Dims, c_int, c_int, c_int, c_int, c_int, c_int, c_int,
                                             P, P, P, P, P, P, P, P, P, P, P, P, P, c_size_t, P]
    L.rehyat_chunk_forward_static.argtypes = [Dims, c_int, c_int, c_int, c_int, c_int, P, P, P, P,
                                              P, P, P, P, P, P, P]
    L.rehyat_chunk_states.argtypes = [Dims, c_int, c_int, c_int, c_int, c_int, P, P, P, P, P, P,
                                      P, c_size_t, P]
    LL = ctypes.c_longlong
    L.rehyat_forward_train.argtypes = [Dims, c_int, c_int, c_int, c_int, c_int, P, P, P, P, P, P,
                                       P, P, P, P, c_size_t, P]
    L.rehyat_backward_workspace_size.argtypes = [Dims, c_int, c_int, c_int, c_int, c_int,
                                                 ctypes.POINTER(c_size_t)]
    L.rehyat_backward.argtypes = [Dims, c_int, c_int, c_int, c_int, c_int] + [P] * 18 + [c_size_t, P]
    L.rehyat_gemm_bf16.argtypes = [c_int, c_int, c_int, c_int, P, LL, LL, c_int, P, LL, LL, c_int,
                                   P, LL, LL, c_int, c_int, ctypes.c_float, P]
    L.rehyat_selftest_wait_timeout.argtypes = [ctypes.c_longlong, P]
    L.rehyat_selftest_bounds.argtypes = [P, ctypes.c_longlong, ctypes.c_longlong, P]
    L.rehyat_debug_bounds.argtypes = []
    for name in ("rotary", "decay_forward", "decay_backward", "decay_step"):
        getattr(L, "rehyat_" + name).argtypes = [ctypes.c_char_p, P]
    L.rehyat_decay_workspace_size.argtypes = [c_int] * 6 + [ctypes.POINTER(c_size_t)]
    L.rehyat_sync_status.argtypes = [P]
    for name in EXPORTED:
        if name not in ("rehyat_last_error",):
            getattr(L, name).restype = c_int
    _lib = L
    return L


def _check(status: int) -> None:
    if status != 0:
        raise RehyatError(status, load().rehyat_last_error().decode())


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return REHYAT_BF16
    if t.dtype == torch.float32:
        return REHYAT_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _ptr(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device: torch.device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _dev(*ts: torch.Tensor) -> torch.device:
    dev = ts[0].device
    for t in ts:
        if t is None:
            continue
        if t.device.type != "cuda" or t.device != dev:
            raise ValueError("all tensors must be on the same CUDA device")
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")
    return dev


def _shape(t: torch.Tensor | None, shape, what: str) -> None:
    """The library reads exactly the sizes the other arguments imply; a tensor of another shape
    is refused here, before anything is enqueued."""
    if t is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _frames(n_rows: int, frame_tokens: int, what: str) -> int:
    if frame_tokens < 1 or n_rows % frame_tokens:
        raise ValueError(f"{what}: {n_rows} rows are not a whole number of frames of "
                         f"{frame_tokens} tokens")
    return n_rows // frame_tokens


def _check_x_w(x: torch.Tensor, W: torch.Tensor, b: torch.Tensor | None, what: str) -> None:
    """x [B,H,n,D]; W [H,G,F/G,D/G]; b [H,F] or None."""
    if x.dim() != 4:
        raise ValueError(f"{what} must be [B,H,rows,D], got {tuple(x.shape)}")
    if W.dim() != 4 or W.shape[0] != x.shape[1] or W.shape[1] * W.shape[3] != x.shape[3]:
        raise ValueError(f"feature-map weights must be [H,G,F/G,D/G] for {what} of shape "
                         f"{tuple(x.shape)}, got {tuple(W.shape)}")
    _shape(b, (W.shape[0], W.shape[1] * W.shape[2]), "feature-map bias")


def _check_step(q, k, v, Wq, bq, Wk, bk, S, Z, out, frame_tokens: int, kv_frames: int | None,
                what_kv: str) -> int:
    """Shapes of a streaming step: q [B,H,cf*L,D]; k, v [B,H,kv_frames*L,D] (the chunk's own
    frames when kv_frames is None); S [B,H,F,D], Z [B,H,F]; out like q.  Returns cf."""
    _check_x_w(q, Wq, bq, "q")
    _check_x_w(q, Wk, bk, "q")
    _shape(Wk, Wq.shape, "Wk")
    cf = _frames(q.shape[2], frame_tokens, "q")
    B, H, _, D = q.shape
    F = Wq.shape[1] * Wq.shape[2]
    rows = (cf if kv_frames is None else kv_frames) * frame_tokens
    _shape(k, (B, H, rows, D), what_kv)
    _shape(v, (B, H, rows, D), what_kv.replace("k", "v", 1))
    _shape(S, (B, H, F, D), "S")
    _shape(Z, (B, H, F), "Z")
    _shape(out, q.shape, "out")
    return cf


def _weights(W: torch.Tensor, b: torch.Tensor | None):
    if W.dtype != torch.float32 or (b is not None and b.dtype != torch.float32):
        raise TypeError("feature-map weights and biases are fp32")
    return W, b


def dims_of(x: torch.Tensor, W: torch.Tensor, P: int, phi: int = 0) -> Dims:
    """Dims from x [B,H,n,D] and W [H,G,F/G,D/G]; phi is PHI_POLY or PHI_ELU1."""
    B, H, _, D = x.shape
    Hw, G, Fg, _ = W.shape
    if Hw != H:
        raise ValueError("W has a different head count than x")
    return Dims(B, H, D, G * Fg, G, P, phi)


def version() -> int:
    return load().rehyat_version()


def featmap(x: torch.Tensor, W: torch.Tensor, bias: torch.Tensor | None, P: int,
            phi: int = 0) -> torch.Tensor:
    """phi(x) for x [B,H,n,D] -> [B,H,n,F] (same dtype as x)."""
    L = load()
    dev = _dev(x, W, bias)
    _weights(W, bias)
    d = dims_of(x, W, P, phi)
    phi = torch.empty(x.shape[0], x.shape[1], x.shape[2], d.F, dtype=x.dtype, device=dev)
    _check(L.rehyat_featmap(d, _dtype_code(x), x.shape[2], _ptr(x), _ptr(W), _ptr(bias),
                            _ptr(phi), _stream(dev)))
    return phi


def forward_workspace_size(d: Dims, dtype_code: int, T: int, L_: int, Tc: int, To: int) -> int:
    n = ctypes.c_size_t(0)
    _check(load().rehyat_forward_workspace_size(d, dtype_code, T, L_, Tc, To, ctypes.byref(n)))
    return n.value


def chunk_workspace_size(d: Dims, dtype_code: int, L_: int, chunk_frames: int, To: int) -> int:
    n = ctypes.c_size_t(0)
    _check(load().rehyat_chunk_workspace_size(d, dtype_code, L_, chunk_frames, To,
                                              ctypes.byref(n)))
    return n.value


def _workspace(nbytes: int, dev: torch.device, workspace: torch.Tensor | None) -> torch.Tensor:
    if workspace is not None and workspace.numel() >= nbytes:
        return workspace
    return torch.empty(max(nbytes, 16), dtype=torch.uint8, device=dev)


def forward(q, k, v, Wq, bq, Wk, bk, *, P: int, phi: int = 0, frame_tokens: int, Tc: int, To: int,
            out: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """Hybrid attention over a whole sequence: q, k, v [B,H,T*frame_tokens,D] -> out."""
    lib = load()
    _check_x_w(q, Wq, bq, "q")
    _check_x_w(q, Wk, bk, "q")
    _shape(Wk, Wq.shape, "Wk")
    for t, n in ((k, "k"), (v, "v"), (out, "out")):
        _shape(t, q.shape, n)
    dev = _dev(q, k, v, Wq, bq, Wk, bk)
    _weights(Wq, bq), _weights(Wk, bk)
    d = dims_of(q, Wq, P, phi)
    N = q.shape[2]
    if N % frame_tokens:
        raise ValueError("sequence length is not a multiple of frame_tokens")
    T = N // frame_tokens
    code = _dtype_code(q)
    ws = _workspace(forward_workspace_size(d, code, T, frame_tokens, Tc, To), dev, workspace)
    if out is None:
        out = torch.empty_like(q)
    _check(lib.rehyat_forward(d, code, T, frame_tokens, Tc, To, _ptr(q), _ptr(k), _ptr(v),
                              _ptr(Wq), _ptr(bq), _ptr(Wk), _ptr(bk), _ptr(out), _ptr(ws),
                              ws.numel(), _stream(dev)))
    return out


def segment_bounds(T: int, Tc: int, To: int, c0: int, c1: int) -> tuple[int, int, int]:
    """(s0, s1, h0) of the segment of chunks [c0, c1): query frames [s0, s1), key/value frames
    [h0, s1)."""
    s0, s1 = c0 * Tc, min(c1 * Tc, T)
    return s0, s1, max(0, s0 - To)


def segment_workspace_size(d: Dims, T: int, frame_tokens: int, Tc: int, To: int, c0: int,
                           c1: int) -> int:
    n = ctypes.c_size_t(0)
    _check(load().rehyat_segment_workspace_size(d, REHYAT_BF16, T, frame_tokens, Tc, To, c0, c1,
                                                ctypes.byref(n)))
    return n.value


def segment_states(k_seg, v_seg, Wk, bk, *, T: int, c0: int, c1: int, P: int, phi: int = 0,
                   frame_tokens: int, Tc: int, To: int, workspace: torch.Tensor,
                   S_seg: torch.Tensor | None = None, Z_seg: torch.Tensor | None = None):
    """First phase of a context-parallel segment (chunks [c0, c1) of a T-frame sequence):
    k_seg, v_seg [B,H,(s1-h0)*frame_tokens,D] bf16 (halo frames first).  Fills `workspace` with
    the segment's folds and returns their sum (S_seg [B,H,F,D], Z_seg [B,H,F] fp32)."""
    lib = load()
    _check_x_w(k_seg, Wk, bk, "k_seg")
    s0, s1, h0 = segment_bounds(T, Tc, To, c0, c1)
    B, H, _, D = k_seg.shape
    F = Wk.shape[1] * Wk.shape[2]
    _shape(k_seg, (B, H, (s1 - h0) * frame_tokens, D), "k_seg")
    _shape(v_seg, k_seg.shape, "v_seg")
    _shape(S_seg, (B, H, F, D), "S_seg")
    _shape(Z_seg, (B, H, F), "Z_seg")
    dev = _dev(k_seg, v_seg, Wk, bk, workspace)
    d = dims_of(k_seg, Wk, P, phi)
    B, H = d.B, d.H
    if S_seg is None:
        S_seg = torch.empty(B, H, d.F, d.D, dtype=torch.float32, device=dev)
    if Z_seg is None:
        Z_seg = torch.empty(B, H, d.F, dtype=torch.float32, device=dev)
    _dev(S_seg, Z_seg)
    _check(lib.rehyat_segment_states(d, _dtype_code(k_seg), T, frame_tokens, Tc, To, c0, c1,
                                     _ptr(k_seg), _ptr(v_seg), _ptr(Wk), _ptr(bk), _ptr(S_seg),
                                     _ptr(Z_seg), _ptr(workspace), workspace.numel(),
                                     _stream(dev)))
    return S_seg, Z_seg


def segment_attend(q_seg, k_seg, v_seg, Wq, bq, *, T: int, c0: int, c1: int, P: int,
                   phi: int = 0, frame_tokens: int, Tc: int, To: int, workspace: torch.Tensor,
                   S_prefix: torch.Tensor | None = None, Z_prefix: torch.Tensor | None = None,
                   out: torch.Tensor | None = None) -> torch.Tensor:
    """Second phase: the segment's outputs.  S_prefix [n,B,H,F,D] / Z_prefix [n,B,H,F] stack
    the segment sums of every earlier segment (None for the first)."""
    lib = load()
    _check_x_w(q_seg, Wq, bq, "q_seg")
    s0, s1, h0 = segment_bounds(T, Tc, To, c0, c1)
    B, H, _, D = q_seg.shape
    F = Wq.shape[1] * Wq.shape[2]
    _shape(q_seg, (B, H, (s1 - s0) * frame_tokens, D), "q_seg")
    _shape(k_seg, (B, H, (s1 - h0) * frame_tokens, D), "k_seg")
    _shape(v_seg, k_seg.shape, "v_seg")
    _shape(out, q_seg.shape, "out")
    if S_prefix is not None:
        _shape(S_prefix, (S_prefix.shape[0], B, H, F, D), "S_prefix")
    if Z_prefix is not None:
        _shape(Z_prefix, (Z_prefix.shape[0], B, H, F), "Z_prefix")
    dev = _dev(q_seg, k_seg, v_seg, Wq, bq, workspace)
    d = dims_of(q_seg, Wq, P, phi)
    n_prefix = 0
    if (S_prefix is None) != (Z_prefix is None):
        raise ValueError("give both S_prefix and Z_prefix or neither")
    if S_prefix is not None:
        _dev(S_prefix, Z_prefix)
        n_prefix = S_prefix.shape[0]
        if S_prefix.dtype != torch.float32 or Z_prefix.dtype != torch.float32:
            raise ValueError("S_prefix/Z_prefix must be float32")
        if Z_prefix.shape[0] != n_prefix:
            raise ValueError("S_prefix and Z_prefix hold different segment counts")
    if out is None:
        out = torch.empty_like(q_seg)
    _dev(out)
    _check(lib.rehyat_segment_attend(d, _dtype_code(q_seg), T, frame_tokens, Tc, To, c0, c1,
                                     _ptr(q_seg), _ptr(k_seg), _ptr(v_seg), _ptr(Wq), _ptr(bq),
                                     n_prefix, _ptr(S_prefix), _ptr(Z_prefix), _ptr(out),
                                     _ptr(workspace), workspace.numel(), _stream(dev)))
    return out


def forward_states(k, v, Wk, bk, *, P: int, phi: int = 0, frame_tokens: int, Tc: int, To: int,
                   workspace: torch.Tensor) -> torch.Tensor:
    """First phase of `forward`: fills `workspace` with the state every chunk reads."""
    lib = load()
    _check_x_w(k, Wk, bk, "k")
    _shape(v, k.shape, "v")
    _frames(k.shape[2], frame_tokens, "k")
    dev = _dev(k, v, Wk, bk, workspace)
    d = dims_of(k, Wk, P, phi)
    T = k.shape[2] // frame_tokens
    _check(lib.rehyat_forward_states(d, _dtype_code(k), T, frame_tokens, Tc, To, _ptr(k), _ptr(v),
                                     _ptr(Wk), _ptr(bk), _ptr(workspace), workspace.numel(),
                                     _stream(dev)))
    return workspace


def forward_phiq(q, Wq, bq, *, P: int, phi: int = 0, frame_tokens: int, Tc: int, To: int,
                 workspace: torch.Tensor) -> torch.Tensor:
    """Second phase of `forward`: phi_q of the query rows that read a state, into `workspace`."""
    lib = load()
    _check_x_w(q, Wq, bq, "q")
    _frames(q.shape[2], frame_tokens, "q")
    dev = _dev(q, Wq, bq, workspace)
    d = dims_of(q, Wq, P, phi)
    T = q.shape[2] // frame_tokens
    _check(lib.rehyat_forward_phiq(d, _dtype_code(q), T, frame_tokens, Tc, To, _ptr(q), _ptr(Wq),
                                   _ptr(bq), _ptr(workspace), workspace.numel(), _stream(dev)))
    return workspace


def forward_attend(q, k, v, *, dims: Dims, frame_tokens: int, Tc: int, To: int,
                   workspace: torch.Tensor, out: torch.Tensor) -> torch.Tensor:
    """Third phase of `forward`: the hybrid output from q, k, v and the workspace."""
    lib = load()
    for t, n in ((k, "k"), (v, "v"), (out, "out")):
        _shape(t, q.shape, n)
    _frames(q.shape[2], frame_tokens, "q")
    dev = _dev(q, k, v, workspace, out)
    T = q.shape[2] // frame_tokens
    _check(lib.rehyat_forward_attend(dims, _dtype_code(q), T, frame_tokens, Tc, To, _ptr(q),
                                     _ptr(k), _ptr(v), _ptr(out), _ptr(workspace),
                                     workspace.numel(), _stream(dev)))
    return out


def chunk_states(k, v, Wk, bk, *, P: int, phi: int = 0, frame_tokens: int, Tc: int, To: int,
                 workspace: torch.Tensor | None = None):
    """States each chunk of `forward` reads: S [B,H,C,F,D], Z [B,H,C,F] (fp32)."""
    lib = load()
    _check_x_w(k, Wk, bk, "k")
    _shape(v, k.shape, "v")
    _frames(k.shape[2], frame_tokens, "k")
    dev = _dev(k, v, Wk, bk)
    d = dims_of(k, Wk, P, phi)
    N = k.shape[2]
    T = N // frame_tokens
    C = -(-T // Tc)
    code = _dtype_code(k)
    ws = _workspace(forward_workspace_size(d, code, T, frame_tokens, Tc, To), dev, workspace)
    S = torch.empty(d.B, d.H, C, d.F, d.D, dtype=torch.float32, device=dev)
    Z = torch.empty(d.B, d.H, C, d.F, dtype=torch.float32, device=dev)
    _check(lib.rehyat_chunk_states(d, code, T, frame_tokens, Tc, To, _ptr(k), _ptr(v), _ptr(Wk),
                                   _ptr(bk), _ptr(S), _ptr(Z), _ptr(ws), ws.numel(),
                                   _stream(dev)))
    return S, Z


def chunk_forward(q, k_win, v_win, Wq, bq, Wk, bk, S, Z, *, P: int, phi: int = 0, frame_tokens: int,
                  frames_before: int, To: int, To_next: int | None = None,
                  out: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """One streaming step; S [B,H,F,D] and Z [B,H,F] (fp32) are updated in place.  To_next (the
    overlap of the next call, for a variable schedule) defaults to To."""
    lib = load()
    cf = _frames(q.shape[2], frame_tokens, "q")
    _check_step(q, k_win, v_win, Wq, bq, Wk, bk, S, Z, out, frame_tokens,
                min(To, frames_before) + cf, "k_win")
    dev = _dev(q, k_win, v_win, Wq, bq, Wk, bk, S, Z)
    d = dims_of(q, Wq, P, phi)
    chunk_frames = q.shape[2] // frame_tokens
    code = _dtype_code(q)
    ws = _workspace(chunk_workspace_size(d, code, frame_tokens, chunk_frames, To), dev, workspace)
    if out is None:
        out = torch.empty_like(q)
    args = (_ptr(q), _ptr(k_win), _ptr(v_win), _ptr(Wq), _ptr(bq), _ptr(Wk), _ptr(bk), _ptr(S),
            _ptr(Z), _ptr(out), _ptr(ws), ws.numel(), _stream(dev))
    if To_next is None:
        _check(lib.rehyat_chunk_forward(d, code, frame_tokens, frames_before, chunk_frames, To,
                                        *args))
    else:
        _check(lib.rehyat_chunk_forward_sched(d, code, frame_tokens, frames_before, chunk_frames,
                                              To, To_next, *args))
    return out


def chunk_carry_workspace_size(d: Dims, dtype_code: int, L_: int, chunk_frames: int, To: int,
                               carry_frames: int) -> int:
    n = ctypes.c_size_t(0)
    _check(load().rehyat_chunk_carry_workspace_size(d, dtype_code, L_, chunk_frames, To,
                                                    carry_frames, ctypes.byref(n)))
    return n.value


def chunk_forward_carry(q, k, v, Wq, bq, Wk, bk, S, Z, k_carry, v_carry, *, P: int, phi: int = 0,
                        frame_tokens: int, frames_before: int, To: int,
                        To_next: int | None = None, out: torch.Tensor | None = None,
                        workspace: torch.Tensor | None = None):
    """Streaming step on the chunk alone; S, Z and the carried frames k_carry, v_carry
    [B,H,carry_frames*L,D] are updated in place."""
    lib = load()
    _check_step(q, k, v, Wq, bq, Wk, bk, S, Z, out, frame_tokens, None, "k")
    _frames(k_carry.shape[2], frame_tokens, "k_carry")
    _shape(k_carry, (q.shape[0], q.shape[1], k_carry.shape[2], q.shape[3]), "k_carry")
    _shape(v_carry, k_carry.shape, "v_carry")
    dev = _dev(q, k, v, Wq, bq, Wk, bk, S, Z, k_carry, v_carry)
    d = dims_of(q, Wq, P, phi)
    chunk_frames = q.shape[2] // frame_tokens
    carry_frames = k_carry.shape[2] // frame_tokens
    code = _dtype_code(q)
    ws = _workspace(chunk_carry_workspace_size(d, code, frame_tokens, chunk_frames, To,
                                               carry_frames), dev, workspace)
    if out is None:
        out = torch.empty_like(q)
    _check(lib.rehyat_chunk_forward_carry(d, code, frame_tokens, frames_before, chunk_frames, To,
                                          To if To_next is None else To_next, carry_frames,
                                          _ptr(q), _ptr(k), _ptr(v), _ptr(Wq), _ptr(bq),
                                          _ptr(Wk), _ptr(bk), _ptr(S), _ptr(Z), _ptr(k_carry),
                                          _ptr(v_carry), _ptr(out), _ptr(ws), ws.numel(),
                                          _stream(dev)))
    return out


def chunk_forward_static(q, k_win, v_win, Wq, bq, Wk, bk, S, Z, *, P: int, phi: int = 0, frame_tokens: int,
                         frames_before: int, To: int, out: torch.Tensor | None = None):
    """chunk_forward without a workspace: the library's own fixed device scratch is used (for
    callers that cannot allocate); bf16 only."""
    lib = load()
    cf = _frames(q.shape[2], frame_tokens, "q")
    _check_step(q, k_win, v_win, Wq, bq, Wk, bk, S, Z, out, frame_tokens,
                min(To, frames_before) + cf, "k_win")
    dev = _dev(q, k_win, v_win, Wq, bq, Wk, bk, S, Z)
    d = dims_of(q, Wq, P, phi)
    chunk_frames = q.shape[2] // frame_tokens
    if out is None:
        out = torch.empty_like(q)
    _check(lib.rehyat_chunk_forward_static(d, _dtype_code(q), frame_tokens, frames_before,
                                           chunk_frames, To, _ptr(q), _ptr(k_win), _ptr(v_win),
                                           _ptr(Wq), _ptr(bq), _ptr(Wk), _ptr(bk), _ptr(S),
                                           _ptr(Z), _ptr(out), _stream(dev)))
    return out


def forward_train(q, k, v, Wq, bq, Wk, bk, *, P: int, phi: int = 0, frame_tokens: int, Tc: int,
                  To: int, out: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """`forward` that also returns lse [B,H,N] fp32 (log2 of every row's denominator), which
    `backward` needs.  bf16 only."""
    lib = load()
    _check_x_w(q, Wq, bq, "q")
    _check_x_w(q, Wk, bk, "q")
    _shape(Wk, Wq.shape, "Wk")
    for t, n in ((k, "k"), (v, "v"), (out, "out")):
        _shape(t, q.shape, n)
    _frames(q.shape[2], frame_tokens, "q")
    dev = _dev(q, k, v, Wq, bq, Wk, bk)
    _weights(Wq, bq), _weights(Wk, bk)
    d = dims_of(q, Wq, P, phi)
    N = q.shape[2]
    T = N // frame_tokens
    code = _dtype_code(q)
    ws = _workspace(forward_workspace_size(d, code, T, frame_tokens, Tc, To), dev, workspace)
    if out is None:
        out = torch.empty_like(q)
    lse = torch.empty(q.shape[0], q.shape[1], N, dtype=torch.float32, device=dev)
    _check(lib.rehyat_forward_train(d, code, T, frame_tokens, Tc, To, _ptr(q), _ptr(k), _ptr(v),
                                    _ptr(Wq), _ptr(bq), _ptr(Wk), _ptr(bk), _ptr(out), _ptr(lse),
                                    _ptr(ws), ws.numel(), _stream(dev)))
    return out, lse


def backward_workspace_size(d: Dims, dtype_code: int, T: int, L_: int, Tc: int, To: int) -> int:
    n = ctypes.c_size_t(0)
    _check(load().rehyat_backward_workspace_size(d, dtype_code, T, L_, Tc, To, ctypes.byref(n)))
    return n.value


GRAD_NAMES = ("dq", "dk", "dv", "dWq", "dbq", "dWk", "dbk")


def backward(q, k, v, Wq, bq, Wk, bk, out, lse, dout, *, P: int, phi: int = 0,
             frame_tokens: int, Tc: int, To: int, workspace: torch.Tensor | None = None,
             grads: dict | None = None) -> dict:
    """Gradients of sum(dout * out) for every input: dict with dq, dk, dv [B,H,N,D], dWq, dWk
    [H,G,F/G,D/G], dbq, dbk [H,F] (fp32).  `grads` may hold those buffers (written, not added
    to)."""
    lib = load()
    _check_x_w(q, Wq, bq, "q")
    _check_x_w(q, Wk, bk, "q")
    _shape(Wk, Wq.shape, "Wk")
    for t, n in ((k, "k"), (v, "v"), (out, "out"), (dout, "dout")):
        _shape(t, q.shape, n)
    _shape(lse, q.shape[:3], "lse")
    _frames(q.shape[2], frame_tokens, "q")
    dev = _dev(q, k, v, Wq, bq, Wk, bk, out, lse, dout)
    d = dims_of(q, Wq, P, phi)
    N = q.shape[2]
    T = N // frame_tokens
    code = _dtype_code(q)
    ws = _workspace(backward_workspace_size(d, code, T, frame_tokens, Tc, To), dev, workspace)
    shapes = {"dq": q.shape, "dk": q.shape, "dv": q.shape, "dWq": Wq.shape, "dWk": Wk.shape,
              "dbq": (d.H, d.F), "dbk": (d.H, d.F)}
    g = {}
    for n in GRAD_NAMES:
        t = grads.get(n) if grads is not None else None
        if t is None:
            t = torch.empty(shapes[n], dtype=torch.float32, device=dev)
        elif tuple(t.shape) != tuple(shapes[n]) or t.dtype != torch.float32:
            raise ValueError(f"grads[{n!r}] must be float32 of shape {tuple(shapes[n])}")
        g[n] = t
    _dev(*g.values())
    _check(lib.rehyat_backward(d, code, T, frame_tokens, Tc, To, _ptr(q), _ptr(k), _ptr(v),
                               _ptr(Wq), _ptr(bq), _ptr(Wk), _ptr(bk), _ptr(out), _ptr(lse),
                               _ptr(dout), _ptr(g["dq"]), _ptr(g["dk"]), _ptr(g["dv"]),
                               _ptr(g["dWq"]), _ptr(g["dbq"]), _ptr(g["dWk"]), _ptr(g["dbk"]),
                               _ptr(ws), ws.numel(), _stream(dev)))
    return g


def gemm(A: torch.Tensor, B: torch.Tensor, *, a_mn: bool = False, b_mn: bool = False,
         out: torch.Tensor | None = None, accumulate: bool = False, alpha: float = 1.0,
         out_dtype: torch.dtype = torch.float32) -> torch.Tensor:
    """Batched bf16 GEMM on the tensor cores.  A [batch, M, K] (or [batch, K, M] with a_mn),
    B [batch, N, K] (or [batch, K, N] with b_mn), both contiguous bf16; returns C [batch, M, N]
    = alpha A B (added to `out` with accumulate)."""
    dev = _dev(A, B)
    batch = A.shape[0]
    M, K = (A.shape[2], A.shape[1]) if a_mn else (A.shape[1], A.shape[2])
    N = B.shape[2] if b_mn else B.shape[1]
    if out is None:
        out = torch.empty(batch, M, N, dtype=out_dtype, device=dev)
    _check(load().rehyat_gemm_bf16(M, N, K, batch, _ptr(A), A.shape[2], A.shape[1] * A.shape[2],
                                   int(a_mn), _ptr(B), B.shape[2], B.shape[1] * B.shape[2],
                                   int(b_mn), _ptr(out), out.shape[2], out.shape[1] * out.shape[2],
                                   int(out.dtype == torch.bfloat16), int(accumulate),
                                   ctypes.c_float(alpha), _stream(dev)))
    return out


def selftest_bounds(buf: torch.Tensor, n: int, bad_index: int) -> None:
    """Enqueue the debug-bounds self test on buf (fp32, at least n + 1 elements past which
    bad_index must stay)."""
    if buf.dtype != torch.float32 or buf.numel() <= max(n, bad_index):
        raise ValueError("buf must be fp32 with room for index max(n, bad_index)")
    dev = _dev(buf)
    _check(load().rehyat_selftest_bounds(_ptr(buf), n, bad_index, _stream(dev)))


def selftest_wait_timeout(limit_ns: int = 20_000_000, device: torch.device | None = None) -> None:
    """Enqueue the bounded-wait failure self test; the next sync_status() then raises
    RehyatError with status REHYAT_ERR_TIMEOUT."""
    dev = device or torch.device("cuda", torch.cuda.current_device())
    _check(load().rehyat_selftest_wait_timeout(ctypes.c_longlong(int(limit_ns)), _stream(dev)))


def sync_status(device: torch.device | None = None) -> None:
    """Synchronise the current stream and raise if a kernel reported a device-side failure."""
    dev = device or torch.device("cuda", torch.cuda.current_device())
    _check(load().rehyat_sync_status(_stream(dev)))


# ---- rotary positions and linear attention with a decay per head ----
# These calls read tensors by their strides: [B, heads, N, D] with contiguous rows of D, so a
# transposed [B, N, heads, D] projection or a slice of a packed qkv needs no copy.

# (a step is host-bound: these checks are a third of its time, so each compares once and leaves the
# reason to _refuse)
def _rows(t: torch.Tensor, dtype: torch.dtype, index: int, shape, what: str):
    """(pointer, strides of sequence, head and row) of a tensor of rows of this type and shape on
    CUDA device `index`."""
    b, h, n, d = t.stride()
    if d != 1 or t.dtype is not dtype or t.get_device() != index or t.shape != shape:
        _refuse(t, dtype, index, shape, what)
        if shape[3] > 1:
            raise ValueError(f"{what}: the last dimension must be contiguous")
    return t.data_ptr(), b, h, n


def _small(t: torch.Tensor, dtype: torch.dtype, index: int, shape, what: str) -> int:
    """Pointer of a contiguous tensor of this type and shape."""
    if t.dtype is not dtype or t.get_device() != index or t.shape != shape or \
            not t.is_contiguous():
        _refuse(t, dtype, index, shape, what)
        raise ValueError(f"{what} must be contiguous")
    return t.data_ptr()


def _refuse(t, dtype, index, shape, what) -> None:
    if t.get_device() != index:
        raise ValueError("all tensors must be on the same CUDA device")
    if t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{what} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _typed(t: torch.Tensor):
    """(dtype, its library code, device index) of the tensor that the others must match."""
    dtype, index = t.dtype, t.get_device()
    if dtype is torch.bfloat16:
        code = REHYAT_BF16
    elif dtype is torch.float32:
        code = REHYAT_F32
    else:
        raise TypeError(f"unsupported dtype {dtype}")
    return dtype, code, index


# (torch.cuda.current_stream builds a Stream object: 2 us of a step's 10)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _scratch(nbytes: int, dev: torch.device, workspace: torch.Tensor | None) -> torch.Tensor:
    if workspace is not None and (workspace.device != dev or workspace.dtype != torch.uint8 or
                                  not workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous uint8 tensor on the tensors' device")
    return _workspace(nbytes, dev, workspace)


def _call(index: int, fn, block: bytes) -> None:
    """Enqueue a library call on the current stream of CUDA device `index`, whichever device is the
    current one."""
    if index < 0:
        raise ValueError("all tensors must be on the same CUDA device")
    if torch.cuda.current_device() == index:
        status = fn(block, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            status = fn(block, _raw_stream(index))
    if status:
        _check(status)


# A tensor of the caller's that a call wrote to: a graph that saved it for its backward pass then says
# so there, instead of taking the new values for the old.
_wrote = torch.autograd.graph.increment_version


def _four(t: torch.Tensor, what: str):
    shape = t.shape
    if len(shape) != 4:
        raise ValueError(f"{what} must be [B, heads, N, D], got {tuple(shape)}")
    return shape


def rotary_frequencies(R: int, *, base: float = 10000.0, scaling: str | None = None,
                       factor: float = 1.0, original_length: int | None = None,
                       turns: tuple[float, float] = (32.0, 1.0),
                       device: torch.device | None = None) -> tuple[torch.Tensor, float]:
    """(freq, scale) for `rotary`: radians per position of the R/2 pairs (fp64), base^(-2p/R), and
    the factor on the rotated values.  A context stretched by `factor`:
      scaling "linear": every frequency divided by the factor;
      scaling "ntk":    the base times factor^(R/(R-2)), so the slowest pair stretches by the
                        factor and the fastest not at all;
      scaling "yarn":   pairs that make at least turns[0] turns over `original_length` positions are
                        kept, those with at most turns[1] divided by the factor, a linear ramp over
                        the pair index between (from pair 0 at the earliest); values times
                        0.1 ln(factor) + 1."""
    if R < 2 or R % 2:
        raise ValueError(f"R={R} must be even and positive")
    if not factor >= 1.0 or not base > 1.0:
        raise ValueError(f"need factor >= 1 and base > 1 (factor={factor}, base={base})")
    scale = 1.0
    if scaling == "ntk":
        if R == 2:
            raise ValueError("scaling 'ntk' needs R > 2")
        base = base * factor ** (R / (R - 2))
    p = torch.arange(R // 2, dtype=torch.float64)
    freq = base ** (-2.0 * p / R)
    if scaling == "linear":
        freq = freq / factor
    elif scaling == "yarn":
        if original_length is None or original_length < 1 or not turns[0] > turns[1] > 0:
            raise ValueError("scaling 'yarn' needs original_length and turns[0] > turns[1] > 0")
        lo, hi = (R * math.log(original_length / (t * 2 * math.pi)) / (2 * math.log(base))
                  for t in turns)
        lo, hi = max(math.floor(lo), 0), min(math.ceil(hi), R - 1)
        # (hi <= 0: no pair makes more than turns[1] turns)
        keep = 1 - ((p - lo) / max(hi - lo, 1e-3)).clamp(0, 1) if hi > 0 else torch.zeros_like(p)
        freq = freq * keep + freq / factor * (1 - keep)
        scale = 0.1 * math.log(factor) + 1.0
    elif scaling not in (None, "ntk"):
        raise ValueError(f"unknown scaling {scaling!r}")
    return freq.to(device), scale


def rotary_axes(pairs: tuple[int, ...], device: torch.device | None = None) -> torch.Tensor:
    """The `axis` argument of `rotary`: the first pairs[0] pairs turn by axis 0, the next pairs[1]
    by axis 1, and so on."""
    return torch.repeat_interleave(torch.arange(len(pairs), dtype=torch.uint8),
                                   torch.tensor(pairs)).to(device)


def video_positions(T: int, frame_h: int, frame_w: int, *, first_frame: int = 0,
                    device: torch.device | None = None) -> torch.Tensor:
    """positions [3, 1, T*frame_h*frame_w] (frame, row, column) of a frame-major token sequence;
    expand the middle dimension to the batch."""
    i = torch.arange(T * frame_h * frame_w, device=device)
    L = frame_h * frame_w
    return torch.stack((first_frame + i // L, i // frame_w % frame_h, i % frame_w))[:, None].to(
        torch.int32)


def rotary(q: torch.Tensor, k: torch.Tensor | None, freq: torch.Tensor, *,
           positions: torch.Tensor | None = None, start=0, axis: torch.Tensor | None = None,
           scale: float = 1.0, interleaved: bool = False, inverse: bool = False,
           q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None):
    """Rotary positions for q [B,H,n,D] and k [B,Hk,n,D] (or None) in one launch: dimension pairs
    of the first R = 2 len(freq) dimensions turn by position * freq[pair] and are scaled by `scale`;
    the rest is copied.  Pairs are (p, p + R/2), or (2p, 2p + 1) when interleaved.

    Token i of sequence b has position positions[b, i] ([B, n]) or, pair by pair,
    positions[axis[pair], b, i] ([A, B, n], axis [R/2] uint8); without `positions`, i.  `start` (an
    int, or without `positions` an int32/int64 tensor [B] on the device) is added.  Positions are
    int32 or int64 tensors of any strides; an axis past the last counts as the last.

    inverse turns the other way: with the same arguments it is the gradient of this call.  Returns
    q_out, or (q_out, k_out); they may be q and k (in place)."""
    lib = _lib or load()
    B, H, n, D = shape = _four(q, "q")
    dtype, code, index = _typed(q)
    qa = _rows(q, dtype, index, shape, "q")
    half = freq.numel()
    fp = _small(freq, torch.float64, index, (half,), "freq")
    pos, axes, add, pa, pb, pn = positions, 1, 0, 0, 0, 0
    if isinstance(start, torch.Tensor):
        if positions is not None:
            raise ValueError("give positions or a start tensor, not both")
        if start.shape != (B,):
            raise ValueError(f"start must have shape {(B,)}, got {tuple(start.shape)}")
        pos, pb, add, start = start, start.stride(0), 1, 0
    elif positions is None:
        add = 1
    elif positions.shape == (B, n):
        pb, pn = positions.stride()
    elif positions.dim() == 3 and positions.shape[1:] == (B, n):
        axes, (pa, pb, pn) = positions.shape[0], positions.stride()
    else:
        raise ValueError(f"positions must have shape {(B, n)} or (axes, {B}, {n}), got "
                         f"{tuple(positions.shape)}")
    pp = pos64 = 0
    if pos is not None:
        pos64 = pos.dtype is torch.int64
        if not pos64 and pos.dtype is not torch.int32:
            raise TypeError(f"positions must be int32 or int64, got {pos.dtype}")
        if pos.get_device() != index:
            raise ValueError("all tensors must be on the same CUDA device")
        pp = pos.data_ptr()
    ap = 0 if axis is None else _small(axis, torch.uint8, index, (half,), "axis")
    given = [t for t in (q_out, k_out) if t is not None]
    Hk, ka, ko = 0, _NO_ROWS, _NO_ROWS
    if k is not None:
        Hk = _four(k, "k")[1]
        ka = _rows(k, dtype, index, (B, Hk, n, D), "k")
        if k_out is None:
            k_out = torch.empty_like(k)
        ko = _rows(k_out, dtype, index, k.shape, "k_out")
    if q_out is None:
        q_out = torch.empty_like(q)
    qo = _rows(q_out, dtype, index, shape, "q_out")
    _call(index, lib.rehyat_rotary, _ROTARY.pack(
        B, n, H, Hk, D, 2 * half, interleaved, inverse, axes, pos64, add, code, pa, pb, pn, start,
        fp, ap, pp, *qa, *ka, *qo, *ko, scale))
    if given:
        _wrote(given)
    return q_out if k is None else (q_out, k_out)


_NO_ROWS = (0, 0, 0, 0)


def _decay_sizes(q, k):
    B, H, N, D = _four(q, "q")
    Hk = _four(k, "k")[1]
    if Hk < 1 or H % Hk:
        raise ValueError(f"k's {Hk} heads must divide q's {H}")
    return B, H, Hk, N, D


@functools.lru_cache(maxsize=1024)
def decay_workspace_size(B: int, H: int, Hk: int, N: int, D: int, backward: bool = False) -> int:
    """Bytes of scratch that decay_forward (or decay_backward) needs for these sizes."""
    n = ctypes.c_size_t(0)
    _check(load().rehyat_decay_workspace_size(B, H, Hk, N, D, int(backward), ctypes.byref(n)))
    return n.value


def decay_forward(q, k, v, log_decay, *, scale: float = 1.0, lengths: torch.Tensor | None = None,
                  state: torch.Tensor | None = None, final_state: bool | torch.Tensor = False,
                  out: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """Linear attention with a decay L = exp(log_decay[h]) per head over a whole prompt:
      out_i = scale * (sum_{j<=i} L^(i-j) (q_i . k_j) v_j + L^(i+1) q_i state)
    q [B,H,N,D]; k, v [B,Hk,N,D] (H a multiple of Hk; query head h reads key/value head
    h // (H/Hk)); bf16 or fp32; D a multiple of 8 up to 128; log_decay [H] fp32, constants <= 0.
    lengths [B] int32: sequence b is its first lengths[b] rows, the others are padding (not read
    into any result, zero in the output).  state [B,H,D,D] fp32: from the rows before.
    final_state True: returns (out, the state after the last row [B,H,D,D] fp32), which
    `decay_step` or the next call goes on from; a tensor: written there (it may be `state`).  In bf16
    asking for it changes the last bits of `out` (the sums between segments are then finer).
    Tensors of rows may have any strides of at least D and whole 16 bytes (none expanded); an output
    that overlaps itself or another argument is refused."""
    lib = _lib or load()
    B, H, Hk, N, D = _decay_sizes(q, k)
    dtype, code, index = _typed(q)
    shape, kv, square = q.shape, (B, Hk, N, D), (B, H, D, D)
    qa = _rows(q, dtype, index, shape, "q")
    ka, va = _rows(k, dtype, index, kv, "k"), _rows(v, dtype, index, kv, "v")
    gp = _small(log_decay, torch.float32, index, (H,), "log_decay")
    lp = 0 if lengths is None else _small(lengths, torch.int32, index, (B,), "lengths")
    sp = 0 if state is None else _small(state, torch.float32, index, square, "state")
    given = [] if out is None else [out]
    if out is None:
        out = torch.empty_like(q)
    oa = _rows(out, dtype, index, shape, "out")
    last, fp = None, 0
    if isinstance(final_state, torch.Tensor):
        last = final_state
        given.append(last)
        fp = _small(last, torch.float32, index, square, "final_state")
    elif final_state:
        last = torch.empty(square, dtype=torch.float32, device=q.device)
        fp = last.data_ptr()
    ws = _scratch(decay_workspace_size(B, H, Hk, N, D), q.device, workspace)
    _call(index, lib.rehyat_decay_forward, _DECAY_FORWARD.pack(
        B, H, Hk, N, D, code, *qa, *ka, *va, *oa, gp, lp, sp, fp, ws.data_ptr(), ws.numel(), scale))
    if given:
        _wrote(given)
    return out if last is None else (out, last)


def decay_backward(q, k, v, log_decay, dout, *, scale: float = 1.0,
                   lengths: torch.Tensor | None = None, state: torch.Tensor | None = None,
                   dfinal: torch.Tensor | None = None,
                   workspace: torch.Tensor | None = None) -> dict:
    """Gradients of sum(dout * out) + sum(dfinal * final state) of `decay_forward`: dict with dq
    [B,H,N,D], dk, dv [B,Hk,N,D] (the inputs' type; dk and dv summed over the query heads that share
    them; zero on padding) and, with `state`, dstate [B,H,D,D] fp32.  dout [B,H,N,D]; dfinal
    [B,H,D,D] fp32 or None (zero)."""
    lib = _lib or load()
    B, H, Hk, N, D = _decay_sizes(q, k)
    dtype, code, index = _typed(q)
    shape, kv, square = q.shape, (B, Hk, N, D), (B, H, D, D)
    qa = _rows(q, dtype, index, shape, "q")
    ka, va = _rows(k, dtype, index, kv, "k"), _rows(v, dtype, index, kv, "v")
    doa = _rows(dout, dtype, index, shape, "dout")
    gp = _small(log_decay, torch.float32, index, (H,), "log_decay")
    lp = 0 if lengths is None else _small(lengths, torch.int32, index, (B,), "lengths")
    sp = 0 if state is None else _small(state, torch.float32, index, square, "state")
    fp = 0 if dfinal is None else _small(dfinal, torch.float32, index, square, "dfinal")
    g = {"dq": torch.empty_like(q), "dk": torch.empty_like(k), "dv": torch.empty_like(v)}
    if state is not None:
        g["dstate"] = torch.empty(square, dtype=torch.float32, device=q.device)
    ws = _scratch(decay_workspace_size(B, H, Hk, N, D, True), q.device, workspace)
    _call(index, lib.rehyat_decay_backward, _DECAY_BACKWARD.pack(
        B, H, Hk, N, D, code, *qa, *ka, *va, *doa, *_rows(g["dq"], dtype, index, shape, "dq"),
        *_rows(g["dk"], dtype, index, kv, "dk"), *_rows(g["dv"], dtype, index, kv, "dv"), gp, lp,
        sp, fp, g["dstate"].data_ptr() if state is not None else 0, ws.data_ptr(), ws.numel(),
        scale))
    return g


def decay_step(q, k, v, log_decay, state, *, scale: float = 1.0,
               slots: torch.Tensor | None = None, out: torch.Tensor | None = None):
    """One token of every sequence: state <- L state + k v^T (in place), out = scale * q state.
    q [B,H,1,D]; k, v [B,Hk,1,D]; state [pool,H,D,D] fp32.  slots [B] int32: sequence b's state
    is state[slots[b]] (without slots: state[b], pool = B); a negative slot is an idle entry (zero
    output, no state touched); a slot listed several times takes its tokens in batch order; one past
    the pool gives zeros and is reported by `sync_status`."""
    lib = _lib or load()
    B, H, Hk, N, D = _decay_sizes(q, k)
    if N != 1:
        raise ValueError(f"a step takes one token of each sequence, got {N}")
    dtype, code, index = _typed(q)
    shape, kv = q.shape, (B, Hk, 1, D)
    pool = state.shape[0] if slots is not None and state.dim() == 4 else B
    qa = _rows(q, dtype, index, shape, "q")
    ka, va = _rows(k, dtype, index, kv, "k"), _rows(v, dtype, index, kv, "v")
    gp = _small(log_decay, torch.float32, index, (H,), "log_decay")
    sp = _small(state, torch.float32, index, (pool, H, D, D), "state")
    lp = 0 if slots is None else _small(slots, torch.int32, index, (B,), "slots")
    given = state if out is None else (state, out)
    if out is None:
        out = torch.empty_like(q)
    _call(index, lib.rehyat_decay_step, _DECAY_STEP.pack(
        B, H, Hk, D, pool, code, *qa, *ka, *va, *_rows(out, dtype, index, shape, "out"), gp, sp, lp,
        scale))
    _wrote(given)
    return out
