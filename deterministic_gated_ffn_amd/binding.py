"""Python binding of libdgf (include/dgf.h): argument marshalling only.

Every step of the path runs in the HIP library; this module turns torch
tensors into device pointers, leading dimensions and the current HIP stream,
allocates outputs and the workspace the library asks for, and raises on any
non-OK status.  There is no fallback: without the built library (or without a
GPU) every call raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from typing import NamedTuple

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libdgf.so")
_lib = None

DGF_NT, DGF_NN, DGF_TN = 0, 1, 2
_LAYOUTS = {"NT": DGF_NT, "NN": DGF_NN, "TN": DGF_TN}

STATUS = {0: "DGF_OK", 1: "DGF_EINVAL", 2: "DGF_EUNSUPPORTED", 3: "DGF_EWORKSPACE", 4: "DGF_EHIP"}

# (name, restype, argtypes) of every exported entry point
_P, _I64, _SZ, _I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int
_F = ctypes.c_float
SIGNATURES = {
    "dgf_abi_version": (_I, []),
    "dgf_leaf_size": (_I, []),
    "dgf_last_error": (ctypes.c_char_p, []),
    "dgf_ffn_fwd_workspace": (_SZ, [_I64, _I64, _I64]),
    "dgf_ffn_fwd": (_I, [_P, _I64, _P, _I64, _P, _I64, _P, _I64, _P, _I64, _P, _P, _I64,
                         _I64, _I64, _I64, _P, _SZ, _P]),
    "dgf_ffn_fwd_static": (_I, [_P, _I64, _P, _I64, _P, _I64, _P, _I64, _P, _I64, _P, _P, _I64,
                                _I64, _I64, _I64, _P]),
    "dgf_ffn_bwd_workspace": (_SZ, [_I64, _I64, _I64]),
    "dgf_ffn_bwd": (_I, [_P, _I64, _P, _I64, _P, _P, _I64, _P, _I64, _P, _I64, _P, _I64,
                         _P, _P, _P, _I64, _P, _I64, _P, _I64, _P, _I64,
                         _I64, _I64, _I64, _P, _SZ, _P]),
    "dgf_tree_combine": (_I, [ctypes.POINTER(_P), _I, _P, _I64, _P]),
    "dgf_tree_combine_typed": (_I, [ctypes.POINTER(_P), _I, _P, _I64, _I, _P]),
    "dgf_gemm_tree_workspace": (_SZ, [_I, _I64, _I64, _I64]),
    "dgf_gemm_tree": (_I, [_I, _P, _I64, _P, _I64, _P, _I64, _I64, _I64, _I64, _P, _SZ, _P]),
    "dgf_act_fwd": (_I, [_P, _P, _P, _I64, _P]),
    "dgf_act_bwd": (_I, [_P, _P, _P, _P, _P, _P, _I64, _P]),
    "dgf_ffn_fwd_typed": (_I, [_P, _I64, _P, _I64, _P, _I64, _P, _I64, _P, _I64, _P, _P, _I64,
                               _I64, _I64, _I64, _P, _SZ, _I, _P]),
    "dgf_ffn_bwd_typed": (_I, [_P, _I64, _P, _I64, _P, _P, _I64, _P, _I64, _P, _I64, _P, _I64,
                               _P, _P, _P, _I64, _P, _I64, _P, _I64, _P, _I64,
                               _I64, _I64, _I64, _P, _SZ, _I, _P]),
    "dgf_gemm_tree_typed": (_I, [_I, _P, _I64, _P, _I64, _P, _I64, _I64, _I64, _I64, _P, _SZ, _I, _P]),
    "dgf_act_fwd_typed": (_I, [_P, _P, _P, _I64, _I, _P]),
    "dgf_act_bwd_typed": (_I, [_P, _P, _P, _P, _P, _P, _I64, _I, _P]),
    "dgf_norm_fwd": (_I, [_P, _I64, _P, _I64, _P, _P, _I64, _F, _P, _F, _P, _I64, _P, _I64, _P, _I64, _I64, _I, _P]),
    "dgf_norm_bwd_workspace": (_SZ, [_I64, _I64]),
    "dgf_norm_bwd": (_I, [_P, _I64, _P, _I64, _P, _I64, _P, _I64, _P, _P, _I64, _F, _P, _P, _P, _I64, _P, _I64,
                          _P, _P, _I64, _P, _I64, _I64, _P, _SZ, _I, _P]),
    "dgf_pack8": (_I, [_P, _I64, _P, _I64, _P, _I64, _I64, _I64, _I, _P]),
    "dgf_unpack8": (_I, [_P, _I64, _P, _I64, _P, _I64, _I64, _I64, _I, _P]),
    "dgf_act_bwd_q8": (_I, [_P, _I64, _P, _P, _P, _P, _I64, _I64, _P, _P, _P, _I64, _I64, _I64, _I, _P]),
    "dgf_ffn_fwd_q8_workspace": (_SZ, [_I64, _I64, _I64]),
    "dgf_ffn_fwd_q8": (_I, [_P, _I64, _P, _I64, _P, _I64, _P, _I64, _P, _I64, _P, _P, _P, _P, _I64, _I64,
                            _I64, _I64, _I64, _P, _SZ, _I, _P]),
    "dgf_ffn_bwd_q8": (_I, [_P, _I64, _P, _I64, _P, _P, _P, _P, _I64, _I64, _P, _I64, _P, _I64, _P, _I64,
                            _P, _P, _P, _I64, _P, _I64, _P, _I64, _P, _I64,
                            _I64, _I64, _I64, _P, _SZ, _I, _P]),
    "dgf_moe_fwd_workspace": (_SZ, [_I64, _I64, _I64, _I64, _I64, _I64]),
    "dgf_moe_fwd": (_I, [_P, _I64, _P, _I64, _P, _I64, _I64, _P, _I64, _I64, _P, _I64, _I64, _P, _I64, _P, _P,
                         _I64, _I64, _I64, _I64, _I64, _I64, _I64, _I, _P, _SZ, _I, _P]),
    "dgf_profile_begin": (_I, [ctypes.POINTER(_P), _I]),
    "dgf_profile_end": (_I, []),
    "dgf_profile_name": (ctypes.c_char_p, [_I]),
}


class DgfError(RuntimeError):
    def __init__(self, status: int, where: str, msg: str):
        super().__init__(f"{where}: {STATUS.get(status, status)}: {msg}")
        self.status = status


def lib_path() -> str:
    return _LIB_PATH


def load() -> ctypes.CDLL:
    """Load libdgf.so; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(f"libdgf.so not built at {_LIB_PATH}: run `python -m deterministic_gated_ffn_amd.build`")
        L = ctypes.CDLL(_LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _check(status: int, where: str):
    if status != 0:
        raise DgfError(status, where, load().dgf_last_error().decode())


def _stream(stream=None) -> int:
    if stream is None:  # the handle alone: building a Stream object costs a small call's kernel time
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return stream.cuda_stream


_ON_CURRENT = contextlib.nullcontext()


def _on(stream):
    """Allocate on the launch stream: outputs and the workspace come from that
    stream's pool, so the caching allocator cannot hand a block to another
    stream while the launched kernels still use it."""
    return torch.cuda.stream(stream) if stream is not None else _ON_CURRENT


DGF_BF16, DGF_FP16, DGF_FP32 = 0, 1, 2
# stored types of the FFN and the tree GEMM: BF16 (the untyped entry points) or FP16
_STORED = {torch.bfloat16: DGF_BF16, torch.float16: DGF_FP16}


def _stored(*ts) -> int:
    """The dtype code shared by every given tensor (BF16 or FP16)."""
    dt = ts[0].dtype
    if dt not in _STORED:
        raise TypeError(f"expected bfloat16 or float16 tensors, got {dt}")
    for t in ts:
        if t.dtype != dt:
            raise TypeError(f"all tensors must share one dtype ({dt} and {t.dtype} given)")
    return _STORED[dt]


def _mat(t: torch.Tensor, name: str):
    """(pointer, leading dimension) of a row-major BF16 or FP16 matrix view on the GPU."""
    if t.dtype not in _STORED:
        raise TypeError(f"{name}: expected bfloat16 or float16, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name}: expected a GPU tensor")
    stride = t.stride()
    if len(stride) != 2 or stride[1] != 1:
        raise ValueError(f"{name}: expected a 2-D row-major view (stride(1) == 1)")
    return t.data_ptr(), stride[0]


def _empty(rows: int, cols: int, like: torch.Tensor, ld: int | None = None) -> torch.Tensor:
    """Row-major [rows, cols] of like's dtype whose leading dimension is a multiple of 8."""
    ld = ld or ((cols + 7) // 8) * 8
    if ld == cols:  # no padding: the cheapest allocation torch has
        return torch.empty_like(like) if like.shape == (rows, cols) and like.is_contiguous() else like.new_empty((rows, cols))
    return like.new_empty((rows, ld))[:, :cols]


def _workspace(nbytes: int, like: torch.Tensor) -> torch.Tensor:
    return like.new_empty(max(int(nbytes), 16), dtype=torch.uint8)


# ---------------------------------------------------------------- entry points
def abi_version() -> int:
    return load().dgf_abi_version()


def leaf_size() -> int:
    return load().dgf_leaf_size()


def ffn_fwd(x, w_gate, w_up, w_down, training: bool = False, out=None, stream=None):
    """y = W_down (silu(W_gate x) * (W_up x)) through the canonical tree, in the
    tensors' stored type (BF16: dgf_ffn_fwd, FP16: dgf_ffn_fwd_typed).
    Returns y, or (y, g, u) when training."""
    with _on(stream):
        return _ffn_fwd(x, w_gate, w_up, w_down, training, out, stream)


def _ffn_fwd(x, w_gate, w_up, w_down, training, out, stream):
    L = load()
    dt = _stored(x, w_gate, w_up, w_down, *([out] if out is not None else []))
    M, H = x.shape
    I = w_gate.shape[0]
    y = out if out is not None else _empty(M, H, x)
    g = u = None
    gp = up = None
    ld_gu = 0
    if training:
        g, u = _empty(M, I, x), _empty(M, I, x)
        gp, up, ld_gu = g.data_ptr(), u.data_ptr(), g.stride(0)
    ws = _workspace(L.dgf_ffn_fwd_workspace(M, H, I), x)
    xp, ldx = _mat(x, "x"); wg, ldwg = _mat(w_gate, "w_gate"); wu, ldwu = _mat(w_up, "w_up")
    wd, ldwd = _mat(w_down, "w_down"); yp, ldy = _mat(y, "y")
    if dt == DGF_BF16:
        _check(L.dgf_ffn_fwd(xp, ldx, wg, ldwg, wu, ldwu, wd, ldwd, yp, ldy, gp, up, ld_gu,
                             M, H, I, ws.data_ptr(), ws.numel(), _stream(stream)), "dgf_ffn_fwd")
    else:
        _check(L.dgf_ffn_fwd_typed(xp, ldx, wg, ldwg, wu, ldwu, wd, ldwd, yp, ldy, gp, up, ld_gu,
                                   M, H, I, ws.data_ptr(), ws.numel(), dt, _stream(stream)), "dgf_ffn_fwd_typed")
    return (y, g, u) if training else y


STATIC_SCRATCH_BYTES = 16 << 20  # DGF_STATIC_SCRATCH_BYTES


def ffn_fwd_static(x, w_gate, w_up, w_down, y, g=None, u=None, stream=None):
    """dgf_ffn_fwd_static: the forward into caller-given y (and g, u when
    training) with the library's own scratch; allocates nothing."""
    L = load()
    if (g is None) != (u is None):
        raise ValueError("give both g and u (training) or neither (inference)")
    if _stored(x, w_gate, w_up, w_down, y, *([g, u] if g is not None else [])) != DGF_BF16:
        raise TypeError("dgf_ffn_fwd_static takes bfloat16 tensors only")
    M, H = x.shape
    I = w_gate.shape[0]
    xp, ldx = _mat(x, "x"); wg, ldwg = _mat(w_gate, "w_gate"); wu, ldwu = _mat(w_up, "w_up")
    wd, ldwd = _mat(w_down, "w_down"); yp, ldy = _mat(y, "y")
    gp = up = None
    ld_gu = 0
    if g is not None:
        (gp, ld_gu), (up, ldu) = _mat(g, "g"), _mat(u, "u")
        if ldu != ld_gu:
            raise ValueError("g and u must share a leading dimension")
    _check(L.dgf_ffn_fwd_static(xp, ldx, wg, ldwg, wu, ldwu, wd, ldwd, yp, ldy, gp, up, ld_gu, M, H, I,
                                _stream(stream)), "dgf_ffn_fwd_static")
    return y


def ffn_bwd(dy, x, g, u, w_gate, w_up, w_down, lanes: bool = False, stream=None):
    """Returns dict dX, dW_gate, dW_up, dW_down (and G, U lanes if lanes=True),
    in the tensors' stored type (BF16: dgf_ffn_bwd, FP16: dgf_ffn_bwd_typed)."""
    with _on(stream):
        return _ffn_bwd(dy, x, g, u, w_gate, w_up, w_down, lanes, stream)


def _ffn_bwd(dy, x, g, u, w_gate, w_up, w_down, lanes, stream):
    L = load()
    dt = _stored(dy, x, g, u, w_gate, w_up, w_down)
    M, H = x.shape
    I = w_gate.shape[0]
    dx = _empty(M, H, x)
    gl = _empty(M, H, x, ld=dx.stride(0)) if lanes else None
    ul = _empty(M, H, x, ld=dx.stride(0)) if lanes else None
    dwg, dwu, dwd = _empty(I, H, x), _empty(I, H, x), _empty(H, I, x)
    ws = _workspace(L.dgf_ffn_bwd_workspace(M, H, I), x)
    dyp, lddy = _mat(dy, "dy"); xp, ldx = _mat(x, "x"); gp, ldg = _mat(g, "g"); upp, ldu = _mat(u, "u")
    if ldg != ldu:
        raise ValueError("g and u must share a leading dimension")
    wg, ldwg = _mat(w_gate, "w_gate"); wu, ldwu = _mat(w_up, "w_up"); wd, ldwd = _mat(w_down, "w_down")
    args = (dyp, lddy, xp, ldx, gp, upp, ldg, wg, ldwg, wu, ldwu, wd, ldwd,
            dx.data_ptr(), gl.data_ptr() if lanes else None, ul.data_ptr() if lanes else None,
            dx.stride(0), dwg.data_ptr(), dwg.stride(0), dwu.data_ptr(), dwu.stride(0),
            dwd.data_ptr(), dwd.stride(0), M, H, I, ws.data_ptr(), ws.numel())
    if dt == DGF_BF16:
        _check(L.dgf_ffn_bwd(*args, _stream(stream)), "dgf_ffn_bwd")
    else:
        _check(L.dgf_ffn_bwd_typed(*args, dt, _stream(stream)), "dgf_ffn_bwd_typed")
    r = {"dX": dx, "dW_gate": dwg, "dW_up": dwu, "dW_down": dwd}
    if lanes:
        r["G"], r["U"] = gl, ul
    return r


_COMBINE_DTYPES = {torch.bfloat16: DGF_BF16, torch.float16: DGF_FP16, torch.float32: DGF_FP32}


def tree_combine(parts, out=None, stream=None):
    """Balanced combine of S in {1,2,4,8} equally sized tensors (rank order);
    BF16, FP16 or FP32, all parts of one dtype."""
    with _on(stream):
        return _tree_combine(parts, out, stream)


def _tree_combine(parts, out, stream):
    L = load()
    parts = list(parts)
    n = parts[0].numel()
    dt = parts[0].dtype
    if dt not in _COMBINE_DTYPES:
        raise ValueError(f"tree_combine takes bfloat16, float16 or float32, not {dt}")
    for t in parts:
        if t.dtype != dt or not t.is_cuda or t.numel() != n or not t.is_contiguous():
            raise ValueError("parts must be contiguous GPU tensors of one dtype and size")
    out = out if out is not None else torch.empty_like(parts[0])
    arr = (ctypes.c_void_p * len(parts))(*[t.data_ptr() for t in parts])
    if dt == torch.bfloat16:
        _check(L.dgf_tree_combine(arr, len(parts), out.data_ptr(), n, _stream(stream)), "dgf_tree_combine")
    else:
        _check(L.dgf_tree_combine_typed(arr, len(parts), out.data_ptr(), n, _COMBINE_DTYPES[dt], _stream(stream)),
               "dgf_tree_combine_typed")
    return out


def tree_combine_ptrs(ptrs, S: int, out_ptr: int, n: int, stream=None, dtype: int = DGF_BF16):
    """Raw-pointer form (offset or unaligned views)."""
    L = load()
    arr = (ctypes.c_void_p * len(ptrs))(*ptrs)
    _check(L.dgf_tree_combine_typed(arr, S, out_ptr, n, dtype, _stream(stream)), "dgf_tree_combine_typed")


def gemm_tree(layout: str, A, B, out=None, stream=None):
    """NT: A [M,K], B [N,K]; NN: A [M,K], B [K,N]; TN: A [K,M], B [K,N] -> C [M,N],
    in the operands' stored type (BF16: dgf_gemm_tree, FP16: dgf_gemm_tree_typed)."""
    with _on(stream):
        return _gemm_tree(layout, A, B, out, stream)


def _gemm_tree(layout, A, B, out, stream):
    L = load()
    dt = _stored(A, B, *([out] if out is not None else []))
    lay = _LAYOUTS[layout]
    if layout == "NT":
        (M, K), N = A.shape, B.shape[0]
    elif layout == "NN":
        (M, K), N = A.shape, B.shape[1]
    else:
        (K, M), N = A.shape, B.shape[1]
    C = out if out is not None else _empty(M, N, A)
    ws = _workspace(L.dgf_gemm_tree_workspace(lay, M, N, K), A)
    ap, lda = _mat(A, "A"); bp, ldb = _mat(B, "B"); cp, ldc = _mat(C, "C")
    if dt == DGF_BF16:
        _check(L.dgf_gemm_tree(lay, ap, lda, bp, ldb, cp, ldc, M, N, K, ws.data_ptr(), ws.numel(), _stream(stream)),
               "dgf_gemm_tree")
    else:
        _check(L.dgf_gemm_tree_typed(lay, ap, lda, bp, ldb, cp, ldc, M, N, K, ws.data_ptr(), ws.numel(), dt,
                                     _stream(stream)), "dgf_gemm_tree_typed")
    return C


def _flat(t: torch.Tensor, name: str) -> int:
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous GPU tensor")
    return t.data_ptr()


def act_fwd(g, u, stream=None):
    """a = rnd(silu(g) u) elementwise in the stored type of g and u."""
    L = load()
    dt = _stored(g, u)
    if u.numel() != g.numel():
        raise ValueError("g and u must have the same size")
    with _on(stream):
        a = torch.empty_like(g)
    gp, up = _flat(g, "g"), _flat(u, "u")
    if dt == DGF_BF16:
        _check(L.dgf_act_fwd(gp, up, a.data_ptr(), g.numel(), _stream(stream)), "dgf_act_fwd")
    else:
        _check(L.dgf_act_fwd_typed(gp, up, a.data_ptr(), g.numel(), dt, _stream(stream)), "dgf_act_fwd_typed")
    return a


def act_bwd(da, g, u, stream=None):
    """dG, dU and the recomputed a elementwise in the stored type of da, g, u."""
    L = load()
    dt = _stored(da, g, u)
    if u.numel() != g.numel() or da.numel() != g.numel():
        raise ValueError("da, g and u must have the same size")
    with _on(stream):
        dg, du, a = torch.empty_like(g), torch.empty_like(g), torch.empty_like(g)
    ptrs = (_flat(da, "da"), _flat(g, "g"), _flat(u, "u"), dg.data_ptr(), du.data_ptr(), a.data_ptr(), g.numel())
    if dt == DGF_BF16:
        _check(L.dgf_act_bwd(*ptrs, _stream(stream)), "dgf_act_bwd")
    else:
        _check(L.dgf_act_bwd_typed(*ptrs, dt, _stream(stream)), "dgf_act_bwd_typed")
    return dg, du, a


# ------------------------------------------------- operators around the FFN
def _vec(t, H: int, like: torch.Tensor, name: str):
    """Pointer of a contiguous [H] vector of like's dtype (None: NULL)."""
    if t is None:
        return None
    if t.dtype is like.dtype and t.get_device() == like.get_device() and t.shape == (H,) and t.is_contiguous():
        return t.data_ptr()
    if t.dtype != like.dtype or t.device != like.device:
        raise TypeError(f"{name}: expected {like.dtype} on {like.device}, got {t.dtype} on {t.device}")
    raise ValueError(f"{name}: expected a contiguous vector of {H} elements")


def _rows(t, shape, like: torch.Tensor, name: str):
    """(pointer, leading dimension) of a matrix of the given shape and like's dtype (None: NULL)."""
    if t is None:
        return None, 0
    if t.dtype is like.dtype and t.get_device() == like.get_device() and t.shape == shape:
        return _mat(t, name)
    if t.dtype != like.dtype or t.device != like.device:
        raise TypeError(f"{name}: expected {like.dtype} on {like.device}, got {t.dtype} on {t.device}")
    raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")


def _gate(gate, M: int, H: int, like: torch.Tensor):
    """(pointer, leading dimension): 0 for one value a channel ([H])."""
    if gate is not None and gate.dim() == 1:
        return _vec(gate, H, like, "gate"), 0
    if gate is not None and gate.dim() == 2 and gate.stride(0) == 0 and M > 0:
        raise ValueError("gate: give one value a channel as a vector, not as an expanded matrix")
    return _rows(gate, (M, H), like, "gate")


def norm_fwd(res, y=None, w_post=None, gate=None, alpha: float = 1.0, w_next=None, eps: float = 1e-6,
             training: bool = False, out=None, stream=None):
    """The norms after a block (of its output y, with gate and the residual res)
    and before the next one, dgf_norm_fwd:

        t = y r_y w_post;  z = alpha res + gate t;  h = z r_z w_next

    res, y [M, H]; w_post, w_next [H]; gate [H] or [M, H]; w_post None: t = y;
    gate None: 1; w_next None: no h; y None: h from res alone (z is res).
    Returns a dict with z, h (w_next given) and rstd [M, 2] FP32 (training).
    out: where z goes (may be res itself)."""
    L = load()
    dt = _stored(res)
    M, H = res.shape
    if y is None and out is not None:
        raise ValueError("out: without y there is no new residual (z is res)")
    rp, ldr = _mat(res, "res")
    yp, ldy = _rows(y, (M, H), res, "y")
    gp, ldg = _gate(gate, M, H, res)
    wp, wn = _vec(w_post, H, res, "w_post"), _vec(w_next, H, res, "w_next")
    with _on(stream):
        z = res if y is None else _empty(M, H, res) if out is None else out
        h = _empty(M, H, res) if w_next is not None else None
        rstd = res.new_empty((M, 2), dtype=torch.float32) if training else None
    zp, ldz = _rows(z, (M, H), res, "out") if out is not None else (z.data_ptr(), z.stride(0))
    hp, ldh = (h.data_ptr(), h.stride(0)) if h is not None else (None, 0)
    _check(L.dgf_norm_fwd(rp, ldr, yp, ldy, wp, gp, ldg, alpha, wn, eps, zp, ldz, hp, ldh,
                          rstd.data_ptr() if training else None, M, H, dt, _stream(stream)), "dgf_norm_fwd")
    r = {"z": z}
    if h is not None:
        r["h"] = h
    if training:
        r["rstd"] = rstd
    return r


def norm_bwd(dz, dh, z, y=None, w_post=None, gate=None, alpha: float = 1.0, w_next=None, rstd=None, stream=None):
    """Backward of norm_fwd (dgf_norm_bwd) from dz and dh (either may be None),
    the forward's z and rstd and its inputs.  Returns a dict: dres, and dy,
    dw_post, dgate, dw_next for the inputs that were given."""
    L = load()
    like = dz if dz is not None else dh
    if like is None or rstd is None:
        raise ValueError("norm_bwd needs dz or dh, and the forward's rstd")
    dt = _stored(like)
    M, H = like.shape
    dzp, lddz = _rows(dz, (M, H), like, "dz")
    dhp, lddh = _rows(dh, (M, H), like, "dh")
    zp, ldz = _rows(z, (M, H), like, "z")
    yp, ldy = _rows(y, (M, H), like, "y")
    gp, ldg = _gate(gate, M, H, like)
    wp, wn = _vec(w_post, H, like, "w_post"), _vec(w_next, H, like, "w_next")
    if (rstd.dtype is not torch.float32 or rstd.shape != (M, 2) or not rstd.is_contiguous()
            or rstd.get_device() != like.get_device()):
        raise ValueError(f"rstd: expected the forward's contiguous float32 [{M}, 2]")
    with _on(stream):
        r = {"dres": _empty(M, H, like)}
        dres, ld_dres = r["dres"].data_ptr(), r["dres"].stride(0)
        dy = dw_post = dgate = dw_next = None
        ld_dy = ld_dgate = 0
        if y is not None:
            t = r["dy"] = _empty(M, H, like)
            dy, ld_dy = t.data_ptr(), t.stride(0)
        if w_post is not None:
            t = r["dw_post"] = torch.empty_like(w_post)
            dw_post = t.data_ptr()
        if gate is not None:
            t = r["dgate"] = torch.empty_like(gate) if ldg == 0 else _empty(M, H, like)
            dgate, ld_dgate = t.data_ptr(), t.stride(0) if ldg else 0
        if w_next is not None:
            t = r["dw_next"] = torch.empty_like(w_next)
            dw_next = t.data_ptr()
        nbytes = L.dgf_norm_bwd_workspace(M, H)
        ws = _workspace(nbytes, like)
    _check(L.dgf_norm_bwd(dzp, lddz, dhp, lddh, zp, ldz, yp, ldy, wp, gp, ldg, alpha, wn, rstd.data_ptr(), dres, ld_dres,
                          dy, ld_dy, dw_post, dgate, ld_dgate, dw_next, M, H, ws.data_ptr(), nbytes, dt, _stream(stream)),
           "dgf_norm_bwd")
    return r


BLOCK8 = 64  # columns that share a scale of an 8-bit checkpoint


class Packed8(NamedTuple):
    """A matrix [M, N] saved in 8 bits: codes (int8 [M, N], row-major), scales
    (FP32 [M, ceil(N/64)]) and the type it reads back as."""

    codes: torch.Tensor
    scales: torch.Tensor
    dtype: torch.dtype


def _packed(M: int, N: int, like: torch.Tensor) -> Packed8:
    ld = (N + 15) // 16 * 16
    codes = like.new_empty((M, ld), dtype=torch.int8)
    scales = like.new_empty((M, -(-N // BLOCK8)), dtype=torch.float32)
    return Packed8(codes if ld == N else codes[:, :N], scales, like.dtype)


def _q8(p: Packed8, shape, dtype, device: int, name: str):
    """(codes, their leading dimension, scales, theirs) of a checkpoint of the given shape and type."""
    q, s, stored = p
    if stored is not dtype or q.dtype is not torch.int8 or s.dtype is not torch.float32:
        raise TypeError(f"{name}: expected an 8-bit checkpoint of {dtype} (int8 codes, float32 scales)")
    if device < 0 or q.get_device() != device or s.get_device() != device:
        raise ValueError(f"{name}: expected GPU tensors of one device")
    M, N = shape
    blocks = -(-N // BLOCK8)
    if q.shape != shape or s.shape != (M, blocks):
        raise ValueError(f"{name}: codes {tuple(q.shape)} and scales {tuple(s.shape)} are not those of a {M} x {N} matrix")
    qs, ss = q.stride(), s.stride()
    if (N > 1 and qs[1] != 1) or (blocks > 1 and ss[1] != 1):
        raise ValueError(f"{name}: expected row-major codes and scales")
    return q.data_ptr(), qs[0], s.data_ptr(), ss[0]


def pack8(t, stream=None) -> Packed8:
    """Saves a BF16 or FP16 matrix in 8 bits, blocks of 64 columns with an FP32 scale each (dgf_pack8)."""
    L = load()
    dt = _stored(t)
    tp, ldt = _mat(t, "t")
    M, N = t.shape
    with _on(stream):
        p = _packed(M, N, t)
    _check(L.dgf_pack8(tp, ldt, p.codes.data_ptr(), p.codes.stride(0), p.scales.data_ptr(), p.scales.stride(0), M, N,
                       dt, _stream(stream)), "dgf_pack8")
    return p


def unpack8(p: Packed8, stream=None) -> torch.Tensor:
    """Reads an 8-bit checkpoint back in its stored type, each value rounded once (dgf_unpack8)."""
    L = load()
    if p.dtype not in _STORED:
        raise TypeError(f"expected a checkpoint of bfloat16 or float16, got {p.dtype}")
    M, N = p.codes.shape
    qp, ldq, sp, lds = _q8(p, (M, N), p.dtype, p.codes.get_device(), "p")
    with _on(stream):
        t = p.codes.new_empty((M, (N + 7) // 8 * 8), dtype=p.dtype)
        t = t if t.shape[1] == N else t[:, :N]
    _check(L.dgf_unpack8(qp, ldq, sp, lds, t.data_ptr(), t.stride(0), M, N, _STORED[p.dtype], _stream(stream)),
           "dgf_unpack8")
    return t


def act_bwd_q8(da, g: Packed8, u: Packed8, stream=None):
    """act_bwd over a matrix [M, N] from g and u saved in 8 bits: dG, dU and the recomputed a."""
    L = load()
    dt = _stored(da)
    M, N = da.shape
    dap, ldda = _mat(da, "da")
    gq, ldq, gs, lds = _q8(g, (M, N), da.dtype, da.get_device(), "g")
    uq, ldq2, us, lds2 = _q8(u, (M, N), da.dtype, da.get_device(), "u")
    if (ldq, lds) != (ldq2, lds2):
        raise ValueError("g and u must share their leading dimensions")
    with _on(stream):
        dg, du, a = _empty(M, N, da), _empty(M, N, da), _empty(M, N, da)
    _check(L.dgf_act_bwd_q8(dap, ldda, gq, gs, uq, us, ldq, lds, dg.data_ptr(), du.data_ptr(), a.data_ptr(),
                            dg.stride(0), M, N, dt, _stream(stream)), "dgf_act_bwd_q8")
    return dg, du, a


def ffn_fwd_q8(x, w_gate, w_up, w_down, stream=None):
    """The training forward with g and u saved in 8 bits (dgf_ffn_fwd_q8): y (the
    bits of ffn_fwd) and the two checkpoints."""
    L = load()
    dt = _stored(x, w_gate, w_up, w_down)
    M, H = x.shape
    I = w_gate.shape[0]
    xp, ldx = _mat(x, "x"); wg, ldwg = _rows(w_gate, (I, H), x, "w_gate"); wu, ldwu = _rows(w_up, (I, H), x, "w_up")
    wd, ldwd = _rows(w_down, (H, I), x, "w_down")
    with _on(stream):
        y, g, u = _empty(M, H, x), _packed(M, I, x), _packed(M, I, x)
        ws = _workspace(L.dgf_ffn_fwd_q8_workspace(M, H, I), x)
    _check(L.dgf_ffn_fwd_q8(xp, ldx, wg, ldwg, wu, ldwu, wd, ldwd, y.data_ptr(), y.stride(0),
                            g.codes.data_ptr(), g.scales.data_ptr(), u.codes.data_ptr(), u.scales.data_ptr(),
                            g.codes.stride(0), g.scales.stride(0), M, H, I, ws.data_ptr(), ws.numel(), dt,
                            _stream(stream)), "dgf_ffn_fwd_q8")
    return y, g, u


def ffn_bwd_q8(dy, x, g: Packed8, u: Packed8, w_gate, w_up, w_down, stream=None):
    """ffn_bwd from the checkpoints of ffn_fwd_q8 (dgf_ffn_bwd_q8): dict dX, dW_gate, dW_up, dW_down."""
    L = load()
    dt = _stored(dy, x, w_gate, w_up, w_down)
    M, H = x.shape
    I = w_gate.shape[0]
    dyp, lddy = _rows(dy, (M, H), x, "dy"); xp, ldx = _mat(x, "x")
    wg, ldwg = _rows(w_gate, (I, H), x, "w_gate"); wu, ldwu = _rows(w_up, (I, H), x, "w_up")
    wd, ldwd = _rows(w_down, (H, I), x, "w_down")
    gq, ldq, gs, lds = _q8(g, (M, I), x.dtype, x.get_device(), "g")
    uq, ldq2, us, lds2 = _q8(u, (M, I), x.dtype, x.get_device(), "u")
    if (ldq, lds) != (ldq2, lds2):
        raise ValueError("g and u must share their leading dimensions")
    with _on(stream):
        dx, dwg, dwu, dwd = _empty(M, H, x), _empty(I, H, x), _empty(I, H, x), _empty(H, I, x)
        ws = _workspace(L.dgf_ffn_bwd_workspace(M, H, I), x)
    _check(L.dgf_ffn_bwd_q8(dyp, lddy, xp, ldx, gq, gs, uq, us, ldq, lds, wg, ldwg, wu, ldwu, wd, ldwd,
                            dx.data_ptr(), None, None, dx.stride(0), dwg.data_ptr(), dwg.stride(0),
                            dwu.data_ptr(), dwu.stride(0), dwd.data_ptr(), dwd.stride(0), M, H, I,
                            ws.data_ptr(), ws.numel(), dt, _stream(stream)), "dgf_ffn_bwd_q8")
    return {"dX": dx, "dW_gate": dwg, "dW_up": dwu, "dW_down": dwd}


def _experts(t: torch.Tensor, shape, like: torch.Tensor, name: str):
    """(pointer, leading dimension, expert stride) of the experts' matrices [El, rows, cols]."""
    if t.dtype is not like.dtype or t.get_device() != like.get_device():
        raise TypeError(f"{name}: expected {like.dtype} on {like.device}, got {t.dtype} on {t.device}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    stride = t.stride()
    if stride[2] != 1:
        raise ValueError(f"{name}: expected row-major matrices (stride(2) == 1)")
    return t.data_ptr(), stride[1], stride[0]


def moe_fwd(x, w_router, w_gate, w_up, w_down, top_k: int, renorm: bool = True, routing: bool = False,
            expert_offset: int = 0, stream=None):
    """A mixture-of-experts layer of gated FFNs for up to 128 tokens (dgf_moe_fwd).

    x [M, H]; w_router [E, H]; w_gate, w_up [El, I, H] and w_down [El, H, I], the
    experts [expert_offset, expert_offset + El) of the E (all of them by default).
    renorm: routing weights over the top_k chosen instead of all E.
    Returns y [M, H], or with routing (y, ids int32 [M, top_k], weights float32 [M, top_k])."""
    L = load()
    dt = _stored(x)
    M, H = x.shape
    E, El, I = w_router.shape[0], w_gate.shape[0], w_gate.shape[1]
    xp, ldx = _mat(x, "x")
    wr, ldr = _rows(w_router, (E, H), x, "w_router")
    wg, ldg, sg = _experts(w_gate, (El, I, H), x, "w_gate")
    wu, ldu, su = _experts(w_up, (El, I, H), x, "w_up")
    wd, ldd, sd = _experts(w_down, (El, H, I), x, "w_down")
    ids = probs = None
    with _on(stream):
        y = _empty(M, H, x)
        if routing:
            ids = x.new_empty((M, max(top_k, 0)), dtype=torch.int32)
            probs = x.new_empty((M, max(top_k, 0)), dtype=torch.float32)
        nbytes = L.dgf_moe_fwd_workspace(M, H, I, E, El, top_k)
        ws = _workspace(nbytes, x)
    _check(L.dgf_moe_fwd(xp, ldx, wr, ldr, wg, ldg, sg, wu, ldu, su, wd, ldd, sd, y.data_ptr(), y.stride(0),
                         ids.data_ptr() if routing else None, probs.data_ptr() if routing else None,
                         M, H, I, E, expert_offset, El, top_k, int(renorm), ws.data_ptr(), nbytes, dt,
                         _stream(stream)), "dgf_moe_fwd")
    return (y, ids, probs) if routing else y


class KernelTimer:
    """Times every kernel the library launches between start() and stop() with
    HIP events recorded on the launch stream (the library's timing hook)."""

    def __init__(self, max_kernels: int = 4096):
        self.n = max_kernels
        self.events = [torch.cuda.Event(enable_timing=True) for _ in range(2 * max_kernels)]
        s = torch.cuda.current_stream()
        for e in self.events:  # materialise the underlying HIP events
            e.record(s)
        torch.cuda.synchronize()
        self._arr = (ctypes.c_void_p * (2 * max_kernels))(*[e.cuda_event for e in self.events])
        self.count = 0
        self.names = []

    def start(self):
        _check(load().dgf_profile_begin(self._arr, self.n), "dgf_profile_begin")

    def stop(self):
        L = load()
        self.count = L.dgf_profile_end()
        self.names = [L.dgf_profile_name(k).decode() for k in range(min(self.count, self.n))]
        return self

    def durations_ms(self):
        """[(name, ms)] for each timed launch (call after synchronising)."""
        return [(self.names[k], self.events[2 * k].elapsed_time(self.events[2 * k + 1]))
                for k in range(min(self.count, self.n))]
