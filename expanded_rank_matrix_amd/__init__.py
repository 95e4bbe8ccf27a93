"""MI355X-native ExTernD decomposition engine: thin Python binding of libexternd.so.

Every step of the decomposition runs in the library's HIP kernels; this module only marshals
torch device tensors (device memory and the current stream) to the C ABI declared in
``include/externd.h``.  There is no CPU fallback: if the library is missing the calls raise.
"""

from __future__ import annotations

import ctypes
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libexternd.so")

OK, EINVAL, ENOMEM, EDEVICE, ENONFINITE = 0, -1, -2, -3, -4

_lib = None


class ExterndError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{status_string(status) if _lib else status}: {message}")
        self.status = status


class Stats(ctypes.Structure):
    _fields_ = [
        ("k", ctypes.c_int64),
        ("passes", ctypes.c_int64),
        ("early_exits", ctypes.c_int64),
        ("fallback_inits", ctypes.c_int64),
        ("zero_components", ctypes.c_int64),
        ("block", ctypes.c_int64),
        ("energy_final_explicit", ctypes.c_double),
        ("seconds", ctypes.c_double),
        ("kernel_ms", ctypes.c_double),
        ("bytes_algorithmic", ctypes.c_double),
        ("flops_algorithmic", ctypes.c_double),
        ("components_used", ctypes.c_int64),
        ("safeguard_activations", ctypes.c_int64),
        ("sweep_reverts", ctypes.c_int64),
        ("residual_lds", ctypes.c_int64),
    ]

    def as_dict(self):
        return {name: getattr(self, name) for name, _ in self._fields_}


class Options(ctypes.Structure):
    _fields_ = [
        ("energy_target", ctypes.c_double),
        ("safeguard", ctypes.c_int),
        ("sweeps", ctypes.c_int),
        ("ablation", ctypes.c_int),
        ("residual_hbm", ctypes.c_int),
    ]


def load():
    """Load libexternd.so (built by ``expanded_rank_matrix_amd.build``); raise if missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is not built; run __graft_entry__.build() or "
                              "python -m expanded_rank_matrix_amd.build")
        lib = ctypes.CDLL(LIB_PATH)
        i64, f32, vp, ci = ctypes.c_int64, ctypes.c_float, ctypes.c_void_p, ctypes.c_int
        lib.externd_rank.restype = i64
        lib.externd_rank.argtypes = [i64, i64, f32]
        lib.externd_packed_words.restype = i64
        lib.externd_packed_words.argtypes = [i64]
        lib.externd_decompose.restype = ci
        lib.externd_decompose.argtypes = [vp, i64, i64, f32, f32, vp, ci, ci, vp, vp, vp, vp, vp,
                                          ctypes.POINTER(Stats)]
        lib.externd_decompose_ex.restype = ci
        lib.externd_decompose_ex.argtypes = [vp, i64, i64, f32, f32, vp, ci, ci, vp, vp, vp, vp,
                                             ctypes.POINTER(Options), vp, ctypes.POINTER(Stats)]
        lib.externd_project.restype = ci
        lib.externd_project.argtypes = [vp, i64, i64, f32, vp, vp, vp, vp]
        lib.externd_matvec.restype = ci
        lib.externd_matvec.argtypes = [vp, i64, i64, vp, vp, ci, vp, vp]
        lib.externd_apply_factors.restype = ci
        lib.externd_apply_factors.argtypes = [vp, vp, vp, i64, i64, i64, vp, i64, vp, vp]
        lib.externd_apply_factors_static.restype = ci
        lib.externd_apply_factors_static.argtypes = [vp, vp, vp, i64, i64, i64, vp, i64, vp, vp]
        lib.externd_quantize_rows.restype = ci
        lib.externd_quantize_rows.argtypes = [vp, ci, i64, i64, i64, vp, i64, vp, vp]
        lib.externd_apply_quantized.restype = ci
        lib.externd_apply_quantized.argtypes = [vp, vp, i64, i64, i64, vp, ci, vp, i64, i64, vp, ci,
                                                i64, vp, vp]
        lib.externd_apply_quantized_workspace.restype = i64
        lib.externd_apply_quantized_workspace.argtypes = [ci, i64, i64, i64]
        lib.externd_distill_loss.restype = ci
        lib.externd_distill_loss.argtypes = [vp, ci, i64, i64, i64, vp, ci, vp, ci, i64, f32, vp, vp, vp,
                                             vp, i64, vp, vp]
        lib.externd_distill_workspace.restype = i64
        lib.externd_distill_workspace.argtypes = [i64, i64]
        lib.externd_distill_grad.restype = ci
        lib.externd_distill_grad.argtypes = [vp, ci, i64, i64, i64, vp, vp, ci, vp, ci, i64, f32, vp, vp,
                                             i64, vp]
        lib.externd_apply_factors_grad.restype = ci
        lib.externd_apply_factors_grad.argtypes = [vp, vp, vp, i64, i64, i64, vp, vp, i64, vp, vp, vp, vp]
        lib.externd_apply_factors_grad_workspace.restype = i64
        lib.externd_apply_factors_grad_workspace.argtypes = [i64, i64, i64, i64]
        lib.externd_quantize_groups.restype = ci
        lib.externd_quantize_groups.argtypes = [vp, ci, i64, i64, i64, i64, vp, vp, vp, ci, vp]
        lib.externd_apply_grouped.restype = ci
        lib.externd_apply_grouped.argtypes = [vp, vp, vp, ci, i64, i64, i64, i64, vp, ci, i64, i64, vp, ci, i64, vp, vp]
        lib.externd_apply_grouped_workspace.restype = i64
        lib.externd_apply_grouped_workspace.argtypes = [ci, i64, i64, i64, i64]
        lib.externd_token_loss.restype = ci
        lib.externd_token_loss.argtypes = [vp, ci, i64, i64, i64, vp, i64, i64, vp, ci, vp, vp, vp, vp, i64, vp, i64,
                                           vp, vp]
        lib.externd_token_grad.restype = ci
        lib.externd_token_grad.argtypes = [vp, ci, i64, i64, i64, vp, i64, i64, vp, vp, ci, vp, vp, i64, vp, i64, vp, vp]
        lib.externd_token_workspace.restype = i64
        lib.externd_token_workspace.argtypes = [ci, i64, i64, i64, vp, i64, ci, ci, ci]
        lib.externd_status_string.restype = ctypes.c_char_p
        lib.externd_status_string.argtypes = [ci]
        lib.externd_last_error.restype = ctypes.c_char_p
        lib.externd_last_error.argtypes = []
        _lib = lib
    return _lib


def status_string(status: int) -> str:
    return load().externd_status_string(status).decode()


def last_error() -> str:
    return load().externd_last_error().decode()


def _check(status: int):
    if status != OK:
        raise ExterndError(status, last_error())


def rank(m: int, n: int, mu: float) -> int:
    return int(load().externd_rank(m, n, mu))


def packed_words(length: int) -> int:
    return int(load().externd_packed_words(length))


def _dev_ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_ptr(stream):
    import torch

    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _require(t, dtype, name, shape=None, device=None):
    """t as the C ABI will read or write it: a contiguous CUDA tensor of ``dtype`` (any of them
    when a tuple), on ``device`` and of exactly ``shape`` when given.  The library gets raw
    pointers and sizes, so a short or mistyped buffer would be read or written out of bounds."""
    if t is None:
        return None
    dtypes = dtype if isinstance(dtype, tuple) else (dtype,)
    if not (t.is_cuda and t.dtype in dtypes and t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous CUDA tensor of {' or '.join(map(str, dtypes))}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t


def decompose(A, mu: float, tau: float = 0.0, h=None, als_iters: int = 4, block: int = 1,
              stream=None, out=None, energy_target: float = 0.0, safeguard: bool = False,
              sweeps: int = 0, ablation: int = 0, residual_hbm: bool = False):
    """Run externd_decompose (externd_decompose_ex when an option is set) on a device fp32
    matrix A (m x n).

    Returns dict(B, C, D, energy, stats): B (k x words(m)) and C (k x words(n)) packed uint32
    stored in int32 tensors, D fp32 (k), energy fp64 (k), stats dict.  ``out`` may supply
    preallocated outputs as a dict with the same keys.  ``energy_target`` in (0, 1] stops after
    the first component whose energy reaches it (stats["components_used"]); ``safeguard`` turns
    on the best single-entry safeguard (sequential path); ``sweeps`` refinement sweeps refit
    every component after the greedy pass; ``ablation`` switches parts of the method off for
    ablation studies (1: block targets without decorrelation, 2: unweighted V-step projection);
    ``residual_hbm`` keeps the sequential path's residual in HBM even where it fits in LDS."""
    import torch

    A = _require(A, torch.float32, "A")
    if A.dim() != 2:
        raise ValueError("A must be a 2-d matrix")
    m, n = A.shape
    dev = A.device
    h = _require(h, torch.float32, "h", shape=(n,), device=dev)
    k = rank(m, n, mu)
    if k < 1:
        raise ExterndError(EINVAL, "mu gives k < 1")
    if out is None:
        out = dict(
            B=torch.empty((k, packed_words(m)), dtype=torch.int32, device=dev),
            C=torch.empty((k, packed_words(n)), dtype=torch.int32, device=dev),
            D=torch.empty(k, dtype=torch.float32, device=dev),
            energy=torch.empty(k, dtype=torch.float64, device=dev),
        )
    words32 = (torch.int32, torch.uint32)
    _require(out["B"], words32, "out['B']", shape=(k, packed_words(m)), device=dev)
    _require(out["C"], words32, "out['C']", shape=(k, packed_words(n)), device=dev)
    _require(out["D"], torch.float32, "out['D']", shape=(k,), device=dev)
    _require(out["energy"], torch.float64, "out['energy']", shape=(k,), device=dev)
    st = Stats()
    if energy_target or safeguard or sweeps or ablation or residual_hbm:
        opt = Options(float(energy_target), int(bool(safeguard)), int(sweeps), int(ablation),
                      int(bool(residual_hbm)))
        rc = load().externd_decompose_ex(_dev_ptr(A), m, n, mu, tau, _dev_ptr(h), als_iters, block,
                                         _dev_ptr(out["B"]), _dev_ptr(out["C"]),
                                         _dev_ptr(out["D"]), _dev_ptr(out["energy"]),
                                         ctypes.byref(opt), _stream_ptr(stream), ctypes.byref(st))
    else:
        rc = load().externd_decompose(_dev_ptr(A), m, n, mu, tau, _dev_ptr(h), als_iters, block,
                                      _dev_ptr(out["B"]), _dev_ptr(out["C"]), _dev_ptr(out["D"]),
                                      _dev_ptr(out["energy"]), _stream_ptr(stream),
                                      ctypes.byref(st))
    _check(rc)
    res = dict(out)
    res["stats"] = st.as_dict()
    res["k"] = k
    return res


def project(X, tau: float = 0.0, h=None, stream=None):
    """Ternary projection of each row of X (count x L, fp32, device).
    Returns (V int8 count x L, PHC fp64 count x 3)."""
    import torch

    X = _require(X, torch.float32, "X")
    if X.dim() != 2:
        raise ValueError("X must be count x L")
    count, L = X.shape
    h = _require(h, torch.float32, "h", shape=(L,), device=X.device)
    V = torch.empty((count, L), dtype=torch.int8, device=X.device)
    PHC = torch.empty((count, 3), dtype=torch.float64, device=X.device)
    rc = load().externd_project(_dev_ptr(X), count, L, tau, _dev_ptr(h), _dev_ptr(V), _dev_ptr(PHC),
                                _stream_ptr(stream))
    _check(rc)
    return V, PHC


def matvec(R, t, h=None, transpose: bool = False, stream=None):
    """R^T t (transpose) or R (h .* t) with fp64 accumulation; R fp32 (m x n), t int8."""
    import torch

    R = _require(R, torch.float32, "R")
    if R.dim() != 2:
        raise ValueError("R must be a 2-d matrix")
    m, n = R.shape
    t = _require(t, torch.int8, "t", shape=(m if transpose else n,), device=R.device)
    if h is not None and transpose:
        raise ValueError("h weights the U-step product R (h .* t) only")
    h = _require(h, torch.float32, "h", shape=(n,), device=R.device)
    out = torch.empty(n if transpose else m, dtype=torch.float64, device=R.device)
    rc = load().externd_matvec(_dev_ptr(R), m, n, _dev_ptr(t), _dev_ptr(h), int(transpose),
                               _dev_ptr(out), _stream_ptr(stream))
    _check(rc)
    return out


def _apply_args(B, C, D, m, n, X, out):
    """Validated (B, C, D, k, X2, Y, single) for the inference entry points."""
    import torch

    D = _require(D, torch.float32, "D")
    if D.dim() != 1:
        raise ValueError("D must be a vector of k scales")
    k = D.shape[0]
    dev = D.device
    words32 = (torch.int32, torch.uint32)
    _require(B, words32, "B", shape=(k, packed_words(m)), device=dev)
    _require(C, words32, "C", shape=(k, packed_words(n)), device=dev)
    X = _require(X, torch.float32, "X", device=dev)
    single = X.dim() == 1
    X2 = X.reshape(1, -1) if single else X
    if X2.dim() != 2 or X2.shape[1] != n:
        raise ValueError("X must be n or batch x n")
    Y = out if out is not None else torch.empty((X2.shape[0], m), dtype=torch.float32, device=dev)
    _require(Y, torch.float32, "out", device=dev)
    if Y.numel() != X2.shape[0] * m:
        raise ValueError("out must hold batch x m values")
    return B, C, D, k, X2, Y, single


def apply_factors(B, C, D, m: int, n: int, X, stream=None, out=None):
    """Y = (B diag(D) C X^T)^T from packed factors (as returned by decompose) for X (n or batch x n,
    fp32, device); returns Y (m or batch x m, fp32).  Enqueued on the stream without waiting (the
    library keeps a workspace per device and stream)."""
    B, C, D, k, X2, Y, single = _apply_args(B, C, D, m, n, X, out)
    rc = load().externd_apply_factors(_dev_ptr(B), _dev_ptr(C), _dev_ptr(D), k, m, n, _dev_ptr(X2),
                                      X2.shape[0], _dev_ptr(Y), _stream_ptr(stream))
    _check(rc)
    return Y[0] if single else Y.reshape(X2.shape[0], m)


def apply_factors_static(B, C, D, m: int, n: int, X, stream=None, out=None):
    """externd_apply_factors_static: as apply_factors, with the library's fixed per-GPU workspace
    (no device allocation) and without waiting for the stream; synchronise before reading Y."""
    B, C, D, k, X2, Y, single = _apply_args(B, C, D, m, n, X, out)
    rc = load().externd_apply_factors_static(_dev_ptr(B), _dev_ptr(C), _dev_ptr(D), k, m, n, _dev_ptr(X2),
                                             X2.shape[0], _dev_ptr(Y), _stream_ptr(stream))
    _check(rc)
    return Y[0] if single else Y.reshape(X2.shape[0], m)


def apply_factors_grad(B, C, D, m: int, n: int, X, dY, need_dX: bool = True, need_dD: bool = True,
                       stream=None, out=None):
    """Gradient of ``apply_factors`` at X (n or batch x n, fp32) for dY (m or batch x m, fp32): the
    ternary factors are fixed, X and the scales have gradients,
    dX = (C^T diag(D) B^T dY^T)^T and dD_i = sum over the batch of (C x)_i (B^T dy)_i.

    Returns (dX, dD) (fp32; dX of X's shape), None for one that is not needed (X may be None where
    dD is not needed).  ``out`` may supply the pair, which must not overlap the inputs
    (dX may be X itself, or dY where m = n).  A NaN or an infinity in a vector of dY gives NaN in that
    vector of dX and throughout dD, one in X throughout dD, one in D throughout dX.  Enqueued on the
    stream without waiting."""
    import torch

    if B is None or C is None or D is None or dY is None:
        _given(B=B, C=C, D=D, dY=dY)
    _require(D, torch.float32, "D")
    if D.dim() != 1:
        raise ValueError("D must be a vector of k scales")
    k, dev = D.shape[0], D.device
    words32 = (torch.int32, torch.uint32)
    _require(B, words32, "B", shape=(k, packed_words(m)), device=dev)
    _require(C, words32, "C", shape=(k, packed_words(n)), device=dev)
    if not (need_dX or need_dD):
        raise ValueError("need_dX or need_dD must be set")
    _require(dY, torch.float32, "dY", device=dev)
    single = dY.dim() == 1
    if dY.dim() not in (1, 2) or dY.shape[-1] != m:
        raise ValueError("dY must be m or batch x m")
    batch = 1 if single else dY.shape[0]
    lead = () if single else (batch,)
    if X is None and need_dD:
        raise ValueError("X is needed for dD")
    _require(X, torch.float32, "X", shape=(*lead, n), device=dev)
    args = (B, C, D, k, m, n, X, dY, batch, lead, need_dX, need_dD, out)
    ptr = _here(dev, stream)
    if ptr is not None:
        return _apply_factors_grad(*args, ptr)
    with _Run(dev, stream, (B, C, D, X, dY, *(out or ()))) as run:
        return _apply_factors_grad(*args, run.ptr)


def _apply_factors_grad(B, C, D, k, m, n, X, dY, batch, lead, need_dX, need_dD, out, stream):
    import torch

    dev = D.device
    lib = load()
    if out is None:
        dX = dD = None
        if need_dX:
            dX = torch.empty((*lead, n), dtype=torch.float32, device=dev) if X is None else torch.empty_like(X)
        if need_dD:
            dD = torch.empty_like(D)
    else:
        dX, dD = (t if need else None for t, need in zip(out, (need_dX, need_dD)))
        if (dX is None) == need_dX or (dD is None) == need_dD:
            raise ValueError("out must hold dX and dD where they are needed")
        _require(dX, torch.float32, "out[0]", shape=(*lead, n), device=dev)
        _require(dD, torch.float32, "out[1]", shape=(k,), device=dev)
    size = lib.externd_apply_factors_grad_workspace(k, m, n, batch)
    ws = torch.empty(size, dtype=torch.uint8, device=dev) if size > 0 else None
    _check(lib.externd_apply_factors_grad(
        B.data_ptr(), C.data_ptr(), D.data_ptr(), k, m, n, None if X is None else X.data_ptr(), dY.data_ptr(), batch,
        None if dX is None else dX.data_ptr(), None if dD is None else dD.data_ptr(),
        None if ws is None else ws.data_ptr(), stream))
    return dX, dD


def _given(**tensors):
    for name, t in tensors.items():
        if t is None:
            raise ValueError(f"{name} is missing")


class _Run:
    """Where one call runs: the device of its tensors made current, the stream, and outputs and
    workspace allocated on that stream, so that their memory is reused in its order.  Inputs that
    belong to another stream are recorded on this one."""

    __slots__ = ("ptr", "guard", "on")

    def __init__(self, device, stream, inputs):
        import torch

        self.guard = self.on = None
        index = device.index
        if index != torch._C._cuda_getDevice():
            self.guard = torch.cuda.device(index)
            self.guard.__enter__()
        self.ptr = torch._C._cuda_getCurrentRawStream(index)
        if stream is not None:
            try:
                if stream.device != device:
                    raise ValueError(f"stream is on {stream.device}, the tensors are on {device}")
                if stream.cuda_stream != self.ptr:
                    for t in inputs:
                        if t is not None:
                            t.record_stream(stream)
                    self.on = torch.cuda.stream(stream)
                    self.on.__enter__()
                    self.ptr = stream.cuda_stream
            except BaseException:
                self.__exit__(None, None, None)
                raise

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        if self.on is not None:
            self.on.__exit__(*exc)
        if self.guard is not None:
            self.guard.__exit__(*exc)
        return False


_TYPE = None  # torch dtype -> the C ABI's number of the type
_FLOAT = ()   # the floating-point ones


def _types():
    global _TYPE, _FLOAT
    if _TYPE is None:
        import torch

        _FLOAT = (torch.float32, torch.float16, torch.bfloat16)
        _TYPE = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2, torch.int8: 3}
    return _TYPE


def _here(device, stream):
    """The pointer of the current stream where a call runs just there, on the current device; None
    where it takes a _Run."""
    import torch

    if stream is None and device.index == torch._C._cuda_getDevice():
        return torch._C._cuda_getCurrentRawStream(device.index)
    return None


def _rows(t, types, name, shape=None, device=None):
    """t as rows of the C ABI: a CUDA matrix of one of ``types`` whose rows are contiguous and do
    not overlap, on ``device`` and of exactly ``shape`` when given.  Returns its row distance."""
    if t is None or not (t.is_cuda and t.dtype in types and t.dim() == 2):
        raise ValueError(f"{name} must be a CUDA matrix of {' or '.join(map(str, types))}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    rows, n = t.shape
    if shape is not None and (rows, n) != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    ld, inner = t.stride()
    if n > 1 and inner != 1:
        raise ValueError(f"{name} must have contiguous rows")
    if rows <= 1:
        return max(n, 1)
    if ld < n:
        raise ValueError(f"{name} must have rows that do not overlap")
    return ld


def quantize_rows(X, stream=None, out=None):
    """Rows of X (rows x n, fp32, fp16 or bf16, device; rows may be strided) to 8-bit integers with
    one scale a row: scale = max |x| / 127 and Q the whole numbers nearest to 127 x / max |x|, ties
    to even.  Returns (Q int8 rows x n, scale fp32 rows); ``out`` may supply that pair, apart from X
    (Q's rows may be strided).  A row of zeros gets scale 0, one with a NaN or an infinity scale NaN; both get
    zeros.  Quantises the weights of ``apply_quantized`` (rows are output channels) and tokens that
    several products share.  Enqueued on the stream without waiting."""
    types = _types()
    ldx = _rows(X, _FLOAT, "X")
    args = (X, types[X.dtype], ldx, out)
    ptr = _here(X.device, stream)
    if ptr is not None:
        return _quantize_rows(*args, ptr)
    with _Run(X.device, stream, (X,) if out is None else (X, *out)) as run:
        return _quantize_rows(*args, run.ptr)


def _quantize_rows(X, x_type, ldx, out, stream):
    import torch

    rows, n = X.shape
    dev = X.device
    if out is None:
        out = (torch.empty((rows, n), dtype=torch.int8, device=dev), torch.empty(rows, dtype=torch.float32, device=dev))
        ldq = n
    else:
        _given(**{"out[1]": out[1]})
        ldq = _rows(out[0], (torch.int8,), "out[0]", shape=(rows, n), device=dev)
        _require(out[1], torch.float32, "out[1]", shape=(rows,), device=dev)
    Q, scale = out
    _check(load().externd_quantize_rows(X.data_ptr(), x_type, rows, n, ldx, Q.data_ptr(), ldq, scale.data_ptr(), stream))
    return Q, scale


def apply_quantized(W, w_scale, X, x_scale=None, out_dtype=None, stream=None, out=None):
    """Y[t][o] = x_scale[t] w_scale[o] sum_j X[t][j] W[o][j]: a layer in 8-bit integers, beside
    ``apply_factors`` for the layers that stay unfactored.  W (m x n int8) and w_scale (m fp32) are
    as ``quantize_rows`` gives them.  X (n or tokens x n) is int8 with x_scale (tokens fp32), or
    fp32, fp16 or bf16 without it: its tokens are then quantised on the way as ``quantize_rows``
    does.  W, X and ``out`` may have strided rows; ``out`` lies apart from the inputs.  Returns Y (m or
    tokens x m) of ``out_dtype`` (fp32, fp16 or bf16; by default X's type, fp32 for int8 tokens).  The
    integer sum is exact; its conversion and the two scales round in fp32, then Y's type does.
    Enqueued on the stream without waiting."""
    types = _types()
    if X is None or w_scale is None:
        _given(X=X, w_scale=w_scale)
    x_type = types.get(X.dtype)
    ldw = _rows(W, _INT8 or _int8(), "W")
    m, n = W.shape
    dev = W.device
    _require(w_scale, _FLOAT[0], "w_scale", shape=(m,), device=dev)
    single = X.dim() == 1
    X2 = X.unsqueeze(0) if single else X
    ldx = _rows(X2, types, "X", device=dev)
    tokens, nx = X2.shape
    if nx != n:
        raise ValueError(f"X must be n or tokens x n with n = {n}")
    if (x_type == 3) != (x_scale is not None):
        raise ValueError("x_scale is given with int8 tokens and only then")
    if x_scale is not None:
        _require(x_scale, _FLOAT[0], "x_scale", shape=(tokens,), device=dev)
    if out is not None:
        if out_dtype is not None and out.dtype != out_dtype:
            raise ValueError("out must be of out_dtype")
        out_dtype = out.dtype
    elif out_dtype is None:
        out_dtype = _FLOAT[0] if x_type == 3 else X.dtype
    if out_dtype not in _FLOAT:
        raise ValueError("out_dtype must be torch.float32, torch.float16 or torch.bfloat16")
    args = (W, w_scale, m, n, ldw, X2, x_type, x_scale, tokens, ldx, out_dtype, out, single)
    ptr = _here(dev, stream)
    if ptr is not None:
        return _apply_quantized(*args, ptr)
    with _Run(dev, stream, (W, w_scale, X, x_scale, out)) as run:
        return _apply_quantized(*args, run.ptr)


_INT8 = ()


def _int8():
    global _INT8
    import torch

    _INT8 = (torch.int8,)
    return _INT8


def _apply_quantized(W, w_scale, m, n, ldw, X, x_type, x_scale, tokens, ldx, y_type, out, single, stream):
    import torch

    dev = W.device
    lib = load()
    if out is None:
        Y = torch.empty((tokens, m), dtype=y_type, device=dev)
        ldy = m
    else:
        Y = out.unsqueeze(0) if single and out.dim() == 1 else out
        ldy = _rows(Y, _FLOAT, "out", shape=(tokens, m), device=dev)
    size = lib.externd_apply_quantized_workspace(x_type, tokens, n, m)
    ws = torch.empty(size, dtype=torch.uint8, device=dev) if size > 0 else None
    _check(lib.externd_apply_quantized(
        W.data_ptr(), w_scale.data_ptr(), m, n, ldw, X.data_ptr(), x_type,
        None if x_scale is None else x_scale.data_ptr(), tokens, ldx, Y.data_ptr(), _TYPE[y_type], ldy,
        None if ws is None else ws.data_ptr(), stream))
    return Y[0] if single else Y


def _distill_args(logits, teacher, index, weight, name, out):
    """Validated arguments of the distillation entry points: the logits', the teacher's, ldd."""
    import torch

    types = _types()
    if teacher is None or index is None:
        _given(teacher=teacher, index=index)
    ldz = _rows(logits, _FLOAT, "logits")
    rows, vocab = logits.shape
    dev = logits.device
    _require(teacher, _FLOAT, "teacher", device=dev)
    if teacher.dim() != 2 or teacher.shape[0] != rows:
        raise ValueError(f"teacher must be rows x top with rows = {rows}")
    _require(index, (torch.int32, torch.int64), "index", shape=teacher.shape, device=dev)
    _require(weight, torch.float32, name, shape=(rows,), device=dev)
    ldd = vocab
    if out is not None:
        ldd = _rows(out, (logits.dtype,), "out", shape=(rows, vocab), device=dev)
    return (logits.data_ptr(), types[logits.dtype], rows, vocab, ldz), (
        teacher.data_ptr(), types[teacher.dtype], index.data_ptr(), index.element_size(), teacher.shape[1]), ldd


def distill_loss(logits, teacher, index, temperature: float = 1.0, weight=None, grad: bool = False,
                 stream=None, out=None):
    """Distillation of a student from a teacher's top logits: for each row (token)
    loss = weight T^2 sum_k p_k (log p_k - log q[index_k]), p the softmax of the row's valid
    teacher logits / T, q the softmax of all its logits / T.

    logits (rows x vocab, fp32, fp16 or bf16; rows may be strided), teacher (rows x top, any of
    these types) and index (rows x top, int32 or int64; an entry outside the vocabulary, such as -1,
    or with a teacher logit of -inf does not count), weight (rows fp32; rows of weight 0 are not
    read).  Returns (loss fp32 rows, stats fp32 rows x 2); with ``grad`` or ``out`` also dlogits, the
    gradient of the losses' sum, formed in the same call (``out`` may be a preallocated tensor apart
    from logits, or logits itself).  ``stats`` feeds ``distill_grad``.  Enqueued on the stream without waiting."""
    args = (logits, *_distill_args(logits, teacher, index, weight, "weight", out), temperature, weight, grad, out)
    ptr = _here(logits.device, stream)
    if ptr is not None:
        return _distill_loss(*args, ptr)
    with _Run(logits.device, stream, (logits, teacher, index, weight, out)) as run:
        return _distill_loss(*args, run.ptr)


def _distill_loss(logits, z, t, ldd, temperature, weight, grad, out, stream):
    import torch

    rows, vocab = logits.shape
    dev = logits.device
    lib = load()
    loss = torch.empty(rows, dtype=torch.float32, device=dev)
    stats = torch.empty((rows, 2), dtype=torch.float32, device=dev)
    if out is None and grad:
        out = torch.empty((rows, vocab), dtype=logits.dtype, device=dev)
    size = lib.externd_distill_workspace(rows, vocab)
    ws = torch.empty(size, dtype=torch.uint8, device=dev) if size > 0 else None
    _check(lib.externd_distill_loss(*z, *t, temperature, None if weight is None else weight.data_ptr(),
                                    loss.data_ptr(), stats.data_ptr(), None if out is None else out.data_ptr(), ldd,
                                    None if ws is None else ws.data_ptr(), stream))
    return (loss, stats) if out is None else (loss, stats, out)


def distill_grad(logits, stats, teacher, index, temperature: float = 1.0, grad_loss=None, stream=None,
                 out=None):
    """The gradient of ``distill_loss`` from its ``stats`` on the same logits:
    dlogits[r][v] = grad_loss[r] T (q[v] - sum of p_k with index_k = v), of logits' type; grad_loss
    (rows fp32, 1 where None) takes the weight's place, and a row where it is 0 is not read.  ``out``
    may be a preallocated tensor apart from logits, or logits itself.  Enqueued on the stream without waiting."""
    if stats is None:
        _given(stats=stats)
    z, t, ldd = _distill_args(logits, teacher, index, grad_loss, "grad_loss", out)
    _require(stats, _FLOAT[0], "stats", shape=(logits.shape[0], 2), device=logits.device)
    args = (logits, z, t, ldd, stats, temperature, grad_loss, out)
    ptr = _here(logits.device, stream)
    if ptr is not None:
        return _distill_grad(*args, ptr)
    with _Run(logits.device, stream, (logits, stats, teacher, index, grad_loss, out)) as run:
        return _distill_grad(*args, run.ptr)


def _distill_grad(logits, z, t, ldd, stats, temperature, grad_loss, out, stream):
    import torch

    if out is None:
        out = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
    _check(load().externd_distill_grad(*z, stats.data_ptr(), *t, temperature,
                                       None if grad_loss is None else grad_loss.data_ptr(), out.data_ptr(), ldd, stream))
    return out


def quantize_groups(W, group: int = 128, offsets: bool = False, scale_dtype=None, stream=None, out=None):
    """Weights W (rows x n, fp32, fp16 or bf16, device; rows may be strided) to 4-bit codes with a scale for each
    ``group`` (32, 64 or 128) of consecutive elements of a row, w = scale c + offset: c in -7 .. 7 and no
    offset (scale = max |w| / 7), or with ``offsets`` c in -8 .. 7 over the group's range
    (scale = (hi - lo) / 15, offset = lo + 8 scale), the whole numbers nearest to the quotients.

    Returns (Q, scale, offset): Q int32 rows x ceil(n / group) group / 8, eight codes a word, the first in the
    lowest four bits; scale and offset rows x ceil(n / group) of ``scale_dtype`` (by default W's type), offset None
    without ``offsets``.  ``out`` may supply the three, apart from W.  A group with a NaN or an infinity gets codes 0
    and scale NaN.  Makes the weights of ``apply_grouped``.  Enqueued on the stream without waiting."""
    types = _types()
    ldw = _rows(W, _FLOAT, "W")
    if group not in (32, 64, 128):
        raise ValueError("group must be 32, 64 or 128")
    if out is not None:
        _given(**{"out[0]": out[0], "out[1]": out[1]})
    if scale_dtype is None:
        scale_dtype = W.dtype if out is None else out[1].dtype
    if scale_dtype not in _FLOAT:
        raise ValueError("scale_dtype must be torch.float32, torch.float16 or torch.bfloat16")
    args = (W, types[W.dtype], ldw, group, offsets, scale_dtype, out)
    ptr = _here(W.device, stream)
    if ptr is not None:
        return _quantize_groups(*args, ptr)
    with _Run(W.device, stream, (W,) if out is None else (W, *out)) as run:
        return _quantize_groups(*args, run.ptr)


def _quantize_groups(W, w_type, ldw, group, offsets, scale_dtype, out, stream):
    import torch

    rows, n = W.shape
    dev, groups = W.device, (n + group - 1) // group
    shapes = ((rows, groups * group // 8), (rows, groups), (rows, groups))
    if out is None:
        Q = torch.empty(shapes[0], dtype=torch.int32, device=dev)
        scale = torch.empty(shapes[1], dtype=scale_dtype, device=dev)
        offset = torch.empty(shapes[2], dtype=scale_dtype, device=dev) if offsets else None
    else:
        Q, scale, offset = out
        if (offset is None) == bool(offsets):
            raise ValueError("out must hold an offset with offsets and only then")
        _require(Q, (torch.int32, torch.uint32), "out[0]", shape=shapes[0], device=dev)
        _require(scale, scale_dtype, "out[1]", shape=shapes[1], device=dev)
        _require(offset, scale_dtype, "out[2]", shape=shapes[2], device=dev)
    _check(load().externd_quantize_groups(W.data_ptr(), w_type, rows, n, ldw, group, Q.data_ptr(), scale.data_ptr(),
                                          None if offset is None else offset.data_ptr(), _TYPE[scale_dtype], stream))
    return Q, scale, offset


def apply_grouped(Q, scale, X, offset=None, group: int = 128, out_dtype=None, stream=None, out=None):
    """Y[t][o] = sum_j (scale[o][j // group] c[o][j] + offset[o][j // group]) X[t][j]: a layer in 4 bits, beside
    ``apply_quantized`` for layers in 8.  Q (int32, m x ceil(n / group) group / 8; rows may be strided), scale and
    offset (m x ceil(n / group), fp32, fp16 or bf16, both of one type) are as ``quantize_groups`` gives them.
    X (n or tokens x n, fp32, fp16 or bf16; rows may be strided) enters exactly.  Returns Y (m or tokens x m) of
    ``out_dtype`` (by default X's type), summed in fp32 and rounded once; ``out`` may supply it, apart from the inputs.
    Enqueued on the stream without waiting."""
    types = _types()
    if scale is None or X is None:
        _given(scale=scale, X=X)
    ldq = _rows(Q, _WORDS or _words(), "Q")
    m, words = Q.shape
    dev = Q.device
    single = X.dim() == 1
    X2 = X.unsqueeze(0) if single else X
    ldx = _rows(X2, _FLOAT, "X", device=dev)
    tokens, n = X2.shape
    if group not in (32, 64, 128):
        raise ValueError("group must be 32, 64 or 128")
    groups = (n + group - 1) // group
    if words != groups * group // 8:
        raise ValueError(f"Q has {words} words a row, {groups * group // 8} hold n = {n} in groups of {group}")
    _require(scale, _FLOAT, "scale", shape=(m, groups), device=dev)
    _require(offset, scale.dtype, "offset", shape=(m, groups), device=dev)
    if out is not None:
        if out_dtype is not None and out.dtype != out_dtype:
            raise ValueError("out must be of out_dtype")
        out_dtype = out.dtype
    elif out_dtype is None:
        out_dtype = X.dtype
    if out_dtype not in _FLOAT:
        raise ValueError("out_dtype must be torch.float32, torch.float16 or torch.bfloat16")
    args = (Q, scale, offset, group, m, n, ldq, X2, types[X.dtype], tokens, ldx, out_dtype, out, single)
    ptr = _here(dev, stream)
    if ptr is not None:
        return _apply_grouped(*args, ptr)
    with _Run(dev, stream, (Q, scale, offset, X, out)) as run:
        return _apply_grouped(*args, run.ptr)


_WORDS = ()


def _words():
    global _WORDS
    import torch

    _WORDS = (torch.int32, torch.uint32)
    return _WORDS


def _apply_grouped(Q, scale, offset, group, m, n, ldq, X, x_type, tokens, ldx, y_type, out, single, stream):
    import torch

    dev = Q.device
    lib = load()
    if out is None:
        Y = torch.empty((tokens, m), dtype=y_type, device=dev)
        ldy = m
    else:
        Y = out.unsqueeze(0) if single and out.dim() == 1 else out
        ldy = _rows(Y, _FLOAT, "out", shape=(tokens, m), device=dev)
    # codes with rows this far apart need none
    size = lib.externd_apply_grouped_workspace(x_type, tokens, n, m, group) if ldq <= 1 << 22 else 0
    ws = torch.empty(size, dtype=torch.uint8, device=dev) if size > 0 else None
    _check(lib.externd_apply_grouped(
        Q.data_ptr(), scale.data_ptr(), None if offset is None else offset.data_ptr(), _TYPE[scale.dtype], group, m, n, ldq,
        X.data_ptr(), x_type, tokens, ldx, Y.data_ptr(), _TYPE[y_type], ldy, None if ws is None else ws.data_ptr(), stream))
    return Y[0] if single else Y


def _token_args(X, W, target, weight, name, out):
    """Validated arguments of the token loss's entry points: X's and W's, the target's, and the row
    distances of given gradients."""
    import torch

    types = _types()
    if W is None or target is None:
        _given(W=W, target=target)
    ldx = _rows(X, _FLOAT, "X")
    rows, n = X.shape
    dev = X.device
    ldw = _rows(W, (X.dtype,), "W", device=dev)
    if W.shape[1] != n:
        raise ValueError(f"W must be vocab x n with n = {n}")
    _require(target, (torch.int32, torch.int64), "target", shape=(rows,), device=dev)
    _require(weight, torch.float32, name, shape=(rows,), device=dev)
    lds = (n, n)
    if out is not None:
        lds = tuple(n if t is None else _rows(t, (X.dtype,), f"out[{i}]", shape=tuple(s.shape), device=dev)
                    for i, (t, s) in enumerate(zip(out, (X, W))))
    return (X.data_ptr(), types[X.dtype], rows, n, ldx, W.data_ptr(), W.shape[0], ldw), (
        target.data_ptr(), target.element_size(), None if weight is None else weight.data_ptr()), lds


def token_loss(X, W, target, weight=None, grad: bool = False, need_dX: bool = True, need_dW: bool = True,
               stream=None, out=None):
    """Softmax cross entropy of tokens through an output matrix, without the logits z = X W^T kept:
    loss[t] = weight[t] (log sum_v exp z[t][v] - z[t][target[t]]), beside ``distill_loss`` where a model
    learns from text instead of from a teacher.

    X (rows x n, fp32, fp16 or bf16: the tokens' hidden rows) and W (vocab x n, of X's type) may have strided rows;
    target (rows, int32 or int64), weight (rows fp32, 1 where None).  A row whose target lies outside
    the vocabulary (such as -100) or whose weight is 0 is not read and has loss and gradient 0.
    Returns (loss fp32 rows, stats fp32 rows x 2); with ``grad`` or ``out`` (loss, stats, dX, dW), the gradients
    of the losses' sum, of X's type, None for one that is not needed (a fixed W: need_dW=False).
    ``out`` may supply the pair (dX, dW), apart from the inputs, but dX may be X itself.  ``stats`` feeds
    ``token_grad``.  Enqueued on the stream without waiting."""
    x, t, lds = _token_args(X, W, target, weight, "weight", out)
    args = (X, W, x, t, None, lds, (grad or out is not None) and need_dX, (grad or out is not None) and need_dW,
            grad or out is not None, out)
    ptr = _here(X.device, stream)
    if ptr is not None:
        return _token(*args, ptr)
    with _Run(X.device, stream, (X, W, target, weight, *(out or ()))) as run:
        return _token(*args, run.ptr)


def token_grad(X, W, stats, target, grad_loss=None, need_dX: bool = True, need_dW: bool = True, stream=None,
               out=None):
    """The gradient of ``token_loss`` from its ``stats`` on the same X and W: with
    P[t][v] = grad_loss[t] (softmax(z[t])[v] - [v = target[t]]), dX = P W and dW = P^T X, of X's type;
    grad_loss (rows fp32, 1 where None) takes the weight's place, and a row where it is 0 is not read.
    Returns (dX, dW), None for one that is not needed.  ``out`` may supply the pair, apart from the inputs, but dX may
    be X itself.  Enqueued on the stream without waiting."""
    if stats is None:
        _given(stats=stats)
    if not (need_dX or need_dW):
        raise ValueError("need_dX or need_dW must be set")
    x, t, lds = _token_args(X, W, target, grad_loss, "grad_loss", out)
    _require(stats, _FLOAT[0], "stats", shape=(X.shape[0], 2), device=X.device)
    args = (X, W, x, t, stats, lds, need_dX, need_dW, True, out)
    ptr = _here(X.device, stream)
    if ptr is not None:
        return _token(*args, ptr)
    with _Run(X.device, stream, (X, W, stats, target, grad_loss, *(out or ()))) as run:
        return _token(*args, run.ptr)


def _token(X, W, x, t, stats, lds, need_dX, need_dW, grad, out, stream):
    import torch

    dev, rows = X.device, X.shape[0]
    lib = load()
    if out is None:
        dX = torch.empty(X.shape, dtype=X.dtype, device=dev) if need_dX else None
        dW = torch.empty(W.shape, dtype=X.dtype, device=dev) if need_dW else None
    else:
        dX, dW = (o if need else None for o, need in zip(out, (need_dX, need_dW)))
        if (dX is None) == need_dX or (dW is None) == need_dW:
            raise ValueError("out must hold dX and dW where they are needed")
    size = lib.externd_token_workspace(x[1], rows, x[3], x[6], x[5], x[7], stats is None, need_dX, need_dW)
    ws = torch.empty(size, dtype=torch.uint8, device=dev) if size > 0 else None
    tail = (None if dX is None else dX.data_ptr(), lds[0], None if dW is None else dW.data_ptr(), lds[1],
            None if ws is None else ws.data_ptr(), stream)
    if stats is not None:
        _check(lib.externd_token_grad(*x, stats.data_ptr(), *t, *tail))
        return dX, dW
    loss = torch.empty(rows, dtype=torch.float32, device=dev)
    stats = torch.empty((rows, 2), dtype=torch.float32, device=dev)
    _check(lib.externd_token_loss(*x, *t, loss.data_ptr(), stats.data_ptr(), *tail))
    return (loss, stats, dX, dW) if grad else (loss, stats)


def unpack(packed, length: int) -> np.ndarray:
    """Packed 2-bit ternary rows (..., words) -> int8 (..., length); accepts torch or numpy.

    Element t is in bits 2(t%16)..2(t%16)+1 of word t//16; 00 -> 0, 01 -> +1, 11 -> -1."""
    if hasattr(packed, "cpu"):
        packed = packed.cpu().numpy()
    w = np.asarray(packed).view(np.uint32)
    codes = (w[..., :, None] >> (2 * np.arange(16, dtype=np.uint32))) & np.uint32(3)
    codes = codes.reshape(*w.shape[:-1], w.shape[-1] * 16)[..., :length]
    out = np.zeros(codes.shape, dtype=np.int8)
    out[codes == 1] = 1
    out[codes == 3] = -1
    return out
