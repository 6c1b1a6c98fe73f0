"""8-bit products with block scales and a mixture of experts, on torch tensors.

    from dense_gemm_elementwise_amd import quantize_fp8, linear_fp8, linear_fp8_backward, moe
    w8, ws, wt8, wts = quantize_fp8(w, block="tile", transpose=True)
    x8, xs, xt8, xts = quantize_fp8(x, transpose=True)
    d, z = linear_fp8(x8, w8, ws, bias, residual, x_scale=xs, act="gelu", save_z=True)
    dx, dw, dbias = linear_fp8_backward(dd, xt8, xts, wt8, wts, z, act="gelu")
    y = moe(x, w_router, up8, down8, top_k=8, up_scale=us, down_scale=ds)

The work runs in the HIP kernels behind include/fp8_ops.h.  Calls, streams,
workspaces and errors are those of operators.py: every call is queued on
`stream` (default: the current stream of the tensors' device) and returns
without waiting; there is no autograd node, and a tensor that requires grad is
refused while gradients are recorded.

8-bit matrices are 2-D torch.float8_e4m3fn or float8_e5m2 tensors with unit
stride along the rows and any row stride; their scales are float8_e8m0fnu
(powers of two), by row blocks (R, ceil(C / 128)) or by tiles (ceil(R / 128),
ceil(C / 128)).  Rows that start at multiples of 16 bytes (scales: of 4), as those of
quantize_fp8 do, are read in place; others are copied first, on every call, but
for products of up to 16 rows and moe, which read all in place.
"""
import ctypes
import operator
import struct

import torch

from . import binding, operators
from .operators import ACTS, _DTYPES, _STREAM_DTYPES, _TAIL, _STREAM, _NO_TAIL, _kind, _matrix, _raise, _run, _vector

FORMATS = {"e4m3": 0, "e5m2": 1}
BLOCKS = {"row": 0, "tile": 1}
FP8_EXPORTS = ("ge_quantize_fp8", "ge_linear_fp8", "ge_linear_fp8_backward", "ge_moe")
_WORKSPACE = {n: n + "_workspace" for n in FP8_EXPORTS if n != "ge_quantize_fp8"}
_FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
_FORMAT_OF = {v: FORMATS[k] for k, v in _FP8.items()}
_SCALE = torch.float8_e8m0fnu

# the argument structures of include/fp8_ops.h, without the trailing workspace and stream
_QUANTIZE = struct.Struct("@2q 2q 2q 2q 2q 2q 3q")
_LINEAR8 = struct.Struct("@3q 2q 2q 2q 2q q 2q 2q 2q 3q")
_LINEAR8_GRAD = struct.Struct("@3q 2q 2q 2q 2q 2q 2q 2q 2q q 3q")
_MOE = struct.Struct("@5q 2q 2q 3q 3q 3q 3q 2q 2q 4q")

_fns = None
_sizes = {}  # workspace sizes by call and sizes


def _functions():
    """The entry points by name; each takes the bytes of its structure."""
    global _fns
    if _fns is None:
        lib = binding.lib()
        fns = {}
        for name in FP8_EXPORTS:
            fns[name] = getattr(lib, name)
            fns[name].argtypes, fns[name].restype = [ctypes.c_char_p], ctypes.c_int
        for name in _WORKSPACE.values():
            fns[name] = getattr(lib, name)
            fns[name].argtypes = [ctypes.c_char_p, ctypes.POINTER(ctypes.c_int64)]
            fns[name].restype = ctypes.c_int
        _fns = fns
    return _fns


def workspace_bytes(name, args):
    """Bytes of workspace that a call of entry point `name` needs for the
    packed argument structure `args`: (status, bytes)."""
    n = ctypes.c_int64(0)
    rc = _functions()[_WORKSPACE[name]](args, ctypes.byref(n))
    return rc, n.value


def _queue(name, head, dev, raw_stream, sizes):
    """Makes one call.  The workspace comes from torch's allocator, in the order
    of the current stream; its size is remembered by the call's sizes, a guess
    that saves the query: the call itself says when it is too small."""
    f = (_fns or _functions())[name]
    key = (name, sizes)
    need = _sizes.get(key, 0)
    ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    rc = f(head + _TAIL.pack(ws.data_ptr() if need else 0, need, raw_stream))
    if rc == 7:
        rc, need = workspace_bytes(name, head + _NO_TAIL)
        if rc == 0:
            if len(_sizes) >= 4096:
                _sizes.clear()
            _sizes[key] = need
            ws = torch.empty(need, dtype=torch.uint8, device=dev)
            rc = f(head + _TAIL.pack(ws.data_ptr(), need, raw_stream))
    if rc != 0:
        _raise(rc)


def _first(name, t, dtypes, dim=2):
    """The type and device of a call, from its first tensor."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be one of {tuple(str(d) for d in dtypes)}, got {t.dtype}")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on a GPU device, got {t.device}")
    if t.dim() != dim:
        raise ValueError(f"{name} must be {dim}-D, got shape {tuple(t.shape)}")
    return t.dtype, t.device


def _blocks(n):
    return -(-n // 128)


def _new8(rows, cols, dtype, multiple, dev):
    """A new matrix of 1-byte elements whose rows start at multiples of `multiple` bytes."""
    pitch = -(-cols // multiple) * multiple
    t = torch.empty((rows, pitch), dtype=dtype, device=dev)
    return (t if pitch == cols else t[:, :cols]), pitch


def _two_d(name, t, what):
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError(f"{name} must be a 2-D tensor {what}")


def quantize_fp8(x, *, block="row", format="e4m3", transpose=False, stream=None):
    """x (R, C), float16, bfloat16 or float32, in 8-bit floating point with a
    power-of-two scale for each block: block "row", 128 consecutive elements of a
    row, or "tile", 128 x 128.  Returns (q, scale), q (R, C) float8_e4m3fn or
    float8_e5m2 (`format`) and scale float8_e8m0fnu, so that x is about q times its
    block's scale; with transpose=True also (qt, scale_t), the same of x
    transposed, (C, R): with "row" blocks along its own rows, with "tile" blocks the
    transpose of q.  The scale is the smallest power of two that keeps the block's
    finite elements in range, and q is rounded to nearest even.  R may be 0."""
    dtype, dev = _first("x", x, _STREAM_DTYPES)
    R, C = x.shape
    b, f = _kind("block", block, BLOCKS), _kind("format", format, FORMATS)
    xp = _matrix("x", x, (R, C), dtype, dev)

    def call(raw):
        q, ldq = _new8(R, C, _FP8[format], 16, dev)
        s, lds = _new8(_blocks(R) if b else R, _blocks(C), _SCALE, 4, dev)
        out, more = (q, s), (0, 0, 0, 0)
        if transpose:
            qt, ldqt = _new8(C, R, _FP8[format], 16, dev)
            st, ldst = _new8(_blocks(C) if b else C, _blocks(R), _SCALE, 4, dev)
            out, more = (q, s, qt, st), (qt.data_ptr(), ldqt, st.data_ptr(), ldst)
        rc = _functions()["ge_quantize_fp8"](_QUANTIZE.pack(R, C, *xp, q.data_ptr(), ldq, s.data_ptr(), lds, *more, b,
                                                            f, _STREAM_DTYPES[dtype]) + _STREAM.pack(raw))
        if rc != 0:
            _raise(rc)
        return out
    return _run(call, (x,), dev, stream)


def linear_fp8(x, w, w_scale, bias=None, residual=None, *, x_scale=None, act="identity", save_z=False, dtype=None,
               stream=None):
    """D = act(x w^T + bias) + residual with 8-bit operands: w (N, K)
    float8_e4m3fn with w_scale by tiles; x (M, K) float8_e4m3fn or float8_e5m2 with
    x_scale by row blocks, or float16 or bfloat16 without: it is then quantised as
    quantize_fp8 does, within the call.  bias (N,) and residual (M, N) or None;
    they and the outputs have `dtype`: x's own where it has 16 bits, bfloat16 by
    default otherwise.  Returns D, or (D, Z) with save_z, Z = x w^T + bias.  act as
    in linear.  M may be 0."""
    xd, dev = _first("x", x, (*_DTYPES, *_FORMAT_OF))
    M, K = x.shape
    _two_d("w", w, "(N, K)")
    N = w.shape[0]
    a = _kind("act", act, ACTS)
    if xd in _DTYPES:
        if x_scale is not None:
            raise ValueError(f"x of {xd} takes no x_scale")
        if dtype not in (None, xd):
            raise TypeError(f"dtype must be x's own, {xd}, got {dtype}")
        dtype, fmt, xs = xd, 0, (0, 0)
    else:
        if x_scale is None:
            raise ValueError(f"x of {xd} needs x_scale")
        dtype = torch.bfloat16 if dtype is None else dtype
        if dtype not in _DTYPES:
            raise TypeError(f"dtype must be float16 or bfloat16, got {dtype}")
        fmt, xs = _FORMAT_OF[xd], _matrix("x_scale", x_scale, (M, _blocks(K)), _SCALE, dev)
    xp = _matrix("x", x, (M, K), xd, dev)
    wp = _matrix("w", w, (N, K), torch.float8_e4m3fn, dev)
    sp = _matrix("w_scale", w_scale, (_blocks(N), _blocks(K)), _SCALE, dev)
    bp = _vector("bias", bias, N, dtype, dev)
    rp = _matrix("residual", residual, (M, N), dtype, dev) if residual is not None else (0, 0)

    def call(raw):
        d = torch.empty((M, N), dtype=dtype, device=dev)
        z = torch.empty_like(d) if save_z else None
        _queue("ge_linear_fp8",
               _LINEAR8.pack(M, N, K, *xp, *xs, *wp, *sp, bp, *rp, d.data_ptr(), N, z.data_ptr() if save_z else 0, N,
                             a, _DTYPES[dtype], fmt), dev, raw, (M, N, K, xs[0] == 0))
        return (d, z) if save_z else d
    return _run(call, (x, x_scale, w, w_scale, bias, residual), dev, stream)


def linear_fp8_backward(dd, xt, xt_scale, wt, wt_scale, z=None, *, act="identity", format="e4m3", need_dx=True,
                        need_dw=True, need_dbias=True, stream=None):
    """Gradients of linear_fp8 at the quantised x and w: dd (M, N) float16 or
    bfloat16, xt (K, M) and wt (K, N) float8_e4m3fn, x and w transposed with their
    scales by row blocks and by tiles (quantize_fp8 with transpose=True), z (M, N) as
    linear_fp8 kept it (may be None for "identity").  Returns (dx, dw, dbias): dx
    (M, K) and dw (N, K) of dd's type, dbias (N,) float32; None in the place of one
    that is not needed (xt and its scale, or wt and its scale, may then be None:
    K comes from the other).  dZ = dd act'(z) is quantised to `format`, along its
    rows for dx and along its columns for dw; dbias sums it unquantised."""
    dtype, dev = _first("dd", dd, _DTYPES)
    M, N = dd.shape
    a, f = _kind("act", act, ACTS), _kind("format", format, FORMATS)
    if not (need_dx or need_dw or need_dbias):
        return None, None, None
    if z is None and a != 0:
        raise ValueError(f"act {act!r} needs z")
    if need_dx:
        _two_d("wt", wt, "(K, N)")
    if need_dw:
        _two_d("xt", xt, "(K, M)")
    K = wt.shape[0] if need_dx else xt.shape[0] if need_dw else 1
    e4m3 = torch.float8_e4m3fn
    dp = _matrix("dd", dd, (M, N), dtype, dev)
    xp = xs = wp = ws = (0, 0)
    if need_dw:
        xp, xs = _matrix("xt", xt, (K, M), e4m3, dev), _matrix("xt_scale", xt_scale, (K, _blocks(M)), _SCALE, dev)
    if need_dx:
        wp = _matrix("wt", wt, (K, N), e4m3, dev)
        ws = _matrix("wt_scale", wt_scale, (_blocks(K), _blocks(N)), _SCALE, dev)
    zp = _matrix("z", z, (M, N), dtype, dev) if z is not None else (0, 0)

    def call(raw):
        dx = dd.new_empty((M, K)) if need_dx else None
        dw = dd.new_empty((N, K)) if need_dw else None
        db = torch.empty((N,), dtype=torch.float32, device=dev) if need_dbias else None
        _queue("ge_linear_fp8_backward",
               _LINEAR8_GRAD.pack(M, N, K, *dp, *xp, *xs, *wp, *ws, *zp, dx.data_ptr() if need_dx else 0, K,
                                  dw.data_ptr() if need_dw else 0, K, db.data_ptr() if need_dbias else 0, a,
                                  _DTYPES[dtype], f), dev, raw, (M, N, K, need_dx, need_dw))
        return dx, dw, db
    return _run(call, (dd, xt if need_dw else None, xt_scale if need_dw else None, wt if need_dx else None,
                       wt_scale if need_dx else None, z), dev, stream)


def _experts(name, t, shape, dtype, dev):
    """(address, row stride, expert stride) of a 3-D tensor with unit stride along its rows."""
    operators._check(name, t, shape, dtype, dev)
    se, s0, s1 = t.stride()
    e, r, c = shape
    if c > 1 and s1 != 1:
        raise ValueError(f"{name} must have unit stride along its rows, got strides {(se, s0, s1)}")
    if r <= 1:
        s0 = c
    if s0 < c or (e > 1 and se < (r - 1) * s0 + c):
        raise ValueError(f"{name}'s rows overlap: strides {(se, s0, s1)} for shape {tuple(shape)}")
    return t.data_ptr(), s0, se


def moe(x, w_router, w_up, w_down, *, top_k, up_scale=None, down_scale=None, residual=None, act="silu",
        renormalize=True, stream=None):
    """A mixture-of-experts layer: x (T, H), w_router (E, H), w_up (E, 2 I, H) for a
    gated layer (each expert's gate rows first) or (E, I, H) for a plain one, w_down
    (E, H, I).  Every token takes the top_k experts with the largest logits
    x w_router^T (ties: the lowest index), weighted by the softmax over all
    experts, divided by the chosen ones' sum with renormalize; logits are fp32
    sums, and a NaN among a token's makes its weights NaN.  An expert's output is
    w_down h, h = act(gate) * up or act(up), h in x's type and 3 bits more (bfloat16:
    where 2^-15 <= |h| < 2^16; float16: an infinity past 65504).
    Returns residual (T, H; None: zero) + the weighted sum, (T, H).  w_up and w_down
    are of x's type, or float8_e4m3fn with up_scale and down_scale by tiles (E,
    ceil(rows / 128), ceil(columns / 128)).  Made for a few tokens: the chosen experts'
    weights are read once for each 64 of them.  T may be 0."""
    dtype, dev = _first("x", x, _DTYPES)
    T, H = x.shape
    _two_d("w_router", w_router, "(E, H)")
    for name, t in (("w_up", w_up), ("w_down", w_down)):
        if not isinstance(t, torch.Tensor) or t.dim() != 3:
            raise ValueError(f"{name} must be a 3-D tensor")
    E, I = w_router.shape[0], w_down.shape[2]  # noqa: E741
    a = _kind("act", act, ACTS)
    gated = w_up.shape[1] == 2 * I
    if not gated and w_up.shape[1] != I:
        raise ValueError(f"w_up has {w_up.shape[1]} rows for each expert, expected {2 * I} (gated) or {I}")
    try:
        top_k = operator.index(top_k)
    except TypeError:
        raise TypeError(f"top_k must be an integer, got {top_k!r}") from None
    if not 1 <= top_k <= min(E, 32):
        raise ValueError(f"top_k must lie in 1 .. {min(E, 32)}, got {top_k}")
    if (up_scale is None) != (down_scale is None):
        raise ValueError("up_scale and down_scale come together")
    xp = _matrix("x", x, (T, H), dtype, dev)
    rp = _matrix("w_router", w_router, (E, H), dtype, dev)
    wide = up_scale is None
    wd = dtype if wide else torch.float8_e4m3fn
    up = _experts("w_up", w_up, (E, (1 + gated) * I, H), wd, dev)
    down = _experts("w_down", w_down, (E, H, I), wd, dev)
    us = ds = (0, 0, 0)
    if not wide:
        us = _experts("up_scale", up_scale, (E, _blocks((1 + gated) * I), _blocks(H)), _SCALE, dev)
        ds = _experts("down_scale", down_scale, (E, _blocks(H), _blocks(I)), _SCALE, dev)
    res = _matrix("residual", residual, (T, H), dtype, dev) if residual is not None else (0, 0)

    def call(raw):
        d = x.new_empty((T, H))
        _queue("ge_moe", _MOE.pack(T, H, E, I, top_k, *xp, *rp, *up, *us, *down, *ds, *res, d.data_ptr(), H, a, gated,
                                   renormalize, _DTYPES[dtype]), dev, raw, (T, H, E, I, top_k))
        return d
    return _run(call, (x, w_router, w_up, w_down, up_scale, down_scale, residual), dev, stream)
