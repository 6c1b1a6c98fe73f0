"""The training and serving operators around a fused product, on torch tensors.

    from dense_gemm_elementwise_amd import linear, linear_xent, norm_residual
    d, z = linear(x, w, bias, residual, act="gelu", save_z=True)
    dx, dw, dbias = linear_backward(dd, x, w, z, act="gelu")
    loss, lse = linear_xent(h, w_vocab, target)
    dh, dw_vocab = linear_xent_backward(dloss, h, w_vocab, target, lse)
    h, x = norm_residual(h, y, w_post=wo, w_pre=wi, gate=g, post="rms", pre="rms")

The work runs in the HIP kernels behind include/linear_ops.h; this module
checks and marshals arguments, and allocates outputs and workspaces from
torch's allocator.  Every call is queued on `stream` (a torch.cuda.Stream;
default: the current stream of the tensors' device) and returns without
waiting.  There is no autograd node: the gradients are calls of their own, and
a tensor that requires grad is refused while gradients are recorded, one with
a forward-mode tangent always.

Matrices are 2-D float16 or bfloat16 GPU tensors with unit stride along the
rows and any row stride of at least the row's length (a column slice of a wider
tensor is read in place).
"""
import ctypes
import struct

import torch
from torch.autograd import forward_ad

from . import binding

ACTS = {"identity": 0, "relu": 1, "gelu": 2, "silu": 3}
NORMS = {"none": 0, "rms": 1, "layer": 2}
OPERATOR_EXPORTS = ("ge_linear", "ge_linear_backward", "ge_linear_xent", "ge_linear_xent_backward",
                    "ge_norm_residual", "ge_norm_residual_backward")
_WORKSPACE = {n: n + "_workspace" for n in OPERATOR_EXPORTS if n != "ge_norm_residual"}
_DTYPES = {torch.float16: 0, torch.bfloat16: 1}
_STREAM_DTYPES = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}

# the argument structures of include/linear_ops.h, without the trailing workspace and stream
_LINEAR = struct.Struct("@3q 2q 2q q 2q 2q 2q 2q")
_LINEAR_GRAD = struct.Struct("@3q 2q 2q 2q 2q 2q 2q q 2q")
_XENT = struct.Struct("@3q 2q 2q 2q 2q q")
_XENT_GRAD = struct.Struct("@3q q 2q 2q 3q 2q 2q q")
_NORM = struct.Struct("@3q 2q 2q 3q 2q 2d 2q 2q 2q")
_NORM_GRAD = struct.Struct("@3q 2q 2q 2q 2q 3q 2q 2d 2q 2q 3q 2q")
_TAIL = struct.Struct("@3q")  # workspace, workspace_bytes, stream
_STREAM = struct.Struct("@q")
_NO_TAIL = _TAIL.pack(0, 0, 0)

_fns = None

# the current stream's address by device index; the plain query where torch has
# it (a torch.cuda.Stream object costs 1.5 us a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _functions():
    """The entry points by name; each takes the bytes of its structure."""
    global _fns
    if _fns is None:
        lib = binding.lib()
        fns = {}
        for name in OPERATOR_EXPORTS:
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


def _raise(rc):
    msg = binding.gemm_epi_status_string(rc)
    if rc == 6:
        msg += f" (hipError_t {binding.gemm_epi_last_hip_error()})"
    raise binding.GemmEpiError(rc, msg)


# workspace sizes by call and sizes (M, N, K / T, V, K / T, H, G): a guess that
# saves the query; the call itself says when it is too small
_sizes = {}


def _queue(name, head, dev, raw_stream, sizes=None):
    """Makes one call.  A workspace, where the call needs one, comes from
    torch's allocator, in the order of the current stream."""
    fns = _fns or _functions()
    f = fns[name]
    if sizes is None:
        rc = f(head + _STREAM.pack(raw_stream))
    else:
        key = (name, sizes)
        need = _sizes.get(key, 0)
        if need:
            ws = torch.empty(need, dtype=torch.uint8, device=dev)
            rc = f(head + _TAIL.pack(ws.data_ptr(), need, raw_stream))
        else:
            rc = f(head + _TAIL.pack(0, 0, raw_stream))
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


def _refuse_tangents(inputs):
    """Tangents of forward-mode differentiation would be dropped silently: they
    are refused, like requires_grad."""
    for t in inputs:
        if t is not None and forward_ad.unpack_dual(t).tangent is not None:
            raise ValueError("an input carries a forward-mode tangent: these calls record no derivative (use "
                             "torch.autograd.forward_ad.unpack_dual(...).primal)")


def _run(call, inputs, dev, stream):
    """Runs call(raw stream) with `dev` current and, if a stream is given, that
    stream current too, so that outputs and workspaces belong to it; the inputs
    are marked as in use there."""
    # (outside every dual level there are no tangents: one comparison a call)
    if getattr(forward_ad, "_current_level", 0) >= 0:
        _refuse_tangents(inputs)
    if stream is not None:
        if stream.device != dev:
            raise ValueError(f"stream is on {stream.device}, the tensors on {dev}")
        with torch.cuda.stream(stream):
            out = call(stream.cuda_stream)
        for t in inputs:
            if t is not None:
                t.record_stream(stream)
        return out
    index = dev.index
    if torch.cuda.current_device() != index:
        with torch.cuda.device(dev):
            return call(_raw_stream(index))
    return call(_raw_stream(index))


def _common(first_name, first, dtypes=_DTYPES):
    """The element type and device of a call, from its first matrix."""
    if not isinstance(first, torch.Tensor):
        raise TypeError(f"{first_name} must be a torch.Tensor")
    if first.dtype not in dtypes:
        raise TypeError(f"{first_name} must be float16 or bfloat16, got {first.dtype}")
    if first.device.type != "cuda":
        raise ValueError(f"{first_name} must be on a GPU device, got {first.device}")
    if first.dim() != 2:
        raise ValueError(f"{first_name} must be 2-D, got shape {tuple(first.shape)}")
    return first.dtype, first.device


def _check(name, t, shape, dtype, dev):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != dev:
        raise ValueError(f"{name} must be on {dev}, got {t.device}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{name} requires grad: these calls record no autograd node (use torch.no_grad() and the "
                         "backward call)")


def _matrix(name, t, shape, dtype, dev):
    """(address, row stride) of a 2-D tensor with unit stride along its rows."""
    # one test for the ordinary case; the messages come after it
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.device == dev and t.shape == shape
            and t.is_contiguous() and not t.requires_grad):
        return t.data_ptr(), shape[1]
    _check(name, t, shape, dtype, dev)
    s0, s1 = t.stride()
    if shape[1] > 1 and s1 != 1:
        raise ValueError(f"{name} must have unit stride along its rows, got strides {(s0, s1)}")
    if shape[0] <= 1:
        s0 = shape[1]
    elif s0 < shape[1]:
        raise ValueError(f"{name}'s rows overlap: row stride {s0} for {shape[1]} columns")
    return t.data_ptr(), s0


def _vector(name, t, n, dtype, dev):
    """The address of a contiguous vector, or 0 for None."""
    if t is None:
        return 0
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.device == dev and t.shape == (n,)
            and t.is_contiguous() and not t.requires_grad):
        return t.data_ptr()
    _check(name, t, (n,), dtype, dev)
    if n > 1 and t.stride(0) != 1:
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _kind(name, value, table):
    if value not in table:
        raise ValueError(f"{name} must be one of {tuple(table)}, got {value!r}")
    return table[value]


def linear(x, w, bias=None, residual=None, *, act="identity", save_z=False, stream=None):
    """D = act(x w^T + bias) + residual: x (M, K), w (N, K), bias (N,) and
    residual (M, N) or None.  Returns D, or (D, Z) with save_z, where
    Z = x w^T + bias is what linear_backward needs for the activation's
    derivative.  act: "identity", "relu", "gelu" (erf form) or "silu", applied to
    the unrounded Z.  M may be 0."""
    dtype, dev = _common("x", x)
    M, K = x.shape
    if not isinstance(w, torch.Tensor) or w.dim() != 2:
        raise ValueError("w must be a 2-D tensor (N, K)")
    N = w.shape[0]
    a = _kind("act", act, ACTS)
    xp = _matrix("x", x, (M, K), dtype, dev)
    wp = _matrix("w", w, (N, K), dtype, dev)
    bp = _vector("bias", bias, N, dtype, dev)
    rp = _matrix("residual", residual, (M, N), dtype, dev) if residual is not None else (0, 0)

    def call(raw):
        d = x.new_empty((M, N))
        z = torch.empty_like(d) if save_z else None
        _queue("ge_linear", _LINEAR.pack(M, N, K, *xp, *wp, bp, *rp, d.data_ptr(), N, z.data_ptr() if save_z else 0,
                                         N, a, _DTYPES[dtype]), dev, raw, (M, N, K))
        return (d, z) if save_z else d
    return _run(call, (x, w, bias, residual), dev, stream)


def linear_backward(dd, x, w, z=None, *, act="identity", need_dx=True, need_dw=True, need_dbias=True, stream=None):
    """Gradients of linear: dd (M, N), x (M, K), w (N, K) and z (M, N) as linear
    kept it (may be None for "identity").  Returns (dx, dw, dbias): dx (M, K) and
    dw (N, K) of the element type, dbias (N,) float32; None in the place of one
    that is not needed.  The residual's gradient is dd itself."""
    dtype, dev = _common("dd", dd)
    M, N = dd.shape
    if not isinstance(w, torch.Tensor) or w.dim() != 2:
        raise ValueError("w must be a 2-D tensor (N, K)")
    K = w.shape[1]
    a = _kind("act", act, ACTS)
    if not (need_dx or need_dw or need_dbias):
        return None, None, None
    if z is None and a != 0:
        raise ValueError(f"act {act!r} needs z")
    dp = _matrix("dd", dd, (M, N), dtype, dev)
    xp = _matrix("x", x, (M, K), dtype, dev)
    wp = _matrix("w", w, (N, K), dtype, dev)
    zp = _matrix("z", z, (M, N), dtype, dev) if z is not None else (0, 0)

    def call(raw):
        dx = dd.new_empty((M, K)) if need_dx else None
        dw = dd.new_empty((N, K)) if need_dw else None
        db = torch.empty((N,), dtype=torch.float32, device=dev) if need_dbias else None
        _queue("ge_linear_backward",
               _LINEAR_GRAD.pack(M, N, K, *dp, *xp, *wp, *zp, dx.data_ptr() if need_dx else 0, K,
                                 dw.data_ptr() if need_dw else 0, K, db.data_ptr() if need_dbias else 0, a,
                                 _DTYPES[dtype]), dev, raw, (M, N, K))
        return dx, dw, db
    return _run(call, (dd, x, w, z), dev, stream)


def linear_xent(x, w, target, *, ignore_index=-100, stream=None):
    """Softmax cross entropy of the logits x w^T, which are never stored: x
    (T, K), w (V, K), target (T,) int64.  Returns (loss, lse), both (T,) float32:
    lse = log sum exp of the row's logits, loss = lse - logit[target], 0 where
    the target is ignore_index, NaN where it is out of range otherwise."""
    dtype, dev = _common("x", x)
    T, K = x.shape
    if not isinstance(w, torch.Tensor) or w.dim() != 2:
        raise ValueError("w must be a 2-D tensor (V, K)")
    V = w.shape[0]
    xp = _matrix("x", x, (T, K), dtype, dev)
    wp = _matrix("w", w, (V, K), dtype, dev)
    if target is None:
        raise TypeError("target must be a torch.Tensor")
    tp = _vector("target", target, T, torch.int64, dev)

    def call(raw):
        loss = torch.empty((T,), dtype=torch.float32, device=dev)
        lse = torch.empty_like(loss)
        _queue("ge_linear_xent", _XENT.pack(T, V, K, *xp, *wp, tp, int(ignore_index), loss.data_ptr(),
                                            lse.data_ptr(), _DTYPES[dtype]), dev, raw, (T, V, K))
        return loss, lse
    return _run(call, (x, w, target), dev, stream)


def linear_xent_backward(dloss, x, w, target, lse, *, ignore_index=-100, need_dx=True, need_dw=True, stream=None):
    """Gradients of linear_xent: dloss (T,) float32, the forward's inputs and its
    lse.  Returns (dx, dw), x's and w's shape and type; None in the place of one
    that is not needed.  The logits are computed again, one piece of the
    vocabulary at a time."""
    dtype, dev = _common("x", x)
    T, K = x.shape
    if not isinstance(w, torch.Tensor) or w.dim() != 2:
        raise ValueError("w must be a 2-D tensor (V, K)")
    V = w.shape[0]
    if not (need_dx or need_dw):
        return None, None
    xp = _matrix("x", x, (T, K), dtype, dev)
    wp = _matrix("w", w, (V, K), dtype, dev)
    for name, t in (("dloss", dloss), ("target", target), ("lse", lse)):
        if t is None:
            raise TypeError(f"{name} must be a torch.Tensor")
    gp = _vector("dloss", dloss, T, torch.float32, dev)
    tp = _vector("target", target, T, torch.int64, dev)
    lp = _vector("lse", lse, T, torch.float32, dev)

    def call(raw):
        dx = x.new_empty((T, K)) if need_dx else None
        dw = x.new_empty((V, K)) if need_dw else None
        _queue("ge_linear_xent_backward",
               _XENT_GRAD.pack(T, V, K, gp, *xp, *wp, tp, lp, int(ignore_index), dx.data_ptr() if need_dx else 0, K,
                               dw.data_ptr() if need_dw else 0, K, _DTYPES[dtype]), dev, raw, (T, V, K))
        return dx, dw
    return _run(call, (dloss, x, w, target, lse), dev, stream)


def _norm_common(h, y, w_post, w_pre, gate, post, pre):
    dtype, dev = _common("y", y)
    T, H = y.shape
    if not isinstance(h, torch.Tensor) or h.dtype not in (dtype, torch.float32):
        raise TypeError(f"the residual stream must be {dtype} or float32")
    po, pr = _kind("post", post, NORMS), _kind("pre", pre, NORMS)
    if pr == 0:
        raise ValueError("pre must be 'rms' or 'layer'")
    if po == 0 and w_post is not None:
        raise ValueError("post 'none' takes no w_post")
    G, gp = 1, 0
    if gate is not None:
        if not isinstance(gate, torch.Tensor) or gate.dim() != 2:
            raise ValueError("gate must be a 2-D tensor (G, H)")
        G = gate.shape[0]
        if G < 1 or T % G:
            raise ValueError(f"gate has {G} rows, which do not divide {T}")
        gp, gs = _matrix("gate", gate, (G, H), dtype, dev)
        if G > 1 and gs != H:
            raise ValueError("gate must be contiguous")
    return dtype, dev, T, H, G, (_vector("w_post", w_post, H, dtype, dev), _vector("w_pre", w_pre, H, dtype, dev),
                                 gp, po, pr)


def norm_residual(h, y, *, w_post=None, w_pre=None, gate=None, scale=1.0, post="rms", pre="rms", eps=1e-5,
                  stream=None):
    """The residual step between two blocks: h' = h + scale * gate *
    norm_post(y), x = norm_pre(h').  h (T, H) of y's type or float32, y (T, H);
    w_post, w_pre (H,) and gate (G, H) of y's type or None (ones); row t takes
    gate row t // (T / G).  Norms: "rms" v / sqrt(mean v^2 + eps), "layer"
    (v - mean) / sqrt(var + eps), each times its weight; post may be "none".
    Returns (h', x): h's and y's type."""
    dtype, dev, T, H, G, mid = _norm_common(h, y, w_post, w_pre, gate, post, pre)
    sd = h.dtype
    hp = _matrix("h", h, (T, H), sd, dev)
    yp = _matrix("y", y, (T, H), dtype, dev)

    def call(raw):
        ho = torch.empty_like(h) if hp[1] == H else h.new_empty((T, H))
        x = torch.empty_like(y) if yp[1] == H else y.new_empty((T, H))
        _queue("ge_norm_residual", _NORM.pack(T, H, G, *hp, *yp, *mid, scale, eps, ho.data_ptr(), H, x.data_ptr(), H,
                                              _DTYPES[dtype], _STREAM_DTYPES[sd]), dev, raw)
        return ho, x
    return _run(call, (h, y, w_post, w_pre, gate), dev, stream)


def norm_residual_backward(dx, dh_out, h_out, y, *, w_post=None, w_pre=None, gate=None, scale=1.0, post="rms",
                           pre="rms", eps=1e-5, stream=None):
    """Gradients of norm_residual from those of its outputs, dx and dh_out, its
    output h_out and its input y.  Returns (dh, dy, dw_post, dw_pre, dgate): dh
    of the stream's type, dy of y's, the rest float32, None for a weight or gate
    that was None."""
    dtype, dev, T, H, G, mid = _norm_common(h_out, y, w_post, w_pre, gate, post, pre)
    sd = h_out.dtype
    dxp = _matrix("dx", dx, (T, H), dtype, dev)
    dhp = _matrix("dh_out", dh_out, (T, H), sd, dev)
    hp = _matrix("h_out", h_out, (T, H), sd, dev)
    yp = _matrix("y", y, (T, H), dtype, dev)

    def call(raw):
        def new32(shape):
            return torch.empty(shape, dtype=torch.float32, device=dev)
        dh, dy = h_out.new_empty((T, H)), y.new_empty((T, H))
        dwo = new32((H,)) if w_post is not None else None
        dwi = new32((H,)) if w_pre is not None else None
        dg = new32((G, H)) if gate is not None else None
        _queue("ge_norm_residual_backward",
               _NORM_GRAD.pack(T, H, G, *dxp, *dhp, *hp, *yp, *mid, scale, eps, dh.data_ptr(), H, dy.data_ptr(), H,
                               *(t.data_ptr() if t is not None else 0 for t in (dwo, dwi, dg)), _DTYPES[dtype],
                               _STREAM_DTYPES[sd]), dev, raw, (T, H, G))
        return dh, dy, dwo, dwi, dg
    return _run(call, (dx, dh_out, h_out, y, w_post, w_pre, gate), dev, stream)
