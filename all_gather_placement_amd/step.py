"""ctypes binding of libtide_step.so (include/tide_step.h): the training-step operators next to the
collectives -- global gradient norm and clipping, layer norm, embedding, with their gradients.

Tensors are torch tensors on the current HIP device.  Outputs and workspaces may be passed in; those
that are not are allocated with torch on the stream the call runs on.  Every call only enqueues
kernels on `stream` (default: torch's current stream), raises ValueError for arguments that do not
fit together and :class:`~all_gather_placement_amd.tide.TideError` for what the library refuses.
There is no fallback: if the library is missing, every call raises.

A caller that passes its own buffers and a stream other than the current one orders their use itself,
as for any call on another stream.
"""
from __future__ import annotations

import ctypes
import os
from array import array

from .tide import TIDE_OK, TideError, _stream_handle

_PKG = os.path.dirname(os.path.abspath(__file__))
TIDE_BF16 = 0
TIDE_FP32 = 1
TIDE_INT32 = 2
TIDE_INT64 = 3
_lib = None
_torch = None
_dtypes = {}
_id_dtypes = {}


def step_library_path() -> str:
    return os.path.join(_PKG, "libtide_step.so")


def load_step_library():
    """Load libtide_step.so (once).  Raises if it is not built, or built from other sources."""
    global _lib, _torch
    if _lib is not None:
        return _lib
    path = step_library_path()
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is not built; run `python -m all_gather_placement_amd.build`")
    import torch

    from .build import STEP_LIB, check_current
    from .tide import load_library

    load_library()  # names the status codes
    lib = ctypes.CDLL(path)
    check_current(STEP_LIB, loaded=lib)
    vp, i32, i64, f32, f64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_double
    sig = {
        "tide_grad_norm_workspace": (i64, [i32, vp, i32]),
        "tide_grad_norm": (i32, [i32, vp, vp, i32, vp, vp, vp, i64, vp]),
        "tide_grad_clip": (i32, [i32, vp, vp, vp, i32, vp, f64, vp, vp]),
        "tide_clip_grad_norm": (i32, [i32, vp, vp, vp, i32, f64, vp, vp, vp, i64, vp]),
        "tide_layer_norm": (i32, [i64, i64, vp, i64, i32, vp, vp, i32, f32, vp, i64, vp, vp, vp]),
        "tide_layer_norm_bwd_workspace": (i64, [i64, i64, i32]),
        "tide_layer_norm_bwd": (i32, [i64, i64, vp, i64, vp, i64, i32, vp, i32, vp, vp, vp, i64, vp, vp, vp, i64, vp]),
        "tide_embedding": (i32, [i64, vp, i32, i64, i64, vp, i32, f32, vp, vp]),
        "tide_embedding_bwd_workspace": (i64, [i64, i64, i64]),
        "tide_embedding_bwd": (i32, [i64, vp, i32, i64, i64, vp, i32, f32, i32, vp, vp, i64, vp]),
        "tide_step_last_hip_error": (i32, []),
        "tide_step_build_id": (ctypes.c_char_p, []),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _torch = torch
    _dtypes.update({torch.bfloat16: TIDE_BF16, torch.float32: TIDE_FP32})
    _id_dtypes.update({torch.int32: TIDE_INT32, torch.int64: TIDE_INT64})
    _lib = lib
    return lib


def _check(status: int, where: str):
    if status != TIDE_OK:
        raise TideError(status, where, _lib.tide_step_last_hip_error() if status == 3 else 0)


def _on(stream):
    """Context in which torch allocates for `stream`."""
    if isinstance(stream, int):
        stream = _torch.cuda.ExternalStream(stream)
    return _torch.cuda.stream(stream)  # None: the current one


def _empty(shape, dtype, device, stream):
    if stream is None:
        return _torch.empty(shape, dtype=dtype, device=device)
    with _on(stream):
        return _torch.empty(shape, dtype=dtype, device=device)


def _need(cond, message):
    if not cond:
        raise ValueError(message)


def _expect(t, name, dtypes, shape=None, contiguous=True):
    """A cuda tensor on the current device, of one of `dtypes` and, if given, of this shape."""
    if not t.is_cuda or t.device.index != _torch.cuda.current_device():
        raise ValueError(f"{name} must be on the current device (cuda:{_torch.cuda.current_device()}), got {t.device}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be of {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _ptr(t):
    return None if t is None else t.data_ptr()


def _workspace(workspace, need, device, stream, where):
    """(tensor, bytes): the caller's workspace if it is large enough, else a new one."""
    if need < 0:
        raise TideError(1, where)
    if workspace is None:
        return _empty((need,), _torch.uint8, device, stream), need
    _expect(workspace, "workspace", (_torch.uint8,))
    _need(workspace.numel() >= need, f"workspace must hold {need} bytes, got {workspace.numel()}")
    return workspace, workspace.numel()


# ------------------------------------------------------------------------------------------------
# Gradient norm and clipping
# ------------------------------------------------------------------------------------------------

def _tensors(grads, name):
    """(addresses, element counts, type code, device) of a list of like tensors, checked."""
    kinds = {(g.dtype, g.device) for g in grads}
    if not kinds:
        return array("Q"), array("q"), TIDE_FP32, _torch.device("cuda", _torch.cuda.current_device())
    _need(len(kinds) == 1, f"all {name} must have one dtype and device, got {sorted(map(str, kinds))}")
    _expect(grads[0], name, tuple(_dtypes))
    _need(all([g.is_contiguous() for g in grads]), f"all {name} must be contiguous")
    dtype, device = kinds.pop()
    return array("Q", [g.data_ptr() for g in grads]), array("q", [g.numel() for g in grads]), _dtypes[dtype], device


def _addr(a):
    return a.buffer_info()[0]


def _scalars(norm, sumsq, device, stream):
    if norm is None:
        norm = _empty((), _torch.float32, device, stream)
    _expect(norm, "norm", (_torch.float32,))
    _need(norm.numel() == 1, "norm must hold one value")
    if sumsq is not None:
        _expect(sumsq, "sumsq", (_torch.float64,))
        _need(sumsq.numel() == 1, "sumsq must hold one value")
    return norm


def grad_norm(grads, norm=None, sumsq=None, workspace=None, stream=None):
    """L2 norm over a list of contiguous bf16 or fp32 tensors, as an fp32 tensor of one value (`norm`
    if given).  `sumsq`, an fp64 tensor of one value, also receives the sum of squares: a data-parallel
    job all-reduces it and clips by :func:`grad_clip`."""
    lib = load_step_library()
    ptrs, numels, dtype, device = _tensors(grads, "grads")
    norm = _scalars(norm, sumsq, device, stream)
    need = lib.tide_grad_norm_workspace(len(ptrs), _addr(numels), dtype)
    ws, size = _workspace(workspace, need, device, stream, "tide_grad_norm")
    _check(lib.tide_grad_norm(len(ptrs), _addr(ptrs), _addr(numels), dtype, _ptr(sumsq), norm.data_ptr(),
                              ws.data_ptr(), size, _stream_handle(stream)), "tide_grad_norm")
    return norm


def _outs(grads, outs, numels):
    if outs is None:
        return None
    optrs, onumels, _, _ = _tensors(outs, "outs")
    _need(len(outs) == len(grads) and onumels == numels, "outs must have the gradients' sizes")
    _need(not grads or (outs[0].dtype == grads[0].dtype and outs[0].device == grads[0].device),
          "outs must have the gradients' dtype and device")
    return optrs


def grad_clip(grads, sumsq, max_norm, outs=None, norm=None, stream=None):
    """outs[i] = grads[i] * min(1, max_norm / (sqrt(sumsq) + 1e-6)); in place without `outs`.  Returns
    sqrt(sumsq) as an fp32 tensor of one value."""
    lib = load_step_library()
    ptrs, numels, dtype, device = _tensors(grads, "grads")
    optrs = _outs(grads, outs, numels)
    norm = _scalars(norm, sumsq, device, stream)
    _check(lib.tide_grad_clip(len(ptrs), _addr(ptrs), _addr(ptrs if optrs is None else optrs), _addr(numels), dtype,
                              sumsq.data_ptr(), max_norm, norm.data_ptr(), _stream_handle(stream)), "tide_grad_clip")
    return norm


def clip_grad_norm(grads, max_norm, outs=None, norm=None, sumsq=None, workspace=None, stream=None):
    """:func:`grad_norm` and :func:`grad_clip` by it in one call, for gradients that are all on this
    device: outs[i] = grads[i] * min(1, max_norm / (norm + 1e-6)); in place without `outs`.  Returns the
    norm before clipping."""
    lib = load_step_library()
    ptrs, numels, dtype, device = _tensors(grads, "grads")
    optrs = _outs(grads, outs, numels)
    norm = _scalars(norm, sumsq, device, stream)
    need = lib.tide_grad_norm_workspace(len(ptrs), _addr(numels), dtype)
    ws, size = _workspace(workspace, need, device, stream, "tide_clip_grad_norm")
    _check(lib.tide_clip_grad_norm(len(ptrs), _addr(ptrs), _addr(ptrs if optrs is None else optrs), _addr(numels),
                                   dtype, max_norm, _ptr(sumsq), norm.data_ptr(), ws.data_ptr(), size,
                                   _stream_handle(stream)), "tide_clip_grad_norm")
    return norm


# ------------------------------------------------------------------------------------------------
# Layer norm
# ------------------------------------------------------------------------------------------------

def _matrix(t, name, dtypes, shape=None):
    """(rows, cols, row stride) of a tensor as rows of its last dimension."""
    _expect(t, name, dtypes, shape, contiguous=False)
    _need(t.dim() >= 1, f"{name} must have at least one dimension")
    cols = t.shape[-1]
    _need(cols >= 1, f"{name} must have a last dimension of at least one")
    rows = t.numel() // cols
    if t.is_contiguous():
        return rows, cols, cols
    _need(t.dim() == 2 and (t.stride(1) == 1 or cols == 1) and t.stride(0) >= cols,
          f"{name} must be contiguous, or a matrix whose rows are")
    return rows, cols, t.stride(0)


def _vector(t, name, cols, dtypes):
    if t is not None:
        _expect(t, name, dtypes, (cols,))


def _param_dtype(x, *params):
    kinds = {p.dtype for p in params if p is not None}
    _need(len(kinds) <= 1, "weight, bias and their gradients must have one dtype")
    return kinds.pop() if kinds else x.dtype


def layer_norm(x, weight=None, bias=None, eps=1e-5, out=None, mean=None, rstd=None, stream=None):
    """Layer norm over the last dimension of a bf16 or fp32 tensor; weight and bias are bf16 or fp32.
    Returns (y, mean, rstd): y of x's dtype and shape, the row statistics in fp32, one for each row."""
    lib = load_step_library()
    rows, cols, xs = _matrix(x, "x", tuple(_dtypes))
    _vector(weight, "weight", cols, tuple(_dtypes))
    _vector(bias, "bias", cols, tuple(_dtypes))
    pdtype = _param_dtype(x, weight, bias)
    if out is None:
        out = _empty(x.shape, x.dtype, x.device, stream)
    ys = _matrix(out, "out", (x.dtype,), x.shape)[2]
    if mean is None:
        mean = _empty(x.shape[:-1], _torch.float32, x.device, stream)
    if rstd is None:
        rstd = _empty(x.shape[:-1], _torch.float32, x.device, stream)
    _expect(mean, "mean", (_torch.float32,), x.shape[:-1])
    _expect(rstd, "rstd", (_torch.float32,), x.shape[:-1])
    _check(lib.tide_layer_norm(rows, cols, x.data_ptr(), xs, _dtypes[x.dtype], _ptr(weight), _ptr(bias),
                               _dtypes[pdtype], eps, out.data_ptr(), ys, mean.data_ptr(), rstd.data_ptr(),
                               _stream_handle(stream)), "tide_layer_norm")
    return out, mean, rstd


def layer_norm_bwd(dy, x, weight, mean, rstd, dx=None, dweight=None, dbias=None, workspace=None, stream=None):
    """Gradients (dx, dweight, dbias) of :func:`layer_norm`.  `weight` may be None (dweight and dbias are
    then of x's dtype); `dx` may be `dy` itself.  dweight and dbias may be gradients of a parameter group
    that the reduce-scatter reads in place."""
    lib = load_step_library()
    rows, cols, xs = _matrix(x, "x", tuple(_dtypes))
    dys = _matrix(dy, "dy", (x.dtype,), x.shape)[2]
    _vector(weight, "weight", cols, tuple(_dtypes))
    _expect(mean, "mean", (_torch.float32,), x.shape[:-1])
    _expect(rstd, "rstd", (_torch.float32,), x.shape[:-1])
    _vector(dweight, "dweight", cols, tuple(_dtypes))
    _vector(dbias, "dbias", cols, tuple(_dtypes))
    pdtype = _param_dtype(x, weight, dweight, dbias)
    if dx is None:
        dx = _empty(x.shape, x.dtype, x.device, stream)
    dxs = _matrix(dx, "dx", (x.dtype,), x.shape)[2]
    if dweight is None:
        dweight = _empty((cols,), pdtype, x.device, stream)
    if dbias is None:
        dbias = _empty((cols,), pdtype, x.device, stream)
    need = lib.tide_layer_norm_bwd_workspace(rows, cols, _dtypes[x.dtype])
    ws, size = _workspace(workspace, need, x.device, stream, "tide_layer_norm_bwd")
    _check(lib.tide_layer_norm_bwd(rows, cols, dy.data_ptr(), dys, x.data_ptr(), xs, _dtypes[x.dtype], _ptr(weight),
                                   _dtypes[pdtype], mean.data_ptr(), rstd.data_ptr(), dx.data_ptr(), dxs,
                                   dweight.data_ptr(), dbias.data_ptr(), ws.data_ptr(), size, _stream_handle(stream)),
           "tide_layer_norm_bwd")
    return dx, dweight, dbias


# ------------------------------------------------------------------------------------------------
# Embedding
# ------------------------------------------------------------------------------------------------

def embedding(ids, table, scale=1.0, out=None, stream=None):
    """table[ids] * scale, of shape ids.shape + (dim,); zeros for ids outside the table.  ids int32 or
    int64 of any shape, table a [vocab, dim] bf16 or fp32 tensor; both contiguous."""
    lib = load_step_library()
    _expect(ids, "ids", tuple(_id_dtypes))
    _expect(table, "table", tuple(_dtypes))
    _need(table.dim() == 2 and table.shape[1] >= 1, "table must be [vocab, dim] with dim at least one")
    vocab, dim = table.shape
    shape = (*ids.shape, dim)
    if out is None:
        out = _empty(shape, table.dtype, table.device, stream)
    _expect(out, "out", (table.dtype,), shape)
    _check(lib.tide_embedding(ids.numel(), ids.data_ptr(), _id_dtypes[ids.dtype], vocab, dim, table.data_ptr(),
                              _dtypes[table.dtype], scale, out.data_ptr(), _stream_handle(stream)), "tide_embedding")
    return out


def embedding_bwd(ids, dy, vocab, scale=1.0, out=None, accumulate=False, workspace=None, stream=None):
    """Gradient of :func:`embedding` with respect to the table: [vocab, dim] of dy's dtype, every row
    written; with `accumulate` it is added to `out`, and rows of no token stay as they are."""
    lib = load_step_library()
    _expect(ids, "ids", tuple(_id_dtypes))
    _expect(dy, "dy", tuple(_dtypes))
    _need(dy.dim() >= 1 and tuple(dy.shape[:-1]) == tuple(ids.shape), "dy must have shape ids.shape + (dim,)")
    dim = dy.shape[-1]
    _need(dim >= 1, "dy must have a last dimension of at least one")
    _need(out is not None or not accumulate, "accumulate needs the gradient to add to as `out`")
    if out is None:
        out = _empty((vocab, dim), dy.dtype, dy.device, stream)
    _expect(out, "out", (dy.dtype,), (vocab, dim))
    need = lib.tide_embedding_bwd_workspace(ids.numel(), vocab, dim)
    ws, size = _workspace(workspace, need, dy.device, stream, "tide_embedding_bwd")
    _check(lib.tide_embedding_bwd(ids.numel(), ids.data_ptr(), _id_dtypes[ids.dtype], vocab, dim, dy.data_ptr(),
                                  _dtypes[dy.dtype], scale, int(accumulate), out.data_ptr(), ws.data_ptr(), size,
                                  _stream_handle(stream)), "tide_embedding_bwd")
    return out
