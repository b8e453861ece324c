"""Binding of libtide_step.so (include/tide_step.h): the training-step operators next to the
collectives -- global gradient norm and clipping, layer norm, embedding, with their gradients.

Tensors are torch tensors on the current HIP device.  Outputs and workspaces may be passed in; those
that are not are allocated with torch on the stream the call runs on.  Every call only enqueues
kernels on `stream` (default: torch's current stream; a torch stream or a hipStream_t as int), raises
ValueError for arguments that do not fit together and :class:`~all_gather_placement_amd.tide.TideError`
for what the library refuses.  There is no fallback: if the library is missing, every call raises.

The functions here are the documentation of a compiled module, ``_step.so``, which checks and allocates;
it calls the C ABI of the library that :func:`load_step_library` loads.

Gradients are calls of their own: no call is recorded by autograd, so what it returns has no history,
whether or not its inputs require grad.  Outputs passed in count as written in place, as by torch's own
in-place functions.

A caller that passes its own buffers and a stream other than the current one orders their use itself,
as for any call on another stream.
"""
from __future__ import annotations

import ctypes
import os

from .tide import TideError

_PKG = os.path.dirname(os.path.abspath(__file__))
TIDE_BF16 = 0
TIDE_FP32 = 1
TIDE_INT32 = 2
TIDE_INT64 = 3
_lib = None
_step = None  # the compiled module


def step_library_path() -> str:
    return os.path.join(_PKG, "libtide_step.so")


def load_step_library():
    """Load libtide_step.so (once).  Raises if it is not built, or built from other sources."""
    global _lib
    if _lib is not None:
        return _lib
    path = step_library_path()
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is not built; run `python -m all_gather_placement_amd.build`")
    import torch  # noqa: F401 (its HIP runtime is loaded first)

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
    _lib = lib
    return lib


def load_step_binding():
    """The compiled module, loaded once together with the library.  Raises if either is not built, or
    built from other sources."""
    global _step
    if _step is None:
        load_step_library()
        import torch

        from .build import STEP_BINDING, check_current

        if not os.path.exists(STEP_BINDING):
            raise RuntimeError(f"{STEP_BINDING} is not built; run `python -m all_gather_placement_amd.build` where "
                               "torch is installed")
        check_current(STEP_BINDING)
        from . import _step as module

        module.configure(TideError, torch._C._cuda_getCurrentRawStream)
        _step = module
    return _step


def _call(name, stream, *args):
    """A call with `stream` as torch's current stream, on which it allocates and runs."""
    import torch

    with torch.cuda.stream(torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream):
        return getattr(load_step_binding(), name)(*args)


def _init(grads):
    try:
        none = len(grads) == 0
    except TypeError:  # an iterator
        none = True
    if none:  # no tensor tells that the device is in use
        import torch

        torch.cuda.init()


# ------------------------------------------------------------------------------------------------
# Gradient norm and clipping
# ------------------------------------------------------------------------------------------------

def grad_norm(grads, norm=None, sumsq=None, workspace=None, stream=None):
    """L2 norm over a list (or other iterable) of contiguous bf16 or fp32 tensors, as an fp32 tensor of one
    value (`norm` if given).  `sumsq`, an fp64 tensor of one value, also receives the sum of squares: a
    data-parallel job all-reduces it and clips by :func:`grad_clip`."""
    _init(grads)
    if stream is None:
        return (_step or load_step_binding()).grad_norm(grads, norm, sumsq, workspace)
    return _call("grad_norm", stream, grads, norm, sumsq, workspace)


def grad_clip(grads, sumsq, max_norm, outs=None, norm=None, stream=None):
    """outs[i] = grads[i] * min(1, max_norm / (sqrt(sumsq) + 1e-6)); in place without `outs`.  Returns
    sqrt(sumsq) as an fp32 tensor of one value."""
    if stream is None:
        return (_step or load_step_binding()).grad_clip(grads, sumsq, max_norm, outs, norm)
    return _call("grad_clip", stream, grads, sumsq, max_norm, outs, norm)


def clip_grad_norm(grads, max_norm, outs=None, norm=None, sumsq=None, workspace=None, stream=None):
    """:func:`grad_norm` and :func:`grad_clip` by it in one call, for gradients that are all on this
    device: outs[i] = grads[i] * min(1, max_norm / (norm + 1e-6)); in place without `outs`.  Returns the
    norm before clipping."""
    _init(grads)
    if stream is None:
        return (_step or load_step_binding()).clip_grad_norm(grads, max_norm, outs, norm, sumsq, workspace)
    return _call("clip_grad_norm", stream, grads, max_norm, outs, norm, sumsq, workspace)


# ------------------------------------------------------------------------------------------------
# Layer norm
# ------------------------------------------------------------------------------------------------

def layer_norm(x, weight=None, bias=None, eps=1e-5, out=None, mean=None, rstd=None, stream=None):
    """Layer norm over the last dimension of a bf16 or fp32 tensor that is contiguous, or a matrix whose
    rows are; weight and bias are bf16 or fp32.  Returns (y, mean, rstd): y of x's dtype and shape, the
    row statistics in fp32, one for each row."""
    if stream is None:
        return (_step or load_step_binding()).layer_norm(x, weight, bias, eps, out, mean, rstd)
    return _call("layer_norm", stream, x, weight, bias, eps, out, mean, rstd)


def layer_norm_bwd(dy, x, weight, mean, rstd, dx=None, dweight=None, dbias=None, workspace=None, stream=None):
    """Gradients (dx, dweight, dbias) of :func:`layer_norm`.  `weight` may be None (dweight and dbias are
    then of x's dtype); `dx` may be `dy` itself.  dweight and dbias may be gradients of a parameter group
    that the reduce-scatter reads in place."""
    if stream is None:
        return (_step or load_step_binding()).layer_norm_bwd(dy, x, weight, mean, rstd, dx, dweight, dbias, workspace)
    return _call("layer_norm_bwd", stream, dy, x, weight, mean, rstd, dx, dweight, dbias, workspace)


# ------------------------------------------------------------------------------------------------
# Embedding
# ------------------------------------------------------------------------------------------------

def embedding(ids, table, scale=1.0, out=None, stream=None):
    """table[ids] * scale, of shape ids.shape + (dim,); zeros for ids outside the table.  ids int32 or
    int64 of any shape, table a [vocab, dim] bf16 or fp32 tensor; both contiguous."""
    if stream is None:
        return (_step or load_step_binding()).embedding(ids, table, scale, out)
    return _call("embedding", stream, ids, table, scale, out)


def embedding_bwd(ids, dy, vocab, scale=1.0, out=None, accumulate=False, workspace=None, stream=None):
    """Gradient of :func:`embedding` with respect to the table: [vocab, dim] of dy's dtype, every row
    written; with `accumulate` it is added to `out`, and rows of no token stay as they are."""
    if stream is None:
        return (_step or load_step_binding()).embedding_bwd(ids, dy, vocab, scale, out, accumulate, workspace)
    return _call("embedding_bwd", stream, ids, dy, vocab, scale, out, accumulate, workspace)
