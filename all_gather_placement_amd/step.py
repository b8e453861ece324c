"""Binding of libtide_step.so (include/tide_step.h): the training-step operators next to the
collectives -- global gradient norm and clipping, layer norm, embedding, tokens sorted by expert and
back, rotary positions, dropout, with their gradients.

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
from typing import NamedTuple

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
        "tide_expert_rows": (i64, [i64, i32, i32, i32]),
        "tide_expert_sort_workspace": (i64, [i64, i32, i32]),
        "tide_expert_sort": (i32, [i64, i32, vp, i32, i32, i32, vp, vp, i64, vp, vp, i64, vp]),
        "tide_expert_dispatch": (i32, [i64, i32, i64, vp, i64, i32, vp, vp, i64, vp, i64, vp]),
        "tide_expert_combine": (i32, [i64, i32, i64, vp, i64, i64, i32, vp, i32, vp, vp, i64, vp]),
        "tide_expert_combine_bwd": (i32, [i64, i32, i64, vp, i64, vp, i64, i64, i32, vp, i32, vp, vp, vp, i64, vp, vp]),
        "tide_rotary": (i32, [i64, i64, i64, vp, i64, i64, i32, vp, i32, i32, vp, vp, i32, i32, vp, i64, i64, vp]),
        "tide_dropout": (i32, [i64, i64, vp, i64, i32, f64, ctypes.c_uint64, vp, i64, vp, i64, vp, i64, vp]),
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


# ------------------------------------------------------------------------------------------------
# Experts of a mixture
# ------------------------------------------------------------------------------------------------

class ExpertSort(NamedTuple):
    """(token, choice) pairs in the order of their experts; int32 tensors.

    place    [..., choices]: each pair's row of the sorted buffer, -1 for a pair without an expert
    source   [rows]: the number token * choices + choice of each row's pair, -1 for a row of no pair
    offsets  [num_experts + 1]: where each expert's rows start
    """
    place: object
    source: object
    offsets: object


def expert_sort(experts, num_experts, align=1, place=None, source=None, offsets=None, workspace=None, stream=None):
    """The order of (token, choice) pairs by expert, as an :class:`ExpertSort`.  `experts`: contiguous int32
    or int64, [..., choices]; ids outside [0, num_experts) -- padded tokens, another rank's experts -- have
    no row.  Each expert's rows start on a multiple of `align`, and its pairs keep their order.  There are
    rows for any ids of this shape; a `source` passed in may have more."""
    if stream is None:
        return ExpertSort._make((_step or load_step_binding()).expert_sort(experts, num_experts, align, place, source,
                                                                           offsets, workspace))
    return ExpertSort._make(_call("expert_sort", stream, experts, num_experts, align, place, source, offsets,
                                  workspace))


def expert_dispatch(x, sort, out=None, stream=None):
    """The tokens' vectors in the order of `sort`, an :class:`ExpertSort`: [rows, dim], zeros in rows of no
    pair.  x is [..., dim], bf16 or fp32, contiguous or a matrix whose rows are."""
    if stream is None:
        return (_step or load_step_binding()).expert_dispatch(x, sort, out)
    return _call("expert_dispatch", stream, x, sort, out)


def expert_dispatch_bwd(drows, sort, out=None, stream=None):
    """Gradient of :func:`expert_dispatch` with respect to x: each token's rows of `drows` [rows, dim], added
    up in fp32 in the order of its choices."""
    return expert_combine(drows, None, sort, out, stream)


def expert_combine(rows, weights, sort, out=None, stream=None):
    """The sorted buffer's rows [rows, dim] back at their tokens, [..., dim]: the sum over a token's choices
    of weights * row, in fp32.  `weights` is [..., choices], bf16 or fp32, or None for ones; those of pairs
    without a row are not used, and a token without rows is zeros."""
    if stream is None:
        return (_step or load_step_binding()).expert_combine(rows, weights, sort, out)
    return _call("expert_combine", stream, rows, weights, sort, out)


def expert_combine_bwd(dy, rows, weights, sort, drows=None, dweights=None, stream=None):
    """Gradients (drows, dweights) of :func:`expert_combine`: weights * dy at each pair's row, zeros in rows
    of no pair (`drows` may be `rows` itself), and the products of dy with the rows, 0 for pairs without one."""
    if stream is None:
        return (_step or load_step_binding()).expert_combine_bwd(dy, rows, weights, sort, drows, dweights)
    return _call("expert_combine_bwd", stream, dy, rows, weights, sort, drows, dweights)


# ------------------------------------------------------------------------------------------------
# Rotary positions
# ------------------------------------------------------------------------------------------------

def rotary_freqs(sections, base=10000.0, shared=False, device=None):
    """Frequencies for :func:`rotary`, fp64 on the current device: with n pairs in an axis's section, pair i
    of it turns by base ** (-i / n) for each step; with `shared` all sections share one such ramp."""
    import torch

    counts = [sum(sections)] if shared else list(sections)
    ramps = [torch.arange(n, dtype=torch.float64) / n for n in counts]
    return (float(base) ** -torch.cat(ramps)).to(device if device is not None else torch.device("cuda"))


def rotary(x, positions, freqs, sections, pairing="halves", out=None, stream=None):
    """Pairs of a head's elements turned by positions[axis] * freqs[pair], the angle (up to 2^64) taken in 64 bits.

    x is [..., heads, dim], bf16 or fp32, contiguous, or [tokens, heads, dim] whose vectors are; `out` may be
    x itself.  positions is [axes, ...] for the tokens, contiguous int32, int64 or fp32 (text: one axis;
    video: time, height, width); sections tells how many pairs turn with each axis, one after the other;
    freqs (fp64) has the pairs' frequencies (:func:`rotary_freqs`).  Of P pairs, pair i is elements i and
    P + i ("halves") or 2 i and 2 i + 1 ("neighbours"); elements from 2 P on are copied."""
    if stream is None:
        return (_step or load_step_binding()).rotary(x, positions, freqs, sections, pairing, False, out)
    return _call("rotary", stream, x, positions, freqs, sections, pairing, False, out)


def rotary_bwd(dy, positions, freqs, sections, pairing="halves", out=None, stream=None):
    """Gradient of :func:`rotary` with respect to x: dy turned back.  `out` may be dy itself.  Heads that were one
    vector read several times (an expanded x) have a gradient each; their sum is that vector's."""
    if stream is None:
        return (_step or load_step_binding()).rotary(dy, positions, freqs, sections, pairing, True, out)
    return _call("rotary", stream, dy, positions, freqs, sections, pairing, True, out)


# ------------------------------------------------------------------------------------------------
# Dropout
# ------------------------------------------------------------------------------------------------

def dropout(x, p, seed, offset=0, residual=None, out=None, stream=None):
    """x / (1 - p) where an element is kept and 0 where it is dropped, plus `residual`; x is bf16 or fp32,
    contiguous or a matrix whose rows are.

    Whether element e of x is dropped depends on `seed` and offset + e alone (Philox4x32-10, 16 bits an
    element: the probability is p rounded to a multiple of 2 ** -16, and the scale is that probability's), so
    the mask is never stored: the same seed and offset give it again.  `seed` is a number of 64 bits or an
    int64 tensor of one value on the device, which a captured call reads at every replay.  `offset` counts
    elements: parts of a tensor, on one rank or several, are dropped as the whole would be, and calls that
    share a seed take numbers apart.  `out` may be x or the residual."""
    if stream is None:
        return (_step or load_step_binding()).dropout(x, p, seed, offset, residual, out)
    return _call("dropout", stream, x, p, seed, offset, residual, out)


def dropout_bwd(dy, p, seed, offset=0, out=None, stream=None):
    """Gradient of :func:`dropout` with respect to x (that of the residual is dy); `out` may be dy itself."""
    return dropout(dy, p, seed, offset, None, out, stream)
