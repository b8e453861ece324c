"""Host-side checks of libtide_step.so (no GPU): exported symbols, workspace sizes, and the refusal of
bad arguments before any work is enqueued (made-up addresses are never touched)."""
import ctypes
import math
import os
import re
import shutil
import subprocess

import pytest

import all_gather_placement_amd as tide
from all_gather_placement_amd import step

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID = 0, 1
A = 1 << 20  # made-up, aligned device addresses, far apart
FAR = 1 << 40


def lib():
    return tide.load_step_library()


def test_library_exports_every_declared_symbol():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "tide_step.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(tide_[a-z0-9_]+)\s*\(", text))
    assert {"tide_grad_norm", "tide_layer_norm_bwd", "tide_embedding_bwd"} <= names
    for n in names:
        assert hasattr(lib(), n), n
    for n in ("grad_norm", "grad_clip", "clip_grad_norm", "layer_norm", "layer_norm_bwd", "embedding", "embedding_bwd"):
        assert callable(getattr(tide, n))


def i64s(*v):
    return (ctypes.c_int64 * max(len(v), 1))(*v)


def ptrs(*v):
    return (ctypes.c_void_p * max(len(v), 1))(*v)


def test_norm_workspace_sizes():
    f = lib().tide_grad_norm_workspace
    assert f(0, None, 0) >= 0 and f(2, i64s(0, 0), 1) >= 0
    assert f(1, i64s(1), 0) >= 8 and f(1000, i64s(*[100] * 1000), 1) >= 8000
    assert f(-1, None, 0) == -1 and f(1, None, 0) == -1 and f(1, i64s(-1), 0) == -1 and f(1, i64s(1), 2) == -1
    assert f(1, i64s(1 << 43), 0) == -1 and f(2, i64s(1 << 62, 1 << 62), 0) == -1


def norm(n=1, grads=None, numels=None, dtype=1, sumsq=8 * A, out=9 * A, ws=10 * A, size=1 << 20):
    return lib().tide_grad_norm(n, ptrs(A) if grads is None else grads, i64s(64) if numels is None else numels, dtype,
                                sumsq, out, ws, size, None)


def test_norm_refusals():
    assert norm(n=-1) == INVALID
    assert norm(dtype=2) == INVALID and norm(dtype=-1) == INVALID
    assert norm(grads=ptrs(None)) == INVALID and norm(grads=ptrs(A + 2)) == INVALID
    assert norm(dtype=0, grads=ptrs(A + 1)) == INVALID
    assert norm(numels=i64s(-5)) == INVALID
    assert norm(sumsq=8 * A + 4) == INVALID and norm(out=9 * A + 2) == INVALID
    assert norm(ws=None) == INVALID and norm(ws=10 * A + 8) == INVALID and norm(size=8) == INVALID
    assert lib().tide_grad_norm(1, None, i64s(4), 1, None, None, 10 * A, 1 << 20, None) == INVALID
    assert lib().tide_grad_norm(1, ptrs(A), None, 1, None, None, 10 * A, 1 << 20, None) == INVALID


def clip(n=2, grads=None, outs=None, numels=None, dtype=1, sumsq=FAR, max_norm=1.0, out=FAR + 64):
    return lib().tide_grad_clip(n, ptrs(A, 2 * A) if grads is None else grads,
                                ptrs(A, 2 * A) if outs is None else outs,
                                i64s(64, 64) if numels is None else numels, dtype, sumsq, max_norm, out, None)


def test_clip_refusals():
    assert clip(max_norm=-1.0) == INVALID and clip(max_norm=math.nan) == INVALID
    assert clip(sumsq=None) == INVALID and clip(sumsq=FAR + 4) == INVALID and clip(out=FAR + 1) == INVALID
    assert clip(outs=ptrs(A, None)) == INVALID and clip(outs=ptrs(A, 2 * A + 1)) == INVALID
    assert clip(outs=ptrs(3 * A, 3 * A + 128)) == INVALID  # outputs over each other
    assert clip(outs=ptrs(A + 128, 3 * A)) == INVALID      # over its own gradient, shifted
    assert clip(outs=ptrs(2 * A, 3 * A)) == INVALID        # over another gradient
    assert clip(grads=ptrs(A, A), outs=ptrs(A, 3 * A)) == INVALID  # in place, but another tensor reads it too
    assert clip(sumsq=A + 64) == INVALID and clip(out=2 * A + 128) == INVALID  # scalars inside an output
    args = [2, ptrs(A, 2 * A), ptrs(A, 2 * A), i64s(64, 64), 1, 1.0, None, FAR, 10 * A, 1 << 20, None]
    f = lib().tide_clip_grad_norm
    for at, bad in ((0, -1), (4, 7), (5, -2.0), (5, math.nan), (6, 12), (7, 2), (8, None), (8, 8), (9, 4), (8, A)):
        assert f(*[bad if i == at else v for i, v in enumerate(args)]) == INVALID, (at, bad)


LN = dict(rows=4, cols=100, x=A, xs=100, dtype=1, w=2 * A, b=3 * A, pdtype=0, eps=1e-5, y=4 * A, ys=100, mean=5 * A,
          rstd=6 * A)


def ln(**kw):
    return lib().tide_layer_norm(*{**LN, **kw}.values(), None)


def test_layer_norm_refusals():
    for kw in (dict(rows=-1), dict(cols=0), dict(cols=-3), dict(cols=1 << 31), dict(rows=1 << 60), dict(x=None),
               dict(x=A + 2), dict(xs=99), dict(xs=-100), dict(xs=1 << 62), dict(y=None), dict(y=4 * A + 1),
               dict(ys=1), dict(dtype=2), dict(dtype=9), dict(pdtype=3), dict(w=2 * A + 1), dict(b=3 * A + 1),
               dict(pdtype=1, w=2 * A + 2), dict(mean=5 * A + 2), dict(rstd=6 * A + 1), dict(eps=-1.0),
               dict(eps=math.nan), dict(eps=math.inf), dict(y=A), dict(y=A + 800), dict(y=2 * A), dict(y=3 * A - 100),
               dict(mean=A), dict(mean=6 * A), dict(rstd=4 * A + 400)):
        assert ln(**kw) == INVALID, kw
    assert ln(rows=0, x=None, y=None, mean=None, rstd=None) == OK  # nothing to do


LNB = dict(rows=4, cols=100, dy=A, dys=100, x=2 * A, xs=100, dtype=0, w=3 * A, pdtype=1, mean=4 * A, rstd=5 * A,
           dx=6 * A, dxs=100, dw=7 * A, db=8 * A, ws=9 * A, size=1 << 19)


def ln_bwd(**kw):
    return lib().tide_layer_norm_bwd(*{**LNB, **kw}.values(), None)


def test_layer_norm_bwd_refusals():
    f = lib().tide_layer_norm_bwd_workspace
    assert f(-1, 4, 0) == -1 and f(4, 0, 0) == -1 and f(4, 4, 2) == -1 and f(0, 4, 0) == 0
    assert f(4, 100, 0) >= 4 * 2 * 100
    for kw in (dict(rows=-1), dict(cols=0), dict(dy=None), dict(x=None), dict(mean=None), dict(rstd=None),
               dict(dy=A + 1), dict(dys=99), dict(xs=7), dict(dxs=99), dict(dtype=4), dict(pdtype=2), dict(w=3 * A + 2),
               dict(dw=7 * A + 2), dict(db=8 * A + 1), dict(ws=None), dict(ws=9 * A + 4), dict(size=16),
               dict(dx=A, dxs=101), dict(dx=A + 2), dict(dx=2 * A), dict(dw=3 * A), dict(dw=8 * A), dict(db=6 * A),
               dict(ws=2 * A), dict(ws=7 * A), dict(dw=4 * A)):
        assert ln_bwd(**kw) == INVALID, kw
    assert ln_bwd(rows=0, dw=None, db=None, ws=None, size=0) == OK


EMB = dict(tokens=10, ids=A, idt=3, vocab=50, dim=16, table=2 * A, dtype=0, scale=1.0, out=3 * A)


def emb(**kw):
    return lib().tide_embedding(*{**EMB, **kw}.values(), None)


def test_embedding_refusals():
    for kw in (dict(tokens=-1), dict(tokens=1 << 31), dict(ids=None), dict(ids=A + 4), dict(idt=0), dict(idt=1),
               dict(vocab=-1), dict(vocab=1 << 31), dict(dim=0), dict(dim=1 << 31), dict(table=None),
               dict(table=2 * A + 1), dict(dtype=2), dict(out=None), dict(out=3 * A + 1), dict(out=2 * A + 32),
               dict(out=A), dict(tokens=(1 << 31) - 1, dim=(1 << 31) - 1)):
        assert emb(**kw) == INVALID, kw
    assert emb(tokens=0, ids=None, out=None) == OK


EMBB = dict(tokens=10, ids=A, idt=3, vocab=50, dim=16, dy=2 * A, dtype=0, scale=1.0, acc=0, dtable=3 * A, ws=4 * A,
            size=1 << 19)


def emb_bwd(**kw):
    return lib().tide_embedding_bwd(*{**EMBB, **kw}.values(), None)


def test_embedding_bwd_refusals():
    f = lib().tide_embedding_bwd_workspace
    assert f(-1, 5, 5) == -1 and f(5, -1, 5) == -1 and f(5, 5, 0) == -1 and f(1 << 31, 5, 5) == -1
    assert f(10, 50, 16) >= 10 * 8
    for kw in (dict(tokens=-1), dict(ids=None), dict(idt=1), dict(vocab=-1), dict(dim=0), dict(dy=None),
               dict(dy=2 * A + 1), dict(dtype=3), dict(acc=2), dict(acc=-1), dict(dtable=None), dict(dtable=3 * A + 1),
               dict(ws=None), dict(ws=4 * A + 8), dict(size=100), dict(dtable=2 * A), dict(dtable=A), dict(ws=3 * A),
               dict(ws=2 * A)):
        assert emb_bwd(**kw) == INVALID, kw
    assert emb_bwd(vocab=0, dtable=None) == OK
    assert emb_bwd(tokens=0, ids=None, dy=None, acc=1) == OK


def test_the_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("checked without a GPU")
    x = torch.zeros(4, 8)
    with pytest.raises((ValueError, RuntimeError)):
        tide.layer_norm(x)
    with pytest.raises((ValueError, RuntimeError)):
        tide.embedding(torch.zeros(3, dtype=torch.int64), x)
    with pytest.raises((ValueError, RuntimeError)):
        tide.grad_norm([x])


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_host_code_under_sanitizers(tmp_path):
    exe = str(tmp_path / "host_step_check")
    csrc = os.path.join(ROOT, "all_gather_placement_amd", "csrc")
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
           "-fno-sanitize-recover=undefined", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
           "-I", os.path.join(ROOT, "include"), os.path.join(ROOT, "tests", "native", "host_step_check.cpp"),
           os.path.join(csrc, "step_api.cpp"), "-L/opt/rocm/lib", "-Wl,-rpath,/opt/rocm/lib", "-lamdhip64", "-o", exe]
    subprocess.run(cmd, check=True, capture_output=True, timeout=300)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=1", UBSAN_OPTIONS="print_stacktrace=1")
    res = subprocess.run([exe], capture_output=True, text=True, timeout=300, env=env)
    assert res.returncode == 0, res.stdout + res.stderr
    assert "0 failures" in res.stdout
