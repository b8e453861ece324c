"""Host-side checks of the block operators of libtide_step.so (no GPU): sizes, and the refusal of bad
arguments before any work is enqueued (made-up addresses are never touched)."""
import ctypes
import math
import os
import shutil
import subprocess

import pytest

import all_gather_placement_amd as tide

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID = 0, 1
A = 1 << 24  # made-up, aligned device addresses, far apart
INT32, INT64 = 2, 3


def lib():
    return tide.load_step_library()


def test_functions_are_there():
    for n in ("expert_sort", "expert_dispatch", "expert_dispatch_bwd", "expert_combine", "expert_combine_bwd", "rotary",
              "rotary_bwd", "rotary_freqs", "dropout", "dropout_bwd"):
        assert callable(getattr(tide, n))


def test_expert_rows():
    f = lib().tide_expert_rows
    assert f(0, 8, 128, 128) == 0 and f(1, 1, 1, 1) == 1 and f(10, 8, 128, 1) == 80
    assert f(10, 8, 3, 16) == 80 + 3 * 15 and f(1, 2, 128, 16) == 2 + 2 * 15
    assert f(-1, 8, 8, 1) == -1 and f(1, 0, 8, 1) == -1 and f(1, 65, 8, 1) == -1 and f(1, 1, 0, 1) == -1
    assert f(1, 1, 2049, 1) == -1 and f(1, 1, 1, 0) == -1 and f(1 << 31, 1, 1, 1) == -1 and f(1 << 30, 2, 1, 1) == -1
    assert f((1 << 31) - 1, 1, 1, 1) == (1 << 31) - 1 and f(1 << 30, 1, 2048, 1 << 20) == -1
    w = lib().tide_expert_sort_workspace
    assert w(0, 1, 1) == 0 and w(1 << 20, 8, 128) >= 0 and w(1 << 20, 65, 128) == -1 and w(4, 2, 4000) == -1


SORT = dict(tokens=100, choices=8, ids=A, idt=INT64, experts=128, align=16, place=2 * A, source=3 * A, rows=4000,
            offsets=4 * A, ws=5 * A, size=1 << 20)


def sort(**kw):
    return lib().tide_expert_sort(*{**SORT, **kw}.values(), None)


def test_sort_refusals():
    for kw in (dict(tokens=-1), dict(tokens=1 << 31), dict(choices=0), dict(choices=65), dict(ids=None), dict(ids=A + 4),
               dict(idt=0), dict(idt=1), dict(idt=7), dict(experts=0), dict(experts=2049), dict(align=0),
               dict(align=(1 << 31) - 1), dict(place=None), dict(place=2 * A + 2), dict(source=None),
               dict(source=3 * A + 1), dict(rows=100 * 8 + 128 * 15 - 1), dict(rows=1 << 31), dict(rows=-1),
               dict(offsets=None), dict(offsets=4 * A + 2), dict(place=A), dict(source=2 * A + 64),
               dict(offsets=3 * A + 400), dict(offsets=A - 8), dict(source=A + 6396)):
        assert sort(**kw) == INVALID, kw
    big = dict(tokens=100000, rows=1 << 20, size=lib().tide_expert_sort_workspace(100000, 8, 128))
    assert big["size"] > 0
    for kw in (dict(ws=None), dict(ws=5 * A + 8), dict(size=big["size"] - 1), dict(ws=A), dict(ws=2 * A), dict(ws=3 * A),
               dict(ws=4 * A)):
        assert sort(**{**big, **kw}) == INVALID, kw


DISPATCH = dict(tokens=10, choices=4, dim=100, x=A, xs=100, dtype=0, place=2 * A, source=3 * A, rows=40, out=4 * A, os=100)


def dispatch(**kw):
    return lib().tide_expert_dispatch(*{**DISPATCH, **kw}.values(), None)


def test_dispatch_refusals():
    for kw in (dict(tokens=-1), dict(choices=0), dict(choices=65), dict(dim=0), dict(dim=1 << 31), dict(x=None),
               dict(x=A + 1), dict(xs=99), dict(xs=-100), dict(xs=1 << 62), dict(dtype=2), dict(dtype=-1),
               dict(place=None), dict(place=2 * A + 2), dict(source=None), dict(source=3 * A + 2), dict(rows=-1),
               dict(rows=1 << 31), dict(out=None), dict(out=4 * A + 1), dict(os=99), dict(out=A), dict(out=A + 1000),
               dict(out=2 * A - 100), dict(out=3 * A + 64), dict(dtype=1, out=A - 400)):
        assert dispatch(**kw) == INVALID, kw
    assert dispatch(rows=0, source=None, out=None) == OK


COMBINE = dict(tokens=10, choices=4, dim=100, x=A, xs=100, rows=40, dtype=1, w=2 * A, wdt=1, place=3 * A, y=4 * A, ys=100)


def combine(**kw):
    return lib().tide_expert_combine(*{**COMBINE, **kw}.values(), None)


def test_combine_refusals():
    for kw in (dict(tokens=-1), dict(choices=0), dict(choices=65), dict(dim=0), dict(x=None), dict(x=A + 2), dict(xs=99),
               dict(rows=-1), dict(rows=1 << 31), dict(dtype=3), dict(wdt=2), dict(w=2 * A + 2), dict(wdt=0, w=2 * A + 1),
               dict(place=None), dict(place=3 * A + 1), dict(y=None), dict(y=4 * A + 2), dict(ys=7), dict(y=A),
               dict(y=A + 15996), dict(y=2 * A), dict(y=3 * A)):
        assert combine(**kw) == INVALID, kw
    assert combine(tokens=0, place=None, y=None, w=None) == OK


COMBINE_BWD = dict(tokens=10, choices=4, dim=100, dy=A, dys=100, x=2 * A, xs=100, rows=40, dtype=0, w=3 * A, wdt=0,
                   place=4 * A, source=5 * A, dx=6 * A, dxs=100, dw=7 * A)


def combine_bwd(**kw):
    return lib().tide_expert_combine_bwd(*{**COMBINE_BWD, **kw}.values(), None)


def test_combine_bwd_refusals():
    for kw in (dict(tokens=-1), dict(choices=65), dict(dim=0), dict(dy=None), dict(dy=A + 1), dict(dys=99), dict(x=None),
               dict(xs=99), dict(rows=-1), dict(dtype=2), dict(w=None), dict(w=3 * A + 1), dict(wdt=3), dict(place=None),
               dict(source=None), dict(source=5 * A + 2), dict(dx=None), dict(dx=6 * A + 1), dict(dxs=98), dict(dw=None),
               dict(dw=7 * A + 1), dict(wdt=1, dw=7 * A + 2), dict(dx=A), dict(dx=2 * A, dxs=101), dict(dx=2 * A + 2),
               dict(dx=3 * A), dict(dx=4 * A), dict(dx=5 * A), dict(dx=7 * A), dict(dw=A), dict(dw=2 * A), dict(dw=3 * A),
               dict(dw=4 * A), dict(dw=5 * A)):
        assert combine_bwd(**kw) == INVALID, kw
    assert combine_bwd(tokens=0, rows=0, dy=None, x=None, w=None, place=None, source=None, dx=None, dw=None) == OK


def i32s(*v):
    return (ctypes.c_int32 * max(len(v), 1))(*v)


ROTARY = dict(tokens=6, heads=5, dim=64, x=A, xt=320, xh=64, dtype=0, pos=2 * A, pdt=INT32, axes=3, sections=i32s(8, 4, 20),
              freqs=3 * A, pairing=0, inverse=0, out=4 * A, ot=320, oh=64)


def rotary(**kw):
    return lib().tide_rotary(*{**ROTARY, **kw}.values(), None)


def test_rotary_refusals():
    for kw in (dict(tokens=-1), dict(tokens=1 << 31), dict(heads=-1), dict(heads=1 << 31), dict(heads=65536, tokens=0), dict(dim=0), dict(dim=1025),
               dict(x=None), dict(x=A + 1), dict(xt=-1), dict(xh=-64), dict(xt=1 << 62), dict(dtype=2), dict(pos=None),
               dict(pos=2 * A + 2), dict(pdt=INT64, pos=2 * A + 4), dict(pdt=0), dict(pdt=5), dict(axes=0), dict(axes=9),
               dict(axes=-1), dict(sections=None), dict(sections=i32s(8, 0, 20)), dict(sections=i32s(8, -4, 20)),
               dict(sections=i32s(8, 4, 21)), dict(sections=i32s((1 << 31) - 1, (1 << 31) - 1, 8)), dict(dim=63),
               dict(freqs=None), dict(freqs=3 * A + 4), dict(pairing=2), dict(pairing=-1), dict(inverse=2), dict(out=None),
               dict(out=4 * A + 1), dict(ot=319), dict(oh=63), dict(oh=0), dict(ot=0), dict(ot=64, oh=128),
               dict(out=A + 2), dict(out=A + 640), dict(out=A, ot=640), dict(out=A, xt=64, xh=384), dict(out=2 * A),
               dict(out=3 * A), dict(out=2 * A - 3838)):
        assert rotary(**kw) == INVALID, kw
    assert rotary(tokens=0, x=None, pos=None, out=None) == OK
    assert rotary(heads=0, x=None, pos=None, out=None) == OK


DROPOUT = dict(rows=6, cols=100, x=A, xs=100, dtype=0, p=0.5, seed=7, dev=None, offset=0, residual=2 * A, rs=100,
               out=3 * A, os=100)


def dropout(**kw):
    return lib().tide_dropout(*{**DROPOUT, **kw}.values(), None)


def test_dropout_refusals():
    for kw in (dict(rows=-1), dict(cols=0), dict(cols=(1 << 44) + 1), dict(rows=1 << 40, cols=1 << 10), dict(x=None),
               dict(x=A + 1), dict(xs=99), dict(dtype=2), dict(p=-0.1), dict(p=1.0001), dict(p=math.nan), dict(p=math.inf),
               dict(dev=8 * A + 4), dict(offset=-1), dict(offset=(1 << 62) - 599), dict(residual=2 * A + 1), dict(rs=99),
               dict(out=None), dict(out=3 * A + 1), dict(os=99), dict(out=A, os=101), dict(out=A + 2), dict(out=2 * A, os=101),
               dict(out=2 * A + 2), dict(dev=3 * A)):
        assert dropout(**kw) == INVALID, kw
    assert dropout(rows=0, x=None, residual=None, out=None) == OK


def test_the_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("checked without a GPU")
    x = torch.zeros(4, 2, 8)
    ids = torch.zeros(4, 2, dtype=torch.int64)
    for call in (lambda: tide.expert_sort(ids, 3), lambda: tide.expert_dispatch(x[:, 0], (ids, ids, ids)),
                 lambda: tide.expert_combine(x[:, 0], None, (ids, ids, ids)), lambda: tide.dropout(x, 0.1, 1),
                 lambda: tide.expert_combine_bwd(x[:, 0], x[:, 0], x[:, 0], (ids, ids, ids)),
                 lambda: tide.rotary(x, ids.T, torch.zeros(4).double(), (2, 2))):
        with pytest.raises((ValueError, RuntimeError)):
            call()


def build(tmp_path, name, sources, flags):
    exe = str(tmp_path / name)
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I",
           os.path.join(ROOT, "include"), os.path.join(ROOT, "tests", "native", name + ".cpp"), *sources, *flags,
           "-L/opt/rocm/lib", "-Wl,-rpath,/opt/rocm/lib", "-lamdhip64", "-o", exe]
    subprocess.run(cmd, check=True, capture_output=True, timeout=300)
    return exe


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_host_code_under_sanitizers(tmp_path):
    csrc = os.path.join(ROOT, "all_gather_placement_amd", "csrc")
    exe = build(tmp_path, "host_block_check", [os.path.join(csrc, "step_block_api.cpp")],
                ["-fno-omit-frame-pointer", "-fsanitize=address,undefined", "-fno-sanitize-recover=undefined"])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=1", UBSAN_OPTIONS="print_stacktrace=1")
    res = subprocess.run([exe], capture_output=True, text=True, timeout=300, env=env)
    assert res.returncode == 0 and "0 failures" in res.stdout, res.stdout + res.stderr
