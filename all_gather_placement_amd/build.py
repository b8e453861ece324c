"""Build libtide.so (C ABI + gfx950 kernels), libtide_step.so with its Python module _step.so, and
libtide_probe.so in-tree with hipcc.

    python -m all_gather_placement_amd.build

The libraries are compiled for gfx950 only.  Packed-fp32 instructions are disabled for device code
(the kernels' fp32 adds must stay plain IEEE adds in a fixed order), and no fast-math flag is
used, so fp32 denormals and rounding are IEEE.

Each library embeds a build id: the first 16 hex digits of the SHA-256 of its sources, the headers
they include and the compile flags (``tide_build_id()`` / ``tide_step_build_id()`` /
``tide_probe_build_id()``); the Python module's also covers the torch and the interpreter it is made for.
:func:`ensure_built` rebuilds a library whose embedded id differs from the sources in the tree, and
the bindings refuse to load one, so a library built from other sources is never run.
"""
from __future__ import annotations

import ctypes
import hashlib
import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libtide.so")
SOURCES = ["layout.cpp", "api.cpp", "kernels.hip"]
PROBE_LIB = os.path.join(PKG, "libtide_probe.so")
PROBE_SOURCES = ["probe.hip"]
STEP_LIB = os.path.join(PKG, "libtide_step.so")
STEP_SOURCES = ["step_api.cpp", "step_norm.hip", "step_layer_norm.hip", "step_embedding.hip"]
STEP_BINDING = os.path.join(PKG, "_step.so")
STEP_BINDING_SOURCES = ["step_binding.cpp"]
ARCH = "gfx950"

# Everything each library is compiled from (its sources and every header they include).
HASHED = {
    LIB: [os.path.join(CSRC, f) for f in ("layout.cpp", "api.cpp", "kernels.hip", "layout.h", "tide_internal.h")]
         + [os.path.join(INCLUDE, "tide.h")],
    PROBE_LIB: [os.path.join(CSRC, f) for f in ("probe.hip", "tide_internal.h")]
               + [os.path.join(INCLUDE, "tide_probe.h")],
    STEP_LIB: [os.path.join(CSRC, f) for f in (*STEP_SOURCES, "step_internal.h", "step_device.h")]
              + [os.path.join(INCLUDE, f) for f in ("tide_step.h", "tide.h")],
    STEP_BINDING: [os.path.join(CSRC, f) for f in STEP_BINDING_SOURCES]
                  + [os.path.join(INCLUDE, f) for f in ("tide_step.h", "tide.h")],
}
ID_SYMBOL = {LIB: "tide_build_id", PROBE_LIB: "tide_probe_build_id", STEP_LIB: "tide_step_build_id"}


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found (looked in $HIPCC, /opt/rocm/bin, PATH)")


def compile_flags(extra=()) -> list:
    return [
        f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-Wall",
        "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
        "-I", INCLUDE, *extra,
    ]


def source_hash(lib: str = LIB, extra=()) -> str:
    """Build id of `lib` for the sources now in the tree (16 hex digits)."""
    h = hashlib.sha256()
    for path in HASHED[lib]:
        h.update(os.path.basename(path).encode() + b"\0")
        with open(path, "rb") as fh:
            h.update(fh.read())
        h.update(b"\0")
    h.update(" ".join(compile_flags(extra)).replace(INCLUDE, "<include>").encode())
    if lib == STEP_BINDING:
        h.update(b"\0" + module_target())
    return h.hexdigest()[:16]


def module_target() -> bytes:
    """What the Python module is compiled against: the interpreter's ABI, torch's version (and revision
    and HIP version, from the file that states them, so that torch is not loaded) and the flags that name
    no place."""
    spec = importlib.util.find_spec("torch") if has_torch() else None
    version = b""
    if spec is not None:
        with open(os.path.join(spec.submodule_search_locations[0], "version.py"), "rb") as fh:
            version = fh.read()
    return b"\0".join((str(sysconfig.get_config_var("SOABI")).encode(), version, " ".join(MODULE_FLAGS).encode()))


MODULE_FLAGS = ["-fvisibility=hidden"]
BINDING_MARK = rb"tide_step_binding build id ([0-9a-f]{16})\0"


def torch_flags() -> list:
    """Compile flags of the Python module: torch's headers and the interpreter's."""
    from torch.utils.cpp_extension import include_paths

    dirs = [*include_paths(), sysconfig.get_paths()["include"]]
    return [*MODULE_FLAGS, *(f for d in dirs for f in ("-isystem", d))]


def torch_link_flags() -> list:
    import torch

    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    return ["-L" + PKG, "-l:" + os.path.basename(STEP_LIB), "-Wl,-rpath,$ORIGIN", "-L" + lib, "-Wl,-rpath," + lib, "-ltorch_python", "-ltorch_cpu", "-lc10"]


def built_id(lib: str = LIB):
    """Build id embedded in the library file at `lib`, or None if it is missing or carries none.
    Loads the library (no HIP call is made by loading or by the id query); the Python module's, which
    would load torch, is found in the file."""
    if not os.path.exists(lib):
        return None
    if lib == STEP_BINDING:
        with open(lib, "rb") as fh:
            found = re.search(BINDING_MARK, fh.read())
        return found.group(1).decode() if found else None
    try:
        fn = getattr(ctypes.CDLL(lib), ID_SYMBOL[lib])
    except (OSError, AttributeError):
        return None
    fn.restype = ctypes.c_char_p
    fn.argtypes = []
    return fn().decode()


def check_current(lib: str = LIB, loaded=None) -> None:
    """Raise if the library (the file, or the already loaded CDLL `loaded`) was not built from the
    sources now in the tree."""
    want = source_hash(lib)
    if loaded is not None:
        fn = getattr(loaded, ID_SYMBOL[lib], None)
        got = None
        if fn is not None:
            fn.restype = ctypes.c_char_p
            fn.argtypes = []
            got = fn().decode()
    else:
        got = built_id(lib)
    if got != want:
        raise RuntimeError(f"{lib} was built from other sources (build id {got}, sources {want}); "
                           f"rebuild it: python -m all_gather_placement_amd.build")


def has_torch() -> bool:
    """Whether the Python module can be built; the libraries' C ABI needs no torch."""
    try:
        return importlib.util.find_spec("torch") is not None
    except (ImportError, ValueError):
        return False


def build(verbose: bool = False, extra=(), out: str = LIB, sources=SOURCES, probe: bool = True) -> str:
    """Compile every source and link the shared library, then the probe and step libraries and, where torch
    is installed, the step operators' Python module; returns the first one's path."""
    compile_library(out, sources, verbose, extra)
    if probe and out == LIB:
        compile_library(PROBE_LIB, PROBE_SOURCES, verbose, extra)
        compile_library(STEP_LIB, STEP_SOURCES, verbose, extra)
        if has_torch():
            compile_library(STEP_BINDING, STEP_BINDING_SOURCES, verbose, extra)
        else:
            print(f"torch is not installed: {os.path.basename(STEP_BINDING)} is not built", flush=True)
    return out


def compile_library(out: str, sources, verbose: bool = False, extra=()) -> None:
    """Compile `sources` and link them to `out`."""
    objdir = os.path.join(PKG, "_build", os.path.splitext(os.path.basename(out))[0])
    os.makedirs(objdir, exist_ok=True)
    cc = hipcc()
    key = out if out in HASHED else LIB
    bid = source_hash(key, extra)
    id_flag = [f"-DTIDE_BUILD_ID=\"{bid}\""]
    objs = []
    running = []
    for src in sources:
        obj = os.path.join(objdir, os.path.splitext(src)[0] + ".o")
        lang = ["-x", "hip"] if src.endswith(".hip") else []
        more = torch_flags() if out == STEP_BINDING else []
        cmd = [cc, *compile_flags(extra), *id_flag, *lang, *more, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        running.append(subprocess.Popen(cmd))
        objs.append(obj)
    for p in running:  # all of them end before an error is raised
        p.wait()
    for p in running:
        if p.returncode != 0:
            raise subprocess.CalledProcessError(p.returncode, p.args)
    tmp = out + ".tmp"
    link = [cc, f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", tmp,
            "-Wl,-rpath,/opt/rocm/lib", "-L/opt/rocm/lib", "-lamdhip64"]
    if out == PROBE_LIB:
        link.append("-lhsa-runtime64")  # the DMA engines' rectangular copy (tide_probe_dma_rect_copies)
    if out == STEP_BINDING:
        link += torch_link_flags()
    if verbose:
        print(" ".join(link), flush=True)
    subprocess.run(link, check=True)
    os.replace(tmp, out)


def is_current(lib: str) -> bool:
    """True when `lib` exists and carries the build id of the sources now in the tree.  The id is
    read in a child process, so a stale file is never mapped into this one (it may be rebuilt)."""
    if not os.path.exists(lib):
        return False
    code = ("import sys; sys.path.insert(0, %r); from all_gather_placement_amd.build import built_id; "
            "print(built_id(%r) or '')" % (ROOT, lib))
    res = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True)
    return res.returncode == 0 and res.stdout.strip() == source_hash(lib)


def ensure_built(verbose: bool = False) -> str:
    """Build the libraries if they are missing or were built from other sources (tests, smoke and
    benchmark entry points); returns the path of libtide.so."""
    if not all(map(is_current, (LIB, PROBE_LIB, STEP_LIB, *((STEP_BINDING,) if has_torch() else ())))):
        build(verbose=verbose)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
