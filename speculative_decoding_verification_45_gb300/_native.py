"""Build and load the sm_103a shared library (libspec_verify.so) in-tree."""
from __future__ import annotations

import ctypes
import importlib.util
import os
import shutil
import subprocess
import sysconfig
import threading
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
INCLUDE = os.path.join(ROOT, "include")
CSRC = os.path.join(PKG, "csrc")
CACHE = os.path.join(CSRC, "cache")
ROWS = os.path.join(CSRC, "rows")
# The host unit, one unit per (dtype, proposal form) of kernels, the cache's four and the rows' two: compiled in parallel.
SOURCES = ([os.path.join(CSRC, f) for f in ("spec_verify.cu", "kernels_bf16.cu", "kernels_bf16_point.cu",
                                             "kernels_f32.cu", "kernels_f32_point.cu")]
           + [os.path.join(CACHE, f) for f in ("spec_cache_move.cu", "spec_cache_attend.cu",
                                               "spec_cache_attend_d64.cu", "spec_cache_attend_d128.cu")]
           + [os.path.join(ROWS, f) for f in ("spec_rows_code.cu", "spec_rows_product.cu")])
HEADERS = [os.path.join(INCLUDE, "spec_verify.h"), os.path.join(CSRC, "spec_verify_kernels.cuh"),
           os.path.join(CACHE, "spec_ptx.cuh"), os.path.join(CACHE, "spec_cache.cuh"),
           os.path.join(CACHE, "spec_cache_attend.cuh"), os.path.join(ROWS, "spec_rows.cuh")]
# The binding's common calls of 8-bit rows, in C: an extension module of this interpreter.
PY_SOURCE = os.path.join(ROWS, "spec_rows_py.c")
BUILD_DIR = os.path.join(PKG, "_build")
LIB_PATH = os.path.join(BUILD_DIR, "libspec_verify.so")
PY_PATH = os.path.join(BUILD_DIR, "spec_rows_py" + sysconfig.get_config_var("EXT_SUFFIX"))
ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]

_lock = threading.Lock()
_lib = None


class Options(ctypes.Structure):
    """spec_verify_options of include/spec_verify.h."""

    _fields_ = [("cluster_size", ctypes.c_int), ("kernel", ctypes.c_int), ("counters", ctypes.c_void_p),
                ("accept_hist", ctypes.c_void_p)]


class Cache(ctypes.Structure):
    """spec_cache of include/spec_verify.h."""

    _fields_ = ([(f, ctypes.c_void_p) for f in ("k", "v", "k_scale", "v_scale", "positions", "block_table")]
                + [("k_stride", ctypes.c_int64 * 3), ("v_stride", ctypes.c_int64 * 3), ("table_stride", ctypes.c_int64)]
                + [(f, ctypes.c_int32) for f in ("batch", "max_blocks", "num_pages", "kv_heads", "block", "dim", "code")])


class CacheForm(ctypes.Structure):
    """spec_cache_form of include/spec_verify.h."""

    _fields_ = [("scale", ctypes.c_float), ("softcap", ctypes.c_float), ("window", ctypes.c_int32),
                ("slopes", ctypes.c_void_p), ("prefix", ctypes.c_void_p), ("parent", ctypes.c_void_p),
                ("num_new", ctypes.c_void_p)]


class Coded(ctypes.Structure):
    """spec_coded of include/spec_verify.h."""

    _fields_ = [("codes", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("stride", ctypes.c_int64),
                ("scale_stride", ctypes.c_int64), ("rows", ctypes.c_int32), ("dim", ctypes.c_int32),
                ("code", ctypes.c_int32)]


def fit(name: str, *sizes: int) -> None:
    """Sizes are handed to the library in 32 bits, into which ctypes cuts larger ones without a word."""
    for n in sizes:
        if not -(1 << 31) <= n < 1 << 31:
            raise ValueError(f"{name}: sizes must be below 2^31, got {n}")


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is needed to build libspec_verify.so")


def _stale() -> bool:
    if not os.path.exists(LIB_PATH) or not os.path.exists(PY_PATH):
        return True
    t = min(os.path.getmtime(LIB_PATH), os.path.getmtime(PY_PATH))
    return any(os.path.getmtime(f) > t for f in SOURCES + HEADERS + [PY_SOURCE])


def _run(cmd):
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"{os.path.basename(cmd[0])} failed ({res.returncode}):\n{' '.join(cmd)}\n{res.stdout}\n{res.stderr}")
    return res.stdout + res.stderr


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile the units of csrc for sm_103a (one nvcc per unit, in parallel), link
    _build/libspec_verify.so, and compile the binding's extension module beside it."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    if not force and not _stale():
        return LIB_PATH
    nvcc, tag = nvcc_path(), f"tmp{os.getpid()}"
    objs = [os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + f".{tag}.o") for src in SOURCES]
    cmds = [[nvcc, "-O3", "-std=c++17", *ARCH_FLAGS, "-lineinfo", "-Xcompiler", "-fPIC", "-I", INCLUDE,
             *(["-Xptxas=-v"] if verbose else []), "-c", "-o", obj, src] for src, obj in zip(SOURCES, objs)]
    tmp, py_tmp = LIB_PATH + f".{tag}", PY_PATH + f".{tag}"
    cmds.append([shutil.which("gcc") or "cc", "-O2", "-Wall", "-shared", "-fPIC", "-I", INCLUDE, "-I", sysconfig.get_paths()["include"],
                 "-o", py_tmp, PY_SOURCE])
    try:
        with ThreadPoolExecutor(max_workers=len(cmds)) as pool:
            logs = list(pool.map(_run, cmds))
        logs.append(_run([nvcc, *ARCH_FLAGS, "-shared", "-o", tmp, *objs, "-ldl"]))
    finally:
        for obj in objs:
            if os.path.exists(obj):
                os.remove(obj)
    if verbose:
        print("".join(logs))
    os.replace(tmp, LIB_PATH)
    os.replace(py_tmp, PY_PATH)
    return LIB_PATH


def load_extension():
    """The binding's extension module; raises if it has not been built."""
    if not os.path.exists(PY_PATH):
        raise RuntimeError(f"{PY_PATH} is missing: run __graft_entry__.build() (or "
                           "speculative_decoding_verification_45_gb300._native.build()) first")
    spec = importlib.util.spec_from_file_location("spec_rows_py", PY_PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def load() -> ctypes.CDLL:
    """Load the built library; raises if it has not been built (no fallback exists)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: run __graft_entry__.build() (or "
                               "speculative_decoding_verification_45_gb300._native.build()) first")
        lib = ctypes.CDLL(LIB_PATH)
        vp, i32 = ctypes.c_void_p, ctypes.c_int
        common = [vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, vp, vp]
        lib.spec_verify.argtypes = common
        lib.spec_verify.restype = i32
        lib.spec_verify_debug.argtypes = common + [vp] * 7
        lib.spec_verify_debug.restype = i32
        lib.spec_verify_ex.argtypes = common + [vp]
        lib.spec_verify_ex.restype = i32
        lib.spec_ngram_propose.argtypes = [vp, ctypes.c_int64, vp, i32, i32, i32, i32, vp, vp, vp]
        lib.spec_ngram_propose.restype = i32
        lib.spec_sample.argtypes = [vp, vp, vp, vp, i32, i32, i32, vp, vp, vp]
        lib.spec_sample.restype = i32
        lib.spec_tree_verify.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, vp, vp, vp]
        lib.spec_tree_verify.restype = i32
        lib.spec_verify_launch_shape.argtypes = [i32, i32, i32, i32, vp, vp, vp, vp]
        lib.spec_verify_launch_shape.restype = i32
        lib.spec_device_pointer.argtypes = [vp, ctypes.POINTER(ctypes.c_void_p)]
        lib.spec_device_pointer.restype = i32
        lib.spec_cache_append.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, vp, vp, vp, vp]
        lib.spec_cache_append.restype = i32
        lib.spec_cache_attend.argtypes = [vp, vp, vp, vp, i32, i32, vp, vp, vp, vp, ctypes.c_int64, vp, vp]
        lib.spec_cache_attend.restype = i32
        lib.spec_cache_attend_workspace.argtypes = [vp, i32, i32, vp]
        lib.spec_cache_attend_workspace.restype = i32
        lib.spec_cache_set_wait_limit.argtypes = [i32]
        lib.spec_cache_set_wait_limit.restype = i32
        lib.spec_cache_weigh.argtypes = [vp, vp, vp, vp, i32, i32, vp, vp, vp, vp, ctypes.c_int64, vp, vp]
        lib.spec_cache_weigh.restype = i32
        lib.spec_cache_evict.argtypes = [vp, vp, vp, i32, i32, vp, ctypes.c_int64, vp, vp, vp, vp]
        lib.spec_cache_evict.restype = i32
        i64, f32 = ctypes.c_int64, ctypes.c_float
        lib.spec_rows_quantise.argtypes = [vp, i64, i32, vp, i32, vp]
        lib.spec_rows_quantise.restype = i32
        lib.spec_rows_norm.argtypes = [vp, i64, i32, vp, i64, i32, vp, i32, f32, vp, i64, vp, vp]
        lib.spec_rows_norm.restype = i32
        lib.spec_rows_gate.argtypes = [vp, i64, vp, i64, i32, i32, vp, vp]
        lib.spec_rows_gate.restype = i32
        lib.spec_rows_product.argtypes = [vp, vp, vp, i64, i32, vp, vp]
        lib.spec_rows_product.restype = i32
        lib.spec_status_string.argtypes = [i32]
        lib.spec_status_string.restype = ctypes.c_char_p
        _lib = lib
        return lib
