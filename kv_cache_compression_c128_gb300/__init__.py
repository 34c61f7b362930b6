"""GB300-native KV-cache window compressor (``c128_256_512_compress``).

The computation runs in the CUDA library ``_lib/libkvc.so`` (sources in
``csrc/``, C ABI in ``include/kvc.h``); this module only marshals arguments
through ctypes.  There is no CPU fallback: if the library is missing or no
CUDA device is present, the calls raise.

The operator is the one of "From Attention to KV Cache Compression: Notes
from a KernelGen Optimization" (KernelGen Challenge 8 write-up), section
"The Compression Operator", with the layout of "Gather and Scatter".
"""
from __future__ import annotations

import contextlib
import ctypes
import hashlib
import importlib.machinery
import importlib.util
import os
import shutil
import subprocess
import sysconfig
import threading
import warnings
from concurrent.futures import ThreadPoolExecutor
from typing import Optional

_HERE = os.path.dirname(os.path.abspath(__file__))
_ROOT = os.path.dirname(_HERE)
_CSRC = os.path.join(_HERE, "csrc")
_INCLUDE = os.path.join(_ROOT, "include")
_LIB_DIR = os.path.join(_HERE, "_lib")
LIB_PATH = os.path.join(_LIB_DIR, "libkvc.so")
_SOURCES = ["kvc_cluster.cu", "kvc_streamk.cu", "kvc_reader.cu", "kvc_api.cu", "kvc_static.cu",
            "kvc_selftest.cu", "kvc_attend.cu", "kvc_join.cu", "kvc_evict.cu", "kvc_operators.cu",
            "kvc_store.cu", "kvc_rotate.cu"]
ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]

KVC_OK = 0
KVC_ERR_INVALID_ARG = 1
KVC_ERR_UNSUPPORTED = 2
KVC_ERR_CUDA = 3
KVC_ERR_BAD_INDEX = 4
KVC_ERR_TIMEOUT = 5
KVC_ERR_SCRATCH_LIMIT = 6
KVC_FLAG_GRID_MASK = 0xFFFF
KVC_DTYPE_F32 = 0
KVC_DTYPE_BF16 = 1
KVC_FORMAT_8BIT = 0
KVC_FORMAT_4BIT = 1
KVC_FLAG_CLUSTER_SHIFT = 16
KVC_FLAG_STREAM_K = 1 << 24
KVC_FLAG_ROW_COPIES = 1 << 25


def make_flags(route: str = "auto", count: int = 0, cluster_size: int = 0,
               row_copies: bool = False) -> int:
    """kvc_compress flags: route 'auto' | 'cluster' | 'streamk', a forced
    launch size (clusters or CTAs; 0 = automatic), cluster size, and, for
    rows apart, row-by-row copies instead of TMA tensor maps."""
    f = int(count) & KVC_FLAG_GRID_MASK
    if route == "streamk":
        f |= KVC_FLAG_STREAM_K
    else:
        f |= (int(cluster_size) & 0x1F) << KVC_FLAG_CLUSTER_SHIFT
    if row_copies:
        f |= KVC_FLAG_ROW_COPIES
    return f

HEAD_DIM = 512
KV_PAGE_BYTES = 64 * (576 + 8)
KV4_PAGE_BYTES = 64 * (352 + 16)  # of 4-bit slots
ROPE_DIM = 64

_lock = threading.Lock()
_lib = None
_quick = None


class KvcError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {kvc_error_string(status)} (status {status})")


# ---- build -------------------------------------------------------------------

def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _stale() -> bool:
    if not os.path.exists(LIB_PATH):
        return True
    t = os.path.getmtime(LIB_PATH)
    deps = [os.path.join(_CSRC, f) for f in os.listdir(_CSRC)]
    deps.append(os.path.join(_INCLUDE, "kvc.h"))
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile csrc/*.cu for sm_103a into _lib/libkvc.so (in-tree)."""
    os.makedirs(_LIB_DIR, exist_ok=True)
    if not force and not _stale():
        _build_call()
        return LIB_PATH
    nvcc = _nvcc()
    common = ARCH_FLAGS + ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC",
                           "-I", _INCLUDE]
    objs = [os.path.join(_LIB_DIR, s.replace(".cu", ".o")) for s in _SOURCES]

    def compile_one(src_obj):
        src, obj = src_obj
        cmd = [nvcc] + common + ["-c", os.path.join(_CSRC, src), "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        return r.stderr

    with ThreadPoolExecutor(len(_SOURCES) + 1) as ex:
        calls = ex.submit(_build_call, force)
        logs = list(ex.map(compile_one, zip(_SOURCES, objs)))
        tmp = LIB_PATH + f".tmp{os.getpid()}"
        r = subprocess.run([nvcc, "-shared"] + ARCH_FLAGS + objs + ["-o", tmp],
                           capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB_PATH)
        calls.result()
    if verbose:
        print("".join(logs))
    return LIB_PATH


def _call_path(torch_dir):
    """Where kvc_call.cpp's module lies that was built for this interpreter, the torch in
    `torch_dir` and the entry points of these sources; None if these cannot be told.  It
    reads tensors and passes arguments as the headers lay them out that it was built with:
    one built beside others has another name, and is not loaded."""
    tag = hashlib.sha256(str(sysconfig.get_config_var("SOABI")).encode())
    try:
        for path in (os.path.join(torch_dir, "version.py"), os.path.join(_CSRC, "kvc_call.cpp"),
                     os.path.join(_INCLUDE, "kvc.h")):
            with open(path, "rb") as f:
                tag.update(hashlib.sha256(f.read()).digest())
        for name in ("libc10.so", "libtorch_python.so"):
            tag.update(b"%d " % os.path.getsize(os.path.join(torch_dir, "lib", name)))
    except OSError:
        return None
    return os.path.join(_LIB_DIR, f"_kvc_call.{tag.hexdigest()[:16]}.so")


def _call_command(root, out):
    """The compiler's command that makes kvc_call.cpp's module of the torch in `root`; None
    without a compiler, torch with CUDA, or a header or library of theirs."""
    libs = os.path.join(root, "lib")
    cuda = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    includes = [sysconfig.get_paths()["include"], os.path.join(root, "include"), cuda]
    needed = [os.path.join(includes[0], "Python.h"), os.path.join(cuda, "cuda_runtime.h"),
              os.path.join(includes[1], "torch", "csrc", "autograd", "python_variable.h"),
              os.path.join(includes[1], "c10", "cuda", "impl", "cuda_cmake_macros.h")]
    linked = ["c10", "c10_cuda", "torch_cpu", "torch_python"]
    needed += [os.path.join(libs, f"lib{name}.so") for name in linked]
    if shutil.which("g++") is None or not all(map(os.path.exists, needed)):
        return None
    try:
        import torch
    except (ImportError, OSError):
        return None
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}"]
    cmd += [f"-I{d}" for d in includes] + [os.path.join(_CSRC, "kvc_call.cpp"), "-o", out, "-L" + libs]
    return cmd + [f"-l{name}" for name in linked] + ["-Wl,-rpath," + libs]


def _build_call(force: bool = False) -> None:
    """Compile csrc/kvc_call.cpp, the operators' calls as the interpreter's own functions,
    unless it is there, and remove what was built beside other sources, another torch or
    interpreter.  Where that cannot be done, calls go through ctypes; a compiler that fails
    is not asked again for the same sources and torch (but with force)."""
    spec = importlib.util.find_spec("torch")
    root = "" if spec is None or spec.origin is None else os.path.dirname(spec.origin)
    path = _call_path(root)
    failed = f"{path}.failed"
    try:
        for name in os.listdir(_LIB_DIR):
            old = os.path.join(_LIB_DIR, name)
            if name.startswith("_kvc_call.") and name.endswith((".so", ".failed")) and (force or old not in (path, failed)):
                with contextlib.suppress(FileNotFoundError):  # (another process was quicker)
                    os.remove(old)
        if path is None or os.path.exists(path) or os.path.exists(failed):
            return
        tmp = path + f".tmp{os.getpid()}"
        cmd = _call_command(root, tmp)
        if cmd is None:
            return
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode == 0:
            os.replace(tmp, path)
            return
        said = f"{r.stdout}\n{r.stderr}"
        with open(failed, "w") as f:
            f.write(said)
    except OSError as e:
        said = str(e)
    warnings.warn(f"kvc_call.cpp was not compiled, calls go through ctypes:\n{said}", RuntimeWarning)


# ---- loading -----------------------------------------------------------------

def lib():
    """The loaded libkvc.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"{LIB_PATH} is missing: build it with "
                    "kv_cache_compression_c128_gb300.build() (there is no CPU fallback)")
            L = ctypes.CDLL(LIB_PATH)
            P, I64, I32, U32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_uint32
            L.kvc_workspace_bytes.argtypes = [I64]
            L.kvc_workspace_bytes.restype = ctypes.c_size_t
            L.kvc_compress.argtypes = [
                P, I64, P, P, I64, P, I64, P, I64, I64, P, P, I64, P, I64, P, I64,
                I32, I32, ctypes.c_float, P, P, ctypes.c_size_t, U32, P]
            L.kvc_compress.restype = ctypes.c_int
            L.kvc_compress_static.argtypes = [
                P, I64, P, P, I64, P, I64, P, I64, I64, P, P, I64, P, I64, P, I64,
                I32, I32, ctypes.c_float, P, U32, P]
            L.kvc_compress_static.restype = ctypes.c_int
            L.kvc_compress_layers.argtypes = [
                I32, P, I64, P, P, I64, P, I64, P, I64, I64, P, P, I64, P, I64, P, I64,
                I32, I32, ctypes.c_float, P, P, ctypes.c_size_t, U32, P]
            L.kvc_compress_layers.restype = ctypes.c_int
            L.kvc_compress_layers_strided.argtypes = [
                I32, P, I32, I64, I64, I64, P, P, I64, P, I64, P, I64, I64, I64, I64, P, P, I64,
                P, I64, P, I64, I32, I32, ctypes.c_float, P, P, ctypes.c_size_t, U32, P]
            L.kvc_compress_layers_strided.restype = ctypes.c_int
            L.kvc_dequantize.argtypes = [P, I64, P, I64, P, I32, P]
            L.kvc_dequantize.restype = ctypes.c_int
            L.kvc_compress_strided.argtypes = [
                P, I32, I64, I64, I64, P, P, I64, P, I64, P, I64, I64, I64, I64, P, P, I64, P,
                I64, P, I64, I32, I32, ctypes.c_float, P, P, ctypes.c_size_t, U32, P]
            L.kvc_compress_strided.restype = ctypes.c_int
            L.kvc_attend_workspace_bytes.argtypes = [I64, I32, I64, I32]
            L.kvc_attend_workspace_bytes.restype = ctypes.c_size_t
            L.kvc_attend.argtypes = [
                P, I64, I64, I64, I32, P, I64, P, I64, I64, P, ctypes.c_float, P, P, P, P, I64,
                P, I64, I64, P, ctypes.c_size_t, U32, P]
            L.kvc_attend.restype = ctypes.c_int
            L.kvc_attend_format.argtypes = [
                P, I64, I64, I64, I32, P, I32, I64, P, I64, I64, P, ctypes.c_float, P, P, P, P,
                I64, P, I64, I64, P, ctypes.c_size_t, U32, P]
            L.kvc_attend_format.restype = ctypes.c_int
            L.kvc_join.argtypes = [P, P, I32, I64, I32, P, P, P]
            L.kvc_join.restype = ctypes.c_int
            L.kvc_evict_workspace_bytes.argtypes = [I64, I64, I64]
            L.kvc_evict_workspace_bytes.restype = ctypes.c_size_t
            L.kvc_evict.argtypes = [
                P, I64, P, I64, I64, I64, P, P, I64, I64, P, I64, I64, I64, P, P, P, I64, P, I64,
                P, ctypes.c_size_t, P]
            L.kvc_evict.restype = ctypes.c_int
            L.kvc_evict_format.argtypes = [
                P, I32, I64, P, I64, I64, I64, P, P, I64, I64, P, I64, I64, I64, P, P, P, I64, P,
                I64, P, ctypes.c_size_t, P]
            L.kvc_evict_format.restype = ctypes.c_int
            L.kvc_store.argtypes = [P, I32, I64, I64, P, I32, I64, P, P, I64, I64, I32,
                                    ctypes.c_char_p, P, I64, P]
            L.kvc_store.restype = ctypes.c_int
            L.kvc_dequantize_format.argtypes = [P, I32, I64, P, I64, P, I32, P]
            L.kvc_dequantize_format.restype = ctypes.c_int
            L.kvc_rotate.argtypes = [P, I32, I64, I64, I64, I32, P, I64, I64, I32,
                                     ctypes.c_char_p, P, I64, I32, P, I64, I64, P]
            L.kvc_rotate.restype = ctypes.c_int
            L.kvc_query_launch.argtypes = [I64, I32, U32, P, P, P, P]
            L.kvc_query_launch.restype = ctypes.c_int
            L.kvc_query_launch_ex.argtypes = [I64, I32, I32, U32, P, P, P, P]
            L.kvc_query_launch_ex.restype = ctypes.c_int
            L.kvc_selftest_wait_timeout.argtypes = [ctypes.c_uint64, P]
            L.kvc_selftest_wait_timeout.restype = ctypes.c_int
            L.kvc_selftest_set_wait_limit.argtypes = [ctypes.c_uint64]
            L.kvc_selftest_set_wait_limit.restype = ctypes.c_int
            L.kvc_selftest_poison_guesses.argtypes = [I32]
            L.kvc_selftest_poison_guesses.restype = ctypes.c_int
            L.kvc_selftest_first_pass_rejections.argtypes = [P, P]
            L.kvc_selftest_first_pass_rejections.restype = ctypes.c_int
            L.kvc_get_device_error.argtypes = [P, P]
            L.kvc_get_device_error.restype = ctypes.c_int
            L.kvc_error_string.argtypes = [ctypes.c_int]
            L.kvc_error_string.restype = ctypes.c_char_p
            L.kvc_version.argtypes = []
            L.kvc_version.restype = ctypes.c_char_p
            _lib = L
    return _lib


def _load_quick():
    """kvc_call.cpp's functions, where they were built (torch is loaded)."""
    global _quick
    path = _call_path(os.path.dirname(_torch.__file__))
    if _quick is None and path is not None and os.path.exists(LIB_PATH) and os.path.exists(path):
        try:
            loader = importlib.machinery.ExtensionFileLoader("_kvc_call", path)
            call = importlib.util.module_from_spec(importlib.util.spec_from_loader("_kvc_call", loader))
            loader.exec_module(call)
        except ImportError:  # (a library that it needs is gone)
            return
        L = lib()
        call.bind(*[ctypes.cast(f, ctypes.c_void_p).value for f in (
            L.kvc_attend_format, L.kvc_evict_format, L.kvc_store, L.kvc_dequantize_format, L.kvc_rotate)])
        _quick = call


def _entry():
    """What the operators call the library through: lib(), or the same with quicker calls."""
    return _quick or lib()


# ---- the C ABI, one Python function per entry point ---------------------------

def kvc_error_string(status: int) -> str:
    return lib().kvc_error_string(int(status)).decode()


def kvc_version() -> str:
    return lib().kvc_version().decode()


def kvc_workspace_bytes(num_outputs: int) -> int:
    return int(lib().kvc_workspace_bytes(int(num_outputs)))


def kvc_query_launch(num_outputs: int, compress_ratio: int, flags: int = 0):
    """(ctas, cluster size, threads, dynamic smem bytes) of the launch."""
    c, k, t, s = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32()
    st = lib().kvc_query_launch(int(num_outputs), int(compress_ratio), int(flags),
                                ctypes.byref(c), ctypes.byref(k), ctypes.byref(t),
                                ctypes.byref(s))
    if st != KVC_OK:
        raise KvcError(st, "kvc_query_launch")
    return c.value, k.value, t.value, s.value


def kvc_query_launch_ex(num_outputs: int, compress_ratio: int, state_dtype: int,
                        flags: int = 0):
    """kvc_query_launch for a state of element type state_dtype (KVC_DTYPE_*)."""
    c, k, t, s = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32()
    st = lib().kvc_query_launch_ex(int(num_outputs), int(compress_ratio), int(state_dtype),
                                   int(flags), ctypes.byref(c), ctypes.byref(k),
                                   ctypes.byref(t), ctypes.byref(s))
    if st != KVC_OK:
        raise KvcError(st, "kvc_query_launch_ex")
    return c.value, k.value, t.value, s.value


def kvc_selftest_wait_timeout(limit_cycles: int, stream: Optional[int] = None) -> int:
    """Launch the bounded-wait self-test (a wait that runs out after
    limit_cycles and records KVC_ERR_TIMEOUT); returns the launch status."""
    return int(lib().kvc_selftest_wait_timeout(int(limit_cycles), ctypes.c_void_p(stream or 0)))


def kvc_selftest_set_wait_limit(limit_cycles: int) -> int:
    """Test hook: the limit (SM cycles) on each pipeline wait of later
    compressions in this process; 0 restores the default.  Returns the
    status."""
    return int(lib().kvc_selftest_set_wait_limit(int(limit_cycles)))


def kvc_selftest_poison_guesses(on: bool) -> int:
    """Test hook: make every guessed first pass of later calls in this
    process fail its check (True) or guess normally (False).  Returns the
    status."""
    return int(lib().kvc_selftest_poison_guesses(1 if on else 0))


def kvc_selftest_first_pass_rejections(stream: Optional[int] = None) -> int:
    """Synchronise `stream`, read and clear the count of guessed first passes
    that failed their check on the current device."""
    n = ctypes.c_uint64()
    st = lib().kvc_selftest_first_pass_rejections(ctypes.c_void_p(stream or 0), ctypes.byref(n))
    if st != KVC_OK:
        raise KvcError(st, "kvc_selftest_first_pass_rejections")
    return int(n.value)


def kvc_get_device_error(stream: Optional[int] = None) -> int:
    """Synchronise `stream` (a cudaStream_t as int), read and clear the
    device error code."""
    code = ctypes.c_uint32()
    st = lib().kvc_get_device_error(ctypes.c_void_p(stream or 0), ctypes.byref(code))
    if st != KVC_OK:
        raise KvcError(st, "kvc_get_device_error")
    return int(code.value)


def kvc_compress(state_cache, num_state_blocks, token_to_req, positions, num_tokens,
                 boundary_token_indices, num_outputs, block_table, num_reqs,
                 max_blocks_per_req, rms_norm_weight, cos_sin_cache, num_positions,
                 kv_slot_mapping, slot_mapping_len, kv_cache, num_kv_pages, block_size,
                 compress_ratio, rms_norm_eps, y_out, workspace, workspace_bytes,
                 flags, stream) -> int:
    """The C entry point with raw integer pointers; returns the status."""
    v = ctypes.c_void_p
    return int(lib().kvc_compress(
        v(state_cache), num_state_blocks, v(token_to_req), v(positions), num_tokens,
        v(boundary_token_indices), num_outputs, v(block_table), num_reqs,
        max_blocks_per_req, v(rms_norm_weight), v(cos_sin_cache), num_positions,
        v(kv_slot_mapping), slot_mapping_len, v(kv_cache), num_kv_pages, block_size,
        compress_ratio, ctypes.c_float(rms_norm_eps), v(y_out), v(workspace),
        workspace_bytes, flags, v(stream)))


def kvc_compress_strided(state_cache, state_dtype, num_state_blocks, state_block_stride,
                         state_row_stride, token_to_req, positions, num_tokens,
                         boundary_token_indices, num_outputs, block_table, num_reqs,
                         max_blocks_per_req, block_table_row_stride, block_table_col_stride,
                         rms_norm_weight, cos_sin_cache, num_positions, kv_slot_mapping,
                         slot_mapping_len, kv_cache, num_kv_pages, block_size, compress_ratio,
                         rms_norm_eps, y_out, workspace, workspace_bytes, flags, stream) -> int:
    """The strided / fp32-state C entry point with raw integer pointers."""
    v = ctypes.c_void_p
    return int(lib().kvc_compress_strided(
        v(state_cache), int(state_dtype), num_state_blocks, state_block_stride,
        state_row_stride, v(token_to_req), v(positions), num_tokens,
        v(boundary_token_indices), num_outputs, v(block_table), num_reqs, max_blocks_per_req,
        block_table_row_stride, block_table_col_stride, v(rms_norm_weight), v(cos_sin_cache),
        num_positions, v(kv_slot_mapping), slot_mapping_len, v(kv_cache), num_kv_pages,
        int(block_size), int(compress_ratio), float(rms_norm_eps), v(y_out), v(workspace),
        int(workspace_bytes), int(flags), v(stream)))


def kvc_compress_static(state_cache, num_state_blocks, token_to_req, positions, num_tokens,
                        boundary_token_indices, num_outputs, block_table, num_reqs,
                        max_blocks_per_req, rms_norm_weight, cos_sin_cache, num_positions,
                        kv_slot_mapping, slot_mapping_len, kv_cache, num_kv_pages, block_size,
                        compress_ratio, rms_norm_eps, y_out, flags, stream) -> int:
    """kvc_compress without a workspace, for callers that cannot allocate
    device memory: the library's built-in 8 MiB scratch buffer is used
    instead (shared by all calls on a device; order overlapping calls).
    Raw integer pointers; returns the status."""
    v = ctypes.c_void_p
    return int(lib().kvc_compress_static(
        v(state_cache), num_state_blocks, v(token_to_req), v(positions), num_tokens,
        v(boundary_token_indices), num_outputs, v(block_table), num_reqs,
        max_blocks_per_req, v(rms_norm_weight), v(cos_sin_cache), num_positions,
        v(kv_slot_mapping), slot_mapping_len, v(kv_cache), num_kv_pages, block_size,
        compress_ratio, ctypes.c_float(rms_norm_eps), v(y_out), flags, v(stream)))


def kvc_compress_layers(num_layers, state_caches, num_state_blocks, token_to_req, positions,
                        num_tokens, boundary_token_indices, num_outputs, block_table, num_reqs,
                        max_blocks_per_req, rms_norm_weights, cos_sin_cache, num_positions,
                        kv_slot_mapping, slot_mapping_len, kv_caches, num_kv_pages, block_size,
                        compress_ratio, rms_norm_eps, y_out, workspace, workspace_bytes, flags,
                        stream) -> int:
    """The multi-layer entry point; the three per-layer arguments are
    sequences of integer device pointers.  Returns the status."""
    v = ctypes.c_void_p
    arr = lambda xs: (ctypes.c_void_p * len(xs))(*[int(x) for x in xs])
    return int(lib().kvc_compress_layers(
        int(num_layers), arr(state_caches), num_state_blocks, v(token_to_req), v(positions),
        num_tokens, v(boundary_token_indices), num_outputs, v(block_table), num_reqs,
        max_blocks_per_req, arr(rms_norm_weights), v(cos_sin_cache), num_positions,
        v(kv_slot_mapping), slot_mapping_len, arr(kv_caches), num_kv_pages, block_size,
        compress_ratio, ctypes.c_float(rms_norm_eps), v(y_out), v(workspace), workspace_bytes,
        flags, v(stream)))


def kvc_compress_layers_strided(num_layers, state_caches, state_dtype, num_state_blocks,
                                state_block_stride, state_row_stride, token_to_req, positions,
                                num_tokens, boundary_token_indices, num_outputs, block_table,
                                num_reqs, max_blocks_per_req, block_table_row_stride,
                                block_table_col_stride, rms_norm_weights, cos_sin_cache,
                                num_positions, kv_slot_mapping, slot_mapping_len, kv_caches,
                                num_kv_pages, block_size, compress_ratio, rms_norm_eps, y_out,
                                workspace, workspace_bytes, flags, stream) -> int:
    """The strided multi-layer entry point (raw integer pointers, per-layer
    sequences for the three per-layer arguments).  Returns the status."""
    v = ctypes.c_void_p
    arr = lambda xs: (ctypes.c_void_p * len(xs))(*[int(x) for x in xs])
    return int(lib().kvc_compress_layers_strided(
        int(num_layers), arr(state_caches), int(state_dtype), num_state_blocks,
        state_block_stride, state_row_stride, v(token_to_req), v(positions), num_tokens,
        v(boundary_token_indices), num_outputs, v(block_table), num_reqs, max_blocks_per_req,
        block_table_row_stride, block_table_col_stride, arr(rms_norm_weights), v(cos_sin_cache),
        num_positions, v(kv_slot_mapping), slot_mapping_len, arr(kv_caches), num_kv_pages,
        int(block_size), int(compress_ratio), ctypes.c_float(rms_norm_eps), v(y_out),
        v(workspace), int(workspace_bytes), int(flags), v(stream)))


def kvc_dequantize(kv_cache, num_kv_pages, slots, num_slots, out, out_dtype, stream) -> int:
    """Decode slots back to vectors (raw integer pointers); returns the status."""
    v = ctypes.c_void_p
    return int(lib().kvc_dequantize(v(kv_cache), num_kv_pages, v(slots), num_slots, v(out),
                                    int(out_dtype), v(stream)))


def kvc_dequantize_format(kv_cache, kv_format, num_kv_pages, slots, num_slots, out, out_dtype,
                          stream) -> int:
    """Decode slots of either form (raw integer pointers); returns the status."""
    return _entry().kvc_dequantize_format(kv_cache, kv_format, num_kv_pages, slots, num_slots, out,
                                       out_dtype, stream)


def kvc_store(x, x_dtype, x_row_stride, num_rows, kv_cache, kv_format, num_kv_pages, slots,
              positions, positions_row_stride, positions_axis_stride, num_axes, pair_axes,
              cos_sin_cache, num_positions, stream) -> int:
    """Vectors into packed slots (raw integer pointers; pair_axes 32 bytes or
    None); returns the status."""
    return _entry().kvc_store(
        x, x_dtype, x_row_stride, num_rows, kv_cache, kv_format, num_kv_pages, slots, positions,
        positions_row_stride, positions_axis_stride, num_axes, pair_axes, cos_sin_cache,
        num_positions, stream)


def kvc_rotate(x, dtype, x_token_stride, x_head_stride, num_tokens, num_heads, positions,
               positions_token_stride, positions_axis_stride, num_axes, pair_axes, cos_sin_cache,
               num_positions, inverse, out, out_token_stride, out_head_stride, stream) -> int:
    """Rotary positions (raw integer pointers; pair_axes 32 bytes or None);
    returns the status."""
    return _entry().kvc_rotate(
        x, dtype, x_token_stride, x_head_stride, num_tokens, num_heads, positions,
        positions_token_stride, positions_axis_stride, num_axes, pair_axes, cos_sin_cache,
        num_positions, inverse, out, out_token_stride, out_head_stride, stream)


def kvc_attend_workspace_bytes(num_reqs: int, num_heads: int, max_pages_per_req: int,
                               with_slot_weights: bool = False) -> int:
    return int(lib().kvc_attend_workspace_bytes(int(num_reqs), int(num_heads),
                                                int(max_pages_per_req), int(with_slot_weights)))


def kvc_attend(q, q_req_stride, q_head_stride, num_reqs, num_heads, kv_cache, num_kv_pages,
               page_table, max_pages_per_req, page_table_row_stride, lengths, scale, sinks, out,
               lse, slot_weights_in, slot_weights_in_row_stride, slot_weights,
               slot_weights_row_stride, max_slots, workspace, workspace_bytes, flags,
               stream) -> int:
    """Attention over packed slots (raw integer pointers); returns the status."""
    return lib().kvc_attend(
        q, q_req_stride, q_head_stride, num_reqs, num_heads, kv_cache, num_kv_pages, page_table,
        max_pages_per_req, page_table_row_stride, lengths, scale, sinks, out, lse,
        slot_weights_in, slot_weights_in_row_stride, slot_weights, slot_weights_row_stride,
        max_slots, workspace, workspace_bytes, flags, stream)


def kvc_attend_format(q, q_req_stride, q_head_stride, num_reqs, num_heads, kv_cache, kv_format,
                      num_kv_pages, page_table, max_pages_per_req, page_table_row_stride, lengths,
                      scale, sinks, out, lse, slot_weights_in, slot_weights_in_row_stride,
                      slot_weights, slot_weights_row_stride, max_slots, workspace,
                      workspace_bytes, flags, stream) -> int:
    """kvc_attend over pages of either form."""
    return _entry().kvc_attend_format(
        q, q_req_stride, q_head_stride, num_reqs, num_heads, kv_cache, kv_format, num_kv_pages,
        page_table, max_pages_per_req, page_table_row_stride, lengths, scale, sinks, out, lse,
        slot_weights_in, slot_weights_in_row_stride, slot_weights, slot_weights_row_stride,
        max_slots, workspace, workspace_bytes, flags, stream)


def kvc_join(outs, lses, num_rows, dtype, out, lse, stream) -> int:
    """Join of attention parts; outs and lses are sequences of integer device
    pointers.  Returns the status."""
    arr = ctypes.c_void_p * len(outs)
    return lib().kvc_join(arr(*outs), arr(*lses), len(outs), num_rows, dtype, out, lse, stream)


def kvc_evict_workspace_bytes(num_reqs: int, max_pages_per_req: int, keep: int) -> int:
    return int(lib().kvc_evict_workspace_bytes(int(num_reqs), int(max_pages_per_req), int(keep)))


def kvc_evict(kv_cache, num_kv_pages, page_table, num_reqs, max_pages_per_req,
              page_table_row_stride, lengths, slot_weights, slot_weights_row_stride, max_slots,
              births, births_row_stride, keep, recent, lengths_out, kept, slot_weights_out,
              slot_weights_out_row_stride, births_out, births_out_row_stride, workspace,
              workspace_bytes, stream) -> int:
    """Eviction of packed slots (raw integer pointers); returns the status."""
    return lib().kvc_evict(
        kv_cache, num_kv_pages, page_table, num_reqs, max_pages_per_req, page_table_row_stride,
        lengths, slot_weights, slot_weights_row_stride, max_slots, births, births_row_stride,
        keep, recent, lengths_out, kept, slot_weights_out, slot_weights_out_row_stride,
        births_out, births_out_row_stride, workspace, workspace_bytes, stream)


def kvc_evict_format(kv_cache, kv_format, num_kv_pages, page_table, num_reqs, max_pages_per_req,
                     page_table_row_stride, lengths, slot_weights, slot_weights_row_stride,
                     max_slots, births, births_row_stride, keep, recent, lengths_out, kept,
                     slot_weights_out, slot_weights_out_row_stride, births_out,
                     births_out_row_stride, workspace, workspace_bytes, stream) -> int:
    """kvc_evict over pages of either form."""
    return _entry().kvc_evict_format(
        kv_cache, kv_format, num_kv_pages, page_table, num_reqs, max_pages_per_req,
        page_table_row_stride, lengths, slot_weights, slot_weights_row_stride, max_slots, births,
        births_row_stride, keep, recent, lengths_out, kept, slot_weights_out,
        slot_weights_out_row_stride, births_out, births_out_row_stride, workspace,
        workspace_bytes, stream)


# ---- torch-facing wrappers ----------------------------------------------------

def dequantize(kv_cache, slots, dtype=None, out=None, stream=None):
    """Read slots of a packed kv_cache back as [len(slots), 512] vectors
    (torch.float32 or torch.bfloat16) on the cache's device.  Pages of 23552
    bytes hold 4-bit slots, pages of 37376 8-bit ones.  `out`, if given, is a
    contiguous tensor of that dtype with room for len(slots) * 512 values."""
    torch = _torch or _load_torch()
    dtype = torch.float32 if dtype is None else dtype
    if out is not None and stream is None and _quick is not None and isinstance(out, torch.Tensor) and out.dtype == dtype:
        st = _quick.dequantize(kv_cache, slots, out)
        if st == KVC_OK:
            return out
        if st is not None:
            raise KvcError(st, "kvc_dequantize")
    if dtype not in _dtype_codes:
        raise TypeError("dtype must be torch.float32 or torch.bfloat16")
    if not kv_cache.is_cuda:
        raise ValueError("kv_cache must be a CUDA tensor (there is no CPU path)")
    device = kv_cache.get_device()
    if not _is_flat(kv_cache, torch.uint8, device):
        _check(kv_cache, "kv_cache", torch.uint8, kv_cache.device)
    if not _is_flat(slots, torch.int64, device):
        _check(slots, "slots", torch.int64, kv_cache.device)
    M = slots.numel()
    if out is not None and not _is_flat(out, dtype, device):
        _check(out, "out", dtype, kv_cache.device)
    shape = kv_cache.shape
    four = len(shape) == 2 and shape[1] == KV4_PAGE_BYTES
    # (of 8-bit slots also pages in several dimensions: [num_pages, 64, 584])
    if not shape or kv_cache.numel() != shape[0] * (KV4_PAGE_BYTES if four else KV_PAGE_BYTES):
        raise ValueError(f"kv_cache must be [num_pages, {KV_PAGE_BYTES}] uint8, or [num_pages, {KV4_PAGE_BYTES}] of 4-bit slots")
    if out is not None and out.numel() < M * HEAD_DIM:
        raise ValueError("out must hold len(slots) * 512 values")

    def call(raw):
        nonlocal out
        if out is None:
            out = torch.empty((M, HEAD_DIM), dtype=dtype, device=kv_cache.device)
        return _entry().kvc_dequantize_format(kv_cache.data_ptr(), KVC_FORMAT_4BIT if four else KVC_FORMAT_8BIT, shape[0],
                                     slots.data_ptr(), M, out.data_ptr(), _dtype_codes[dtype], raw)

    st = _run(call, device, stream)
    if st != KVC_OK:
        raise KvcError(st, "kvc_dequantize")
    return out


# ---- torch-facing wrapper with the statement's signature ----------------------

_workspaces = {}


def workspace_for(device, stream_ptr: int, num_outputs: int):
    """A zero-initialised workspace cached per (device, stream)."""
    import torch

    need = kvc_workspace_bytes(num_outputs)
    key = (device.index, stream_ptr)
    ws = _workspaces.get(key)
    if ws is None or ws.numel() < need:
        ws = torch.zeros(max(need, 1 << 20), dtype=torch.uint8, device=device)
        _workspaces[key] = ws
    return ws


def _check(t, name, dtype, device, contiguous=True):
    import torch

    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    dtypes = dtype if isinstance(dtype, tuple) else (dtype,)
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must have dtype {' or '.join(map(str, dtypes))}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def c128_256_512_compress(state_cache, token_to_req, positions, boundary_token_indices,
                          block_table, rms_norm_weight, cos_sin_cache, kv_slot_mapping,
                          kv_cache, block_size, compress_ratio, rms_norm_eps=1.0e-6, *,
                          y_out=None, flags: int = 0, stream=None, workspace=None):
    """Compress every boundary token's window into its kv_cache slot, in place.

    state_cache bf16 or fp32 [blocks, block_size, 1024] (any block and row
    strides, columns contiguous); token_to_req int32 [T]; positions int64
    [T]; boundary_token_indices int64 [N]; block_table int32 [R, Lb] (any
    strides); rms_norm_weight fp32 [512]; cos_sin_cache fp32 [P, 64];
    kv_slot_mapping int64 [T] (or [N]); kv_cache uint8 [pages, 37376].  All
    on one CUDA device.  Optional y_out fp32 [N, 512] receives the
    normalised vectors.  A contiguous bf16 state with a contiguous table goes
    through kvc_compress, anything else through kvc_compress_strided.
    Returns kv_cache.
    """
    import torch

    dev = state_cache.device
    if dev.type != "cuda":
        raise ValueError("state_cache must be a CUDA tensor (there is no CPU path)")
    _check(state_cache, "state_cache", (torch.bfloat16, torch.float32), dev, contiguous=False)
    _check(token_to_req, "token_to_req", torch.int32, dev)
    _check(positions, "positions", torch.int64, dev)
    _check(boundary_token_indices, "boundary_token_indices", torch.int64, dev)
    _check(block_table, "block_table", torch.int32, dev, contiguous=False)
    _check(rms_norm_weight, "rms_norm_weight", torch.float32, dev)
    _check(cos_sin_cache, "cos_sin_cache", torch.float32, dev)
    _check(kv_slot_mapping, "kv_slot_mapping", torch.int64, dev)
    _check(kv_cache, "kv_cache", torch.uint8, dev)
    if state_cache.dim() != 3 or state_cache.shape[2] != 2 * HEAD_DIM:
        raise ValueError("state_cache must be [num_blocks, block_size, 1024]")
    if state_cache.stride(2) != 1:
        raise ValueError("state_cache columns must be contiguous (stride(2) == 1)")
    if state_cache.shape[1] != block_size:
        raise ValueError("state_cache.shape[1] must equal block_size")
    if block_table.dim() != 2 or cos_sin_cache.dim() != 2 or cos_sin_cache.shape[1] != 64:
        raise ValueError("block_table must be 2-D and cos_sin_cache [P, 64]")
    if rms_norm_weight.numel() != HEAD_DIM:
        raise ValueError("rms_norm_weight must have 512 elements")
    if kv_cache.dim() != 2 or kv_cache.shape[1] != KV_PAGE_BYTES:
        raise ValueError(f"kv_cache must be [num_pages, {KV_PAGE_BYTES}] uint8")
    if token_to_req.numel() != positions.numel():
        raise ValueError("token_to_req and positions must have one entry per token")
    N = boundary_token_indices.numel()
    if y_out is not None:
        _check(y_out, "y_out", torch.float32, dev)
        if y_out.numel() < N * HEAD_DIM:
            raise ValueError("y_out must hold num_outputs * 512 floats")
    with torch.cuda.device(dev):
        s = stream if stream is not None else torch.cuda.current_stream(dev)
        sp = int(s.cuda_stream)
        ws = workspace if workspace is not None else workspace_for(dev, sp, N)
        y_ptr = 0 if y_out is None else y_out.data_ptr()
        if (state_cache.dtype == torch.bfloat16 and state_cache.is_contiguous()
                and block_table.is_contiguous()):
            name = "kvc_compress"
            st = kvc_compress(
                state_cache.data_ptr(), state_cache.shape[0], token_to_req.data_ptr(),
                positions.data_ptr(), positions.numel(), boundary_token_indices.data_ptr(), N,
                block_table.data_ptr(), block_table.shape[0], block_table.shape[1],
                rms_norm_weight.data_ptr(), cos_sin_cache.data_ptr(), cos_sin_cache.shape[0],
                kv_slot_mapping.data_ptr(), kv_slot_mapping.numel(), kv_cache.data_ptr(),
                kv_cache.shape[0], int(block_size), int(compress_ratio), float(rms_norm_eps),
                y_ptr, ws.data_ptr(), ws.numel(), int(flags), sp)
        else:
            name = "kvc_compress_strided"
            st = kvc_compress_strided(
                state_cache.data_ptr(),
                KVC_DTYPE_F32 if state_cache.dtype == torch.float32 else KVC_DTYPE_BF16,
                state_cache.shape[0], state_cache.stride(0), state_cache.stride(1),
                token_to_req.data_ptr(), positions.data_ptr(), positions.numel(),
                boundary_token_indices.data_ptr(), N, block_table.data_ptr(),
                block_table.shape[0], block_table.shape[1], block_table.stride(0),
                block_table.stride(1), rms_norm_weight.data_ptr(), cos_sin_cache.data_ptr(),
                cos_sin_cache.shape[0], kv_slot_mapping.data_ptr(), kv_slot_mapping.numel(),
                kv_cache.data_ptr(), kv_cache.shape[0], int(block_size), int(compress_ratio),
                float(rms_norm_eps), y_ptr, ws.data_ptr(), ws.numel(), int(flags), sp)
    if st != KVC_OK:
        raise KvcError(st, name)
    return kv_cache


def compress_layers(state_caches, token_to_req, positions, boundary_token_indices, block_table,
                    rms_norm_weights, cos_sin_cache, kv_slot_mapping, kv_caches, block_size,
                    compress_ratio, rms_norm_eps=1.0e-6, *, y_out=None, flags: int = 0,
                    stream=None, workspace=None):
    """c128_256_512_compress for several layers in one launch: lists of
    per-layer state caches, RMSNorm weights and kv caches (same shapes and
    dtypes as the single-layer call) sharing every index array.  The state
    caches are bf16 or fp32, all of one dtype and one set of strides (any
    block and row strides, columns contiguous); the block table may have any
    strides.  y_out, if given, is fp32 [L * N, 512] (layer-major).  Returns
    kv_caches."""
    import torch

    L = len(state_caches)
    if not (len(rms_norm_weights) == L == len(kv_caches)) or L < 1:
        raise ValueError("state_caches, rms_norm_weights and kv_caches need one entry per layer")
    dev = state_caches[0].device
    if dev.type != "cuda":
        raise ValueError("state caches must be CUDA tensors (there is no CPU path)")
    s0 = state_caches[0]
    for l in range(L):
        _check(state_caches[l], f"state_caches[{l}]", (torch.bfloat16, torch.float32), dev,
               contiguous=False)
        _check(rms_norm_weights[l], f"rms_norm_weights[{l}]", torch.float32, dev)
        _check(kv_caches[l], f"kv_caches[{l}]", torch.uint8, dev)
        if state_caches[l].shape != s0.shape or kv_caches[l].shape != kv_caches[0].shape:
            raise ValueError("all layers need the same state and kv_cache shapes")
        if state_caches[l].dtype != s0.dtype or state_caches[l].stride() != s0.stride():
            raise ValueError("all layers need the same state dtype and strides")
    if s0.dim() != 3 or s0.shape[2] != 2 * HEAD_DIM or s0.stride(2) != 1:
        raise ValueError("state caches must be [num_blocks, block_size, 1024] with contiguous columns")
    for name, t, dt in (("token_to_req", token_to_req, torch.int32), ("positions", positions, torch.int64),
                        ("boundary_token_indices", boundary_token_indices, torch.int64),
                        ("cos_sin_cache", cos_sin_cache, torch.float32),
                        ("kv_slot_mapping", kv_slot_mapping, torch.int64)):
        _check(t, name, dt, dev)
    _check(block_table, "block_table", torch.int32, dev, contiguous=False)
    if s0.shape[1] < block_size:
        raise ValueError("state caches must have block_size rows a block")
    if block_table.dim() != 2 or cos_sin_cache.dim() < 1 or cos_sin_cache.numel() < 64 * cos_sin_cache.shape[0]:
        raise ValueError("block_table must be 2-D and cos_sin_cache [P, 64]")
    if any(w.numel() < HEAD_DIM for w in rms_norm_weights):
        raise ValueError("rms_norm_weights must have 512 elements each")
    kv_shape = kv_caches[0].shape  # (pages of 4-bit slots are shorter than what is written)
    if not kv_shape or kv_caches[0].numel() != kv_shape[0] * KV_PAGE_BYTES:
        raise ValueError(f"kv_caches must be [num_pages, {KV_PAGE_BYTES}] uint8")
    if token_to_req.numel() < positions.numel():
        raise ValueError("token_to_req and positions must have one entry per token")
    N = boundary_token_indices.numel()
    if y_out is not None:
        _check(y_out, "y_out", torch.float32, dev)
        if y_out.numel() < L * N * HEAD_DIM:
            raise ValueError("y_out must hold num_layers * num_outputs * 512 floats")
    with torch.cuda.device(dev):
        s = stream if stream is not None else torch.cuda.current_stream(dev)
        sp = int(s.cuda_stream)
        ws = workspace if workspace is not None else workspace_for(dev, sp, N)
        y_ptr = 0 if y_out is None else y_out.data_ptr()
        if s0.dtype == torch.bfloat16 and s0.is_contiguous() and block_table.is_contiguous():
            name = "kvc_compress_layers"
            st = kvc_compress_layers(
                L, [t.data_ptr() for t in state_caches], s0.shape[0],
                token_to_req.data_ptr(), positions.data_ptr(), positions.numel(),
                boundary_token_indices.data_ptr(), N, block_table.data_ptr(), block_table.shape[0],
                block_table.shape[1], [t.data_ptr() for t in rms_norm_weights],
                cos_sin_cache.data_ptr(), cos_sin_cache.shape[0], kv_slot_mapping.data_ptr(),
                kv_slot_mapping.numel(), [t.data_ptr() for t in kv_caches], kv_caches[0].shape[0],
                int(block_size), int(compress_ratio), float(rms_norm_eps), y_ptr, ws.data_ptr(),
                ws.numel(), int(flags), sp)
        else:
            name = "kvc_compress_layers_strided"
            st = kvc_compress_layers_strided(
                L, [t.data_ptr() for t in state_caches],
                KVC_DTYPE_F32 if s0.dtype == torch.float32 else KVC_DTYPE_BF16, s0.shape[0],
                s0.stride(0), s0.stride(1), token_to_req.data_ptr(), positions.data_ptr(),
                positions.numel(), boundary_token_indices.data_ptr(), N, block_table.data_ptr(),
                block_table.shape[0], block_table.shape[1], block_table.stride(0),
                block_table.stride(1), [t.data_ptr() for t in rms_norm_weights],
                cos_sin_cache.data_ptr(), cos_sin_cache.shape[0], kv_slot_mapping.data_ptr(),
                kv_slot_mapping.numel(), [t.data_ptr() for t in kv_caches], kv_caches[0].shape[0],
                int(block_size), int(compress_ratio), float(rms_norm_eps), y_ptr, ws.data_ptr(),
                ws.numel(), int(flags), sp)
    if st != KVC_OK:
        raise KvcError(st, name)
    return kv_caches


# ---- operators on packed slots ------------------------------------------------
#
# These are called once per layer and token, with little work in a small batch:
# the checks below read each attribute once and make no objects in passing.

_torch = None
_dtype_codes = {}  # of the element types, KVC_DTYPE_*


def _load_torch():
    global _torch
    if _torch is None:
        import torch

        _dtype_codes.update({torch.float32: KVC_DTYPE_F32, torch.bfloat16: KVC_DTYPE_BF16})
        _torch = torch
        _load_quick()
    return _torch


def _is_flat(t, dtype, device):
    return isinstance(t, _torch.Tensor) and t.dtype == dtype and t.get_device() == device and t.is_contiguous()


def _refuse(name, t, dtype, dim, device):
    """Raise for the first property of `t` that is not as an operator needs it."""
    if not isinstance(t, _torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must have dtype {dtype}, got {t.dtype}")
    if t.get_device() != device:
        raise ValueError(f"{name} must be on cuda:{device}, got {t.device}")
    if t.dim() != dim:
        raise ValueError(f"{name} must have {dim} dimensions, got {t.dim()}")
    raise ValueError(f"{name} must have contiguous columns")


def _rows(name, t, dtype, device):
    """(rows, columns, row stride) of a 2-D tensor with contiguous columns."""
    if not isinstance(t, _torch.Tensor) or t.dtype != dtype or t.get_device() != device or t.dim() != 2:
        _refuse(name, t, dtype, 2, device)
    rows, cols = t.shape
    row, col = t.stride()
    if col != 1 and cols > 1 and rows > 0:
        _refuse(name, t, dtype, 2, device)
    return rows, cols, row


def _dense(name, t, dtype, device, shape):
    """A contiguous tensor of a given shape."""
    if not isinstance(t, _torch.Tensor) or t.dtype != dtype or t.get_device() != device or t.dim() != len(shape):
        _refuse(name, t, dtype, len(shape), device)
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous {tuple(shape)}, got {tuple(t.shape)}")


def _pages(kv_cache):
    """(device index, pages, their form)"""
    if not isinstance(kv_cache, _torch.Tensor) or not kv_cache.is_cuda:
        raise ValueError("kv_cache must be a CUDA tensor (there is no CPU path)")
    device = kv_cache.get_device()
    if kv_cache.dtype != _torch.uint8 or kv_cache.dim() != 2:
        _refuse("kv_cache", kv_cache, _torch.uint8, 2, device)
    pages, width = kv_cache.shape
    if (width != KV_PAGE_BYTES and width != KV4_PAGE_BYTES) or not kv_cache.is_contiguous():
        raise ValueError(f"kv_cache must be contiguous [num_pages, {KV_PAGE_BYTES}] uint8, or "
                         f"[num_pages, {KV4_PAGE_BYTES}] of 4-bit slots")
    return device, pages, KVC_FORMAT_8BIT if width == KV_PAGE_BYTES else KVC_FORMAT_4BIT


def _cache(kv_cache, page_table, lengths):
    """(device index, pages, their form, requests, page table columns, its row stride)"""
    device, pages, form = _pages(kv_cache)
    reqs, columns, row = _rows("page_table", page_table, _torch.int32, device)
    _dense("lengths", lengths, _torch.int32, device, (reqs,))
    return device, pages, form, reqs, columns, row


class _on:
    """Context of an operator call where the caller's device is not current, or
    a stream is given: both current while results and workspaces are allocated
    (memory of another stream's pool could still be in use there)."""

    def __init__(self, device, stream):
        cuda = _torch.cuda
        self.entered = [cuda.device(device)] + ([] if stream is None else [cuda.stream(stream)])

    def __enter__(self):
        for c in self.entered:
            c.__enter__()

    def __exit__(self, *exc):
        for c in reversed(self.entered):
            c.__exit__(*exc)


def _run(call, device, stream):
    """call(raw stream), on the operator's device and stream."""
    cuda = _torch.cuda
    if stream is None:
        if _torch._C._cuda_getDevice() == device:  # (a tensor of the device is there: CUDA is up)
            return call(_torch._C._cuda_getCurrentRawStream(device))
    elif stream.device.index != device:  # (its context would make the other device current)
        raise ValueError(f"stream must be one of cuda:{device}, got one of {stream.device}")
    with _on(device, stream):
        return call(cuda.current_stream(device).cuda_stream)


_known_axes = {None: (1, None)}  # of what `axes` was found right for: (axes that positions have at least, bytes)


def _axes(axes):
    """(axes that positions have at least, the 32 bytes of a C call)"""
    pairs = bytes(list(axes))  # (bytes(32), and those of an array of 4 numbers of 8 bytes, are 32 zeros)
    if len(pairs) != 32:
        raise ValueError("axes must name an axis of positions for each of the 32 pairs")
    known = (max(pairs) + 1, pairs)
    if len(_known_axes) < 64:
        _known_axes[pairs] = known
    return known


def _rotation(positions, cos_sin_cache, axes, rows, device):
    """(positions, row stride, axis stride, axes, pair axes, table, its rows) of a
    C call that turns `rows` rows."""
    int64, float32 = _torch.int64, _torch.float32
    if not isinstance(positions, _torch.Tensor) or positions.dtype != int64 or positions.get_device() != device:
        _refuse("positions", positions, int64, 2, device)
    shape, stride = positions.shape, positions.stride()
    count, apart = 1, 0
    if len(shape) == 2:
        count, apart = shape[1], stride[1]
    elif len(shape) != 1:
        raise ValueError("positions must be [rows] or [rows, axes]")
    if shape[0] != rows:
        raise ValueError("positions must have one row for each of x")
    if not 1 <= count <= 4:
        raise ValueError("positions must have 1 to 4 axes")
    least, pairs = (_known_axes.get(axes) if axes is None or type(axes) is bytes else None) or _axes(axes)
    if least > count:
        raise ValueError("axes must name an axis of positions for each of the 32 pairs")
    if pairs is None and count > 1:
        raise ValueError("positions of several axes need axes, one for each of the 32 pairs")
    if not _is_flat(cos_sin_cache, float32, device) or cos_sin_cache.dim() != 2:
        _refuse("cos_sin_cache", cos_sin_cache, float32, 2, device)
    entries, width = cos_sin_cache.shape
    if width != ROPE_DIM:
        raise ValueError("cos_sin_cache must be contiguous [num_positions, 64]")
    return positions.data_ptr(), stride[0], apart, count, pairs, cos_sin_cache.data_ptr(), entries


def store(x, kv_cache, slots, *, positions=None, cos_sin_cache=None, axes=None, stream=None):
    """Write vectors into packed slots as they come, in place.

    x bf16 or fp32 [N, 512] (any row stride that is a multiple of 16 bytes,
    columns contiguous); kv_cache uint8 [pages, 37376] of 8-bit slots or
    [pages, 23552] of 4-bit ones; slots int64 [N], a negative one skips its row,
    none may be named twice.  Dims 0..447 are rounded to bf16 and quantised: in
    8 bits as the compressor does, in 4 bits to 15 levels with a scale for every
    32 dims.  Dims 448..511 are kept in bf16, turned to `positions` if given
    (with cos_sin_cache and axes as for `rotate`).

    A slot beyond the cache or a position outside the table leaves its slot as
    it was and raises the device error word (kvc_get_device_error).  Returns
    kv_cache.  No gradient is recorded.
    """
    torch = _torch or _load_torch()
    if stream is None and _quick is not None:
        st = _quick.store(x, kv_cache, slots, positions, cos_sin_cache, axes)
        if st == KVC_OK:
            return kv_cache
        if st is not None:
            raise KvcError(st, "kvc_store")
    device, pages, form = _pages(kv_cache)
    if not isinstance(x, torch.Tensor) or x.dtype not in _dtype_codes:
        raise TypeError("x must be a tensor of dtype torch.float32 or torch.bfloat16")
    dtype = x.dtype
    N, D, row = _rows("x", x, dtype, device)
    if D != HEAD_DIM:
        raise ValueError("x must be [rows, 512]")
    _dense("slots", slots, torch.int64, device, (N,))
    turn = (None, 0, 0, 0, None, None, 0)
    if positions is not None:
        turn = _rotation(positions, cos_sin_cache, axes, N, device)
    elif axes is not None or cos_sin_cache is not None:
        raise ValueError("axes and cos_sin_cache need positions")

    def call(raw):
        return _entry().kvc_store(x.data_ptr(), _dtype_codes[dtype], row if N > 1 else 0, N, kv_cache.data_ptr(), form, pages,
                         slots.data_ptr(), *turn, raw)

    st = _run(call, device, stream)
    if st != KVC_OK:
        raise KvcError(st, "kvc_store")
    return kv_cache


def rotate(x, positions, cos_sin_cache, *, axes=None, inverse: bool = False, out=None, stream=None):
    """Rotary positions, with one axis or several.

    x bf16 or fp32 [T, H, 64] or [T, 64] (any token and head strides that are
    multiples of 16 bytes, columns contiguous: the last 64 dims of queries
    [T, H, 512], for instance); positions int64 [T] or [T, 1..4 axes] (any
    strides); cos_sin_cache fp32 [P, 64], cos in columns 0..31, sin 32..63.  Pair
    i (dims 2 i, 2 i + 1) is turned by the angle in column i at the position of
    axis axes[i]: 32 numbers (quickest as bytes), not needed for one axis.

    `inverse` turns by the opposite angles: attention's rows back, whose last 64
    dims are sums of rotated ones, and the gradient with respect to x from the
    one with respect to the result.  Returns `out`, which may be x itself, and whose
    rows share no memory with x's else (a new contiguous tensor if None).  A position outside the table leaves its token's
    rows of out as they were and raises the device error word.  No gradient is
    recorded.
    """
    torch = _torch or _load_torch()
    if out is not None and stream is None and _quick is not None:
        st = _quick.rotate(x, positions, cos_sin_cache, axes, inverse, out)
        if st == KVC_OK:
            return out
        if st is not None:
            raise KvcError(st, "kvc_rotate")
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise ValueError("x must be a CUDA tensor (there is no CPU path)")
    device, dtype, shape, strides = x.get_device(), x.dtype, x.shape, x.stride()
    code = _dtype_codes.get(dtype)
    if code is None:
        raise TypeError("x must have dtype torch.float32 or torch.bfloat16")
    T, H, D, by_token, by_head, by_dim = 0, 1, 0, 0, 0, 0
    if len(shape) == 3:
        T, H, D = shape
        by_token, by_head, by_dim = strides
    elif len(shape) == 2:
        T, D = shape
        by_token, by_dim = strides
    if D != ROPE_DIM or (by_dim != 1 and T * H > 0):
        raise ValueError("x must be [tokens, heads, 64] or [tokens, 64] with contiguous columns")
    at, at_row, at_axis, axis_count, pairs, table, entries = _rotation(positions, cos_sin_cache, axes, T, device)
    if out is not None:
        if not isinstance(out, torch.Tensor) or out.dtype != dtype or out.get_device() != device:
            _refuse("out", out, dtype, len(shape), device)
        if out.shape != shape or (out.stride(-1) != 1 and T * H > 0):
            raise ValueError(f"out must be {tuple(shape)} with contiguous columns")

    def call(raw):
        nonlocal out
        if out is None:
            out = torch.empty(shape, dtype=dtype, device=x.device)
        to = out.stride()
        return _entry().kvc_rotate(
            x.data_ptr(), code, by_token if T > 1 else 0, by_head if H > 1 else 0, T, H, at, at_row, at_axis, axis_count,
            pairs, table, entries, 1 if inverse else 0, out.data_ptr(), to[0] if T > 1 else 0, to[1] if H > 1 else 0, raw)

    st = _run(call, device, stream)
    if st != KVC_OK:
        raise KvcError(st, "kvc_rotate")
    return out


def attend(q, kv_cache, page_table, lengths, scale=None, *, sinks=None, out=None, lse=None,
           slot_weights=None, slot_weights_in=None, flags: int = 0, stream=None, workspace=None):
    """Attention of one new token per request over its packed slots.

    q bf16 [R, H, 512] (any request and head strides that are multiples of 8
    elements, columns contiguous; H up to 128); kv_cache uint8 [pages, 37376], or
    [pages, 23552] of 4-bit slots; page_table int32 [R, max_pages] (any row stride), 64 slots to a page;
    lengths int32 [R], slots of each request.  A slot's decoded vector is the
    key and the value of every head; `scale` defaults to 512 ** -0.5; optional
    sinks fp32 [H] join the softmax as a score without a value.

    Returns (out bf16 [R, H, 512], lse fp32 [R, H]).  With slot_weights (fp32
    [R, S]), entry [r, n] of every slot also receives slot_weights_in[r, n]
    (zero without it; may be the same tensor) plus the slot's softmax weight
    summed over the heads: what `evict` goes by.  They are shares among these
    slots and the sink; what a head gives to tokens that are joined later does
    not lower them.  A request whose length or pages are out of range keeps its
    rows as they were (undefined in results that the call allocates) and raises
    the device error word (kvc_get_device_error).  A workspace given by the
    caller (kvc_attend_workspace_bytes) serves calls that do not overlap; with
    slot_weights it holds a score for every slot of the page table's width and
    every head.  A serving form: no gradient is recorded.
    """
    torch = _torch or _load_torch()
    if workspace is not None and stream is None and _quick is not None:  # (out and lse are looked at there)
        st = _quick.attend(q, kv_cache, page_table, lengths, scale, sinks, out, lse, slot_weights, slot_weights_in, flags, workspace)
        if st == KVC_OK:
            return out, lse
        if st is not None:
            raise KvcError(st, "kvc_attend")
    device, pages, form, R, columns, row = _cache(kv_cache, page_table, lengths)
    if not isinstance(q, torch.Tensor) or q.dtype != torch.bfloat16 or q.get_device() != device or q.dim() != 3:
        _refuse("q", q, torch.bfloat16, 3, device)
    shape = q.shape
    reqs, H, D = shape
    if D != HEAD_DIM or not 1 <= H <= 128:
        raise ValueError("q must be [num_reqs, 1..128 heads, 512]")
    if reqs != R:
        raise ValueError("q and page_table must have one row per request")
    by_req, by_head, by_dim = q.stride()
    if by_dim != 1:
        _refuse("q", q, torch.bfloat16, 3, device)
    if sinks is not None:
        _dense("sinks", sinks, torch.float32, device, (H,))
    S = weights_row = in_row = 0
    if slot_weights is not None:
        rows, S, weights_row = _rows("slot_weights", slot_weights, torch.float32, device)
        if rows != R:
            raise ValueError("slot_weights must have one row per request")
        if S == 0 and R != 0:
            raise ValueError("slot_weights must have at least one column")
    if slot_weights_in is not None:
        rows, cols, in_row = _rows("slot_weights_in", slot_weights_in, torch.float32, device)
        if slot_weights is None or (rows, cols) != (R, S):
            raise ValueError("slot_weights_in needs slot_weights of the same shape")
    if out is not None:
        _dense("out", out, torch.bfloat16, device, shape)
    if lse is not None:
        _dense("lse", lse, torch.float32, device, shape[:2])
    if workspace is not None:
        if not isinstance(workspace, torch.Tensor):
            _refuse("workspace", workspace, torch.uint8, 1, device)
        _dense("workspace", workspace, torch.uint8, device, (workspace.numel(),))
    if R != 0 and columns == 0:
        raise ValueError("page_table must have at least one column")

    def call(raw):
        nonlocal q, by_req, by_head, out, lse, workspace
        if H > 1 and by_head == 0:  # one query for all heads
            q = q.contiguous()
            by_req, by_head, _ = q.stride()
        if out is None:
            out = torch.empty((R, H, HEAD_DIM), dtype=torch.bfloat16, device=kv_cache.device)
        if lse is None:
            lse = torch.empty((R, H), dtype=torch.float32, device=kv_cache.device)
        if R == 0:
            return KVC_OK
        if workspace is None:
            workspace = torch.empty(kvc_attend_workspace_bytes(R, H, columns, slot_weights is not None),
                                    dtype=torch.uint8, device=kv_cache.device)
        return _entry().kvc_attend_format(
            q.data_ptr(), by_req, by_head, R, H, kv_cache.data_ptr(), form, pages,
            page_table.data_ptr(), columns, row, lengths.data_ptr(), HEAD_DIM ** -0.5 if scale is None else scale,
            None if sinks is None else sinks.data_ptr(), out.data_ptr(), lse.data_ptr(),
            None if slot_weights_in is None else slot_weights_in.data_ptr(), in_row,
            None if slot_weights is None else slot_weights.data_ptr(), weights_row, S,
            workspace.data_ptr(), workspace.numel(), flags, raw)

    st = _run(call, device, stream)
    if st != KVC_OK:
        raise KvcError(st, "kvc_attend")
    return out, lse


def join(outs, lses, *, out=None, lse=None, stream=None):
    """Join attention parts whose softmax ran over disjoint keys.

    outs: 1 to 8 contiguous [..., 512] tensors, all bf16 or all fp32, of one
    shape; lses: as many contiguous fp32 tensors of that shape without the 512
    (-inf: the part held no key for the row).  Returns (out, lse); `out` may
    be one of outs and `lse` one of lses.  No gradient is recorded.
    """
    torch = _torch or _load_torch()
    if not 1 <= len(outs) <= 8 or len(lses) != len(outs):
        raise ValueError("outs and lses need one entry per part, 1 to 8 parts")
    first = outs[0]
    if not isinstance(first, torch.Tensor) or not first.is_cuda:
        raise ValueError("outs must be CUDA tensors (there is no CPU path)")
    device, dtype, shape = first.get_device(), first.dtype, first.shape
    if dtype != torch.bfloat16 and dtype != torch.float32:
        raise TypeError("outs must have dtype torch.float32 or torch.bfloat16")
    if len(shape) < 1 or shape[-1] != HEAD_DIM:
        raise ValueError("outs must be [..., 512]")
    rows = shape[:-1]
    for o, x in zip(outs, lses):
        _dense("every part of outs", o, dtype, device, shape)
        _dense("every part of lses", x, torch.float32, device, rows)
    if out is not None:
        _dense("out", out, dtype, device, shape)
    if lse is not None:
        _dense("lse", lse, torch.float32, device, rows)

    def call(raw):
        nonlocal out, lse
        if out is None:
            out = torch.empty(shape, dtype=dtype, device=first.device)
        if lse is None:
            lse = torch.empty(rows, dtype=torch.float32, device=first.device)
        return kvc_join([t.data_ptr() for t in outs], [t.data_ptr() for t in lses], lse.numel(),
                        KVC_DTYPE_BF16 if dtype == torch.bfloat16 else KVC_DTYPE_F32, out.data_ptr(),
                        lse.data_ptr(), raw)

    st = _run(call, device, stream)
    if st != KVC_OK:
        raise KvcError(st, "kvc_join")
    return out, lse


def evict(kv_cache, page_table, lengths, slot_weights, keep, *, recent: int = 0, births=None,
          lengths_out=None, kept=None, slot_weights_out=None, births_out=None, stream=None,
          workspace=None):
    """Evict, in place, the slots that gathered the least attention.

    Of the first lengths[r] slots of request r (of either form, as for attend),
    min(keep, lengths[r]) stay:
    the `recent` newest by birth number (births int32 [R, S], needed if recent
    > 0), then those of largest slot_weights[r, n] (fp32 [R, S]), the lowest
    index first among equals, NaN last.  Slots that stay below the new length
    keep their places; the i-th place that falls free takes the i-th slot that
    stays from behind.  The slots' bytes move within kv_cache; no page may
    belong to two requests or stand twice in one's table.

    Returns (lengths_out int32 [R], kept int32 [R, keep]): the new lengths,
    and the former place of the slot at each place (-1 behind the new length).
    slot_weights_out and births_out, if given, receive those arrays in the new
    order; entries behind the new length are left as they were, so whoever adds a
    slot there sets its weight and birth anew.  lengths_out, slot_weights_out and
    births_out may be the inputs themselves.  A request whose length or pages are
    out of range stays as it is, its rows of these results too (undefined in
    results that the call allocates), and raises the device error word.
    """
    torch = _torch or _load_torch()
    device, pages, form, R, columns, row = _cache(kv_cache, page_table, lengths)
    keep, recent = int(keep), int(recent)
    if keep < 0 or not 0 <= recent <= keep:
        raise ValueError("keep must be >= 0 and recent between 0 and keep")
    rows, S, weights_row = _rows("slot_weights", slot_weights, torch.float32, device)
    if rows != R:
        raise ValueError("slot_weights must have one row per request")
    births_row = weights_out_row = births_out_row = 0
    if births is not None:
        rows, cols, births_row = _rows("births", births, torch.int32, device)
        if (rows, cols) != (R, S):
            raise ValueError("births must have the shape of slot_weights")
    elif recent > 0 or births_out is not None:
        raise ValueError("recent and births_out need births")
    if slot_weights_out is not None:
        rows, cols, weights_out_row = _rows("slot_weights_out", slot_weights_out, torch.float32, device)
        if rows != R or cols < min(keep, S):
            raise ValueError("slot_weights_out must be [num_reqs, at least min(keep, slots)]")
    if births_out is not None:
        rows, cols, births_out_row = _rows("births_out", births_out, torch.int32, device)
        if rows != R or cols < min(keep, S):
            raise ValueError("births_out must be [num_reqs, at least min(keep, slots)]")
    if lengths_out is not None:
        _dense("lengths_out", lengths_out, torch.int32, device, (R,))
    if kept is not None:
        _dense("kept", kept, torch.int32, device, (R, keep))
    if workspace is not None:
        if not isinstance(workspace, torch.Tensor):
            _refuse("workspace", workspace, torch.uint8, 1, device)
        _dense("workspace", workspace, torch.uint8, device, (workspace.numel(),))
    if R != 0 and columns == 0:
        raise ValueError("page_table must have at least one column")

    def call(raw):
        nonlocal lengths_out, kept, workspace
        if lengths_out is None:
            lengths_out = torch.empty((R,), dtype=torch.int32, device=kv_cache.device)
        if kept is None:
            kept = torch.empty((R, keep), dtype=torch.int32, device=kv_cache.device)
        if R == 0:
            return KVC_OK
        if workspace is None:
            workspace = torch.empty(kvc_evict_workspace_bytes(R, columns, keep), dtype=torch.uint8,
                                    device=kv_cache.device)
        return _entry().kvc_evict_format(
            kv_cache.data_ptr(), form, pages, page_table.data_ptr(), R, columns, row, lengths.data_ptr(),
            slot_weights.data_ptr(), weights_row, S, None if births is None else births.data_ptr(),
            births_row, keep, recent, lengths_out.data_ptr(), kept.data_ptr() if keep else None,
            None if slot_weights_out is None else slot_weights_out.data_ptr(), weights_out_row,
            None if births_out is None else births_out.data_ptr(), births_out_row,
            workspace.data_ptr(), workspace.numel(), raw)

    st = _run(call, device, stream)
    if st != KVC_OK:
        raise KvcError(st, "kvc_evict")
    return lengths_out, kept
