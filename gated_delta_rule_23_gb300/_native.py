"""Build and load the CUDA library (libkda.so) and expose its C ABI through ctypes.

The library is compiled in-tree with nvcc for sm_103a only.  Loading fails loudly
when the library is missing or cannot be built: there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os
import subprocess
import threading
from typing import List, Optional

_PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(_PKG)
CSRC = os.path.join(_PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(_PKG, "_build")
LIB_PATH = os.path.join(BUILD_DIR, "libkda.so")
UNITS = ["kda_api", "kda_prep", "kda_recur", "kda_recurrent", "kda_decode", "kda_host", "kda_noalloc", "kda_scan",
         "kda_step", "kda_append", "kda_attn", "kda_attn_tiles", "kda_attn_decode", "kda_beam", "kda_reorder",
         "kda_linear", "kda_linear_tokens", "kda_linear_chunks", "kda_verify"]
SOURCES = [os.path.join(CSRC, u + ".cu") for u in UNITS]
HEADERS = [os.path.join(INCLUDE, "kda.h"), os.path.join(CSRC, "kda_device.cuh"), os.path.join(CSRC, "kda_internal.h"),
           os.path.join(CSRC, "kda_plan.h"), os.path.join(CSRC, "kda_step.cuh"), os.path.join(CSRC, "kda_attn.cuh"),
           os.path.join(CSRC, "kda_linear.cuh"), os.path.join(CSRC, "kda_tc.cuh")]
BINDING_SOURCE = os.path.join(CSRC, "kda_binding.cpp")
BINDING_PATH = os.path.join(BUILD_DIR, "kda_binding.so")
ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]

_lock = threading.Lock()
_lib: Optional[ctypes.CDLL] = None


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _stale() -> bool:
    if not os.path.exists(LIB_PATH) or not os.path.exists(BINDING_PATH):
        return True
    t = min(os.path.getmtime(LIB_PATH), os.path.getmtime(BINDING_PATH))
    return any(os.path.getmtime(s) > t for s in SOURCES + HEADERS + [BINDING_SOURCE])


def _binding_command(out: str) -> List[str]:
    """The host compiler's command for csrc/kda_binding.cpp, a Python module over torch's C++ tensors."""
    import sysconfig

    import torch
    t = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc())) or "/usr/local/cuda"
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
            "-I" + INCLUDE, "-I" + os.path.join(t, "include"),
            "-I" + os.path.join(t, "include", "torch", "csrc", "api", "include"),
            "-I" + sysconfig.get_paths()["include"], "-I" + os.path.join(cuda, "include"), "-o", out, BINDING_SOURCE,
            "-L" + os.path.join(t, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"]


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile csrc/*.cu (sm_103a, -O3, -lineinfo), one process per unit, and link _build/libkda.so; compile the
    decoder-step operators' Python module (csrc/kda_binding.cpp) beside it."""
    with _lock:
        if not force and not _stale():
            return LIB_PATH
        os.makedirs(BUILD_DIR, exist_ok=True)
        tag = f".tmp{os.getpid()}"
        common = [nvcc(), *ARCH_FLAGS, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I" + INCLUDE]
        if verbose:
            common.append("-Xptxas=-v")
        objs, procs = [], []
        for u, src in zip(UNITS, SOURCES):
            obj = os.path.join(BUILD_DIR, u + tag + ".o")
            objs.append(obj)
            procs.append(subprocess.Popen(common + ["-c", "-o", obj, src]))
        binding = BINDING_PATH + tag
        procs.append(subprocess.Popen(_binding_command(binding)))
        codes = [pr.wait() for pr in procs]
        try:
            for src, rc in zip(SOURCES + [BINDING_SOURCE], codes):
                if rc != 0:
                    raise subprocess.CalledProcessError(rc, f"compiling {src}")
            tmp = LIB_PATH + tag
            subprocess.run([nvcc(), *ARCH_FLAGS, "-shared", "-o", tmp, *objs], check=True)
            os.replace(tmp, LIB_PATH)
            os.replace(binding, BINDING_PATH)
        finally:
            for o in objs + [binding]:
                if os.path.exists(o):
                    os.remove(o)
        return LIB_PATH


def load() -> ctypes.CDLL:
    """Load libkda.so (building it first if it is missing or older than its sources)."""
    global _lib
    if _lib is None:
        path = build()
        lib = ctypes.CDLL(path)
        P, I, I64, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float
        lib.kda_fwd.argtypes = [P, P, P, P, P, F, P, P, P, F, P, P, I, P, I, I64, I, P]
        lib.kda_fwd.restype = I
        lib.kda_fwd_noalloc.argtypes = [P, P, P, P, P, F, P, P, P, F, P, P, I, P, I, I64, I, P]
        lib.kda_fwd_noalloc.restype = I
        lib.kda_fwd_recurrent.argtypes = [P, P, P, P, P, F, P, P, P, F, P, P, I, P, I, I64, I, P]
        lib.kda_fwd_recurrent.restype = I
        lib.kda_fwd_host.argtypes = [P, P, P, P, P, F, P, P, P, F, P, P, I, P, I, I64, I]
        lib.kda_fwd_host.restype = I
        lib.kda_fwd_host_plan.argtypes = [I, I64, P, P, P, P, P, I]
        lib.kda_fwd_host_plan.restype = I
        lib.kda_fwd_ws.argtypes = [P, P, P, P, P, F, P, P, P, F, P, P, I, P, I, I64, I, P, ctypes.c_size_t, P]
        lib.kda_fwd_ws.restype = I
        lib.kda_fwd_ws_profiled.argtypes = [P, P, P, P, P, F, P, P, P, F, P, P, I, P, I, I64, I, P, ctypes.c_size_t,
                                             P, P]
        lib.kda_fwd_ws_profiled.restype = I
        lib.kda_fwd_ws_variant.argtypes = [P, P, P, P, P, F, P, P, P, F, P, P, I, P, I, I64, I, P, ctypes.c_size_t,
                                           ctypes.c_uint, P]
        lib.kda_fwd_ws_variant.restype = I
        lib.kda_fwd_workspace_size.argtypes = [I, I64, I, I]
        lib.kda_fwd_workspace_size.restype = ctypes.c_size_t
        lib.kda_fwd_pieces.argtypes = [I, I64, I, I]
        lib.kda_fwd_pieces.restype = I
        lib.kda_fwd_scan_groups.argtypes = [I, I64, I, I]
        lib.kda_fwd_scan_groups.restype = I
        lib.kda_workspace_trim.argtypes = []
        lib.kda_workspace_trim.restype = I
        lib.kda_check_cu_seqlens.argtypes = [P, I, I64]
        lib.kda_check_cu_seqlens.restype = I
        lib.kda_status_string.argtypes = [I]
        lib.kda_status_string.restype = ctypes.c_char_p
        lib.kda_device_status.argtypes = [P]
        lib.kda_device_status.restype = I
        lib.kda_set_wait_limit.argtypes = [ctypes.c_uint32]
        lib.kda_set_wait_limit.restype = None
        lib.kda_fwd_smem_bytes.argtypes = []
        lib.kda_fwd_smem_bytes.restype = ctypes.c_size_t
        Z = ctypes.c_size_t
        cache = [P, I, I64, I, I, I, I64, I, I]      # cu_seqlens, N, T, Hq, Hkv, D, pages, page, max_pages
        lib.kda_kv_append.argtypes = [P, I64, P, I64, P, P, P, P, P, P, I, I64, I, P, I64, P] + cache + [P]
        lib.kda_kv_append.restype = I
        attn = [P, I64, P, P, P, P, P, P, F, I, I] + cache
        lib.kda_window_attn.argtypes = attn + [P]
        lib.kda_window_attn.restype = I
        lib.kda_window_attn_ws.argtypes = attn + [P, Z, P]
        lib.kda_window_attn_ws.restype = I
        lib.kda_window_attn_workspace_size.argtypes = [I, I, I, I, I64, I, I, I, I, I]
        lib.kda_window_attn_workspace_size.restype = Z
        beam = [P, I, I64, P, P, I, P, P, P, I, I, I, I]
        lib.kda_beam_select.argtypes = beam + [P]
        lib.kda_beam_select.restype = I
        lib.kda_beam_select_ws.argtypes = beam + [P, Z, P]
        lib.kda_beam_select_ws.restype = I
        lib.kda_beam_select_workspace_size.argtypes = [I, I, I, I]
        lib.kda_beam_select_workspace_size.restype = Z
        lib.kda_state_reorder.argtypes = [P, P, P, I, P, I, I, P]
        lib.kda_state_reorder.restype = I
        linear = [P, I64, P, I64, P, I64, P, P, F, P, P, P, I, P, P, I, I64, I, I, I]
        lib.kda_linear_attn.argtypes = linear + [P]
        lib.kda_linear_attn.restype = I
        lib.kda_linear_attn_ws.argtypes = linear + [P, Z, P]
        lib.kda_linear_attn_ws.restype = I
        lib.kda_linear_attn_workspace_size.argtypes = [I, I, I64, I, I]
        lib.kda_linear_attn_workspace_size.restype = Z
        verify = [P, I, I64, P, P, P, P, P, P, P, P, I, I, I]
        lib.kda_verify_drafts.argtypes = verify + [P]
        lib.kda_verify_drafts.restype = I
        lib.kda_verify_drafts_ws.argtypes = verify + [P, Z, P]
        lib.kda_verify_drafts_ws.restype = I
        lib.kda_verify_drafts_opt.argtypes = verify + [ctypes.c_uint32, P, Z, P]
        lib.kda_verify_drafts_opt.restype = I
        lib.kda_verify_drafts_workspace_size.argtypes = [I, I, I, I]
        lib.kda_verify_drafts_workspace_size.restype = Z
        _lib = lib
    return _lib


_binding = None


def binding():
    """The module kda_binding (csrc/kda_binding.cpp), bound to libkda.so."""
    global _binding
    if _binding is None:
        import importlib.util
        lib = load()
        spec = importlib.util.spec_from_file_location("kda_binding", BINDING_PATH)
        mod = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(mod)
        mod.bind(*(ctypes.cast(getattr(lib, f), ctypes.c_void_p).value
                   for f in ("kda_kv_append", "kda_window_attn", "kda_window_attn_ws", "kda_beam_select",
                             "kda_beam_select_ws", "kda_state_reorder", "kda_linear_attn", "kda_linear_attn_ws",
                             "kda_verify_drafts_opt")))
        _binding = mod
    return _binding


def declared_functions() -> List[str]:
    """Names of the functions include/kda.h declares (for export checks)."""
    import re
    text = open(HEADERS[0]).read()
    return sorted(set(re.findall(r"^\s*(?:const\s+)?[a-z_0-9]+\s*\*?\s*(kda_[a-z_0-9]+)\s*\(", text, re.M)))


KDA_DEFAULT_WAIT_POLLS = 16777216
KDA_VARIANT_BF16_STATE, KDA_VARIANT_NEUMANN_INVERSE = 1, 2
# status codes, as in include/kda.h
KDA_OK, KDA_ERR_INVALID_ARGUMENT, KDA_ERR_UNSUPPORTED, KDA_ERR_CUDA, KDA_ERR_TIMEOUT, KDA_ERR_NONFINITE = range(6)
KDA_DTYPE_NONE, KDA_DTYPE_BF16, KDA_DTYPE_FP32 = range(3)
KDA_VERIFY_FIRST_LARGEST = 1


class KDAError(RuntimeError):
    def __init__(self, status: int):
        self.status = status
        super().__init__(f"kda: {load().kda_status_string(status).decode()} (status {status})")
