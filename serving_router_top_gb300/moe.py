"""ctypes binding of libmoe (``include/moe.h``): same names, argument marshalling only.

Every step of the layer runs in the library's CUDA kernels; this module only
turns torch tensors into device pointers and streams into handles.  If the
library has not been built (``python -m serving_router_top_gb300.build``) the
first call raises -- there is no fallback.
"""
from __future__ import annotations

import ctypes as C
import functools
import os
from typing import Optional

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "lib", "libmoe.so")

MOE_OK, MOE_EINVAL, MOE_ENOMEM, MOE_ECUDA, MOE_EMISSING, MOE_ERANGE, MOE_ENAN, MOE_ETIMEOUT = range(8)
MOE_SRC_MISSING, MOE_SRC_RESIDENT, MOE_SRC_STAGED, MOE_SRC_SKIPPED = -1, 0, 1, 2
MOE_MODE_AUTO, MOE_MODE_DECODE, MOE_MODE_PREFILL = 0, 1, 2
MOE_DECODE_FUSED, MOE_DECODE_CHAIN = 0, 1

# Every symbol include/moe.h declares.
EXPORTED = (
    "moe_blob_bytes", "moe_pack_expert", "moe_cache_create", "moe_cache_destroy", "moe_cache_admit",
    "moe_cache_fill", "moe_cache_get_view", "moe_get_stats", "moe_ws_create", "moe_ws_destroy", "moe_ws_get_view",
    "moe_sync_status", "moe_strerror", "moe_route", "moe_group", "moe_layer_forward", "cache_heat_update",
    "cache_plan_swaps", "moe_cache_apply_swaps", "moe_ws_set_profiling", "moe_ws_kernel_times",
    "cache_plan_swaps_noalloc", "moe_residual_rmsnorm", "moe_layer_forward_streamed", "moe_ws_set_tail_skip",
    "moe_ws_set_fused_heat", "cache_lru_plan", "moe_cache_apply_lru", "moe_ws_set_decode_path",
    "moe_ws_set_wait_test", "moe_nvfp4_split", "moe_layers_forward_streamed", "moe_rope_create", "moe_rope_destroy",
    "moe_kv_append", "moe_attn_ws_create", "moe_attn_ws_destroy", "moe_attn_ws_get_view", "moe_attn_sync_status",
    "moe_paged_attention", "moe_block_norm", "moe_attn_ws_set_wait_test", "moe_tree_prepare", "moe_kv_append_norm",
    "moe_tree_attention", "moe_verify_drafts", "moe_kv_compact", "moe_kv_copy_pages",
)


class MoeError(RuntimeError):
    def __init__(self, code: int, what: str = ""):
        self.code = code
        super().__init__(f"{what}: {strerror(code)} ({code})" if what else f"{strerror(code)} ({code})")


class moe_layer_shape(C.Structure):
    _fields_ = [("H", C.c_int), ("I", C.c_int), ("E", C.c_int), ("k", C.c_int), ("I_shared", C.c_int)]


class moe_layer_desc(C.Structure):
    _fields_ = [("w_router", C.c_void_p), ("bias", C.c_void_p), ("w_shared_gate", C.c_void_p),
                ("shared_blob", C.c_void_p), ("layer", C.c_int), ("s", moe_layer_shape)]


class moe_cache_view(C.Structure):
    _fields_ = [("resid", C.c_void_p), ("stage", C.c_void_p), ("heat", C.c_void_p), ("slot_owner", C.c_void_p),
                ("slots", C.c_void_p), ("staging", C.c_void_p), ("blob_bytes", C.c_size_t), ("L", C.c_int),
                ("E", C.c_int), ("nslots", C.c_int), ("nstaging", C.c_int), ("lru_tick", C.c_void_p),
                ("lru_clock", C.c_void_p)]


class moe_ws_view(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("num_groups", "grp_expert", "grp_off", "grp_slot", "grp_src", "ent_tok",
                                           "ent_pos", "logits", "topk_ids", "topk_w", "error")]


class moe_swap(C.Structure):
    _fields_ = [("layer", C.c_int), ("hot_expert", C.c_int), ("cold_expert", C.c_int), ("slot", C.c_int),
                ("diff", C.c_float)]


class moe_policy_cfg(C.Structure):
    _fields_ = [("threshold", C.c_float), ("max_swaps", C.c_int), ("decay", C.c_float)]


class moe_kv_pages(C.Structure):
    _fields_ = [("k", C.c_void_p), ("v", C.c_void_p), ("e4m3", C.c_int), ("Hkv", C.c_int), ("D", C.c_int),
                ("page", C.c_int), ("npages", C.c_int), ("page_stride", C.c_longlong), ("head_stride", C.c_longlong),
                ("tok_stride", C.c_longlong), ("k_scale", C.c_void_p), ("v_scale", C.c_void_p)]


class moe_kv_batch(C.Structure):
    _fields_ = [("q_start", C.c_void_p), ("kv_len", C.c_void_p), ("page_table", C.c_void_p), ("B", C.c_int),
                ("T", C.c_int), ("max_n", C.c_int), ("table_stride", C.c_int)]


class moe_attn_ws_view(C.Structure):
    _fields_ = [("error", C.c_void_p)]


class moe_tree(C.Structure):
    _fields_ = [("parent", C.c_void_p), ("depth", C.c_void_p), ("above", C.c_void_p), ("below", C.c_void_p),
                ("words", C.c_int)]


class moe_head_norm(C.Structure):
    _fields_ = [("w_q", C.c_void_p), ("w_k", C.c_void_p), ("eps", C.c_float)]


class moe_verify_desc(C.Structure):
    _fields_ = [("target", C.c_void_p), ("target_stride", C.c_longlong), ("draft", C.c_void_p),
                ("draft_stride", C.c_longlong), ("token", C.c_void_p), ("parent", C.c_void_p), ("u", C.c_void_p),
                ("u_last", C.c_void_p), ("V", C.c_int)]


class moe_block_norm_desc(C.Structure):
    _fields_ = [("y", C.c_void_p), ("y_stride", C.c_longlong), ("post_norm", C.c_int), ("w_post", C.c_void_p),
                ("gate", C.c_void_p), ("gate_stride", C.c_longlong), ("gate_sigmoid", C.c_int),
                ("res_scale", C.c_float), ("w_pre", C.c_void_p), ("eps", C.c_float)]


SWAP_DTYPE = np.dtype([("layer", "<i4"), ("hot_expert", "<i4"), ("cold_expert", "<i4"), ("slot", "<i4"),
                       ("diff", "<f4")])

_lib = None


def load() -> C.CDLL:
    """Load libmoe.so (raises if it was not built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"libmoe.so not built ({LIB_PATH}); run python -m serving_router_top_gb300.build")
    lib = C.CDLL(LIB_PATH)
    P, I, Z, F, Q, D = C.c_void_p, C.c_int, C.c_size_t, C.c_float, C.c_longlong, C.c_double
    sig = {
        "moe_blob_bytes": (Z, [I, I]),
        "moe_pack_expert": (I, [P, P, P, I, I, F, F, F, P]),
        "moe_cache_create": (I, [C.POINTER(P), I, I, I, I, I, I, P, I]),
        "moe_cache_destroy": (I, [P]),
        "moe_cache_admit": (I, [P, I, I, C.POINTER(C.c_int32)]),
        "moe_cache_fill": (I, [P, P, I]),
        "moe_cache_get_view": (I, [P, C.POINTER(moe_cache_view)]),
        "moe_get_stats": (I, [P, P]),
        "moe_ws_create": (I, [C.POINTER(P), I, moe_layer_shape]),
        "moe_ws_destroy": (I, [P]),
        "moe_ws_get_view": (I, [P, C.POINTER(moe_ws_view)]),
        "moe_sync_status": (I, [P, P]),
        "moe_strerror": (C.c_char_p, [I]),
        "moe_route": (I, [P, P, P, P, I, I, I, I, P, P, P, P]),
        "moe_group": (I, [P, I, I, I, I, P, P, P]),
        "moe_layer_forward": (I, [C.POINTER(moe_layer_desc), P, P, I, I, P, P, I, P]),
        "moe_layer_forward_streamed": (I, [C.POINTER(moe_layer_desc), P, P, I, I, P, P, I, I, P, P]),
        "cache_heat_update": (I, [P, P, I, I, I, P, P]),
        "cache_plan_swaps": (I, [P, C.POINTER(moe_policy_cfg), P, P, P]),
        "cache_plan_swaps_noalloc": (I, [P, P, I, I, C.POINTER(moe_policy_cfg), P, P, P]),
        "moe_residual_rmsnorm": (I, [P, P, P, I, I, F, P]),
        "moe_cache_apply_swaps": (I, [P, P, P, P, P]),
        "moe_ws_set_profiling": (I, [P, I]),
        "moe_ws_set_tail_skip": (I, [P, I]),
        "moe_ws_set_fused_heat": (I, [P, I]),
        "moe_ws_set_decode_path": (I, [P, I]),
        "moe_ws_set_wait_test": (I, [P, C.c_ulonglong, I]),
        "moe_nvfp4_split": (I, [P, I, I, I, I, I, P, P, P, P]),
        "moe_layers_forward_streamed": (I, [P, I, P, P, P, I, P, P, I, F, P, P]),
        "cache_lru_plan": (I, [P, P, I, I, P, P, P]),
        "moe_cache_apply_lru": (I, [P, P, P, P, P]),
        "moe_ws_kernel_times": (I, [P, I, P, P, C.POINTER(C.c_int)]),
        "moe_rope_create": (I, [C.POINTER(P), I, I, D, P]),
        "moe_rope_destroy": (I, [P]),
        "moe_kv_append": (I, [P, P, P, P, Q, P, Q, I, P, Q, P, Q, P, P]),
        "moe_attn_ws_create": (I, [C.POINTER(P), I, I, I]),
        "moe_attn_ws_destroy": (I, [P]),
        "moe_attn_ws_get_view": (I, [P, C.POINTER(moe_attn_ws_view)]),
        "moe_attn_sync_status": (I, [P, P]),
        "moe_attn_ws_set_wait_test": (I, [P, I]),
        "moe_paged_attention": (I, [P, P, P, Q, I, P, Q, F, I, P, P]),
        "moe_block_norm": (I, [P, P, Q, P, Q, P, Q, I, I, P]),
        "moe_tree_prepare": (I, [P, P, P, P]),
        "moe_kv_append_norm": (I, [P, P, P, P, P, P, Q, P, Q, I, P, Q, P, Q, P, P]),
        "moe_tree_attention": (I, [P, P, P, P, Q, I, P, Q, F, I, P, P]),
        "moe_verify_drafts": (I, [P, P, P, I, P, P, P, P]),
        "moe_kv_compact": (I, [P, I, P, P, I, P, P, P, P]),
        "moe_kv_copy_pages": (I, [P, I, P, P, P, I, P, P]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def strerror(code: int) -> str:
    try:
        return load().moe_strerror(int(code)).decode()
    except RuntimeError:
        return f"error {code}"


def _check(rc: int, what: str) -> None:
    if rc != MOE_OK:
        raise MoeError(rc, what)


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


_raw_stream = _device = None  # device index -> the handle of its current stream; the current device


def _find_stream() -> None:
    global _raw_stream, _device
    import torch
    torch.cuda.current_device()  # sets CUDA up
    _device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    # torch.cuda.current_stream() builds a Stream object, 3 us a call on a Grace core
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda device: torch.cuda.current_stream(device).cuda_stream)


def _stream(stream) -> Optional[int]:
    if stream is not None:
        return stream.cuda_stream or None
    if _raw_stream is None:
        _find_stream()
    return _raw_stream(_device()) or None


class _CudaArray:
    """Minimal __cuda_array_interface__ holder so torch can view library-owned memory."""

    def __init__(self, ptr: int, shape, typestr: str, owner):
        self.__cuda_array_interface__ = {"shape": tuple(shape), "typestr": typestr, "data": (ptr, False),
                                         "version": 3, "strides": None}
        self._owner = owner


def device_view(ptr: int, shape, dtype: str, owner=None):
    """A torch tensor aliasing library device memory (no copy)."""
    import torch
    typestr = {"int32": "<i4", "float32": "<f4", "uint8": "|u1"}[dtype]
    return torch.as_tensor(_CudaArray(ptr, shape, typestr, owner), device="cuda")


# ------------------------------------------------------------------ blobs

def moe_blob_bytes(H: int, I: int) -> int:
    return int(load().moe_blob_bytes(H, I))


def moe_pack_expert(gate_rows: np.ndarray, up_rows: np.ndarray, down_rows: np.ndarray, H: int, I: int,
                    gscale=(1.0, 1.0, 1.0), out: Optional[np.ndarray] = None) -> np.ndarray:
    """Canonical packed rows (host numpy uint8) -> one slot blob (host numpy uint8)."""
    nb = moe_blob_bytes(H, I)
    if out is None:
        out = np.empty(nb, dtype=np.uint8)
    g, u, d = (np.ascontiguousarray(a, dtype=np.uint8) for a in (gate_rows, up_rows, down_rows))
    _check(load().moe_pack_expert(g.ctypes.data, u.ctypes.data, d.ctypes.data, H, I, float(gscale[0]),
                                  float(gscale[1]), float(gscale[2]), out.ctypes.data), "moe_pack_expert")
    return out


# ------------------------------------------------------------------ cache

class Cache:
    """Owner of a moe_cache handle and (a reference to) its backing store tensor."""

    def __init__(self, L: int, E: int, H: int, I: int, nslots: int, nstaging: int, backing, backing_on_device: bool):
        h = C.c_void_p()
        _check(load().moe_cache_create(C.byref(h), L, E, H, I, nslots, nstaging, _ptr(backing),
                                       1 if backing_on_device else 0), "moe_cache_create")
        self.handle = h
        self.backing = backing
        self.L, self.E, self.H, self.I, self.nslots, self.nstaging = L, E, H, I, nslots, nstaging
        v = moe_cache_view()
        _check(load().moe_cache_get_view(h, C.byref(v)), "moe_cache_get_view")
        self.view = v

    def close(self):
        if self.handle:
            load().moe_cache_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def admit(self, layer: int, expert: int) -> int:
        s = C.c_int32()
        _check(load().moe_cache_admit(self.handle, layer, expert, C.byref(s)), "moe_cache_admit")
        return int(s.value)

    def fill(self, mask: np.ndarray, staging: bool = False) -> None:
        m = np.ascontiguousarray(mask, dtype=np.uint8).ravel()
        assert m.size == self.L * self.E
        _check(load().moe_cache_fill(self.handle, m.ctypes.data, 1 if staging else 0), "moe_cache_fill")

    def tables(self):
        """Torch views of resid, stage, heat (device, aliasing the library's memory)."""
        LE = self.L * self.E
        return (device_view(self.view.resid, (LE,), "int32", self), device_view(self.view.stage, (LE,), "int32", self),
                device_view(self.view.heat, (LE,), "float32", self))

    def lru_tables(self):
        """Torch views of the global LRU's slot ticks (uint32 as int32 [nslots]) and clock (int32 [1])."""
        return (device_view(self.view.lru_tick, (max(1, self.view.nslots),), "int32", self),
                device_view(self.view.lru_clock, (1,), "int32", self))

    def stats(self) -> np.ndarray:
        """int64 [L, 5]: groups looked up, resident hits, staged, missing, skipped by the tail skip."""
        out = np.zeros((self.L, 5), dtype=np.int64)
        _check(load().moe_get_stats(self.handle, out.ctypes.data), "moe_get_stats")
        return out


# -------------------------------------------------------------- workspace

class Workspace:
    def __init__(self, maxT: int, H: int, I: int, E: int, k: int, I_shared: int):
        h = C.c_void_p()
        self.shape = moe_layer_shape(H, I, E, k, I_shared)
        _check(load().moe_ws_create(C.byref(h), maxT, self.shape), "moe_ws_create")
        self.handle = h
        self.maxT = maxT
        v = moe_ws_view()
        _check(load().moe_ws_get_view(h, C.byref(v)), "moe_ws_get_view")
        self.view = v

    def close(self):
        if self.handle:
            load().moe_ws_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def groups(self, T: int):
        """Copy the last grouping to host numpy: (experts, off, slot, src, ent_tok, ent_pos)."""
        import torch
        torch.cuda.synchronize()
        k = self.shape.k
        G = int(device_view(self.view.num_groups, (1,), "int32", self).cpu()[0])
        n = T * k
        get = lambda p, m: device_view(p, (m,), "int32", self).cpu().numpy().copy()
        return (get(self.view.grp_expert, G), get(self.view.grp_off, G + 1), get(self.view.grp_slot, G),
                get(self.view.grp_src, G), get(self.view.ent_tok, n), get(self.view.ent_pos, n))

    def routing(self, T: int):
        """(logits [T,E], ids [T,k], w [T,k]) of the last forward (device tensors)."""
        E, k = self.shape.E, self.shape.k
        return (device_view(self.view.logits, (T, E), "float32", self),
                device_view(self.view.topk_ids, (T, k), "int32", self),
                device_view(self.view.topk_w, (T, k), "float32", self))

    def set_tail_skip(self, min_rank: int) -> None:
        """Drop non-resident experts that every choosing token ranks at or past min_rank (0: off)."""
        _check(load().moe_ws_set_tail_skip(self.handle, int(min_rank)), "moe_ws_set_tail_skip")

    def set_fused_heat(self, enable: bool) -> None:
        """Let the grouping of later calls with a cache also add the window's counts to the layer's heat."""
        _check(load().moe_ws_set_fused_heat(self.handle, 1 if enable else 0), "moe_ws_set_fused_heat")

    def set_decode_path(self, path: int) -> None:
        """MOE_DECODE_FUSED (one cooperative kernel where the shapes fit) or MOE_DECODE_CHAIN."""
        _check(load().moe_ws_set_decode_path(self.handle, int(path)), "moe_ws_set_decode_path")

    def set_wait_test(self, wait_ns: int, phantom_arrivals: int) -> None:
        """Bound of the decode kernel's grid-barrier waits, and arrivals they wait for that never come."""
        _check(load().moe_ws_set_wait_test(self.handle, int(wait_ns), int(phantom_arrivals)), "moe_ws_set_wait_test")

    def set_profiling(self, enable: bool) -> None:
        _check(load().moe_ws_set_profiling(self.handle, 1 if enable else 0), "moe_ws_set_profiling")

    def kernel_times(self):
        """[(name, ms)] of the kernels of the most recent call (profiling must be on)."""
        ms = (C.c_float * 16)()
        names = (C.c_char_p * 16)()
        n = C.c_int()
        _check(load().moe_ws_kernel_times(self.handle, 16, ms, names, C.byref(n)), "moe_ws_kernel_times")
        return [(names[i].decode(), float(ms[i])) for i in range(n.value)]

    @property
    def error_ptr(self) -> int:
        return self.view.error


# ------------------------------------------------------------- hot path

def moe_sync_status(ws: Workspace, stream=None) -> int:
    return int(load().moe_sync_status(ws.handle, _stream(stream)))


def moe_route(x, w_router, bias, logits_io, T: int, H: int, E: int, k: int, topk_ids, topk_w, err=None,
              stream=None) -> None:
    _check(load().moe_route(_ptr(x), _ptr(w_router), _ptr(bias), _ptr(logits_io), T, H, E, k, _ptr(topk_ids),
                            _ptr(topk_w), _ptr(err), _stream(stream)), "moe_route")


def moe_group(topk_ids, T: int, k: int, E: int, layer: int, cache: Cache, ws: Workspace, stream=None) -> None:
    _check(load().moe_group(_ptr(topk_ids), T, k, E, layer, cache.handle, ws.handle, _stream(stream)), "moe_group")


def layer_desc(w_router, bias, w_shared_gate, shared_blob, layer: int, H: int, I: int, E: int, k: int,
               I_shared: int) -> moe_layer_desc:
    return moe_layer_desc(_ptr(w_router), _ptr(bias), _ptr(w_shared_gate), _ptr(shared_blob), layer,
                          moe_layer_shape(H, I, E, k, I_shared))


def moe_layer_forward(desc: moe_layer_desc, x, y, y_is_fp32: bool, T: int, cache: Cache, ws: Workspace,
                      mode: int = MOE_MODE_AUTO, stream=None) -> None:
    _check(load().moe_layer_forward(C.byref(desc), _ptr(x), _ptr(y), 1 if y_is_fp32 else 0, T, cache.handle,
                                    ws.handle, mode, _stream(stream)), "moe_layer_forward")


def moe_layer_forward_streamed(desc: moe_layer_desc, x, y, y_is_fp32: bool, T: int, cache: Cache, ws: Workspace,
                               U: int, stream=None, copy_stream=None, buffers: int = 2) -> None:
    _check(load().moe_layer_forward_streamed(C.byref(desc), _ptr(x), _ptr(y), 1 if y_is_fp32 else 0, T, cache.handle,
                                             ws.handle, U, buffers, _stream(stream), _stream(copy_stream)),
           "moe_layer_forward_streamed")


def moe_layers_forward_streamed(descs, x_res, xn, y, T: int, cache: Cache, ws: Workspace, buffers: int = 2,
                                eps: float = 1e-6, stream=None, copy_stream=None) -> None:
    """Layers of a prefill chunk on a residual stream, each layer's experts streamed one layer ahead."""
    arr = (moe_layer_desc * len(descs))(*descs)
    _check(load().moe_layers_forward_streamed(arr, len(descs), _ptr(x_res), _ptr(xn), _ptr(y), T, cache.handle,
                                              ws.handle, buffers, eps, _stream(stream), _stream(copy_stream)),
           "moe_layers_forward_streamed")


def moe_nvfp4_split(src, src_is_fp32: bool, rows: int, K: int, ld: int, R: int, codes, scales, gscale,
                    stream=None) -> None:
    """Rows of activations -> R NVFP4 terms each (codes, block scales, global scales)."""
    _check(load().moe_nvfp4_split(_ptr(src), 1 if src_is_fp32 else 0, rows, K, ld, R, _ptr(codes), _ptr(scales),
                                  _ptr(gscale), _stream(stream)), "moe_nvfp4_split")


def cache_heat_update(cache: Cache, topk_ids, T: int, k: int, layer: int, err=None, stream=None) -> None:
    _check(load().cache_heat_update(cache.handle, _ptr(topk_ids), T, k, layer, _ptr(err), _stream(stream)),
           "cache_heat_update")


def cache_plan_swaps(cache: Cache, threshold: float, max_swaps: int, decay: float, plan_dev, n_dev,
                     stream=None) -> None:
    cfg = moe_policy_cfg(threshold, max_swaps, decay)
    _check(load().cache_plan_swaps(cache.handle, C.byref(cfg), _ptr(plan_dev), _ptr(n_dev), _stream(stream)),
           "cache_plan_swaps")


def moe_residual_rmsnorm(x_res, y_prev, xn_out, T: int, H: int, eps: float = 1e-6, stream=None) -> None:
    """x_res (fp32 [T,H]) += y_prev (bf16 bits, or None); xn_out (bf16 bits) = RMSNorm(x_res)."""
    _check(load().moe_residual_rmsnorm(_ptr(x_res), _ptr(y_prev), _ptr(xn_out), T, H, eps, _stream(stream)),
           "moe_residual_rmsnorm")


# Capacity of the static scratch behind cache_plan_swaps_noalloc.
NOALLOC_MAX_L, NOALLOC_MAX_E, NOALLOC_MAX_LE, NOALLOC_MAX_KEYS = 1024, 1024, 32768, 16384


def cache_plan_swaps_noalloc(heat_dev, resid_dev, L: int, E: int, threshold: float, max_swaps: int, decay: float,
                             plan_dev, n_dev, stream=None) -> None:
    """Swap planning on caller-owned heat [L, E] (decayed in place) and residency [L, E] tables; allocates nothing."""
    if not (1 <= L <= NOALLOC_MAX_L and 1 <= E <= NOALLOC_MAX_E and L * E <= NOALLOC_MAX_LE
            and L * ((E + 1) // 2) <= NOALLOC_MAX_KEYS):
        raise ValueError(f"cache_plan_swaps_noalloc: L={L}, E={E} exceed the static scratch (L <= {NOALLOC_MAX_L}, "
                         f"E <= {NOALLOC_MAX_E}, L*E <= {NOALLOC_MAX_LE}, L*ceil(E/2) <= {NOALLOC_MAX_KEYS})")
    cfg = moe_policy_cfg(threshold, max_swaps, decay)
    _check(load().cache_plan_swaps_noalloc(_ptr(heat_dev), _ptr(resid_dev), L, E, C.byref(cfg), _ptr(plan_dev),
                                           _ptr(n_dev), _stream(stream)), "cache_plan_swaps_noalloc")


def cache_lru_plan(cache: Cache, ws: Workspace, layer: int, K: int, plan_dev, n_dev, stream=None) -> None:
    """After a layer call's grouping on ws: refresh its hits, plan its admissions into the K LRU victims."""
    _check(load().cache_lru_plan(cache.handle, ws.handle, layer, K, _ptr(plan_dev), _ptr(n_dev), _stream(stream)),
           "cache_lru_plan")


def moe_cache_apply_lru(cache: Cache, plan_dev, n_dev, compute=None, copy=None) -> None:
    _check(load().moe_cache_apply_lru(cache.handle, _ptr(plan_dev), _ptr(n_dev), _stream(compute), _stream(copy)),
           "moe_cache_apply_lru")


def moe_cache_apply_swaps(cache: Cache, plan_dev, n_dev, compute=None, copy=None) -> None:
    _check(load().moe_cache_apply_swaps(cache.handle, _ptr(plan_dev), _ptr(n_dev), _stream(compute),
                                        _stream(copy)), "moe_cache_apply_swaps")


# ------------------------------------------------- the attention half of a layer

@functools.cache
def _row_types():
    """The types of row arguments: fp32; bf16, or its bits as integers."""
    import torch
    return (torch.float32,), (torch.bfloat16, torch.int16, torch.uint16)


def _on_gpu(*tensors) -> bool:
    return all(t is None or t.is_cuda for t in tensors)


_ELSEWHERE = "the attention half's kernels read and write GPU tensors; an argument is on another device"


class KvPages:
    """A layer's key and value page pools: torch tensors [npages, Hkv, page, D], bf16 (or their
    bits as int16) or float8_e4m3fn with the scales of each head (fp32 [Hkv]); any strides with
    contiguous columns, the same in both."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        import torch
        if k.dim() != 4 or k.shape != v.shape or k.stride() != v.stride() or k.dtype != v.dtype or k.stride(3) != 1:
            raise ValueError("KvPages: k and v are [npages, Hkv, page, D] of one shape, type and layout, columns contiguous")
        if k.dtype not in (torch.bfloat16, torch.int16, torch.float8_e4m3fn):
            raise ValueError(f"KvPages: bf16 or float8_e4m3fn pools, not {k.dtype}")
        for t in (k_scale, v_scale):
            if t is not None and (t.dtype != torch.float32 or t.numel() != k.shape[1] or not t.is_contiguous()):
                raise ValueError("KvPages: the scales are contiguous float32 [Hkv]")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        npages, self.Hkv, page, self.D = k.shape
        self.c = moe_kv_pages(k.data_ptr(), v.data_ptr(), 1 if k.dtype == torch.float8_e4m3fn else 0, self.Hkv, self.D,
                              page, npages, k.stride(0), k.stride(1), k.stride(2), _ptr(k_scale), _ptr(v_scale))
        self.on_gpu = _on_gpu(k, v, k_scale, v_scale)
        self.ref = C.addressof(self.c)


class KvBatch:
    """The requests of one call: q_start int32 [B+1], kv_len int32 [B], page_table int32 [B, pages]
    (device tensors, read when the kernels run), T token rows, about max_n new tokens a request."""

    def __init__(self, q_start, kv_len, page_table, T: int, max_n: int):
        import torch
        B = kv_len.numel()
        if (any(t.dtype != torch.int32 for t in (q_start, kv_len, page_table)) or q_start.numel() != B + 1
                or page_table.dim() != 2 or page_table.shape[0] != B or not q_start.is_contiguous()
                or not kv_len.is_contiguous() or (page_table.numel() and page_table.stride(1) != 1)):
            raise ValueError("KvBatch: int32 q_start [B+1], kv_len [B] and page_table [B, pages], rows contiguous")
        if B > 1 and page_table.stride(0) != page_table.shape[1]:
            raise ValueError("KvBatch: the rows of page_table follow one another")
        self.q_start, self.kv_len, self.page_table = q_start, kv_len, page_table
        self.c = moe_kv_batch(q_start.data_ptr(), kv_len.data_ptr(), page_table.data_ptr(), B, T, max_n,
                              page_table.shape[1])
        self.on_gpu = _on_gpu(q_start, kv_len, page_table)
        self.ref = C.addressof(self.c)


class Rope:
    """Rotation frequencies: theta^(-2i/rot), or inv_freq (float64 [rot/2])."""

    def __init__(self, rot: int, theta: float = 10000.0, inv_freq: Optional[np.ndarray] = None,
                 interleaved: bool = False):
        f = None
        if inv_freq is not None:
            f = np.ascontiguousarray(inv_freq, dtype=np.float64)
            if f.shape != (rot // 2,):
                raise ValueError("Rope: inv_freq is [rot/2]")
        h = C.c_void_p()
        _check(load().moe_rope_create(C.byref(h), rot, 1 if interleaved else 0, float(theta),
                                      None if f is None else f.ctypes.data), "moe_rope_create")
        self.handle, self.rot = h, rot

    def close(self):
        if self.handle:
            load().moe_rope_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class AttnWorkspace:
    def __init__(self, Hq: int, Hkv: int, D: int):
        h = C.c_void_p()
        _check(load().moe_attn_ws_create(C.byref(h), Hq, Hkv, D), "moe_attn_ws_create")
        self.handle = h
        self.Hq, self.Hkv, self.D = Hq, Hkv, D
        v = moe_attn_ws_view()
        _check(load().moe_attn_ws_get_view(h, C.byref(v)), "moe_attn_ws_get_view")
        self.view = v

    def close(self):
        if self.handle:
            load().moe_attn_ws_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @property
    def error_ptr(self) -> int:
        return self.view.error

    def set_wait_test(self, stage: int) -> None:
        """Fault-injection hook for tests of the bounded waits (see include/moe.h)."""
        _check(load().moe_attn_ws_set_wait_test(self.handle, int(stage)), "moe_attn_ws_set_wait_test")


def _heads(t, shape, types, what: str):
    """Address and token stride of [T, H, D] bf16 rows whose heads follow one another."""
    if t.dtype in types and t.shape == shape:
        tok, head, col = t.stride()
        if col == 1 and (head == shape[2] or shape[1] <= 1):
            return t.data_ptr(), tok
    raise ValueError(f"{what}: bf16 {list(shape)} with heads {shape[2]} apart, got {list(t.shape)} {t.dtype} "
                     f"strides {t.stride()}")


def moe_kv_append(pages: KvPages, batch: KvBatch, rope: Optional[Rope], q, q_out, k, v, err=None, stream=None) -> None:
    """Rotate q into q_out and the keys by position; write keys and values into their pages."""
    T, D, bf16 = batch.c.T, pages.D, _row_types()[1]
    kv = (T, pages.Hkv, D)
    kp, ks = _heads(k, kv, bf16, "k")
    vp, vs = _heads(v, kv, bf16, "v")
    on_gpu = pages.on_gpu and batch.on_gpu and k.is_cuda and v.is_cuda
    Hq, qp, qs, op, os_ = 0, None, 0, None, 0
    if q is not None:
        Hq = q.shape[1]
        rows = (T, Hq, D)
        qp, qs = _heads(q, rows, bf16, "q")
        # in place: looked at already
        op, os_ = (qp, qs) if q_out is q else _heads(q_out, rows, bf16, "q_out")
        on_gpu = on_gpu and q.is_cuda and q_out.is_cuda
    if err is not None and not isinstance(err, int):
        on_gpu = on_gpu and err.is_cuda
        err = err.data_ptr()
    if not on_gpu:
        raise ValueError(_ELSEWHERE)
    _check(load().moe_kv_append(pages.ref, batch.ref, None if rope is None else rope.handle, qp, qs, op, os_, Hq, kp, ks,
                                vp, vs, err, _stream(stream)), "moe_kv_append")


def moe_paged_attention(pages: KvPages, batch: KvBatch, q, o, ws: AttnWorkspace, scale: float, window: int = 0,
                        stream=None) -> None:
    """o (bf16 [T, Hq, D]) = attention of every new token over its request's pages."""
    rows, bf16 = (batch.c.T, ws.Hq, pages.D), _row_types()[1]
    qp, qs = _heads(q, rows, bf16, "q")
    op, os_ = _heads(o, rows, bf16, "o")
    if not (pages.on_gpu and batch.on_gpu and q.is_cuda and o.is_cuda):
        raise ValueError(_ELSEWHERE)
    _check(load().moe_paged_attention(pages.ref, batch.ref, qp, qs, ws.Hq, op, os_, scale, window, ws.handle,
                                      _stream(stream)), "moe_paged_attention")


def moe_attn_sync_status(ws: AttnWorkspace, stream=None) -> int:
    return int(load().moe_attn_sync_status(ws.handle, _stream(stream)))


class BlockNormDesc:
    """Owner of a moe_block_norm_desc and references to its tensors (bf16 or their bits)."""

    def __init__(self, **kw):
        self.tensors = kw
        y, gate, bf16 = kw["y"], kw["gate"], _row_types()[1]
        for t in (y, gate):
            if t is not None and (t.dim() != 2 or t.dtype not in bf16 or t.stride(1) != 1):
                raise ValueError("block_norm_desc: y is bf16 [T, H], gate bf16 [T, H] or [1, H], columns contiguous")
        for t in (kw["w_post"], kw["w_pre"]):
            if t is not None and (t.dim() != 1 or t.dtype not in bf16 or not t.is_contiguous()):
                raise ValueError("block_norm_desc: the weights are contiguous bf16 [H]")
        self.T = None if y is None else y.shape[0]
        widths = {t.shape[-1] for t in (y, gate, kw["w_post"], kw["w_pre"]) if t is not None}
        if len(widths) > 1 or (gate is not None and gate.shape[0] not in (1, self.T)):
            raise ValueError("block_norm_desc: y, gate and the weights differ in size")
        self.H = widths.pop() if widths else None
        self.c = moe_block_norm_desc(
            _ptr(y), 0 if y is None else y.stride(0), 1 if kw["post_norm"] else 0, _ptr(kw["w_post"]), _ptr(gate),
            0 if gate is None or gate.shape[0] == 1 else gate.stride(0), 1 if kw["gate_sigmoid"] else 0,
            kw["res_scale"], _ptr(kw["w_pre"]), kw["eps"])
        self.on_gpu = _on_gpu(y, gate, kw["w_post"], kw["w_pre"])
        self.ref = C.addressof(self.c)


def block_norm_desc(y=None, post_norm: bool = False, w_post=None, gate=None, gate_sigmoid: bool = False,
                    res_scale: float = 1.0, w_pre=None, eps: float = 1e-6) -> BlockNormDesc:
    return BlockNormDesc(y=y, post_norm=post_norm, w_post=w_post, gate=gate, gate_sigmoid=gate_sigmoid,
                         res_scale=res_scale, w_pre=w_pre, eps=eps)


def _columns(t, rows, types, what: str):
    """Address and row stride of [T, H] rows with contiguous columns."""
    if t.shape == rows and t.dtype in types:
        row, col = t.stride()
        if col == 1 or rows[1] == 1:
            return t.data_ptr(), row
    raise ValueError(f"{what}: {types[0]} {list(rows)}, columns contiguous, got {list(t.shape)} {t.dtype} strides {t.stride()}")


def moe_block_norm(desc: BlockNormDesc, x, x_out, xn, T: int, H: int, stream=None) -> None:
    """x_out (fp32) = x + res_scale * gate * post-norm(y); xn (bf16) = pre-norm of the next block of x_out."""
    if desc.H not in (None, H) or desc.T not in (None, T):
        raise ValueError(f"moe_block_norm: y, gate and the weights are [{T}, {H}]")
    rows = (T, H)
    fp32, bf16 = _row_types()
    xp, xs = _columns(x, rows, fp32, "x")
    # in place: looked at already
    op, os_ = (xp, xs) if x_out is x else (None, 0) if x_out is None else _columns(x_out, rows, fp32, "x_out")
    np_, ns = (None, 0) if xn is None else _columns(xn, rows, bf16, "xn")
    if not (desc.on_gpu and x.is_cuda and (x_out is None or x_out.is_cuda) and (xn is None or xn.is_cuda)):
        raise ValueError(_ELSEWHERE)
    _check(load().moe_block_norm(desc.ref, xp, xs, op, os_, np_, ns, T, H, _stream(stream)), "moe_block_norm")


# --------------------------------------------- a step of drafted token trees

def _ints(t, shape, what: str):
    """Address of a contiguous int32 tensor."""
    import torch
    if t.dtype != torch.int32 or tuple(t.shape) != shape or not t.is_contiguous():
        raise ValueError(f"{what}: contiguous int32 {list(shape)}, got {list(t.shape)} {t.dtype}")
    return t.data_ptr()


def _error_word(err):
    """Address of an error word, and whether it is where the kernels can write it."""
    if err is None or isinstance(err, int):
        return err, True
    return err.data_ptr(), err.is_cuda


class Tree:
    """The trees of a batch's new tokens: parent int32 [T], an index among the request's own rows or -1;
    depth int32 [T] and the masks above and below int32 [T, words], which moe_tree_prepare fills.  The masks
    have room for the batch's max_n nodes, in whole words of 32."""

    def __init__(self, batch: KvBatch, parent):
        import torch
        T, words = batch.c.T, max(1, -(-batch.c.max_n // 32))
        if words > 8:
            raise ValueError(f"Tree: at most 256 nodes a request, max_n is {batch.c.max_n}")
        p = _ints(parent, (T,), "parent")
        self.parent, self.words = parent, words
        self.depth = torch.zeros(T, dtype=torch.int32, device=parent.device)
        self.above, self.below = (torch.zeros(T, words, dtype=torch.int32, device=parent.device) for _ in range(2))
        self.c = moe_tree(p, self.depth.data_ptr(), self.above.data_ptr(), self.below.data_ptr(), words)
        self.T, self.on_gpu = T, parent.is_cuda
        self.ref = C.addressof(self.c)


def _same_rows(batch: KvBatch, tree: "Tree") -> None:
    if tree.T != batch.c.T:
        raise ValueError(f"the tree has {tree.T} rows, the batch {batch.c.T}")


def moe_tree_prepare(batch: KvBatch, tree: Tree, err=None, stream=None) -> None:
    """Depths and masks of the trees from their parents, once for all layers of a step."""
    _same_rows(batch, tree)
    ep, there = _error_word(err)
    if not (batch.on_gpu and tree.on_gpu and there):
        raise ValueError(_ELSEWHERE)
    _check(load().moe_tree_prepare(batch.ref, tree.ref, ep, _stream(stream)), "moe_tree_prepare")


class HeadNorm:
    """Norms of each head's queries and keys: weights bf16 [D] (or their bits) or None, for ones."""

    def __init__(self, w_q=None, w_k=None, eps: float = 1e-6):
        bf16 = _row_types()[1]
        for w in (w_q, w_k):
            if w is not None and (w.dim() != 1 or w.dtype not in bf16 or not w.is_contiguous()):
                raise ValueError("HeadNorm: the weights are contiguous bf16 [D]")
        widths = {w.numel() for w in (w_q, w_k) if w is not None}
        if len(widths) > 1:
            raise ValueError("HeadNorm: the weights differ in size")
        self.w_q, self.w_k, self.D = w_q, w_k, widths.pop() if widths else None
        self.c = moe_head_norm(_ptr(w_q), _ptr(w_k), eps)
        self.on_gpu = _on_gpu(w_q, w_k)
        self.ref = C.addressof(self.c)


def moe_kv_append_norm(pages: KvPages, batch: KvBatch, rope: Optional[Rope], norm: Optional[HeadNorm], q, q_out, k, v,
                       tree: Optional[Tree] = None, err=None, stream=None) -> None:
    """moe_kv_append behind norms of the queries' and keys' heads, at the positions of a tree's nodes."""
    T, D, bf16 = batch.c.T, pages.D, _row_types()[1]
    kv = (T, pages.Hkv, D)
    kp, ks = _heads(k, kv, bf16, "k")
    vp, vs = _heads(v, kv, bf16, "v")
    on_gpu = pages.on_gpu and batch.on_gpu and k.is_cuda and v.is_cuda
    Hq, qp, qs, op, os_ = 0, None, 0, None, 0
    if q is not None:
        Hq = q.shape[1]
        rows = (T, Hq, D)
        qp, qs = _heads(q, rows, bf16, "q")
        op, os_ = (qp, qs) if q_out is q else _heads(q_out, rows, bf16, "q_out")
        on_gpu = on_gpu and q.is_cuda and q_out.is_cuda
    if norm is not None:
        if norm.D not in (None, D):
            raise ValueError(f"moe_kv_append_norm: the norms' weights are [{D}]")
        on_gpu = on_gpu and norm.on_gpu
    if tree is not None:
        _same_rows(batch, tree)
        on_gpu = on_gpu and tree.on_gpu
    ep, there = _error_word(err)
    if not (on_gpu and there):
        raise ValueError(_ELSEWHERE)
    _check(load().moe_kv_append_norm(pages.ref, batch.ref, None if tree is None else tree.ref,
                                     None if rope is None else rope.handle, None if norm is None else norm.ref, qp, qs, op,
                                     os_, Hq, kp, ks, vp, vs, ep, _stream(stream)), "moe_kv_append_norm")


def moe_tree_attention(pages: KvPages, batch: KvBatch, tree: Tree, q, o, ws: AttnWorkspace, scale: float, window: int = 0,
                       stream=None) -> None:
    """o (bf16 [T, Hq, D]) = attention of every tree node over its request's pages and the nodes above it."""
    rows, bf16 = (batch.c.T, ws.Hq, pages.D), _row_types()[1]
    qp, qs = _heads(q, rows, bf16, "q")
    op, os_ = _heads(o, rows, bf16, "o")
    _same_rows(batch, tree)
    if not (pages.on_gpu and batch.on_gpu and tree.on_gpu and q.is_cuda and o.is_cuda):
        raise ValueError(_ELSEWHERE)
    _check(load().moe_tree_attention(pages.ref, batch.ref, tree.ref, qp, qs, ws.Hq, op, os_, scale, window, ws.handle,
                                     _stream(stream)), "moe_tree_attention")


class VerifyDesc:
    """Owner of a moe_verify_desc and references to its tensors."""

    def __init__(self, target, token, parent, u, u_last, draft=None):
        import torch
        if target.dim() != 2:
            raise ValueError("verify_desc: target is float32 [T, V]")
        T, V = target.shape
        fp32 = _row_types()[0]
        tp, ts = _columns(target, (T, V), fp32, "target")
        dp, ds = (None, 0) if draft is None else _columns(draft, (T, V), fp32, "draft")
        for t, n in ((u, (T,)), (u_last, (u_last.numel(),))):
            if t.dtype != torch.float32 or tuple(t.shape) != n or not t.is_contiguous():
                raise ValueError("verify_desc: u and u_last are contiguous float32 [T] and [B]")
        self.tensors = (target, token, parent, u, u_last, draft)
        self.T, self.B = T, u_last.numel()
        self.c = moe_verify_desc(tp, ts, dp, ds, _ints(token, (T,), "token"), _ints(parent, (T,), "parent"), u.data_ptr(),
                                 u_last.data_ptr(), V)
        self.on_gpu = _on_gpu(*self.tensors)
        self.ref = C.addressof(self.c)


def verify_desc(target, token, parent, u, u_last, draft=None) -> VerifyDesc:
    return VerifyDesc(target, token, parent, u, u_last, draft)


def moe_verify_drafts(batch: KvBatch, desc: VerifyDesc, path, count, token, err=None, stream=None) -> None:
    """path int32 [B, most], count and token int32 [B]: the nodes the target keeps and the next token."""
    B = batch.c.B
    if desc.T != batch.c.T or desc.B != B:
        raise ValueError(f"moe_verify_drafts: {desc.T} rows and {desc.B} requests, the batch has {batch.c.T} and {B}")
    if path.dim() != 2:
        raise ValueError("path: int32 [B, most nodes kept]")
    pp, cp, tp = _ints(path, (B, path.shape[1]), "path"), _ints(count, (B,), "count"), _ints(token, (B,), "token")
    ep, there = _error_word(err)
    if not (batch.on_gpu and desc.on_gpu and path.is_cuda and count.is_cuda and token.is_cuda and there):
        raise ValueError(_ELSEWHERE)
    _check(load().moe_verify_drafts(batch.ref, desc.ref, pp, path.shape[1], cp, tp, ep, _stream(stream)),
           "moe_verify_drafts")


class KvLayers:
    """The pools of a model's layers, of one geometry, for the calls that move keys and values in all of them; one that
    layers share counts once."""

    def __init__(self, layers):
        self.layers = list(layers)
        if not self.layers or any(not isinstance(p, KvPages) for p in self.layers):
            raise ValueError("KvLayers: a list of KvPages, one a layer")
        self.c = (moe_kv_pages * len(self.layers))(*[p.c for p in self.layers])
        self.on_gpu = all(p.on_gpu for p in self.layers)
        self.ref = C.addressof(self.c)


def moe_kv_compact(layers: KvLayers, batch: KvBatch, path, count, kv_len_out=None, err=None, stream=None) -> None:
    """Keys and values of the kept nodes to the front of their trees in every layer; kv_len_out int32 [B]: the new lengths."""
    B = batch.c.B
    if path.dim() != 2:
        raise ValueError("path: int32 [B, most nodes kept]")
    pp, cp = _ints(path, (B, path.shape[1]), "path"), _ints(count, (B,), "count")
    lp = None if kv_len_out is None else _ints(kv_len_out, (B,), "kv_len_out")
    ep, there = _error_word(err)
    if not (layers.on_gpu and batch.on_gpu and path.is_cuda and count.is_cuda and (kv_len_out is None or kv_len_out.is_cuda)
            and there):
        raise ValueError(_ELSEWHERE)
    _check(load().moe_kv_compact(layers.ref, len(layers.layers), batch.ref, pp, path.shape[1], cp, lp, ep, _stream(stream)),
           "moe_kv_compact")


def moe_kv_copy_pages(layers: KvLayers, src, dst, tokens=None, err=None, stream=None) -> None:
    """Page src[i] to page dst[i] in every layer, or its first tokens[i] places."""
    n = src.numel()
    sp, dp = _ints(src, (n,), "src"), _ints(dst, (n,), "dst")
    tp = None if tokens is None else _ints(tokens, (n,), "tokens")
    ep, there = _error_word(err)
    if not (layers.on_gpu and src.is_cuda and dst.is_cuda and (tokens is None or tokens.is_cuda) and there):
        raise ValueError(_ELSEWHERE)
    _check(load().moe_kv_copy_pages(layers.ref, len(layers.layers), sp, dp, tp, n, ep, _stream(stream)), "moe_kv_copy_pages")
