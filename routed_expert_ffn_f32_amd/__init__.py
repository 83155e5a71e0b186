"""Python binding of libcoli_moe, the gfx950 routed-MoE layer library.

Argument marshalling only: every step of the layer runs in the library's HIP
kernels (include/coli_moe.h documents the C ABI).  The functions keep the C
names; pointers are passed as integers (device addresses, e.g. a torch
tensor's data_ptr()) and streams as integer hipStream_t handles (e.g.
torch.cuda.current_stream().cuda_stream).  Non-zero return codes raise
ColiMoeError.

`MoELayer` is a convenience wrapper that uses PyTorch for what PyTorch is
here for: device memory (weights, workspace, outputs) and streams.

There is no fallback: if the library is not built, importing works but the
first call raises, naming the build command.
"""
from __future__ import annotations

import contextlib
import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
# The in-tree build (routed_expert_ffn_f32_amd/build.py), and only that.
LIB_PATH = os.path.join(_HERE, "_lib", "libcoli_moe.so")

COLI_MOE_OK = 0
COLI_MOE_ECAPACITY = -1
COLI_MOE_EROUTING = -2
COLI_MOE_EDEVICE = -3
COLI_MOE_EARG = -4
COLI_MOE_N_KERNELS = 10
COLI_MOE_STATIC_SCRATCH_BYTES = 64 << 20
COLI_MOE_DEFAULT_SPIN_LIMIT = 1 << 22


class ColiMoeError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: error {code} ({coli_moe_error_string(code)})")


class coli_moe_config_t(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("n_experts", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("inter", ctypes.c_int32), ("n_shared", ctypes.c_int32), ("group_size", ctypes.c_int32),
                ("n_group", ctypes.c_int32), ("max_tokens", ctypes.c_int32),
                ("prefill_threshold", ctypes.c_int32), ("routed_scaling_factor", ctypes.c_float),
                ("weight_format", ctypes.c_int32)]


class coli_moe_weights_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "router_w", "sel_bias", "gate_q", "gate_s", "up_q", "up_s", "down_q", "down_s",
        "sh_gate_q", "sh_gate_s", "sh_up_q", "sh_up_s", "sh_down_q", "sh_down_s")]


class coli_moe_host_experts_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("gate_q", "gate_s", "up_q", "up_s", "down_q", "down_s")]


class coli_moe_cache_config_t(ctypes.Structure):
    _fields_ = [("n_slots", ctypes.c_int32), ("repin_every", ctypes.c_int32), ("decay", ctypes.c_float)]


class coli_moe_cache_stats_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("calls", "needed", "hits", "misses", "prefetched", "prefetch_hits",
                                               "evictions", "repin_swaps", "bytes_copied")] + \
               [("pinned", ctypes.c_int32), ("resident", ctypes.c_int32)]

    def as_dict(self):
        return {n: int(getattr(self, n)) for n, _ in self._fields_}


# Element types and score kinds of the operators around the layer.
COLI_MOE_F32 = 0
COLI_MOE_BF16 = 1
COLI_MOE_F16 = 2
COLI_MOE_INT8 = 3
COLI_MOE_E4M3 = 4
COLI_MOE_SCORES_SIGMOID = 0
COLI_MOE_SCORES_SOFTMAX = 1


class coli_moe_rmsnorm_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("rows", "hidden", "x_type", "residual_type", "weight_type", "out_type",
                                              "group")] + \
               [("eps", ctypes.c_float), ("x", ctypes.c_void_p), ("x_stride", ctypes.c_int64),
                ("residual", ctypes.c_void_p), ("residual_stride", ctypes.c_int64),
                ("residual_out", ctypes.c_void_p), ("residual_out_stride", ctypes.c_int64),
                ("weight", ctypes.c_void_p), ("out", ctypes.c_void_p), ("out_stride", ctypes.c_int64),
                ("scales", ctypes.c_void_p), ("scales_stride", ctypes.c_int64)]


COLI_MOE_ACT_NONE = 0
COLI_MOE_ACT_RELU = 1
COLI_MOE_ACT_SILU = 2
COLI_MOE_ACT_GELU = 3
COLI_MOE_ACT_GELU_TANH = 4
COLI_MOE_ACT_SWIGLU = 5


class coli_moe_linear_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("m", "n", "k", "type", "out_type", "bias_type", "act")] + \
               [("x", ctypes.c_void_p), ("ldx", ctypes.c_int64), ("w", ctypes.c_void_p), ("ldw", ctypes.c_int64),
                ("x_scale", ctypes.c_void_p), ("w_scale", ctypes.c_void_p), ("bias", ctypes.c_void_p),
                ("residual", ctypes.c_void_p), ("ldr", ctypes.c_int64), ("out", ctypes.c_void_p),
                ("ldo", ctypes.c_int64)]


class coli_moe_balance_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("tokens", "n_experts", "top_k", "n_seqs", "scores")] + \
               [("alpha", ctypes.c_float), ("logits", ctypes.c_void_p), ("logits_stride", ctypes.c_int64),
                ("idx", ctypes.c_void_p), ("seq_offsets", ctypes.c_void_p), ("mask", ctypes.c_void_p)]


_lib = None


def load_library():
    """Load the built library (raises if it was never built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m routed_expert_ffn_f32_amd.build` (hipcc, gfx950)")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
        cfgp, wp = ctypes.POINTER(coli_moe_config_t), ctypes.POINTER(coli_moe_weights_t)
        L.coli_moe_workspace_bytes.argtypes = [cfgp]
        L.coli_moe_workspace_bytes.restype = sz
        L.coli_moe_init.argtypes = [ctypes.POINTER(vp), cfgp, wp, vp, sz, vp]
        L.coli_moe_init.restype = ctypes.c_int
        L.coli_moe_forward.argtypes = [vp, vp, vp, i32, vp]
        L.coli_moe_forward.restype = ctypes.c_int
        L.coli_moe_forward_noalloc.argtypes = [cfgp, wp, vp, vp, i32, vp]
        L.coli_moe_forward_noalloc.restype = ctypes.c_int
        L.coli_moe_free.argtypes = [vp]
        L.coli_moe_free.restype = None
        L.coli_moe_set_routing.argtypes = [vp, i32, ctypes.c_float]
        L.coli_moe_set_routing.restype = ctypes.c_int
        L.coli_moe_last_routing.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp]
        L.coli_moe_last_routing.restype = ctypes.c_int
        L.coli_moe_status.argtypes = [vp, vp]
        L.coli_moe_status.restype = ctypes.c_int
        L.coli_moe_test_spin_limit.argtypes = [vp, i32]
        L.coli_moe_test_spin_limit.restype = ctypes.c_int
        L.coli_moe_test_batch_kernels.argtypes = [vp, i32]
        L.coli_moe_test_batch_kernels.restype = ctypes.c_int
        L.coli_moe_test_dispatch.argtypes = [vp, i32, i32, i32, vp, vp, vp, vp, vp, vp]
        L.coli_moe_test_dispatch.restype = ctypes.c_int
        L.coli_moe_probe_read.argtypes = [vp, vp, i32, vp]
        L.coli_moe_probe_read.restype = ctypes.c_int
        L.coli_moe_probe_read_down.argtypes = [vp, vp, i32, vp]
        L.coli_moe_probe_read_down.restype = ctypes.c_int
        L.coli_moe_probe_stream.argtypes = [vp, ctypes.c_size_t, vp, vp]
        L.coli_moe_probe_stream.restype = ctypes.c_int
        L.coli_moe_probe_mfma.argtypes = [i32, i32, vp, vp]
        L.coli_moe_probe_mfma.restype = ctypes.c_int
        L.coli_moe_probe_mfma_f16.argtypes = [i32, i32, ctypes.c_uint32, vp, vp]
        L.coli_moe_probe_mfma_f16.restype = ctypes.c_int
        L.coli_moe_profile_begin.argtypes = [vp, i32]
        L.coli_moe_profile_begin.restype = ctypes.c_int
        L.coli_moe_profile_end.argtypes = [vp, vp, vp]
        L.coli_moe_profile_end.restype = ctypes.c_int
        L.coli_moe_kernel_name.argtypes = [i32]
        L.coli_moe_kernel_name.restype = ctypes.c_char_p
        L.coli_moe_error_string.argtypes = [i32]
        L.coli_moe_error_string.restype = ctypes.c_char_p
        hp, ccp = ctypes.POINTER(coli_moe_host_experts_t), ctypes.POINTER(coli_moe_cache_config_t)
        L.coli_moe_cache_slot_bytes.argtypes = [cfgp, i32]
        L.coli_moe_cache_slot_bytes.restype = sz
        L.coli_moe_cache_init.argtypes = [ctypes.POINTER(vp), cfgp, ccp, wp, hp, vp, sz, vp, sz, vp]
        L.coli_moe_cache_init.restype = ctypes.c_int
        L.coli_moe_cache_forward.argtypes = [vp, vp, vp, i32, vp]
        L.coli_moe_cache_forward.restype = ctypes.c_int
        L.coli_moe_cache_prefetch.argtypes = [vp, vp, i32, i32, vp]
        L.coli_moe_cache_prefetch.restype = ctypes.c_int
        L.coli_moe_cache_pin.argtypes = [vp, vp, i32, vp]
        L.coli_moe_cache_pin.restype = ctypes.c_int
        L.coli_moe_cache_stats.argtypes = [vp, ctypes.POINTER(coli_moe_cache_stats_t)]
        L.coli_moe_cache_stats.restype = ctypes.c_int
        L.coli_moe_cache_usage.argtypes = [vp, vp]
        L.coli_moe_cache_usage.restype = ctypes.c_int
        L.coli_moe_cache_slots.argtypes = [vp, vp]
        L.coli_moe_cache_slots.restype = ctypes.c_int
        L.coli_moe_cache_layer.argtypes = [vp]
        L.coli_moe_cache_layer.restype = vp
        L.coli_moe_cache_free.argtypes = [vp]
        L.coli_moe_cache_free.restype = None
        L.coli_moe_usage_engine_id.argtypes = []
        L.coli_moe_usage_engine_id.restype = ctypes.c_uint32
        L.coli_moe_usage_write.argtypes = [ctypes.c_char_p, i32, i32, vp]
        L.coli_moe_usage_write.restype = ctypes.c_int
        L.coli_moe_usage_read.argtypes = [ctypes.c_char_p, i32, i32, vp]
        L.coli_moe_usage_read.restype = ctypes.c_int
        L.coli_moe_test_cache_policy.argtypes = [i32, i32, i32, ctypes.c_float, i32, vp, i32, vp, vp, i32, vp, vp]
        L.coli_moe_test_cache_policy.restype = ctypes.c_int
        L.coli_moe_rmsnorm.argtypes = [ctypes.POINTER(coli_moe_rmsnorm_t), vp]
        L.coli_moe_rmsnorm.restype = ctypes.c_int
        L.coli_moe_linear.argtypes = [ctypes.POINTER(coli_moe_linear_t), vp]
        L.coli_moe_linear.restype = ctypes.c_int
        bp = ctypes.POINTER(coli_moe_balance_t)
        L.coli_moe_balance_workspace_bytes.argtypes = [i32, i32, i32]
        L.coli_moe_balance_workspace_bytes.restype = sz
        L.coli_moe_balance.argtypes = [bp, vp, vp, vp, vp, sz, vp]
        L.coli_moe_balance.restype = ctypes.c_int
        L.coli_moe_balance_grad.argtypes = [bp, vp, vp, vp, ctypes.c_int64, vp]
        L.coli_moe_balance_grad.restype = ctypes.c_int
        L.coli_moe_last_logits.argtypes = [vp, vp, vp]
        L.coli_moe_last_logits.restype = ctypes.c_int
        _lib = L
    return _lib


def _check(rc: int, where: str) -> int:
    if rc < 0:
        raise ColiMoeError(rc, where)
    return rc


def coli_moe_error_string(code: int) -> str:
    return load_library().coli_moe_error_string(int(code)).decode()


def coli_moe_kernel_name(i: int) -> str:
    return load_library().coli_moe_kernel_name(int(i)).decode()


def coli_moe_workspace_bytes(cfg: coli_moe_config_t) -> int:
    return int(load_library().coli_moe_workspace_bytes(ctypes.byref(cfg)))


def coli_moe_init(cfg: coli_moe_config_t, weights: coli_moe_weights_t, workspace: int,
                  workspace_bytes: int, stream: int = 0) -> ctypes.c_void_p:
    h = ctypes.c_void_p()
    _check(load_library().coli_moe_init(ctypes.byref(h), ctypes.byref(cfg), ctypes.byref(weights),
                                        workspace, workspace_bytes, stream), "coli_moe_init")
    return h


def coli_moe_forward(handle, hidden: int, out: int, T: int, stream: int = 0) -> int:
    return _check(load_library().coli_moe_forward(handle, hidden, out, int(T), stream), "coli_moe_forward")


def coli_moe_forward_noalloc(cfg: coli_moe_config_t, weights: coli_moe_weights_t, hidden: int, out: int, T: int,
                             stream: int = 0) -> int:
    """The forward without handle or workspace: the library's own device
    array (COLI_MOE_STATIC_SCRATCH_BYTES per device) is the workspace."""
    return _check(load_library().coli_moe_forward_noalloc(ctypes.byref(cfg), ctypes.byref(weights), hidden, out,
                                                          int(T), stream), "coli_moe_forward_noalloc")


def coli_moe_free(handle) -> None:
    load_library().coli_moe_free(handle)


def coli_moe_set_routing(handle, k_use: int, top_p: float = 1.0) -> int:
    """Run-time routing limits (explicit smaller k, adaptive expert top-p) of
    the handle's later forwards; (top_k, 1.0) is the plain routing."""
    return _check(load_library().coli_moe_set_routing(handle, int(k_use), float(top_p)), "coli_moe_set_routing")


def _warn_lossy(k_use: int, top_k: int, top_p: float) -> None:
    if k_use < top_k or top_p < 1.0:
        import warnings
        warnings.warn(f"lossy routing override: k {k_use} of {top_k}, expert top-p {top_p}: outputs differ from the "
                      f"layer's plain routing", stacklevel=3)


def coli_moe_last_routing(handle, idx=None, w=None, offsets=None, sorted_ids=None, inv=None,
                          active=None, n_active=None, stream: int = 0) -> int:
    return _check(load_library().coli_moe_last_routing(handle, idx, w, offsets, sorted_ids, inv, active,
                                                       n_active, stream), "coli_moe_last_routing")


def coli_moe_test_dispatch(idx: int, T: int, k: int, E: int, offsets: int, sorted_ids: int, inv: int,
                           active: int, n_active: int, stream: int = 0) -> int:
    return _check(load_library().coli_moe_test_dispatch(idx, int(T), int(k), int(E), offsets, sorted_ids,
                                                        inv, active, n_active, stream),
                  "coli_moe_test_dispatch")


def coli_moe_probe_read(handle, experts: int, n: int, stream: int = 0) -> int:
    """Pure-load probe of the gate/up rows of n experts (device int32 ids, -1
    = shared): the read ceiling of the gate/up access pattern."""
    return _check(load_library().coli_moe_probe_read(handle, experts, int(n), stream), "coli_moe_probe_read")


def coli_moe_probe_read_down(handle, experts: int, n: int, stream: int = 0) -> int:
    """Pure-load probe of the down rows of n experts with the one-token down +
    combine launch's grid: the read ceiling of that access pattern."""
    return _check(load_library().coli_moe_probe_read_down(handle, experts, int(n), stream),
                  "coli_moe_probe_read_down")


def coli_moe_probe_stream(buf: int, nbytes: int, sink: int, stream: int = 0) -> int:
    """XOR of every 32-bit word of a device buffer into the device word at
    sink, each byte read once (the HBM read rate of this GPU)."""
    return _check(load_library().coli_moe_probe_stream(buf, int(nbytes), sink, stream), "coli_moe_probe_stream")


MFMA_PROBE_MFMAS_PER_ROUND = 8


def coli_moe_probe_mfma(iters: int, blocks: int, sink: int, stream: int = 0) -> int:
    """blocks x 4 waves of iters x 8 back-to-back bf16 MFMAs (32768 flops
    each); each wave whose results check adds 1 to the device word at sink."""
    return _check(load_library().coli_moe_probe_mfma(int(iters), int(blocks), sink, stream), "coli_moe_probe_mfma")


MFMA_F16_PROBE_MFMAS_PER_ROUND = 16


def coli_moe_probe_mfma_f16(iters: int, blocks: int, seed: int, sink: int, stream: int = 0) -> int:
    """blocks x 4 waves of iters x 16 back-to-back f16 MFMAs on operands that
    change from one MFMA to the next; each wave whose accumulators are all
    finite adds 1 to the device word at sink."""
    return _check(load_library().coli_moe_probe_mfma_f16(int(iters), int(blocks), int(seed) & 0xFFFFFFFF, sink, stream),
                  "coli_moe_probe_mfma_f16")


def coli_moe_profile_begin(handle, max_calls: int) -> int:
    return _check(load_library().coli_moe_profile_begin(handle, int(max_calls)), "coli_moe_profile_begin")


def coli_moe_profile_end(handle):
    """Returns (calls, {kernel name: (total ms, launches)})."""
    ms = (ctypes.c_float * COLI_MOE_N_KERNELS)()
    n = (ctypes.c_int32 * COLI_MOE_N_KERNELS)()
    calls = _check(load_library().coli_moe_profile_end(handle, ms, n), "coli_moe_profile_end")
    return calls, {coli_moe_kernel_name(i): (float(ms[i]), int(n[i])) for i in range(COLI_MOE_N_KERNELS)}


def coli_moe_cache_slot_bytes(cfg: coli_moe_config_t, n_slots: int) -> int:
    return int(load_library().coli_moe_cache_slot_bytes(ctypes.byref(cfg), int(n_slots)))


def coli_moe_cache_init(cfg, cache_cfg, resident, host, slots: int, slot_bytes: int, workspace: int,
                        workspace_bytes: int, stream: int = 0):
    h = ctypes.c_void_p()
    _check(load_library().coli_moe_cache_init(ctypes.byref(h), ctypes.byref(cfg), ctypes.byref(cache_cfg),
                                              ctypes.byref(resident), ctypes.byref(host), slots, slot_bytes,
                                              workspace, workspace_bytes, stream), "coli_moe_cache_init")
    return h


def coli_moe_cache_forward(cache, hidden: int, out: int, T: int, stream: int = 0) -> int:
    return _check(load_library().coli_moe_cache_forward(cache, hidden, out, int(T), stream), "coli_moe_cache_forward")


def coli_moe_cache_prefetch(cache, hidden: int, T: int, n_predict: int, stream: int = 0) -> int:
    return _check(load_library().coli_moe_cache_prefetch(cache, hidden, int(T), int(n_predict), stream),
                  "coli_moe_cache_prefetch")


def coli_moe_cache_pin(cache, experts, stream: int = 0) -> int:
    arr = (ctypes.c_int32 * len(experts))(*[int(e) for e in experts])
    return _check(load_library().coli_moe_cache_pin(cache, arr, len(experts), stream), "coli_moe_cache_pin")


def coli_moe_cache_stats(cache) -> dict:
    st = coli_moe_cache_stats_t()
    _check(load_library().coli_moe_cache_stats(cache, ctypes.byref(st)), "coli_moe_cache_stats")
    return st.as_dict()


def coli_moe_cache_usage(cache, n_experts: int):
    arr = (ctypes.c_int64 * n_experts)()
    _check(load_library().coli_moe_cache_usage(cache, arr), "coli_moe_cache_usage")
    return [int(v) for v in arr]


def coli_moe_cache_slots(cache, n_experts: int):
    arr = (ctypes.c_int32 * n_experts)()
    _check(load_library().coli_moe_cache_slots(cache, arr), "coli_moe_cache_slots")
    return [int(v) for v in arr]


def coli_moe_cache_layer(cache):
    return load_library().coli_moe_cache_layer(cache)


def coli_moe_cache_free(cache) -> None:
    load_library().coli_moe_cache_free(cache)


def coli_moe_usage_engine_id() -> int:
    return int(load_library().coli_moe_usage_engine_id())


def coli_moe_usage_write(path: str, counts) -> int:
    """counts: int64 array [n_layers][n_experts] (numpy)."""
    import numpy as np
    c = np.ascontiguousarray(counts, dtype=np.int64)
    return _check(load_library().coli_moe_usage_write(path.encode(), c.shape[0], c.shape[1], c.ctypes.data),
                  "coli_moe_usage_write")


def coli_moe_usage_read(path: str, n_layers: int, n_experts: int):
    """Returns (records, counts int64 [n_layers][n_experts])."""
    import numpy as np
    c = np.zeros((n_layers, n_experts), np.int64)
    n = _check(load_library().coli_moe_usage_read(path.encode(), n_layers, n_experts, c.ctypes.data),
               "coli_moe_usage_read")
    return n, c


def coli_moe_test_cache_policy(n_experts, n_slots, reserve, decay, repin_every, pins, calls):
    """The residency policy alone; `calls` is a list of expert lists.
    Returns (repin swaps, misses per call, final slot per expert)."""
    flat = [int(e) for c in calls for e in c]
    lens = [len(c) for c in calls]
    pa = (ctypes.c_int32 * max(1, len(pins)))(*[int(e) for e in pins])
    ca = (ctypes.c_int32 * max(1, len(flat)))(*flat)
    la = (ctypes.c_int32 * max(1, len(lens)))(*lens)
    miss = (ctypes.c_int32 * max(1, len(calls)))()
    slots = (ctypes.c_int32 * n_experts)()
    rc = _check(load_library().coli_moe_test_cache_policy(n_experts, n_slots, reserve, decay, repin_every, pa,
                                                          len(pins), ca, la, len(calls), miss, slots),
                "coli_moe_test_cache_policy")
    return rc, [int(miss[i]) for i in range(len(calls))], [int(v) for v in slots]


def coli_moe_rmsnorm(args: coli_moe_rmsnorm_t, stream: int = 0) -> int:
    return _check(load_library().coli_moe_rmsnorm(args, stream), "coli_moe_rmsnorm")


def coli_moe_linear(args: coli_moe_linear_t, stream: int = 0) -> int:
    return _check(load_library().coli_moe_linear(args, stream), "coli_moe_linear")


def coli_moe_balance_workspace_bytes(tokens: int, n_experts: int, n_seqs: int) -> int:
    return int(load_library().coli_moe_balance_workspace_bytes(int(tokens), int(n_experts), int(n_seqs)))


def coli_moe_balance(args: coli_moe_balance_t, loss: int, counts: int, coef: int, workspace: int,
                     workspace_bytes: int, stream: int = 0) -> int:
    return _check(load_library().coli_moe_balance(args, loss, counts, coef, workspace, workspace_bytes, stream),
                  "coli_moe_balance")


def coli_moe_balance_grad(args: coli_moe_balance_t, coef: int, dloss, dlogits: int, dlogits_stride: int,
                          stream: int = 0) -> int:
    return _check(load_library().coli_moe_balance_grad(args, coef, dloss, dlogits, dlogits_stride, stream),
                  "coli_moe_balance_grad")


def coli_moe_last_logits(handle, logits: int, stream: int = 0) -> int:
    return _check(load_library().coli_moe_last_logits(handle, logits, stream), "coli_moe_last_logits")


# ---------------------------------------------------------------------------
# The operators around the layer on torch device tensors.  Work is enqueued on
# the current stream of the tensors' device; results are allocated there
# unless given.  Tensors of other devices, shapes or types than described
# raise ValueError; sizes and alignments that the library refuses raise
# ColiMoeError.  Results carry no autograd history whatever the arguments do;
# tensors written in place are marked as changed, so that a backward pass that
# needs what stood there before raises.
# ---------------------------------------------------------------------------

_DTYPES: dict = {}  # torch dtype -> COLI_MOE_* element type


def _dtype_code(dtype, what: str, bytes_too: bool = False) -> int:
    if not _DTYPES:
        import torch
        _DTYPES.update({torch.float32: COLI_MOE_F32, torch.bfloat16: COLI_MOE_BF16, torch.float16: COLI_MOE_F16,
                        torch.int8: COLI_MOE_INT8, torch.float8_e4m3fn: COLI_MOE_E4M3})
    code = _DTYPES.get(dtype)
    if code is None or (code > COLI_MOE_F16 and not bytes_too):
        raise ValueError(f"{what}: unsupported type {dtype}")
    return code


def _matrix(t, what: str, device, rows=None, cols=None, dtype=None):
    """Checks a 2-D device tensor whose rows are contiguous; its row stride."""
    shape, strides = t.shape, t.stride()
    if len(shape) != 2 or (strides[1] != 1 and shape[1] > 1):
        raise ValueError(f"{what}: expected a 2-D tensor with contiguous rows, got shape {tuple(shape)}, "
                         f"strides {tuple(strides)}")
    if (rows is not None and shape[0] != rows) or (cols is not None and shape[1] != cols):
        raise ValueError(f"{what}: expected shape {(rows, cols)}, got {tuple(shape)}")
    if (shape[0] | shape[1]) >> 31:  # a size is an int32 in the C structs, where it would wrap around
        raise ValueError(f"{what}: at most 2^31 - 1 rows and columns, got shape {tuple(shape)}")
    if t.device != device or (dtype is not None and t.dtype != dtype):
        _refuse_place(t, what, device, dtype)
    return strides[0]


def _vector(t, what: str, device, n: int, dtype=None):
    """Checks a contiguous 1-D device tensor of n elements."""
    if t.dim() != 1 or t.shape[0] != n or not t.is_contiguous():
        raise ValueError(f"{what}: expected {n} contiguous elements, got shape {tuple(t.shape)}, "
                         f"strides {tuple(t.stride())}")
    if t.device != device or (dtype is not None and t.dtype != dtype):
        _refuse_place(t, what, device, dtype)


def _scale_vector(t, what: str, device, n: int):
    """Checks contiguous float32 scales [n] or [n, 1]."""
    import torch
    if t.shape not in ((n,), (n, 1)) or not t.is_contiguous():
        raise ValueError(f"{what}: expected {n} contiguous scales, got shape {tuple(t.shape)}, "
                         f"strides {tuple(t.stride())}")
    if t.device != device or t.dtype != torch.float32:
        _refuse_place(t, what, device, torch.float32)


def _refuse_place(t, what: str, device, dtype):
    if t.device != device:
        raise ValueError(f"{what}: expected a tensor on {device}, got one on {t.device}")
    raise ValueError(f"{what}: expected {dtype}, got {t.dtype}")


def _gpu(t, what: str):
    """The tensor's device, which has to be a GPU."""
    device = t.device
    if device.type != "cuda":
        raise ValueError(f"{what}: expected a tensor on the GPU, got one on {device}")
    return device


def _enqueue(entry: str, device, *args) -> None:
    """Calls a C entry point, whose last argument is the stream, with `device`
    current and on its current stream."""
    import torch
    index = device.index
    call = getattr(_lib or load_library(), entry)
    if torch._C._cuda_getDevice() == index:
        rc = call(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(device):
            rc = call(*args, torch._C._cuda_getCurrentRawStream(index))
    if rc < 0:
        raise ColiMoeError(rc, entry)


def rms_norm(x, weight=None, eps: float = 1e-6, residual=None, residual_out=None, out=None, scales=None,
             out_dtype=None, group: int = 0):
    """Root-mean-square norm of the rows of x [rows, hidden] (float32, bf16 or
    f16), of x + residual if a residual is given; the sum is stored in
    residual_out (default: in the residual itself).

    Returns the normed rows in out_dtype (default: x's type), or for int8 and
    float8_e4m3fn the pair (codes, scales) with scales [rows, 1], or
    [rows, ceil(hidden / group)] for a group of 64 or 128 columns (linear reads
    scales of rows); for other types there are no scales and group is not used.
    Forward only: no gradient goes through it.  coli_moe_rmsnorm in
    include/coli_moe.h gives the formulas."""
    import torch
    written = ()  # the caller's tensors that this call writes
    dev = _gpu(x, "x")
    ldx = _matrix(x, "x", dev)
    rows, hidden = x.shape
    if out_dtype is None:
        out_dtype = x.dtype if out is None else out.dtype
    xt, ot = _dtype_code(x.dtype, "x"), _dtype_code(out_dtype, "out", True)
    if out is None:
        out, ldo = x.new_empty((rows, hidden), dtype=out_dtype), hidden
    else:
        ldo = _matrix(out, "out", dev, rows, hidden, out_dtype)
        written = (out,)
    rt = wt = ldr = ldro = lds = 0
    rp = rop = wp = sp = None
    if residual is not None:
        rt = _dtype_code(residual.dtype, "residual")
        ldr = ldro = _matrix(residual, "residual", dev, rows, hidden)
        rp = rop = residual.data_ptr()
        if residual_out is not None:
            ldro = _matrix(residual_out, "residual_out", dev, rows, hidden, residual.dtype)
            rop = residual_out.data_ptr()
        written += (residual if residual_out is None else residual_out,)
    elif residual_out is not None:
        raise ValueError("residual_out without a residual")
    if weight is not None:
        wt = _dtype_code(weight.dtype, "weight")
        _vector(weight, "weight", dev, hidden)
        wp = weight.data_ptr()
    if ot > COLI_MOE_F16:
        if group not in (0, 64, 128):
            raise ValueError(f"group: 0, 64 or 128, got {group}")
        n = -(-hidden // group) if group else 1
        if scales is None:
            scales, lds = x.new_empty((rows, n), dtype=torch.float32), n
        else:
            lds = _matrix(scales, "scales", dev, rows, n, torch.float32)
            written += (scales,)
        sp = scales.data_ptr()
    else:
        if scales is not None:
            raise ValueError("scales belong to 8-bit outputs")
        group = 0
    if rows and hidden:
        _enqueue("coli_moe_rmsnorm", dev,
                 coli_moe_rmsnorm_t(rows, hidden, xt, rt, wt, ot, group, eps, x.data_ptr(), ldx, rp, ldr, rop, ldro,
                                    wp, out.data_ptr(), ldo, sp, lds))
        if written:
            torch._C._increment_version(written)
    return out if scales is None else (out, scales)


_ACTS = {"none": COLI_MOE_ACT_NONE, "relu": COLI_MOE_ACT_RELU, "silu": COLI_MOE_ACT_SILU, "gelu": COLI_MOE_ACT_GELU,
         "gelu_tanh": COLI_MOE_ACT_GELU_TANH, "swiglu": COLI_MOE_ACT_SWIGLU}


def linear(x, w, x_scale=None, w_scale=None, bias=None, act: str = "none", residual=None, out=None, out_dtype=None):
    """act(x w^T [* x_scale w_scale] + bias) + residual for x [m, k] and w
    [n, k] of one type (bf16, f16, int8 or float8_e4m3fn; 8 bits with float32
    scales per row, [m] or [m, 1] and [n] or [n, 1]).  act is one of none,
    relu, silu, gelu, gelu_tanh and swiglu; for swiglu w, w_scale and bias
    hold the gate rows and then as many up rows, and n is half of w's rows.
    The result [m, n] has out_dtype (float32, bf16 or f16; default: the
    residual's type, else x's, or bf16 for 8 bits), which is also the
    residual's type; out may be the residual.  Forward only: no gradient goes
    through it.  coli_moe_linear in include/coli_moe.h gives the formulas."""
    import torch
    given = out is not None
    dev = _gpu(x, "x")
    ldx = _matrix(x, "x", dev)
    m, k = x.shape
    ldw = _matrix(w, "w", dev, None, k, x.dtype)
    code = _dtype_code(x.dtype, "x", True)
    if code == COLI_MOE_F32:
        raise ValueError("x: unsupported type torch.float32 (bf16, f16, int8 or float8_e4m3fn)")
    if act not in _ACTS:
        raise ValueError(f"act: one of {', '.join(_ACTS)}, got {act!r}")
    n = rows = w.shape[0]
    if act == "swiglu":
        if rows % 2:
            raise ValueError(f"w: an even number of rows for swiglu, got {rows}")
        n = rows // 2
    sxp = swp = bp = rp = None
    bt = ldr = 0
    if code > COLI_MOE_F16:
        if x_scale is None or w_scale is None:
            raise ValueError("x_scale and w_scale: 8-bit rows carry scales")
        _scale_vector(x_scale, "x_scale", dev, m)
        _scale_vector(w_scale, "w_scale", dev, rows)
        sxp, swp = x_scale.data_ptr(), w_scale.data_ptr()
    elif x_scale is not None or w_scale is not None:
        raise ValueError("x_scale, w_scale: only 8-bit rows carry scales")
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else residual.dtype if residual is not None else \
            torch.bfloat16 if code > COLI_MOE_F16 else x.dtype
    ot = _dtype_code(out_dtype, "out")
    if out is None:
        out, ldo = x.new_empty((m, n), dtype=out_dtype), n
    else:
        ldo = _matrix(out, "out", dev, m, n, out_dtype)
    if residual is not None:
        ldr = _matrix(residual, "residual", dev, m, n, out_dtype)
        rp = residual.data_ptr()
    if bias is not None:
        bt = _dtype_code(bias.dtype, "bias")
        _vector(bias, "bias", dev, rows)
        bp = bias.data_ptr()
    if m and n:
        _enqueue("coli_moe_linear", dev,
                 coli_moe_linear_t(m, n, k, code, ot, bt, _ACTS[act], x.data_ptr(), ldx, w.data_ptr(), ldw, sxp, swp,
                                   bp, rp, ldr, out.data_ptr(), ldo))
        if given:
            torch._C._increment_version((out,))
    return out


_SCORES = {"sigmoid": COLI_MOE_SCORES_SIGMOID, "softmax": COLI_MOE_SCORES_SOFTMAX}


def _balance_args(logits, idx, alpha, scores, offsets, mask):
    """(struct, device, tokens, experts, sequences) of checked arguments."""
    import torch
    dev = _gpu(logits, "logits")
    ld = _matrix(logits, "logits", dev, dtype=torch.float32)
    T, E = logits.shape
    if scores not in _SCORES:
        raise ValueError(f"scores: 'sigmoid' or 'softmax', got {scores!r}")
    n_seqs, k, ip, op, mp = 1, 1, None, None, None
    if idx is not None:
        if _matrix(idx, "idx", dev, T, None, torch.int32) != idx.shape[1] and T > 1:
            raise ValueError("idx: expected a contiguous tensor")
        k, ip = idx.shape[1], idx.data_ptr()
    if offsets is not None:
        n_seqs = offsets.numel() - 1
        _vector(offsets, "offsets", dev, n_seqs + 1, torch.int32)
        if n_seqs < 1 or n_seqs >> 31:
            raise ValueError(f"offsets: expected the bounds of 1 to 65536 sequences, got {n_seqs + 1} elements")
        op = offsets.data_ptr()
    if mask is not None:
        if mask.dtype not in (torch.bool, torch.uint8):
            raise ValueError(f"mask: expected bool or uint8, got {mask.dtype}")
        _vector(mask, "mask", dev, T)
        mp = mask.data_ptr()
    a = coli_moe_balance_t(T, E, k, n_seqs, _SCORES[scores], alpha, logits.data_ptr(), ld, ip, op, mp)
    return a, dev, T, E, n_seqs


def _balance_loss(logits, idx, alpha, scores, offsets, mask):
    """(results, enqueue) of a balance_loss call: arguments checked and buffers
    allocated, the launch left to enqueue()."""
    import torch
    a, dev, T, E, S = _balance_args(logits, idx, alpha, scores, offsets, mask)
    loss, coef = logits.new_empty((S,)), logits.new_empty((S, E))
    counts = logits.new_empty((S, E), dtype=torch.int32)
    nbytes = coli_moe_balance_workspace_bytes(T, E, S)
    ws = logits.new_empty(((nbytes + 3) // 4,))

    def enqueue():
        _enqueue("coli_moe_balance", dev, a, loss.data_ptr(), counts.data_ptr(), coef.data_ptr(), ws.data_ptr(), nbytes)
    return (loss, counts, coef), enqueue


def balance_loss(logits, idx, alpha: float, scores: str = "sigmoid", offsets=None, mask=None):
    """Balance loss of router choices idx [T, k] (int32, -1 in dropped slots)
    with logits [T, E] (float32), per sequence: offsets int32 [S + 1] gives
    the sequences' rows (default: one sequence of all tokens), mask [T] the
    valid tokens (default: all).

    Returns (loss [S], counts [S, E] int32, coef [S, E]).  The loss is a number
    without history, also where the logits have one: its gradient comes from
    balance_grad, which takes coef, and
    logits.backward(balance_grad(logits, coef, ...)) carries it to the router.
    coli_moe_balance in include/coli_moe.h gives the formulas."""
    results, enqueue = _balance_loss(logits, idx, alpha, scores, offsets, mask)
    enqueue()
    return results


def balance_grad(logits, coef, dloss=None, scores: str = "sigmoid", offsets=None, mask=None, out=None):
    """Gradient [T, E] of sum_s dloss[s] * loss[s] (dloss default: ones) with
    respect to the logits, from balance_loss's coef and the same logits,
    scores, offsets and mask.  Rows of tokens in no sequence are left as they
    were in `out` (a fresh result holds zeros there)."""
    import torch
    a, dev, T, E, S = _balance_args(logits, None, 0.0, scores, offsets, mask)
    if _matrix(coef, "coef", dev, S, E, torch.float32) != E and S > 1:
        raise ValueError("coef: expected a contiguous tensor")
    if dloss is not None:
        _vector(dloss, "dloss", dev, S, torch.float32)
    given = out is not None
    if out is None:
        out, ldo = (logits.new_empty if offsets is None else logits.new_zeros)((T, E)), E
    else:
        ldo = _matrix(out, "out", dev, T, E, torch.float32)
    _enqueue("coli_moe_balance_grad", dev, a, coef.data_ptr(), None if dloss is None else dloss.data_ptr(),
             out.data_ptr(), ldo)
    if given:
        torch._C._increment_version((out,))
    return out


# ---------------------------------------------------------------------------
# Convenience wrapper over torch device tensors.
# ---------------------------------------------------------------------------

_WEIGHT_KEYS = ("gate_q", "gate_s", "up_q", "up_s", "down_q", "down_s")


COLI_MOE_WEIGHTS_INT4_GS64 = 0
COLI_MOE_WEIGHTS_INT8_ROW = 1


def make_config(hidden, n_experts, top_k, inter, n_shared, routed_scaling_factor, max_tokens,
                prefill_threshold=0, group_size=None, n_group=1,
                weight_format=COLI_MOE_WEIGHTS_INT4_GS64) -> coli_moe_config_t:
    if group_size is None:
        group_size = 0 if weight_format == COLI_MOE_WEIGHTS_INT8_ROW else 64
    return coli_moe_config_t(hidden=hidden, n_experts=n_experts, top_k=top_k, inter=inter, n_shared=n_shared,
                             group_size=group_size, n_group=n_group, max_tokens=max_tokens,
                             prefill_threshold=prefill_threshold,
                             routed_scaling_factor=routed_scaling_factor, weight_format=weight_format)


def _layer_stream(stream: int, device):
    """Context in which a layer's device is current and work goes to its
    `stream`.  Where torch's current stream of that device is another one, the
    layer's first waits for it and it then waits for the layer's, so that
    tensors may be allocated (before the context), made, used and freed on the
    current stream as if all were one stream."""
    import torch
    current = torch.cuda.current_stream(device)
    if current.cuda_stream != stream:
        return _crossing(current, torch.cuda.ExternalStream(stream, device=device))
    # every device's default stream has the handle 0
    return contextlib.nullcontext() if torch._C._cuda_getDevice() == device.index else torch.cuda.device(device)


@contextlib.contextmanager
def _crossing(current, own):
    import torch
    own.wait_stream(current)
    try:
        with torch.cuda.stream(own):
            yield
    finally:
        current.wait_stream(own)


class _RoutedCalls:
    """What a resident and a cached layer have in common beside their forward:
    needs `cfg`, `workspace`, `stream` and `_layer()`.  These calls run on the
    layer's stream; on another current stream they wait for its work, and its
    later work for them (_layer_stream)."""

    def forward_normed(self, x, norm_weight=None, eps: float = 1e-6, residual=None, out=None):
        """The layer on the norm of x (of x + residual, stored in the residual,
        if one is given): forward(rms_norm(x, norm_weight, eps, residual)), on
        the layer's stream.  x and the residual may be float32, bf16 or f16;
        the result is the layer's float32 output, to be added to the residual
        by the next norm.  A call that is refused leaves the residual as it
        was."""
        import torch
        dev, h = self.workspace.device, self.cfg.hidden
        _matrix(x, "x", dev, None, h)
        T, given = x.shape[0], out is not None
        if out is None:
            out = torch.empty((T, h), dtype=torch.float32, device=dev)
        elif _matrix(out, "out", dev, T, h, torch.float32) != h and T > 1:
            raise ValueError("out: expected a contiguous tensor")
        # what the layer would refuse, while the residual is still as it was
        if T > self.cfg.max_tokens:
            raise ColiMoeError(COLI_MOE_ECAPACITY, "forward_normed")
        if not self.handle or out.data_ptr() % 16:
            raise ColiMoeError(COLI_MOE_EARG, "forward_normed")
        hidden = torch.empty((T, h), dtype=torch.float32, device=dev)
        with _layer_stream(self.stream, dev):
            rms_norm(x, norm_weight, eps, residual=residual, out=hidden)
            self.forward(hidden, out)
        if given:
            torch._C._increment_version((out,))
        return out

    def last_logits(self):
        """Router logits [T, E] of the last forward.  Refused (ColiMoeError)
        between a prefetch, which routes into the same arrays, and the next
        forward."""
        import torch
        dev = self.workspace.device
        T = coli_moe_last_routing(self._layer())
        z = torch.empty((T, self.cfg.n_experts), dtype=torch.float32, device=dev)
        with _layer_stream(self.stream, dev):
            if T:
                coli_moe_last_logits(self._layer(), z.data_ptr(), self.stream)
        return z

    def balance(self, alpha: float, scores: str = "sigmoid", offsets=None, mask=None):
        """balance_loss of the last forward's routing: (loss [S], counts
        [S, E], coef [S, E]).  Refused after a prefetch, as last_logits."""
        import torch
        dev = self.workspace.device
        T = coli_moe_last_routing(self._layer())
        z = torch.empty((T, self.cfg.n_experts), dtype=torch.float32, device=dev)
        idx = torch.empty((T, self.cfg.top_k), dtype=torch.int32, device=dev)
        results, enqueue = _balance_loss(z, idx, alpha, scores, offsets, mask)
        with _layer_stream(self.stream, dev):
            if T:
                coli_moe_last_logits(self._layer(), z.data_ptr(), self.stream)
                coli_moe_last_routing(self._layer(), idx.data_ptr(), stream=self.stream)
            enqueue()
        return results


class MoELayer(_RoutedCalls):
    """One layer on the current torch device.

    `tensors` maps names to device tensors: router_w [h,E] f32, sel_bias [E]
    f32 (optional), gate_q/up_q [E,I,h/2] u8, gate_s/up_s [E,I,h/64] f32,
    down_q [E,h,I/2] u8, down_s [E,h,I/64] f32, and sh_* for the shared
    expert.  The tensors are borrowed: keep them alive with the layer.
    """

    def __init__(self, cfg: coli_moe_config_t, tensors: dict, stream: int | None = None):
        import torch
        self.cfg = cfg
        self.tensors = tensors
        w = coli_moe_weights_t()
        for name, _ in coli_moe_weights_t._fields_:
            t = tensors.get(name)
            setattr(w, name, None if t is None else t.data_ptr())
        self.weights = w
        nbytes = coli_moe_workspace_bytes(cfg)
        if nbytes == 0:
            raise ColiMoeError(COLI_MOE_EARG, "coli_moe_workspace_bytes")
        dev = tensors["router_w"].device
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        self.stream = torch.cuda.current_stream(dev).cuda_stream if stream is None else stream
        self.handle = coli_moe_init(cfg, w, self.workspace.data_ptr(), nbytes, self.stream)

    def forward(self, hidden, out=None):
        import torch
        T = hidden.shape[0]
        if out is None:
            out = torch.empty_like(hidden)
        coli_moe_forward(self.handle, hidden.data_ptr(), out.data_ptr(), T, self.stream)
        return out

    __call__ = forward

    def _layer(self):
        return self.handle

    def set_routing(self, k_use: int | None = None, top_p: float = 1.0):
        """Lossy run-time routing limits for later forwards (warns when they
        change the routing); no arguments restore the plain routing."""
        k_use = self.cfg.top_k if k_use is None else int(k_use)
        coli_moe_set_routing(self.handle, k_use, top_p)
        _warn_lossy(k_use, self.cfg.top_k, top_p)

    def status(self) -> int:
        """Waits for the layer's stream; COLI_MOE_OK unless a launch since the
        last check gave up its bounded wait (COLI_MOE_EDEVICE).  Clears the
        error word."""
        return int(load_library().coli_moe_status(self.handle, ctypes.c_void_p(self.stream)))

    def last_routing(self):
        """Device tensors of the last forward's routing and dispatch."""
        import torch
        dev = self.workspace.device
        T, k, E = None, self.cfg.top_k, self.cfg.n_experts
        T = coli_moe_last_routing(self.handle, stream=self.stream)
        n = T * k
        i32 = dict(dtype=torch.int32, device=dev)
        r = dict(idx=torch.empty(n, **i32), w=torch.empty(n, dtype=torch.float32, device=dev),
                 offsets=torch.empty(E + 1, **i32), sorted_ids=torch.empty(n, **i32),
                 inv=torch.empty(n, **i32), active=torch.empty(E, **i32), n_active=torch.empty(1, **i32))
        with _layer_stream(self.stream, dev):
            coli_moe_last_routing(self.handle, *(r[key].data_ptr() for key in
                                                 ("idx", "w", "offsets", "sorted_ids", "inv", "active",
                                                  "n_active")), stream=self.stream)
        return T, r

    def close(self):
        if getattr(self, "handle", None) is not None:
            coli_moe_free(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class ExpertCache(_RoutedCalls):
    """One layer whose routed experts live in pinned host memory, copied on
    demand into `n_slots` HBM slots (torch device tensors hold the slots and
    the workspace).  `resident` maps router_w, sel_bias and sh_* to device
    tensors; `host` maps gate_q ... down_s to pinned host tensors."""

    def __init__(self, cfg: coli_moe_config_t, resident: dict, host: dict, n_slots: int, repin_every: int = 0,
                 decay: float = 0.0, stream: int | None = None):
        import torch
        self.cfg, self.resident, self.host = cfg, resident, host
        dev = resident["router_w"].device
        w = coli_moe_weights_t()
        for name, _ in coli_moe_weights_t._fields_:
            t = resident.get(name)
            setattr(w, name, None if t is None else t.data_ptr())
        hx = coli_moe_host_experts_t()
        for name, _ in coli_moe_host_experts_t._fields_:
            setattr(hx, name, host[name].data_ptr())
        self.weights, self.hx = w, hx
        sb = coli_moe_cache_slot_bytes(cfg, n_slots)
        wb = coli_moe_workspace_bytes(cfg)
        if sb == 0 or wb == 0:
            raise ColiMoeError(COLI_MOE_EARG, "coli_moe_cache_slot_bytes")
        self.slots = torch.empty(sb, dtype=torch.uint8, device=dev)
        self.workspace = torch.empty(wb, dtype=torch.uint8, device=dev)
        self.stream = torch.cuda.current_stream(dev).cuda_stream if stream is None else stream
        cc = coli_moe_cache_config_t(n_slots=n_slots, repin_every=repin_every, decay=decay)
        self.handle = coli_moe_cache_init(cfg, cc, w, hx, self.slots.data_ptr(), sb, self.workspace.data_ptr(), wb,
                                          self.stream)

    def forward(self, hidden, out=None):
        import torch
        if out is None:
            out = torch.empty_like(hidden)
        coli_moe_cache_forward(self.handle, hidden.data_ptr(), out.data_ptr(), hidden.shape[0], self.stream)
        return out

    __call__ = forward

    def _layer(self):
        return coli_moe_cache_layer(self.handle)

    def prefetch(self, hidden, n_predict: int):
        return coli_moe_cache_prefetch(self.handle, hidden.data_ptr(), hidden.shape[0], n_predict, self.stream)

    def pin(self, experts):
        return coli_moe_cache_pin(self.handle, experts, self.stream)

    def stats(self) -> dict:
        return coli_moe_cache_stats(self.handle)

    def usage(self):
        return coli_moe_cache_usage(self.handle, self.cfg.n_experts)

    def slot_map(self):
        return coli_moe_cache_slots(self.handle, self.cfg.n_experts)

    def set_routing(self, k_use: int | None = None, top_p: float = 1.0):
        """Lossy run-time routing limits of the cached layer (see
        MoELayer.set_routing)."""
        k_use = self.cfg.top_k if k_use is None else int(k_use)
        coli_moe_set_routing(coli_moe_cache_layer(self.handle), k_use, top_p)
        _warn_lossy(k_use, self.cfg.top_k, top_p)

    def last_routing(self):
        """Device tensors of the last forward's routing and dispatch."""
        import torch
        layer = coli_moe_cache_layer(self.handle)
        dev = self.workspace.device
        k, E = self.cfg.top_k, self.cfg.n_experts
        T = coli_moe_last_routing(layer, stream=self.stream)
        n = T * k
        i32 = dict(dtype=torch.int32, device=dev)
        r = dict(idx=torch.empty(n, **i32), w=torch.empty(n, dtype=torch.float32, device=dev),
                 offsets=torch.empty(E + 1, **i32), sorted_ids=torch.empty(n, **i32),
                 inv=torch.empty(n, **i32), active=torch.empty(E, **i32), n_active=torch.empty(1, **i32))
        with _layer_stream(self.stream, dev):
            coli_moe_last_routing(layer, *(r[key].data_ptr() for key in
                                           ("idx", "w", "offsets", "sorted_ids", "inv", "active", "n_active")),
                                  stream=self.stream)
        return T, r

    def close(self):
        if getattr(self, "handle", None) is not None:
            coli_moe_cache_free(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
