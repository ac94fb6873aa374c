"""Thin Python binding of the C ABI in include/fs.h (argument marshalling only).

Every step of the decode path runs inside ``_build/libfs.so``; this module
only converts Python/numpy/torch arguments to pointers and sizes. If the
library is missing the import of any entry point raises: there is no
fallback implementation.
"""
from __future__ import annotations

import ctypes as C
import os

import numpy as np

from . import build as _build

FS_OK = 0
ERRORS = {-1: "FS_ERR_ARG", -2: "FS_ERR_LANE", -3: "FS_ERR_DUP_LANE",
          -4: "FS_ERR_POSITION", -5: "FS_ERR_TOKEN", -6: "FS_ERR_KV_FULL",
          -7: "FS_ERR_OOM", -8: "FS_ERR_CUDA", -9: "FS_ERR_STATE",
          -10: "FS_ERR_DEVICE", -11: "FS_ERR_SCRATCH", -12: "FS_ERR_QUEUE_FULL",
          -13: "FS_ERR_KV_BUDGET"}
CODES = {v: k for k, v in ERRORS.items()}
FS_DTYPE_F32, FS_DTYPE_BF16, FS_DTYPE_Q8_0, FS_DTYPE_Q8_ROW = 0, 1, 2, 3


class FsError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{ERRORS.get(code, code)}: {msg}")
        self.code = code
        self.name = ERRORS.get(code, str(code))


class fs_model_desc(C.Structure):
    _fields_ = [("n_layers", C.c_int32), ("d_model", C.c_int32),
                ("n_heads", C.c_int32), ("n_kv_heads", C.c_int32),
                ("head_dim", C.c_int32), ("d_ffn", C.c_int32),
                ("vocab", C.c_int32), ("rms_eps", C.c_float),
                ("rope_theta", C.c_double), ("tied_embeddings", C.c_int32),
                ("weight_dtype", C.c_int32), ("kv_dtype", C.c_int32),
                ("max_lanes", C.c_int32), ("page_size", C.c_int32),
                ("n_pages", C.c_int32), ("max_pos", C.c_int32),
                ("act_split", C.c_int32)]


class fs_layer_weights(C.Structure):
    _fields_ = [(k, C.c_void_p) for k in ("wq", "wk", "wv", "wo", "w_gate",
                                          "w_up", "w_down", "attn_norm",
                                          "ffn_norm")]


class fs_weights(C.Structure):
    _fields_ = [("embed", C.c_void_p), ("lm_head", C.c_void_p),
                ("final_norm", C.c_void_p),
                ("layers", C.POINTER(fs_layer_weights))]


class fs_sched_config(C.Structure):
    _fields_ = [("lanes", C.c_int32), ("max_prefill_tokens_per_tick", C.c_int32),
                ("max_queue", C.c_int32), ("prefill_chunk", C.c_int32),
                ("kv_budget_tokens", C.c_int64), ("prefix_reuse_min", C.c_int32)]


class fs_job(C.Structure):
    _fields_ = [("prompt", C.c_void_p), ("prompt_len", C.c_int32),
                ("max_new_tokens", C.c_int32), ("temperature", C.c_float),
                ("seed", C.c_uint64), ("stop_token", C.c_int32)]


class fs_sched_stats(C.Structure):
    _fields_ = [("steps", C.c_int64), ("prefill_tokens", C.c_int64),
                ("decode_tokens", C.c_int64), ("jobs_submitted", C.c_int64),
                ("jobs_done", C.c_int64), ("rejected", C.c_int64),
                ("active", C.c_int32), ("queued", C.c_int32),
                ("occupancy_last", C.c_int32), ("occupancy_max", C.c_int32),
                ("occupancy_avg", C.c_double),
                ("rejected_queue_full", C.c_int64), ("rejected_kv_budget", C.c_int64),
                ("kv_reserved_tokens", C.c_int64), ("kv_reserved_max", C.c_int64),
                ("kv_budget_tokens", C.c_int64), ("kv_wait_steps", C.c_int64),
                ("seconds", C.c_double), ("prefill_tok_s", C.c_double),
                ("decode_tok_s", C.c_double),
                ("prefix_hits", C.c_int64), ("prefix_tokens", C.c_int64),
                ("jobs_cancelled", C.c_int64)]


class fs_kv_q8(C.Structure):
    _fields_ = [("k", C.c_void_p), ("v", C.c_void_p), ("k_scale", C.c_void_p),
                ("v_scale", C.c_void_p), ("page_table", C.c_void_p),
                ("n_pages", C.c_int32), ("n_kv_heads", C.c_int32),
                ("page_size", C.c_int32), ("head_dim", C.c_int32),
                ("n_lanes", C.c_int32), ("max_pages", C.c_int32)]


class fs_rope_scaling(C.Structure):
    _fields_ = [("kind", C.c_int32), ("original", C.c_int32), ("factor", C.c_double),
                ("low", C.c_double), ("high", C.c_double)]


LIB_PATH = _build.LIB
_lib = None


def lib():
    """Loads libfs.so (built by ``build.build()``); raises if it is absent."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"CUDA library not built: {LIB_PATH} is missing "
                          "(run __graft_entry__.build())")
    L = C.CDLL(LIB_PATH)
    p, i32, i64, u64 = C.c_void_p, C.c_int32, C.c_int64, C.c_uint64
    f32, kv8 = C.c_float, C.POINTER(fs_kv_q8)
    sig = {
        "fs_create": (C.c_int, [C.POINTER(fs_model_desc),
                                C.POINTER(fs_weights), C.POINTER(p)]),
        "fs_destroy": (C.c_int, [p]),
        "fs_last_error": (C.c_char_p, [p]),
        "fs_set_stream": (C.c_int, [p, p]),
        "fs_lane_reset": (C.c_int, [p, i32]),
        "fs_lane_clone": (C.c_int, [p, i32, i32]),
        "fs_trace_enable": (C.c_int, [p, i64]),
        "fs_selftest_bounded_wait": (C.c_int, [p, i32, p]),
        "fs_trace_read": (C.c_int, [p, p, i64, p, C.c_int]),
        "fs_lane_evict": (C.c_int, [p, i32, i32, i32]),
        "fs_decode_step_batch": (C.c_int, [p, p, p, p, i32, p]),
        "fs_step_batch_chunked": (C.c_int, [p, p, p, p, i32, p]),
        "fs_decode_step_greedy": (C.c_int, [p, p, p, p, i32, p]),
        "fs_sample": (C.c_int, [p, i32, p, p, p, p]),
        "fs_lane_length": (C.c_int, [p, i32, p]),
        "fs_lane_pages": (C.c_int, [p, i32, p, i32, p]),
        "fs_lane_export_kv": (C.c_int, [p, i32, i32, p, p]),
        "fs_lane_import_kv": (C.c_int, [p, i32, p, p, i32]),
        "fs_lane_fill_random_kv": (C.c_int, [p, i32, i32, u64]),
        "fs_quantize_q8_0": (C.c_int, [p, i64, p, p]),
        "fs_sample_device": (C.c_int, [p, i32, p, p, p, p]),
        "fs_profile_enable": (C.c_int, [p, i32]),
        "fs_profile_read": (C.c_int, [p, i32, p, p, p]),
        "fs_kernel_launches": (C.c_int, [p, p]),
        "fs_gemm_path": (C.c_char_p, [p]),
        "fs_gemm_plan": (C.c_int, [i64, i64, i32, i32, i32, i32, p]),
        "fs_lane_capacity": (C.c_int, [p, p]),
        "fs_attention_path": (C.c_char_p, [p]),
        "fs_device_error": (C.c_int, [p, p]),
        "fs_copy_logits": (C.c_int, [p, p]),
        "fs_gemm_bf16_noalloc": (C.c_int, [p, i32, i32, p, i32, p, i32, p]),
        "fs_sched_create": (C.c_int, [p, C.POINTER(fs_sched_config), C.POINTER(p)]),
        "fs_sched_create_model_free": (C.c_int, [C.POINTER(fs_sched_config), i32,
                                                 C.POINTER(p)]),
        "fs_sched_destroy": (C.c_int, [p]),
        "fs_sched_submit": (C.c_int, [p, C.POINTER(fs_job), p]),
        "fs_sched_step": (C.c_int, [p, p]),
        "fs_sched_run": (C.c_int, [p, i64, p]),
        "fs_sched_take": (C.c_int, [p, i64, p, i32, p]),
        "fs_sched_get_stats": (C.c_int, [p, C.POINTER(fs_sched_stats)]),
        "fs_sched_status": (C.c_int, [p, i64, p]),
        "fs_sched_cancel": (C.c_int, [p, i64]),
        "fs_sched_last_batch": (C.c_int, [p, p, i32, p]),
        "fs_sched_last_error": (C.c_char_p, [p]),
        "fs_sched_model_free_fail_resets": (C.c_int, [p, i32]),
        "fs_kv_q8_append": (C.c_int, [kv8, p, p, i64, i64, i32, p, p, i32, p, p, i32, p]),
        "fs_kv_q8_read": (C.c_int, [kv8, p, p, i32, p, p, i64, i64, i32, p]),
        "fs_kv_q8_attention_workspace": (i64, [kv8, i32, i32, i32, i32]),
        "fs_kv_q8_attention": (C.c_int, [kv8, p, i64, p, p, i32, i32, i32, f32, p, p, i32, p, i64,
                                         i32, i32, p, i64, p]),
        "fs_verify_draft": (C.c_int, [p, i64, i32, i32, p, i32, p, p, i64, p, p, p, p, p, p]),
        "fs_pages_update": (C.c_int, [p, i32, p, p, i32, i32, i32, p, p, p, p, p, p, p, i32, p, p]),
        "fs_rope_frequencies": (C.c_int, [i32, C.c_double, C.POINTER(fs_rope_scaling), p, p]),
        "fs_rope": (C.c_int, [p, i64, i32, p, i64, i32, i32, i32, i32, p, p, i32, C.c_double, i32, p,
                              i64, p, i64, p]),
        "fs_lora_add": (C.c_int, [p, i64, i32, p, i32, i32, i32, p, p, p, i32, i32, p, i64, p, i64,
                                  i32, p]),
        "fs_sample_filtered": (C.c_int, [p, i64, i32, i32, p, p, p, p, p, p, p, p]),
        "fs_gemm_bf16": (C.c_int, [p, i32, i32, p, i32, p, i32, i32, p]),
        "fs_gemm_bf16_width": (C.c_int, [p, i32, i32, p, i32, p, i32, p]),
        "fs_gemm_bf16_time": (C.c_int, [p, i32, i32, p, i32, p, i32, i32, p, p]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    _lib = L
    return L


def exported_symbols() -> list:
    """Names of the entry points declared in include/fs.h."""
    return ["fs_create", "fs_destroy", "fs_last_error", "fs_set_stream",
            "fs_lane_reset", "fs_lane_clone", "fs_lane_evict", "fs_trace_enable", "fs_trace_read", "fs_selftest_bounded_wait", "fs_decode_step_batch", "fs_step_batch_chunked", "fs_decode_step_greedy", "fs_sample",
            "fs_lane_length", "fs_lane_pages", "fs_lane_export_kv",
            "fs_lane_import_kv", "fs_lane_fill_random_kv", "fs_quantize_q8_0",
            "fs_kernel_launches", "fs_gemm_path", "fs_gemm_plan", "fs_lane_capacity", "fs_attention_path", "fs_sample_device",
            "fs_profile_enable", "fs_profile_read", "fs_device_error",
            "fs_kv_q8_append", "fs_kv_q8_read", "fs_kv_q8_attention_workspace",
            "fs_kv_q8_attention", "fs_verify_draft",
            "fs_pages_update", "fs_rope_frequencies", "fs_rope", "fs_lora_add",
            "fs_sample_filtered",
            "fs_gemm_bf16", "fs_gemm_bf16_width", "fs_gemm_bf16_time", "fs_copy_logits", "fs_gemm_bf16_noalloc",
            "fs_sched_create", "fs_sched_create_model_free", "fs_sched_destroy",
            "fs_sched_submit", "fs_sched_step", "fs_sched_run", "fs_sched_take",
            "fs_sched_get_stats", "fs_sched_status", "fs_sched_cancel", "fs_sched_last_batch",
            "fs_sched_last_error", "fs_sched_model_free_fail_resets"]


def _check(h, rc: int) -> None:
    if rc != FS_OK:
        msg = lib().fs_last_error(h)
        raise FsError(rc, msg.decode() if msg else "")


def _i32(a) -> np.ndarray:
    return np.ascontiguousarray(np.asarray(a, dtype=np.int32))


def _ptr(a: np.ndarray):
    return a.ctypes.data_as(C.c_void_p)


def _dptr(x):
    """Address of a host numpy array, a torch tensor (host or device) or None."""
    if x is None:
        return None
    if isinstance(x, np.ndarray):
        assert x.flags["C_CONTIGUOUS"]
        return x.ctypes.data
    if hasattr(x, "data_ptr"):
        assert x.is_contiguous()
        return x.data_ptr()
    return int(x)


def make_desc(cfg: dict, weight_dtype: int, kv_dtype: int, max_lanes: int,
              n_pages: int, max_pos: int, page_size: int = 16,
              act_split: int = 0) -> fs_model_desc:
    return fs_model_desc(cfg["L"], cfg["d"], cfg["H"], cfg["Hkv"], cfg["hd"],
                         cfg["F"], cfg["V"], cfg["rms_eps"], cfg["rope_theta"],
                         1 if cfg["tied"] else 0, weight_dtype, kv_dtype,
                         max_lanes, page_size, n_pages, max_pos, act_split)


LAYER_KEYS = ("wq", "wk", "wv", "wo", "w_gate", "w_up", "w_down",
              "attn_norm", "ffn_norm")


def fs_create(desc: fs_model_desc, weights: dict):
    """weights: dict of host numpy arrays or torch tensors (host or device):
    embed, lm_head (or None), final_norm, layers[list of LAYER_KEYS dicts]."""
    layers = (fs_layer_weights * len(weights["layers"]))()
    for i, ly in enumerate(weights["layers"]):
        for k in LAYER_KEYS:
            setattr(layers[i], k, _dptr(ly[k]))
    w = fs_weights(_dptr(weights["embed"]), _dptr(weights.get("lm_head")),
                   _dptr(weights["final_norm"]), layers)
    h = C.c_void_p()
    _check(None, lib().fs_create(C.byref(desc), C.byref(w), C.byref(h)))
    return h


def fs_destroy(h) -> None:
    lib().fs_destroy(h)


def fs_last_error(h) -> str:
    m = lib().fs_last_error(h)
    return m.decode() if m else ""


def fs_set_stream(h, stream) -> None:
    """stream: a torch.cuda.Stream, a raw cudaStream_t int, or None."""
    raw = getattr(stream, "cuda_stream", stream)
    _check(h, lib().fs_set_stream(h, raw))


def fs_lane_reset(h, lane: int) -> None:
    _check(h, lib().fs_lane_reset(h, int(lane)))


TRACE_TAGS = {1: "embed", 2: "rmsnorm", 3: "sample", 4: "argmax_tiles",
              5: "attn_mma", 6: "attn_tma", 7: "attn_tiled", 8: "attn_warp",
              9: "rope_append", 10: "gemv", 11: "attn_partial", 12: "attn_combine",
              13: "gemv_swiglu", 14: "kv_q8_append", 15: "attn_q8",
              16: "gemm_store", 17: "gemm_resid",
              18: "gemm_swiglu", 19: "gemm_argmax", 20: "attn_q8_join"}


def fs_trace_enable(h, capacity: int) -> None:
    """Kernel timeline tracing into a device buffer of ``capacity`` records
    (0 turns it off)."""
    _check(h, lib().fs_trace_enable(h, int(capacity)))


def fs_trace_read(h, reset: bool = True):
    """Returns (records [n, 4] uint64, appended count)."""
    n = C.c_int64()
    _check(h, lib().fs_trace_read(h, None, 0, C.byref(n), 0))
    out = np.zeros((max(1, n.value), 4), dtype=np.uint64)
    _check(h, lib().fs_trace_read(h, _ptr(out), n.value, C.byref(n), int(bool(reset))))
    return out[:min(n.value, out.shape[0])], n.value


def fs_lane_clone(h, src: int, dst: int) -> None:
    """Empty lane ``dst`` takes lane ``src``'s history (full pages shared,
    the partial last page copied)."""
    _check(h, lib().fs_lane_clone(h, int(src), int(dst)))


def fs_lane_evict(h, lane: int, start: int, end: int) -> None:
    """Positions [start, end) leave the lane; later entries move down, their
    keys rotated back by end - start positions."""
    _check(h, lib().fs_lane_evict(h, int(lane), int(start), int(end)))


def fs_decode_step_batch(h, lanes, positions, tokens, logits_out=None):
    """Advances lanes by one token. ``positions`` (np.int32) is incremented
    in place on success and returned. logits_out: torch CUDA f32 [n, V]."""
    la = _i32(lanes)
    to = _i32(tokens)
    if (isinstance(positions, np.ndarray) and positions.dtype == np.int32
            and positions.flags["C_CONTIGUOUS"]):
        po = positions
    else:
        po = _i32(positions)
    n = la.size
    assert po.size == n and to.size == n
    _check(h, lib().fs_decode_step_batch(h, _ptr(la), _ptr(po), _ptr(to), n,
                                         _dptr(logits_out)))
    return po


def fs_decode_step_greedy(h, lanes, positions, tokens, tokens_out=None):
    """Decode step + greedy token per lane without materialising logits.
    tokens_out: torch CUDA int32 [n] (no synchronisation) or None for a host
    numpy array. ``positions`` (np.int32) is incremented in place."""
    la = _i32(lanes)
    to = _i32(tokens)
    if (isinstance(positions, np.ndarray) and positions.dtype == np.int32
            and positions.flags["C_CONTIGUOUS"]):
        po = positions
    else:
        po = _i32(positions)
    n = la.size
    assert po.size == n and to.size == n
    host = tokens_out is None
    out = np.empty(n, dtype=np.int32) if host else tokens_out
    _check(h, lib().fs_decode_step_greedy(h, _ptr(la), _ptr(po), _ptr(to), n,
                                          _ptr(out) if host else _dptr(out)))
    return out


def fs_step_batch_chunked(h, lanes, positions, tokens, logits_out=None):
    """Chunked prefill step: a lane may appear on several rows at its next
    consecutive positions. ``positions`` (np.int32) is incremented in place
    on success and returned. logits_out: torch CUDA f32 [n, V]."""
    la = _i32(lanes)
    to = _i32(tokens)
    if (isinstance(positions, np.ndarray) and positions.dtype == np.int32
            and positions.flags["C_CONTIGUOUS"]):
        po = positions
    else:
        po = _i32(positions)
    n = la.size
    assert po.size == n and to.size == n
    _check(h, lib().fs_step_batch_chunked(h, _ptr(la), _ptr(po), _ptr(to), n,
                                          _dptr(logits_out)))
    return po


def fs_sample(h, temps, seeds, counters) -> np.ndarray:
    t = np.ascontiguousarray(np.asarray(temps, dtype=np.float32))
    s = np.ascontiguousarray(np.asarray(seeds, dtype=np.uint64))
    c = np.ascontiguousarray(np.asarray(counters, dtype=np.uint64))
    out = np.empty(t.size, dtype=np.int32)
    _check(h, lib().fs_sample(h, t.size, _ptr(t), _ptr(s), _ptr(c), _ptr(out)))
    return out


def fs_sample_device(h, temps, seeds, counters, tokens_out) -> None:
    """All four are torch CUDA tensors (f32, int64/uint64, int64/uint64,
    int32) of n entries; no synchronisation."""
    _check(h, lib().fs_sample_device(h, tokens_out.numel(), _dptr(temps),
                                     _dptr(seeds), _dptr(counters),
                                     _dptr(tokens_out)))


FS_PROF_GEMM, FS_PROF_ATTN, FS_PROF_OTHER = 0, 1, 2


def fs_profile_enable(h, enable: bool) -> None:
    _check(h, lib().fs_profile_enable(h, 1 if enable else 0))


def fs_profile_read(h, cls: int):
    """(ms, launches, algorithmic bytes) of kernel class `cls` since the
    last read."""
    ms, n, b = C.c_double(), C.c_int64(), C.c_double()
    _check(h, lib().fs_profile_read(h, int(cls), C.byref(ms), C.byref(n),
                                    C.byref(b)))
    return ms.value, n.value, b.value


def fs_lane_length(h, lane: int) -> int:
    v = C.c_int32()
    _check(h, lib().fs_lane_length(h, int(lane), C.byref(v)))
    return v.value


def fs_lane_pages(h, lane: int) -> list:
    n = C.c_int32()
    _check(h, lib().fs_lane_pages(h, int(lane), None, 0, C.byref(n)))
    out = np.empty(max(1, n.value), dtype=np.int32)
    _check(h, lib().fs_lane_pages(h, int(lane), _ptr(out), n.value, C.byref(n)))
    return out[:n.value].tolist()


def fs_lane_export_kv(h, lane: int, layer: int, Hkv: int, hd: int):
    n = fs_lane_length(h, lane)
    k = np.empty((n, Hkv, hd), dtype=np.float32)
    v = np.empty((n, Hkv, hd), dtype=np.float32)
    _check(h, lib().fs_lane_export_kv(h, int(lane), int(layer), _ptr(k), _ptr(v)))
    return k, v


def fs_lane_import_kv(h, lane: int, k: np.ndarray, v: np.ndarray) -> None:
    """k, v: f32 [n_layers, n, Hkv, hd] (K already rotated)."""
    k = np.ascontiguousarray(k, dtype=np.float32)
    v = np.ascontiguousarray(v, dtype=np.float32)
    _check(h, lib().fs_lane_import_kv(h, int(lane), _ptr(k), _ptr(v),
                                      k.shape[1]))


def fs_lane_fill_random_kv(h, lane: int, n: int, seed: int) -> None:
    _check(h, lib().fs_lane_fill_random_kv(h, int(lane), int(n), int(seed)))


def fs_quantize_q8_0(src, blocks_out, stream=None) -> None:
    """src: torch CUDA f32 tensor; blocks_out: torch CUDA uint8 [n/32, 34]."""
    raw = getattr(stream, "cuda_stream", stream)
    rc = lib().fs_quantize_q8_0(_dptr(src), src.numel(), _dptr(blocks_out), raw)
    if rc != FS_OK:
        raise FsError(rc, "fs_quantize_q8_0 failed")


def fs_kernel_launches(h) -> int:
    v = C.c_int64()
    _check(h, lib().fs_kernel_launches(h, C.byref(v)))
    return v.value


def fs_gemm_path(h) -> str:
    return lib().fs_gemm_path(h).decode()


PLAN_KEYS = ("P", "lanes_per_group", "groups", "tmem_cols", "q8_copy_kept",
             "q8_copy_used", "m_tiles", "k_blocks")


def fs_gemm_plan(n_rows: int, k_inputs: int, max_lanes: int, n: int, sms: int,
                 weight_dtype: int) -> dict:
    """The tcgen05 GEMM's work split for one matrix and call (host only)."""
    out = (C.c_int32 * 8)()
    _check(None, lib().fs_gemm_plan(n_rows, k_inputs, max_lanes, n, sms, weight_dtype, out))
    return dict(zip(PLAN_KEYS, [int(v) for v in out]))


def fs_attention_path(h) -> str:
    return lib().fs_attention_path(h).decode()


def fs_device_error(h) -> int:
    v = C.c_int32()
    _check(h, lib().fs_device_error(h, C.byref(v)))
    return v.value


def fs_selftest_bounded_wait(h, timeout_us: int = 2000) -> int:
    """Failure-detection check: a kernel's bounded wait on a barrier nothing
    arrives on gives up after timeout_us; returns the device error code it
    set (99), which is then cleared."""
    v = C.c_int32()
    _check(h, lib().fs_selftest_bounded_wait(h, int(timeout_us), C.byref(v)))
    return v.value


def fs_gemm_bf16(W, X, Y, splits: int = 1, path: int = 1, stream=None) -> None:
    """Test hook: Y = X @ W^T on the device (torch bf16 W [N, K], X [B, K],
    f32 Y [B, N])."""
    raw = getattr(stream, "cuda_stream", stream)
    N, K = W.shape
    B = X.shape[0]
    rc = lib().fs_gemm_bf16(_dptr(W), N, K, _dptr(X), B, _dptr(Y), splits,
                            path, raw)
    if rc != FS_OK:
        raise FsError(rc, "fs_gemm_bf16 failed")


def fs_gemm_bf16_width(W, X, Y, width: int, stream=None) -> None:
    """Test hook: the tcgen05 GEMM with the stream-K width given directly."""
    raw = getattr(stream, "cuda_stream", stream)
    N, K = W.shape
    B = X.shape[0]
    rc = lib().fs_gemm_bf16_width(_dptr(W), N, K, _dptr(X), B, _dptr(Y), width, raw)
    if rc != FS_OK:
        raise FsError(rc, "fs_gemm_bf16_width failed")


def fs_gemm_bf16_time(W, X, Y, width: int, reps: int = 10, stream=None) -> float:
    """Tuning hook: mean device ms of one tcgen05 GEMM launch with the given
    stream-K width, over `reps` launches each after an L2-evicting memset."""
    raw = getattr(stream, "cuda_stream", stream)
    N, K = W.shape
    B = X.shape[0]
    ms = C.c_double()
    rc = lib().fs_gemm_bf16_time(_dptr(W), N, K, _dptr(X), B, _dptr(Y), width, reps,
                                 C.byref(ms), raw)
    if rc != FS_OK:
        raise FsError(rc, "fs_gemm_bf16_time failed")
    return ms.value


def fs_copy_logits(h, dst) -> None:
    """Copies the last step's logits [n, V] f32 into dst (numpy or torch)."""
    _check(h, lib().fs_copy_logits(h, _dptr(dst)))


def fs_gemm_bf16_noalloc(W, X, Y, splits: int = 1, stream=None) -> None:
    """fs_gemm_bf16 (tcgen05 path) with its workspace in the library's static
    device scratch instead of allocations (see include/fs.h)."""
    raw = getattr(stream, "cuda_stream", stream)
    N, K = W.shape
    B = X.shape[0]
    rc = lib().fs_gemm_bf16_noalloc(_dptr(W), N, K, _dptr(X), B, _dptr(Y),
                                    splits, raw)
    if rc != FS_OK:
        raise FsError(rc, "fs_gemm_bf16_noalloc failed")


# ------------------------------------------------------- 8-bit paged KV cache
# The calls of this section and the next two take CUDA tensors and a stream (a
# torch.cuda.Stream or an address; None: torch's current stream) and return once
# their work is enqueued there. As with any kernel on a stream of the caller's,
# tensors that were made or are freed on another stream are the caller's to order.
class _Types:
    """torch and its types, once torch is there (this module does not import it)."""
    torch = f32 = bf16 = i32 = i64 = u8 = None
    rows = {}  # of rows: FS_DTYPE


def _types():
    if _Types.f32 is None:
        import torch
        _Types.torch = torch
        _Types.bf16, _Types.i32, _Types.u8 = torch.bfloat16, torch.int32, torch.uint8
        _Types.i64 = torch.int64
        _Types.f32 = torch.float32
        _Types.rows = {torch.float32: FS_DTYPE_F32, torch.bfloat16: FS_DTYPE_BF16}
    return _Types


def _refuse(why: str):
    raise FsError(CODES["FS_ERR_ARG"], why)


def _op_check(rc: int) -> None:
    if rc:
        raise FsError(rc, fs_last_error(None))


def _raw(stream, x):
    """Address of the stream: without one, torch's current stream of x's device, as
    torch's own calls take it."""
    if stream is not None:
        return getattr(stream, "cuda_stream", stream)
    device = x.get_device()
    if device < 0:  # host memory, refused by the C call
        return None
    return _types().torch._C._cuda_getCurrentRawStream(device)


def _vec(x, n: int, dtype, what: str):
    """Address of a contiguous tensor of n values (that it is the current
    device's memory the C call checks)."""
    if x.dtype is dtype and x.numel() == n and x.is_contiguous():
        return x.data_ptr()
    _refuse(f"{what}: a contiguous CUDA tensor of {n} {dtype} values is needed")


def _rows(x, n: int, heads: int, hd: int, what: str):
    """(address, row stride, dtype) of n rows [heads, hd], each contiguous."""
    dt = _Types.rows.get(x.dtype)
    if dt is not None and x.shape == (n, heads, hd):
        if x.is_contiguous():
            return x.data_ptr(), heads * hd, dt
        s0, s1, s2 = x.stride()
        if n == 0 or (s2 == 1 and (heads == 1 or s1 == hd)):
            return x.data_ptr(), s0 if n > 1 else heads * hd, dt
    _refuse(f"{what}: a CUDA tensor [{n}, {heads}, {hd}] of f32 or bf16 whose rows are "
            "contiguous is needed")


def _rope_args(rope, hd: int):
    if rope is None:
        return None, None, 0
    cos, sin = rope
    n = cos.shape[0] if cos.dim() == 2 else 0
    if n < 1 or cos.shape != (n, hd // 2) or sin.shape != cos.shape:
        _refuse(f"rope: two tables [rope_len, {hd // 2}] are needed")
    return (_vec(cos, n * (hd // 2), _Types.f32, "rope cos"),
            _vec(sin, n * (hd // 2), _Types.f32, "rope sin"), n)


def fs_kv_q8_view(k, v, k_scale, v_scale, page_table) -> fs_kv_q8:
    """The 8-bit paged cache in the caller's CUDA tensors: codes k, v uint8
    [n_pages, Hkv, page_size, hd], scales f32 [n_pages, Hkv, page_size],
    page_table int32 [n_lanes, max_pages], all contiguous. The view keeps them
    alive; page-table entries may change between calls."""
    if k.dim() != 4 or page_table.dim() != 2:
        _refuse("codes are [n_pages, Hkv, page_size, hd], the page table [n_lanes, max_pages]")
    if v.shape != k.shape or k_scale.shape != k.shape[:3] or v_scale.shape != k.shape[:3]:
        _refuse("v has the shape of k, the scales all but its last dimension")
    if not all(t.is_cuda for t in (k, v, k_scale, v_scale, page_table)):
        _refuse("a cache in CUDA tensors is needed")
    ty = _types()
    n_pages, Hkv, ps, hd = k.shape
    n_lanes, max_pages = page_table.shape
    rows = n_pages * Hkv * ps
    c = fs_kv_q8(_vec(k, rows * hd, ty.u8, "k codes"),
                 _vec(v, rows * hd, ty.u8, "v codes"),
                 _vec(k_scale, rows, ty.f32, "k scales"),
                 _vec(v_scale, rows, ty.f32, "v scales"),
                 _vec(page_table, n_lanes * max_pages, ty.i32, "page table"),
                 n_pages, Hkv, ps, hd, n_lanes, max_pages)
    c.tensors = (k, v, k_scale, v_scale, page_table)
    return c


def fs_kv_q8_append(cache: fs_kv_q8, k, v, lanes, positions, rope=None, stream=None) -> None:
    """Quantises rows k, v [n, Hkv, hd] (f32 or bf16, any row stride) into
    tokens positions[i] of lanes lanes[i] (int32 CUDA vectors); rope: (cos, sin)
    f32 [rope_len, hd / 2] that rotate the keys."""
    ty = _types()
    n = lanes.numel()
    hd = cache.head_dim
    kp, ks, dt = _rows(k, n, cache.n_kv_heads, hd, "k")
    vp, vs, dv = _rows(v, n, cache.n_kv_heads, hd, "v")
    if dt != dv:
        _refuse("k and v have different types")
    rc, rs, rl = _rope_args(rope, hd)
    _op_check(lib().fs_kv_q8_append(C.byref(cache), kp, vp, ks, vs, dt,
                                    _vec(lanes, n, ty.i32, "lanes"),
                                    _vec(positions, n, ty.i32, "positions"), n, rc, rs, rl,
                                    _raw(stream, lanes)))


def fs_kv_q8_read(cache: fs_kv_q8, lanes, positions, k_out=None, v_out=None, stream=None) -> None:
    """Reads tokens back into k_out, v_out [n, Hkv, hd] (f32 or bf16; either
    may be None)."""
    ty = _types()
    n = lanes.numel()
    kp, ks, dt = (None, 0, None) if k_out is None else \
        _rows(k_out, n, cache.n_kv_heads, cache.head_dim, "k_out")
    vp, vs, dv = (None, 0, None) if v_out is None else \
        _rows(v_out, n, cache.n_kv_heads, cache.head_dim, "v_out")
    if dt is not None and dv is not None and dt != dv:
        _refuse("k_out and v_out have different types")
    if dt is None:
        dt = FS_DTYPE_F32 if dv is None else dv
    _op_check(lib().fs_kv_q8_read(C.byref(cache), _vec(lanes, n, ty.i32, "lanes"),
                                  _vec(positions, n, ty.i32, "positions"), n, kp, vp, ks,
                                  vs, dt, _raw(stream, lanes)))


def fs_kv_q8_attention_workspace(cache: fs_kv_q8, n: int, n_heads: int, max_len: int = 0,
                                 split_len: int = 0) -> int:
    """Bytes of workspace fs_kv_q8_attention needs for the same arguments."""
    b = lib().fs_kv_q8_attention_workspace(C.byref(cache), n, n_heads, max_len, split_len)
    if b < 0:
        _op_check(int(b))
    return b


def fs_kv_q8_attention(cache: fs_kv_q8, q, lanes, lengths, out, max_len: int = 0,
                       scale: float | None = None, rope=None, split_len: int = 0,
                       workspace=None, stream=None) -> None:
    """out[i] = attention of q[i] (both [n, H, hd], f32 or bf16) over tokens
    0 .. lengths[i] - 1 of lane lanes[i]. max_len: an upper bound of the lengths;
    scale: 1 / sqrt(hd) by default; rope: (cos, sin) that rotate q by
    lengths[i] - 1; workspace: a CUDA tensor of at least
    fs_kv_q8_attention_workspace bytes, not shared with a call that may run at
    the same time."""
    ty = _types()
    n = lanes.numel()
    hd = cache.head_dim
    H = q.shape[1] if q.dim() == 3 else 0
    qp, qs, dt = _rows(q, n, H, hd, "q")
    op, os_, do = _rows(out, n, H, hd, "out")
    if dt != do:
        _refuse("q and out have different types")
    rc, rs, rl = _rope_args(rope, hd)
    wp, wb = None, 0
    if workspace is not None:
        if not workspace.is_contiguous():
            _refuse("workspace: a contiguous CUDA tensor is needed")
        wp, wb = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    _op_check(lib().fs_kv_q8_attention(
        C.byref(cache), qp, qs, _vec(lanes, n, ty.i32, "lanes"),
        _vec(lengths, n, ty.i32, "lengths"), n, H, max_len,
        hd ** -0.5 if scale is None else scale, rc, rs, rl, op, os_, dt, split_len, wp, wb,
        _raw(stream, lanes)))


# --------------------------------------------------------- draft verification
def fs_verify_draft(logits, row_start, draft, draft_probs, temps, u_accept, u_sample, n_accepted,
                    next_token, stream=None) -> None:
    """Speculative sampling's accept / resample rule (see include/fs.h). logits
    f32 [rows, vocab] (any row stride), row_start int32 [seqs + 1], draft int32
    [rows], draft_probs f32 [rows, vocab] or None, temps and u_sample f32 [seqs],
    u_accept f32 [rows]; n_accepted and next_token int32 [seqs] are written. All
    CUDA tensors."""
    ty = _types()
    if logits.dim() != 2 or logits.dtype is not ty.f32:
        _refuse("logits: a CUDA tensor [rows, vocab] of f32 is needed")
    rows, V = logits.shape
    if draft_probs is not None and (draft_probs.shape != (rows, V) or
                                    draft_probs.dtype is not ty.f32):
        _refuse("draft_probs: a CUDA tensor [rows, vocab] of f32 is needed")
    for t in (logits, draft_probs):
        if t is not None and V > 1 and t.numel() and t.stride(1) != 1:
            _refuse("rows of logits and draft_probs must be contiguous")
    n = temps.numel()
    ld = lambda t: 0 if t is None else t.stride(0) if rows > 1 else V
    _op_check(lib().fs_verify_draft(
        logits.data_ptr(), ld(logits), rows, V,
        _vec(row_start, n + 1, ty.i32, "row_start"), n,
        _vec(draft, rows, ty.i32, "draft"),
        None if draft_probs is None else draft_probs.data_ptr(), ld(draft_probs),
        _vec(temps, n, ty.f32, "temps"),
        _vec(u_accept, rows, ty.f32, "u_accept"),
        _vec(u_sample, n, ty.f32, "u_sample"),
        _vec(n_accepted, n, ty.i32, "n_accepted"),
        _vec(next_token, n, ty.i32, "next_token"),
        _raw(stream, temps)))


# ------------------------------------ what differs from request to request
def _or_none(x, n: int, dtype, what: str):
    return None if x is None else _vec(x, n, dtype, what)


def fs_pages_update(holders, page_table, lengths, grow, page_size: int, status, keep=None,
                    row_start=None, row_lane=None, row_position=None, row_length=None,
                    row_slot=None, max_rows: int | None = None, stream=None) -> None:
    """Lanes keep keep[l] tokens (all without it) and take grow[l] new ones; pages are
    let go and taken, and each new token gets its row (see include/fs.h). int32 CUDA
    tensors, contiguous: holders [n_pages], page_table [n_lanes, max_pages], lengths,
    keep, grow [n_lanes], row_start [n_lanes + 1], status [4]; row_lane, row_position,
    row_length int32 and row_slot int64 [max_rows], each or None. max_rows: the rows'
    length where none of the four is given."""
    ty = _types()
    shape = page_table.shape
    if len(shape) != 2:
        _refuse("the page table is [n_lanes, max_pages]")
    n, wide = shape
    if row_start is None:
        _refuse(f"row_start: a contiguous CUDA tensor of {n + 1} values is needed")
    m = max_rows
    if m is None:
        rows = [t for t in (row_lane, row_position, row_length, row_slot) if t is not None]
        m = rows[0].numel() if rows else 0
    n_pages = holders.numel()
    _op_check(lib().fs_pages_update(
        _vec(holders, n_pages, ty.i32, "holders"), n_pages,
        _vec(page_table, n * wide, ty.i32, "page table"), _vec(lengths, n, ty.i32, "lengths"), n,
        wide, page_size, _or_none(keep, n, ty.i32, "keep"), _vec(grow, n, ty.i32, "grow"),
        _vec(row_start, n + 1, ty.i32, "row_start"), _or_none(row_lane, m, ty.i32, "row_lane"),
        _or_none(row_position, m, ty.i32, "row_position"),
        _or_none(row_length, m, ty.i32, "row_length"), _or_none(row_slot, m, ty.i64, "row_slot"),
        m, _vec(status, 4, ty.i32, "status"), _raw(stream, lengths)))


ROPE_SCALINGS = {"none": 0, "linear": 1, "base": 2, "ramp": 3, "bands": 4}


def fs_rope_frequencies(rotary_dim: int, theta: float = 10000.0, scaling: dict | None = None):
    """(angles a position of the rotary_dim / 2 pairs as f64, factor of the turned values)
    for fs_rope. scaling: {"kind": "linear" | "base", "factor"}, {"kind": "ramp", "factor",
    "original", "beta_fast" (32), "beta_slow" (1)} or {"kind": "bands", "factor",
    "original", "low" (1), "high" (4)}; see include/fs.h."""
    c = None
    if scaling is not None:
        s = dict(scaling)
        kind = s.pop("kind", None)
        if kind not in ROPE_SCALINGS:
            _refuse(f"scaling: kind is one of {', '.join(ROPE_SCALINGS)}")
        c = fs_rope_scaling(ROPE_SCALINGS[kind], 0, float(s.pop("factor", 1.0)), 0.0, 0.0)
        if kind in ("ramp", "bands"):
            c.original = int(s.pop("original", 0))
            names = ("beta_slow", "beta_fast", 1.0, 32.0) if kind == "ramp" else ("low", "high", 1.0, 4.0)
            c.low, c.high = float(s.pop(names[0], names[2])), float(s.pop(names[1], names[3]))
        if s:
            _refuse(f"scaling: {kind} has no {', '.join(s)}")
    f = np.empty(max(0, rotary_dim // 2), np.float64)
    m = C.c_double()
    _op_check(lib().fs_rope_frequencies(rotary_dim, theta, None if c is None else C.byref(c),
                                        f.ctypes.data, C.byref(m)))
    return f, m.value


def fs_rope(q, positions, inv_freq, k=None, q_out=None, k_out=None, interleaved: bool = False,
            factor: float = 1.0, inverse: bool = False, stream=None) -> None:
    """Turns the first 2 * len(inv_freq) values of each head of q [n, H, hd] and k
    [n, Hkv, hd] (f32 or bf16 CUDA tensors, any row stride) by positions (int32 [n]; a
    negative one skips its row). inv_freq and factor from fs_rope_frequencies (inv_freq: a
    host array of f64). Without q_out / k_out in place."""
    ty = _types()
    n = positions.numel()
    shape, k_shape = q.shape, (0, 0, 0) if k is None else k.shape
    if len(shape) != 3 or len(k_shape) != 3:
        _refuse("q and k are [n, heads, head_dim]")
    _, H, hd = shape
    qp, qs, dt = _rows(q, n, H, hd, "q")
    op, os_, do = (qp, qs, dt) if q_out is None else _rows(q_out, n, H, hd, "q_out")
    kp, ks, dk, Hkv, okp, oks, dko = None, 0, dt, 0, None, 0, dt
    if k is not None:
        Hkv = k_shape[1]
        kp, ks, dk = _rows(k, n, Hkv, hd, "k")
        okp, oks, dko = (kp, ks, dk) if k_out is None else _rows(k_out, n, Hkv, hd, "k_out")
    elif k_out is not None:
        _refuse("k_out without k")
    if not dt == do == dk == dko:
        _refuse("q, k and their outputs have different types")
    f = np.asarray(inv_freq, np.float64)
    if f.ndim != 1:
        _refuse("inv_freq: a vector of f64 is needed")
    _op_check(lib().fs_rope(qp, qs, H, kp, ks, Hkv, n, hd, dt, _vec(positions, n, ty.i32, "positions"),
                            f.tobytes(), 2 * f.size, factor, bool(interleaved) | bool(inverse) << 1,
                            op, os_, okp, oks, _raw(stream, positions)))


def _panel(x, n: int, width: int, what: str):
    """(address, row stride, dtype) of n contiguous rows of `width` f32 or bf16 values."""
    dt = _Types.rows.get(x.dtype)
    if dt is not None and x.shape == (n, width):
        if x.is_contiguous():
            return x.data_ptr(), width, dt
        s0, s1 = x.stride()
        if width == 1 or s1 == 1:
            return x.data_ptr(), s0 if n > 1 else width, dt
    _refuse(f"{what}: a CUDA tensor [{n}, {width}] of f32 or bf16 whose rows are contiguous is needed")


def fs_lora_add(x, adapter, A, B, scale, out, base=None, stream=None) -> None:
    """out[i] = base[i] + scale[a] * B[a] (A[a] x[i]) with a = adapter[i] (int32 [n];
    outside [0, adapters): out[i] = base[i]). x [n, K], base and out [n, N] (f32 or bf16,
    any row stride; base may be out, None is 0), A bf16 [adapters, rank, K], B bf16
    [adapters, N, rank], contiguous, scale f32 [adapters]. All CUDA tensors."""
    ty = _types()
    a, b = A.shape, B.shape
    if len(a) != 3 or len(b) != 3:
        _refuse("A is [adapters, rank, K], B [adapters, N, rank]")
    n, (ad, r, K), N = adapter.numel(), a, b[1]
    if b != (ad, N, r):
        _refuse(f"B: [{ad}, N, {r}] is needed")
    xp, xs, dx = _panel(x, n, K, "x")
    op, os_, do = _panel(out, n, N, "out")
    bp, bs, db = (None, 0, do) if base is None else _panel(base, n, N, "base")
    if db != do:
        _refuse("base and out have different types")
    _op_check(lib().fs_lora_add(xp, xs, dx, _vec(adapter, n, ty.i32, "adapter"), n, K, N,
                                _vec(A, ad * r * K, ty.bf16, "A"), _vec(B, ad * N * r, ty.bf16, "B"),
                                _vec(scale, ad, ty.f32, "scale"), ad, r, bp, bs, op, os_, do,
                                _raw(stream, adapter)))


def fs_sample_filtered(logits, temps, u, tokens, top_k=None, top_p=None, min_p=None, kept=None,
                       stream=None) -> None:
    """One token a row of logits f32 [n, vocab] (any row stride) with the row's temps,
    top_p, min_p (f32 [n]), top_k (int32 [n]) and random number u (f32 [n]): see
    include/fs.h. tokens int32 [n] is written, and kept int32 [n] (how many tokens
    stayed) if given. top_k, top_p, min_p: None for all tokens. All CUDA tensors."""
    ty = _types()
    n = temps.numel()
    shape = logits.shape
    if len(shape) != 2 or logits.dtype is not ty.f32 or shape[0] != n:
        _refuse(f"logits: a CUDA tensor [{n}, vocab] of f32 is needed")
    V = ld = shape[1]
    if not logits.is_contiguous():
        s0, s1 = logits.stride()
        if V > 1 and s1 != 1:
            _refuse("rows of logits must be contiguous")
        ld = s0 if n > 1 else V
    _op_check(lib().fs_sample_filtered(
        logits.data_ptr(), ld, n, V, _vec(temps, n, ty.f32, "temps"),
        _or_none(top_k, n, ty.i32, "top_k"), _or_none(top_p, n, ty.f32, "top_p"),
        _or_none(min_p, n, ty.f32, "min_p"), _vec(u, n, ty.f32, "u"),
        _vec(tokens, n, ty.i32, "tokens"), _or_none(kept, n, ty.i32, "kept"), _raw(stream, temps)))


# ------------------------------------------------------------------ scheduler
def _sched_check(s, rc: int) -> None:
    if rc != FS_OK:
        msg = lib().fs_sched_last_error(s)
        raise FsError(rc, msg.decode() if msg else "")


def fs_sched_create(h, lanes: int, max_prefill_tokens_per_tick: int = 1,
                    max_queue: int = 0, prefill_chunk: int = 1, kv_budget_tokens: int = 0,
                    prefix_reuse_min: int = 0):
    s = C.c_void_p()
    cfg = fs_sched_config(lanes, max_prefill_tokens_per_tick, max_queue, prefill_chunk,
                          kv_budget_tokens, prefix_reuse_min)
    rc = lib().fs_sched_create(h, C.byref(cfg), C.byref(s))
    if rc != FS_OK:
        raise FsError(rc, "fs_sched_create failed")
    return s


def fs_sched_create_model_free(lanes: int, vocab: int,
                               max_prefill_tokens_per_tick: int = 1,
                               max_queue: int = 0, prefill_chunk: int = 1,
                               kv_budget_tokens: int = 0, prefix_reuse_min: int = 0):
    s = C.c_void_p()
    cfg = fs_sched_config(lanes, max_prefill_tokens_per_tick, max_queue, prefill_chunk,
                          kv_budget_tokens, prefix_reuse_min)
    rc = lib().fs_sched_create_model_free(C.byref(cfg), vocab, C.byref(s))
    if rc != FS_OK:
        raise FsError(rc, "fs_sched_create_model_free failed")
    return s


def fs_sched_destroy(s) -> None:
    lib().fs_sched_destroy(s)


def fs_sched_submit(s, prompt, max_new_tokens: int, temperature: float = 0.0,
                    seed: int = 0, stop_token: int = -1) -> int:
    p = _i32(prompt)
    job = fs_job(p.ctypes.data, p.size, max_new_tokens, temperature,
                 int(seed) & (2**64 - 1), stop_token)
    jid = C.c_int64()
    _sched_check(s, lib().fs_sched_submit(s, C.byref(job), C.byref(jid)))
    return jid.value


def fs_sched_step(s) -> int:
    n = C.c_int32()
    _sched_check(s, lib().fs_sched_step(s, C.byref(n)))
    return n.value


def fs_sched_run(s, max_steps: int = 10**9) -> int:
    n = C.c_int64()
    _sched_check(s, lib().fs_sched_run(s, max_steps, C.byref(n)))
    return n.value


def fs_sched_take(s, job_id: int) -> list:
    n = C.c_int32()
    buf = np.empty(1 << 16, dtype=np.int32)
    _sched_check(s, lib().fs_sched_take(s, job_id, _ptr(buf), buf.size, C.byref(n)))
    return buf[:n.value].tolist()


def fs_sched_get_stats(s) -> dict:
    st = fs_sched_stats()
    _sched_check(s, lib().fs_sched_get_stats(s, C.byref(st)))
    return {k: getattr(st, k) for k, _ in st._fields_}


JOB_UNKNOWN, JOB_QUEUED, JOB_RUNNING, JOB_DONE_LENGTH, JOB_DONE_STOP, JOB_CANCELLED = (
    -1, 0, 1, 2, 3, 4)


def fs_sched_status(s, job_id: int) -> int:
    """One of the JOB_* states."""
    v = C.c_int32()
    _sched_check(s, lib().fs_sched_status(s, int(job_id), C.byref(v)))
    return v.value


def fs_sched_cancel(s, job_id: int) -> None:
    _sched_check(s, lib().fs_sched_cancel(s, int(job_id)))


def fs_sched_last_batch(s) -> list:
    n = C.c_int32()
    buf = np.empty(4096, dtype=np.int32)
    _sched_check(s, lib().fs_sched_last_batch(s, _ptr(buf), buf.size, C.byref(n)))
    return buf[:n.value].tolist()


def fs_sched_model_free_fail_resets(s, n: int) -> None:
    """Test hook: the model-free engine fails its next n lane resets."""
    _sched_check(s, lib().fs_sched_model_free_fail_resets(s, int(n)))


def fs_sched_last_error(s) -> str:
    m = lib().fs_sched_last_error(s)
    return m.decode() if m else ""
