"""Python binding of the ftmoe C ABI (include/ftmoe.h): argument marshalling only.

Every step of the MoE layer runs in libftmoe.so (HIP kernels for gfx950 and the
library's host workers).  The functions here carry the C names and take device
pointers as integers (e.g. ``tensor.data_ptr()``) and a HIP stream as an
integer (``torch.cuda.current_stream().cuda_stream``); PyTorch is only used by
callers for device memory and streams.  If the shared library has not been
built, loading fails loudly: there is no fallback implementation.
"""
import ctypes
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libftmoe.so")

FT_OK, FT_ERR_ARG, FT_ERR_NOMEM, FT_ERR_HIP, FT_ERR_STATE, FT_ERR_UNSUPPORTED = range(6)
FT_FMT_BF16, FT_FMT_FP8_B128, FT_FMT_MXFP4_B32 = 0, 1, 2
FMT = {"bf16": FT_FMT_BF16, "fp8": FT_FMT_FP8_B128, "mxfp4": FT_FMT_MXFP4_B32}
FT_HIT, FT_FILL, FT_CPU = 0, 1, 2
FT_MODE_CACHED, FT_MODE_STREAMED, FT_PREFETCH_NEXT, FT_SINGLE_BUFFER, FT_WARM_DECODE = 0, 1, 0x100, 0x200, 0x400
ROUTE_INVALID = -(2 ** 31)

i32, i64, u32, u64, vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32, ctypes.c_uint64, ctypes.c_void_p


class FtShape(ctypes.Structure):
    _fields_ = [("layers", i32), ("experts", i32), ("top_k", i32), ("d_model", i32), ("d_ff", i32), ("fmt", i32)]


class FtProfile(ctypes.Structure):
    _fields_ = [("bp_mbps", u32), ("bh_mbps", u32), ("max_fetch", i32)]


class FtClassifyOut(ctypes.Structure):
    _fields_ = [("counts", vp), ("uniq", vp), ("cls", vp), ("slot", vp), ("ev_slot", vp), ("ev_old", vp),
                ("ev_new", vp), ("cpu_ids", vp), ("capacity", i32)]


class FtStats(ctypes.Structure):
    _fields_ = [("calls", u64), ("routes", u64), ("unique", u64), ("hits", u64), ("misses", u64), ("fills", u64),
                ("cpu_experts", u64), ("evictions", u64), ("bytes_filled", u64), ("layers_streamed", u64),
                ("clock", u64), ("error_flags", i32), ("num_slots", i32), ("host_experts", u64),
                ("host_bytes", u64), ("host_seconds", ctypes.c_double)]

    def as_dict(self):
        return {k: getattr(self, k) for k, _ in self._fields_}


FT_K_GEMV_GU, FT_K_GEMV_DOWN, FT_K_GEMM_GU, FT_K_GEMM_DOWN, FT_K_FILL = range(5)


class FtTiming(ctypes.Structure):
    _fields_ = [("launches", u64 * 5), ("ms", ctypes.c_double * 5), ("gemv_experts", u64), ("gemv_rows", u64),
                ("gemm_experts", u64), ("gemm_rows", u64)]


class FtLora(ctypes.Structure):
    _fields_ = [("count", i32), ("max_rank", i32), ("rank", vp), ("scale", vp), ("a", vp), ("b", vp)]


class FtMatrix(ctypes.Structure):
    _fields_ = [("n", i32), ("K", i32), ("fmt", i32), ("reserved", i32), ("codes", vp), ("scales", vp)]


FT_KV_BF16, FT_KV_E4M3 = 0, 1
KV_FMT = {"bf16": FT_KV_BF16, "e4m3": FT_KV_E4M3}
FT_GATE_NONE, FT_GATE_CHANNEL, FT_GATE_TOKEN, FT_GATE_FULL, FT_GATE_SIGMOID = 0, 1, 2, 3, 0x10
GATE = {"none": FT_GATE_NONE, "channel": FT_GATE_CHANNEL, "token": FT_GATE_TOKEN, "full": FT_GATE_FULL}


class FtKvCache(ctypes.Structure):
    _fields_ = [("pages", i32), ("page_tokens", i32), ("kv_heads", i32), ("head_dim", i32), ("fmt", i32),
                ("reserved", i32), ("page_stride", i64), ("k", vp), ("v", vp), ("k_scale", vp), ("v_scale", vp)]


class FtKvBatch(ctypes.Structure):
    _fields_ = [("requests", i32), ("pages", i32), ("page_tokens", i32), ("width", i32), ("tokens", i32),
                ("row_tokens", i32), ("context", vp), ("add", vp), ("table", vp), ("free_pages", vp),
                ("free_count", vp), ("kv_len", vp), ("start", vp), ("slot", vp), ("pos", vp), ("counts", vp)]


class FtAppend(ctypes.Structure):
    _fields_ = [("tokens", i32), ("q_heads", i32), ("rot", i32), ("positions", i32), ("q", vp), ("k", vp), ("v", vp),
                ("q_stride", i64), ("k_stride", i64), ("v_stride", i64), ("slot", vp), ("pos", vp), ("cos_sin", vp),
                ("q_out", vp), ("q_out_stride", i64)]


class FtAttend(ctypes.Structure):
    _fields_ = [("requests", i32), ("q_heads", i32), ("width", i32), ("window", i32), ("scale", ctypes.c_float),
                ("reserved", i32), ("q", vp), ("q_stride", i64), ("table", vp), ("kv_len", vp), ("sinks", vp),
                ("out", vp), ("out_stride", i64)]


class FtNorm(ctypes.Structure):
    _fields_ = [("T", i32), ("d", i32), ("gate_kind", i32), ("eps", ctypes.c_float),
                ("residual_scale", ctypes.c_float), ("weight_offset", ctypes.c_float), ("block", vp),
                ("residual", vp), ("post_w", vp), ("pre_w", vp), ("gate", vp), ("sum", vp), ("normed", vp),
                ("block_stride", i64), ("residual_stride", i64), ("gate_stride", i64), ("sum_stride", i64),
                ("normed_stride", i64)]


class FtError(RuntimeError):
    def __init__(self, status, msg):
        super().__init__(f"ftmoe status {status}: {msg}")
        self.status = status


_lib = None

# name -> (restype, argtypes)
_SIGS = {
    "ft_cache_create": (i32, [ctypes.POINTER(FtShape), ctypes.POINTER(FtProfile), vp, i64, i32, ctypes.POINTER(vp)]),
    "ft_cache_create_layers": (i32, [ctypes.POINTER(FtShape), ctypes.POINTER(FtProfile), ctypes.POINTER(vp), i64, i32,
                                     ctypes.POINTER(vp)]),
    "ft_cache_destroy": (i32, [vp]),
    "ft_record_bytes": (i64, [ctypes.POINTER(FtShape)]),
    "ft_moe_route": (i32, [ctypes.POINTER(FtShape), vp, vp, i32, vp, vp, vp]),
    "ft_cache_classify": (i32, [vp, i32, vp, i32, ctypes.POINTER(FtClassifyOut), vp]),
    "ft_moe_forward": (i32, [vp, i32, i32, vp, vp, vp, i32, vp, vp]),
    "ft_moe_forward_noalloc": (i32, [vp, i32, vp, vp, vp, i32, vp, vp]),
    "ft_cache_resize": (i32, [vp, i64]),
    "ft_cache_profile": (i32, [vp, i32, ctypes.POINTER(FtProfile)]),
    "ft_cache_set_profile": (i32, [vp, ctypes.POINTER(FtProfile)]),
    "ft_cache_stats": (i32, [vp, ctypes.POINTER(FtStats)]),
    "ft_cache_snapshot": (i32, [vp, vp, vp, vp, vp]),
    "ft_cache_set_timing": (i32, [vp, i32]),
    "ft_cache_timing": (i32, [vp, ctypes.POINTER(FtTiming)]),
    "ft_cache_read_slot": (i32, [vp, i64, vp]),
    "ft_workspace_create": (i32, [ctypes.c_size_t, ctypes.POINTER(vp)]),
    "ft_workspace_destroy": (i32, [vp]),
    "ft_moe_layer_workspace": (i64, [ctypes.POINTER(FtShape), i32]),
    "ft_moe_layer": (i32, [ctypes.POINTER(FtShape), vp, vp, vp, i64, i32, vp, vp, vp, vp, vp, vp]),
    "ft_lora_project_workspace": (i64, [ctypes.POINTER(FtMatrix), i32, i32]),
    "ft_lora_project": (i32, [ctypes.POINTER(FtMatrix), ctypes.POINTER(FtLora), vp, vp, i32, vp, vp, vp, vp]),
    "ft_lora_expert_workspace": (i64, [ctypes.POINTER(FtShape), i32, i32]),
    "ft_lora_expert": (i32, [ctypes.POINTER(FtShape), vp, ctypes.POINTER(FtLora), ctypes.POINTER(FtLora),
                             ctypes.POINTER(FtLora), vp, vp, i32, vp, vp, vp, vp]),
    "ft_kv_plan": (i32, [ctypes.POINTER(FtKvBatch), vp, vp]),
    "ft_kv_append": (i32, [ctypes.POINTER(FtKvCache), ctypes.POINTER(FtAppend), vp]),
    "ft_kv_attend_workspace": (i64, [ctypes.POINTER(FtKvCache), i32, i32]),
    "ft_kv_attend": (i32, [ctypes.POINTER(FtKvCache), ctypes.POINTER(FtAttend), vp, vp]),
    "ft_block_norm": (i32, [ctypes.POINTER(FtNorm), vp]),
    "ft_host_alloc": (i32, [ctypes.c_size_t, ctypes.POINTER(vp)]),
    "ft_host_free": (i32, [vp]),
    "ft_last_error": (ctypes.c_char_p, []),
}


def lib():
    """Load libftmoe.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m moe_expert_execution_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def ft_last_error() -> str:
    return lib().ft_last_error().decode()


def _check(status):
    if status != FT_OK:
        raise FtError(status, ft_last_error())


def shape(layers, experts, top_k, d_model, d_ff, fmt="bf16") -> FtShape:
    return FtShape(layers, experts, top_k, d_model, d_ff, FMT[fmt] if isinstance(fmt, str) else fmt)


def profile(bp_mbps, bh_mbps, max_fetch=-1) -> FtProfile:
    return FtProfile(bp_mbps, bh_mbps, max_fetch)


def matrix(n, K, fmt, codes: int, scales: int = 0) -> FtMatrix:
    """A resident matrix [n x K]: device addresses of its codes and (fp8, mxfp4) scales."""
    return FtMatrix(n, K, FMT[fmt] if isinstance(fmt, str) else fmt, 0, codes, scales)


def ft_record_bytes(shp: FtShape) -> int:
    return lib().ft_record_bytes(ctypes.byref(shp))


def ft_host_alloc(nbytes: int) -> int:
    p = vp()
    _check(lib().ft_host_alloc(nbytes, ctypes.byref(p)))
    return p.value


def ft_host_free(ptr: int) -> None:
    _check(lib().ft_host_free(ptr))


def host_array(ptr: int, nbytes: int) -> np.ndarray:
    """A uint8 NumPy view of `nbytes` of (pinned) host memory at `ptr`."""
    return np.ctypeslib.as_array(ctypes.cast(ptr, ctypes.POINTER(ctypes.c_uint8)), shape=(nbytes,))


def ft_cache_create(shp: FtShape, prof: FtProfile, host_bank: int, num_slots: int, max_tokens: int) -> int:
    h = vp()
    _check(lib().ft_cache_create(ctypes.byref(shp), ctypes.byref(prof), host_bank, num_slots, max_tokens,
                                 ctypes.byref(h)))
    return h.value


def ft_cache_create_layers(shp: FtShape, prof: FtProfile, layer_banks, num_slots: int, max_tokens: int) -> int:
    """`layer_banks`: one pinned host address per layer (entries may repeat)."""
    table = (vp * len(layer_banks))(*layer_banks)
    h = vp()
    _check(lib().ft_cache_create_layers(ctypes.byref(shp), ctypes.byref(prof), table, num_slots, max_tokens,
                                        ctypes.byref(h)))
    return h.value


def ft_cache_destroy(h: int) -> None:
    _check(lib().ft_cache_destroy(h))


def ft_moe_route(shp: FtShape, x: int, wr: int, T: int, ids: int, w: int, stream: int = 0) -> None:
    _check(lib().ft_moe_route(ctypes.byref(shp), x, wr, T, ids, w, stream))


def ft_cache_classify(h: int, layer: int, ids: int, T: int, out=None, stream: int = 0) -> None:
    _check(lib().ft_cache_classify(h, layer, ids, T, ctypes.byref(out) if out is not None else None, stream))


def ft_moe_forward(h: int, layer: int, mode: int, x: int, routes: int, w: int, T: int, y: int,
                   stream: int = 0) -> None:
    _check(lib().ft_moe_forward(h, layer, mode, x, routes, w, T, y, stream))


def ft_moe_forward_noalloc(h: int, layer: int, x: int, routes: int, w: int, T: int, y: int, stream: int = 0) -> None:
    _check(lib().ft_moe_forward_noalloc(h, layer, x, routes, w, T, y, stream))


def ft_cache_resize(h: int, num_slots: int) -> None:
    _check(lib().ft_cache_resize(h, num_slots))


def ft_cache_profile(h: int, records: int) -> FtProfile:
    out = FtProfile()
    _check(lib().ft_cache_profile(h, records, ctypes.byref(out)))
    return out


def ft_cache_set_profile(h: int, prof: FtProfile) -> None:
    _check(lib().ft_cache_set_profile(h, ctypes.byref(prof)))


def ft_cache_stats(h: int) -> FtStats:
    s = FtStats()
    _check(lib().ft_cache_stats(h, ctypes.byref(s)))
    return s


def ft_cache_set_timing(h: int, enable: bool) -> None:
    _check(lib().ft_cache_set_timing(h, 1 if enable else 0))


def ft_cache_timing(h: int) -> FtTiming:
    t = FtTiming()
    _check(lib().ft_cache_timing(h, ctypes.byref(t)))
    return t


def ft_cache_snapshot(h: int, n_ids: int, n_slots: int):
    sfi = np.empty(n_ids, np.int32)
    ios = np.empty(n_slots, np.int32)
    st = np.empty(n_slots, np.uint64)
    clk = np.zeros(1, np.uint64)
    _check(lib().ft_cache_snapshot(h, sfi.ctypes.data, ios.ctypes.data, st.ctypes.data, clk.ctypes.data))
    return sfi, ios, st, int(clk[0])


def ft_cache_read_slot(h: int, slot: int, nbytes: int) -> np.ndarray:
    out = np.empty(nbytes, np.uint8)
    _check(lib().ft_cache_read_slot(h, slot, out.ctypes.data))
    return out


def ft_workspace_create(nbytes: int) -> int:
    h = vp()
    _check(lib().ft_workspace_create(nbytes, ctypes.byref(h)))
    return h.value


def ft_workspace_destroy(ws: int) -> None:
    _check(lib().ft_workspace_destroy(ws))


def ft_moe_layer_workspace(shp: FtShape, max_tokens: int) -> int:
    return lib().ft_moe_layer_workspace(ctypes.byref(shp), max_tokens)


def ft_moe_layer(shp: FtShape, x: int, wr: int, records: int, record_stride: int, T: int, base: int, ids: int, w: int,
                 y: int, ws: int, stream: int = 0) -> None:
    """`base` may be 0 (no addend)."""
    _check(lib().ft_moe_layer(ctypes.byref(shp), x, wr, records, record_stride, T, base, ids, w, y, ws, stream))


def _opt(struct):
    return ctypes.byref(struct) if struct is not None else None


def ft_lora_project_workspace(m: FtMatrix, max_rank: int, max_tokens: int) -> int:
    return lib().ft_lora_project_workspace(ctypes.byref(m), max_rank, max_tokens)


def ft_lora_project(m: FtMatrix, lora, x: int, adapter: int, T: int, base: int, y: int, ws: int,
                    stream: int = 0) -> None:
    """`lora`: an FtLora or None; `base` and (without adapters) `adapter` may be 0."""
    _check(lib().ft_lora_project(ctypes.byref(m), _opt(lora), x, adapter, T, base, y, ws, stream))


def ft_lora_expert_workspace(shp: FtShape, max_rank: int, max_tokens: int) -> int:
    return lib().ft_lora_expert_workspace(ctypes.byref(shp), max_rank, max_tokens)


def ft_lora_expert(shp: FtShape, record: int, gate, up, down, x: int, adapter: int, T: int, base: int, y: int, ws: int,
                   stream: int = 0) -> None:
    """`gate`, `up`, `down`: FtLora or None; `base` and (without adapters) `adapter` may be 0."""
    _check(lib().ft_lora_expert(ctypes.byref(shp), record, _opt(gate), _opt(up), _opt(down), x, adapter, T, base, y,
                                ws, stream))


def kv_cache(pages, page_tokens, kv_heads, head_dim, fmt, k: int, v: int, k_scale: int = 0, v_scale: int = 0,
             page_stride: int = 0) -> FtKvCache:
    """A paged key-value cache; page_stride 0: pages back to back."""
    f = KV_FMT[fmt] if isinstance(fmt, str) else fmt
    stride = page_stride or kv_heads * page_tokens * head_dim * (2 if f == FT_KV_BF16 else 1)
    return FtKvCache(pages, page_tokens, kv_heads, head_dim, f, 0, stride, k, v, k_scale, v_scale)


def kv_batch(requests, pages, page_tokens, width, tokens, row_tokens, context: int, add: int, table: int,
             free_pages: int, free_count: int, kv_len: int, start: int, slot: int, pos: int, counts: int) -> FtKvBatch:
    return FtKvBatch(requests, pages, page_tokens, width, tokens, row_tokens, context, add, table, free_pages,
                     free_count, kv_len, start, slot, pos, counts)


def kv_append(tokens, k: int, k_stride, v: int, v_stride, slot: int, pos: int = 0, rot=0, positions=0,
              cos_sin: int = 0, q_heads=0, q: int = 0, q_stride=0, q_out: int = 0, q_out_stride=0) -> FtAppend:
    return FtAppend(tokens, q_heads, rot, positions, q, k, v, q_stride, k_stride, v_stride, slot, pos, cos_sin, q_out,
                    q_out_stride)


def kv_attend(requests, q_heads, width, scale, q: int, q_stride, table: int, kv_len: int, out: int, out_stride,
              window=0, sinks: int = 0) -> FtAttend:
    return FtAttend(requests, q_heads, width, window, scale, 0, q, q_stride, table, kv_len, sinks, out, out_stride)


def block_norm(T, d, eps, block: int = 0, residual: int = 0, post_w: int = 0, pre_w: int = 0, gate: int = 0,
               gate_kind="none", sigmoid=False, sum: int = 0, normed: int = 0, residual_scale=1.0, weight_offset=0.0,
               block_stride=0, residual_stride=0, gate_stride=0, sum_stride=0, normed_stride=0) -> FtNorm:
    """Strides of 0 mean d."""
    kind = GATE[gate_kind] if isinstance(gate_kind, str) else gate_kind
    kind |= FT_GATE_SIGMOID if sigmoid and kind else 0
    return FtNorm(T, d, kind, eps, residual_scale, weight_offset, block, residual, post_w, pre_w, gate, sum, normed,
                  block_stride or d, residual_stride or d, gate_stride or d, sum_stride or d, normed_stride or d)


def ft_kv_plan(batch: FtKvBatch, ws: int, stream: int = 0) -> None:
    _check(lib().ft_kv_plan(ctypes.byref(batch), ws, stream))


def ft_kv_append(cache: FtKvCache, args: FtAppend, stream: int = 0) -> None:
    _check(lib().ft_kv_append(ctypes.byref(cache), ctypes.byref(args), stream))


def ft_kv_attend_workspace(cache: FtKvCache, q_heads: int, max_requests: int) -> int:
    return lib().ft_kv_attend_workspace(ctypes.byref(cache), q_heads, max_requests)


def ft_kv_attend(cache: FtKvCache, args: FtAttend, ws: int, stream: int = 0) -> None:
    _check(lib().ft_kv_attend(ctypes.byref(cache), ctypes.byref(args), ws, stream))


def ft_block_norm(args: FtNorm, stream: int = 0) -> None:
    _check(lib().ft_block_norm(ctypes.byref(args), stream))
