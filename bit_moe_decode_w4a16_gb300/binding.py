"""ctypes binding of libbitmoe.so: argument marshalling only.

Every function here has the name of the C entry point it calls (see
include/bitmoe.h) and does nothing but convert arguments: torch tensors to
device pointers, torch streams to cudaStream_t handles, and a non-OK status
to a ``BitMoeError``.  All of the decode step's work runs in the CUDA
library; when the library has not been built this module raises on import
of the library rather than running anything else in its place.
"""

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libbitmoe.so")

BM_OK = 0
STATUS_NAMES = {
    0: "BM_OK", 1: "BM_ERR_INVALID_ARG", 2: "BM_ERR_CTX_CAP", 3: "BM_ERR_NO_SLOT",
    4: "BM_ERR_SLOT_FREE", 5: "BM_ERR_CUDA", 6: "BM_ERR_OOM", 7: "BM_ERR_NOT_READY",
    8: "BM_ERR_DEVICE_CHECK", 9: "BM_ERR_UNSUPPORTED",
}
KV8_E4M3, KV8_INT8 = 0, 1
KV8_DRAFTS = 64
POLICY_AUTO, POLICY_SIMT, POLICY_TC, POLICY_MMA = 0, 1, 2, 3


class BitMoeError(RuntimeError):
    def __init__(self, status, message):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status
        self.message = message


class bm_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("hidden", "q_heads", "kv_heads", "head_dim", "experts", "top_k",
                                            "ffn", "group", "vocab", "layers")] + \
               [("rope_base", ctypes.c_float), ("rms_eps", ctypes.c_float)] + \
               [(n, ctypes.c_int) for n in ("max_streams", "ctx_cap", "renorm_topk", "kernel_policy",
                                            "use_graph", "prefill_tc", "persistent_step")]


_P = ctypes.c_void_p


class bm_layer_weights(ctypes.Structure):
    _fields_ = [(n, _P) for n in ("wqkv", "wqkv_s", "wo", "wo_s", "wr", "wg", "wg_s", "wu", "wu_s",
                                  "wd", "wd_s", "attn_norm", "ffn_norm")]


class bm_moe_weights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("experts", "top_k", "hidden", "ffn", "group", "renorm_topk")] + \
               [(n, _P) for n in ("wr", "wg", "wg_s", "wu", "wu_s", "wd", "wd_s")]


class bm_kv8_cache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("format", "slots", "ctx_cap", "kv_heads", "head_dim")] + \
               [(n, _P) for n in ("K", "V", "Ks", "Vs")]


class bm_kv8_rope(ctypes.Structure):
    _fields_ = [("norm", ctypes.c_int), ("eps", ctypes.c_float)] + [(n, _P) for n in ("q_norm", "k_norm", "inv_freq")]


class bm_kernel_profile(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char * 24), ("launches", ctypes.c_int), ("ms", ctypes.c_float),
                ("bytes", ctypes.c_double), ("flops", ctypes.c_double)]


class bm_stats(ctypes.Structure):
    _fields_ = [(n, ctypes.c_uint64) for n in ("steps", "tokens", "graph_launches", "graph_captures",
                                               "kernel_launches", "kernels_per_step")] + \
               [(n, ctypes.c_size_t) for n in ("weight_bytes", "arena_bytes", "scratch_bytes")]


_lib = None


def lib():
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"libbitmoe.so is not built ({LIB_PATH}); run __graft_entry__.build()")
        L = ctypes.CDLL(LIB_PATH)
        I, V, S, SZ = ctypes.c_int, ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        PI = ctypes.POINTER(ctypes.c_int)
        sig = {
            "bm_last_error": ([], ctypes.c_char_p),
            "bm_engine_create": ([ctypes.POINTER(bm_config), ctypes.POINTER(V)], S),
            "bm_engine_destroy": ([V], None),
            "bm_engine_set_layer": ([V, I, ctypes.POINTER(bm_layer_weights), V], S),
            "bm_engine_set_embeddings": ([V, V, V, V, V], S),
            "bm_engine_sync": ([V, V], S),
            "bm_engine_stats": ([V, ctypes.POINTER(bm_stats)], S),
            "bm_engine_kernel_family": ([V], I),
            "kv_slot_seed": ([V, V, V, I, PI, V], S),
            "kv_slot_append": ([V, I, V, V, V, I, V], S),
            "kv_slot_attend": ([V, I, V, V, V, I, V], S),
            "kv_slot_advance": ([V, V, I, V], S),
            "kv_slot_release": ([V, I], S),
            "kv_slot_length": ([V, I, PI], S),
            "kv_slot_read": ([V, I, I, I, V, V, V], S),
            "w4_gemm_batched": ([V, V, V, V, V, I, I, I, I, V], S),
            "bm_moe_workspace_bytes": ([I, I, I, I, I], SZ),
            "bm_w4_repack_tc": ([V, V, I, I, I, V, V, V], S),
            "w4_gemm_batched_tc": ([V, V, V, V, V, I, I, I, I, V], S),
            "bm_w4_repack_mma": ([V, V, I, I, I, V, V, V], S),
            "w4_gemm_batched_mma": ([V, V, V, V, V, I, I, I, I, V], S),
            "w4_gemm_prompt_tc": ([V, V, V, V, V, I, I, I, I, V], S),
            "moe_grouped_w4": ([ctypes.POINTER(bm_moe_weights), V, V, V, V, V, I, V, SZ, V], S),
            "moe_grouped_w4_noalloc": ([ctypes.POINTER(bm_moe_weights), V, V, V, V, V, I, V], S),
            "bm_moe_noalloc_max_bytes": ([], SZ),
            "decode_step": ([V, I, V, V, V, V, V], S),
            "kv_slot_prefill": ([V, I, I, V, V, V, V], S),
            "bm_engine_profile_step": ([V, I, V, V, V, ctypes.POINTER(bm_kernel_profile), I, PI, V], S),
            "kv8_append": ([V, V, ctypes.c_int64, I, V, V, V, V, V, I, V], S),
            "kv8_read": ([V, I, I, I, V, V, V], S),
            "kv8_workspace_bytes": ([I, I, I, I, I, I], SZ),
            "kv8_attend": ([V, V, V, V, I, ctypes.c_float, V, I, V, SZ, V], S),
            "kv8_attend_prefix": ([V, V, I, I, V, V, V, I, ctypes.c_float, V, I, V, SZ, V], S),
            "kv8_plan_bytes": ([I, I, I, I], SZ),
            "kv8_plan": ([V, I, V, V, V, V, V, V, V, V, V, I, I, V, SZ, V], S),
            "kv8_rows_workspace_bytes": ([I, I, I, I, I, I], SZ),
            "kv8_attend_rows": ([V, V, SZ, V, I, ctypes.c_float, V, I, I, V, SZ, V], S),
            "kv8_rows_status": ([V], S),
            "bm_test_kv8_rows_hold": ([I, I, I], S),
            "kv8_tree_accept": ([V, SZ, V, V, V, V, V, V, V, I, I, V], S),
            "kv8_tree_keep": ([V, V, SZ, V, V, I, V], S),
            "bm_sample": ([V, I, ctypes.c_int64, I, I, V, V, V, V, V, V, V, V], S),
            "bm_w4_quantize": ([V, I, I, I, V, V, V], S),
            "bm_engine_moe": ([V, I, V, V, V, V, I, V], S),
            "bm_probe_tcgen05_mma": ([I, I, I, I, I, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_double)], S),
            "bm_engine_attention": ([V, I, V, V, V, I, V], S),
            "bm_engine_read_hidden": ([V, I, V, V], S),
            "bm_engine_test_drop_expert_item": ([V, I], S),
            "bm_engine_test_drop_persist_unit": ([V, I], S),
            "bm_engine_set_persistent_step": ([V, I], S),
            "bm_slot_map_create": ([I, I, ctypes.POINTER(V)], S),
            "bm_slot_map_destroy": ([V], None),
            "bm_slot_map_acquire": ([V, I, PI], S),
            "bm_slot_map_release": ([V, I], S),
            "bm_slot_map_check_batch": ([V, V, I], S),
            "bm_slot_map_advance": ([V, V, I], S),
            "bm_slot_map_length": ([V, I, PI], S),
            "bm_slot_map_active_count": ([V], I),
        }
        for name, (args, res) in sig.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = res
        _lib = L
    return _lib


def last_error():
    return lib().bm_last_error().decode()


def _check(status):
    if status != BM_OK:
        raise BitMoeError(status, last_error())
    return status


def ptr(x):
    """Device/host address of a torch tensor, an int address, or None."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if hasattr(x, "data_ptr"):
        return x.data_ptr()
    if isinstance(x, ctypes.Array):
        return ctypes.addressof(x)
    raise TypeError(f"cannot take the address of {type(x)}")


def stream_handle(s):
    if s is None:
        import torch
        return torch.cuda.current_stream().cuda_stream if torch.cuda.is_available() else None
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _i32_array(values):
    arr = (ctypes.c_int32 * len(values))(*[int(v) for v in values])
    return arr


# --------------------------------------------------------------- engine

def bm_engine_create(cfg):
    """cfg: a bm_config or a dict of its fields.  Returns the engine handle."""
    if isinstance(cfg, dict):
        c = bm_config()
        for k, v in cfg.items():
            setattr(c, k, v)
        cfg = c
    h = ctypes.c_void_p()
    _check(lib().bm_engine_create(ctypes.byref(cfg), ctypes.byref(h)))
    return h.value


def bm_engine_destroy(e):
    lib().bm_engine_destroy(e)


def bm_engine_set_layer(e, layer, weights, stream=None):
    """weights: dict with the bm_layer_weights field names -> tensors/addresses."""
    w = bm_layer_weights(**{k: ptr(weights.get(k)) for k, _ in bm_layer_weights._fields_})
    _check(lib().bm_engine_set_layer(e, layer, ctypes.byref(w), stream_handle(stream)))


def bm_engine_set_embeddings(e, embed, lm_head, final_norm=None, stream=None):
    _check(lib().bm_engine_set_embeddings(e, ptr(embed), ptr(lm_head), ptr(final_norm), stream_handle(stream)))


def bm_engine_sync(e, stream=None):
    _check(lib().bm_engine_sync(e, stream_handle(stream)))


def bm_engine_stats(e):
    s = bm_stats()
    _check(lib().bm_engine_stats(e, ctypes.byref(s)))
    return {k: getattr(s, k) for k, _ in bm_stats._fields_}


def bm_engine_kernel_family(e):
    return lib().bm_engine_kernel_family(e)


# --------------------------------------------------------------- slots

def kv_slot_seed(e, K, V, length, stream=None):
    slot = ctypes.c_int(-1)
    _check(lib().kv_slot_seed(e, ptr(K), ptr(V), int(length), ctypes.byref(slot), stream_handle(stream)))
    return slot.value


def kv_slot_append(e, layer, slots, Knew, Vnew, stream=None):
    arr = _i32_array(slots)
    _check(lib().kv_slot_append(e, layer, ctypes.addressof(arr), ptr(Knew), ptr(Vnew), len(slots),
                                stream_handle(stream)))


def kv_slot_attend(e, layer, slots, Q, O, stream=None):
    arr = _i32_array(slots)
    _check(lib().kv_slot_attend(e, layer, ctypes.addressof(arr), ptr(Q), ptr(O), len(slots),
                                stream_handle(stream)))


def kv_slot_advance(e, slots, stream=None):
    arr = _i32_array(slots)
    _check(lib().kv_slot_advance(e, ctypes.addressof(arr), len(slots), stream_handle(stream)))


def kv_slot_release(e, slot):
    _check(lib().kv_slot_release(e, int(slot)))


def kv_slot_length(e, slot):
    n = ctypes.c_int(0)
    _check(lib().kv_slot_length(e, int(slot), ctypes.byref(n)))
    return n.value


def kv_slot_read(e, layer, slot, count, K_out, V_out, stream=None):
    _check(lib().kv_slot_read(e, layer, slot, count, ptr(K_out), ptr(V_out), stream_handle(stream)))


# --------------------------------------------------------------- ops

def w4_gemm_batched(W, S, X, Y, R, M, N, K, g, stream=None):
    _check(lib().w4_gemm_batched(ptr(W), ptr(S), ptr(X), ptr(Y), ptr(R), M, N, K, g, stream_handle(stream)))


def bm_w4_repack_tc(W, S, N, K, g, Wtc, Stc, stream=None):
    _check(lib().bm_w4_repack_tc(ptr(W), ptr(S), N, K, g, ptr(Wtc), ptr(Stc), stream_handle(stream)))


def w4_gemm_batched_tc(Wtc, Stc, X, Y, R, M, N, K, g, stream=None):
    _check(lib().w4_gemm_batched_tc(ptr(Wtc), ptr(Stc), ptr(X), ptr(Y), ptr(R), M, N, K, g, stream_handle(stream)))


def bm_w4_repack_mma(W, S, N, K, g, Wm, Sm, stream=None):
    _check(lib().bm_w4_repack_mma(ptr(W), ptr(S), N, K, g, ptr(Wm), ptr(Sm), stream_handle(stream)))


def w4_gemm_batched_mma(Wm, Sm, X, Y, R, M, N, K, g, stream=None):
    _check(lib().w4_gemm_batched_mma(ptr(Wm), ptr(Sm), ptr(X), ptr(Y), ptr(R), M, N, K, g, stream_handle(stream)))


def w4_gemm_prompt_tc(Wm, Sm, X16, Y, R, M, N, K, g, stream=None):
    _check(lib().w4_gemm_prompt_tc(ptr(Wm), ptr(Sm), ptr(X16), ptr(Y), ptr(R), M, N, K, g, stream_handle(stream)))


def bm_moe_workspace_bytes(B, experts, top_k, hidden, ffn):
    return lib().bm_moe_workspace_bytes(B, experts, top_k, hidden, ffn)


def moe_grouped_w4(weights, X, Hres, Y, topk_ids, topk_w, B, ws, ws_bytes, stream=None):
    """weights: dict with bm_moe_weights field names."""
    w = bm_moe_weights(**{k: (weights[k] if t is ctypes.c_int else ptr(weights[k]))
                          for k, t in bm_moe_weights._fields_})
    _check(lib().moe_grouped_w4(ctypes.byref(w), ptr(X), ptr(Hres), ptr(Y), ptr(topk_ids), ptr(topk_w), B,
                                ptr(ws), ws_bytes, stream_handle(stream)))


def moe_grouped_w4_noalloc(weights, X, Hres, Y, topk_ids, topk_w, B, stream=None):
    """The grouped expert op with the library's built-in workspace (no
    allocation); weights as for moe_grouped_w4."""
    w = bm_moe_weights(**{k: (weights[k] if t is ctypes.c_int else ptr(weights[k]))
                          for k, t in bm_moe_weights._fields_})
    _check(lib().moe_grouped_w4_noalloc(ctypes.byref(w), ptr(X), ptr(Hres), ptr(Y), ptr(topk_ids), ptr(topk_w), B,
                                        stream_handle(stream)))


def bm_moe_noalloc_max_bytes():
    return lib().bm_moe_noalloc_max_bytes()


def decode_step(e, slots, tokens, next_tokens, logits=None, stream=None):
    """slots: host sequence of ints; tokens / next_tokens: host or device int32."""
    arr = _i32_array(slots)
    _check(lib().decode_step(e, len(slots), ctypes.addressof(arr), ptr(tokens), ptr(next_tokens), ptr(logits),
                             stream_handle(stream)))


def kv_slot_prefill(e, slot, tokens, next_token, logits=None, stream=None):
    """tokens: host or device int32 [n]; next_token: host or device int32 [1]."""
    _check(lib().kv_slot_prefill(e, int(slot), int(tokens.numel()), ptr(tokens), ptr(next_token), ptr(logits),
                                 stream_handle(stream)))


def bm_engine_profile_step(e, slots, tokens, next_tokens, stream=None):
    """One eager decode step with per-kernel CUDA-event times; returns a list
    of dicts (name, launches, ms, bytes, flops), one per kernel class."""
    arr = _i32_array(slots)
    out = (bm_kernel_profile * 32)()
    n = ctypes.c_int(0)
    _check(lib().bm_engine_profile_step(e, len(slots), ctypes.addressof(arr), ptr(tokens), ptr(next_tokens), out,
                                        32, ctypes.byref(n), stream_handle(stream)))
    return [{"name": out[i].name.decode(), "launches": out[i].launches, "ms": out[i].ms,
             "bytes": out[i].bytes, "flops": out[i].flops} for i in range(n.value)]


def bm_engine_moe(e, layer, h, y, topk_ids=None, topk_w=None, stream=None):
    """The decode step's routing and expert kernels on one layer; h, y: bf16 [B][H]."""
    _check(lib().bm_engine_moe(e, layer, ptr(h), ptr(y), ptr(topk_ids), ptr(topk_w), int(h.shape[0]),
                               stream_handle(stream)))


def bm_engine_attention(e, layer, slots, qkv, out, stream=None):
    """The decode step's fused attention on one layer; qkv: bf16 rows, out: fp16 [B][qh][d]."""
    arr = _i32_array(slots)
    _check(lib().bm_engine_attention(e, layer, ctypes.addressof(arr), ptr(qkv), ptr(out), len(slots),
                                     stream_handle(stream)))


def bm_engine_read_hidden(e, B, out, stream=None):
    _check(lib().bm_engine_read_hidden(e, int(B), ptr(out), stream_handle(stream)))


def bm_engine_test_drop_expert_item(e, item):
    _check(lib().bm_engine_test_drop_expert_item(e, int(item)))


def bm_engine_set_persistent_step(e, enable):
    _check(lib().bm_engine_set_persistent_step(e, int(enable)))


def bm_engine_test_drop_persist_unit(e, unit):
    _check(lib().bm_engine_test_drop_persist_unit(e, int(unit)))


def bm_probe_tcgen05_mma(n, a_in_tmem, swizzle128, iters, roundtrip=0):
    """SM cycles per tcgen05 MMA (M 128 x N n x K 16): (to issue, to complete)."""
    a, b = ctypes.c_double(0), ctypes.c_double(0)
    _check(lib().bm_probe_tcgen05_mma(int(n), int(a_in_tmem), int(swizzle128), int(iters), int(roundtrip),
                                      ctypes.byref(a), ctypes.byref(b)))
    return a.value, b.value


def bm_w4_quantize(W, N, K, g, packed, scales, stream=None):
    _check(lib().bm_w4_quantize(ptr(W), N, K, g, ptr(packed), ptr(scales), stream_handle(stream)))


# --------------------------------------------------------------- 8-bit K/V cache, sampling
# These calls take torch tensors and check what the C side cannot see: type,
# shape, contiguity, and that the memory is on the current CUDA device.  A
# decode step makes several of them, so the checks take the short way through
# and only a failing one works out what is wrong.

_torch = None


def _t():
    global _torch
    if _torch is None:
        import torch
        if torch.cuda.is_available():
            torch.cuda.init()
        _torch = torch
    return _torch


def _here():
    """Index of the current CUDA device; -2 without one (a CPU tensor's is -1)."""
    t = _t()
    return t._C._cuda_getDevice() if t.cuda.is_initialized() else -2


def _stream(s, dev):
    return _t()._C._cuda_getCurrentRawStream(dev) if s is None else s if isinstance(s, int) else s.cuda_stream


def _tensor(x, call, name, dtype, shape, dev):
    """Address of a contiguous tensor of that type and shape (None: any) on device dev."""
    if x is None or x.dtype is not dtype or x.get_device() != dev or not x.is_contiguous() or (shape is not None and x.shape != shape):
        _refuse(x, f"{call}: {name}", dtype, shape)
    return x.data_ptr()


def _optional(x, call, name, dtype, shape, dev):
    return None if x is None else _tensor(x, call, name, dtype, shape, dev)


def _refuse(x, what, dtype, shape):
    if x is None:
        raise BitMoeError(1, f"{what}: null tensor")
    if x.dtype is not dtype:
        raise BitMoeError(1, f"{what}: dtype {x.dtype}, expected {dtype}")
    if shape is not None and x.shape != shape:
        raise BitMoeError(1, f"{what}: shape {tuple(x.shape)}, expected {tuple(shape)}")
    if not x.is_contiguous():
        raise BitMoeError(1, f"{what}: not contiguous")
    raise BitMoeError(1, f"{what}: on {x.device}, expected the current CUDA device")


def kv8_cache(format, slots, ctx_cap, kv_heads, head_dim, K, V, Ks, Vs):
    """The bm_kv8_cache of four tensors: codes uint8 [slots][kv_heads][ctx_cap][head_dim],
    scales fp32 [slots][kv_heads][ctx_cap].  It keeps the tensors alive."""
    t, dev, rows = _t(), _here(), (slots, kv_heads, ctx_cap)
    c = bm_kv8_cache(format, slots, ctx_cap, kv_heads, head_dim,
                     *[_tensor(x, "kv8_cache", n, t.uint8, rows + (head_dim,), dev) for n, x in (("K", K), ("V", V))],
                     *[_tensor(x, "kv8_cache", n, t.float32, rows, dev) for n, x in (("Ks", Ks), ("Vs", Vs))])
    c.tensors, c.device, c.address = (K, V, Ks, Vs), dev, ctypes.addressof(c)
    return c


def kv8_rope(norm=False, q_norm=None, k_norm=None, eps=1e-6, inv_freq=None):
    """The bm_kv8_rope of its tensors (bf16 norm weights [head_dim], fp32 inv_freq [head_dim / 2]), which it keeps alive."""
    t, dev = _t(), _here()
    r = bm_kv8_rope(int(norm), eps, _optional(q_norm, "kv8_rope", "q_norm", t.bfloat16, None, dev),
                    _optional(k_norm, "kv8_rope", "k_norm", t.bfloat16, None, dev),
                    _optional(inv_freq, "kv8_rope", "inv_freq", t.float32, None, dev))
    r.tensors, r.device, r.address = (q_norm, k_norm, inv_freq), dev, ctypes.addressof(r)
    # the head_dim each tensor fits
    r.fits = {x.numel() * f for x, f in ((q_norm, 1), (k_norm, 1), (inv_freq, 2)) if x is not None}
    return r


def _on_device(c, what, dev):
    if getattr(c, "device", None) != dev:
        if not hasattr(c, "device"):
            raise BitMoeError(1, f"{what}: {type(c).__name__}, expected one that kv8_cache() or kv8_rope() made")
        raise BitMoeError(1, f"{what}: its tensors are on cuda:{c.device}, expected the current CUDA device")


def _shape(x, call, name, dims):
    """Shape of a tensor of that many dimensions."""
    if x is None or x.dim() != dims:
        raise BitMoeError(1, f"{call}: {name}: " + ("null tensor" if x is None else f"{x.dim()} dimensions, expected {dims}"))
    return x.shape


def kv8_append(cache, qkv, rope, slots, index, Q, rope_pos=None, stream=None):
    """qkv: bf16 [T][>= (q_heads + 2 kv_heads) * head_dim], rows may be strided; Q: bf16 [T][q_heads][head_dim]."""
    t, dev = _t(), _here()
    _on_device(cache, "kv8_append: cache", dev)
    _on_device(rope, "kv8_append: rope", dev)
    T, qh, d = _shape(Q, "kv8_append", "Q", 3)
    rows, width = _shape(qkv, "kv8_append", "qkv", 2)
    if rows != T or width < (qh + 2 * cache.kv_heads) * d or d != cache.head_dim:
        raise BitMoeError(1, f"kv8_append: qkv {tuple(qkv.shape)} and Q {tuple(Q.shape)} do not fit the cache")
    if qkv.dtype is not t.bfloat16 or qkv.stride(1) != 1 or qkv.get_device() != dev:
        raise BitMoeError(1, "kv8_append: qkv must be bf16 rows of unit stride on the current CUDA device")
    if rope.fits and rope.fits != {d}:
        raise BitMoeError(1, f"kv8_append: q_norm and k_norm need {d} elements, inv_freq {d // 2}")
    ld = qkv.stride(0) if T > 1 else width + -width % 8
    i32, n = t.int32, (T,)
    _check(lib().kv8_append(cache.address, qkv.data_ptr(), ld, qh, rope.address, _tensor(slots, "kv8_append", "slots", i32, n, dev),
                            _tensor(index, "kv8_append", "index", i32, n, dev),
                            _optional(rope_pos, "kv8_append", "rope_pos", i32, n, dev),
                            _tensor(Q, "kv8_append", "Q", t.bfloat16, None, dev), T, _stream(stream, dev)))


def kv8_read(cache, slot, first, count, K_out, V_out, stream=None):
    """K_out, V_out: bf16 [kv_heads][count][head_dim]."""
    t, dev = _t(), _here()
    _on_device(cache, "kv8_read: cache", dev)
    shape = (cache.kv_heads, count, cache.head_dim)
    _check(lib().kv8_read(cache.address, slot, first, count, _tensor(K_out, "kv8_read", "K_out", t.bfloat16, shape, dev),
                          _tensor(V_out, "kv8_read", "V_out", t.bfloat16, shape, dev), _stream(stream, dev)))


def kv8_workspace_bytes(B, q_heads, kv_heads, head_dim, ctx_cap, prefix_len=0):
    return lib().kv8_workspace_bytes(B, q_heads, kv_heads, head_dim, ctx_cap, prefix_len)


def _attend_args(what, cache, Q, slots, lens, O, ws, scale, dev):
    t = _t()
    _on_device(cache, what, dev)
    shape = _shape(Q, what, "Q", 3)
    B, qh, d = shape
    if d != cache.head_dim:
        raise BitMoeError(1, f"{what}: Q of head_dim {d}, the cache of {cache.head_dim}")
    return (_tensor(Q, what, "Q", t.bfloat16, None, dev), _tensor(slots, what, "slots", t.int32, (B,), dev),
            _tensor(lens, what, "lens", t.int32, (B,), dev), qh, d ** -0.5 if scale is None else scale,
            _tensor(O, what, "O", t.bfloat16, shape, dev), B, _tensor(ws, what, "ws", t.uint8, None, dev), ws.numel())


def kv8_attend(cache, Q, slots, lens, O, ws, scale=None, stream=None):
    """Q, O: bf16 [B][q_heads][head_dim]; ws: uint8 tensor of kv8_workspace_bytes(...); scale: 1 / sqrt(head_dim) if None."""
    dev = _here()
    args = _attend_args("kv8_attend", cache, Q, slots, lens, O, ws, scale, dev)
    _check(lib().kv8_attend(cache.address, *args, _stream(stream, dev)))


def kv8_attend_prefix(cache, prefix, prefix_slot, prefix_len, Q, slots, lens, O, ws, scale=None, stream=None):
    """kv8_attend behind positions 0..prefix_len-1 of slot prefix_slot of `prefix` (a kv8_cache, or `cache` itself)."""
    dev = _here()
    _on_device(prefix, "kv8_attend_prefix: prefix", dev)
    args = _attend_args("kv8_attend_prefix", cache, Q, slots, lens, O, ws, scale, dev)
    _check(lib().kv8_attend_prefix(cache.address, prefix.address, prefix_slot, prefix_len, *args, _stream(stream, dev)))


def kv8_plan_bytes(B, T, q_heads, kv_heads):
    return lib().kv8_plan_bytes(B, T, q_heads, kv_heads)


def kv8_plan(cache, q_heads, slots, lens, counts, row_start, after, row_slot, row_index, row_pos, plan, parents=None, stream=None):
    """slots, lens, counts, after: int32 [B]; row_start: int32 [B + 1]; row_slot, row_index, parents, row_pos (the last two
    or None): int32 [T]; plan: uint8 tensor of kv8_plan_bytes(...)."""
    t, dev, w = _t(), _here(), "kv8_plan"
    _on_device(cache, "kv8_plan: cache", dev)
    (B,), (T,) = _shape(slots, w, "slots", 1), _shape(row_slot, w, "row_slot", 1)
    i32, b, r = t.int32, (B,), (T,)
    _check(lib().kv8_plan(cache.address, q_heads, _tensor(slots, w, "slots", i32, b, dev), _tensor(lens, w, "lens", i32, b, dev),
                          _tensor(counts, w, "counts", i32, b, dev), _optional(parents, w, "parents", i32, r, dev),
                          _tensor(row_start, w, "row_start", i32, (B + 1,), dev), _tensor(after, w, "after", i32, b, dev),
                          _tensor(row_slot, w, "row_slot", i32, r, dev), _tensor(row_index, w, "row_index", i32, r, dev),
                          _optional(row_pos, w, "row_pos", i32, r, dev), B, T, _tensor(plan, w, "plan", t.uint8, None, dev),
                          plan.numel(), _stream(stream, dev)))


def kv8_rows_workspace_bytes(B, T, q_heads, kv_heads, head_dim, ctx_cap):
    return lib().kv8_rows_workspace_bytes(B, T, q_heads, kv_heads, head_dim, ctx_cap)


def kv8_attend_rows(cache, plan, Q, O, B, ws, scale=None, stream=None):
    """Q, O: bf16 [T][q_heads][head_dim], plan: of kv8_plan for B streams and T rows; ws: uint8 tensor of
    kv8_rows_workspace_bytes(...); scale: 1 / sqrt(head_dim) if None."""
    t, dev, w = _t(), _here(), "kv8_attend_rows"
    _on_device(cache, "kv8_attend_rows: cache", dev)
    shape = _shape(Q, w, "Q", 3)
    T, qh, d = shape
    if d != cache.head_dim:
        raise BitMoeError(1, f"{w}: Q of head_dim {d}, the cache of {cache.head_dim}")
    _check(lib().kv8_attend_rows(cache.address, _tensor(plan, w, "plan", t.uint8, None, dev), plan.numel(),
                                 _tensor(Q, w, "Q", t.bfloat16, None, dev), qh, d ** -0.5 if scale is None else scale,
                                 _tensor(O, w, "O", t.bfloat16, shape, dev), B, T, _tensor(ws, w, "ws", t.uint8, None, dev),
                                 ws.numel(), _stream(stream, dev)))


def kv8_rows_status(stream=None):
    """Waits for the stream; raises if a wait inside kv8_attend_rows gave up on this device since the last call."""
    dev = _here()
    _check(lib().kv8_rows_status(_stream(stream, dev) if dev >= 0 else None))   # without a device: BM_ERR_CUDA


def bm_test_kv8_rows_hold(what, cta=0, at=0):
    _check(lib().bm_test_kv8_rows_hold(int(what), int(cta), int(at)))


def kv8_tree_accept(plan, tokens, ids, path, kept, fresh, n_fresh, lens, stream=None):
    """tokens, ids: int32 [T]; path, fresh: int32 [B][KV8_DRAFTS]; kept, n_fresh, lens: int32 [B]."""
    t, dev, w = _t(), _here(), "kv8_tree_accept"
    (T,), (B,) = _shape(tokens, w, "tokens", 1), _shape(kept, w, "kept", 1)
    i32, b, many = t.int32, (B,), (B, KV8_DRAFTS)
    _check(lib().kv8_tree_accept(_tensor(plan, w, "plan", t.uint8, None, dev), plan.numel(), _tensor(tokens, w, "tokens", i32, None, dev),
                                 _tensor(ids, w, "ids", i32, (T,), dev), _tensor(path, w, "path", i32, many, dev),
                                 _tensor(kept, w, "kept", i32, b, dev), _tensor(fresh, w, "fresh", i32, many, dev),
                                 _tensor(n_fresh, w, "n_fresh", i32, b, dev), _tensor(lens, w, "lens", i32, b, dev), B, T,
                                 _stream(stream, dev)))


def kv8_tree_keep(cache, plan, path, kept, stream=None):
    """path: int32 [B][KV8_DRAFTS]; kept: int32 [B]."""
    t, dev, w = _t(), _here(), "kv8_tree_keep"
    _on_device(cache, "kv8_tree_keep: cache", dev)
    (B,) = _shape(kept, w, "kept", 1)
    _check(lib().kv8_tree_keep(cache.address, _tensor(plan, w, "plan", t.uint8, None, dev), plan.numel(),
                               _tensor(path, w, "path", t.int32, (B, KV8_DRAFTS), dev), _tensor(kept, w, "kept", t.int32, (B,), dev), B,
                               _stream(stream, dev)))


def bm_sample(logits, temperature, top_k, top_p, min_p, u, ids, logprobs=None, stream=None):
    """logits: fp32 or bf16 [B][V], rows may be strided; temperature, top_p, min_p (fp32) and top_k (int32) [B] or
    None; u: fp32 [B]; ids: int32 [B]; logprobs: fp32 [B] or None."""
    t, dev = _t(), _here()
    B, V = _shape(logits, "bm_sample", "logits", 2)
    half = logits.dtype is t.bfloat16
    if not (half or logits.dtype is t.float32) or logits.stride(1) != 1 or logits.get_device() != dev:
        raise BitMoeError(1, "bm_sample: logits must be fp32 or bf16 rows of unit stride on the current CUDA device")
    f32, n = t.float32, (B,)
    _check(lib().bm_sample(logits.data_ptr(), int(half), logits.stride(0) if B > 1 else V, V, B,
                           _optional(temperature, "bm_sample", "temperature", f32, n, dev),
                           _optional(top_k, "bm_sample", "top_k", t.int32, n, dev),
                           _optional(top_p, "bm_sample", "top_p", f32, n, dev),
                           _optional(min_p, "bm_sample", "min_p", f32, n, dev), _tensor(u, "bm_sample", "u", f32, n, dev),
                           _tensor(ids, "bm_sample", "ids", t.int32, n, dev),
                           _optional(logprobs, "bm_sample", "logprobs", f32, n, dev), _stream(stream, dev)))


# --------------------------------------------------------------- host slot map

def bm_slot_map_create(max_streams, ctx_cap):
    h = ctypes.c_void_p()
    _check(lib().bm_slot_map_create(max_streams, ctx_cap, ctypes.byref(h)))
    return h.value


def bm_slot_map_destroy(m):
    lib().bm_slot_map_destroy(m)


def bm_slot_map_acquire(m, length):
    s = ctypes.c_int(-1)
    _check(lib().bm_slot_map_acquire(m, int(length), ctypes.byref(s)))
    return s.value


def bm_slot_map_release(m, slot):
    _check(lib().bm_slot_map_release(m, int(slot)))


def bm_slot_map_check_batch(m, slots):
    arr = _i32_array(slots)
    _check(lib().bm_slot_map_check_batch(m, ctypes.addressof(arr), len(slots)))


def bm_slot_map_advance(m, slots):
    arr = _i32_array(slots)
    _check(lib().bm_slot_map_advance(m, ctypes.addressof(arr), len(slots)))


def bm_slot_map_length(m, slot):
    n = ctypes.c_int(0)
    _check(lib().bm_slot_map_length(m, int(slot), ctypes.byref(n)))
    return n.value


def bm_slot_map_active_count(m):
    return lib().bm_slot_map_active_count(m)
