"""Python binding of libmoe_v41 (include/moe_v41.h, moe_v41_cache.h,
moe_v41_ops.h and moe_v41_attn.h): argument marshalling, and the types that
an address does not say (lengths, positions, angles).

Every step of the MoE layer runs in the library's sm_103a kernels; this
module converts torch tensors (device memory) and streams into the C-ABI's
plain pointers and raises on a non-zero return code.  There is no fallback:
if the compiled library is missing, loading fails loudly.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
SO = os.path.join(_HERE, "_lib", "libmoe_v41.so")

MOE_PATH_AUTO, MOE_PATH_DECODE, MOE_PATH_PREFILL = 0, 1, 2
MOE_SCORE_SQRTSOFTPLUS, MOE_SCORE_SIGMOID, MOE_SCORE_SOFTMAX = 0, 1, 2
MOE_SHARED_BF16, MOE_SHARED_KQUANT = 0, 1
MOE_OK, MOE_ERR_ARG, MOE_ERR_ALIGN, MOE_ERR_WORKSPACE, MOE_ERR_CUDA = 0, 1, 2, 3, 4
MOE_STATUS_NAN_KEY, MOE_STATUS_MISSING_EXPERT, MOE_STATUS_TIMEOUT, MOE_STATUS_BAD_PAGE = 1, 2, 4, 8
MOE_T_F32, MOE_T_BF16, MOE_T_F16 = 0, 1, 2
MOE_NORM_NONE, MOE_NORM_RMS, MOE_NORM_LAYER = 0, 1, 2
MOE_GATE_NONE, MOE_GATE_ROW, MOE_GATE_TOKEN = 0, 1, 2
MOE_ROPE_HALF, MOE_ROPE_INTERLEAVED = 0, 1
MOE_ROPE_SCALE_NONE, MOE_ROPE_SCALE_LINEAR, MOE_ROPE_SCALE_BASE, MOE_ROPE_SCALE_PARTS = 0, 1, 2, 3


class MoeError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: moe_v41 error {code} ({strerror(code)})")
        self.code = code


class moe_v41_cfg(ctypes.Structure):
    _fields_ = [("dim", ctypes.c_int32), ("inter", ctypes.c_int32), ("n_routed", ctypes.c_int32),
                ("topk", ctypes.c_int32), ("gate_temp", ctypes.c_float), ("norm_topk_prob", ctypes.c_int32),
                ("route_scale", ctypes.c_float), ("swiglu_limit", ctypes.c_float), ("max_tokens", ctypes.c_int32),
                ("path", ctypes.c_int32), ("wait_timeout_us", ctypes.c_uint32), ("score_func", ctypes.c_int32)]


class moe_v41_cache_cfg(ctypes.Structure):
    _fields_ = [("n_layers", ctypes.c_int32), ("n_routed", ctypes.c_int32), ("n_slots", ctypes.c_int32),
                ("slot_bytes", ctypes.c_uint64), ("off_w1", ctypes.c_uint64), ("off_w3", ctypes.c_uint64),
                ("off_w2", ctypes.c_uint64), ("arena", ctypes.c_void_p), ("slots", ctypes.c_void_p),
                ("tables", ctypes.c_void_p)]


class moe_v41_cache_stats(ctypes.Structure):
    _fields_ = [("hits", ctypes.c_uint64), ("misses", ctypes.c_uint64), ("evictions", ctypes.c_uint64),
                ("bytes_copied", ctypes.c_uint64), ("prefetched", ctypes.c_uint64),
                ("prefetch_hits", ctypes.c_uint64)]


class moe_v41_q4_cfg(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int32), ("k", ctypes.c_int32), ("group", ctypes.c_int32), ("x_type", ctypes.c_int32),
                ("scale_type", ctypes.c_int32), ("out_type", ctypes.c_int32), ("max_tokens", ctypes.c_int32)]


class moe_v41_norm_cfg(ctypes.Structure):
    _fields_ = [("dim", ctypes.c_int32), ("post_kind", ctypes.c_int32), ("pre_kind", ctypes.c_int32),
                ("y_type", ctypes.c_int32), ("h_type", ctypes.c_int32), ("x_type", ctypes.c_int32),
                ("w_type", ctypes.c_int32), ("gate_kind", ctypes.c_int32), ("gate_type", ctypes.c_int32),
                ("gate_group", ctypes.c_int32), ("eps", ctypes.c_float), ("residual_scale", ctypes.c_float),
                ("block_scale", ctypes.c_float)]


class moe_v41_logprob_cfg(ctypes.Structure):
    _fields_ = [("vocab", ctypes.c_int32), ("logit_type", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("temperature", ctypes.c_float)]


class moe_v41_rope_cfg(ctypes.Structure):
    _fields_ = [("head_dim", ctypes.c_int32), ("rot_dim", ctypes.c_int32), ("rot_first", ctypes.c_int32),
                ("layout", ctypes.c_int32), ("x_type", ctypes.c_int32), ("inverse", ctypes.c_int32),
                ("magnitude", ctypes.c_float)]


class moe_v41_kv_cfg(ctypes.Structure):
    _fields_ = [("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("n_pages", ctypes.c_int32), ("type", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("page_pitch", ctypes.c_int64), ("token_pitch", ctypes.c_int64), ("head_pitch", ctypes.c_int64)]


class moe_v41_seqs(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("max_pages", ctypes.c_int32), ("cu_new", ctypes.c_void_p),
                ("kv_len", ctypes.c_void_p), ("table", ctypes.c_void_p), ("ld_table", ctypes.c_int64)]


class moe_v41_attn_cfg(ctypes.Structure):
    _fields_ = [("kv", moe_v41_kv_cfg), ("heads", ctypes.c_int32), ("causal", ctypes.c_int32),
                ("window", ctypes.c_int32), ("scale", ctypes.c_float)]


_lib = None


def lib():
    global _lib
    if _lib is None:
        if not os.path.exists(SO):
            raise RuntimeError(f"{SO} is missing: the CUDA library must be built (__graft_entry__.build())")
        L = ctypes.CDLL(SO)
        vp, i32, sz, cfgp = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.POINTER(moe_v41_cfg)
        L.moe_v41_workspace_bytes.restype = sz
        L.moe_v41_workspace_bytes.argtypes = [cfgp]
        L.moe_v41_workspace_init.argtypes = [vp, sz, vp]
        L.moe_v41_quantize_q8_1.argtypes = [vp, i32, i32, i32, vp, vp]
        L.moe_v41_select_from_logits.argtypes = [cfgp, vp, i32, vp, vp, vp, vp, sz, vp]
        L.moe_v41_route.argtypes = [cfgp, vp, i32, vp, vp, vp, vp, vp, vp, sz, vp]
        L.moe_v41_forward.argtypes = [cfgp, vp, i32, vp, vp, vp, i32, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.moe_v41_select_from_logits_vl.argtypes = [cfgp, vp, i32, vp, vp, vp, vp, vp, vp, sz, vp]
        L.moe_v41_route_vl.argtypes = [cfgp, vp, i32, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.moe_v41_forward_vl.argtypes = [cfgp, vp, i32, vp, vp, vp, vp, vp, i32, vp, vp, vp, vp, vp, vp, vp, vp, sz,
                                         vp]
        L.moe_v41_read_status.argtypes = [vp, vp, ctypes.POINTER(ctypes.c_uint32), i32]
        L.moe_v41_forward_noalloc.argtypes = [cfgp, vp, i32, vp, vp, vp, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp]
        L.moe_v41_kernel_launches.argtypes = [cfgp, i32, i32]
        L.moe_v41_kernel_launches.restype = i32
        L.moe_v41_strerror.restype = ctypes.c_char_p
        L.moe_v41_strerror.argtypes = [i32]
        cp = ctypes.c_void_p
        L.moe_v41_cache_create.argtypes = [ctypes.POINTER(moe_v41_cache_cfg), vp, ctypes.POINTER(cp)]
        L.moe_v41_cache_destroy.argtypes = [cp]
        L.moe_v41_cache_fetch.argtypes = [cp, i32, vp, i32, i32, vp]
        L.moe_v41_cache_wait.argtypes = [cp, i32, vp]
        L.moe_v41_cache_reads.argtypes = [cp, i32, vp, i32, vp]
        L.moe_v41_cache_slot_of.argtypes = [cp, i32, i32]
        L.moe_v41_cache_get_stats.argtypes = [cp, ctypes.POINTER(moe_v41_cache_stats)]
        L.moe_v41_forward_streamed.argtypes = [cfgp, cp, i32, vp, i32, vp, vp, vp, vp, i32, i32, vp, vp, vp, vp, vp,
                                               vp, vp, sz, vp, vp, vp]
        i64 = ctypes.c_int64
        q4p, nmp, lpp = (ctypes.POINTER(c) for c in (moe_v41_q4_cfg, moe_v41_norm_cfg, moe_v41_logprob_cfg))
        L.moe_v41_q4_workspace_bytes.restype = sz
        L.moe_v41_q4_workspace_bytes.argtypes = [q4p]
        L.moe_v41_q4_linear.argtypes = [q4p, vp, i32, i64, vp, vp, vp, vp, i64, vp, sz, vp]
        L.moe_v41_block_norm.argtypes = [nmp, i32, vp, i64, vp, vp, vp, i64, vp, i64, vp, i64, vp, vp, vp, i64, vp]
        L.moe_v41_token_logprobs.argtypes = [lpp, vp, i32, i64, vp, i64, vp, vp, vp, vp, vp, vp, vp, vp]
        rpp, kvp, sqp, atp = (ctypes.POINTER(c) for c in (moe_v41_rope_cfg, moe_v41_kv_cfg, moe_v41_seqs,
                                                          moe_v41_attn_cfg))
        f64 = ctypes.c_double
        L.moe_v41_rope_freqs.argtypes = [i32, f64, i32, f64, i32, vp, vp]
        L.moe_v41_rope.argtypes = [rpp, i32, i32, vp, i64, i64, vp, vp, vp, i64, i64, vp]
        L.moe_v41_kv_append.argtypes = [kvp, rpp, sqp, i32, vp, i64, vp, i64, vp, vp, i32, vp, i64, vp, i64, vp, vp,
                                        vp, vp]
        L.moe_v41_attn_workspace_bytes.restype = sz
        L.moe_v41_attn_workspace_bytes.argtypes = [atp]
        L.moe_v41_paged_attention.argtypes = [atp, sqp, i32, i32, vp, i64, vp, vp, vp, i64, vp, i64, vp, sz, vp]
        for f in ("moe_v41_workspace_init", "moe_v41_quantize_q8_1", "moe_v41_select_from_logits", "moe_v41_route",
                  "moe_v41_forward", "moe_v41_read_status", "moe_v41_forward_noalloc",
                  "moe_v41_select_from_logits_vl", "moe_v41_route_vl", "moe_v41_forward_vl", "moe_v41_cache_create",
                  "moe_v41_cache_destroy", "moe_v41_cache_fetch", "moe_v41_cache_wait", "moe_v41_cache_reads",
                  "moe_v41_cache_slot_of", "moe_v41_cache_get_stats", "moe_v41_forward_streamed",
                  "moe_v41_q4_linear", "moe_v41_block_norm", "moe_v41_token_logprobs", "moe_v41_rope_freqs",
                  "moe_v41_rope", "moe_v41_kv_append", "moe_v41_paged_attention"):
            getattr(L, f).restype = i32
        _lib = L
    return _lib


def strerror(code: int) -> str:
    return lib().moe_v41_strerror(code).decode()


def _p(t):
    """device address of a tensor, or an int address, or None"""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


_raw = None


def _current_stream() -> int:
    """torch's current stream as an address; without the stream object that
    torch.cuda.current_stream() builds, which costs as much as a launch"""
    global _raw
    if _raw is None:
        import torch
        torch.cuda.init()
        get = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if get is None:
            _raw = lambda: torch.cuda.current_stream().cuda_stream  # noqa: E731
        else:
            _raw = lambda: get(torch.cuda.current_device())  # noqa: E731
    return _raw()


def _s(stream):
    if stream is None:
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _nbytes(t):
    return t.numel() * t.element_size()


def _check(rc: int, what: str):
    if rc != MOE_OK:
        raise MoeError(rc, what)


def make_cfg(dim, inter, n_routed, topk, gate_temp=1.0, norm_topk_prob=True, route_scale=1.5, swiglu_limit=10.0,
             max_tokens=1, path=MOE_PATH_AUTO, wait_timeout_us=0, score_func=MOE_SCORE_SQRTSOFTPLUS) -> moe_v41_cfg:
    return moe_v41_cfg(dim, inter, n_routed, topk, gate_temp, int(bool(norm_topk_prob)), route_scale, swiglu_limit,
                       max_tokens, path, wait_timeout_us, score_func)


def moe_v41_workspace_bytes(cfg: moe_v41_cfg) -> int:
    return int(lib().moe_v41_workspace_bytes(ctypes.byref(cfg)))


def moe_v41_workspace_init(ws, stream=None):
    _check(lib().moe_v41_workspace_init(_p(ws), _nbytes(ws), _s(stream)), "moe_v41_workspace_init")


def moe_v41_quantize_q8_1(x, x_is_f32: bool, rows: int, cols: int, q8_out, stream=None):
    _check(lib().moe_v41_quantize_q8_1(_p(x), int(x_is_f32), rows, cols, _p(q8_out), _s(stream)),
           "moe_v41_quantize_q8_1")


def moe_v41_select_from_logits(cfg, logits, m, bias, topk_w, topk_idx, ws, stream=None):
    _check(lib().moe_v41_select_from_logits(ctypes.byref(cfg), _p(logits), m, _p(bias), _p(topk_w), _p(topk_idx),
                                            _p(ws), _nbytes(ws), _s(stream)), "moe_v41_select_from_logits")


def moe_v41_select_from_logits_vl(cfg, logits, m, bias, bias_vl, image_mask, topk_w, topk_idx, ws, stream=None):
    _check(lib().moe_v41_select_from_logits_vl(ctypes.byref(cfg), _p(logits), m, _p(bias), _p(bias_vl),
                                               _p(image_mask), _p(topk_w), _p(topk_idx), _p(ws), _nbytes(ws),
                                               _s(stream)), "moe_v41_select_from_logits_vl")


def moe_v41_route_vl(cfg, x, m, router_w, bias, bias_vl, image_mask, logits_out, topk_w, topk_idx, ws, stream=None):
    _check(lib().moe_v41_route_vl(ctypes.byref(cfg), _p(x), m, _p(router_w), _p(bias), _p(bias_vl), _p(image_mask),
                                  _p(logits_out), _p(topk_w), _p(topk_idx), _p(ws), _nbytes(ws), _s(stream)),
           "moe_v41_route_vl")


def moe_v41_route(cfg, x, m, router_w, bias, logits_out, topk_w, topk_idx, ws, stream=None):
    _check(lib().moe_v41_route(ctypes.byref(cfg), _p(x), m, _p(router_w), _p(bias), _p(logits_out), _p(topk_w),
                               _p(topk_idx), _p(ws), _nbytes(ws), _s(stream)), "moe_v41_route")


def moe_v41_forward(cfg, x, m, router_w, bias, expert_ptrs, shared_kind, sh_w1, sh_w3, sh_w2, out, topk_w, topk_idx,
                    logits_out, ws, stream=None):
    _check(lib().moe_v41_forward(ctypes.byref(cfg), _p(x), m, _p(router_w), _p(bias), _p(expert_ptrs), shared_kind,
                                 _p(sh_w1), _p(sh_w3), _p(sh_w2), _p(out), _p(topk_w), _p(topk_idx), _p(logits_out),
                                 _p(ws), _nbytes(ws), _s(stream)), "moe_v41_forward")


def moe_v41_forward_vl(cfg, x, m, router_w, bias, bias_vl, image_mask, expert_ptrs, shared_kind, sh_w1, sh_w3, sh_w2,
                       out, topk_w, topk_idx, logits_out, ws, stream=None):
    _check(lib().moe_v41_forward_vl(ctypes.byref(cfg), _p(x), m, _p(router_w), _p(bias), _p(bias_vl), _p(image_mask),
                                    _p(expert_ptrs), shared_kind, _p(sh_w1), _p(sh_w3), _p(sh_w2), _p(out),
                                    _p(topk_w), _p(topk_idx), _p(logits_out), _p(ws), _nbytes(ws), _s(stream)),
           "moe_v41_forward_vl")


NOALLOC_SCRATCH_BYTES = 512 << 10


def moe_v41_forward_noalloc(cfg, x, m, router_w, bias, expert_ptrs, shared_kind, sh_w1, sh_w3, sh_w2, out, topk_w,
                            topk_idx, logits_out=None, status_out=None, stream=None):
    """moe_v41_forward without a workspace: the library's own fixed scratch
    array (512 KiB per device) is used.  For callers that cannot allocate device
    memory when they call; see include/moe_v41.h for the limits."""
    _check(lib().moe_v41_forward_noalloc(ctypes.byref(cfg), _p(x), m, _p(router_w), _p(bias), _p(expert_ptrs),
                                         shared_kind, _p(sh_w1), _p(sh_w3), _p(sh_w2), _p(out), _p(topk_w),
                                         _p(topk_idx), _p(logits_out), _p(status_out), _s(stream)),
           "moe_v41_forward_noalloc")


def moe_v41_kernel_launches(cfg, m: int, shared_kind: int) -> int:
    return int(lib().moe_v41_kernel_launches(ctypes.byref(cfg), int(m), int(shared_kind)))


def moe_v41_read_status(ws, stream=None, clear: bool = False) -> int:
    v = ctypes.c_uint32(0)
    _check(lib().moe_v41_read_status(_p(ws), _s(stream), ctypes.byref(v), int(clear)), "moe_v41_read_status")
    return v.value


# ------------------------------------------------------------ expert cache

def _ids(experts):
    a = [int(e) for e in experts]
    return (ctypes.c_int32 * max(1, len(a)))(*a), len(a)


class ExpertCache:
    """include/moe_v41_cache.h: routed experts of a host arena held in a
    least-recently-used set of HBM slots, with the per-layer slot pointer
    tables moe_v41_forward reads.  arena: page-locked host tensor (or address)
    of [n_layers, n_routed, slot_bytes]; slots: device [n_slots, slot_bytes];
    tables: device int64 [n_layers, n_routed, 3].  With slots and tables None
    the cache only simulates the replacement policy (no CUDA call)."""

    def __init__(self, n_layers, n_routed, n_slots, slot_bytes, off_w1, off_w3, off_w2, arena=None, slots=None,
                 tables=None, stream=None):
        self.sim = slots is None and tables is None
        self.cfg = moe_v41_cache_cfg(n_layers, n_routed, n_slots, slot_bytes, off_w1, off_w3, off_w2, _p(arena),
                                     _p(slots), _p(tables))
        self._keep = (arena, slots, tables)
        self._h = ctypes.c_void_p()
        _check(lib().moe_v41_cache_create(ctypes.byref(self.cfg), None if self.sim else _s(stream),
                                          ctypes.byref(self._h)), "moe_v41_cache_create")
        self.tables = tables

    def _st(self, stream):
        return None if self.sim else _s(stream)

    def fetch(self, layer, experts, prefetch=False, copy_stream=None):
        a, n = _ids(experts)
        _check(lib().moe_v41_cache_fetch(self._h, layer, a, n, int(bool(prefetch)), self._st(copy_stream)),
               "moe_v41_cache_fetch")

    def wait(self, layer, stream=None):
        _check(lib().moe_v41_cache_wait(self._h, layer, self._st(stream)), "moe_v41_cache_wait")

    def reads(self, layer, experts=None, stream=None):
        if experts is None:
            _check(lib().moe_v41_cache_reads(self._h, layer, None, 0, self._st(stream)), "moe_v41_cache_reads")
        else:
            a, n = _ids(experts)
            _check(lib().moe_v41_cache_reads(self._h, layer, a, n, self._st(stream)), "moe_v41_cache_reads")

    def slot_of(self, layer, expert) -> int:
        return int(lib().moe_v41_cache_slot_of(self._h, layer, expert))

    def stats(self) -> dict:
        st = moe_v41_cache_stats()
        _check(lib().moe_v41_cache_get_stats(self._h, ctypes.byref(st)), "moe_v41_cache_get_stats")
        return {f: int(getattr(st, f)) for f, _ in moe_v41_cache_stats._fields_}

    def table(self, layer):
        """the device slot pointer table of one layer ([n_routed, 3] int64 view)"""
        return self.tables[layer]

    def close(self):
        if self._h:
            lib().moe_v41_cache_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def moe_v41_forward_streamed(cfg, cache: ExpertCache, layer, x, m, router_w, bias, next_router_w, next_bias,
                             prefetch_k, shared_kind, sh_w1, sh_w3, sh_w2, out, topk_w, topk_idx, ws, host_picks,
                             stream=None, copy_stream=None):
    _check(lib().moe_v41_forward_streamed(ctypes.byref(cfg), cache._h, layer, _p(x), m, _p(router_w), _p(bias),
                                          _p(next_router_w), _p(next_bias), prefetch_k, shared_kind, _p(sh_w1),
                                          _p(sh_w3), _p(sh_w2), _p(out), _p(topk_w), _p(topk_idx), _p(ws),
                                          _nbytes(ws), _p(host_picks), _s(stream), _s(copy_stream)),
           "moe_v41_forward_streamed")


# ------------------------------------- operators around the MoE layer (moe_v41_ops.h)

def make_q4_cfg(n, k, group=128, x_type=MOE_T_BF16, scale_type=MOE_T_F16, out_type=MOE_T_F32,
                max_tokens=1) -> moe_v41_q4_cfg:
    return moe_v41_q4_cfg(n, k, group, x_type, scale_type, out_type, max_tokens)


def moe_v41_q4_workspace_bytes(cfg: moe_v41_q4_cfg) -> int:
    return int(lib().moe_v41_q4_workspace_bytes(ctypes.byref(cfg)))


def moe_v41_q4_linear(cfg, x, m, ldx, w, scales, zeros, out, ldo, ws, stream=None):
    _check(lib().moe_v41_q4_linear(ctypes.byref(cfg), _p(x), m, ldx, _p(w), _p(scales), _p(zeros), _p(out), ldo,
                                   _p(ws), _nbytes(ws), _s(stream)), "moe_v41_q4_linear")


def make_norm_cfg(dim, post_kind=MOE_NORM_RMS, pre_kind=MOE_NORM_RMS, y_type=MOE_T_F32, h_type=MOE_T_BF16,
                  x_type=MOE_T_BF16, w_type=MOE_T_F32, gate_kind=MOE_GATE_NONE, gate_type=MOE_T_F32, gate_group=1,
                  eps=1e-6, residual_scale=1.0, block_scale=1.0) -> moe_v41_norm_cfg:
    return moe_v41_norm_cfg(dim, post_kind, pre_kind, y_type, h_type, x_type, w_type, gate_kind, gate_type,
                            gate_group, eps, residual_scale, block_scale)


def moe_v41_block_norm(cfg, m, y, ldy, post_w, post_b, gate, ldg, h, ldh, h_out, ldh_out, pre_w, pre_b, x_out, ldx,
                       stream=None):
    _check(lib().moe_v41_block_norm(ctypes.byref(cfg), m, _p(y), ldy, _p(post_w), _p(post_b), _p(gate), ldg, _p(h),
                                    ldh, _p(h_out), ldh_out, _p(pre_w), _p(pre_b), _p(x_out), ldx, _s(stream)),
           "moe_v41_block_norm")


def make_logprob_cfg(vocab, logit_type=MOE_T_F32, top_k=0, temperature=1.0) -> moe_v41_logprob_cfg:
    return moe_v41_logprob_cfg(vocab, logit_type, top_k, temperature)


def moe_v41_token_logprobs(cfg, logits, m, ld, allowed, ld_allowed, target, logprob, rank, lse, entropy,
                           top_logprob, top_id, stream=None):
    _check(lib().moe_v41_token_logprobs(ctypes.byref(cfg), _p(logits), m, ld, _p(allowed), ld_allowed, _p(target),
                                        _p(logprob), _p(rank), _p(lse), _p(entropy), _p(top_logprob), _p(top_id),
                                        _s(stream)), "moe_v41_token_logprobs")


# ------------------------------------- operators of an attention block (moe_v41_attn.h)

_I32, _F32, _F64 = "int32", "float32", "float64"
_dtypes = {}  # by torch's dtype, its name as above (a look-up costs a tenth of making the name)


def _typed(t, dtype, what):
    """_p of lengths, positions or angles, which are refused in another type than the kernels read (an address does not
    say which, and torch's default types are others)"""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if _dtypes.get(t.dtype) is not dtype:
        if str(t.dtype) != "torch." + dtype:
            raise MoeError(MOE_ERR_ARG, f"{what} is {t.dtype}, not {dtype}")
        _dtypes[t.dtype] = dtype
    return t.data_ptr()


def moe_v41_rope_freqs(rot_dim, base=10000.0, kind=MOE_ROPE_SCALE_NONE, factor=1.0, trained=0):
    """(angles per position of each pair, magnitude) on the host; the angles go to the device as f64"""
    out, magnitude = (ctypes.c_double * max(1, rot_dim // 2))(), ctypes.c_float(1.0)
    _check(lib().moe_v41_rope_freqs(rot_dim, base, kind, factor, trained, out, ctypes.byref(magnitude)),
           "moe_v41_rope_freqs")
    return list(out)[:rot_dim // 2], magnitude.value


def make_rope_cfg(head_dim, rot_dim=None, rot_first=0, layout=MOE_ROPE_HALF, x_type=MOE_T_BF16, inverse=False,
                  magnitude=1.0) -> moe_v41_rope_cfg:
    return moe_v41_rope_cfg(head_dim, head_dim if rot_dim is None else rot_dim, rot_first, layout, x_type,
                            int(bool(inverse)), magnitude)


def moe_v41_rope(cfg, m, heads, x, ldx, ldx_head, pos, freqs, out, ldo, ldo_head, stream=None):
    _check(lib().moe_v41_rope(ctypes.byref(cfg), m, heads, _p(x), ldx, ldx_head, _typed(pos, _I32, "moe_v41_rope: pos"),
                              _typed(freqs, _F64, "moe_v41_rope: freqs"), _p(out), ldo, ldo_head, _s(stream)),
           "moe_v41_rope")


def make_kv_cfg(kv_heads, head_dim, page_size, n_pages, type=MOE_T_BF16, page_pitch=None, token_pitch=None,
                head_pitch=None) -> moe_v41_kv_cfg:
    """without pitches: a cache of [n_pages, page_size, kv_heads, head_dim] in memory"""
    token_pitch = kv_heads * head_dim if token_pitch is None else token_pitch
    return moe_v41_kv_cfg(kv_heads, head_dim, page_size, n_pages, type, 0,
                          page_size * token_pitch if page_pitch is None else page_pitch, token_pitch,
                          head_dim if head_pitch is None else head_pitch)


def make_seqs(batch, cu_new, kv_len, table, max_pages, ld_table=None) -> moe_v41_seqs:
    """int32 tensors on the device; holds their addresses, and the tensors themselves as long as it lives"""
    given = {"cu_new": cu_new, "kv_len": kv_len, "table": table}
    at = [_typed(t, _I32, f"make_seqs: {name}") for name, t in given.items()]
    for name, t in given.items():
        if t is not None and not isinstance(t, int) and t.dim() and t.shape[-1] > 1 and t.stride(-1) != 1:
            raise MoeError(MOE_ERR_ARG, f"make_seqs: {name} has gaps")
    s = moe_v41_seqs(batch, max_pages, *at, max_pages if ld_table is None else ld_table)
    s.keep = (cu_new, kv_len, table)
    return s


def moe_v41_kv_append(kv, rope, seqs, m, k, ldk, v, ldv, k_cache, v_cache, q_heads, q, ldq, q_out, ldq_out, freqs,
                      pos, status, stream=None):
    _check(lib().moe_v41_kv_append(ctypes.byref(kv), ctypes.byref(rope), ctypes.byref(seqs), m, _p(k), ldk, _p(v),
                                   ldv, _p(k_cache), _p(v_cache), q_heads, _p(q), ldq, _p(q_out), ldq_out,
                                   _typed(freqs, _F64, "moe_v41_kv_append: freqs"),
                                   _typed(pos, _I32, "moe_v41_kv_append: pos"), _p(status), _s(stream)),
           "moe_v41_kv_append")


def make_attn_cfg(kv, heads, causal=True, window=0, scale=1.0) -> moe_v41_attn_cfg:
    return moe_v41_attn_cfg(kv, heads, int(bool(causal)), window, scale)


def moe_v41_attn_workspace_bytes(cfg: moe_v41_attn_cfg) -> int:
    return int(lib().moe_v41_attn_workspace_bytes(ctypes.byref(cfg)))


def moe_v41_paged_attention(cfg, seqs, m, max_new, q, ldq, k_cache, v_cache, out, ldo, lse, ld_lse, ws, stream=None):
    _check(lib().moe_v41_paged_attention(ctypes.byref(cfg), ctypes.byref(seqs), m, max_new, _p(q), ldq, _p(k_cache),
                                         _p(v_cache), _p(out), ldo,
                                         _typed(lse, _F32, "moe_v41_paged_attention: lse"), ld_lse, _p(ws), _nbytes(ws),
                                         _s(stream)), "moe_v41_paged_attention")
