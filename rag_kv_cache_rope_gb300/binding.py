"""Thin Python binding of libblend's C ABI (include/blend.h).

Functions carry the C names and only marshal arguments: torch tensors become device
pointers, Python lists become host arrays, and a non-zero status raises BlendError.
Every step of the method runs in the library's CUDA kernels.  If libblend.so is
missing, lib() raises: there is no fallback implementation.
"""
from __future__ import annotations

import ctypes as C
import os
import struct
from typing import Optional, Sequence

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libblend.so")

OK, EINVAL, ENOMEM, ECUDA, EMISS, ETIMEOUT, EDEVICE, EUNSUPPORTED = 0, -1, -2, -3, -4, -5, -6, -7
F32, BF16 = 0, 1
SEL_EXT, SEL_HKVD, SEL_FORCED, SEL_FULL, SEL_EPIC = 0, 1, 2, 3, 4
BUDGET_FINAL, BUDGET_CANDIDATE = 0, 1
DEV_KV, DEV_V = 0, 1
GROUP_WINDOW, GROUP_SPAN = 0, 1
POOL_DEVICE, POOL_HOST = 0, 1
MAX_BATCH = 64
MAX_SPAN = 64
MAX_ALIGN_TARGETS = 131072
GU_BLOCK = 16
PAGES_MODEL, PAGES_INT4 = 0, 1
MAX_SEQS = 1024
MAX_TOP = 32
W4_STORE, W4_ADD, W4_SWIGLU = 0, 1, 2
ROPE_HALF, ROPE_PAIRS = 0, 1
ROPE_NONE, ROPE_LINEAR, ROPE_BASE, ROPE_BANDS, ROPE_YARN = 0, 1, 2, 3, 4

MODES = {"ext": SEL_EXT, "hkvd": SEL_HKVD, "forced": SEL_FORCED, "full": SEL_FULL, "epic": SEL_EPIC}
BUDGETS = {"final": BUDGET_FINAL, "candidate": BUDGET_CANDIDATE}
DEVMODES = {"kv": DEV_KV, "v": DEV_V}
GROUP_RULES = {"window": GROUP_WINDOW, "span": GROUP_SPAN}
W4_EPIS = {"store": W4_STORE, "add": W4_ADD, "swiglu": W4_SWIGLU}
ROPE_LAYOUTS = {"half": ROPE_HALF, "pairs": ROPE_PAIRS}
ROPE_SCALINGS = {"none": ROPE_NONE, "linear": ROPE_LINEAR, "base": ROPE_BASE, "bands": ROPE_BANDS, "yarn": ROPE_YARN}


class BlendError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"libblend error {code}: {msg}")
        self.code = code


# ---------------------------------------------------------------- C structs
class ModelCfg(C.Structure):
    _fields_ = [("n_layers", C.c_int32), ("hidden", C.c_int32), ("n_q_heads", C.c_int32),
                ("n_kv_heads", C.c_int32), ("head_dim", C.c_int32), ("ffn", C.c_int32),
                ("vocab", C.c_int32), ("dtype", C.c_int32), ("rope_theta", C.c_double),
                ("rms_eps", C.c_float), ("max_pos", C.c_int32)]


class Weights(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("embed", "attn_norm", "w_qkv", "w_o", "mlp_norm", "w_gu",
                                          "w_down", "final_norm")]


class Limits(C.Structure):
    _fields_ = [("max_rows", C.c_int32), ("max_tokens", C.c_int32), ("max_chunk_rows", C.c_int32),
                ("max_batch", C.c_int32)]


class Pool(C.Structure):
    _fields_ = [("n_entries", C.c_int32), ("prefix_len", C.c_int32),
                ("entry_len", C.POINTER(C.c_int32)), ("entry_row", C.POINTER(C.c_int64)),
                ("present", C.POINTER(C.c_uint8)), ("n_rows", C.c_int64), ("k", C.c_void_p),
                ("v", C.c_void_p), ("tokens", C.c_void_p), ("location", C.c_int32)]


class Request(C.Structure):
    _fields_ = [("n_chunks", C.c_int32), ("chunk_ids", C.POINTER(C.c_int32)),
                ("query_len", C.c_int32), ("query_tokens", C.c_void_p), ("mode", C.c_int32),
                ("rho_bp", C.c_int32), ("r1_bp", C.c_int32), ("window", C.c_int32),
                ("tau", C.c_int32), ("budget_mode", C.c_int32), ("dev_mode", C.c_int32),
                ("scores", C.c_void_p), ("n_stages", C.c_int32), ("stage_layer", C.c_int32 * 3),
                ("stage_pos", C.c_void_p * 3), ("stage_n", C.c_int32 * 3), ("group_rule", C.c_int32),
                ("tau_smooth", C.c_float), ("tau_cover_bp", C.c_int32), ("max_span", C.c_int32),
                ("cap_bp", C.c_int32), ("epic_m", C.c_int32), ("focus_layer", C.c_int32),
                ("focus_bp", C.c_int32)]


class Outputs(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("k", "v", "hidden", "sel", "n_sel", "c1", "n_c1", "dev1",
                                          "dev2", "q_last")]


class Pages(C.Structure):
    _fields_ = [("format", C.c_int32), ("page_tokens", C.c_int32), ("n_pages", C.c_int32), ("n_seq", C.c_int32),
                ("max_pages", C.c_int32), ("table", C.c_void_p), ("k", C.c_void_p), ("v", C.c_void_p),
                ("k_scale", C.c_void_p), ("v_scale", C.c_void_p)]


class W4(C.Structure):
    _fields_ = [("n", C.c_int32), ("k", C.c_int32), ("group", C.c_int32), ("codes", C.c_void_p), ("scale", C.c_void_p)]


class Rope(C.Structure):
    _fields_ = [("layout", C.c_int32), ("rot_dim", C.c_int32), ("scaling", C.c_int32), ("trained_len", C.c_int32),
                ("theta", C.c_double), ("factor", C.c_double), ("low", C.c_double), ("high", C.c_double),
                ("magnitude", C.c_float)]


class RopeRows(C.Structure):
    _fields_ = [("src", C.c_void_p), ("dst", C.c_void_p), ("src_row", C.c_int64), ("src_layer", C.c_int64),
                ("dst_row", C.c_int64), ("dst_layer", C.c_int64), ("heads", C.c_int32), ("n_layers", C.c_int32)]


_lib = None


def lib() -> C.CDLL:
    """Loads libblend.so (built by build.build()); raises if it is not there."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "rag_kv_cache_rope_gb300.build.build() (needs nvcc)")
        L = C.CDLL(LIB_PATH)
        vp, i32, i64 = C.c_void_p, C.c_int32, C.c_int64
        sig = {
            "blend_workspace_size": (C.c_size_t, [C.POINTER(ModelCfg), C.POINTER(Limits)]),
            "blend_init": (C.c_int, [C.POINTER(ModelCfg), C.POINTER(Weights), C.POINTER(Limits), vp,
                                     C.c_size_t, vp, C.POINTER(vp)]),
            "blend_destroy": (C.c_int, [vp]),
            "blend_last_error": (C.c_char_p, [vp]),
            "blend_device_status": (C.c_int, [vp, vp]),
            "blend_set_tensor_cores": (C.c_int, [vp, C.c_int]),
            "rope_realign": (C.c_int, [vp, vp, vp, i32, vp, i32, i64, i64, vp]),
            "blend_assemble": (C.c_int, [vp, i32, C.POINTER(Request), C.POINTER(Pool),
                                         C.POINTER(Outputs), vp]),
            "kv_deviation": (C.c_int, [vp, vp, vp, vp, vp, vp, vp, i32, i64, i32, vp, vp]),
            "topk_select_dilate": (C.c_int, [vp, vp, i32, i32, i32, i32, i32, i32, vp, vp, vp, vp]),
            "gather_rows": (C.c_int, [vp, vp, i64, i64, vp, vp, i32, vp, vp]),
            "scatter_kv": (C.c_int, [vp, vp, vp, vp, vp, i32, i64, vp, vp, vp]),
            "selective_layer": (C.c_int, [vp, i32, vp, vp, vp, i32, vp, vp, i32, vp, i32, vp]),
            "blend_prefill": (C.c_int, [vp, i32, C.POINTER(Request), C.POINTER(Pool),
                                        C.POINTER(Outputs), vp]),
            "importance_scores": (C.c_int, [vp, i32, i32, i32, i32, vp, vp]),
            "blend_profile": (C.c_int, [vp, C.c_int]),
            "blend_profile_stages": (C.c_int, [vp, C.c_uint32]),
            "blend_wait_flag": (C.c_int, [vp, vp, i64, vp]),
            "blend_profile_read": (C.c_int, [vp, C.POINTER(C.c_double), C.POINTER(C.c_int64), i32]),
            "blend_profile_name": (C.c_char_p, [i32]),
            "blend_launch_count": (C.c_int64, []),
            "topk_select_dilate_noalloc": (C.c_int, [vp, i32, i32, i32, i32, i32, i32, vp, vp, vp, vp]),
            "span_select": (C.c_int, [vp, vp, i32, i32, i32, i32, C.c_float, i32, i32, i32, vp, vp, vp]),
            "aux_attention_scores": (C.c_int, [vp, i32, C.POINTER(Request), C.POINTER(Pool),
                                               C.POINTER(Outputs), vp, vp]),
            "blend_ratio_controller": (C.c_int, [C.c_double, C.c_double, C.c_double, i32, C.POINTER(i32)]),
            "blend_pick_storage": (C.c_int, [C.c_double, C.c_double, i32, i32, C.POINTER(C.c_double),
                                             C.POINTER(C.c_double), C.POINTER(i32)]),
            "align_expand": (C.c_int, [vp, vp, vp, i32, i32, vp, vp, i32, i32, i32, vp, vp, vp]),
            "paged_append": (C.c_int, [vp, C.POINTER(Pages), vp, i64, vp, i64, vp, i64, vp, vp, vp, vp, vp, i32, vp]),
            "paged_gather": (C.c_int, [vp, C.POINTER(Pages), vp, vp, vp, vp, i32, vp, vp, vp]),
            "paged_attention": (C.c_int, [vp, C.POINTER(Pages), vp, i64, vp, vp, i32, i32, i32, i32, vp, vp]),
            "w4_pack": (C.c_int, [vp, C.POINTER(W4), vp, i64, vp]),
            "w4_unpack": (C.c_int, [vp, C.POINTER(W4), vp, i64, vp]),
            "w4_linear": (C.c_int, [vp, C.POINTER(W4), vp, i64, i32, vp, i64, i32, i32, vp]),
            "token_logprobs": (C.c_int, [vp, vp, i64, i32, i32, i32, C.c_float, vp, i32, vp, vp, i32, vp, vp, vp]),
            "rope_rows": (C.c_int, [vp, C.POINTER(Rope), vp, i32, vp, vp, i32, vp]),
        }
        for name, (res, args) in sig.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


EXPORTED = ("blend_workspace_size", "blend_init", "blend_destroy", "blend_last_error",
            "blend_device_status", "blend_set_tensor_cores", "rope_realign", "blend_assemble",
            "kv_deviation", "topk_select_dilate", "gather_rows", "scatter_kv", "selective_layer",
            "blend_prefill", "importance_scores", "blend_profile", "blend_profile_stages", "blend_wait_flag", "blend_profile_read",
            "blend_profile_name", "blend_launch_count", "topk_select_dilate_noalloc", "span_select",
            "align_expand", "aux_attention_scores", "blend_ratio_controller", "blend_pick_storage",
            "paged_append", "paged_gather", "paged_attention", "w4_pack", "w4_unpack", "w4_linear",
            "token_logprobs", "rope_rows")


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    return C.c_void_p(t.data_ptr())


def _stream(stream=None):
    if stream is None:
        stream = torch.cuda.current_stream()
    return C.c_void_p(stream.cuda_stream)


def _check(rc: int, h=None):
    if rc != OK:
        msg = lib().blend_last_error(h.ptr if h is not None else None)
        raise BlendError(rc, msg.decode() if msg else "")
    return rc


# ---------------------------------------------------------------- handle
class Handle:
    """A libblend handle plus the tensors it points into (kept alive here)."""

    def __init__(self, ptr, cfg: ModelCfg, lim: Limits, keep, index: int = 0):
        self.ptr = ptr
        self.cfg = cfg
        self.lim = lim
        self._keep = keep
        self.index = index  # the GPU that holds its workspace and error word

    def __del__(self):
        if getattr(self, "ptr", None) and _lib is not None:
            _lib.blend_destroy(self.ptr)
            self.ptr = None


def model_cfg(shape, max_pos: int) -> ModelCfg:
    return ModelCfg(shape.n_layers, shape.hidden, shape.n_q_heads, shape.n_kv_heads, shape.head_dim,
                    shape.ffn, shape.vocab, F32 if shape.dtype == "f32" else BF16,
                    float(shape.rope_theta), float(shape.rms_eps), int(max_pos))


def blend_workspace_size(cfg: ModelCfg, lim: Limits) -> int:
    return int(lib().blend_workspace_size(C.byref(cfg), C.byref(lim)))


def blend_init(cfg: ModelCfg, packed: dict, lim: Limits, workspace: Optional[torch.Tensor] = None,
               stream=None) -> Handle:
    need = blend_workspace_size(cfg, lim)
    if need == 0:
        raise BlendError(EINVAL, "bad model configuration or limits")
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=packed["embed"].device)
    w = Weights(*[packed[k].data_ptr() for k in ("embed", "attn_norm", "w_qkv", "w_o", "mlp_norm",
                                                  "w_gu", "w_down", "final_norm")])
    out = C.c_void_p()
    rc = lib().blend_init(C.byref(cfg), C.byref(w), C.byref(lim), _ptr(workspace), workspace.numel(),
                          _stream(stream), C.byref(out))
    _check(rc)
    return Handle(out, cfg, lim, (packed, workspace), workspace.get_device())


def blend_destroy(h: Handle):
    if h.ptr:
        _check(lib().blend_destroy(h.ptr))
        h.ptr = None


def blend_device_status(h: Handle, stream=None) -> int:
    return _check(lib().blend_device_status(h.ptr, _stream(stream)), h)


def blend_wait_flag(h: Handle, flag: torch.Tensor, max_polls: int, stream=None):
    """Bounded device-side wait until flag (device int32 scalar) is nonzero; on expiry the
    handle's error word records BLEND_ETIMEOUT (raised by blend_device_status)."""
    _check(lib().blend_wait_flag(h.ptr, _ptr(flag), int(max_polls), _stream(stream)), h)


def blend_set_tensor_cores(h: Handle, on: bool) -> int:
    return int(lib().blend_set_tensor_cores(h.ptr, 1 if on else 0))


def blend_profile(h: Handle, enable: bool):
    _check(lib().blend_profile(h.ptr, 1 if enable else 0), h)


def blend_profile_stages(h: Handle, stages: Sequence[str]):
    """Record only the named stages (an empty list stops recording)."""
    names = [lib().blend_profile_name(i).decode() for i in range(32)]
    mask = 0
    for st in stages:
        if st not in names:
            raise ValueError(f"unknown profiler stage {st!r}")
        mask |= 1 << names.index(st)
    _check(lib().blend_profile_stages(h.ptr, mask), h)


def blend_profile_read(h: Handle) -> dict:
    """{stage: (total ms, kernel launches)} since blend_profile(h, True)."""
    n = 32
    ms = (C.c_double * n)()
    cnt = (C.c_int64 * n)()
    k = lib().blend_profile_read(h.ptr, ms, cnt, n)
    if k < 0:
        _check(k, h)
    return {lib().blend_profile_name(i).decode(): (ms[i], int(cnt[i])) for i in range(k)}


def blend_launch_count() -> int:
    return int(lib().blend_launch_count())


def rope_realign(h, k_src, k_dst, n_rows, delta, n_layers, src_layer_rows, dst_layer_rows, stream=None):
    _check(lib().rope_realign(h.ptr, _ptr(k_src), _ptr(k_dst), n_rows, _ptr(delta), n_layers,
                              src_layer_rows, dst_layer_rows, _stream(stream)), h)


def kv_deviation(h, k_new, v_new, k_cache, v_cache, pos, n_rows, max_rows, mode, dev_out, stream=None):
    """n_rows: device int32 count; the cache row count is taken from k_cache's first dimension."""
    _check(lib().kv_deviation(h.ptr, _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache), _ptr(pos),
                              _ptr(n_rows), max_rows, k_cache.shape[0], mode, _ptr(dev_out), _stream(stream)), h)


def span_select(h, scores, n, base, budget, cap, tau_smooth, tau_cover_bp, max_span, budget_mode, idx_out,
                n_out, stream=None):
    _check(lib().span_select(h.ptr, _ptr(scores), n, base, budget, cap, float(tau_smooth), tau_cover_bp, max_span,
                             budget_mode, _ptr(idx_out), _ptr(n_out), _stream(stream)), h)


def align_expand(h, sel, n_sel, max_sel, sel_base, a_start, a_end, n_spec, n_target, out_base, idx_out, n_out,
                 stream=None):
    _check(lib().align_expand(h.ptr, _ptr(sel), _ptr(n_sel), max_sel, sel_base, _ptr(a_start), _ptr(a_end), n_spec,
                              n_target, out_base, _ptr(idx_out), _ptr(n_out), _stream(stream)), h)


def topk_select_dilate(h, scores, n, base, budget, window, tau, budget_mode, allowed, idx_out, n_out,
                       stream=None):
    _check(lib().topk_select_dilate(h.ptr, _ptr(scores), n, base, budget, window, tau, budget_mode,
                                    _ptr(allowed), _ptr(idx_out), _ptr(n_out), _stream(stream)), h)


def topk_select_dilate_noalloc(scores, n, base, budget, window, tau, budget_mode, allowed, idx_out, n_out,
                               stream=None):
    """topk_select_dilate without a handle or any allocation (fixed 32768-entry device
    scratch shared by every call; see include/blend.h)."""
    _check(lib().topk_select_dilate_noalloc(_ptr(scores), n, base, budget, window, tau, budget_mode,
                                            _ptr(allowed), _ptr(idx_out), _ptr(n_out), _stream(stream)))


def gather_rows(h, src, row_bytes, idx, n, max_n, dst, stream=None):
    """src's first dimension is its row count (src_rows of the C call)."""
    _check(lib().gather_rows(h.ptr, _ptr(src), row_bytes, src.shape[0], _ptr(idx), _ptr(n), max_n, _ptr(dst),
                             _stream(stream)), h)


def scatter_kv(h, k_new, v_new, pos, n, max_n, k_cache, v_cache, stream=None):
    """The cache row count (n_ctx of the C call) is k_cache's first dimension."""
    _check(lib().scatter_kv(h.ptr, _ptr(k_new), _ptr(v_new), _ptr(pos), _ptr(n), max_n, k_cache.shape[0],
                            _ptr(k_cache), _ptr(v_cache), _stream(stream)), h)


def selective_layer(h, layer, x, pos, n, k_cache, v_cache, n_ctx, dev_out=None, dev_mode=DEV_KV,
                    stream=None, max_n=None):
    """n: a device int32 count (then max_n bounds it) or a host int (copied into a device
    scalar, max_n = n)."""
    if isinstance(n, torch.Tensor):
        n_dev = n
        if max_n is None:
            raise ValueError("max_n is required with a device count")
    else:
        n_dev = torch.tensor([int(n)], dtype=torch.int32, device=x.device)
        max_n = int(n) if max_n is None else max_n
    _check(lib().selective_layer(h.ptr, layer, _ptr(x), _ptr(pos), _ptr(n_dev), max_n, _ptr(k_cache),
                                 _ptr(v_cache), n_ctx, _ptr(dev_out), dev_mode, _stream(stream)), h)


def importance_scores(hidden, n, n_layers, dim, out, stream=None):
    dt = BF16 if hidden.dtype == torch.bfloat16 else F32
    _check(lib().importance_scores(_ptr(hidden), n, n_layers, dim, dt, _ptr(out), _stream(stream)))


# ---------------------------------------------------------------- pool / requests / outputs
class PoolRef:
    """Host-side description of a chunk-KV pool (see blend_pool): tensors on the GPU, or
    pinned CPU tensors (location "host") that the GPU reads in place."""

    def __init__(self, k, v, tokens, prefix_len, entry_len, entry_row, present=None, location: str = "device"):
        self.k, self.v, self.tokens = k, v, tokens
        self._len = (C.c_int32 * len(entry_len))(*entry_len)
        self._row = (C.c_int64 * len(entry_row))(*entry_row)
        self._present = None if present is None else (C.c_uint8 * len(present))(*present)
        self.c = Pool(len(entry_len), prefix_len, self._len, self._row, self._present, k.shape[1],
                      k.data_ptr(), v.data_ptr(), tokens.data_ptr(),
                      {"device": POOL_DEVICE, "host": POOL_HOST}[location])
        self.entry_len = list(entry_len)
        self.prefix_len = prefix_len


class RequestRef:
    def __init__(self, chunk_ids: Sequence[int], query_tokens: torch.Tensor, mode: str = "ext",
                 rho_bp: int = 0, r1_bp: int = 0, window: int = 1, tau: int = 1,
                 budget_mode: str = "final", dev_mode: str = "kv", scores: Optional[torch.Tensor] = None,
                 stages: Optional[list] = None, group_rule: str = "window", tau_smooth: float = 0.4,
                 tau_cover_bp: int = 7000, max_span: int = 16, cap_bp: int = 0, epic_m: int = 0,
                 focus_layer: int = 0, focus_bp: int = 0):
        self.chunk_ids = list(chunk_ids)
        self._ids = (C.c_int32 * len(self.chunk_ids))(*self.chunk_ids)
        self.query = query_tokens
        self.scores = scores
        self.stages = stages or []
        st_layer = (C.c_int32 * 3)(*([int(f) for f, _ in self.stages] + [0] * (3 - len(self.stages))))
        st_pos = (C.c_void_p * 3)(*([p.data_ptr() if p.numel() else None for _, p in self.stages]
                                     + [None] * (3 - len(self.stages))))
        st_n = (C.c_int32 * 3)(*([int(p.numel()) for _, p in self.stages] + [0] * (3 - len(self.stages))))
        self.c = Request(len(self.chunk_ids), self._ids, int(query_tokens.numel()), query_tokens.data_ptr(),
                         MODES[mode], rho_bp, r1_bp, window, tau, BUDGETS[budget_mode], DEVMODES[dev_mode],
                         scores.data_ptr() if scores is not None else None, len(self.stages), st_layer,
                         st_pos, st_n, GROUP_RULES[group_rule], float(tau_smooth), tau_cover_bp, max_span, cap_bp,
                         epic_m, focus_layer, focus_bp)


class OutputsRef:
    def __init__(self, k, v, hidden, sel=None, n_sel=None, c1=None, n_c1=None, dev1=None, dev2=None,
                 q_last=None):
        self.t = dict(k=k, v=v, hidden=hidden, sel=sel, n_sel=n_sel, c1=c1, n_c1=n_c1, dev1=dev1, dev2=dev2,
                      q_last=q_last)
        self.c = Outputs(*[None if self.t[n] is None else self.t[n].data_ptr()
                           for n in ("k", "v", "hidden", "sel", "n_sel", "c1", "n_c1", "dev1", "dev2",
                                     "q_last")])

    def __getitem__(self, k):
        return self.t[k]


def _req_array(reqs):
    arr = (Request * len(reqs))()
    for i, r in enumerate(reqs):
        arr[i] = r.c
    return arr


def blend_assemble(h, reqs: Sequence[RequestRef], pool: PoolRef, out: OutputsRef, stream=None):
    _check(lib().blend_assemble(h.ptr, len(reqs), _req_array(reqs), C.byref(pool.c), C.byref(out.c),
                                _stream(stream)), h)


def blend_prefill(h, reqs: Sequence[RequestRef], pool: PoolRef, out: OutputsRef, stream=None):
    _check(lib().blend_prefill(h.ptr, len(reqs), _req_array(reqs), C.byref(pool.c), C.byref(out.c),
                               _stream(stream)), h)


def aux_attention_scores(h, reqs: Sequence[RequestRef], pool: PoolRef, out: OutputsRef, scores: torch.Tensor,
                         stream=None):
    _check(lib().aux_attention_scores(h.ptr, len(reqs), _req_array(reqs), C.byref(pool.c), C.byref(out.c),
                                      _ptr(scores), _stream(stream)), h)


def blend_ratio_controller(full_prefill_s: float, kv_bytes: float, load_bytes_per_s: float,
                           floor_bp: int = 1500) -> int:
    out = C.c_int32()
    _check(lib().blend_ratio_controller(full_prefill_s, kv_bytes, load_bytes_per_s, floor_bp, C.byref(out)))
    return out.value


def blend_pick_storage(full_prefill_s: float, kv_bytes: float, floor_bp: int, bytes_per_s, cost_per_byte) -> int:
    n = len(bytes_per_s)
    bw = (C.c_double * max(n, 1))(*bytes_per_s)
    cost = (C.c_double * max(n, 1))(*cost_per_byte)
    out = C.c_int32()
    _check(lib().blend_pick_storage(full_prefill_s, kv_bytes, floor_bp, n, bw, cost, C.byref(out)))
    return out.value


# ---------------------------------------------------------------- paged cache
class PagesRef:
    """Host-side description of one layer's paged cache (see blend_pages): k, v contiguous
    [n_pages][hkv][page_tokens][d] of the model's dtype, or uint8 [..][d / 2] with bf16 scales
    [..][d / 32] for 4-bit pages; table int32 [n_seq][max_pages].  All on one GPU."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, table: torch.Tensor, k_scale: Optional[torch.Tensor] = None,
                 v_scale: Optional[torch.Tensor] = None):
        int4 = k.dtype == torch.uint8
        if k.dim() != 4 or v.shape != k.shape or v.dtype != k.dtype:
            raise ValueError("k and v must be alike: [n_pages][kv heads][page tokens][head dim]")
        if table.dim() != 2 or table.dtype != torch.int32:
            raise ValueError("table must be int32 [n_seq][max_pages]")
        if int4:
            want = (*k.shape[:3], k.shape[3] * 2 // 32)
            for s in (k_scale, v_scale):
                if s is None or s.dtype != torch.bfloat16 or tuple(s.shape) != want:
                    raise ValueError(f"4-bit pages need bf16 scales of shape {want}")
        elif k_scale is not None or v_scale is not None:
            raise ValueError("scales go with 4-bit pages (uint8 k and v)")
        self.t = tuple(x for x in (k, v, table, k_scale, v_scale) if x is not None)
        if any(not x.is_contiguous() or x.device != k.device for x in self.t):
            raise ValueError("the tensors of a paged cache must be contiguous and on one device")
        self.device, self.dtype, self.n_kv_heads, self.n_seq = k.device, k.dtype, k.shape[1], table.shape[0]
        self.index = k.get_device()  # -1: not on a GPU
        self._fit = (None, None, 0)  # the model these pages were last found to fit, its element type and query heads
        self.head_dim = k.shape[3] * (2 if int4 else 1)
        self.c = Pages(PAGES_INT4 if int4 else PAGES_MODEL, k.shape[2], k.shape[0], table.shape[0], table.shape[1],
                       *[None if x is None else x.data_ptr() for x in (table, k, v, k_scale, v_scale)])
        self.ref = C.byref(self.c)


# A decode step makes these calls once per layer with kernels of a few microseconds: the checks below
# read each property once, and what holds for a pair of handle and pages is remembered in the pages.
def _paged_stream(h: Handle, pages: PagesRef, stream):
    """The call's stream, the model's element type and query heads, after a look at the pages: they must
    be the handle's model's and on the stream's GPU."""
    fit = pages._fit
    if fit[0] is not h.cfg:
        model = torch.bfloat16 if h.cfg.dtype == BF16 else torch.float32
        if pages.dtype != (torch.uint8 if pages.c.format == PAGES_INT4 else model) or pages.n_kv_heads != h.cfg.n_kv_heads or pages.head_dim != h.cfg.head_dim:
            raise ValueError("the pages are not of the handle's model")
        if pages.index < 0:
            raise ValueError("the pages are not on a GPU")
        pages._fit = fit = (h.cfg, model, h.cfg.n_q_heads)
    dev = pages.index
    if torch.cuda.current_device() != dev or (stream is not None and stream.device_index != dev):
        raise ValueError(f"the pages are on {pages.device}: make it the current device and use a stream of it")
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream, fit[1], fit[2]


def _paged_rows(pages: PagesRef, dtype, t: torch.Tensor, heads: int, what: str) -> int:
    """Distance between the rows of t [rows][heads][head dim] in elements."""
    d = pages.head_dim
    st, sh = t.stride(), t.shape
    if len(sh) == 3:
        ok = sh[1] == heads and sh[2] == d and st[2] == 1 and (st[1] == d or heads == 1)
    else:
        ok = len(sh) == 2 and sh[1] == heads * d and st[1] == 1
    if not ok:
        raise ValueError(f"{what} must be [rows][{heads}][{d}] with adjacent heads")
    if t.dtype is not dtype or t.get_device() != pages.index:
        raise ValueError(f"{what} must be of the model's dtype and on {pages.device}")
    return st[0] if sh[0] > 1 else heads * d


def _paged_index(pages: PagesRef, n: int, what: str, t: torch.Tensor):
    if t.dtype is not torch.int32 or t.numel() < n or not t.is_contiguous() or t.get_device() != pages.index:
        raise ValueError(f"{what} must be contiguous int32 of at least {n} entries on {pages.device}")
    return t.data_ptr()


def paged_append(h: Handle, pages: PagesRef, k_new, v_new, seq, pos, n, max_n, q=None, q_out=None, rot=None,
                 stream=None):
    """k_new, v_new (and q): [rows][heads][head dim], rows at any stride of 16 bytes; seq, pos, rot
    int32 per row; n a device int32 count of at most max_n rows."""
    s, dt, hq = _paged_stream(h, pages, stream)
    hkv = pages.n_kv_heads
    ld_k, ld_v = _paged_rows(pages, dt, k_new, hkv, "k_new"), _paged_rows(pages, dt, v_new, hkv, "v_new")
    seq, pos = _paged_index(pages, max_n, "seq", seq), _paged_index(pages, max_n, "pos", pos)
    if rot is not None:
        rot = _paged_index(pages, max_n, "rot", rot)
    n = _paged_index(pages, 1, "n", n)
    if k_new.shape[0] < max_n or v_new.shape[0] < max_n:
        raise ValueError("fewer rows than max_n")
    ld_q = pq = po = None
    if q is not None and q_out is not None:
        ld_q = _paged_rows(pages, dt, q, hq, "q")
        if _paged_rows(pages, dt, q_out, hq, "q_out") != hq * pages.head_dim or min(q.shape[0], q_out.shape[0]) < max_n:
            raise ValueError("q_out must hold max_n adjacent rows, and q as many")
        pq, po = q.data_ptr(), q_out.data_ptr()
    elif q is not None or q_out is not None:
        raise ValueError("q and q_out go together")
    if max_n == 0:
        return
    rc = lib().paged_append(h.ptr, pages.ref, k_new.data_ptr(), ld_k, v_new.data_ptr(), ld_v, pq, ld_q or 0, po, seq,
                            pos, rot, n, max_n, s)
    if rc:
        _check(rc, h)


def paged_gather(h: Handle, pages: PagesRef, seq, pos, n, max_n, k_out, v_out, rot=None, stream=None):
    """k_out, v_out: [rows][kv heads][head dim], rows adjacent, of the model's dtype."""
    s, dt, _ = _paged_stream(h, pages, stream)
    hkv = pages.n_kv_heads
    for t in (k_out, v_out):
        if _paged_rows(pages, dt, t, hkv, "k_out and v_out") != hkv * pages.head_dim or t.shape[0] < max_n:
            raise ValueError("k_out and v_out must hold max_n adjacent rows")
    seq, pos = _paged_index(pages, max_n, "seq", seq), _paged_index(pages, max_n, "pos", pos)
    if rot is not None:
        rot = _paged_index(pages, max_n, "rot", rot)
    n = _paged_index(pages, 1, "n", n)
    if max_n == 0:
        return
    rc = lib().paged_gather(h.ptr, pages.ref, seq, pos, rot, n, max_n, k_out.data_ptr(), v_out.data_ptr(), s)
    if rc:
        _check(rc, h)


def paged_attention(h: Handle, pages: PagesRef, q, q_start, kv_len, max_q, out, window=0, n_sink=0, stream=None):
    """q: [rows][hq][head dim] (rows at any stride of 16 bytes); out: [rows][hq * head dim], rows
    adjacent; q_start int32 [n_seq + 1], kv_len int32 [n_seq] on the device; max_q: most query rows of
    one sequence."""
    s, dt, hq = _paged_stream(h, pages, stream)
    n_seq, rows = pages.n_seq, q.shape[0]
    ld_q = _paged_rows(pages, dt, q, hq, "q")
    if _paged_rows(pages, dt, out, hq, "out") != hq * pages.head_dim or out.shape[0] < rows:
        raise ValueError("out must hold as many adjacent rows as q")
    kv_len = _paged_index(pages, n_seq, "kv_len", kv_len)
    q_start = _paged_index(pages, n_seq + 1, "q_start", q_start)
    if max(window, n_sink, max_q) >= 1 << 31:  # (the call takes 32 bits, and more would wrap)
        raise ValueError("window, n_sink and max_q must be below 2^31")
    if rows == 0:
        return
    rc = lib().paged_attention(h.ptr, pages.ref, q.data_ptr(), ld_q, q_start, kv_len, rows, max_q, window, n_sink,
                               out.data_ptr(), s)
    if rc:
        _check(rc, h)


# ---------------------------------------------------------------- behind the cache: tokens
# (Called once or more per layer and token, as the paged calls: each property is read once.)
def _token_stream(h: Handle, index: int, stream):
    """The call's stream: the tensors' GPU must be the handle's, the current one, and the stream's."""
    if index < 0:
        raise ValueError("the tensors are not on a GPU")
    if h.index != index:
        raise ValueError(f"the tensors are on cuda:{index}, the handle on cuda:{h.index}")
    if torch.cuda.current_device() != index or (stream is not None and stream.device_index != index):
        raise ValueError(f"the tensors are on cuda:{index}: make it the current device and use a stream of it")
    return torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream


def _matrix(t: torch.Tensor, what: str, dtype, index: int, rows: Optional[int], cols: int) -> int:
    """Distance between the rows of t [rows][cols] in elements (neighbouring columns adjacent)."""
    sh, st = t.shape, t.stride()
    if len(sh) != 2 or sh[1] != cols or (rows is not None and sh[0] != rows) or (st[1] != 1 and cols > 1):
        raise ValueError(f"{what} must be [{'rows' if rows is None else rows}][{cols}] with adjacent columns")
    if t.dtype is not dtype or t.get_device() != index:
        raise ValueError(f"{what} must be {dtype} on cuda:{index}")
    return st[0] if sh[0] > 1 else cols


def _model_dtype(h: Handle):
    return torch.bfloat16 if h.cfg.dtype == BF16 else torch.float32


class W4Ref:
    """Host-side description of 4-bit weights [n][k] (see blend_w4): codes uint8 [n][chunks * 64], scale
    bf16 [n][chunks * 128 / group], chunks = ceil(k / 128), contiguous and on one GPU."""

    def __init__(self, codes: torch.Tensor, scale: torch.Tensor, k: int, group: int = 128):
        if group not in (32, 64, 128):
            raise ValueError("group must be 32, 64 or 128")
        chunks = (k + 127) // 128
        n = codes.shape[0]
        if codes.dtype != torch.uint8 or tuple(codes.shape) != (n, chunks * 64):
            raise ValueError(f"codes must be uint8 [n][{chunks * 64}]")
        if scale.dtype != torch.bfloat16 or tuple(scale.shape) != (n, chunks * (128 // group)):
            raise ValueError(f"scale must be bf16 [{n}][{chunks * (128 // group)}]")
        if not codes.is_contiguous() or not scale.is_contiguous() or codes.device != scale.device:
            raise ValueError("codes and scale must be contiguous and on one device")
        self.codes, self.scale, self.n, self.k, self.group = codes, scale, n, k, group
        self.index = codes.get_device()
        self.c = W4(n, k, group, codes.data_ptr(), scale.data_ptr())
        self.ref = C.byref(self.c)

    @classmethod
    def empty(cls, n: int, k: int, group: int = 128, device="cuda") -> "W4Ref":
        chunks = (k + 127) // 128
        return cls(torch.empty(n, chunks * 64, dtype=torch.uint8, device=device),
                   torch.empty(n, chunks * (128 // group), dtype=torch.bfloat16, device=device), k, group)


def w4_layout(codes: torch.Tensor) -> torch.Tensor:
    """Codes 0..15 [n][k] (integers; weight = (code - 8) * scale) in the packed rows of blend_w4."""
    n, k = codes.shape
    u = torch.nn.functional.pad(codes.to(torch.uint8), (0, -k % 128), value=8)
    u = u.reshape(n, -1, 4, 4, 4, 2).permute(0, 1, 3, 2, 5, 4).reshape(n, -1, 2)  # chunk, part, step, half, pair
    return (u[..., 0] | (u[..., 1] << 4)).contiguous()


def w4_pack(h: Handle, w: torch.Tensor, w4: W4Ref, stream=None):
    """w: [n][k] of the model's dtype (rows at any stride of 16 bytes)."""
    s = _token_stream(h, w4.index, stream)
    ld = _matrix(w, "w", _model_dtype(h), w4.index, w4.n, w4.k)
    rc = lib().w4_pack(h.ptr, w4.ref, w.data_ptr(), ld, s)
    if rc:
        _check(rc, h)


def w4_unpack(h: Handle, w4: W4Ref, out: torch.Tensor, stream=None):
    """out: [n][k] of the model's dtype (rows at any stride of 16 bytes)."""
    s = _token_stream(h, w4.index, stream)
    ld = _matrix(out, "out", _model_dtype(h), w4.index, w4.n, w4.k)
    rc = lib().w4_unpack(h.ptr, w4.ref, out.data_ptr(), ld, s)
    if rc:
        _check(rc, h)


def w4_linear(h: Handle, w4: W4Ref, x: torch.Tensor, y: torch.Tensor, epi: str = "store", stream=None):
    """x: [rows][k] of the model's dtype (rows at any stride of 16 bytes); y: [rows][n] ([n / 2] for
    "swiglu"), fp32 or bf16 (fp32 for "add"), rows at any stride."""
    s = _token_stream(h, w4.index, stream)
    code = W4_EPIS.get(epi)
    if code is None:
        raise ValueError(f"epi must be one of {', '.join(W4_EPIS)}")
    dt = y.dtype
    if dt is not torch.float32 and dt is not torch.bfloat16:
        raise ValueError("y must be fp32 or bf16")
    rows = x.shape[0]
    ld_x = _matrix(x, "x", _model_dtype(h), w4.index, None, w4.k)
    ld_y = _matrix(y, "y", dt, w4.index, rows, w4.n // 2 if code == W4_SWIGLU else w4.n)
    if rows == 0:
        return
    rc = lib().w4_linear(h.ptr, w4.ref, x.data_ptr(), ld_x, rows, y.data_ptr(), ld_y, F32 if dt is torch.float32 else BF16,
                         code, s)
    if rc:
        _check(rc, h)


def token_logprobs(h: Handle, logits: torch.Tensor, ids=None, logp=None, entropy=None, top_id=None, top_logp=None,
                   scale: float = 1.0, stream=None):
    """logits: [rows][vocab], fp32 or bf16, rows at any stride; ids int32 and logp fp32 [rows][n_ids]; entropy
    fp32 [rows]; top_id int32 and top_logp fp32 [rows][top].  What is None is left out."""
    dt, index = logits.dtype, logits.get_device()
    s = _token_stream(h, index, stream)
    if dt is not torch.float32 and dt is not torch.bfloat16:
        raise ValueError("logits must be fp32 or bf16")
    if logits.dim() != 2:
        raise ValueError("logits must be [rows][vocab]")
    rows, vocab = logits.shape
    ld = _matrix(logits, "logits", dt, index, rows, vocab)
    if (ids is None) != (logp is None):
        raise ValueError("ids and logp go together")

    def flat(t, what, dtype, width):
        if t.dtype is not dtype or t.get_device() != index or not t.is_contiguous() or tuple(t.shape) != width:
            raise ValueError(f"{what} must be contiguous {dtype} of shape {width} on cuda:{index}")
        return t.data_ptr()

    n_ids = top = 0
    p_ids = p_logp = p_ent = p_top = p_top_logp = None
    if ids is not None:
        n_ids = ids.shape[1] if ids.dim() == 2 else -1
        p_ids, p_logp = flat(ids, "ids", torch.int32, (rows, n_ids)), flat(logp, "logp", torch.float32, (rows, n_ids))
    if entropy is not None:
        p_ent = flat(entropy, "entropy", torch.float32, (rows,))
    if top_id is not None:
        top = top_id.shape[1] if top_id.dim() == 2 else -1
        p_top = flat(top_id, "top_id", torch.int32, (rows, top))
    if top_logp is not None:
        if top_id is None:
            raise ValueError("top_logp goes with top_id")
        p_top_logp = flat(top_logp, "top_logp", torch.float32, (rows, top))
    if rows == 0:
        return
    rc = lib().token_logprobs(h.ptr, logits.data_ptr(), ld, F32 if dt is torch.float32 else BF16, rows, vocab, scale, p_ids,
                              n_ids, p_logp, p_ent, top, p_top, p_top_logp, s)
    if rc:
        _check(rc, h)


def rope_desc(theta: float, rot_dim: int, layout: str = "half", scaling: str = "none", factor: float = 1.0,
              low: float = 0.0, high: float = 0.0, trained_len: int = 0, magnitude: float = 1.0) -> Rope:
    """Rotary layout and frequencies of a model (see blend_rope)."""
    if layout not in ROPE_LAYOUTS or scaling not in ROPE_SCALINGS:
        raise ValueError(f"layout must be one of {', '.join(ROPE_LAYOUTS)}, scaling one of {', '.join(ROPE_SCALINGS)}")
    return Rope(ROPE_LAYOUTS[layout], rot_dim, ROPE_SCALINGS[scaling], trained_len, theta, factor, low, high, magnitude)


_ROPE_ROWS = struct.Struct("@QQqqqqii")  # a blend_rope_rows


def _rope_part(src: torch.Tensor, dst: torch.Tensor, dtype, index: int, heads: int, d: int, max_n: int, what: str) -> bytes:
    """src, dst: [rows][heads][head dim] or [layers][rows][heads][head dim]."""
    (s_row, s_layer, layers), (d_row, d_layer, d_layers) = (_rope_strides(t, dtype, index, heads, d, max_n, what) for t in (src, dst))
    if layers != d_layers:
        raise ValueError(f"{what} and its output must have the same layers")
    return _ROPE_ROWS.pack(src.data_ptr(), dst.data_ptr(), s_row, s_layer, d_row, d_layer, heads, layers)


def _rope_strides(t: torch.Tensor, dtype, index: int, heads: int, d: int, max_n: int, what: str):
    sh, sr = t.shape, t.stride()
    if len(sh) == 3:
        (rows, n, dim), (row, head, one), layers, layer = sh, sr, 1, 0
    elif len(sh) == 4:
        (layers, rows, n, dim), (layer, row, head, one) = sh, sr
    else:
        n = -1
    if n != heads or dim != d or one != 1 or (heads > 1 and head != d):
        raise ValueError(f"{what} must be [rows][{heads}][{d}] or [layers][rows][{heads}][{d}] with adjacent heads")
    if t.dtype is not dtype or t.get_device() != index:
        raise ValueError(f"{what} must be of the model's dtype and on cuda:{index}")
    if rows < max_n:
        raise ValueError("fewer rows than max_n")
    return (row if rows > 1 else heads * d), layer, layers


def rope_rows(h: Handle, rope: Rope, k, k_out, rot, n, max_n, q=None, q_out=None, stream=None):
    """k, k_out: [rows][kv heads][head dim], or [layers][rows][..], of the model's dtype (rows at any stride
    of 16 bytes); q, q_out the same with the model's query heads; rot int32 per row; n a device int32 count of
    at most max_n rows.  An output may be its own input."""
    index = k.get_device()
    s = _token_stream(h, index, stream)
    cfg, dt = h.cfg, _model_dtype(h)
    d = cfg.head_dim
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out go together")
    for t, what, least in ((rot, "rot", max_n), (n, "n", 1)):
        if t.dtype is not torch.int32 or t.numel() < least or not t.is_contiguous() or t.get_device() != index:
            raise ValueError(f"{what} must be contiguous int32 of at least {least} entries on cuda:{index}")
    parts = _rope_part(k, k_out, dt, index, cfg.n_kv_heads, d, max_n, "k")
    if q is not None:
        parts += _rope_part(q, q_out, dt, index, cfg.n_q_heads, d, max_n, "q")
    if max_n == 0 or 0 in k.shape or (q is not None and 0 in q.shape):
        return
    rc = lib().rope_rows(h.ptr, C.byref(rope), parts, 1 if q is None else 2, rot.data_ptr(), n.data_ptr(), max_n, s)
    if rc:
        _check(rc, h)


# ---------------------------------------------------------------- weight layout
def pack_weights(w: dict, device=None) -> dict:
    """Plain per-layer weights (synth.model_weights layout) -> the layout blend_weights
    documents: fused [q; k; v] rows, gate/up rows interleaved in blocks of GU_BLOCK."""
    dev = device or w["embed"].device
    wq, wk, wv = w["wq"], w["wk"], w["wv"]
    L, F, H = w["wg"].shape
    gu = torch.stack([w["wg"].reshape(L, F // GU_BLOCK, GU_BLOCK, H),
                      w["wu"].reshape(L, F // GU_BLOCK, GU_BLOCK, H)], dim=2).reshape(L, 2 * F, H)
    return {
        "embed": w["embed"].to(dev).contiguous(),
        "attn_norm": w["attn_norm"].to(dev).contiguous(),
        "w_qkv": torch.cat([wq, wk, wv], dim=1).to(dev).contiguous(),
        "w_o": w["wo"].to(dev).contiguous(),
        "mlp_norm": w["mlp_norm"].to(dev).contiguous(),
        "w_gu": gu.to(dev).contiguous(),
        "w_down": w["wd"].to(dev).contiguous(),
        "final_norm": w["final_norm"].to(dev).contiguous(),
    }
