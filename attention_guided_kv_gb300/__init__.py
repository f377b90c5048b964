"""Python binding of libkvsel.so (attention-guided KV selection on GB300).

Argument marshalling only: every function takes torch CUDA tensors, checks
their dtype/device/contiguity, and hands raw device pointers and the current
stream to the C ABI declared in ``include/kvsel.h``.  Every step of the path
runs in the library's CUDA kernels; there is no CPU or PyTorch fallback.  If
the shared library is missing this module raises instead of degrading.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkvsel.so")

KVSEL_OK = 0
KVSEL_ERR_INVALID_ARG = 1
KVSEL_ERR_UNSUPPORTED = 2
KVSEL_ERR_CUDA = 3
KVSEL_ERR_TIMEOUT = 4
KVSEL_ERR_BAD_INDEX = 5
KVSEL_BF16 = 0
KVSEL_F32 = 1
KVSEL_AGG_MAX, KVSEL_AGG_MEAN, KVSEL_AGG_TOPP, KVSEL_AGG_FRAC_HOT, KVSEL_AGG_ALL_COLD = 0, 1, 2, 3, 4
KVSEL_NORM_NONE, KVSEL_NORM_PERCENTILE = 0, 1
KVSEL_UPDATE_DECAY, KVSEL_UPDATE_MAX, KVSEL_UPDATE_WINDOW = 0, 1, 2
KVSEL_SNAP_GROUP_SUM, KVSEL_SNAP_HEAD_UNION = 0, 1

_STATUS = {0: "OK", 1: "INVALID_ARG", 2: "UNSUPPORTED", 3: "CUDA", 4: "TIMEOUT", 5: "BAD_INDEX"}


class KvselError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"kvsel status {_STATUS.get(code, code)}: {msg}")
        self.code = code


class PagedKV(ctypes.Structure):
    _fields_ = [("k_pool", ctypes.c_void_p), ("v_pool", ctypes.c_void_p),
                ("num_pages", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("num_q_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page_size", ctypes.c_int32)]


class PagedKV4(ctypes.Structure):
    _fields_ = [("k_codes", ctypes.c_void_p), ("v_codes", ctypes.c_void_p), ("k_scales", ctypes.c_void_p),
                ("v_scales", ctypes.c_void_p), ("num_pages", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("num_q_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32)]


class ScoreMod(ctypes.Structure):
    _fields_ = [("softcap", ctypes.c_float), ("slopes", ctypes.c_void_p), ("window", ctypes.c_int32),
                ("n_sink", ctypes.c_int32)]


class BpOptions(ctypes.Structure):
    _fields_ = [("update", ctypes.c_int), ("history", ctypes.c_void_p), ("window", ctypes.c_int),
                ("step", ctypes.c_int64), ("history_tokens", ctypes.c_int64), ("threshold", ctypes.c_float)]


class BlockSignal(ctypes.Structure):
    _fields_ = [("topk_blocks", ctypes.c_int), ("step", ctypes.c_int32), ("block_score", ctypes.c_void_p),
                ("block_step", ctypes.c_void_p), ("topk_out", ctypes.c_void_p), ("mass_out", ctypes.c_void_p)]


class SnapOptions(ctypes.Structure):
    _fields_ = [("mode", ctypes.c_int), ("keep_count", ctypes.c_void_p), ("seed_out", ctypes.c_void_p),
                ("seed_layer_stride", ctypes.c_int64), ("seed_head_stride", ctypes.c_int64)]


_vp, _i, _f, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
_PKV = ctypes.POINTER(PagedKV)
_PKV4 = ctypes.POINTER(PagedKV4)

# name -> (restype, argtypes)
_SIGS = {
    "kvsel_last_error_string": (ctypes.c_char_p, []),
    "kvsel_clear_status": (_i, [_vp, _vp]),
    "kvsel_read_status": (_i, [_vp, _vp]),
    "kvsel_set_wait_limit": (_i, [_vp, ctypes.c_uint, _vp]),
    "kvsel_trace_start": (_i, [ctypes.POINTER(ctypes.c_void_p), _i]),
    "kvsel_trace_stop": (_i, [ctypes.POINTER(ctypes.c_char_p), _i]),
    "kvsel_decode_attn_workspace": (_sz, [_PKV, _i, _i, _i]),
    "kvsel_decode_attn": (_i, [_PKV, _vp, _i, _vp, _i, _vp, _vp, _vp, _vp, _vp, _f, _vp, _i, _vp,
                               _vp, _i, _i, _vp, _sz, _vp, _sz, _vp]),
    "kvsel_decode_attn_noalloc": (_i, [_PKV, _vp, _i, _vp, _i, _vp, _vp, _vp, _vp, _vp, _f, _vp, _i,
                                       _vp, _vp, _i, _i, _vp]),
    "kvsel_h2o_evict_workspace": (_sz, [_PKV, _i, _i]),
    "kvsel_h2o_link_bytes": (_sz, [_i, _i]),
    "kvsel_h2o_link_reset": (_i, [_vp, _i, _i, _vp]),
    "kvsel_h2o_evict": (_i, [_PKV, _vp, _i, _vp, _i, _vp, _vp, _i, _i, _i, _i, _i, _vp, _vp, _vp,
                             _sz, _vp]),
    "kvsel_kv_compact_workspace": (_sz, [_i, _i]),
    "kvsel_kv_compact": (_i, [_PKV, _vp, _i, _vp, _i, _vp, _i, _vp, _vp, _vp, _i, _vp, _vp, _sz, _vp]),
    "kvsel_block_priority_workspace": (_sz, [_i, ctypes.c_int64]),
    "kvsel_block_priority": (_i, [_vp, _vp, _f, _vp, _i, _i, _i, _f, _i, _f, _vp, ctypes.c_int64, _vp,
                                  ctypes.c_int64, _vp, _vp, _sz, _vp]),
    "kvsel_block_priority_ex": (_i, [_vp, _vp, _f, _vp, _i, _i, _i, _f, _i, _f, _vp, ctypes.c_int64, _vp,
                                     ctypes.c_int64, _vp, _vp, _sz, ctypes.POINTER(BpOptions), _vp]),
    "kvsel_sparse_decode_workspace": (_sz, [_PKV, _i, _i, _i, _i]),
    "kvsel_sparse_decode": (_i, [_PKV, _vp, _i, _vp, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i,
                                 _i, _f, _vp, _i, _vp, _vp, _vp, _sz, _vp]),
    "kvsel_snapkv_select_workspace": (_sz, [_PKV, _i, _i, _i, _i]),
    "kvsel_snapkv_select": (_i, [_PKV, _vp, _i, _i, _i, _vp, _i, _f, _i, _i, _vp, _vp, _vp, _sz, _vp]),
    "kvsel_snapkv_select_ex_workspace": (_sz, [_PKV, _i, _i, _i, _i, _i]),
    "kvsel_decode_attn_ex_workspace": (_sz, [_PKV, _i, _i, _i, _i]),
    "kvsel_decode_attn_ex": (_i, [_PKV, _vp, _i, _vp, _i, _vp, _vp, _vp, _vp, _vp, _f, _vp, _i, _vp, _vp, _i, _i,
                                  ctypes.POINTER(BlockSignal), _vp, _sz, _vp, _sz, _vp]),
    "kvsel_quest_page_meta": (_i, [_PKV, _vp, _i, _vp, _i, _vp, _vp, _vp]),
    "kvsel_quest_decode_workspace": (_sz, [_PKV, _i, _i, _i, _i, _i]),
    "kvsel_quest_decode": (_i, [_PKV, _vp, _i, _vp, _i, _vp, _vp, _vp, _vp, _i, _f, _vp, _i, _vp, _vp, _vp, _sz,
                                _vp]),
    "kvsel_kv4_append_workspace": (_sz, [_PKV4, _i]),
    "kvsel_kv4_append": (_i, [_PKV4, _vp, _i, _vp, _i, _vp, _i, _vp, _vp, _vp, _vp, _vp, _i, _vp, _sz, _vp]),
    "kvsel_kv4_read": (_i, [_PKV4, _vp, _i, _vp, _i, _vp, _i, _vp, _vp, _vp, _vp, _sz, _vp]),
    "kvsel_kv4_decode_attn_workspace": (_sz, [_PKV4, _i, _i, _i, _i]),
    "kvsel_kv4_decode_attn": (_i, [_PKV4, _vp, _i, _vp, _i, _vp, _vp, _vp, _vp, _vp, _f, ctypes.POINTER(ScoreMod),
                                   _vp, _i, _vp, _vp, _i, _vp, _sz, _vp]),
    "kvsel_kv4_evict_workspace": (_sz, [_PKV4, _i, _i]),
    "kvsel_kv4_evict": (_i, [_PKV4, _vp, _i, _vp, _i, _vp, _vp, _i, _i, _i, _i, _i, _vp, _vp, _vp, _sz, _vp]),
    "kvsel_prefill_attn_workspace": (_sz, [_PKV, _i, _i]),
    "kvsel_prefill_attn": (_i, [_PKV, _vp, _i, _vp, _i, _vp, _vp, _i, _f, _f, _vp, _i, _vp, _vp, _vp, _i, _vp, _vp,
                                _sz, _vp]),
    "kvsel_snapkv_select_ex": (_i, [_PKV, _vp, _i, _i, _i, _vp, _i, _f, _i, _i, ctypes.POINTER(SnapOptions), _vp,
                                    _vp, _vp, _sz, _vp]),
}

_lib = None


def lib() -> ctypes.CDLL:
    """Load libkvsel.so once (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                               "(nvcc, sm_103a); there is no fallback path")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def exported_symbols():
    return list(_SIGS)


def _check(code: int):
    if code != KVSEL_OK:
        raise KvselError(code, lib().kvsel_last_error_string().decode())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _need(t, dtype, name, allow_none=False):
    if t is None:
        if allow_none:
            return
        raise ValueError(f"{name} is required")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def paged_kv(k_pool: torch.Tensor, v_pool: torch.Tensor, num_q_heads: int) -> PagedKV:
    """Descriptor of bf16 pools shaped [num_pages][num_kv_heads][page_size][head_dim]."""
    _need(k_pool, torch.bfloat16, "k_pool")
    _need(v_pool, torch.bfloat16, "v_pool")
    if k_pool.shape != v_pool.shape or k_pool.dim() != 4:
        raise ValueError("k_pool and v_pool must share one [pages][Hkv][page][d] shape")
    P, H, pg, d = k_pool.shape
    return PagedKV(k_pool.data_ptr(), v_pool.data_ptr(), P, H, num_q_heads, d, pg)


def clear_status(workspace: torch.Tensor, stream=None):
    _check(lib().kvsel_clear_status(_ptr(workspace), _stream(stream)))


def read_status(workspace: torch.Tensor, stream=None) -> int:
    """Synchronise and return (and clear) the device status word of a workspace."""
    return int(lib().kvsel_read_status(_ptr(workspace), _stream(stream)))


def set_wait_limit(workspace: torch.Tensor, spins: int, stream=None):
    """Bound the cross-CTA waits of kernels using this workspace (0 = the default of a few seconds)."""
    _check(lib().kvsel_set_wait_limit(_ptr(workspace), int(spins), _stream(stream)))


class LaunchTrace:
    """Record CUDA events around every library kernel launched by this thread.

    with LaunchTrace(capacity) as tr: ...   then tr.durations() -> [(name, ms)].
    """

    def __init__(self, capacity: int):
        self.capacity = capacity
        self.events = [torch.cuda.Event(enable_timing=True) for _ in range(2 * capacity)]
        for e in self.events:
            e.record()                       # materialise the cudaEvent_t handles
        self._handles = (ctypes.c_void_p * (2 * capacity))(*[e.cuda_event for e in self.events])
        self.names = []

    def __enter__(self):
        _check(lib().kvsel_trace_start(self._handles, self.capacity))
        return self

    def __exit__(self, *exc):
        buf = (ctypes.c_char_p * self.capacity)()
        n = lib().kvsel_trace_stop(buf, self.capacity)
        self.names = [buf[i].decode() for i in range(min(n, self.capacity))]
        return False

    def durations(self):
        torch.cuda.synchronize()
        return [(nm, self.events[2 * i].elapsed_time(self.events[2 * i + 1]))
                for i, nm in enumerate(self.names)]


# ----------------------------------------------------------------------------
# decode attention
# ----------------------------------------------------------------------------
def kvsel_decode_attn_workspace(kv: PagedKV, batch: int, max_len: int, with_probs: bool) -> int:
    return int(lib().kvsel_decode_attn_workspace(ctypes.byref(kv), batch, max_len, int(with_probs)))


def kvsel_decode_attn_ex_workspace(kv: PagedKV, batch: int, max_len: int, with_probs: bool,
                                   with_signal: bool) -> int:
    return int(lib().kvsel_decode_attn_ex_workspace(ctypes.byref(kv), batch, max_len, int(with_probs),
                                                    int(with_signal)))


def kvsel_decode_attn(kv: PagedKV, block_table, seq_lens, q, out, workspace, *, k_new=None,
                      v_new=None, pos_map=None, next_pos=None, scale=None, probs=None,
                      h2o_cum=None, max_len=None, num_ctas=0, h2o_link=None, block_score=None,
                      block_step=None, signal_topk=512, signal_step=0, signal_topk_out=None,
                      signal_mass_out=None, stream=None):
    """Append (optional) + decode attention + probabilities + H2O score update.

    h2o_link: the workspace of the kvsel_h2o_evict calls that follow (same
    batch); the step then hands them its heavy-hitter candidates.
    block_score / block_step (per physical block, fp32 / int32): given, the
    same launch also emits the step's top-k block signal (signal_topk blocks
    per sequence; optional outputs signal_topk_out [batch][signal_topk] and
    signal_mass_out [batch][ceil(max_len / 16)]); the workspace must then be
    sized by kvsel_decode_attn_ex_workspace(..., with_signal=True).
    """
    _need(block_table, torch.int32, "block_table")
    _need(seq_lens, torch.int32, "seq_lens")
    _need(q, torch.bfloat16, "q")
    _need(k_new, torch.bfloat16, "k_new", True)
    _need(v_new, torch.bfloat16, "v_new", True)
    _need(pos_map, torch.int32, "pos_map", True)
    _need(next_pos, torch.int32, "next_pos", True)
    _need(probs, torch.float32, "probs", True)
    _need(h2o_cum, torch.float32, "h2o_cum", True)
    _need(workspace, workspace.dtype, "workspace")
    if out.dtype not in (torch.bfloat16, torch.float32) or not out.is_contiguous():
        raise ValueError("out must be a contiguous bf16 or fp32 CUDA tensor")
    batch = seq_lens.shape[0]
    if max_len is None:
        for t in (probs, h2o_cum, pos_map):
            if t is not None:
                max_len = t.shape[-1]
                break
        else:
            max_len = block_table.shape[1] * kv.page_size
    if scale is None:
        scale = kv.head_dim ** -0.5
    odt = KVSEL_F32 if out.dtype == torch.float32 else KVSEL_BF16
    sig = None
    if block_score is not None or block_step is not None:
        _need(block_score, torch.float32, "block_score")
        _need(block_step, torch.int32, "block_step")
        _need(signal_topk_out, torch.int32, "signal_topk_out", True)
        _need(signal_mass_out, torch.float32, "signal_mass_out", True)
        sig = BlockSignal(int(signal_topk), int(signal_step), block_score.data_ptr(), block_step.data_ptr(),
                          signal_topk_out.data_ptr() if signal_topk_out is not None else None,
                          signal_mass_out.data_ptr() if signal_mass_out is not None else None)
    _check(lib().kvsel_decode_attn_ex(
        ctypes.byref(kv), _ptr(block_table), block_table.shape[1], _ptr(seq_lens), batch, _ptr(q),
        _ptr(k_new), _ptr(v_new), _ptr(pos_map), _ptr(next_pos), float(scale), _ptr(out), odt,
        _ptr(probs), _ptr(h2o_cum), int(max_len), int(num_ctas), ctypes.byref(sig) if sig is not None else None,
        _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(h2o_link),
        0 if h2o_link is None else h2o_link.numel() * h2o_link.element_size(), _stream(stream)))


def kvsel_decode_attn_noalloc(kv: PagedKV, block_table, seq_lens, q, out, *, k_new=None,
                              v_new=None, pos_map=None, next_pos=None, scale=None, probs=None,
                              h2o_cum=None, max_len=None, num_ctas=0, stream=None):
    """kvsel_decode_attn without a workspace, for callers that cannot allocate.

    The library's built-in 8 MiB device array serves as scratch; calls that
    need more are rejected, and calls that overlap on the GPU race.
    """
    for t, dt, nm, opt in ((block_table, torch.int32, "block_table", False),
                           (seq_lens, torch.int32, "seq_lens", False), (q, torch.bfloat16, "q", False),
                           (k_new, torch.bfloat16, "k_new", True), (v_new, torch.bfloat16, "v_new", True),
                           (pos_map, torch.int32, "pos_map", True), (next_pos, torch.int32, "next_pos", True),
                           (probs, torch.float32, "probs", True), (h2o_cum, torch.float32, "h2o_cum", True)):
        _need(t, dt, nm, opt)
    if out.dtype not in (torch.bfloat16, torch.float32) or not out.is_contiguous():
        raise ValueError("out must be a contiguous bf16 or fp32 CUDA tensor")
    if max_len is None:
        for t in (probs, h2o_cum, pos_map):
            if t is not None:
                max_len = t.shape[-1]
                break
        else:
            max_len = block_table.shape[1] * kv.page_size
    if scale is None:
        scale = kv.head_dim ** -0.5
    odt = KVSEL_F32 if out.dtype == torch.float32 else KVSEL_BF16
    _check(lib().kvsel_decode_attn_noalloc(
        ctypes.byref(kv), _ptr(block_table), block_table.shape[1], _ptr(seq_lens), seq_lens.shape[0],
        _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(pos_map), _ptr(next_pos), float(scale), _ptr(out), odt,
        _ptr(probs), _ptr(h2o_cum), int(max_len), int(num_ctas), _stream(stream)))


# ----------------------------------------------------------------------------
# H2O select / evict
# ----------------------------------------------------------------------------
def kvsel_h2o_link_reset(workspace, batch: int, num_kv_heads: int, stream=None):
    """Clear the decode -> select hand-off in an H2O evict workspace (after an outside write to h2o_cum)."""
    _check(lib().kvsel_h2o_link_reset(_ptr(workspace), int(batch), int(num_kv_heads), _stream(stream)))


def kvsel_h2o_evict_workspace(kv: PagedKV, batch: int, budget: int) -> int:
    return int(lib().kvsel_h2o_evict_workspace(ctypes.byref(kv), batch, budget))


def kvsel_h2o_evict(kv: PagedKV, block_table, seq_lens, h2o_cum, workspace, *, budget, n_sink,
                    window, compact=False, pos_map=None, keep_out=None, freed_pages=None,
                    stream=None):
    """H2O heavy hitters + StreamingLLM sinks/window; optional in-place compaction."""
    _need(block_table, torch.int32, "block_table")
    _need(seq_lens, torch.int32, "seq_lens")
    _need(h2o_cum, torch.float32, "h2o_cum")
    _need(pos_map, torch.int32, "pos_map", True)
    _need(keep_out, torch.int32, "keep_out", True)
    _need(freed_pages, torch.int32, "freed_pages", True)
    batch = seq_lens.shape[0]
    _check(lib().kvsel_h2o_evict(
        ctypes.byref(kv), _ptr(block_table), block_table.shape[1], _ptr(seq_lens), batch,
        _ptr(h2o_cum), _ptr(pos_map), h2o_cum.shape[-1], int(budget), int(n_sink), int(window),
        int(bool(compact)), _ptr(keep_out), _ptr(freed_pages), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))


def kvsel_kv_compact_workspace(batch: int, num_kv_heads: int) -> int:
    return int(lib().kvsel_kv_compact_workspace(batch, num_kv_heads))


def kvsel_kv_compact(kv: PagedKV, block_table, seq_lens, keep, workspace, *, keep_count=None, scores=None,
                     pos_map=None, freed_pages=None, stream=None):
    """Move each row's kept slots (keep [batch][Hkv][stride], ascending) to the front, in place."""
    _need(block_table, torch.int32, "block_table")
    _need(seq_lens, torch.int32, "seq_lens")
    _need(keep, torch.int32, "keep")
    _need(keep_count, torch.int32, "keep_count", True)
    _need(scores, torch.float32, "scores", True)
    _need(pos_map, torch.int32, "pos_map", True)
    _need(freed_pages, torch.int32, "freed_pages", True)
    max_len = next((t.shape[-1] for t in (scores, pos_map) if t is not None), 0)
    _check(lib().kvsel_kv_compact(
        ctypes.byref(kv), _ptr(block_table), block_table.shape[-1], _ptr(seq_lens), seq_lens.shape[0],
        _ptr(keep), keep.shape[-1], _ptr(keep_count), _ptr(scores), _ptr(pos_map), int(max_len),
        _ptr(freed_pages), _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))


def workspace(nbytes: int, device="cuda") -> torch.Tensor:
    """A zeroed, 256-byte aligned workspace buffer (status word cleared)."""
    return torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=device)


# ----------------------------------------------------------------------------
# block offload priority
# ----------------------------------------------------------------------------
def kvsel_block_priority_workspace(num_requests: int, max_total_blocks: int) -> int:
    return int(lib().kvsel_block_priority_workspace(num_requests, max_total_blocks))


def kvsel_block_priority(token_scores, req_offsets, order_out, n_out, workspace, *, block_size, agg,
                         norm, evict_frac, increment=None, decay=1.0, top_p=0.1, block_score_out=None,
                         max_total_blocks=None, update=KVSEL_UPDATE_DECAY, history=None, window=1, step=0,
                         threshold=0.0, stream=None):
    """Score update (decay, max over steps or sliding-window sum) + token->block fold + per-request
    percentile + global evict order (kvsel_block_priority_ex)."""
    _need(token_scores, torch.float32, "token_scores")
    _need(increment, torch.float32, "increment", True)
    _need(history, torch.float32, "history", True)
    _need(req_offsets, torch.int64, "req_offsets")
    _need(order_out, torch.int64, "order_out")
    _need(n_out, torch.int64, "n_out")
    _need(block_score_out, torch.float32, "block_score_out", True)
    if max_total_blocks is None:
        max_total_blocks = block_score_out.numel() if block_score_out is not None else token_scores.numel()
    opt = BpOptions(int(update), _ptr(history), int(window), int(step),
                    (history.numel() // max(1, int(window))) if history is not None else 0, float(threshold))
    _check(lib().kvsel_block_priority_ex(
        _ptr(token_scores), _ptr(increment), float(decay), _ptr(req_offsets), req_offsets.numel() - 1,
        int(block_size), int(agg), float(top_p), int(norm), float(evict_frac), _ptr(block_score_out),
        int(max_total_blocks), _ptr(order_out), order_out.numel(), _ptr(n_out), _ptr(workspace),
        workspace.numel() * workspace.element_size(), ctypes.byref(opt), _stream(stream)))


# ----------------------------------------------------------------------------
# DSA-style sparse decode
# ----------------------------------------------------------------------------
def kvsel_sparse_decode_workspace(kv: PagedKV, batch: int, max_len: int, top_k: int,
                                  with_scores_out: bool) -> int:
    return int(lib().kvsel_sparse_decode_workspace(ctypes.byref(kv), batch, max_len, top_k,
                                                   int(with_scores_out)))


def kvsel_sparse_decode(kv: PagedKV, block_table, seq_lens, q, idx_q, idx_w, idx_k, out, workspace, *,
                        top_k=2048, k_new=None, v_new=None, idx_k_new=None, scale=None, topk_out=None,
                        scores_out=None, stream=None):
    """Indexer scores -> top-k positions -> attention over the selected keys."""
    for t, dt, nm, opt in ((block_table, torch.int32, "block_table", False),
                           (seq_lens, torch.int32, "seq_lens", False), (q, torch.bfloat16, "q", False),
                           (idx_q, torch.bfloat16, "idx_q", False), (idx_w, torch.float32, "idx_w", False),
                           (idx_k, torch.bfloat16, "idx_k", False), (k_new, torch.bfloat16, "k_new", True),
                           (v_new, torch.bfloat16, "v_new", True), (idx_k_new, torch.bfloat16, "idx_k_new", True),
                           (topk_out, torch.int32, "topk_out", True), (scores_out, torch.float32, "scores_out", True)):
        _need(t, dt, nm, opt)
    if out.dtype not in (torch.bfloat16, torch.float32) or not out.is_contiguous():
        raise ValueError("out must be a contiguous bf16 or fp32 CUDA tensor")
    B, Hi, Di = idx_q.shape
    max_len = idx_k.shape[1]
    if scale is None:
        scale = kv.head_dim ** -0.5
    odt = KVSEL_F32 if out.dtype == torch.float32 else KVSEL_BF16
    _check(lib().kvsel_sparse_decode(
        ctypes.byref(kv), _ptr(block_table), block_table.shape[1], _ptr(seq_lens), B, _ptr(q), _ptr(k_new),
        _ptr(v_new), _ptr(idx_q), _ptr(idx_w), _ptr(idx_k), _ptr(idx_k_new), Hi, Di, max_len, int(top_k),
        float(scale), _ptr(out), odt, _ptr(topk_out), _ptr(scores_out), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))


# ----------------------------------------------------------------------------
# SnapKV prefill selection
# ----------------------------------------------------------------------------
def kvsel_snapkv_select_workspace(kv: PagedKV, num_layers: int, seq_len: int, obs_window: int,
                                  with_vote_out: bool) -> int:
    return int(lib().kvsel_snapkv_select_workspace(ctypes.byref(kv), num_layers, seq_len, obs_window,
                                                   int(with_vote_out)))


def kvsel_snapkv_select(kv: PagedKV, block_table, q_obs, keep_out, workspace, *, seq_len, keep_k,
                        pool_kernel=7, scale=None, vote_out=None, stream=None):
    """Observation-window votes, max-pool and top-k keep per layer and kv head."""
    _need(block_table, torch.int32, "block_table")
    _need(q_obs, torch.bfloat16, "q_obs")
    _need(keep_out, torch.int32, "keep_out")
    _need(vote_out, torch.float32, "vote_out", True)
    L, Hq, W, d = q_obs.shape
    if scale is None:
        scale = kv.head_dim ** -0.5
    _check(lib().kvsel_snapkv_select(
        ctypes.byref(kv), _ptr(block_table), block_table.shape[-1], L, int(seq_len), _ptr(q_obs), W,
        float(scale), int(pool_kernel), int(keep_k), _ptr(keep_out), _ptr(vote_out), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))


def kvsel_snapkv_select_ex_workspace(kv: PagedKV, num_layers: int, seq_len: int, obs_window: int,
                                     with_vote_out: bool, mode: int = KVSEL_SNAP_GROUP_SUM) -> int:
    return int(lib().kvsel_snapkv_select_ex_workspace(ctypes.byref(kv), num_layers, seq_len, obs_window,
                                                      int(with_vote_out), int(mode)))


def kvsel_snapkv_select_ex(kv: PagedKV, block_table, q_obs, keep_out, workspace, *, seq_len, keep_k,
                           mode=KVSEL_SNAP_GROUP_SUM, pool_kernel=7, scale=None, vote_out=None,
                           keep_count=None, seed_out=None, seed_layer_stride=0, seed_head_stride=0,
                           stream=None):
    """SnapKV selection with the union keep mode, keep counts and cold-start seeds.

    seed_out is a float32 tensor (or a view into one) addressed with the given
    element strides: entry i of (layer l, kv head h) at l * seed_layer_stride +
    h * seed_head_stride + i from its first element.
    """
    _need(block_table, torch.int32, "block_table")
    _need(q_obs, torch.bfloat16, "q_obs")
    _need(keep_out, torch.int32, "keep_out")
    _need(vote_out, torch.float32, "vote_out", True)
    _need(keep_count, torch.int32, "keep_count", True)
    if seed_out is not None and (seed_out.dtype != torch.float32 or seed_out.device.type != "cuda"):
        raise ValueError("seed_out must be a CUDA float32 tensor")
    L, Hq, W, d = q_obs.shape
    if scale is None:
        scale = kv.head_dim ** -0.5
    opt = SnapOptions(int(mode), keep_count.data_ptr() if keep_count is not None else None,
                      seed_out.data_ptr() if seed_out is not None else None,
                      int(seed_layer_stride), int(seed_head_stride))
    _check(lib().kvsel_snapkv_select_ex(
        ctypes.byref(kv), _ptr(block_table), block_table.shape[-1], L, int(seq_len), _ptr(q_obs), W,
        float(scale), int(pool_kernel), int(keep_k), ctypes.byref(opt), _ptr(keep_out), _ptr(vote_out),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))


def kvsel_quest_page_meta(kv: PagedKV, block_table, seq_lens, page_meta, workspace, stream=None):
    """Per-page key min / max for every page of each sequence (status in the workspace's first word)."""
    _need(block_table, torch.int32, "block_table")
    _need(seq_lens, torch.int32, "seq_lens")
    _need(page_meta, torch.bfloat16, "page_meta")
    _check(lib().kvsel_quest_page_meta(ctypes.byref(kv), _ptr(block_table), block_table.shape[-1],
                                       _ptr(seq_lens), seq_lens.shape[0], _ptr(page_meta), _ptr(workspace),
                                       _stream(stream)))


def kvsel_quest_decode_workspace(kv: PagedKV, batch: int, max_pages: int, budget_pages: int,
                                 with_bounds_out: bool = False, with_pages_out: bool = False) -> int:
    return int(lib().kvsel_quest_decode_workspace(ctypes.byref(kv), batch, max_pages, budget_pages,
                                                  int(with_bounds_out), int(with_pages_out)))


def kvsel_quest_decode(kv: PagedKV, block_table, seq_lens, q, page_meta, out, workspace, *, budget_pages,
                       k_new=None, v_new=None, scale=None, pages_out=None, bounds_out=None, stream=None):
    """One decode step with Quest page selection per q head."""
    _need(block_table, torch.int32, "block_table")
    _need(seq_lens, torch.int32, "seq_lens")
    _need(q, torch.bfloat16, "q")
    _need(page_meta, torch.bfloat16, "page_meta")
    _need(k_new, torch.bfloat16, "k_new", True)
    _need(v_new, torch.bfloat16, "v_new", True)
    _need(pages_out, torch.int32, "pages_out", True)
    _need(bounds_out, torch.float32, "bounds_out", True)
    if out.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("out must be bfloat16 or float32")
    if scale is None:
        scale = kv.head_dim ** -0.5
    _check(lib().kvsel_quest_decode(
        ctypes.byref(kv), _ptr(block_table), block_table.shape[-1], _ptr(seq_lens), seq_lens.shape[0], _ptr(q),
        _ptr(k_new), _ptr(v_new), _ptr(page_meta), int(budget_pages), float(scale), _ptr(out),
        KVSEL_F32 if out.dtype == torch.float32 else KVSEL_BF16, _ptr(pages_out), _ptr(bounds_out),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))


# ----------------------------------------------------------------------------
# the paged 4-bit cache
# ----------------------------------------------------------------------------
def _shaped(t, shape, name):
    if t is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _same_device(ref, **tensors):
    for name, t in tensors.items():
        if t is not None and t.device != ref.device:
            raise ValueError(f"{name} must be on {ref.device}")


def paged_kv4(k_codes: torch.Tensor, v_codes: torch.Tensor, k_scales: torch.Tensor, v_scales: torch.Tensor,
              num_q_heads: int) -> PagedKV4:
    """Descriptor of a 4-bit cache: codes uint8 [num_pages][num_kv_heads][page_size][64], scales bf16
    [num_pages][num_kv_heads][page_size][4][2] ({scale, minimum} of each group of 32 values)."""
    for t, name in ((k_codes, "k_codes"), (v_codes, "v_codes")):
        _need(t, torch.uint8, name)
    for t, name in ((k_scales, "k_scales"), (v_scales, "v_scales")):
        _need(t, torch.bfloat16, name)
    if k_codes.dim() != 4:
        raise ValueError("k_codes must be [pages][Hkv][page][head_dim / 2]")
    P, H, pg, half = k_codes.shape
    _shaped(v_codes, k_codes.shape, "v_codes")
    _shaped(k_scales, (P, H, pg, half // 16, 2), "k_scales")
    _shaped(v_scales, (P, H, pg, half // 16, 2), "v_scales")
    _same_device(k_codes, v_codes=v_codes, k_scales=k_scales, v_scales=v_scales)
    return PagedKV4(k_codes.data_ptr(), v_codes.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(), P, H, num_q_heads,
                    2 * half, pg)


def _table_of(block_table, seq_lens):
    _need(block_table, torch.int32, "block_table")
    _need(seq_lens, torch.int32, "seq_lens")
    if block_table.dim() != 2 or seq_lens.dim() != 1 or block_table.shape[0] != seq_lens.shape[0]:
        raise ValueError("block_table must be [batch][max_pages] and seq_lens [batch]")
    return seq_lens.shape[0]


def _nbytes(t):
    return t.numel() * t.element_size()


def _per_slot(kv, batch, max_len, **tensors):
    """The common row length of the given [batch][num_kv_heads][max_len] tensors (0 without any)."""
    for name, t in tensors.items():
        if t is not None:
            max_len = t.shape[-1] if max_len is None else max_len
            _shaped(t, (batch, kv.num_kv_heads, max_len), name)
    return max_len


def kvsel_kv4_append_workspace(kv: PagedKV4, batch: int) -> int:
    return int(lib().kvsel_kv4_append_workspace(ctypes.byref(kv), int(batch)))


def kvsel_kv4_append(kv: PagedKV4, block_table, seq_lens, tok_off, k, v, workspace, *, pos_map=None, next_pos=None,
                     h2o_cum=None, stream=None):
    """Quantise packed new tokens (k, v bf16 [total][Hkv][128]; sequence b's are rows tok_off[b]..tok_off[b + 1])
    into the cache behind each sequence's live ones; seq_lens (and next_pos) grow."""
    batch = _table_of(block_table, seq_lens)
    _need(tok_off, torch.int32, "tok_off")
    _shaped(tok_off, (batch + 1,), "tok_off")
    _need(k, torch.bfloat16, "k")
    _need(v, torch.bfloat16, "v")
    _shaped(k, (k.shape[0], kv.num_kv_heads, kv.head_dim), "k")
    _shaped(v, k.shape, "v")
    _need(pos_map, torch.int32, "pos_map", True)
    _need(next_pos, torch.int32, "next_pos", True)
    _shaped(next_pos, (batch,), "next_pos")
    _need(h2o_cum, torch.float32, "h2o_cum", True)
    _need(workspace, workspace.dtype, "workspace")
    max_len = _per_slot(kv, batch, None, pos_map=pos_map, h2o_cum=h2o_cum) or 0
    _same_device(block_table, seq_lens=seq_lens, tok_off=tok_off, k=k, v=v, pos_map=pos_map, next_pos=next_pos,
                 h2o_cum=h2o_cum, workspace=workspace)
    with torch.cuda.device(block_table.device):
        _check(lib().kvsel_kv4_append(
            ctypes.byref(kv), _ptr(block_table), block_table.shape[1], _ptr(seq_lens), batch, _ptr(tok_off), k.shape[0],
            _ptr(k), _ptr(v), _ptr(pos_map), _ptr(next_pos), _ptr(h2o_cum), max_len, _ptr(workspace), _nbytes(workspace),
            _stream(stream)))


def kvsel_kv4_read(kv: PagedKV4, block_table, seq_lens, tok_off, k_out, v_out, workspace, *, start=None, stream=None):
    """Read cached tokens back as bf16: packed row tok_off[b] + i is slot start[b] + i (or i) of sequence b."""
    batch = _table_of(block_table, seq_lens)
    _need(tok_off, torch.int32, "tok_off")
    _shaped(tok_off, (batch + 1,), "tok_off")
    _need(start, torch.int32, "start", True)
    _shaped(start, (batch,), "start")
    _need(k_out, torch.bfloat16, "k_out")
    _need(v_out, torch.bfloat16, "v_out")
    _shaped(k_out, (k_out.shape[0], kv.num_kv_heads, kv.head_dim), "k_out")
    _shaped(v_out, k_out.shape, "v_out")
    _need(workspace, workspace.dtype, "workspace")
    _same_device(block_table, seq_lens=seq_lens, tok_off=tok_off, start=start, k_out=k_out, v_out=v_out,
                 workspace=workspace)
    with torch.cuda.device(block_table.device):
        _check(lib().kvsel_kv4_read(
            ctypes.byref(kv), _ptr(block_table), block_table.shape[1], _ptr(seq_lens), batch, _ptr(tok_off),
            k_out.shape[0], _ptr(start), _ptr(k_out), _ptr(v_out), _ptr(workspace), _nbytes(workspace), _stream(stream)))


def kvsel_kv4_decode_attn_workspace(kv: PagedKV4, batch: int, max_len: int, with_probs: bool, with_cum: bool) -> int:
    return int(lib().kvsel_kv4_decode_attn_workspace(ctypes.byref(kv), int(batch), int(max_len), int(bool(with_probs)),
                                                     int(bool(with_cum))))


def kvsel_kv4_decode_attn(kv: PagedKV4, block_table, seq_lens, q, out, workspace, *, k_new=None, v_new=None,
                          pos_map=None, next_pos=None, scale=None, softcap=0.0, slopes=None, window=0, n_sink=0,
                          probs=None, h2o_cum=None, max_len=None, stream=None):
    """Append (optional) + decode attention over the 4-bit cache + probabilities + H2O score update.

    softcap: scores become softcap * tanh(score / softcap).  slopes (fp32 [num_q_heads]): slopes[h] times the
    distance is taken off the score.  window: only the last `window` positions and the first `n_sink` are seen.
    Positions are pos_map's where it is given, else the slots.
    """
    batch = _table_of(block_table, seq_lens)
    _need(q, torch.bfloat16, "q")
    _shaped(q, (batch, kv.num_q_heads, kv.head_dim), "q")
    for t, name in ((k_new, "k_new"), (v_new, "v_new")):
        _need(t, torch.bfloat16, name, True)
        _shaped(t, (batch, kv.num_kv_heads, kv.head_dim), name)
    _need(pos_map, torch.int32, "pos_map", True)
    _need(next_pos, torch.int32, "next_pos", True)
    _shaped(next_pos, (batch,), "next_pos")
    _need(slopes, torch.float32, "slopes", True)
    _shaped(slopes, (kv.num_q_heads,), "slopes")
    _need(probs, torch.float32, "probs", True)
    _need(h2o_cum, torch.float32, "h2o_cum", True)
    _need(workspace, workspace.dtype, "workspace")
    if out.dtype not in (torch.bfloat16, torch.float32) or not out.is_contiguous() or out.device.type != "cuda":
        raise ValueError("out must be a contiguous bf16 or fp32 CUDA tensor")
    _shaped(out, q.shape, "out")
    if max_len is None and probs is not None:
        max_len = probs.shape[-1]
    max_len = _per_slot(kv, batch, max_len, pos_map=pos_map, h2o_cum=h2o_cum)
    if max_len is None:
        max_len = block_table.shape[1] * kv.page_size
    _shaped(probs, (batch, kv.num_q_heads, max_len), "probs")
    _same_device(block_table, seq_lens=seq_lens, q=q, out=out, k_new=k_new, v_new=v_new, pos_map=pos_map,
                 next_pos=next_pos, slopes=slopes, probs=probs, h2o_cum=h2o_cum, workspace=workspace)
    mod = None
    if softcap != 0 or slopes is not None or window != 0 or n_sink != 0:
        mod = ScoreMod(float(softcap), slopes.data_ptr() if slopes is not None else None, int(window), int(n_sink))
    with torch.cuda.device(block_table.device):
        _check(lib().kvsel_kv4_decode_attn(
            ctypes.byref(kv), _ptr(block_table), block_table.shape[1], _ptr(seq_lens), batch, _ptr(q), _ptr(k_new),
            _ptr(v_new), _ptr(pos_map), _ptr(next_pos), float(kv.head_dim ** -0.5 if scale is None else scale),
            ctypes.byref(mod) if mod is not None else None, _ptr(out),
            KVSEL_F32 if out.dtype == torch.float32 else KVSEL_BF16, _ptr(probs), _ptr(h2o_cum), int(max_len),
            _ptr(workspace), _nbytes(workspace), _stream(stream)))


def kvsel_kv4_evict_workspace(kv: PagedKV4, batch: int, budget: int) -> int:
    return int(lib().kvsel_kv4_evict_workspace(ctypes.byref(kv), int(batch), int(budget)))


def kvsel_kv4_evict(kv: PagedKV4, block_table, seq_lens, h2o_cum, workspace, *, budget, n_sink, window, compact=False,
                    pos_map=None, keep_out=None, freed_pages=None, stream=None):
    """kvsel_h2o_evict for the 4-bit cache: select by accumulated weight; optional in-place compaction."""
    batch = _table_of(block_table, seq_lens)
    _need(h2o_cum, torch.float32, "h2o_cum")
    _need(pos_map, torch.int32, "pos_map", True)
    _need(keep_out, torch.int32, "keep_out", True)
    _shaped(keep_out, (batch, kv.num_kv_heads, int(budget)), "keep_out")
    _need(freed_pages, torch.int32, "freed_pages", True)
    _shaped(freed_pages, block_table.shape, "freed_pages")
    _need(workspace, workspace.dtype, "workspace")
    max_len = _per_slot(kv, batch, None, h2o_cum=h2o_cum, pos_map=pos_map)
    _same_device(block_table, seq_lens=seq_lens, h2o_cum=h2o_cum, pos_map=pos_map, keep_out=keep_out,
                 freed_pages=freed_pages, workspace=workspace)
    with torch.cuda.device(block_table.device):
        _check(lib().kvsel_kv4_evict(
            ctypes.byref(kv), _ptr(block_table), block_table.shape[1], _ptr(seq_lens), batch, _ptr(h2o_cum), _ptr(pos_map),
            max_len, int(budget), int(n_sink), int(window), int(bool(compact)), _ptr(keep_out), _ptr(freed_pages),
            _ptr(workspace), _nbytes(workspace), _stream(stream)))


# ----------------------------------------------------------------------------
# attention of prompt tokens
# ----------------------------------------------------------------------------
def kvsel_prefill_attn_workspace(kv: PagedKV, batch: int, total_q: int) -> int:
    return int(lib().kvsel_prefill_attn_workspace(ctypes.byref(kv), int(batch), int(total_q)))


def kvsel_prefill_attn(kv: PagedKV, block_table, seq_lens, q, q_off, out, workspace, *, scale=None, softcap=0.0,
                       slopes=None, window=0, prefix=None, doc_start=None, lse=None, stream=None):
    """Attention of packed prompt tokens (q bf16 [total][Hq][128]; sequence b's are rows q_off[b]..q_off[b + 1], the
    last of its seq_lens[b] cached tokens) over the paged bf16 cache.

    Causal; softcap: scores become softcap * tanh(score / softcap).  slopes (fp32 [Hq]): slopes[h] times the distance
    is taken off the score.  window: only the last `window` positions are seen, and the prefix.  prefix (int32
    [batch]): positions that every query of the sequence sees.  doc_start (int32 [total]): the first position each
    query may see.  lse (fp32 [total][Hq]): log-sum-exp of each row's scores, -inf for a row that sees nothing.
    """
    batch = _table_of(block_table, seq_lens)
    _need(q, torch.bfloat16, "q")
    _shaped(q, (q.shape[0], kv.num_q_heads, kv.head_dim), "q")
    total = q.shape[0]
    _need(q_off, torch.int32, "q_off")
    _shaped(q_off, (batch + 1,), "q_off")
    if out.dtype not in (torch.bfloat16, torch.float32) or not out.is_contiguous() or out.device.type != "cuda":
        raise ValueError("out must be a contiguous bf16 or fp32 CUDA tensor")
    _shaped(out, q.shape, "out")
    _need(slopes, torch.float32, "slopes", True)
    _shaped(slopes, (kv.num_q_heads,), "slopes")
    _need(prefix, torch.int32, "prefix", True)
    _shaped(prefix, (batch,), "prefix")
    _need(doc_start, torch.int32, "doc_start", True)
    _shaped(doc_start, (total,), "doc_start")
    _need(lse, torch.float32, "lse", True)
    _shaped(lse, q.shape[:2], "lse")
    _need(workspace, workspace.dtype, "workspace")
    _same_device(block_table, seq_lens=seq_lens, q=q, q_off=q_off, out=out, slopes=slopes, prefix=prefix,
                 doc_start=doc_start, lse=lse, workspace=workspace)
    with torch.cuda.device(block_table.device):
        _check(lib().kvsel_prefill_attn(
            ctypes.byref(kv), _ptr(block_table), block_table.shape[1], _ptr(seq_lens), batch, _ptr(q), _ptr(q_off), total,
            float(kv.head_dim ** -0.5 if scale is None else scale), float(softcap), _ptr(slopes), int(window),
            _ptr(prefix), _ptr(doc_start), _ptr(out), KVSEL_F32 if out.dtype == torch.float32 else KVSEL_BF16, _ptr(lse),
            _ptr(workspace), _nbytes(workspace), _stream(stream)))
