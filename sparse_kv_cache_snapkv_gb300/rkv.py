"""Thin ctypes binding of librkv.so (include/rkv.h), one Python function per C entry point.

Argument marshalling only: shapes are read from the tensors, pointers and the current CUDA
stream are passed through, and any non-OK status raises RkvError. Every step of the hot path
runs in the library's kernels; there is no fallback of any kind. If the library is missing the
import fails with an explanation.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

from . import _build

_lib = None

RKV_OK = 0
_STATUS = {0: "RKV_OK", 1: "RKV_ERR_INVALID_ARG", 2: "RKV_ERR_UNSUPPORTED",
           3: "RKV_ERR_WORKSPACE", 4: "RKV_ERR_CUDA", 5: "RKV_ERR_DEVICE_STATUS",
           6: "RKV_ERR_TOO_LARGE"}
STATUS_BYTES = 256
HEAD_DIM = 128

SYMBOLS = [
    "rkv_status_string", "rkv_check_status", "rkv_plan", "rkv_snapkv_workspace_bytes",
    "rkv_snapkv_compress", "rkv_summaries_workspace_bytes", "rkv_build_page_summaries",
    "rkv_hybrid_decode_workspace_bytes", "rkv_hybrid_decode",
    "rkv_dense_decode_workspace_bytes", "rkv_dense_decode", "rkv_dense_decode_noalloc",
    "rkv_build_page_summaries_mt", "rkv_hybrid_decode_mt", "rkv_plan_even_split",
    "rkv_snapkv_per_head_workspace_bytes", "rkv_snapkv_compress_per_head",
    "rkv_snapkv_compress_paged", "rkv_build_page_summaries_paged", "rkv_hybrid_decode_paged",
    "rkv_snapkv_compress_summarized", "rkv_snapkv_compress_avg_pool", "rkv_snapkv_select",
    "rkv_snapkv_scores", "rkv_testing_scores_wait_timeout", "rkv_testing_decode_layout",
    "rkv_kv4_append_workspace_bytes", "rkv_kv4_append", "rkv_kv4_append_paged",
    "rkv_kv4_decode_workspace_bytes", "rkv_kv4_decode", "rkv_kv4_decode_paged",
    "rkv_dense_decode_weights_workspace_bytes", "rkv_dense_decode_weights",
    "rkv_prompt_weights_workspace_bytes", "rkv_prompt_weights", "rkv_evict_workspace_bytes",
    "rkv_evict", "rkv_evict_kv4", "rkv_testing_prompt_wait_timeout",
    "rkv_reserve_slots_workspace_bytes", "rkv_reserve_slots", "rkv_release_blocks_workspace_bytes",
    "rkv_release_blocks", "rkv_rope_frequencies", "rkv_rope_append_workspace_bytes",
    "rkv_rope_append", "rkv_prompt_attention_workspace_bytes", "rkv_prompt_attention",
    "rkv_prompt_attention_paged", "rkv_tree_attention", "rkv_tree_attention_paged",
    "rkv_testing_attention_wait_timeout",
]


class RkvError(RuntimeError):
    def __init__(self, fn: str, code: int, bits: int = 0):
        self.code = code
        self.bits = bits
        extra = f" (device bits 0x{bits:x})" if bits else ""
        super().__init__(f"{fn} -> {_STATUS.get(code, code)}{extra}")


def lib_path() -> str:
    return _build.LIB


def load(build_if_missing: bool = False) -> ctypes.CDLL:
    """Load librkv.so (optionally building it first)."""
    global _lib
    if _lib is not None:
        return _lib
    path = _build.LIB
    if not os.path.exists(path):
        if not build_if_missing:
            raise ImportError(f"librkv.so not found at {path}: run "
                              "`python -c 'import __graft_entry__ as g; g.build()'` first")
        _build.build()
    lib = ctypes.CDLL(path)
    vp, sz, i32, f32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_float
    u32p = ctypes.POINTER(ctypes.c_uint32)
    ip = ctypes.POINTER(ctypes.c_int)
    i64, f64 = ctypes.c_int64, ctypes.c_double
    sigs = {
        "rkv_status_string": ([i32], ctypes.c_char_p),
        "rkv_check_status": ([vp, vp, u32p], i32),
        "rkv_plan": ([i32, i32, i32, i32, i32, ip, ip, ip, ip], i32),
        "rkv_snapkv_workspace_bytes": ([i32, i32, i32, i32, i32], sz),
        "rkv_snapkv_compress": ([vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, i32, i32, f32,
                                 vp, vp, i32, vp, vp, vp, vp, sz, vp], i32),
        "rkv_snapkv_compress_avg_pool": ([vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, i32,
                                          i32, f32, vp, vp, i32, vp, vp, vp, vp, sz, vp], i32),
        "rkv_testing_scores_wait_timeout": ([vp, vp, vp, i32, i32, i32, i32, i32, i32, f32,
                                             vp, ctypes.c_uint64, vp, sz, vp], i32),
        "rkv_snapkv_scores": ([vp, vp, vp, i32, i32, i32, i32, i32, i32, f32, vp, vp, sz, vp],
                              i32),
        "rkv_testing_decode_layout": ([i32], i32),
        "rkv_snapkv_select": ([vp, vp, vp, i32, i32, i32, i32, i32, i32, i32, i32, f32, vp, i32,
                               vp, vp, vp, sz, vp], i32),
        "rkv_summaries_workspace_bytes": ([], sz),
        "rkv_build_page_summaries": ([vp, vp, i32, i32, i32, i32, i32, i32, i32, vp, vp, vp,
                                      sz, vp], i32),
        "rkv_hybrid_decode_workspace_bytes": ([i32, i32, i32, i32, i32, i32], sz),
        "rkv_hybrid_decode": ([vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32,
                               i32, i32, i32, f32, vp, vp, vp, vp, vp, sz, vp], i32),
        "rkv_dense_decode_workspace_bytes": ([i32, i32, i32, i32], sz),
        "rkv_dense_decode": ([vp, vp, vp, vp, i32, i32, i32, i32, i32, f32, vp, vp, sz, vp],
                             i32),
        "rkv_dense_decode_noalloc": ([vp, vp, vp, vp, i32, i32, i32, i32, i32, f32, vp, vp],
                                     i32),
        "rkv_plan_even_split": ([i32, i32, i32, ip, ip, ip, ip], i32),
        "rkv_snapkv_per_head_workspace_bytes": ([i32, i32, i32, i32, i32], sz),
        "rkv_snapkv_compress_per_head": ([vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, i32, i32,
                                          f32, vp, vp, i32, vp, vp, vp, vp, sz, vp], i32),
        "rkv_snapkv_compress_summarized": ([vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, i32,
                                            i32, f32, vp, vp, i32, vp, vp, vp, i32, i32, vp, vp,
                                            vp, sz, vp], i32),
        "rkv_snapkv_compress_paged": ([vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, i32, i32,
                                       f32, vp, vp, i32, i32, vp, i32, vp, vp, vp, vp, sz, vp],
                                      i32),
        "rkv_build_page_summaries_paged": ([vp, vp, vp, i32, i32, i32, i32, i32, i32, i32, i32,
                                            i32, vp, vp, vp, sz, vp], i32),
        "rkv_hybrid_decode_paged": ([vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32,
                                     i32, i32, i32, i32, i32, i32, f32, vp, vp, vp, vp, vp, sz,
                                     vp], i32),
        "rkv_build_page_summaries_mt": ([vp, vp, vp, i32, i32, i32, i32, i32, i32, i32, i32, vp,
                                         vp, vp, sz, vp], i32),
        "rkv_hybrid_decode_mt": ([vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32,
                                  i32, i32, i32, i32, i32, i32, f32, vp, vp, vp, vp, vp, sz, vp],
                                 i32),
        "rkv_kv4_append_workspace_bytes": ([i32], sz),
        "rkv_kv4_append": ([vp, vp, vp, i32, i32, i32, i32, vp, vp, vp, vp, i32, vp, vp, vp, vp,
                            vp, sz, vp], i32),
        "rkv_kv4_append_paged": ([vp, vp, vp, i32, i32, i32, i32, vp, vp, vp, vp, i32, i32, vp,
                                  i32, vp, vp, vp, vp, vp, sz, vp], i32),
        "rkv_kv4_decode_workspace_bytes": ([i32, i32, i32, i32, i32], sz),
        "rkv_kv4_decode": ([vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, f32, vp,
                            vp, vp, sz, vp], i32),
        "rkv_kv4_decode_paged": ([vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32,
                                  i32, i32, f32, vp, vp, vp, sz, vp], i32),
        "rkv_dense_decode_weights_workspace_bytes": ([i32, i32, i32, i32], sz),
        "rkv_dense_decode_weights": ([vp, vp, vp, vp, i32, i32, i32, i32, i32, f32, vp, vp, vp,
                                      sz, vp], i32),
        "rkv_prompt_weights_workspace_bytes": ([i32, i32, i32, i32, i32], sz),
        "rkv_prompt_weights": ([vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, f32, vp, vp, sz,
                                vp], i32),
        "rkv_testing_prompt_wait_timeout": ([vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, f32, vp,
                                             i32, ctypes.c_uint64, vp, sz, vp], i32),
        "rkv_evict_workspace_bytes": ([i32, i32, i32, i32], sz),
        "rkv_evict": ([vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, vp, vp,
                       sz, vp], i32),
        "rkv_evict_kv4": ([vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32,
                           i32, vp, vp, sz, vp], i32),
        "rkv_reserve_slots_workspace_bytes": ([i32], sz),
        "rkv_reserve_slots": ([vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, vp, vp, vp, vp, vp,
                               vp, vp, sz, vp], i32),
        "rkv_release_blocks_workspace_bytes": ([i32], sz),
        "rkv_release_blocks": ([vp, vp, vp, vp, vp, i32, i32, i32, i32, vp, vp, vp, sz, vp], i32),
        "rkv_rope_frequencies": ([i32, i32, f64, f64, i32, f64, f64, vp, ctypes.POINTER(f32)],
                                 i32),
        "rkv_rope_append_workspace_bytes": ([], sz),
        "rkv_rope_append": ([vp, i64, vp, i64, vp, i64, vp, vp, vp, i32, i32, i32, i32, i32, i32,
                             f32, vp, vp, vp, i32, i32, vp, sz, vp], i32),
        "rkv_prompt_attention_workspace_bytes": ([i32, i32, i32, i32], sz),
        "rkv_prompt_attention": ([vp, i64, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, f32, vp,
                                  vp, sz, vp], i32),
        "rkv_prompt_attention_paged": ([vp, i64, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32,
                                        i32, i32, f32, vp, vp, sz, vp], i32),
        "rkv_tree_attention": ([vp, i64, vp, vp, i32, vp, vp, vp, i32, i32, i32, i32, i32, i32,
                                f32, vp, vp, sz, vp], i32),
        "rkv_tree_attention_paged": ([vp, i64, vp, vp, i32, vp, vp, vp, vp, i32, i32, i32, i32,
                                      i32, i32, i32, i32, f32, vp, vp, sz, vp], i32),
        "rkv_testing_attention_wait_timeout": ([vp, i64, vp, vp, vp, vp, i32, i32, i32, i32, i32,
                                                i32, f32, vp, i32, ctypes.c_uint64, vp, sz, vp],
                                               i32),
    }
    for name, (args, res) in sigs.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    _lib = lib
    return lib


# ------------------------------------------------------------------------------- helpers
def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("librkv takes device tensors only")
    if not t.is_contiguous():
        raise ValueError("librkv takes contiguous tensors only")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _check(fn: str, code: int):
    if code != RKV_OK:
        raise RkvError(fn, code)


def _bf16(t: torch.Tensor, name: str):
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be bfloat16")


def _i32(t: torch.Tensor, name: str):
    if t.dtype != torch.int32:
        raise TypeError(f"{name} must be int32")


def _group(hq: int, n_kv: int) -> int:
    """Query heads per KV head; the query heads must split evenly over the KV heads."""
    if n_kv <= 0 or hq % n_kv != 0:
        raise ValueError(f"{hq} query heads do not split over {n_kv} KV heads")
    return hq // n_kv


def workspace(nbytes: int, device) -> torch.Tensor:
    """A zeroed workspace (the device status word must start at zero)."""
    return torch.zeros(max(int(nbytes), STATUS_BYTES), dtype=torch.uint8, device=device)


def rkv_status_string(code: int) -> str:
    return load().rkv_status_string(code).decode()


def rkv_check_status(ws: torch.Tensor, stream=None) -> int:
    """Sync, read and clear the device status word; raise RkvError if it was non-zero."""
    bits = ctypes.c_uint32(0)
    code = load().rkv_check_status(_ptr(ws), _stream(stream), ctypes.byref(bits))
    if code != RKV_OK:
        raise RkvError("rkv_check_status", code, bits.value)
    return bits.value


def rkv_plan(ctx: int, budget: int, head_dim: int = HEAD_DIM, page: int = 0, channels: int = 0):
    """(keep, page, channels, kernel_size) for one sequence."""
    out = [ctypes.c_int(0) for _ in range(4)]
    code = load().rkv_plan(ctx, budget, head_dim, page, channels, *[ctypes.byref(o) for o in out])
    _check("rkv_plan", code)
    return tuple(o.value for o in out)


def rkv_plan_even_split(ctx: int, budget: int, head_dim: int = HEAD_DIM):
    """(keep, page, channels, kernel_size) from the even split of ctx / budget."""
    out = [ctypes.c_int(0) for _ in range(4)]
    code = load().rkv_plan_even_split(ctx, budget, head_dim, *[ctypes.byref(o) for o in out])
    _check("rkv_plan_even_split", code)
    return tuple(o.value for o in out)


# ------------------------------------------------------------------------------- stage 1
def rkv_snapkv_workspace_bytes(n: int, n_kv: int, gqa: int, max_len: int, window: int) -> int:
    return int(load().rkv_snapkv_workspace_bytes(n, n_kv, gqa, max_len, window))


def rkv_snapkv_compress(k, v, seq_lens, q_win, kernel_size: int, keep: int, scale: float,
                        k_out, v_out, kept_idx, out_len, scores_out=None, ws=None,
                        stream=None):
    """SnapKV++ compression of every (unit, KV head); see include/rkv.h."""
    _bf16(k, "k"), _bf16(v, "v"), _bf16(q_win, "q_win"), _i32(seq_lens, "seq_lens")
    _i32(kept_idx, "kept_idx"), _i32(out_len, "out_len")
    n, n_kv, max_len, d = k.shape
    hq, window = q_win.shape[1], q_win.shape[2]
    gqa = _group(hq, n_kv)
    cap = k_out.shape[2]
    if ws is None:
        ws = workspace(rkv_snapkv_workspace_bytes(n, n_kv, gqa, max_len, window), k.device)
    code = load().rkv_snapkv_compress(
        _ptr(k), _ptr(v), _ptr(seq_lens), _ptr(q_win), n, n_kv, gqa, d, max_len, window,
        kernel_size, keep, float(scale), _ptr(k_out), _ptr(v_out), cap, _ptr(kept_idx),
        _ptr(out_len), _ptr(scores_out), _ptr(ws), ws.numel(), _stream(stream))
    _check("rkv_snapkv_compress", code)
    return ws


def rkv_snapkv_compress_avg_pool(k, v, seq_lens, q_win, kernel_size: int, keep: int,
                                 scale: float, k_out, v_out, kept_idx, out_len, scores_out=None,
                                 ws=None, stream=None):
    """SnapKV++ compression with average instead of max pooling; see include/rkv.h."""
    _bf16(k, "k"), _bf16(v, "v"), _bf16(q_win, "q_win"), _i32(seq_lens, "seq_lens")
    _i32(kept_idx, "kept_idx"), _i32(out_len, "out_len")
    n, n_kv, max_len, d = k.shape
    hq, window = q_win.shape[1], q_win.shape[2]
    gqa = _group(hq, n_kv)
    cap = k_out.shape[2]
    if ws is None:
        ws = workspace(rkv_snapkv_workspace_bytes(n, n_kv, gqa, max_len, window), k.device)
    code = load().rkv_snapkv_compress_avg_pool(
        _ptr(k), _ptr(v), _ptr(seq_lens), _ptr(q_win), n, n_kv, gqa, d, max_len, window,
        kernel_size, keep, float(scale), _ptr(k_out), _ptr(v_out), cap, _ptr(kept_idx),
        _ptr(out_len), _ptr(scores_out), _ptr(ws), ws.numel(), _stream(stream))
    _check("rkv_snapkv_compress_avg_pool", code)
    return ws


def rkv_snapkv_select(k, seq_lens, q_win, kernel_size: int, keep: int, scale: float, kept_idx,
                      out_len, scores_out=None, ws=None, stream=None):
    """RocketKV-MT stage 1: scores, pooling and top-k over the full history, kept indices only
    (kept_idx [n][n_kv][kept_stride], kept_stride >= keep); see include/rkv.h."""
    _bf16(k, "k"), _bf16(q_win, "q_win"), _i32(seq_lens, "seq_lens")
    _i32(kept_idx, "kept_idx"), _i32(out_len, "out_len")
    n, n_kv, max_len, d = k.shape
    hq, window = q_win.shape[1], q_win.shape[2]
    gqa = _group(hq, n_kv)
    if ws is None:
        ws = workspace(rkv_snapkv_workspace_bytes(n, n_kv, gqa, max_len, window), k.device)
    code = load().rkv_snapkv_select(
        _ptr(k), _ptr(seq_lens), _ptr(q_win), n, n_kv, gqa, d, max_len, window, kernel_size,
        keep, float(scale), _ptr(kept_idx), kept_idx.shape[2], _ptr(out_len), _ptr(scores_out),
        _ptr(ws), ws.numel(), _stream(stream))
    _check("rkv_snapkv_select", code)
    return ws


def rkv_snapkv_scores(k, seq_lens, q_win, scale: float, scores_out, ws=None, stream=None):
    """Stage-1 window scores only (no pooling, selection or gather) into
    scores_out [n][n_kv][max_len - window] fp32; see include/rkv.h."""
    _bf16(k, "k"), _bf16(q_win, "q_win"), _i32(seq_lens, "seq_lens")
    n, n_kv, max_len, d = k.shape
    hq, window = q_win.shape[1], q_win.shape[2]
    gqa = _group(hq, n_kv)
    if ws is None:
        ws = workspace(rkv_snapkv_workspace_bytes(n, n_kv, gqa, max_len, window), k.device)
    code = load().rkv_snapkv_scores(
        _ptr(k), _ptr(seq_lens), _ptr(q_win), n, n_kv, gqa, d, max_len, window, float(scale),
        _ptr(scores_out), _ptr(ws), ws.numel(), _stream(stream))
    _check("rkv_snapkv_scores", code)
    return ws


def rkv_testing_scores_wait_timeout(k, seq_lens, q_win, scale: float, scores_out,
                                    wait_limit_ns: int, ws=None, stream=None):
    """Test hook (include/rkv_testing.h): the score passes with one K tile of block 0 never
    loaded, so that its bounded waits run out after wait_limit_ns."""
    _bf16(k, "k"), _bf16(q_win, "q_win"), _i32(seq_lens, "seq_lens")
    n, n_kv, max_len, d = k.shape
    hq, window = q_win.shape[1], q_win.shape[2]
    gqa = _group(hq, n_kv)
    if ws is None:
        ws = workspace(rkv_snapkv_workspace_bytes(n, n_kv, gqa, max_len, window), k.device)
    code = load().rkv_testing_scores_wait_timeout(
        _ptr(k), _ptr(seq_lens), _ptr(q_win), n, n_kv, gqa, d, max_len, window, float(scale),
        _ptr(scores_out), int(wait_limit_ns), _ptr(ws), ws.numel(), _stream(stream))
    _check("rkv_testing_scores_wait_timeout", code)
    return ws


def rkv_testing_decode_layout(layout: int) -> None:
    """Test hook (include/rkv_testing.h): the hybrid decode's shared-memory layout for later
    calls in this process (0 automatic, 1 ordinary, 2 wide wherever it fits)."""
    _check("rkv_testing_decode_layout", load().rkv_testing_decode_layout(int(layout)))


def rkv_snapkv_per_head_workspace_bytes(n: int, n_kv: int, gqa: int, max_len: int,
                                        window: int) -> int:
    return int(load().rkv_snapkv_per_head_workspace_bytes(n, n_kv, gqa, max_len, window))


def rkv_snapkv_compress_per_head(k, v, seq_lens, q_win, kernel_size: int, keep: int,
                                 scale: float, k_out, v_out, kept_idx, out_len, scores_out=None,
                                 ws=None, stream=None):
    """SnapKV without the GQA sum: every query head scored and filtered on its own; outputs per
    query head ([n][n_kv*gqa][...]); see include/rkv.h."""
    _bf16(k, "k"), _bf16(v, "v"), _bf16(q_win, "q_win"), _i32(seq_lens, "seq_lens")
    _i32(kept_idx, "kept_idx"), _i32(out_len, "out_len")
    n, n_kv, max_len, d = k.shape
    hq, window = q_win.shape[1], q_win.shape[2]
    gqa = _group(hq, n_kv)
    cap = k_out.shape[2]
    if ws is None:
        ws = workspace(rkv_snapkv_per_head_workspace_bytes(n, n_kv, gqa, max_len, window),
                       k.device)
    code = load().rkv_snapkv_compress_per_head(
        _ptr(k), _ptr(v), _ptr(seq_lens), _ptr(q_win), n, n_kv, gqa, d, max_len, window,
        kernel_size, keep, float(scale), _ptr(k_out), _ptr(v_out), cap, _ptr(kept_idx),
        _ptr(out_len), _ptr(scores_out), _ptr(ws), ws.numel(), _stream(stream))
    _check("rkv_snapkv_compress_per_head", code)
    return ws


def rkv_snapkv_compress_summarized(k, v, seq_lens, q_win, kernel_size: int, keep: int,
                                   scale: float, k_out, v_out, kept_idx, out_len, page: int,
                                   kmin, kmax, scores_out=None, ws=None, stream=None):
    """rkv_snapkv_compress + page summaries of the compact cache in one pass."""
    _bf16(k, "k"), _bf16(v, "v"), _bf16(q_win, "q_win"), _i32(seq_lens, "seq_lens")
    _i32(kept_idx, "kept_idx"), _i32(out_len, "out_len"), _bf16(kmin, "kmin")
    n, n_kv, max_len, d = k.shape
    hq, window = q_win.shape[1], q_win.shape[2]
    gqa = _group(hq, n_kv)
    cap = k_out.shape[2]
    page_cap = kmin.shape[-1]
    if ws is None:
        ws = workspace(rkv_snapkv_workspace_bytes(n, n_kv, gqa, max_len, window), k.device)
    code = load().rkv_snapkv_compress_summarized(
        _ptr(k), _ptr(v), _ptr(seq_lens), _ptr(q_win), n, n_kv, gqa, d, max_len, window,
        kernel_size, keep, float(scale), _ptr(k_out), _ptr(v_out), cap, _ptr(kept_idx),
        _ptr(out_len), _ptr(scores_out), page, page_cap, _ptr(kmin), _ptr(kmax), _ptr(ws),
        ws.numel(), _stream(stream))
    _check("rkv_snapkv_compress_summarized", code)
    return ws


# ------------------------------------------------------------------------------- stage 2
def rkv_build_page_summaries(k_cache, length, page: int, kmin, kmax, first_token: int = 0,
                             ws=None, stream=None):
    _bf16(k_cache, "k_cache"), _i32(length, "len")
    n, n_kv, cap, d = k_cache.shape
    page_cap = kmin.shape[-1]
    if ws is None:
        ws = workspace(STATUS_BYTES, k_cache.device)
    code = load().rkv_build_page_summaries(
        _ptr(k_cache), _ptr(length), n, n_kv, d, cap, page, page_cap, first_token, _ptr(kmin),
        _ptr(kmax), _ptr(ws), ws.numel(), _stream(stream))
    _check("rkv_build_page_summaries", code)
    return ws


def rkv_hybrid_decode_workspace_bytes(n, n_kv, gqa, page_cap, budget, page) -> int:
    return int(load().rkv_hybrid_decode_workspace_bytes(n, n_kv, gqa, page_cap, budget, page))


def rkv_hybrid_decode(q, k_cache, v_cache, length, kmin, kmax, budget: int, page: int,
                      channels: int, scale: float, out, new_k=None, new_v=None,
                      sel_channels=None, sel_pages=None, approx_scores=None, ws=None,
                      stream=None):
    """One hybrid sparse decode step (optionally appending new_k / new_v first)."""
    _bf16(q, "q"), _bf16(k_cache, "k_cache"), _i32(length, "len")
    n, n_kv, cap, d = k_cache.shape
    gqa = _group(q.shape[1], n_kv)
    page_cap = kmin.shape[-1]
    if ws is None:
        ws = workspace(rkv_hybrid_decode_workspace_bytes(n, n_kv, gqa, page_cap, budget, page),
                       q.device)
    code = load().rkv_hybrid_decode(
        _ptr(q), _ptr(new_k), _ptr(new_v), _ptr(k_cache), _ptr(v_cache), _ptr(length),
        _ptr(kmin), _ptr(kmax), n, n_kv, gqa, d, cap, page_cap, budget, page, channels,
        float(scale), _ptr(out), _ptr(sel_channels), _ptr(sel_pages), _ptr(approx_scores),
        _ptr(ws), ws.numel(), _stream(stream))
    _check("rkv_hybrid_decode", code)
    return ws


def rkv_build_page_summaries_mt(k_full, kept_idx, kept_len, page: int, kmin, kmax,
                                first_token: int = 0, ws=None, stream=None):
    """Page summaries of the kept sequence k_full[u][g][kept_idx[u][g][j]] (RocketKV-MT)."""
    _bf16(k_full, "k_full"), _i32(kept_idx, "kept_idx"), _i32(kept_len, "kept_len")
    n, n_kv, full_cap, d = k_full.shape
    kcap = kept_idx.shape[-1]
    page_cap = kmin.shape[-1]
    if ws is None:
        ws = workspace(STATUS_BYTES, k_full.device)
    code = load().rkv_build_page_summaries_mt(
        _ptr(k_full), _ptr(kept_idx), _ptr(kept_len), n, n_kv, d, full_cap, kcap, page, page_cap,
        first_token, _ptr(kmin), _ptr(kmax), _ptr(ws), ws.numel(), _stream(stream))
    _check("rkv_build_page_summaries_mt", code)
    return ws


def rkv_hybrid_decode_mt(q, k_full, v_full, full_len, kept_idx, kept_len, kmin, kmax,
                         budget: int, page: int, channels: int, scale: float, out, new_k=None,
                         new_v=None, sel_channels=None, sel_pages=None, approx_scores=None,
                         ws=None, stream=None):
    """One hybrid decode step over the kept sequence of the full cache (RocketKV-MT),
    optionally appending new_k / new_v to the full cache and the kept list first."""
    _bf16(q, "q"), _bf16(k_full, "k_full"), _i32(full_len, "full_len")
    _i32(kept_idx, "kept_idx"), _i32(kept_len, "kept_len")
    n, n_kv, full_cap, d = k_full.shape
    gqa = _group(q.shape[1], n_kv)
    kcap = kept_idx.shape[-1]
    page_cap = kmin.shape[-1]
    if ws is None:
        ws = workspace(rkv_hybrid_decode_workspace_bytes(n, n_kv, gqa, page_cap, budget, page),
                       q.device)
    code = load().rkv_hybrid_decode_mt(
        _ptr(q), _ptr(new_k), _ptr(new_v), _ptr(k_full), _ptr(v_full), _ptr(full_len),
        _ptr(kept_idx), _ptr(kept_len), _ptr(kmin), _ptr(kmax), n, n_kv, gqa, d, full_cap, kcap,
        page_cap, budget, page, channels, float(scale), _ptr(out), _ptr(sel_channels),
        _ptr(sel_pages), _ptr(approx_scores), _ptr(ws), ws.numel(), _stream(stream))
    _check("rkv_hybrid_decode_mt", code)
    return ws


# ------------------------------------------------------------------------------- paged cache
def rkv_snapkv_compress_paged(k, v, seq_lens, q_win, kernel_size: int, keep: int, scale: float,
                              k_pool, v_pool, block_table, kept_idx, out_len, scores_out=None,
                              ws=None, stream=None):
    """SnapKV++ compression whose kept rows go to the pools through the block table."""
    _bf16(k, "k"), _bf16(k_pool, "k_pool"), _i32(block_table, "block_table")
    _i32(kept_idx, "kept_idx"), _i32(out_len, "out_len"), _i32(seq_lens, "seq_lens")
    n, n_kv, max_len, d = k.shape
    hq, window = q_win.shape[1], q_win.shape[2]
    gqa = _group(hq, n_kv)
    num_blocks, _, block, _ = k_pool.shape
    max_blocks = block_table.shape[-1]
    if ws is None:
        ws = workspace(rkv_snapkv_workspace_bytes(n, n_kv, gqa, max_len, window), k.device)
    code = load().rkv_snapkv_compress_paged(
        _ptr(k), _ptr(v), _ptr(seq_lens), _ptr(q_win), n, n_kv, gqa, d, max_len, window,
        kernel_size, keep, float(scale), _ptr(k_pool), _ptr(v_pool), num_blocks, block,
        _ptr(block_table), max_blocks, _ptr(kept_idx), _ptr(out_len), _ptr(scores_out), _ptr(ws),
        ws.numel(), _stream(stream))
    _check("rkv_snapkv_compress_paged", code)
    return ws


def rkv_build_page_summaries_paged(k_pool, block_table, length, page: int, kmin, kmax,
                                   first_token: int = 0, ws=None, stream=None):
    _bf16(k_pool, "k_pool"), _i32(block_table, "block_table"), _i32(length, "len")
    num_blocks, n_kv, block, d = k_pool.shape
    n, max_blocks = block_table.shape
    page_cap = kmin.shape[-1]
    if ws is None:
        ws = workspace(STATUS_BYTES, k_pool.device)
    code = load().rkv_build_page_summaries_paged(
        _ptr(k_pool), _ptr(block_table), _ptr(length), n, n_kv, d, num_blocks, block, max_blocks,
        page, page_cap, first_token, _ptr(kmin), _ptr(kmax), _ptr(ws), ws.numel(),
        _stream(stream))
    _check("rkv_build_page_summaries_paged", code)
    return ws


def rkv_hybrid_decode_paged(q, k_pool, v_pool, block_table, length, kmin, kmax, budget: int,
                            page: int, channels: int, scale: float, out, new_k=None, new_v=None,
                            sel_channels=None, sel_pages=None, approx_scores=None, ws=None,
                            stream=None):
    """One hybrid decode step over a paged cache (appending new_k / new_v first if given)."""
    _bf16(q, "q"), _bf16(k_pool, "k_pool"), _i32(block_table, "block_table"), _i32(length, "len")
    num_blocks, n_kv, block, d = k_pool.shape
    n, max_blocks = block_table.shape
    gqa = _group(q.shape[1], n_kv)
    page_cap = kmin.shape[-1]
    if ws is None:
        ws = workspace(rkv_hybrid_decode_workspace_bytes(n, n_kv, gqa, page_cap, budget, page),
                       q.device)
    code = load().rkv_hybrid_decode_paged(
        _ptr(q), _ptr(new_k), _ptr(new_v), _ptr(k_pool), _ptr(v_pool), _ptr(block_table),
        _ptr(length), _ptr(kmin), _ptr(kmax), n, n_kv, gqa, d, num_blocks, block, max_blocks,
        page_cap, budget, page, channels, float(scale), _ptr(out), _ptr(sel_channels),
        _ptr(sel_pages), _ptr(approx_scores), _ptr(ws), ws.numel(), _stream(stream))
    _check("rkv_hybrid_decode_paged", code)
    return ws


def rkv_dense_decode_workspace_bytes(n, n_kv, gqa, max_len) -> int:
    return int(load().rkv_dense_decode_workspace_bytes(n, n_kv, gqa, max_len))


def rkv_dense_decode(q, k, v, length, scale: float, out, ws=None, stream=None):
    """Full-KV decode attention over len[u] tokens."""
    _bf16(q, "q"), _bf16(k, "k"), _i32(length, "len")
    n, n_kv, max_len, d = k.shape
    gqa = _group(q.shape[1], n_kv)
    if ws is None:
        ws = workspace(rkv_dense_decode_workspace_bytes(n, n_kv, gqa, max_len), q.device)
    code = load().rkv_dense_decode(_ptr(q), _ptr(k), _ptr(v), _ptr(length), n, n_kv, gqa, d,
                                   max_len, float(scale), _ptr(out), _ptr(ws), ws.numel(),
                                   _stream(stream))
    _check("rkv_dense_decode", code)
    return ws


def rkv_dense_decode_noalloc(q, k, v, length, scale: float, out, stream=None):
    """Dense decode without a workspace: the library's fixed device scratch holds the partials.
    For callers that cannot allocate; calls sharing the scratch must not overlap on the GPU."""
    _bf16(q, "q"), _bf16(k, "k"), _i32(length, "len")
    n, n_kv, max_len, d = k.shape
    gqa = _group(q.shape[1], n_kv)
    code = load().rkv_dense_decode_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(length), n, n_kv, gqa,
                                           d, max_len, float(scale), _ptr(out), _stream(stream))
    _check("rkv_dense_decode_noalloc", code)


# ------------------------------------------------------------------------------- 4-bit cache
CODE_BYTES = HEAD_DIM // 2
ROW_SCALES = HEAD_DIM // 16
_BF16, _F32, _I32, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


def _refuse(t, name, dtype, shape, dev):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {str(dtype).replace('torch.', '')}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.get_device() < 0:
        raise ValueError(f"{name}: librkv takes device tensors only")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on cuda:{t.get_device()}, others on cuda:{dev}")
    raise ValueError(f"{name}: librkv takes contiguous tensors only")


def _at(t, name, dtype, shape, dev):
    """Address of a tensor of the call, after its type, shape, layout and device (a call's own
    cost is what a small step waits for, so this is one chain of cheap tests)."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape
            and t.is_contiguous() and t.get_device() == dev):
        return t.data_ptr()
    _refuse(t, name, dtype, shape, dev)


def _weights16(t, shape, dev, given=True):
    """Address of a decode's weights, which begin on 16 bytes: a slice of a larger array need not.
    given: they have to be (else None: not asked for)."""
    p = (_at if given else _at_or_none)(t, "weights", _F32, shape, dev)
    if p is not None and p % 16:
        raise ValueError("weights must begin on a 16-byte boundary: a slice of units does where "
                         "n_kv * cap is a multiple of 4")
    return p


def _first(t, name, dtype, rank, dev):
    """Shape and address of a tensor that others' shapes follow from."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a tensor of {rank} dimensions")
    shape = t.shape
    if len(shape) != rank:
        raise ValueError(f"{name} must be a tensor of {rank} dimensions")
    if t.dtype is dtype and t.is_contiguous() and t.get_device() == dev:
        return shape, t.data_ptr()
    _refuse(t, name, dtype, shape, dev)


def _at_or_none(t, name, dtype, shape, dev):
    return None if t is None else _at(t, name, dtype, shape, dev)


def _dims(t, name, rank):
    if not isinstance(t, torch.Tensor) or t.dim() != rank:
        raise ValueError(f"{name} must be a tensor of {rank} dimensions")
    return t.shape


def _call(fn, args, ws, nbytes, dev, stream):
    """Run entry point `fn` on the device of its tensors and the stream given (or that device's
    current one). nbytes(): the workspace to make where none is given; it is made on that stream."""
    if dev < 0:
        raise ValueError("librkv takes device tensors only")
    if stream is not None or torch._C._cuda_getDevice() != dev:
        if stream is not None and stream.device.index != dev:
            raise ValueError(f"stream of {stream.device} for tensors on cuda:{dev}")
        with torch.cuda.stream(stream or torch.cuda.current_stream(dev)):
            return _call(fn, args, ws, nbytes, dev, None)
    if ws is None:
        ws = workspace(nbytes(), torch.device("cuda", dev))
    elif ws.dtype is not _U8 or ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError("the workspace must be contiguous bytes on the tensors' device")
    code = getattr(load(), fn)(*args, ws.data_ptr(), ws.numel(),
                               torch._C._cuda_getCurrentRawStream(dev))
    if code != RKV_OK:
        raise RkvError(fn, code)
    return ws


def kv4_cache(n: int, n_kv: int, cap: int, device="cuda"):
    """Zeroed arrays of a 4-bit cache: (k_codes, k_scales, v_codes, v_scales)."""
    z = lambda w: torch.zeros(n, n_kv, cap, w, dtype=torch.uint8, device=device)  # noqa: E731
    return z(CODE_BYTES), z(ROW_SCALES), z(CODE_BYTES), z(ROW_SCALES)


def _kv4(k_codes, k_scales, v_codes, v_scales, dev):
    """Leading dimensions and addresses of a 4-bit cache."""
    a, b, c, _ = _dims(k_codes, "k_codes", 4)
    codes, scales = (a, b, c, CODE_BYTES), (a, b, c, ROW_SCALES)
    return a, b, c, (_at(k_codes, "k_codes", _U8, codes, dev),
                     _at(k_scales, "k_scales", _U8, scales, dev),
                     _at(v_codes, "v_codes", _U8, codes, dev),
                     _at(v_scales, "v_scales", _U8, scales, dev))


def rkv_kv4_append_workspace_bytes(n: int) -> int:
    return int(load().rkv_kv4_append_workspace_bytes(n))


def _kv4_append(fn, new_k, new_v, cache, table, length, length_out, new_len, k_values, v_values,
                ws, stream):
    n, n_kv, max_new, d = shape = _dims(new_k, "new_k", 4)
    dev = new_k.get_device()
    lead, heads, rows, ptrs = _kv4(*cache, dev)
    if heads != n_kv:
        raise ValueError(f"new_k has {n_kv} KV heads, the cache {heads}")
    if table is None:
        if lead != n:
            raise ValueError(f"{n} units of new rows for a cache of {lead}")
        size = (rows,)
    else:
        max_blocks = _dims(table, "block_table", 2)[1]
        size = (lead, rows, _at(table, "block_table", _I32, (n, max_blocks), dev), max_blocks)
    args = (_at(new_k, "new_k", _BF16, shape, dev), _at(new_v, "new_v", _BF16, shape, dev),
            _at_or_none(new_len, "new_len", _I32, (n,), dev), n, n_kv, d, max_new, *ptrs, *size,
            _at(length, "len", _I32, (n,), dev), _at(length_out, "len_out", _I32, (n,), dev),
            _at_or_none(k_values, "k_values", _BF16, shape, dev),
            _at_or_none(v_values, "v_values", _BF16, shape, dev))
    return _call(fn, args, ws, lambda: rkv_kv4_append_workspace_bytes(n), dev, stream)


def rkv_kv4_append(new_k, new_v, k_codes, k_scales, v_codes, v_scales, length, length_out,
                   new_len=None, k_values=None, v_values=None, ws=None, stream=None):
    """Quantise new rows ([n][n_kv][max_new][128] bf16) behind each unit's length[u] rows; see
    include/rkv.h. length_out may be length."""
    return _kv4_append("rkv_kv4_append", new_k, new_v, (k_codes, k_scales, v_codes, v_scales),
                       None, length, length_out, new_len, k_values, v_values, ws, stream)


def rkv_kv4_append_paged(new_k, new_v, k_codes, k_scales, v_codes, v_scales, block_table, length,
                         length_out, new_len=None, k_values=None, v_values=None, ws=None,
                         stream=None):
    """rkv_kv4_append into pools [num_blocks][n_kv][block][..] through block_table [n][max_blocks]."""
    _dims(block_table, "block_table", 2)
    return _kv4_append("rkv_kv4_append_paged", new_k, new_v,
                       (k_codes, k_scales, v_codes, v_scales), block_table, length, length_out,
                       new_len, k_values, v_values, ws, stream)


def rkv_kv4_decode_workspace_bytes(n: int, n_kv: int, gqa: int, cap: int,
                                   with_weights: bool) -> int:
    return int(load().rkv_kv4_decode_workspace_bytes(n, n_kv, gqa, cap, int(with_weights)))


def rkv_kv4_decode(q, k_codes, k_scales, v_codes, v_scales, length, scale: float, out, new_k=None,
                   new_v=None, length_out=None, weights=None, ws=None, stream=None):
    """One decode step over the 4-bit cache, optionally appending new_k / new_v first and adding
    each token's softmax weight to weights; see include/rkv.h. length_out may be length."""
    shape = _dims(q, "q", 3)
    dev = q.get_device()
    n, n_kv, cap, ptrs = _kv4(k_codes, k_scales, v_codes, v_scales, dev)
    gqa, d = _group(shape[1], n_kv), shape[2]
    args = (_at(q, "q", _BF16, (n, shape[1], d), dev),
            _at_or_none(new_k, "new_k", _BF16, (n, n_kv, d), dev),
            _at_or_none(new_v, "new_v", _BF16, (n, n_kv, d), dev), *ptrs,
            _at(length, "len", _I32, (n,), dev),
            _at_or_none(length_out, "len_out", _I32, (n,), dev), n, n_kv, gqa, d, cap, scale,
            _at(out, "out", _BF16, shape, dev),
            _weights16(weights, (n, n_kv, cap), dev, given=False))
    return _call("rkv_kv4_decode", args, ws,
                 lambda: rkv_kv4_decode_workspace_bytes(n, n_kv, gqa, cap, weights is not None),
                 dev, stream)


def rkv_kv4_decode_paged(q, k_codes, k_scales, v_codes, v_scales, block_table, length,
                         scale: float, out, new_k=None, new_v=None, length_out=None, weights=None,
                         ws=None, stream=None):
    """rkv_kv4_decode over pools [num_blocks][n_kv][block][..] through block_table
    [n][max_blocks]; weights [n][n_kv][max_blocks * block]."""
    n, hq, d = shape = _dims(q, "q", 3)
    dev = q.get_device()
    num_blocks, n_kv, block, ptrs = _kv4(k_codes, k_scales, v_codes, v_scales, dev)
    max_blocks = _dims(block_table, "block_table", 2)[1]
    gqa, cap = _group(hq, n_kv), max_blocks * block
    args = (_at(q, "q", _BF16, shape, dev),
            _at_or_none(new_k, "new_k", _BF16, (n, n_kv, d), dev),
            _at_or_none(new_v, "new_v", _BF16, (n, n_kv, d), dev), *ptrs,
            _at(block_table, "block_table", _I32, (n, max_blocks), dev),
            _at(length, "len", _I32, (n,), dev),
            _at_or_none(length_out, "len_out", _I32, (n,), dev), n, n_kv, gqa, d, num_blocks,
            block, max_blocks, scale, _at(out, "out", _BF16, shape, dev),
            _weights16(weights, (n, n_kv, cap), dev, given=False))
    return _call("rkv_kv4_decode_paged", args, ws,
                 lambda: rkv_kv4_decode_workspace_bytes(n, n_kv, gqa, cap, weights is not None),
                 dev, stream)


# ------------------------------------------------------------------------------- weights, eviction
def rkv_dense_decode_weights_workspace_bytes(n: int, n_kv: int, gqa: int, max_len: int) -> int:
    return int(load().rkv_dense_decode_weights_workspace_bytes(n, n_kv, gqa, max_len))


def rkv_dense_decode_weights(q, k, v, length, scale: float, out, weights, ws=None, stream=None):
    """Full-KV decode attention that adds each token's softmax weight (summed over the query heads
    of its group) to weights [n][n_kv][max_len] fp32."""
    n, n_kv, max_len, d = shape = _dims(k, "k", 4)
    hq = _dims(q, "q", 3)[1]
    gqa, dev = _group(hq, n_kv), q.get_device()
    args = (_at(q, "q", _BF16, (n, hq, d), dev), _at(k, "k", _BF16, shape, dev),
            _at(v, "v", _BF16, shape, dev), _at(length, "len", _I32, (n,), dev), n, n_kv, gqa, d,
            max_len, scale, _at(out, "out", _BF16, (n, hq, d), dev),
            _weights16(weights, (n, n_kv, max_len), dev))
    return _call("rkv_dense_decode_weights", args, ws,
                 lambda: rkv_dense_decode_weights_workspace_bytes(n, n_kv, gqa, max_len), dev,
                 stream)


def rkv_prompt_weights_workspace_bytes(n: int, n_kv: int, gqa: int, max_q: int,
                                       max_len: int) -> int:
    return int(load().rkv_prompt_weights_workspace_bytes(n, n_kv, gqa, max_q, max_len))


def _prompt(fn, hook, q, q_len, k, length, scale, weights, ws, stream):
    n, n_kv, max_len, d = shape = _dims(k, "k", 4)
    _, hq, max_q, _ = _dims(q, "q", 4)
    gqa, dev = _group(hq, n_kv), q.get_device()
    args = (_at(q, "q", _BF16, (n, hq, max_q, d), dev), _at(q_len, "q_len", _I32, (n,), dev),
            _at(k, "k", _BF16, shape, dev), _at(length, "len", _I32, (n,), dev), n, n_kv, gqa, d,
            max_q, max_len, scale, _at(weights, "weights", _F32, (n, n_kv, max_len), dev), *hook)
    return _call(fn, args, ws,
                 lambda: rkv_prompt_weights_workspace_bytes(n, n_kv, gqa, max_q, max_len), dev,
                 stream)


def rkv_prompt_weights(q, q_len, k, length, scale: float, weights, ws=None, stream=None):
    """Adds the softmax weight that every key gets from the last q_len[u] positions' queries
    (q [n][Hq][max_q][128]) to weights [n][n_kv][max_len] fp32; see include/rkv.h."""
    return _prompt("rkv_prompt_weights", (), q, q_len, k, length, scale, weights, ws, stream)


def rkv_testing_prompt_wait_timeout(q, q_len, k, length, scale: float, weights, what: int,
                                    wait_limit_ns: int, ws=None, stream=None):
    """Test hook (include/rkv_testing.h): rkv_prompt_weights with one load of block 0 never
    requested, so that its bounded waits run out after wait_limit_ns."""
    return _prompt("rkv_testing_prompt_wait_timeout", (int(what), int(wait_limit_ns)), q, q_len, k,
                   length, scale, weights, ws, stream)


def rkv_evict_workspace_bytes(n: int, n_kv: int, cap: int, keep: int) -> int:
    return int(load().rkv_evict_workspace_bytes(n, n_kv, cap, keep))


def _evict(fn, ptrs, n, n_kv, cap, d, length, weights, pos, seen, keep, recent, length_out,
           weights_out, pos_out, src_rows, ws, dev, stream):
    rows = (n, n_kv, cap)
    args = (*ptrs, _at(length, "len", _I32, (n,), dev), _at(length_out, "len_out", _I32, (n,), dev),
            _at(weights, "weights", _F32, rows, dev), _at(weights_out, "weights_out", _F32, rows, dev),
            _at(pos, "pos", _I32, rows, dev), _at(pos_out, "pos_out", _I32, rows, dev),
            _at(seen, "seen", _I32, (n,), dev), n, n_kv, d, cap, keep, recent,
            _at_or_none(src_rows, "src_rows", _I32, (n, n_kv, keep), dev))
    return _call(fn, args, ws, lambda: rkv_evict_workspace_bytes(n, n_kv, cap, keep), dev, stream)


def rkv_evict(k, v, length, weights, pos, seen, keep: int, recent: int, length_out, weights_out,
              pos_out, src_rows=None, ws=None, stream=None):
    """Keep the `keep` rows of largest weight (the last `recent` positions always) of every
    (unit, KV head), in place; the *_out arrays may be the inputs. See include/rkv.h."""
    n, n_kv, cap, d = shape = _dims(k, "k", 4)
    dev = k.get_device()
    ptrs = (_at(k, "k", _BF16, shape, dev), _at(v, "v", _BF16, shape, dev))
    return _evict("rkv_evict", ptrs, n, n_kv, cap, d, length, weights, pos, seen, keep, recent,
                  length_out, weights_out, pos_out, src_rows, ws, dev, stream)


def rkv_evict_kv4(k_codes, k_scales, v_codes, v_scales, length, weights, pos, seen, keep: int,
                  recent: int, length_out, weights_out, pos_out, src_rows=None, ws=None,
                  stream=None):
    """rkv_evict of a 4-bit cache."""
    _dims(k_codes, "k_codes", 4)
    dev = k_codes.get_device()
    n, n_kv, cap, ptrs = _kv4(k_codes, k_scales, v_codes, v_scales, dev)
    return _evict("rkv_evict_kv4", ptrs, n, n_kv, cap, HEAD_DIM, length, weights, pos, seen, keep,
                  recent, length_out, weights_out, pos_out, src_rows, ws, dev, stream)


# ------------------------------------------------------------------------------- a serving step
def _tokens(t, name, heads, dev, tokens):
    """Address and token stride (elements) of packed rows [tokens][heads][128] bf16: contiguous, or a
    slice of rows that hold more (the strides of tokens free, a token's heads side by side)."""
    if (isinstance(t, torch.Tensor) and t.dtype is _BF16 and t.shape == (tokens, heads, HEAD_DIM)
            and t.get_device() == dev):
        stride, head, one = t.stride()
        if one == 1 and (head == HEAD_DIM or heads == 1):
            if tokens <= 1:
                stride = heads * HEAD_DIM
            p = t.data_ptr()
            if p % 16 or stride % 8 or stride < heads * HEAD_DIM:
                raise ValueError(f"{name}: tokens must begin on 16 bytes and not overlap")
            return p, stride
        raise ValueError(f"{name}: the heads of a token must lie side by side")
    _refuse(t, name, _BF16, (tokens, heads, HEAD_DIM), dev)


def rkv_reserve_slots_workspace_bytes(n: int) -> int:
    return int(load().rkv_reserve_slots_workspace_bytes(n))


def rkv_reserve_slots(new_len, length, held, block_table, free_blocks, free_count, block: int, q_start,
                      slots, positions, length_out, held_out, free_count_out, ws=None, stream=None):
    """Places for new_len[u] more tokens of every unit: blocks off the free stack into block_table,
    q_start [n + 1], and slots and positions [max_tokens] of the packed tokens; see include/rkv.h.
    length_out, held_out and free_count_out may be the inputs."""
    _dims(block_table, "block_table", 2)
    dev = block_table.get_device()
    (n, max_blocks), table = _first(block_table, "block_table", _I32, 2, dev)
    (num_blocks,), free = _first(free_blocks, "free_blocks", _I32, 1, dev)
    (room,), places = _first(slots, "slots", _I32, 1, dev)
    each, one = (n,), (1,)
    args = (_at(new_len, "new_len", _I32, each, dev), _at(length, "len", _I32, each, dev),
            _at(held, "held", _I32, each, dev), table, free,
            _at(free_count, "free_count", _I32, one, dev), n, num_blocks, block, max_blocks, room,
            _at(q_start, "q_start", _I32, (n + 1,), dev), places,
            _at(positions, "positions", _I32, (room,), dev),
            _at(length_out, "len_out", _I32, each, dev), _at(held_out, "held_out", _I32, each, dev),
            _at(free_count_out, "free_count_out", _I32, one, dev))
    return _call("rkv_reserve_slots", args, ws, lambda: rkv_reserve_slots_workspace_bytes(n), dev,
                 stream)


def rkv_release_blocks_workspace_bytes(n: int) -> int:
    return int(load().rkv_release_blocks_workspace_bytes(n))


def rkv_release_blocks(length, held, block_table, free_blocks, free_count, block: int, held_out,
                       free_count_out, ws=None, stream=None):
    """Blocks that length[u] tokens do not need go back to the free stack; see include/rkv.h."""
    n, max_blocks = _dims(block_table, "block_table", 2)
    num_blocks = _dims(free_blocks, "free_blocks", 1)[0]
    dev = block_table.get_device()
    args = (_at(length, "len", _I32, (n,), dev), _at(held, "held", _I32, (n,), dev),
            _at(block_table, "block_table", _I32, (n, max_blocks), dev),
            _at(free_blocks, "free_blocks", _I32, (num_blocks,), dev),
            _at(free_count, "free_count", _I32, (1,), dev), n, num_blocks, block, max_blocks,
            _at(held_out, "held_out", _I32, (n,), dev),
            _at(free_count_out, "free_count_out", _I32, (1,), dev))
    return _call("rkv_release_blocks", args, ws, lambda: rkv_release_blocks_workspace_bytes(n), dev,
                 stream)


ROPE_KINDS = {"plain": 0, "linear": 1, "base": 2, "by_parts": 3, "smooth": 4, "by_whole_parts": 5}


def rkv_rope_frequencies(rot_dim: int = HEAD_DIM, base: float = 10000.0, kind: str = "plain",
                         factor: float = 1.0, ctx: int = 0, fast: float = 32.0, slow: float = 1.0):
    """(inv_freq fp32 [rot_dim / 2] on the host, mscale) of the rotary positions; see include/rkv.h."""
    if kind not in ROPE_KINDS:
        raise ValueError(f"kind must be one of {sorted(ROPE_KINDS)}")
    freq = torch.empty(max(int(rot_dim), 2) // 2, dtype=torch.float32)
    mscale = ctypes.c_float(0.0)
    _check("rkv_rope_frequencies", load().rkv_rope_frequencies(
        ROPE_KINDS[kind], rot_dim, base, factor, ctx, fast, slow, freq.data_ptr(),
        ctypes.byref(mscale)))
    return freq, mscale.value


def rkv_rope_append_workspace_bytes() -> int:
    return int(load().rkv_rope_append_workspace_bytes())


def rkv_rope_append(q, k, v, positions, inv_freq, slots, q_out, k_cache, v_cache,
                    interleaved: bool = False, mscale: float = 1.0, ws=None, stream=None):
    """Turns packed q [tokens][Hq][128] (into q_out) and k [tokens][n_kv][128] to their positions and
    stores k and v in row slots[t] of the caches ([num_blocks][n_kv][block][128], or
    [n][n_kv][cap][128] with slots u * cap + row); see include/rkv.h."""
    tokens, hq, _ = _dims(q, "q", 3)
    dev = q.get_device()
    shape, k_rows = _first(k_cache, "k_cache", _BF16, 4, dev)
    num_blocks, n_kv, block, d = shape
    (pairs,), freq = _first(inv_freq, "inv_freq", _F32, 1, dev)
    each = (tokens,)
    args = (*_tokens(q, "q", hq, dev, tokens), *_tokens(k, "k", n_kv, dev, tokens),
            *_tokens(v, "v", n_kv, dev, tokens), _at(positions, "positions", _I32, each, dev), freq,
            _at(slots, "slots", _I32, each, dev), tokens, hq, n_kv, d, 2 * pairs, int(interleaved),
            mscale, _at(q_out, "q_out", _BF16, (tokens, hq, HEAD_DIM), dev), k_rows,
            _at(v_cache, "v_cache", _BF16, shape, dev), num_blocks, block)
    return _call("rkv_rope_append", args, ws, rkv_rope_append_workspace_bytes, dev, stream)


def rkv_prompt_attention_workspace_bytes(n: int, n_kv: int, gqa: int, tokens: int) -> int:
    return int(load().rkv_prompt_attention_workspace_bytes(n, n_kv, gqa, tokens))


def _attention(fn, q, q_start, mask, k, v, table, length, scale, out, ws, stream, hook=()):
    tokens, hq, _ = _dims(q, "q", 3)
    dev = q.get_device()
    shape, k_rows = _first(k, "k", _BF16, 4, dev)
    lead, n_kv, rows, d = shape
    (n,), lens = _first(length, "len", _I32, 1, dev)
    gqa = _group(hq, n_kv)
    tree = ()
    if mask is not None:
        (lines, words), bits = _first(mask, "mask", _I32, 2, dev)
        if lines != tokens:
            raise ValueError(f"mask has {lines} rows, expected {tokens}")
        tree = (bits, words)
    if table is None:
        if lead != n:
            raise ValueError(f"{n} lengths for a cache of {lead} units")
        paged, sizes = (), (tokens, rows)
    else:
        (lines, max_blocks), blocks = _first(table, "block_table", _I32, 2, dev)
        if lines != n:
            raise ValueError(f"block_table has {lines} rows, expected {n}")
        paged, sizes = (blocks,), (tokens, lead, rows, max_blocks)
    args = (*_tokens(q, "q", hq, dev, tokens), _at(q_start, "q_start", _I32, (n + 1,), dev), *tree,
            k_rows, _at(v, "v", _BF16, shape, dev), *paged, lens, n, n_kv, gqa, d, *sizes, scale,
            _at(out, "out", _BF16, (tokens, hq, HEAD_DIM), dev), *hook)
    return _call(fn, args, ws, lambda: rkv_prompt_attention_workspace_bytes(n, n_kv, gqa, tokens),
                 dev, stream)


def rkv_prompt_attention(q, q_start, k, v, length, scale: float, out, ws=None, stream=None):
    """Causal attention of packed new tokens (q, out [tokens][Hq][128]; unit u's are
    q_start[u] .. q_start[u + 1] - 1) over the unit's length[u] cached rows, theirs included and
    last; see include/rkv.h."""
    return _attention("rkv_prompt_attention", q, q_start, None, k, v, None, length, scale, out, ws,
                      stream)


def rkv_prompt_attention_paged(q, q_start, k_pool, v_pool, block_table, length, scale: float, out,
                               ws=None, stream=None):
    """rkv_prompt_attention over pools [num_blocks][n_kv][block][128] through block_table."""
    _dims(block_table, "block_table", 2)
    return _attention("rkv_prompt_attention_paged", q, q_start, None, k_pool, v_pool, block_table,
                      length, scale, out, ws, stream)


def rkv_tree_attention(q, q_start, mask, k, v, length, scale: float, out, ws=None, stream=None):
    """Attention of a tree of drafted tokens: each sees the rows before the drafted ones, and of
    those the ones that its bits in mask [tokens][words] int32 name; see include/rkv.h."""
    _dims(mask, "mask", 2)
    return _attention("rkv_tree_attention", q, q_start, mask, k, v, None, length, scale, out, ws,
                      stream)


def rkv_tree_attention_paged(q, q_start, mask, k_pool, v_pool, block_table, length, scale: float,
                             out, ws=None, stream=None):
    """rkv_tree_attention over pools [num_blocks][n_kv][block][128] through block_table."""
    _dims(mask, "mask", 2), _dims(block_table, "block_table", 2)
    return _attention("rkv_tree_attention_paged", q, q_start, mask, k_pool, v_pool, block_table,
                      length, scale, out, ws, stream)


def rkv_testing_attention_wait_timeout(q, q_start, k, v, length, scale: float, out, what: int,
                                       wait_limit_ns: int, ws=None, stream=None):
    """Test hook (include/rkv_testing.h): rkv_prompt_attention with one load of block 0 never
    requested, so that its bounded waits run out after wait_limit_ns."""
    return _attention("rkv_testing_attention_wait_timeout", q, q_start, None, k, v, None, length,
                      scale, out, ws, stream, (int(what), int(wait_limit_ns)))
