"""Python binding of libzp, the Compressed PagedAttention hot path for GB300.

Argument marshalling only: every function forwards torch tensors' device
pointers and sizes to the C ABI declared in ``include/zp.h`` and raises
``ZPError`` on a non-OK status.  All arithmetic runs in the CUDA kernels of
libzp.so; there is no CPU fallback.  The library must have been built (see
``compressed_paged_kv_zp_gb300/_build.py`` or ``__graft_entry__.build()``):
importing this package without it raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libzp.so")

ZP_BF16 = 0
ZP_F32 = 1
_DTYPES = {torch.bfloat16: ZP_BF16, torch.float32: ZP_F32}
_TORCH = {code: t for t, code in _DTYPES.items()}

STATUS = {0: "ZP_OK", 1: "ZP_ERR_INVALID_ARG", 2: "ZP_ERR_SHAPE", 3: "ZP_ERR_DTYPE",
          4: "ZP_ERR_CAPACITY", 5: "ZP_ERR_CUDA", 6: "ZP_ERR_TIMEOUT", 7: "ZP_ERR_DEVICE"}

# every symbol include/*.h declares
EXPORTS = [
    "zp_last_error", "zp_status_string", "zp_version", "zp_device_status",
    "zp_decode_workspace_size", "zp_paged_decode_attn", "zp_paged_decode_attn_rho", "zp_paged_decode_attn_noalloc",
    "zp_debug_noalloc_preset_ctl", "zp_append_kv", "zp_needs_compression",
    "zp_needs_compression_batch",
    "zp_build_slots", "zp_write_kv", "zp_prefix_plan", "zp_prefix_decode_workspace_size", "zp_prefix_decode_attn",
    "zp_window_score_workspace_size", "zp_window_score",
    "zp_score_workspace_size", "zp_score_tokens", "zp_select_topk", "zp_compact_pages",
    "zp_compress_workspace_size", "zp_compress_layers", "zp_compress_layers_rho", "zp_compress_rho_supported",
    "zp_pool_create", "zp_pool_destroy", "zp_pool_num_free", "zp_pool_refcount", "zp_pool_alloc",
    "zp_pool_incref", "zp_pool_release", "zp_plan_compaction", "zp_plan_compaction_batch",
    "zp_plan_capacity",
    "zp_q4_tile_bytes", "zp_q4_write_kv", "zp_q4_append_kv", "zp_q4_read_kv", "zp_q4_decode_workspace_size",
    "zp_q4_decode_attn", "zp_q4_compact_pages",
    # include/zp_sched.h
    "zp_sched_create", "zp_sched_destroy", "zp_sched_add_request", "zp_sched_schedule", "zp_sched_commit",
    "zp_sched_take_compressions", "zp_sched_compression_done", "zp_sched_counts", "zp_sched_request_info",
]


class ZPError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__("%s: %s" % (STATUS.get(status, status), msg))
        self.status = status


class CacheDesc(ctypes.Structure):
    _fields_ = [("h_q", ctypes.c_int32), ("h_kv", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("block_size", ctypes.c_int32), ("n_total_blocks", ctypes.c_int32),
                ("dtype", ctypes.c_int32)]


class ScoreParams(ctypes.Structure):
    _fields_ = [("window", ctypes.c_int32), ("use_global", ctypes.c_int32), ("alpha", ctypes.c_float),
                ("pool_kernel", ctypes.c_int32), ("pool_policy", ctypes.c_int32),
                ("use_similarity", ctypes.c_int32), ("lightning", ctypes.c_int32),
                ("threshold", ctypes.c_float), ("lambda_", ctypes.c_float), ("tau", ctypes.c_float)]


class ScoreRows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("stride", ctypes.c_int64), ("layer_stride", ctypes.c_int64),
                ("rows", ctypes.c_void_p)]


class RhoRows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("stride", ctypes.c_int64), ("layer_stride", ctypes.c_int64),
                ("rows", ctypes.c_void_p), ("n_rows", ctypes.c_int32), ("threshold", ctypes.c_float)]


class _PrefixGroups(ctypes.Structure):
    _fields_ = [("prefix_lens", ctypes.c_void_p), ("n_groups", ctypes.c_void_p), ("group_start", ctypes.c_void_p),
                ("members", ctypes.c_void_p), ("group_blocks", ctypes.c_void_p)]


def _rho_rows(rho, rows, threshold=0.0):
    """rho: float32 [R][h_kv][stride] or [layers][R][h_kv][stride]; rows: int32 device or None."""
    if rho.dtype != torch.float32 or rho.dim() not in (3, 4):
        raise ValueError("redundancy rows must be float32 [R][h_kv][stride] or [layers][R][h_kv][stride]")
    if rows is not None and rows.dtype != torch.int32:
        raise ValueError("rho_rows must be int32")
    layer_stride = rho.stride(0) if rho.dim() == 4 else 0
    return ctypes.byref(RhoRows(_dev(rho, "rho").value, int(rho.shape[-1]), int(layer_stride),
                                _dev(rows, "rho_rows").value if rows is not None else None,
                                int(rho.shape[-3]), float(threshold)))


def _score_rows(attn, rows):
    """attn: float32 [R][h_kv][stride] or [layers][R][h_kv][stride]; rows: int32 [n] or None."""
    if attn is None:
        return None
    if attn.dtype != torch.float32 or attn.dim() not in (3, 4):
        raise ValueError("score rows must be float32 [R][h_kv][stride] or [layers][R][h_kv][stride]")
    if rows is not None and rows.dtype != torch.int32:
        raise ValueError("rows must be int32")
    layer_stride = attn.stride(0) if attn.dim() == 4 else 0
    return ctypes.byref(ScoreRows(_dev(attn, "attn").value, int(attn.shape[-1]), int(layer_stride),
                                  _dev(rows, "rows").value if rows is not None else None))


def score_params(window=16, use_global=True, alpha=0.8, pool_kernel=7, pool_policy=1,
                 use_similarity=True, lightning=True, threshold=0.9, lam=0.2, tau=0.4) -> ScoreParams:
    return ScoreParams(int(window), int(bool(use_global)), float(alpha), int(pool_kernel),
                       int(pool_policy), int(bool(use_similarity)), int(bool(lightning)),
                       float(threshold), float(lam), float(tau))


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError("libzp.so is not built (expected at %s); run "
                          "compressed_paged_kv_zp_gb300._build.build()" % LIB_PATH)
    lib = ctypes.CDLL(LIB_PATH)
    P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    D = ctypes.POINTER(CacheDesc)
    lib.zp_last_error.restype = ctypes.c_char_p
    lib.zp_status_string.restype = ctypes.c_char_p
    lib.zp_status_string.argtypes = [ctypes.c_int]
    lib.zp_device_status.argtypes = [P, P, I32]
    lib.zp_decode_workspace_size.restype = SZ
    lib.zp_decode_workspace_size.argtypes = [D, I32, I32]
    lib.zp_paged_decode_attn.argtypes = [D, P, P, P, P, I32, P, I32, P, P, P, I32, I32, P, SZ, P]
    lib.zp_paged_decode_attn_rho.argtypes = [D, P, P, P, P, I32, P, I32, P, P, P, I32, I32, P, P, SZ, P]
    lib.zp_paged_decode_attn_noalloc.argtypes = [D, P, P, P, P, I32, P, I32, P, P, P, I32, I32, P]
    lib.zp_debug_noalloc_preset_ctl.argtypes = [I32, ctypes.c_uint64]
    lib.zp_append_kv.argtypes = [D, P, P, P, P, P, I32, P, I32, P]
    G = ctypes.POINTER(_PrefixGroups)
    lib.zp_build_slots.argtypes = [D, P, P, I32, P, P, I32, P, I32, P, P, I32, P, P, P]
    lib.zp_write_kv.argtypes = [D, P, P, I64, I64, P, I32, P, P, I64, I32, P]
    lib.zp_prefix_plan.argtypes = [D, P, I32, P, I32, I32, I32, G, P]
    lib.zp_prefix_decode_workspace_size.restype = SZ
    lib.zp_prefix_decode_workspace_size.argtypes = [D, I32, I32]
    lib.zp_prefix_decode_attn.argtypes = [D, P, P, P, P, I32, P, I32, G, P, P, P, I32, I32, P, SZ, P]
    lib.zp_needs_compression.argtypes = [I32, I32, I32]
    lib.zp_needs_compression_batch.argtypes = [P, P, I32, I32, I32, P, P, P]
    lib.zp_score_workspace_size.restype = SZ
    lib.zp_score_workspace_size.argtypes = [D, I32, I32]
    lib.zp_window_score_workspace_size.restype = SZ
    lib.zp_window_score_workspace_size.argtypes = [D, I32, I32, I32]
    lib.zp_window_score.argtypes = [D, P, I32, P, P, I32, P, I32, P, I32, P, SZ, P]
    lib.zp_score_tokens.argtypes = [D, ctypes.POINTER(ScoreParams), P, P, I32, P, P, I32, P, P, P,
                                    I32, P, SZ, P]
    lib.zp_select_topk.argtypes = [P, I32, I32, P, I32, I32, P, P, P, P]
    lib.zp_compact_pages.argtypes = [D, P, P, I64, I32, P, I64, P, P, I32, P, I32, P, P, I32, P, I32, P]
    lib.zp_compress_workspace_size.restype = SZ
    lib.zp_compress_workspace_size.argtypes = [D, I32, I32, I32]
    lib.zp_compress_layers.argtypes = [D, ctypes.POINTER(ScoreParams), P, P, I64, I32, P, I32, P, P, I32, P, P,
                                       I64, P, I32, I32, P, P, P, P, I32, P, SZ, P]
    lib.zp_compress_rho_supported.restype = I32
    lib.zp_compress_rho_supported.argtypes = [D, ctypes.POINTER(ScoreParams), I32, I32]
    lib.zp_compress_layers_rho.argtypes = [D, ctypes.POINTER(ScoreParams), P, P, I64, I32, P, I32, P, P, I32, P,
                                           P, I64, P, I32, I32, P, P, P, P, I32, P, P]
    lib.zp_q4_tile_bytes.restype = SZ
    lib.zp_q4_tile_bytes.argtypes = [D, I32]
    lib.zp_q4_write_kv.argtypes = [D, I32, P, P, I64, I64, P, I32, P, P, I64, I32, P]
    lib.zp_q4_append_kv.argtypes = [D, I32, P, P, P, P, P, I32, P, I32, P]
    lib.zp_q4_read_kv.argtypes = [D, I32, P, P, I64, P, I32, P, P, I64, I64, I32, P]
    lib.zp_q4_decode_workspace_size.restype = SZ
    lib.zp_q4_decode_workspace_size.argtypes = [D, I32, I32, I32, I32]
    lib.zp_q4_decode_attn.argtypes = [D, I32, P, P, P, P, I32, P, I32, P, P, P, I32, I32, P, SZ, P]
    lib.zp_q4_compact_pages.argtypes = [D, I32, P, P, I64, I32, P, I64, P, P, I32, P, I32, P, P, I32, P, I32, P]
    lib.zp_pool_create.restype = P
    lib.zp_pool_create.argtypes = [I32]
    lib.zp_pool_destroy.argtypes = [P]
    lib.zp_pool_num_free.argtypes = [P]
    lib.zp_pool_refcount.argtypes = [P, I32]
    lib.zp_pool_alloc.argtypes = [P, I32, P]
    lib.zp_pool_incref.argtypes = [P, I32, P]
    lib.zp_pool_release.argtypes = [P, I32, P]
    lib.zp_plan_compaction.argtypes = [P, P, I32, I32, P, P, P, P, P]
    lib.zp_plan_compaction_batch.argtypes = [P, P, I32, P, I32, I32, P, P, P, P, P, P]
    lib.zp_plan_capacity.argtypes = [I64, I64, I64, I32, I64, I64, P, P]
    return lib


lib = _load()


def _check(status: int) -> None:
    if status != 0:
        raise ZPError(status, lib.zp_last_error().decode())


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to libzp must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _dev(t: Optional[torch.Tensor], name: str):
    if t is not None and not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    return _ptr(t)


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def cache_desc(h_q, h_kv, head_dim, block_size, n_total_blocks, dtype) -> CacheDesc:
    code = _DTYPES[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    return CacheDesc(int(h_q), int(h_kv), int(head_dim), int(block_size), int(n_total_blocks), code)


# ----------------------------------------------------------------------------- decode
def zp_decode_workspace_size(desc: CacheDesc, B: int, table_stride: int) -> int:
    n = lib.zp_decode_workspace_size(ctypes.byref(desc), int(B), int(table_stride))
    if n == 0 and B > 0:
        raise ZPError(2, lib.zp_last_error().decode() or "unsupported decode shape")
    return int(n)


def _slot_map(score_accum, score_rows):
    """(pointer, row count) of an optional int32 [B] slot map into score_accum [R][h_kv][stride]."""
    if score_rows is None:
        return None, 0
    if score_rows.dtype != torch.int32:
        raise ValueError("score_rows must be int32")
    if score_accum is None:
        raise ValueError("score_rows needs score_accum")
    return _dev(score_rows, "score_rows"), int(score_accum.shape[0])


def zp_paged_decode_attn(desc, q, k_cache, v_cache, block_table, seq_lens, out, score_accum=None,
                         window=0, workspace=None, stream=None, score_rows=None, rho=None, rho_rows=None,
                         rho_threshold=0.9) -> None:
    """score_rows: optional int32 [B] device map of batch entries to rows of
    score_accum (query slots); -1 = no slot, the entry is not scored.
    rho (optional float32 [R][h_kv][stride]) with rho_rows (int32 [B] device,
    -1 = none): the lightning redundancy row sums of the entries that have a
    row, at threshold rho_threshold (zp_paged_decode_attn_rho)."""
    B, table_stride = int(block_table.shape[0]), int(block_table.shape[1])
    rows_p, n_rows = _slot_map(score_accum, score_rows)
    if workspace is None:
        workspace = torch.empty(zp_decode_workspace_size(desc, B, table_stride), dtype=torch.uint8,
                                device=q.device)
    args = (ctypes.byref(desc), _dev(q, "q"), _dev(k_cache, "k_cache"), _dev(v_cache, "v_cache"),
            _dev(block_table, "block_table"), table_stride, _dev(seq_lens, "seq_lens"), B, _dev(out, "out"),
            _dev(score_accum, "score_accum"), rows_p, n_rows, int(window))
    tail = (_dev(workspace, "workspace"), workspace.numel(), _stream(stream))
    if rho is None:
        _check(lib.zp_paged_decode_attn(*args, *tail))
    else:
        if rho_rows is None or rho_rows.numel() != B:
            raise ValueError("rho needs rho_rows: one int32 entry per batch entry")
        _check(lib.zp_paged_decode_attn_rho(*args, _rho_rows(rho, rho_rows, rho_threshold), *tail))


def zp_paged_decode_attn_noalloc(desc, q, k_cache, v_cache, block_table, seq_lens, out,
                                 score_accum=None, window=0, stream=None, score_rows=None) -> None:
    """zp_paged_decode_attn with the library's built-in scratch (no workspace)."""
    B, table_stride = int(block_table.shape[0]), int(block_table.shape[1])
    rows_p, n_rows = _slot_map(score_accum, score_rows)
    _check(lib.zp_paged_decode_attn_noalloc(ctypes.byref(desc), _dev(q, "q"), _dev(k_cache, "k_cache"),
                                            _dev(v_cache, "v_cache"), _dev(block_table, "block_table"),
                                            table_stride, _dev(seq_lens, "seq_lens"), B, _dev(out, "out"),
                                            _dev(score_accum, "score_accum"), rows_p, n_rows, int(window),
                                            _stream(stream)))


def zp_append_kv(desc, k_new, v_new, k_cache, v_cache, block_table, seq_lens, stream=None) -> None:
    B, table_stride = int(block_table.shape[0]), int(block_table.shape[1])
    _check(lib.zp_append_kv(ctypes.byref(desc), _dev(k_new, "k_new"), _dev(v_new, "v_new"),
                            _dev(k_cache, "k_cache"), _dev(v_cache, "v_cache"),
                            _dev(block_table, "block_table"), table_stride, _dev(seq_lens, "seq_lens"),
                            B, _stream(stream)))


# ----------------------------------------------------------------------------- shared prompts
# These calls run before or inside every decode step, so their checks are kept to
# a few attribute reads per tensor: pointers go to ctypes as ints.
def _ptr_on(t, dev: int, name: str):
    """Address of a contiguous tensor on CUDA device `dev`, the current one (None stays None)."""
    if t is None:
        return None
    if t.get_device() != dev:
        raise ValueError("%s must be a CUDA tensor on the current device, is on %s" % (name, t.device))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


def _ints(t, dev: int, name: str, numel=None):
    """_ptr_on of an int32 tensor, of `numel` elements where given."""
    if t is None:
        return None
    if t.dtype is not torch.int32:
        raise ValueError("%s must be int32" % name)
    if numel is not None and t.numel() != numel:
        raise ValueError("%s must have %d elements, has %d" % (name, numel, t.numel()))
    return _ptr_on(t, dev, name)


def _device() -> int:
    return torch.cuda.current_device() if torch.cuda.is_initialized() or torch.cuda.is_available() else -2


def _raw_stream(stream, dev: int) -> int:
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _table(block_table):
    if block_table.dim() != 2:
        raise ValueError("block_table must be [B][table_stride]")
    return block_table.shape


def _check_cache(desc, k_cache, v_cache, layers=1) -> None:
    n = layers * desc.n_total_blocks * desc.block_size * desc.h_kv * desc.head_dim
    if k_cache.numel() != n or v_cache.numel() != n:
        raise ValueError("k_cache and v_cache must be [N_total][b][h_kv][d] (or one of these per layer), are %s and %s"
                         % (tuple(k_cache.shape), tuple(v_cache.shape)))


def zp_build_slots(desc, block_table, old_lens, new_lens, slots, cu_tokens, fresh=None, table_out=None, positions=None,
                   n_used=None, stream=None) -> None:
    """Grow the block table from old_lens to new_lens with the blocks of `fresh`
    (int32, in the order they go out) and write the slot map of the new tokens:
    slots and positions int32 [max_tokens] (padded with -1), cu_tokens [B+1],
    n_used [1].  table_out: a separate table for the result (None: in place)."""
    B, table_stride = _table(block_table)
    dev, room = _device(), slots.numel()
    table = _ints(block_table, dev, "block_table")
    if table_out is not None and table_out.shape != block_table.shape:
        raise ValueError("table_out must have block_table's shape")
    rc = lib.zp_build_slots(desc, table, table if table_out is None else _ints(table_out, dev, "table_out"),
                            table_stride, _ints(old_lens, dev, "old_lens", B), _ints(new_lens, dev, "new_lens", B), B,
                            _ints(fresh, dev, "fresh"), 0 if fresh is None else fresh.numel(),
                            _ints(slots, dev, "slots"), _ints(positions, dev, "positions", room), room,
                            _ints(cu_tokens, dev, "cu_tokens", B + 1), _ints(n_used, dev, "n_used", 1),
                            _raw_stream(stream, dev))
    if rc:
        _check(rc)


def zp_write_kv(desc, k_new, v_new, slots, k_cache, v_cache, stream=None) -> None:
    """Store the rows of n tokens into their slots (int32 [n]; negative: skipped).
    k_new, v_new: [n][h_kv][d] for one layer, or [layers][n][h_kv][d] with caches
    [layers][N_total][b][h_kv][d].  The rows [h_kv][d] are contiguous; the token
    and layer strides are free (a slice of a fused projection)."""
    n, h_kv, d = slots.numel(), desc.h_kv, desc.head_dim
    several = k_cache.dim() == 5
    layers = k_cache.shape[0] if several else 1
    shape = (layers, n, h_kv, d) if several else (n, h_kv, d)
    dev, dt = _device(), _TORCH.get(desc.dtype)
    if k_new.shape != shape or v_new.shape != shape:
        raise ValueError("k_new and v_new must be %s, are %s and %s" % (shape, tuple(k_new.shape), tuple(v_new.shape)))
    if not (k_new.dtype is v_new.dtype is k_cache.dtype is v_cache.dtype is dt):
        raise ValueError("k_new, v_new, k_cache and v_cache must have the cache's type")
    if k_new.get_device() != dev or v_new.get_device() != dev:
        raise ValueError("k_new and v_new must be CUDA tensors on the current device")
    # (layer, token, head, element); a stride along a dimension of one entry means nothing
    row = h_kv * d
    strides = [(x.stride(0) if layers > 1 else 0, x.stride(-3) if n > 1 else row, x.stride(-2) if h_kv > 1 else d, x.stride(-1))
               for x in (k_new, v_new)]
    if n and (strides[0][2:] != (d, 1) or strides[1] != strides[0]):
        raise ValueError("the row [h_kv][d] of a token must be contiguous, and k_new and v_new must have the same strides")
    _check_cache(desc, k_cache, v_cache, layers)
    if n == 0:
        return
    rc = lib.zp_write_kv(desc, k_new.data_ptr(), v_new.data_ptr(), strides[0][1], strides[0][0], _ints(slots, dev, "slots"), n,
                         _ptr_on(k_cache, dev, "k_cache"),
                         _ptr_on(v_cache, dev, "v_cache"), k_cache.stride(0) if layers > 1 else 0, layers,
                         _raw_stream(stream, dev))
    if rc:
        _check(rc)


class PrefixPlan:
    """Groups of batch entries that share leading blocks: int32 CUDA tensors
    prefix_lens [B], n_groups [1], group_start [B+1], members [B], group_blocks
    [B] (see zp_prefix_groups in zp.h).  zp_prefix_plan fills them from the block
    table; a scheduler that knows its groups may fill them itself, in place: the
    library is given their addresses when the plan is made."""

    def __init__(self, prefix_lens, n_groups, group_start, members, group_blocks):
        B, dev = prefix_lens.numel(), _device()
        c = _PrefixGroups(_ints(prefix_lens, dev, "prefix_lens", B), _ints(n_groups, dev, "n_groups", 1),
                          _ints(group_start, dev, "group_start", B + 1), _ints(members, dev, "members", B),
                          _ints(group_blocks, dev, "group_blocks", B))
        self.__dict__.update(B=B, prefix_lens=prefix_lens, n_groups=n_groups, group_start=group_start, members=members,
                             group_blocks=group_blocks, _dev=dev, _c=c)

    def __setattr__(self, name, value):
        raise AttributeError("a plan's arrays are filled in place, not replaced (%s)" % name)


def _groups_for(plan: PrefixPlan, B: int, dev: int):
    """The plan's arrays for a call on device `dev` with B batch entries."""
    if plan.B != B:
        raise ValueError("the plan is for %d batch entries, the table has %d" % (plan.B, B))
    if plan._dev != dev:
        raise ValueError("the plan is on CUDA device %d, the current one is %d" % (plan._dev, dev))
    return plan._c


def prefix_plan(B: int, device="cuda") -> PrefixPlan:
    """An empty plan (no groups) for B batch entries."""
    buf = torch.zeros(4 * B + 2, dtype=torch.int32, device=device)
    buf[2 * B + 2:3 * B + 2] = -1
    return PrefixPlan(buf[:B], buf[B:B + 1], buf[B + 1:2 * B + 2], buf[2 * B + 2:3 * B + 2], buf[3 * B + 2:])


def zp_prefix_plan(desc, block_table, seq_lens, plan: PrefixPlan, min_blocks=1, min_members=2, stream=None) -> None:
    """Find the groups that share at least min_blocks leading blocks among at least min_members entries."""
    B, table_stride = _table(block_table)
    dev = _device()
    groups = _groups_for(plan, B, dev)
    rc = lib.zp_prefix_plan(desc, _ints(block_table, dev, "block_table"), table_stride, _ints(seq_lens, dev, "seq_lens", B),
                            B, min_blocks, min_members, groups, _raw_stream(stream, dev))
    if rc:
        _check(rc)


def zp_prefix_decode_workspace_size(desc: CacheDesc, B: int, table_stride: int) -> int:
    n = lib.zp_prefix_decode_workspace_size(desc, B, table_stride)
    if n == 0 and B > 0:
        raise ZPError(2, lib.zp_last_error().decode() or "unsupported decode shape")
    return n


def zp_prefix_decode_attn(desc, q, k_cache, v_cache, block_table, seq_lens, plan: PrefixPlan, out, score_accum=None,
                          window=0, workspace=None, stream=None, score_rows=None) -> None:
    """zp_paged_decode_attn with every group's shared prefix computed once for all its members."""
    B, table_stride = _table(block_table)
    dev = _device()
    groups = _groups_for(plan, B, dev)
    shape, dt = (B, desc.h_q, desc.head_dim), _TORCH.get(desc.dtype)
    if q.shape != shape or out.shape != shape:
        raise ValueError("q and out must be [B][h_q][d] = %s, are %s and %s" % (shape, tuple(q.shape), tuple(out.shape)))
    if not (q.dtype is out.dtype is k_cache.dtype is v_cache.dtype is dt):
        raise ValueError("q, out, k_cache and v_cache must have the cache's type")
    _check_cache(desc, k_cache, v_cache)
    n_rows = 0
    if score_accum is not None:
        n_rows = score_accum.shape[0]
        if (score_accum.dtype is not torch.float32 or score_accum.dim() != 3 or (score_rows is None and n_rows < B) or
                score_accum.shape[1:] != (desc.h_kv, table_stride * desc.block_size)):
            raise ValueError("score_accum must be float32 [R][h_kv][table_stride*b] with a row per batch entry or a slot map")
    elif score_rows is not None:
        raise ValueError("score_rows needs score_accum")
    args = (desc, _ptr_on(q, dev, "q"), _ptr_on(k_cache, dev, "k_cache"), _ptr_on(v_cache, dev, "v_cache"),
            _ints(block_table, dev, "block_table"), table_stride, _ints(seq_lens, dev, "seq_lens", B), B, groups,
            _ptr_on(out, dev, "out"), _ptr_on(score_accum, dev, "score_accum"), _ints(score_rows, dev, "score_rows", B),
            n_rows, window)
    on = _raw_stream(stream, dev)
    if workspace is None:
        # memory of the stream that the work runs on, given back behind it: torch's
        # allocator hands it to later work of that stream only
        n = max(zp_prefix_decode_workspace_size(desc, B, table_stride), 16)
        at = torch.cuda.caching_allocator_alloc(n, dev, on)
        try:
            rc = lib.zp_prefix_decode_attn(*args, at, n, on)
        finally:
            torch.cuda.caching_allocator_delete(at)
    else:
        rc = lib.zp_prefix_decode_attn(*args, _ptr_on(workspace, dev, "workspace"), workspace.nbytes, on)
    if rc:
        _check(rc)


# ----------------------------------------------------------------------------- 4-bit cache
def zp_q4_tile_bytes(desc: CacheDesc, group: int = 32) -> int:
    """Bytes of a tile (16 tokens of one kv head) of a 4-bit cache."""
    n = lib.zp_q4_tile_bytes(desc, group)
    if n == 0:
        raise ZPError(2, lib.zp_last_error().decode())
    return n


def zp_q4_cache(desc: CacheDesc, group: int = 32, layers=None, device="cuda"):
    """An empty 4-bit cache (all values 0): k_cache, v_cache uint8 [N_total][h_kv][b/16][tile], with a
    leading dimension of `layers` where given."""
    shape = (desc.n_total_blocks, desc.h_kv, desc.block_size // 16, zp_q4_tile_bytes(desc, group))
    if layers is not None:
        shape = (layers,) + shape
    return torch.zeros(shape, dtype=torch.uint8, device=device), torch.zeros(shape, dtype=torch.uint8, device=device)


def _q4_shape(desc, group):
    """Shape of one layer of a 4-bit cache.  (The library refuses the groups and head sizes it does not know.)"""
    d = desc.head_dim
    return desc.n_total_blocks, desc.h_kv, desc.block_size >> 4, (d << 3) + 64 * (d // group if group > 0 else 0)


def _q4_check(k_cache, v_cache, shape):
    """Refuses cache tensors of other types or shapes."""
    if not (k_cache.dtype is v_cache.dtype is torch.uint8 and k_cache.shape == shape and v_cache.shape == shape):
        raise ValueError("k_cache and v_cache must be uint8 [N_total][h_kv][b/16][tile] = %s, are %s %s and %s %s"
                         % (shape, k_cache.dtype, tuple(k_cache.shape), v_cache.dtype, tuple(v_cache.shape)))


def _q4_here(dev: int, tensors, names) -> None:
    """Refuses tensors that are not contiguous on CUDA device `dev`, the current one.  (One loop for all:
    a call's checks are a good part of its time where the batch is small.)"""
    for t in tensors:
        if t.get_device() != dev or not t.is_contiguous():
            for t, name in zip(tensors, names):
                _ptr_on(t, dev, name)


def _q4_ints(block_table, seq_lens, B) -> None:
    if not (block_table.dtype is seq_lens.dtype is torch.int32 and seq_lens.numel() == B):
        raise ValueError("block_table and seq_lens must be int32, with an entry of seq_lens per row of block_table")


def _q4_caches(desc, group, k_cache, v_cache, dev):
    """(address, address, layers, bytes between layers) of a 4-bit cache of one layer (layers: None) or, with a
    fifth dimension, of several."""
    shape = _q4_shape(desc, group)
    layers = None
    if k_cache.dim() == 5:
        layers = k_cache.shape[0]
        shape = (layers,) + shape
    _q4_check(k_cache, v_cache, shape)
    _q4_here(dev, (k_cache, v_cache), ("k_cache", "v_cache"))
    return k_cache.data_ptr(), v_cache.data_ptr(), layers, 0 if layers is None else k_cache.stride(0)


def _q4_rows(desc, k, v, n, layers, dev, names):
    """(address, address, token stride, layer stride) of rows [n][h_kv][d] or [layers][n][h_kv][d]."""
    h_kv, d = desc.h_kv, desc.head_dim
    shape = (n, h_kv, d) if layers is None else (layers, n, h_kv, d)
    if k.shape != shape or v.shape != shape:
        raise ValueError("%s and %s must be %s, are %s and %s" % (*names, shape, tuple(k.shape), tuple(v.shape)))
    if not (k.dtype is v.dtype is _TORCH.get(desc.dtype)):
        raise ValueError("%s and %s must have the descriptor's type" % names)
    if k.get_device() != dev or v.get_device() != dev:
        raise ValueError("%s and %s must be CUDA tensors on the current device" % names)
    # (layer, token, head, element); a stride along a dimension of one entry means nothing
    row = h_kv * d
    ks, vs = k.stride(), v.stride()
    if n and (ks[-1] != 1 or vs[-1] != 1 or (h_kv > 1 and (ks[-2] != d or vs[-2] != d)) or (n > 1 and ks[-3] != vs[-3]) or
              (layers is not None and layers > 1 and ks[0] != vs[0])):
        raise ValueError("the row [h_kv][d] of a token must be contiguous, and %s and %s must have the same strides" % names)
    return k.data_ptr(), v.data_ptr(), ks[-3] if n > 1 else row, ks[0] if layers is not None and layers > 1 else 0


def zp_q4_write_kv(desc, k_new, v_new, slots, k_cache, v_cache, group=32, stream=None) -> None:
    """zp_write_kv into a 4-bit cache: rows [n][h_kv][d] (or [layers][n][h_kv][d]) quantised into their
    slots (int32 [n]; negative: skipped)."""
    dev, n = _device(), slots.numel()
    K, V, layers, layer_bytes = _q4_caches(desc, group, k_cache, v_cache, dev)
    k, v, token, layer = _q4_rows(desc, k_new, v_new, n, layers, dev, ("k_new", "v_new"))
    rc = lib.zp_q4_write_kv(desc, group, k, v, token, layer, _ints(slots, dev, "slots"), n, K, V, layer_bytes,
                            1 if layers is None else layers, _raw_stream(stream, dev))
    if rc:
        _check(rc)


_Q4_APPEND = ("k_new", "v_new", "k_cache", "v_cache", "block_table", "seq_lens")


def zp_q4_append_kv(desc, k_new, v_new, k_cache, v_cache, block_table, seq_lens, group=32, stream=None) -> None:
    """zp_append_kv into a 4-bit cache: k_new, v_new [B][h_kv][d], one token per sequence."""
    B, table_stride = _table(block_table)
    dev = _device()
    _q4_check(k_cache, v_cache, _q4_shape(desc, group))
    shape = (B, desc.h_kv, desc.head_dim)
    if k_new.shape != shape or v_new.shape != shape or not (k_new.dtype is v_new.dtype is _TORCH.get(desc.dtype)):
        raise ValueError("k_new and v_new must be [B][h_kv][d] = %s of the descriptor's type" % (shape,))
    _q4_ints(block_table, seq_lens, B)
    _q4_here(dev, (k_new, v_new, k_cache, v_cache, block_table, seq_lens), _Q4_APPEND)
    rc = lib.zp_q4_append_kv(desc, group, k_new.data_ptr(), v_new.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                             block_table.data_ptr(), table_stride, seq_lens.data_ptr(), B, _raw_stream(stream, dev))
    if rc:
        _check(rc)


def zp_q4_read_kv(desc, k_cache, v_cache, slots, k_out, v_out, group=32, stream=None) -> None:
    """Rows of a 4-bit cache as bf16 or fp32: k_out, v_out [n][h_kv][d] (or [layers][n][h_kv][d]) receive
    the rows at `slots` (int32 [n]; negative: the row is left as it was)."""
    dev, n = _device(), slots.numel()
    K, V, layers, layer_bytes = _q4_caches(desc, group, k_cache, v_cache, dev)
    k, v, token, layer = _q4_rows(desc, k_out, v_out, n, layers, dev, ("k_out", "v_out"))
    rc = lib.zp_q4_read_kv(desc, group, K, V, layer_bytes, _ints(slots, dev, "slots"), n, k, v, token, layer,
                           1 if layers is None else layers, _raw_stream(stream, dev))
    if rc:
        _check(rc)


def zp_q4_decode_workspace_size(desc: CacheDesc, B: int, table_stride: int, group: int = 32, scored: bool = True) -> int:
    n = lib.zp_q4_decode_workspace_size(desc, group, B, table_stride, scored)
    if n == 0:
        raise ZPError(2, lib.zp_last_error().decode() or "unsupported decode shape")
    return n


_Q4_SIZES = {}  # workspace sizes by shape and device
_Q4_DECODE = ("q", "out", "k_cache", "v_cache", "block_table", "seq_lens")


def zp_q4_decode_attn(desc, q, k_cache, v_cache, block_table, seq_lens, out, score_accum=None, window=0, workspace=None,
                      stream=None, score_rows=None, group=32) -> None:
    """zp_paged_decode_attn over a 4-bit cache."""
    B, table_stride = _table(block_table)
    dev = _device()
    shape, dt = (B, desc.h_q, desc.head_dim), _TORCH.get(desc.dtype)
    if q.shape != shape or out.shape != shape:
        raise ValueError("q and out must be [B][h_q][d] = %s, are %s and %s" % (shape, tuple(q.shape), tuple(out.shape)))
    if not (q.dtype is out.dtype is dt):
        raise ValueError("q and out must have the descriptor's type")
    _q4_check(k_cache, v_cache, _q4_shape(desc, group))
    _q4_ints(block_table, seq_lens, B)
    _q4_here(dev, (q, out, k_cache, v_cache, block_table, seq_lens), _Q4_DECODE)
    n_rows, S, rows = 0, None, None
    if score_accum is not None:
        n_rows = score_accum.shape[0]
        if (score_accum.dtype is not torch.float32 or score_accum.dim() != 3 or (score_rows is None and n_rows < B) or
                score_accum.shape[1:] != (desc.h_kv, table_stride * desc.block_size)):
            raise ValueError("score_accum must be float32 [R][h_kv][table_stride*b] with a row per batch entry or a slot map")
        S, rows = _ptr_on(score_accum, dev, "score_accum"), _ints(score_rows, dev, "score_rows", B)
    elif score_rows is not None:
        raise ValueError("score_rows needs score_accum")
    args = (desc, group, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_table.data_ptr(), table_stride,
            seq_lens.data_ptr(), B, out.data_ptr(), S, rows, n_rows, window)
    on = _raw_stream(stream, dev)
    if workspace is None:
        # memory of the stream that the work runs on, given back behind it
        key = (bytes(desc), group, B, table_stride, score_accum is not None, dev)
        n = _Q4_SIZES.get(key)
        if n is None:
            if len(_Q4_SIZES) > 1000:
                _Q4_SIZES.clear()
            n = _Q4_SIZES[key] = zp_q4_decode_workspace_size(desc, B, table_stride, group, score_accum is not None)
        at = torch.cuda.caching_allocator_alloc(n, dev, on)
        try:
            rc = lib.zp_q4_decode_attn(*args, at, n, on)
        finally:
            torch.cuda.caching_allocator_delete(at)
    else:
        rc = lib.zp_q4_decode_attn(*args, _ptr_on(workspace, dev, "workspace"), workspace.nbytes, on)
    if rc:
        _check(rc)


def zp_q4_compact_pages(desc, k_cache, v_cache, src_table, dst_targets, seq_lens, keep_idx, global_F=None, scores=None,
                        rows=None, k_seq=None, group=32, stream=None) -> None:
    """zp_compact_pages of a 4-bit cache of one or several layers: keep_idx int32 [n][h_kv][k] or
    [layers][n][h_kv][k]; global_F float32 like the slots, [N_total][b][h_kv] (or one per layer), with the
    score rows `scores` that zp_score_tokens left."""
    n, table_stride = _table(src_table)
    dev = _device()
    K, V, layers, layer_bytes = _q4_caches(desc, group, k_cache, v_cache, dev)
    lead = () if layers is None else (layers,)
    k = keep_idx.shape[-1]
    if keep_idx.shape != lead + (n, desc.h_kv, k):
        raise ValueError("keep_idx must be %s, is %s" % (lead + (n, desc.h_kv, "k"), tuple(keep_idx.shape)))
    if dst_targets.dim() != 2 or dst_targets.shape[0] != n:
        raise ValueError("dst_targets must be [n][target_stride]")
    score = None
    if global_F is not None:
        if global_F.dtype is not torch.float32 or global_F.shape != lead + (desc.n_total_blocks, desc.block_size, desc.h_kv):
            raise ValueError("global_F must be float32 [N_total][b][h_kv] (or one of these per layer)")
        if scores is None:
            raise ValueError("global_F needs the score rows")
        if scores.dim() != 3 + len(lead) or scores.shape[-2] != desc.h_kv or (layers and scores.shape[0] != layers):
            raise ValueError("scores must be float32 [R][h_kv][stride] (or one of these per layer)")
        if rows is None and scores.shape[-3] < n:
            raise ValueError("scores must have a row per sequence or a row map")
        if rows is not None and rows.numel() != n:
            raise ValueError("rows must have one entry per sequence")
        _ptr_on(scores, dev, "scores")
        score = _score_rows(scores, rows)
    rc = lib.zp_q4_compact_pages(desc, group, K, V, layer_bytes, 1 if layers is None else layers,
                                 _ptr_on(global_F, dev, "global_F"), 0 if global_F is None or not lead else global_F.stride(0),
                                 score, _ints(src_table, dev, "src_table"), table_stride,
                                 _ints(dst_targets, dev, "dst_targets"), dst_targets.shape[1],
                                 _ints(seq_lens, dev, "seq_lens", n), _ints(keep_idx, dev, "keep_idx"), k,
                                 _ints(k_seq, dev, "k_seq", n), n, _raw_stream(stream, dev))
    if rc:
        _check(rc)


# ----------------------------------------------------------------------------- compression
def zp_needs_compression(seq_len: int, block_size: int, max_blocks: int) -> bool:
    return bool(lib.zp_needs_compression(int(seq_len), int(block_size), int(max_blocks)))


def zp_needs_compression_batch(seq_lens, block_size: int, max_blocks: int, active=None,
                               max_blocks_seq=None):
    """Indices (int64 numpy array, ascending) of the sequences whose trigger
    holds; host numpy arrays in, no device work."""
    import numpy as np
    lens = np.ascontiguousarray(seq_lens, dtype=np.int32)
    n = int(lens.shape[0])
    act = None if active is None else np.ascontiguousarray(active, dtype=np.uint8)
    per = None if max_blocks_seq is None else np.ascontiguousarray(max_blocks_seq, dtype=np.int32)
    out = np.empty(max(n, 1), dtype=np.int32)
    cnt = ctypes.c_int32(0)
    _check(lib.zp_needs_compression_batch(lens.ctypes.data, None if act is None else act.ctypes.data, n,
                                          int(block_size), int(max_blocks),
                                          None if per is None else per.ctypes.data, out.ctypes.data,
                                          ctypes.byref(cnt)))
    return out[:cnt.value].astype(np.int64)


def zp_score_workspace_size(desc: CacheDesc, n: int, Lmax: int) -> int:
    return int(lib.zp_score_workspace_size(ctypes.byref(desc), int(n), int(Lmax)))


def zp_window_score_workspace_size(desc: CacheDesc, n: int, Lmax: int, window: int) -> int:
    return int(lib.zp_window_score_workspace_size(ctypes.byref(desc), int(n), int(Lmax), int(window)))


def zp_window_score(desc, q_window, k_cache, block_table, seq_lens, scores_out, workspace=None,
                    stream=None) -> None:
    n, table_stride = int(block_table.shape[0]), int(block_table.shape[1])
    window = int(q_window.shape[1])
    Lmax = int(scores_out.shape[-1])
    if workspace is None:
        workspace = torch.empty(max(zp_window_score_workspace_size(desc, n, Lmax, window), 1),
                                dtype=torch.uint8, device=scores_out.device)
    _check(lib.zp_window_score(ctypes.byref(desc), _dev(q_window, "q_window"), window,
                               _dev(k_cache, "k_cache"), _dev(block_table, "block_table"), table_stride,
                               _dev(seq_lens, "seq_lens"), n, _dev(scores_out, "scores_out"), Lmax,
                               _dev(workspace, "workspace"), workspace.numel(), _stream(stream)))


def zp_score_tokens(desc, params: ScoreParams, k_cache, block_table, seq_lens, first_compression,
                    attn, global_F, scores_out, rows=None, workspace=None, stream=None) -> None:
    """attn: the attention-score rows, float32 [R][h_kv][stride] (the decode
    score_accum, or the output of zp_window_score); sequence i reads row
    rows[i] (rows None: row i).  On return the rows hold the global score."""
    n, table_stride = int(block_table.shape[0]), int(block_table.shape[1])
    Lmax = int(scores_out.shape[-1])
    if workspace is None:
        workspace = torch.empty(max(zp_score_workspace_size(desc, n, Lmax), 1), dtype=torch.uint8,
                                device=scores_out.device)
    if attn is None:
        raise ValueError("attn (the attention-score rows) is required")
    _check(lib.zp_score_tokens(ctypes.byref(desc), ctypes.byref(params), _dev(k_cache, "k_cache"),
                               _dev(block_table, "block_table"), table_stride,
                               _dev(seq_lens, "seq_lens"), _dev(first_compression, "first_compression"),
                               n, _score_rows(attn, rows), _dev(global_F, "global_F"),
                               _dev(scores_out, "scores_out"), Lmax, _dev(workspace, "workspace"),
                               workspace.numel(), _stream(stream)))


def zp_select_topk(scores, seq_lens, k, keep_idx, tie_count=None, k_seq=None, stream=None) -> None:
    """k_seq: optional int32 [n] device array of per-request budgets k_i <= k;
    keep_idx rows keep stride k and are padded with -1 after k_i."""
    n, h_kv, Lmax = (int(x) for x in scores.shape)
    _check(lib.zp_select_topk(_dev(scores, "scores"), h_kv, Lmax, _dev(seq_lens, "seq_lens"), n,
                              int(k), _dev(k_seq, "k_seq"), _dev(keep_idx, "keep_idx"),
                              _dev(tie_count, "tie_count"), _stream(stream)))


def zp_compact_pages(desc, k_base, v_base, layer_stride, layer_count, global_F, F_layer_stride,
                     src_table, dst_targets, seq_lens, keep_idx, k, scores=None, rows=None,
                     k_seq=None, stream=None) -> None:
    """scores/rows: the score rows zp_score_tokens left (float32 [R][h_kv][stride],
    or [layers][R][h_kv][stride] for several layers); needed when global_F is set."""
    n, table_stride = int(src_table.shape[0]), int(src_table.shape[1])
    _check(lib.zp_compact_pages(ctypes.byref(desc), _dev(k_base, "k_base"), _dev(v_base, "v_base"),
                                int(layer_stride), int(layer_count), _dev(global_F, "global_F"),
                                int(F_layer_stride), _score_rows(scores, rows),
                                _dev(src_table, "src_table"), table_stride,
                                _dev(dst_targets, "dst_targets"), int(dst_targets.shape[1]),
                                _dev(seq_lens, "seq_lens"), _dev(keep_idx, "keep_idx"), int(k),
                                _dev(k_seq, "k_seq"), n, _stream(stream)))


def zp_compress_workspace_size(desc: CacheDesc, n: int, Lmax: int, layer_count: int = 1) -> int:
    return int(lib.zp_compress_workspace_size(ctypes.byref(desc), int(n), int(Lmax), int(layer_count)))


def zp_compress_layers(desc, params: ScoreParams, k_cache, v_cache, block_table, seq_lens, first_compression,
                       attn, global_F, dst_targets, k, keep_idx, Lmax, rows=None, tie_count=None, scores_out=None,
                       workspace=None, k_seq=None, stream=None, rho=None, rho_rows=None) -> None:
    """Scores, keep sets and moves of one or several layers in one call.
    k_cache/v_cache: one layer [N_total][b][h_kv][d] or several
    [layers][N_total][b][h_kv][d]; global_F and attn (score rows) alike;
    keep_idx int32 [layers][n][h_kv][k] (or [n][h_kv][k] for one layer);
    k_seq: optional int32 [n] device array of per-request budgets k_i <= k.
    rho (optional float32 [R][h_kv][stride], or [layers][R][h_kv][stride]) with
    rho_rows (int32 [n] device or None: row i): lightning row sums written by
    the decode; the call then runs zp_compress_layers_rho (no workspace)."""
    n, table_stride = int(block_table.shape[0]), int(block_table.shape[1])
    layers = int(k_cache.shape[0]) if k_cache.dim() == 5 else 1
    layer_stride = int(k_cache.stride(0)) if layers > 1 else 0
    F_layer = int(global_F.stride(0)) if (global_F is not None and global_F.dim() == 4) else 0
    if layers > 1 and attn.dim() != 4:
        raise ValueError("several layers need score rows [layers][R][h_kv][stride]")
    if rho is not None:
        if layers > 1 and rho.dim() != 4:
            raise ValueError("several layers need redundancy rows [layers][R][h_kv][stride]")
        _check(lib.zp_compress_layers_rho(ctypes.byref(desc), ctypes.byref(params), _dev(k_cache, "k_cache"),
                                          _dev(v_cache, "v_cache"), layer_stride, layers,
                                          _dev(block_table, "block_table"), table_stride, _dev(seq_lens, "seq_lens"),
                                          _dev(first_compression, "first_compression"), n, _score_rows(attn, rows),
                                          _dev(global_F, "global_F"), F_layer, _dev(dst_targets, "dst_targets"),
                                          int(dst_targets.shape[1]), int(k), _dev(k_seq, "k_seq"),
                                          _dev(keep_idx, "keep_idx"), _dev(tie_count, "tie_count"),
                                          _dev(scores_out, "scores_out"), int(Lmax), _rho_rows(rho, rho_rows),
                                          _stream(stream)))
        return
    if workspace is None:
        workspace = torch.empty(max(zp_compress_workspace_size(desc, n, Lmax, layers), 1), dtype=torch.uint8,
                                device=k_cache.device)
    _check(lib.zp_compress_layers(ctypes.byref(desc), ctypes.byref(params), _dev(k_cache, "k_cache"),
                                  _dev(v_cache, "v_cache"), layer_stride, layers, _dev(block_table, "block_table"),
                                  table_stride, _dev(seq_lens, "seq_lens"),
                                  _dev(first_compression, "first_compression"), n, _score_rows(attn, rows),
                                  _dev(global_F, "global_F"), F_layer, _dev(dst_targets, "dst_targets"),
                                  int(dst_targets.shape[1]), int(k), _dev(k_seq, "k_seq"),
                                  _dev(keep_idx, "keep_idx"),
                                  _dev(tie_count, "tie_count"), _dev(scores_out, "scores_out"), int(Lmax),
                                  _dev(workspace, "workspace"), workspace.numel(), _stream(stream)))


def zp_compress_rho_supported(desc, params: ScoreParams, Lmax: int, k: int) -> bool:
    """Whether zp_compress_layers_rho (the decode's row sums, one kernel) covers
    this cache, these switches, Lmax and k on the current device."""
    return bool(lib.zp_compress_rho_supported(ctypes.byref(desc), ctypes.byref(params), int(Lmax), int(k)))


def zp_plan_capacity(m_available: int, m_kv_block: int, m_q_request: int, max_blocks: int,
                     extra=(0, 1)):
    """(M, N_total) of eq. (1) / (2): the largest request concurrency and the
    block count for a memory budget; extra = (num, den) per-block overhead of
    the global score cache relative to K and V."""
    M, N = ctypes.c_int64(0), ctypes.c_int64(0)
    _check(lib.zp_plan_capacity(int(m_available), int(m_kv_block), int(m_q_request), int(max_blocks),
                                int(extra[0]), int(extra[1]), ctypes.byref(M), ctypes.byref(N)))
    return M.value, N.value


def zp_device_status(clear: bool = True):
    code, detail = ctypes.c_int32(0), ctypes.c_int32(0)
    _check(lib.zp_device_status(ctypes.byref(code), ctypes.byref(detail), int(bool(clear))))
    return code.value, detail.value


# ----------------------------------------------------------------------------- host pool
def _i32buf(n):
    return (ctypes.c_int32 * max(int(n), 1))()


class Pool:
    """Host block pool (zp_pool_*): reference counts and the free list."""

    def __init__(self, n_total: int):
        self._p = lib.zp_pool_create(int(n_total))
        if not self._p:
            raise ZPError(1, lib.zp_last_error().decode())
        self.n_total = int(n_total)

    def __del__(self):
        p = getattr(self, "_p", None)
        if p:
            lib.zp_pool_destroy(p)
            self._p = None

    @property
    def num_free(self) -> int:
        return int(lib.zp_pool_num_free(self._p))

    def refcount(self, block: int) -> int:
        return int(lib.zp_pool_refcount(self._p, int(block)))

    def alloc(self, n: int):
        buf = _i32buf(n)
        _check(lib.zp_pool_alloc(self._p, int(n), buf))
        return list(buf)[: int(n)]

    def incref(self, ids):
        ids = list(ids)
        buf = (ctypes.c_int32 * max(len(ids), 1))(*ids)
        _check(lib.zp_pool_incref(self._p, len(ids), buf))

    def release(self, ids):
        ids = list(ids)
        buf = (ctypes.c_int32 * max(len(ids), 1))(*ids)
        _check(lib.zp_pool_release(self._p, len(ids), buf))

    def plan_compaction(self, table, max_blocks: int):
        table = [int(x) for x in table]
        tb = (ctypes.c_int32 * max(len(table), 1))(*table)
        targets, new_table = _i32buf(max_blocks - 1), _i32buf(max_blocks)
        dropped = _i32buf(len(table))
        nd, nf = ctypes.c_int32(0), ctypes.c_int32(0)
        _check(lib.zp_plan_compaction(self._p, tb, len(table), int(max_blocks), targets, new_table,
                                      dropped, ctypes.byref(nd), ctypes.byref(nf)))
        return {"targets": list(targets)[: max_blocks - 1], "new_table": list(new_table)[:max_blocks],
                "dropped": list(dropped)[: nd.value], "n_fresh": nf.value}

    def plan_compaction_batch(self, tables, n_blocks, max_blocks: int, out=None, max_blocks_seq=None):
        """Plans of n sequences in one C call; tables int32 [n][stride] and
        n_blocks int32 [n] as numpy arrays; max_blocks_seq: optional int32 [n]
        per-request block budgets in [2, max_blocks] (rows padded with -1).
        Returns numpy arrays (reused from ``out`` when given): targets
        [n][max_blocks-1], new_tables [n][max_blocks], dropped [n][stride],
        n_dropped [n], n_fresh [n]."""
        import numpy as np
        tables = np.ascontiguousarray(tables, dtype=np.int32)
        n_blocks = np.ascontiguousarray(n_blocks, dtype=np.int32)
        n, stride = tables.shape
        if out is None:
            out = {"targets": np.empty((n, max_blocks - 1), np.int32),
                   "new_tables": np.empty((n, max_blocks), np.int32),
                   "dropped": np.empty((n, stride), np.int32), "n_dropped": np.empty(n, np.int32),
                   "n_fresh": np.empty(n, np.int32)}
        P = lambda a: ctypes.c_void_p(a.ctypes.data)  # noqa: E731
        mbs = None
        if max_blocks_seq is not None:
            mbs = np.ascontiguousarray(max_blocks_seq, dtype=np.int32)
            if mbs.shape != (n,):
                raise ValueError("max_blocks_seq must have one entry per sequence")
        _check(lib.zp_plan_compaction_batch(self._p, P(tables), stride, P(n_blocks), n, int(max_blocks),
                                            None if mbs is None else P(mbs), P(out["targets"]), P(out["new_tables"]), P(out["dropped"]),
                                            P(out["n_dropped"]), P(out["n_fresh"])))
        return out


__all__ = ["lib", "LIB_PATH", "EXPORTS", "ZPError", "CacheDesc", "ScoreParams", "ScoreRows", "RhoRows", "score_params",
           "cache_desc", "zp_decode_workspace_size", "zp_paged_decode_attn",
           "zp_paged_decode_attn_noalloc", "zp_append_kv",
           "zp_build_slots", "zp_write_kv", "PrefixPlan", "prefix_plan", "zp_prefix_plan",
           "zp_prefix_decode_workspace_size", "zp_prefix_decode_attn",
           "zp_needs_compression", "zp_needs_compression_batch", "zp_window_score_workspace_size", "zp_window_score",
           "zp_score_workspace_size", "zp_score_tokens", "zp_select_topk",
           "zp_compact_pages", "zp_compress_workspace_size", "zp_compress_layers", "zp_compress_rho_supported", "zp_plan_capacity", "zp_device_status", "Pool",
           "ZP_BF16", "ZP_F32"]
