"""Thin Python binding of ``libds_ragged.so`` (argument marshalling only).

The functions keep the C ABI's names (``include/ds_ragged.h``); every step of
the layer runs in the library's CUDA kernels.  PyTorch supplies device memory,
pinned host memory and streams.  There is no fallback: if the library is
missing, importing the binding's functions raises.
"""
from __future__ import annotations

import ctypes
import math
import os
from typing import Optional, Sequence

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libds_ragged.so")

DS_OK, DS_ERR_INVALID_ARG, DS_ERR_CAPACITY, DS_ERR_BAD_BLOCK = 0, 1, 2, 3
DS_ERR_UNSUPPORTED, DS_ERR_WORKSPACE, DS_ERR_CUDA = 4, 5, 6
DS_DEVERR_BLOCK_ID, DS_DEVERR_POSITION, DS_DEVERR_WORKLIST, DS_DEVERR_TOKEN = 1, 2, 4, 8
DS_FP16, DS_BF16, DS_FP32 = 0, 1, 2
DS_ROPE_HALF, DS_ROPE_INTERLEAVED = 0, 1
DS_META_CAPACITY = 1
STATUS_NAMES = {0: "DS_OK", 1: "DS_ERR_INVALID_ARG", 2: "DS_ERR_CAPACITY", 3: "DS_ERR_BAD_BLOCK",
                4: "DS_ERR_UNSUPPORTED", 5: "DS_ERR_WORKSPACE", 6: "DS_ERR_CUDA"}

P = ctypes.c_void_p
i32 = ctypes.c_int32


class ds_seq_desc(ctypes.Structure):
    _fields_ = [("seen_tokens", i32), ("new_tokens", i32),
                ("block_ids", ctypes.POINTER(i32)), ("n_blocks", i32)]


class ds_attn_params(ctypes.Structure):
    _fields_ = [("n_q_heads", i32), ("n_kv_heads", i32), ("head_dim", i32), ("block_size", i32),
                ("dtype", i32), ("rope_style", i32), ("rope_theta", ctypes.c_float),
                ("softmax_scale", ctypes.c_float)]


class ds_kv_pool(ctypes.Structure):
    _fields_ = [("base", P), ("num_blocks", i32)]


class ds_kv8_pool(ctypes.Structure):
    _fields_ = [("codes", P), ("scales", P), ("num_blocks", i32)]


class ds_rope_table(ctypes.Structure):
    _fields_ = [("table", P), ("max_positions", i32), ("head_dim", i32),
                ("rope_theta", ctypes.c_float)]


class ds_qk_norm(ctypes.Structure):
    _fields_ = [("q_weight", P), ("k_weight", P), ("per_head", i32), ("eps", ctypes.c_float)]


class ds_sampler(ctypes.Structure):
    _fields_ = [("uniforms", P), ("temperature", P), ("top_k", P), ("top_p", P), ("min_p", P)]


class ds_logit_rules(ctypes.Structure):
    _fields_ = [("history", P), ("history_stride", ctypes.c_int64), ("history_len", P), ("prompt_len", P), ("repetition", P),
                ("frequency", P), ("presence", P), ("bias_ids", P), ("bias_values", P), ("bias_stride", ctypes.c_int64),
                ("bias_len", P), ("mask", P), ("mask_stride", ctypes.c_int64), ("n_masks", i32), ("mask_row", P)]


class ds_lora_weights(ctypes.Structure):
    _fields_ = [("a", P), ("b", P), ("scale", P), ("n_adapters", i32), ("rank", i32), ("in_dim", i32),
                ("out_dim", i32), ("dtype", i32)]


class ds_lora_plan(ctypes.Structure):
    _fields_ = [("device_buf", P), ("device_bytes", ctypes.c_size_t),
                ("host_staging", P), ("staging_bytes", ctypes.c_size_t),
                ("max_seqs", i32), ("max_tokens", i32), ("flags", i32),
                ("n_seqs", i32), ("n_tokens", i32), ("n_adapters", i32),
                ("n_small_tiles", i32), ("n_large_tiles", i32), ("used_bytes", ctypes.c_size_t),
                ("header", P), ("order", P), ("small_tiles", P), ("large_tiles", P)]


class ds_ragged_meta(ctypes.Structure):
    _fields_ = [("device_buf", P), ("device_bytes", ctypes.c_size_t),
                ("host_staging", P), ("staging_bytes", ctypes.c_size_t),
                ("max_seqs", i32), ("max_tokens", i32), ("max_blocks", i32), ("flags", i32),
                ("n_seqs", i32), ("n_tokens", i32), ("n_blocks", i32),
                ("n_prefill_seqs", i32), ("n_decode_seqs", i32), ("n_prefill_tiles", i32),
                ("n_decode_items", i32), ("max_len", i32), ("pool_num_blocks", i32),
                ("split_blocks", i32), ("prefill_sms", ctypes.c_float), ("used_bytes", ctypes.c_size_t),
                ("header", P), ("cu_seqlens", P), ("seq_seen", P), ("seq_new", P),
                ("blk_off", P), ("block_table", P), ("tok_seq", P), ("tok_pos", P),
                ("prefill_tiles", P), ("decode_items", P), ("decode_seqs", P)]


class ds_block_allocator(ctypes.Structure):
    _fields_ = [("stack", P), ("state", P), ("num_blocks", i32), ("n_free", i32)]


class ds_splitfuse(ctypes.Structure):
    _fields_ = [("mem", P), ("mem_bytes", ctypes.c_size_t), ("max_requests", i32),
                ("max_blocks_per_request", i32), ("token_budget", i32), ("max_seqs", i32),
                ("block_size", i32), ("n_active", i32), ("n_planned", i32)]


# name -> (restype, argtypes); every entry point of include/ds_ragged.h
SIGNATURES = {
    "ds_last_error": (ctypes.c_char_p, []),
    "ds_version": (ctypes.c_char_p, []),
    "ds_meta_buffer_sizes": (i32, [i32, i32, i32, P, P, P]),
    "ds_ragged_meta_pack": (i32, [P, i32, P, i32, P]),
    "ds_ragged_meta_build": (i32, [P, i32, P, i32, P, P]),
    "ds_rope_table_size": (i32, [P, i32, P]),
    "ds_rope_table_build": (i32, [P, i32, P, ctypes.c_size_t, P, P]),
    "ds_kv_rotary_append": (i32, [P, P, P, P, P, P, P]),
    "ds_kv_norm_rotary_append": (i32, [P, P, P, P, P, P, P, P, P]),
    "ds_blocked_attention_workspace_size": (i32, [P, i32, i32, i32, P]),
    "ds_blocked_attention": (i32, [P, P, P, P, P, P, P, ctypes.c_size_t, P]),
    "ds_get_device_error": (i32, [P, P, P]),
    "ds_kv8_rotary_append": (i32, [P, P, P, P, P, P]),
    "ds_kv8_blocked_attention": (i32, [P, P, P, P, P, P, P, ctypes.c_size_t, P]),
    "ds_blocked_attention_static_ws": (i32, [P, P, P, P, P, P, P]),
    "ds_fused_workspace_size": (i32, [P, i32, i32, i32, P]),
    "ds_fused_workspace_init": (i32, [P, P, P, ctypes.c_size_t, P]),
    "ds_fused_append_attention": (i32, [P, P, P, P, P, P, P, ctypes.c_size_t, P]),
    "ds_block_allocator_init": (i32, [P, P, P, i32, P]),
    "ds_block_allocator_allocate": (i32, [P, i32, P]),
    "ds_block_allocator_free": (i32, [P, P, i32]),
    "ds_kv_blocks_required": (i32, [i32, i32, i32, i32, P]),
    "ds_splitfuse_mem_size": (i32, [i32, i32, P]),
    "ds_splitfuse_init": (i32, [P, P, ctypes.c_size_t, i32, i32, i32, i32, i32]),
    "ds_splitfuse_add": (i32, [P, i32, i32, i32]),
    "ds_splitfuse_next": (i32, [P, P, P, P, P]),
    "ds_splitfuse_commit": (i32, [P, P, P, P]),
    "ds_kv_block_bytes": (i32, [P, P]),
    "ds_kv_offload": (i32, [P, P, P, i32, P, P]),
    "ds_kv_restore": (i32, [P, P, P, i32, P, P]),
    "ds_ragged_embedding": (i32, [P, P, P, i32, i32, i32, P, P]),
    "ds_ragged_logits_gather": (i32, [P, P, i32, i32, P, P]),
    "ds_lora_plan_size": (i32, [i32, i32, P, P]),
    "ds_lora_plan_pack": (i32, [P, P, i32, i32, P]),
    "ds_lora_plan_build": (i32, [P, P, i32, i32, P, P]),
    "ds_ragged_lora": (i32, [P, P, P, ctypes.c_int64, P, ctypes.c_int64, P, ctypes.c_int64, P]),
    "ds_lora_get_device_error": (i32, [P, P, P]),
    "ds_ragged_adjust_logits": (i32, [P, P, i32, i32, ctypes.c_int64, P, P, ctypes.c_int64, P]),
    "ds_ragged_sample": (i32, [P, P, i32, i32, ctypes.c_int64, P, P, P, P]),
}

DS_STATIC_WORKSPACE_BYTES = 32 << 20

_lib = None


class DSError(RuntimeError):
    def __init__(self, status: int, where: str, msg: str):
        super().__init__("%s: %s (%s)" % (where, msg, STATUS_NAMES.get(status, status)))
        self.status = status


def load():
    """Load the library (raises if it was not built: there is no fallback)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libds_ragged.so is not built (%s); run __graft_entry__.build()" % LIB_PATH)
        lib = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def _ref(x):
    return ctypes.byref(x) if x is not None else None


def _check(status: int, where: str):
    if status != DS_OK:
        raise DSError(status, where, load().ds_last_error().decode())


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if isinstance(t, np.ndarray):
        return t.ctypes.data
    return t.data_ptr()


def _stream(s) -> Optional[int]:
    if s is None:
        return None
    if isinstance(s, int):
        return s
    return s.cuda_stream


def make_params(n_q_heads: int, n_kv_heads: int, head_dim: int, dtype: str = "bf16",
                rope_theta: float = 1.0e4, rope_style: int = DS_ROPE_HALF,
                block_size: int = 64, softmax_scale: float = 0.0) -> ds_attn_params:
    return ds_attn_params(n_q_heads, n_kv_heads, head_dim, block_size,
                          {"fp16": DS_FP16, "bf16": DS_BF16}[dtype] if isinstance(dtype, str) else dtype,
                          rope_style, rope_theta, softmax_scale)


def params_for(wl, rope_style: int = DS_ROPE_HALF) -> ds_attn_params:
    return make_params(wl.n_q_heads, wl.n_kv_heads, wl.head_dim, wl.dtype, wl.rope_theta,
                       rope_style, wl.block_size)


class SeqDescs:
    """ds_seq_desc[] for a workload (keeps the id arrays alive)."""

    def __init__(self, seen: Sequence[int], new: Sequence[int], block_ids: Sequence[np.ndarray]):
        self.ids = [np.ascontiguousarray(b, dtype=np.int32) for b in block_ids]
        n = len(self.ids)
        self.arr = (ds_seq_desc * max(n, 1))()
        for i in range(n):
            self.arr[i].seen_tokens = int(seen[i])
            self.arr[i].new_tokens = int(new[i])
            self.arr[i].block_ids = self.ids[i].ctypes.data_as(ctypes.POINTER(i32))
            self.arr[i].n_blocks = len(self.ids[i])
        self.n = n

    @classmethod
    def of(cls, wl):
        return cls(wl.seen, wl.new, wl.block_ids)


# ------------------------------------------------------------ thin wrappers --

def ds_meta_buffer_sizes(max_seqs: int, max_tokens: int, max_blocks: int, params: ds_attn_params):
    dev, stg = ctypes.c_size_t(0), ctypes.c_size_t(0)
    _check(load().ds_meta_buffer_sizes(max_seqs, max_tokens, max_blocks, _ref(params),
                                       _ref(dev), _ref(stg)), "ds_meta_buffer_sizes")
    return dev.value, stg.value


def ds_ragged_meta_pack(descs: SeqDescs, params: ds_attn_params, pool_num_blocks: int,
                        meta: ds_ragged_meta) -> int:
    return load().ds_ragged_meta_pack(_ref(descs.arr), descs.n, _ref(params), pool_num_blocks, _ref(meta))


def ds_ragged_meta_build(descs: SeqDescs, params: ds_attn_params, pool_num_blocks: int,
                         meta: ds_ragged_meta, stream=None):
    _check(load().ds_ragged_meta_build(_ref(descs.arr), descs.n, _ref(params), pool_num_blocks,
                                       _ref(meta), _stream(stream)), "ds_ragged_meta_build")


def ds_rope_table_size(params: ds_attn_params, max_positions: int) -> int:
    b = ctypes.c_size_t(0)
    _check(load().ds_rope_table_size(_ref(params), max_positions, _ref(b)), "ds_rope_table_size")
    return b.value


def ds_rope_table_build(params: ds_attn_params, max_positions: int, table, stream=None) -> ds_rope_table:
    out = ds_rope_table()
    nbytes = table.numel() * table.element_size()
    _check(load().ds_rope_table_build(_ref(params), max_positions, _ptr(table), nbytes, _ref(out),
                                      _stream(stream)), "ds_rope_table_build")
    return out


def ds_kv_rotary_append(meta: ds_ragged_meta, params: ds_attn_params, rope: ds_rope_table, qkv,
                        q_out, pool: ds_kv_pool, stream=None):
    _check(load().ds_kv_rotary_append(_ref(meta), _ref(params), _ref(rope), _ptr(qkv), _ptr(q_out),
                                      _ref(pool), _stream(stream)), "ds_kv_rotary_append")


def _require(ok: bool, where: str, msg: str):
    if not ok:
        raise DSError(DS_ERR_INVALID_ARG, where, msg)


def make_qk_norm(q_weight, k_weight, eps: float = 1e-6, per_head: bool = False) -> ds_qk_norm:
    """ds_qk_norm of two CUDA tensors of the layer's storage type (None: ones):
    [head_dim], or with per_head [heads][head_dim].  Keeps them alive."""
    import torch
    given = [w for w in (q_weight, k_weight) if w is not None]
    for w in given:
        _require(w.is_cuda and w.is_contiguous() and w.dtype in (torch.float16, torch.bfloat16) and w.dtype == given[0].dtype,
                 "make_qk_norm", "weights must be contiguous CUDA tensors of the storage type, fp16 or bf16")
    norm = ds_qk_norm(_ptr(q_weight), _ptr(k_weight), int(per_head), eps)
    norm.tensors = (q_weight, k_weight)
    # type, device and elements of the weights, None and 0 for ones
    norm.given = (given[0].dtype if given else None, _device_of("make_qk_norm", *given),
                  *(0 if w is None else w.numel() for w in norm.tensors))
    return norm


def _current_device():
    """The device that the library launches on; None where there is none."""
    import torch
    try:
        return torch.cuda.current_device()
    except (RuntimeError, AssertionError):
        return None


def _device_of(where: str, *given):
    """The one device of some CUDA tensors, None where there are none."""
    at = [t.get_device() for t in given if t is not None]
    _require(not at or min(at) == max(at), where, "tensors are on several devices")
    return at[0] if at else None


def _elsewhere(where: str, device):
    raise DSError(DS_ERR_INVALID_ARG, where, "tensors are on device %d, which is not the current one" % device)


def _storage(params: ds_attn_params, known={}):
    """Torch's type of a layer's storage type."""
    if not known:
        import torch
        known.update({DS_FP16: torch.float16, DS_BF16: torch.bfloat16})
    return known.get(params.dtype)


def _rows_ptr(where: str, t, dtype, elements: int, here):
    """Address of a contiguous tensor of `dtype` on device `here` that holds `elements`, or an address as it is
    (None: NULL)."""
    if t is None or isinstance(t, int):
        return t
    if t.get_device() == here and t.dtype is dtype and t.numel() >= elements and t.is_contiguous():
        return t.data_ptr()
    _require(t.is_cuda and t.is_contiguous(), where, "tensors must be contiguous and on the GPU")
    if t.get_device() != here:
        _elsewhere(where, t.get_device())
    raise DSError(DS_ERR_INVALID_ARG, where, "tensors must be of the layer's storage type and hold a whole row for each token (the pool: whole blocks)")


def ds_kv_norm_rotary_append(meta: ds_ragged_meta, params: ds_attn_params, rope: ds_rope_table,
                             norm: ds_qk_norm, qkv, qkv_out, q_out, pool: ds_kv_pool, stream=None, pool_t=None):
    """pool_t: the pool as a tensor [blocks, 2, KV heads, 64, head_dim], in the place of pool."""
    where = "ds_kv_norm_rotary_append"
    if meta is None or params is None or norm is None:  # the library's to refuse
        qkv = qkv_out = q_out = None
    else:
        dt, here = _storage(params), _current_device()
        hq, hkv, d = params.n_q_heads, params.n_kv_heads, params.head_dim
        kind, device, nq, nk = getattr(norm, "given", (None, here, 0, 0))  # not known of a struct filled by hand
        if kind is not None:
            per_head = norm.per_head
            if (nq and nq != (d * hq if per_head else d)) or (nk and nk != (d * hkv if per_head else d)):
                raise DSError(DS_ERR_INVALID_ARG, where, "norm weights have head_dim elements, with per_head for each head")
            if kind is not dt:
                raise DSError(DS_ERR_INVALID_ARG, where, "norm weights are not of the layer's storage type")
            if device != here:
                _elsewhere(where, device)
        n = meta.max_tokens if meta.flags & DS_META_CAPACITY else meta.n_tokens
        width = n * (hq + 2 * hkv) * d
        qkv = _rows_ptr(where, qkv, dt, width, here)
        qkv_out = qkv_out if qkv_out is None else _rows_ptr(where, qkv_out, dt, width, here)
        q_out = q_out if q_out is None else _rows_ptr(where, q_out, dt, n * hq * d, here)
        if pool_t is not None:
            blocks = pool_t.shape[0]
            pool = ds_kv_pool(_rows_ptr(where, pool_t, dt, blocks * 2 * hkv * params.block_size * d, here), blocks)
    _check(load().ds_kv_norm_rotary_append(_ref(meta), _ref(params), _ref(rope), _ref(norm), qkv, qkv_out, q_out, _ref(pool),
                                           _stream(stream)), where)


def ds_blocked_attention_workspace_size(params: ds_attn_params, max_seqs: int, max_tokens: int,
                                        max_blocks: int) -> int:
    b = ctypes.c_size_t(0)
    _check(load().ds_blocked_attention_workspace_size(_ref(params), max_seqs, max_tokens, max_blocks,
                                                      _ref(b)), "ds_blocked_attention_workspace_size")
    return b.value


def ds_blocked_attention(meta: ds_ragged_meta, params: ds_attn_params, rope: ds_rope_table, qkv,
                         pool: ds_kv_pool, out, workspace, stream=None):
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(load().ds_blocked_attention(_ref(meta), _ref(params), _ref(rope), _ptr(qkv), _ref(pool),
                                       _ptr(out), _ptr(workspace), ws_bytes, _stream(stream)),
           "ds_blocked_attention")


def make_kv8_pool(codes, scales) -> ds_kv8_pool:
    """ds_kv8_pool of two contiguous CUDA tensors: codes [blocks, 2, KV heads, 64, head_dim] of a type of one byte
    (uint8 or float8_e4m3fn), scales float32 [blocks, 2, KV heads].  Keeps them alive."""
    import torch
    _require(codes.is_cuda and scales.is_cuda and codes.is_contiguous() and scales.is_contiguous()
             and codes.dtype in (torch.uint8, torch.float8_e4m3fn) and scales.dtype is torch.float32
             and len(codes.shape) == 5 and codes.shape[1] == 2 and tuple(scales.shape) == tuple(codes.shape[:3]),
             "make_kv8_pool", "codes must be a contiguous CUDA tensor of bytes [blocks, 2, KV heads, 64, head_dim], scales "
             "one of float32 [blocks, 2, KV heads]")
    pool = ds_kv8_pool(codes.data_ptr(), scales.data_ptr(), codes.shape[0])
    pool.tensors = (codes, scales)
    pool.device = _device_of("make_kv8_pool", codes, scales)
    pool.tile = tuple(codes.shape[2:])
    return pool


def _kv8_args(where: str, meta, params, qkv, pool):
    """(address of qkv, the device) for a call on an 8-bit pool; a pool filled by hand is taken as it is."""
    here = _current_device()
    tile = getattr(pool, "tile", None)
    if tile is not None:
        if tile != (params.n_kv_heads, params.block_size, params.head_dim):
            raise DSError(DS_ERR_INVALID_ARG, where, "the pool is for another layer shape")
        if pool.device != here:
            _elsewhere(where, pool.device)
    n = meta.max_tokens if meta.flags & DS_META_CAPACITY else meta.n_tokens
    width = (params.n_q_heads + 2 * params.n_kv_heads) * params.head_dim
    return _rows_ptr(where, qkv, _storage(params), n * width, here), here


def ds_kv8_rotary_append(meta: ds_ragged_meta, params: ds_attn_params, rope: ds_rope_table, qkv, pool: ds_kv8_pool, stream=None):
    where = "ds_kv8_rotary_append"
    if meta is not None and params is not None:  # else the library's to refuse
        qkv, _ = _kv8_args(where, meta, params, qkv, pool)
    _check(load().ds_kv8_rotary_append(_ref(meta), _ref(params), _ref(rope), _ptr(qkv), _ref(pool), _stream(stream)), where)


def ds_kv8_blocked_attention(meta: ds_ragged_meta, params: ds_attn_params, rope: ds_rope_table, qkv, pool: ds_kv8_pool, out,
                             workspace, stream=None):
    where = "ds_kv8_blocked_attention"
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    if meta is not None and params is not None:
        qkv, here = _kv8_args(where, meta, params, qkv, pool)
        n = meta.max_tokens if meta.flags & DS_META_CAPACITY else meta.n_tokens
        out = _rows_ptr(where, out, _storage(params), n * params.n_q_heads * params.head_dim, here)
        if workspace is not None and (workspace.get_device() != here or not workspace.is_contiguous()):
            raise DSError(DS_ERR_INVALID_ARG, where, "the workspace must be contiguous and on the current device")
    _check(load().ds_kv8_blocked_attention(_ref(meta), _ref(params), _ref(rope), _ptr(qkv), _ref(pool), _ptr(out),
                                           _ptr(workspace), ws_bytes, _stream(stream)), where)


def ds_fused_workspace_size(params: ds_attn_params, max_seqs: int, max_tokens: int, max_blocks: int) -> int:
    b = ctypes.c_size_t(0)
    _check(load().ds_fused_workspace_size(_ref(params), max_seqs, max_tokens, max_blocks, _ref(b)),
           "ds_fused_workspace_size")
    return b.value


def ds_fused_workspace_init(meta: ds_ragged_meta, params: ds_attn_params, workspace, stream=None):
    ws_bytes = workspace.numel() * workspace.element_size()
    _check(load().ds_fused_workspace_init(_ref(meta), _ref(params), _ptr(workspace), ws_bytes, _stream(stream)),
           "ds_fused_workspace_init")


def ds_fused_append_attention(meta: ds_ragged_meta, params: ds_attn_params, rope: ds_rope_table, qkv,
                              pool: ds_kv_pool, out, workspace, stream=None):
    """The append and the attention of one batch (a decode-only batch is one launch)."""
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(load().ds_fused_append_attention(_ref(meta), _ref(params), _ref(rope), _ptr(qkv), _ref(pool),
                                            _ptr(out), _ptr(workspace), ws_bytes, _stream(stream)),
           "ds_fused_append_attention")


def ds_blocked_attention_static_ws(meta: ds_ragged_meta, params: ds_attn_params, rope: ds_rope_table,
                                   qkv, pool: ds_kv_pool, out, stream=None):
    """ds_blocked_attention with the split partials in the library's built-in
    scratch array (no workspace argument; nothing is allocated)."""
    _check(load().ds_blocked_attention_static_ws(_ref(meta), _ref(params), _ref(rope), _ptr(qkv),
                                                 _ref(pool), _ptr(out), _stream(stream)),
           "ds_blocked_attention_static_ws")


def ds_kv_block_bytes(params: ds_attn_params) -> int:
    b = ctypes.c_size_t(0)
    _check(load().ds_kv_block_bytes(_ref(params), _ref(b)), "ds_kv_block_bytes")
    return b.value


def ds_kv_offload(params: ds_attn_params, pool: ds_kv_pool, block_ids, host_dst, stream=None):
    ids = np.ascontiguousarray(block_ids, np.int32)
    _check(load().ds_kv_offload(_ref(params), _ref(pool), ids.ctypes.data if len(ids) else None, len(ids),
                                _ptr(host_dst), _stream(stream)), "ds_kv_offload")


def ds_kv_restore(params: ds_attn_params, pool: ds_kv_pool, block_ids, host_src, stream=None):
    ids = np.ascontiguousarray(block_ids, np.int32)
    _check(load().ds_kv_restore(_ref(params), _ref(pool), ids.ctypes.data if len(ids) else None, len(ids),
                                _ptr(host_src), _stream(stream)), "ds_kv_restore")


def ds_ragged_embedding(meta: ds_ragged_meta, token_ids, table, out, stream=None):
    vocab, hidden = table.shape
    _check(load().ds_ragged_embedding(_ref(meta), _ptr(token_ids), _ptr(table), vocab, hidden,
                                      table.element_size(), _ptr(out), _stream(stream)), "ds_ragged_embedding")


def ds_ragged_logits_gather(meta: ds_ragged_meta, hidden_states, out, stream=None):
    hidden = hidden_states.shape[1]
    _check(load().ds_ragged_logits_gather(_ref(meta), _ptr(hidden_states), hidden,
                                          hidden_states.element_size(), _ptr(out), _stream(stream)),
           "ds_ragged_logits_gather")


def make_lora(a, b, scale=None) -> ds_lora_weights:
    """ds_lora_weights of contiguous CUDA tensors of one 16-bit type, a [adapters][rank]
    [in] and b [adapters][out][rank], and float32 scale [adapters].  Keeps them alive."""
    import torch
    kinds = {torch.float16: DS_FP16, torch.bfloat16: DS_BF16}
    n, rank, width_in = a.shape
    _require(a.dtype in kinds and a.dtype == b.dtype and a.is_cuda and b.is_cuda and a.is_contiguous() and b.is_contiguous()
             and b.shape[0] == n and b.shape[2] == rank, "make_lora", "a and b must be contiguous CUDA tensors of fp16 or bf16, "
             "[adapters][rank][in] and [adapters][out][rank]")
    _require(scale is None or (scale.is_cuda and scale.is_contiguous() and scale.dtype == torch.float32 and scale.numel() == n),
             "make_lora", "scale must be a contiguous CUDA tensor of float32, one for each adapter")
    w = ds_lora_weights(_ptr(a), _ptr(b), _ptr(scale), n, rank, width_in, b.shape[1], kinds[a.dtype])
    w.tensors = (a, b, scale)
    w.device = _device_of("make_lora", a, b, scale)
    return w


class LoraPlan:
    """A ds_lora_plan with its buffers (allocated with torch) for batches within the capacities."""

    def __init__(self, max_seqs: int, max_tokens: int, device: str = "cuda", stream=None, flags: int = 0):
        import torch
        self.stream = stream
        dev, stg = ctypes.c_size_t(0), ctypes.c_size_t(0)
        _check(load().ds_lora_plan_size(max_seqs, max_tokens, _ref(dev), _ref(stg)), "ds_lora_plan_size")
        self.device_buf = torch.empty(dev.value, dtype=torch.uint8, device=device)
        self.staging = torch.empty(stg.value, dtype=torch.uint8, pin_memory=True)
        self.plan = ds_lora_plan(_ptr(self.device_buf), dev.value, _ptr(self.staging), stg.value, max_seqs, max_tokens, flags)
        self.plan.device = self.device_buf.get_device()

    def _args(self, new_tokens, adapters, n_adapters):
        new, which = (np.ascontiguousarray(v, np.int32) for v in (new_tokens, adapters))
        _require(new.shape == which.shape and new.ndim == 1, "LoraPlan", "one adapter for each sequence")
        return new, which, (new.ctypes.data, which.ctypes.data, len(new), n_adapters, _ref(self.plan))

    def build(self, new_tokens, adapters, n_adapters: int):
        """Pack and upload: adapters[i] (-1: none) for sequence i of new_tokens[i] tokens."""
        keep = self._args(new_tokens, adapters, n_adapters)
        _check(load().ds_lora_plan_build(*keep[2], _stream(self.stream)), "ds_lora_plan_build")

    def pack(self, new_tokens, adapters, n_adapters: int):
        """Host half of build: with DS_META_CAPACITY, what a captured graph's upload copies next."""
        keep = self._args(new_tokens, adapters, n_adapters)
        _check(load().ds_lora_plan_pack(*keep[2]), "ds_lora_plan_pack")

    def device_error(self) -> int:
        v = ctypes.c_int32(0)
        _check(load().ds_lora_get_device_error(_ref(self.plan), _ref(v), _stream(self.stream)), "ds_lora_get_device_error")
        return v.value


def ds_ragged_lora(plan: ds_lora_plan, lora: ds_lora_weights, x, base, out, stream=None):
    where = "ds_ragged_lora"
    n = plan.max_tokens if plan.flags & DS_META_CAPACITY else plan.n_tokens
    dt, here, wi, wo = lora.tensors[0].dtype, _current_device(), lora.in_dim, lora.out_dim
    strides = []
    for t, width in ((x, wi), (base, wo), (out, wo)):
        rows, cols = t.shape
        if not t.is_cuda or t.dtype is not dt or rows < n or cols != width or (t.stride(1) != 1 and cols != 1):
            raise DSError(DS_ERR_INVALID_ARG, where, "x, base and out must be CUDA tensors of the adapters' type and widths, "
                          "with a contiguous row for each token")
        if t.get_device() != here:
            _elsewhere(where, t.get_device())
        strides.append(t.stride(0) if rows != 1 else width)  # a tensor of one row may give any stride for it
    if getattr(lora, "device", here) != here:
        _elsewhere(where, lora.device)
    if getattr(plan, "device", here) != here:
        _elsewhere(where, plan.device)
    _check(load().ds_ragged_lora(_ref(plan), _ref(lora), x.data_ptr(), strides[0], base.data_ptr(), strides[1], out.data_ptr(),
                                 strides[2], _stream(stream)), where)


def make_logit_rules(history=None, history_len=None, prompt_len=None, repetition=None, frequency=None, presence=None,
                     bias_ids=None, bias_values=None, bias_len=None, mask=None, mask_row=None) -> ds_logit_rules:
    """ds_logit_rules of contiguous CUDA tensors: int32 history [sequences][ids] and bias_ids [sequences][pairs], float32
    bias_values as bias_ids, int32 mask [masks][words] of 32 bits; int32 history_len, prompt_len, bias_len, mask_row
    and float32 repetition, frequency, presence with a value for each sequence.  None leaves a rule out.  Keeps them
    alive."""
    import torch
    where = "make_logit_rules"
    given = dict(history=history, history_len=history_len, prompt_len=prompt_len, repetition=repetition, frequency=frequency,
                 presence=presence, bias_ids=bias_ids, bias_values=bias_values, bias_len=bias_len, mask=mask, mask_row=mask_row)
    rows = []
    for name, t in given.items():
        if t is None:
            continue
        want = torch.float32 if name in ("repetition", "frequency", "presence", "bias_values") else torch.int32
        dims = 2 if name in ("history", "bias_ids", "bias_values", "mask") else 1
        _require(t.is_cuda and t.is_contiguous() and t.dtype == want and len(t.shape) == dims, where,
                 "%s must be a contiguous CUDA tensor of %s in %d dimensions" % (name, want, dims))
        if name != "mask":
            rows.append(t.shape[0])
    width = lambda t: 0 if t is None else t.shape[1]  # noqa: E731
    _require((history is None) == (history_len is None), where, "history and history_len go together")
    _require(history is not None or (prompt_len is None and repetition is None and frequency is None and presence is None), where,
             "penalties need a history")
    _require((bias_ids is None) == (bias_values is None) and (bias_ids is None or tuple(bias_ids.shape) == tuple(bias_values.shape)),
             where, "bias_ids and bias_values go together, in one shape")
    _require(bias_len is None or bias_ids is not None, where, "bias_len needs bias_ids")
    _require(mask_row is None or mask is not None, where, "mask_row needs a mask")
    r = ds_logit_rules(_ptr(history), width(history), _ptr(history_len), _ptr(prompt_len), _ptr(repetition), _ptr(frequency),
                       _ptr(presence), _ptr(bias_ids), _ptr(bias_values), width(bias_ids), _ptr(bias_len), _ptr(mask),
                       width(mask), 0 if mask is None else mask.shape[0], _ptr(mask_row))
    r.tensors = given
    r.device = _device_of(where, *given.values())
    r.rows = min(rows, default=None)
    return r


def ds_ragged_adjust_logits(meta: ds_ragged_meta, logits, rules: ds_logit_rules, out, stream=None):
    """out: rows of logits' type and width; it may be logits itself."""
    import torch
    where = "ds_ragged_adjust_logits"
    rows, vocab = logits.shape
    n = meta.max_seqs if meta.flags & DS_META_CAPACITY else meta.n_seqs
    dt, here = logits.dtype, _current_device()
    kind = DS_FP32 if dt is torch.float32 else DS_BF16 if dt is torch.bfloat16 else DS_FP16 if dt is torch.float16 else None
    if kind is None:
        raise DSError(DS_ERR_INVALID_ARG, where, "logits must be of fp16, bf16 or fp32")
    for t in (logits, out):
        if not t.is_cuda or t.dtype is not dt or t.shape[1] != vocab or t.shape[0] < n or (vocab > 1 and t.stride(1) != 1):
            raise DSError(DS_ERR_INVALID_ARG, where, "logits and out must be CUDA tensors of one type and width, with a contiguous row for each sequence")
        if t.get_device() != here:
            _elsewhere(where, t.get_device())
    if getattr(rules, "device", None) not in (None, here):
        _elsewhere(where, rules.device)
    if getattr(rules, "rows", None) is not None and rules.rows < n:
        raise DSError(DS_ERR_INVALID_ARG, where, "%d sequences need as many rows of rules" % n)
    _check(load().ds_ragged_adjust_logits(_ref(meta), logits.data_ptr(), kind, vocab, logits.stride(0) if rows > 1 else vocab,
                                          _ref(rules), out.data_ptr(), out.stride(0) if out.shape[0] > 1 else vocab, _stream(stream)),
           where)


def make_sampler(uniforms, temperature=None, top_k=None, top_p=None, min_p=None) -> ds_sampler:
    """ds_sampler of CUDA tensors with a value for each sequence: float32, top_k
    int32; None leaves a setting off.  Keeps them alive."""
    import torch
    given = dict(uniforms=uniforms, temperature=temperature, top_k=top_k, top_p=top_p, min_p=min_p)
    for name, t in given.items():
        want = torch.int32 if name == "top_k" else torch.float32
        _require((t is None and name != "uniforms") or (t is not None and t.is_cuda and t.is_contiguous() and t.dtype == want),
                 "make_sampler", "%s must be a contiguous CUDA tensor of %s" % (name, want))
    sp = ds_sampler(*[_ptr(t) for t in given.values()])
    sp.tensors = given
    sp.device = _device_of("make_sampler", *given.values())
    sp.rows = min(t.numel() for t in given.values() if t is not None)
    return sp


def ds_ragged_sample(meta: ds_ragged_meta, logits, sampler: ds_sampler, out_tokens, out_logprobs=None, stream=None):
    import torch
    where = "ds_ragged_sample"
    rows, vocab = logits.shape
    n = meta.max_seqs if meta.flags & DS_META_CAPACITY else meta.n_seqs
    dt, here = logits.dtype, _current_device()
    kind = DS_FP32 if dt is torch.float32 else DS_BF16 if dt is torch.bfloat16 else DS_FP16 if dt is torch.float16 else None
    if kind is None or not logits.is_cuda or (vocab > 1 and logits.stride(1) != 1):
        raise DSError(DS_ERR_INVALID_ARG, where, "logits must be a CUDA tensor of fp16, bf16 or fp32 with contiguous rows")
    if logits.get_device() != here:
        _elsewhere(where, logits.get_device())
    for t, dt in ((out_tokens, torch.int32), (out_logprobs, torch.float32)):
        if t is None:
            continue
        if not (t.is_cuda and t.dtype is dt and t.is_contiguous() and t.numel() >= n):
            raise DSError(DS_ERR_INVALID_ARG, where, "outputs must be contiguous CUDA tensors (int32, float32) with a value for each sequence")
        if t.get_device() != here:
            _elsewhere(where, t.get_device())
    if getattr(sampler, "device", here) != here:
        _elsewhere(where, sampler.device)
    if rows < n or sampler.rows < n:
        raise DSError(DS_ERR_INVALID_ARG, where, "%d sequences need as many logits rows and settings" % n)
    _check(load().ds_ragged_sample(_ref(meta), logits.data_ptr(), kind, vocab, logits.stride(0) if rows > 1 else vocab,
                                   _ref(sampler), _ptr(out_tokens), _ptr(out_logprobs), _stream(stream)), where)


def ds_get_device_error(meta: ds_ragged_meta, stream=None) -> int:
    v = ctypes.c_int32(0)
    _check(load().ds_get_device_error(_ref(meta), _ref(v), _stream(stream)), "ds_get_device_error")
    return v.value


class BlockAllocator:
    """The C-ABI block ledger with its two host arrays."""

    def __init__(self, num_blocks: int, initial_order=None):
        self.stack = np.zeros(max(num_blocks, 1), np.int32)
        self.state = np.zeros(max(num_blocks, 1), np.uint8)
        self.a = ds_block_allocator()
        order = None if initial_order is None else np.ascontiguousarray(initial_order, np.int32)
        self._order = order
        _check(load().ds_block_allocator_init(_ref(self.a), self.stack.ctypes.data, self.state.ctypes.data,
                                              num_blocks, None if order is None else order.ctypes.data),
               "ds_block_allocator_init")

    @property
    def n_free(self) -> int:
        return self.a.n_free

    def allocate(self, n: int) -> np.ndarray:
        out = np.zeros(max(n, 1), np.int32)
        _check(load().ds_block_allocator_allocate(_ref(self.a), n, out.ctypes.data), "ds_block_allocator_allocate")
        return out[:n].copy()

    def free(self, ids) -> None:
        ids = np.ascontiguousarray(ids, np.int32)
        _check(load().ds_block_allocator_free(_ref(self.a), ids.ctypes.data if len(ids) else None, len(ids)),
               "ds_block_allocator_free")


def ds_kv_blocks_required(seen: int, new: int, owned: int, block_size: int = 64) -> int:
    e = ctypes.c_int32(0)
    _check(load().ds_kv_blocks_required(seen, new, owned, block_size, _ref(e)), "ds_kv_blocks_required")
    return e.value


# ------------------------------------------------------- buffer management --

class RaggedLayer:
    """Caller-side buffers for one layer shape and capacity (all allocated with
    torch), plus the three calls of a forward pass."""

    def __init__(self, params: ds_attn_params, max_seqs: int, max_tokens: int, max_blocks: int,
                 max_positions: int, device: str = "cuda", stream=None, workspace=None, flags: int = 0):
        import torch
        self.params = params
        self.device = device
        self.stream = stream
        dev_b, stg_b = ds_meta_buffer_sizes(max_seqs, max_tokens, max_blocks, params)
        self.meta_dev = torch.empty(dev_b, dtype=torch.uint8, device=device)
        self.meta_stage = torch.empty(stg_b, dtype=torch.uint8, pin_memory=True)
        self.meta = ds_meta_init(self.meta_dev, self.meta_stage, max_seqs, max_tokens, max_blocks)
        self.meta.flags = flags
        rb = ds_rope_table_size(params, max_positions)
        self.rope_buf = torch.empty(max(rb, 16), dtype=torch.uint8, device=device)
        self.rope = ds_rope_table_build(params, max_positions, self.rope_buf, stream)
        wb = ds_blocked_attention_workspace_size(params, max_seqs, max_tokens, max_blocks)
        # a caller may share one workspace between layers whose calls are ordered on one stream
        self.workspace = workspace if workspace is not None else torch.empty(wb, dtype=torch.uint8, device=device)
        self.fused_ws = None  # made (and its counters zeroed) on the first fused call

    def build(self, descs: SeqDescs, pool_num_blocks: int):
        ds_ragged_meta_build(descs, self.params, pool_num_blocks, self.meta, self.stream)

    def pack(self, descs: SeqDescs, pool_num_blocks: int):
        """Host half of build (validate and pack into the staging buffer; no
        upload): with DS_META_CAPACITY, what a captured graph's upload then
        copies for the next replay."""
        _check(ds_ragged_meta_pack(descs, self.params, pool_num_blocks, self.meta), "ds_ragged_meta_pack")

    def append(self, qkv, pool_t, q_out=None):
        pool = ds_kv_pool(pool_t.data_ptr(), pool_t.shape[0])
        ds_kv_rotary_append(self.meta, self.params, self.rope, qkv, q_out, pool, self.stream)

    def norm_append(self, norm: ds_qk_norm, qkv, pool_t, qkv_out=None, q_out=None):
        """append() of a layer that norms its query and key heads; attention()
        then takes qkv_out (which may be qkv itself) in the place of qkv."""
        ds_kv_norm_rotary_append(self.meta, self.params, self.rope, norm, qkv, qkv_out, q_out, None, self.stream, pool_t)

    def attention(self, qkv, pool_t, out):
        pool = ds_kv_pool(pool_t.data_ptr(), pool_t.shape[0])
        ds_blocked_attention(self.meta, self.params, self.rope, qkv, pool, out, self.workspace, self.stream)

    def append8(self, qkv, pool: ds_kv8_pool):
        """append() to an 8-bit pool (make_kv8_pool)."""
        ds_kv8_rotary_append(self.meta, self.params, self.rope, qkv, pool, self.stream)

    def attention8(self, qkv, pool: ds_kv8_pool, out):
        """attention() over an 8-bit pool."""
        ds_kv8_blocked_attention(self.meta, self.params, self.rope, qkv, pool, out, self.workspace, self.stream)

    def fused(self, qkv, pool_t, out):
        """Append + attention in one call (ds_fused_append_attention)."""
        import torch
        if self.fused_ws is None:
            m = self.meta
            fb = ds_fused_workspace_size(self.params, m.max_seqs, m.max_tokens, m.max_blocks)
            self.fused_ws = torch.empty(fb, dtype=torch.uint8, device=self.device)
            ds_fused_workspace_init(self.meta, self.params, self.fused_ws, self.stream)
        pool = ds_kv_pool(pool_t.data_ptr(), pool_t.shape[0])
        ds_fused_append_attention(self.meta, self.params, self.rope, qkv, pool, out, self.fused_ws, self.stream)

    def device_error(self) -> int:
        return ds_get_device_error(self.meta, self.stream)

    def read_meta(self) -> dict:
        """Copy the uploaded metadata back and split it into named arrays."""
        import torch
        n = self.meta.used_bytes
        raw = self.meta_dev[:n].cpu().numpy().view(np.int32)
        return unpack_meta(self.meta, raw, int(self.meta_dev.data_ptr()))


def ds_meta_init(dev_buf, staging, max_seqs: int, max_tokens: int, max_blocks: int) -> ds_ragged_meta:
    m = ds_ragged_meta()
    m.device_buf = _ptr(dev_buf)
    m.device_bytes = dev_buf.numel() * dev_buf.element_size() if hasattr(dev_buf, "numel") else dev_buf.nbytes
    m.host_staging = _ptr(staging)
    m.staging_bytes = staging.numel() * staging.element_size() if hasattr(staging, "numel") else staging.nbytes
    m.max_seqs, m.max_tokens, m.max_blocks = max_seqs, max_tokens, max_blocks
    return m


def unpack_meta(meta: ds_ragged_meta, words: np.ndarray, base_addr: int) -> dict:
    """Named views of a packed metadata image (staging or device copy)."""
    def at(ptr, count, width=1):
        off = (ptr - base_addr) // 4
        return words[off:off + count * width].reshape(-1, width) if width > 1 else words[off:off + count]
    S, N = meta.n_seqs, meta.n_tokens
    return dict(
        header=at(meta.header, 16),
        cu_seqlens=at(meta.cu_seqlens, S + 1), seq_seen=at(meta.seq_seen, S),
        seq_new=at(meta.seq_new, S), blk_off=at(meta.blk_off, S + 1),
        block_table=at(meta.block_table, meta.n_blocks), tok_seq=at(meta.tok_seq, N),
        tok_pos=at(meta.tok_pos, N),
        prefill_tiles=at(meta.prefill_tiles, meta.n_prefill_tiles, 4),
        decode_items=at(meta.decode_items, meta.n_decode_items, 4),
        decode_seqs=at(meta.decode_seqs, meta.n_decode_seqs, 4))
