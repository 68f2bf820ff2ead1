"""Thin ctypes binding of libmq (include/mq.h), same call names as the C ABI.

Argument marshalling only: every step of the compute path runs in the CUDA
kernels of libmq.so.  There is no CPU fallback: importing this module raises
if the in-tree library has not been built, and every compute call raises
``MQError`` on a non-zero status.

Raw calls (``mq_*``) take integer device addresses and a stream handle.
The tensor-level helpers below them (``quantize_q8_0``, ``matvec_q4K_q8_0``,
``ffn_gu_silu_down``, ``StepBuffers``) only compute pointers from torch
tensors, build the descriptor structs and upload them.
"""
from __future__ import annotations

import ctypes
import os
from typing import Dict, List, Optional, Sequence

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libmq.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"libmq.so is not built ({LIB_PATH}); run `python -c 'import __graft_entry__ as g; g.build()'`")

_lib = ctypes.CDLL(LIB_PATH)

c_i32 = ctypes.c_int32
c_i64 = ctypes.c_int64
c_u32 = ctypes.c_uint32
c_vp = ctypes.c_void_p

MQ_OK = 0
MQ_ERR_INVALID_ARG = 1
MQ_ERR_SHAPE = 2
MQ_ERR_ALIGN = 3
MQ_ERR_CUDA = 4
MQ_ERR_UNSUPPORTED = 5
MQ_ERR_NOT_INITIALIZED = 6
MQ_DEV_DESC_MISMATCH = 1
MQ_DEV_DESC_ALIGN = 2
MQ_DEV_TIMEOUT = 4
MQ_DEV_ALIAS = 8
MQ_DEV_KV_RANGE = 16
MQ_DEV_KV_FULL = 32
MQ_VARIANT_AUTO = 0
MQ_VARIANT_FORCE_REGISTER = 1
MQ_FAULT_NONE = 0
MQ_FAULT_WITHHOLD_TILE = 1
MQ_FAULT_WITHHOLD_RECORDS = 2
MQ_FAULT_WITHHOLD_COUNT = 3
MQ_TYPE_Q4_K = 1
MQ_TYPE_Q8_0 = 2
MQ_TYPE_Q4_0 = 3
MQ_TYPE_F16 = 4
MQ_MAX_NCOLS = 8
MQ_MAX_K = 131072
MQ_MAX_K_TIMES_NCOLS = 163840
MQ_STEP_PDL = 1
MQ_STEP_PERSISTENT = 2
MQ_STEP_CHAINED = 4
MQ_STEP_WORKSPACE_BYTES = 4352
MQ_NOALLOC_HQ8_MAX_BYTES = 131072
MQ_MMQ_MAX_NCOLS = 64
MQ_KV_PAGE_TOKENS = 64
MQ_TREE_MAX_TOKENS = 64
MQ_ROPE_INTERLEAVED = 1
MQ_MAX_SEQS = 4096
MQ_VERIFY_GREEDY = 1
MQ_PLAN_MATVEC = 0
MQ_PLAN_DOWN = 1
MQ_PLAN_GATE_UP = 2
MQ_PLAN_FIELDS = 20
MQ_STEP_PLAN_FIELDS = 8


class MvDesc(ctypes.Structure):
    _fields_ = [("W", c_vp), ("x", c_vp), ("xq", c_vp), ("xq_out", c_vp), ("y", c_vp),
                ("rows", c_i32), ("K", c_i32), ("ncols", c_i32), ("y_ld", c_i32)]


class FfnDesc(ctypes.Structure):
    _fields_ = [("W_gu", c_vp), ("W_down", c_vp), ("x", c_vp), ("xq", c_vp), ("h_q8", c_vp),
                ("gu_dbg", c_vp), ("h_dbg", c_vp), ("y", c_vp),
                ("H", c_i32), ("I", c_i32), ("ncols", c_i32), ("y_ld", c_i32)]


class LayerDesc(ctypes.Structure):
    _fields_ = [("qkv", MvDesc), ("o", MvDesc), ("ffn", FfnDesc)]


class StepShape(ctypes.Structure):
    _fields_ = [("n_layers", c_i32), ("H", c_i32), ("I", c_i32), ("qkv_rows", c_i32), ("o_rows", c_i32),
                ("o_K", c_i32), ("ncols", c_i32), ("flags", c_u32), ("workspace", c_vp)]


class KvCacheStruct(ctypes.Structure):
    _fields_ = [("pages", c_vp), ("table", c_vp), ("n_pages", c_i64), ("n_seqs", c_i32), ("table_ld", c_i32),
                ("type", c_i32), ("n_kv_heads", c_i32), ("head_dim", c_i32), ("reserved", c_i32)]


class KvAppendArgs(ctypes.Structure):
    _fields_ = [("qkv", c_vp), ("q_norm", c_vp), ("k_norm", c_vp), ("inv_freq", c_vp), ("pos", c_vp), ("seq", c_vp),
                ("slot", c_vp), ("q_out", c_vp), ("qkv_ld", c_i64), ("q_ld", c_i64), ("n_tokens", c_i32),
                ("n_heads", c_i32), ("rot_dims", c_i32), ("flags", c_u32), ("eps", ctypes.c_float),
                ("reserved", c_i32)]


class AttnArgs(ctypes.Structure):
    _fields_ = [("q", c_vp), ("out", c_vp), ("tok_start", c_vp), ("ctx_len", c_vp), ("mask", c_vp), ("q_ld", c_i64),
                ("out_ld", c_i64), ("n_tokens", c_i32), ("n_heads", c_i32), ("max_len", c_i32),
                ("max_tokens", c_i32), ("out_type", c_i32), ("scale", ctypes.c_float)]


class AttnGroups(ctypes.Structure):
    _fields_ = [("grp_start", c_vp), ("grp_pages", c_vp), ("n_groups", c_i32), ("max_pages", c_i32)]


class VerifyArgs(ctypes.Structure):
    _fields_ = [("target", c_vp), ("draft", c_vp), ("tok_start", c_vp), ("token", c_vp), ("parent", c_vp), ("u", c_vp),
                ("path", c_vp), ("n_path", c_vp), ("next", c_vp), ("target_ld", c_i64), ("draft_ld", c_i64),
                ("n_tokens", c_i32), ("n_seqs", c_i32), ("vocab", c_i32), ("path_ld", c_i32), ("flags", c_u32),
                ("reserved", c_i32)]


class KvPoolStruct(ctypes.Structure):
    _fields_ = [("refs", c_vp), ("free_list", c_vp), ("n_free", c_vp), ("seq_pages", c_vp), ("scratch", c_vp)]


def _sig(name, res, *args):
    f = getattr(_lib, name)
    f.restype = res
    f.argtypes = list(args)
    return f


_sig("mq_status_string", ctypes.c_char_p, c_i32)
_sig("mq_abi_version", c_i32)
_sig("mq_last_cuda_error", c_i32)
_sig("mq_init", c_i32, c_i32)
_sig("mq_read_device_status", c_i32, ctypes.POINTER(c_u32), c_vp)
_sig("mq_q4K_row_bytes", ctypes.c_size_t, c_i64)
_sig("mq_q8_0_bytes", ctypes.c_size_t, c_i64)
_sig("mq_quant_block_elems", c_i32, c_i32)
_sig("mq_quant_block_bytes", c_i32, c_i32)
_sig("mq_concat_rows_feasible", c_i32, c_i32, ctypes.POINTER(c_i32), ctypes.POINTER(c_i64),
     ctypes.POINTER(c_i64), ctypes.POINTER(ctypes.c_uint64))
_sig("mq_concat_rows", c_i32, c_vp, ctypes.POINTER(c_vp), ctypes.POINTER(c_i64), c_i32, c_i32, c_i64, c_vp)
_sig("mq_quantize_q8_0", c_i32, c_vp, c_vp, c_i64, c_i32, c_vp)
_sig("mq_check_mv_desc", c_i32, ctypes.POINTER(MvDesc))
_sig("mq_matvec_q4K_q8_0", c_i32, c_vp, c_i32, c_i32, c_i32, c_vp)
_sig("mq_matvec_q4_0_q8_0", c_i32, c_vp, c_i32, c_i32, c_i32, c_vp)
_sig("mq_matvec_q8_0_q8_0", c_i32, c_vp, c_i32, c_i32, c_i32, c_vp)
_sig("mq_check_ffn_desc", c_i32, ctypes.POINTER(FfnDesc))
_sig("mq_ffn_gu_silu_down", c_i32, c_vp, c_i32, c_i32, c_i32, c_vp)
_sig("mq_ffn_gate_up", c_i32, c_vp, c_i32, c_i32, c_i32, c_vp)
_sig("mq_step", c_i32, c_vp, ctypes.POINTER(StepShape), c_vp)
_sig("mq_step_workspace_bytes", c_i32, ctypes.POINTER(StepShape), ctypes.POINTER(ctypes.c_size_t))
_sig("mq_ffn_gu_silu_down_noalloc", c_i32, c_vp, c_vp, c_vp, c_vp, c_vp, c_i32, c_i32, c_i32, c_i32, c_vp)
_sig("mq_mmq_workspace_bytes", c_i32, c_i32, c_i32, c_i32, ctypes.POINTER(ctypes.c_size_t))
_sig("mq_mmq_q4K_q8_0", c_i32, c_vp, c_i32, c_i32, c_i32, c_vp, ctypes.c_size_t, c_vp)
_sig("mq_dequant_q4K_f16", c_i32, c_vp, c_vp, c_i64, c_i64, c_vp)
_sig("mq_convert_f32_f16", c_i32, c_vp, c_vp, c_i64, c_vp)
_sig("mq_gemm_f16", c_i32, c_vp, c_vp, c_vp, c_i32, c_i32, c_i32, c_vp)
_sig("mq_kv_page_bytes", ctypes.c_size_t, c_i32, c_i32, c_i32)
_sig("mq_check_kv_cache", c_i32, ctypes.POINTER(KvCacheStruct))
_sig("mq_kv_append", c_i32, ctypes.POINTER(KvCacheStruct), ctypes.POINTER(KvAppendArgs), c_vp)
_sig("mq_kv_read", c_i32, ctypes.POINTER(KvCacheStruct), c_vp, c_vp, c_i32, c_vp, c_vp, c_vp)
_sig("mq_kv_accept", c_i32, ctypes.POINTER(KvCacheStruct), c_vp, c_vp, c_vp, c_i32, c_vp)
_sig("mq_attn_workspace_bytes", c_i32, ctypes.POINTER(KvCacheStruct), c_i32, c_i32, ctypes.POINTER(ctypes.c_size_t))
_sig("mq_attn_tree", c_i32, ctypes.POINTER(KvCacheStruct), ctypes.POINTER(AttnArgs), c_vp, ctypes.c_size_t, c_vp)
_sig("mq_attn_shared_workspace_bytes", c_i32, ctypes.POINTER(KvCacheStruct), c_i32, c_i32, c_i32, c_i32,
     ctypes.POINTER(ctypes.c_size_t))
_sig("mq_attn_shared", c_i32, ctypes.POINTER(KvCacheStruct), ctypes.POINTER(AttnArgs), ctypes.POINTER(AttnGroups), c_vp,
     ctypes.c_size_t, c_vp)
_sig("mq_softmax", c_i32, c_vp, c_vp, c_i32, c_i32, c_i64, c_i64, ctypes.c_float, c_vp)
_sig("mq_verify_tree", c_i32, ctypes.POINTER(VerifyArgs), c_vp)
_sig("mq_kv_pool_scratch", c_i64, ctypes.POINTER(KvCacheStruct))
_sig("mq_kv_grow", c_i32, ctypes.POINTER(KvCacheStruct), ctypes.POINTER(KvPoolStruct), c_vp, c_vp)
_sig("mq_kv_fork", c_i32, ctypes.POINTER(KvCacheStruct), ctypes.POINTER(KvPoolStruct), c_vp, c_vp, c_vp, c_i32, c_vp)
_sig("mq_kv_free", c_i32, ctypes.POINTER(KvCacheStruct), ctypes.POINTER(KvPoolStruct), c_vp, c_vp, c_i32, c_vp)
_sig("mq_kv_compact", c_i32, ctypes.POINTER(KvCacheStruct), ctypes.POINTER(KvPoolStruct), c_vp)
_sig("mq_debug_block_sums_q4K_q8_0", c_i32, c_vp, c_i32, c_i32, c_i32, c_vp, c_vp, c_vp)
_sig("mq_debug_set_variant", c_i32, c_i32)
_sig("mq_debug_set_fault", c_i32, c_i32)
_sig("mq_debug_plan_mv", c_i32, c_i32, c_i64, c_i32, c_i32, c_i32, c_i32, c_i64, c_i32, ctypes.POINTER(c_i64), c_i32)
_sig("mq_debug_plan_step", c_i32, ctypes.POINTER(StepShape), c_i32, c_i64, c_i32, ctypes.POINTER(c_i64), c_i32)

# the exported names, one per declaration in include/mq.h
EXPORTS = ["mq_status_string", "mq_abi_version", "mq_last_cuda_error", "mq_init", "mq_read_device_status",
           "mq_q4K_row_bytes", "mq_q8_0_bytes", "mq_quant_block_elems", "mq_quant_block_bytes",
           "mq_concat_rows_feasible", "mq_concat_rows", "mq_quantize_q8_0", "mq_check_mv_desc",
           "mq_matvec_q4K_q8_0", "mq_matvec_q4_0_q8_0", "mq_matvec_q8_0_q8_0", "mq_check_ffn_desc", "mq_ffn_gu_silu_down", "mq_ffn_gate_up", "mq_step", "mq_step_workspace_bytes",
           "mq_ffn_gu_silu_down_noalloc", "mq_dequant_q4K_f16", "mq_convert_f32_f16", "mq_gemm_f16",
           "mq_mmq_workspace_bytes", "mq_mmq_q4K_q8_0",
           "mq_kv_page_bytes", "mq_check_kv_cache", "mq_kv_append", "mq_kv_read", "mq_kv_accept",
           "mq_attn_workspace_bytes", "mq_attn_tree",
           "mq_attn_shared_workspace_bytes", "mq_attn_shared", "mq_softmax", "mq_verify_tree", "mq_kv_pool_scratch",
           "mq_kv_grow", "mq_kv_fork", "mq_kv_free", "mq_kv_compact",
           "mq_debug_block_sums_q4K_q8_0", "mq_debug_set_variant", "mq_debug_set_fault", "mq_debug_plan_mv",
           "mq_debug_plan_step"]


class MQError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = f"{where}: {mq_status_string(status)} (status {status})"
        if status == MQ_ERR_CUDA:
            msg += f", cudaError {mq_last_cuda_error()}"
        super().__init__(msg)


def status_string(s: int) -> str:
    return _lib.mq_status_string(s).decode()


# ---- raw calls, same names as the C ABI -------------------------------------------------------------

def mq_status_string(s: int) -> str:
    return status_string(s)


def mq_abi_version() -> int:
    return _lib.mq_abi_version()


def mq_last_cuda_error() -> int:
    return _lib.mq_last_cuda_error()


def mq_init(device: int) -> int:
    return _lib.mq_init(device)


def mq_read_device_status(stream: int = 0) -> int:
    v = c_u32(0)
    _check(_lib.mq_read_device_status(ctypes.byref(v), c_vp(stream)), "mq_read_device_status")
    return v.value


def mq_q4K_row_bytes(K: int) -> int:
    return _lib.mq_q4K_row_bytes(K)


def mq_q8_0_bytes(K: int) -> int:
    return _lib.mq_q8_0_bytes(K)


def mq_quant_block_elems(t: int) -> int:
    return _lib.mq_quant_block_elems(t)


def mq_quant_block_bytes(t: int) -> int:
    return _lib.mq_quant_block_bytes(t)


def mq_concat_rows_feasible(ttypes: Sequence[int], ne0: Sequence[int], ne1: Sequence[int],
                            nbytes: Sequence[int]) -> bool:
    n = len(ttypes)
    if not (len(ne0) == len(ne1) == len(nbytes) == n):
        return False
    A = lambda ct, v: (ct * n)(*v)
    return bool(_lib.mq_concat_rows_feasible(n, A(c_i32, ttypes), A(c_i64, ne0), A(c_i64, ne1),
                                             A(ctypes.c_uint64, nbytes)))


def mq_concat_rows(dst: int, srcs: Sequence[int], rows: Sequence[int], ttype: int, ne0: int,
                   stream: int = 0) -> int:
    n = len(srcs)
    return _lib.mq_concat_rows(c_vp(dst), (c_vp * n)(*srcs), (c_i64 * n)(*rows), n, ttype, ne0, c_vp(stream))


def mq_quantize_q8_0(x: int, xq: int, K: int, ncols: int, stream: int = 0) -> int:
    return _lib.mq_quantize_q8_0(c_vp(x), c_vp(xq), K, ncols, c_vp(stream))


def mq_check_mv_desc(d: MvDesc) -> int:
    return _lib.mq_check_mv_desc(ctypes.byref(d))


def mq_matvec_q4K_q8_0(d_desc: int, rows: int, K: int, ncols: int, stream: int = 0) -> int:
    return _lib.mq_matvec_q4K_q8_0(c_vp(d_desc), rows, K, ncols, c_vp(stream))


def mq_matvec_q4_0_q8_0(d_desc: int, rows: int, K: int, ncols: int, stream: int = 0) -> int:
    return _lib.mq_matvec_q4_0_q8_0(c_vp(d_desc), rows, K, ncols, c_vp(stream))


def mq_matvec_q8_0_q8_0(d_desc: int, rows: int, K: int, ncols: int, stream: int = 0) -> int:
    return _lib.mq_matvec_q8_0_q8_0(c_vp(d_desc), rows, K, ncols, c_vp(stream))


def mq_check_ffn_desc(d: FfnDesc) -> int:
    return _lib.mq_check_ffn_desc(ctypes.byref(d))


def mq_ffn_gu_silu_down(d_desc: int, H: int, I: int, ncols: int, stream: int = 0) -> int:
    return _lib.mq_ffn_gu_silu_down(c_vp(d_desc), H, I, ncols, c_vp(stream))


def mq_ffn_gate_up(d_desc: int, H: int, I: int, ncols: int, stream: int = 0) -> int:
    return _lib.mq_ffn_gate_up(c_vp(d_desc), H, I, ncols, c_vp(stream))


def mq_step(d_layers: int, shape: StepShape, stream: int = 0) -> int:
    return _lib.mq_step(c_vp(d_layers), ctypes.byref(shape), c_vp(stream))


def mq_step_workspace_bytes(shape: StepShape) -> int:
    n = ctypes.c_size_t(0)
    _check(_lib.mq_step_workspace_bytes(ctypes.byref(shape), ctypes.byref(n)), "mq_step_workspace_bytes")
    return int(n.value)


def mq_ffn_gu_silu_down_noalloc(W_gu: int, W_down: int, x: int, xq: int, y: int, H: int, I: int, ncols: int,
                                y_ld: int, stream: int = 0) -> int:
    return _lib.mq_ffn_gu_silu_down_noalloc(c_vp(W_gu), c_vp(W_down), c_vp(x), c_vp(xq), c_vp(y), H, I, ncols,
                                            y_ld, c_vp(stream))


def mq_mmq_workspace_bytes(rows: int, K: int, ncols: int) -> int:
    n = ctypes.c_size_t(0)
    _check(_lib.mq_mmq_workspace_bytes(rows, K, ncols, ctypes.byref(n)), "mq_mmq_workspace_bytes")
    return int(n.value)


def mq_mmq_q4K_q8_0(d_desc: int, rows: int, K: int, ncols: int, workspace: int, ws_bytes: int,
                    stream: int = 0) -> int:
    return _lib.mq_mmq_q4K_q8_0(c_vp(d_desc), rows, K, ncols, c_vp(workspace), ws_bytes, c_vp(stream))


def mq_dequant_q4K_f16(W: int, W16: int, rows: int, K: int, stream: int = 0) -> int:
    return _lib.mq_dequant_q4K_f16(c_vp(W), c_vp(W16), rows, K, c_vp(stream))


def mq_convert_f32_f16(x: int, y: int, n: int, stream: int = 0) -> int:
    return _lib.mq_convert_f32_f16(c_vp(x), c_vp(y), n, c_vp(stream))


def mq_gemm_f16(W16: int, X16: int, Y: int, R: int, K: int, T: int, stream: int = 0) -> int:
    return _lib.mq_gemm_f16(c_vp(W16), c_vp(X16), c_vp(Y), R, K, T, c_vp(stream))


def mq_kv_page_bytes(ttype: int, n_kv_heads: int, head_dim: int) -> int:
    return _lib.mq_kv_page_bytes(ttype, n_kv_heads, head_dim)


def mq_check_kv_cache(cache: KvCacheStruct) -> int:
    return _lib.mq_check_kv_cache(cache)


def mq_kv_append(cache: KvCacheStruct, args: KvAppendArgs, stream: int = 0) -> int:
    return _lib.mq_kv_append(cache, args, stream)


def mq_kv_read(cache: KvCacheStruct, seq: int, slot: int, n: int, k_out: int, v_out: int, stream: int = 0) -> int:
    return _lib.mq_kv_read(cache, seq, slot, n, k_out, v_out, stream)


def mq_kv_accept(cache: KvCacheStruct, ctx_len: int, path: int, n_path: int, path_ld: int, stream: int = 0) -> int:
    return _lib.mq_kv_accept(cache, ctx_len, path, n_path, path_ld, stream)


def mq_attn_workspace_bytes(cache: KvCacheStruct, n_heads: int, max_tokens: int) -> int:
    n = ctypes.c_size_t(0)
    _check(_lib.mq_attn_workspace_bytes(cache, n_heads, max_tokens, ctypes.byref(n)), "mq_attn_workspace_bytes")
    return int(n.value)


def mq_attn_tree(cache: KvCacheStruct, args: AttnArgs, workspace: int, ws_bytes: int, stream: int = 0) -> int:
    return _lib.mq_attn_tree(cache, args, workspace, ws_bytes, stream)


def mq_attn_shared_workspace_bytes(cache: KvCacheStruct, n_heads: int, n_tokens: int, max_tokens: int, n_groups: int) -> int:
    n = ctypes.c_size_t()
    _check(_lib.mq_attn_shared_workspace_bytes(cache, n_heads, n_tokens, max_tokens, n_groups, ctypes.byref(n)),
           "mq_attn_shared_workspace_bytes")
    return n.value


def mq_attn_shared(cache: KvCacheStruct, args: AttnArgs, groups: AttnGroups, workspace: int, ws_bytes: int,
                   stream: int = 0) -> int:
    return _lib.mq_attn_shared(cache, args, groups, workspace, ws_bytes, stream)


def mq_softmax(x: int, y: int, rows: int, vocab: int, x_ld: int, y_ld: int, scale: float, stream: int = 0) -> int:
    return _lib.mq_softmax(x, y, rows, vocab, x_ld, y_ld, scale, stream)


def mq_verify_tree(args: VerifyArgs, stream: int = 0) -> int:
    return _lib.mq_verify_tree(args, stream)


def mq_kv_pool_scratch(cache: KvCacheStruct) -> int:
    return _lib.mq_kv_pool_scratch(cache)


def mq_kv_grow(cache: KvCacheStruct, pool: KvPoolStruct, length: int, stream: int = 0) -> int:
    return _lib.mq_kv_grow(cache, pool, length, stream)


def mq_kv_fork(cache: KvCacheStruct, pool: KvPoolStruct, src: int, dst: int, length: int, n: int, stream: int = 0) -> int:
    return _lib.mq_kv_fork(cache, pool, src, dst, length, n, stream)


def mq_kv_free(cache: KvCacheStruct, pool: KvPoolStruct, seq: int, keep: int, n: int, stream: int = 0) -> int:
    return _lib.mq_kv_free(cache, pool, seq, keep, n, stream)


def mq_kv_compact(cache: KvCacheStruct, pool: KvPoolStruct, stream: int = 0) -> int:
    return _lib.mq_kv_compact(cache, pool, stream)


def mq_debug_block_sums_q4K_q8_0(d_desc: int, rows: int, K: int, ncols: int, sumi: int, sumq: int,
                                 stream: int = 0) -> int:
    return _lib.mq_debug_block_sums_q4K_q8_0(c_vp(d_desc), rows, K, ncols, c_vp(sumi), c_vp(sumq), c_vp(stream))


def mq_debug_set_variant(policy: int) -> int:
    return _lib.mq_debug_set_variant(policy)


def mq_debug_set_fault(fault: int) -> int:
    return _lib.mq_debug_set_fault(fault)


# the planner's fields, in the order mq.h gives them
PLAN_FIELDS = ("variant", "grid", "block", "smem", "C", "L", "S", "nseg", "nwc", "rg", "T", "ns", "stage_bytes",
               "rows_per_cta", "cmap", "cgw", "cgu", "hu", "ksplit", "kpn")
STEP_PLAN_FIELDS = ("grid", "block", "smem", "nwc", "ns", "stage_bytes", "pf_tiles", "ws_bytes")
PHASES = ("qkv", "o", "gu", "down")


def mq_debug_plan_mv(kind: int, rows: int, K: int, ncols: int, I: int, num_sms: int, l2_bytes: int,
                     max_smem: int, out, n_out: int) -> int:
    return _lib.mq_debug_plan_mv(kind, rows, K, ncols, I, num_sms, l2_bytes, max_smem, out, n_out)


def mq_debug_plan_step(shape: StepShape, num_sms: int, l2_bytes: int, max_smem: int, out, n_out: int) -> int:
    return _lib.mq_debug_plan_step(ctypes.byref(shape), num_sms, l2_bytes, max_smem, out, n_out)


def debug_plan_mv(kind: int, rows: int, K: int, ncols: int, I: int = 0, *, num_sms: int, l2_bytes: int,
                  max_smem: int) -> dict:
    """The plan a q4_K projection call takes on the stated device (host only), as a dict."""
    out = (c_i64 * MQ_PLAN_FIELDS)()
    _check(mq_debug_plan_mv(kind, rows, K, ncols, I, num_sms, l2_bytes, max_smem, out, MQ_PLAN_FIELDS),
           "mq_debug_plan_mv")
    return dict(zip(PLAN_FIELDS, list(out)))


def debug_plan_step(shape: StepShape, *, num_sms: int, l2_bytes: int, max_smem: int) -> dict:
    """The persistent step's plan on the stated device (host only): the kernel's fields and one
    dict per phase under "qkv", "o", "gu", "down"."""
    n = MQ_STEP_PLAN_FIELDS + 4 * MQ_PLAN_FIELDS
    out = (c_i64 * n)()
    _check(mq_debug_plan_step(shape, num_sms, l2_bytes, max_smem, out, n), "mq_debug_plan_step")
    v = list(out)
    d = dict(zip(STEP_PLAN_FIELDS, v[:MQ_STEP_PLAN_FIELDS]))
    for i, ph in enumerate(PHASES):
        o = MQ_STEP_PLAN_FIELDS + i * MQ_PLAN_FIELDS
        d[ph] = dict(zip(PLAN_FIELDS, v[o:o + MQ_PLAN_FIELDS]))
    return d


def _check(st: int, where: str):
    if st != MQ_OK:
        raise MQError(st, where)


# ---- tensor-level marshalling (torch owns memory and streams) ------------------------------------------

_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _ptr(t) -> int:
    return 0 if t is None else t.data_ptr()


def _stream(stream) -> int:
    torch = _torch()
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


_initialized = set()


def init(device: Optional[int] = None) -> None:
    """mq_init for a device (default: torch's current device), once."""
    torch = _torch()
    dev = torch.cuda.current_device() if device is None else int(device)
    if dev in _initialized:
        return
    torch.cuda.init()
    _check(mq_init(dev), "mq_init")
    _initialized.add(dev)


def upload_struct(s: ctypes.Structure, device) -> "torch.Tensor":
    """Copy a descriptor struct to a new device buffer (8-byte aligned)."""
    torch = _torch()
    raw = bytes(s) if not isinstance(s, (bytes, bytearray)) else s
    host = torch.frombuffer(bytearray(raw), dtype=torch.uint8)
    return host.to(device)


def quantize_q8_0(x, out=None, stream=None):
    """fp32 [ncols, K] cuda tensor -> uint8 [ncols, K/32*34] q8_0."""
    torch = _torch()
    x2 = x if x.dim() == 2 else x.reshape(1, -1)
    ncols, K = x2.shape
    if out is None:
        out = torch.empty((ncols, K // 32 * 34), dtype=torch.uint8, device=x.device)
    _check(mq_quantize_q8_0(_ptr(x2), _ptr(out), K, ncols, _stream(stream)), "mq_quantize_q8_0")
    return out


def mv_desc(W, rows: int, K: int, y, x=None, xq=None, xq_out=None, ncols: int = 1,
            y_ld: Optional[int] = None) -> MvDesc:
    return MvDesc(_ptr(W), _ptr(x), _ptr(xq), _ptr(xq_out), _ptr(y), rows, K, ncols,
                  rows if y_ld is None else y_ld)


def matvec_q4K_q8_0(W, rows: int, K: int, x=None, xq=None, y=None, xq_out=None, ncols: Optional[int] = None,
                    stream=None):
    """y [ncols, rows] fp32 = W . q8_0(x) (or W . xq).  Returns (y, desc_buffer)."""
    torch = _torch()
    act = x if x is not None else xq
    if ncols is None:
        ncols = act.shape[0] if act.dim() == 2 else 1
    if y is None:
        y = torch.empty((ncols, rows), dtype=torch.float32, device=W.device)
    d = mv_desc(W, rows, K, y, x=x, xq=xq, xq_out=xq_out, ncols=ncols, y_ld=y.shape[-1])
    _check(mq_check_mv_desc(d), "mq_check_mv_desc")
    dd = upload_struct(d, W.device)
    _check(mq_matvec_q4K_q8_0(_ptr(dd), rows, K, ncols, _stream(stream)), "mq_matvec_q4K_q8_0")
    return y, dd


def matvec_w(wtype: str, W, rows: int, K: int, x=None, xq=None, y=None, ncols: Optional[int] = None, stream=None):
    """y [ncols, rows] fp32 = W . q8_0(x) (or W . xq) for q4_0 (``wtype="q4_0"``) or q8_0
    (``"q8_0"``) weights.  Returns (y, desc_buffer)."""
    torch = _torch()
    act = x if x is not None else xq
    if ncols is None:
        ncols = act.shape[0] if act.dim() == 2 else 1
    if y is None:
        y = torch.empty((ncols, rows), dtype=torch.float32, device=W.device)
    d = mv_desc(W, rows, K, y, x=x, xq=xq, ncols=ncols, y_ld=y.shape[-1])
    _check(mq_check_mv_desc(d), "mq_check_mv_desc")
    dd = upload_struct(d, W.device)
    fn = {"q4_0": mq_matvec_q4_0_q8_0, "q8_0": mq_matvec_q8_0_q8_0}[wtype]
    _check(fn(_ptr(dd), rows, K, ncols, _stream(stream)), f"mq_matvec_{wtype}_q8_0")
    return y, dd


def block_sums(W, rows: int, K: int, x=None, xq=None, ncols: Optional[int] = None, stream=None):
    """Test export: (sumi int32 [ncols, rows, K/32], sumq int32 [ncols, K/32])."""
    torch = _torch()
    act = x if x is not None else xq
    if ncols is None:
        ncols = act.shape[0] if act.dim() == 2 else 1
    y = torch.empty((ncols, rows), dtype=torch.float32, device=W.device)
    d = mv_desc(W, rows, K, y, x=x, xq=xq, ncols=ncols)
    _check(mq_check_mv_desc(d), "mq_check_mv_desc")
    dd = upload_struct(d, W.device)
    sumi = torch.empty((ncols, rows, K // 32), dtype=torch.int32, device=W.device)
    sumq = torch.empty((ncols, K // 32), dtype=torch.int32, device=W.device)
    _check(mq_debug_block_sums_q4K_q8_0(_ptr(dd), rows, K, ncols, _ptr(sumi), _ptr(sumq), _stream(stream)),
           "mq_debug_block_sums_q4K_q8_0")
    return sumi, sumq


def ffn_desc(W_gu, W_down, H: int, I: int, h_q8, y, x=None, xq=None, gu_dbg=None, h_dbg=None, ncols: int = 1,
             y_ld: Optional[int] = None) -> FfnDesc:
    return FfnDesc(_ptr(W_gu), _ptr(W_down), _ptr(x), _ptr(xq), _ptr(h_q8), _ptr(gu_dbg), _ptr(h_dbg), _ptr(y),
                   H, I, ncols, H if y_ld is None else y_ld)


def ffn_gu_silu_down(W_gu, W_down, H: int, I: int, x=None, xq=None, debug: bool = False, stream=None):
    """Fused FFN.  Returns dict with y [ncols, H], h_q8 and (debug) gu, h, plus the descriptor buffer."""
    torch = _torch()
    act = x if x is not None else xq
    ncols = act.shape[0] if act.dim() == 2 else 1
    dev = W_gu.device
    out = {
        "y": torch.empty((ncols, H), dtype=torch.float32, device=dev),
        "h_q8": torch.empty((ncols, I // 32 * 34), dtype=torch.uint8, device=dev),
    }
    if debug:
        out["gu"] = torch.empty((ncols, 2 * I), dtype=torch.float32, device=dev)
        out["h"] = torch.empty((ncols, I), dtype=torch.float32, device=dev)
    d = ffn_desc(W_gu, W_down, H, I, out["h_q8"], out["y"], x=x, xq=xq, gu_dbg=out.get("gu"), h_dbg=out.get("h"),
                 ncols=ncols)
    _check(mq_check_ffn_desc(d), "mq_check_ffn_desc")
    out["desc"] = upload_struct(d, dev)
    _check(mq_ffn_gu_silu_down(_ptr(out["desc"]), H, I, ncols, _stream(stream)), "mq_ffn_gu_silu_down")
    return out


def ffn_gu_silu_down_noalloc(W_gu, W_down, H: int, I: int, x=None, xq=None, y=None, stream=None):
    """mq_ffn_gu_silu_down_noalloc: the fused FFN with the library's own fixed
    scratch instead of a caller-owned h_q8 and descriptor.  Returns y [ncols, H]
    (allocated here by torch unless given)."""
    torch = _torch()
    act = x if x is not None else xq
    ncols = act.shape[0] if act.dim() == 2 else 1
    if y is None:
        y = torch.empty((ncols, H), dtype=torch.float32, device=W_gu.device)
    _check(mq_ffn_gu_silu_down_noalloc(_ptr(W_gu), _ptr(W_down), _ptr(x), _ptr(xq), _ptr(y), H, I, ncols,
                                       y.shape[-1], _stream(stream)), "mq_ffn_gu_silu_down_noalloc")
    return y


def mmq_q4K_q8_0(W, rows: int, K: int, x=None, xq=None, y=None, xq_out=None, ncols: Optional[int] = None,
                 workspace=None, stream=None):
    """The matmul for more columns on the tensor cores: y [ncols, rows] fp32 = W . q8_0(x) (or W . xq).
    Returns (y, desc_buffer, workspace)."""
    torch = _torch()
    act = x if x is not None else xq
    if ncols is None:
        ncols = act.shape[0] if act.dim() == 2 else 1
    if y is None:
        y = torch.empty((ncols, rows), dtype=torch.float32, device=W.device)
    nbytes = mq_mmq_workspace_bytes(rows, K, ncols)
    if workspace is None:
        workspace = torch.empty(max(nbytes, 128), dtype=torch.uint8, device=W.device)
    d = mv_desc(W, rows, K, y, x=x, xq=xq, xq_out=xq_out, ncols=ncols, y_ld=y.shape[-1])
    dd = upload_struct(d, W.device)
    _check(mq_mmq_q4K_q8_0(_ptr(dd), rows, K, ncols, _ptr(workspace), workspace.numel(), _stream(stream)),
           "mq_mmq_q4K_q8_0")
    return y, dd, workspace


def dequant_q4K_f16(W, rows: int, K: int, out=None, stream=None):
    """The resident f16 weight cache: uint8 q4_K [rows, K/256*144] -> f16 [rows, K]."""
    torch = _torch()
    if out is None:
        out = torch.empty((rows, K), dtype=torch.float16, device=W.device)
    _check(mq_dequant_q4K_f16(_ptr(W), _ptr(out), rows, K, _stream(stream)), "mq_dequant_q4K_f16")
    return out


def convert_f32_f16(x, out=None, stream=None):
    """fp32 tensor -> f16 tensor of the same shape (round to nearest-even)."""
    torch = _torch()
    if out is None:
        out = torch.empty(x.shape, dtype=torch.float16, device=x.device)
    _check(mq_convert_f32_f16(_ptr(x), _ptr(out), x.numel(), _stream(stream)), "mq_convert_f32_f16")
    return out


def gemm_f16(W16, X16, out=None, stream=None):
    """Prefill GEMM on the tensor cores: Y [T, R] fp32 = X16 [T, K] . W16 [R, K]^T."""
    torch = _torch()
    R, K = W16.shape
    T = X16.shape[0]
    if out is None:
        out = torch.empty((T, R), dtype=torch.float32, device=W16.device)
    _check(mq_gemm_f16(_ptr(W16), _ptr(X16), _ptr(out), R, K, T, _stream(stream)), "mq_gemm_f16")
    return out


KV_TYPES = {"f16": MQ_TYPE_F16, "q8_0": MQ_TYPE_Q8_0}


def _want(t, name: str, dtype, shape=None, device=None):
    """Address of a tensor; refuses one that the raw call would misread (the C ABI sees addresses only)."""
    if t.dtype is not dtype or not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous {dtype} tensor is wanted, got {t.dtype} with strides {t.stride()}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name}: shape {shape} is wanted, got {tuple(t.shape)}")
    if device is not None and t.device != device:
        raise ValueError(f"{name}: on {t.device}, the cache is on {device}")
    return t.data_ptr()


def _rows(t, name: str, dtype, device, width: int, n: Optional[int] = None):
    """Address and row stride of a 2-D tensor with dense rows of ``width`` (the row stride is free)."""
    if t.dtype is not dtype or t.dim() != 2 or t.device != device:
        raise ValueError(f"{name}: a 2-D {dtype} tensor on {device} is wanted, got {t.dtype} {tuple(t.shape)} on {t.device}")
    rows, cols = t.shape
    if cols != width or (n is not None and rows != n):
        raise ValueError(f"{name}: rows of {width}{'' if n is None else f', {n} of them,'} are wanted, got {tuple(t.shape)}")
    if t.is_contiguous():
        return t.data_ptr(), cols
    if t.stride(1) != 1 and cols > 1:
        raise ValueError(f"{name}: dense rows are wanted, got strides {t.stride()}")
    return t.data_ptr(), t.stride(0)


def _new(shape, dtype, device, stream):
    """A tensor for the call's result, allocated on the stream that will write it."""
    torch = _torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    on = torch.cuda.ExternalStream(stream, device=device) if isinstance(stream, int) else stream
    with torch.cuda.stream(on):
        return torch.empty(shape, dtype=dtype, device=device)


def _stream_on(stream, device, what: str = "the cache is") -> int:
    """The stream handle of a call on ``device`` (None: torch's current stream there).  The library launches on the
    current CUDA device, so a call whose memory is anywhere else is refused."""
    torch = _torch()
    if device.type != "cuda" or torch.cuda.current_device() != device.index:
        raise ValueError(f"{what} on {device}: the current CUDA device is wanted")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device.index)
    if isinstance(stream, int):
        return stream
    if stream.device != device:
        raise ValueError(f"a stream of {stream.device}, {what} on {device}")
    return stream.cuda_stream


class KVCache:
    """A paged key/value cache (mq_kv_cache): the page pool and the page table.

    ``pages``: uint8 cuda tensor of n_pages * mq_kv_page_bytes bytes; ``table``: int32
    [n_seqs, pages per sequence].  ``type`` is "f16" or "q8_0".  The tensors are the
    caller's; the handle keeps references to them.  Calls on a cache are made with its device current.
    """

    def __init__(self, pages, table, type: str, n_kv_heads: int, head_dim: int):
        torch = _torch()
        self.type_name, self.n_kv_heads, self.head_dim = type, n_kv_heads, head_dim
        self.pages, self.table, self.device = pages, table, pages.device
        if type not in KV_TYPES:
            raise ValueError(f"cache type {type!r}: one of {sorted(KV_TYPES)}")
        page = mq_kv_page_bytes(KV_TYPES[type], n_kv_heads, head_dim)
        if not page:
            raise MQError(MQ_ERR_SHAPE, "mq_kv_page_bytes")
        if table.dim() != 2:
            raise ValueError("table: a 2-D tensor is wanted")
        if pages.numel() % page:
            raise ValueError(f"pages: {pages.numel()} bytes are no whole number of {page}-byte pages")
        self.n_seqs = table.shape[0]
        self.struct = KvCacheStruct(_want(pages, "pages", torch.uint8), _want(table, "table", torch.int32, device=pages.device),
                                    pages.numel() // page, table.shape[0], table.shape[1], KV_TYPES[type], n_kv_heads,
                                    head_dim, 0)
        _check(mq_check_kv_cache(self.struct), "mq_check_kv_cache")

    @classmethod
    def alloc(cls, n_pages: int, table, type: str, n_kv_heads: int, head_dim: int) -> "KVCache":
        """A cache with a new (unwritten) pool of n_pages pages."""
        torch = _torch()
        page = mq_kv_page_bytes(KV_TYPES.get(type, 0), n_kv_heads, head_dim)
        if not page:
            raise MQError(MQ_ERR_SHAPE, "mq_kv_page_bytes")
        return cls(torch.empty(n_pages * page, dtype=torch.uint8, device=table.device), table, type, n_kv_heads, head_dim)


def kv_append(cache: KVCache, qkv, pos, seq, slot, n_heads: int, inv_freq=None, interleaved: bool = False,
              q_norm=None, k_norm=None, eps: float = 1e-6, q_out=None, stream=None):
    """Norms and rotation of y_qkv [n, (n_heads + 2 n_kv_heads) * head_dim] (fp32, rows may be strided), K and V into
    the cache.  Returns q, f16 [n, n_heads * head_dim].  rot_dims is twice inv_freq's length (None: no rotation, and
    pos is not read)."""
    torch = _torch()
    dev, D, i32, f32 = cache.device, cache.head_dim, torch.int32, torch.float32
    width = n_heads * D
    x, ld = _rows(qkv, "qkv", f32, dev, width + 2 * cache.n_kv_heads * D)
    n = qkv.shape[0]
    if q_out is None:
        q_out = _new((n, width), torch.float16, dev, stream)
        q, q_ld = q_out.data_ptr(), width
    else:
        q, q_ld = _rows(q_out, "q_out", torch.float16, dev, width, n)
    rot, f, at = 0, None, None
    if inv_freq is not None and inv_freq.numel():
        rot, f = 2 * inv_freq.numel(), _want(inv_freq, "inv_freq", f32, None, dev)
        at = _want(pos, "pos", i32, (n,), dev)
    a = KvAppendArgs(x, None if q_norm is None else _want(q_norm, "q_norm", f32, (D,), dev),
                     None if k_norm is None else _want(k_norm, "k_norm", f32, (D,), dev), f, at,
                     _want(seq, "seq", i32, (n,), dev), _want(slot, "slot", i32, (n,), dev), q, ld, q_ld,
                     n, n_heads, rot, MQ_ROPE_INTERLEAVED if interleaved else 0, eps, 0)
    st = _lib.mq_kv_append(cache.struct, a, _stream_on(stream, dev))
    if st:
        raise MQError(st, "mq_kv_append")
    return q_out


def kv_read(cache: KVCache, seq, slot, k_out=None, v_out=None, stream=None):
    """Cached keys and values of (sequence, slot) pairs: two f16 tensors [n, n_kv_heads, head_dim]."""
    torch = _torch()
    n, dev, i32 = seq.numel(), cache.device, torch.int32
    shape = (n, cache.n_kv_heads, cache.head_dim)
    k_out = _new(shape, torch.float16, dev, stream) if k_out is None else k_out
    v_out = _new(shape, torch.float16, dev, stream) if v_out is None else v_out
    st = _lib.mq_kv_read(cache.struct, _want(seq, "seq", i32, (n,), dev), _want(slot, "slot", i32, (n,), dev), n,
                         _want(k_out, "k_out", torch.float16, shape, dev),
                         _want(v_out, "v_out", torch.float16, shape, dev), _stream_on(stream, dev))
    if st:
        raise MQError(st, "mq_kv_read")
    return k_out, v_out


def kv_accept(cache: KVCache, ctx_len, path, n_path, stream=None) -> None:
    """Move each sequence's accepted nodes path[s, :n_path[s]] to the slots from ctx_len[s] on."""
    i32, dev, S = _torch().int32, cache.device, cache.n_seqs
    if path.dim() != 2 or path.shape[0] != S:
        raise ValueError(f"path: [{S}, path_ld] is wanted, got {tuple(path.shape)}")
    st = _lib.mq_kv_accept(cache.struct, _want(ctx_len, "ctx_len", i32, (S,), dev), _want(path, "path", i32, None, dev),
                           _want(n_path, "n_path", i32, (S,), dev), path.shape[1], _stream_on(stream, dev))
    if st:
        raise MQError(st, "mq_kv_accept")


def attn_workspace(cache: KVCache, n_heads: int, max_tokens: int = MQ_TREE_MAX_TOKENS, stream=None):
    """A zeroed workspace for attn_tree calls with up to max_tokens tokens per sequence (one per stream that runs them).
    It serves any number of sequences, and any cache and heads whose workspace is no larger."""
    torch = _torch()
    handle = _stream_on(stream, cache.device)  # before the size, which goes by the current device
    out = _new(mq_attn_workspace_bytes(cache.struct, n_heads, max_tokens), torch.uint8, cache.device, stream)
    with torch.cuda.stream(None if stream is None else torch.cuda.ExternalStream(handle, device=cache.device)):
        return out.zero_()


def _attn_args(cache: KVCache, q, tok_start, ctx_len, mask, scale, max_len, max_tokens, out_type, out, stream):
    """The arguments that attn_tree and attn_shared have in common, and the output tensor."""
    torch = _torch()
    dev, D, S, i32 = cache.device, cache.head_dim, cache.n_seqs, torch.int32
    if q.dim() != 2 or q.shape[1] % D:
        raise ValueError(f"q: rows of whole heads of {D} are wanted, got {tuple(q.shape)}")
    n, width = q.shape
    qp, q_ld = _rows(q, "q", torch.float16, dev, width)
    if out_type == "f16":
        if out is None:
            out = _new((n, width), torch.float16, dev, stream)
            op, out_ld = out.data_ptr(), width
        else:
            op, out_ld = _rows(out, "out", torch.float16, dev, width, n)
        kind = MQ_TYPE_F16
    elif out_type == "q8_0":
        shape = (n, width // 32 * 34)
        out = _new(shape, torch.uint8, dev, stream) if out is None else out
        op, out_ld, kind = _want(out, "out", torch.uint8, shape, dev), 0, MQ_TYPE_Q8_0
    else:
        raise ValueError(f"out_type {out_type!r}: \"f16\" or \"q8_0\"")
    if max_len is None:
        max_len = cache.table.shape[1] * MQ_KV_PAGE_TOKENS
    a = AttnArgs(qp, op, _want(tok_start, "tok_start", i32, (S + 1,), dev), _want(ctx_len, "ctx_len", i32, (S,), dev),
                 None if mask is None else _want(mask, "mask", torch.int64, (n,), dev), q_ld, out_ld, n, width // D,
                 max_len, max_tokens, kind, D ** -0.5 if scale is None else scale)
    return a, out


def attn_tree(cache: KVCache, q, tok_start, ctx_len, mask=None, scale: Optional[float] = None,
              max_len: Optional[int] = None, max_tokens: int = MQ_TREE_MAX_TOKENS, out_type: str = "f16", out=None,
              workspace=None, stream=None):
    """Attention of every tree's nodes (q: f16 [n, n_heads * head_dim], rows may be strided) over the cache.

    ``mask``: int64 [n], bit j = node j of the token's tree is seen (None: a chain).  ``max_len`` bounds context plus
    tree of any sequence (default: what the table can hold).  ``max_tokens`` bounds the tokens of any sequence, picks the
    kernel and sizes the workspace: a decode step says 1, with the default it takes the kernel for large trees.  Returns
    f16 [n, n_heads * head_dim], or with ``out_type="q8_0"`` uint8 [n, n_heads * head_dim / 32 * 34], the ``xq`` of a
    projection.  A program that calls this every step keeps the workspace (attn_workspace)."""
    a, out = _attn_args(cache, q, tok_start, ctx_len, mask, scale, max_len, max_tokens, out_type, out, stream)
    if workspace is None:
        workspace = attn_workspace(cache, a.n_heads, max_tokens, stream)
    st = _lib.mq_attn_tree(cache.struct, a, _want(workspace, "workspace", _torch().uint8, None, cache.device),
                           workspace.numel(), _stream_on(stream, cache.device))
    if st:
        raise MQError(st, "mq_attn_tree")
    return out


def attn_shared_workspace(cache: KVCache, n_heads: int, n_tokens: int, n_groups: int, max_tokens: int = MQ_TREE_MAX_TOKENS,
                          stream=None):
    """A zeroed workspace for attn_shared calls with up to n_tokens tokens in all, n_groups groups and max_tokens tokens
    per sequence (one per stream that runs them).  It serves any call of attn_shared or attn_tree whose workspace is no
    larger."""
    torch = _torch()
    handle = _stream_on(stream, cache.device)  # before the size, which goes by the current device
    out = _new(mq_attn_shared_workspace_bytes(cache.struct, n_heads, n_tokens, max_tokens, n_groups), torch.uint8,
               cache.device, stream)
    with torch.cuda.stream(None if stream is None else torch.cuda.ExternalStream(handle, device=cache.device)):
        return out.zero_()


def attn_shared(cache: KVCache, q, tok_start, ctx_len, grp_start, grp_pages, mask=None, scale: Optional[float] = None,
                max_len: Optional[int] = None, max_tokens: int = MQ_TREE_MAX_TOKENS, max_pages: Optional[int] = None,
                out_type: str = "f16", out=None, workspace=None, stream=None):
    """attn_tree of a batch whose sequences share the pages of a prefix, each prefix attended once for all.

    ``grp_start``: int32 [n_groups + 1], group g are the sequences grp_start[g]..grp_start[g + 1] - 1; ``grp_pages``:
    int32 [n_groups], the pages at the start of their table rows that are the same for all of them that have tokens (every
    such context reaches past them).  ``max_pages`` bounds grp_pages (default: what the table can hold).  The rest is attn_tree's;
    the workspace is attn_shared_workspace's."""
    i32, dev = _torch().int32, cache.device
    a, out = _attn_args(cache, q, tok_start, ctx_len, mask, scale, max_len, max_tokens, out_type, out, stream)
    n = grp_pages.numel()
    g = AttnGroups(_want(grp_start, "grp_start", i32, (n + 1,), dev), _want(grp_pages, "grp_pages", i32, (n,), dev), n,
                   cache.table.shape[1] if max_pages is None else max_pages)
    if workspace is None:
        workspace = attn_shared_workspace(cache, a.n_heads, a.n_tokens, n, max_tokens, stream)
    st = _lib.mq_attn_shared(cache.struct, a, g, _want(workspace, "workspace", _torch().uint8, None, dev),
                             workspace.numel(), _stream_on(stream, dev))
    if st:
        raise MQError(st, "mq_attn_shared")
    return out


def softmax(x, scale: float = 1.0, out=None, stream=None):
    """exp(scale * x) / sum of it, along the rows of x (fp32 [n, vocab], rows may be strided); ``out`` may be x."""
    torch = _torch()
    if x.dim() != 2:
        raise ValueError(f"x: a 2-D tensor is wanted, got {tuple(x.shape)}")
    n, vocab = x.shape
    xp, x_ld = _rows(x, "x", torch.float32, x.device, vocab)
    handle = _stream_on(stream, x.device, "x is")
    if out is None:
        out = _new((n, vocab), torch.float32, x.device, stream)
    yp, y_ld = _rows(out, "out", torch.float32, x.device, vocab, n)
    st = _lib.mq_softmax(xp, yp, n, vocab, x_ld, y_ld, scale, handle)
    if st:
        raise MQError(st, "mq_softmax")
    return out


def verify_tree(target, tok_start, token, parent, u=None, draft=None, greedy: bool = False, path_ld: Optional[int] = None,
                path=None, n_path=None, next_token=None, stream=None):
    """Verify drafted trees: (path int32 [n_seqs, path_ld], n_path int32 [n_seqs], next int32 [n_seqs]).

    ``target``: fp32 [n, vocab], the target's probabilities behind every node (mq.softmax of the logits); ``draft``: fp32
    [n, vocab], those that a node's children were drawn from (None: the drafts are looked up, not drawn).  ``token`` and
    ``parent``: int32 [n], the drafted tokens and their parents' numbers in the tree (node 0, the root, is the token
    that the step before ended with).  ``u``: fp32 [n] in [0, 1), a root's is what ``next`` is drawn with.  ``greedy``:
    the largest target value instead of a draw (target may be logits; u and draft are not read).  ``path_ld`` bounds
    the nodes of a path, the root included.  path (zeros behind the nodes) and n_path are what kv_accept takes."""
    torch = _torch()
    dev, i32, f32 = target.device, torch.int32, torch.float32
    if target.dim() != 2:
        raise ValueError(f"target: a 2-D tensor is wanted, got {tuple(target.shape)}")
    n, vocab = target.shape
    S = tok_start.numel() - 1
    if S < 0:
        raise ValueError("tok_start: n_seqs + 1 values are wanted")
    handle = _stream_on(stream, dev, "target is")
    tp, t_ld = _rows(target, "target", f32, dev, vocab)
    dp, d_ld = (None, 0) if draft is None or greedy else _rows(draft, "draft", f32, dev, vocab, n)
    if u is None and not greedy:
        raise ValueError("u: random numbers are wanted (or greedy)")
    if path is None:
        path = _new((S, MQ_TREE_MAX_TOKENS if path_ld is None else path_ld), i32, dev, stream)
    elif path.dim() != 2 or path_ld not in (None, path.shape[1]):
        raise ValueError(f"path: [{S}, path_ld] is wanted, got {tuple(path.shape)}")
    n_path = _new((S,), i32, dev, stream) if n_path is None else n_path
    next_token = _new((S,), i32, dev, stream) if next_token is None else next_token
    a = VerifyArgs(tp, dp, _want(tok_start, "tok_start", i32, (S + 1,), dev), _want(token, "token", i32, (n,), dev),
                   _want(parent, "parent", i32, (n,), dev), None if u is None else _want(u, "u", f32, (n,), dev),
                   _want(path, "path", i32, (S, path.shape[1]), dev), _want(n_path, "n_path", i32, (S,), dev),
                   _want(next_token, "next_token", i32, (S,), dev), t_ld, d_ld, n, S, vocab, path.shape[1],
                   MQ_VERIFY_GREEDY if greedy else 0, 0)
    st = _lib.mq_verify_tree(a, handle)
    if st:
        raise MQError(st, "mq_verify_tree")
    return path, n_path, next_token


class KVPool:
    """A cache's pages as a pool (mq_kv_pool), for kv_grow, kv_fork, kv_free and kv_compact, which keep its tensors and
    the cache's table.  ``seq_pages``: int32 [n_seqs], pages of every sequence; ``refs``: int32 [n_pages], table entries
    that name a page; ``free_list``: int32 [n_pages], of which the first ``n_free`` (int32 [1]) are the free pages, the
    last of them the next to be taken.  Calls on one pool must not overlap on the GPU."""

    def __init__(self, cache: KVCache, seq_pages, refs, free_list, n_free):
        torch = _torch()
        i32, dev, P = torch.int32, cache.device, cache.struct.n_pages
        self.seq_pages, self.refs, self.free_list, self.n_free = seq_pages, refs, free_list, n_free
        self.scratch = torch.empty(mq_kv_pool_scratch(cache.struct), dtype=i32, device=dev)
        self.struct = KvPoolStruct(_want(refs, "refs", i32, (P,), dev), _want(free_list, "free_list", i32, (P,), dev),
                                   _want(n_free, "n_free", i32, (1,), dev),
                                   _want(seq_pages, "seq_pages", i32, (cache.n_seqs,), dev), self.scratch.data_ptr())

    @classmethod
    def alloc(cls, cache: KVCache) -> "KVPool":
        """A pool with every page of the cache free, the lowest taken first; the table is emptied."""
        torch = _torch()
        i32, dev, P = torch.int32, cache.device, cache.struct.n_pages
        cache.table.fill_(-1)
        return cls(cache, torch.zeros(cache.n_seqs, dtype=i32, device=dev), torch.zeros(P, dtype=i32, device=dev),
                   torch.arange(P - 1, -1, -1, dtype=i32, device=dev), torch.full((1,), P, dtype=i32, device=dev))


def kv_grow(cache: KVCache, pool: KVPool, length, stream=None) -> None:
    """Give every sequence the pages that length[s] tokens need (int32 [n_seqs]); none loses one."""
    st = _lib.mq_kv_grow(cache.struct, pool.struct, _want(length, "length", _torch().int32, (cache.n_seqs,), cache.device),
                         _stream_on(stream, cache.device))
    if st:
        raise MQError(st, "mq_kv_grow")


def kv_fork(cache: KVCache, pool: KVPool, src, dst, length, stream=None) -> None:
    """Sequence dst[i] (without pages) continues the first length[i] tokens of src[i]: full pages are shared, the
    tokens of a begun one are copied."""
    i32, dev, n = _torch().int32, cache.device, src.numel()
    st = _lib.mq_kv_fork(cache.struct, pool.struct, _want(src, "src", i32, (n,), dev), _want(dst, "dst", i32, (n,), dev),
                         _want(length, "length", i32, (n,), dev), n, _stream_on(stream, dev))
    if st:
        raise MQError(st, "mq_kv_fork")


def kv_free(cache: KVCache, pool: KVPool, seq, keep=None, stream=None) -> None:
    """Sequences seq[i] give up their pages but the first keep[i] (None: all)."""
    i32, dev, n = _torch().int32, cache.device, seq.numel()
    st = _lib.mq_kv_free(cache.struct, pool.struct, _want(seq, "seq", i32, (n,), dev),
                         None if keep is None else _want(keep, "keep", i32, (n,), dev), n, _stream_on(stream, dev))
    if st:
        raise MQError(st, "mq_kv_free")


def kv_compact(cache: KVCache, pool: KVPool, stream=None) -> None:
    """Move the pages in use to the front of the pool; the table, the counts and the free pages follow."""
    st = _lib.mq_kv_compact(cache.struct, pool.struct, _stream_on(stream, cache.device))
    if st:
        raise MQError(st, "mq_kv_compact")


class StepBuffers:
    """Device buffers and the descriptor table of one layer stack for mq_step.

    weights: per layer dict with 'qkv' (concatenated q|k|v rows), 'o', 'gu', 'down'
    (uint8 cuda tensors); a stack of FFN layers only (qkv_rows == o_rows == 0)
    needs only 'gu' and 'down'.  Inputs a/b/c and outputs are allocated here, one
    buffer per layer, so a captured graph reads fresh inputs from the same
    addresses on every replay.

    chained: build the descriptors of a decode chain (MQ_STEP_CHAINED): the o
    projection reads the q|k|v output (its first o_K values), the FFN reads the
    o output, and layer l+1's q|k|v reads layer l's FFN output; only layer 0's
    first input (a[0], or c[0] for an FFN-only stack) comes from the caller.
    """

    def __init__(self, weights: List[Dict[str, "torch.Tensor"]], H: int, I: int, qkv_rows: int, o_rows: int,
                 o_K: int, ncols: int = 1, device=None, debug: bool = False, chained: bool = False):
        torch = _torch()
        self.n_layers = len(weights)
        self.H, self.I, self.qkv_rows, self.o_rows, self.o_K, self.ncols = H, I, qkv_rows, o_rows, o_K, ncols
        self.chained = chained
        dev = device if device is not None else weights[0]["gu"].device
        self.device = dev
        n = self.n_layers
        self.weights = weights
        if chained and ncols > 1 and ((qkv_rows and o_rows and qkv_rows != o_K) or (o_rows and o_rows != H)
                                      or (qkv_rows and not o_rows and qkv_rows != H)):
            raise ValueError("a chain of ncols > 1 needs each producer's rows equal to its consumer's K")
        # inputs [layer, ncols, K]: views of one buffer, so that a step's inputs
        # arrive in one host-to-device copy (each view starts on a 16-byte
        # boundary: H and o_K are multiples of 256)
        na, nb = n * ncols * H, n * ncols * o_K
        self.inputs = torch.zeros(na + nb + na, dtype=torch.float32, device=dev)
        self.a = self.inputs[:na].view(n, ncols, H)
        self.b = self.inputs[na:na + nb].view(n, ncols, o_K)
        self.c = self.inputs[na + nb:].view(n, ncols, H)
        # outputs: views of one buffer too (one device-to-host copy)
        nq, no = n * ncols * qkv_rows, n * ncols * o_rows
        self.outputs = torch.zeros(nq + no + n * ncols * H, dtype=torch.float32, device=dev)
        self.y_qkv = self.outputs[:nq].view(n, ncols, qkv_rows)
        self.y_o = self.outputs[nq:nq + no].view(n, ncols, o_rows)
        self.y_ffn = self.outputs[nq + no:].view(n, ncols, H)
        self.h_q8 = torch.zeros((n, ncols, I // 32 * 34), dtype=torch.uint8, device=dev)
        self.debug = debug
        if debug:
            self.xq_a = torch.zeros((n, ncols, H // 32 * 34), dtype=torch.uint8, device=dev)
            self.xq_b = torch.zeros((n, ncols, o_K // 32 * 34), dtype=torch.uint8, device=dev)
        table = (LayerDesc * n)()
        prev = None  # the fp32 output the next phase of a chain reads
        for l, w in enumerate(weights):
            if qkv_rows:
                xa = prev if (chained and prev is not None) else self.a[l]
                table[l].qkv = mv_desc(w["qkv"], qkv_rows, H, self.y_qkv[l], x=xa,
                                       xq_out=self.xq_a[l] if debug else None, ncols=ncols, y_ld=qkv_rows)
                prev = self.y_qkv[l]
            if o_rows:
                xb = prev if (chained and prev is not None) else self.b[l]
                table[l].o = mv_desc(w["o"], o_rows, o_K, self.y_o[l], x=xb,
                                     xq_out=self.xq_b[l] if debug else None, ncols=ncols, y_ld=o_rows)
                prev = self.y_o[l]
            xc = prev if (chained and prev is not None) else self.c[l]
            table[l].ffn = ffn_desc(w["gu"], w["down"], H, I, self.h_q8[l], self.y_ffn[l], x=xc,
                                    ncols=ncols, y_ld=H)
            prev = self.y_ffn[l]
            for rows, part in ((qkv_rows, table[l].qkv), (o_rows, table[l].o)):
                if rows:
                    _check(mq_check_mv_desc(part), "mq_check_mv_desc")
            _check(mq_check_ffn_desc(table[l].ffn), "mq_check_ffn_desc")
        self.table_host = table
        self.table = upload_struct(bytes(table), dev)
        # dependency words and records of the persistent step (zeroed by mq_step itself)
        nbytes = mq_step_workspace_bytes(StepShape(n, H, I, qkv_rows, o_rows, o_K, ncols,
                                                   MQ_STEP_CHAINED if chained else 0, None))
        self.workspace = torch.zeros(nbytes, dtype=torch.uint8, device=dev)

    def shape(self, flags: int = 0) -> StepShape:
        if self.chained:
            flags |= MQ_STEP_CHAINED
        return StepShape(self.n_layers, self.H, self.I, self.qkv_rows, self.o_rows, self.o_K, self.ncols, flags,
                         _ptr(self.workspace))

    def step(self, stream=None, flags: int = 0) -> None:
        _check(mq_step(_ptr(self.table), self.shape(flags), _stream(stream)), "mq_step")
