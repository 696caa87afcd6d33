"""ctypes binding of libdsa.so — argument marshalling only.

Every entry point here forwards torch CUDA tensors (as raw device pointers)
and the current CUDA stream to the C ABI declared in ``include/dsa.h``; all
arithmetic happens in the library's kernels.  There is no CPU fallback: if
the library is missing or fails to load, every call raises.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdsa.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_BOUNDS, ERR_TIMEOUT, ERR_CUDA, ERR_WORKSPACE = range(7)
KEY_FP8_E4M3, KEY_MXFP4, KEY_MXFP4_NATIVE = 0, 1, 2
LATENT_FP8_E4M3, LATENT_NVFP4 = 0, 1
BLOCK, IDX_HEADS, IDX_DIM, MLA_HEADS, LATENT, VALUE, MAX_TOPK = 64, 32, 128, 96, 576, 512, 2048
DELTA_DIM = 128


class DsaError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        extra = ""
        if code == ERR_CUDA:
            extra = f" [{lib().dsa_last_cuda_error().decode()}]"
        super().__init__(f"{what}: {status_string(code)}{extra}")


class PagedCacheT(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("row_stride", ctypes.c_int64), ("latent_off", ctypes.c_int64),
                ("index_off", ctypes.c_int64), ("block_size", ctypes.c_int32), ("num_blocks", ctypes.c_int32),
                ("key_format", ctypes.c_int32), ("latent_scale", ctypes.c_float), ("latent_format", ctypes.c_int32)]


class BatchT(ctypes.Structure):
    _fields_ = [("block_table", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p),
                ("max_blocks_per_seq", ctypes.c_int32), ("batch", ctypes.c_int32),
                ("queries_per_seq", ctypes.c_int32), ("max_seq_len", ctypes.c_int32)]


class StatePoolT(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("slot_stride", ctypes.c_int64), ("num_slots", ctypes.c_int32),
                ("heads", ctypes.c_int32)]


class DeltaRowsT(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("q", "k", "v", "gate", "beta")] + [
        (n, ctypes.c_int64) for n in ("ld_q", "ld_k", "ld_v", "ld_gate", "ld_beta")] + [
        ("qk_heads", ctypes.c_int32), ("gate_dim", ctypes.c_int32), ("scale", ctypes.c_float)]


_lib = None

EXPORTS = ["dsa_api_version", "dsa_status_string", "dsa_last_cuda_error", "dsa_kernel_launches",
           "dsa_translate_pages", "dsa_index_scores", "dsa_index_scores_bf16", "dsa_topk_bf16",
           "dsa_decode_step_bf16",
           "dsa_topk_workspace_size", "dsa_topk", "dsa_topk_noalloc", "dsa_topk_force_multipass", "dsa_topk_paged",
           "dsa_dcp_topk_workspace_size", "dsa_dcp_topk", "sparse_mla_workspace_size",
           "sparse_mla_decode", "dense_mla_workspace_size", "dense_mla_decode",
           "dsa_attention_mass_workspace_size", "dsa_attention_mass", "dsa_cache_evict_workspace_size",
           "dsa_cache_evict", "dsa_dcp_sparse_mla_workspace_size", "dsa_dcp_sparse_mla", "dsa_batch_invariant",
           "dsa_workspace_size", "dsa_decode_step", "dsa_cache_append", "dsa_quantize_index_query",
           "dsa_index_frontend", "dsa_frontend_workspace_size", "dsa_decode_step_frontend",
           "dsa_assign_slots", "dsa_cache_append_slots", "gated_delta_decode", "gated_delta_prefill_workspace_size",
           "gated_delta_prefill", "dsa_selftest_wait_timeout"]


def lib():
    """Load libdsa.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libdsa.so not found at {LIB_PATH}: build it with "
                               "dsa_sparse_attention_index_gb300.build.build()")
        L = ctypes.CDLL(LIB_PATH)
        P, i32, i64, sz, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
        pc, pb = ctypes.POINTER(PagedCacheT), ctypes.POINTER(BatchT)
        ps, pd = ctypes.POINTER(StatePoolT), ctypes.POINTER(DeltaRowsT)
        sig = {
            "dsa_api_version": (i32, []),
            "dsa_status_string": (ctypes.c_char_p, [i32]),
            "dsa_last_cuda_error": (ctypes.c_char_p, []),
            "dsa_kernel_launches": (ctypes.c_uint64, []),
            "dsa_translate_pages": (i32, [pc, pb, P, P, P, P]),
            "dsa_index_scores": (i32, [pc, pb, P, P, P, i64, P, P]),
            "dsa_topk_workspace_size": (sz, [i32, i32, i32]),
            "dsa_topk": (i32, [P, i64, P, i32, i32, i32, P, P, sz, P, P]),
            "dsa_topk_noalloc": (i32, [P, i64, P, i32, i32, i32, P, P, P]),
            "dsa_topk_force_multipass": (i32, [i32]),
            "dsa_dcp_topk_workspace_size": (sz, [i32, i32, i32]),
            "dsa_dcp_topk": (i32, [P, i64, P, i32, i32, i32, i32, P, P, P, sz, P, P]),
            "sparse_mla_workspace_size": (sz, [i32, i32]),
            "sparse_mla_decode": (i32, [pc, pb, P, P, i32, f32, P, P, P, sz, P, P]),
            "dense_mla_workspace_size": (sz, [i32, i32]),
            "dense_mla_decode": (i32, [pc, pb, P, f32, P, P, P, sz, P, P]),
            "dsa_attention_mass_workspace_size": (sz, [i32, i32, i32]),
            "dsa_attention_mass": (i32, [pc, pb, P, P, P, i32, f32, P, P, i64, P, sz, P, P]),
            "dsa_cache_evict_workspace_size": (sz, [i32, i32, i32]),
            "dsa_cache_evict": (i32, [pc, pb, P, i64, i32, i32, i32, pc, P, i32, P, P, i64, P, P, sz, P, P]),
            "dsa_dcp_sparse_mla_workspace_size": (sz, [i32, i32, i32]),
            "dsa_batch_invariant": (i32, [i32]),
            "dsa_dcp_sparse_mla": (i32, [pc, pb, P, P, i32, i32, f32, P, P, P, P, P, sz, P, P]),
            "dsa_workspace_size": (sz, [pb, i32]),
            "dsa_decode_step": (i32, [pc, pb, P, P, P, i32, f32, P, P, P, i64, P, P, P, sz, P, P]),
            "dsa_decode_step_bf16": (i32, [pc, pb, P, P, P, i32, f32, P, P, P, i64, P, P, P, sz, P, P]),
            "dsa_topk_paged": (i32, [pc, pb, P, i64, i32, P, P, P, sz, P, P]),
            "dsa_index_scores_bf16": (i32, [pc, pb, P, P, P, i64, P, P]),
            "dsa_topk_bf16": (i32, [P, i64, P, i32, i32, i32, P, P, P]),
            "dsa_cache_append": (i32, [pc, pb, P, P, P, P]),
            "dsa_quantize_index_query": (i32, [P, P, i32, P, P, P]),
            "dsa_index_frontend": (i32, [pc, pb, P, i32, P, f32, P, P, P, P, P, P, P, P, P]),
            "dsa_frontend_workspace_size": (sz, [pb, i32]),
            "dsa_decode_step_frontend": (i32, [pc, pb, P, i32, P, f32, P, P, P, P, P, i32, f32, P, P, P, i64, P, P,
                                               P, sz, P, P]),
            "dsa_assign_slots": (i32, [P, P, i32, P, i32, P, P, i32, P, i32, P, P, P, P, i32, P, P]),
            "dsa_cache_append_slots": (i32, [pc, P, i32, P, P, P, P]),
            "gated_delta_decode": (i32, [ps, pd, i32, i32, P, P, P, P, P]),
            "gated_delta_prefill_workspace_size": (sz, [i32, i32, i32]),
            "gated_delta_prefill": (i32, [ps, pd, P, i32, i32, P, P, P, P, sz, P, P]),
            "dsa_selftest_wait_timeout": (i32, [i64, P, P]),
        }
        for name, (res, args) in sig.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def topk_force_multipass(on: bool) -> bool:
    """Route rows longer than 245,760 tokens through the four-kernel top-k
    (True) or the automatic choice (False); returns the previous setting."""
    return bool(lib().dsa_topk_force_multipass(int(bool(on))))


def kernel_launches() -> int:
    """Kernels libdsa has launched in this process so far."""
    return int(lib().dsa_kernel_launches())


def status_string(code: int) -> str:
    return lib().dsa_status_string(int(code)).decode()


def _check(code: int, what: str) -> None:
    if code != OK:
        raise DsaError(code, what)


def _ptr(t) -> int | None:
    if t is None:
        return None
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError("tensors passed to libdsa must be contiguous CUDA tensors")
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is not None:
        return stream.cuda_stream
    # the current stream's handle, without building a Stream object (3 us a call)
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


_BITS16 = (torch.int16, torch.uint16, torch.bfloat16)
_I32, _F32 = (torch.int32,), (torch.float32,)


def _want(name: str, t, shape, dtypes) -> int | None:
    """The address of a tensor that must have this shape and one of these types, or of None."""
    if t is None:
        return None
    if t.shape != shape or t.dtype not in dtypes:
        raise ValueError(f"{name}: expected {list(shape)} of {dtypes[0]}, got {list(t.shape)} of {t.dtype}")
    return _ptr(t)


def _one_device(*tensors) -> None:
    """Every tensor on the current device: the library launches there."""
    at = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.get_device() != at:
            raise ValueError(f"tensors must be on the current device (cuda:{at}), got {t.device}")


@dataclass
class PagedCache:
    """One layer's packed paged cache: ``pool`` is a uint8 CUDA tensor
    [num_blocks, row_stride]; offsets locate the latent and index pages."""

    pool: torch.Tensor
    row_stride: int
    latent_off: int
    index_off: int
    key_format: int
    latent_scale: float
    latent_format: int = 0

    def struct(self) -> PagedCacheT:
        return PagedCacheT(_ptr(self.pool), self.row_stride, self.latent_off, self.index_off, BLOCK,
                           int(self.pool.shape[0]), self.key_format, float(self.latent_scale),
                           int(self.latent_format))


@dataclass
class Batch:
    """block_table int32 [batch, max_blocks] and seq_lens int32 [batch] on the GPU."""

    block_table: torch.Tensor
    seq_lens: torch.Tensor
    queries_per_seq: int
    max_seq_len: int

    @property
    def batch(self) -> int:
        return int(self.seq_lens.shape[0])

    @property
    def rows(self) -> int:
        return self.batch * self.queries_per_seq

    def struct(self) -> BatchT:
        return BatchT(_ptr(self.block_table), _ptr(self.seq_lens), int(self.block_table.shape[1]), self.batch,
                      self.queries_per_seq, int(self.max_seq_len))


def _structs(batch: Batch, *caches: PagedCache):
    """The descriptors of a batch and caches whose tensors hold all that the library reads through them."""
    table, lens = batch.block_table, batch.seq_lens
    if (table.dtype not in _I32 or lens.dtype not in _I32 or table.dim() != 2 or lens.dim() != 1
            or table.shape[0] < lens.shape[0]):
        raise ValueError(f"block_table and seq_lens: expected int32 [batch, max_blocks] and [batch], got "
                         f"{list(table.shape)} of {table.dtype} and {list(lens.shape)} of {lens.dtype}")
    for c in caches:
        if c.pool.nbytes < c.pool.shape[0] * c.row_stride:
            raise ValueError(f"pool: {c.pool.nbytes} bytes for {c.pool.shape[0]} rows of {c.row_stride}")
    return batch.struct(), *(c.struct() for c in caches)


def _status(status) -> int | None:
    if status is not None and (status.dtype not in _I32 or status.numel() < 1):
        raise ValueError(f"status: expected one int32, got {list(status.shape)} of {status.dtype}")
    return _ptr(status)


def translate_pages(cache: PagedCache, batch: Batch, latent_pages, index_pages, status, stream=None):
    c, b = cache.struct(), batch.struct()
    _check(lib().dsa_translate_pages(ctypes.byref(c), ctypes.byref(b), _ptr(latent_pages), _ptr(index_pages),
                                     _ptr(status), _stream(stream)), "dsa_translate_pages")


def index_scores(cache: PagedCache, batch: Batch, q_index, head_w, scores, status, stream=None):
    c, b = cache.struct(), batch.struct()
    _check(lib().dsa_index_scores(ctypes.byref(c), ctypes.byref(b), _ptr(q_index), _ptr(head_w), _ptr(scores),
                                  int(scores.shape[1]), _ptr(status), _stream(stream)), "dsa_index_scores")


def index_scores_bf16(cache: PagedCache, batch: Batch, q_index, head_w, scores, status, stream=None):
    """Indexer scores rounded to bf16; `scores` holds the bits (int16 or bfloat16 [rows, ld], ld % 8 == 0)."""
    c, b = cache.struct(), batch.struct()
    _check(lib().dsa_index_scores_bf16(ctypes.byref(c), ctypes.byref(b), _ptr(q_index), _ptr(head_w), _ptr(scores),
                                       int(scores.shape[1]), _ptr(status), _stream(stream)), "dsa_index_scores_bf16")


def topk_bf16(scores, row_lens, max_row_len: int, k: int, idx_out, status, stream=None):
    """Top-k over bf16 scores (bits [rows, ld], ld % 8 == 0); no workspace."""
    rows = int(scores.shape[0])
    _check(lib().dsa_topk_bf16(_ptr(scores), int(scores.shape[1]), _ptr(row_lens), rows, int(max_row_len), int(k),
                               _ptr(idx_out), _ptr(status), _stream(stream)), "dsa_topk_bf16")


def topk_workspace_size(rows: int, max_row_len: int, k: int) -> int:
    return int(lib().dsa_topk_workspace_size(rows, max_row_len, k))


def topk(scores, row_lens, max_row_len: int, k: int, idx_out, workspace, status, stream=None):
    rows = int(scores.shape[0])
    _check(lib().dsa_topk(_ptr(scores), int(scores.shape[1]), _ptr(row_lens), rows, int(max_row_len), int(k),
                          _ptr(idx_out), _ptr(workspace), workspace.numel() * workspace.element_size(),
                          _ptr(status), _stream(stream)), "dsa_topk")


def topk_noalloc(scores, row_lens, max_row_len: int, k: int, idx_out, status, stream=None):
    """dsa_topk with the library's built-in scratch: no workspace, no allocation (rows <= 64)."""
    rows = int(scores.shape[0])
    _check(lib().dsa_topk_noalloc(_ptr(scores), int(scores.shape[1]), _ptr(row_lens), rows, int(max_row_len),
                                  int(k), _ptr(idx_out), _ptr(status), _stream(stream)), "dsa_topk_noalloc")


def dcp_topk_workspace_size(rows: int, k: int, shards: int) -> int:
    return int(lib().dsa_dcp_topk_workspace_size(rows, k, shards))


def dcp_topk(scores, row_lens, max_row_len: int, k: int, shards: int, idx_out, workspace, status, stats_out=None,
             stream=None):
    """The decode-context-parallel top-k merge of `shards` token shards (bf16-keyed candidates, global
    selection, resends); stats_out: optional int32 [rows, 3] (words sent, shards that resent, words resent)."""
    rows = int(scores.shape[0])
    _check(lib().dsa_dcp_topk(_ptr(scores), int(scores.shape[1]), _ptr(row_lens), rows, int(max_row_len), int(k),
                              int(shards), _ptr(idx_out), _ptr(stats_out), _ptr(workspace),
                              workspace.numel() * workspace.element_size(), _ptr(status), _stream(stream)),
           "dsa_dcp_topk")


def sparse_mla_workspace_size(rows: int, k: int) -> int:
    return int(lib().sparse_mla_workspace_size(rows, k))


def sparse_mla_decode(cache: PagedCache, batch: Batch, q_mla, idx, sm_scale: float, out, lse, workspace, status,
                      stream=None):
    c, b = cache.struct(), batch.struct()
    _check(lib().sparse_mla_decode(ctypes.byref(c), ctypes.byref(b), _ptr(q_mla), _ptr(idx), int(idx.shape[1]),
                                   float(sm_scale), _ptr(out), _ptr(lse), _ptr(workspace),
                                   workspace.numel() * workspace.element_size(), _ptr(status), _stream(stream)),
           "sparse_mla_decode")


def dense_mla_workspace_size(rows: int, max_seq_len: int) -> int:
    return int(lib().dense_mla_workspace_size(rows, max_seq_len))


def dense_mla_decode(cache: PagedCache, batch: Batch, q_mla, sm_scale: float, out, lse, workspace, status,
                     stream=None):
    """Exact MLA over every token each row sees (no selection): q_mla bf16 bits [rows, 96, 576], out bf16 bits
    [rows, 96, 512], lse fp32 [rows, 96]."""
    b, c = _structs(batch, cache)
    rows = batch.rows
    _one_device(cache.pool, batch.block_table, batch.seq_lens, q_mla, out, lse, workspace, status)
    _check(lib().dense_mla_decode(ctypes.byref(c), ctypes.byref(b),
                                  _want("q_mla", q_mla, (rows, MLA_HEADS, LATENT), _BITS16), float(sm_scale),
                                  _want("out", out, (rows, MLA_HEADS, VALUE), _BITS16),
                                  _want("lse", lse, (rows, MLA_HEADS), _F32), _ptr(workspace),
                                  workspace.nbytes, _status(status), _stream(stream)),
           "dense_mla_decode")


def attention_mass_workspace_size(rows: int, max_seq_len: int, k: int = 0) -> int:
    return int(lib().dsa_attention_mass_workspace_size(rows, max_seq_len, k))


def attention_mass(cache: PagedCache, batch: Batch, q_mla, lse, sm_scale: float, mass_in, mass_out, workspace, status,
                   idx=None, stream=None):
    """mass_out = mass_in (or 0) + every token's attention weight, summed over the rows of its sequence and the heads:
    fp32 [batch, ld]; over every visible token, or over the top-k's entries when idx (int32 [rows, k]) is given."""
    b, c = _structs(batch, cache)
    rows = batch.rows
    _one_device(cache.pool, batch.block_table, batch.seq_lens, q_mla, lse, mass_in, mass_out, workspace, status, idx)
    ld, k = mass_out.shape[-1], 0 if idx is None else idx.shape[-1]
    if idx is not None and k < 1:
        raise ValueError("idx: expected at least one entry a row; None stands for every visible token")
    totals = (batch.batch, ld)
    _check(lib().dsa_attention_mass(ctypes.byref(c), ctypes.byref(b),
                                    _want("q_mla", q_mla, (rows, MLA_HEADS, LATENT), _BITS16),
                                    _want("lse", lse, (rows, MLA_HEADS), _F32), _want("idx", idx, (rows, k), _I32), k,
                                    float(sm_scale), _want("mass_in", mass_in, totals, _F32),
                                    _want("mass_out", mass_out, totals, _F32), ld, _ptr(workspace),
                                    workspace.nbytes, _status(status), _stream(stream)), "dsa_attention_mass")


def cache_evict_workspace_size(batch: int, max_seq_len: int, keep: int) -> int:
    return int(lib().dsa_cache_evict_workspace_size(batch, max_seq_len, keep))


def cache_evict(cache: PagedCache, batch: Batch, mass, keep: int, sink: int, recent: int, dst_cache: PagedCache,
                dst_block_table, kept_idx, mass_out, new_lens, workspace, status, stream=None):
    """Keep each sequence's first `sink`, last `recent` and, between them, heaviest tokens (`keep` in all) and move
    their records into the pages of dst_block_table.  kept_idx int32 [batch, keep], mass_out fp32 [batch, >= keep]
    or None, new_lens int32 [batch]."""
    b, c, d = _structs(batch, cache, dst_cache)
    n = batch.batch
    ld, blocks, ld_out = mass.shape[-1], dst_block_table.shape[-1], 0 if mass_out is None else mass_out.shape[-1]
    _one_device(cache.pool, batch.block_table, batch.seq_lens, mass, dst_cache.pool, dst_block_table, kept_idx, mass_out,
                new_lens, workspace, status)
    _check(lib().dsa_cache_evict(ctypes.byref(c), ctypes.byref(b), _want("mass", mass, (n, ld), _F32),
                                 ld, int(keep), int(sink), int(recent), ctypes.byref(d),
                                 _want("dst_block_table", dst_block_table, (n, blocks), _I32), blocks,
                                 _want("kept_idx", kept_idx, (n, int(keep)), _I32),
                                 _want("mass_out", mass_out, (n, ld_out), _F32), ld_out,
                                 _want("new_lens", new_lens, (n,), _I32), _ptr(workspace),
                                 workspace.nbytes, _status(status), _stream(stream)),
           "dsa_cache_evict")


def batch_invariant(on: bool) -> bool:
    """Switch the process-wide batch-invariant mode (MLA chunks of 512 selected tokens, dense parts of 3,840 tokens);
    returns the previous one."""
    return bool(lib().dsa_batch_invariant(1 if on else 0))


def dcp_sparse_mla_workspace_size(rows: int, k: int, shards: int) -> int:
    return int(lib().dsa_dcp_sparse_mla_workspace_size(rows, k, shards))


def dcp_sparse_mla(cache: PagedCache, batch: Batch, q_mla, idx, shards: int, sm_scale: float, out, lse, workspace,
                   status, part_out=None, part_lse=None, stream=None):
    """Sparse MLA as `shards` token shards would compute it: per-shard partial attention over the selected
    tokens each holds, bf16 partial outputs and fp32 LSEs, merged through their log-sum-exp.  part_out
    (bf16 [shards, rows, 96, 512]) and part_lse (fp32 [shards, rows, 96]) optionally receive the partials."""
    c, b = cache.struct(), batch.struct()
    _check(lib().dsa_dcp_sparse_mla(ctypes.byref(c), ctypes.byref(b), _ptr(q_mla), _ptr(idx), int(idx.shape[1]),
                                    int(shards), float(sm_scale), _ptr(out), _ptr(lse), _ptr(part_out),
                                    _ptr(part_lse), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                    _ptr(status), _stream(stream)),
           "dsa_dcp_sparse_mla")


def workspace_size(batch: Batch, k: int) -> int:
    b = batch.struct()
    return int(lib().dsa_workspace_size(ctypes.byref(b), int(k)))


def decode_step(cache: PagedCache, batch: Batch, q_index, head_w, q_mla, k: int, sm_scale: float, out, lse,
                workspace, status, scores_out=None, idx_out=None, stream=None, phys_out=None):
    c, b = cache.struct(), batch.struct()
    ld = int(scores_out.shape[1]) if scores_out is not None else 0
    _check(lib().dsa_decode_step(ctypes.byref(c), ctypes.byref(b), _ptr(q_index), _ptr(head_w), _ptr(q_mla),
                                 int(k), float(sm_scale), _ptr(out), _ptr(lse), _ptr(scores_out), ld,
                                 _ptr(idx_out), _ptr(phys_out), _ptr(workspace),
                                 workspace.numel() * workspace.element_size(), _ptr(status), _stream(stream)),
           "dsa_decode_step")


def topk_paged(cache: PagedCache, batch: Batch, scores, k: int, idx_out, workspace, status, phys_out=None,
               stream=None):
    """The fused step's top-k on its own (row lengths from the batch), with the
    selected tokens' physical KV rows when phys_out is given."""
    c, b = cache.struct(), batch.struct()
    nbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib().dsa_topk_paged(ctypes.byref(c), ctypes.byref(b), _ptr(scores), int(scores.shape[1]), int(k),
                                _ptr(idx_out), _ptr(phys_out), _ptr(workspace), nbytes, _ptr(status),
                                _stream(stream)), "dsa_topk_paged")


def decode_step_bf16(cache: PagedCache, batch: Batch, q_index, head_w, q_mla, k: int, sm_scale: float, out, lse,
                     workspace, status, scores_out=None, idx_out=None, stream=None, phys_out=None):
    """The fused step with bf16 scores between the indexer and the top-k."""
    c, b = cache.struct(), batch.struct()
    ld = int(scores_out.shape[1]) if scores_out is not None else 0
    _check(lib().dsa_decode_step_bf16(ctypes.byref(c), ctypes.byref(b), _ptr(q_index), _ptr(head_w), _ptr(q_mla),
                                      int(k), float(sm_scale), _ptr(out), _ptr(lse), _ptr(scores_out), ld,
                                      _ptr(idx_out), _ptr(phys_out), _ptr(workspace),
                                      workspace.numel() * workspace.element_size(), _ptr(status), _stream(stream)),
           "dsa_decode_step_bf16")


def cache_append(cache: PagedCache, batch: Batch, new_latent, new_index_key, status, stream=None):
    """Write every sequence's queries_per_seq new tokens (bf16 bits, [rows, 576] and
    [rows, 128]) into their pages."""
    c, b = cache.struct(), batch.struct()
    _check(lib().dsa_cache_append(ctypes.byref(c), ctypes.byref(b), _ptr(new_latent), _ptr(new_index_key),
                                  _ptr(status), _stream(stream)), "dsa_cache_append")


def assign_slots(cached_lens, new_lens, free_blocks, free_count, num_blocks: int, block_table, seq_lens, row_starts,
                 positions, slots, free_left, status, stream=None):
    """Pages off the free stack and cache slots for every request's new tokens: cached_lens and new_lens int32 [batch],
    free_blocks int32 [n] with its count in free_count; fills in block_table int32 [batch, max_blocks], seq_lens
    [batch], row_starts [batch + 1], positions and slots [max_rows] (-1 behind the last row) and free_left."""
    n, blocks, rows = cached_lens.shape[0], block_table.shape[-1], slots.shape[0]
    _one_device(cached_lens, new_lens, free_blocks, free_count, block_table, seq_lens, row_starts, positions, slots,
                free_left, status)
    _check(lib().dsa_assign_slots(_want("cached_lens", cached_lens, (n,), _I32), _want("new_lens", new_lens, (n,), _I32),
                                  n, _want("free_blocks", free_blocks, (free_blocks.shape[0],), _I32),
                                  free_blocks.shape[0], _want("free_count", free_count, (1,), _I32),
                                  _want("free_left", free_left, (1,), _I32), int(num_blocks),
                                  _want("block_table", block_table, (n, blocks), _I32), blocks,
                                  _want("seq_lens", seq_lens, (n,), _I32),
                                  _want("row_starts", row_starts, (n + 1,), _I32),
                                  _want("positions", positions, (rows,), _I32), _want("slots", slots, (rows,), _I32),
                                  rows, _status(status), _stream(stream)), "dsa_assign_slots")


def cache_append_slots(cache: PagedCache, slots, new_latent, new_index_key, status, stream=None):
    """Write new tokens (bf16 bits, [rows, 576] and [rows, 128]) into the cache rows slots [rows]; -1: none."""
    rows = slots.shape[0]
    if cache.pool.nbytes < cache.pool.shape[0] * cache.row_stride:
        raise ValueError(f"pool: {cache.pool.nbytes} bytes for {cache.pool.shape[0]} rows of {cache.row_stride}")
    c = cache.struct()
    _one_device(cache.pool, slots, new_latent, new_index_key, status)
    _check(lib().dsa_cache_append_slots(ctypes.byref(c), _want("slots", slots, (rows,), _I32), rows,
                                        _want("new_latent", new_latent, (rows, LATENT), _BITS16),
                                        _want("new_index_key", new_index_key, (rows, IDX_DIM), _BITS16),
                                        _status(status), _stream(stream)), "dsa_cache_append_slots")


def _rows_of(name: str, t, shape, dtypes):
    """Address and row stride of a tensor of this shape whose rows are contiguous but may lie apart."""
    if tuple(t.shape) != shape or t.dtype not in dtypes or not t.is_cuda:
        raise ValueError(f"{name}: expected {list(shape)} of {dtypes[0]} on the GPU, got {list(t.shape)} of {t.dtype}")
    inner = 1
    for size, stride in zip(reversed(shape[1:]), reversed(t.stride()[1:])):
        if size > 1 and stride != inner:
            raise ValueError(f"{name}: rows must be contiguous, got strides {list(t.stride())}")
        inner *= size
    return t.data_ptr(), t.stride(0) if shape[0] > 1 else inner


class _Descriptor:
    """A descriptor's `layout`, made from its tensors and made again, with all checks, once one of them has another
    address (resized, set_() or with new .data), or the rows' number has changed; a tensor's other sizes and its strides
    have to stay as long as its address does (looking at all of them takes 2 us a call).  `seen`: what it was made from."""

    def __post_init__(self):
        self.read()

    def read(self):
        seen = self.places()
        if getattr(self, "seen", None) != seen:
            layout = self.describe()
            object.__setattr__(self, "layout", layout)
            object.__setattr__(self, "seen", seen)
        return self.layout


@dataclass(frozen=True)
class StatePool(_Descriptor):
    """The recurrent layers' states, fp32 [slots, heads, 128 values, 128 keys] on the GPU: a tensor of its own, or a
    view into the packed cache's block rows (slots may lie apart)."""

    states: torch.Tensor

    def places(self):
        return self.states.data_ptr(), self.states.shape

    def describe(self):
        t = self.states
        if t.dim() != 4:
            raise ValueError(f"states: expected [slots, heads, {DELTA_DIM}, {DELTA_DIM}], got {list(t.shape)}")
        ptr, stride = _rows_of("states", t, (t.shape[0], t.shape[1], DELTA_DIM, DELTA_DIM), _F32)
        return StatePoolT(ptr, 4 * stride, t.shape[0], t.shape[1])


@dataclass(frozen=True)
class DeltaRows(_Descriptor):
    """The rows of a gated delta layer: q and k bf16 bits [rows, qk_heads, 128], v [rows, heads, 128], the log decays
    gate fp32 [rows, heads, 128] (per key channel) or [rows, heads], beta fp32 [rows, heads].  Rows may lie apart.
    Making one takes longer than a decode call (its tensors' layouts are checked), so keep it where the tensors stay;
    what they hold is read at every call."""

    q: torch.Tensor
    k: torch.Tensor
    v: torch.Tensor
    gate: torch.Tensor
    beta: torch.Tensor
    scale: float

    def places(self):
        return (self.q.data_ptr(), self.k.data_ptr(), self.v.data_ptr(), self.gate.data_ptr(), self.beta.data_ptr(),
                self.v.shape)

    def describe(self):
        if self.q.dim() != 3 or self.v.dim() != 3:
            raise ValueError(f"q and v: expected [rows, heads, {DELTA_DIM}], got {list(self.q.shape)}, {list(self.v.shape)}")
        rows, heads, qk, wide = self.v.shape[0], self.v.shape[1], self.q.shape[1], self.gate.dim() == 3
        got = [_rows_of("q", self.q, (rows, qk, DELTA_DIM), _BITS16), _rows_of("k", self.k, (rows, qk, DELTA_DIM), _BITS16),
               _rows_of("v", self.v, (rows, heads, DELTA_DIM), _BITS16),
               _rows_of("gate", self.gate, (rows, heads, DELTA_DIM) if wide else (rows, heads), _F32),
               _rows_of("beta", self.beta, (rows, heads), _F32)]
        at = {t.get_device() for t in (self.q, self.k, self.v, self.gate, self.beta)}
        if len(at) != 1:
            raise ValueError(f"the rows' tensors must be on one device, got {sorted(at)}")
        return DeltaRowsT(*(p for p, _ in got), *(ld for _, ld in got), qk, DELTA_DIM if wide else 1, float(self.scale))

    @property
    def rows(self) -> int:
        return self.v.shape[0]


def _delta(pool: StatePool, x: DeltaRows, *others):
    states, layout = pool.read(), x.read()
    if x.v.shape[1] != states.heads:
        raise ValueError(f"rows of {x.v.shape[1]} heads and states of {states.heads}")
    _one_device(pool.states, x.v, *others)
    return ctypes.byref(states), ctypes.byref(layout), (x.v.shape[0], x.v.shape[1], DELTA_DIM)


def gated_delta_decode(pool: StatePool, x: DeltaRows, queries_per_seq: int, slots_in, slots_out, out, status,
                       stream=None):
    """The gated delta rule for queries_per_seq rows a sequence: states from slots_in int32 [batch] (-1: zeros), the
    state after each row to slots_out int32 [batch, queries_per_seq] (-1: nowhere); out bf16 bits [rows, heads, 128]."""
    p, r, shape = _delta(pool, x, slots_in, slots_out, out, status)
    batch, nq = slots_in.shape[0], int(queries_per_seq)
    if shape[0] != batch * nq:
        raise ValueError(f"{shape[0]} rows for {batch} sequences of {nq}")
    _check(lib().gated_delta_decode(p, r, batch, nq, _want("slots_in", slots_in, (batch,), _I32),
                                    _want("slots_out", slots_out, (batch, nq), _I32), _want("out", out, shape, _BITS16),
                                    _status(status), _stream(stream)), "gated_delta_decode")


def gated_delta_prefill_workspace_size(rows: int, batch: int, heads: int) -> int:
    return int(lib().gated_delta_prefill_workspace_size(rows, batch, heads))


def gated_delta_prefill(pool: StatePool, x: DeltaRows, row_starts, slots_in, slots_out, out, workspace, status,
                        stream=None):
    """The gated delta rule over ragged prompts: sequence b has the rows row_starts[b] .. row_starts[b + 1] - 1 (int32
    [batch + 1]); its state comes from slots_in[b] (-1: zeros) and goes to slots_out[b] (-1: nowhere)."""
    p, r, shape = _delta(pool, x, row_starts, slots_in, slots_out, out, workspace, status)
    batch = slots_in.shape[0]
    _check(lib().gated_delta_prefill(p, r, _want("row_starts", row_starts, (batch + 1,), _I32), batch, shape[0],
                                     _want("slots_in", slots_in, (batch,), _I32),
                                     _want("slots_out", slots_out, (batch,), _I32), _want("out", out, shape, _BITS16),
                                     _ptr(workspace), workspace.nbytes, _status(status), _stream(stream)),
           "gated_delta_prefill")


def quantize_index_query(q_bf16, head_w, q_index, head_w_out, stream=None):
    """FP8 indexer query per (row, head), its scale folded into the head weight."""
    rows = int(q_bf16.shape[0])
    _check(lib().dsa_quantize_index_query(_ptr(q_bf16), _ptr(head_w), rows, _ptr(q_index), _ptr(head_w_out),
                                          _stream(stream)), "dsa_quantize_index_query")


def index_frontend(cache: PagedCache, batch: Batch, c_q, gamma, eps: float, w_iq, head_w, new_latent, new_index_key,
                   q_index, head_w_out, status, q_proj=None, stream=None):
    """The fused indexer front end: RMSNorm of c_q (bf16 bits [rows, D]), the
    projection by w_iq (bf16 bits [4096, D]), the FP8 query (q_index [rows, 32,
    128]) with its scale folded into head_w_out, optionally the fp32 projected
    values (q_proj [rows, 4096]), and the new tokens into the cache."""
    c, b = cache.struct(), batch.struct()
    _check(lib().dsa_index_frontend(ctypes.byref(c), ctypes.byref(b), _ptr(c_q), int(c_q.shape[1]), _ptr(gamma),
                                    float(eps), _ptr(w_iq), _ptr(head_w), _ptr(new_latent), _ptr(new_index_key),
                                    _ptr(q_index), _ptr(head_w_out), _ptr(q_proj), _ptr(status), _stream(stream)),
           "dsa_index_frontend")


def frontend_workspace_size(batch: Batch, k: int) -> int:
    b = batch.struct()
    return int(lib().dsa_frontend_workspace_size(ctypes.byref(b), int(k)))


def decode_step_frontend(cache: PagedCache, batch: Batch, c_q, gamma, eps: float, w_iq, head_w, new_latent,
                         new_index_key, q_mla, k: int, sm_scale: float, out, lse, workspace, status, scores_out=None,
                         idx_out=None, stream=None, phys_out=None):
    """The front end, then the fused step over the updated cache (one call)."""
    c, b = cache.struct(), batch.struct()
    ld = int(scores_out.shape[1]) if scores_out is not None else 0
    _check(lib().dsa_decode_step_frontend(ctypes.byref(c), ctypes.byref(b), _ptr(c_q), int(c_q.shape[1]), _ptr(gamma),
                                          float(eps), _ptr(w_iq), _ptr(head_w), _ptr(new_latent),
                                          _ptr(new_index_key), _ptr(q_mla), int(k), float(sm_scale), _ptr(out),
                                          _ptr(lse), _ptr(scores_out), ld, _ptr(idx_out), _ptr(phys_out),
                                          _ptr(workspace),
                                          workspace.numel() * workspace.element_size(), _ptr(status),
                                          _stream(stream)), "dsa_decode_step_frontend")


def selftest_wait_timeout(limit_ns: int, status, stream=None):
    _check(lib().dsa_selftest_wait_timeout(int(limit_ns), _ptr(status), _stream(stream)),
           "dsa_selftest_wait_timeout")


def workspace(nbytes: int, device="cuda") -> torch.Tensor:
    """A 256-byte aligned uint8 device buffer (torch's allocator aligns to 512 B)."""
    return torch.empty(max(int(nbytes), 1), dtype=torch.uint8, device=device)
