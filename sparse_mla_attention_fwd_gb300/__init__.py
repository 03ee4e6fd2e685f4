"""GB300-native sparse MLA attention forward and backward (DeepSeek-style DSA top-k), sm_103a.

Python names mirror the C ABI of include/sparse_mla.h.  Tensors are torch CUDA tensors (torch
supplies device memory and streams only); outputs are allocated here when not given.

    out, lse, max_logits = sparse_mla_fwd(q, kv, indices, topk_length=None, attn_sink=None,
                                          sm_scale=None, d_v=512)

Semantics (FlashMLA PR #196 "Problem"/"Fix", PR #216 "Summary", PR #198 "Summary" item 2): each
query row attends to the slots j < L_t of its index list whose index lies in [0, s_kv); L_t is
topk_length[t] clamped to [0, topk] when given, else topk.  O is bf16; lse (natural log, sink
excluded) and max_logits (max of sm_scale * q.k) are fp32; a row without a counted slot gives
O = 0, lse = +inf, max_logits = -inf.

    dq, dkv, dsink = sparse_mla_bwd(q, kv, out, dout, indices, lse, topk_length, attn_sink)

returns the gradients of sum(dout * out) (FlashMLA PR #198, "Summary" item 1) in fp32.

A serving step on the paged cache that :func:`sparse_mla_fwd_paged` reads:

    seqlens_k, cu, slots, positions, counts = sparse_mla_plan_pages(seqlens, new_lens, block_table,
                                                                    free_pages, n_tokens)
    sparse_mla_append_kv(c_kv, k_pe, slots, kv_pool, norm_weight, positions=positions, rope=rope,
                         q_pe=q_pe, q=q)
    out, lse, max_logits = sparse_mla_chunk_fwd_paged(q, kv_pool, block_table, cu, seqlens_k)

gives the step's tokens their pages and rows, writes the rows, and attends to every cached key (the
dense form, one token to whole prompts per request).
"""
from __future__ import annotations

import math

import torch

from ._native import EXPORTED, SmlaError, load_library, status_string
from .native_build import LIB_PATH, build as build_library

__all__ = ["sparse_mla_fwd", "sparse_mla_fwd_paged", "sparse_mla_fwd_paged_splitkv_static", "sparse_mla_fwd_host",
           "row_shard", "sparse_mla_fwd_sharded", "auto_splits",
           "sparse_mla_bwd", "sparse_mla_plan_pages", "sparse_mla_append_kv", "sparse_mla_chunk_fwd_paged",
           "sparse_mla_device_status",
           "sparse_mla_status_string", "SmlaError", "load_library", "build_library", "LIB_PATH"]


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream_handle(stream, device):
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return stream.cuda_stream


# the current stream's handle on a device; a stream object in between costs two microseconds
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)
# torch.empty on the current device without its argument parsing, which is nearly half of its 1.5 microseconds
try:
    from torch._C._dynamo.guards import _empty_strided_cuda as _empty_strided
except ImportError:
    def _empty_strided(size, stride, dtype):
        return torch.empty_strided(size, stride, dtype=dtype, device="cuda")


def _check(t, name, dtype, device=None):
    if t is None:
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _outputs(q, h_q, d_v, out, lse, max_logits):
    s_q = q.shape[0]
    if out is None:
        out = torch.empty((s_q, h_q, d_v), dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((s_q, h_q), dtype=torch.float32, device=q.device)
    if max_logits is None:
        max_logits = torch.empty((s_q, h_q), dtype=torch.float32, device=q.device)
    _check(out, "out", torch.bfloat16, q.device)
    _check(lse, "lse", torch.float32, q.device)
    _check(max_logits, "max_logits", torch.float32, q.device)
    if tuple(out.shape) != (s_q, h_q, d_v) or tuple(lse.shape) != (s_q, h_q) \
            or tuple(max_logits.shape) != (s_q, h_q):
        raise ValueError("output tensors have the wrong shape")
    return out, lse, max_logits


def _host(t, name, dtype):
    if t is None:
        return
    if not isinstance(t, torch.Tensor) or t.is_cuda or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} host tensor")


def sparse_mla_fwd_host(q, kv, indices, topk_length=None, attn_sink=None, sm_scale=None, d_v=512,
                        out=None, lse=None, max_logits=None, device=None, dev_buffers=None, n_chunks=8,
                        stream=None, copy_streams=None):
    """The forward for host tensors (pinned for the copies to overlap), end to end: the C entry
    copies each row chunk's inputs to the device, runs the forward on it and copies its outputs
    back, with the copies of one chunk overlapping the compute of another.  Outputs are host
    tensors (pinned, allocated here when not given).  `dev_buffers` (a dict with the keys q, kv,
    indices, topk_length, attn_sink, out, lse, max_logits) and `copy_streams` (two streams: in,
    out) are allocated here when not given.  The call is asynchronous on `stream`: synchronise
    it before reading the outputs."""
    lib = load_library()
    dev = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
    _host(q, "q", torch.bfloat16)
    _host(kv, "kv", torch.bfloat16)
    _host(indices, "indices", torch.int32)
    _host(topk_length, "topk_length", torch.int32)
    _host(attn_sink, "attn_sink", torch.float32)
    s_q, h_q, d_qk = q.shape
    s_kv = kv.shape[0]
    topk = indices.shape[-1]
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(d_qk)
    if out is None:
        out = torch.empty((s_q, h_q, d_v), dtype=torch.bfloat16).pin_memory()
    if lse is None:
        lse = torch.empty((s_q, h_q), dtype=torch.float32).pin_memory()
    if max_logits is None:
        max_logits = torch.empty((s_q, h_q), dtype=torch.float32).pin_memory()
    _host(out, "out", torch.bfloat16)
    _host(lse, "lse", torch.float32)
    _host(max_logits, "max_logits", torch.float32)
    if dev_buffers is None:
        def like(t, shape=None):
            return None if t is None else torch.empty(t.shape if shape is None else shape, dtype=t.dtype, device=dev)
        dev_buffers = dict(q=like(q), kv=like(kv), indices=like(indices), topk_length=like(topk_length),
                           attn_sink=like(attn_sink), out=like(out), lse=like(lse), max_logits=like(max_logits))
    d = dev_buffers
    for k, dt in (("q", torch.bfloat16), ("kv", torch.bfloat16), ("indices", torch.int32),
                  ("topk_length", torch.int32), ("attn_sink", torch.float32), ("out", torch.bfloat16),
                  ("lse", torch.float32), ("max_logits", torch.float32)):
        _check(d.get(k), "dev_buffers[" + k + "]", dt, dev)
    if copy_streams is None:
        copy_streams = (torch.cuda.Stream(dev), torch.cuda.Stream(dev))
    with torch.cuda.device(dev):
        rc = lib.sparse_mla_fwd_host(
            _ptr(q), _ptr(kv), _ptr(indices), _ptr(topk_length), _ptr(attn_sink), float(sm_scale), int(d_v),
            _ptr(out), _ptr(lse), _ptr(max_logits), int(s_q), int(s_kv), int(h_q), int(d_qk), int(topk),
            _ptr(d["q"]), _ptr(d["kv"]), _ptr(d["indices"]), _ptr(d.get("topk_length")), _ptr(d.get("attn_sink")),
            _ptr(d["out"]), _ptr(d["lse"]), _ptr(d["max_logits"]), int(n_chunks), _stream_handle(stream, dev),
            copy_streams[0].cuda_stream, copy_streams[1].cuda_stream)
    if rc != 0:
        raise SmlaError(rc, "sparse_mla_fwd_host")
    return out, lse, max_logits


def row_shard(s_q, rank, world):
    """The contiguous query rows [r0, r1) that rank `rank` of `world` owns in a batch of s_q rows.
    Rows are independent, so a batch splits across GPUs with no exchange; the first s_q % world
    ranks take one row more."""
    if world < 1 or not 0 <= rank < world or s_q < 0:
        raise ValueError("need 0 <= rank < world and s_q >= 0")
    base, extra = divmod(int(s_q), int(world))
    r0 = rank * base + min(rank, extra)
    return r0, r0 + base + (1 if rank < extra else 0)


def sparse_mla_fwd_sharded(q, kv, indices, rank, world, topk_length=None, attn_sink=None, sm_scale=None,
                           d_v=512, stream=None, n_split=1):
    """The forward on this rank's rows of the batch (see row_shard): every GPU holds the whole
    shared KV and the batch's tensors, computes its own contiguous rows, and keeps its outputs
    (an all-gather is needed only if a caller wants them replicated).  Returns (r0, r1) and the
    outputs of those rows."""
    r0, r1 = row_shard(q.shape[0], rank, world)
    tl = None if topk_length is None else topk_length[r0:r1]
    out = sparse_mla_fwd(q[r0:r1], kv, indices[r0:r1], tl, attn_sink, sm_scale=sm_scale, d_v=d_v,
                         stream=stream, n_split=n_split)
    return (r0, r1), out


def auto_splits(s_q, h_q, topk, device=None):
    """Split-KV factor for a call: 1 when the (row, 64-head group) items already fill more than
    half the SMs, else as many ranges per row as keep every (item, range) unit in one wave (at
    least one 64-slot block per range, at most 64 ranges)."""
    items = s_q * (h_q // 64)
    sms = torch.cuda.get_device_properties(device).multi_processor_count
    if items == 0 or 2 * items > sms:
        return 1
    # one wave of (item, range) units, each range at least one 64-slot block
    return int(max(1, min(64, sms // items, -(-topk // 64))))


def _workspace(lib, s_q, h_q, n_split, device):
    n = int(lib.sparse_mla_splitkv_workspace_size(int(s_q), int(h_q), int(n_split)))
    if n == 0:
        return None, 0
    return torch.empty(n, dtype=torch.uint8, device=device), n


def sparse_mla_fwd(q, kv, indices, topk_length=None, attn_sink=None, sm_scale=None, d_v=512,
                   out=None, lse=None, max_logits=None, stream=None, n_split=1):
    """q [s_q, h_q, d_qk] bf16; kv [s_kv, 1, d_qk] (or [s_kv, d_qk]) bf16; indices [s_q, 1, topk]
    (or [s_q, topk]) int32; topk_length [s_q] int32 or None; attn_sink [h_q] fp32 or None.
    Returns (out [s_q, h_q, d_v] bf16, lse [s_q, h_q] fp32, max_logits [s_q, h_q] fp32).
    n_split > 1 (or "auto": see auto_splits) runs the split-KV variant with a workspace
    allocated here."""
    lib = load_library()
    _check(q, "q", torch.bfloat16)
    dev = q.device
    _check(kv, "kv", torch.bfloat16, dev)
    _check(indices, "indices", torch.int32, dev)
    _check(topk_length, "topk_length", torch.int32, dev)
    _check(attn_sink, "attn_sink", torch.float32, dev)
    s_q, h_q, d_qk = q.shape
    s_kv = kv.shape[0]
    if kv.numel() != s_kv * d_qk:
        raise ValueError("kv must be [s_kv, 1, d_qk] with the d_qk of q")
    topk = indices.shape[-1] if indices.dim() else 0
    if indices.numel() != s_q * topk:
        raise ValueError("indices must be [s_q, 1, topk]")
    if topk_length is not None and topk_length.numel() != s_q:
        raise ValueError("topk_length must have s_q entries")
    if attn_sink is not None and attn_sink.numel() != h_q:
        raise ValueError("attn_sink must have h_q entries")
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(d_qk)
    out, lse, max_logits = _outputs(q, h_q, d_v, out, lse, max_logits)
    if n_split == "auto":
        n_split = auto_splits(s_q, h_q, topk, dev)
    with torch.cuda.device(dev):
        if n_split == 1:
            rc = lib.sparse_mla_fwd(_ptr(q), _ptr(kv), _ptr(indices), _ptr(topk_length), _ptr(attn_sink),
                                    float(sm_scale), int(d_v), _ptr(out), _ptr(lse), _ptr(max_logits),
                                    int(s_q), int(s_kv), int(h_q), int(d_qk), int(topk),
                                    _stream_handle(stream, dev))
        else:
            ws, nbytes = _workspace(lib, s_q, h_q, n_split, dev)
            rc = lib.sparse_mla_fwd_splitkv(_ptr(q), _ptr(kv), _ptr(indices), _ptr(topk_length),
                                            _ptr(attn_sink), float(sm_scale), int(d_v), _ptr(out), _ptr(lse),
                                            _ptr(max_logits), int(s_q), int(s_kv), int(h_q), int(d_qk),
                                            int(topk), int(n_split), _ptr(ws), int(nbytes),
                                            _stream_handle(stream, dev))
    if rc != 0:
        raise SmlaError(rc, "sparse_mla_fwd")
    return out, lse, max_logits


def sparse_mla_fwd_paged(q, kv_pool, block_table, indices, page_block=64, seqlens_k=None,
                         s_kv_per_req=None, s_q_per_req=1, topk_length=None, attn_sink=None,
                         sm_scale=None, d_v=512, out=None, lse=None, max_logits=None, stream=None,
                         n_split=1):
    """Paged-KV variant: kv_pool [n_pages*page_block, 1, d_qk] bf16, block_table [n_req,
    max_blocks] int32, seqlens_k [n_req] int32 or None (then every request has s_kv_per_req
    tokens); indices hold token positions within the row's request."""
    lib = load_library()
    _check(q, "q", torch.bfloat16)
    dev = q.device
    _check(kv_pool, "kv_pool", torch.bfloat16, dev)
    _check(block_table, "block_table", torch.int32, dev)
    _check(indices, "indices", torch.int32, dev)
    _check(seqlens_k, "seqlens_k", torch.int32, dev)
    _check(topk_length, "topk_length", torch.int32, dev)
    _check(attn_sink, "attn_sink", torch.float32, dev)
    s_q, h_q, d_qk = q.shape
    pool_rows = kv_pool.shape[0]
    if kv_pool.numel() != pool_rows * d_qk:
        raise ValueError("kv_pool must be [rows, 1, d_qk] with the d_qk of q")
    if block_table.dim() != 2:
        raise ValueError("block_table must be [n_req, max_blocks]")
    max_blocks = block_table.shape[1]
    if s_kv_per_req is None:
        s_kv_per_req = max_blocks * page_block
    topk = indices.shape[-1] if indices.dim() else 0
    if indices.numel() != s_q * topk:
        raise ValueError("indices must be [s_q, 1, topk]")
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(d_qk)
    out, lse, max_logits = _outputs(q, h_q, d_v, out, lse, max_logits)
    if n_split == "auto":
        n_split = auto_splits(s_q, h_q, topk, dev)
    with torch.cuda.device(dev):
        if n_split == 1:
            rc = lib.sparse_mla_fwd_paged(_ptr(q), _ptr(kv_pool), int(pool_rows), _ptr(block_table),
                                          int(max_blocks), int(page_block), _ptr(seqlens_k),
                                          int(s_kv_per_req), int(s_q_per_req), _ptr(indices),
                                          _ptr(topk_length), _ptr(attn_sink), float(sm_scale), int(d_v),
                                          _ptr(out), _ptr(lse), _ptr(max_logits), int(s_q), int(h_q),
                                          int(d_qk), int(topk), _stream_handle(stream, dev))
        else:
            ws, nbytes = _workspace(lib, s_q, h_q, n_split, dev)
            rc = lib.sparse_mla_fwd_paged_splitkv(
                _ptr(q), _ptr(kv_pool), int(pool_rows), _ptr(block_table), int(max_blocks), int(page_block),
                _ptr(seqlens_k), int(s_kv_per_req), int(s_q_per_req), _ptr(indices), _ptr(topk_length),
                _ptr(attn_sink), float(sm_scale), int(d_v), _ptr(out), _ptr(lse), _ptr(max_logits), int(s_q),
                int(h_q), int(d_qk), int(topk), int(n_split), _ptr(ws), int(nbytes), _stream_handle(stream, dev))
    if rc != 0:
        raise SmlaError(rc, "sparse_mla_fwd_paged")
    return out, lse, max_logits


def sparse_mla_fwd_paged_splitkv_static(q, kv_pool, block_table, indices, n_split, page_block=64,
                                        seqlens_k=None, s_kv_per_req=None, s_q_per_req=1, topk_length=None,
                                        attn_sink=None, sm_scale=None, d_v=512, out=None, lse=None,
                                        max_logits=None, stream=None):
    """Split-KV paged forward whose partial results use the library's own 32 MiB scratch array
    (no workspace is allocated anywhere).  Calls on one device must not overlap; see the C
    header."""
    lib = load_library()
    _check(q, "q", torch.bfloat16)
    dev = q.device
    _check(kv_pool, "kv_pool", torch.bfloat16, dev)
    _check(block_table, "block_table", torch.int32, dev)
    _check(indices, "indices", torch.int32, dev)
    _check(seqlens_k, "seqlens_k", torch.int32, dev)
    _check(topk_length, "topk_length", torch.int32, dev)
    _check(attn_sink, "attn_sink", torch.float32, dev)
    s_q, h_q, d_qk = q.shape
    pool_rows = kv_pool.shape[0]
    max_blocks = block_table.shape[1]
    if s_kv_per_req is None:
        s_kv_per_req = max_blocks * page_block
    topk = indices.shape[-1] if indices.dim() else 0
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(d_qk)
    out, lse, max_logits = _outputs(q, h_q, d_v, out, lse, max_logits)
    with torch.cuda.device(dev):
        rc = lib.sparse_mla_fwd_paged_splitkv_static(
            _ptr(q), _ptr(kv_pool), int(pool_rows), _ptr(block_table), int(max_blocks), int(page_block),
            _ptr(seqlens_k), int(s_kv_per_req), int(s_q_per_req), _ptr(indices), _ptr(topk_length),
            _ptr(attn_sink), float(sm_scale), int(d_v), _ptr(out), _ptr(lse), _ptr(max_logits), int(s_q),
            int(h_q), int(d_qk), int(topk), int(n_split), _stream_handle(stream, dev))
    if rc != 0:
        raise SmlaError(rc, "sparse_mla_fwd_paged_splitkv_static")
    return out, lse, max_logits


def sparse_mla_bwd(q, kv, out, dout, indices, lse, topk_length=None, attn_sink=None, sm_scale=None,
                   d_v=512, dq=None, dkv=None, dsink=None, stream=None):
    """Gradients of sum(dout * out) through the forward: q, kv, indices, topk_length, attn_sink and
    sm_scale as passed to :func:`sparse_mla_fwd`; out [s_q, h_q, d_v] bf16 and lse [s_q, h_q]
    fp32 as it returned them; dout [s_q, h_q, d_v] bf16.  Returns (dq [s_q, h_q, d_qk] fp32,
    dkv [s_kv, d_qk] fp32, dsink [h_q] fp32 or None)."""
    lib = load_library()
    _check(q, "q", torch.bfloat16)
    dev = q.device
    _check(kv, "kv", torch.bfloat16, dev)
    _check(out, "out", torch.bfloat16, dev)
    _check(dout, "dout", torch.bfloat16, dev)
    _check(indices, "indices", torch.int32, dev)
    _check(lse, "lse", torch.float32, dev)
    _check(topk_length, "topk_length", torch.int32, dev)
    _check(attn_sink, "attn_sink", torch.float32, dev)
    s_q, h_q, d_qk = q.shape
    s_kv = kv.shape[0]
    if kv.numel() != s_kv * d_qk:
        raise ValueError("kv must be [s_kv, 1, d_qk] with the d_qk of q")
    topk = indices.shape[-1] if indices.dim() else 0
    if indices.numel() != s_q * topk:
        raise ValueError("indices must be [s_q, 1, topk]")
    if out.numel() != s_q * h_q * d_v or dout.numel() != s_q * h_q * d_v or lse.numel() != s_q * h_q:
        raise ValueError("out / dout must be [s_q, h_q, d_v] and lse [s_q, h_q]")
    if topk_length is not None and topk_length.numel() != s_q:
        raise ValueError("topk_length must have s_q entries")
    if attn_sink is not None and attn_sink.numel() != h_q:
        raise ValueError("attn_sink must have h_q entries")
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(d_qk)
    if dq is None:
        dq = torch.empty((s_q, h_q, d_qk), dtype=torch.float32, device=dev)
    if dkv is None:
        dkv = torch.empty((s_kv, d_qk), dtype=torch.float32, device=dev)
    if dsink is None and attn_sink is not None:
        dsink = torch.empty((h_q,), dtype=torch.float32, device=dev)
    _check(dq, "dq", torch.float32, dev)
    _check(dkv, "dkv", torch.float32, dev)
    _check(dsink, "dsink", torch.float32, dev)
    with torch.cuda.device(dev):
        rc = lib.sparse_mla_bwd(_ptr(q), _ptr(kv), _ptr(out), _ptr(dout), _ptr(indices), _ptr(topk_length),
                                _ptr(attn_sink), _ptr(lse), float(sm_scale), int(d_v), _ptr(dq), _ptr(dkv),
                                _ptr(dsink), int(s_q), int(s_kv), int(h_q), int(d_qk), int(topk),
                                _stream_handle(stream, dev))
    if rc != 0:
        raise SmlaError(rc, "sparse_mla_bwd")
    return dq, dkv, dsink


def _dense(t, name, dtype, dev=None):
    """_check for a required tensor, with one test in the usual case; returns its device."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.is_contiguous():
        at = t.device
        if at == dev or (dev is None and t.is_cuda):
            return at
    _check(t, name, dtype, dev)
    raise TypeError(f"{name} must be a torch.Tensor")


def _int_output(t, name, n, dev):
    """An int32 output [n]: the caller's, or a new one on the current device."""
    if t is None:
        return _empty_strided((n,), (1,), torch.int32)
    _dense(t, name, torch.int32, dev)
    if t.shape != (n,):
        raise ValueError(f"{name} must be [{n}], got {list(t.shape)}")
    return t


def _strided(t, name, shape, dev):
    """The strides of a bf16 tensor of this shape whose last dimension is contiguous."""
    if isinstance(t, torch.Tensor) and t.dtype is torch.bfloat16 and t.device == dev and t.shape == shape:
        strides = t.stride()
        if strides[-1] == 1 or t.numel() == 0:
            return strides
        raise ValueError(f"{name} must be contiguous in its last dimension")
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be a torch.bfloat16 tensor")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")


def _on_device(fn, dev, stream, *args, **kwargs):
    """Calls fn again with `stream` as the current one, so that what it allocates belongs to the stream
    that uses it, or with the tensors' device as the current one."""
    if stream is not None:
        if stream.device != dev:
            raise ValueError(f"stream is on {stream.device}, the tensors are on {dev}")
        with torch.cuda.stream(stream):
            return fn(*args, **kwargs)
    with torch.cuda.device(dev):
        return fn(*args, **kwargs)


def sparse_mla_plan_pages(seqlens, new_lens, block_table, free_pages, n_tokens, page_block=64, free_start=None,
                          seqlens_k=None, cu_seqlens_q=None, slots=None, positions=None, counts=None, stream=None):
    """Pages and rows of one step's new tokens, planned on the device.  seqlens [n_req] and new_lens
    [n_req] int32: cached and new tokens of each request; block_table [n_req, max_blocks] int32:
    updated in place with the new pages; free_pages [n_free] int32, handed out from index
    free_start [1] (int32, None: 0); n_tokens: length of the token arrays, at least the step's
    tokens (the rest is padding).  Returns int32 tensors (allocated here when not given):
    seqlens_k [n_req], cu_seqlens_q [n_req + 1], slots [n_tokens] and positions [n_tokens] (-1 for
    padding; a slot is also -1 where there is no page), counts [3] = tokens placed, next free_start,
    pages that were missing.  See the C header for the exact rules."""
    lib = load_library()
    i32 = torch.int32
    dev = _dense(seqlens, "seqlens", i32)
    if stream is not None or torch.cuda.current_device() != dev.index:
        return _on_device(sparse_mla_plan_pages, dev, stream, seqlens, new_lens, block_table, free_pages, n_tokens, page_block,
                          free_start, seqlens_k, cu_seqlens_q, slots, positions, counts)
    _dense(new_lens, "new_lens", i32, dev)
    _dense(block_table, "block_table", i32, dev)
    _dense(free_pages, "free_pages", i32, dev)
    n_req, n_tokens = seqlens.numel(), int(n_tokens)
    if n_tokens < 0:
        raise ValueError("n_tokens must be at least 0")
    if new_lens.numel() != n_req:
        raise ValueError("new_lens must have one entry per request")
    table_shape = block_table.shape
    if len(table_shape) != 2 or table_shape[0] != n_req:
        raise ValueError("block_table must be [n_req, max_blocks]")
    if free_start is not None:
        _dense(free_start, "free_start", i32, dev)
        if free_start.numel() != 1:
            raise ValueError("free_start must have one entry")
    k, cu = _int_output(seqlens_k, "seqlens_k", n_req, dev), _int_output(cu_seqlens_q, "cu_seqlens_q", n_req + 1, dev)
    sl, pos = _int_output(slots, "slots", n_tokens, dev), _int_output(positions, "positions", n_tokens, dev)
    cnt = _int_output(counts, "counts", 3, dev)
    rc = lib.sparse_mla_plan_pages(
        seqlens.data_ptr(), new_lens.data_ptr(), block_table.data_ptr(), free_pages.data_ptr(), _ptr(free_start),
        k.data_ptr(), cu.data_ptr(), sl.data_ptr(), pos.data_ptr(), cnt.data_ptr(), n_req, free_pages.numel(), n_tokens,
        table_shape[1], int(page_block), _raw_stream(dev.index))
    if rc != 0:
        raise SmlaError(rc, "sparse_mla_plan_pages")
    return k, cu, sl, pos, cnt


def sparse_mla_append_kv(c_kv, k_pe, slots, kv_pool, norm_weight=None, eps=1e-6, positions=None, rope=None, q_pe=None,
                         q=None, stream=None, past_rope=None):
    """Writes the rows of n new tokens into the paged cache: the latent part c_kv [n, 512] bf16
    (RMS-normalised with norm_weight [512] bf16 and eps when given) and, for d_qk 576, the rotary
    part k_pe [n, 64] bf16 (turned pair by pair when rope is given), to row slots[t] (int32; a
    token whose slot lies outside the pool is not written) of kv_pool [rows, 1, d_qk] bf16.  rope
    [max_pos, 64] fp32 holds 32 cosines and 32 sines per position, positions [n] int32 the tokens'.
    Outside the table nothing is written: negative positions are padding; one at or past max_pos
    leaves its request without that row, and past_rope [1] int32, when given, is increased by the
    number of such tokens (a table of max_blocks * page_block positions covers every row that the
    planner gives).  With q_pe [n, h, 64] bf16, q[..., 512:] of q
    [n, h, 576] gets the queries' columns turned by the same angles.  c_kv, k_pe and q_pe may be
    strided views (slices of a projection's output) with a contiguous last dimension, the other strides
    even for k_pe and multiples of eight for c_kv and q_pe.  Returns kv_pool."""
    lib = load_library()
    bf16 = torch.bfloat16
    dev = _dense(kv_pool, "kv_pool", bf16)
    if stream is not None or torch.cuda.current_device() != dev.index:
        return _on_device(sparse_mla_append_kv, dev, stream, c_kv, k_pe, slots, kv_pool, norm_weight, eps, positions, rope, q_pe, q,
                          past_rope=past_rope)
    _dense(slots, "slots", torch.int32, dev)
    pool_shape = kv_pool.shape
    n, d_qk, pool_rows = slots.numel(), pool_shape[-1] if len(pool_shape) > 1 else 0, pool_shape[0]
    if d_qk not in (512, 576) or kv_pool.numel() != pool_rows * d_qk:
        raise ValueError("kv_pool must be [rows, 1, d_qk] with d_qk 512 or 576")
    c_stride, k_stride, q_strides, h_q, max_pos = _strided(c_kv, "c_kv", (n, 512), dev)[0], 0, (0, 0), 0, 0
    if (k_pe is not None) != (d_qk == 576):
        raise ValueError("k_pe must be given exactly when d_qk is 576")
    if k_pe is not None:
        k_stride = _strided(k_pe, "k_pe", (n, 64), dev)[0]
    if norm_weight is not None:
        _dense(norm_weight, "norm_weight", bf16, dev)
        if norm_weight.numel() != 512:
            raise ValueError("norm_weight must have 512 entries")
    if rope is not None:
        if d_qk != 576 or positions is None:
            raise ValueError("rope needs positions and d_qk 576")
        _dense(rope, "rope", torch.float32, dev)
        _dense(positions, "positions", torch.int32, dev)
        rope_shape = rope.shape
        if len(rope_shape) != 2 or rope_shape[1] != 64 or rope_shape[0] < 1:
            raise ValueError("rope must be [max_pos, 64]")
        max_pos = rope_shape[0]
        if positions.numel() != n:
            raise ValueError("positions must have one entry per token")
    else:
        positions = None
    if (q_pe is None) != (q is None) or (q_pe is not None and rope is None):
        raise ValueError("q_pe and q come together, and need rope")
    if q is not None:
        _dense(q, "q", bf16, dev)
        q_shape = q.shape
        if len(q_shape) != 3 or q_shape[0] != n or q_shape[2] != 576:
            raise ValueError("q must be [n, h, 576]")
        h_q = q_shape[1]
        q_strides = _strided(q_pe, "q_pe", (n, h_q, 64), dev)
    if past_rope is not None:
        _dense(past_rope, "past_rope", torch.int32, dev)
        if past_rope.numel() != 1:
            raise ValueError("past_rope must have one entry")
    if n == 0:
        return kv_pool
    append, last = (lib.sparse_mla_append_kv, ()) if past_rope is None else \
        (lib.sparse_mla_append_kv_counted, (past_rope.data_ptr(),))
    rc = append(
        c_kv.data_ptr(), c_stride, _ptr(k_pe), k_stride, slots.data_ptr(), _ptr(positions), _ptr(rope), max_pos,
        _ptr(norm_weight), float(eps), _ptr(q_pe), q_strides[0], q_strides[1], _ptr(q), h_q, kv_pool.data_ptr(), pool_rows,
        d_qk, n, *last, _raw_stream(dev.index))
    if rc != 0:
        raise SmlaError(rc, "sparse_mla_append_kv")
    return kv_pool


def sparse_mla_chunk_fwd_paged(q, kv_pool, block_table, cu_seqlens_q, seqlens_k, page_block=64, causal=True,
                               attn_sink=None, sm_scale=None, d_v=512, out=None, lse=None, max_logits=None,
                               workspace=None, stream=None):
    """Dense attention of each request's new tokens over its paged cache.  q [n_tok, h, d_qk] bf16
    (any h up to 1024), rows cu_seqlens_q[b] .. cu_seqlens_q[b+1]-1 being request b's new tokens;
    kv_pool, block_table and page_block as for :func:`sparse_mla_fwd_paged`; seqlens_k [n_req] int32
    counts the cached keys with the new tokens' own; causal: a token sees the positions up to its
    own, else every key.  Returns (out [n_tok, h, d_v] bf16, lse [n_tok, h] fp32, max_logits [n_tok,
    h] fp32); rows of no request are not written.  `workspace` (uint8, at least
    sparse_mla_chunk_workspace_size bytes, 256-byte aligned) is allocated here when not given; calls
    that may overlap must not share one."""
    lib = load_library()
    bf16, i32, f32 = torch.bfloat16, torch.int32, torch.float32
    dev = _dense(q, "q", bf16)
    if stream is not None or torch.cuda.current_device() != dev.index:
        return _on_device(sparse_mla_chunk_fwd_paged, dev, stream, q, kv_pool, block_table, cu_seqlens_q, seqlens_k, page_block,
                          causal, attn_sink, sm_scale, d_v, out, lse, max_logits, workspace)
    _dense(kv_pool, "kv_pool", bf16, dev)
    _dense(block_table, "block_table", i32, dev)
    _dense(cu_seqlens_q, "cu_seqlens_q", i32, dev)
    _dense(seqlens_k, "seqlens_k", i32, dev)
    q_shape, pool_shape, table_shape = q.shape, kv_pool.shape, block_table.shape
    if len(q_shape) != 3:
        raise ValueError("q must be [n_tok, h, d_qk]")
    n_tok, h_q, d_qk = q_shape
    pool_rows = pool_shape[0] if len(pool_shape) else 0
    if kv_pool.numel() != pool_rows * d_qk:
        raise ValueError("kv_pool must be [rows, 1, d_qk] with the d_qk of q")
    if len(table_shape) != 2:
        raise ValueError("block_table must be [n_req, max_blocks]")
    n_req, max_blocks = table_shape
    if seqlens_k.numel() != n_req or cu_seqlens_q.numel() != n_req + 1:
        raise ValueError("seqlens_k must have n_req entries and cu_seqlens_q n_req + 1")
    if attn_sink is not None:
        _dense(attn_sink, "attn_sink", f32, dev)
        if attn_sink.numel() != h_q:
            raise ValueError("attn_sink must have h entries")
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(d_qk) if d_qk else 1.0
    if out is None and lse is None and max_logits is None:
        out = _empty_strided((n_tok, h_q, d_v), (h_q * d_v, d_v, 1), bf16)
        lse = _empty_strided((n_tok, h_q), (h_q, 1), f32)
        max_logits = _empty_strided((n_tok, h_q), (h_q, 1), f32)
    else:
        out, lse, max_logits = _outputs(q, h_q, d_v, out, lse, max_logits)
    if workspace is None:
        ws_bytes = lib.sparse_mla_chunk_workspace_size(n_tok, h_q)
        workspace = _empty_strided((ws_bytes,), (1,), torch.uint8)
    else:
        _dense(workspace, "workspace", torch.uint8, dev)
        ws_bytes = workspace.numel()
    rc = lib.sparse_mla_chunk_fwd_paged(
        q.data_ptr(), kv_pool.data_ptr(), pool_rows, block_table.data_ptr(), max_blocks, int(page_block),
        cu_seqlens_q.data_ptr(), seqlens_k.data_ptr(), n_req, 1 if causal else 0, _ptr(attn_sink), float(sm_scale), int(d_v),
        out.data_ptr(), lse.data_ptr(), max_logits.data_ptr(), n_tok, h_q, d_qk, workspace.data_ptr(), ws_bytes,
        _raw_stream(dev.index))
    if rc != 0:
        raise SmlaError(rc, "sparse_mla_chunk_fwd_paged")
    return out, lse, max_logits


def sparse_mla_device_status(reset=False) -> int:
    """Device-side status (0, or 5 = a bounded wait of some kernel gave up); synchronises."""
    lib, reset = load_library(), 1 if reset else 0
    words = int(lib.sparse_mla_device_status(reset)), int(lib.sparse_mla_chunk_device_status(reset))
    return words[0] or words[1]


def sparse_mla_status_string(code: int) -> str:
    return status_string(code)
