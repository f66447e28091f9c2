"""PyTorch-facing binding of the C ABI (include/mla_qcache.h).

The functions carry the C entry points' names and only marshal arguments:
they check dtypes, devices and contiguity, allocate outputs and workspace
through PyTorch when the caller passes none, and hand raw pointers plus the
current CUDA stream to the library. Nothing is computed here.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os

import torch

from . import _lib
from ._lib import MlaError, check, make_desc, mla_qcache_desc  # noqa: F401

D_C, D_R, PAGE = 512, 64, 64


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _need(t: torch.Tensor, name: str, dtype, shape=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t.data_ptr()


def mla_qcache_page_bytes(desc: mla_qcache_desc) -> int:
    return int(_lib.load().mla_qcache_page_bytes(ctypes.byref(desc)))


def mla_qcache_segment_offsets(desc: mla_qcache_desc):
    out = (ctypes.c_size_t * 5)()
    check("mla_qcache_segment_offsets", _lib.load().mla_qcache_segment_offsets(ctypes.byref(desc), out))
    return tuple(int(v) for v in out)


def new_qcache_pool(desc: mla_qcache_desc, device="cuda") -> torch.Tensor:
    """uint8 pool [num_pages, page_bytes] (PyTorch allocations are 256-byte aligned)."""
    return torch.zeros((desc.num_pages, mla_qcache_page_bytes(desc)), dtype=torch.uint8, device=device)


def new_bf16_pool(num_pages: int, device="cuda") -> torch.Tensor:
    return torch.zeros((num_pages, PAGE, D_C + D_R), dtype=torch.bfloat16, device=device)


def mla_qcache_append(desc, pool, block_table, seq_lens_before, c_new, kr_new, stream=None) -> None:
    B, n = c_new.shape[0], c_new.shape[1]
    args = (_need(pool, "pool", torch.uint8), _need(block_table, "block_table", torch.int32),
            block_table.shape[1], _need(seq_lens_before, "seq_lens_before", torch.int32, (B,)),
            _need(c_new, "c_new", torch.bfloat16, (B, n, D_C)), _need(kr_new, "kr_new", torch.bfloat16, (B, n, D_R)))
    check("mla_qcache_append",
          _lib.load().mla_qcache_append(ctypes.byref(desc), *args, B, n, _stream(stream)))


def mla_bf16cache_append(pool, block_table, seq_lens_before, c_new, kr_new, stream=None) -> None:
    B, n = c_new.shape[0], c_new.shape[1]
    check("mla_bf16cache_append", _lib.load().mla_bf16cache_append(
        _need(pool, "pool", torch.bfloat16), pool.shape[0], pool.shape[1],
        _need(block_table, "block_table", torch.int32), block_table.shape[1],
        _need(seq_lens_before, "seq_lens_before", torch.int32, (B,)),
        _need(c_new, "c_new", torch.bfloat16, (B, n, D_C)), _need(kr_new, "kr_new", torch.bfloat16, (B, n, D_R)),
        B, n, _stream(stream)))


def mla_decode_num_splits(B, s_q, H, max_seq_len, num_splits=0) -> int:
    return int(_lib.load().mla_decode_num_splits(B, s_q, H, max_seq_len, num_splits))


def mla_decode_workspace_bytes(B, s_q, H, max_seq_len, num_splits=0) -> int:
    return int(_lib.load().mla_decode_workspace_bytes(B, s_q, H, max_seq_len, num_splits))


def _decode_io(q_c, q_r, out, out_dtype, lse, workspace, max_seq_len, num_splits):
    B, s_q, H = q_c.shape[:3]
    qc = _need(q_c, "q_c", torch.bfloat16, (B, s_q, H, D_C))
    qr = _need(q_r, "q_r", torch.bfloat16, (B, s_q, H, D_R))
    if out is None:
        out = torch.empty((B, s_q, H, D_C), dtype=out_dtype, device=q_c.device)
    if out.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("out must be bfloat16 or float32")
    po = _need(out, "out", out.dtype, (B, s_q, H, D_C))
    pl = None
    if lse is not None:
        pl = _need(lse, "lse", torch.float32, (B, s_q, H))
    need = mla_decode_workspace_bytes(B, s_q, H, max_seq_len, num_splits)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=q_c.device)
    pw, nw = (None, 0) if workspace is None else (_need(workspace, "workspace", torch.uint8), workspace.numel())
    return (B, s_q, H), qc, qr, out, po, pl, pw, nw, int(out.dtype == torch.float32), workspace


def mla_qdecode(desc, pool, block_table, seq_lens, max_seq_len, q_c, q_r, scale, *, out=None,
                out_dtype=torch.bfloat16, lse=None, num_splits=0, workspace=None, flags=0, stream=None):
    """Returns (out, lse). See include/mla_qcache.h for the contract."""
    (B, s_q, H), qc, qr, out, po, pl, pw, nw, f32, _ = _decode_io(
        q_c, q_r, out, out_dtype, lse, workspace, max_seq_len, num_splits)
    B_ = seq_lens.shape[0]
    if B_ != B:
        raise ValueError("seq_lens must have one entry per request")
    check("mla_qdecode", _lib.load().mla_qdecode(
        ctypes.byref(desc), _need(pool, "pool", torch.uint8), _need(block_table, "block_table", torch.int32),
        block_table.shape[1], _need(seq_lens, "seq_lens", torch.int32), int(max_seq_len), qc, qr, B, s_q, H,
        float(scale), int(num_splits), pw, nw, po, f32, pl, int(flags), _stream(stream)))
    return out, lse


def mla_qdecode_noalloc(desc, pool, block_table, seq_lens, max_seq_len, q_c, q_r, scale, out, lse=None, *,
                        num_splits=0, flags=0, stream=None):
    """mla_qdecode without a workspace argument, for callers that cannot
    allocate: the split-KV scratch is a fixed array inside the library (see
    include/mla_qcache.h). `out` must be given; nothing is allocated here."""
    B, s_q, H = q_c.shape[:3]
    f32 = {torch.float32: 1, torch.bfloat16: 0}[out.dtype]
    check("mla_qdecode_noalloc", _lib.load().mla_qdecode_noalloc(
        ctypes.byref(desc), _need(pool, "pool", torch.uint8), _need(block_table, "block_table", torch.int32),
        block_table.shape[1], _need(seq_lens, "seq_lens", torch.int32, (B,)), int(max_seq_len),
        _need(q_c, "q_c", torch.bfloat16, (B, s_q, H, D_C)), _need(q_r, "q_r", torch.bfloat16, (B, s_q, H, D_R)),
        B, s_q, H, float(scale), int(num_splits), _need(out, "out", out.dtype, (B, s_q, H, D_C)), f32,
        None if lse is None else _need(lse, "lse", torch.float32, (B, s_q, H)), int(flags), _stream(stream)))
    return out, lse


def mla_qdecode_fused_append(desc, pool, block_table, seq_lens, max_seq_len, c_new, kr_new, q_c, q_r, scale, *,
                             out=None, out_dtype=torch.bfloat16, lse=None, num_splits=0, workspace=None, flags=0,
                             stream=None):
    """Append the step's new tokens (c_new [B, n, 512], kr_new [B, n, 64]; seq_lens count them) and
    decode, in one call. Returns (out, lse). See include/mla_qcache.h for the contract."""
    (B, s_q, H), qc, qr, out, po, pl, pw, nw, f32, _ = _decode_io(
        q_c, q_r, out, out_dtype, lse, workspace, max_seq_len, num_splits)
    if seq_lens.shape[0] != B or c_new.shape[0] != B:
        raise ValueError("seq_lens and c_new must have one entry per request")
    n = c_new.shape[1]
    check("mla_qdecode_fused_append", _lib.load().mla_qdecode_fused_append(
        ctypes.byref(desc), _need(pool, "pool", torch.uint8), _need(block_table, "block_table", torch.int32),
        block_table.shape[1], _need(seq_lens, "seq_lens", torch.int32), int(max_seq_len),
        _need(c_new, "c_new", torch.bfloat16, (B, n, D_C)), _need(kr_new, "kr_new", torch.bfloat16, (B, n, D_R)), n,
        qc, qr, B, s_q, H, float(scale), int(num_splits), pw, nw, po, f32, pl, int(flags), _stream(stream)))
    return out, lse


def mla_decode_bf16(pool, block_table, seq_lens, max_seq_len, q_c, q_r, scale, *, out=None,
                    out_dtype=torch.bfloat16, lse=None, num_splits=0, workspace=None, flags=0, stream=None):
    (B, s_q, H), qc, qr, out, po, pl, pw, nw, f32, _ = _decode_io(
        q_c, q_r, out, out_dtype, lse, workspace, max_seq_len, num_splits)
    check("mla_decode_bf16", _lib.load().mla_decode_bf16(
        _need(pool, "pool", torch.bfloat16), pool.shape[0], pool.shape[1],
        _need(block_table, "block_table", torch.int32), block_table.shape[1],
        _need(seq_lens, "seq_lens", torch.int32), int(max_seq_len), qc, qr, B, s_q, H, float(scale),
        int(num_splits), pw, nw, po, f32, pl, int(flags), _stream(stream)))
    return out, lse


def mla_qcache_append_bf16_pages(desc, pool, block_table, seq_lens_before, bf16_pool, src_pages, stream=None) -> None:
    """Quantize whole BF16 pages (src_pages[b] of bf16_pool, or -1) into the quantized cache at
    positions seq_lens_before[b] .. + 63. See include/mla_qcache.h."""
    B = src_pages.shape[0]
    check("mla_qcache_append_bf16_pages", _lib.load().mla_qcache_append_bf16_pages(
        ctypes.byref(desc), _need(pool, "pool", torch.uint8), _need(block_table, "block_table", torch.int32),
        block_table.shape[1], _need(seq_lens_before, "seq_lens_before", torch.int32, (B,)),
        _need(bf16_pool, "bf16_pool", torch.bfloat16), bf16_pool.shape[0],
        _need(src_pages, "src_pages", torch.int32, (B,)), B, _stream(stream)))


def mla_qdecode_hybrid_workspace_bytes(B, s_q, H, max_hist_len, max_prot_len) -> int:
    return int(_lib.load().mla_qdecode_hybrid_workspace_bytes(B, s_q, H, max_hist_len, max_prot_len))


def mla_qdecode_hybrid(desc, pool, block_table, hist_lens, max_hist_len, bf16_pool, prot_table, prot_lens,
                       max_prot_len, q_c, q_r, scale, *, out=None, out_dtype=torch.bfloat16, lse=None,
                       workspace=None, stream=None):
    """Decode over a hybrid cache (quantized history + BF16 sink and window). Returns (out, lse)."""
    B, s_q, H = q_c.shape[:3]
    qc = _need(q_c, "q_c", torch.bfloat16, (B, s_q, H, D_C))
    qr = _need(q_r, "q_r", torch.bfloat16, (B, s_q, H, D_R))
    if out is None:
        out = torch.empty((B, s_q, H, D_C), dtype=out_dtype, device=q_c.device)
    po = _need(out, "out", out.dtype, (B, s_q, H, D_C))
    pl = None if lse is None else _need(lse, "lse", torch.float32, (B, s_q, H))
    need = mla_qdecode_hybrid_workspace_bytes(B, s_q, H, max_hist_len, max_prot_len)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q_c.device)
    check("mla_qdecode_hybrid", _lib.load().mla_qdecode_hybrid(
        ctypes.byref(desc), _need(pool, "pool", torch.uint8), _need(block_table, "block_table", torch.int32),
        block_table.shape[1], _need(hist_lens, "hist_lens", torch.int32, (B,)), int(max_hist_len),
        _need(bf16_pool, "bf16_pool", torch.bfloat16), bf16_pool.shape[0],
        _need(prot_table, "prot_table", torch.int32), prot_table.shape[1],
        _need(prot_lens, "prot_lens", torch.int32, (B,)), int(max_prot_len), qc, qr, B, s_q, H, float(scale),
        _need(workspace, "workspace", torch.uint8), workspace.numel(), po, int(out.dtype == torch.float32), pl,
        _stream(stream)))
    return out, lse


# The operators around the decode are bound in C++ (csrc/torch_binding.cpp): same checks, a
# quarter of the host time a call.
_binding = None


def _ext():
    global _binding
    if _binding is None:
        _lib.load()
        path = _lib.binding_path()
        if not os.path.exists(path) and os.environ.get("MLA_BUILD_ON_IMPORT") == "1":
            _lib.build_binding()
        if not os.path.exists(path):
            raise ImportError(f"PyTorch binding {path} is missing: build it with "
                              "`python -m bit_mla_kv_qdecode_b200.build`")
        spec = importlib.util.spec_from_file_location("_mla_torch", path)
        m = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(m)
        m.set_error(MlaError)
        _binding = m
    return _binding


def _handle(stream):
    return None if stream is None else stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


_ROPE_PAIRS = {"interleaved": _lib.MLA_ROPE_INTERLEAVED, "half": _lib.MLA_ROPE_HALF}


def mla_qcache_append_norm_rope(desc, pool, block_table, seq_lens_before, kv, norm_weight, eps, cos_sin, *,
                                convention="interleaved", q=None, q_out=None, positions=None, new_lens=None,
                                rows_out=None, stream=None):
    """Append from the raw projections: RMS norm of the latent, rotation of the key and of the
    queries, quantize and write. kv [B, n, 576] and q [B, n, H, 64] may be column ranges of wider
    tensors; norm_weight may be None (ones); convention names the rotary pairs as in
    fold.rotary_pairs. Returns q_out [B, n, H, 64] (None without q). See include/mla_qcache.h."""
    pairs = _ROPE_PAIRS.get(convention)
    if pairs is None:
        raise ValueError(f"unknown rotary convention {convention!r}")
    return _ext().append_norm_rope(ctypes.addressof(desc), pool, block_table, seq_lens_before, kv, norm_weight, eps, cos_sin,
                                   pairs, q, q_out, positions, new_lens, rows_out, _handle(stream))


def mla_qcache_read(desc, pool, block_table, start, cu_rows, max_rows, out_c=None, out_kr=None, stream=None) -> None:
    """Read dequantized rows back: tokens start[b] + i (start None: 0) of request b into row
    cu_rows[b] + i of out_c [rows, 512] and out_kr [rows, 64] (bf16; either may be None, and both may
    be column ranges of one buffer). max_rows bounds the rows of one request."""
    _ext().qcache_read(ctypes.addressof(desc), pool, block_table, start, cu_rows, max_rows, out_c, out_kr, _handle(stream))


def mla_page_digest(desc, pool, block_table, seq_lens_before, n_new, digests, *, new_lens=None, stream=None) -> None:
    """Mean keys of the pages that appending new_lens[b] (None: n_new) tokens completed, into the
    pages' rows of digests [num_pages, 576] (bf16). Call it after the append."""
    _ext().page_digest(ctypes.addressof(desc), pool, block_table, seq_lens_before, n_new, digests, new_lens, _handle(stream))


def new_digests(desc: mla_qcache_desc, device="cuda") -> torch.Tensor:
    """Zeroed bf16 digests [num_pages, 576] of a pool's pages."""
    return torch.zeros((desc.num_pages, D_C + D_R), dtype=torch.bfloat16, device=device)


def mla_page_scores(block_table, seq_lens, max_seq_len, digests, q_c, q_r, scale, *, out=None, stream=None):
    """Expected attention mass of every candidate page, fp32 [B, s_q, ceil(max_seq_len / 64)] (-inf
    for pages that are no candidates). See include/mla_qcache.h."""
    return _ext().page_scores(block_table, seq_lens, max_seq_len, digests, q_c, q_r, scale, out, _handle(stream))


def mla_select_pages(block_table, seq_lens, max_seq_len, scores, k_pages, *, n_sink=1, n_recent=1, s_q=None,
                     sel_table=None, sel_pages=None, sel_lens=None, stream=None):
    """Pages each query attends: (sel_table [B, s_q, k_pages] pages of the pool, sel_pages their
    indexes in the request, sel_lens [B, s_q] keys), int32, -1 behind the last page. scores
    [B, s_q, ceil(max_seq_len / 64)] may be None when k_pages covers every page (then s_q is needed).
    sel_table and sel_lens, flattened to B * s_q requests, are what mla_qdecode takes."""
    return _ext().select_pages(block_table, seq_lens, max_seq_len, scores, k_pages, n_sink, n_recent, s_q, sel_table,
                               sel_pages, sel_lens, _handle(stream))


def mla_qdecode_sparse_workspace_bytes(B, s_q, H, max_seq_len, k_pages, num_splits=0) -> int:
    return _lib.load().mla_qdecode_sparse_workspace_bytes(B, s_q, H, int(max_seq_len), int(k_pages), int(num_splits))


def mla_qdecode_sparse(desc, pool, block_table, seq_lens, max_seq_len, digests, q_c, q_r, scale, k_pages, *, n_sink=1,
                       n_recent=1, out=None, out_dtype=torch.bfloat16, lse=None, num_splits=0, workspace=None, flags=0,
                       stream=None):
    """One decode step over the pages that the digests' scores select (scores, selection, decode).
    digests may be None when k_pages covers every page. Returns (out, lse). See include/mla_qcache.h."""
    if out is None and out_dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("out must be bfloat16 or float32")
    return _ext().qdecode_sparse(ctypes.addressof(desc), pool, block_table, seq_lens, max_seq_len, digests, q_c, q_r, scale,
                                 k_pages, n_sink, n_recent, out, out_dtype is torch.float32, lse, num_splits, workspace,
                                 flags, _handle(stream)), lse


def mla_cache_bytes_per_request(desc, seq_len, sink=0, window=0) -> int:
    """Bytes one request holds (desc None: the BF16 cache). See include/mla_qcache.h."""
    return int(_lib.load().mla_cache_bytes_per_request(None if desc is None else ctypes.byref(desc),
                                                       int(seq_len), int(sink), int(window)))


def mla_cache_max_requests(desc, seq_len, budget_bytes, sink=0, window=0) -> int:
    return int(_lib.load().mla_cache_max_requests(None if desc is None else ctypes.byref(desc), int(seq_len),
                                                  int(sink), int(window), int(budget_bytes)))


def mla_get_device_status(stream=None) -> int:
    v = ctypes.c_int(0)
    check("mla_get_device_status", _lib.load().mla_get_device_status(ctypes.byref(v), _stream(stream)))
    return int(v.value)
