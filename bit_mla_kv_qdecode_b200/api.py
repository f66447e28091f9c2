"""PyTorch-facing binding of the C ABI (include/mla_qcache.h).

The functions carry the C entry points' names and only marshal arguments:
they check dtypes, devices and contiguity, allocate outputs and workspace
through PyTorch when the caller passes none, and hand raw pointers plus the
current CUDA stream to the library. Nothing is computed here.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from ._lib import MlaError, check, make_desc, mla_qcache_desc  # noqa: F401

D_C, D_R, PAGE = 512, 64, 64
_Tensor, _U8, _I32, _BF16, _F32 = torch.Tensor, torch.uint8, torch.int32, torch.bfloat16, torch.float32


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


def _refuse(t, name, dtype, shape, index):
    """Raise the error of an argument that does not fit (the contiguity check comes last)."""
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on cuda:{index}, got {t.device}")
    raise ValueError(f"{name} must be contiguous")


def _arg(t, name, dtype, shape, index):
    """Address of a dense tensor of this type and shape on CUDA device `index`."""
    if isinstance(t, _Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == index \
            and t.is_contiguous():
        return t.data_ptr()
    _refuse(t, name, dtype, shape, index)


def _opt(t, name, dtype, shape, index):
    return None if t is None else _arg(t, name, dtype, shape, index)


def _device_index(t, name, dtype, dims):
    """CUDA device of the tensor that the other arguments have to join, which has `dims` dimensions."""
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got shape {tuple(t.shape)}")
    if not t.is_cuda or t.dtype is not dtype:
        _refuse(t, name, dtype, t.shape, 0)
    return t.get_device()


def _dense(shape):
    """Strides of a dense tensor of one to four dimensions."""
    if len(shape) == 3:
        return shape[1] * shape[2], shape[2], 1
    if len(shape) == 2:
        return shape[1], 1
    if len(shape) == 1:
        return (1,)
    return shape[1] * shape[2] * shape[3], shape[2] * shape[3], shape[3], 1


def _empty(shape, dtype, index, stream):
    """Uninitialised tensor for a kernel on `stream` (None: the current stream): taken from that
    stream's memory, and not given back while the current stream may still read it."""
    if stream is not None:
        device = torch.device("cuda", index)
        cur = torch.cuda.current_stream(device)
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(int(stream), device) if int(stream) else torch.cuda.default_stream(device)
        if stream.cuda_stream != cur.cuda_stream:
            with torch.cuda.stream(stream):
                t = torch.empty(shape, dtype=dtype, device=device)
            t.record_stream(cur)
            return t
    return torch.empty_strided(shape, _dense(shape), dtype=dtype, device=index)


def _call(name, index, stream, *args):
    """Run a library call with CUDA device `index` current, on `stream` or that device's current stream."""
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(index)
    elif isinstance(stream, torch.cuda.Stream):
        stream = stream.cuda_stream
    else:
        stream = int(stream)
    fn = getattr(_lib.load(), name)
    if torch.cuda.current_device() == index:
        code = fn(*args, stream)
    else:
        with torch.cuda.device(index):
            code = fn(*args, stream)
    if code:
        check(name, code)


def _pool(desc, pool, index):
    """Address of a quantized pool, which must hold every page of desc."""
    if not (isinstance(pool, _Tensor) and pool.dtype is _U8 and pool.get_device() == index and pool.is_contiguous()):
        _refuse(pool, "pool", _U8, getattr(pool, "shape", ()), index)
    if pool.numel() < desc.num_pages * _lib.load().mla_qcache_page_bytes(ctypes.byref(desc)):
        raise ValueError("pool is smaller than desc.num_pages pages")
    return pool.data_ptr()


def _table(block_table, B, index):
    """(address, row length) of a block table of B requests."""
    if isinstance(block_table, _Tensor):
        shape = block_table.shape
        if len(shape) == 2 and shape[0] == B:
            return _arg(block_table, "block_table", _I32, shape, index), shape[1]
        raise ValueError(f"block_table must have shape ({B}, max_pages), got {tuple(shape)}")
    raise TypeError("block_table must be a torch.Tensor")


def _rows(t, name, shape, index):
    """(address, row stride) of a bf16 tensor [B, n, ...] whose B * n rows are evenly spaced."""
    if not isinstance(t, _Tensor) or t.dtype is not _BF16 or t.shape != shape or t.get_device() != index:
        _refuse(t, name, _BF16, shape, index)
    B, n = shape[0], shape[1]
    stride = t.stride()
    if t.numel() and (stride[-1] != 1 or (B > 1 and n > 1 and stride[0] != n * stride[1])):
        raise ValueError(f"{name} must have unit stride in its last dimension and evenly spaced rows")
    return t.data_ptr(), (stride[1] if n > 1 else stride[0] if B > 1 else 0)


def _out_rows(t, name, rows, width, index):
    """(address, row stride) of a bf16 output [rows, width] with unit stride in a row."""
    if not isinstance(t, _Tensor) or t.dtype is not _BF16 or t.shape != (rows, width) \
            or t.get_device() != index:
        _refuse(t, name, _BF16, (rows, width), index)
    stride = t.stride()
    if stride[1] != 1 or (rows > 1 and stride[0] < width):
        raise ValueError(f"{name} must have unit stride in a row and rows that do not overlap")
    return t.data_ptr(), stride[0] if rows > 1 else width


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
    dev = _device_index(kv, "kv", _BF16, 3)
    B, n = kv.shape[0], kv.shape[1]
    pkv, kv_stride = _rows(kv, "kv", (B, n, D_C + D_R), dev)
    H, pq, q_token, q_head, pqo = 0, None, 0, 0, None
    if q is not None:
        if not isinstance(q, _Tensor) or q.dim() != 4:
            raise ValueError("q must be a tensor [B, n, H, 64]")
        H = q.shape[2]
        pq, q_token = _rows(q, "q", (B, n, H, D_R), dev)
        q_head = q.stride(2) if H > 1 else 0
        if q_out is None:
            q_out = _empty((B, n, H, D_R), _BF16, dev, stream)
        pqo = _arg(q_out, "q_out", _BF16, (B, n, H, D_R), dev)
        if H == 0:
            pq = pqo = None
    elif q_out is not None:
        raise ValueError("q_out needs q")
    if not isinstance(cos_sin, _Tensor) or cos_sin.dim() != 2:
        raise ValueError(f"cos_sin must be a tensor [positions, {D_R}]")
    positions_held = cos_sin.shape[0]
    _call("mla_qcache_append_norm_rope", dev, stream, ctypes.byref(desc), _pool(desc, pool, dev),
          *_table(block_table, B, dev), _arg(seq_lens_before, "seq_lens_before", _I32, (B,), dev),
          _opt(new_lens, "new_lens", _I32, (B,), dev), pkv, kv_stride,
          _opt(norm_weight, "norm_weight", _BF16, (D_C,), dev), float(eps), pq, q_token, q_head, H, pqo,
          _arg(cos_sin, "cos_sin", _F32, (positions_held, D_R), dev), positions_held,
          _opt(positions, "positions", _I32, (B, n), dev), pairs,
          _opt(rows_out, "rows_out", _BF16, (B, n, D_C + D_R), dev), B, n)
    return q_out


def mla_qcache_read(desc, pool, block_table, start, cu_rows, max_rows, out_c=None, out_kr=None, stream=None) -> None:
    """Read dequantized rows back: tokens start[b] + i (start None: 0) of request b into row
    cu_rows[b] + i of out_c [rows, 512] and out_kr [rows, 64] (bf16; either may be None, and both may
    be column ranges of one buffer). max_rows bounds the rows of one request."""
    out = out_c if out_c is not None else out_kr
    if not isinstance(out, _Tensor) or out.dim() != 2:
        raise ValueError("out_c or out_kr must be given, as tensors [rows, width]")
    dev = _device_index(cu_rows, "cu_rows", _I32, 1)
    B = cu_rows.shape[0] - 1
    if B < 0:
        raise ValueError("cu_rows must have one entry more than there are requests")
    rows = out.shape[0]
    pc, sc = (None, 0) if out_c is None else _out_rows(out_c, "out_c", rows, D_C, dev)
    pr, sr = (None, 0) if out_kr is None else _out_rows(out_kr, "out_kr", rows, D_R, dev)
    _call("mla_qcache_read", dev, stream, ctypes.byref(desc), _pool(desc, pool, dev), *_table(block_table, B, dev),
          _opt(start, "start", _I32, (B,), dev), _arg(cu_rows, "cu_rows", _I32, (B + 1,), dev),
          int(max_rows), rows, pc, sc, pr, sr, B)


def mla_page_digest(desc, pool, block_table, seq_lens_before, n_new, digests, *, new_lens=None, stream=None) -> None:
    """Mean keys of the pages that appending new_lens[b] (None: n_new) tokens completed, into the
    pages' rows of digests [num_pages, 576] (bf16). Call it after the append."""
    dev = _device_index(seq_lens_before, "seq_lens_before", _I32, 1)
    B = seq_lens_before.shape[0]
    _call("mla_page_digest", dev, stream, ctypes.byref(desc), _pool(desc, pool, dev), *_table(block_table, B, dev),
          _arg(seq_lens_before, "seq_lens_before", _I32, (B,), dev),
          _opt(new_lens, "new_lens", _I32, (B,), dev), int(n_new),
          _arg(digests, "digests", _BF16, (desc.num_pages, D_C + D_R), dev), B)


def new_digests(desc: mla_qcache_desc, device="cuda") -> torch.Tensor:
    """Zeroed bf16 digests [num_pages, 576] of a pool's pages."""
    return torch.zeros((desc.num_pages, D_C + D_R), dtype=_BF16, device=device)


def _page_count(max_seq_len) -> int:
    return max(0, -(-max_seq_len // PAGE))


def _queries(q_c, q_r):
    """(B, s_q, H, device index, addresses of q_c and q_r)."""
    dev = _device_index(q_c, "q_c", _BF16, 4)
    B, s_q, H = q_c.shape[:3]
    return B, s_q, H, dev, _arg(q_c, "q_c", _BF16, (B, s_q, H, D_C), dev), \
        _arg(q_r, "q_r", _BF16, (B, s_q, H, D_R), dev)


def mla_page_scores(block_table, seq_lens, max_seq_len, digests, q_c, q_r, scale, *, out=None, stream=None):
    """Expected attention mass of every candidate page, fp32 [B, s_q, ceil(max_seq_len / 64)] (-inf
    for pages that are no candidates). See include/mla_qcache.h."""
    B, s_q, H, dev, pc, pr = _queries(q_c, q_r)
    max_seq_len = int(max_seq_len)
    pages = digests.shape[0] if isinstance(digests, _Tensor) and digests.dim() == 2 else 0
    pd = _arg(digests, "digests", _BF16, (pages, D_C + D_R), dev)
    shape = (B, s_q, _page_count(max_seq_len))
    if out is None:
        out = _empty(shape, _F32, dev, stream)
    _call("mla_page_scores", dev, stream, pd, pages, *_table(block_table, B, dev),
          _arg(seq_lens, "seq_lens", _I32, (B,), dev), max_seq_len, pc, pr, B, s_q, H, float(scale),
          _arg(out, "out", _F32, shape, dev))
    return out


def mla_select_pages(block_table, seq_lens, max_seq_len, scores, k_pages, *, n_sink=1, n_recent=1, s_q=None,
                     sel_table=None, sel_pages=None, sel_lens=None, stream=None):
    """Pages each query attends: (sel_table [B, s_q, k_pages] pages of the pool, sel_pages their
    indexes in the request, sel_lens [B, s_q] keys), int32, -1 behind the last page. scores
    [B, s_q, ceil(max_seq_len / 64)] may be None when k_pages covers every page (then s_q is needed).
    sel_table and sel_lens, flattened to B * s_q requests, are what mla_qdecode takes."""
    if scores is None:
        if s_q is None:
            raise ValueError("s_q is needed without scores")
    elif not isinstance(scores, _Tensor) or scores.dim() != 3:
        raise ValueError("scores must be a tensor [B, s_q, pages]")
    else:
        s_q = scores.shape[1]
    dev = _device_index(seq_lens, "seq_lens", _I32, 1)
    B, max_seq_len, k_pages = seq_lens.shape[0], int(max_seq_len), int(k_pages)
    if k_pages < 1 or s_q < 1:
        raise MlaError("mla_select_pages", _lib.MLA_ERR_INVALID_ARG)
    shape = (B, s_q, k_pages)
    if sel_table is None:
        sel_table = _empty(shape, _I32, dev, stream)
    if sel_pages is None:
        sel_pages = _empty(shape, _I32, dev, stream)
    if sel_lens is None:
        sel_lens = _empty((B, s_q), _I32, dev, stream)
    _call("mla_select_pages", dev, stream, *_table(block_table, B, dev),
          _arg(seq_lens, "seq_lens", _I32, (B,), dev), max_seq_len,
          _opt(scores, "scores", _F32, (B, s_q, _page_count(max_seq_len)), dev), B, s_q, k_pages, int(n_sink), int(n_recent),
          _arg(sel_table, "sel_table", _I32, shape, dev), _arg(sel_pages, "sel_pages", _I32, shape, dev),
          _arg(sel_lens, "sel_lens", _I32, (B, s_q), dev))
    return sel_table, sel_pages, sel_lens


def mla_qdecode_sparse_workspace_bytes(B, s_q, H, max_seq_len, k_pages, num_splits=0) -> int:
    return _lib.load().mla_qdecode_sparse_workspace_bytes(B, s_q, H, int(max_seq_len), int(k_pages), int(num_splits))


def mla_qdecode_sparse(desc, pool, block_table, seq_lens, max_seq_len, digests, q_c, q_r, scale, k_pages, *, n_sink=1,
                       n_recent=1, out=None, out_dtype=torch.bfloat16, lse=None, num_splits=0, workspace=None, flags=0,
                       stream=None):
    """One decode step over the pages that the digests' scores select (scores, selection, decode).
    digests may be None when k_pages covers every page. Returns (out, lse). See include/mla_qcache.h."""
    B, s_q, H, dev, pc, pr = _queries(q_c, q_r)
    max_seq_len, k_pages = int(max_seq_len), int(k_pages)
    if out is None:
        out = _empty((B, s_q, H, D_C), out_dtype, dev, stream)
    f32 = out.dtype is _F32
    if not f32 and out.dtype is not _BF16:
        raise TypeError("out must be bfloat16 or float32")
    if workspace is None:
        with torch.cuda.device(dev):  # the split plan is the device's
            need = mla_qdecode_sparse_workspace_bytes(B, s_q, H, max_seq_len, k_pages, num_splits)
        workspace = _empty((max(need, 1),), _U8, dev, stream)
    nw = workspace.numel()
    _call("mla_qdecode_sparse", dev, stream, ctypes.byref(desc), _pool(desc, pool, dev), *_table(block_table, B, dev),
          _arg(seq_lens, "seq_lens", _I32, (B,), dev), max_seq_len,
          _opt(digests, "digests", _BF16, (desc.num_pages, D_C + D_R), dev), pc, pr, B, s_q, H, float(scale),
          k_pages, int(n_sink), int(n_recent), int(num_splits), _arg(workspace, "workspace", _U8, (nw,), dev), nw,
          _arg(out, "out", out.dtype, (B, s_q, H, D_C), dev), f32, _opt(lse, "lse", _F32, (B, s_q, H), dev),
          int(flags))
    return out, lse


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
