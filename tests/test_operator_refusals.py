"""Argument errors of the operators around the cache; nothing here reaches a device.

Every refused call returns before a launch (fake device addresses are never
dereferenced), and the binding refuses before it calls the library.
"""
import ctypes

import pytest
import torch

from bit_mla_kv_qdecode_b200 import _lib, api
from bit_mla_kv_qdecode_b200 import build as _build

INV, UNS, CAP, WS = (_lib.MLA_ERR_INVALID_ARG, _lib.MLA_ERR_UNSUPPORTED, _lib.MLA_ERR_CAPACITY, _lib.MLA_ERR_WORKSPACE)
A = 0x7000000  # a 256-byte aligned address that nothing reads
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return _lib.load()


def _desc(**kw):
    return ctypes.byref(_lib.make_desc(**{"num_pages": 10, **kw}))


def _caller(lib, name, defaults):
    def call(**kw):
        unknown = set(kw) - set(defaults)
        assert not unknown, unknown
        return getattr(lib, name)(*{**defaults, **kw}.values())
    return call


NORM_ROPE = dict(desc=_desc(), pool=A, table=A, max_pages=4, before=A, new_lens=None, kv=A, kv_stride=576, weight=A,
                 eps=1e-6, q=A, q_token=1024, q_head=64, H=16, q_out=A, cos_sin=A, max_positions=100, positions=None,
                 pairs=0, rows=None, B=2, n=3, stream=None)


@pytest.mark.parametrize("bad,code", [
    (dict(desc=None), INV), (dict(desc=_desc(bits_c=3)), UNS), (dict(pool=None), INV), (dict(pool=A + 16), INV),
    (dict(table=None), INV), (dict(max_pages=0), INV), (dict(before=None), INV), (dict(kv=None), INV), (dict(kv=A + 8), INV),
    (dict(kv_stride=572), INV), (dict(kv_stride=-576), INV), (dict(weight=A + 2), INV), (dict(eps=0.0), INV),
    (dict(eps=-1e-6), INV), (dict(eps=NAN), INV), (dict(eps=INF), INV), (dict(q=None), INV), (dict(q_out=None), INV),
    (dict(H=0), INV), (dict(q=None, q_out=None), INV), (dict(q=A + 4), INV), (dict(q_token=4), INV), (dict(q_head=-64), INV),
    (dict(H=-1), INV), (dict(q_out=A + 8), INV), (dict(cos_sin=None), INV), (dict(cos_sin=A + 4), INV),
    (dict(max_positions=-1), INV), (dict(pairs=2), INV), (dict(pairs=-1), INV), (dict(rows=A + 8), INV), (dict(B=-1), INV),
    (dict(n=-1), INV), (dict(B=1 << 20, n=1 << 10), UNS), (dict(H=1 << 17), UNS), (dict(B=1 << 14, n=1 << 12, H=4096), UNS)])
def test_norm_rope(lib, bad, code):
    assert _caller(lib, "mla_qcache_append_norm_rope", NORM_ROPE)(**bad) == code


READ = dict(desc=_desc(), pool=A, table=A, max_pages=4, start=A, cu=A, max_rows=100, total=200, c=A, c_stride=512, kr=A,
            kr_stride=64, B=2, stream=None)


@pytest.mark.parametrize("bad,code", [
    (dict(desc=None), INV), (dict(desc=_desc(group_c=16)), UNS), (dict(pool=None), INV), (dict(pool=A + 128), INV),
    (dict(table=None), INV), (dict(cu=None), INV), (dict(max_pages=0), INV), (dict(c=None, kr=None), INV), (dict(c=A + 2), INV),
    (dict(kr=A + 2), INV), (dict(c_stride=511), INV), (dict(c_stride=516), INV), (dict(c_stride=-512), INV),
    (dict(kr_stride=56), INV), (dict(kr_stride=68), INV), (dict(max_rows=-1), INV), (dict(total=-1), INV), (dict(B=-1), INV),
    (dict(B=65536), UNS)])
def test_read(lib, bad, code):
    assert _caller(lib, "mla_qcache_read", READ)(**bad) == code


DIGEST = dict(desc=_desc(), pool=A, table=A, max_pages=4, before=A, new_lens=None, n=3, digests=A, B=2, stream=None)


@pytest.mark.parametrize("bad,code", [
    (dict(desc=None), INV), (dict(desc=_desc(bits_r=8)), UNS), (dict(pool=None), INV), (dict(pool=A + 16), INV),
    (dict(table=None), INV), (dict(max_pages=0), INV), (dict(before=None), INV), (dict(digests=None), INV),
    (dict(digests=A + 8), INV), (dict(n=-1), INV), (dict(B=-1), INV), (dict(B=65536), UNS)])
def test_digest(lib, bad, code):
    assert _caller(lib, "mla_page_digest", DIGEST)(**bad) == code


SCORES = dict(digests=A, num_pages=10, table=A, max_pages=4, lens=A, max_len=256, q_c=A, q_r=A, B=2, s_q=1, H=16, scale=0.1,
              out=A, stream=None)


@pytest.mark.parametrize("bad,code", [
    (dict(digests=None), INV), (dict(digests=A + 8), INV), (dict(num_pages=-1), INV), (dict(table=None), INV),
    (dict(max_pages=0), INV), (dict(lens=None), INV), (dict(max_len=-1), INV), (dict(max_len=257), CAP), (dict(q_c=None), INV),
    (dict(q_c=A + 2), INV), (dict(q_r=None), INV), (dict(q_r=A + 2), INV), (dict(B=-1), INV), (dict(s_q=0), INV), (dict(H=0), INV),
    (dict(H=129), UNS), (dict(B=65536), UNS), (dict(B=40000, s_q=2), UNS), (dict(scale=NAN), INV), (dict(scale=INF), INV),
    (dict(out=None), INV), (dict(out=A + 2), INV)])
def test_scores(lib, bad, code):
    assert _caller(lib, "mla_page_scores", SCORES)(**bad) == code


SELECT = dict(table=A, max_pages=4, lens=A, max_len=256, scores=A, B=2, s_q=1, k=3, n_sink=1, n_recent=1, sel_table=A,
              sel_pages=None, sel_lens=A, stream=None)


@pytest.mark.parametrize("bad,code", [
    (dict(table=None), INV), (dict(max_pages=0), INV), (dict(lens=None), INV), (dict(max_len=-1), INV), (dict(max_len=257), CAP),
    (dict(scores=None), INV), (dict(scores=A + 2), INV), (dict(B=-1), INV), (dict(s_q=0), INV), (dict(k=0), INV),
    (dict(k=(1 << 20) + 1), INV), (dict(n_sink=-1), INV), (dict(n_recent=0), INV), (dict(n_sink=2, n_recent=2), INV),
    (dict(n_sink=2 ** 31 - 1), INV), (dict(sel_table=None), INV), (dict(sel_table=A + 1), INV), (dict(sel_pages=A + 2), INV),
    (dict(sel_lens=None), INV), (dict(B=65536), UNS), (dict(B=30000, s_q=3), UNS)])
def test_select(lib, bad, code):
    assert _caller(lib, "mla_select_pages", SELECT)(**bad) == code


SPARSE = dict(desc=_desc(), pool=A, table=A, max_pages=4, lens=A, max_len=256, digests=A, q_c=A, q_r=A, B=2, s_q=1, H=16,
              scale=0.1, k=3, n_sink=1, n_recent=1, splits=0, ws=A, ws_bytes=1 << 24, out=A, out_dtype=0, lse=None, flags=0, stream=None)


@pytest.mark.parametrize("bad,code", [
    (dict(desc=None), INV), (dict(desc=_desc(bits_c=8)), UNS), (dict(pool=None), INV), (dict(pool=A + 16), INV),
    (dict(table=None), INV), (dict(max_pages=0), INV), (dict(lens=None), INV), (dict(max_len=-1), INV), (dict(max_len=257), CAP),
    (dict(digests=None), INV), (dict(digests=A + 4), INV), (dict(q_c=None), INV), (dict(q_c=A + 8), INV), (dict(q_r=None), INV),
    (dict(B=-1), INV), (dict(s_q=0), INV), (dict(H=0), INV), (dict(H=129), UNS), (dict(B=65536), UNS), (dict(scale=NAN), INV),
    (dict(k=0), INV), (dict(n_sink=3), INV), (dict(n_recent=0), INV), (dict(splits=-1), INV), (dict(ws=None), WS), (dict(ws=A + 16), WS),
    (dict(ws_bytes=100), WS), (dict(out=None), INV), (dict(out=A + 8), INV), (dict(out_dtype=2), INV), (dict(lse=A + 2), INV),
    (dict(flags=8), INV), (dict(flags=_lib.MLA_DECODE_TEST_STALL), INV)])
def test_sparse(lib, bad, code):
    assert _caller(lib, "mla_qdecode_sparse", SPARSE)(**bad) == code


def test_empty_batches_need_nothing(lib):
    none = dict(pool=None, table=None)
    assert _caller(lib, "mla_qcache_append_norm_rope", NORM_ROPE)(B=0, kv=None, before=None, cos_sin=None, **none) == 0
    assert _caller(lib, "mla_qcache_append_norm_rope", NORM_ROPE)(n=0, kv=None, before=None, cos_sin=None, **none) == 0
    assert _caller(lib, "mla_qcache_read", READ)(B=0, cu=None, c=None, kr=None, **none) == 0
    assert _caller(lib, "mla_qcache_read", READ)(max_rows=0, **none) == 0
    assert _caller(lib, "mla_page_digest", DIGEST)(B=0, before=None, digests=None, **none) == 0
    assert _caller(lib, "mla_page_digest", DIGEST)(n=0, **none) == 0
    assert _caller(lib, "mla_page_scores", SCORES)(B=0, table=None, lens=None, out=None) == 0
    assert _caller(lib, "mla_page_scores", SCORES)(max_len=0, table=None, lens=None, out=None) == 0
    assert _caller(lib, "mla_select_pages", SELECT)(B=0, table=None, lens=None, sel_table=None) == 0
    assert _caller(lib, "mla_qdecode_sparse", SPARSE)(B=0, lens=None, out=None, ws=None, **none) == 0


def test_sparse_workspace(lib):
    ws = lib.mla_qdecode_sparse_workspace_bytes
    for bad in ((0, 1, 16, 100, 4, 0), (2, 0, 16, 100, 4, 0), (2, 1, 0, 100, 4, 0), (2, 1, 16, -1, 4, 0), (2, 1, 16, 100, 0, 0),
                (40000, 2, 16, 100, 4, 0), (1, 1, (1 << 20) + 1, 100, 4, 0), (2, 1, 16, 100, 4, -1),
                (2, 1, 16, 100, (1 << 20) + 1, 0)):
        assert ws(*bad) == 0, bad
    # scores of 128 pages a query, 6 of them selected, and the scratch of 6 requests of 384 keys
    B, s_q, H, T, k = 2, 3, 128, 8192, 6
    up = lambda n: (n + 255) // 256 * 256  # noqa: E731
    for n in (1, 2, 3):
        inner = lib.mla_decode_workspace_bytes(B * s_q, 1, H, 64 * k, n)
        assert ws(B, s_q, H, T, k, n) == up(6 * 128 * 4) + up(6 * k * 4) + up(6 * 4) + inner
        # every page selected: no scores
        assert ws(B, s_q, H, 300, k, n) == up(6 * k * 4) + up(6 * 4) + lib.mla_decode_workspace_bytes(6, 1, H, 300, n)
    # up to 16 rows the choice is mla_qdecode's; else its own: many short selections are not split, few are
    assert ws(B, 1, 16, T, k, 0) == up(2 * 128 * 4) + up(2 * k * 4) + up(2 * 4) + lib.mla_decode_workspace_bytes(2, 1, 16, 64 * k, 0)
    assert ws(128, 2, 128, 32768, 32, 0) == ws(128, 2, 128, 32768, 32, 1)
    assert ws(4, 1, 128, 131072, 64, 0) == ws(4, 1, 128, 131072, 64, 16)
    # a selection of more than 8,192 keys is split whatever is asked for
    assert ws(64, 1, 128, 65536, 200, 1) == ws(64, 1, 128, 65536, 200, 2)


def test_sparse_workspace_is_no_wider_than_the_pages(lib):
    """k_pages above the page count is the way to attend everything; its rows cost no more than the pages."""
    ws = lib.mla_qdecode_sparse_workspace_bytes
    for T in (0, 1, 64, 300, 8192):
        pages = max(1, -(-T // 64))
        for k in (pages, pages + 1, 1 << 20):
            assert ws(256, 1, 128, T, k, 1) == ws(256, 1, 128, T, pages, 1), (T, k)
    assert ws(256, 1, 128, 64, 1 << 20, 1) == 2 * 1024  # a page and a length a query


def test_binding_refuses_host_tensors_types_and_shapes():
    desc = api.make_desc(4, 64, 4, 64, num_pages=2)
    pool = torch.zeros((2, 20736), dtype=torch.uint8)
    table, ints = torch.zeros((1, 2), dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    kv = torch.zeros((1, 1, 576), dtype=torch.bfloat16)
    cs = torch.zeros((4, 64))
    q_c, q_r = torch.zeros((1, 1, 2, 512), dtype=torch.bfloat16), torch.zeros((1, 1, 2, 64), dtype=torch.bfloat16)
    dig = torch.zeros((2, 576), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        api.mla_qcache_append_norm_rope(desc, pool, table, ints, kv, None, 1e-6, cs)
    with pytest.raises(TypeError):
        api.mla_qcache_append_norm_rope(desc, pool, table, ints, kv.float(), None, 1e-6, cs)
    with pytest.raises(ValueError, match="convention"):
        api.mla_qcache_append_norm_rope(desc, pool, table, ints, kv, None, 1e-6, cs, convention="pairs")
    with pytest.raises(ValueError, match="kv"):
        api.mla_qcache_append_norm_rope(desc, pool, table, ints, kv[0], None, 1e-6, cs)
    with pytest.raises(ValueError, match="out_c or out_kr"):
        api.mla_qcache_read(desc, pool, table, None, torch.zeros(2, dtype=torch.int32), 4)
    with pytest.raises(ValueError, match="CUDA"):
        api.mla_qcache_read(desc, pool, table, None, torch.zeros(2, dtype=torch.int32), 4,
                            torch.zeros((4, 512), dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="CUDA"):
        api.mla_page_digest(desc, pool, table, ints, 1, dig)
    with pytest.raises(ValueError, match="CUDA"):
        api.mla_page_scores(table, ints, 100, dig, q_c, q_r, 1.0)
    with pytest.raises(ValueError, match="s_q"):
        api.mla_select_pages(table, ints, 100, None, 2)
    with pytest.raises(ValueError, match="scores"):
        api.mla_select_pages(table, ints, 100, torch.zeros((1, 2)), 1)
    with pytest.raises(ValueError, match="CUDA"):
        api.mla_qdecode_sparse(desc, pool, table, ints, 100, dig, q_c, q_r, 1.0, 2)


def test_binding_refuses_wrong_kinds_of_arguments():
    desc = api.make_desc(4, 64, 4, 64, num_pages=2)
    table, ints = torch.zeros((1, 2), dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    dig = torch.zeros((2, 576), dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        api.mla_page_digest(None, dig, table, ints, 1, dig)        # no description
    with pytest.raises(TypeError):
        api.mla_page_digest(desc, "pool", table, ints, 1, dig)     # no tensor
    with pytest.raises(TypeError):
        api.mla_page_digest(desc, dig, table, ints, 1.5, dig)      # no whole number
    with pytest.raises(TypeError):
        api.mla_page_digest(desc, dig, table, ints.long(), 1, dig)
    with pytest.raises(TypeError):
        api.mla_qdecode_sparse(desc, dig, table, ints, 100, dig, dig, dig, 1.0, 2, out_dtype=torch.float16)
    with pytest.raises(ValueError, match="dimensions"):
        api.mla_page_scores(table, ints, 100, dig, dig, dig, 1.0)
