"""GPU tests of the launch sizes under loose host bounds: max_rows and n_new may be any int, the work
launched for them is what the outputs and the block table allow.

The calls are captured into a graph and their grids read from its nodes, before anything runs. The scores'
grids show which cluster sizes their tests reach.
"""
import ctypes

import numpy as np
import pytest
import torch

from bit_mla_kv_qdecode_b200 import api
from tests import operator_refs as ref

pytestmark = pytest.mark.gpu
ANY = 2 ** 31 - 1


class _KernelNode(ctypes.Structure):  # CUDA_KERNEL_NODE_PARAMS of the driver's interface
    _fields_ = [("func", ctypes.c_void_p), ("grid", ctypes.c_uint * 3), ("block", ctypes.c_uint * 3), ("smem", ctypes.c_uint),
                ("params", ctypes.c_void_p), ("extra", ctypes.c_void_p), ("kern", ctypes.c_void_p), ("ctx", ctypes.c_void_p)]


def _grids(call):
    """CTAs of each kernel that `call` launches; nothing runs."""
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        call()
    cu, g, n = ctypes.CDLL("libcuda.so.1"), ctypes.c_void_p(graph.raw_cuda_graph()), ctypes.c_size_t(0)
    assert cu.cuGraphGetNodes(g, None, ctypes.byref(n)) == 0
    nodes = (ctypes.c_void_p * n.value)()
    assert cu.cuGraphGetNodes(g, nodes, ctypes.byref(n)) == 0
    out = []
    for node in nodes:
        kind, p = ctypes.c_int(-1), _KernelNode()
        assert cu.cuGraphNodeGetType(ctypes.c_void_p(node), ctypes.byref(kind)) == 0
        if kind.value == 0:  # a kernel
            assert cu.cuGraphKernelNodeGetParams_v2(ctypes.c_void_p(node), ctypes.byref(p)) == 0
            out.append(p.grid[0] * p.grid[1] * p.grid[2])
    return out


def _i32(a):
    return torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()


@pytest.mark.parametrize("B,max_pages", [(1, 2), (3, 40), (700, 2)])
def test_read_launches_no_more_than_rows_and_pages_allow(B, max_pages):
    rng = np.random.default_rng(B)
    fmt = (4, 64, 4, 64)
    desc = api.make_desc(*fmt, num_pages=4)
    pool = torch.from_numpy(ref.random_pool(rng, fmt, 4)).cuda()
    table = _i32(rng.integers(0, 4, (B, max_pages)))
    start = _i32(rng.integers(0, 60, B))
    cu = _i32(5 * np.arange(B + 1))
    tight, loose = (torch.full((5 * B + 3, 512), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    read = lambda bound, out: api.mla_qcache_read(desc, pool, table, start, cu, bound, out)  # noqa: E731
    # a page more than the rows fill, and at most four CTAs a page
    most = 4 * B * (min(5 * B + 3, 64 * max_pages + 1) // 64 + 2)
    (ctas,) = _grids(lambda: read(ANY, loose))
    assert ctas <= most, (ctas, most)
    read(5, tight)
    read(ANY, loose)
    assert api.mla_get_device_status() == 0 and torch.equal(tight, loose)


def test_read_of_many_rows_flags_the_position_behind_the_table():
    fmt = (4, 64, 4, 64)
    desc = api.make_desc(*fmt, num_pages=3)
    pool = torch.from_numpy(ref.random_pool(np.random.default_rng(1), fmt, 3)).cuda()
    table = _i32([[2, 0]])
    good, out = (torch.full((1000, 512), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    api.mla_qcache_read(desc, pool, table, _i32([5]), _i32([0, 123]), 123, good)
    assert api.mla_get_device_status() == 0
    for count in (124, 1000):  # one position too many, and many
        out.fill_(7.0)
        api.mla_qcache_read(desc, pool, table, _i32([5]), _i32([0, count]), ANY, out)
        assert api.mla_get_device_status() == api._lib.MLA_ERR_INVALID_ARG
        assert torch.equal(out, good)


@pytest.mark.parametrize("B,max_pages", [(1, 2), (3, 40), (700, 3)])
def test_digest_launches_no_more_than_pages_allow(B, max_pages):
    rng = np.random.default_rng(B)
    fmt, pages = (2, 32, 4, 64), 8
    desc = api.make_desc(*fmt, num_pages=pages)
    pool = torch.from_numpy(ref.random_pool(rng, fmt, pages)).cuda()
    table = _i32(rng.integers(0, pages, (B, max_pages)))
    before, given = _i32(rng.integers(0, 64, B)), _i32(np.full(B, 64))
    tight, loose = (torch.full((pages, 576), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    digest = lambda bound, out: api.mla_page_digest(desc, pool, table, before, bound, out, new_lens=given)  # noqa: E731
    (ctas,) = _grids(lambda: digest(ANY, loose))
    assert ctas <= max(B * (max_pages + 1), 2 * torch.cuda.get_device_properties(0).multi_processor_count), ctas
    digest(64, tight)
    digest(ANY, loose)
    assert api.mla_get_device_status() == 0 and torch.equal(tight, loose)


def test_digest_flags_the_page_behind_the_table():
    fmt = (4, 64, 4, 64)
    desc = api.make_desc(*fmt, num_pages=3)
    pool = torch.from_numpy(ref.random_pool(np.random.default_rng(1), fmt, 3)).cuda()
    table = _i32([[2, 0]])
    good, out = api.new_digests(desc), api.new_digests(desc)
    api.mla_page_digest(desc, pool, table, _i32([0]), 128, good)
    assert api.mla_get_device_status() == 0
    for new in (192, ANY):
        out.zero_()
        api.mla_page_digest(desc, pool, table, _i32([0]), ANY, out, new_lens=_i32([new]))
        assert api.mla_get_device_status() == api._lib.MLA_ERR_INVALID_ARG
        assert torch.equal(out, good)


def test_scores_reach_every_cluster_size():
    """The shapes of the scores' cluster-size test take one CTA a query up to sixteen, a size each."""
    got = []
    for tokens, B in ((64 * 100, 150), (64 * 200, 60), (64 * 500, 30), (64 * 1000, 12), (64 * 2040 + 1, 3)):
        pages = -(-tokens // 64)
        table, lens = torch.zeros((B, pages), dtype=torch.int32, device="cuda"), _i32(np.full(B, tokens))
        dig = torch.zeros((1, 576), dtype=torch.bfloat16, device="cuda")
        q_c, q_r = (torch.zeros((B, 1, 8, d), dtype=torch.bfloat16, device="cuda") for d in (512, 64))
        (ctas,) = _grids(lambda: api.mla_page_scores(table, lens, tokens, dig, q_c, q_r, 0.1))
        got.append(ctas / B)
    assert got == [1, 2, 4, 8, 16]
