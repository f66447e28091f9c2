"""GPU tests of mla_qcache_read and mla_page_digest against float64."""
import numpy as np
import pytest
import torch

from bit_mla_kv_qdecode_b200 import api
from oracle import layout
from tests import operator_refs as ref

pytestmark = pytest.mark.gpu


def _i32(a):
    return torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()


def _read_case(fmt, start, count, seed=0, gaps=(), one_buffer=True):
    """Read ranges [start, start + count) into consecutive rows, with unused rows in front and behind."""
    rng = np.random.default_rng(seed)
    start, count = np.asarray(start), np.asarray(count)
    table, pages = ref.random_table(rng, start + count)
    pool = ref.random_pool(rng, fmt, pages)
    lead = 3
    cu = lead + np.concatenate([[0], np.cumsum(count)])
    rows = int(cu[-1]) + 5
    desc = api.make_desc(*fmt, num_pages=pages)
    if one_buffer:
        buf = torch.full((rows, 584), 7.0, dtype=torch.bfloat16, device="cuda")
        out_c, out_kr = buf[:, :512], buf[:, 512:576]
    else:
        out_c = torch.full((rows, 512), 7.0, dtype=torch.bfloat16, device="cuda")
        out_kr = torch.full((rows, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    api.mla_qcache_read(desc, torch.from_numpy(pool).cuda(), _i32(table), _i32(start), _i32(cu), max(int(count.max()), 1),
                        out_c, out_kr)
    assert api.mla_get_device_status() == 0
    want = np.full((rows, 576), 7.0)
    for b in range(len(start)):
        C, R = layout.gather_tokens(ref.np_desc(fmt), pool, table[b], int(start[b] + count[b]))
        want[cu[b]:cu[b + 1]] = np.concatenate([C, R], 1)[start[b]:]
    got = np.concatenate([ref.f32(out_c), ref.f32(out_kr)], 1)
    # u*s + z rounded to fp32, then to bf16
    assert np.all(np.abs(got - want) <= np.abs(want) * (ref.BF16_HALF + 2 * ref.FP32_HALF))
    if one_buffer:
        assert bool((buf[:, 576:] == 7.0).all())


@pytest.mark.parametrize("fmt", ref.FORMATS)
def test_read_formats(fmt):
    _read_case(fmt, [0, 5, 70], [129, 1, 66])


@pytest.mark.parametrize("start,count", [([0], [1]), ([63], [1]), ([63, 64], [2, 64]), ([0, 0, 9], [0, 64, 0]),
                                         ([100, 0, 1, 2], [300, 65, 63, 0]), ([17] * 9, [200] * 9)])
def test_read_ranges(start, count):
    _read_case((2, 32, 4, 64), start, count, seed=len(start))
    _read_case((4, 64, 4, 64), start, count, seed=len(start), one_buffer=False)


def test_read_parts_and_defaults():
    rng = np.random.default_rng(4)
    fmt = (4, 64, 4, 64)
    pool = torch.from_numpy(ref.random_pool(rng, fmt, 3)).cuda()
    desc = api.make_desc(*fmt, num_pages=3)
    table, cu = _i32([[2, 0]]), _i32([0, 100])
    c, kr = torch.zeros((100, 512), dtype=torch.bfloat16).cuda(), torch.zeros((100, 64), dtype=torch.bfloat16).cuda()
    c2, kr2 = c.clone(), kr.clone()
    api.mla_qcache_read(desc, pool, table, None, cu, 100, c, kr)
    api.mla_qcache_read(desc, pool, table, _i32([0]), cu, 100, out_c=c2)
    api.mla_qcache_read(desc, pool, table, None, cu, 100, out_kr=kr2)
    assert torch.equal(c, c2) and torch.equal(kr, kr2) and bool((c != 0).any())
    api.mla_qcache_read(desc, pool, table[:0], None, cu[:1], 100, c, kr)  # no requests
    assert api.mla_get_device_status() == 0


def test_read_loose_bound_and_shared_pages():
    """The bound on a request's rows may be any int; requests may share pages."""
    rng = np.random.default_rng(5)
    fmt = (4, 32, 2, 64)
    pool = torch.from_numpy(ref.random_pool(rng, fmt, 3)).cuda()
    desc = api.make_desc(*fmt, num_pages=3)
    out = torch.full((260, 576), 7.0, dtype=torch.bfloat16).cuda()
    api.mla_qcache_read(desc, pool, _i32([[2, 0], [2, 1]]), _i32([0, 10]), _i32([0, 128, 246]), 2 ** 31 - 1, out[:, :512],
                        out[:, 512:])
    assert api.mla_get_device_status() == 0
    assert torch.equal(out[10:64], out[128:182]) and bool((out[246:] == 7.0).all())
    assert not bool((out[:246] == 7.0).all(1).any())


def test_read_bad_data_is_skipped():
    rng = np.random.default_rng(4)
    fmt = (2, 64, 2, 32)
    pool = torch.from_numpy(ref.random_pool(rng, fmt, 3)).cuda()
    desc = api.make_desc(*fmt, num_pages=3)
    good = torch.full((200, 512), 7.0, dtype=torch.bfloat16).cuda()
    api.mla_qcache_read(desc, pool, _i32([[2, 0]]), None, _i32([0, 128]), 128, good)
    assert api.mla_get_device_status() == 0
    for table, start, cu, most, same in (
            ([[2, 9]], [0], [0, 128], 128, range(0, 64)),          # a page past the pool
            ([[2, -1]], [0], [0, 128], 128, range(0, 64)),
            ([[2, 0]], [0], [0, 130], 130, range(0, 128)),         # past the table row
            ([[2, 0]], [0], [0, 128], 100, range(0, 100)),         # more rows than max_rows
            ([[2, 0]], [0], [0, 0x7fffffff], 128, range(0, 128)),  # more rows than the output has
            ([[2, 0]], [-3], [0, 3], 128, ()),                     # before the first token
            ([[2, 0]], [0x7fffffff], [0, 3], 128, ()),
            ([[2, 0]], [0], [-5, 0], 128, ()),                     # rows before the output
            ([[2, 0]], [0], [50, 10], 128, ())):                   # decreasing
        out = torch.full((200, 512), 7.0, dtype=torch.bfloat16).cuda()
        api.mla_qcache_read(desc, pool, _i32(table), _i32(start), _i32(cu), most, out)
        assert api.mla_get_device_status() == api._lib.MLA_ERR_INVALID_ARG, (table, start, cu, most)
        same = list(same)
        other = [r for r in range(200) if r not in set(same)]
        assert torch.equal(out[same], good[same]) and bool((out[other] == 7.0).all()), (table, start, cu, most)


@pytest.mark.parametrize("fmt", ref.FORMATS)
def test_digest_formats(fmt):
    _digest_case(fmt, [0, 63, 128], 130)


@pytest.mark.parametrize("before,n,new_lens", [([63], 1, None), ([62, 63, 64], 1, None), ([0, 127, 100], 2, None),
                                               ([10, 60, 0, 5], 200, [200, 4, 0, 59]), ([0] * 5, 64, None), ([1], 700, None)])
def test_digest_completed_pages(before, n, new_lens):
    _digest_case((4, 64, 4, 64), before, n, new_lens, seed=n)


def _digest_case(fmt, before, n, new_lens=None, seed=0):
    rng = np.random.default_rng(seed)
    before = np.asarray(before)
    count = np.full(len(before), n) if new_lens is None else np.asarray(new_lens)
    table, pages = ref.random_table(rng, before + n, spare=1)
    pool = ref.random_pool(rng, fmt, pages)
    desc = api.make_desc(*fmt, num_pages=pages)
    out = torch.full((pages, 576), 7.0, dtype=torch.bfloat16).cuda()
    api.mla_page_digest(desc, torch.from_numpy(pool).cuda(), _i32(table), _i32(before), n, out,
                        new_lens=None if new_lens is None else _i32(new_lens))
    assert api.mla_get_device_status() == 0
    got = ref.f32(out)
    done = [int(table[b, p]) for b in range(len(before)) for p in range(before[b] // 64, (before[b] + count[b]) // 64)]
    for p in range(pages):
        if p not in set(done):
            assert np.all(got[p] == 7.0)
            continue
        v = ref.page_values(fmt, pool, p)
        want = v.mean(0)
        # 64 fp32 terms of one rounding each, at most 64 roundings of partial sums below sum|v|, then bf16
        tol = np.abs(want) * ref.BF16_HALF + (1 + ref.BF16_HALF) * 66 * ref.FP32_HALF * np.abs(v).mean(0)
        assert np.all(np.abs(got[p] - want) <= tol)


@pytest.mark.parametrize("fmt", [(4, 64, 4, 64), (2, 32, 4, 64), (2, 64, 2, 32)])
def test_digest_many_pages(fmt):
    """More pages than one CTA each would do at once: ragged prompts, some of them empty."""
    rng = np.random.default_rng(6)
    n, B = 64 * 40, 24
    given = rng.integers(0, n + 1, B)
    given[:4] = n, 0, 63, 64
    _digest_case(fmt, rng.integers(0, 200, B), n, list(given), seed=3)


def test_digest_many_pages_with_bad_ones():
    rng = np.random.default_rng(7)
    fmt, B, n = (4, 64, 4, 64), 40, 64 * 20
    pages = 30
    pool = torch.from_numpy(ref.random_pool(rng, fmt, pages)).cuda()
    desc = api.make_desc(*fmt, num_pages=pages)
    table = np.full((B, 20), pages + 1)
    table[3, :20] = np.arange(20)
    table[7, 5] = 25
    before = np.zeros(B)
    before[9] = -1
    out = torch.full((pages, 576), 7.0, dtype=torch.bfloat16).cuda()
    api.mla_page_digest(desc, pool, _i32(table), _i32(before), n, out)
    assert api.mla_get_device_status() == api._lib.MLA_ERR_INVALID_ARG
    alone = torch.full_like(out, 7.0)
    api.mla_page_digest(desc, pool, _i32(np.arange(20)[None]), _i32([0]), n, alone)
    api.mla_page_digest(desc, pool, _i32([[25]]), _i32([0]), 64, alone)
    assert api.mla_get_device_status() == 0
    assert torch.equal(out, alone)


def test_digest_of_a_page_two_requests_share():
    rng = np.random.default_rng(5)
    fmt = (2, 32, 4, 64)
    pool = torch.from_numpy(ref.random_pool(rng, fmt, 3)).cuda()
    desc = api.make_desc(*fmt, num_pages=3)
    a, b = api.new_digests(desc), api.new_digests(desc)
    api.mla_page_digest(desc, pool, _i32([[2, 0], [2, 1]]), _i32([0, 0]), 128, a)
    api.mla_page_digest(desc, pool, _i32([[0, 1, 2]]), _i32([0]), 192, b)
    assert torch.equal(a, b) and api.mla_get_device_status() == 0


def test_digest_bad_data_is_skipped():
    rng = np.random.default_rng(4)
    fmt = (4, 64, 4, 64)
    pool = torch.from_numpy(ref.random_pool(rng, fmt, 2)).cuda()
    desc = api.make_desc(*fmt, num_pages=2)
    for table, before, new in (([[9]], [0], [64]), ([[0]], [-1], [64]), ([[0]], [64], [64]), ([[0]], [0], [65]),
                               ([[0]], [0], [-1]), ([[0]], [0x7fffffff], [64])):
        out = torch.full((2, 576), 7.0, dtype=torch.bfloat16).cuda()
        api.mla_page_digest(desc, pool, _i32(table), _i32(before), 64, out, new_lens=_i32(new))
        assert api.mla_get_device_status() == api._lib.MLA_ERR_INVALID_ARG, (table, before, new)
        assert bool((out == 7.0).all())
