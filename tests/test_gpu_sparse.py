"""GPU tests of the sparse decode: page scores, page selection, and the step, against float64."""
import math

import numpy as np
import pytest
import torch

from bit_mla_kv_qdecode_b200 import api
from oracle import attention, layout
from tests import mla_cases as mc
from tests import operator_refs as ref

pytestmark = pytest.mark.gpu
SCALE = 1.0 / math.sqrt(192.0)


def _i32(a):
    return torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()


def _score_tol(size, H, P):
    """Relative bound on a score. A logit is 576 exact products accumulated in fp32; the tensor
    cores may truncate rather than round, so each of the 576 additions is off by at most
    2^-23 of the products' absolute sum (`size`, scale included); scaling and 2^x add 4 more.
    A weight is a quotient of such exponentials, and a score a sum of H weights."""
    d = 580 * 2.0 ** -23 * size
    return math.expm1(2 * d) + (H + P + 8) * 2.0 ** -24


def _scores_case(lens, s_q, H, seed=0, scale=SCALE, gain=3.0, bad=()):
    rng = np.random.default_rng(seed)
    lens = np.asarray(lens)
    B = len(lens)
    table, pages = ref.random_table(rng, lens, spare=1)
    u = rng.standard_normal((B, 1, 1, 576))
    q = torch.from_numpy((u + 0.5 * rng.standard_normal((B, s_q, H, 576))).astype(np.float32)).bfloat16()
    dig = rng.standard_normal((pages, 576)) * 0.125
    for b in range(B):
        for p in table[b][table[b] >= 0]:
            if rng.random() < 0.2:
                dig[p] += u[b, 0, 0] / np.linalg.norm(u[b]) * rng.uniform(1, gain)
    dig = torch.from_numpy(dig.astype(np.float32)).bfloat16()
    for b, p in bad:
        table[b, p] = pages + 3
    W = -(-int(lens.max()) // 64)
    q_c, q_r = q[..., :512].contiguous().cuda(), q[..., 512:].contiguous().cuda()
    out = torch.full((B, s_q, W), 7.0, device="cuda")
    api.mla_page_scores(_i32(table), _i32(lens), int(lens.max()), dig.cuda(), q_c, q_r, scale, out=out)
    assert api.mla_get_device_status() == (api._lib.MLA_ERR_INVALID_ARG if bad else 0)
    got = out.cpu().numpy()
    dig, qf = ref.f32(dig), ref.f32(q)
    for b in range(B):
        for i in range(s_q):
            L = int(lens[b]) - s_q + 1 + i
            P = (L - 1) // 64 if L > 0 else 0
            row = table[b].copy()
            ok = [p for p in range(P) if 0 <= row[p] < pages]
            want = np.full(W, -np.inf)
            s, size = ref.page_scores(row[ok], dig, qf[b, i, :, :512], qf[b, i, :, 512:], scale, 64 * len(ok) + 1)
            want[ok] = s
            assert np.array_equal(np.isneginf(got[b, i]), np.isneginf(want)), (b, i)
            tol = _score_tol(size, H, P)
            # fp32 has no normal number below 2^-126: each of the H weights under it may become 0
            assert np.all(np.abs(got[b, i, ok] - s) <= tol * s + H * 2.0 ** -126), (b, i, np.max(np.abs(got[b, i, ok] / s - 1)), tol)


@pytest.mark.parametrize("H", [1, 7, 8, 16, 20, 33, 64, 100, 128])
def test_scores_heads(H):
    _scores_case([1000, 64, 65, 1, 130], 1, H, seed=H)


@pytest.mark.parametrize("lens,s_q,H", [([1], 1, 16), ([64], 1, 16), ([65], 1, 16), ([2, 300], 3, 16), ([8192, 77, 8193], 2, 128),
                                        ([40000], 1, 128), ([70000, 100], 1, 32), ([300] * 70, 1, 16)])
def test_scores_lengths(lens, s_q, H):
    _scores_case(lens, s_q, H, seed=len(lens) + H)


def test_scores_in_every_cluster_size():
    """One query to many, short to long: one CTA a query up to sixteen."""
    for lens in ([64 * 100] * 150, [64 * 200] * 60, [64 * 500] * 30, [64 * 1000] * 12, [64 * 2040 + 1] * 3):
        _scores_case(lens, 1, 8, seed=len(lens))


def test_scores_beyond_one_sweep():
    """More pages than a query's accumulators hold at once."""
    _scores_case([64 * 9000 + 5], 1, 128, seed=2)
    _scores_case([64 * 9000 + 5, 3000], 1, 16, seed=3)


def test_scores_large_logits_and_zero_scale():
    _scores_case([2000, 500], 1, 16, scale=2.0, gain=6.0, seed=4)   # logits of +-300: a few pages hold everything
    _scores_case([2000, 500], 1, 16, scale=0.0, seed=5)             # every page the same
    _scores_case([2000, 500], 1, 16, scale=-SCALE, seed=6)


def test_scores_bad_pages_do_not_count():
    _scores_case([2000, 500], 2, 16, bad=[(0, 3), (0, 16), (1, 0)], seed=7)
    _scores_case([100], 1, 16, bad=[(0, 0)], seed=8)  # the only candidate


def test_scores_bad_length_is_clamped():
    rng = np.random.default_rng(1)
    table = _i32([[0, 1, 2]])
    dig = torch.from_numpy(rng.standard_normal((3, 576)).astype(np.float32)).bfloat16().cuda()
    q = torch.from_numpy(rng.standard_normal((1, 1, 4, 576)).astype(np.float32)).bfloat16().cuda()
    q_c, q_r = q[..., :512].contiguous(), q[..., 512:].contiguous()
    good = api.mla_page_scores(table, _i32([150]), 150, dig, q_c, q_r, SCALE)
    assert api.mla_get_device_status() == 0
    assert torch.equal(api.mla_page_scores(table, _i32([9999]), 150, dig, q_c, q_r, SCALE), good)
    assert api.mla_get_device_status() == api._lib.MLA_ERR_INVALID_ARG
    none = api.mla_page_scores(table, _i32([-5]), 150, dig, q_c, q_r, SCALE)
    assert api.mla_get_device_status() == api._lib.MLA_ERR_INVALID_ARG
    assert bool(torch.isneginf(none).all())


def _select_case(scores, lens, k, n_sink, n_recent, seed=0):
    rng = np.random.default_rng(seed)
    lens = np.asarray(lens)
    B, s_q, W = scores.shape
    table, _ = ref.random_table(rng, lens)
    t, p, n = api.mla_select_pages(_i32(table), _i32(lens), int(lens.max()), torch.from_numpy(scores).cuda(), k,
                                   n_sink=n_sink, n_recent=n_recent)
    assert api.mla_get_device_status() == 0
    t, p, n = t.cpu().numpy(), p.cpu().numpy(), n.cpu().numpy()
    for b in range(B):
        for i in range(s_q):
            pages, keys = ref.select(scores[b, i], int(lens[b]) - s_q + 1 + i, k, n_sink, n_recent)
            pad = [-1] * (k - len(pages))
            assert list(p[b, i]) == pages + pad, (b, i)
            assert list(t[b, i]) == [int(table[b, x]) for x in pages] + pad, (b, i)
            assert n[b, i] == keys


@pytest.mark.parametrize("lens,s_q,k,n_sink,n_recent", [
    ([1], 1, 1, 0, 1), ([5000, 64, 65, 3], 1, 8, 1, 2), ([5000, 200], 3, 16, 0, 1), ([70000], 1, 300, 4, 8),
    ([64 * 1025, 64 * 1024, 64 * 256 + 1], 2, 64, 2, 2), ([4096] * 3, 1, 64, 1, 1), ([4096] * 3, 1, 63, 31, 32),
    ([64 * 20000 + 9], 1, 777, 1, 1), ([64 * 70000], 1, 66000, 1, 1), ([64 * 7000], 1, 500, 1, 1), ([1, 2, 3], 4, 5, 0, 1), ([64 * 300], 1, 1, 0, 1), ([64 * 5000] * 2, 1, 4096, 3, 3)])
def test_select(lens, s_q, k, n_sink, n_recent):
    rng = np.random.default_rng(len(lens) + k)
    W = -(-max(lens) // 64)
    _select_case(rng.random((len(lens), s_q, W)).astype(np.float32), lens, k, n_sink, n_recent)


def test_select_ties_and_special_values():
    rng = np.random.default_rng(5)
    W, lens = 300, [64 * 300, 64 * 299 + 1, 64 * 200]
    few = rng.integers(0, 3, (3, 1, W)).astype(np.float32)
    for k in (3, 17, 128, 299, 300, 301):
        _select_case(few, lens, k, 1, 2)
    _select_case(np.zeros((3, 1, W), np.float32), lens, 50, 0, 1)
    odd = rng.standard_normal((3, 1, W)).astype(np.float32)
    odd[rng.random(odd.shape) < 0.3] = -np.inf
    odd[rng.random(odd.shape) < 0.1] = np.inf
    odd[rng.random(odd.shape) < 0.3] = np.nan
    odd[rng.random(odd.shape) < 0.1] = -0.0
    odd[rng.random(odd.shape) < 0.1] = 0.0
    odd[rng.random(odd.shape) < 0.05] = 1e-42
    for k in (5, 60, 200, 280):
        _select_case(odd, lens, k, 1, 1)
    _select_case(np.full((3, 1, W), np.nan, np.float32), lens, 9, 0, 1)


def test_select_without_scores():
    t, p, n = api.mla_select_pages(_i32([[4, 2, 7]]), _i32([130]), 192, None, 3, s_q=2)
    assert t.tolist() == [[[4, 2, 7], [4, 2, 7]]] and p.tolist() == [[[0, 1, 2]] * 2] and n.tolist() == [[129, 130]]
    t, p, n = api.mla_select_pages(_i32([[4, 2, 7]]), _i32([1]), 192, None, 4, s_q=2)
    assert t.tolist() == [[[-1] * 4, [4, -1, -1, -1]]] and n.tolist() == [[0, 1]]


def _sparse_case(fmt, lens, s_q, H, k, n_sink, n_recent, seed=0, out_dtype=torch.float32, num_splits=1):
    """The step against float64 over the pages that the library's own scores and selection name
    (each of them is tested on its own): the decode's error bound holds over the selection."""
    rng = np.random.default_rng(seed)
    lens = np.asarray(lens)
    B = len(lens)
    table, pages = ref.random_table(rng, lens)
    u = rng.standard_normal((B, 1, 1, 576))
    q = torch.from_numpy((u + 0.5 * rng.standard_normal((B, s_q, H, 576))).astype(np.float32)).bfloat16()
    off = np.zeros((pages, 576))
    for b in range(B):
        for p in table[b][table[b] >= 0]:
            if rng.random() < 0.3:
                off[p] = u[b, 0, 0] / np.linalg.norm(u[b]) * rng.uniform(1, 3)
    pool = ref.random_pool(rng, fmt, pages, off)
    desc = api.make_desc(*fmt, num_pages=pages)
    pool_t, table_t, lens_t, L = torch.from_numpy(pool).cuda(), _i32(table), _i32(lens), int(lens.max())
    dig = api.new_digests(desc)
    api.mla_page_digest(desc, pool_t, table_t, torch.zeros_like(lens_t), L, dig, new_lens=lens_t)
    q_c, q_r = q[..., :512].contiguous().cuda(), q[..., 512:].contiguous().cuda()
    lse = torch.empty((B, s_q, H), device="cuda")
    out, _ = api.mla_qdecode_sparse(desc, pool_t, table_t, lens_t, L, dig, q_c, q_r, SCALE, k, n_sink=n_sink,
                                    n_recent=n_recent, out_dtype=out_dtype, lse=lse, num_splits=num_splits)
    scores = api.mla_page_scores(table_t, lens_t, L, dig, q_c, q_r, SCALE) if k < -(-L // 64) else None
    t, p, n = api.mla_select_pages(table_t, lens_t, L, scores, k, n_sink=n_sink, n_recent=n_recent, s_q=s_q)
    # the parts give the step's own result
    lse2 = torch.empty((B * s_q, 1, H), device="cuda")
    out2, _ = api.mla_qdecode(desc, pool_t, t.view(B * s_q, k), n.view(-1), min(64 * k, L), q_c.view(B * s_q, 1, H, 512),
                              q_r.view(B * s_q, 1, H, 64), SCALE, out_dtype=out_dtype, lse=lse2, num_splits=num_splits)
    assert api.mla_get_device_status() == 0
    assert torch.equal(out.view(-1), out2.view(-1)) and torch.equal(lse.view(-1), lse2.view(-1))
    want = {}
    p, n, qf = p.cpu().numpy(), n.cpu().numpy(), ref.f32(q)
    for b in range(B):
        o, l = np.zeros((s_q, H, 512)), np.full((s_q, H), -np.inf)
        for i in range(s_q):
            keys = int(n[b, i])
            if keys:
                row = [int(table[b, x]) for x in p[b, i] if x >= 0]
                C, R = layout.gather_tokens(ref.np_desc(fmt), pool, row, keys)
                o[i], l[i] = attention.attend(qf[b, i, :, :512], qf[b, i, :, 512:], C, R, SCALE, np.full(H, keys))
        want[b] = (o, l)
    err, lerr = mc.parity(out, lse, want, bf16_out=out_dtype == torch.bfloat16)
    assert err <= mc.RTOL_RMS and lerr <= mc.LSE_ATOL, (err, lerr)


@pytest.mark.parametrize("fmt,lens,s_q,H,k,n_sink,n_recent", [
    ((4, 64, 4, 64), [1000, 70, 1, 64], 1, 128, 4, 1, 1),
    ((2, 32, 4, 64), [900, 300, 2], 3, 128, 5, 1, 2),
    ((4, 64, 4, 64), [2000, 64, 700], 1, 16, 6, 0, 1),
    ((4, 32, 2, 64), [700, 650], 2, 20, 3, 1, 1),
    ((2, 64, 2, 32), [1500], 1, 1, 8, 2, 2),
    ((4, 64, 4, 64), [500, 130], 2, 64, 100, 1, 1),     # every page: no scores
    ((2, 32, 4, 64), [64 * 40], 1, 128, 33, 1, 1)])
def test_sparse_step(fmt, lens, s_q, H, k, n_sink, n_recent):
    _sparse_case(fmt, lens, s_q, H, k, n_sink, n_recent, seed=H + k)


@pytest.mark.parametrize("num_splits", [2, 5])
def test_sparse_step_split(num_splits):
    _sparse_case((4, 64, 4, 64), [1500, 900, 20], 2, 128, 9, 1, 2, num_splits=num_splits)
    _sparse_case((4, 64, 4, 64), [1500, 900, 20], 1, 16, 9, 1, 2, num_splits=num_splits)


def test_sparse_step_bf16_out():
    _sparse_case((4, 64, 4, 64), [800, 90], 1, 128, 4, 1, 1, out_dtype=torch.bfloat16)


def test_sparse_covering_every_page_is_the_dense_decode():
    rng = np.random.default_rng(3)
    fmt, lens, H = (4, 64, 4, 64), np.array([300, 64, 1]), 128
    table, pages = ref.random_table(rng, lens)
    pool = torch.from_numpy(ref.random_pool(rng, fmt, pages)).cuda()
    desc = api.make_desc(*fmt, num_pages=pages)
    q_c, q_r = ref.bf16_randn(rng, (3, 1, H, 512)).cuda(), ref.bf16_randn(rng, (3, 1, H, 64)).cuda()
    a, _ = api.mla_qdecode(desc, pool, _i32(table), _i32(lens), 300, q_c, q_r, SCALE, num_splits=1)
    b, _ = api.mla_qdecode_sparse(desc, pool, _i32(table), _i32(lens), 300, None, q_c, q_r, SCALE, 5, num_splits=1)
    assert torch.equal(a, b)


def test_select_all_and_dense_window_only():
    """n_sink + n_recent = k: nothing is left to the scores."""
    _select_case(np.random.default_rng(1).random((1, 1, 40)).astype(np.float32), [64 * 40], 10, 4, 6)


def _serving_state(fmt=(4, 64, 4, 64), B=3, H=16, T=700):
    rng = np.random.default_rng(8)
    desc = api.make_desc(*fmt, num_pages=B * 14)
    table = torch.from_numpy(rng.permutation(B * 14).astype(np.int32)).cuda().view(B, 14)
    cs = torch.from_numpy(ref.angle_table(1000)).cuda()
    w = (1 + 0.1 * ref.bf16_randn(rng, (512,))).cuda()
    return rng, desc, table, cs, w


def test_serving_run():
    """Prefill in two chunks, read back, then decode steps that append, complete pages and attend
    sparsely: each step against float64 over the tokens fed so far."""
    fmt, B, H, k = (4, 64, 4, 64), 3, 16, 5
    rng, desc, table, cs, w = _serving_state(fmt, B, H)
    pool, dig = api.new_qcache_pool(desc), api.new_digests(desc)
    d, want = ref.np_desc(fmt), layout.new_pool(ref.np_desc(fmt), desc.num_pages)
    lens = np.zeros(B, dtype=np.int64)
    tab = table.cpu().numpy()
    for n, given in ((400, [400, 250, 37]), (300, [200, 300, 31]), (1, None), (2, None), (1, None), (1, None)):
        kv, q = ref.bf16_randn(rng, (B, n, 576)), ref.bf16_randn(rng, (B, n, H, 64))
        before, new = _i32(lens), None if given is None else _i32(given)
        rows = torch.zeros((B, n, 576), dtype=torch.bfloat16, device="cuda")
        q_r = api.mla_qcache_append_norm_rope(desc, pool, table, before, kv.cuda(), w, 1e-6, cs, q=q.cuda(), new_lens=new,
                                              rows_out=rows)
        api.mla_page_digest(desc, pool, table, before, n, dig, new_lens=new)
        count = np.full(B, n) if given is None else np.asarray(given)
        x = ref.f32(kv)
        pos = lens[:, None] + np.arange(n)
        c = ref.to_bf16_f32(ref.rms_norm(x[..., :512], ref.f32(w), 1e-6))
        kr = ref.to_bf16_f32(ref.rotate(x[..., 512:], ref.angle_table(1000)[pos], "interleaved"))
        for b in range(B):
            layout.append(d, want, tab[b:b + 1], [lens[b]], c[b:b + 1, :count[b]], kr[b:b + 1, :count[b]])
        lens = lens + count
        assert np.array_equal(pool.cpu().numpy(), want)
        lens_t, L = _i32(lens), int(lens.max())
        if n > 2:  # read everything back: the newest rows are those the append returned
            cu = np.concatenate([[0], np.cumsum(lens)])
            buf = torch.zeros((int(cu[-1]), 576), dtype=torch.bfloat16, device="cuda")
            api.mla_qcache_read(desc, pool, table, None, _i32(cu), L, buf[:, :512], buf[:, 512:])
            for b in range(B):
                assert torch.equal(buf[cu[b + 1] - count[b]:cu[b + 1]], rows[b, :count[b]])
            continue
        q_c = ref.bf16_randn(rng, (B, n, H, 512)).cuda()
        lse = torch.empty((B, n, H), device="cuda")
        out, _ = api.mla_qdecode_sparse(desc, pool, table, lens_t, L, dig, q_c, q_r, SCALE, k, n_sink=1, n_recent=1,
                                        out_dtype=torch.float32, lse=lse)
        scores = api.mla_page_scores(table, lens_t, L, dig, q_c, q_r, SCALE)
        _, pages, keys = api.mla_select_pages(table, lens_t, L, scores, k, n_sink=1, n_recent=1)
        assert api.mla_get_device_status() == 0
        pages, keys, res = pages.cpu().numpy(), keys.cpu().numpy(), {}
        for b in range(B):
            o, l = np.zeros((n, H, 512)), np.zeros((n, H))
            for i in range(n):
                row = [int(tab[b, p]) for p in pages[b, i] if p >= 0]
                C, R = layout.gather_tokens(d, want, row, int(keys[b, i]))
                o[i], l[i] = attention.attend(ref.f32(q_c)[b, i], ref.f32(q_r)[b, i], C, R, SCALE, np.full(H, keys[b, i]))
            res[b] = (o, l)
        err, lerr = mc.parity(out, lse, res)
        assert err <= mc.RTOL_RMS and lerr <= mc.LSE_ATOL, (err, lerr)


def test_step_captured_in_a_graph_and_on_another_stream():
    """append + digest + sparse decode captured once and replayed as the lengths grow gives the eager
    calls' results; and the same on a stream that is not the current one."""
    fmt, B, H, k = (2, 32, 4, 64), 3, 128, 4
    rng, desc, table, cs, w = _serving_state(fmt, B, H)
    pool, dig = api.new_qcache_pool(desc), api.new_digests(desc)
    first = ref.bf16_randn(rng, (B, 600, 576)).cuda()
    zero = torch.zeros(B, dtype=torch.int32, device="cuda")
    api.mla_qcache_append_norm_rope(desc, pool, table, zero, first, w, 1e-6, cs)
    api.mla_page_digest(desc, pool, table, zero, 600, dig)
    kv, q = ref.bf16_randn(rng, (B, 1, 576)).cuda(), ref.bf16_randn(rng, (B, 1, H, 64)).cuda()
    q_c = ref.bf16_randn(rng, (B, 1, H, 512)).cuda()

    def step(state, stream=None):
        pool, dig, before, after = state
        qr = api.mla_qcache_append_norm_rope(desc, pool, table, before, kv, w, 1e-6, cs, q=q, stream=stream)
        api.mla_page_digest(desc, pool, table, before, 1, dig, stream=stream)
        return api.mla_qdecode_sparse(desc, pool, table, after, 896, dig, q_c, qr, SCALE, k, stream=stream)[0]

    def state():
        before = torch.tensor([637, 600, 639], dtype=torch.int32, device="cuda")
        return pool.clone(), dig.clone(), before, before + 1

    eager, want = state(), []
    for _ in range(4):
        want.append(step(eager).clone())
        eager[2].add_(1), eager[3].add_(1)
    live = state()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        warm = state()
        step(warm)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(live)
    live[0].copy_(pool), live[1].copy_(dig)
    for r in range(4):
        graph.replay()
        assert torch.equal(out, want[r]), r
        live[2].add_(1), live[3].add_(1)
    assert torch.equal(live[0], eager[0]) and torch.equal(live[1], eager[1])
    other = state()
    side.wait_stream(torch.cuda.current_stream())
    got = step(other, stream=side)
    side.synchronize()
    assert torch.equal(got, want[0])
    raw = state()
    torch.cuda.synchronize()
    got = step(raw, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(got, want[0])
    assert api.mla_get_device_status() == 0


def test_steps_at_once_on_two_streams():
    """Two batches' steps in flight together, each with its own workspace, give what they give alone."""
    rng = np.random.default_rng(21)
    fmt, H, k = (4, 64, 4, 64), 128, 6
    jobs = []
    for lens in ([4000, 300, 2500], [1800, 3900, 64, 1]):
        lens = np.array(lens)
        table, pages = ref.random_table(rng, lens)
        desc = api.make_desc(*fmt, num_pages=pages)
        pool, dig = torch.from_numpy(ref.random_pool(rng, fmt, pages)).cuda(), api.new_digests(desc)
        api.mla_page_digest(desc, pool, _i32(table), torch.zeros(len(lens), dtype=torch.int32).cuda(), int(lens.max()), dig,
                            new_lens=_i32(lens))
        q_c, q_r = ref.bf16_randn(rng, (len(lens), 1, H, 512)).cuda(), ref.bf16_randn(rng, (len(lens), 1, H, 64)).cuda()
        jobs.append((desc, pool, _i32(table), _i32(lens), int(lens.max()), dig, q_c, q_r, SCALE, k))
    alone = [api.mla_qdecode_sparse(*j)[0] for j in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        outs = [api.mla_qdecode_sparse(*j, stream=s)[0] for j, s in zip(jobs, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(alone, outs))
    assert api.mla_get_device_status() == 0


def test_two_graphs_take_turns():
    """Two captured steps of different batches, replayed alternately and with new inputs."""
    rng = np.random.default_rng(22)
    fmt, H, k = (2, 32, 4, 64), 16, 4
    graphs = []
    for lens in ([2000, 130], [900, 700, 5]):
        lens = np.array(lens)
        table, pages = ref.random_table(rng, lens + 64)
        desc = api.make_desc(*fmt, num_pages=pages)
        pool, dig = torch.from_numpy(ref.random_pool(rng, fmt, pages)).cuda(), api.new_digests(desc)
        lens_t, L = _i32(lens), int(lens.max()) + 64
        api.mla_page_digest(desc, pool, _i32(table), torch.zeros_like(lens_t), L, dig, new_lens=lens_t)
        q = ref.bf16_randn(rng, (len(lens), 1, H, 576)).cuda()
        q_c, q_r = q[..., :512].contiguous(), q[..., 512:].contiguous()
        args = (desc, pool, _i32(table), lens_t, L, dig, q_c, q_r, SCALE, k)
        api.mla_qdecode_sparse(*args)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = api.mla_qdecode_sparse(*args)[0]
        graphs.append((g, out, args, q_c, lens_t))
    for step in range(3):
        for g, _, _, _, _ in graphs:
            g.replay()
        for g, out, args, q_c, lens_t in graphs:
            assert torch.equal(out, api.mla_qdecode_sparse(*args)[0]), step
            q_c.copy_(torch.flip(q_c, [0]))
            lens_t += 7
    assert api.mla_get_device_status() == 0


def test_batches_of_nothing():
    desc = api.make_desc(4, 64, 4, 64, num_pages=1)
    pool, dig = api.new_qcache_pool(desc), api.new_digests(desc)
    for B, L in ((0, 100), (2, 64), (2, 0)):
        table = torch.zeros((B, 2), dtype=torch.int32, device="cuda")
        lens = torch.zeros(B, dtype=torch.int32, device="cuda")
        q_c = torch.ones((B, 1, 4, 512), dtype=torch.bfloat16, device="cuda")
        q_r = torch.ones((B, 1, 4, 64), dtype=torch.bfloat16, device="cuda")
        lse = torch.zeros((B, 1, 4), device="cuda")
        out, _ = api.mla_qdecode_sparse(desc, pool, table, lens, L, dig, q_c, q_r, SCALE, 1, n_sink=0, lse=lse)
        assert bool((out == 0).all()) and bool(torch.isneginf(lse).all())
        sc = api.mla_page_scores(table, lens, L, dig, q_c, q_r, SCALE)
        assert sc.shape == (B, 1, -(-L // 64)) and bool(torch.isneginf(sc).all())
        t, p, n = api.mla_select_pages(table, lens, L, sc, 1, n_sink=0)
        assert bool((t == -1).all()) and bool((p == -1).all()) and bool((n == 0).all())
    assert api.mla_get_device_status() == 0


def test_sparse_with_more_pages_asked_for_than_there_are():
    """The largest k_pages, with first and newest pages beyond the context too, is the dense decode, in a
    workspace no larger than the pages need."""
    rng = np.random.default_rng(33)
    fmt, lens = (4, 64, 4, 64), np.array([300, 64, 1])
    table, pages = ref.random_table(rng, lens)
    pool = torch.from_numpy(ref.random_pool(rng, fmt, pages)).cuda()
    desc = api.make_desc(*fmt, num_pages=pages)
    for H, k, sink, recent in ((128, 2 ** 20, 1, 1), (16, 2 ** 20, 2 ** 19, 2 ** 19), (20, 6, 3, 3)):
        q_c, q_r = ref.bf16_randn(rng, (3, 2, H, 512)).cuda(), ref.bf16_randn(rng, (3, 2, H, 64)).cuda()
        need = api.mla_qdecode_sparse_workspace_bytes(3, 2, H, 300, k, 1)
        assert need <= 4096
        ws = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
        out, lse = None, torch.empty((3, 2, H), device="cuda")
        out, _ = api.mla_qdecode_sparse(desc, pool, _i32(table), _i32(lens), 300, None, q_c, q_r, SCALE, k, n_sink=sink,
                                        n_recent=recent, num_splits=1, lse=lse, workspace=ws[:need])
        assert api.mla_get_device_status() == 0 and bool((ws[need:] == 0xA5).all())
        # query i of request b as a request of its own
        own = _i32([n - 1 + i for n in lens for i in range(2)])
        rows = _i32(np.repeat(table, 2, 0))
        lse2 = torch.empty((6, 1, H), device="cuda")
        want, _ = api.mla_qdecode(desc, pool, rows, own, 300, q_c.view(6, 1, H, 512), q_r.view(6, 1, H, 64), SCALE,
                                  num_splits=1, lse=lse2)
        assert api.mla_get_device_status() == 0
        assert torch.equal(out.view(-1), want.view(-1)) and torch.equal(lse.view(-1), lse2.view(-1))


def test_impossible_calls_are_refused_before_anything_is_allocated():
    B, H, k = 64, 2, 2 ** 20
    desc = api.make_desc(4, 64, 4, 64, num_pages=2)
    pool, dig = api.new_qcache_pool(desc), api.new_digests(desc)
    table, lens = torch.zeros((B, 2), dtype=torch.int32, device="cuda"), torch.ones(B, dtype=torch.int32, device="cuda")
    q_c = torch.zeros((B, 1, H, 512), dtype=torch.bfloat16, device="cuda")
    q_r = torch.zeros((B, 1, H, 64), dtype=torch.bfloat16, device="cuda")
    inv, cap, uns = api._lib.MLA_ERR_INVALID_ARG, api._lib.MLA_ERR_CAPACITY, api._lib.MLA_ERR_UNSUPPORTED
    bad = [(k, dict(n_sink=-1), 128, inv), (k, dict(n_recent=0), 128, inv), (k, dict(n_sink=k), 128, inv), (0, {}, 128, inv),
           (k + 1, {}, 128, inv), (k, dict(n_sink=2 ** 40), 128, inv), (k, dict(n_recent=2 ** 62, n_sink=2 ** 62), 128, inv),
           (k, {}, 129, cap), (2, {}, 2 ** 31 - 1, cap)]
    torch.cuda.synchronize()
    held = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    for pages, kw, L, code in bad:
        with pytest.raises(api.MlaError) as e:
            api.mla_select_pages(table, lens, L, None, pages, s_q=1, **kw)
        assert e.value.code == code
        with pytest.raises(api.MlaError) as e:
            api.mla_qdecode_sparse(desc, pool, table, lens, L, dig, q_c, q_r, SCALE, pages, **kw)
        assert e.value.code == code
    with pytest.raises(api.MlaError) as e:
        api.mla_select_pages(table, lens, 128, None, k, s_q=1024)
    assert e.value.code == uns
    with pytest.raises(api.MlaError) as e:
        api.mla_page_scores(table, lens, 2 ** 31 - 1, dig, q_c, q_r, SCALE)
    assert e.value.code == cap
    assert torch.cuda.max_memory_allocated() == held
    api.mla_select_pages(table, lens, 128, None, 2, s_q=1)
    assert api.mla_get_device_status() == 0
