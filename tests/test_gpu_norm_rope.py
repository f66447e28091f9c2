"""GPU tests of mla_qcache_append_norm_rope: bytes, rotated queries and rows against float64."""
import numpy as np
import pytest
import torch

from bit_mla_kv_qdecode_b200 import api
from oracle import layout
from tests import operator_refs as ref

pytestmark = pytest.mark.gpu
EPS = 1e-6


def _run(fmt, conv, before, n, H, new_lens=None, positions=None, weight=True, wide=True, seed=0, rows=True,
         q_inplace=False, scale=1.0):
    rng = np.random.default_rng(seed)
    B = len(before)
    table, pages = ref.random_table(rng, np.asarray(before) + n, spare=2)
    mag = np.exp(rng.normal(0, 0.5, 576)) * scale
    kv_w = ref.bf16_randn(rng, (B, n, 96 + 576 if wide else 576))
    kv_w[..., -576:] = (kv_w[..., -576:].float() * torch.from_numpy(mag).float()).bfloat16()
    q_w = ref.bf16_randn(rng, (B, n, H, 192 if wide and not q_inplace else 64))
    w = ref.bf16_randn(rng, (512,)) * 0.2 + 1.0 if weight else None
    limit = int(max(before)) + n if positions is None else int(positions.max()) + 1
    cs = ref.angle_table(limit)
    desc = api.make_desc(*fmt, num_pages=pages)
    pool = torch.randint(0, 256, (pages, api.mla_qcache_page_bytes(desc)), dtype=torch.uint8,
                         generator=torch.Generator().manual_seed(seed)).cuda()
    start = pool.cpu().numpy().copy()
    dev = lambda a: None if a is None else torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()  # noqa: E731
    kv, q = kv_w.cuda()[..., -576:], q_w.cuda()[..., -64:]
    fill = torch.full((B, n, H, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    rows_t = torch.full((B, n, 576), 7.0, dtype=torch.bfloat16, device="cuda") if rows else None
    q_out = api.mla_qcache_append_norm_rope(
        desc, pool, dev(table), dev(before), kv, None if w is None else w.cuda(), EPS, torch.from_numpy(cs).cuda(),
        convention=conv, q=q, q_out=q if q_inplace else fill, positions=dev(positions), new_lens=dev(new_lens),
        rows_out=rows_t)
    torch.cuda.synchronize()
    assert api.mla_get_device_status() == 0
    # float64
    x = ref.f32(kv_w)[..., -576:]
    c = ref.to_bf16_f32(ref.rms_norm(x[..., :512], None if w is None else ref.f32(w), EPS))
    count = np.full(B, n) if new_lens is None else np.asarray(new_lens)
    pos = np.asarray(before)[:, None] + np.arange(n) if positions is None else positions
    cs_t = cs[np.where(np.arange(n) < count[:, None], pos, 0)]
    kr = ref.to_bf16_f32(ref.rotate(x[..., 512:], cs_t, conv))
    d = ref.np_desc(fmt)
    want = start.copy()
    hat = np.full((B, n, 576), 7.0)
    for b in range(B):
        m = int(count[b])
        if m:
            layout.append(d, want, table[b:b + 1], [before[b]], c[b:b + 1, :m], kr[b:b + 1, :m])
            with np.errstate(invalid="ignore"):  # older slots hold random bytes
                C, R = layout.gather_tokens(d, want, table[b], before[b] + m)
            hat[b, :m] = np.concatenate([C, R], 1)[before[b]:]
    assert np.array_equal(pool.cpu().numpy(), want)
    live = (np.arange(n) < count[:, None])
    if rows:
        err = np.abs(ref.f32(rows_t) - hat)
        # u*s + z rounded to fp32, then to bf16
        assert np.all(err <= np.abs(hat) * (ref.BF16_HALF + 2 * ref.FP32_HALF))
    if H:
        v = ref.f32(q_w)[..., -64:]
        r64 = ref.rotate(v, cs_t[:, :, None], conv)
        # one product and one sum rounded in fp32, then bf16; the terms' size bounds the first
        size = np.abs(v).max(-1, keepdims=True) * 2
        got = ref.f32(q_out)
        tol = np.abs(r64) * ref.BF16_HALF + 2 * ref.FP32_HALF * size
        assert np.all(np.abs(got - r64)[live] <= tol[live])
        if not q_inplace:
            assert np.all(got[~live] == 7.0)
        else:
            assert np.array_equal(got[~live], v[~live])


@pytest.mark.parametrize("fmt", ref.FORMATS)
@pytest.mark.parametrize("conv", ["interleaved", "half"])
def test_formats_and_conventions(fmt, conv):
    _run(fmt, conv, [0, 61, 200], 9, 16)


@pytest.mark.parametrize("before,n,H", [([0], 1, 128), ([4095] * 5, 1, 128), ([63, 64, 0, 127], 1, 20), ([10], 130, 1),
                                        ([5, 700], 67, 40), ([0, 1], 3, 0), ([33] * 9, 2, 8), ([8190], 3, 33)])
def test_shapes(before, n, H):
    _run((4, 64, 4, 64), "interleaved", before, n, H, seed=n + H)


def test_padded_batch_positions_and_options():
    fmt = (2, 32, 4, 64)
    _run(fmt, "half", [0, 64, 30, 7], 70, 32, new_lens=[70, 0, 1, 69])
    pos = np.random.default_rng(3).integers(0, 5000, (2, 6)).astype(np.int32)
    _run(fmt, "half", [3, 100], 6, 16, positions=pos)
    _run(fmt, "interleaved", [3, 100], 6, 16, weight=False, wide=False, rows=False)
    _run(fmt, "interleaved", [3, 100], 6, 16, q_inplace=True, new_lens=[6, 2])
    _run(fmt, "half", [3, 100], 6, 16, q_inplace=True)


def test_magnitudes():
    # latents of any scale are brought to the quantizer's range: 1e-18 (eps dominates) to 1e18
    for scale in (1e-18, 1e-3, 1e3, 60000.0):
        _run((4, 64, 4, 64), "interleaved", [2], 5, 4, scale=scale if scale < 1e4 else 1e4, seed=5)
    rng = np.random.default_rng(1)
    kv = ref.bf16_randn(rng, (1, 1, 576))
    kv[0, 0, :512] *= 1e18
    kv[0, 0, 100:140] = 0
    desc = api.make_desc(4, 64, 4, 64, num_pages=1)
    pool = api.new_qcache_pool(desc)
    z = torch.zeros(1, dtype=torch.int32, device="cuda")
    cs = ref.angle_table(1)
    api.mla_qcache_append_norm_rope(desc, pool, z[None], z, kv.cuda(), None, EPS, torch.from_numpy(cs).cuda())
    x = ref.f32(kv)
    d = ref.np_desc((4, 64, 4, 64))
    want = layout.new_pool(d, 1)
    layout.append(d, want, np.zeros((1, 1), int), [0], ref.to_bf16_f32(ref.rms_norm(x[..., :512], None, EPS)), x[..., 512:])
    assert np.array_equal(pool.cpu().numpy(), want)


def test_same_bytes_as_append():
    """Ones and a position of angle 0 after a norm done outside: the bytes of mla_qcache_append."""
    rng = np.random.default_rng(11)
    fmt = (4, 32, 2, 64)
    kv = ref.bf16_randn(rng, (2, 80, 576))
    c = torch.from_numpy(ref.to_bf16_f32(ref.rms_norm(ref.f32(kv)[..., :512], None, EPS))).bfloat16().cuda()
    desc = api.make_desc(*fmt, num_pages=6)
    table = torch.arange(6, dtype=torch.int32, device="cuda").view(2, 3)
    before = torch.tensor([5, 60], dtype=torch.int32, device="cuda")
    a, b = api.new_qcache_pool(desc), api.new_qcache_pool(desc)
    api.mla_qcache_append(desc, a, table, before, c, kv[..., 512:].contiguous().cuda())
    cs = torch.from_numpy(ref.angle_table(1)).cuda()
    api.mla_qcache_append_norm_rope(desc, b, table, before, kv.cuda(), None, EPS, cs,
                                    positions=torch.zeros((2, 80), dtype=torch.int32, device="cuda"))
    assert torch.equal(a, b)


@pytest.mark.parametrize("fmt", [(4, 64, 4, 64), (2, 32, 2, 32), (4, 32, 2, 64), (2, 64, 4, 32)])
def test_codes_on_borders(fmt):
    """The division-free codes against mla_qcache_append's, where quotients meet borders: values that are
    multiples of half a step, steps from fp16's smallest to large, constant groups. The key part carries
    them (angle 0 leaves it as it is); the latent is what the norm makes of such values."""
    rng = np.random.default_rng(sum(fmt))
    n = 4096
    step = 2.0 ** rng.integers(-26, 8, (n, 1)) * rng.choice([1.0, 1.5, 1.0625, 1.984375, 0.0], (n, 1), p=[.4, .2, .2, .15, .05])
    kv = torch.from_numpy((step * rng.integers(-40, 41, (n, 576)) / 2).astype(np.float32)).bfloat16()
    kv[: n // 2, 512:] += torch.from_numpy((step[: n // 2] * rng.standard_normal((n // 2, 64)) * 4).astype(np.float32)).bfloat16()
    kv = kv.view(1, n, 576)
    c = torch.from_numpy(ref.to_bf16_f32(ref.rms_norm(ref.f32(kv)[..., :512], None, EPS))).bfloat16().cuda()
    desc = api.make_desc(*fmt, num_pages=n // 64)
    table = torch.arange(n // 64, dtype=torch.int32, device="cuda").view(1, -1)
    before = torch.zeros(1, dtype=torch.int32, device="cuda")
    a, b = api.new_qcache_pool(desc), api.new_qcache_pool(desc)
    api.mla_qcache_append(desc, a, table, before, c, kv[..., 512:].contiguous().cuda())
    api.mla_qcache_append_norm_rope(desc, b, table, before, kv.cuda(), None, EPS, torch.from_numpy(ref.angle_table(1)).cuda(),
                                    positions=torch.zeros((1, n), dtype=torch.int32, device="cuda"))
    assert torch.equal(a, b)


def test_bad_slots_and_positions_are_skipped():
    desc = api.make_desc(4, 64, 4, 64, num_pages=2)
    pool = api.new_qcache_pool(desc)
    kv = torch.ones((3, 1, 576), dtype=torch.bfloat16, device="cuda")
    q = torch.ones((3, 1, 4, 64), dtype=torch.bfloat16, device="cuda")
    cs = torch.from_numpy(ref.angle_table(64)).cuda()
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    rows = torch.full((3, 1, 576), 7.0, dtype=torch.bfloat16, device="cuda")
    q_out = torch.full_like(q, 7.0)
    # a table entry outside the pool, a position past the table row, an angle past the table of angles
    api.mla_qcache_append_norm_rope(desc, pool, i32([[9], [0], [1]]), i32([0, 64, 1]), kv, None, EPS, cs, q=q, q_out=q_out,
                                    rows_out=rows, positions=i32([[3], [3], [64]]))
    assert api.mla_get_device_status() == api._lib.MLA_ERR_INVALID_ARG
    assert int(pool.sum()) == 0 and bool((rows == 7.0).all())
    assert bool((q_out[2] == 7.0).all()) and bool((q_out[:2] != 7.0).all())
    for bad in (-1, -(2 ** 31)):
        api.mla_qcache_append_norm_rope(desc, pool, i32([[0], [0], [1]]), i32([bad] * 3), kv, None, EPS, cs)
        assert api.mla_get_device_status() == api._lib.MLA_ERR_INVALID_ARG
        assert int(pool.sum()) == 0


def test_empty_calls():
    desc = api.make_desc(4, 64, 4, 64, num_pages=1)
    pool = api.new_qcache_pool(desc)
    cs = torch.from_numpy(ref.angle_table(4)).cuda()
    for B, n in ((0, 3), (2, 0)):
        kv = torch.ones((B, n, 576), dtype=torch.bfloat16, device="cuda")
        table = torch.zeros((B, 1), dtype=torch.int32, device="cuda")
        z = torch.zeros(B, dtype=torch.int32, device="cuda")
        out = api.mla_qcache_append_norm_rope(desc, pool, table, z, kv, None, EPS, cs, q=kv.new_zeros((B, n, 2, 64)))
        assert out.shape == (B, n, 2, 64)
    assert api.mla_get_device_status() == 0 and int(pool.sum()) == 0


@pytest.mark.parametrize("fmt", [(4, 64, 4, 64), (2, 32, 2, 32), (4, 32, 2, 64), (2, 64, 4, 32)])
def test_same_bytes_as_append_beyond_the_range_of_fp16(fmt):
    """Offsets that overflow to an infinity, under steps that do and steps that do not: still the bytes of
    mla_qcache_append, and the oracle's wherever the step is finite. Weights carry the latent out there."""
    rng = np.random.default_rng(sum(fmt) + 1)
    n = 256
    kv = ref.f32(ref.bf16_randn(rng, (1, n, 576)))
    center = rng.choice([-7e4, -66000.0, -65520.0, -3e5, 7e4, 1e6, 0.0], (n, 1))
    width = rng.choice([0.0, 600.0, 5e3, 9e4, 3e6], (n, 1))
    kv[0, :, 512:] = center + width * rng.uniform(-1, 1, (n, 64))
    kv[0, 0, 512:], kv[0, 1, 512:] = -7e4 + 1000 * (np.arange(64) % 8), -1e38  # a finite step; a step of zero
    kv = torch.from_numpy(kv).bfloat16()
    w = torch.from_numpy(np.where(np.arange(512) // 64 % 2, 3e4, 1.0).astype(np.float32)).bfloat16()
    c = ref.to_bf16_f32(ref.rms_norm(ref.f32(kv)[..., :512], ref.f32(w), EPS))
    desc = api.make_desc(*fmt, num_pages=n // 64)
    table = torch.arange(n // 64, dtype=torch.int32, device="cuda").view(1, -1)
    before = torch.zeros(1, dtype=torch.int32, device="cuda")
    a, b = api.new_qcache_pool(desc), api.new_qcache_pool(desc)
    api.mla_qcache_append(desc, a, table, before, torch.from_numpy(c).bfloat16().cuda(), kv[..., 512:].contiguous().cuda())
    api.mla_qcache_append_norm_rope(desc, b, table, before, kv.cuda(), w.cuda(), EPS, torch.from_numpy(ref.angle_table(1)).cuda(),
                                    positions=torch.zeros((1, n), dtype=torch.int32, device="cuda"))
    assert api.mla_get_device_status() == 0
    assert torch.equal(a, b)
    d = ref.np_desc(fmt)
    want = layout.new_pool(d, 1)
    x = ref.f32(kv)[:, :1, 512:]
    with np.errstate(over="ignore"):
        layout.append(d, want, np.zeros((1, 1), int), [0], c[:, :1], x)
    off = 64 * 512 * fmt[0] // 8  # the key's codes of the first token: every one the largest
    assert np.all(b[0, off:off + 64 * fmt[2] // 8].cpu().numpy() == 255)
    assert np.array_equal(b[0, off:off + 64 * fmt[2] // 8].cpu().numpy(), want[0, off:off + 64 * fmt[2] // 8])


def test_counts_out_of_range_skip_the_request():
    """new_lens below 0 or above n_new: the append and the digests both leave the request as it is and flag it;
    the other requests are served."""
    rng = np.random.default_rng(31)
    fmt, n, H = (4, 64, 4, 64), 65, 3
    desc = api.make_desc(*fmt, num_pages=8)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    table, before = i32([[0, 1], [2, 3], [4, 5], [6, 7]]), i32([3, 0, 5, 60])
    kv, q = ref.bf16_randn(rng, (4, n, 576)).cuda(), ref.bf16_randn(rng, (4, n, H, 64)).cuda()
    cs = torch.from_numpy(ref.angle_table(200)).cuda()

    def run(new):
        pool, dig = api.new_qcache_pool(desc), api.new_digests(desc)
        rows, q_out = torch.full_like(kv, 7.0), torch.full_like(q, 7.0)
        api.mla_qcache_append_norm_rope(desc, pool, table, before, kv, None, EPS, cs, q=q, q_out=q_out, rows_out=rows,
                                        new_lens=i32(new))
        status = api.mla_get_device_status()
        api.mla_page_digest(desc, pool, table, before, n, dig, new_lens=i32(new))
        assert api.mla_get_device_status() == status
        return status, pool, dig, rows, q_out

    ok, *want = run([65, 0, 64, 0])
    assert ok == 0
    for a, b in ((66, -1), (-(2 ** 31), 2 ** 31 - 1)):
        bad, *got = run([65, a, 64, b])
        assert bad == api._lib.MLA_ERR_INVALID_ARG
        for x, y in zip(want, got):
            assert torch.equal(x, y)
