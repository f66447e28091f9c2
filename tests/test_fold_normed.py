"""Folding where the latent is normed between its projection and the cache: equivalence in float64 (CPU), and
through the append that norms, rotates and quantizes (GPU)."""
import numpy as np
import pytest
import torch

from bit_mla_kv_qdecode_b200 import api, fold
from oracle import attention
from tests import operator_refs as ref
from tests.test_fold import D_C, D_H, D_Q, D_R, D_V, H, _orth, _weights

EPS = 1e-6


def _norm(x, w=None):
    return ref.rms_norm(x, w, EPS)


def _attend(W, c, cq, convention):
    """The library's absorbed form over the cache c [T, d_c], k_r: outputs [H, D_V] of the last position."""
    T = len(c)
    kr = fold.rope(W["kr"], np.arange(T), convention=convention)
    qc = np.stack([W["W_uk"][h].T @ (W["W_uq"][h] @ cq) for h in range(H)])
    qr = np.stack([fold.rope(W["W_qr"][h] @ cq, T - 1, convention=convention) for h in range(H)])
    o, _ = attention.attend(qc, qr, c, kr, 1.0 / np.sqrt(D_H + D_R), np.full(H, T))
    return np.stack([W["W_uv"][h] @ o[h] for h in range(H)])


@pytest.mark.parametrize("convention", ["interleaved", "half"])
@pytest.mark.parametrize("weight", [True, False])
def test_folded_normed_layer_is_equivalent(convention, weight):
    rng = np.random.default_rng(51)
    W = _weights(rng)
    w = rng.uniform(0.2, 3.0, D_C) if weight else None
    R, D = _orth(rng, D_C), rng.uniform(0.2, 5.0, D_C)
    M = fold.rope_pair_transform(rng.uniform(-np.pi, np.pi, D_R // 2), rng.uniform(0.2, 5.0, D_R // 2), convention)
    h, cq = rng.standard_normal((33, W["W_dkv"].shape[1])), rng.standard_normal(D_Q)
    # the model: keys and values up-projected from w * norm(W_dkv h), head by head
    c = _norm(h @ W["W_dkv"].T, w)
    kr = fold.rope(h @ W["W_kr"].T, np.arange(33), convention=convention)
    want = np.zeros((H, D_V))
    for a in range(H):
        s = c @ W["W_uk"][a].T @ (W["W_uq"][a] @ cq) + kr @ fold.rope(W["W_qr"][a] @ cq, 32, convention=convention)
        p = np.exp((s - s.max()) / np.sqrt(D_H + D_R))
        want[a] = (p / p.sum()) @ (c @ W["W_uv"][a].T)
    F = dict(W)
    F["W_dkv"], scale, F["W_uk"], F["W_uv"] = fold.fold_normed_content(W["W_dkv"], W["W_uk"], W["W_uv"], w, R, D)
    F["W_kr"], F["W_qr"] = fold.fold_rope(W["W_kr"], W["W_qr"], M)
    F["kr"] = h @ F["W_kr"].T
    cache = _norm(h @ F["W_dkv"].T, scale)
    assert np.allclose(_attend(F, cache, cq, convention), want, rtol=1e-10, atol=1e-12)
    # the cache holds the transform of the normed latent
    assert np.allclose(cache, _norm(h @ W["W_dkv"].T) @ fold.content_transform(R, D).T, rtol=1e-10, atol=1e-12)
    # negative control: the fold for latents that are not normed, with the norm left in between
    X = dict(F)
    W_dkv, X["W_uk"], X["W_uv"] = fold.fold_content(W["W_dkv"], W["W_uk"], W["W_uv"], fold.content_transform(R, D))
    assert not np.allclose(_attend(X, _norm(h @ W_dkv.T, w), cq, convention), want, rtol=1e-2)


def test_bad_shapes_are_rejected():
    rng = np.random.default_rng(52)
    W = _weights(rng)
    with pytest.raises(ValueError):
        fold.fold_normed_content(W["W_dkv"], W["W_uk"], W["W_uv"], np.ones(D_C - 1), np.eye(D_C), np.ones(D_C))
    with pytest.raises(ValueError):
        fold.fold_normed_content(W["W_dkv"], W["W_uk"], W["W_uv"], None, np.eye(D_C), -np.ones(D_C))
    with pytest.raises(ValueError):
        fold.fold_normed_content(W["W_dkv"], W["W_uk"], W["W_uv"], None, 2 * np.eye(D_C), np.ones(D_C))


@pytest.mark.gpu
@pytest.mark.parametrize("convention", ["interleaved", "half"])
def test_append_of_folded_projections_holds_the_transformed_latent(convention):
    """kv from the folded projections through the append: the cache holds T norm(W_dkv h) and the rotated M k_r."""
    rng = np.random.default_rng(53)
    d_model, n, fmt = 96, 70, (4, 32, 4, 32)
    W_dkv, W_kr = rng.standard_normal((512, d_model)) / 7, rng.standard_normal((64, d_model)) / 7
    R = _orth(rng, 512)
    D = ref.to_bf16_f32(rng.uniform(0.2, 5.0, 512)).astype(np.float64)
    M = fold.rope_pair_transform(rng.uniform(-np.pi, np.pi, 32), rng.uniform(0.3, 3.0, 32), convention)
    up = np.zeros((1, 1, 512))
    F_dkv, scale, _, _ = fold.fold_normed_content(W_dkv, up, up, None, R, D)
    F_kr, _ = fold.fold_rope(W_kr, np.zeros((1, 64, 1)), M)
    h = rng.standard_normal((n, d_model))
    kv = torch.from_numpy(np.concatenate([h @ F_dkv.T, h @ F_kr.T], 1).astype(np.float32)).bfloat16().view(1, n, 576).cuda()
    desc = api.make_desc(*fmt, num_pages=2)
    pool, rows = api.new_qcache_pool(desc), torch.zeros_like(kv)
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    cs = ref.angle_table(n)
    api.mla_qcache_append_norm_rope(desc, pool, torch.tensor([[1, 0]], dtype=torch.int32, device="cuda"), zero, kv,
                                    torch.from_numpy(scale.astype(np.float32)).bfloat16().cuda(), EPS,
                                    torch.from_numpy(cs).cuda(), convention=convention, rows_out=rows)
    assert api.mla_get_device_status() == 0
    got = ref.f32(rows)[0].astype(np.float64)
    c = _norm(h @ W_dkv.T) @ fold.content_transform(R, D).T
    k = ref.rotate(h @ W_kr.T, cs, convention) @ M.T
    # Before the quantizer: kv rounded to bf16 (each channel, hence also the root mean square, by 2^-8 of itself),
    # the result again; a rotated channel comes of two, of its pair's length. Then half a step of a group of 32 and the
    # fp16 rounding of the offset (2^-11 of it) and of fifteen steps (2^-11 of the range); rows are rounded to bf16.
    pr = fold.rotary_pairs(64, convention)
    length = np.empty_like(k)
    length[:, pr[:, 0]] = length[:, pr[:, 1]] = np.hypot(k[:, pr[:, 0]], k[:, pr[:, 1]])
    unlike = _norm(h @ (fold.content_transform(R, D) @ W_dkv).T)  # the fold for latents that are not normed
    for x, size, out, wrong in ((c, np.abs(c), got[:, :512], unlike), (k, length, got[:, 512:], None)):
        e = 3.05 * ref.BF16_HALF * size
        g = lambda a: a.reshape(n, -1, 32)  # noqa: E731
        span = (g(x + e).max(-1) - g(x - e).min(-1))[..., None]
        tol = g(e) + span / 30 * 1.001 + 2.0 ** -11 * (np.abs(g(x)).max(-1, keepdims=True) * 1.05 + 2 * span)
        tol = tol + ref.BF16_HALF * (g(np.abs(x)) + tol)
        assert np.all(np.abs(g(out) - g(x)) <= tol)
        assert wrong is None or np.mean(np.abs(g(wrong) - g(x)) > tol) > 0.5
