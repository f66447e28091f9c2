"""Plain float64 implementations of the operators around the cache, for the tests:
norm and rotation, read-back, page digests, page scores, page selection."""
from __future__ import annotations

import numpy as np
import torch

from bit_mla_kv_qdecode_b200 import fold, synth
from oracle import layout

FORMATS = [(4, 64, 4, 64), (2, 32, 4, 64), (4, 32, 2, 64), (2, 64, 2, 32), (4, 64, 2, 32), (2, 32, 4, 32)]
BF16_HALF = 2.0 ** -8   # half a step of bf16, relative to the value
FP32_HALF = 2.0 ** -24


def to_bf16_f32(x64) -> np.ndarray:
    """float64 -> fp32 -> bf16, each rounded to nearest, as fp32 values."""
    return synth.bf16_bits_to_f32(synth.f32_to_bf16_bits(np.asarray(x64).astype(np.float32)))


def f32(t: torch.Tensor) -> np.ndarray:
    return t.detach().float().cpu().numpy()


def bf16_randn(rng, shape, mag=None) -> torch.Tensor:
    x = rng.standard_normal(shape)
    if mag is not None:
        x = x * mag
    return torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16)


def angle_table(n, base=10000.0) -> np.ndarray:
    """fp32 [n, 64]: cosines, then sines, of the 32 pairs' angles."""
    th = np.arange(n, dtype=np.float64)[:, None] * base ** (-2.0 * np.arange(32) / 64)
    return np.concatenate([np.cos(th), np.sin(th)], 1).astype(np.float32)


def rotate(x, cs, convention) -> np.ndarray:
    """Rotary pairs of x [..., 64] turned by cs [..., 64] (cosines, sines), float64."""
    pr = fold.rotary_pairs(64, convention)
    x, c, s = x.astype(np.float64), cs[..., :32].astype(np.float64), cs[..., 32:].astype(np.float64)
    out = np.empty_like(x)
    a, b = x[..., pr[:, 0]], x[..., pr[:, 1]]
    out[..., pr[:, 0]] = a * c - b * s
    out[..., pr[:, 1]] = a * s + b * c
    return out


def rms_norm(x, w, eps) -> np.ndarray:
    x = x.astype(np.float64)
    y = x * (1.0 / np.sqrt((x * x).sum(-1, keepdims=True) / x.shape[-1] + float(np.float32(eps))))
    return y if w is None else y * w.astype(np.float64)


def np_desc(fmt):
    return layout.Desc(bits_c=fmt[0], group_c=fmt[1], bits_r=fmt[2], group_r=fmt[3])


def random_table(rng, lens, spare=0):
    """(block table int32 [B, max_pages], pages) of shuffled pages, `spare` pages unused."""
    pages = np.maximum((np.asarray(lens) + 63) // 64, 1)
    perm = rng.permutation(int(pages.sum()) + spare).astype(np.int32)
    table = np.full((len(pages), int(pages.max())), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, len(perm)


def random_pool(rng, fmt, num_pages, offset=None):
    """uint8 pool of quantized random tokens; offset [num_pages, 576] is added to every token of a page."""
    d = np_desc(fmt)
    pool = layout.new_pool(d, num_pages)
    mag = np.exp(rng.normal(0, 0.5, 576))
    for p in range(num_pages):
        x = rng.standard_normal((1, 64, 576)) * mag
        if offset is not None:
            x = x + offset[p]
        x = to_bf16_f32(x)
        layout.append(d, pool, np.array([[p]]), [0], x[..., :512], x[..., 512:])
    return pool


def page_values(fmt, pool, page) -> np.ndarray:
    """float64 [64, 576] of one page."""
    return np.concatenate(layout.gather_tokens(np_desc(fmt), pool, [page], 64), 1)


def digests(fmt, pool, pages) -> np.ndarray:
    return np.stack([page_values(fmt, pool, p).mean(0) for p in pages])


def page_scores(table_row, dig, q_c, q_r, scale, L):
    """(float64 score [P], largest sum of |products| of a logit) for one query of H heads."""
    P = (L - 1) // 64 if L > 0 else 0
    if P == 0:
        return np.zeros(0), 0.0
    d = dig[table_row[:P]].astype(np.float64)
    q = np.concatenate([q_c, q_r], -1).astype(np.float64)
    s = scale * (q @ d.T)
    w = np.exp(s - s.max(1, keepdims=True))
    return (w / w.sum(1, keepdims=True)).sum(0), float((np.abs(q) @ np.abs(d).T).max() * abs(scale))


def select(scores, L, k, n_sink, n_recent):
    """Indexes of the pages a query of L keys attends, ascending, and their keys."""
    if L <= 0:
        return [], 0
    n = (L - 1) // 64 + 1
    if n <= k:
        return list(range(n)), L
    must = [p for p in range(n) if p < n_sink or p >= n - n_recent]
    key = np.where(np.isnan(scores), -np.inf, scores)
    rest = [p for p in range(n) if p not in set(must)]
    # NaN below every number, -inf included; equal scores: the lower page first
    rest.sort(key=lambda p: (bool(np.isnan(scores[p])), -key[p], p))
    pages = sorted(must + rest[:k - len(must)])
    return pages, (len(pages) - 1) * 64 + (L - 1) % 64 + 1
