"""GPU tests of what the other tests of the sparse decode leave open: the precision that the scores'
accumulators are for, and the step's own choice of key splits where it splits."""
import pytest
import torch

import perf.operators as cases
from bit_mla_kv_qdecode_b200 import api
from tests import test_gpu_sparse as sparse

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,H,tokens,bound", [(8, 16, 32768, 7e-7), (2, 128, 131072, 1.2e-6)])
@pytest.mark.parametrize("seed", [1, 2])
def test_scores_keep_the_precision_of_their_accumulators(B, H, tokens, bound, seed):
    """Norm of the scores' error, relative, at ordinary logits (a few pages hold most of the mass). Measured
    against float64 on three seeds each: 3.4e-7 and 6.8e-7 with three accumulators a logit, 1.1e-6 and 1.8e-6
    with one, which the derived bound of the other tests (1e-3) cannot tell apart. (What one accumulator of
    36 steps truncates, 36 / 4 units of 2^-23 of the logit on average, becomes a third of it with three of 12.)"""
    case = dict(op="scores", B=B, s_q=1, H=H, t_lo=tokens, t_hi=tokens)
    st = cases.prepare(case, seed)
    got = api.mla_page_scores(st["table"], st["lens"], st["max_len"], st["digests"], st["q_c"], st["q_r"], cases.SCALE)
    want = cases.exact(case, seed)
    assert api.mla_get_device_status() == 0
    assert torch.equal(torch.isfinite(got), torch.isfinite(want))
    some = torch.isfinite(want)
    err = float((got.double() - want)[some].norm() / want[some].norm())
    assert err <= bound, err


@pytest.mark.parametrize("fmt,lens,s_q,H,k", [((4, 64, 4, 64), [64 * 20, 64 * 18 + 7, 64 * 13], 1, 128, 12),
                                              ((2, 32, 4, 64), [64 * 30 + 1, 64 * 9], 2, 40, 24),
                                              ((4, 32, 2, 64), [64 * 40], 1, 20, 33)])
def test_own_choice_of_splits(monkeypatch, fmt, lens, s_q, H, k):
    """num_splits = 0 above 16 rows, with selections long enough to be split: the result of the number of splits
    that the workspace shows it to have chosen, bit for bit, and within the decode's bound of float64."""
    need = lambda n: api.mla_qdecode_sparse_workspace_bytes(len(lens), s_q, H, max(lens), k, n)  # noqa: E731
    chosen = [n for n in range(1, 65) if need(n) == need(0)]
    assert chosen and chosen[0] > 1, chosen
    step = api.mla_qdecode_sparse
    used = []

    def own(*args, **kw):
        used.append(kw.pop("num_splits"))
        return step(*args, **kw, num_splits=0)

    monkeypatch.setattr(api, "mla_qdecode_sparse", own)
    sparse._sparse_case(fmt, lens, s_q, H, k, 1, 2, seed=k, num_splits=chosen[0])
    assert used == [chosen[0]]
