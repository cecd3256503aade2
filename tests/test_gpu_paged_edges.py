"""Paged cache: scores of any magnitude, thread blocks with several runs of
work, long waits, and first calls from several threads, against fp64 (bounds
as in paged_ref)."""
import numpy as np
import pytest
import torch

import long_context_mask_gb300 as bsa
import paged_ref as ref
from gpu_util import status_ok
from test_gpu_paged import bits, check_select, lists_for, mean_keys, run_forward, run_select

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ selection

@pytest.mark.parametrize("kind", ["equal", "steps", "close", "shuffled"])
@pytest.mark.parametrize("q_exp,m_exp", [(0, -76), (0, -80), (-80, 0), (-50, -50), (0, -100), (-90, 60), (70, 70)])
def test_close_and_equal_scores_of_any_magnitude(kind, q_exp, m_exp):
    """Powers of two change no order: the lists are those of the unscaled scores.
    shuffled: the same values in another order against a query of equal ones, so
    that the exact scores are equal and their fp32 sums are not."""
    b = ref.make([30], [128 * 400 + 7], H=4, H_kv=2, D=128, page=128, seed=54, poison=False)
    q, km = ref.rows(b, 4, 55), mean_keys(b, 56)
    at = b.table[0].long()
    if kind == "steps":
        for j in range(400):
            km[at[j]] = km[at[j % 9]]
    else:
        km[:] = km[0]
    if kind == "shuffled":
        q[:] = q[..., :1].clone()
        g = torch.Generator().manual_seed(59)
        for j in range(400):
            km[at[j]] = km[at[j]][:, torch.randperm(128, generator=g).cuda()]
    if kind == "close":
        q[..., 5] = 2.0 ** -22
        for j in range(400):
            km[at[j], :, 5] = 1.0 + (j * 37 % 101) / 128
    kw = dict(topk=16, sink_blocks=1, local_blocks=1)
    want = ref.select(b, q, km, *kw.values())
    q, km = q * 2.0 ** q_exp, km * 2.0 ** m_exp
    assert q.isfinite().all() and km.isfinite().all()
    sel, cnt = run_select(b, q, km, **kw)
    status_ok()
    for t in range(30):
        for h in range(2):
            assert sel[t, h].tolist() == want[t][h] and int(cnt[t, h]) == 18, (t, h)
