"""GPU parity of the bf16 tree decode in groups of 128 columns (one rounded P term for long sequences) where a few
rows carry the softmax: their rounding must not stay in O (the parity bar of tests/parity.py)."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import mla_decode_attention_etap_b200 as m
from mla_decode_attention_etap_b200 import workloads as W
from tests import uneven_softmax as U
from tests import verify_reference as ref
from tests.parity import assert_parity
from tests.test_tree_gpu import tree_masks

pytestmark = pytest.mark.gpu


def _check(q, kv, lens, n_sms, what, softmax_scale=U.SCALE):
    B, q_len, h, _ = q.shape
    q, kv = q.cuda(), kv.cuda()
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    masks = tree_masks(np.random.default_rng(q_len), B, q_len)
    words = torch.from_numpy(ref.mask_words(masks, q_len).copy()).cuda()
    sees = torch.tensor([[[bool(v >> u & 1) for u in range(q_len)] for v in row] for row in masks], device="cuda")
    dec = m.MlaDecoder(B, q_len, h, device="cuda", n_sms=n_sms)
    dec.plan(sl)
    o, lse = dec.fwd_tree(q, kv, sl, words, softmax_scale=softmax_scale)
    assert dec.status() == 0
    o_ref, lse_ref = U.attention(q, kv, None, lens, sees, softmax_scale)
    return assert_parity(o.float().cpu().numpy(), lse.cpu().numpy(), o_ref.cpu().numpy(), lse_ref.cpu().numpy(),
                         what=what)


@pytest.mark.parametrize("columns", [(9, 8), (16, 16), (4, 128)])
@pytest.mark.parametrize("seed", range(4))
@pytest.mark.parametrize("L", [8192, 20000, 32768])
def test_spiky_rows_in_long_ranges(L, seed, columns):
    """5 % of the rows scaled by 8, the whole sequence in one range of a work unit and spread over all."""
    w = W.make_workload(1, columns[1], [L], q_len=columns[0], seed=200 + seed, spike_frac=0.05)
    for n_sms in (2, 12, 148):
        _check(w.q, w.kv, [L], n_sms, f"spikes L={L} n_sms={n_sms}", w.softmax_scale)


@pytest.mark.parametrize("columns", [(9, 8), (16, 16), (4, 128)])
@pytest.mark.parametrize("kind,gap", [("even", 0), ("first", 10.7), ("first", 14.6), ("first_equal", 12.3),
                                      ("first_equal", 13.9), ("every128", 7), ("last", 13), ("heavy_start", 12),
                                      ("falling", 20), ("rising", 20), ("spikes", 9)])
def test_heavy_rows(kind, gap, columns):
    lens = [8192, 16001]
    q, kv, _ = U.make(kind, lens, gap, columns, seed=int(10 * gap) + 3, fp8=False)
    for n_sms in (2, 148):
        _check(q, kv, lens, n_sms, f"{kind} gap={gap} n_sms={n_sms}")


@pytest.mark.parametrize("columns", [(9, 8), (16, 16)])
def test_long_and_short_sequences_in_one_batch(columns):
    """Short sequences' P is multiplied as two terms, long ones' as one: each divides by its own sum."""
    lens = [9000, 300, 8192, 8191, 64, 12000]
    for kind, gap in (("even", 0), ("first", 8.4), ("spikes", 6)):
        q, kv, _ = U.make(kind, lens, gap, columns, seed=int(10 * gap) + 5, fp8=False)
        for n_sms in (2, 8, 148):
            _check(q, kv, lens, n_sms, f"{kind} gap={gap} n_sms={n_sms}")
