"""GPU parity of the E4M3 cache's decodes where a few rows carry much of the softmax and the many others the rest:
their probabilities lie far below the column's largest and must not be rounded away (the parity bar of
tests/parity.py, which both decodes meet on even rows)."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import mla_decode_attention_etap_b200 as m
from tests import uneven_softmax as U
from tests import verify_reference as ref
from tests.parity import MAXABS_REL, LSE_ABS, RMSE_REL, assert_parity, parity_metrics
from tests.test_tree_gpu import tree_masks

pytestmark = pytest.mark.gpu


def _check(q, kv8, scale, lens, tree, n_sms, what, softmax_scale=U.SCALE, few_values=False):
    B, q_len, h, _ = q.shape
    q, kv8, scale = q.cuda(), kv8.cuda(), scale.cuda()
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    dec = m.MlaDecoder(B, q_len, h, device="cuda", n_sms=n_sms)
    dec.plan(sl)
    sees = None
    if tree:
        masks = tree_masks(np.random.default_rng(q_len), B, q_len)
        words = torch.from_numpy(ref.mask_words(masks, q_len).copy()).cuda()
        sees = torch.tensor([[[bool(v >> u & 1) for u in range(q_len)] for v in row] for row in masks], device="cuda")
        o, lse = dec.fwd_tree_fp8(q, kv8, scale, sl, words, softmax_scale=softmax_scale)
    else:
        o, lse = dec.fwd_fp8(q, kv8, scale, sl, softmax_scale=softmax_scale)
    assert dec.status() == 0
    o_ref, lse_ref = U.attention(q, kv8, scale, lens, sees, softmax_scale)
    got = o.float().cpu().numpy(), lse.cpu().numpy(), o_ref.cpu().numpy(), lse_ref.cpu().numpy()
    if not few_values:
        return assert_parity(*got, what=what)
    # The bar leaves 0.35e-3 above the 1.65e-3 that the rounding of many numbers to bf16 costs on average.  Where O
    # is a single cache row in every column, 512 numbers a sequence, that rounding's error is not the average: it may
    # be anything up to 2^-8 / sqrt(3) = 2.26e-3 (half a step, uniform within it, is 2^-8 of a number just above
    # a power of 2).  It is taken from the reference itself, and the kernel gets the 0.35e-3 over it.
    r = parity_metrics(*got)
    rounding = ((o_ref.float().bfloat16().double() - o_ref).pow(2).mean() / o_ref.pow(2).mean()).sqrt().item()
    assert rounding <= 2.0 ** -8 / 3 ** 0.5
    assert r["nan_o"] == 0 and r["inf_lse_mismatch"] == 0 and r["lse_err"] <= LSE_ABS, f"{what}: {r}"
    assert r["rmse_rel"] <= max(RMSE_REL, rounding + 0.35e-3) and r["maxabs"] <= MAXABS_REL * r["max_ref"], f"{what}: {r}"


# columns of one CTA (16, 32), of one group (64) and of several (72, 256): the pair kernel's and the tree kernel's
COLUMNS = [(1, 16), (4, 4), (2, 16), (4, 16), (9, 8), (16, 16)]


@pytest.mark.parametrize("tree", [True, False])
@pytest.mark.parametrize("columns", COLUMNS)
@pytest.mark.parametrize("L,gap", [(300, 8), (4096, 8), (4096, 12.3), (32768, 10.7), (32768, 13.6), (32768, 15.2)])
@pytest.mark.parametrize("kind", ["first", "first_equal"])
def test_a_first_row_with_much_of_the_softmax(kind, L, gap, columns, tree):
    q, kv8, scale = U.make(kind, [L], gap, columns, seed=int(10 * gap) + L)
    _check(q, kv8, scale, [L], tree, n_sms=2, what=f"{kind} L={L} gap={gap}")  # one range


@pytest.mark.parametrize("tree", [True, False])
@pytest.mark.parametrize("columns", [(1, 16), (2, 16), (4, 16), (16, 16)])
@pytest.mark.parametrize("kind,gap", [("even", 0), ("every128", 5), ("every128", 9.4), ("last", 13), ("heavy_start", 7),
                                      ("heavy_start", 12), ("falling", 20), ("rising", 20), ("spikes", 9)])
def test_heavy_rows_elsewhere(kind, gap, columns, tree):
    lens = [8192, 1025, 130]
    q, kv8, scale = U.make(kind, lens, gap, columns, seed=int(10 * gap) + 7)
    for n_sms in (2, 148):
        _check(q, kv8, scale, lens, tree, n_sms, what=f"{kind} gap={gap} n_sms={n_sms}")


@pytest.mark.parametrize("tree", [True, False])
@pytest.mark.parametrize("columns", [(1, 16), (2, 16), (4, 16), (16, 16)])
@pytest.mark.parametrize("gap", [25, 40, 70, 100])
def test_a_row_with_all_of_the_softmax(gap, columns, tree):
    lens = [3000, 257]
    for kind in ("first", "last", "falling"):
        q, kv8, scale = U.make(kind, lens, gap, columns, seed=gap)
        _check(q, kv8, scale, lens, tree, 2, what=f"{kind} gap={gap}", few_values=kind != "falling")


@pytest.mark.parametrize("tree", [True, False])
@pytest.mark.parametrize("columns", [(1, 16), (2, 16), (4, 16), (16, 16)])
@pytest.mark.parametrize("log2_scale", [-85, -40, 20])
def test_far_row_scales(log2_scale, columns, tree):
    """All row scales times a power of two, and the softmax scale divided by it: the same softmax, an O as much
    smaller or larger, with log2 of the row scales far from 0."""
    lens = [4096, 200]
    q, kv8, scale = U.make("first", lens, 11.0, columns, seed=31, page_scale=2.0 ** log2_scale)
    _check(q, kv8, scale, lens, tree, 2, what=f"scales 2^{log2_scale}", softmax_scale=U.SCALE * 2.0 ** -log2_scale)


@pytest.mark.parametrize("tree", [True, False])
@pytest.mark.parametrize("columns", [(1, 16), (2, 16), (4, 16), (16, 16)])
def test_rows_of_scale_zero_between_others(columns, tree):
    """A scale of 0 stands for a row of zeros, whatever its codes: score 0, no value."""
    lens = [2500, 190]
    q, kv8, scale = U.make("first", lens, 10.0, columns, seed=33)
    scale[:, 3::5] = 0.0
    scale[:, 128:256] = 0.0  # a whole tile
    _check(q, kv8, scale, lens, tree, 2, what="zero scales")
