"""GPU tests of the plan at the edges of its arithmetic: batches without a row, and the longest lengths."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import mla_decode_attention_etap_b200 as m
from tests.test_parity_gpu import _sched_offsets

pytestmark = pytest.mark.gpu


def _tree_tables(lens, heads, q_len):
    """Device tree schedule of these lengths, compared with the host's."""
    batch = len(lens)
    dec = m.MlaDecoder(batch, q_len, heads, device="cuda")
    dec.workspace.fill_(0x3f)
    dec.plan(torch.from_numpy(lens).cuda())
    torch.cuda.synchronize()
    ws = dec.workspace.view(torch.int32).cpu().numpy()
    ncols, sms = heads * q_len, dec.n_sms
    g64, c_max = (ncols + 63) // 64, max(1, sms // 2 // ((ncols + 127) // 128))
    _, size = _sched_offsets(0, batch, c_max, g64)
    tab, _ = _sched_offsets(dec.workspace.numel() - size, batch, c_max, g64)
    ranges, info, nct, ngr, rows, gcols = m.mla_decode_plan_host(lens, q_len, heads, sms, schedule=2)
    assert ws[0] == 0 and ws[24] == nct and ws[25] == ngr and ws[28] == gcols
    np.testing.assert_array_equal(ws[tab["ranges"] // 4:][:2 * nct].reshape(-1, 2), ranges)
    np.testing.assert_array_equal(ws[tab["info"] // 4:][:4 * batch].reshape(-1, 4), info)
    first = np.concatenate([[0], np.cumsum((lens.astype(np.int64) + rows - 1) // rows)])
    np.testing.assert_array_equal(ws[tab["tile"] // 4:][:batch + 1], first)
    return ranges, info


@pytest.mark.parametrize("batch", [1, 5, 32, 33])
@pytest.mark.parametrize("heads,q_len", [(16, 4), (16, 8), (128, 4)])
def test_plan_of_a_batch_without_rows(batch, heads, q_len):
    ranges, info = _tree_tables(np.zeros(batch, np.int32), heads, q_len)
    assert (ranges == 0).all() and (info[:, 0] == 0).all() and (info[:, 2] == 0).all()


@pytest.mark.parametrize("batch", [1, 31, 32])
@pytest.mark.parametrize("heads,q_len", [(16, 4), (128, 4)])
def test_plan_of_the_longest_lengths(batch, heads, q_len):
    lens = np.full(batch, np.iinfo(np.int32).max, np.int32)
    lens[1::3] = 0
    lens[2::3] -= 300
    ranges, _ = _tree_tables(lens, heads, q_len)
    assert ranges[-1, 1] == ((lens.astype(np.int64) + 255) // 256).sum()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("heads", [4, 16, 32])
def test_tree_decode_of_a_batch_without_rows(heads, fp8):
    B, q_len = 5, 4
    dec = m.MlaDecoder(B, q_len, heads, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    q = torch.randn(B, q_len, heads, 576, device="cuda").bfloat16()
    kv = torch.zeros(B, 64, 576, dtype=torch.uint8 if fp8 else torch.bfloat16, device="cuda")
    mask = torch.ones(B, q_len, 1, dtype=torch.int32, device="cuda")
    o = torch.full((B, q_len, heads, 512), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, q_len, heads), float("nan"), device="cuda")
    dec.plan(lens)
    if fp8:
        dec.fwd_tree_fp8(q, kv, torch.ones(B, 64, device="cuda"), lens, mask, o=o, lse=lse, q_lens=lens)
    else:
        dec.fwd_tree(q, kv, lens, mask, o=o, lse=lse, q_lens=lens)
    assert dec.status() == 0
    assert (o == 0).all() and torch.isneginf(lse).all()
