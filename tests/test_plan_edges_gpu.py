"""GPU tests of the plan at the edges of its arithmetic: the longest lengths."""

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


@pytest.mark.parametrize("batch", [1, 31, 32])
@pytest.mark.parametrize("heads,q_len", [(16, 4), (128, 4)])
def test_plan_of_the_longest_lengths(batch, heads, q_len):
    lens = np.full(batch, np.iinfo(np.int32).max, np.int32)
    lens[1::3] = 0
    lens[2::3] -= 300
    ranges, _ = _tree_tables(lens, heads, q_len)
    assert ranges[-1, 1] == ((lens.astype(np.int64) + 255) // 256).sum()
