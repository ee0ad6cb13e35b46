"""GPU test: where kernel and schedule are those of the causal decode, the tree decode of a chain gives its bits."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import mla_decode_attention_etap_b200 as m
from mla_decode_attention_etap_b200 import workloads as W
from tests.parity import run_cuda
from tests.test_tree_gpu import run_tree

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("heads,q_len", [(16, 2), (16, 4), (5, 7), (20, 3), (1, 33)])
def test_chain_on_one_range(heads, q_len, paged):
    """bf16, 17 to 64 columns, all of the batch in one range: the two schedules' costs of a sequence's end play no part."""
    lens = [q_len, 40 + q_len, 3000, 128, 255, 257, 9000]
    plans = [m.mla_decode_plan_host(lens, q_len, heads, 2, schedule) for schedule in (1, 2)]
    np.testing.assert_array_equal(plans[0][0], plans[1][0])
    np.testing.assert_array_equal(plans[0][1], plans[1][1])
    w = W.make_workload(len(lens), heads, lens, q_len=q_len, causal=True, paged=paged, seed=17, spike_frac=0.05)
    o, lse, st, _ = run_tree(w, [[(2 << t) - 1 for t in range(q_len)]] * len(lens), n_sms=2)
    o2, lse2, st2, _ = run_cuda(w, n_sms=2)
    assert st == st2 == 0
    np.testing.assert_array_equal(o.float().cpu().numpy(), o2)
    np.testing.assert_array_equal(lse.cpu().numpy(), lse2)
