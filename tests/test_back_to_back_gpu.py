"""GPU tests of decodes enqueued one behind the other on one workspace, each with its own plan and nothing
between them: a plan must not touch the tables, counters or status word of a decode that still runs."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import mla_decode_attention_etap_b200 as m
from mla_decode_attention_etap_b200 import workloads as W
from tests import verify_reference as ref
from tests.test_tree_gpu import tree_masks

pytestmark = pytest.mark.gpu


def _lengths(rng, batch, longs):
    """Mostly sequences of one unit (never split), and a few long ones (split) at places drawn anew."""
    lens = rng.integers(16, 257, batch)
    lens[rng.choice(batch, longs, replace=False)] = rng.integers(6000, 12001, longs)
    return lens


@pytest.mark.parametrize("kind", ["tree", "tree_fp8", "causal"])
@pytest.mark.parametrize("heads,q_len", [(16, 4), (16, 16)])
def test_plans_and_decodes_in_a_row(kind, heads, q_len):
    rng = np.random.default_rng(61 + heads * q_len)
    batch, steps, dev = 24, 6, torch.device("cuda")
    fp8 = kind == "tree_fp8"
    w = W.make_workload(batch, heads, [12000] * batch, q_len=q_len, seed=62, paged=False,
                        kv_dtype="e4m3" if fp8 else "bf16")
    q, kv = w.q.to(dev), (w.kv8 if fp8 else w.kv).to(dev)
    scale = w.kv_scale.to(dev) if fp8 else None
    masks = tree_masks(rng, batch, q_len)
    mask = torch.from_numpy(ref.mask_words(masks, q_len).copy()).to(dev)
    lens = [torch.from_numpy(_lengths(rng, batch, 4 if i % 2 else 1)).int().to(dev) for i in range(steps)]

    def step(dec, i, o, lse):
        dec.plan(lens[i])
        if kind == "causal":
            dec.fwd(q, kv, lens[i], None, w.softmax_scale, True, o=o, lse=lse)
        elif fp8:
            dec.fwd_tree_fp8(q, kv, scale, lens[i], mask, None, w.softmax_scale, o=o, lse=lse)
        else:
            dec.fwd_tree(q, kv, lens[i], mask, None, w.softmax_scale, o=o, lse=lse)

    def outputs(n):
        return (torch.full((n, batch, q_len, heads, 512), float("nan"), dtype=torch.bfloat16, device=dev),
                torch.full((n, batch, q_len, heads), float("nan"), device=dev))

    want_o, want_l = outputs(steps)
    for i in range(steps):  # one at a time, each on a workspace of its own
        dec = m.MlaDecoder(batch, q_len, heads, device=dev)
        step(dec, i, want_o[i], want_l[i])
        torch.cuda.synchronize()
        assert dec.status() == 0
    rounds = 5
    o, lse = outputs(rounds * steps)
    dec = m.MlaDecoder(batch, q_len, heads, device=dev)
    torch.cuda.synchronize()
    for r in range(rounds):
        for i in range(steps):
            step(dec, i, o[r * steps + i], lse[r * steps + i])
    torch.cuda.synchronize()
    assert dec.status() == 0
    for r in range(rounds):
        assert torch.equal(o[r * steps:(r + 1) * steps], want_o), (kind, r)
        assert torch.equal(lse[r * steps:(r + 1) * steps], want_l), (kind, r)
