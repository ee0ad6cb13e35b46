"""A decode on a workspace whose plan is for another shape, or that holds no plan: refused by the decoder on the
host, and by the kernels, the combine included, through the status word."""

from __future__ import annotations

import time

import pytest
import torch

import mla_decode_attention_etap_b200 as m

BF16, I32 = torch.bfloat16, torch.int32


@pytest.mark.parametrize("shape", [(2, 4, 16), (2, 8, 8), (3, 8, 16), (1, 8, 16)])
@pytest.mark.parametrize("fp8", [False, True])
def test_decoder_refuses_another_shape(shape, fp8):
    dec = m.MlaDecoder(4, 8, 16, device="cpu", n_sms=148)
    dec._planned = 2  # as after a plan of two sequences
    q = torch.zeros(*shape, 576, dtype=BF16)
    with pytest.raises(ValueError, match="planned for 2 of 8 and 16"):
        if fp8:
            dec.fwd_tree_fp8(q, None, None, None, None)
        else:
            dec.fwd_tree(q, None, None, None)


def test_decoder_takes_the_planned_shape():
    dec = m.MlaDecoder(4, 8, 16, device="cpu", n_sms=148)
    for planned, batch in ((None, 3), (2, 2)):
        dec._planned = planned
        assert dec._tree_shape(torch.zeros(batch, 8, 16, 576, dtype=BF16)) == (batch, 8, 16)


def _refused(dec, B, q_len, h, n_sms, fp8, call):
    """Runs `call` on poisoned outputs: status MLA_ERR_INVALID_ARG at once, outputs as they were."""
    o = torch.full((B, q_len, h, 512), 7.0, dtype=BF16, device="cuda")
    lse = torch.full((B, q_len, h), 7.0, device="cuda")
    torch.cuda.synchronize()
    t0 = time.monotonic()
    call(o, lse)
    torch.cuda.synchronize()
    assert time.monotonic() - t0 < 1.0  # no bounded wait ran out
    assert dec.status() == -1
    assert (o == 7).all() and (lse == 7).all()


def _inputs(B, q_len, h, fp8):
    q = torch.randn(B, q_len, h, 576, device="cuda").to(BF16)
    kv = torch.randn(B, 4096, 576, device="cuda").to(BF16)
    scale = torch.ones(B, 4096, device="cuda") if fp8 else None
    if fp8:
        kv = torch.zeros(B, 4096, 576, dtype=torch.uint8, device="cuda")
    lens = torch.full((B,), 4000, dtype=I32, device="cuda")
    mask = torch.full((B, q_len, 1), -1, dtype=I32, device="cuda")
    return q, kv, scale, lens, mask


def _tree(q, kv, scale, lens, mask, o, lse, ws, n_sms):
    if scale is None:
        m.mla_decode_fwd_tree(q, kv, lens, None, 0.04, mask, o, lse, ws, n_sms)
    else:
        m.mla_decode_fwd_tree_fp8(q, kv, scale, lens, None, 0.04, mask, o, lse, ws, n_sms)


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("planned,used", [((2, 8, 16), (2, 4, 16)), ((2, 16, 16), (2, 8, 16)), ((4, 4, 16), (2, 4, 16))])
def test_tree_on_a_plan_of_another_shape(planned, used, fp8):
    n_sms = m.num_sms()
    dec = m.MlaDecoder(*planned, device="cuda")
    dec.workspace.fill_(0x3f)  # words that no table may be taken from
    B, q_len, h = used
    q, kv, scale, lens, mask = _inputs(B, q_len, h, fp8)
    dec.plan(torch.full((planned[0],), 4000, dtype=I32, device="cuda"))
    _refused(dec, B, q_len, h, n_sms, fp8,
             lambda o, lse: _tree(q, kv, scale, lens, mask, o, lse, dec.workspace, n_sms))


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
def test_tree_on_a_plan_without_tree_tables(fp8):
    """A plan given a workspace too small for the tree tables plans the other decodes only."""
    n_sms = m.num_sms()
    dec = m.MlaDecoder(2, 4, 16, device="cuda")
    dec.workspace.fill_(0x3f)
    q, kv, scale, lens, mask = _inputs(2, 4, 16, fp8)
    m.mla_decode_plan(lens, 4, 16, dec.workspace[:-256], n_sms)
    _refused(dec, 2, 4, 16, n_sms, fp8,
             lambda o, lse: _tree(q, kv, scale, lens, mask, o, lse, dec.workspace, n_sms))


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
def test_tree_on_a_plan_for_other_sms(fp8):
    dec = m.MlaDecoder(2, 4, 16, device="cuda", n_sms=148)
    dec.workspace.fill_(0x3f)
    q, kv, scale, lens, mask = _inputs(2, 4, 16, fp8)
    m.mla_decode_plan(lens, 4, 16, dec.workspace, 64)
    _refused(dec, 2, 4, 16, 148, fp8, lambda o, lse: _tree(q, kv, scale, lens, mask, o, lse, dec.workspace, 148))


@pytest.mark.gpu
@pytest.mark.parametrize("used", [0, 1, 2, 5])
def test_combine_without_a_plan(used):
    dec = m.MlaDecoder(2, 4, 16, device="cuda")
    dec.workspace.fill_(0x3f)
    dec.workspace.view(I32)[:64] = 0
    dec.workspace.view(I32)[4] = used  # the schedule that a decode would have recorded
    _refused(dec, 2, 4, 16, dec.n_sms, False,
             lambda o, lse: m.mla_combine(dec.workspace, 2, 4, 16, dec.n_sms, o, lse))
