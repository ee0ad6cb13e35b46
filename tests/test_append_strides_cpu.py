"""Strides of an append's inputs: a dimension of one entry has any stride, the others' are passed on as they are."""

from __future__ import annotations

import pytest
import torch

import mla_decode_attention_etap_b200 as m

BF16, I32 = torch.bfloat16, torch.int32


def _arguments(latent, q_rope):
    T, h = latent.shape[0], q_rope.shape[1]
    return m.check_append_args(latent, None, torch.zeros(4, 64), torch.zeros(T, dtype=I32), torch.zeros(T, dtype=I32),
                               torch.zeros(1, 64, 576, dtype=BF16), torch.zeros(64, dtype=I32), q_rope,
                               torch.zeros(T, h, 576, dtype=BF16))


@pytest.mark.parametrize("T,h,strides,want", [
    (1, 1, (3, 5, 1), (0, 0)),
    (1, 2, (3, 72, 1), (0, 72)),
    (2, 1, (80, 5, 1), (80, 0)),
    (2, 2, (400, 192, 1), (400, 192)),
    (2, 2, (0, 64, 1), (0, 64)),  # one token's columns for both
])
def test_query_strides(T, h, strides, want):
    room = torch.zeros(4096, dtype=BF16)
    ahead, table, where, cache, behind = _arguments(torch.zeros(T, 576, dtype=BF16), room.as_strided((T, h, 64), strides))
    assert tuple(behind[1:4]) == (*want, h)


@pytest.mark.parametrize("T,stride,want", [(1, 7, 576), (2, 1000, 1000)])
def test_latent_stride(T, stride, want):
    latent = torch.zeros(4096, dtype=BF16).as_strided((T, 576), (stride, 1))
    ahead, *_ = _arguments(latent, torch.zeros(T, 1, 64, dtype=BF16))
    assert ahead[1] == want
