"""GPU tests of an append's edges: the E4M3 codes it stores are those of the fp32 quotient row / scale, rounded to
nearest even (as the framework's own quantiser of workloads has them), and every bad position is reported."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import mla_decode_attention_etap_b200 as m
from tests import verify_reference as ref

pytestmark = pytest.mark.gpu


def _nearest_even(y):
    """The E4M3 value nearest to y (64 bits, |y| <= 448): steps of 2^(e - 3) in [2^e, 2^(e+1)), 2^-9 at least."""
    step = np.exp2(np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -6))) - 3)
    return np.rint(y / step) * step


@pytest.mark.parametrize("exponent", [-40, 0, 30])
def test_codes_at_every_border(exponent):
    """Rows with every bf16 mantissa as their largest value, and every mantissa over twelve octaves below it: among
    these quotients many lie on the border of two codes exactly, and many next to one."""
    values = np.concatenate([np.arange(128, 256) * 2.0 ** -e for e in range(12)])  # 1536 of them
    rows = []
    for top in range(128, 256):
        v = np.where(values <= top, values, -values / 2)
        for part in range(0, len(v), 575):
            rows.append(np.concatenate([[top], v[part:part + 575], np.zeros(max(0, part + 575 - len(v)))]))
    x = np.stack(rows) * 2.0 ** exponent
    latent = torch.from_numpy(x).bfloat16().cuda()
    assert (latent.double().cpu().numpy() == x).all()
    T = len(x)
    kv = torch.zeros(-(-T // 64), 64, 576, dtype=torch.uint8, device="cuda")
    scale = torch.zeros(kv.shape[:2], device="cuda")
    status = torch.zeros(64, dtype=torch.int32, device="cuda")
    still = torch.cat([torch.ones(1, 32), torch.zeros(1, 32)], 1).cuda()  # no rotation
    m.mla_cache_append_fp8(latent, None, 0.0, still, False, torch.zeros(T, dtype=torch.int32, device="cuda"),
                           torch.arange(T, dtype=torch.int32, device="cuda"), kv, scale, status)
    assert int(status[0]) == 0
    s = scale.view(-1)[:T].double().cpu().numpy()
    np.testing.assert_array_equal(s, (np.abs(x).max(1).astype(np.float32) / np.float32(448)).astype(np.float64))
    got = ref.e4m3_values()[kv.view(-1, 576)[:T].cpu().numpy()]
    # The quotient is an fp32 one, rounded once: every code is that quotient's.
    q = (x.astype(np.float32) / s[:, None].astype(np.float32)).astype(np.float64)
    np.testing.assert_array_equal(got, _nearest_even(q))
    # Against the quotient without end a code may therefore differ only where that lies within half a step of
    # fp32, 2^-24 of it, of the border between two codes (a scale that is itself rounded puts it there): the middle
    # of the two codes' values.
    y = x / s[:, None]
    exact = _nearest_even(y)
    off = got != exact
    border = (got + exact) / 2
    assert (np.abs(y - border)[off] <= 2.0 ** -24 * np.abs(y)[off]).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("heads", [0, 2])
def test_a_position_past_the_table_is_reported_without_a_slot_too(heads, fp8):
    latent = torch.randn(3, 576, device="cuda").bfloat16()
    kv = torch.zeros(1, 64, 576, dtype=torch.uint8 if fp8 else torch.bfloat16, device="cuda")
    scale = torch.zeros(1, 64, device="cuda")
    table = torch.cat([torch.ones(5, 32), torch.zeros(5, 32)], 1).cuda()
    slots = torch.tensor([-1, -1, 7], dtype=torch.int32, device="cuda")
    q_rope = torch.randn(3, heads, 64, device="cuda").bfloat16() if heads else None
    for bad, want in ((4, 0), (5, -1), (2 ** 31 - 1, -1)):
        positions = torch.tensor([0, bad, 1], dtype=torch.int32, device="cuda")
        status = torch.zeros(64, dtype=torch.int32, device="cuda")
        q = torch.zeros(3, heads, 576, dtype=torch.bfloat16, device="cuda") if heads else None
        front = (latent, None, 0.0, table, True, positions, slots, kv)
        if fp8:
            m.mla_cache_append_fp8(*front, scale, status, q_rope=q_rope, q=q)
        else:
            m.mla_cache_append(*front, status, q_rope=q_rope, q=q)
        assert int(status[0]) == want
        rows = kv.view(-1, 576).float().abs().sum(1)
        assert rows[7] > 0 and rows.count_nonzero() == 1  # the good token's row and no other
        if heads:
            assert (q[1, :, 512:].abs().sum() > 0).item() == (want == 0)
