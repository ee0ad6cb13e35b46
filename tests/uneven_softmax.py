"""Inputs whose softmax is carried by few rows while many others hold the rest of it, and the 64-bit attention of a
cache: scores are set through one rope column (the values do not see it), on top of random ones."""

from __future__ import annotations

import math

import torch

from mla_decode_attention_etap_b200.workloads import quantize_e4m3_rows

SCALE = 1.0 / 24.0
Q_ROPE = 8.0  # the queries' entry in rope column 512, times 1 .. 1.125 by column


def octaves(kind: str, L: int, gap: float, g: torch.Generator) -> torch.Tensor:
    """What is added to the score of each of L rows, in octaves (factors of 2)."""
    x = torch.zeros(L, dtype=torch.float64)
    if kind in ("first", "first_equal"):
        x[0] = gap                        # an attention sink
    elif kind == "every128":
        x[torch.arange(L // 128 + (L % 128 > 5)) * 128 + 5] = gap
    elif kind == "last":
        x[L - 1] = gap
    elif kind == "heavy_start":
        x[:L // 16] = gap                 # many heavy rows, then as many light ones as matter
    elif kind == "falling":
        x = torch.linspace(gap, 0, L, dtype=torch.float64)
    elif kind == "rising":
        x = torch.linspace(0, gap, L, dtype=torch.float64)
    elif kind == "spikes":
        x[torch.rand(L, generator=g) < 0.05] = gap
    else:
        assert kind == "even", kind
    return x


def make(kind, lens, gap, columns, seed, mean=0.5, fp8=True, page_scale=1.0):
    """q bf16 [B, *columns, 576], cache [B, L_max, 576] (bf16, or E4M3 codes and row scales); columns (q_len, heads)."""
    g = torch.Generator().manual_seed(seed)
    B, L_max = len(lens), max(lens)
    q = torch.randn(B, *columns, 576, generator=g)
    k = torch.randn(B, L_max, 576, generator=g)
    k[..., :512] += mean
    if kind.endswith("equal"):
        q[..., :512] = 0.0
    q[..., 512:] = 0.0
    q[..., 512] = Q_ROPE * (1 + torch.rand(B, *columns, generator=g) / 8)
    k[..., 512:] = 0.0
    for b, L in enumerate(lens):
        k[b, :L, 512] = (octaves(kind, L, gap, g) * math.log(2) / (SCALE * Q_ROPE)).float()
    q, k = q.bfloat16(), k.bfloat16()
    if not fp8:
        return q, k, None
    kv8, scale = quantize_e4m3_rows(k)
    return q, kv8, scale * page_scale


def attention(q, kv, scale, lens, sees=None, softmax_scale=SCALE):
    """64-bit O [B, q_len, h, 512] and LSE; sees: bool [B, q_len, n] of the last n rows (None: every row)."""
    B, q_len, h, _ = q.shape
    o = torch.zeros(B, q_len, h, 512, dtype=torch.float64, device=q.device)
    lse = torch.full((B, q_len, h), -math.inf, dtype=torch.float64, device=q.device)
    for b, L in enumerate(int(v) for v in lens):
        k = kv[b, :L].view(torch.float8_e4m3fn).double() * scale[b, :L, None].double() if scale is not None \
            else kv[b, :L].double()
        x = (q[b].double().flatten(0, 1) @ k.T * softmax_scale).view(q_len, h, L)
        if sees is not None:
            hide = torch.zeros(q_len, L, dtype=torch.bool, device=q.device)
            hide[:, L - sees.shape[2]:] = ~sees[b]
            x = x.masked_fill(hide[:, None], -math.inf)
        lse[b] = torch.logsumexp(x, -1)
        o[b] = (torch.softmax(x, -1).flatten(0, 1) @ k[:, :512]).view(q_len, h, 512)
    return o, lse
