"""Plain 64-bit references of the verify step's operators (numpy and Python integers, no shared code
with the CUDA path): extend, append, tree attention, accept."""

from __future__ import annotations

import math

import numpy as np

PAGE, D_QK, D_V = 64, 576, 512


def pages(n: int) -> int:
    return (n + PAGE - 1) // PAGE


def extend(seqlens, new_lens, table, stack, nfree, parents, q_len):
    """-> (table, slots, positions, masks [B][q_len] as Python integers, lengths, nfree)."""
    table = [list(r) for r in table]
    slots, positions, masks, lens = [], [], [], []
    for b, (L, n) in enumerate(zip(seqlens, new_lens)):
        for p in range(pages(L), pages(L + n)):
            nfree -= 1
            table[b][p] = stack[nfree]
        s, q, m = [], [], []
        for t in range(q_len):
            up, seen = t, 0
            while t < n and up >= 0:
                seen |= 1 << up
                up = parents[b][up] if parents is not None else -1
            depth = t if parents is None else bin(seen).count("1") - 1
            s.append(table[b][(L + t) // PAGE] * PAGE + (L + t) % PAGE if t < n else -1)
            q.append(L + depth if t < n else -1)
            m.append(seen)
        slots.append(s)
        positions.append(q)
        masks.append(m)
        lens.append(L + n)
    return table, slots, positions, masks, lens, nfree


def mask_words(masks, q_len):
    """Python integers [B][q_len] -> int32 [B, q_len, ceil(q_len / 32)]."""
    words = (q_len + 31) // 32
    out = np.zeros((len(masks), q_len, words), np.uint32)
    for b, row in enumerate(masks):
        for t, v in enumerate(row):
            for w in range(words):
                out[b, t, w] = (v >> (32 * w)) & 0xFFFFFFFF
    return out.view(np.int32)


def rotate(x, angles, interleaved):
    """x [..., 64], angles [..., 64] as 32 cosines and 32 sines."""
    c, s = angles[..., :32], angles[..., 32:]
    y = np.empty_like(x)
    a, b = (slice(0, None, 2), slice(1, None, 2)) if interleaved else (slice(0, 32), slice(32, 64))
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def append_rows(latent, weight, eps, table, positions, interleaved):
    """fp64 cache rows of all tokens (rows of padding tokens are meaningless)."""
    x = np.asarray(latent, np.float64)
    lat = x[:, :D_V]
    if weight is not None:
        lat = lat / np.sqrt((lat ** 2).mean(1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    ang = np.asarray(table, np.float64)[np.clip(positions, 0, len(table) - 1)]
    return np.concatenate([lat, rotate(x[:, D_V:], ang, interleaved)], 1)


def e4m3_values():
    """The 256 values of the E4M3 codes, from the format's definition."""
    v = np.empty(256)
    for c in range(256):
        s, e, m = c >> 7, (c >> 3) & 15, c & 7
        x = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v[c] = math.nan if e == 15 and m == 7 else (-x if s else x)
    return v


def tree_attention(q, rows, masks, q_lens, scale):
    """q [B, q_len, h, 576], rows: list of [L_b, 576] fp64 -> (O [B, q_len, h, 512], LSE [B, q_len, h])."""
    B, q_len, h, _ = q.shape
    o = np.zeros((B, q_len, h, D_V))
    lse = np.full((B, q_len, h), -math.inf)
    for b in range(B):
        k, n = np.asarray(rows[b], np.float64), int(q_lens[b])
        L = len(k)
        for t in range(n):
            first = L - n
            see = [j for j in range(max(first, 0), L) if masks[b][t] >> (j - first) & 1]
            kk = np.concatenate([k[:max(first, 0)], k[see]])
            if not len(kk):
                continue
            x = scale * (np.asarray(q[b, t], np.float64) @ kk.T)
            top = x.max(1, keepdims=True)
            p = np.exp(x - top)
            total = p.sum(1, keepdims=True)
            o[b, t] = (p / total) @ kk[:, :D_V]
            lse[b, t] = (top + np.log(total))[:, 0]
    return o, lse


def accept(seqlens, new_lens, path, path_lens, table, stack, nfree):
    """-> (moves as (source row, target row) of the pool, lengths, stack, nfree)."""
    moves, lens, stack = [], [], list(stack)
    for b, (L, n, keep) in enumerate(zip(seqlens, new_lens, path_lens)):
        end = 0 if keep < 0 else L - n + keep
        for i in range(max(keep, 0)):
            src, dst = L - n + path[b][i], L - n + i
            moves.append(tuple(table[b][r // PAGE] * PAGE + r % PAGE for r in (src, dst)))
        for p in range(pages(end), pages(L)):
            stack[nfree] = table[b][p]
            nfree += 1
        lens.append(end)
    return moves, lens, stack, nfree


def random_parents(rng, B, q_len, shape="tree"):
    """parents [B][q_len]: 'tree' any earlier token or the context, 'chain', 'star' (all follow the context)."""
    if shape == "chain":
        return [[t - 1 for t in range(q_len)] for _ in range(B)]
    if shape == "star":
        return [[-1] * q_len for _ in range(B)]
    return [[int(rng.integers(-1, t)) if t else -1 for t in range(q_len)] for _ in range(B)]


def paged_setup(rng, lens, max_blocks, num_blocks):
    """A table whose pages come from a permutation of the pool, and the stack of the rest."""
    perm = [int(x) for x in rng.permutation(num_blocks)]
    table, at = [], 0
    for L in lens:
        table.append(perm[at:at + pages(L)] + [-1] * (max_blocks - pages(L)))
        at += pages(L)
    left = perm[at:]
    return table, left + [-1] * (num_blocks - len(left)), len(left)
