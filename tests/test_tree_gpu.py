"""GPU tests of the tree decode (mla_decode_fwd_tree, mla_decode_fwd_tree_fp8) against the 64-bit
reference, and of the whole verify step: extend, append, tree decode, accept."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import mla_decode_attention_etap_b200 as m
from mla_decode_attention_etap_b200 import workloads as W
from tests import verify_reference as ref
from tests.parity import assert_parity
from tests.test_parity_gpu import _poison_padding

pytestmark = pytest.mark.gpu


def run_tree(w, masks, n_sms=None, flags=0, q_lens="workload", mask_words=None):
    """Plan + tree decode, outputs poisoned first -> (o, lse, status, decoder)."""
    dev = torch.device("cuda")
    dec = m.MlaDecoder(w.batch, w.q_len, w.num_heads, device=dev, n_sms=n_sms)
    words = ref.mask_words(masks, w.q_len) if mask_words is None else mask_words
    mask = torch.from_numpy(words.copy()).to(dev)
    sl = w.seqlens.to(dev)
    bt = None if w.block_table is None else w.block_table.to(dev)
    ql = None if w.q_lens is None else w.q_lens.to(dev)
    o = torch.full((w.batch, w.q_len, w.num_heads, 512), float("nan"), dtype=torch.bfloat16, device=dev)
    lse = torch.full((w.batch, w.q_len, w.num_heads), float("nan"), dtype=torch.float32, device=dev)
    dec.plan(sl)
    if w.fp8:
        dec.fwd_tree_fp8(w.q.to(dev), w.kv8.to(dev), w.kv_scale.to(dev), sl, mask, bt, w.softmax_scale, o=o, lse=lse,
                         flags=flags, q_lens=ql)
    else:
        dec.fwd_tree(w.q.to(dev), w.kv.to(dev), sl, mask, bt, w.softmax_scale, o=o, lse=lse, flags=flags, q_lens=ql)
    torch.cuda.synchronize()
    return o, lse, dec.status(), dec


def rows_of(w, b):
    if not w.fp8:
        return w.kv_rows(b).double().numpy()
    L = int(w.seqlens[b])
    if w.block_table is None:
        codes, sc = w.kv8[b, :L], w.kv_scale[b, :L]
    else:
        pages = w.block_table[b, :(L + 63) // 64].long()
        codes, sc = w.kv8[pages].reshape(-1, 576)[:L], w.kv_scale[pages].reshape(-1)[:L]
    return ref.e4m3_values()[codes.numpy()] * sc.double().numpy()[:, None]


def check(w, masks, what, **kw):
    o, lse, st, _ = run_tree(w, masks, **kw)
    assert st == 0
    q_lens = [w.q_len] * w.batch if w.q_lens is None else w.q_lens.tolist()
    o_ref, lse_ref = ref.tree_attention(w.q.double().numpy(), [rows_of(w, b) for b in range(w.batch)], masks, q_lens,
                                        w.softmax_scale)
    assert_parity(o.float().cpu().numpy(), lse.cpu().numpy(), o_ref, lse_ref, what=what)
    dead = np.isneginf(lse_ref)
    assert (o.float().cpu().numpy()[dead] == 0).all()
    return o, lse


def tree_masks(rng, B, q_len, shape="tree"):
    return ref.extend([0] * B, [q_len] * B, [[0] * (ref.pages(q_len) + 1)] * B, [0] * 9999, 9999,
                      ref.random_parents(rng, B, q_len, shape), q_len)[3]


def random_masks(rng, B, q_len, density=0.5):
    """Any mask: not a tree's, some tokens without their own bit, some with none."""
    return [[sum(1 << u for u in range(q_len) if rng.random() < density) if rng.random() > 0.2 else 0
             for _ in range(q_len)] for _ in range(B)]


DTYPES = ["bf16", "e4m3"]


@pytest.mark.parametrize("kv", DTYPES)
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("heads,q_len", [(16, 1), (1, 16), (3, 5), (16, 2), (16, 4), (5, 33), (20, 7), (16, 16),
                                         (1, 64), (128, 2), (2, 100)])
def test_trees(heads, q_len, paged, kv):
    rng = np.random.default_rng(heads * 100 + q_len)
    lens = [q_len, q_len + 1, 64 + q_len, 127 + q_len, 700, 333]
    w = W.make_workload(len(lens), heads, lens, q_len=q_len, paged=paged, seed=q_len, kv_dtype=kv)
    check(w, tree_masks(rng, len(lens), q_len), f"h={heads} q={q_len} {kv}")


@pytest.mark.parametrize("kv", DTYPES)
@pytest.mark.parametrize("heads,q_len", [(16, 1), (8, 2), (16, 4), (16, 9), (1, 70)])
def test_any_mask(heads, q_len, kv):
    """Rows that no token sees, tokens that see nothing new, and (without context) nothing at all."""
    rng = np.random.default_rng(q_len)
    lens = [q_len, q_len, 300, 129 + q_len, 64 + q_len // 2]
    w = W.make_workload(len(lens), heads, lens, q_len=q_len, paged=True, seed=3, kv_dtype=kv)
    for density in (0.0, 0.1, 0.6, 1.0):
        masks = random_masks(rng, len(lens), q_len, density)
        masks[0] = [0] * q_len
        check(w, masks, f"any mask {density}")


@pytest.mark.parametrize("kv", DTYPES)
@pytest.mark.parametrize("heads,q_len", [(2, 8), (16, 8), (16, 40)])
def test_ragged_drafts(heads, q_len, kv):
    """0 .. q_len real tokens; masks and bits past them hold anything."""
    rng = np.random.default_rng(heads)
    q_lens = [0, 1, q_len, q_len // 2, 3, q_len - 1]
    lens = [500, 1, q_len + 5, 200, 64, 1000]
    w = W.make_workload(len(lens), heads, lens, q_len=q_len, paged=True, seed=4, q_lens=q_lens, kv_dtype=kv)
    masks = tree_masks(rng, len(lens), q_len)
    for b, n in enumerate(q_lens):
        for t in range(q_len):
            junk = int(rng.integers(0, 2 ** 62)) << n
            masks[b][t] = (masks[b][t] & ((1 << n) - 1) if t < n else 0) | (junk & ((1 << q_len) - 1))
    check(w, masks, "ragged")


@pytest.mark.parametrize("heads,q_len", [(16, 4), (4, 4), (16, 12)])
def test_fewer_rows_than_tokens_and_empty_sequences(heads, q_len):
    lens = [0, 1, 2, q_len - 1, q_len, 0]
    rng = np.random.default_rng(1)
    w = W.make_workload(len(lens), heads, lens, q_len=q_len, seed=5)
    o, lse, st, _ = run_tree(w, [[(1 << q_len) - 1] * q_len] * len(lens))
    assert st == 0 and (o[0] == 0).all() and torch.isneginf(lse[0]).all() and (o[5] == 0).all()
    # rows that exist are the last ones of the draft: token u is row L - n + u
    masks = tree_masks(rng, len(lens), q_len)
    for b, L in enumerate(lens):
        gone = max(q_len - L, 0)
        for t in range(q_len):
            masks[b][t] = masks[b][t] >> gone << gone
    o, lse, st, _ = run_tree(w, masks)
    for b, L in enumerate(lens):
        gone = max(q_len - L, 0)
        shifted = [[v >> gone for v in masks[b]]]
        k = [rows_of(w, b)]
        if L >= q_len or L == 0:
            continue
        # the reference on L tokens whose rows all are drafted: any token, the surviving bits
        for t in range(q_len):
            ro, rl = ref.tree_attention(w.q[b:b + 1, t:t + 1].double().numpy().repeat(L, 1), k,
                                        [[shifted[0][t]] * L], [L], w.softmax_scale)
            assert np.abs(o[b, t].float().cpu().numpy() - ro[0, 0]).max() <= 1e-2 * max(np.abs(ro[0, 0]).max(), 1e-6)
            got = lse[b, t].cpu().numpy()
            assert (np.isneginf(got) == np.isneginf(rl[0, 0])).all()


@pytest.mark.parametrize("kv", DTYPES)
@pytest.mark.parametrize("batch,heads,q_len", [(40, 16, 4), (40, 16, 9), (1100, 10, 3), (1030, 2, 2)])
def test_large_batches(batch, heads, q_len, kv):
    """More than 32 sequences, and more than 1024: every way that the plan is made."""
    lens = np.random.default_rng(batch).integers(0, 400, batch).tolist()
    lens[3] = 5000
    q_lens = [min(L, b % (q_len + 1)) for b, L in enumerate(lens)]
    w = W.make_workload(batch, heads, lens, q_len=q_len, paged=True, seed=24, q_lens=q_lens, kv_dtype=kv)
    check(w, random_masks(np.random.default_rng(17), batch, q_len), f"batch of {batch}")


@pytest.mark.parametrize("kv", DTYPES)
@pytest.mark.parametrize("heads,q_len", [(2, 5), (16, 4), (16, 9), (128, 4), (5, 33)])
def test_padding_queries_and_mask_bits_do_not_matter(heads, q_len, kv):
    """NaN, infinite and huge queries of padding tokens, and mask bits at or past the count: the same bits."""
    lens = [700, 9000, q_len, 257]
    q_lens = [1, q_len - 1, q_len, 0]
    w = W.make_workload(len(lens), heads, lens, q_len=q_len, paged=True, seed=22, q_lens=q_lens, kv_dtype=kv)
    masks = random_masks(np.random.default_rng(15), len(lens), q_len)
    want = run_tree(w, masks)
    assert want[2] == 0
    stuff = torch.tensor([float("nan"), float("inf"), -float("inf"), 3e38], dtype=torch.bfloat16)
    for b, n in enumerate(q_lens):
        w.q[b, n:] = stuff[torch.arange(w.q[b, n:].numel()) % 4].view(w.q[b, n:].shape)
        masks[b] = [(row if t < n else 0) | -(1 << n) & (1 << q_len) - 1 for t, row in enumerate(masks[b])]
    got = run_tree(w, masks)
    assert got[2] == 0 and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("kv", DTYPES)
def test_nan_past_the_end(kv):
    lens = [5, 64, 130, 1000]
    w = W.make_workload(4, 16, lens, q_len=5, paged=True, seed=6, extra_blocks=3, kv_dtype=kv)
    if kv == "bf16":
        _poison_padding(w)
    else:
        owned = torch.zeros(w.kv8.shape[:2], dtype=torch.bool)
        for b, L in enumerate(lens):
            for j in range(L):
                owned[int(w.block_table[b, j // 64]), j % 64] = True
        w.kv8[~owned] = 0x7F
        w.kv_scale[~owned] = float("nan")
    check(w, tree_masks(np.random.default_rng(2), 4, 5), "NaN past the end")


@pytest.mark.parametrize("kv", DTYPES)
@pytest.mark.parametrize("heads,q_len", [(16, 1), (4, 4), (16, 4), (16, 20), (128, 3)])
def test_a_chain_is_the_causal_decode(heads, q_len, kv):
    """The same values: the same bits where kernel and schedule are the same (at most 16 columns), else both
    are within the parity bar of them."""
    lens = [q_len, 40 + q_len, 900, 128]
    w = W.make_workload(4, heads, lens, q_len=q_len, causal=True, paged=True, seed=7, kv_dtype=kv, spike_frac=0.05)
    from tests.parity import run_cuda
    o, lse, st, _ = run_tree(w, [[(2 << t) - 1 for t in range(q_len)]] * 4)
    o2, lse2, st2, _ = run_cuda(w)
    assert st == st2 == 0
    if heads * q_len > 16:
        d = o.double().cpu().numpy() - o2
        assert np.sqrt((d ** 2).mean()) <= 2 * 2e-3 * np.sqrt((o2.astype(np.float64) ** 2).mean())
        np.testing.assert_allclose(lse.cpu().numpy(), lse2, rtol=0, atol=2e-3)
    else:
        np.testing.assert_array_equal(o.float().cpu().numpy(), o2)
        np.testing.assert_array_equal(lse.cpu().numpy(), lse2)


@pytest.mark.parametrize("kv", DTYPES)
@pytest.mark.parametrize("n_sms", [1, 2, 5, 148, 400])
def test_split_counts(n_sms, kv):
    w = W.make_workload(3, 16, [3000, 257, 1536], q_len=6, seed=8, kv_dtype=kv)
    check(w, tree_masks(np.random.default_rng(n_sms), 3, 6), f"n_sms={n_sms}", n_sms=n_sms)


@pytest.mark.parametrize("heads,kv", [(4, "bf16"), (16, "bf16"), (16, "e4m3")])
def test_combine_apart_gives_the_same_bits(heads, kv):
    w = W.make_workload(2, heads, [5000, 700], q_len=4, seed=9, kv_dtype=kv)
    masks = tree_masks(np.random.default_rng(3), 2, 4)
    o, lse, _, _ = run_tree(w, masks)
    o2, lse2, st, dec = run_tree(w, masks, flags=m.FLAG_SKIP_COMBINE)
    m.mla_combine(dec.workspace, 2, 4, heads, dec.n_sms, o2, lse2)
    torch.cuda.synchronize()
    assert st == 0 and torch.equal(o, o2) and torch.equal(lse, lse2)


def test_long_rows_one_probability_term():
    """128-column groups with one bf16 P term (every sequence holds 8192 rows or more), spiked rows."""
    w = W.make_workload(2, 16, [8192, 9001], q_len=9, paged=True, seed=10, spike_frac=0.05)
    check(w, tree_masks(np.random.default_rng(4), 2, 9), "mode 1")


@pytest.mark.parametrize("heads,q_len", [(16, 9), (128, 2), (16, 16)])
@pytest.mark.parametrize("kv", DTYPES)
def test_short_sequences_among_enough_units(heads, q_len, kv):
    """128-column groups with short sequences in them: theirs are multiplied by both bf16 terms of P."""
    lens = [9000, 700, q_len, 64 + q_len, 3000, 0, 8191, 8192]
    w = W.make_workload(len(lens), heads, lens, q_len=q_len, paged=True, seed=21, spike_frac=0.03, kv_dtype=kv)
    q_lens = [q_len if L >= q_len else 0 for L in lens]
    w.q_lens = torch.tensor(q_lens, dtype=torch.int32)
    assert m.mla_decode_plan_host(lens, q_len, heads, 148, schedule=2)[5] == 128
    masks = tree_masks(np.random.default_rng(14), len(lens), q_len)
    o, lse = check(w, masks, "short among long")
    # each short sequence by itself, to the same bar
    o = o.float().cpu().numpy()
    for b, L in enumerate(lens):
        if q_lens[b] and L < 8192:
            r = ref.tree_attention(w.q[b:b + 1].double().numpy(), [rows_of(w, b)], masks[b:b + 1], q_lens[b:b + 1],
                                   w.softmax_scale)
            assert_parity(o[b:b + 1], lse[b:b + 1].cpu().numpy(), *r, what=f"L={L}")


@pytest.mark.parametrize("batch", [1, 5, 31, 32, 33, 300, 1024, 1025, 3000])
def test_device_tree_schedule_matches_the_host(batch):
    from tests.test_parity_gpu import _a256, _sched_offsets
    rng = np.random.default_rng(batch)
    for heads, q_len in ((16, 4), (16, 8), (128, 4)):
        lens = rng.integers(0, 1500, batch).astype(np.int32)
        dec = m.MlaDecoder(batch, q_len, heads, device="cuda")
        dec.plan(torch.from_numpy(lens).cuda())
        torch.cuda.synchronize()
        ws = dec.workspace.view(torch.int32).cpu().numpy()
        ncols, sms = heads * q_len, dec.n_sms
        g64, g128 = (ncols + 63) // 64, (ncols + 127) // 128
        c_max = max(1, sms // 2 // g128)
        # the tables are the workspace's last: their size, from the end
        _, size = _sched_offsets(0, batch, c_max, g64)
        tab, end = _sched_offsets(dec.workspace.numel() - size, batch, c_max, g64)
        assert end == dec.workspace.numel()
        ranges, info, nct, ngr, rows, gcols = m.mla_decode_plan_host(lens, q_len, heads, sms, schedule=2)
        assert ws[24] == nct and ws[25] == ngr and ws[28] == gcols
        np.testing.assert_array_equal(ws[tab["ranges"] // 4:][:2 * nct].reshape(-1, 2), ranges)
        np.testing.assert_array_equal(ws[tab["info"] // 4:][:4 * batch].reshape(-1, 4), info)
        first = np.concatenate([[0], np.cumsum((lens.astype(np.int64) + rows - 1) // rows)])
        np.testing.assert_array_equal(ws[tab["tile"] // 4:][:batch + 1], first)


def test_bad_pages_are_reported():
    w = W.make_workload(2, 16, [200, 300], q_len=4, paged=True, seed=11)
    w.block_table[1, 2] = 10 ** 6
    _, _, st, _ = run_tree(w, tree_masks(np.random.default_rng(5), 2, 4))
    assert st == -7


def test_same_inputs_same_bits():
    w = W.make_workload(5, 16, [4000, 9, 700, 64, 2000], q_len=8, seed=12)
    masks = tree_masks(np.random.default_rng(6), 5, 8)
    first = run_tree(w, masks)
    for _ in range(3):
        again = run_tree(w, masks)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("heads,q_len", [(16, 9), (128, 2), (5, 26), (64, 16)])
def test_long_rows_on_the_e4m3_cache(heads, q_len):
    """128-column groups, whose two CTAs take 64 columns each; rows scaled x8 move the maxima."""
    w = W.make_workload(2, heads, [8192, 9001], q_len=q_len, paged=True, seed=13, spike_frac=0.05, kv_dtype="e4m3")
    check(w, tree_masks(np.random.default_rng(7), 2, q_len), "e4m3 mode 1")


@pytest.mark.parametrize("heads,q_len", [(16, 1), (16, 4), (20, 5)])
def test_e4m3_rows_of_very_unequal_scale(heads, q_len):
    """Row scales over twelve orders of two, rising and falling along the sequence, and rows of zeros."""
    lens = [1500, 333, 640]
    w = W.make_workload(3, heads, lens, q_len=q_len, seed=14, kv_dtype="e4m3")
    rows = torch.arange(w.kv_scale.shape[1])
    w.kv_scale *= torch.exp2(6.0 * torch.sin(rows / 70.0)).float()
    w.kv8[:, 100:130] = 0
    check(w, tree_masks(np.random.default_rng(8), 3, q_len), "unequal scales")


@pytest.mark.parametrize("kv", DTYPES)
def test_splits_of_a_long_sequence(kv):
    """One sequence over all SMs, and a neighbour of one tile."""
    w = W.make_workload(2, 16, [40000, 100], q_len=4, paged=True, seed=15, spike_frac=0.01, kv_dtype=kv)
    check(w, tree_masks(np.random.default_rng(9), 2, 4), "long split")


@pytest.mark.parametrize("heads,q_len,lens,kv", [(16, 4, [6000, 3000, 9000, 500], "e4m3"),
                                                 (128, 2, [8200, 9000], "e4m3"), (16, 4, [6000, 3000, 700], "bf16"),
                                                 (4, 4, [6000, 500], "bf16"), (4, 4, [6000, 500], "e4m3")])
def test_repeated_trees_are_bitwise_identical(heads, q_len, lens, kv):
    """Stress of the hand-offs between roles and CTAs: 200 plan + decode calls give one result."""
    w = W.make_workload(len(lens), heads, lens, q_len=q_len, seed=16, kv_dtype=kv, spike_frac=0.02)
    masks = tree_masks(np.random.default_rng(10), len(lens), q_len)
    o, lse = check(w, masks, "first of many")
    dec = m.MlaDecoder(w.batch, q_len, heads, device="cuda")
    sl, q = w.seqlens.cuda(), w.q.cuda()
    mask = torch.from_numpy(ref.mask_words(masks, q_len).copy()).cuda()
    kvs = (w.kv8.cuda(), w.kv_scale.cuda()) if kv == "e4m3" else (w.kv.cuda(),)
    fwd = dec.fwd_tree_fp8 if kv == "e4m3" else dec.fwd_tree
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(200):
        dec.plan(sl)
        o2, lse2 = fwd(q, *kvs, sl, mask)
        differ += (o2 != o).sum() + (lse2 != lse).sum()
    assert int(differ) == 0 and dec.status() == 0


@pytest.mark.parametrize("heads,q_len,kv", [(4, 4, "bf16"), (16, 4, "bf16"), (4, 4, "e4m3"), (16, 4, "e4m3")])
def test_bounded_waits_of_the_tree_kernels(heads, q_len, kv):
    """Q withheld: the waits run out, the status says so, and the next decode on the workspace is right."""
    w = W.make_workload(2, heads, [700, 300], q_len=q_len, seed=17, kv_dtype=kv)
    masks = tree_masks(np.random.default_rng(11), 2, q_len)
    assert run_tree(w, masks, flags=m.FLAG_TEST_EXPIRE_WAITS)[2] == -6
    check(w, masks, "after a timeout")


@pytest.mark.parametrize("heads,kv", [(4, "bf16"), (16, "bf16"), (16, "e4m3")])
def test_lengths_out_of_range_are_reported(heads, kv):
    w = W.make_workload(2, heads, [100, 300], q_len=4, seed=18, kv_dtype=kv)
    masks = tree_masks(np.random.default_rng(12), 2, 4)
    for q_lens in ([-1, 2], [2, 5]):
        w.q_lens = torch.tensor(q_lens, dtype=torch.int32)
        assert run_tree(w, masks)[2] == -1
    w.q_lens = None
    w.seqlens = torch.tensor([100, 301], dtype=torch.int32)
    assert run_tree(w, masks)[2] == -1


def test_two_streams_two_workspaces():
    """Two decodes at once, on streams and workspaces of their own, give what each gives alone."""
    ws = [W.make_workload(3, 16, [3000, 257, 1536], q_len=4, seed=s, kv_dtype=kv) for s, kv in ((19, "bf16"), (20, "e4m3"))]
    masks = tree_masks(np.random.default_rng(13), 3, 4)
    alone = [run_tree(w, masks)[:2] for w in ws]
    mask = torch.from_numpy(ref.mask_words(masks, 4).copy()).cuda()
    decs = [m.MlaDecoder(3, 4, 16, device="cuda") for _ in ws]
    streams = [torch.cuda.Stream() for _ in ws]
    args = [(w.q.cuda(), *((w.kv8.cuda(), w.kv_scale.cuda()) if w.fp8 else (w.kv.cuda(),)), w.seqlens.cuda(), mask)
            for w in ws]
    torch.cuda.synchronize()
    for _ in range(20):
        outs = []
        for w, dec, s, a in zip(ws, decs, streams, args):
            dec.plan(a[-2], stream=s)
            with torch.cuda.stream(s):
                outs.append((dec.fwd_tree_fp8 if w.fp8 else dec.fwd_tree)(*a, stream=s))
        torch.cuda.synchronize()
        for (o, lse), (o2, lse2) in zip(alone, outs):
            assert torch.equal(o, o2) and torch.equal(lse, lse2)


# ------------------------------------------------------------------------------------ the whole step
@pytest.mark.parametrize("kv,heads,captured", [("bf16", 16, False), ("e4m3", 16, False), ("bf16", 4, True),
                                               ("e4m3", 16, True)])
def test_verify_steps(kv, heads, captured):
    """Three serving steps over a paged cache that fills, shrinks and frees pages, each checked against
    the references on the cache as it stands; with `captured`, one graph replayed on new inputs."""
    dev, B, q, P, fp8 = "cuda", 4, 6, 3, kv == "e4m3"
    rng = np.random.default_rng(20)
    lens, num_blocks, max_blocks = [60, 0, 126, 333], 24, 8
    table, stack, nfree = ref.paged_setup(rng, lens, max_blocks, num_blocks)
    i32 = lambda x: torch.as_tensor(np.asarray(x), dtype=torch.int32, device=dev)  # noqa: E731
    w = W.make_workload(1, 1, [num_blocks * 64], seed=21, kv_dtype=kv)
    cache = (w.kv8 if fp8 else w.kv).reshape(num_blocks, 64, 576).to(dev)
    scale = w.kv_scale.reshape(num_blocks, 64).to(dev) if fp8 else None
    rope = torch.rand(1024, 32, dtype=torch.float64, generator=torch.Generator().manual_seed(1)) * 6
    rope = torch.cat([rope.cos(), rope.sin()], 1).float().to(dev)
    d = dict(lens=i32(lens), table=i32(table), stack=i32(stack), nfree=i32([nfree]), new=i32([0] * B),
             parents=i32([[-1] * q] * B), path=i32([[-1] * P] * B), keep=i32([0] * B), slots=i32([[0] * q] * B),
             pos=i32([[0] * q] * B), mask=i32([[[0]] * q] * B), status=i32([0]))
    latent = torch.zeros(B * q, 576, dtype=torch.bfloat16, device=dev)
    weight = (1 + 0.1 * torch.randn(512, generator=torch.Generator().manual_seed(2))).bfloat16().to(dev)
    q_rope = torch.zeros(B * q, heads, 64, dtype=torch.bfloat16, device=dev)
    queries = torch.zeros(B, q, heads, 576, dtype=torch.bfloat16, device=dev)
    dec = m.MlaDecoder(B, q, heads, device=dev)
    o = torch.zeros(B, q, heads, 512, dtype=torch.bfloat16, device=dev)
    lse = torch.zeros(B, q, heads, dtype=torch.float32, device=dev)

    def verify():
        m.mla_cache_extend(d["lens"], d["new"], d["table"], d["stack"], d["nfree"], num_blocks * 64, d["slots"],
                           d["pos"], d["lens"], d["nfree"], d["status"], parents=d["parents"], tree_mask=d["mask"])
        front = (latent, weight, 1e-6, rope, True, d["pos"].view(-1), d["slots"].view(-1), cache)
        if fp8:
            m.mla_cache_append_fp8(*front, scale, d["status"], q_rope=q_rope, q=queries)
        else:
            m.mla_cache_append(*front, d["status"], q_rope=q_rope, q=queries)
        dec.plan(d["lens"])
        if fp8:
            dec.fwd_tree_fp8(queries, cache, scale, d["lens"], d["mask"], d["table"], o=o, lse=lse, q_lens=d["new"])
        else:
            dec.fwd_tree(queries, cache, d["lens"], d["mask"], d["table"], o=o, lse=lse, q_lens=d["new"])

    def accept():
        m.mla_cache_accept(cache, d["lens"], d["new"], d["path"], d["keep"], d["table"], d["stack"], d["nfree"],
                           d["lens"], d["nfree"], d["status"], kv_scale=scale)

    graphs = []
    if captured:
        verify(), accept()  # no new tokens yet: nothing changes
        torch.cuda.synchronize()
        for call in (verify, accept):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                call()
            graphs.append(g.replay)
    steps = graphs or [verify, accept]
    for step in range(3):
        new = [q, 1 + step, 0 if step == 1 else 4, q]
        parents = ref.random_parents(rng, B, q)
        g = torch.Generator().manual_seed(30 + step)
        latent.copy_(torch.randn(B * q, 576, generator=g))
        q_rope.copy_(torch.randn(B * q, heads, 64, generator=g))
        queries[..., :512] = torch.randn(B, q, heads, 512, generator=g).to(dev).bfloat16()
        d["new"].copy_(i32(new))
        d["parents"].copy_(i32(parents))
        before = cache.clone()
        steps[0]()
        torch.cuda.synchronize()
        assert int(d["status"]) == 0 and dec.status() == 0
        table, slots, pos, masks, lens, nfree = ref.extend(lens, new, table, stack, nfree, parents, q)
        assert d["slots"].tolist() == slots and d["table"].tolist() == table and d["lens"].tolist() == lens
        assert int(d["nfree"]) == nfree
        # the new rows, from the inputs; every other row as before
        want = ref.append_rows(latent.double().cpu().numpy(), weight.double().cpu().numpy(), 1e-6,
                               rope.double().cpu().numpy(), np.asarray(pos).reshape(-1), True)
        at = np.asarray(slots).reshape(-1)
        codes = cache.view(-1, 576).cpu()
        vals = (ref.e4m3_values()[codes.numpy()] * scale.view(-1).double().cpu().numpy()[:, None] if fp8
                else codes.double().numpy())
        live = at >= 0
        # bf16: half a step (2^-8) and the fp32 arithmetic; E4M3: 2^-4, and 2^-10 of the scale near zero
        rel, floor = (2.0 ** -4 + 2.0 ** -12, np.abs(want[live]).max(1, keepdims=True) / 448 * 2.0 ** -9) if fp8 else (
            2.0 ** -8 + 2.0 ** -13, 1e-5)
        assert (np.abs(vals[at[live]] - want[live]) <= np.abs(want[live]) * rel + floor).all()
        other = np.ones(len(vals), bool)
        other[at[live]] = False
        assert torch.equal(cache.view(-1, 576).cpu()[torch.from_numpy(other)],
                           before.view(-1, 576).cpu()[torch.from_numpy(other)])
        rows = [vals[[table[b][j // 64] * 64 + j % 64 for j in range(lens[b])]].reshape(-1, 576) for b in range(B)]
        o_ref, lse_ref = ref.tree_attention(queries.double().cpu().numpy(), rows, masks, new, 576 ** -0.5)
        assert_parity(o.float().cpu().numpy(), lse.cpu().numpy(), o_ref, lse_ref, what=f"step {step}")
        # a path from a root down, at most P long; the third request ends after the last step
        path, keep = [], []
        for b in range(B):
            t, way = new[b] - 1, []
            while t >= 0:
                way.append(t)
                t = parents[b][t]
            way = way[::-1][:P]
            keep.append(-1 if (b == 3 and step == 2) else len(way))
            path.append(way + [-1] * (P - len(way)))
        d["path"].copy_(i32(path))
        d["keep"].copy_(i32(keep))
        steps[1]()
        torch.cuda.synchronize()
        moves, lens, stack, nfree = ref.accept(lens, new, path, keep, table, stack, nfree)
        assert int(d["status"]) == 0 and d["lens"].tolist() == lens and int(d["nfree"]) == nfree
        assert d["stack"].tolist()[:nfree] == stack[:nfree]
        order = np.arange(len(vals))
        for src, dst in moves:
            order[dst] = src
        assert torch.equal(cache.view(-1, 576).cpu(), codes[torch.from_numpy(order)])
    used = sorted(p for b in range(B) for p in table[b][:ref.pages(lens[b])])
    assert sorted(used + stack[:nfree]) == list(range(num_blocks))  # no page lost, none held twice
