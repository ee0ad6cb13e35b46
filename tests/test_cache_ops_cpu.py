"""Host side of the verify step's operators: references against hand-worked cases, argument checks of
the C entry points (nothing is launched) and of the binding."""

from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

import mla_decode_attention_etap_b200 as m
from tests import verify_reference as ref

A = 1 << 20  # a fake, suitably aligned device address: every call below is refused before it is used
vp = ctypes.c_void_p


def opt(x):
    return vp(x) if x else None


# ------------------------------------------------------------------------------------- references
def test_reference_extend_by_hand():
    """63 rows + 2 tokens cross into a new page; 64 + 1 open one; an empty request takes its first."""
    table, slots, pos, masks, lens, nfree = ref.extend([63, 64, 0], [2, 1, 0], [[5, -1], [6, -1], [-1, -1]],
                                                       [9, 8, 7], 3, [[-1, 0], [-1, 0], [-1, 0]], 2)
    assert table == [[5, 7], [6, 8], [-1, -1]] and nfree == 1 and lens == [65, 65, 0]
    assert slots == [[5 * 64 + 63, 7 * 64], [8 * 64, -1], [-1, -1]]
    assert pos == [[63, 64], [64, -1], [-1, -1]] and masks == [[1, 3], [1, 0], [0, 0]]


def test_reference_tree_masks_and_words():
    _, _, pos, masks, _, _ = ref.extend([10], [5], [[0]], [], 0, [[-1, 0, 0, 1, -1]], 5)
    assert masks == [[0b1, 0b11, 0b101, 0b1011, 0b10000]] and pos == [[10, 11, 11, 12, 10]]
    w = ref.mask_words([[1 << 33 | 1 << 31]], 40)
    assert w.shape == (1, 40, 2) and w[0, 0].tolist() == [-2 ** 31, 2]


def test_reference_rotation_is_a_rotation():
    rng = np.random.default_rng(0)
    x, a = rng.standard_normal((3, 64)), rng.uniform(-9, 9, (3, 32))
    cs = np.concatenate([np.cos(a), np.sin(a)], 1)
    for inter in (False, True):
        y = ref.rotate(x, cs, inter)
        np.testing.assert_allclose((y ** 2).sum(1), (x ** 2).sum(1), rtol=1e-13)
        back = np.concatenate([np.cos(a), -np.sin(a)], 1)
        np.testing.assert_allclose(ref.rotate(y, back, inter), x, atol=1e-13)
    # the first pair by hand
    y = ref.rotate(x, cs, False)
    assert y[0, 0] == pytest.approx(x[0, 0] * np.cos(a[0, 0]) - x[0, 32] * np.sin(a[0, 0]), abs=1e-14)


def test_reference_attention_of_a_chain_is_causal():
    from oracle import mla_oracle as om
    from mla_decode_attention_etap_b200 import workloads as W
    w = W.make_workload(2, 2, [9, 40], q_len=4, causal=True, seed=1)
    masks = [[(2 << t) - 1 for t in range(4)]] * 2
    rows = [w.kv_rows(b).double().numpy() for b in range(2)]
    o, lse = ref.tree_attention(w.q.double().numpy(), rows, masks, [4, 4], w.softmax_scale)
    o2, lse2 = om.mla_decode(W.bf16_bits(w.q), W.bf16_bits(w.kv), w.seqlens.numpy(), None, w.softmax_scale, True)
    np.testing.assert_allclose(o, o2, atol=1e-6)
    np.testing.assert_allclose(lse, lse2, atol=1e-5)


def test_reference_e4m3_values_match_torch():
    v = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(ref.e4m3_values(), v)


def test_reference_accept_by_hand():
    moves, lens, stack, nfree = ref.accept([66, 130], [3, 4], [[1, 2], [0, -1]], [2, -1], [[4, 7, 0], [1, 2, 3]],
                                           [9, -1, -1, -1, -1], 1)
    assert moves == [(7 * 64, 4 * 64 + 63), (7 * 64 + 1, 7 * 64)] and lens == [65, 0]
    assert stack == [9, 1, 2, 3, -1] and nfree == 4


# ------------------------------------------------------------------------------------ C entry points
def extend(**kw):
    a = dict(seqlens=A, new_lens=A, parents=A, batch=2, q_len=4, block_table=A, max_blocks=3, free_pages=A, cap=6,
             num_free=A, kv_rows=384, slots=A, positions=A, tree_mask=A, seqlens_out=A, num_free_out=A, status=A)
    a.update(kw)
    return m.lib().mla_cache_extend(opt(a["seqlens"]), opt(a["new_lens"]), opt(a["parents"]), a["batch"], a["q_len"],
                                    opt(a["block_table"]), a["max_blocks"], opt(a["free_pages"]), a["cap"],
                                    opt(a["num_free"]), a["kv_rows"], opt(a["slots"]), opt(a["positions"]),
                                    opt(a["tree_mask"]), opt(a["seqlens_out"]), opt(a["num_free_out"]),
                                    opt(a["status"]), None)


@pytest.mark.parametrize("kw,code", [
    (dict(seqlens=0), -1), (dict(slots=0), -1), (dict(positions=0), -1), (dict(seqlens_out=0), -1),
    (dict(status=0), -1), (dict(batch=0), -1), (dict(batch=65537), -1), (dict(q_len=0), -1),
    (dict(parents=0), -1), (dict(tree_mask=0), -1),            # parents and tree_mask come together
    (dict(free_pages=0), -1), (dict(num_free=0), -1), (dict(num_free_out=0), -1), (dict(cap=-1), -1),
    (dict(max_blocks=0), -1), (dict(kv_rows=100), -1), (dict(kv_rows=0), -1),
    (dict(q_len=1025), -2),                                    # a tree of more than MLA_MAX_COLUMNS tokens
    (dict(batch=65536, q_len=65536, parents=0, tree_mask=0), -2),
    (dict(max_blocks=1 << 26), -2), (dict(kv_rows=1 << 32), -2),
    (dict(block_table=0, batch=65536, kv_rows=1 << 20), -2),   # contiguous rows past int32
    (dict(seqlens=A + 2), -3), (dict(parents=A + 1), -3), (dict(tree_mask=A + 2), -3), (dict(status=A + 2), -3),
])
def test_extend_refuses(kw, code):
    assert extend(**kw) == code


def append(fp8=False, **kw):
    a = dict(latent=A, stride=576, weight=A, eps=1e-6, table=A, max_pos=16, inter=0, positions=A, slots=A, tokens=4,
             kv=A, scale=A, rows=128, q_rope=A, ts=1024, hs=64, heads=16, q=A, status=A)
    a.update(kw)
    ahead = [opt(a["latent"]), a["stride"], opt(a["weight"]), a["eps"], opt(a["table"]), a["max_pos"], a["inter"],
             opt(a["positions"]), opt(a["slots"]), a["tokens"], opt(a["kv"])]
    behind = [a["rows"], opt(a["q_rope"]), a["ts"], a["hs"], a["heads"], opt(a["q"]), opt(a["status"]), None]
    if fp8:
        return m.lib().mla_cache_append_fp8(*ahead, opt(a["scale"]), *behind)
    return m.lib().mla_cache_append(*ahead, *behind)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(latent=0), -1), (dict(table=0), -1), (dict(positions=0), -1), (dict(slots=0), -1), (dict(kv=0), -1),
    (dict(status=0), -1), (dict(tokens=-1), -1), (dict(max_pos=0), -1), (dict(rows=0), -1), (dict(inter=2), -1),
    (dict(eps=-1e-6), -1), (dict(eps=float("nan")), -1), (dict(eps=float("inf")), -1), (dict(stride=568), -1),
    (dict(q=0), -1), (dict(q_rope=0), -1), (dict(heads=0), -1), (dict(ts=-64), -1), (dict(hs=-64), -1),
    (dict(rows=1 << 31), -2), (dict(heads=1025), -2),
    (dict(latent=A + 8), -3), (dict(stride=580), -3), (dict(weight=A + 2), -3), (dict(table=A + 8), -3),
    (dict(kv=A + 8), -3), (dict(q_rope=A + 8), -3), (dict(q=A + 8), -3), (dict(ts=1028), -3), (dict(hs=68), -3),
    (dict(positions=A + 2), -3), (dict(slots=A + 1), -3), (dict(status=A + 2), -3),
])
def test_append_refuses(fp8, kw, code):
    assert append(fp8, **kw) == code


def test_append_fp8_needs_scales_and_nothing_is_launched_for_no_tokens():
    assert append(True, scale=0) == -1 and append(True, scale=A + 2) == -3
    assert append(False, tokens=0) == 0 and append(True, tokens=0) == 0


def accept(**kw):
    a = dict(kv=A, scale=0, seqlens=A, new_lens=A, path=A, path_lens=A, batch=2, q_len=4, max_path=4, block_table=A,
             max_blocks=3, free_pages=A, cap=6, num_free=A, kv_rows=384, seqlens_out=A, num_free_out=A, status=A)
    a.update(kw)
    return m.lib().mla_cache_accept(opt(a["kv"]), opt(a["scale"]), opt(a["seqlens"]), opt(a["new_lens"]),
                                    opt(a["path"]), opt(a["path_lens"]), a["batch"], a["q_len"], a["max_path"],
                                    opt(a["block_table"]), a["max_blocks"], opt(a["free_pages"]), a["cap"],
                                    opt(a["num_free"]), a["kv_rows"], opt(a["seqlens_out"]), opt(a["num_free_out"]),
                                    opt(a["status"]), None)


@pytest.mark.parametrize("kw,code", [
    (dict(kv=0), -1), (dict(seqlens=0), -1), (dict(new_lens=0), -1), (dict(path=0), -1), (dict(path_lens=0), -1),
    (dict(seqlens_out=0), -1), (dict(status=0), -1), (dict(batch=0), -1), (dict(q_len=0), -1), (dict(max_path=0), -1),
    (dict(free_pages=0), -1), (dict(num_free=0), -1), (dict(num_free_out=0), -1), (dict(cap=-1), -1),
    (dict(max_blocks=0), -1), (dict(kv_rows=100), -1),
    (dict(kv_rows=1 << 32), -2), (dict(block_table=0, batch=65536, kv_rows=1 << 20), -2),
    (dict(kv=A + 8), -3), (dict(scale=A + 2), -3), (dict(path=A + 2), -3), (dict(num_free_out=A + 1), -3),
])
def test_accept_refuses(kw, code):
    assert accept(**kw) == code


def tree(fp8=False, **kw):
    a = dict(q=A, kv=A, scale=A, seqlens=A, q_lens=0, mask=A, block_table=0, batch=2, q_len=4, heads=16, kv_rows=128,
             max_blocks=0, sm=1 / 24, o=A, lse=A, ws=A, ws_bytes=1 << 30, n_sms=148, flags=0)
    a.update(kw)
    mid = [opt(a["seqlens"]), opt(a["q_lens"]), opt(a["mask"]), opt(a["block_table"]), a["batch"], a["q_len"],
           a["heads"], a["kv_rows"], a["max_blocks"], a["sm"], opt(a["o"]), opt(a["lse"]), opt(a["ws"]),
           a["ws_bytes"], a["n_sms"], a["flags"], None]
    if fp8:
        return m.lib().mla_decode_fwd_tree_fp8(opt(a["q"]), opt(a["kv"]), opt(a["scale"]), *mid)
    return m.lib().mla_decode_fwd_tree(opt(a["q"]), opt(a["kv"]), *mid)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(q=0), -1), (dict(kv=0), -1), (dict(seqlens=0), -1), (dict(mask=0), -1), (dict(o=0), -1), (dict(lse=0), -1),
    (dict(ws=0), -1), (dict(sm=0.0), -1), (dict(sm=float("nan")), -1), (dict(flags=8), -1), (dict(q_len=0), -1),
    (dict(heads=257), -2), (dict(mask=A + 2), -3), (dict(q=A + 8), -3), (dict(q_lens=A + 2), -3),
    (dict(ws_bytes=100), -4), (dict(block_table=A, kv_rows=100, max_blocks=2), -1),
])
def test_tree_refuses(fp8, kw, code):
    assert tree(fp8, **kw) == code


def test_tree_fp8_needs_scales():
    assert tree(True, scale=0) == -1


# ---------------------------------------------------------------------------------- tree schedule
@pytest.mark.parametrize("lens,q,h,want", [
    ([1024], 8, 16, (37, 2, 256, 64)),            # 4 units: too few for 74 clusters, groups of 64
    ([300] * 74, 8, 16, (74, 1, 256, 128)),       # short sequences, but two units for every cluster
    ([9000], 8, 16, (74, 1, 256, 128)),           # long enough for the duo schedule's groups of 128
    ([32768] * 16, 4, 16, (74, 1, 256, 64)),      # 64 columns: one group
    ([64], 64, 16, (4, 16, 256, 64)),             # 1024 columns
    ([700] * 3, 1, 16, (74, 1, 128, 16)),         # 16 columns: the pair schedule
])
def test_tree_schedule_grouping(lens, q, h, want):
    ranges, info, *rest = m.mla_decode_plan_host(lens, q, h, 148, schedule=2)
    assert tuple(rest) == want
    units = sum(-(-L // want[2]) for L in lens)
    assert ranges[0, 0] == 0 and ranges[-1, 1] == units and (ranges[1:, 0] == ranges[:-1, 1]).all()
    assert info[:, 0].sum() == units


@pytest.mark.parametrize("lens,q,h", [([1024], 8, 16), ([100, 20], 8, 16), ([5000] * 3, 4, 16), ([64], 1, 17),
                                      ([300, 0, 1], 64, 16)])
def test_tree_schedule_gives_every_unit_its_own_work_unit(lens, q, h):
    """As long as there are enough of them."""
    ranges, info, ctas, *_ = m.mla_decode_plan_host(lens, q, h, 148, schedule=2)
    units = sum(-(-L // 256) for L in lens)
    assert units <= ctas
    assert [tuple(r) for r in ranges] == [(c, c + 1) if c < units else (units, units) for c in range(ctas)]
    assert info[:, 2].tolist() == [-(-L // 256) for L in lens]


def test_tree_schedule_is_the_duo_schedule_in_groups_of_128():
    for lens, q, h in (([9000, 8192, 10000], 8, 16), ([30000] * 8, 4, 128)):
        a, b = (m.mla_decode_plan_host(lens, q, h, 148, schedule=s) for s in (1, 2))
        assert a[5] == 128 and a[2:] == b[2:]
        np.testing.assert_array_equal(a[0], b[0])
        np.testing.assert_array_equal(a[1], b[1])


def test_tree_schedule_end_costs():
    """64-column groups: a sequence's end counts as four units, in the duo schedule as two."""
    lens = [3000, 5000, 40000, 256, 0, 17]
    units = [-(-L // 256) for L in lens]
    for schedule, E in ((1, 2), (2, 4)):
        ranges, info, ctas, *_ = m.mla_decode_plan_host(lens, 4, 16, 148, schedule=schedule)
        cost = sum(u + E for u in units if u)
        # the last unit of every sequence ends a range or lies in one whose cost is at most an even share
        share = -(-cost // ctas)
        for lo, hi in ranges:
            ends = sum(lo < e <= hi for e, u in zip(np.cumsum(units), units) if u)
            assert hi - lo + E * max(ends - 1, 0) <= share


def test_static_workspace_takes_what_it_took():
    """The tree schedule's tables come behind what the other decodes need: a workspace without them
    still serves those, and a tree decode refuses it."""
    need = m.mla_decode_workspace_size(2, 8, 16, 148)
    assert tree(q_len=8, ws_bytes=need - 256) == -4 and tree(True, q_len=8, ws_bytes=need - 256) == -4


# ------------------------------------------------------------------------------------------ binding
def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def extend_args(B=3, q=5, tree=True, paged=True):
    return dict(seqlens=i32(B), new_lens=i32(B), block_table=i32(B, 4) if paged else None,
                free_pages=i32(12) if paged else None, num_free=i32(1) if paged else None, slots=i32(B, q),
                positions=i32(B, q), seqlens_out=i32(B), num_free_out=i32(1) if paged else None, status=i32(1),
                parents=i32(B, q) if tree else None, tree_mask=i32(B, q, 1) if tree else None)


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("paged", [False, True])
def test_extend_guards_accept(tree, paged):
    m.check_extend_args(**extend_args(tree=tree, paged=paged))
    m.check_extend_args(**dict(extend_args(tree=tree, paged=paged), new_lens=None))


@pytest.mark.parametrize("name,value,exc", [
    ("seqlens", i32(2), ValueError), ("seqlens", i32(3).long(), TypeError), ("seqlens", None, ValueError),
    ("seqlens", i32(6)[::2], ValueError), ("new_lens", i32(4), ValueError), ("slots", i32(15), ValueError),
    ("slots", i32(3, 10)[:, ::2], ValueError), ("slots", [1], TypeError), ("positions", i32(3, 4), ValueError),
    ("parents", None, ValueError), ("tree_mask", i32(3, 5, 2), ValueError), ("tree_mask", None, ValueError),
    ("block_table", i32(2, 4), ValueError), ("block_table", i32(3, 8)[:, ::2], ValueError),
    ("free_pages", i32(3, 4), ValueError), ("free_pages", None, TypeError), ("num_free", i32(2), ValueError),
    ("num_free_out", None, ValueError), ("status", i32(0), ValueError), ("status", i32(1).float(), TypeError),
])
def test_extend_guards_reject(name, value, exc):
    with pytest.raises(exc):
        m.check_extend_args(**dict(extend_args(), **{name: value}))


def append_args(T=6, h=2, fp8=False):
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    return dict(latent=bf(T, 700)[:, 100:676], norm_weight=bf(512), rope_table=torch.zeros(9, 64), positions=i32(T),
                slots=i32(T), kv=torch.zeros(2, 64, 576, dtype=torch.uint8) if fp8 else bf(2, 64, 576), status=i32(1),
                q_rope=bf(T, h, 192)[..., 128:], q=bf(2, T // 2, h, 576),
                kv_scale=torch.zeros(2, 64) if fp8 else None)


@pytest.mark.parametrize("fp8", [False, True])
def test_append_guards_accept(fp8):
    a = append_args(fp8=fp8)
    ahead, _, where, cache, behind = m.check_append_args(**a)
    assert ahead[1] == 700 and where[-1] == 6 and cache[-1] == 128 and behind[1:4] == [384, 192, 2]
    m.check_append_args(**dict(a, q=None, q_rope=None, norm_weight=None))
    m.check_append_args(**append_args(T=0, fp8=fp8))


@pytest.mark.parametrize("name,value,exc", [
    ("latent", torch.zeros(6, 576), TypeError), ("latent", torch.zeros(6, 500, dtype=torch.bfloat16), ValueError),
    ("latent", torch.zeros(6, 1152, dtype=torch.bfloat16)[:, ::2], ValueError), ("latent", None, TypeError),
    ("norm_weight", torch.zeros(511, dtype=torch.bfloat16), ValueError), ("norm_weight", torch.zeros(512), TypeError),
    ("rope_table", torch.zeros(9, 32), ValueError), ("rope_table", torch.zeros(9, 64).double(), TypeError),
    ("positions", i32(5), ValueError), ("slots", i32(6).long(), TypeError), ("slots", None, ValueError),
    ("kv", torch.zeros(2, 64, 576), TypeError), ("kv", torch.zeros(2, 64, 512, dtype=torch.bfloat16), ValueError),
    ("q", None, ValueError), ("q_rope", None, ValueError),
    ("q", torch.zeros(6, 3, 576, dtype=torch.bfloat16), ValueError),
    ("q", torch.zeros(12, 576, dtype=torch.bfloat16), ValueError),
    ("q_rope", torch.zeros(6, 2, 128, dtype=torch.bfloat16)[..., ::2], ValueError),
    ("q_rope", torch.zeros(5, 2, 64, dtype=torch.bfloat16), ValueError), ("status", None, TypeError),
])
def test_append_guards_reject(name, value, exc):
    with pytest.raises(exc):
        m.check_append_args(**dict(append_args(), **{name: value}))


def accept_args(B=3, P=2, paged=True, fp8=False):
    shape = (12, 64, 576) if paged else (B, 200, 576)
    return dict(kv=torch.zeros(shape, dtype=torch.uint8 if fp8 else torch.bfloat16), seqlens=i32(B), new_lens=i32(B),
                path=i32(B, P), path_lens=i32(B), block_table=i32(B, 4) if paged else None,
                free_pages=i32(12) if paged else None, num_free=i32(1) if paged else None, seqlens_out=i32(B),
                num_free_out=i32(1) if paged else None, status=i32(1), kv_scale=torch.zeros(shape[:2]) if fp8 else None)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("paged", [False, True])
def test_accept_guards_accept(paged, fp8):
    assert m.check_accept_args(**accept_args(paged=paged, fp8=fp8))[1] == (768 if paged else 200)


@pytest.mark.parametrize("name,value,exc", [
    ("path", i32(6), ValueError), ("path", i32(3, 2).long(), TypeError), ("path", None, TypeError),
    ("path_lens", i32(2), ValueError), ("new_lens", None, ValueError), ("seqlens_out", i32(4), ValueError),
    ("kv", torch.zeros(12, 32, 576, dtype=torch.bfloat16), ValueError), ("kv", torch.zeros(12, 64, 576), TypeError),
    ("num_free", None, ValueError), ("free_pages", i32(12).float(), TypeError), ("block_table", i32(4, 4), ValueError),
])
def test_accept_guards_reject(name, value, exc):
    with pytest.raises(exc):
        m.check_accept_args(**dict(accept_args(), **{name: value}))


def test_accept_guards_reject_too_few_contiguous_sequences():
    a = accept_args(paged=False)
    a["kv"] = a["kv"][:2]
    with pytest.raises(ValueError):
        m.check_accept_args(**a)


def test_tree_guards():
    q = torch.zeros(2, 5, 4, 576, dtype=torch.bfloat16)
    kv = torch.zeros(2, 90, 576, dtype=torch.bfloat16)
    o, lse = torch.zeros(2, 5, 4, 512, dtype=torch.bfloat16), torch.zeros(2, 5, 4)
    ws = torch.zeros(1024, dtype=torch.uint8)
    m.check_tree_args(q, kv, i32(2), None, i32(2, 5, 1), o, lse, ws, i32(2))
    for bad in (i32(2, 5, 2), i32(2, 5), i32(2, 4, 1), i32(2, 10, 1)[:, ::2]):
        with pytest.raises(ValueError):
            m.check_tree_args(q, kv, i32(2), None, bad, o, lse, ws)
    with pytest.raises(TypeError):
        m.check_tree_args(q, kv, i32(2), None, i32(2, 5, 1).long(), o, lse, ws)
    with pytest.raises(ValueError, match="pages"):
        m.check_tree_args(q, kv, i32(2), i32(2, 3), i32(2, 5, 1), o, lse, ws)


def test_wrappers_refuse_host_tensors():
    with pytest.raises(ValueError, match="CUDA"):
        a = extend_args()
        m.mla_cache_extend(a["seqlens"], None, a["block_table"], a["free_pages"], a["num_free"], 768, a["slots"],
                           a["positions"], a["seqlens_out"], a["num_free_out"], a["status"])
    a = append_args()
    with pytest.raises(ValueError, match="CUDA"):
        m.mla_cache_append(a["latent"], None, 0.0, a["rope_table"], False, a["positions"], a["slots"], a["kv"],
                           a["status"])
    with pytest.raises(TypeError, match="kv_scale"):
        m.mla_cache_append_fp8(a["latent"], None, 0.0, a["rope_table"], False, a["positions"], a["slots"], a["kv"],
                               None, a["status"])
    a = accept_args()
    with pytest.raises(ValueError, match="CUDA"):
        m.mla_cache_accept(**a)
    q = torch.zeros(2, 5, 4, 576, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        m.mla_decode_fwd_tree(q, q, q, None, 1.0, q, q, q, q, 148)
