"""GPU tests of mla_cache_extend, mla_cache_append(_fp8) and mla_cache_accept against the 64-bit
references of tests/verify_reference.py."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import mla_decode_attention_etap_b200 as m
from tests import verify_reference as ref

pytestmark = pytest.mark.gpu

INVALID, BLOCK_TABLE, PAGES = -1, -7, -8


def dev(x, dtype=torch.int32):
    return torch.as_tensor(np.asarray(x), dtype=dtype).cuda()


def status_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------------------------------ extend
class Extend:
    """One extend call on copies of host lists, outputs poisoned first."""

    def __init__(self, lens, new_lens, table, stack, nfree, q_len, parents=None, kv_rows=None, in_place=False,
                 num_blocks=None):
        B = len(lens)
        self.lens, self.stack, self.nfree = dev(lens), dev(stack), dev([nfree])
        self.table = None if table is None else dev(table).reshape(B, -1)
        junk = lambda *s: torch.full(s, 12345, dtype=torch.int32, device="cuda")  # noqa: E731
        self.slots, self.positions = junk(B, q_len), junk(B, q_len)
        self.mask = None if parents is None else junk(B, q_len, (q_len + 31) // 32)
        self.lens_out = self.lens if in_place else junk(B)
        self.nfree_out = self.nfree if in_place else junk(1)
        self.status = status_word()
        self.args = (self.lens, None if new_lens is None else dev(new_lens), self.table, self.stack, self.nfree,
                     kv_rows if kv_rows is not None else len(stack) * 64, self.slots, self.positions, self.lens_out,
                     self.nfree_out, self.status)
        self.kw = dict(parents=None if parents is None else dev(parents), tree_mask=self.mask)

    def run(self):
        m.mla_cache_extend(*self.args, **self.kw)
        torch.cuda.synchronize()
        return self


def check_extend(lens, new_lens, q_len, parents=None, seed=0, in_place=False, spare=3, all_new=False):
    rng = np.random.default_rng(seed)
    max_blocks = max(ref.pages(L + q_len) for L in lens) + 1
    num = sum(ref.pages(L + n) for L, n in zip(lens, new_lens)) + spare
    table, stack, nfree = ref.paged_setup(rng, lens, max_blocks, num)
    e = Extend(lens, None if all_new else new_lens, table, stack, nfree, q_len, parents, in_place=in_place).run()
    want = ref.extend(lens, new_lens, table, stack, nfree, parents, q_len)
    assert int(e.status) == 0
    assert e.table.tolist() == want[0]
    np.testing.assert_array_equal(e.slots.cpu().numpy(), np.asarray(want[1]).reshape(len(lens), q_len))
    np.testing.assert_array_equal(e.positions.cpu().numpy(), np.asarray(want[2]).reshape(len(lens), q_len))
    if parents is not None:
        np.testing.assert_array_equal(e.mask.cpu().numpy(), ref.mask_words(want[3], q_len))
    assert e.lens_out.tolist() == want[4] and int(e.nfree_out) == want[5] and e.stack.tolist() == stack
    return e


@pytest.mark.parametrize("lens,new,q_len", [
    ([0], [1], 1), ([63], [1], 1), ([64], [1], 1), ([0, 1, 63, 64, 65, 127, 128], [4, 0, 4, 1, 3, 2, 4], 4),
    ([5, 700, 64], [200, 64, 129], 200), ([0], [0], 3), ([1000], [1000], 1000)])
@pytest.mark.parametrize("in_place", [False, True])
def test_extend_pages_and_slots(lens, new, q_len, in_place):
    check_extend(lens, new, q_len, in_place=in_place, seed=q_len)


@pytest.mark.parametrize("q_len", [1, 2, 5, 31, 32, 33, 64, 100, 1024])
@pytest.mark.parametrize("shape", ["tree", "chain", "star"])
def test_extend_tree_masks(q_len, shape):
    rng = np.random.default_rng(q_len)
    lens = [0, 77, 64]
    check_extend(lens, [q_len, (q_len + 1) // 2, q_len - 1], q_len, ref.random_parents(rng, 3, q_len, shape))


def test_extend_ignores_the_parents_of_padding():
    check_extend([10, 20], [2, 0], 4, [[-1, 0, 99, -7], [55, 55, 55, 55]])


@pytest.mark.parametrize("B,q_len", [(1, 20000), (300, 64), (1024, 9), (1025, 3), (1500, 17), (5000, 2), (3000, 70)])
def test_extend_large_batches_use_every_cta(B, q_len):
    """Above 4096 tokens the cluster grows; above 1024 sequences they are taken in chunks."""
    rng = np.random.default_rng(B)
    lens = [int(x) for x in rng.integers(0, 300, B)]
    new = [int(x) for x in rng.integers(0, q_len + 1, B)]
    for in_place in (False, True):
        check_extend(lens, new, q_len, in_place=in_place)
    if q_len <= 1024:
        check_extend(lens, new, q_len, ref.random_parents(rng, B, q_len))


def test_extend_without_new_lens_takes_q_len():
    check_extend([3, 62], [4, 4], 4, all_new=True)


def test_extend_contiguous_cache():
    e = Extend([0, 5, 96], [4, 1, 4], None, [], 0, 4, [[-1, 0, 0, 2]] * 3, kv_rows=100).run()
    assert int(e.status) == 0 and e.lens_out.tolist() == [4, 6, 100]
    assert e.slots.tolist() == [[0, 1, 2, 3], [105, -1, -1, -1], [296, 297, 298, 299]]
    assert e.positions.tolist() == [[0, 1, 1, 2], [5, -1, -1, -1], [96, 97, 97, 98]]


def unchanged(e, lens, table, nfree, code, B, q_len):
    assert int(e.status) == code
    assert e.lens_out.tolist() == lens and int(e.nfree_out) == nfree and e.table.tolist() == table
    assert (e.slots == -1).all() and (e.positions == -1).all() and e.slots.shape == (B, q_len)


@pytest.mark.parametrize("in_place", [False, True])
def test_extend_with_too_few_pages_changes_nothing(in_place):
    table = [[0, -1, -1], [1, -1, -1]]
    e = Extend([64, 64], [4, 4], table, [2, 3], 1, 4, kv_rows=256, in_place=in_place).run()
    unchanged(e, [64, 64], table, 1, PAGES, 2, 4)
    # the exact number is enough
    e = Extend([64, 64], [4, 4], table, [2, 3], 2, 4, kv_rows=256, in_place=in_place).run()
    assert int(e.status) == 0 and int(e.nfree_out) == 0 and e.table.tolist() == [[0, 3, -1], [1, 2, -1]]


@pytest.mark.parametrize("lens,nfree", [([-1, 5], 2), ([190, 5], 2), ([2 ** 31 - 1, 5], 2), ([5, 5], 3), ([5, 5], -1)])
def test_extend_refuses_bad_lengths_and_counts(lens, nfree):
    """A negative length, one past the table's 3 pages, and a page count outside the stack."""
    table = [[0, 2, 3], [1, -1, -1]]
    e = Extend(lens, [4, 4], table, [4, 5], nfree, 4, kv_rows=512).run()
    unchanged(e, lens, table, nfree, INVALID, 2, 4)


def test_extend_flags_clamped_lengths_bad_parents_and_bad_pages():
    e = Extend([5, 5], [9, -3], [[0, -1], [1, -1]], [2, 3], 2, 4, kv_rows=256).run()
    assert int(e.status) == INVALID and e.lens_out.tolist() == [9, 5]
    assert e.slots.tolist() == [[5, 6, 7, 8], [-1] * 4]
    e = Extend([5], [4], [[0]], [], 0, 4, [[-1, 0, 2, -9]], kv_rows=64).run()
    assert int(e.status) == INVALID and e.positions.tolist() == [[5, 6, 5, 5]]
    assert e.mask.tolist() == [[[1], [3], [4], [8]]]
    for bad in (-1, 4, 2 ** 31 - 1):
        e = Extend([62], [4], [[0, -1]], [bad], 1, 4, kv_rows=256).run()      # a bad page on the stack
        assert int(e.status) == BLOCK_TABLE and e.slots.tolist() == [[62, 63, -1, -1]]
        e = Extend([62], [4], [[bad, -1]], [2], 1, 4, kv_rows=256).run()      # and in the table
        assert int(e.status) == BLOCK_TABLE and e.slots.tolist() == [[-1, -1, 128, 129]]


# ------------------------------------------------------------------------------------------ append
def rope_table(max_pos, seed=0):
    a = torch.rand(max_pos, 32, generator=torch.Generator().manual_seed(seed), dtype=torch.float64) * 40 - 20
    return torch.cat([a.cos(), a.sin()], 1).float()


class Append:
    """Inputs of an append call: strided latents and queries, slots from a permutation of the pool."""

    def __init__(self, T, heads, fp8, norm=True, seed=0, max_pos=50, pad=0.2, scale=1.0):
        g = torch.Generator().manual_seed(seed)
        self.T, self.heads, self.fp8 = T, heads, fp8
        self.latent = (scale * torch.randn(T, 1536 + 576, generator=g)).bfloat16().cuda()[:, 1536:]
        self.weight = (1 + 0.2 * torch.randn(512, generator=g)).bfloat16().cuda() if norm else None
        self.table = rope_table(max_pos).cuda()
        self.rows = -(-T // 64) * 64 + 128
        pos = torch.randint(0, max_pos, (T,), generator=g)
        slots = torch.randperm(self.rows, generator=g)[:T]
        gone = torch.rand(T, generator=g) < pad
        self.positions, self.slots = torch.where(gone, -1, pos).int().cuda(), torch.where(gone, -1, slots).int().cuda()
        self.kv = torch.randint(0, 120, (self.rows // 64, 64, 576), generator=g, dtype=torch.uint8)
        if not fp8:
            self.kv = self.kv.bfloat16()
        self.kv = self.kv.cuda()
        self.kv_scale = torch.full((self.rows // 64, 64), 7.0).cuda() if fp8 else None
        self.q_rope = self.q = None
        if heads:
            self.q_rope = torch.randn(T, heads, 192, generator=g).bfloat16().cuda()[..., 128:]
            self.q = torch.full((T, heads, 576), 3.0, dtype=torch.bfloat16, device="cuda")
        self.status = status_word()

    def run(self, interleaved, eps=1e-6):
        front = (self.latent, self.weight, eps, self.table, interleaved, self.positions, self.slots, self.kv)
        if self.fp8:
            m.mla_cache_append_fp8(*front, self.kv_scale, self.status, q_rope=self.q_rope, q=self.q)
        else:
            m.mla_cache_append(*front, self.status, q_rope=self.q_rope, q=self.q)
        torch.cuda.synchronize()
        return self


# fp32 arithmetic of a row, worst case: the sum of 512 squares (512 * 2^-24), rsqrt (2^-22) and two
# products stay under 2^-14 relative; a rotated pair is off by at most 3 * 2^-24 (|x| + |y|).
NORM_REL, ROT = 2.0 ** -14, 3 * 2.0 ** -24


def check_append(a: Append, interleaved, eps=1e-6):
    kv0 = a.kv.clone()
    sc0 = None if a.kv_scale is None else a.kv_scale.clone()
    q0 = None if a.q is None else a.q.clone()
    rope0 = None if a.q_rope is None else a.q_rope.double().cpu().numpy()
    latent = a.latent.double().cpu().numpy()
    a.run(interleaved, eps)
    assert int(a.status) == 0
    pos, slots = a.positions.cpu().numpy(), a.slots.cpu().numpy()
    want = ref.append_rows(latent, None if a.weight is None else a.weight.double().cpu().numpy(), eps,
                           a.table.double().cpu().numpy(), pos, interleaved)
    live = (pos >= 0) & (slots >= 0)
    # rows that no slot names stay as they were
    touched = np.zeros(a.rows, bool)
    touched[slots[live]] = True
    flat, flat0 = a.kv.view(-1, 576), kv0.view(-1, 576)
    keep = torch.from_numpy(~touched).cuda()
    assert torch.equal(flat[keep], flat0[keep])
    mag = np.abs(latent[live][:, 512:])  # |x| + |y| of each rope column's pair
    pair = mag[:, np.arange(64) ^ 1] if interleaved else mag[:, (np.arange(64) + 32) % 64]
    abs_err = np.concatenate([np.abs(want[live][:, :512]) * NORM_REL, ROT * (mag + pair)], 1)
    if not a.fp8:
        got = flat.double().cpu().numpy()[slots[live]]
        tol = np.abs(want[live]) * 2.0 ** -8 + abs_err * (1 + 2.0 ** -8)
        assert (np.abs(got - want[live]) <= tol).all()
    else:
        scale = a.kv_scale.view(-1).double().cpu().numpy()
        assert torch.equal(a.kv_scale.view(-1)[keep], sc0.view(-1)[keep])
        amax = np.abs(want[live]).max(1)
        sc = scale[slots[live]]
        np.testing.assert_allclose(sc, amax / 448, rtol=NORM_REL + 2.0 ** -22)
        got = ref.e4m3_values()[flat.cpu().numpy()[slots[live]]] * sc[:, None]
        # half a step of the code (2^-4 relative, 2^-10 of the scale below the normal range), taken at
        # the fp32 value; the division by the scale adds 2^-23
        tol = (np.abs(want[live]) + abs_err) * (2.0 ** -4 + 2.0 ** -22) + abs_err + sc[:, None] * 2.0 ** -10
        assert (np.abs(got - want[live]) <= tol).all()
    if a.q is not None:
        qw = ref.rotate(rope0, a.table.double().cpu().numpy()[np.clip(pos, 0, None)][:, None], interleaved)
        real = pos >= 0
        if a.q_rope.data_ptr() != a.q.data_ptr() + 1024:
            assert torch.equal(a.q[..., :512], q0[..., :512])
        assert torch.equal(a.q[torch.from_numpy(~real).cuda()], q0[torch.from_numpy(~real).cuda()])
        got = a.q.view(-1, a.heads, 576)[..., 512:].double().cpu().numpy()[real]
        mag = np.abs(rope0[real])
        pair = mag[..., np.arange(64) ^ 1] if interleaved else mag[..., (np.arange(64) + 32) % 64]
        tol = np.abs(qw[real]) * 2.0 ** -8 + ROT * (mag + pair) * (1 + 2.0 ** -8)
        assert (np.abs(got - qw[real]) <= tol).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,heads,norm", [(1, 16, True), (1, 0, True), (5, 1, False), (64, 16, True), (33, 3, True),
                                          (7, 128, False), (130, 20, True), (1000, 5, True)])
def test_append(T, heads, norm, interleaved, fp8):
    check_append(Append(T, heads, fp8, norm, seed=T), interleaved)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("scale", [1e-12, 1e-3, 3e4])
def test_append_extreme_magnitudes(scale, fp8):
    check_append(Append(40, 4, fp8, norm=False, scale=scale), True)
    check_append(Append(40, 4, fp8, norm=True, scale=scale), False)


def test_append_rotates_queries_in_place():
    a = Append(50, 8, False)
    a.q = torch.randn(50, 8, 576, device="cuda").bfloat16()
    a.q_rope = a.q[..., 512:]
    for interleaved in (True, False):
        check_append(a, interleaved)


def test_append_no_tokens_and_all_padding():
    a = Append(4, 2, False, pad=1.1)
    check_append(a, True)
    z = Append(4, 2, True)
    before = z.kv.clone()
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    m.mla_cache_append_fp8(z.latent[:0], z.weight, 1e-6, z.table, True, e, e, z.kv, z.kv_scale, z.status)
    torch.cuda.synchronize()
    assert torch.equal(z.kv, before) and int(z.status) == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_append_negative_slot_still_rotates_the_query(fp8):
    a = Append(9, 3, fp8, pad=0)
    a.slots[4] = -1
    check_append(a, True)


@pytest.mark.parametrize("fp8", [False, True])
def test_append_bad_positions_and_slots_write_nothing(fp8):
    for field, value, code in (("positions", 50, INVALID), ("positions", 2 ** 31 - 1, INVALID),
                               ("slots", 10 ** 6, BLOCK_TABLE), ("slots", 2 ** 31 - 1, BLOCK_TABLE)):
        a = Append(9, 3, fp8, pad=0)
        a.slots[2] = -1 if field == "positions" else a.slots[2]
        getattr(a, field)[2] = value
        kv0, q0 = a.kv.clone(), a.q.clone()
        a.run(True)
        assert int(a.status) == code
        free = torch.ones(a.rows, dtype=torch.bool, device="cuda")
        others = a.slots[torch.arange(9) != 2]
        free[others.long()] = False
        assert torch.equal(a.kv.view(-1, 576)[free], kv0.view(-1, 576)[free])
        assert torch.equal(a.q[2], q0[2]) == (field == "positions")


def test_append_fp8_special_rows():
    """Zeros get scale 1, tiny rows the least scale, values that are not finite the NaN code."""
    a = Append(4, 0, True, norm=False, pad=0)
    a.latent[0] = 0
    a.latent[1] = 1e-38
    a.latent[2, 5], a.latent[2, 6], a.latent[2, 7] = float("inf"), float("nan"), float("-inf")
    a.table[:] = torch.cat([torch.ones(32), torch.zeros(32)])
    a.run(False)
    rows, sc = a.kv.view(-1, 576)[a.slots.long()].cpu(), a.kv_scale.view(-1)[a.slots.long()].cpu()
    assert sc[0] == 1 and int(rows[0].sum()) == 0
    assert sc[1] == 2.0 ** -100
    vals = ref.e4m3_values()[rows.numpy()]
    assert abs(vals[1, 0] * 2.0 ** -100 - float(torch.tensor(1e-38).bfloat16())) <= 2.0 ** -110
    assert np.isnan(vals[2, 5:8]).all() and np.isnan(vals[2]).sum() == 3
    x = a.latent[2].double().cpu().numpy()
    fin = np.isfinite(x)
    np.testing.assert_allclose(float(sc[2]), np.abs(x[fin]).max() / 448, rtol=2.0 ** -23)


def test_append_past_two_gib():
    """Rows of the pool past 2^31 bytes (and elements): slots near its end and its start."""
    rows = 4_000_000 // 64 * 64
    kv = torch.zeros(rows // 64, 64, 576, dtype=torch.bfloat16, device="cuda")
    a = Append(8, 2, False, pad=0)
    a.kv, a.rows = kv, rows
    assert 2 ** 31 // 576 == 2 ** 32 // 1152  # the byte border of one is the element border of the other
    a.slots = dev([rows - 1, 0, rows - 64, 2 ** 31 // 1152, 2 ** 31 // 1152 + 1, 2 ** 31 // 576,
                   2 ** 32 // 1152 + 1, 7])
    a.run(True)
    assert int(a.status) == 0
    want = ref.append_rows(a.latent.double().cpu().numpy(), a.weight.double().cpu().numpy(), 1e-6,
                           a.table.double().cpu().numpy(), a.positions.cpu().numpy(), True)
    got = kv.view(-1, 576)[a.slots.long()].double().cpu().numpy()
    assert np.abs(got - want).max() <= 2.0 ** -7 * np.abs(want).max()
    assert int((kv.view(-1, 576).abs().amax(1) > 0).sum()) == 8


# ------------------------------------------------------------------------------------------ accept
def random_path(rng, n, keep, max_path):
    return sorted(int(x) for x in rng.permutation(n)[:max(keep, 0)]) + [-5] * (max_path - max(keep, 0))


def check_accept(lens, new, keeps, max_path, fp8, seed=0, in_place=False, paged=True, junk_len=None):
    rng = np.random.default_rng(seed)
    B = len(lens)
    g = torch.Generator().manual_seed(seed)
    if paged:
        max_blocks = max(ref.pages(L) for L in lens) + 1
        num = sum(ref.pages(L) for L in lens) + 4
        table, stack, nfree = ref.paged_setup(rng, lens, max_blocks, num)
        shape = (num, 64)
    else:
        shape = (B, max(lens) + 3)
        table = None
    kv = torch.randint(0, 255, (*shape, 576), generator=g, dtype=torch.uint8)
    kv = (kv if fp8 else kv.bfloat16()).cuda()
    scale = torch.rand(shape, generator=g).cuda() if fp8 else None
    path = [random_path(rng, n, k, max_path) for n, k in zip(new, keeps)]
    kv0, sc0 = kv.clone(), None if scale is None else scale.clone()
    d_lens = dev(lens)
    out = d_lens if in_place else torch.full((B,), 99, dtype=torch.int32, device="cuda")
    status = status_word()
    d_path = dev(path).reshape(B, max_path)
    if paged:
        d_stack, d_nfree = dev(stack), dev([nfree])
        nf_out = d_nfree if in_place else dev([77])
        m.mla_cache_accept(kv, d_lens, dev(new), d_path, dev(keeps), dev(table), d_stack, d_nfree, out, nf_out,
                           status, kv_scale=scale)
        moves, want, want_stack, want_nfree = ref.accept(lens, new, path, keeps, table, stack, nfree)
        torch.cuda.synchronize()
        assert d_stack.tolist() == want_stack and int(nf_out) == want_nfree
    else:
        m.mla_cache_accept(kv, d_lens, dev(new), d_path, dev(keeps), None, None, None, out, None, status,
                           kv_scale=scale)
        big = ref.pages(shape[1])
        pages = [[b * big + i for i in range(big)] for b in range(B)]
        moves, want, _, _ = ref.accept(lens, new, path, keeps, pages, [0] * (B * big + 1), 0)
        moves = [tuple(r // (big * 64) * shape[1] + r % (big * 64) for r in mv) for mv in moves]
        torch.cuda.synchronize()
    assert int(status) == 0 and out.tolist() == want
    at = np.arange(shape[0] * shape[1])
    for src, dst in moves:
        at[dst] = src
    at = torch.from_numpy(at).cuda()
    assert torch.equal(kv.view(-1, 576), kv0.view(-1, 576)[at])
    if fp8:
        assert torch.equal(scale.view(-1), sc0.view(-1)[at])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("lens,new,keeps,max_path", [
    ([1], [1], [1], 1), ([1], [1], [0], 1), ([70], [8], [3], 4), ([64, 65, 128, 4], [4, 4, 4, 4], [1, 2, 4, 3], 4),
    ([200, 64, 300], [64, 64, 64], [20, 64, -1], 64), ([700, 900], [600, 600], [590, 17], 600),
    ([2000], [1024], [513], 1024), ([5, 0], [0, 0], [0, -1], 2), ([130, 64], [100, 3], [0, 0], 2)])
def test_accept(lens, new, keeps, max_path, paged, fp8):
    check_accept(lens, new, keeps, max_path, fp8, seed=max_path, paged=paged)
    check_accept(lens, new, keeps, max_path, fp8, seed=max_path + 1, paged=paged, in_place=True)


def test_accept_large_batches():
    rng = np.random.default_rng(4)
    B = 2500
    lens = [int(x) for x in rng.integers(9, 200, B)]
    new = [int(x) for x in rng.integers(0, 9, B)]
    keeps = [int(rng.integers(-1, n + 1)) for n in new]
    for in_place in (False, True):
        check_accept(lens, new, keeps, 8, True, in_place=in_place)


@pytest.mark.parametrize("L,n,keep,path", [
    (70, 4, 2, [1, 1]), (70, 4, 2, [2, 1]), (70, 4, 2, [-1, 1]), (70, 4, 2, [0, 4]), (70, 4, 2, [0, 2 ** 31 - 1]),
    (70, 1, 2, [0, 1]), (70, 4, 3, [0, 1]), (70, 4, -2, [0, 1]), (70, -1, 0, [0, 1]), (70, 71, 0, [0, 1]),
    (-3, 0, 0, [0, 1]), (129, 4, 1, [0, 1])])
def test_accept_leaves_a_sequence_with_a_bad_path_as_it_is(L, n, keep, path):
    kv = torch.randn(6, 64, 576, device="cuda").bfloat16()
    kv0, status, out, nf = kv.clone(), status_word(), dev([0, 0]), dev([1])
    stack = dev([5, -1, -1, -1, -1, -1])
    m.mla_cache_accept(kv, dev([L, 66]), dev([n, 3]), dev([path, [2, 0]]), dev([keep, 1]), dev([[0, 1], [2, 3]]),
                       stack, nf, out, nf, status)
    torch.cuda.synchronize()
    assert int(status) == INVALID and out.tolist() == [L, 64]
    assert int(nf) == 2 and stack.tolist() == [5, 3, -1, -1, -1, -1]  # the other sequence is served
    want = kv0.clone()
    want[2, 63] = kv0[3, 1]
    assert torch.equal(kv, want)


def test_accept_bad_pages_and_a_full_stack():
    kv = torch.zeros(4, 64, 576, device="cuda").bfloat16()
    for bad in (-1, 4, 2 ** 31 - 1):
        status, nf = status_word(), dev([0])
        m.mla_cache_accept(kv, dev([66]), dev([3]), dev([[1, 2]]), dev([2]), dev([[0, bad]]), dev([9, 9]), nf,
                           dev([0]), nf, status)
        torch.cuda.synchronize()
        assert int(status) == BLOCK_TABLE
    for count, left in ((2, 2), (1, 2), (-1, -1), (3, 3)):
        status, nf, out, stack = status_word(), dev([count]), dev([0]), dev([7, 8])
        m.mla_cache_accept(kv, dev([130]), dev([0]), dev([[0]]), dev([-1]), dev([[0, 1, 2]]), stack, nf, out, nf,
                           status)
        torch.cuda.synchronize()
        assert int(status) == INVALID and int(nf) == left and out.tolist() == [0]
        assert stack.tolist() == ([7, 0] if count == 1 else [7, 8])


# --------------------------------------------------------------------------------- streams and graphs
def test_calls_follow_their_stream():
    """On a side stream behind work that produces their inputs."""
    s = torch.cuda.Stream()
    e = Extend([64], [2], [[0, -1]], [1], 1, 2, kv_rows=128)
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        e.lens.fill_(63)
        m.mla_cache_extend(*e.args)
    torch.cuda.synchronize()
    assert e.slots.tolist() == [[63, 64]]
    e = Extend([64], [2], [[0, -1]], [1], 1, 2, kv_rows=128)
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        e.lens.fill_(63)
    m.mla_cache_extend(*e.args, stream=s)
    torch.cuda.synchronize()
    assert e.slots.tolist() == [[63, 64]]


def test_captured_calls_replay_on_new_inputs():
    """extend, append and accept in one graph, in place: each replay is one more step."""
    a = Append(4, 2, True, pad=0)
    a.kv = torch.zeros(8, 64, 576, dtype=torch.uint8, device="cuda")
    a.kv_scale = torch.zeros(8, 64, device="cuda")
    lens, nfree, table = dev([126, 3]), dev([5]), dev([[0, 1, -1, -1], [2, -1, -1, -1]])
    stack = dev([3, 4, 5, 6, 7, -1, -1, -1])
    new, path, keep = dev([2, 2]), dev([[1], [0]]), dev([1, 1])
    slots, pos = torch.zeros(2, 2, dtype=torch.int32, device="cuda"), torch.zeros(2, 2, dtype=torch.int32, device="cuda")
    pos_flat, slots_flat = pos.view(-1), slots.view(-1)
    a.table = rope_table(512).cuda()

    def step():
        m.mla_cache_extend(lens, new, table, stack, nfree, 512, slots, pos, lens, nfree, a.status)
        m.mla_cache_append_fp8(a.latent, a.weight, 1e-6, a.table, True, pos_flat, slots_flat, a.kv, a.kv_scale,
                               a.status, q_rope=a.q_rope, q=a.q)
        m.mla_cache_accept(a.kv, lens, new, path, keep, table, stack, nfree, lens, nfree, a.status,
                           kv_scale=a.kv_scale)

    step()
    torch.cuda.synchronize()
    assert lens.tolist() == [127, 4]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    assert lens.tolist() == [127, 4]  # captured, not run
    for k in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert lens.tolist() == [128 + k, 5 + k] and int(a.status) == 0
    assert table.tolist()[0][:3] == [0, 1, 7] and int(nfree) == 4
    # row 127 of sequence 0 was appended by the second token of its step and moved down by one
    assert int(a.kv_scale[1, 63].count_nonzero()) == 1
