"""The speculative-verify operators over the latent cache: workloads, plain forms and 64-bit values.

One serving step with a tree of drafted tokens runs four operators in this order:

* extend: pages, row slots, positions and ancestor masks of the new tokens, from the request lengths;
* append: RMS norm of the new latents, rotation of the key's and the queries' rope columns, rows stored
  into the bf16 or E4M3 cache at their slots;
* tree:   attention of the drafted tokens over the cache, each seeing the context and its own ancestors;
* accept: the accepted path's rows moved behind the context, the rest dropped, pages handed back.

``run`` computes one of them, in its plain form (elementary torch operations) or, with ``own`` set,
through the package's entry points.  ``exact`` computes the same from the definitions in 64 bits.
"""

from __future__ import annotations

import math

import torch

own = False

D_QK, D_V, D_ROPE, PAGE = 576, 512, 64, 64
E4M3_MAX = 448.0
SCALE = 1.0 / math.sqrt(D_QK)
EPS = 1e-6


# ------------------------------------------------------------------------------------------- cases
def _extend(name, batch, q_len, lo, hi, tree, ragged):
    return dict(name=name, op="extend", batch=batch, q_len=q_len, lo=lo, hi=hi, tree=tree, ragged=ragged)


def _append(name, batch, q_len, heads, kv, interleaved, ragged):
    return dict(name=name, op="append", batch=batch, q_len=q_len, heads=heads, kv=kv, interleaved=interleaved,
                ragged=ragged)


def _tree(name, batch, heads, q_len, lo, hi, kv, paged, ragged, spikes=False):
    return dict(name=name, op="tree", batch=batch, heads=heads, q_len=q_len, lo=lo, hi=hi, kv=kv, paged=paged,
                ragged=ragged, spikes=spikes)


def _accept(name, batch, q_len, keep, lo, hi, kv):
    return dict(name=name, op="accept", batch=batch, q_len=q_len, keep=keep, lo=lo, hi=hi, kv=kv)


def listed():
    return [
        # the bookkeeping of one verify step of the q_len = 4 decode: 64 new rows, latency only
        _extend("extend_verify_b16_q4", 16, 4, 1, 32768, True, False),
        # a chunk of up to 2048 prompt tokens for each of 32 requests: many new pages, no tree
        _extend("extend_prompt_b32_q2048", 32, 2048, 0, 30000, False, True),
        # the new rows of that verify step: 64 tokens of 16 heads into the bf16 cache
        _append("append_verify_b16_q4_h16", 16, 4, 16, "bf16", False, False),
        # a prompt chunk into the E4M3 cache (keys only: the queries of a prompt do not run the decode)
        _append("append_prompt_e4m3_t8192", 4, 2048, 0, "e4m3", True, False),
        # many ragged requests with all 128 heads on one GPU: the queries' rope columns dominate
        _append("append_b256_q16_h128", 256, 16, 128, "bf16", True, True),
        # one short request with 8 drafted tokens: latency
        _tree("tree_b1_h16_l1024_q8", 1, 16, 8, 1024, 1024, "bf16", False, False),
        # the q_len = 4 verify shape on a contiguous cache, 5% of the rows scaled x8
        _tree("tree_b16_h16_l32k_q4", 16, 16, 4, 32768, 32768, "bf16", False, False, True),
        # ragged trees of up to 16 tokens over very unequal paged requests
        _tree("tree_b16_h16_q16_ragged", 16, 16, 16, 1, 32768, "bf16", True, True),
        # the verify shape on the E4M3 cache
        _tree("tree_e4m3_b16_h16_q4", 16, 16, 4, 16384, 32768, "e4m3", True, False),
        # all 128 heads on one GPU: 512 query columns a request, bound by the tensor cores
        _tree("tree_b8_h128_q4", 8, 128, 4, 8192, 32768, "bf16", True, False),
        # the end of a verify step: at most 4 of 4 drafted tokens kept, E4M3 cache
        _accept("accept_e4m3_b16_q4", 16, 4, 4, 4, 32768, "e4m3"),
        # wide trees: up to 16 of 64 drafted tokens kept, many pages handed back
        _accept("accept_b64_q64", 64, 64, 16, 64, 4000, "bf16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("extend", "append", "tree", "tree", "accept"))
    kv = rng.choice(("bf16", "e4m3"))
    if op == "extend":
        tree = rng.random() < 0.6
        q_len = _log(rng, 1, 128) if tree else _log(rng, 1, 2048)
        c = _extend("", _log(rng, 1, 256 if q_len <= 256 else 32), q_len, 0, _log(rng, 64, 32768), tree,
                    rng.random() < 0.5)
    elif op == "append":
        q_len = _log(rng, 1, 2048)
        c = _append("", _log(rng, 1, 2048 // q_len), q_len, rng.choice((0, 1, 5, 8, 16, 32, 64, 128)), kv,
                    rng.random() < 0.5, rng.random() < 0.5)
    elif op == "tree":
        heads = rng.choice((1, 3, 8, 16, 16, 20, 64, 128))
        q_len = _log(rng, 1, max(1, min(64, 512 // heads)))
        batch = _log(rng, 1, 32)
        hi = _log(rng, 64, min(32768, 16 * 32768 // batch, 80_000_000 // (batch * heads * q_len)))
        lo = rng.choice((1, (hi + 1) // 2, hi))
        paged = rng.random() < 0.7
        c = _tree("", batch, heads, q_len, max(lo, min(q_len, hi)), max(hi, q_len), kv, paged, rng.random() < 0.5,
                  rng.random() < 0.3)
    else:
        q_len = _log(rng, 1, 64)
        c = _accept("", _log(rng, 1, 64), q_len, rng.randint(1, min(16, q_len)), q_len, _log(rng, 128, 4000), kv)
    del c["name"]
    return c


# ------------------------------------------------------------------------------------------ inputs
def _lens(g, batch, lo, hi):
    return torch.randint(lo, hi + 1, (batch,), generator=g, device="cuda").int()


def _ragged(g, c):
    if not c["ragged"]:
        return None
    return _lens(g, c["batch"], 1, c["q_len"])


def _parents(g, batch, q_len):
    """A random tree over each request's drafted tokens: parents[t] < t, or -1 behind the context."""
    t = torch.arange(q_len, device="cuda")
    u = torch.rand(batch, q_len, generator=g, device="cuda", dtype=torch.float64)
    return (torch.minimum((u * (t + 1)).long(), t) - 1).int()


def _sees(parents):
    """bool [B, q_len, q_len]: token t sees drafted token u (itself and its ancestors)."""
    batch, q_len = parents.shape
    u = torch.arange(q_len, device=parents.device)
    sees = ((parents[:, :, None] == u) | (u[:, None] == u)).float()
    for _ in range(q_len.bit_length()):  # paths of length 1, 2, 4, ...
        sees = (torch.bmm(sees, sees) > 0).float()
    return sees > 0


def _pack(sees):
    """bool [B, q_len, q_len] -> int32 words [B, q_len, ceil(q_len / 32)], bit u % 32 of word u / 32."""
    batch, q_len, _ = sees.shape
    words = -(-q_len // 32)
    bits = torch.zeros(batch, q_len, words * 32, dtype=torch.int64, device=sees.device)
    bits[:, :, :q_len] = sees.long()
    w = (bits.view(batch, q_len, words, 32) << torch.arange(32, device=sees.device)).sum(-1)
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).int()


def _unpack(mask, q_len):
    bits = (mask.long()[..., None] >> torch.arange(32, device=mask.device)) & 1
    return bits.flatten(-2)[..., :q_len] > 0


def _page_table(g, lens, max_blocks, num_blocks):
    """Pages drawn from a permutation of the pool, in request order; unused entries are -1."""
    pages = torch.randperm(num_blocks, generator=g, device="cuda").int()
    need = (lens.long() + PAGE - 1) // PAGE
    first = need.cumsum(0) - need
    i = torch.arange(max_blocks, device="cuda")
    at = (first[:, None] + i).clamp(max=num_blocks - 1)
    table = torch.where(i < need[:, None], pages[at], -1).int().contiguous()
    left = pages[int(need.sum()):]
    return table, left


def _free_stack(left, num_blocks):
    stack = torch.full((num_blocks,), -1, dtype=torch.int32, device="cuda")
    stack[:left.numel()] = left
    return stack, torch.tensor([left.numel()], dtype=torch.int32, device="cuda")


def _rope_table(max_pos):
    inv = 10000.0 ** (-torch.arange(0, D_ROPE, 2, device="cuda", dtype=torch.float64) / D_ROPE)
    a = torch.arange(max_pos, device="cuda", dtype=torch.float64)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float().contiguous()


def _cache(g, shape, kv):
    """A cache of N(0, 1) rows: (bf16 rows, None) or (E4M3 codes, row scales)."""
    x = torch.randn(*shape, D_QK, generator=g, device="cuda", dtype=torch.bfloat16)
    if kv == "bf16":
        return x, None
    scale = x.abs().amax(-1).float() / E4M3_MAX
    codes = (x / scale[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes.contiguous(), scale.contiguous()


def _status():
    return torch.zeros(64, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    B, q = c["batch"], c["q_len"]
    s = dict(case=c, status=_status())
    if c["op"] == "extend":
        max_blocks = (c["hi"] + q + PAGE - 1) // PAGE
        lens = _lens(g, B, c["lo"], c["hi"])
        num_blocks = B * max_blocks
        table, left = _page_table(g, lens, max_blocks, num_blocks)
        stack, nfree = _free_stack(left, num_blocks)
        i32 = lambda *n: torch.zeros(*n, dtype=torch.int32, device="cuda")  # noqa: E731
        s.update(seqlens=lens, new_lens=_ragged(g, c), table=table, stack=stack, nfree=nfree,
                 kv_rows=num_blocks * PAGE, slots=i32(B, q), positions=i32(B, q), seqlens_out=i32(B),
                 nfree_out=i32(1), parents=_parents(g, B, q) if c["tree"] else None,
                 mask=i32(B, q, -(-q // 32)) if c["tree"] else None)
    elif c["op"] == "append":
        T, h = B * q, c["heads"]
        n = _ragged(g, c)
        # the latents are the last columns of a wider projection's output; the slots a permutation of the pool
        proj = torch.randn(T, 1536 + D_QK, generator=g, device="cuda", dtype=torch.bfloat16)
        rows = -(-T // PAGE) * PAGE + 8 * PAGE
        slots = torch.randperm(rows, generator=g, device="cuda")[:T].int().view(B, q)
        t = torch.arange(q, device="cuda")
        positions = (_lens(g, B, 0, 32768)[:, None] + t).int()
        if n is not None:
            slots = torch.where(t < n[:, None], slots, -1)
            positions = torch.where(t < n[:, None], positions, -1)
        kv, scale = _cache(g, (rows // PAGE, PAGE), c["kv"])
        s.update(latent=proj[:, 1536:], weight=1 + 0.1 * torch.randn(D_V, generator=g, device="cuda").bfloat16(),
                 table=_rope_table(32768 + 2048), positions=positions.contiguous().view(-1),
                 slots=slots.contiguous().view(-1), kv=kv, kv_scale=scale, q_rope=None, q=None)
        if h:
            qp = torch.randn(T, h, 128 + D_ROPE, generator=g, device="cuda", dtype=torch.bfloat16)
            s.update(q_rope=qp[..., 128:],
                     q=torch.randn(T, h, D_QK, generator=g, device="cuda", dtype=torch.bfloat16))
    elif c["op"] == "tree":
        h = c["heads"]
        lens = _lens(g, B, c["lo"], c["hi"])
        n = _ragged(g, c)
        lens = torch.maximum(lens, torch.full_like(lens, q) if n is None else n)
        table = None
        if c["paged"]:
            max_blocks = (max(c["hi"], q) + PAGE - 1) // PAGE
            num_blocks = int(((lens.long() + PAGE - 1) // PAGE).sum()) + 3
            table, _ = _page_table(g, lens, max_blocks, num_blocks)
            kv, scale = _cache(g, (num_blocks, PAGE), c["kv"])
        else:
            kv, scale = _cache(g, (B, max(c["hi"], q)), c["kv"])
        if c["spikes"]:
            big = torch.rand(kv.shape[:2], generator=g, device="cuda") < 0.05
            if scale is None:
                kv = torch.where(big[..., None], kv * 8, kv)
            else:
                scale = torch.where(big, scale * 8, scale)
        s.update(q=torch.randn(B, q, h, D_QK, generator=g, device="cuda", dtype=torch.bfloat16), kv=kv,
                 kv_scale=scale, seqlens=lens, q_lens=n, table=table, mask=_pack(_sees(_parents(g, B, q))),
                 o=torch.zeros(B, q, h, D_V, dtype=torch.bfloat16, device="cuda"),
                 lse=torch.zeros(B, q, h, dtype=torch.float32, device="cuda"))
        if own:  # the workspace that a serving loop keeps
            from mla_decode_attention_etap_b200 import MlaDecoder
            s.update(dec=MlaDecoder(B, q, h, device="cuda"))
    else:
        lens = _lens(g, B, c["lo"], max(c["lo"], c["hi"]))
        max_blocks = (max(c["lo"], c["hi"]) + PAGE - 1) // PAGE
        num_blocks = B * max_blocks
        table, left = _page_table(g, lens, max_blocks, num_blocks)
        stack, nfree = _free_stack(left, num_blocks)
        kv, scale = _cache(g, (num_blocks, PAGE), c["kv"])
        # an accepted path: an increasing choice among the drafted tokens; one request in 16 has finished
        P = c["keep"]
        kept = _lens(g, B, 1, P)
        rank = torch.rand(B, q, generator=g, device="cuda").argsort(-1).argsort(-1)
        t = torch.arange(q, device="cuda")
        path = torch.where(rank < kept[:, None], t, q).sort(-1).values[:, :P]
        path = torch.where(path < q, path, -1).int().contiguous()
        kept = torch.where(torch.rand(B, generator=g, device="cuda") < 1 / 16, -1, kept).int()
        s.update(kv=kv, kv_scale=scale, seqlens=lens, new_lens=torch.full_like(lens, q), path=path, path_lens=kept,
                 table=table, stack=stack, nfree=nfree, seqlens_out=torch.zeros_like(lens),
                 nfree_out=torch.zeros_like(nfree))
    return s


# ------------------------------------------------------------------------------------- plain forms
def _plain_extend(s):
    c = s["case"]
    q, table, stack = c["q_len"], s["table"], s["stack"]
    L = s["seqlens"].long()
    n = torch.full_like(L, q) if s["new_lens"] is None else s["new_lens"].long()
    have, want = (L + PAGE - 1) // PAGE, (L + n + PAGE - 1) // PAGE
    need = want - have
    first = need.cumsum(0) - need
    i = torch.arange(q // PAGE + 2, device=L.device)
    page, new = have[:, None] + i, i < need[:, None]
    b = torch.arange(L.numel(), device=L.device)[:, None].expand_as(page)
    taken = stack[(s["nfree"].long() - 1 - first[:, None] - i).clamp(min=0)]
    table[b[new], page[new]] = taken[new]
    t = torch.arange(q, device=L.device)
    row, real = L[:, None] + t, t < n[:, None]
    blk = table.gather(1, (row // PAGE).clamp(max=table.shape[1] - 1)).long()
    slots = torch.where(real, blk * PAGE + row % PAGE, -1).int()
    out = [table, slots, (L + n).int(), (s["nfree"] - need.sum()).int()]
    if s["parents"] is None:
        return out + [torch.where(real, row, -1).int()]
    sees = _sees(s["parents"])
    return out + [torch.where(real, L[:, None] + sees.sum(-1) - 1, -1).int(), _pack(sees & real[:, :, None])]


def _rotate(x, cs, interleaved):
    """Rotate the 64 columns of x (32 bits) by the angles whose cosines and sines are cs [T, 64]."""
    cos, sin = cs[..., :32], cs[..., 32:]
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    a, b = x[..., :32], x[..., 32:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _plain_append(s):
    c = s["case"]
    live = s["positions"] >= 0
    cs = s["table"][s["positions"].clamp(min=0).long()]
    x = s["latent"].float()
    lat = x[:, :D_V]
    lat = lat / torch.sqrt((lat * lat).mean(-1, keepdim=True) + EPS) * s["weight"].float()
    row = torch.cat([lat, _rotate(x[:, D_V:], cs, c["interleaved"])], 1)[live]
    at = s["slots"][live].long()
    if c["kv"] == "bf16":
        s["kv"].view(-1, D_QK)[at] = row.bfloat16()
        out = [s["kv"]]
    else:
        scale = row.abs().amax(-1) / E4M3_MAX
        codes = (row / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        s["kv"].view(-1, D_QK)[at] = codes.view(torch.uint8)
        s["kv_scale"].view(-1)[at] = scale
        out = [s["kv"].view(torch.float8_e4m3fn), s["kv_scale"]]
    if s["q"] is None:
        return out
    s["q"][..., D_V:][live] = _rotate(s["q_rope"].float(), cs[:, None], c["interleaved"]).bfloat16()[live]
    return out + [s["q"]]


def _plain_tree(s):
    c = s["case"]
    B, q, h = c["batch"], c["q_len"], c["heads"]
    k = s["kv"].float() if s["kv_scale"] is None else (
        s["kv"].view(torch.float8_e4m3fn).float() * s["kv_scale"][..., None])
    if s["table"] is not None:
        k = k[s["table"].clamp(min=0).long()].flatten(1, 2)
    x = torch.bmm(s["q"].float().view(B, q * h, D_QK), k.transpose(1, 2)).view(B, q, h, -1) * SCALE
    L = s["seqlens"].long()[:, None, None]
    n = torch.full_like(L, q) if s["q_lens"] is None else s["q_lens"].long()[:, None, None]
    j, t = torch.arange(k.shape[1], device=k.device), torch.arange(q, device=k.device)[:, None]
    u = j - (L - n)  # the drafted token in cache row j
    sees = _unpack(s["mask"], q).gather(2, u.clamp(0, q - 1).expand(B, q, -1))
    vis = ((j < L) & (t < n) & ((u < 0) | sees))[:, :, None]
    x = torch.where(vis, x, -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    o = torch.bmm(p.view(B, q * h, -1), k[..., :D_V]).view(B, q, h, D_V)
    o = torch.where(total > 0, o / torch.where(total > 0, total, 1.0), 0.0)
    return [o.bfloat16(), (top + torch.log(total))[..., 0]]


def _plain_accept(s):
    table, path = s["table"], s["path"].long()
    L, n, keep = s["seqlens"].long(), s["new_lens"].long(), s["path_lens"].long()
    ctx = L - n
    i = torch.arange(path.shape[1], device=L.device)
    moved = i < keep[:, None]
    b = torch.arange(L.numel(), device=L.device)[:, None].expand_as(path)[moved]
    src, dst = (ctx[:, None] + path)[moved], (ctx[:, None] + i)[moved]
    src = table[b, src // PAGE].long() * PAGE + src % PAGE
    dst = table[b, dst // PAGE].long() * PAGE + dst % PAGE
    flat = s["kv"].view(-1, D_QK)
    flat[dst] = flat[src]
    out = [s["kv"]]
    if s["kv_scale"] is not None:
        sc = s["kv_scale"].view(-1)
        sc[dst] = sc[src]
        out = [s["kv"].view(torch.float8_e4m3fn), s["kv_scale"]]
    new_len = torch.where(keep < 0, 0, ctx + keep)
    have, want = (L + PAGE - 1) // PAGE, (new_len + PAGE - 1) // PAGE
    p = torch.arange(table.shape[1], device=L.device)
    back = table[(p >= want[:, None]) & (p < have[:, None])]
    stack = s["stack"]
    stack[s["nfree"].long() + torch.arange(back.numel(), device=L.device)] = back
    return out + [stack, new_len.int(), s["nfree"] + back.numel()]


# --------------------------------------------------------------------------- the package's own calls
def _own(s):
    import mla_decode_attention_etap_b200 as mla

    c = s["case"]
    if c["op"] == "extend":
        mla.mla_cache_extend(s["seqlens"], s["new_lens"], s["table"], s["stack"], s["nfree"], s["kv_rows"],
                             s["slots"], s["positions"], s["seqlens_out"], s["nfree_out"], s["status"],
                             parents=s["parents"], tree_mask=s["mask"])
        out = [s["table"], s["slots"], s["seqlens_out"], s["nfree_out"], s["positions"]]
        return out if s["mask"] is None else out + [s["mask"]]
    if c["op"] == "append":
        if c["kv"] == "bf16":
            mla.mla_cache_append(s["latent"], s["weight"], EPS, s["table"], c["interleaved"], s["positions"],
                                 s["slots"], s["kv"], s["status"], q_rope=s["q_rope"], q=s["q"])
            out = [s["kv"]]
        else:
            mla.mla_cache_append_fp8(s["latent"], s["weight"], EPS, s["table"], c["interleaved"], s["positions"],
                                     s["slots"], s["kv"], s["kv_scale"], s["status"], q_rope=s["q_rope"], q=s["q"])
            out = [s["kv"].view(torch.float8_e4m3fn), s["kv_scale"]]
        return out if s["q"] is None else out + [s["q"]]
    if c["op"] == "tree":
        s["dec"].plan(s["seqlens"])
        if c["kv"] == "bf16":
            s["dec"].fwd_tree(s["q"], s["kv"], s["seqlens"], s["mask"], block_table=s["table"], softmax_scale=SCALE,
                              o=s["o"], lse=s["lse"], q_lens=s["q_lens"])
        else:
            s["dec"].fwd_tree_fp8(s["q"], s["kv"], s["kv_scale"], s["seqlens"], s["mask"], block_table=s["table"],
                                  softmax_scale=SCALE, o=s["o"], lse=s["lse"], q_lens=s["q_lens"])
        return [s["o"], s["lse"]]
    mla.mla_cache_accept(s["kv"], s["seqlens"], s["new_lens"], s["path"], s["path_lens"], s["table"], s["stack"],
                         s["nfree"], s["seqlens_out"], s["nfree_out"], s["status"], kv_scale=s["kv_scale"])
    out = [s["kv"]] if s["kv_scale"] is None else [s["kv"].view(torch.float8_e4m3fn), s["kv_scale"]]
    return out + [s["stack"], s["seqlens_out"], s["nfree_out"]]


def run(state):
    if own:
        return _own(state)
    return {"extend": _plain_extend, "append": _plain_append, "tree": _plain_tree,
            "accept": _plain_accept}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------------- work
def work(case):
    """Inputs read once, outputs written once; random lengths count with their means."""
    c = case
    B, q = c["batch"], c["q_len"]
    row = D_QK * 2 if c.get("kv") == "bf16" else D_QK + 4
    n = (1 + q) / 2 if c.get("ragged") else q
    if c["op"] == "extend":
        words = -(-q // 32)
        tree = B * q * 4 * (1 + words) if c["tree"] else 0
        # lengths in and out, new pages from the stack into the table, the last page read, slots and positions
        return {"bytes": B * 12 + B * (n / PAGE) * 8 + B * 4 + 2 * B * q * 4 + tree + 8, "flops": 0}
    if c["op"] == "append":
        T = B * n
        one = D_QK * 2 + row + 8 + D_ROPE * 4 + c["heads"] * D_ROPE * 4
        return {"bytes": T * one + D_V * 2, "flops": T * (4 * D_V + 6 * 32 * (1 + c["heads"]))}
    if c["op"] == "tree":
        h = c["heads"]
        L = max((c["lo"] + c["hi"]) / 2, q)
        io = B * q * h * (D_QK * 2 + D_V * 2 + 4) + B * q * -(-q // 32) * 4
        return {"bytes": B * L * row + io, "flops": B * L * n * h * 2 * (D_QK + D_V)}
    keep = (1 + c["keep"]) / 2 * 15 / 16
    back = B * ((q - keep) / PAGE + (c["lo"] + c["hi"]) / 2 / PAGE / 16)
    return {"bytes": B * (keep * (2 * row + 4) + 16) + back * 8, "flops": 0}


# ------------------------------------------------------------------------------------ 64-bit values
def _exact_extend(s):
    q = s["case"]["q_len"]
    table, stack = s["table"].tolist(), s["stack"].tolist()
    lens = s["seqlens"].tolist()
    new = [q] * len(lens) if s["new_lens"] is None else s["new_lens"].tolist()
    parents = None if s["parents"] is None else s["parents"].tolist()
    top, slots, positions, masks = int(s["nfree"]), [], [], []
    for b, L in enumerate(lens):
        slots.append([-1] * q)
        positions.append([-1] * q)
        masks.append([[0] * -(-q // 32) for _ in range(q)])
        for p in range((L + PAGE - 1) // PAGE, (L + new[b] + PAGE - 1) // PAGE):
            top -= 1
            table[b][p] = stack[top]
        for t in range(q):
            up, depth = t if t < new[b] else -1, -1
            while parents is not None and up >= 0:
                w = masks[b][t][up // 32] | 1 << up % 32
                masks[b][t][up // 32] = w
                up, depth = parents[b][up], depth + 1
            if t < new[b]:
                slots[b][t] = table[b][(L + t) // PAGE] * PAGE + (L + t) % PAGE
                positions[b][t] = L + (t if parents is None else depth)
    i32 = lambda v: torch.tensor(v, dtype=torch.int64, device="cuda").to(torch.int32)  # noqa: E731
    out = [i32(table), i32(slots), i32([a + b for a, b in zip(lens, new)]), i32([top]), i32(positions)]
    if parents is None:
        return out
    words = torch.tensor(masks, dtype=torch.int64, device="cuda")
    return out + [((words + 2 ** 31) % 2 ** 32 - 2 ** 31).to(torch.int32)]


def _exact_append(s):
    c = s["case"]
    pos, at = s["positions"].long(), s["slots"].long()
    real = (pos >= 0).nonzero()[:, 0]
    angle = s["table"].double()[pos[real]]  # the cosines and sines are inputs
    turn = torch.complex(angle[:, :32], angle[:, 32:])

    def turned(x):  # [..., 64] as 32 complex numbers, multiplied by the unit numbers of the angles
        z = torch.view_as_complex((x.unflatten(-1, (32, 2)) if c["interleaved"]
                                   else x.unflatten(-1, (2, 32)).transpose(-1, -2)).contiguous())
        y = torch.view_as_real(z * (turn if x.dim() == 2 else turn[:, None]))
        return (y if c["interleaved"] else y.transpose(-1, -2)).flatten(-2)

    x = s["latent"][real].double()
    norm = x[:, :D_V].pow(2).mean(1).add(EPS).rsqrt()
    rows = torch.empty_like(x)
    rows[:, :D_V] = x[:, :D_V] * norm[:, None] * s["weight"].double()
    rows[:, D_V:] = turned(x[:, D_V:])
    if c["kv"] == "bf16":
        pool = s["kv"].double().view(-1, D_QK)
        pool[at[real]] = rows
        out = [pool.view(s["kv"].shape)]
    else:
        scale = rows.abs().max(1).values / E4M3_MAX
        y = rows / scale[:, None]
        # the nearest E4M3 value: a step of 2^(e - 3) in [2^e, 2^(e+1)), never under 2^-9
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
        pool = s["kv"].view(torch.float8_e4m3fn).double().view(-1, D_QK)
        pool[at[real]] = (torch.round(y / step) * step).clamp(-E4M3_MAX, E4M3_MAX)
        scales = s["kv_scale"].double().view(-1)
        scales[at[real]] = scale
        out = [pool.view(s["kv"].shape), scales.view(s["kv_scale"].shape)]
    if s["q"] is None:
        return out
    q = s["q"].double()
    q[real, :, D_V:] = turned(s["q_rope"][real].double())
    return out + [q]


def _exact_tree(s):
    c = s["case"]
    B, q, h = c["batch"], c["q_len"], c["heads"]
    o = torch.zeros(B, q, h, D_V, dtype=torch.float64, device="cuda")
    lse = torch.full((B, q, h), -math.inf, dtype=torch.float64, device="cuda")
    for b, L in enumerate(s["seqlens"].tolist()):
        n = q if s["q_lens"] is None else int(s["q_lens"][b])
        if s["table"] is None:
            pick = lambda x: x[b, :L]  # noqa: E731
        else:
            blocks = s["table"][b, :(L + PAGE - 1) // PAGE].long()
            pick = lambda x: x[blocks].flatten(0, 1)[:L]  # noqa: E731
        if s["kv_scale"] is None:
            k = pick(s["kv"]).double()
        else:
            k = pick(s["kv"]).view(torch.float8_e4m3fn).double() * pick(s["kv_scale"]).double()[:, None]
        hide = torch.zeros(n, L, dtype=torch.bool, device="cuda")
        u = torch.arange(n, device="cuda")
        hide[:, L - n:] = (s["mask"][b, :n].long()[:, u // 32] // 2 ** (u % 32)) % 2 == 0
        x = (s["q"][b, :n].double().flatten(0, 1) @ k.T / math.sqrt(D_QK)).view(n, h, L)
        x = x.masked_fill(hide[:, None], -math.inf)
        lse[b, :n] = torch.logsumexp(x, -1)
        o[b, :n] = (torch.softmax(x, -1).flatten(0, 1) @ k[:, :D_V]).view(n, h, D_V)
    return [o, lse]


def _exact_accept(s):
    table, path = s["table"].tolist(), s["path"].tolist()
    stack, top = s["stack"].tolist(), int(s["nfree"])
    src, dst, lens = [], [], []
    for b, (L, n, keep) in enumerate(zip(s["seqlens"].tolist(), s["new_lens"].tolist(), s["path_lens"].tolist())):
        end = 0 if keep < 0 else L - n + keep
        for i in range(max(keep, 0)):
            for rows, r in ((src, L - n + path[b][i]), (dst, L - n + i)):
                rows.append(table[b][r // PAGE] * PAGE + r % PAGE)
        for p in range((end + PAGE - 1) // PAGE, (L + PAGE - 1) // PAGE):
            stack[top] = table[b][p]
            top += 1
        lens.append(end)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    at = torch.arange(s["kv"].shape[0] * PAGE, device="cuda")
    at[i32(dst).long()] = i32(src).long()
    kv = s["kv"] if s["kv_scale"] is None else s["kv"].view(torch.float8_e4m3fn)
    out = [kv.double().view(-1, D_QK)[at].view(kv.shape)]
    if s["kv_scale"] is not None:
        out.append(s["kv_scale"].double().view(-1)[at].view(s["kv_scale"].shape))
    return out + [i32(stack), i32(lens), i32([top])]


def exact(case, seed):
    s = prepare(case, seed)
    return {"extend": _exact_extend, "append": _exact_append, "tree": _exact_tree, "accept": _exact_accept}[
        case["op"]](s)
