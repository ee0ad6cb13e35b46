// The steps around the decode that keep its latent cache: pages, slots and masks of new tokens
// (extend_kernel), their rows and rotated queries (append_kernel), and the accepted path of a verified tree
// (accept_kernel; accept_rows_kernel with accept_pages_kernel).  No kernel here waits on another CTA except through the
// hardware cluster barrier; every index read from memory is checked before it is used.
#pragma once

#include <cuda_bf16.h>
#include <cstdint>

#include "block_scan.cuh"
#include "etap_common.cuh"
#include "plan_core.h"
#include "ptx_sm100.cuh"

namespace mla {

constexpr int kStatusPages = -8;  // MLA_ERR_PAGES
constexpr int kCacheThreads = 1024;

__device__ __forceinline__ void raise_status(int32_t *status, int code) { atomicCAS(status, 0, code); }
__device__ __forceinline__ int pages_of(int64_t rows) { return (int)((rows + kPage - 1) / kPage); }

// ------------------------------------------------------------------------------------------ extend
struct ExtendParams {
    const int32_t *seqlens, *new_lens, *parents;
    int32_t *block_table;  // or NULL: contiguous cache of kv_rows rows a sequence
    const int32_t *free_pages, *num_free;
    int32_t *slots, *positions, *tree_mask, *seqlens_out, *num_free_out, *status;
    int64_t kv_rows;
    int batch, q_len, max_blocks, free_capacity, tree_words;
    int vector_out;  // slots and positions may be stored four at a time
};

// One cluster of up to 8 CTAs.  Every CTA computes the page offsets of all sequences (a prefix sum of
// the pages each needs), then, once all have read the lengths (the cluster barrier, so that lengths and
// the page count may be updated in place), writes its share.  Sequences are taken kCacheThreads at a
// time; a batch that fits one such chunk is read once, and its tokens are dealt over all CTAs.
// A thread handles TOKENS neighbouring tokens at a time: 4 for many tokens (their lookups in flight
// together and stored as one; 65536 tokens took 8.2 us with one each and 5.5 us with four), 1 for few
// (64 tokens of a tree: 3.6 us against 4.9 us, the walks of a thread's tokens running one by one).
// What bounds it is the chain launch, lengths, sums, barrier, page, stores: 65536 tokens write 0.5 MB, 0.08 us
// of the measured copy bandwidth.  With parents it is the depth: each token follows its own ancestors, a dependent
// load a step.  Random trees are shallow (16 x 128 tokens: 8.7 us); chains of 4, 64, 128 tokens in 16 sequences take
// 3.7, 16 and 62 us, one chain of 1024 tokens 213.  (Times replayed from a graph.)
template <int TOKENS>
__global__ void __launch_bounds__(kCacheThreads) extend_kernel(const __grid_constant__ ExtendParams p) {
    __shared__ int64_t scan_smem[32];
    __shared__ int s_len[kCacheThreads], s_new[kCacheThreads], s_first[kCacheThreads];
    const int tid = threadIdx.x;
    const int rank = (int)blockIdx.x, ctas = (int)gridDim.x;
    const bool paged = p.block_table != nullptr;
    const int64_t cap = paged ? (int64_t)p.max_blocks * kPage : p.kv_rows;
    bool bad = false;  // a length this call cannot take: nothing is changed
    // length and new tokens of sequence b, and the pages it needs
    auto read = [&](int b, int &L, int &n) -> int {
        L = p.seqlens[b];
        n = p.new_lens ? p.new_lens[b] : p.q_len;
        if (n < 0 || n > p.q_len) {
            if (rank == 0) raise_status(p.status, kStatusInvalid);
            n = n < 0 ? 0 : p.q_len;
        }
        if (L < 0 || (int64_t)L + n > cap) {
            bad = true;
            return 0;
        }
        return paged ? pages_of((int64_t)L + n) - pages_of(L) : 0;
    };
    // Mask words of new token t of sequence b (t < 0, padding: none), at `at` in tree_mask; returns its
    // depth.  The walk to the root visits falling indices, so the words are finished from the top down.
    auto ancestors = [&](int b, int t, int64_t at) -> int {
        int32_t *m = p.tree_mask + at;
        int w = p.tree_words - 1, depth = -1;
        uint32_t bits = 0;
        for (int u = t; u >= 0;) {
            for (; w > u >> 5; --w) {
                m[w] = (int32_t)bits;
                bits = 0;
            }
            bits |= 1u << (u & 31);
            ++depth;
            const int up = __ldg(p.parents + (int64_t)b * p.q_len + u);
            if (up >= u || up < -1) {
                raise_status(p.status, kStatusInvalid);
                break;
            }
            u = up;
        }
        for (; w >= 0; --w) {
            m[w] = (int32_t)bits;
            bits = 0;
        }
        return depth;
    };
    const bool one_chunk = p.batch <= kCacheThreads;
    // this CTA's sequences (all of them when they fit one chunk)
    const int s0 = one_chunk ? 0 : (int)((int64_t)p.batch * rank / ctas);
    const int s1 = one_chunk ? p.batch : (int)((int64_t)p.batch * (rank + 1) / ctas);
    const int nfree = paged ? *p.num_free : 0;
    int64_t total = 0, base = 0;
    if (one_chunk) {
        int L = 0, n = 0;
        const int need = tid < p.batch ? read(tid, L, n) : 0;
        const int64_t first = block_exclusive_scan(need, scan_smem, &total);
        s_len[tid] = L;
        s_new[tid] = n;
        s_first[tid] = (int)first;
    } else {
        int64_t all = 0, before = 0;
        for (int b = tid; b < p.batch; b += kCacheThreads) {
            int L, n;
            const int need = read(b, L, n);
            all += need;
            before += b < s0 ? need : 0;
        }
        block_exclusive_scan(all, scan_smem, &total);
        block_exclusive_scan(before, scan_smem, &base);
    }
    bad = __syncthreads_or(bad);
    const bool no_pages = paged && (nfree < 0 || nfree > p.free_capacity || total > nfree);
    const bool ok = !bad && !no_pages;
    if (!ok && rank == 0 && tid == 0)
        raise_status(p.status, bad || nfree < 0 || nfree > p.free_capacity ? kStatusInvalid : kStatusPages);
    if (ctas > 1) cluster_sync();  // every CTA has read the lengths and the page count

    for (int c0 = s0; c0 < s1; c0 += kCacheThreads) {
        const int cn = min(s1 - c0, kCacheThreads);
        if (!one_chunk) {
            int L = 0, n = 0;
            const int need = tid < cn ? read(c0 + tid, L, n) : 0;
            int64_t sum;
            const int64_t first = base + block_exclusive_scan(need, scan_smem, &sum);
            base += sum;
            s_len[tid] = L;
            s_new[tid] = n;
            s_first[tid] = (int)first;
            __syncthreads();
        }
        // page i of the new ones: taken from the top of the stack, sequence by sequence
        auto taken = [&](int c, int i) -> int { return p.free_pages[nfree - 1 - (s_first[c] + i)]; };
        if (paged && ok) {
            const int warp = tid >> 5, lane = tid & 31, warps = kCacheThreads / 32;
            const int w0 = one_chunk ? rank * warps + warp : warp, step = one_chunk ? ctas * warps : warps;
            for (int c = w0; c < cn; c += step) {
                const int have = pages_of(s_len[c]), need = pages_of((int64_t)s_len[c] + s_new[c]) - have;
                for (int i = lane; i < need; i += 32) {
                    const int page = taken(c, i);
                    if (page < 0 || (int64_t)page * kPage >= p.kv_rows) raise_status(p.status, kStatusBlockTable);
                    p.block_table[(int64_t)(c0 + c) * p.max_blocks + have + i] = page;
                }
            }
        }
        if (tid < cn && (!one_chunk || rank == 0)) p.seqlens_out[c0 + tid] = s_len[tid] + (ok ? s_new[tid] : 0);
        // slots, positions and ancestor masks: TOKENS tokens of one sequence a thread, whose page
        // lookups are in flight together
        const uint32_t per_seq = (uint32_t)(p.q_len + TOKENS - 1) / TOKENS;
        const uint32_t items = (uint32_t)cn * per_seq;  // batch * q_len fits an int32
        const uint32_t estep = one_chunk ? ctas * kCacheThreads : kCacheThreads;
        for (uint32_t e = one_chunk ? rank * kCacheThreads + tid : tid; e < items; e += estep) {
            const int c = (int)(e / per_seq), t0 = (int)(e - (uint32_t)c * per_seq) * TOKENS;
            const int b = c0 + c, L = s_len[c], n = s_new[c];
            const int have = pages_of(L);
            const int64_t at = (int64_t)b * p.q_len + t0;
            int pos[TOKENS], page[TOKENS];
#pragma unroll
            for (int u = 0; u < TOKENS; ++u) {
                const int t = t0 + u;
                pos[u] = page[u] = -1;
                if (t >= n || !ok) continue;
                pos[u] = L + t;
                if (paged) {
                    const int i = (L + t) / kPage;
                    page[u] = i < have ? p.block_table[(int64_t)b * p.max_blocks + i] : taken(c, i - have);
                }
            }
            if (p.tree_mask) {
#pragma unroll
                for (int u = 0; u < TOKENS; ++u)
                    if (t0 + u < p.q_len) {
                        const int depth = ancestors(b, t0 + u < n ? t0 + u : -1, (at + u) * p.tree_words);
                        if (pos[u] >= 0) pos[u] = L + depth;
                    }
            }
            int slot[TOKENS];
#pragma unroll
            for (int u = 0; u < TOKENS; ++u) {
                slot[u] = -1;
                if (pos[u] < 0) continue;
                if (!paged)
                    slot[u] = (int)((int64_t)b * p.kv_rows + L + t0 + u);
                else if (page[u] < 0 || (int64_t)page[u] * kPage >= p.kv_rows)
                    raise_status(p.status, kStatusBlockTable);
                else
                    slot[u] = page[u] * kPage + (L + t0 + u) % kPage;
            }
            bool stored = false;
            if constexpr (TOKENS == 4) {
                if (p.vector_out) {
                    *reinterpret_cast<int4 *>(p.slots + at) = make_int4(slot[0], slot[1], slot[2], slot[3]);
                    *reinterpret_cast<int4 *>(p.positions + at) = make_int4(pos[0], pos[1], pos[2], pos[3]);
                    stored = true;
                }
            }
            if (!stored) {
#pragma unroll
                for (int u = 0; u < TOKENS; ++u)
                    if (t0 + u < p.q_len) {
                        p.slots[at + u] = slot[u];
                        p.positions[at + u] = pos[u];
                    }
            }
        }
        if (!one_chunk) __syncthreads();  // the shared arrays are rewritten for the next chunk
    }
    if (paged && rank == 0 && tid == 0) *p.num_free_out = nfree - (ok ? (int)total : 0);
}

// ------------------------------------------------------------------------------------------ append
struct AppendParams {
    const __nv_bfloat16 *latent;  // [tokens] rows of 576, row_stride elements apart
    const __nv_bfloat16 *norm_weight;  // [512] or NULL: no norm
    const float *rope_table;      // [max_pos][64]: 32 cosines, 32 sines
    const int32_t *positions, *slots;
    __nv_bfloat16 *kv;            // bf16 cache, or NULL
    uint8_t *kv8;                 // E4M3 cache, or NULL
    float *kv_scale;
    const __nv_bfloat16 *q_rope;  // [tokens][heads] rows of 64, or NULL
    __nv_bfloat16 *q;             // [tokens][heads][576]: the last 64 columns are written
    int32_t *status;
    int64_t row_stride, q_token_stride, q_head_stride, cache_rows;
    int tokens, heads, max_pos;
    int key_blocks;               // blocks of rows ahead of the queries' blocks
    float eps;
};

constexpr int kAppendThreads = 128;
constexpr int kQueryHeads = 4;  // heads a thread of the queries' part rotates

__device__ __forceinline__ void unpack8(const uint4 &v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                      pack_bf16x2(x[6], x[7]));
}

// E4M3 codes of 8 values divided by the row's scale, given its reciprocal too: the product is corrected by its
// residual, which leaves the quotient rounded once, so that the border between two codes, where quotients
// of bf16 values do lie, falls as it does for the quotient (8192 rows: 6.8 -> 7.3 us).  A value that
// is not finite becomes the NaN code.
__device__ __forceinline__ uint2 codes8(const float (&x)[8], float scale, float inv) {
    const float2 scale2 = make_float2(scale, scale), inv2 = make_float2(inv, inv);
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = make_float2(x[2 * i], x[2 * i + 1]);
        const float2 q = mul2(v, inv2);
        const float2 y = fma2(fma2(make_float2(-q.x, -q.y), scale2, v), inv2, q);
        const float nan = __uint_as_float(0x7FFFFFFFu);
        w[i >> 1] |= (uint32_t)f32x2_to_e4m3x2(fabsf(v.x) < INFINITY ? y.x : nan, fabsf(v.y) < INFINITY ? y.y : nan)
                     << (16 * (i & 1));
    }
    return make_uint2(w[0], w[1]);
}

// The two 16-byte chunks of a 64-column rope row that thread i of 4 rotates: INTERLEAVED pairs (2k, 2k+1)
// lie within them, else chunk i holds the first and chunk i + 4 the second elements of its 8 pairs.
// Either way the pairs are 8i .. 8i + 7, and a thread writes exactly the elements that it read.
template <bool INTERLEAVED>
__device__ __forceinline__ void rotate16(float (&a)[8], float (&b)[8], const float (&c)[8], const float (&s)[8]) {
    if constexpr (INTERLEAVED) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float x = a[2 * k], y = a[2 * k + 1];
            a[2 * k] = x * c[k] - y * s[k];
            a[2 * k + 1] = y * c[k] + x * s[k];
            const float z = b[2 * k], w = b[2 * k + 1];
            b[2 * k] = z * c[4 + k] - w * s[4 + k];
            b[2 * k + 1] = w * c[4 + k] + z * s[4 + k];
        }
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float x = a[k], y = b[k];
            a[k] = x * c[k] - y * s[k];
            b[k] = y * c[k] + x * s[k];
        }
    }
}
template <bool INTERLEAVED>
__device__ __forceinline__ int rope_chunk(int i, int second) {
    return INTERLEAVED ? 2 * i + second : i + 4 * second;
}
__device__ __forceinline__ void load_angles(const float *table, int pos, int i, float (&c)[8], float (&s)[8]) {
    const float4 *t = reinterpret_cast<const float4 *>(table + (int64_t)pos * 64 + 8 * i);
    const float4 c0 = __ldg(t), c1 = __ldg(t + 1), s0 = __ldg(t + 8), s1 = __ldg(t + 9);
    c[0] = c0.x, c[1] = c0.y, c[2] = c0.z, c[3] = c0.w, c[4] = c1.x, c[5] = c1.y, c[6] = c1.z, c[7] = c1.w;
    s[0] = s0.x, s[1] = s0.y, s[2] = s0.z, s[3] = s0.w, s[4] = s1.x, s[5] = s1.y, s[6] = s1.z, s[7] = s1.w;
}

// One launch for both parts.  Rows: a warp per token; a lane holds two 16-byte chunks of the latent (the
// sum of squares is one warp reduction) and two of the rope columns (eight lanes alike), so that the row
// is read once, kept in registers through norm, rotation and quantisation, and written once.  Queries:
// four threads per head's 64 columns, each for kQueryHeads heads of one token, with the angles kept in
// registers across them.  Replayed from a graph: many tokens are bound by HBM, 256 ragged sequences of up to 16 with 128
// heads (half of the 4096 rows padding) move 77 MB in 13.3 us, 5.8 TB/s (0.88 of a copy); 8192 E4M3 rows without
// queries, 16 MB, take 7.4 us in 1.7 waves (64 registers leave room for 4736 of the 8192 warps; 9.1 with the
// position waited for before the loads), 64 tokens 2.4 us, most of it launch.
template <bool FP8, bool INTERLEAVED>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const __grid_constant__ AppendParams p) {
    if ((int)blockIdx.x < p.key_blocks) {
        const int lane = threadIdx.x & 31;
        const int tok = blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
        if (tok >= p.tokens) return;
        // everything that does not hang on the position is in flight before the position is known
        const uint4 *src = reinterpret_cast<const uint4 *>(p.latent + (int64_t)tok * p.row_stride);
        const int pos = p.positions[tok], slot = p.slots[tok];
        const uint4 l0 = __ldg(src + lane), l1 = __ldg(src + 32 + lane);
        const int i = lane & 3;
        const uint4 k0 = __ldg(src + 64 + rope_chunk<INTERLEAVED>(i, 0));
        const uint4 k1 = __ldg(src + 64 + rope_chunk<INTERLEAVED>(i, 1));
        if (pos < 0 || (slot < 0 && pos < p.max_pos)) return;  // padding, or no cache row wanted
        if (pos >= p.max_pos || slot >= p.cache_rows) {
            if (lane == 0) raise_status(p.status, pos >= p.max_pos ? kStatusInvalid : kStatusBlockTable);
            return;
        }
        float x0[8], x1[8], ra[8], rb[8], c[8], s[8];
        load_angles(p.rope_table, pos, i, c, s);
        unpack8(l0, x0);
        unpack8(l1, x1);
        unpack8(k0, ra);
        unpack8(k1, rb);
        rotate16<INTERLEAVED>(ra, rb, c, s);  // in every lane, of chunk pair lane % 4
        if (p.norm_weight) {
            float sum = 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) sum += x0[k] * x0[k] + x1[k] * x1[k];
#pragma unroll
            for (int d = 16; d >= 1; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
            const float r = __frsqrt_rn(sum * (1.f / kDv) + p.eps);
            float w0[8], w1[8];
            unpack8(__ldg(reinterpret_cast<const uint4 *>(p.norm_weight) + lane), w0);
            unpack8(__ldg(reinterpret_cast<const uint4 *>(p.norm_weight) + 32 + lane), w1);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                x0[k] = x0[k] * r * w0[k];
                x1[k] = x1[k] * r * w1[k];
            }
        }
        if constexpr (FP8) {
            float amax = 0.f;
            auto widen = [&](const float (&x)[8]) {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float a = fabsf(x[k]);
                    amax = fmaxf(amax, a < INFINITY ? a : 0.f);  // false for NaN too
                }
            };
            widen(x0);
            widen(x1);
            widen(ra);
            widen(rb);
#pragma unroll
            for (int d = 16; d >= 1; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, d));
            // 1 for a row of zeros; never under 2^-100, the least scale the decode tells apart
            const float scale = amax > 0.f ? fmaxf(amax / 448.f, 0x1p-100f) : 1.f;
            const float inv = 1.f / scale;
            uint2 *dst = reinterpret_cast<uint2 *>(p.kv8 + (int64_t)slot * kDqk);
            dst[lane] = codes8(x0, scale, inv);
            dst[32 + lane] = codes8(x1, scale, inv);
            if (lane < 4) {
                dst[64 + rope_chunk<INTERLEAVED>(lane, 0)] = codes8(ra, scale, inv);
                dst[64 + rope_chunk<INTERLEAVED>(lane, 1)] = codes8(rb, scale, inv);
            }
            if (lane == 0) p.kv_scale[slot] = scale;
        } else {
            uint4 *dst = reinterpret_cast<uint4 *>(p.kv + (int64_t)slot * kDqk);
            dst[lane] = pack8(x0);
            dst[32 + lane] = pack8(x1);
            if (lane < 4) {
                dst[64 + rope_chunk<INTERLEAVED>(lane, 0)] = pack8(ra);
                dst[64 + rope_chunk<INTERLEAVED>(lane, 1)] = pack8(rb);
            }
        }
        return;
    }
    const int groups = (p.heads + kQueryHeads - 1) / kQueryHeads;  // threads of a token: 4 per group of heads
    const int64_t idx = (int64_t)(blockIdx.x - p.key_blocks) * kAppendThreads + threadIdx.x;
    const int i = (int)(idx & 3);
    const int64_t tok = (idx >> 2) / groups;
    const int hg = (int)((idx >> 2) - tok * groups);
    if (tok >= p.tokens) return;
    const int pos = p.positions[tok];
    if (pos < 0) return;
    if (pos >= p.max_pos) {
        raise_status(p.status, kStatusInvalid);
        return;
    }
    float c[8], s[8];
    load_angles(p.rope_table, pos, i, c, s);
    uint4 v[kQueryHeads][2];
#pragma unroll
    for (int u = 0; u < kQueryHeads; ++u) {
        const int h = hg + u * groups;
        if (h >= p.heads) break;
        const uint4 *src = reinterpret_cast<const uint4 *>(p.q_rope + tok * p.q_token_stride + h * p.q_head_stride);
        v[u][0] = src[rope_chunk<INTERLEAVED>(i, 0)];
        v[u][1] = src[rope_chunk<INTERLEAVED>(i, 1)];
    }
#pragma unroll
    for (int u = 0; u < kQueryHeads; ++u) {
        const int h = hg + u * groups;
        if (h >= p.heads) break;
        float a[8], b[8];
        unpack8(v[u][0], a);
        unpack8(v[u][1], b);
        rotate16<INTERLEAVED>(a, b, c, s);
        uint4 *dst = reinterpret_cast<uint4 *>(p.q + (tok * p.heads + h) * (int64_t)kDqk + kDv);
        dst[rope_chunk<INTERLEAVED>(i, 0)] = pack8(a);
        dst[rope_chunk<INTERLEAVED>(i, 1)] = pack8(b);
    }
}

// ------------------------------------------------------------------------------------------ accept
struct AcceptParams {
    void *kv;         // bf16 or E4M3 rows
    float *kv_scale;  // E4M3 cache, or NULL
    const int32_t *seqlens, *new_lens, *path, *path_lens, *block_table;
    int32_t *free_pages;
    const int32_t *num_free;
    int32_t *seqlens_out, *num_free_out, *status;
    int64_t kv_rows;
    int batch, q_len, max_path, max_blocks, free_capacity;
};

// Sequence b's lengths, valid when its path may be taken: 0 <= new tokens <= min(q_len, L), and a path
// length of -1 (finished) or 0 .. min(max_path, new tokens).  The path's entries are checked apart.
struct AcceptSeq {
    int L, n, keep;
    bool valid;
};
__device__ __forceinline__ AcceptSeq accept_seq(const AcceptParams &p, int b) {
    AcceptSeq s;
    s.L = p.seqlens[b];
    s.n = p.new_lens[b];
    s.keep = p.path_lens[b];
    const int64_t cap = p.block_table ? (int64_t)p.max_blocks * kPage : p.kv_rows;
    s.valid = s.L >= 0 && s.L <= cap && s.n >= 0 && s.n <= p.q_len && s.n <= s.L && s.keep >= -1 &&
              s.keep <= p.max_path && s.keep <= s.n;
    return s;
}
// Lengths and path of sequence b, read together by a warp: lane i gets entry i of the path in `v`.  False
// where the sequence has to stay as it is; the entries must rise and lie inside the new tokens.
__device__ __forceinline__ bool accept_read(const AcceptParams &p, int b, AcceptSeq &s, int &v) {
    const int lane = threadIdx.x & 31;
    const int32_t *path = p.path + (int64_t)b * p.max_path;
    v = lane < p.max_path ? path[lane] : 0;
    s = accept_seq(p, b);
    bool bad = !s.valid;
    int before = -1;  // the last entry of the 32 ahead
    for (int i0 = 0; !bad && i0 < s.keep; i0 += 32) {
        const int i = i0 + lane;
        const int e = i0 == 0 ? v : i < s.keep ? path[i] : 0;
        const int up = __shfl_up_sync(0xffffffffu, e, 1);
        bad = __any_sync(0xffffffffu, i < s.keep && (e >= s.n || e <= (lane == 0 ? before : up)));
        before = __shfl_sync(0xffffffffu, e, 31);
    }
    return !bad;
}

// A warp moves one slice of a sequence's accepted rows: 32 of the 16-byte columns of a row (E4M3: the last
// slice also the row scales, in lane 4).  Row ctx + path[i] goes to row ctx + i; path[i] >= i, so a lane
// that carries its column through the rows in rising order, kAcceptBatch read before the first of them
// is written, never overwrites a row that it has yet to read, and lanes and warps never meet.  The
// path's rows are looked up by the warp 32 at a time, one a lane.  `lengths_read` is called once the
// lengths have been read.
constexpr int kAcceptBatch = 8;
template <bool FP8>
constexpr int kAcceptSlices = FP8 ? 2 : 3;
template <bool FP8, class Read>
__device__ __forceinline__ void accept_rows(const AcceptParams &p, int b, int slice, Read lengths_read) {
    const int lane = threadIdx.x & 31;
    AcceptSeq s;
    int v0;
    const bool good = accept_read(p, b, s, v0);
    lengths_read();
    if (!good) {
        if (lane == 0 && slice == 0) raise_status(p.status, kStatusInvalid);
        return;
    }
    const int ctx = s.L - s.n;
    auto locate = [&](int row) -> int {  // cache row, or -1 behind a bad page
        if (!p.block_table) return (int)((int64_t)b * p.kv_rows + row);
        const int page = p.block_table[(int64_t)b * p.max_blocks + row / kPage];
        if (page < 0 || (int64_t)page * kPage >= p.kv_rows) {
            raise_status(p.status, kStatusBlockTable);
            return -1;
        }
        return page * kPage + row % kPage;
    };
    constexpr int kChunks = FP8 ? kDqk / 16 : kDqk * 2 / 16;  // 16-byte columns of a row
    const int col = 32 * slice + lane;
    const bool data = col < kChunks, scale = FP8 && col == kChunks;
    uint4 *rows = reinterpret_cast<uint4 *>(p.kv) + col;
    for (int i0 = 0; i0 < s.keep; i0 += 32) {
        int src = -1, dst = -1;
        if (i0 + lane < s.keep) {
            const int from = i0 == 0 ? v0 : p.path[(int64_t)b * p.max_path + i0 + lane];
            if (from != i0 + lane) {
                src = locate(ctx + from);
                dst = locate(ctx + i0 + lane);
                if (dst < 0) src = -1;
            }
        }
        const int end = min(s.keep - i0, 32);
        for (int j0 = 0; j0 < end; j0 += kAcceptBatch) {
            uint4 v[kAcceptBatch];
#pragma unroll
            for (int u = 0; u < kAcceptBatch; ++u) {
                const int64_t r = __shfl_sync(0xffffffffu, src, j0 + u);  // -1 past the path's end
                if (r >= 0 && data) v[u] = rows[r * kChunks];
                if (r >= 0 && scale) v[u].x = __float_as_uint(p.kv_scale[r]);
            }
#pragma unroll
            for (int u = 0; u < kAcceptBatch; ++u) {
                const int64_t r = __shfl_sync(0xffffffffu, src, j0 + u);
                const int64_t w = __shfl_sync(0xffffffffu, dst, j0 + u);
                if (r >= 0 && data) rows[w * kChunks] = v[u];
                if (r >= 0 && scale) p.kv_scale[w] = __uint_as_float(v[u].x);
            }
        }
    }
}

// One CTA: the new lengths, and the pages past them pushed on the stack in sequence order.  It reads
// nothing that accept_rows writes; `others_have_read` returns once every reader of the lengths is done,
// and only then is anything written, so that lengths and page count may be updated in place.
template <class Wait>
__device__ __forceinline__ void accept_pages(const AcceptParams &p, Wait others_have_read) {
    __shared__ int64_t scan_smem[32];
    __shared__ int s_len[kCacheThreads], s_want[kCacheThreads], s_first[kCacheThreads];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const bool paged = p.block_table != nullptr;
    const int nfree = paged ? *p.num_free : 0;
    const bool stack_ok = nfree >= 0 && nfree <= p.free_capacity;
    int64_t base = 0;
    for (int c0 = 0; c0 < p.batch; c0 += kCacheThreads) {
        const int cn = min(p.batch - c0, kCacheThreads);
        for (int c = warp; c < cn; c += kCacheThreads / 32) {
            AcceptSeq s;
            int v;
            const bool good = accept_read(p, c0 + c, s, v);
            if (lane == 0) {
                s_len[c] = s.L;
                s_want[c] = !good ? s.L : (s.keep < 0 ? 0 : s.L - s.n + s.keep);  // a bad path keeps its rows
            }
        }
        __syncthreads();
        int back = 0;
        if (tid < cn && paged && s_len[tid] > s_want[tid]) back = pages_of(s_len[tid]) - pages_of(s_want[tid]);
        int64_t sum;
        // (an int32: more pages than that go back only where a page stands in a table twice)
        s_first[tid] = (int)(base + block_exclusive_scan(back, scan_smem, &sum));
        __syncthreads();
        if (c0 == 0) others_have_read();
        if (tid < cn) p.seqlens_out[c0 + tid] = s_want[tid];
        for (int c = warp; c < cn && paged; c += kCacheThreads / 32) {
            const int want = pages_of(s_want[c]), more = pages_of(s_len[c]) - want;
            for (int i = lane; i < more; i += 32) {
                const int page = p.block_table[(int64_t)(c0 + c) * p.max_blocks + want + i];
                if (page < 0 || (int64_t)page * kPage >= p.kv_rows) raise_status(p.status, kStatusBlockTable);
                const int64_t at = (int64_t)nfree + s_first[c] + i;
                if (stack_ok && at < p.free_capacity) p.free_pages[at] = page;
            }
        }
        base += sum;
        __syncthreads();
    }
    if (paged && tid == 0) {
        const int64_t total = nfree + base;
        if (!stack_ok || total > p.free_capacity) raise_status(p.status, kStatusInvalid);
        *p.num_free_out = !stack_ok ? nfree : (int)(total > p.free_capacity ? p.free_capacity : total);
    }
}

// A small batch: one cluster.  CTA 0 takes lengths and pages, the warps of the others the rows; they
// arrive on the cluster barrier as soon as they have read the lengths (all that CTA 0 waits for: the
// values have been used by then, so the arrival needs no ordering of its own).  16 sequences of 4 tokens,
// E4M3: 5.5..6.6 us, the chain lengths, path, page, row, store.
template <bool FP8>
__global__ void __launch_bounds__(kCacheThreads) accept_kernel(const __grid_constant__ AcceptParams p) {
    auto arrive = [] { asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory"); };
    auto wait = [] { asm volatile("barrier.cluster.wait;" ::: "memory"); };
    if (blockIdx.x == 0) {
        accept_pages(p, [&] {
            arrive();
            wait();
        });
        return;
    }
    constexpr int kSlices = kAcceptSlices<FP8>;
    const int i = ((int)blockIdx.x - 1) * (kCacheThreads / 32) + (int)(threadIdx.x >> 5);
    if (i < p.batch * kSlices)
        accept_rows<FP8>(p, i / kSlices, i % kSlices, arrive);
    else
        arrive();
    __syncwarp();
    wait();
}

// A large one: a grid of warps, and beside it (a programmatic dependent, which waits for the grid's end
// before it writes) the CTA for lengths and pages.  64 sequences of up to 64 rows: 6.2 us.
constexpr int kAcceptThreads = 128;
template <bool FP8>
__global__ void __launch_bounds__(kAcceptThreads) accept_rows_kernel(const __grid_constant__ AcceptParams p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    constexpr int kSlices = kAcceptSlices<FP8>;
    const int i = (int)blockIdx.x * (kAcceptThreads / 32) + (int)(threadIdx.x >> 5);
    if (i < p.batch * kSlices) accept_rows<FP8>(p, i / kSlices, i % kSlices, [] {});
}
__global__ void __launch_bounds__(kCacheThreads) accept_pages_kernel(const __grid_constant__ AcceptParams p) {
    accept_pages(p, [] { asm volatile("griddepcontrol.wait;" ::: "memory"); });
}

}  // namespace mla
