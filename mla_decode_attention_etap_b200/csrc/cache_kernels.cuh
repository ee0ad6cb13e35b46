// The steps around the decode that keep its latent cache: pages, slots and masks of new tokens
// (extend_kernel), their rows (append_kernel, rotate_queries), and the accepted path of a verified tree
// (accept_rows_kernel, accept_pages_kernel).  No kernel here waits on another CTA except through the
// hardware cluster barrier; every index read from memory is checked before it is used.
#pragma once

#include <cuda_bf16.h>
#include <cstdint>
#include <type_traits>

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
};

// One cluster of up to 8 CTAs.  Every CTA computes the page offsets of all sequences (a prefix sum of
// the pages each needs), then, once all have read the lengths (the cluster barrier, so that lengths and
// the page count may be updated in place), writes its share.  Sequences are taken kCacheThreads at a
// time; a batch that fits one such chunk is read once, and its tokens are dealt over all CTAs.
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
        // slots, positions and ancestor masks, token by token
        const uint32_t tokens = (uint32_t)cn * p.q_len;  // batch * q_len fits an int32
        const uint32_t estep = one_chunk ? ctas * kCacheThreads : kCacheThreads;
        for (uint32_t e = one_chunk ? rank * kCacheThreads + tid : tid; e < tokens; e += estep) {
            const int c = (int)(e / (uint32_t)p.q_len), t = (int)(e - (uint32_t)c * p.q_len);
            const int b = c0 + c;
            const int64_t at = (int64_t)b * p.q_len + t;
            const bool real = t < s_new[c];
            int depth = t;
            if (p.tree_mask) {
                // the walk to the root visits falling indices, so the words are finished from the top down
                int32_t *m = p.tree_mask + at * p.tree_words;
                int w = p.tree_words - 1;
                uint32_t bits = 0;
                depth = -1;
                for (int u = real ? t : -1; u >= 0;) {
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
            }
            int slot = -1, pos = -1;
            if (real && ok) {
                const int row = s_len[c] + t;
                pos = s_len[c] + depth;
                if (paged) {
                    const int have = pages_of(s_len[c]), i = row / kPage;
                    const int page = i < have ? p.block_table[(int64_t)b * p.max_blocks + i] : taken(c, i - have);
                    if (page < 0 || (int64_t)page * kPage >= p.kv_rows)
                        raise_status(p.status, kStatusBlockTable);
                    else
                        slot = page * kPage + row % kPage;
                } else {
                    slot = (int)((int64_t)b * p.kv_rows + row);
                }
            }
            p.slots[at] = slot;
            p.positions[at] = pos;
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

// E4M3 codes of 8 values divided by the row's scale (round to nearest even, as a cache quantised on the
// host holds them); a value that is not finite becomes the NaN code.
__device__ __forceinline__ uint2 codes8(const float (&x)[8], float scale) {
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float y[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float v = x[2 * i + j];
            y[j] = fabsf(v) < INFINITY ? v / scale : __uint_as_float(0x7FFFFFFFu);
        }
        w[i >> 1] |= (uint32_t)f32x2_to_e4m3x2(y[0], y[1]) << (16 * (i & 1));
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
// sum of squares is one warp reduction) and lanes 0..3 two chunks of the rope columns, so that the row
// is read once, kept in registers through norm, rotation and quantisation, and written once.  Queries:
// four threads per head's 64 columns, each for kQueryHeads heads of one token, with the angles kept in
// registers across them.
template <bool FP8, bool INTERLEAVED>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const __grid_constant__ AppendParams p) {
    if ((int)blockIdx.x < p.key_blocks) {
        const int lane = threadIdx.x & 31;
        const int tok = blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
        if (tok >= p.tokens) return;
        const int pos = p.positions[tok], slot = p.slots[tok];
        const uint4 *src = reinterpret_cast<const uint4 *>(p.latent + (int64_t)tok * p.row_stride);
        if (pos < 0 || slot < 0) return;  // padding
        if (pos >= p.max_pos || slot >= p.cache_rows) {
            if (lane == 0) raise_status(p.status, pos >= p.max_pos ? kStatusInvalid : kStatusBlockTable);
            return;
        }
        float x0[8], x1[8], ra[8], rb[8];
        unpack8(__ldg(src + lane), x0);
        unpack8(__ldg(src + 32 + lane), x1);
        if (lane < 4) {
            float c[8], s[8];
            load_angles(p.rope_table, pos, lane, c, s);
            unpack8(__ldg(src + 64 + rope_chunk<INTERLEAVED>(lane, 0)), ra);
            unpack8(__ldg(src + 64 + rope_chunk<INTERLEAVED>(lane, 1)), rb);
            rotate16<INTERLEAVED>(ra, rb, c, s);
        }
        if (p.norm_weight) {
            float sum = 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) sum += x0[k] * x0[k] + x1[k] * x1[k];
#pragma unroll
            for (int d = 16; d >= 1; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
            const float r = rsqrtf(sum * (1.f / kDv) + p.eps);
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
            if (lane < 4) {
                widen(ra);
                widen(rb);
            }
#pragma unroll
            for (int d = 16; d >= 1; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, d));
            // 1 for a row of zeros; never under 2^-100, the least scale the decode tells apart
            const float scale = amax > 0.f ? fmaxf(amax / 448.f, 0x1p-100f) : 1.f;
            uint2 *dst = reinterpret_cast<uint2 *>(p.kv8 + (int64_t)slot * kDqk);
            dst[lane] = codes8(x0, scale);
            dst[32 + lane] = codes8(x1, scale);
            if (lane < 4) {
                dst[64 + rope_chunk<INTERLEAVED>(lane, 0)] = codes8(ra, scale);
                dst[64 + rope_chunk<INTERLEAVED>(lane, 1)] = codes8(rb, scale);
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
// Entry i of a path: inside the new tokens and above entry i - 1.
__device__ __forceinline__ bool path_entry_ok(const int32_t *path, int i, int n) {
    const int v = path[i];
    return v < n && v > (i > 0 ? path[i - 1] : -1);
}

// One CTA per sequence moves the accepted rows: row ctx + path[i] to row ctx + i.  path[i] >= i, so a
// thread that carries one 16-byte column (or the row scale) through all rows in rising order never
// overwrites a row that it has yet to read, and threads never meet: no barrier between rows.
constexpr int kAcceptThreads = 96;
constexpr int kAcceptBatch = 8;   // rows in flight per thread
constexpr int kAcceptChunk = 512; // rows whose places are looked up at a time
template <bool FP8>
__global__ void __launch_bounds__(kAcceptThreads) accept_rows_kernel(const __grid_constant__ AcceptParams p) {
    __shared__ int s_src[kAcceptChunk], s_dst[kAcceptChunk];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int b = blockIdx.x, tid = threadIdx.x;
    const AcceptSeq s = accept_seq(p, b);
    if (!s.valid) {
        if (tid == 0) raise_status(p.status, kStatusInvalid);
        return;
    }
    if (s.keep <= 0) return;
    const int32_t *path = p.path + (int64_t)b * p.max_path;
    bool bad = false;
    for (int i = tid; i < s.keep; i += kAcceptThreads) bad |= !path_entry_ok(path, i, s.n);
    if (__syncthreads_or(bad)) {
        if (tid == 0) raise_status(p.status, kStatusInvalid);
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
    for (int c0 = 0; c0 < s.keep; c0 += kAcceptChunk) {
        const int cn = min(s.keep - c0, kAcceptChunk);
        if (c0 > 0) __syncthreads();
        for (int i = tid; i < cn; i += kAcceptThreads) {
            const int from = path[c0 + i], to = c0 + i;
            int src = -1, dst = -1;
            if (from != to) {
                src = locate(ctx + from);
                dst = locate(ctx + to);
            }
            s_src[i] = dst < 0 ? -1 : src;
            s_dst[i] = dst;
        }
        __syncthreads();
        // kAcceptBatch rows are read before the first of them is written: their places lie below every
        // later source
        auto carry = [&](auto *rows, int pitch) {
            for (int i0 = 0; i0 < cn; i0 += kAcceptBatch) {
                std::remove_reference_t<decltype(*rows)> v[kAcceptBatch];
#pragma unroll
                for (int u = 0; u < kAcceptBatch; ++u)
                    if (i0 + u < cn && s_src[i0 + u] >= 0) v[u] = rows[(int64_t)s_src[i0 + u] * pitch];
#pragma unroll
                for (int u = 0; u < kAcceptBatch; ++u)
                    if (i0 + u < cn && s_src[i0 + u] >= 0) rows[(int64_t)s_dst[i0 + u] * pitch] = v[u];
            }
        };
        if (tid < kChunks)
            carry(reinterpret_cast<uint4 *>(p.kv) + tid, kChunks);
        else if (FP8 && tid == kChunks)
            carry(p.kv_scale, 1);
    }
}

// One CTA: the new lengths, and the pages past them pushed on the stack in sequence order.  It reads
// nothing that the rows' kernel writes, so it runs beside it (a programmatic dependent) and waits for
// it only before it writes, which is what makes an update in place safe.
__global__ void __launch_bounds__(kCacheThreads) accept_pages_kernel(const __grid_constant__ AcceptParams p) {
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
            const AcceptSeq s = accept_seq(p, c0 + c);
            bool bad = !s.valid;
            if (!bad)
                for (int i = lane; i < s.keep; i += 32)
                    bad |= !path_entry_ok(p.path + (int64_t)(c0 + c) * p.max_path, i, s.n);
            bad = __any_sync(0xffffffffu, bad);
            if (lane == 0) {
                s_len[c] = s.L;
                s_want[c] = bad ? s.L : (s.keep < 0 ? 0 : s.L - s.n + s.keep);  // a bad path keeps its rows
            }
        }
        __syncthreads();
        int back = 0;
        if (tid < cn && paged && s_len[tid] > s_want[tid]) back = pages_of(s_len[tid]) - pages_of(s_want[tid]);
        int64_t sum;
        // (an int32: more pages than that go back only where a page stands in a table twice)
        s_first[tid] = (int)(base + block_exclusive_scan(back, scan_smem, &sum));
        __syncthreads();
        if (c0 == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
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

}  // namespace mla
