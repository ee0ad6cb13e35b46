// ETAP decode of an E4M3 cache in groups of 64 query columns, sm_100a: the tree decode of more than 16
// columns.
//
// Computation as in etap_pair_kernel.cuh's E4M3 configurations: S^T = K Q^T with Q as two E4M3 terms
// times a power of two per column, P^T as two E4M3 terms of 2^(score + log2 s - m + PSCALE) (s: the row's
// scale; m follows the tiles' largest both ways, see etap_common.cuh), O^T = V^T P^T, fp32 accumulation.  What differs is the layout, made for 64 columns:
//
//   * A CTA holds whole 128-row tiles (72 KB of codes) and all of its 64 columns' Q (72 KB: [Q_hi; Q_lo]
//     are the 128 B-operand rows of one N = 128 MMA), so that neither scores nor probabilities cross
//     CTAs.  Its ring keeps two tiles: the loads and scores of tile k + 1 run under the softmax and the
//     output contraction of tile k, and a tile's value columns are the codes that its scores read.
//   * P_hi and P_lo are multiplied one after the other into the same accumulators (N = 64 each): four
//     M-tiles of 64 columns leave the TMEM room for two score buffers of 128.
//   * Sixteen softmax warps, four per TMEM lane quadrant: a thread holds one row and 16 columns, and
//     its row's scale is read a tile ahead.
//   * It runs on the M = 256 kernel's schedules (256-row units, one range per 2-CTA cluster).  In its 64-column
//     groups the two CTAs take the two tiles of a unit and merge their results once per segment through
//     distributed shared memory; in its 128-column groups each takes 64 of the columns and both tiles,
//     and nothing is merged.
//
// B=16, h=16, q_len=4, 16384..32768 rows (230 MB of cache): 83..84 us with its plan, replayed from a graph at full
// clock, 2.8 TB/s (90..94 called in a row from Python); 32 columns 81 us.  The 32-column groups of the pair kernel,
// causal, take 160 and 116 us on these shapes.  A tile takes a CTA 2.7 us: 1.5 us of matrix
// instructions, but the chain of its loads (1.2 us after a slot comes free), scores (0.5), softmax (2.0) and
// step 3 (1.25) runs over a ring of two tiles; shared memory and TMEM are full.
//
// Warps per CTA (20): 0 TMA producer, 1 step-1 issuer and TMEM owner, 2 and 3 step-3 issuers (two M-tiles
// each), 4..19 softmax and epilogue.  Every wait is bounded; see etap_common.cuh.
#pragma once

#include "etap_common.cuh"
#include "etap_pair_kernel.cuh"  // swz_off
#include "plan_check.cuh"

namespace mla {

struct Wide8 {
    static constexpr int NC = 64;                      // query columns of a CTA
    static constexpr int NV = 8;                       // 16 KB slots: 128 rows x 128 codes
    static constexpr int THREADS = 640, NSM = 512;     // softmax threads: warps 4..19
    static constexpr uint32_t CHUNK = 16384, HALF = 8192;
    static constexpr uint32_t R_ROW = 64, R_DATA = 128 * R_ROW, R_HALF = 64 * R_ROW;
    static constexpr uint32_t Q_CHUNK = 2 * NC * 128, P_TERM = 128 * NC;
    static constexpr uint32_t OFF_V = 0;
    static constexpr uint32_t OFF_R = OFF_V + NV * CHUNK;
    static constexpr uint32_t OFF_Q = OFF_R + R_DATA;
    static constexpr uint32_t OFF_QR = OFF_Q + 4 * Q_CHUNK;
    static constexpr uint32_t OFF_P = OFF_QR + 2 * NC * R_ROW;  // P_hi, then P_lo
    static constexpr uint32_t OFF_BAR = OFF_P + 2 * P_TERM;
    static constexpr uint32_t OFF_MISC = OFF_BAR + 256;  // +0 TMEM address, +16 WaitCtl
    static constexpr uint32_t OFF_M = OFF_MISC + 64;     // float[64] PSCALE - m (log2 units)
    static constexpr uint32_t OFF_ALPHA = OFF_M + 256;   // float[64] rescale factors; the epilogue's factors of this CTA's part
    static constexpr uint32_t OFF_QV = OFF_ALPHA + 256;  // float[64] 2^-c; the epilogue's of the peer's
    static constexpr uint32_t OFF_MX = OFF_QV + 256;     // int[2][64] column maxima of a tile's halves (ordered_bits)
    static constexpr uint32_t BYTES = OFF_MX + 512;
    static constexpr uint32_t SMEM_ALLOC = BYTES + 1024;  // slack for 1024-byte alignment
    // the Q area receives the peer's part of a segment: 2 M-tiles x 16 column quads x 128 rows x 16 bytes,
    // then its (m, l) per column
    static constexpr uint32_t OFF_XM = OFF_Q, XM_TILE = 128 * NC * 4, OFF_XML = OFF_XM + 2 * XM_TILE;
    static constexpr uint32_t X_BYTES = 2 * XM_TILE + 2 * NC * 4;
    // and behind that the column sums of the four lane quadrants
    static constexpr uint32_t OFF_SUM = OFF_XML + 2 * NC * 4;
    static constexpr uint32_t O_COL = 0, S_COL = 4 * NC;  // 4 M-tiles; 2 buffers of [hi | lo] scores
    static constexpr uint32_t IDESC_S = idesc_e4m3_f32(128, 2 * NC, 0, 0);
    static constexpr uint32_t IDESC_O = idesc_e4m3_f32(128, NC, 1, 1);
    // barriers
    static constexpr int VF = 0, VE = VF + NV, RF = VE + NV, RE = RF + 1, QF = RE + 1, SF = QF + 1, SE = SF + 2,
                         PF = SE + 2, PE = PF + 1, TAIL = PE + 1, FIN1 = TAIL + 1, FIN3 = FIN1 + 1, XFREE = FIN3 + 2,
                         XFULL = XFREE + 1, BARS = XFULL + 1;
};
static_assert(Wide8::SMEM_ALLOC <= 232448 && Wide8::BARS * 8 <= 256 && Wide8::S_COL + 4 * Wide8::NC <= 512 &&
                  Wide8::OFF_SUM + 4 * Wide8::NC * 4 <= Wide8::OFF_P && Wide8::OFF_P % 1024 == 0,
              "shared memory / TMEM plan");

// An int that orders as the float does (its own inverse), for a maximum over warps by atomicMax.
__device__ __forceinline__ int ordered_bits(int bits) { return bits < 0 ? bits ^ 0x7fffffff : bits; }
constexpr int kOrderedLowest = (int)0x80000000;  // below every float's

// The 128-row tiles of a CTA, segment by segment: tile t of the segments' sequence b.
struct WideTiles {
    SegIter it;
    int b, t, t_end, step, L;
    bool first, valid;
    template <class Len>
    __device__ void segment(const int32_t *tile_off, int rank, int mode, Len len) {
        int t0, t1;
        valid = it.next(tile_off, b, t0, t1);
        if (!valid) return;
        L = len(b);
        step = mode ? 1 : 2;
        t = 2 * t0 + (mode ? 0 : rank);
        t_end = mode ? min(2 * t1, tiles_of(L)) : 2 * t1;
        first = true;
    }
    template <class Len>
    __device__ void init(const int32_t *tile_off, int b0, int64_t fb, int64_t fe, int rank, int mode, Len len) {
        it.init_at(b0, fb, fe);
        segment(tile_off, rank, mode, len);
    }
    // true when the next tile opens another segment (or there is none)
    template <class Len>
    __device__ bool advance(const int32_t *tile_off, int rank, int mode, Len len) {
        t += step;
        first = false;
        if (t < t_end) return false;
        segment(tile_off, rank, mode, len);
        return true;
    }
};

__global__ void __launch_bounds__(Wide8::THREADS, 1)
    etap_wide8_kernel(const __grid_constant__ CUtensorMap tm_kv, const __grid_constant__ CUtensorMap tm_kvr,
                      const __grid_constant__ DecodeParams p) {
    using C = Wide8;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_addr(smem_raw);
    const uint32_t sbase = (raw_addr + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (sbase - raw_addr);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank(), peer = rank ^ 1u;
    int32_t *status = p.ws + kHdrStatus;
    auto bar = [&](int i) -> uint32_t { return sbase + C::OFF_BAR + 8u * (uint32_t)i; };
    volatile WaitCtl *wc = reinterpret_cast<volatile WaitCtl *>(smem + C::OFF_MISC + 16);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::OFF_MISC);

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::BARS; ++i) {
            const bool warps = i == C::QF || i == C::SE || i == C::SE + 1 || i == C::PF;
            mbar_init(bar(i), warps ? C::NSM / 32 : i == C::PE ? 2 : 1);  // PE: both step-3 issuers commit
        }
        wc->abort = 0;
        wc->limit_ns = p.wait_limit_ns;
        fence_barrier_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&tm_kv);
        tma_prefetch_desc(&tm_kvr);
    }
    if (warp == 1) {
        tmem_alloc(smem_addr(tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    cluster_sync();  // both CTAs' barriers exist before any remote operation
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);  // (known to be the same in all lanes)
    // Launched as a programmatic dependent of the plan: nothing above read global memory.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // The schedule must come from a plan for this same shape (uniform in the whole cluster).
    const PlanHeader plan = read_plan_header(p.ws, p.sched_hdr);
    const int mode = plan.mode, groups = plan.groups, ctas = plan.ctas;
    const bool plan_ok = duo_plan_matches(plan, p.batch, p.ncols, p.slots, p.ctas) &&
                         ctas * groups <= (int)(gridDim.x >> 1);
    if (!plan_ok && threadIdx.x == 0) atomicCAS(status, 0, kStatusInvalid);
    if (blockIdx.x == 0 && threadIdx.x == 0) p.ws[kHdrSchedUsed] = p.sched_id;  // the partials' schedule
    const int cluster = (int)(blockIdx.x >> 1);
    const int unit = plan_ok ? cluster / groups : 0;
    const int grp = plan_ok ? cluster % groups : 0;
    const bool has_work = plan_ok && unit < ctas;
    const int c0 = grp * duo_group_cols(mode) + (mode == 1 ? C::NC * (int)rank : 0);  // this CTA's first column
    const int32_t *ranges = p.ws + p.cta_ranges_off;
    const int32_t *tile_off = p.ws + p.tile_off_off;
    const int32_t *seq_info = p.ws + p.seq_info_off;
    const int64_t fb = has_work ? ranges[2 * unit] : 0, fe = has_work ? ranges[2 * unit + 1] : 0;
    const int seq0 = has_work ? p.ws[p.cta_seq_off + unit] : 0;
    const int64_t l_cap = p.paged ? (int64_t)p.max_blocks * kPage : p.kv_rows;
    auto seq_len = [&](int b) -> int {
        int L = p.seqlens[b];
        if ((int64_t)L > l_cap) {
            if (lane == 0) atomicCAS(status, 0, kStatusInvalid);
            L = (int)l_cap;
        }
        return L < 0 ? 0 : L;
    };
    // Cache row of the first of 64 rows `row0` (a multiple of 64) of sequence b, or -1 behind a bad page.
    auto locate = [&](int b, int row0) -> int {
        if (!p.paged) return (int)((int64_t)b * p.kv_rows + row0);
        const int blk = __ldg(p.block_table + (int64_t)b * p.max_blocks + (row0 >> 6));
        return blk < 0 || (int64_t)blk * kPage >= p.kv_rows ? -1 : blk * kPage;
    };

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        // The whole warp runs the loop, one lane issues.
        const bool lead = elect_one();
        bool ok = true;
        uint32_t g = 0;  // value chunks so far
        int k = 0, tail_uses = 0;
        uint32_t tma_slots = 0;  // bit s: the last load of slot s was a TMA counted on its VF
        WideTiles w;
        w.valid = false;
        if (fb < fe) w.init(tile_off, seq0, fb, fe, (int)rank, mode, seq_len);
        int y0 = 0, y1 = 0, valid = 0;  // cache rows of the tile's two 64-row boxes (-1: not loaded), valid rows
        auto look_up = [&] {
            if (!w.valid) return;
            const int row0 = w.t * kTileRows;
            valid = min(max(w.L - row0, 0), kTileRows);
            y0 = valid > 0 ? locate(w.b, row0) : -1;
            y1 = valid > 64 ? locate(w.b, row0 + 64) : -1;
            if (lead && ((valid > 0 && y0 < 0) || (valid > 64 && y1 < 0))) atomicCAS(status, 0, kStatusBlockTable);
        };
        look_up();
        while (__all_sync(0xffffffffu, ok && w.valid)) {
            const int ya = __shfl_sync(0xffffffffu, y0, 0), yb = __shfl_sync(0xffffffffu, y1, 0);
            const int rows = __shfl_sync(0xffffffffu, valid, 0);
            const uint32_t nload = (ya >= 0 ? 1u : 0u) + (yb >= 0 ? 1u : 0u);
            const bool whole = rows == kTileRows && nload == 2;
            // rope codes: rows past the end are masked in S^T, no zeroing needed
            ok = poll_phase(bar(C::RE), (k & 1) ^ 1, wc, status);
            if (!__all_sync(0xffffffffu, ok)) break;
            if (lead) {
                mbar_arrive_expect_tx(bar(C::RF), nload * C::R_HALF);
                if (ya >= 0) tma_load_2d(sbase + C::OFF_R, &tm_kvr, bar(C::RF), kDv, ya);
                if (yb >= 0) tma_load_2d(sbase + C::OFF_R + C::R_HALF, &tm_kvr, bar(C::RF), kDv, yb);
            }
            __syncwarp();
            ++k;
            w.advance(tile_off, (int)rank, mode, seq_len);
            look_up();  // of the next tile, while this one's slots come free
            if (lead) {
                // bring it into L2, so that its loads, a tile later, do not wait on HBM (95.7 -> 93.5 us at
                // B=16, h=16, q_len=4, 16384..32768 rows)
#pragma unroll
                for (int i = 0; i < 4 && w.valid; ++i) {
                    if (y0 >= 0) tma_prefetch_l2_2d(&tm_kv, 128 * i, y0);
                    if (y1 >= 0) tma_prefetch_l2_2d(&tm_kv, 128 * i, y1);
                }
                if (w.valid && y0 >= 0) tma_prefetch_l2_2d(&tm_kvr, kDv, y0);
                if (w.valid && y1 >= 0) tma_prefetch_l2_2d(&tm_kvr, kDv, y1);
            }
            __syncwarp();
            if (whole) {
#pragma unroll 1
                for (int i = 0; i < 4; ++i, ++g) {
                    const uint32_t s = g % C::NV;
                    ok = poll_phase(bar(C::VE + (int)s), ((g / C::NV) & 1) ^ 1, wc, status);
                    if (!__all_sync(0xffffffffu, ok)) break;
                    if (lead) {
                        const uint32_t dst = sbase + C::OFF_V + s * C::CHUNK, on = bar(C::VF + (int)s);
                        mbar_arrive_expect_tx(on, C::CHUNK);
                        tma_load_2d(dst, &tm_kv, on, 128 * i, ya);
                        tma_load_2d(dst + C::HALF, &tm_kv, on, 128 * i, yb);
                    }
                    __syncwarp();
                    tma_slots |= 1u << s;
                }
            } else {
                // a tail: land the valid rows, zero all others, so that whatever the cache (or the slot) holds
                // there meets P = 0 as an exact 0
                for (int i = 0; i < 4; ++i, ++g) {
                    const uint32_t s = g % C::NV;
                    ok = poll_phase(bar(C::VE + (int)s), ((g / C::NV) & 1) ^ 1, wc, status);
                    if (!__all_sync(0xffffffffu, ok)) break;
                    const uint32_t dst = sbase + C::OFF_V + s * C::CHUNK;
                    tma_slots &= ~(1u << s);
                    if (nload > 0) {
                        if (lead) {
                            mbar_arrive_expect_tx(bar(C::TAIL), nload * C::HALF);
                            if (ya >= 0) tma_load_2d(dst, &tm_kv, bar(C::TAIL), 128 * i, ya);
                            if (yb >= 0) tma_load_2d(dst + C::HALF, &tm_kv, bar(C::TAIL), 128 * i, yb);
                        }
                        __syncwarp();
                        ok = wait_phase(bar(C::TAIL), tail_uses & 1, wc, status);
                        ++tail_uses;
                        if (!__all_sync(0xffffffffu, ok)) break;
                    }
                    for (int idx = lane; idx < kTileRows * 8; idx += 32) {
                        const int r = idx >> 3;
                        if (r < rows && (r < 64 ? ya : yb) >= 0) continue;
                        *reinterpret_cast<uint4 *>(smem + C::OFF_V + s * C::CHUNK + idx * 16) = make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lead) mbar_arrive(bar(C::VF + (int)s));
                    __syncwarp();
                }
            }
            ok = __all_sync(0xffffffffu, ok);
        }
        if (!ok && lead) {
            // every load issued has landed before this CTA leaves: the last use of each barrier
            if (k > 0) drain_phase(bar(C::RF), (k - 1) & 1);
            for (int s = 0; s < C::NV; ++s) {
                const uint32_t uses = g > (uint32_t)s ? (g - s + C::NV - 1) / C::NV : 0;
                if (uses > 0 && (tma_slots >> s & 1)) drain_phase(bar(C::VF + s), (uses - 1) & 1);
            }
            if (tail_uses > 0) drain_phase(bar(C::TAIL), (tail_uses - 1) & 1);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ step 1: S^T of each tile
        // The whole warp runs the loop, one lane issues (see umma_e4m3_elected).
        WideTiles w;
        w.valid = false;
        if (fb < fe) w.init(tile_off, seq0, fb, fe, (int)rank, mode, seq_len);
        const bool lead = elect_one();
        bool ok = true;
        uint32_t g = 0;
        int k = 0, seg = 0;
        while (__all_sync(0xffffffffu, ok && w.valid)) {
            const uint32_t d_s = tmem + C::S_COL + (uint32_t)(k & 1) * 2 * C::NC;
            ok = poll_phase(bar(C::SE + (k & 1)), ((k >> 1) & 1) ^ 1, wc, status);
            if (ok && w.first) ok = poll_phase(bar(C::QF), seg & 1, wc, status);
            ok = ok && poll_phase(bar(C::RF), k & 1, wc, status);
            if (!__all_sync(0xffffffffu, ok)) break;
            tc_fence_after();
#pragma unroll
            for (int j = 0; j < 2; ++j)
                umma_e4m3_elected(lead, d_s, smem_desc(sbase + C::OFF_R + 32u * j, 16, 8 * C::R_ROW, kSwizzle64B),
                                  smem_desc(sbase + C::OFF_QR + 32u * j, 16, 8 * C::R_ROW, kSwizzle64B), C::IDESC_S,
                                  j == 0 ? 0u : 1u);
            if (lead) umma_commit(bar(C::RE));
            __syncwarp();
#pragma unroll 1
            for (int i = 0; i < 4; ++i, ++g) {
                const uint32_t s = g % C::NV;
                ok = poll_phase(bar(C::VF + (int)s), (g / C::NV) & 1, wc, status);
                if (!__all_sync(0xffffffffu, ok)) break;
                tc_fence_after();
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    umma_e4m3_elected(lead, d_s,
                                      smem_desc(sbase + C::OFF_V + s * C::CHUNK + 32u * j, 16, 1024, kSwizzle128B),
                                      smem_desc(sbase + C::OFF_Q + i * C::Q_CHUNK + 32u * j, 16, 1024, kSwizzle128B),
                                      C::IDESC_S, 1u);
            }
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            if (lead) umma_commit(bar(C::SF + (k & 1)));
            __syncwarp();
            ++k;
            if (__any_sync(0xffffffffu, w.advance(tile_off, (int)rank, mode, seq_len))) ++seg;
        }
        if (lead) {
            umma_commit(bar(C::FIN1));
            drain_phase(bar(C::FIN1), 0);
        }
        __syncwarp();
    } else if (warp == 2 || warp == 3) {
        // ------------------------------------------------------------ step 3: O^T (+)= V^T P^T
        // M-tiles 0, 1 (warp 2) and 2, 3 (warp 3); the whole warp runs the loop, one lane issues.
        WideTiles w;
        w.valid = false;
        if (fb < fe) w.init(tile_off, seq0, fb, fe, (int)rank, mode, seq_len);
        const bool lead = elect_one();
        const int i0 = __shfl_sync(0xffffffffu, 2 * (warp - 2), 0);
        bool ok = true;
        int k = 0;
        while (__all_sync(0xffffffffu, ok && w.valid)) {
            ok = poll_phase(bar(C::PF), k & 1, wc, status);
            if (!__all_sync(0xffffffffu, ok)) break;
            const uint32_t fresh = __any_sync(0xffffffffu, w.first) ? 0u : 1u;
#pragma unroll 1
            for (int i = i0; i < i0 + 2; ++i) {
                const uint32_t g = 4u * k + i, s = g % C::NV;
                ok = poll_phase(bar(C::VF + (int)s), (g / C::NV) & 1, wc, status);  // landed for step 1 already
                if (!__all_sync(0xffffffffu, ok)) break;
                tc_fence_after();
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    // A = V^T: M = 128 latent columns (one 128-byte swizzle row), K = 32 KV rows (MN-major)
                    const uint64_t a = smem_desc(sbase + C::OFF_V + s * C::CHUNK + 4096u * r, C::CHUNK, 1024, kSwizzle128B);
#pragma unroll
                    for (int term = 0; term < 2; ++term)
                        umma_e4m3_elected(lead, tmem + C::O_COL + (uint32_t)i * C::NC, a,
                                          smem_desc(sbase + C::OFF_P + term * C::P_TERM + 32u * C::NC * r, C::P_TERM,
                                                    8 * C::NC, kSwizzle64B),
                                          C::IDESC_O, (r == 0 && term == 0) ? fresh : 1u);
                }
                if (lead) umma_commit(bar(C::VE + (int)s));
                __syncwarp();
            }
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            if (lead) umma_commit(bar(C::PE));
            __syncwarp();
            ++k;
            w.advance(tile_off, (int)rank, mode, seq_len);
        }
        if (lead) {
            umma_commit(bar(C::FIN3 + i0 / 2));
            drain_phase(bar(C::FIN3 + i0 / 2), 0);
        }
        __syncwarp();
    } else if (warp >= 4) {
        // ------------------------------------------------------------ softmax + epilogue (warps 4..19)
        constexpr uint32_t SMX = 1, NSM = C::NSM;
        const int quad = warp & 3;          // TMEM lane quadrant this warp may access
        const int cq = (warp - 4) >> 2;     // columns 16 cq .. 16 cq + 15 of this CTA
        const int row = quad * 32 + lane;   // KV row within the tile (= TMEM lane)
        const int tid = (int)threadIdx.x - 128;
        const uint32_t lane_addr = (uint32_t)(quad * 32) << 16;
        float *m_s = reinterpret_cast<float *>(smem + C::OFF_M);
        float *alpha_s = reinterpret_cast<float *>(smem + C::OFF_ALPHA);
        float *qv_s = reinterpret_cast<float *>(smem + C::OFF_QV);
        int *mx_s = reinterpret_cast<int *>(smem + C::OFF_MX);
        if (tid < 2 * C::NC) mx_s[tid] = kOrderedLowest;
        bool ok = true, stop = false;
        int k = 0, seg = 0, merges = 0;
        WideTiles w;
        w.valid = false;
        if (fb < fe) w.init(tile_off, seq0, fb, fe, (int)rank, mode, seq_len);
        // The scale of this thread's row of a tile (1 for rows that are not loaded), in two steps so that
        // neither load is waited for: the row's page, then what stands there.
        auto page_of = [&](const WideTiles &at) -> int {
            const int rg = at.t * kTileRows + row;
            return p.paged && at.valid && rg < at.L ? __ldg(p.block_table + (int64_t)at.b * p.max_blocks + (rg >> 6)) : 0;
        };
        auto read_scale = [&](const WideTiles &at, int page) -> float {
            const int rg = at.t * kTileRows + row;
            if (!at.valid || rg >= at.L || page < 0 || (int64_t)page * kPage >= p.kv_rows) return 1.f;
            return __ldg(p.kv_scale + (p.paged ? (int64_t)page * kPage + (rg & 63) : (int64_t)at.b * p.kv_rows + rg));
        };
        float sig_next = read_scale(w, page_of(w));
        while (!stop && w.valid) {
            // ---- one segment: tiles of sequence b
            const int b = w.b, L = w.L;
            const int nsplit = seq_info[4 * b + 2];
            const int slot = seq_info[4 * b + 3] + (unit - seq_info[4 * b + 1]);
            int qlen_b = p.q_len;
            if (p.q_lens) {
                qlen_b = p.q_lens[b];
                if (qlen_b < 0 || qlen_b > p.q_len) {
                    if (tid == 0) atomicCAS(status, 0, kStatusInvalid);
                    qlen_b = qlen_b < 0 ? 0 : p.q_len;
                }
            }
            // Q of this segment as E4M3 codes [Q_hi ; Q_lo], column n scaled by 2^c_n with
            // 128 < max|q_n| 2^c_n <= 256.  The area is free: the last segment's scores are complete, and
            // its merge data have been read by everyone once this barrier is passed.
            named_bar_sync(SMX, NSM);
            {
                // eight neighbouring threads per column, nine 16-byte loads each
                constexpr int TPC = NSM / C::NC, LOADS = kDqk / 8 / TPC;
                const int n = tid / TPC, part = tid % TPC;
                uint4 raw[LOADS];
                const uint4 *q4 = reinterpret_cast<const uint4 *>(p.q + ((int64_t)b * p.ncols + c0 + n) * kDqk) + part;
#pragma unroll
                for (int i = 0; i < LOADS; ++i)
                    raw[i] = c0 + n < p.ncols ? __ldg(q4 + TPC * i) : make_uint4(0u, 0u, 0u, 0u);
                float amax = 0.f;
#pragma unroll
                for (int i = 0; i < LOADS; ++i) {
                    const uint32_t wv[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(wv[j] << 16)),
                                                 fabsf(__uint_as_float(wv[j] & 0xFFFF0000u))));
                }
#pragma unroll
                for (int o = TPC / 2; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                int c = 0;
                if (amax > 0.f && amax < INFINITY) {
                    // c = 8 - ceil(log2 amax), read off the fp32 exponent and mantissa fields
                    const uint32_t bits = __float_as_uint(amax);
                    c = 8 - ((int)(bits >> 23) - 127 + ((bits & 0x7FFFFFu) != 0u ? 1 : 0));
                    c = c < -100 ? -100 : (c > 100 ? 100 : c);
                }
                if (part == 0) {
                    qv_s[n] = __uint_as_float((uint32_t)(127 - c) << 23);
                    m_s[n] = kNoRow;
                }
                const float sc = __uint_as_float((uint32_t)(127 + c) << 23);
#pragma unroll
                for (int i = 0; i < LOADS; ++i) {
                    const int v8 = part + TPC * i;  // columns 8 v8 .. 8 v8 + 7
                    const uint32_t wv[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
                    uint32_t hi[2] = {0u, 0u}, lo[2] = {0u, 0u};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float a0 = __uint_as_float(wv[j] << 16) * sc;
                        const float a1 = __uint_as_float(wv[j] & 0xFFFF0000u) * sc;
                        const uint16_t h = f32x2_to_e4m3x2(a0, a1);
                        const float2 hf = e4m3x2_to_f32x2(h);
                        const uint16_t l = f32x2_to_e4m3x2(a0 - hf.x, a1 - hf.y);
                        hi[j >> 1] |= (uint32_t)h << (16 * (j & 1));
                        lo[j >> 1] |= (uint32_t)l << (16 * (j & 1));
                    }
                    uint32_t dh, dl;
                    const uint32_t sub = (uint32_t)(v8 & 1) * 8u;
                    if (i < LOADS - 1) {  // latent columns: chunk v8 / 16 (128 codes a row, 128B swizzle)
                        const uint32_t base = C::OFF_Q + (uint32_t)(v8 >> 4) * C::Q_CHUNK;
                        const uint32_t j16 = (uint32_t)(v8 & 15) >> 1;
                        dh = base + swz_off(n, j16, 128, 7) + sub;
                        dl = base + swz_off(C::NC + n, j16, 128, 7) + sub;
                    } else {  // rope columns: 64-byte rows, 64B swizzle
                        const uint32_t j16 = (uint32_t)(v8 - 64) >> 1;
                        dh = C::OFF_QR + swz_off(n, j16, C::R_ROW, 3) + sub;
                        dl = C::OFF_QR + swz_off(C::NC + n, j16, C::R_ROW, 3) + sub;
                    }
                    *reinterpret_cast<uint2 *>(smem + dh) = make_uint2(hi[0], hi[1]);
                    *reinterpret_cast<uint2 *>(smem + dl) = make_uint2(lo[0], lo[1]);
                }
                static_assert(TPC * (LOADS - 1) == 64 && LOADS * TPC * 8 == kDqk, "the last load is the rope columns'");
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0 && !p.withhold_q) mbar_arrive(bar(C::QF));
            named_bar_sync(SMX, NSM);  // qv_s and m_s
            float lpart[16], rq[16];  // column sums of this thread's rows; 2^-c_n * softmax_scale * log2 e
#pragma unroll
            for (int n = 0; n < 16; ++n) {
                lpart[n] = 0.f;
                rq[n] = qv_s[16 * cq + n] * p.scale_log2;
            }
            bool more = true;
            // of this thread's column, if it has one (see etap_common.cuh)
            int seen_tiles = 0;
            Look8 looks;
            if (tid >= C::NC) looks.at = -1;
            float highest = -INFINITY;
            for (; more; ++k, ++seen_tiles) {
                const bool first = w.first;
                const int rg = w.t * kTileRows + row;
                const float sig = fmaxf(sig_next, 0x1p-100f);
                const bool full = (w.t + 1) * kTileRows <= L - qlen_b && c0 + C::NC <= qlen_b * p.num_heads;
                uint32_t seen = 0u;
                if (!full) seen = (uint32_t)tree_sees(p, b, L, qlen_b, rg, c0 + 16 * cq, 16);
                more = !w.advance(tile_off, (int)rank, mode, seq_len);
                const int next_page = page_of(w);  // of the next tile: looked up until the vote
                ok = ok && spin_phase<false>(bar(C::SF + (k & 1)), (k >> 1) & 1, wc, status);
                tc_fence_after();
                float x[16], xl[16];
                tmem_ld16(tmem + lane_addr + C::S_COL + (uint32_t)(k & 1) * 2 * C::NC + 16 * cq, x);
                tmem_ld16(tmem + lane_addr + C::S_COL + (uint32_t)(k & 1) * 2 * C::NC + C::NC + 16 * cq, xl);
                tmem_wait_ld();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(C::SE + (k & 1)));
                // x = score + log2 s; does any pass its column's maximum?
                const float lgs = __log2f(sig);
                const float2 sig2 = make_float2(sig, sig), lgs2 = make_float2(lgs, lgs);
                const float4 *m4 = reinterpret_cast<const float4 *>(m_s + 16 * cq);  // PSCALE - m per column
                float over = -INFINITY;
#pragma unroll
                for (int n = 0; n < 16; n += 2) {
                    const float2 r = mul2(make_float2(rq[n], rq[n + 1]), sig2);
                    const float2 s = add2(make_float2(x[n], x[n + 1]), make_float2(xl[n], xl[n + 1]));
                    const float2 v = fma2(s, r, lgs2);
                    x[n] = v.x;
                    x[n + 1] = v.y;
                }
                if (!full) {
#pragma unroll
                    for (int n = 0; n < 16; ++n) x[n] = (seen >> n) & 1u ? x[n] : -INFINITY;
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float4 mm = m4[q];
                    const float2 d0 = add2(make_float2(x[4 * q], x[4 * q + 1]), make_float2(mm.x, mm.y));
                    const float2 d1 = add2(make_float2(x[4 * q + 2], x[4 * q + 3]), make_float2(mm.z, mm.w));
                    over = fmaxf(over, fmaxf(fmaxf(d0.x, d0.y), fmaxf(d1.x, d1.y)));
                }
                const bool need = seen_tiles == looks.at || !ok || over > kTopLog2_8;
                if (named_bar_or(SMX, NSM, need)) {
                    // ---- the tile's column maxima, m moved where it has to, O^T rescaled
                    if (!named_bar_and(SMX, NSM, ok)) {
                        stop = true;
                        break;
                    }
                    const float wmax = warp_colreduce16<true>(x, lane);
                    if ((lane & 1) == 0)
                        atomicMax(mx_s + (quad >> 1) * C::NC + 16 * cq + col16(lane), ordered_bits(__float_as_int(wmax)));
                    named_bar_sync(SMX, NSM);
                    bool moved = false;
                    if (tid < C::NC) {
                        const float h0 = __int_as_float(ordered_bits(mx_s[tid]));
                        const float h1 = __int_as_float(ordered_bits(mx_s[C::NC + tid]));
                        mx_s[tid] = mx_s[C::NC + tid] = kOrderedLowest;
                        highest = fmaxf(highest, fmaxf(h0, h1));
                        const float from = m_s[tid];
                        const float to = follow_maximum8(from, h0, h1, highest, seen_tiles == looks.at);
                        alpha_s[tid] = fast_exp2(to - from);  // 0 for a column that saw no row so far
                        m_s[tid] = to;
                        moved = to != from && !first;  // (a first tile's O^T does not exist yet)
                        looks.next(seen_tiles, fmaxf(h0, h1) + from);
                    }
                    if (named_bar_or(SMX, NSM, moved)) {
                        // step 3 of the last tile completes first
                        ok = ok && spin_phase<false>(bar(C::PE), (k - 1) & 1, wc, status);
                        tc_fence_after();
                        const float *al = alpha_s + 16 * cq;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            float v[16];
                            const uint32_t addr = tmem + lane_addr + C::O_COL + (uint32_t)i * C::NC + 16 * cq;
                            tmem_ld16(addr, v);
                            tmem_wait_ld();
#pragma unroll
                            for (int n = 0; n < 16; ++n) v[n] *= al[n];
                            tmem_st16(addr, v);
                        }
                        tmem_wait_st();
#pragma unroll
                        for (int n = 0; n < 16; ++n) lpart[n] *= al[n];
                    }
                }
                sig_next = read_scale(w, next_page);  // in flight until the next tile
                // ---- P^T: stored 2^(score + log2 s - m + PSCALE), summed as 2^(score - m)
                const float inv = kPUnit8 / sig;
                const float2 inv2 = make_float2(inv, inv), dith = make_float2(dither8(row), dither8(row));
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float4 mm = m4[q];
                    uint32_t h2[2], l2[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int n = 4 * q + 2 * e;
                        const float2 nm = e == 0 ? make_float2(mm.x, mm.y) : make_float2(mm.z, mm.w);
                        const float2 d = add2(make_float2(x[n], x[n + 1]), nm);
                        const float2 pv = make_float2(fast_exp2(d.x), fast_exp2(d.y));
                        const float2 sum = fma2(pv, inv2, make_float2(lpart[n], lpart[n + 1]));
                        lpart[n] = sum.x;
                        lpart[n + 1] = sum.y;
                        const uint16_t h = f32x2_to_e4m3x2(pv.x, pv.y);
                        const float2 f = e4m3x2_to_f32x2(h);
                        h2[e] = h;
                        const float2 rest = add2(pv, dith);
                        l2[e] = f32x2_to_e4m3x2(rest.x - f.x, rest.y - f.y);
                    }
                    hi[q] = h2[0] | h2[1] << 16;
                    lo[q] = l2[0] | l2[1] << 16;
                }
                if (k > 0) ok = ok && spin_phase<false>(bar(C::PE), (k - 1) & 1, wc, status);
                uint8_t *dst = smem + C::OFF_P + swz_off(row, cq, C::NC, 3);
                *reinterpret_cast<uint4 *>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                *reinterpret_cast<uint4 *>(dst + C::P_TERM) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(C::PF));
            }
            if (stop) break;
            // ---------------------------------------------------- epilogue of the segment
            // Its scores are complete, so the Q area is idle: the peer may send its part there (it hears so
            // ahead of time), and the column sums are added up behind that, while step 3 of the last tile runs.
            if (mode == 0 && tid == 0) mbar_arrive_remote(map_to_rank(bar(C::XFREE), peer));
            float *sums = reinterpret_cast<float *>(smem + C::OFF_SUM);  // [4][64]
            {
                const float wsum = warp_colreduce16<false>(lpart, lane);
                if ((lane & 1) == 0) sums[quad * C::NC + 16 * cq + col16(lane)] = wsum;
            }
            ok = ok && spin_phase<false>(bar(C::PE), (k - 1) & 1, wc, status);
            if (!named_bar_and(SMX, NSM, ok)) {
                stop = true;
                break;
            }
            tc_fence_after();
            // one thread per column: its sum, (mode 0) both CTAs' parts merged by the log-sum-exp rule, its LSE
            // and the factors of the two parts in the output, P^T's 2^PSCALE included
            float l_own = 0.f;
            if (tid < C::NC)
                l_own = (sums[tid] + sums[C::NC + tid]) + (sums[2 * C::NC + tid] + sums[3 * C::NC + tid]);
            auto finish_column = [&](float mm, float l, float as, float ap) {
                const bool empty = !(l > 0.f);
                const float inv = empty ? 0.f : kPUnit8 / l;
                alpha_s[tid] = as * inv;
                qv_s[tid] = ap * inv;
                if (c0 + tid < p.ncols && (mode == 1 || rank == 0)) {
                    const float v = empty ? -INFINITY : (mm + __log2f(l)) * 0.69314718055994531f;
                    if (nsplit == 1)
                        p.lse[(int64_t)b * p.ncols + c0 + tid] = v;
                    else
                        p.lsepart[(int64_t)slot * p.ncols + c0 + tid] = v;
                }
            };
            // 16 columns of latent row d: outputs of an unsplit sequence, else partials
            const int cols = min(p.ncols - (c0 + 16 * cq), 16);
            auto store16 = [&](int d, const float (&v)[16]) {
                if (nsplit == 1) {
                    __nv_bfloat16 *o = p.o + ((int64_t)b * p.ncols + c0 + 16 * cq) * kDv + d;
#pragma unroll
                    for (int n = 0; n < 16; ++n)
                        if (n < cols) o[n * kDv] = __float2bfloat16_rn(v[n]);
                } else {
                    float *o = p.opart + ((int64_t)slot * p.ncols + c0 + 16 * cq) * kDv + d;
#pragma unroll
                    for (int n = 0; n < 16; ++n)
                        if (n < cols) o[n * kDv] = v[n];
                }
            };
            const float4 *fa = reinterpret_cast<const float4 *>(alpha_s + 16 * cq);
            const float4 *fb = reinterpret_cast<const float4 *>(qv_s + 16 * cq);
            if (mode == 1) {
                if (tid < C::NC) finish_column(kPScaleLog2_8 - m_s[tid], l_own, 1.f, 0.f);
                named_bar_sync(SMX, NSM);
#pragma unroll 1
                for (int i = 0; i < 4; ++i) {
                    float v[16];
                    tmem_ld16(tmem + lane_addr + C::O_COL + (uint32_t)i * C::NC + 16 * cq, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float4 a = fa[q];
                        v[4 * q] *= a.x, v[4 * q + 1] *= a.y, v[4 * q + 2] *= a.z, v[4 * q + 3] *= a.w;
                    }
                    store16(128 * i + row, v);
                }
            } else {
                // The two CTAs hold disjoint rows of the same columns: each finishes latent rows
                // 256 rank .., so it sends the other two M-tiles and its (m, l) to the peer, into its Q area,
                // once the peer has said that this area is idle (above).
                const uint32_t x_peer = map_to_rank(sbase + C::OFF_XM, peer);
                const uint32_t ml_peer = map_to_rank(sbase + C::OFF_XML, peer);
                const uint32_t xfull_peer = map_to_rank(bar(C::XFULL), peer);
                ok = ok && spin_phase<true>(bar(C::XFREE), merges & 1, wc, status);
                if (tid < C::NC && ok) {
                    st_async_b32(ml_peer + 4u * tid, __float_as_uint(m_s[tid]), xfull_peer);
                    st_async_b32(ml_peer + 4u * (C::NC + tid), __float_as_uint(l_own), xfull_peer);
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float v[16];
                    tmem_ld16(tmem + lane_addr + C::O_COL + (2u * peer + j) * C::NC + 16 * cq, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int q = 0; q < 4 && ok; ++q)
                        st_async_v4(x_peer + (uint32_t)j * C::XM_TILE + (uint32_t)(4 * cq + q) * 2048u +
                                        (uint32_t)row * 16u,
                                    __float_as_uint(v[4 * q]), __float_as_uint(v[4 * q + 1]),
                                    __float_as_uint(v[4 * q + 2]), __float_as_uint(v[4 * q + 3]), xfull_peer);
                }
                if (tid == 0) mbar_arrive_expect_tx(bar(C::XFULL), C::X_BYTES);
                ok = ok && spin_phase<true>(bar(C::XFULL), merges & 1, wc, status);
                ++merges;
                const float4 *xs = reinterpret_cast<const float4 *>(smem + C::OFF_XM);
                const float *ml = reinterpret_cast<const float *>(smem + C::OFF_XML);
                if (tid < C::NC) {
                    const float m = kPScaleLog2_8 - m_s[tid], mp = kPScaleLog2_8 - ml[tid], lp = ml[C::NC + tid];
                    const float mm = fmaxf(m, mp);
                    const float as = fast_exp2(m - mm), ap = fast_exp2(mp - mm);  // 0 for a part without rows
                    // rank 0's term first in both CTAs, so that both compute the same l
                    const float l = rank == 0 ? __fmaf_rn(l_own, as, __fmul_rn(lp, ap))
                                              : __fmaf_rn(lp, ap, __fmul_rn(l_own, as));
                    finish_column(mm, l, as, ap);
                }
                if (!named_bar_and(SMX, NSM, ok)) {
                    stop = true;
                    break;
                }
#pragma unroll 1
                for (int j = 0; j < 2; ++j) {
                    float v[16];
                    tmem_ld16(tmem + lane_addr + C::O_COL + (2u * rank + j) * C::NC + 16 * cq, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float4 a = fa[q], c = fb[q], x = xs[(j * C::XM_TILE >> 4) + (4 * cq + q) * 128 + row];
                        v[4 * q] = v[4 * q] * a.x + x.x * c.x;
                        v[4 * q + 1] = v[4 * q + 1] * a.y + x.y * c.y;
                        v[4 * q + 2] = v[4 * q + 2] * a.z + x.z * c.z;
                        v[4 * q + 3] = v[4 * q + 3] * a.w + x.w * c.w;
                    }
                    store16(256 * (int)rank + 128 * j + row, v);
                }
            }
            if (nsplit >= 2 && p.signal_combine) {
                // this CTA's part of the split is stored: count it for the combine kernel (release: the CTA
                // barrier and one thread's release add cover every thread's stores)
                named_bar_sync(SMX, NSM);
                if (tid == 0) red_add_release_gpu(p.counters + ((int64_t)b * groups + grp) * 2 + rank, 1);
            }
            tc_fence_before();
            ++seg;
        }
        if (stop || !ok) wc->abort = 1;
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // no CTA leaves while its peer may still write into its shared memory
    if (wc->abort) {
        // After an abort a peer's last st.async may not have been waited for: let it land before either
        // CTA leaves (no thread sends after the barrier above).
        const uint64_t t_q = global_timer_ns();
        while (global_timer_ns() - t_q < 20000ull) {
        }
    }
    cluster_sync();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

}  // namespace mla
