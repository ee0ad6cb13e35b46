// ETAP decode on a pair of SMs with M = 256 KV rows per tensor-core instruction, sm_100a.
//
// Computation (FlashMLA-ETAP technical summary, "Methodology", ETAP steps 1-4): S^T = K Q^T with
// the KV rows as the UMMA M dimension and the query columns (heads x tokens) as N; P^T = softmax
// of S^T down each column; O^T = V^T P^T; O = (O^T)^T.  The pages keep a producer that streams
// KV into a circular shared-memory buffer and consumers that compute scores and softmax
// statistics block by block ("Integration and Implementation"); this kernel keeps those roles
// and lays the two contractions out for Blackwell's CTA-pair tensor cores:
//
//   * A cluster of two CTAs owns 256-row units of one sequence: CTA r holds rows 128r..128r+127
//     of every unit.  Step 1 is tcgen05.mma.cta_group::2 with M = 256: each CTA supplies its 128
//     K rows (A) and half of the group's query columns (B = Q^T, split by columns, so that a
//     128-column group costs each CTA 72 KB of Q); each CTA's TMEM receives S^T of its own rows
//     for all columns.
//   * Step 3 is also M = 256 across the pair, now over latent rows: CTA r accumulates O^T for
//     latent rows 256r..256r+255 (two M-blocks of 128, paired with the peer's) and supplies, as
//     B, P^T of its half of the columns for all 256 KV rows of the unit.  So each CTA sends the
//     peer P^T of its rows for the peer's columns (st.async, 16 KB per unit) and loads, from L2,
//     the value columns of the peer's rows that its M-blocks need (the scores pass streamed its
//     own rows through a separate ring: nothing is held between the two steps).
//   * The softmax is taken down each column over the rows of both CTAs with one running maximum
//     per column, kept identical in both CTAs: it moves only when some score exceeds it by
//     2^THRESH; the vote travels with the P^T exchange, so the common case needs no extra
//     round trip.  When a vote is raised, both CTAs exchange their tile maxima, rescale their
//     O^T in TMEM and redo the tile's P^T.
//   * Column groups of 64 store P as bf16 hi + lo (N = 128 for step 3: [hi | lo] per CTA);
//     groups of 128 store one bf16 term, used when every sequence of the batch is long enough
//     (the plan decides; see plan_core.h).  Tree decodes (TREE) test mask bits in the tiles that
//     reach into the new rows, and may take groups of 128 with short sequences among them, whose
//     P is then multiplied as hi and lo in two passes.  In their groups of 128 the sums of P's terms are taken by
//     mma.sync (sum_columns8), so that O of one pass can be divided by the sum of what was multiplied: 512 columns at
//     B=8, 8192..32768 rows 178 -> 189 us for it.
//
// Measured, kernel and combine: B=32 h=128, 786 MB: 0.216 ms, 3.6 TB/s, 879 TFLOP/s, 0.56 of the HBM
// roof; B=16 q_len=4 h=16, 604 MB: 0.144 ms, 4.2 TB/s, 0.64; 256 columns on 32768 rows: 1051 TFLOP/s,
// 0.64 of the tensor roof.  Neither is reached: at 64 columns a unit takes 4.1 us, its nine K chunks 3.7
// (1.3 us from a load's issue to its use, four slots) and the chain P^T, step 3, P^T's release 4.0 (step 3
// waits 0.7 for its third value pair); deeper rings for both do not fit.  16 softmax warps instead of 8
// took 152 us instead of 150, at 512 columns 196 instead of 185 (these, and the rings' figures below, replayed from a
// graph).  The tensor pipe is 40..50 % busy.
//
// The roles that issue loads and matrix instructions run as whole warps, one elected lane per
// instruction: a loop run by one lane alone takes 80..130 cycles per instruction, a warp's about 50
// (B=32 h=128 0.267 -> 0.22 ms with the shorter softmax that it made worth while).
// Warp roles per CTA (12 warps): 0 loads K tiles and Q (TMA; the bytes of both CTAs count on
// the even CTA's barriers), 1 issues step 1 (even CTA only) and owns TMEM, 2 loads the value
// columns for step 3, 3..10 run the softmax and the epilogue (two warps per TMEM lane quadrant,
// one KV row and half of the columns per thread), 11 issues step 3 in the even CTA (a thread that
// issues MMAs blocks while the tensor pipe drains, so step 1's chunks are not queued behind it) and
// in the odd CTA tells the even one when the even CTA's P^T part has landed here.
// Every wait is bounded; see etap_common.cuh.
#pragma once

#include <type_traits>

#include "etap_common.cuh"
#include "plan_check.cuh"

namespace mla {

// Shared-memory control block (identical in both configurations, so that one prologue serves both).
constexpr uint32_t kDuoCtlBar = 0;        // mbarriers
constexpr uint32_t kDuoCtlMisc = 512;     // +0 TMEM address, +16 WaitCtl, +64 received votes (2 x 16 B)
constexpr uint32_t kDuoCtlM = 1024;       // float[128] running maximum per column (log2 units)
constexpr uint32_t kDuoCtlAlpha = 1536;   // float[128] rescale factor of the current tile pair
constexpr uint32_t kDuoCtlRed = 2048;     // float[4][128] per-quadrant partial maxima / sums
constexpr uint32_t kDuoCtlMx = 4096;      // float[128] peer's tile maxima (received)
constexpr uint32_t kDuoCtlLx = 4608;      // float[128] peer's row sums (received)
constexpr uint32_t kDuoCtlMt = 5120;      // float[128] this CTA's tile maxima / row sums
constexpr uint32_t kDuoCtlVis = 5632;     // int[128] visible rows per column of the current sequence
constexpr uint32_t kDuoCtlNm = 6144;      // float[128] minus the running maximum (kNoRow: no row seen yet)
constexpr uint32_t kDuoCtlLr = 6656;      // float[128] peer's sums of rounded P (received; one-term trees)
constexpr uint32_t kDuoCtlEnd = 7168;     // data regions start here (1024-aligned)
constexpr int kDuoThreads = 384;
constexpr int kDuoMaxSlots = 4;           // slots per operand ring that have barriers

// NC query columns per cluster, P as hi + lo (SPLIT), NS1 K-chunk slots, NS3 value-pair slots.
template <int NC_, bool SPLIT_, int NS1_, int NS3_>
struct DuoCfg {
    static constexpr int NC = NC_;
    static constexpr bool SPLIT = SPLIT_;
    static constexpr int NH = NC / 2;               // columns of Q^T / P^T this CTA holds (its half)
    static constexpr int NP = SPLIT ? 2 * NC : NC;  // UMMA N of step 3
    static constexpr int NPH = NP / 2;              // step-3 B columns per CTA
    static constexpr int NS1 = NS1_, NS3 = NS3_;
    static constexpr uint32_t CHUNK = 16384;        // 128 rows x 64 bf16, 128B swizzle
    static constexpr uint32_t HALF = 8192;          // 64 rows of a chunk: one TMA box
    static constexpr uint32_t VPAIR = 2 * CHUNK;    // 128 rows x 128 latent columns (two chunks)
    static constexpr uint32_t Q_CHUNK = NH * 128;   // NH rows x 64 columns
    static constexpr uint32_t P_PITCH = NPH * 2;    // bytes per KV row of a P^T buffer
    static constexpr uint32_t P_BUF = 128 * P_PITCH;
    static constexpr uint32_t OFF_S1 = kDuoCtlEnd;
    static constexpr uint32_t OFF_S3 = OFF_S1 + NS1 * CHUNK;
    static constexpr uint32_t OFF_Q = OFF_S3 + NS3 * VPAIR;
    static constexpr uint32_t OFF_P = OFF_Q + 9 * Q_CHUNK;  // P^T buffer of K-half 0 (rows of CTA 0), then 1
    static constexpr uint32_t BYTES = OFF_P + 2 * P_BUF;
    static constexpr uint32_t O_COL = 0;                   // 2 M-blocks x NP columns
    static constexpr uint32_t S_COL = 2 * NP;              // 2 buffers x NC columns
    static constexpr uint32_t IDESC_S = idesc_bf16_f32(256, NC, 0, 0);
    static constexpr uint32_t IDESC_O = idesc_bf16_f32(256, NP, 1, 1);
};
// Ring slots, measured: 64 columns at B=16, q_len*h=64, 32768 rows: 4 K chunks + 2 value pairs 152 us, 3 + 3
// 158 us, 5 + 2 154 us (value slots of half the size, 4 + 5: no gain over 4 + 2); 128 columns at B=8,
// h=128, q_len=4: 5 + 1 slots take 12 % longer than 3 + 2, half-size slots 3 + 4 4 % longer.
using DuoCfg64 = DuoCfg<64, true, 4, 2>;     // 64 columns, P as bf16 hi + lo
using DuoCfg128 = DuoCfg<128, false, 3, 2>;  // 128 columns, one bf16 P term
constexpr uint32_t kDuoSmemAlloc =
    (DuoCfg64::BYTES > DuoCfg128::BYTES ? DuoCfg64::BYTES : DuoCfg128::BYTES) + 1024;  // + alignment slack

template <class C>
constexpr bool duo_cfg_fits() {
    return C::BYTES + 1024 <= 232448 && kDuoCtlNm + 512 <= kDuoCtlLr && kDuoCtlLr + 512 <= kDuoCtlEnd && C::S_COL + 2 * C::NC <= 512 && C::P_PITCH == 128 &&
           C::NS1 <= kDuoMaxSlots && C::NS3 <= kDuoMaxSlots && C::OFF_Q % 1024 == 0 && C::OFF_P % 1024 == 0 && C::NC <= 128 && C::NH % 16 == 0;
}
static_assert(duo_cfg_fits<DuoCfg64>() && duo_cfg_fits<DuoCfg128>(), "shared memory / TMEM plan");

// Barrier indices (the same in both configurations; slot barriers sized for kDuoMaxSlots slots).  Barriers
// that gather both CTAs (S1F, S3F, QF, SE, PF0, PF1) are used in the even CTA only.  Step 3 runs in
// two K-halves: K-half h reads the P^T buffers that CTA h's softmax fills (its own columns in place,
// the peer's columns through st.async), so PF_h / PE_h track them separately and CTA h refills
// them as soon as the previous unit's K-half h is done.
struct DuoBars {
    static constexpr int S1F = 0, S1E = S1F + kDuoMaxSlots, S3F = S1E + kDuoMaxSlots, S3E = S3F + kDuoMaxSlots,
                         QF = S3E + kDuoMaxSlots, QE = QF + 1, SF = QF + 2, SE = QF + 4, PF0 = QF + 6, PF1 = QF + 7,
                         PE0 = QF + 8, PE1 = QF + 9, XF = QF + 10, XV = QF + 11, XM = QF + 12, XL = QF + 13,
                         TAIL = QF + 14, FINAL = QF + 15, FINAL3 = QF + 16, COUNT = QF + 17;
};
static_assert(DuoBars::COUNT * 8 <= kDuoCtlMisc, "barrier area");

struct DuoMaps {
    CUtensorMap q32, q64, kv;  // Q with 32- and 64-row boxes; the latent cache with 64 x 64 boxes
};

// Trace events (mla_decode_fwd_trace): role 0 K-tile producer, 1 step-1 issuer, 2 value producer,
// 3 softmax (its first thread), 4 step-3 issuer.
enum : int {
    kEvKChunk = 1,      // a K chunk's slot is free and its loads are issued (index: chunk count)
    kEvQ = 2,           // a segment's Q loads are issued
    kEvS1Begin = 10,    // step 1 of a unit may start (S^T buffer free, Q landed)
    kEvS1Chunk = 11,    // step-1 MMAs of one chunk issued (index: chunk 0..8)
    kEvS1Done = 12,     // step 1 of a unit committed (index: unit count)
    kEvPReady = 13,     // both CTAs' P^T of a unit observed
    kEvS3Pair = 14,     // step-3 MMAs of one value pair issued (index 0..3)
    kEvS3Done = 15,     // step 3 of a unit committed
    kEvVPair = 20,      // a value pair's slot is free and its loads are issued (index: pair count)
    kEvSmS = 30,        // softmax: S^T of a unit observed
    kEvSmVote = 31,     // softmax: vote taken
    kEvSmPe = 32,       // softmax: previous unit's step 3 observed complete
    kEvSmX = 33,        // softmax: exchange round complete
    kEvSmSlow = 34,     // softmax: the slow path begins
    kEvSmDone = 35,     // softmax: P^T ready and S^T released
    kEvSmEpi = 36,      // softmax: epilogue begins
    kEvSmEpiDone = 37,  // softmax: epilogue ends
    kEvEpiS3 = 38,      // epilogue: the segment's last step 3 observed complete
    kEvEpiL = 39,       // epilogue: column sums of both CTAs known
    kEvEpiO = 40        // epilogue: outputs (or partials) stored
};

// Adds to acc the column sums of 8 columns of bf16 pairs over the rows (lanes) of a warp, four rows a lane group: lane
// (g, q) = (lane / 4, lane % 4) gives, as rows g and g + 8 of the 16 x 16 operand, words 0, 2 and 1, 3 of its KV row
// (places 2q, 2q + 1 and 8 + 2q, 9 + 2q), and the other operand sends places of equal parity and half to one
// result column each: columns 0..3 of the result for `second` = 0, 4..7 for 1.  So acc[0..3] of lanes with q = 0, 1 are
// columns 4q .. 4q + 3 of the first eight, with q = 2, 3 those of the second.  (8 instructions for 64 columns of a
// warp's rows, instead of 64 additions and as many registers a thread.)
__device__ __forceinline__ void sum_columns8(float (&acc)[4], const uint32_t (&w)[4], int lane, int second) {
    const int n = (lane >> 2) - 4 * second;
    const uint32_t b0 = n == 0 ? 0x3F80u : n == 1 ? 0x3F800000u : 0u, b1 = n == 2 ? 0x3F80u : n == 3 ? 0x3F800000u : 0u;
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(acc[0]), "+f"(acc[1]), "+f"(acc[2]), "+f"(acc[3])
        : "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(b0), "r"(b1));
}

template <class C, bool TR, bool TREE>
__device__ __forceinline__ void duo_body(const DuoMaps &tm, const DecodeParams &p, uint8_t *smem, uint32_t sbase,
                                         uint32_t tmem, uint32_t rank, int unit, int grp, int groups, bool has_work,
                                         volatile WaitCtl *wc, int32_t *status, bool &pv_pending) {
    using BR = DuoBars;
    constexpr int NC = C::NC, NH = C::NH;
    // One-term groups of a tree decode: O is divided by the sum of P's rounded terms
    constexpr bool TWO_SUMS = TREE && !C::SPLIT;
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t peer = rank ^ 1u;
    const bool leader = rank == 0;
    auto bar = [&](int i) -> uint32_t { return sbase + kDuoCtlBar + 8u * (uint32_t)i; };
    // the even CTA's barrier i as a cluster address (its own barrier when this is the even CTA)
    auto bar0 = [&](int i) -> uint32_t { return map_to_rank(bar(i), 0); };
    // announce transaction bytes on the even CTA's barrier i
    auto expect0 = [&](int i, uint32_t bytes) {
        if (leader)
            mbar_arrive_expect_tx(bar(i), bytes);
        else
            mbar_arrive_expect_tx_remote(bar0(i), bytes);
    };
    // plain arrival on the even CTA's barrier i, ordering this thread's (and, after a barrier,
    // its CTA's) earlier shared-memory accesses before the even CTA's acquire
    auto arrive0 = [&](int i) {
        if (leader) {
            mbar_arrive(bar(i));
        } else {
            mbar_arrive_remote(bar0(i));
        }
    };
    const int32_t *ranges = p.ws + p.cta_ranges_off;
    const int32_t *tile_off = p.ws + p.tile_off_off;
    const int32_t *seq_info = p.ws + p.seq_info_off;
    const int64_t fb = has_work ? ranges[2 * unit] : 0, fe = has_work ? ranges[2 * unit + 1] : 0;
    const int seq0 = has_work ? p.ws[p.cta_seq_off + unit] : 0;
    const int64_t l_cap = p.paged ? (int64_t)p.max_blocks * kPage : p.kv_rows;
    const CUtensorMap *tm_q = NH == 32 ? &tm.q32 : &tm.q64;

    // Cache rows of the 64-row boxes [row0, row0 + 128) of sequence b: y coordinates, which boxes
    // exist, and how many rows are valid.  A block-table entry outside the pool is not used and
    // raises the status word.
    auto locate = [&](int b, int row0, int L, int (&y)[2], bool (&loaded)[2]) -> int {
        int valid = L - row0;
        valid = valid < 0 ? 0 : (valid > kTileRows ? kTileRows : valid);
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            loaded[hh] = valid > 64 * hh;
            y[hh] = 0;
            if (loaded[hh]) {
                if (p.paged) {
                    const int blk = p.block_table[(int64_t)b * p.max_blocks + (row0 >> 6) + hh];
                    if (blk < 0 || (int64_t)blk * kPage >= p.kv_rows) {
                        if (lane == 0) atomicCAS(status, 0, kStatusBlockTable);
                        loaded[hh] = false;
                    } else {
                        y[hh] = blk * kPage;
                    }
                } else {
                    y[hh] = (int)((int64_t)b * p.kv_rows + row0 + 64 * hh);
                }
            }
        }
        return valid;
    };
    auto seq_len = [&](int b) -> int {
        int L = p.seqlens[b];
        if ((int64_t)L > l_cap) {
            if (lane == 0) atomicCAS(status, 0, kStatusInvalid);
            L = (int)l_cap;
        }
        return L < 0 ? 0 : L;
    };

    // Passes of step 3 over a unit of sequence b.  In 128-column groups the tree schedule also holds
    // sequences for which one bf16 P term is not accurate enough: their units are multiplied twice, by
    // P_hi and then by what its rounding left (the value columns are loaded again, from L2).
    auto passes_of = [&](int L) -> int {
        if constexpr (TREE && !C::SPLIT)
            return L < kSingleP_MinRows ? 2 : 1;
        else
            return 1;
    };

    if (warp == 0) {
        // ------------------------------------------------------------ K tiles and Q (step-1 operands)
        // The loops of warps 0, 1, 2 and 11 are run by the whole warp; one lane issues (see elect_one).
        const bool lead = elect_one();
        bool ok = true;
        TraceRowT<TR> tr;
        tr.init(p, 0);
        if (!lead) tr.row = nullptr;
        TileCursor w;
        w.valid = false;
        if (fb < fe) w.init(tile_off, seq0, fb, fe);
        int seg = 0, y[2];
        bool loaded[2];
        uint32_t g1 = 0;
        if (w.valid) locate(w.b, w.t * kDuoRows + kTileRows * (int)rank, seq_len(w.b), y, loaded);
        while (__all_sync(0xffffffffu, ok && w.valid)) {
            const int y0 = __shfl_sync(0xffffffffu, loaded[0] ? y[0] : -1, 0);
            const int y1 = __shfl_sync(0xffffffffu, loaded[1] ? y[1] : -1, 0);
            const uint32_t nload = (y0 >= 0 ? 1u : 0u) + (y1 >= 0 ? 1u : 0u);
            if (__any_sync(0xffffffffu, w.first())) {
                if (seg > 0) ok = poll_phase(bar(BR::QE), (seg - 1) & 1, wc, status);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if (!p.withhold_q && lead) {
                    expect0(BR::QF, 9 * C::Q_CHUNK);
                    const int qrow = w.b * p.ncols + grp * NC + (int)rank * NH;
                    for (int i = 0; i < 9; ++i)
                        tma_load_2d_pair(sbase + C::OFF_Q + i * C::Q_CHUNK, tm_q, bar0(BR::QF), 64 * i, qrow);
                    tr.put(kEvQ, seg);
                }
                __syncwarp();
                ++seg;
            }
            // the next unit's rows are looked up while this one's slots come free
            w.advance(tile_off);
            if (w.valid) locate(w.b, w.t * kDuoRows + kTileRows * (int)rank, seq_len(w.b), y, loaded);
            // rows past the end need no zeroing here: their scores are masked to -inf
#pragma unroll 1
            for (int i = 0; i < 9; ++i, ++g1) {
                const uint32_t s = g1 % C::NS1;
                ok = poll_phase(bar(BR::S1E + (int)s), ((g1 / C::NS1) & 1) ^ 1, wc, status);
                if (!__all_sync(0xffffffffu, ok)) break;
                if (lead) {
                    expect0(BR::S1F + (int)s, nload * C::HALF);
                    const uint32_t dst = sbase + C::OFF_S1 + s * C::CHUNK;
                    if (y0 >= 0) tma_load_2d_pair(dst, &tm.kv, bar0(BR::S1F + (int)s), 64 * i, y0);
                    if (y1 >= 0) tma_load_2d_pair(dst + C::HALF, &tm.kv, bar0(BR::S1F + (int)s), 64 * i, y1);
                    tr.put(kEvKChunk, (int)g1);
                }
                __syncwarp();
            }
            ok = __all_sync(0xffffffffu, ok);
        }
        // Tail: the last releases of the slots and of Q arrive by multicast commit; wait for them
        // so that nothing lands in this CTA's shared memory after it leaves.
        if (fb < fe) {
            for (uint32_t g = g1; ok && g < g1 + C::NS1; ++g)
                ok = poll_phase(bar(BR::S1E + (int)(g % C::NS1)), ((g / C::NS1) & 1) ^ 1, wc, status);
            if (ok && seg > 0) ok = poll_phase(bar(BR::QE), (seg - 1) & 1, wc, status);
        }
        __syncwarp();
    } else if (warp == 2) {
        // ------------------------------------------------------------ value columns (step-3 operands)
        // Unit tp, K-half h (rows 256 tp + 128 h ..), M-block j: this CTA's latent columns
        // 256 rank + 128 j .. + 127 of those rows, as one 32 KB slot of two 64-column chunks.
        const bool lead = elect_one();
        bool ok = true;
        TraceRowT<TR> tr;
        tr.init(p, 2);
        if (!lead) tr.row = nullptr;
        TileCursor w;
        w.valid = false;
        if (fb < fe) w.init(tile_off, seq0, fb, fe);
        int tail_uses = 0, L = 0, t = 0, y[2][2];
        bool loaded[2][2];
        uint32_t g3 = 0;
        auto look_up = [&] {  // both K-halves of the unit
            if (!w.valid) return;
            L = seq_len(w.b);
            t = w.t;
            locate(w.b, t * kDuoRows, L, y[0], loaded[0]);
            locate(w.b, t * kDuoRows + kTileRows, L, y[1], loaded[1]);
        };
        look_up();
        while (__all_sync(0xffffffffu, ok && w.valid)) {
            int ya[2], yb[2], valid[2];
            const int passes = __shfl_sync(0xffffffffu, passes_of(L), 0);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                ya[h] = __shfl_sync(0xffffffffu, loaded[h][0] ? y[h][0] : -1, 0);
                yb[h] = __shfl_sync(0xffffffffu, loaded[h][1] ? y[h][1] : -1, 0);
                valid[h] = __shfl_sync(0xffffffffu, min(max(L - t * kDuoRows - kTileRows * h, 0), kTileRows), 0);
            }
            w.advance(tile_off);
            look_up();  // of the next unit, while this one's slots come free
#pragma unroll 1
            for (int pass = 0; pass < passes && ok; ++pass)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll 1
                for (int j = 0; j < 2; ++j, ++g3) {
                    const uint32_t s = g3 % C::NS3;
                    ok = poll_phase(bar(BR::S3E + (int)s), ((g3 / C::NS3) & 1) ^ 1, wc, status);
                    if (!__all_sync(0xffffffffu, ok)) break;
                    const int x0 = 256 * (int)rank + 128 * j;
                    const uint32_t dst = sbase + C::OFF_S3 + s * C::VPAIR;
                    if (valid[h] == kTileRows && ya[h] >= 0 && yb[h] >= 0) {
                        if (lead) {
                            expect0(BR::S3F + (int)s, C::VPAIR);
#pragma unroll
                            for (int hc = 0; hc < 2; ++hc) {
                                tma_load_2d_pair(dst + hc * C::CHUNK, &tm.kv, bar0(BR::S3F + (int)s), x0 + 64 * hc, ya[h]);
                                tma_load_2d_pair(dst + hc * C::CHUNK + C::HALF, &tm.kv, bar0(BR::S3F + (int)s),
                                                 x0 + 64 * hc, yb[h]);
                            }
                            tr.put(kEvVPair, (int)g3);
                        }
                        __syncwarp();
                    } else {
                        // a tail: land the valid rows, zero all others, so that whatever the cache (or
                        // the slot) holds there meets P = 0 as an exact 0
                        const int nload = (ya[h] >= 0 ? 1 : 0) + (yb[h] >= 0 ? 1 : 0);
                        if (nload > 0) {
                            if (lead) {
                                mbar_arrive_expect_tx(bar(BR::TAIL), 2 * nload * C::HALF);
                                for (int hc = 0; hc < 2; ++hc) {
                                    if (ya[h] >= 0)
                                        tma_load_2d(dst + hc * C::CHUNK, &tm.kv, bar(BR::TAIL), x0 + 64 * hc, ya[h]);
                                    if (yb[h] >= 0)
                                        tma_load_2d(dst + hc * C::CHUNK + C::HALF, &tm.kv, bar(BR::TAIL), x0 + 64 * hc,
                                                    yb[h]);
                                }
                            }
                            __syncwarp();
                            ok = wait_phase(bar(BR::TAIL), tail_uses & 1, wc, status);
                            ++tail_uses;
                            if (!__all_sync(0xffffffffu, ok)) break;
                        }
                        for (int idx = lane; idx < 2 * kTileRows * 8; idx += 32) {
                            const int hc = idx / (kTileRows * 8);
                            const int r = (idx / 8) % kTileRows;
                            const int c16 = idx % 8;
                            if (r < valid[h] && (r < 64 ? ya[h] : yb[h]) >= 0) continue;
                            *reinterpret_cast<uint4 *>(smem + C::OFF_S3 + s * C::VPAIR + hc * C::CHUNK + r * 128 +
                                                       c16 * 16) = make_uint4(0u, 0u, 0u, 0u);
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lead) arrive0(BR::S3F + (int)s);
                        __syncwarp();
                    }
                }
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
            }
        }
        // Tail: the last slot releases (multicast commits) land before this CTA leaves.
        if (fb < fe)
            for (uint32_t g = g3; ok && g < g3 + C::NS3; ++g)
                ok = poll_phase(bar(BR::S3E + (int)(g % C::NS3)), ((g / C::NS3) & 1) ^ 1, wc, status);
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ step-1 issuer (even CTA)
        // Step 1 of each unit chunk by chunk as its K tiles land in both CTAs.
        if (leader && fb < fe) {
            const bool lead = elect_one();
            const uint64_t q_desc0 = smem_desc(sbase + C::OFF_Q, 16, 1024, kSwizzle128B);
            const uint64_t k_desc0 = smem_desc(sbase + C::OFF_S1, 16, 1024, kSwizzle128B);
            TileCursor qc;
            qc.init(tile_off, seq0, fb, fe);
            bool ok = true;
            int kq = 0, seg_q = 0;
            uint32_t g1 = 0;
            TraceRowT<TR> tr;
            tr.init(p, 1);
            if (!lead) tr.row = nullptr;
            while (__all_sync(0xffffffffu, ok && qc.valid)) {
                const uint32_t d_s = tmem + C::S_COL + (uint32_t)(kq & 1) * NC;
                ok = poll_phase_cluster(bar(BR::SE + (kq & 1)), ((kq >> 1) & 1) ^ 1, wc, status);
                if (ok && qc.first()) ok = poll_phase_cluster(bar(BR::QF), seg_q & 1, wc, status);
                if (!__all_sync(0xffffffffu, ok)) break;
                tr.put(kEvS1Begin, kq);
#pragma unroll 1
                for (uint32_t i = 0; i < 9; ++i, ++g1) {
                    const uint32_t s = g1 % C::NS1;
                    ok = poll_phase_cluster(bar(BR::S1F + (int)s), (g1 / C::NS1) & 1, wc, status);
                    if (!__all_sync(0xffffffffu, ok)) break;
                    tc_fence_after();
#pragma unroll
                    for (uint32_t j = 0; j < 4; ++j) {
                        // A = K tile chunk (K-major, 128 rows per CTA), B = Q^T chunk (K-major, NH per CTA)
                        const uint64_t a = k_desc0 + ((s * C::CHUNK + 32 * j) >> 4);
                        const uint64_t bq = q_desc0 + ((i * C::Q_CHUNK + 32 * j) >> 4);
                        umma_bf16_pair_elected(lead, d_s, a, bq, C::IDESC_S, j == 0 ? (i == 0 ? 0u : 1u) : 1u);
                    }
                    if (lead) umma_commit_pair_both(bar(BR::S1E + (int)s));
                    __syncwarp();
                    tr.put(kEvS1Chunk, (int)i);
                }
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if (lead) umma_commit_pair_both(bar(BR::SF + (kq & 1)));
                __syncwarp();
                tr.put(kEvS1Done, kq);
                if (__any_sync(0xffffffffu, qc.last())) {
                    if (lead) umma_commit_pair_both(bar(BR::QE));
                    __syncwarp();
                    ++seg_q;
                }
                qc.advance(tile_off);
                ++kq;
            }
            // Tail: both CTAs' last releases of the score buffers (the odd CTA's arrive is remote)
            // land before this CTA leaves.
            for (int k = kq; ok && k < kq + 2 && !wc->abort; ++k)
                ok = poll_phase(bar(BR::SE + (k & 1)), ((k >> 1) & 1) ^ 1, wc, status);
            pv_pending = lead;  // FINAL is committed (and drained) at the end of the kernel
        }
        __syncwarp();
    } else if (warp == 11) {
        if (leader) {
            // -------------------------------------------------------- step-3 issuer (even CTA)
            // Per unit: K-half 0 once PF0 (both CTAs hold the even CTA's P^T part), value pair by value
            // pair as they land, then PE0; K-half 1 once PF1 and this CTA's XF (the odd CTA's part
            // landed here), then PE1.  Each value slot is freed as its MMAs complete.
            if (fb < fe) {
                const bool lead = elect_one();
                const uint64_t v_desc0 = smem_desc(sbase + C::OFF_S3, C::CHUNK, 1024, kSwizzle128B);
                const uint64_t p_desc0 = smem_desc(sbase + C::OFF_P, C::P_BUF, 1024, kSwizzle128B);
                TileCursor pc;
                pc.init(tile_off, seq0, fb, fe);
                bool ok = true;
                int kp = 0;
                uint32_t g3 = 0;
                TraceRowT<TR> tr;
                tr.init(p, 4);
                if (!lead) tr.row = nullptr;
                int pass = 0;  // kp counts passes
                while (__all_sync(0xffffffffu, ok && pc.valid)) {
                    if (lead) mbar_arrive_expect_tx(bar(BR::XF), C::P_BUF);  // the odd CTA's part of pass kp
                    __syncwarp();
                    const uint32_t fresh = __any_sync(0xffffffffu, pc.first() && pass == 0) ? 0u : 1u;
#pragma unroll 1
                    for (uint32_t h = 0; h < 2; ++h) {
                        ok = poll_phase_cluster(bar(h == 0 ? BR::PF0 : BR::PF1), kp & 1, wc, status);
                        if (ok && h == 1) {
                            ok = poll_phase_cluster(bar(BR::XF), kp & 1, wc, status);
                            fence_proxy_async_smem();  // the st.async writes are read by the tensor core next
                        }
                        if (!__all_sync(0xffffffffu, ok)) break;
                        tr.put(kEvPReady, 2 * kp + (int)h);
#pragma unroll 1
                        for (uint32_t j = 0; j < 2; ++j, ++g3) {
                            const uint32_t s = g3 % C::NS3;
                            ok = poll_phase_cluster(bar(BR::S3F + (int)s), (g3 / C::NS3) & 1, wc, status);
                            if (!__all_sync(0xffffffffu, ok)) break;
                            tc_fence_after();
                            const uint32_t d_o = tmem + C::O_COL + j * C::NP;
#pragma unroll
                            for (uint32_t k8 = 0; k8 < 8; ++k8) {
                                // A = V^T: M = 128 latent rows of this CTA (two chunks), K = 16 KV rows
                                const uint64_t a = v_desc0 + ((s * C::VPAIR + 2048 * k8) >> 4);
                                // B = P^T of K-half h: K = 16 KV rows, N = this CTA's NPH columns
                                const uint64_t bp = p_desc0 + ((h * C::P_BUF + 2048 * k8) >> 4);
                                umma_bf16_pair_elected(lead, d_o, a, bp, C::IDESC_O, k8 == 0 ? (h == 0 ? fresh : 1u) : 1u);
                            }
                            if (lead) umma_commit_pair_both(bar(BR::S3E + (int)s));
                            __syncwarp();
                            tr.put(kEvS3Pair, (int)(2 * h + j));
                        }
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok) break;
                        if (lead) umma_commit_pair_both(bar(h == 0 ? BR::PE0 : BR::PE1));
                        __syncwarp();
                    }
                    tr.put(kEvS3Done, kp);
                    ++kp;
                    if (++pass == passes_of(seq_len(pc.b))) {
                        pc.advance(tile_off);
                        pass = 0;
                    }
                }
                pv_pending = lead;  // FINAL3 is committed (and drained) at the end of the kernel
            }
        } else if (lane == 0 && fb < fe) {
            // -------------------------------------------------------- relay (odd CTA)
            // The even CTA's P^T part of each unit lands here through st.async; once it has, tell the
            // even CTA (its PF0 counts this arrival and its own softmax's).
            TileCursor rc;
            rc.init(tile_off, seq0, fb, fe);
            const uint32_t pf0_remote = map_to_rank(bar(BR::PF0), 0);
            int kr = 0, pass = 0;  // kr counts passes
            bool ok = true;
            while (rc.valid && ok) {
                mbar_arrive_expect_tx(bar(BR::XF), C::P_BUF);
                if (!mbar_test_wait_cluster(bar(BR::XF), kr & 1)) {
                    const uint64_t t0 = global_timer_ns();
                    for (uint32_t spin = 1;; ++spin) {
                        if (mbar_test_wait_cluster(bar(BR::XF), kr & 1)) break;
                        if ((spin & 255u) == 0) {
                            if (wc->abort || global_timer_ns() - t0 > wc->limit_ns) {
                                if (!wc->abort) atomicCAS(status, 0, kStatusTimeout);
                                wc->abort = 1;
                                ok = false;
                                break;
                            }
                        }
                    }
                }
                if (!ok) break;
                fence_acquire_cluster_smem();
                fence_proxy_async_smem();  // the st.async writes are read by the tensor core next
                mbar_arrive_remote(pf0_remote);
                ++kr;
                if (++pass == passes_of(seq_len(rc.b))) {
                    rc.advance(tile_off);
                    pass = 0;
                }
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ softmax + epilogue (warps 3..10)
        constexpr uint32_t SMX = 1, NSM = 256;
        const int sw = warp - 3;
        const int quad = warp & 3;                // TMEM lane quadrant this warp may access
        const int half = sw >> 2;                 // columns [half*NH, half*NH + NH) of the group
        const int row = quad * 32 + lane;         // KV row within this CTA's 128-row tile (= TMEM lane)
        const int tid = sw * 32 + lane;
        const uint32_t lane_addr = (uint32_t)(quad * 32) << 16;
        const bool own = half == (int)rank;       // these columns are this CTA's half of step 3's B operand
        float *m_s = reinterpret_cast<float *>(smem + kDuoCtlM);
        float *nm_s = reinterpret_cast<float *>(smem + kDuoCtlNm);
        float *alpha_s = reinterpret_cast<float *>(smem + kDuoCtlAlpha);
        float *red = reinterpret_cast<float *>(smem + kDuoCtlRed);
        const float *mx = reinterpret_cast<const float *>(smem + kDuoCtlMx);
        const float *lx = reinterpret_cast<const float *>(smem + kDuoCtlLx);
        const float *lr = reinterpret_cast<const float *>(smem + kDuoCtlLr);
        float *mt = reinterpret_cast<float *>(smem + kDuoCtlMt);
        int *vis_s = reinterpret_cast<int *>(smem + kDuoCtlVis);
        // the peer's vote number v lands in slot v & 1 (its next vote may arrive before this CTA has read
        // this one)
        const volatile uint32_t *vote_in = reinterpret_cast<const volatile uint32_t *>(smem + kDuoCtlMisc + 64);
        // this thread's P^T row goes to K-half `rank` of the CTA that owns its columns
        const uint32_t p_row_local = C::OFF_P + rank * C::P_BUF + (uint32_t)row * C::P_PITCH;
        const uint32_t p_row_remote = map_to_rank(sbase + p_row_local, peer);
        const uint32_t xf_remote = map_to_rank(bar(BR::XF), peer);
        const uint32_t xv_remote = map_to_rank(bar(BR::XV), peer);
        const uint32_t xm_remote = map_to_rank(bar(BR::XM), peer);
        const uint32_t xl_remote = map_to_rank(bar(BR::XL), peer);
        const uint32_t vote_remote = map_to_rank(sbase + kDuoCtlMisc + 64, peer);
        const uint32_t mx_remote = map_to_rank(sbase + kDuoCtlMx, peer);
        const uint32_t lx_remote = map_to_rank(sbase + kDuoCtlLx, peer);
        const uint32_t lr_remote = map_to_rank(sbase + kDuoCtlLr, peer);
        bool ok = true, stop = false;
        int k = 0, kv = 0, votes = 0, xmr = 0, xlr = 0;  // units, passes of step 3, votes, exchange rounds
        TraceRowT<TR> tr;
        tr.init(p, 3);
        if (tid != 0) tr.row = nullptr;
        // Scores of 32 columns of this thread's row (block cc of its half), scaled to log2 units
        // and masked; one TMEM round trip.
        uint32_t seen[NH / 32] = {};  // TREE: bit n of word cc: column 32 cc + n of this half sees this thread's row
        auto load_scores = [&](int cc, bool full, int rg, float (&x)[32]) {
            tmem_ld32_wait(tmem + lane_addr + C::S_COL + (uint32_t)(k & 1) * NC + half * NH + 32 * cc, x);
            const float2 sc = make_float2(p.scale_log2, p.scale_log2);
#pragma unroll
            for (int n = 0; n < 32; n += 2) {
                const float2 v = mul2(make_float2(x[n], x[n + 1]), sc);
                x[n] = v.x;
                x[n + 1] = v.y;
            }
            if (full) return;
            if constexpr (TREE) {
                const uint32_t bits = cc == 0 ? seen[0] : seen[NH / 32 - 1];
#pragma unroll
                for (int n = 0; n < 32; ++n) x[n] = (bits >> n) & 1u ? x[n] : -INFINITY;
            } else {
                const int4 *v4 = reinterpret_cast<const int4 *>(vis_s + half * NH + 32 * cc);
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const int4 vv = v4[q];
                    x[4 * q] = rg < vv.x ? x[4 * q] : -INFINITY;
                    x[4 * q + 1] = rg < vv.y ? x[4 * q + 1] : -INFINITY;
                    x[4 * q + 2] = rg < vv.z ? x[4 * q + 2] : -INFINITY;
                    x[4 * q + 3] = rg < vv.w ? x[4 * q + 3] : -INFINITY;
                }
            }
        };
        // P^T of this thread's row for its columns, with the final maxima of the unit: into this
        // CTA's buffer (own columns) or the peer's (st.async, counted on its XF barrier); the
        // probabilities are added to lpart.
        float lpart[TWO_SUMS ? 1 : NH];
        // TWO_SUMS: the sums of P's rounded terms and of what their rounding left, taken over the warp's rows by
        // matrix instructions whose other operand picks columns (sum_columns8): word i of block c: column
        // 16 c + 4 (lane % 4) + i of this half, summed over the four rows of the lanes alike in lane / 4.
        float sum_hi[TWO_SUMS ? NH / 16 : 1][4], sum_lo[TWO_SUMS ? NH / 16 : 1][4];
        // (rest: the term that P_hi's rounding left, for a second pass of step 3)
        auto write_p = [&](bool full, int rg, auto rest) {
#pragma unroll
            for (int cc = 0; cc < NH / 32; ++cc) {
                float x[32];
                load_scores(cc, full, rg, x);
                const float4 *nm4 = reinterpret_cast<const float4 *>(nm_s + half * NH + 32 * cc);
                // one 16-byte chunk (8 columns) at a time: hi at chunk 4cc+u, lo (split) at NH/8 + that
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const float4 nm = nm4[2 * u + q];
#pragma unroll
                        for (int e = 0; e < 4; e += 2) {
                            const int n = 8 * u + 4 * q + e;
                            const float2 d = add2(make_float2(x[n], x[n + 1]),
                                                  e == 0 ? make_float2(nm.x, nm.y) : make_float2(nm.z, nm.w));
                            const float2 pv = make_float2(fast_exp2(d.x), fast_exp2(d.y));
                            const uint32_t h = pack_bf16x2(pv.x, pv.y);
                            if constexpr (!decltype(rest)::value) hi[2 * q + e / 2] = h;
                            if constexpr (!decltype(rest)::value && !TWO_SUMS) {
                                const float2 l = add2(make_float2(lpart[32 * cc + n], lpart[32 * cc + n + 1]), pv);
                                lpart[32 * cc + n] = l.x;
                                lpart[32 * cc + n + 1] = l.y;
                            }
                            if constexpr (C::SPLIT || TWO_SUMS || decltype(rest)::value) {
                                // p - hi, exactly rounded as a subtraction
                                const float2 r = fma2(make_float2(__uint_as_float(h << 16), __uint_as_float(h & 0xFFFF0000u)),
                                                      make_float2(-1.f, -1.f), pv);
                                (decltype(rest)::value && !C::SPLIT ? hi : lo)[2 * q + e / 2] = pack_bf16x2(r.x, r.y);
                            }
                        }
                    }
                    if constexpr (TWO_SUMS && !decltype(rest)::value) {
                        sum_columns8(sum_hi[2 * cc + u / 2], hi, lane, u & 1);
                        sum_columns8(sum_lo[2 * cc + u / 2], lo, lane, u & 1);
                    }
#pragma unroll
                    for (int hl = 0; hl < (C::SPLIT ? 2 : 1); ++hl) {
                        const uint32_t *w = hl == 0 ? hi : lo;
                        const uint32_t j16 = (uint32_t)(hl * (NH / 8) + 4 * cc + u);
                        const uint32_t off = (j16 ^ ((uint32_t)row & 7u)) << 4;
                        if (own) {
                            *reinterpret_cast<uint4 *>(smem + p_row_local + off) = make_uint4(w[0], w[1], w[2], w[3]);
                        } else if (ok) {
                            st_async_v4(p_row_remote + off, w[0], w[1], w[2], w[3], xf_remote);
                        }
                    }
                }
            }
        };
        if (fb < fe) {
            SegIter it;
            it.init_at(seq0, fb, fe);
            int b, t0, t1;
            while (!stop && it.next(tile_off, b, t0, t1)) {
                int L = p.seqlens[b];
                if ((int64_t)L > l_cap) L = (int)l_cap;
                if (L < 0) L = 0;
                const int passes = passes_of(L);
                const int seg_nsplit = seq_info[4 * b + 2];
                const int seg_slot = seq_info[4 * b + 3] + (unit - seq_info[4 * b + 1]);
                int qlen_b = p.q_len;
                if (p.q_lens) {
                    qlen_b = p.q_lens[b];
                    if (qlen_b < 0 || qlen_b > p.q_len) {
                        if (tid == 0) atomicCAS(status, 0, kStatusInvalid);
                        qlen_b = qlen_b < 0 ? 0 : p.q_len;
                    }
                }
                // per-column visible rows and a fresh running maximum (after everyone is done with the
                // previous segment's values)
                named_bar_sync(SMX, NSM);
                if (tid < NC) {
                    const int ng = grp * NC + tid;
                    int vis = 0;
                    if (ng < p.ncols) {
                        const int tok = ng / p.num_heads;
                        vis = tok >= qlen_b ? 0 : (p.causal ? (L - qlen_b + tok + 1) : L);
                        vis = vis < 0 ? 0 : vis;
                    }
                    vis_s[tid] = vis;
                    m_s[tid] = -INFINITY;
                    nm_s[tid] = kNoRow;
                }
                named_bar_sync(SMX, NSM);
                if constexpr (TWO_SUMS) {
#pragma unroll
                    for (int c = 0; c < NH / 16; ++c)
#pragma unroll
                        for (int i = 0; i < 4; ++i) sum_hi[c][i] = sum_lo[c][i] = 0.f;
                } else {
#pragma unroll
                    for (int n = 0; n < NH; ++n) lpart[n] = 0.f;
                }
                for (int tp = t0; tp < t1 && !stop; ++tp, ++k) {
                    const bool first = tp == t0;
                    ok = ok && spin_phase<false>(bar(BR::SF + (k & 1)), (k >> 1) & 1, wc, status);
                    tc_fence_after();
                    tr.put(kEvSmS, k);
                    const int rg = tp * kDuoRows + kTileRows * (int)rank + row;
                    // every row of this CTA's tile visible to every column: no per-column mask
                    bool full;
                    if constexpr (TREE) {
                        full = tp * kDuoRows + kTileRows * ((int)rank + 1) <= L - qlen_b &&
                               grp * NC + NC <= qlen_b * p.num_heads;
                        if (!full) {
                            const uint64_t s = tree_sees(p, b, L, qlen_b, rg, grp * NC + half * NH, NH);
                            seen[0] = (uint32_t)s;
                            if constexpr (NH > 32) seen[1] = (uint32_t)(s >> 32);
                        }
                    } else {
                        full = qlen_b == p.q_len &&
                               tp * kDuoRows + kTileRows * ((int)rank + 1) <= (p.causal ? L - qlen_b + 1 : L) &&
                               grp * NC + NC <= p.ncols;
                    }
                    // ---- pass 1: does any score exceed its column's running maximum by > 2^THRESH?  (A segment's
                    // first unit sets the maxima: nothing to ask.)
                    bool slow = first;
                    if (!first) {
                        float over = -INFINITY;
                        // rolled: one copy of the score read and test (instruction cache; measured faster)
#pragma unroll 1
                        for (int cc = 0; cc < NH / 32; ++cc) {
                            float x[32];
                            load_scores(cc, full, rg, x);
                            const float4 *nm4 = reinterpret_cast<const float4 *>(nm_s + half * NH + 32 * cc);
#pragma unroll
                            for (int q = 0; q < 8; ++q) {
                                const float4 nm = nm4[q];
                                const float2 d0 = add2(make_float2(x[4 * q], x[4 * q + 1]), make_float2(nm.x, nm.y));
                                const float2 d1 = add2(make_float2(x[4 * q + 2], x[4 * q + 3]), make_float2(nm.z, nm.w));
                                over = fmaxf(over, fmaxf(fmaxf(d0.x, d0.y), fmaxf(d1.x, d1.y)));
                            }
                        }
                        const bool need = !ok || over > kRescaleThreshold;
                        const bool vote = named_bar_or(SMX, NSM, need);
                        // ---- votes of both CTAs (a small exchange ahead of P^T, so that P^T is final when written)
                        if (tid == 0) {
                            mbar_arrive_expect_tx(bar(BR::XV), 16);
                            if (ok)
                                st_async_v4(vote_remote + 16u * (uint32_t)(votes & 1), vote ? 1u : 0u, (uint32_t)k, 0u, 0u,
                                            xv_remote);
                        }
                        ok = ok && spin_phase<true>(bar(BR::XV), votes & 1, wc, status);
                        slow = vote || vote_in[4 * (votes & 1)] != 0u;
                        ++votes;
                    }
                    tr.put(kEvSmVote, k);
                    // a timed-out wait stops every warp here, before any branch on the peer's vote
                    if (!named_bar_and(SMX, NSM, ok)) {
                        stop = true;
                        break;
                    }
                    if (slow) {  // the same in every thread of both CTAs
                        tr.put(kEvSmSlow, k);
                        // ---- slow path, taken by both CTAs together: tile maxima over all 256 rows
#pragma unroll 1
                        for (int cc = 0; cc < NH / 32; ++cc) {
                            float x[32];
                            load_scores(cc, full, rg, x);
#pragma unroll
                            for (int g = 0; g < 2; ++g) {
                                float x16[16];
#pragma unroll
                                for (int n = 0; n < 16; ++n) x16[n] = x[16 * g + n];
                                const float wmax = warp_colreduce16<true>(x16, lane);
                                if ((lane & 1) == 0) red[quad * NC + half * NH + 32 * cc + 16 * g + col16(lane)] = wmax;
                            }
                        }
                        named_bar_sync(SMX, NSM);
                        if (tid == 0) mbar_arrive_expect_tx(bar(BR::XM), 4 * NC);
                        if (tid < NC) {
                            const float v = fmaxf(fmaxf(red[tid], red[NC + tid]), fmaxf(red[2 * NC + tid], red[3 * NC + tid]));
                            mt[tid] = v;
                            if (ok) st_async_b32(mx_remote + 4u * tid, __float_as_uint(v), xm_remote);
                        }
                        ok = ok && spin_phase<true>(bar(BR::XM), xmr & 1, wc, status);
                        ++xmr;
                        bool resc = false;
                        if (tid < NC) {
                            // the same inputs and arithmetic in both CTAs: identical maxima and factors
                            const float mtot = fmaxf(mt[tid], mx[tid]);
                            const float mo = m_s[tid];
                            float a = 1.f;
                            if (mo == -INFINITY) {
                                m_s[tid] = mtot == -INFINITY ? -INFINITY : mtot + kRescaleHeadroom;
                                nm_s[tid] = mtot == -INFINITY ? kNoRow : -(mtot + kRescaleHeadroom);
                            } else if (mtot > mo + kRescaleThreshold) {
                                const float mn = mtot + kRescaleHeadroom;
                                a = fast_exp2(mo - mn);
                                m_s[tid] = mn;
                                nm_s[tid] = -mn;
                                resc = true;
                            }
                            alpha_s[tid] = a;
                        }
                        const bool any_resc = named_bar_or(SMX, NSM, resc);
                        if (any_resc) {
                            // O^T holds step 3 up to the previous unit once both of its K-halves completed;
                            // rescale this thread's lane of both M-blocks for its half's columns
                            if (kv > 0) {
                                ok = ok && spin_phase<false>(bar(BR::PE0), (kv - 1) & 1, wc, status);
                                ok = ok && spin_phase<false>(bar(BR::PE1), (kv - 1) & 1, wc, status);
                            }
                            tc_fence_after();
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
#pragma unroll
                                for (int g = 0; g < 4; ++g) {
                                    float v[16];
                                    const uint32_t addr = tmem + lane_addr + C::O_COL + (uint32_t)j * C::NP + half * 64 + 16 * g;
                                    tmem_ld16(addr, v);
                                    tmem_wait_ld();
#pragma unroll
                                    for (int n = 0; n < 16; ++n) v[n] *= alpha_s[half * NH + ((16 * g + n) % NH)];
                                    tmem_st16(addr, v);
                                }
                            }
                            tmem_wait_st();
                            if constexpr (TWO_SUMS) {
#pragma unroll
                                for (int c = 0; c < NH / 16; ++c)
#pragma unroll
                                    for (int i = 0; i < 4; ++i) {
                                        const float a = alpha_s[half * NH + 16 * c + 4 * (lane & 3) + i];
                                        sum_hi[c][i] *= a;
                                        sum_lo[c][i] *= a;
                                    }
                            } else {
#pragma unroll
                                for (int n = 0; n < NH; ++n) lpart[n] *= alpha_s[half * NH + n];
                            }
                        }
                    }
                    // ---- P^T of this CTA's rows (K-half `rank`) once the previous pass of step 3 released that
                    // K-half's buffers in both CTAs
#pragma unroll 1
                    for (int pass = 0; pass < passes; ++pass, ++kv) {
                        if (kv > 0)
                            ok = ok && spin_phase<false>(bar(rank == 0 ? BR::PE0 : BR::PE1), (kv - 1) & 1, wc, status);
                        tc_fence_after();
                        tr.put(kEvSmPe, k);
                        if constexpr (TREE && !C::SPLIT) {
                            if (pass == 0)
                                write_p(full, rg, std::false_type{});
                            else
                                write_p(full, rg, std::true_type{});
                        } else {
                            write_p(full, rg, std::false_type{});
                        }
                        // this CTA's P^T writes are seen by the tensor core's reads; the S^T reads are complete
                        fence_proxy_async_smem();
                        tc_fence_before();
                        if (!named_bar_and(SMX, NSM, ok)) {
                            stop = true;
                            break;
                        }
                        if (tid == 0) {
                            // K-half `rank` is ready on this side (the receiving side reports its part)
                            if (leader)
                                mbar_arrive(bar(BR::PF0));
                            else
                                mbar_arrive_remote(map_to_rank(bar(BR::PF1), 0));
                            if (pass == passes - 1) arrive0(BR::SE + (k & 1));
                            tr.put(kEvSmDone, k);
                        }
                    }
                }
                if (stop) break;
                // ---------------------------------------------------- epilogue for this CTA's 256 latent rows
                // The column sums are summed and exchanged while the last pass of step 3 runs.
                const int kl = kv - 1;  // that pass
                tr.put(kEvSmEpi, kl);
                // this CTA's sum of column tid over the four lane quadrants (rows of warps that share columns)
                auto quadrants = [&] { return (red[tid] + red[NC + tid]) + (red[2 * NC + tid] + red[3 * NC + tid]); };
                float rounded = 0.f;  // TWO_SUMS: column tid's sum of rounded P, of this CTA, then of both
                if constexpr (TWO_SUMS) {
                    // every lane's four rows joined with the other seven groups'; lanes 0..3 hold the columns
#pragma unroll
                    for (int c = 0; c < NH / 16; ++c)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
#pragma unroll
                            for (int d = 4; d <= 16; d <<= 1) {
                                sum_hi[c][i] += __shfl_xor_sync(0xffffffffu, sum_hi[c][i], d);
                                sum_lo[c][i] += __shfl_xor_sync(0xffffffffu, sum_lo[c][i], d);
                            }
                        }
                    auto put = [&](const float (&v)[NH / 16][4]) {
                        if (lane < 4) {
#pragma unroll
                            for (int c = 0; c < NH / 16; ++c)
                                *reinterpret_cast<float4 *>(red + quad * NC + half * NH + 16 * c + 4 * lane) =
                                    make_float4(v[c][0], v[c][1], v[c][2], v[c][3]);
                        }
                        named_bar_sync(SMX, NSM);
                    };
                    put(sum_hi);
                    if (tid < NC) rounded = quadrants();
                    named_bar_sync(SMX, NSM);
                    put(sum_lo);
                } else {
#pragma unroll
                    for (int ch = 0; ch < NH / 16; ++ch) {
                        float v16[16];
#pragma unroll
                        for (int n = 0; n < 16; ++n) v16[n] = lpart[16 * ch + n];
                        const float wsum = warp_colreduce16<false>(v16, lane);
                        if ((lane & 1) == 0) red[quad * NC + half * NH + 16 * ch + col16(lane)] = wsum;
                    }
                    named_bar_sync(SMX, NSM);
                }
                if (tid == 0) mbar_arrive_expect_tx(bar(BR::XL), (TWO_SUMS ? 8 : 4) * NC);
                if (tid < NC) {
                    const float v = TWO_SUMS ? rounded + quadrants() : quadrants();
                    mt[tid] = v;
                    if (ok) {
                        st_async_b32(lx_remote + 4u * tid, __float_as_uint(v), xl_remote);
                        if constexpr (TWO_SUMS) st_async_b32(lr_remote + 4u * tid, __float_as_uint(rounded), xl_remote);
                    }
                }
                ok = ok && spin_phase<true>(bar(BR::XL), xlr & 1, wc, status);
                ++xlr;
                tr.put(kEvEpiL, kl);
                ok = ok && spin_phase<false>(bar(BR::PE0), kl & 1, wc, status);
                ok = ok && spin_phase<false>(bar(BR::PE1), kl & 1, wc, status);
                if (!named_bar_and(SMX, NSM, ok)) {  // also orders the mt writes before the reads
                    stop = true;
                    break;
                }
                tc_fence_after();
                tr.put(kEvEpiS3, kl);
                const int nsplit = seg_nsplit;
                const int slot = seg_slot;
                // column sum over both CTAs, rank 0's part first in both (identical values)
                auto col_l = [&](int c) -> float { return rank == 0 ? mt[c] + lx[c] : lx[c] + mt[c]; };
                // 1 / l per column (0 for a column that saw no row), once, in the idle alpha area.  TWO_SUMS with one
                // pass: over the sum of what was multiplied, so that a rounding that many of the column's rows share, or
                // that the one row has which carries it, cancels; the LSE keeps the sum of P itself.
                if (tid < NC) {
                    const float l = col_l(tid);
                    float over = l;
                    if constexpr (TWO_SUMS)
                        if (passes == 1) over = rank == 0 ? rounded + lr[tid] : lr[tid] + rounded;
                    alpha_s[tid] = (!(l > 0.f) || m_s[tid] == -INFINITY) ? 0.f : 1.f / over;
                }
                named_bar_sync(SMX, NSM);
                // 16 columns of latent row d: outputs of an unsplit sequence, else partials
                auto store16 = [&](int c, int d, const float (&v)[16]) {
                    const int cols = min(p.ncols - (grp * NC + c), 16);
                    if (nsplit == 1) {
                        __nv_bfloat16 *o = p.o + ((int64_t)b * p.ncols + grp * NC + c) * kDv + d;
#pragma unroll
                        for (int n = 0; n < 16; ++n)
                            if (n < cols) o[n * kDv] = __float2bfloat16_rn(v[n]);
                    } else {
                        float *o = p.opart + ((int64_t)slot * p.ncols + grp * NC + c) * kDv + d;
#pragma unroll
                        for (int n = 0; n < 16; ++n)
                            if (n < cols) o[n * kDv] = v[n];
                    }
                };
#pragma unroll 1
                for (int j = 0; j < 2; ++j) {
#pragma unroll 1
                    for (int g = 0; g < NH / 16; ++g) {
                        float hi[16], lo[16];
                        tmem_ld16(tmem + lane_addr + C::O_COL + (uint32_t)j * C::NP + half * 64 + 16 * g, hi);
                        if constexpr (C::SPLIT)
                            tmem_ld16(tmem + lane_addr + C::O_COL + (uint32_t)j * C::NP + half * 64 + NH + 16 * g, lo);
                        tmem_wait_ld();
                        const int c = half * NH + 16 * g;
#pragma unroll
                        for (int n = 0; n < 16; ++n) {
                            const float val = C::SPLIT ? hi[n] + lo[n] : hi[n];
                            hi[n] = val * alpha_s[c + n];
                        }
                        store16(c, 256 * (int)rank + 128 * j + row, hi);
                    }
                }
                if (rank == 0 && tid < NC) {
                    const int ng = grp * NC + tid;
                    if (ng < p.ncols) {
                        const float l = col_l(tid);
                        const bool empty = !(l > 0.f) || m_s[tid] == -INFINITY;
                        const float lse = empty ? -INFINITY : (m_s[tid] + __log2f(l)) * 0.69314718055994531f;
                        if (nsplit == 1)
                            p.lse[(int64_t)b * p.ncols + ng] = lse;
                        else
                            p.lsepart[((int64_t)rank * p.slots + slot) * p.ncols + ng] = lse;
                    }
                }
                tr.put(kEvEpiO, nsplit);
                if (nsplit >= 2 && p.signal_combine) {
                    // this CTA's partial of the split is stored: count it for the combine kernel
                    // (release: the CTA barrier and one thread's release add cover every thread's
                    // stores)
                    named_bar_sync(SMX, NSM);
                    if (tid == 0) red_add_release_gpu(p.counters + ((int64_t)b * groups + grp) * 2 + rank, 1);
                }
                tr.put(kEvSmEpiDone, kl);
                tc_fence_before();
            }
        }
        if (stop || !ok) wc->abort = 1;
        __syncwarp();
    }
}

// TREE: the new rows' visibility comes from per-token ancestor masks (tree_sees) instead of a length
// per column.
template <class C64, class C128, bool TR = false, bool TREE = false>
__global__ void __launch_bounds__(kDuoThreads, 1)
    etap_duo_kernel(const __grid_constant__ DuoMaps tm, const __grid_constant__ DecodeParams p) {
    using BR = DuoBars;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_addr(smem_raw);
    const uint32_t sbase = (raw_addr + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (sbase - raw_addr);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    int32_t *status = p.ws + kHdrStatus;
    auto bar = [&](int i) -> uint32_t { return sbase + kDuoCtlBar + 8u * (uint32_t)i; };
    volatile WaitCtl *wc = reinterpret_cast<volatile WaitCtl *>(smem + kDuoCtlMisc + 16);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + kDuoCtlMisc);
    // trace: every CTA's entry, start of work (after the plan), end of work and exit
    unsigned long long *span = trace_span<TR>(p);
    if (span && threadIdx.x == 0) span[0] = global_timer_ns();

    if (threadIdx.x == 0) {
        for (int i = 0; i < kDuoMaxSlots; ++i) {
            mbar_init(bar(BR::S1F + i), 2);  // both CTAs' producers (expect_tx) + their TMA bytes
            mbar_init(bar(BR::S1E + i), 1);  // the MMA commit
            mbar_init(bar(BR::S3F + i), 2);
            mbar_init(bar(BR::S3E + i), 1);
        }
        mbar_init(bar(BR::QF), 2);
        mbar_init(bar(BR::QE), 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(BR::SF + i), 1);
            mbar_init(bar(BR::SE + i), 2);  // one arrival per CTA once its softmax warps read S^T
        }
        // K-half 0: the even CTA's softmax (its writes) + the odd CTA's relay (it received the rest);
        // K-half 1: the odd CTA's softmax; the step-3 issuer checks its own XF for the rest
        mbar_init(bar(BR::PF0), 2);
        mbar_init(bar(BR::PF1), 1);
        mbar_init(bar(BR::PE0), 1);
        mbar_init(bar(BR::PE1), 1);
        mbar_init(bar(BR::XF), 1);  // the peer's P^T part: armed by this CTA's step-3 issuer or relay
        mbar_init(bar(BR::XV), 1);  // the peer's vote
        mbar_init(bar(BR::XM), 1);
        mbar_init(bar(BR::XL), 1);
        mbar_init(bar(BR::TAIL), 1);
        mbar_init(bar(BR::FINAL), 1);
        mbar_init(bar(BR::FINAL3), 1);
        wc->abort = 0;
        wc->limit_ns = p.wait_limit_ns;
        fence_barrier_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&tm.q32);
        tma_prefetch_desc(&tm.q64);
        tma_prefetch_desc(&tm.kv);
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_addr(tmem_slot), 512);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    cluster_sync();  // both CTAs' barriers and TMEM exist before any remote operation
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
    bool pv_pending = false;
    if (span && threadIdx.x == 0) span[1] = global_timer_ns();
    if (mode == 1)
        duo_body<C128, TR, TREE>(tm, p, smem, sbase, tmem, rank, unit, grp, groups, has_work, wc, status, pv_pending);
    else
        duo_body<C64, TR, TREE>(tm, p, smem, sbase, tmem, rank, unit, grp, groups, has_work, wc, status, pv_pending);
    if (pv_pending) {
        // every MMA issued completes before TMEM is released (one barrier per issuing thread)
        const int fin = warp == 1 ? BR::FINAL : BR::FINAL3;
        umma_commit_pair_local(bar(fin));
        drain_phase(bar(fin), 0);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (span && threadIdx.x == 0) span[2] = global_timer_ns();
    // No CTA leaves while its peer may still write into its shared memory.  Every operation that
    // targets a CTA's shared memory (TMA bytes, st.async, remote and multicast arrivals) has been
    // waited for by that CTA above (the producers' tails included), so the barrier needs no
    // ordering of its own.
    cluster_sync_relaxed_arrive();
    if (wc->abort) {
        // After an abort a peer's last st.async or bulk copy may not have been waited for: let it
        // land before either CTA leaves (no thread sends after the barrier above).
        const uint64_t t_q = global_timer_ns();
        while (global_timer_ns() - t_q < 20000ull) {
        }
    }
    cluster_sync_relaxed_arrive();
    tc_fence_after();
    if (warp == 1) tmem_dealloc_pair(tmem, 512);
    if (span && threadIdx.x == 32) span[3] = global_timer_ns();
}

}  // namespace mla
