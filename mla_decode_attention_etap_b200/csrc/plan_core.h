// Split-KV schedules and workspace layout, shared by the device plan kernel,
// the decode/combine kernels and the host mirror (mla_decode_plan_host).
//
// The KV units of all sequences are concatenated in sequence order and cut into one
// contiguous range per work unit and column group, balanced by cost (plan_cut.h).  A
// sequence touched by several ranges is "split": each writes an fp32 partial (O_s,
// lse_s) into its slot and the merge (in the decode kernel, or the combine kernel)
// combines them.  Not on the pages: it exists so that a batch of few long
// sequences still spreads over every SM.
//
// Up to three schedules live in one workspace:
//   pair  128-row units, column groups of 16 or 32: the CTA-pair kernel (etap_pair_kernel),
//         used by the FP8 cache for every shape and by the bf16 cache when q_len*h <= 16;
//   duo   256-row units (a tile of 128 rows per CTA of the pair), column groups of 64 (P as
//         bf16 hi + lo) or 128 (one bf16 P term): the M = 256 kernel (etap_duo_kernel), used
//         by the bf16 cache when q_len*h > 16.  Groups of 128 are chosen by the plan, on the
//         device, when q_len*h > 64 and every nonempty sequence holds at least
//         kSingleP_MinRows rows; the decode kernel reads the choice from the header;
//   tree  as duo, for tree decodes of more than 16 columns (bf16 and E4M3 cache), with other end
//         costs (plan_cut.h) and groups of 128 also when some sequences are shorter, if there are
//         units enough (tree_mode); the bf16 kernel then multiplies the short sequences' P as hi
//         and lo, one after the other.
#pragma once

#include <cstddef>
#include <cstdint>

#ifdef __CUDACC__
#define MLA_HD __host__ __device__ __forceinline__
#else
#define MLA_HD inline
#endif

namespace mla {

constexpr int kTileRows = 128;   // KV rows per tile = UMMA M of S^T = K Q^T in one CTA
constexpr int kDuoRows = 256;    // KV rows per unit of the duo kernel = UMMA M across the CTA pair
constexpr int kDqk = 576;
constexpr int kDv = 512;
constexpr int kPage = 64;
// One bf16 P term (half a step: 2^-9 of a power of 2, 1.65e-3 RMS, as much again as O's own rounding) averages out in
// what many rows share: RMSE of O over its RMS at 8192 / 32768 N(0,1) rows 1.78e-3 / 1.70e-3 against the
// 2e-3 bar (1.65e-3 with P as hi + lo).  Where few rows carry the softmax their rounding stays: with 5 % of the rows
// scaled x8, all of a sequence in one range, 2.22e-3 / 2.26e-3.  A tree decode divides O by the sum of the rounded terms
// instead of P's, which takes that out (1.69e-3 / 1.72e-3); the causal form does not.  Neither helps where values have
// nothing to do with scores and no mean, so that O is what the rows' weights happen to leave: 2.34e-3.
constexpr int kSingleP_MinRows = 8192;

// header words (int32) at the start of the workspace
enum : int {
    kHdrStatus = 0,
    kHdrBatch = 1,
    kHdrCols = 2,
    kHdrSlotsMax = 3,
    kHdrSchedUsed = 4,   // written by the decode kernel: 0 pair, 1 duo, 2 tree (the partials' schedule)
    kHdrPair = 8,        // + kSch*: the pair schedule
    kHdrDuo = 16,        // + kSch*: the duo schedule
    kHdrTree = 24,       // + kSch*: the tree schedule (0 units per group: not planned)
    kHdrWords = 64
};
enum : int { kSchCtas = 0, kSchGroups = 1, kSchTotal = 2, kSchSlotsUsed = 3, kSchGroupCols = 4, kSchMode = 5 };

// Column groups of the pair kernel: one group of 16 when they fit, otherwise groups of 32.
MLA_HD int group_cols(int ncols) { return ncols <= 16 ? 16 : 32; }
MLA_HD int num_groups(int ncols) { return (ncols + group_cols(ncols) - 1) / group_cols(ncols); }
// The bf16 cache runs the duo kernel for more than 16 query columns.
MLA_HD bool uses_duo(int ncols) { return ncols > 16; }
// Duo column group: mode 0 = 64 columns (P as bf16 hi + lo), mode 1 = 128 columns (one bf16 P term).
MLA_HD int duo_group_cols(int mode) { return mode ? 128 : 64; }
MLA_HD bool duo_mode1_possible(int ncols) { return ncols > 64; }
MLA_HD int duo_groups(int ncols, int mode) { return (ncols + duo_group_cols(mode) - 1) / duo_group_cols(mode); }
// Work units per column group: one per pair of SMs (a 2-CTA cluster).
MLA_HD int num_ctas(int num_sms, int groups) {
    int c = num_sms / 2 / groups;
    return c < 1 ? 1 : c;
}
MLA_HD int units_of(int L, int unit_rows) { return L <= 0 ? 0 : (L - 1) / unit_rows + 1; }  // (no sum past INT32_MAX)
MLA_HD int tiles_of(int L) { return units_of(L, kTileRows); }
// The duo mode the plan picks for these lengths (min_len: shortest nonempty sequence, 0 if none).
MLA_HD int duo_mode(int ncols, int min_len) { return duo_mode1_possible(ncols) && min_len >= kSingleP_MinRows ? 1 : 0; }

// The grouping of the tree schedule: for more than 64 columns groups of 128 wherever the duo schedule takes them, and when every work
// unit of that grouping gets a unit of KV rows (`units` of kDuoRows in all).  Batches of 16 ragged trees of
// up to 16 tokens, 16 heads, lengths drawn from 1 to 32768 (three draws each): 194..224 us in groups of
// 128, 224..269 us in groups of 64 (replayed from a graph, on the kernel of that time).
MLA_HD int tree_mode(int ncols, int min_len, int64_t units, int num_sms) {
    if (!duo_mode1_possible(ncols)) return 0;
    return duo_mode(ncols, min_len) || units >= num_ctas(num_sms, duo_groups(ncols, 1)) ? 1 : 0;
}

// Work units that receive ranges: never more than there are units.
MLA_HD int used_ctas(int64_t total, int ctas) { return total < (int64_t)ctas ? (int)total : ctas; }
// Near-equal cut of [0, total) into `used` ranges: range c is [cta_begin(c), cta_begin(c+1)).
// The plan cuts the cost axis of plan_cut.h this way.
MLA_HD int64_t cta_begin(int64_t total, int used, int c) {
    return c >= used ? total : total * (int64_t)c / used;
}
// The range that holds position f (0 <= f < total, used >= 1).
MLA_HD int cta_of(int64_t total, int used, int64_t f) { return (int)(((f + 1) * (int64_t)used - 1) / total); }

MLA_HD size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// One schedule's tables (byte offsets into the workspace), sized for its largest grouping.
struct Sched {
    size_t cta_ranges;  // int32 [ctas][2] (one range per work unit = SM pair)
    size_t cta_seq;     // int32 [ctas]: the sequence that holds the unit's first tile (batch if none)
    size_t tile_off;    // int32 [batch + 1]: first flattened unit of each sequence
    size_t seq_info;    // int32 [batch][4]: units, first CTA, splits, slot offset
    size_t counters;    // int32 [batch][groups][2 ranks]: split CTAs done (in-kernel merge, or the combine's wait)
    size_t done;        // int32 [batch]: combine CTAs done with a sequence (the last one rearms its counters)
    int ctas_max, groups_max, unit_rows;
};

struct WsLayout {
    Sched pair, duo, tree;  // duo is meaningful only when has_duo, tree when has_tree
    int has_duo, has_tree;
    size_t opart;    // fp32 [slots][ncols][512] (shared: one decode runs per plan at a time)
    size_t lsepart;  // fp32 [2 ranks][slots][ncols] (the two CTAs of a pair compute equal values)
    size_t base;     // bytes of everything but the tree schedule's tables, which come last
    size_t total;
    int slots;       // batch + the most work units any schedule can have
    // pair schedule grouping (fixed by the shape)
    int ctas, groups;
};

MLA_HD size_t sched_tables(Sched &s, size_t off, int batch, int ctas_max, int groups_max, int unit_rows) {
    s.ctas_max = ctas_max;
    s.groups_max = groups_max;
    s.unit_rows = unit_rows;
    s.cta_ranges = off;
    off += align256(sizeof(int32_t) * 2 * (size_t)ctas_max);
    s.cta_seq = off;
    off += align256(sizeof(int32_t) * (size_t)ctas_max);
    s.tile_off = off;
    off += align256(sizeof(int32_t) * ((size_t)batch + 1));
    s.seq_info = off;
    off += align256(sizeof(int32_t) * 4 * (size_t)batch);
    s.counters = off;
    off += align256(sizeof(int32_t) * 2 * (size_t)batch * groups_max);
    s.done = off;
    off += align256(sizeof(int32_t) * (size_t)batch);
    return off;
}

MLA_HD WsLayout ws_layout(int batch, int q_len, int num_heads, int num_sms) {
    WsLayout w{};
    const int ncols = q_len * num_heads;
    w.groups = num_groups(ncols);
    w.ctas = num_ctas(num_sms, w.groups);
    w.has_duo = uses_duo(ncols) ? 1 : 0;
    size_t off = align256(sizeof(int32_t) * kHdrWords);
    off = sched_tables(w.pair, off, batch, w.ctas, w.groups, kTileRows);
    int units_max = w.ctas;
    if (w.has_duo) {
        // mode 0 has the most groups; mode 1 (when possible) the most units per group
        const int g0 = duo_groups(ncols, 0);
        const int c_max = num_ctas(num_sms, duo_mode1_possible(ncols) ? duo_groups(ncols, 1) : g0);
        off = sched_tables(w.duo, off, batch, c_max, g0, kDuoRows);
        if (c_max > units_max) units_max = c_max;
    }
    w.slots = batch + units_max;  // sum over split sequences of their split counts is < batch + units
    w.opart = off;
    off += align256(sizeof(float) * (size_t)w.slots * ncols * kDv);
    w.lsepart = off;
    off += align256(sizeof(float) * 2 * (size_t)w.slots * ncols);
    w.base = off;
    w.has_tree = w.has_duo;
    if (w.has_tree) off = sched_tables(w.tree, off, batch, w.duo.ctas_max, w.duo.groups_max, kDuoRows);
    w.total = off;
    return w;
}

}  // namespace mla
