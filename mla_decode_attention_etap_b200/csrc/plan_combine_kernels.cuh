// Split-KV plan kernel and the log-sum-exp combine kernel.
#pragma once

#include <cuda_bf16.h>
#include <cstdint>

#include "block_scan.cuh"
#include "etap_common.cuh"
#include "merge.cuh"
#include "plan_check.cuh"
#include "plan_core.h"
#include "plan_cut.h"

namespace mla {

constexpr int kPlanThreads = 1024;

// One schedule: unit prefix sums, per-CTA flattened ranges (cut by cost, see plan_core.h),
// per-sequence split info and zeroed merge counters, plus its header words.  Every thread of the
// block calls it; thread i owns the consecutive sequences [b0, b1).
__device__ void plan_schedule(const int32_t *__restrict__ seqlens, int batch, int b0, int b1, int ctas, int groups,
                              int sched, int unit_rows, int gcols, int mode, int32_t *__restrict__ ws,
                              const Sched &sc, int hdr, int64_t *scan_smem) {
    int32_t *tile_off = ws + sc.tile_off / 4;
    int32_t *ranges = ws + sc.cta_ranges / 4;
    int32_t *seq_info = ws + sc.seq_info / 4;
    int32_t *counters = ws + sc.counters / 4;
    int32_t *cta_seq = ws + sc.cta_seq / 4;
    // flattened unit offsets and cost offsets: exclusive prefix sums per sequence
    int64_t mine = 0, ends = 0;
    for (int b = b0; b < b1; ++b) {
        const int u = units_of(seqlens[b], unit_rows);
        mine += u;
        ends += u > 0;
    }
    int64_t total, total_ends;
    int64_t f = block_exclusive_scan(mine, scan_smem, &total);
    ends = block_exclusive_scan(ends, scan_smem, &total_ends);
    const int E = end_cost_units(sched, mode, total, ctas);
    int64_t g = f + E * ends;
    const int64_t total_cost = total + E * total_ends;
    const int used = used_ctas(total, ctas);
    for (int c = threadIdx.x; c < ctas; c += blockDim.x) {
        cta_seq[c] = batch;  // no units, unless a sequence below claims it
        if (c >= used) ranges[2 * c] = (int32_t)total;
    }
    // range starts that fall inside each sequence's cost interval, and its split CTAs
    int64_t split_slots = 0;
    for (int b = b0; b < b1; ++b) {
        const int64_t units = units_of(seqlens[b], unit_rows);
        const int64_t t0 = f, t1 = f + units;
        const int64_t gend = g + units + (units > 0 ? E : 0);
        int first = -1, nsplit = 0;
        if (units > 0) {
            first = cta_of(total_cost, used, g);
            nsplit = cta_of(total_cost, used, g + units - 1) - first + 1;
            for (int c = first_range_at_or_after(total_cost, used, g); c < used; ++c) {
                const int64_t x = cta_begin(total_cost, used, c);
                if (x >= gend) break;
                ranges[2 * c] = (int32_t)unit_at_cost(x, g, t0, units);
            }
        }
        tile_off[b] = (int32_t)t0;
        seq_info[4 * b + 0] = (int32_t)units;
        seq_info[4 * b + 1] = first;
        seq_info[4 * b + 2] = nsplit;
        if (nsplit >= 2) split_slots += nsplit;
        f = t1;
        g = gend;
    }
    // partial-output slots: exclusive prefix sum of the split counts of split sequences (the scan's
    // barriers also publish every range start written above)
    int64_t slots;
    int64_t sl = block_exclusive_scan(split_slots, scan_smem, &slots);
    for (int b = b0; b < b1; ++b) {
        seq_info[4 * b + 3] = (int32_t)sl;
        const int nsplit = seq_info[4 * b + 2];
        if (nsplit >= 2) sl += nsplit;
        // the units whose range starts inside this sequence start their walk here
        const int first = seq_info[4 * b + 1];
        for (int c = first; c >= 0 && c < first + nsplit; ++c)
            if (ranges[2 * c] >= tile_off[b]) cta_seq[c] = b;
    }
    for (int c = threadIdx.x; c < ctas; c += blockDim.x)
        ranges[2 * c + 1] = c + 1 < ctas ? ranges[2 * (c + 1)] : (int32_t)total;
    for (int i = threadIdx.x; i < 2 * batch * groups; i += blockDim.x) counters[i] = 0;
    for (int i = threadIdx.x; i < batch; i += blockDim.x) ws[sc.done / 4 + i] = 0;
    if (threadIdx.x == 0) {
        tile_off[batch] = (int32_t)total;
        ws[hdr + kSchCtas] = ctas;
        ws[hdr + kSchGroups] = groups;
        ws[hdr + kSchTotal] = (int32_t)total;
        ws[hdr + kSchSlotsUsed] = (int32_t)slots;
        ws[hdr + kSchGroupCols] = gcols;
        ws[hdr + kSchMode] = mode;
    }
}

// The same tables for up to kPlanThreads sequences (thread b owns sequence b, of length L) and work
// units: lengths and offsets stay in registers and shared memory, and the range starts are found by a
// thread per range (a search for the sequence that holds its cost position) instead of by the
// sequence's thread, range after range.
struct PlanSmem {
    int64_t scan[64];
    int64_t f[kPlanThreads], g[kPlanThreads];  // first flattened unit, first cost position
    int32_t start[kPlanThreads + 1];           // first flattened unit of each range
};
__device__ void plan_schedule_small(int L, int batch, int ctas, int groups, int sched, int unit_rows, int gcols,
                                    int mode, int32_t *__restrict__ ws, const Sched &sc, int hdr, PlanSmem &sm) {
    const int b = threadIdx.x, c = threadIdx.x;
    const bool is_seq = b < batch;
    const int64_t units = is_seq ? units_of(L, unit_rows) : 0;
    int64_t f = units, ends = units > 0, total, total_ends;
    block_exclusive_scan2(f, ends, sm.scan, &total, &total_ends);
    const int E = end_cost_units(sched, mode, total, ctas);
    const int64_t g = f + E * ends, total_cost = total + E * total_ends;
    const int used = used_ctas(total, ctas);
    sm.f[b] = f;
    sm.g[b] = g;
    // the last of the sequences whose offset is at most x (those without units share their successor's)
    auto find = [&](const int64_t *off, int64_t x) -> int {
        int lo = 0, hi = batch;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (off[mid] <= x)
                lo = mid;
            else
                hi = mid;
        }
        return lo;
    };
    int first = -1, nsplit = 0;
    if (units > 0) {
        first = cta_of(total_cost, used, g);
        nsplit = cta_of(total_cost, used, g + units - 1) - first + 1;
    }
    int64_t slot = nsplit >= 2 ? nsplit : 0, slots;
    slot = block_exclusive_scan(slot, sm.scan, &slots);  // (its barriers publish f and g)
    if (c < ctas) {
        int64_t s = total;
        if (c < used) {
            const int64_t x = cta_begin(total_cost, used, c);
            const int q = find(sm.g, x);
            const int64_t end = q + 1 < batch ? sm.f[q + 1] : total;
            s = unit_at_cost(x, sm.g[q], sm.f[q], end - sm.f[q]);
        }
        sm.start[c] = (int32_t)s;
    }
    if (c == 0) sm.start[ctas] = (int32_t)total;
    __syncthreads();
    int32_t *counters = ws + sc.counters / 4;
    if (is_seq) {
        ws[sc.tile_off / 4 + b] = (int32_t)f;
        reinterpret_cast<int4 *>(ws + sc.seq_info / 4)[b] = make_int4((int)units, first, nsplit, (int)slot);
        ws[sc.done / 4 + b] = 0;
    }
    if (c < ctas) {
        const int32_t s = sm.start[c], e = sm.start[c + 1];
        reinterpret_cast<int2 *>(ws + sc.cta_ranges / 4)[c] = make_int2(s, e);
        ws[sc.cta_seq / 4 + c] = s < e ? find(sm.f, s) : batch;
    }
    for (int i = threadIdx.x; i < 2 * batch * groups; i += kPlanThreads) counters[i] = 0;
    if (threadIdx.x == 0) {
        ws[sc.tile_off / 4 + batch] = (int32_t)total;
        ws[hdr + kSchCtas] = ctas;
        ws[hdr + kSchGroups] = groups;
        ws[hdr + kSchTotal] = (int32_t)total;
        ws[hdr + kSchSlotsUsed] = (int32_t)slots;
        ws[hdr + kSchGroupCols] = gcols;
        ws[hdr + kSchMode] = mode;
    }
}

// The schedules share no table, so a CTA makes each and they run side by side: CTA 0 the pair schedule, for
// more than 16 query columns CTA 1 the duo schedule and CTA 2 the tree schedule (whose column-group
// widths depend on the lengths).  CTA 0 writes the header (and clears the status word) so that
// the decode kernels can check that they run on a plan for their own grid.
//
// What bounds a plan is its chain of launch, lengths, sums and table writes.  Three schedules at B = 16,
// q_len = 4..8, h = 16 (device time of plans in a row): one after the other 9.5 us; a CTA each 6.3; ranges
// found by a thread each (plan_schedule_small) 4.1..4.4; within warps (plan_warps_kernel) 2.5.
__device__ __forceinline__ void plan_header(int batch, int ncols, int slots, int32_t *ws) {
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        ws[kHdrStatus] = 0;
        ws[kHdrBatch] = batch;
        ws[kHdrCols] = ncols;
        ws[kHdrSlotsMax] = slots;
        ws[kHdrSchedUsed] = 0;
        if (gridDim.x < 3) ws[kHdrTree + kSchCtas] = 0;
    }
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const int32_t *__restrict__ seqlens, int batch, int ncols,
                                                            int num_sms, int32_t *__restrict__ ws, WsLayout lay) {
    // Launched as a programmatic dependent: nothing is read (seqlens may come from the
    // preceding kernel) or written (that kernel may still read the workspace) before it
    // completes.  Then the decode kernel may start its prologue: it waits for this grid in
    // turn before reading the workspace.  Both are no-ops without programmatic launch.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __shared__ PlanSmem sm;
    __shared__ int min_smem[32];
    const int per = (batch + kPlanThreads - 1) / kPlanThreads;
    const int b0 = min(batch, (int)threadIdx.x * per), b1 = min(batch, b0 + per);
    int mn = 0x7fffffff;  // this thread's shortest nonempty sequence
    int64_t units = 0;    // and its sequences' units of kDuoRows
    for (int b = b0; b < b1; ++b) {
        const int L = seqlens[b];
        if (L > 0) mn = min(mn, L);
        units += units_of(L, kDuoRows);
    }
    const int L = per == 1 && b0 < b1 && mn != 0x7fffffff ? mn : 0;  // its only sequence
    int ctas = lay.ctas, groups = lay.groups, mode = 0;
    if (blockIdx.x >= 1) {
        mn = block_min(mn, min_smem);
        mn = mn == 0x7fffffff ? 0 : mn;
        mode = duo_mode(ncols, mn);
        if (blockIdx.x == 2) {
            int64_t all;
            block_exclusive_scan(units, sm.scan, &all);
            mode = tree_mode(ncols, mn, all, num_sms);
        }
        groups = duo_groups(ncols, mode);
        ctas = num_ctas(num_sms, groups);
    }
    const Sched &sc = blockIdx.x == 0 ? lay.pair : blockIdx.x == 1 ? lay.duo : lay.tree;
    const int hdr = blockIdx.x == 0 ? kHdrPair : blockIdx.x == 1 ? kHdrDuo : kHdrTree;
    const int unit_rows = blockIdx.x == 0 ? kTileRows : kDuoRows;
    const int gcols = blockIdx.x == 0 ? group_cols(ncols) : duo_group_cols(mode);
    if (per == 1 && ctas <= kPlanThreads)
        plan_schedule_small(L, batch, ctas, groups, blockIdx.x, unit_rows, gcols, mode, ws, sc, hdr, sm);
    else
        plan_schedule(seqlens, batch, b0, b1, ctas, groups, blockIdx.x, unit_rows, gcols, mode, ws, sc, hdr, sm.scan);
    plan_header(batch, ncols, lay.slots, ws);
}

// The same plan for at most kWarpPlanSeqs sequences and kWarpPlanThreads work units: lane b of every warp owns
// sequence b, so that sums and searches stay within warps and nothing waits for another warp.  Warp 0
// writes the sequences' entries, thread c work unit c's range.  2.5 us for three schedules, 2.35 for one,
// most of it launch; the blocks of plan_kernel take 4.1..4.4 and 2.9 (33 sequences: 3.7).
constexpr int kWarpPlanThreads = 128, kWarpPlanSeqs = 32;
__global__ void __launch_bounds__(kWarpPlanThreads) plan_warps_kernel(const int32_t *__restrict__ seqlens, int batch,
                                                                      int ncols, int num_sms, int32_t *__restrict__ ws,
                                                                      WsLayout lay) {
    asm volatile("griddepcontrol.wait;" ::: "memory");  // as in plan_kernel
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    constexpr uint32_t kAll = 0xffffffffu;
    const int lane = threadIdx.x & 31, c = threadIdx.x;
    const int L = lane < batch ? seqlens[lane] : 0;
    const bool pair = blockIdx.x == 0;
    const int unit_rows = pair ? kTileRows : kDuoRows;
    // positions on the cost axis fit 32 bits: at most ceil(INT32_MAX / kTileRows) units and 4 end positions a sequence
    static_assert(kWarpPlanSeqs <= 32 && (int64_t)kWarpPlanSeqs * (0x7fffffff / kTileRows + 1 + 4) <= 0x7fffffff &&
                      kTileRows <= kDuoRows,
                  "32-bit sums");
    const int units = units_of(L, unit_rows);
    int f = units;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(kAll, f, d);
        if (lane >= d) f += v;
    }
    const int total = __shfl_sync(kAll, f, 31);
    f -= units;  // first flattened unit
    const uint32_t nonempty = __ballot_sync(kAll, units > 0);
    int ctas = lay.ctas, groups = lay.groups, gcols = group_cols(ncols), mode = 0;
    if (!pair) {
        const int shortest = __reduce_min_sync(kAll, L > 0 ? L : 0x7fffffff);
        const int mn = shortest == 0x7fffffff ? 0 : shortest;
        mode = blockIdx.x == 1 ? duo_mode(ncols, mn) : tree_mode(ncols, mn, total, num_sms);
        groups = duo_groups(ncols, mode);
        ctas = num_ctas(num_sms, groups);
        gcols = duo_group_cols(mode);
    }
    const Sched &sc = pair ? lay.pair : blockIdx.x == 1 ? lay.duo : lay.tree;
    const int hdr = pair ? kHdrPair : blockIdx.x == 1 ? kHdrDuo : kHdrTree;
    const int used = used_ctas(total, ctas), E = end_cost_units(blockIdx.x, mode, total, ctas);
    const int g = f + E * __popc(nonempty & ((1u << lane) - 1)), total_cost = total + E * __popc(nonempty);
    // the last of the sequences whose offset (`off` of its lane) is at most x; every lane calls it
    auto find = [&](int off, int x) -> int {
        int lo = 0;
#pragma unroll
        for (int step = 16; step >= 1; step >>= 1) {
            const int at = lo + step, v = __shfl_sync(kAll, off, at);
            if (at < batch && v <= x) lo = at;
        }
        return lo;
    };
    auto range_start = [&](int r) -> int {
        // (past the used ranges, and with no rows at all, there is no position to look for)
        const int64_t x = r < used ? cta_begin(total_cost, used, r) : 0;
        const int q = find(g, (int)x);
        const int gq = __shfl_sync(kAll, g, q), fq = __shfl_sync(kAll, f, q), uq = __shfl_sync(kAll, units, q);
        return r < used ? (int)unit_at_cost(x, gq, fq, uq) : total;
    };
    const int s = range_start(c), e = range_start(c + 1);
    const int seq = find(f, s);
    if (c < ctas) {
        reinterpret_cast<int2 *>(ws + sc.cta_ranges / 4)[c] = make_int2(s, e);
        ws[sc.cta_seq / 4 + c] = s < e ? seq : batch;
    }
    if (c < 32) {
        int first = -1, nsplit = 0;
        if (units > 0) {
            first = cta_of(total_cost, used, g);
            nsplit = cta_of(total_cost, used, g + units - 1) - first + 1;
        }
        const int mine = nsplit >= 2 ? nsplit : 0;
        int slot = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int v = __shfl_up_sync(kAll, slot, d);
            if (lane >= d) slot += v;
        }
        if (lane < batch) {
            ws[sc.tile_off / 4 + lane] = f;
            reinterpret_cast<int4 *>(ws + sc.seq_info / 4)[lane] = make_int4(units, first, nsplit, slot - mine);
            ws[sc.done / 4 + lane] = 0;
        }
        if (lane == 31) {  // (the inclusive sums of all lanes)
            ws[sc.tile_off / 4 + batch] = total;
            ws[hdr + kSchCtas] = ctas;
            ws[hdr + kSchGroups] = groups;
            ws[hdr + kSchTotal] = total;
            ws[hdr + kSchSlotsUsed] = slot;
            ws[hdr + kSchGroupCols] = gcols;
            ws[hdr + kSchMode] = mode;
        }
    }
    for (int i = threadIdx.x; i < 2 * batch * groups; i += kWarpPlanThreads) ws[sc.counters / 4 + i] = 0;
    plan_header(batch, ncols, lay.slots, ws);
}

// Stand-alone split merge: one CTA of 128 threads per (column, sequence), 4 latent rows per
// thread.  Up to 8 splits' partial LSEs and outputs are loaded at once, so that a sequence with
// at most 8 splits costs one round trip to L2 once its partials are complete.  Also writes
// O = 0, LSE = -inf for sequences without rows.
//   sched = 0: launched after the decode (or by the caller after MLA_FLAG_SKIP_COMBINE): waits
//             for the whole previous grid (griddepcontrol.wait) and reads the schedule the
//             decode recorded.
//   sched = 1 or 2 (duo or tree): a programmatic dependent of the decode kernel on that schedule
//             (two CTAs per work unit) that starts on the SMs its CTAs leave: each CTA waits only for the split counters of its own sequence and column
//             group (both CTAs of every split add 1 with release semantics once their partials
//             are stored), so early sequences merge while the decode still runs.  The grid as a whole does not
//             complete before the decode does: its last CTA waits for that grid before it exits.  What follows
//             on the stream (the next plan is a programmatic dependent too) waits for this grid only, and
//             without that CTA could clear the status word and rewrite the tables under a running decode.
// Either way, for the duo schedule the last combine CTA of a sequence rearms its counters.
constexpr int kCombineBatch = 8;
__device__ __forceinline__ int ld_acquire_gpu(const int32_t *p) {
    int v;
    asm volatile("ld.acquire.gpu.global.b32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void combine_column(int32_t *__restrict__ ws, const float *__restrict__ opart,
                                               const float *__restrict__ lsepart, int ncols, const WsLayout &lay,
                                               __nv_bfloat16 *__restrict__ o, float *__restrict__ lse, int sched,
                                               unsigned long long wait_limit_ns) {
    const bool spin = sched != 0;
    const int n = blockIdx.x, b = blockIdx.y;
    // the schedule of the decode that wrote the partials (the plan's tables: complete before the
    // decode started)
    const int used = spin ? sched : __ldcg(ws + kHdrSchedUsed);
    const bool duo = used != 0;  // the schedules whose splits are counted for this kernel
    const Sched &sc = used == 0 ? lay.pair : used == 1 ? lay.duo : lay.tree;
    const int32_t *seq_info = ws + sc.seq_info / 4;
    // (behind a decode the host has measured the workspace: this word is inside it, whatever it holds)
    int nsplit = spin ? __ldcg(seq_info + 4 * b + 2) : 0;
    const PlanHeader plan = read_plan_header(ws, used == 0 ? kHdrPair : used == 2 ? kHdrTree : kHdrDuo);
    // Tables of another shape, or of no plan at all, are not used: the decode has refused them too.
    const bool planned = used == 0 ? plan.batch == (int)gridDim.y && plan.ctas == lay.ctas && plan.groups == lay.groups
                                   : (used == 1 || used == 2) && lay.has_duo &&
                                         duo_plan_matches(plan, (int)gridDim.y, ncols, lay.slots, sc.ctas_max);
    if (!planned) {
        if (threadIdx.x == 0) atomicCAS(ws + kHdrStatus, 0, kStatusInvalid);
        return;
    }
    if (!spin) nsplit = __ldcg(seq_info + 4 * b + 2);
    if (nsplit == 1) return;  // written by the decode kernel
    int32_t *cnt = nullptr;
    if (duo && nsplit >= 2)
        cnt = ws + sc.counters / 4 + ((int64_t)b * plan.groups + n / duo_group_cols(plan.mode)) * 2;
    if (spin && nsplit >= 2) {
        __shared__ int ready;
        if (threadIdx.x == 0) {
            const uint64_t t0 = global_timer_ns();
            int ok = 1;
            while (ld_acquire_gpu(cnt) < nsplit || ld_acquire_gpu(cnt + 1) < nsplit) {
                if (global_timer_ns() - t0 > wait_limit_ns) {
                    atomicCAS(ws + kHdrStatus, 0, kStatusTimeout);
                    ok = 0;
                    break;
                }
                __nanosleep(256);
            }
            ready = ok;
        }
        __syncthreads();  // with thread 0's acquire, orders every thread's reads of the partials
        if (!ready) return;
    }
    const int64_t orow = ((int64_t)b * ncols + n) * kDv + 4 * threadIdx.x;
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    float lse_tot = -INFINITY;
    if (nsplit >= 2) {
        const int s0 = seq_info[4 * b + 3];
        const float *l = lsepart + (int64_t)s0 * ncols + n;
        const float *op = opart + ((int64_t)s0 * ncols + n) * kDv + 4 * threadIdx.x;
        float ls[kCombineBatch];
        float4 v[kCombineBatch];
#pragma unroll
        for (int u = 0; u < kCombineBatch; ++u) {
            const int su = u < nsplit ? u : nsplit - 1;
            ls[u] = __ldcg(l + (int64_t)su * ncols);
            v[u] = __ldcg(reinterpret_cast<const float4 *>(op + (int64_t)su * ncols * kDv));
        }
        if (nsplit <= kCombineBatch) {
            lse_tot = merged_lse([&](int s) { return ls[s]; }, nsplit);
        } else {
            lse_tot = merged_lse([&](int s) { return __ldcg(l + (int64_t)s * ncols); }, nsplit);
        }
        // the sum runs in split order, as in the decode kernel's own merge
        if (lse_tot != -INFINITY) {
#pragma unroll
            for (int u = 0; u < kCombineBatch; ++u) {
                if (u < nsplit) {
                    const float w = merge_weight(ls[u], lse_tot);
                    acc[0] = fmaf(w, v[u].x, acc[0]);
                    acc[1] = fmaf(w, v[u].y, acc[1]);
                    acc[2] = fmaf(w, v[u].z, acc[2]);
                    acc[3] = fmaf(w, v[u].w, acc[3]);
                }
            }
            for (int s = kCombineBatch; s < nsplit; ++s) {
                const float w = merge_weight(__ldcg(l + (int64_t)s * ncols), lse_tot);
                const float4 vs = __ldcg(reinterpret_cast<const float4 *>(op + (int64_t)s * ncols * kDv));
                acc[0] = fmaf(w, vs.x, acc[0]);
                acc[1] = fmaf(w, vs.y, acc[1]);
                acc[2] = fmaf(w, vs.z, acc[2]);
                acc[3] = fmaf(w, vs.w, acc[3]);
            }
        }
    }
    const __nv_bfloat162 lo = __floats2bfloat162_rn(acc[0], acc[1]);
    const __nv_bfloat162 hi = __floats2bfloat162_rn(acc[2], acc[3]);
    uint2 packed;
    packed.x = *reinterpret_cast<const uint32_t *>(&lo);
    packed.y = *reinterpret_cast<const uint32_t *>(&hi);
    *reinterpret_cast<uint2 *>(o + orow) = packed;
    if (threadIdx.x == 0) {
        lse[(int64_t)b * ncols + n] = lse_tot;
        if (cnt && atomicAdd(ws + sc.done / 4 + b, 1) == ncols - 1) {
            // every combine CTA of this sequence is past its wait: rearm for the next decode
            const int groups = plan.groups;
            for (int i = 0; i < 2 * groups; ++i) ws[sc.counters / 4 + (int64_t)b * groups * 2 + i] = 0;
            ws[sc.done / 4 + b] = 0;
        }
    }
}

__global__ void __launch_bounds__(128) combine_kernel(int32_t *__restrict__ ws, const float *__restrict__ opart,
                                                      const float *__restrict__ lsepart, int ncols, WsLayout lay,
                                                      __nv_bfloat16 *__restrict__ o, float *__restrict__ lse, int sched,
                                                      unsigned long long wait_limit_ns) {
    if (sched == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
    combine_column(ws, opart, lsepart, ncols, lay, o, lse, sched, wait_limit_ns);
    if (sched != 0 && blockIdx.x == gridDim.x - 1 && blockIdx.y == gridDim.y - 1)
        asm volatile("griddepcontrol.wait;" ::: "memory");
}

}  // namespace mla
