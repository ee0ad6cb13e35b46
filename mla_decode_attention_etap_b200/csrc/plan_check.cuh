// The question every kernel on the duo or tree schedule asks before it uses the plan's tables.
#pragma once

#include <cstdint>

#include "plan_core.h"

namespace mla {

// Header words of a schedule.  They are read together: one after the other, as a chain of conditions reads them,
// costs an L2 round trip each (a combine CTA lives for little more than three).
struct PlanHeader {
    int batch, cols, slots;              // of the plan
    int ctas, groups, group_cols, mode;  // of the schedule whose words start at `hdr`
};
__device__ __forceinline__ PlanHeader read_plan_header(const int32_t *ws, int hdr) {
    static_assert(kHdrStatus == 0 && kHdrBatch == 1 && kHdrCols == 2 && kHdrSlotsMax == 3 && kHdrPair % 8 == 0 &&
                      kHdrDuo % 8 == 0 && kHdrTree % 8 == 0 && kSchCtas == 0 && kSchGroups == 1 &&
                      kSchGroupCols == 4 && kSchMode == 5,
                  "header words read as vectors");
    const int4 a = __ldcg(reinterpret_cast<const int4 *>(ws));
    const int4 s = __ldcg(reinterpret_cast<const int4 *>(ws + hdr));
    const int2 t = __ldcg(reinterpret_cast<const int2 *>(ws + hdr + 4));
    return {a.y, a.z, a.w, s.x, s.y, t.x, t.y};
}
// Is it a duo or tree schedule made for this shape and this number of SMs, with at most ctas_max work units?  The
// tables lie where `slots` and the shape put them, so nothing in them may be used before this has been asked.
__device__ __forceinline__ bool duo_plan_matches(const PlanHeader &h, int batch, int ncols, int slots, int ctas_max) {
    return (h.batch == batch) & (h.cols == ncols) & (h.slots == slots) & (h.mode == 0 || h.mode == 1) &
           (h.group_cols == duo_group_cols(h.mode)) & (h.groups == duo_groups(ncols, h.mode)) & (h.ctas >= 1) &
           (h.ctas <= ctas_max);
}

}  // namespace mla
