// The 8-bit forms of the grouped products (grouped_tile.h).
#include <hip/hip_runtime.h>

#include "grouped.h"
#include "grouped_stream.h"
#include "grouped_tile.h"

namespace dsmoe {

hipError_t launch_grouped_int8(GroupedShape shape, const GroupedArgs& t, uint64_t tiles, hipStream_t s) {
  return t.p.kind == GroupedKind::kGated ? launch_grouped_tiles<Elem::kI8, GroupedKind::kGated>(shape, t, tiles, s)
                                         : launch_grouped_tiles<Elem::kI8, GroupedKind::kLinear>(shape, t, tiles, s);
}

}  // namespace dsmoe
