// Tiled kernel of the grouped linears (grouped_tile.h): one weight per group.
#include "grouped_tile.h"

namespace convrot {

hipError_t launch_grouped_tile(GroupedArgs a, const RowPlan& plan, Elt out, hipStream_t stream) {
  switch (static_cast<Act>(a.act)) {
    case Act::GeluErf: return launch_tile_act<1, false>(a, plan, out, stream);
    case Act::GeluTanh: return launch_tile_act<2, false>(a, plan, out, stream);
    case Act::Silu: return launch_tile_act<3, false>(a, plan, out, stream);
    default: return launch_tile_act<0, false>(a, plan, out, stream);
  }
}

}  // namespace convrot
