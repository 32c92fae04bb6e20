// Tiled kernel of the grouped linears (grouped_tile.h): the gated pair.
#include "grouped_tile.h"

namespace convrot {

hipError_t launch_grouped_tile_gated(GroupedArgs a, const RowPlan& plan, Elt out, hipStream_t stream) {
  switch (static_cast<Act>(a.act)) {
    case Act::GeluErf: return launch_tile_act<1, true>(a, plan, out, stream);
    case Act::GeluTanh: return launch_tile_act<2, true>(a, plan, out, stream);
    default: return launch_tile_act<3, true>(a, plan, out, stream);
  }
}

}  // namespace convrot
