// bfloat16 products, the gated one: the tiles, with adapters and without.
#include "bf16_tile.h"

namespace moe {

hipError_t tiles_gated(const MatBf16Params& p, hipStream_t s) {
    return p.ad.s ? bf16_tiles<MAT_GATED, true>(p, s) : bf16_tiles<MAT_GATED, false>(p, s);
}

}  // namespace moe
