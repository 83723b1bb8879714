// bfloat16 products, a layer's product: the tiles, with adapters and without.
#include "bf16_tile.h"

namespace moe {

hipError_t tiles_nt(const MatBf16Params& p, hipStream_t s) {
    return p.ad.s ? bf16_tiles<MAT_NT, true>(p, s) : bf16_tiles<MAT_NT, false>(p, s);
}

}  // namespace moe
