#include "bf16_tile.h"
namespace moe {
hipError_t tiles_nt(const MatBf16Params& p, hipStream_t s) {
    return p.ad.s ? bf16_tiles<MAT_NT, true>(BF16_TILES, p, s) : bf16_tiles<MAT_NT, false>(BF16_TILES, p, s);
}
}  // namespace moe
