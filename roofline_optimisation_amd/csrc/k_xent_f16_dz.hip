// dZ of binary16 heads, tile by tile of logits (xent_dma.hpp).
#include "xent_dma.hpp"

namespace g355 {

hipError_t launch_xent_dz_f16(int tile, const HeadArgs &h, const RowGrad *rows, int v0, uint16_t *dZ, uint16_t *lo,
                              int ldz, hipStream_t s) {
    return launch_head<f16_t>(tile, h, DzEpilogue<f16_t>{h.M, h.N, v0, rows, dZ, lo, ldz}, s);
}

}  // namespace g355
