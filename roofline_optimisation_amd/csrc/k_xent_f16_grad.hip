// The products of binary16 dZ with the head and with the hidden rows (xent_dma.hpp).
#include "xent_dma.hpp"

namespace g355 {

hipError_t launch_xent_dx_f16(int tile, bool b_mn, const ProductArgs &p, hipStream_t s) {
    return launch_dx<f16_t>(tile, b_mn, p, s);
}

hipError_t launch_xent_dw_f16(int tile, const ProductArgs &p, hipStream_t s) {
    return launch_dw<f16_t>(tile, p, s);
}

}  // namespace g355
