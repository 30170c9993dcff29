// Row statistics of bfloat16 logits' tiles (xent_dma.hpp).
#include "xent_dma.hpp"

namespace g355 {

hipError_t launch_xent_stats_bf16(int tile, const HeadArgs &h, const int64_t *labels, int v0, float2 *part,
                                 int ldp, float *zl, hipStream_t s) {
    return launch_head<bf16_t>(tile, h, StatsEpilogue{h.M, h.N, v0, labels, part, ldp, zl}, s);
}

}  // namespace g355
