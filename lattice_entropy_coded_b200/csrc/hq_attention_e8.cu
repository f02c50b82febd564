// hq_attention_e8.cu -- attention over E8 caches (hq_attention.cuh), instantiated apart so that the
// lattices compile in parallel.
#include "hq_attention.cuh"

namespace hq {

cudaError_t launch_attention_e8(int dither, const AttnArgs &a, cudaStream_t s) {
    return dither ? launch_lat<HQ_E8, true>(a, s) : launch_lat<HQ_E8, false>(a, s);
}

}  // namespace hq
