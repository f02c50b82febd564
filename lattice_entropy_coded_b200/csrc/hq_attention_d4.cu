// hq_attention_d4.cu -- attention over D4 caches (hq_attention.cuh), instantiated apart so that the
// lattices compile in parallel.
#include "hq_attention.cuh"

namespace hq {

cudaError_t launch_attention_d4(int dither, const AttnArgs &a, cudaStream_t s) {
    return dither ? launch_lat<HQ_D4, true>(a, s) : launch_lat<HQ_D4, false>(a, s);
}

}  // namespace hq
