// hq_attention_a2.cu -- attention over A2 caches (hq_attention.cuh), instantiated apart so that the
// lattices compile in parallel.
#include "hq_attention.cuh"

namespace hq {

cudaError_t launch_attention_a2(int dither, const AttnArgs &a, cudaStream_t s) {
    return dither ? launch_lat<HQ_A2, true>(a, s) : launch_lat<HQ_A2, false>(a, s);
}

}  // namespace hq
