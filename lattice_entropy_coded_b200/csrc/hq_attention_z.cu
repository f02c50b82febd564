// hq_attention_z.cu -- attention over Z caches (hq_attention.cuh), instantiated apart so that the
// lattices compile in parallel.
#include "hq_attention.cuh"

namespace hq {

cudaError_t launch_attention_z(int dither, const AttnArgs &a, cudaStream_t s) {
    return dither ? launch_lat<HQ_Z, true>(a, s) : launch_lat<HQ_Z, false>(a, s);
}

}  // namespace hq
