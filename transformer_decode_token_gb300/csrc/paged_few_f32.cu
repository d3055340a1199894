// Attention over a paged fp32 cache, on the CUDA cores.
#include "paged_few.cuh"

namespace gpt2 {

cudaError_t paged_few_f32(const PagedArgs &a, int r, int ctas, cudaStream_t s)
{
    return paged::few_dims<GPT2_F32>(a, r, ctas, s);
}

}  // namespace gpt2
