// Attention over a paged 16-bit cache, on the CUDA cores.
#include "paged_few.cuh"

namespace gpt2 {

cudaError_t paged_few_16(const PagedArgs &a, int r, int ctas, cudaStream_t s)
{
    return a.kv.dtype == GPT2_F16 ? paged::few_dims<GPT2_F16>(a, r, ctas, s) : paged::few_dims<GPT2_BF16>(a, r, ctas, s);
}

}  // namespace gpt2
