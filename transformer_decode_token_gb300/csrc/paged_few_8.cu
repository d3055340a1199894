// Attention over a paged 8-bit cache, on the CUDA cores.
#include "paged_few.cuh"

namespace gpt2 {

cudaError_t paged_few_8(const PagedArgs &a, int r, int ctas, cudaStream_t s)
{
    return a.kv.dtype == GPT2_INT8 ? paged::few_dims<GPT2_INT8>(a, r, ctas, s) : paged::few_dims<GPT2_E4M3>(a, r, ctas, s);
}

}  // namespace gpt2
