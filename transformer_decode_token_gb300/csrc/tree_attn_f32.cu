// Tree attention over an fp32 cache (tree_attn.cuh).
#include "tree_attn.cuh"

namespace gpt2 {

cudaError_t tree_attn_f32(const TreeArgs &a, int mt, cudaStream_t s)
{
    return tree::launch_shape<tree::Traits<tree::kTf32, 4, 2, 2>>(a, mt, s);
}

}  // namespace gpt2
