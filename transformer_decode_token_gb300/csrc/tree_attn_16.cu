// Tree attention over fp16 and bf16 caches (tree_attn.cuh).
#include "tree_attn.cuh"

namespace gpt2 {

cudaError_t tree_attn_16(const TreeArgs &a, int mt, cudaStream_t s)
{
    using namespace tree;
    const bool f32 = a.q_dtype == GPT2_F32;
    if (a.kv.dtype == GPT2_BF16)
        return f32 ? launch_shape<Traits<kBf16, 2, 3, 3>>(a, mt, s) : launch_shape<Traits<kBf16, 2, 1, 2>>(a, mt, s);
    return f32 ? launch_shape<Traits<kF16, 2, 2, 2>>(a, mt, s) : launch_shape<Traits<kF16, 2, 1, 2>>(a, mt, s);
}

}  // namespace gpt2
