// Tree attention over int8 and e4m3 caches (tree_attn.cuh).
#include "tree_attn.cuh"

namespace gpt2 {

cudaError_t tree_attn_8(const TreeArgs &a, int mt, cudaStream_t s)
{
    using namespace tree;
    const bool f32 = a.q_dtype == GPT2_F32;
    if (a.kv.dtype == GPT2_INT8)
        return f32 ? launch_shape<Traits<kF16, 1, 2, 2>>(a, mt, s) : launch_shape<Traits<kF16, 1, 1, 2>>(a, mt, s);
    return f32 ? launch_shape<Traits<kF16, 1, 2, 2, true>>(a, mt, s)
               : launch_shape<Traits<kF16, 1, 1, 2, true>>(a, mt, s);
}

}  // namespace gpt2
