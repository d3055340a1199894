// Internal interface of the speculative-decoding operations: what the C entry
// points (kv_ops.cu, tree_attn.cu, verify.cu) and the batched engine share.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/gpt2.h"

namespace gpt2 {

inline int spec_rc(cudaError_t e)
{
    if (e == cudaSuccess) return GPT2_OK;
    cudaGetLastError();
    return e == cudaErrorMemoryAllocation ? GPT2_ERR_OUT_OF_MEMORY : GPT2_ERR_CUDA;
}

// Launches a kernel as a programmatic dependent of the stream's last one: its
// CTAs may be placed before that one has ended (right away where it was one of
// these, which let the next one go as soon as they all run), and every thread
// calls pdl_wait(), and then pdl_launch_dependents(), before it touches memory
// (but for k_verify, see there).
// cluster: CTAs of a cluster along x, 1: none.
template <typename... P, typename... A>
inline cudaError_t spec_launch(void (*fn)(P...), dim3 grid, unsigned threads, size_t smem, int cluster, cudaStream_t s,
                               A &&...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = unsigned(cluster);
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, fn, static_cast<P>(args)...);
}

inline bool is_row_type(int t) { return t == GPT2_F32 || t == GPT2_F16 || t == GPT2_BF16; }
inline bool is_scaled(int t) { return t == GPT2_INT8 || t == GPT2_E4M3; }
inline int elem_size(int t) { return t == GPT2_F32 ? 4 : is_scaled(t) ? 1 : 2; }
inline bool aligned16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }
// int32 and fp32 arrays (a NULL one is aligned)
template <typename... P>
inline bool aligned4(const P *...p)
{
    return ((reinterpret_cast<uintptr_t>(p) | ...) & 3) == 0;
}

inline bool kv_ok(const gpt2_kv *kv)
{
    if (!kv || !kv->k || !kv->v || !aligned16(kv->k) || !aligned16(kv->v)) return false;
    if (!is_row_type(kv->dtype) && !is_scaled(kv->dtype)) return false;
    if (is_scaled(kv->dtype) && (!kv->k_scale || !kv->v_scale || !aligned4(kv->k_scale, kv->v_scale))) return false;
    if (kv->n_slots < 1 || kv->n_head < 1 || kv->n_positions < 1) return false;
    if (kv->head_dim != 32 && kv->head_dim != 64 && kv->head_dim != 128) return false;
    // (slot, head, position) rows are counted in 64 bits; heads x positions of
    // a slot in 32
    return (long long)kv->n_head * kv->n_positions < (1ll << 31);
}

// Clusters of 2, 4, 8 and 16 CTAs that run at once, per resident CTA of an SM: what
// the runtime reports for a GB300 of 152 SMs, where a cluster stays within a group
// of 16 to 20 of them.  On other groups of SMs the shares of work are not the best
// ones; clusters of 16 are taken only where few units leave room for them, and
// would be refused by a device that has no group of 16 SMs.
constexpr int kClustersFit[] = {76, 36, 17, 7};

// Multiprocessors of the current device (0 and *rc on failure, also where it
// is not of compute capability 10.3).  Looked up once per device.
int spec_sms(int *rc);

}  // namespace gpt2
