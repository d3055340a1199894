// gpt2_op_paged_attention: argument checks, the shape of the launch, and the
// kernel that joins the parts of the units that were cut.
#include "paged.cuh"

#include <cmath>

namespace gpt2 {
namespace paged {
namespace {

// One CTA per warp of the attention's kernel: where a cut unit's parts begin with
// that warp, joins them (the first part is its second place, the others are the
// first places of the warps that follow).  KIND: the cache's type where the parts
// come from the matrix instructions, whose results that are not finite are
// computed anew; -1 otherwise.
template <int KIND, int D, int R>
__global__ void __launch_bounds__(kThreads) k_paged_join(const __grid_constant__ PagedArgs a)
{
    constexpr int kLanes = R * D / 4, kGroups = kLanes < kThreads ? kThreads / kLanes : 1;
    constexpr int kTurns = kLanes > kThreads ? kLanes / kThreads : 1;
    __shared__ float s_top[R], s_inv[R];
    __shared__ float4 s_sum[kGroups > 1 ? kThreads : 1];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_wait();
    pdl_launch_dependents();
    const int4 head = a.heads[blockIdx.x];
    const int n = head.z;
    if (n == 0) return;
    const uint32_t w = blockIdx.x;
    auto place = [&](int i) { return size_t(i == 0 ? w * 2 + 1 : (w + i) * 2); };
    const int heads = heads_of<R>(a, head.y);
    for (int r = warp; r < heads; r += kNW) {
        float top = -INFINITY, l = 0.f;
        for (int i = lane; i < n; i += 32) {
            const float2 v = a.ml[place(i) * R + r];
            const float mn = fmaxf(top, v.x), safe = mn == -INFINITY ? 0.f : mn;
            l = l * exp2_approx(top - safe) + v.y * exp2_approx(v.x - safe);
            top = mn;
        }
        const float all = warp_max(top), safe = all == -INFINITY ? 0.f : all;
        l = warp_sum(l * exp2_approx(top - safe));
        if (lane == 0) {
            s_top[r] = safe;
            s_inv[r] = l == 0.f ? 0.f : 1.f / l;
        }
    }
    __syncthreads();
    bool odd = false;
    const int grp = tid / kLanes;
#pragma unroll
    for (int turn = 0; turn < kTurns; ++turn) {
        const int e = (kLanes < kThreads ? tid % kLanes : tid + turn * kThreads) * 4, r = e / D;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < heads) {
            const float top = s_top[r];
#pragma unroll 4
            for (int i = grp; i < n; i += kGroups) {
                const float4 y = *reinterpret_cast<const float4 *>(a.sums + place(i) * (R * D) + e);
                const float f = exp2_approx(a.ml[place(i) * R + r].x - top);
                v.x = fmaf(y.x, f, v.x), v.y = fmaf(y.y, f, v.y), v.z = fmaf(y.z, f, v.z), v.w = fmaf(y.w, f, v.w);
            }
        }
        if constexpr (kGroups > 1) {
            s_sum[tid] = v;
            __syncthreads();
            if (grp == 0)
#pragma unroll
                for (int k = 1; k < kGroups; ++k) {
                    const float4 y = s_sum[k * kLanes + tid];
                    v.x += y.x, v.y += y.y, v.z += y.z, v.w += y.w;
                }
        }
        if (grp == 0 && r < heads) {
            const float inv = s_inv[r];
            put4(a, row_at<D, R>(a, head.x, head.y, a.out_stride) + e, v.x * inv, v.y * inv, v.z * inv, v.w * inv);
            const float sum = (v.x + v.y + v.z + v.w) * inv;
            odd = odd || !is_finite(sum);
        }
    }
    if constexpr (KIND >= 0) {
        if (!__syncthreads_or(odd)) return;
        for (int r = warp; r < heads; r += kNW) row_anew<KIND, D, R>(a, head.x, head.y, r);
    }
}

template <int KIND, int R>
cudaError_t join_dims(const PagedArgs &a, cudaStream_t s)
{
    switch (a.kv.head_dim) {
    case 32: return spec_launch(k_paged_join<KIND, 32, R>, dim3(a.warps), kThreads, 0, 1, s, a);
    case 64: return spec_launch(k_paged_join<KIND, 64, R>, dim3(a.warps), kThreads, 0, 1, s, a);
    default: return spec_launch(k_paged_join<KIND, 128, R>, dim3(a.warps), kThreads, 0, 1, s, a);
    }
}

// Query heads of a tile: 1, 2 or 4 on the CUDA cores, 8 on the matrix instructions.
int tile_heads(int q_dtype, int group)
{
    if (group <= 2) return group;
    return q_dtype == GPT2_F32 ? 4 : 8;
}

// CTAs that an SM holds of the kernel for these tiles.
int resident(int r)
{
    return r == 4 ? 2 : 3;
}

// Cache rows of a tile, as the kernels have them.
int tile_rows(const gpt2_kv &kv)
{
    const int n = 4096 / (kv.head_dim * elem_size(kv.dtype));
    return n > 32 ? 32 : n;
}

struct Layout {
    int warps;
    size_t heads, ml, total;          // bytes: of the heads, of (m, l), of everything
    Layout(const gpt2_kv &kv, int r, int sms)
    {
        warps = sms * resident(r) * tree::kNW;
        heads = size_t(warps) * sizeof(int4);
        ml = (size_t(warps) * 2 * r * sizeof(float2) + 15) / 16 * 16;
        total = heads + ml + size_t(warps) * 2 * r * kv.head_dim * sizeof(float);
    }
};

bool shape_ok(const gpt2_kv *kv, int q_dtype, int n_head)
{
    if (!kv_ok(kv) || !is_row_type(q_dtype)) return false;
    if (q_dtype != GPT2_F32 && q_dtype != kv->dtype && !is_scaled(kv->dtype)) return false;
    if ((long long)kv->n_head * kv->n_positions * kv->n_slots >= (1ll << 32) - 1) return false;
    return n_head >= 1 && n_head % kv->n_head == 0 && n_head <= (1 << 16);
}

}  // namespace
}  // namespace paged

cudaError_t paged_join(const PagedArgs &a, int r, cudaStream_t s)
{
    switch (r) {
    case 1: return paged::join_dims<-1, 1>(a, s);
    case 2: return paged::join_dims<-1, 2>(a, s);
    case 4: return paged::join_dims<-1, 4>(a, s);
    default: break;
    }
    switch (a.kv.dtype) {
    case GPT2_F16: return paged::join_dims<GPT2_F16, 8>(a, s);
    case GPT2_BF16: return paged::join_dims<GPT2_BF16, 8>(a, s);
    case GPT2_INT8: return paged::join_dims<GPT2_INT8, 8>(a, s);
    default: return paged::join_dims<GPT2_E4M3, 8>(a, s);
    }
}

}  // namespace gpt2

using namespace gpt2;

extern "C" size_t gpt2_op_paged_attention_workspace(const gpt2_kv *kv, int32_t q_dtype, int32_t n_head)
{
    if (!paged::shape_ok(kv, q_dtype, n_head)) return 0;
    int rc;
    const int sms = spec_sms(&rc);
    return sms ? paged::Layout(*kv, paged::tile_heads(q_dtype, n_head / kv->n_head), sms).total : 0;
}

extern "C" int gpt2_op_paged_attention(const gpt2_kv *kv, const void *q, int32_t q_dtype, int64_t q_stride, int32_t n_head,
                                       const int32_t *table, int32_t n_seqs, int32_t max_blocks, const int32_t *seq,
                                       const int32_t *position, int32_t n_rows, float scale, void *out,
                                       int64_t out_stride, void *workspace, size_t workspace_bytes, void *stream)
{
    if (!paged::shape_ok(kv, q_dtype, n_head)) return GPT2_ERR_INVALID_ARG;
    if (!q || !table || !position || !out || !std::isfinite(scale)) return GPT2_ERR_INVALID_ARG;
    if (n_seqs < 0 || n_rows < 0 || max_blocks < 1 || (!seq && n_rows > n_seqs)) return GPT2_ERR_INVALID_ARG;
    const int64_t E = int64_t(n_head) * kv->head_dim;
    if (q_stride < E || out_stride < E || q_stride % 8 || out_stride % 8) return GPT2_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(out) || !aligned4(table, seq, position)) return GPT2_ERR_INVALID_ARG;
    const long long longest = (long long)max_blocks * kv->n_positions;
    if (longest >= (1ll << 31)) return GPT2_ERR_INVALID_ARG;
    PagedArgs a{};
    a.kv = *kv;
    a.group = n_head / kv->n_head;
    const int r = paged::tile_heads(q_dtype, a.group);
    a.row_tiles = (a.group + r - 1) / r;
    const int ks = paged::tile_rows(*kv);
    const double tiles = double(n_rows) * kv->n_head * a.row_tiles * double((longest + ks - 1) / ks);
    if (tiles >= 4.0e9) return GPT2_ERR_INVALID_ARG;
    if (n_rows == 0) return GPT2_OK;
    int rc;
    const int sms = spec_sms(&rc);
    if (!sms) return rc;
    const paged::Layout at(*kv, r, sms);
    if (!workspace || !aligned16(workspace) || workspace_bytes < at.total) return GPT2_ERR_INVALID_ARG;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    a.heads = reinterpret_cast<int4 *>(ws);
    a.ml = reinterpret_cast<float2 *>(ws + at.heads);
    a.sums = reinterpret_cast<float *>(ws + at.heads + at.ml);
    a.warps = at.warps;
    a.q = q;
    a.out = out;
    a.q_stride = q_stride;
    a.out_stride = out_stride;
    a.table = table;
    a.seq = seq;
    a.position = position;
    a.n_seqs = n_seqs;
    a.n_rows = n_rows;
    a.max_blocks = max_blocks;
    a.q_dtype = q_dtype;
    a.per_block = (65536 + kv->n_positions - 1) / kv->n_positions;
    a.scale_log2 = scale * 1.4426950408889634f;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int ctas = at.warps / tree::kNW;
    if (r == 8) rc = spec_rc(paged_mma(a, ctas, s));
    else if (kv->dtype == GPT2_F32) rc = spec_rc(paged_few_f32(a, r, ctas, s));
    else if (is_scaled(kv->dtype)) rc = spec_rc(paged_few_8(a, r, ctas, s));
    else rc = spec_rc(paged_few_16(a, r, ctas, s));
    return rc != GPT2_OK ? rc : spec_rc(paged_join(a, r, s));
}
