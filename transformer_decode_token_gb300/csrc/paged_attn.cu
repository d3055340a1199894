// gpt2_op_paged_attention: argument checks, the shape of the launch, and the
// kernel that joins the parts of the units that were cut.
#include "paged.cuh"

#include <cmath>

namespace gpt2 {
namespace paged {
namespace {

// Joins the parts of the units that were cut: a warp per unit whose parts begin with
// that warp of the attention's kernel, or, for four or more query heads, a CTA.
template <int KIND, int D, int R>
__global__ void __launch_bounds__(kThreads) k_paged_join(const __grid_constant__ PagedArgs a)
{
    pdl_wait();
    pdl_launch_dependents();
    const int warp = threadIdx.x >> 5;
    const uint32_t w = R >= kNW ? blockIdx.x : blockIdx.x * kNW + warp;
    const int4 h = a.heads[w];
    if (h.z == 0) return;
    const int heads = heads_of<R>(a, h.y);
    for (int r = R >= kNW ? warp : 0; r < heads; r += R >= kNW ? kNW : 1)
        join_row<KIND, D, R>(a, h.x, h.y, w, uint32_t(h.z), r);
}

template <int KIND, int R>
cudaError_t join_dims(const PagedArgs &a, cudaStream_t s)
{
    switch (a.kv.head_dim) {
    case 32: return spec_launch(k_paged_join<KIND, 32, R>, dim3(R >= kNW ? a.warps : a.warps / kNW), kThreads, 0, 1, s, a);
    case 64: return spec_launch(k_paged_join<KIND, 64, R>, dim3(R >= kNW ? a.warps : a.warps / kNW), kThreads, 0, 1, s, a);
    default: return spec_launch(k_paged_join<KIND, 128, R>, dim3(R >= kNW ? a.warps : a.warps / kNW), kThreads, 0, 1, s, a);
    }
}

template <int R>
cudaError_t join_kinds(const PagedArgs &a, cudaStream_t s)
{
    switch (a.kv.dtype) {
    case GPT2_F16: return join_dims<GPT2_F16, R>(a, s);
    case GPT2_BF16: return join_dims<GPT2_BF16, R>(a, s);
    case GPT2_INT8: return join_dims<GPT2_INT8, R>(a, s);
    default: return join_dims<GPT2_E4M3, R>(a, s);
    }
}

// Query heads of a tile: 1, 2 or 4 on the CUDA cores, 8 or 16 on the matrix instructions.
int tile_heads(int q_dtype, int group)
{
    if (group <= 2) return group;
    return q_dtype == GPT2_F32 ? 4 : group <= 8 ? 8 : 16;
}

struct Layout {
    int warps;
    size_t heads, ml, total;          // bytes: of the heads, of (m, l), of everything
    Layout(const gpt2_kv &kv, int r, int sms)
    {
        const int size = elem_size(kv.dtype);
        warps = sms * ring_ctas(r, size, kv.head_dim * size) * tree::kNW;
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
    case 8: return paged::join_kinds<8>(a, s);
    default: return paged::join_kinds<16>(a, s);
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
    if (n_seqs < 0 || n_rows < 0 || n_rows >= (1 << 30) || max_blocks < 1 || (!seq && n_rows > n_seqs))
        return GPT2_ERR_INVALID_ARG;
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
    const int size = elem_size(kv->dtype), ks = paged::tile_rows(r, size, kv->head_dim * size);
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
    a.per_block = 65535 / kv->n_positions + 1;
    a.scale_log2 = scale * 1.4426950408889634f;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int ctas = at.warps / tree::kNW;
    if (r >= 8) rc = spec_rc(paged_mma(a, r, ctas, s));
    else if (kv->dtype == GPT2_F32) rc = spec_rc(paged_few_f32(a, r, ctas, s));
    else if (is_scaled(kv->dtype)) rc = spec_rc(paged_few_8(a, r, ctas, s));
    else rc = spec_rc(paged_few_16(a, r, ctas, s));
    return rc != GPT2_OK ? rc : spec_rc(paged_join(a, r, s));
}
