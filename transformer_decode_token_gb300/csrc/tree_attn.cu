// gpt2_op_tree_attention: argument checks, and the shape of the launch.
#include "tree_attn.cuh"

#include <algorithm>
#include <cmath>

using namespace gpt2;

extern "C" int gpt2_op_tree_attention(const gpt2_kv *kv, const void *q, int32_t q_dtype, int64_t q_stride,
                                      int32_t n_head, const int32_t *slot, const int32_t *cached, const int32_t *first,
                                      const uint64_t *mask, int32_t n_seqs, int32_t n_rows, int32_t max_nodes,
                                      float scale, void *out, int64_t out_stride, void *stream)
{
    if (!kv_ok(kv) || !q || !slot || !cached || !first || !mask || !out) return GPT2_ERR_INVALID_ARG;
    if (!is_row_type(q_dtype) || n_seqs < 0 || n_rows < 0 || !std::isfinite(scale)) return GPT2_ERR_INVALID_ARG;
    if (q_dtype != GPT2_F32 && q_dtype != kv->dtype && !is_scaled(kv->dtype)) return GPT2_ERR_INVALID_ARG;
    if (max_nodes < 1 || max_nodes > GPT2_MAX_NODES) return GPT2_ERR_INVALID_ARG;
    if (n_head < 1 || n_head % kv->n_head || n_head > (1 << 16)) return GPT2_ERR_INVALID_ARG;
    const int64_t E = int64_t(n_head) * kv->head_dim;
    if (q_stride < E || out_stride < E || q_stride % 8 || out_stride % 8) return GPT2_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(out)) return GPT2_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(mask) % 8) return GPT2_ERR_INVALID_ARG;
    TreeArgs a{};
    a.kv = *kv;
    a.q = q;
    a.out = out;
    a.q_stride = q_stride;
    a.out_stride = out_stride;
    a.slot = slot;
    a.cached = cached;
    a.first = first;
    a.mask = mask;
    a.n_seqs = n_seqs;
    a.n_rows = n_rows;
    a.max_nodes = max_nodes;
    a.q_dtype = q_dtype;
    a.group = n_head / kv->n_head;
    a.scale_log2 = scale * 1.4426950408889634f;
    // 16 rows of a (sequence, cache head) per warp, or 32 where there are more
    const int rows = max_nodes * a.group, mt = rows <= 16 ? 1 : 2;
    a.row_tiles = (rows + 16 * mt - 1) / (16 * mt);
    const long long units = (long long)n_seqs * kv->n_head * a.row_tiles;
    if (units * 16 >= (1ll << 31)) return GPT2_ERR_INVALID_ARG;
    if (units == 0 || n_rows == 0) return GPT2_OK;
    int rc;
    const int sms = spec_sms(&rc);
    if (!sms) return rc;
    // split the cache between up to 16 CTAs (a cluster) until there are about
    // four per SM, as long as each has 128 positions or more
    a.splits = 1;
    while (a.splits < 16 && units * a.splits < 2ll * sms && kv->n_positions >= 256 * a.splits) a.splits *= 2;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (kv->dtype == GPT2_F32) return spec_rc(tree_attn_f32(a, mt, s));
    if (is_scaled(kv->dtype)) return spec_rc(tree_attn_8(a, mt, s));
    return spec_rc(tree_attn_16(a, mt, s));
}
