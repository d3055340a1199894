// gpt2_op_tree_attention: argument checks, and the shape of the launch.
#include "tree_attn.cuh"

#include <algorithm>
#include <cmath>

using namespace gpt2;

namespace {

// The lengths are on the device, so the rules below go by the cache's positions, and
// were measured with caches that are nearly full: short sequences in a long cache
// get the kernel and the clusters of long ones.

// The 5th-generation tensor cores (tree_attn_tc.cu), in tiles of 32 or 64 query
// rows (0: not): for more than 16 query rows on a cache head over a 16-bit cache
// of the rows' own type, of 1,536 positions or more (in shorter ones the units are
// a few tiles each: 24 rows x 12 heads x 64 sequences, 540 positions, took 56 us
// against 35).
int tensor_tile(const gpt2_kv &kv, int q_dtype, int rows)
{
    if (rows <= 16 || q_dtype != kv.dtype || q_dtype == GPT2_F32 || kv.head_dim < 64) return 0;
    if (kv.n_positions < 1536) return 0;
    if ((long long)kv.n_slots * kv.n_head * kv.n_positions >= (1ll << 31) - 128) return 0;   // TMA's row coordinates
    return rows <= 32 ? 32 : 64;
}

// They pay for their second kernel and for the change from one unit to the next
// where there is much of the cache, sooner with more rows per tile and with
// longer rows of the cache.  Measured in us against the other kernel (query rows x
// cache heads x sequences, positions, dimensions; in millions of elements of k):
//   64 x 12 x 32, 4,096, 64 (101): 94 / 170;  64 x 12 x 16, 1,600 (20): 42 / 53;
//   64 x 12 x 4, 4,096 (13): 31 / 36;  64 x 12 x 8, 1,600 (10): 32 / 30
//   32 x 12 x 8, 4,096, 64 (25): 31 / 38;  32 x 12 x 8, 2,400 (15): 27 / 26
//   32 x 8 x 2, 4,096, 128 (8): 20 / 28;  32 x 8 x 1, 4,096 (4): 18 / 20;
//   32 x 8 x 2, 1,600 (3): 17 / 16
bool tensor_pays(const gpt2_kv &kv, int n_seqs, int tile)
{
    const long long least = kv.head_dim == 128 ? 4000000 : tile == 64 ? 11000000 : 16000000;
    return (long long)n_seqs * kv.n_head * kv.n_positions * kv.head_dim >= least;
}

// Query rows per tile on the CUDA cores (tree_attn_few.cu; 0: the matrix
// instructions): all rows of a single token or a pair, up to four over an fp32
// cache (whose matrix products take three instructions each), and tiles of two
// where there are few rows and sequences, and all that counts is how soon one
// pass is over.  Measured in us against the matrix instructions (sequences x 12
// heads of 64, up to so many positions, cache type):
//   1 row: 64 x 575 bf16 14.5 / 23.7, int8 14.3 / 22.7, fp32 22.7 / 37.5;
//     1 x 1,000 bf16 4.9 / 6.5, fp32 4.8 / 7.3
//   2 rows: 64 x 575 bf16 17.3 / 24.4, int8 18.6 / 22.9
//   4 rows in one tile: 64 x 575 fp32 28.7 / 38.4, but bf16 26.0 / 24.9, int8 29.3 / 23.1
//   8 rows in tiles of two: 1 x 1,000 fp32 6.7 / 7.9, bf16 6.6 / 7.2, int8 7.0 / 7.2;
//     2 x 1,000 fp32 7.7 / 9.5, bf16 7.3 / 7.8; but 1 x 16,000 bf16 25.4 / 21.5,
//     4 x 1,000 bf16 9.4 / 8.9
int few_rows(const gpt2_kv &kv, int n_seqs, int rows)
{
    if (rows <= 2) return rows;
    if (rows <= 8 && kv.n_positions <= 2048 && (long long)n_seqs * kv.n_head * ((rows + 1) / 2) <= 108) return 2;
    return rows <= 4 && kv.dtype == GPT2_F32 ? 4 : 0;
}

// CTAs (of a cluster) that share a unit's cache: twice as many while all clusters
// still run at once (one too many costs a second round: 24 units of 8 fp32 rows
// over 1,024 positions took 9.4 us with 8 CTAs each, 15.3 with 16), and each CTA has
// 128 positions or more.
int splits_for(long long units, int positions, int resident)
{
    int n = 1;
    for (int i = 0; i < 4 && units <= kClustersFit[i] * resident && positions >= 256 * n; ++i) n *= 2;
    return n;
}

bool shape_ok(const gpt2_kv *kv, int q_dtype, int n_head, int max_nodes)
{
    if (!kv_ok(kv) || !is_row_type(q_dtype)) return false;
    if (q_dtype != GPT2_F32 && q_dtype != kv->dtype && !is_scaled(kv->dtype)) return false;
    if (max_nodes < 1 || max_nodes > GPT2_MAX_NODES) return false;
    return n_head >= 1 && n_head % kv->n_head == 0 && n_head <= (1 << 16);
}

}  // namespace

extern "C" size_t gpt2_op_tree_attention_workspace(const gpt2_kv *kv, int32_t q_dtype, int32_t n_head,
                                                   int32_t max_nodes)
{
    if (!shape_ok(kv, q_dtype, n_head, max_nodes)) return 0;
    const int tile = tensor_tile(*kv, q_dtype, max_nodes * (n_head / kv->n_head));
    if (!tile) return 0;
    int rc;
    const int sms = spec_sms(&rc);
    return sms ? tree_attn_tc_workspace(kv->head_dim, tile, sms) : 0;
}

extern "C" int gpt2_op_tree_attention(const gpt2_kv *kv, const void *q, int32_t q_dtype, int64_t q_stride,
                                      int32_t n_head, const int32_t *slot, const int32_t *cached, const int32_t *first,
                                      const uint64_t *mask, int32_t n_seqs, int32_t n_rows, int32_t max_nodes,
                                      float scale, void *out, int64_t out_stride, void *workspace,
                                      size_t workspace_bytes, void *stream)
{
    if (!shape_ok(kv, q_dtype, n_head, max_nodes)) return GPT2_ERR_INVALID_ARG;
    if (!q || !slot || !cached || !first || !mask || !out) return GPT2_ERR_INVALID_ARG;
    if (n_seqs < 0 || n_rows < 0 || !std::isfinite(scale)) return GPT2_ERR_INVALID_ARG;
    const int64_t E = int64_t(n_head) * kv->head_dim;
    if (q_stride < E || out_stride < E || q_stride % 8 || out_stride % 8) return GPT2_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(out)) return GPT2_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(mask) % 8 || !aligned4(slot, cached, first)) return GPT2_ERR_INVALID_ARG;
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
    const int rows = max_nodes * a.group, can = tensor_tile(*kv, q_dtype, rows);
    const int tc = can && tensor_pays(*kv, n_seqs, can) ? can : 0;
    const int few = few_rows(*kv, n_seqs, rows);
    const int tile = tc ? tc : few ? few : rows <= 16 ? 16 : 32;   // (matrix instructions: 16 or 32 query rows per warp)
    a.row_tiles = (rows + tile - 1) / tile;
    const long long units = (long long)n_seqs * kv->n_head * a.row_tiles;
    if (units * 16 >= (1ll << 31)) return GPT2_ERR_INVALID_ARG;
    if (units == 0 || n_rows == 0) return GPT2_OK;
    int rc;
    const int sms = spec_sms(&rc);
    if (!sms) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (can && (!workspace || !aligned16(workspace) ||
                workspace_bytes < tree_attn_tc_workspace(kv->head_dim, can, sms)))
        return GPT2_ERR_INVALID_ARG;
    if (tc) return spec_rc(tree_attn_tc(a, tile, sms, workspace, s));
    // (the CTAs per SM that each kernel is compiled for)
    const int resident = tile == 1 ? 4 : tile == 2 || (tile == 16 && kv->head_dim <= 64) ? 3 : 2;
    a.splits = splits_for(units, kv->n_positions, resident);
    if (few) return spec_rc(tree_attn_few(a, few, s));
    const int mt = tile / 16;
    if (kv->dtype == GPT2_F32) return spec_rc(tree_attn_f32(a, mt, s));
    if (is_scaled(kv->dtype)) return spec_rc(tree_attn_8(a, mt, s));
    return spec_rc(tree_attn_16(a, mt, s));
}
