// Tree attention of few query rows (single tokens, short chains and trees of one
// or two sequences), on the CUDA cores in fp32.
//
// The same pass over the cache as tree_attn.cuh's kernel, whose matrix
// instructions take 16 rows at a time: with one or two rows most of that work is
// thrown away, and it bounds the kernel (which rows come here, and what both
// take: tree_attn.cu).  A row of the cache lies in kLPR neighbouring lanes, 16
// bytes in each; a lane multiplies its piece of kLoads keys with its piece of q,
// and the products are summed over the lanes by halving: after it every lane
// holds keys of its own, so that the softmax is computed once per key.  The
// weighted sum takes the weights from the lanes that hold them.  The steps across
// lanes are made for all query rows together, so that their latencies overlap
// (four fp32 rows of one sequence: 6.1 us instead of 6.8).  No rounding but
// fp32's: two products and additions per instruction.
// What bounds it: for 64 sequences of 32 to 575 bf16 rows, 12 heads of 64, 14.2 us
// (4.2 TB/s): 768 CTAs for 608 places, so that the last ones, whatever their
// lengths, start when the first have ended, and each is a chain of dependent loads
// (int8, half the bytes: 13.4 us; fp32, twice: 22.2, 5.4 TB/s); with
// long caches HBM: 64 x 2,000 to 4,000 rows 93.7 us, 6.3 TB/s; fp32 176.6 us, 6.7.
// Four CTAs per SM: with five, registers spill (one sequence 5.2 us instead of 4.8;
// 64 short ones 13.9 instead of 14.3); half the accesses per tile were no better (int8
// 83 us instead of 72 for the long caches).
#include "tree_attn.cuh"

#include <type_traits>

namespace gpt2 {
namespace tree {
namespace {

template <int KIND, int D, int R>
struct Few {
    static constexpr int kES = KIND == GPT2_F32 ? 4 : KIND == GPT2_INT8 || KIND == GPT2_E4M3 ? 1 : 2;
    static constexpr bool kScaled = kES == 1;
    static constexpr int kRowB = D * kES;
    static constexpr int kLPR = kRowB / 16;              // lanes per cache row
    static constexpr int kRPL = 32 / kLPR;               // cache rows per access of a warp
    static constexpr int kE = 16 / kES;                  // elements of a lane
    static constexpr int kLoads = kRPL >= 4 ? 32 / kRPL : 8;   // accesses per tile: 32 rows, or 4 KB
    static constexpr int KS = kLoads * kRPL;
    static constexpr int kSplit = kLPR < kLoads ? kLPR : kLoads;   // lanes that a row's scores are spread over
    static constexpr int kNV = kLoads / kSplit;          // scores of a lane
    static constexpr int kSame = kLPR / kSplit;          // lanes with the same scores
};

template <int KIND, int D, int R>
__global__ void __launch_bounds__(kNW * 32, R == 1 ? 4 : R == 2 ? 3 : 2) k_tree_few(const __grid_constant__ TreeArgs a)
{
    using F = Few<KIND, D, R>;
    constexpr int E = F::kE, I = F::kLoads, NV = F::kNV, KS = F::KS, LPR = F::kLPR;
    __shared__ __align__(16) float so[kNW * R * D];
    __shared__ float sm_m[kNW][R], sm_l[kNW][R];
    __shared__ int sm_bad;
    __shared__ float sm_f[kMaxSplits][R];

    const int rank = blockIdx.x % a.splits, unit = blockIdx.x / a.splits;
    const int rt = unit % a.row_tiles, bh = unit / a.row_tiles;
    const int kvh = bh % a.kv.n_head, b = bh / a.kv.n_head;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, c = lane % LPR, grp = lane / LPR;
    const int P = a.kv.n_positions, G = a.group;
    pdl_wait();
    pdl_launch_dependents();
    const int f0 = min(max(a.first[b], 0), a.n_rows), f1 = min(max(a.first[b + 1], f0), a.n_rows);
    const int nodes = min(f1 - f0, a.max_nodes);
    const int row0 = rt * R, rows = min(nodes * G - row0, R);
    if (rows <= 0) return;                         // the whole cluster leaves
    const int slot = a.slot[b];
    const bool there = slot >= 0 && slot < a.kv.n_slots;
    const int pre = there ? min(max(a.cached[b], 0), P) : 0;
    const int total = there ? min(pre + nodes, P) : 0;
    const size_t row_base = (size_t(there ? slot : 0) * a.kv.n_head + kvh) * P;
    const uint8_t *kbase = static_cast<const uint8_t *>(a.kv.k) + row_base * F::kRowB + c * 16;
    const uint8_t *vbase = static_cast<const uint8_t *>(a.kv.v) + row_base * F::kRowB + c * 16;

    const int tiles = (total + KS - 1) / KS, per = (tiles + a.splits - 1) / a.splits;
    const int t0 = rank * per + warp, t1 = min(tiles, (rank + 1) * per);   // this warp's: t0, t0 + kNW, ..
    // access i of a tile holds cache rows i * kRPL + grp; after the halving this
    // lane holds the scores of accesses i0 .. i0 + NV - 1
    const int i0 = c / F::kSame * NV;
    uint32_t kr[I][4], vr[I][4];
    float ks[NV], vs[NV];
    auto load_keys = [&](int t) {
#pragma unroll
        for (int i = 0; i < I; ++i) {
            const int j = t * KS + i * F::kRPL + grp;
            load_piece<16>(kr[i], kbase + size_t(j) * F::kRowB, j < total);
        }
    };
    auto load_values = [&](int t) {
#pragma unroll
        for (int i = 0; i < I; ++i) {
            const int j = t * KS + i * F::kRPL + grp;
            load_piece<16>(vr[i], vbase + size_t(j) * F::kRowB, j < total);
        }
        if constexpr (F::kScaled) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int j = t * KS + (i0 + k) * F::kRPL + grp;
                ks[k] = load_scale(a.kv.k_scale + row_base + j, j < total);
                vs[k] = load_scale(a.kv.v_scale + row_base + j, j < total);
            }
        }
    };
    if (t0 < t1) {
        load_keys(t0);
        load_values(t0);
    }
    float2 q[R][E / 2], o[R][E / 2];
    float m[R], l[R];
    uint64_t see[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int rr = row0 + (r < rows ? r : 0);
        const size_t at = size_t(f0 + rr / G) * a.q_stride + size_t(kvh * G + rr % G) * D + c * E;
        see[r] = a.mask[f0 + rr / G];
#pragma unroll
        for (int e = 0; e < E; e += 4) {
            const float4 v = load_row4(a.q, at + e, a.q_dtype);
            q[r][e / 2] = make_float2(v.x * a.scale_log2, v.y * a.scale_log2);
            q[r][e / 2 + 1] = make_float2(v.z * a.scale_log2, v.w * a.scale_log2);
        }
#pragma unroll
        for (int e = 0; e < E / 2; ++e) o[r][e] = make_float2(0.f, 0.f);
        m[r] = -INFINITY;
        l[r] = 0.f;
    }

    for (int t = t0; t < t1; t += kNW) {
        if (t > t0) load_values(t);
        float s[R][I];
#pragma unroll
        for (int i = 0; i < I; ++i) {
            float2 x[E / 2];
            widen<KIND, E>(kr[i], x);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                float2 y = make_float2(x[0].x * q[r][0].x, x[0].y * q[r][0].y);
#pragma unroll
                for (int e = 1; e < E / 2; ++e) y = fma2(x[e], q[r][e], y);
                s[r][i] = y.x + y.y;
            }
        }
        if (t + kNW < t1) load_keys(t + kNW);
        // sums over a cache row's lanes (a step of every query row before the next
        // step: the shuffles' latencies overlap)
        int n = I;
#pragma unroll
        for (int x = LPR / 2; x > 0; x /= 2) {
            const bool halve = n > NV, up = c & x;
            if (halve) n /= 2;
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int i = 0; i < I; ++i)
                    if (i < n) {
                        if (halve) {
                            const float mine = up ? s[r][i + n] : s[r][i], other = up ? s[r][i] : s[r][i + n];
                            s[r][i] = mine + __shfl_xor_sync(0xffffffffu, other, x);
                        } else {
                            s[r][i] += __shfl_xor_sync(0xffffffffu, s[r][i], x);
                        }
                    }
        }
        uint32_t seen[R][NV];                      // lanes whose key the row sees (tiles with nodes)
        const bool tail = (t + 1) * KS > pre;
        float top[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            top[r] = -INFINITY;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                if constexpr (F::kScaled) s[r][k] *= ks[k];
                if (tail) {
                    const int j = t * KS + (i0 + k) * F::kRPL + grp;
                    const bool yes = j < pre || (j < total && (see[r] >> (j - pre) & 1));
                    if (!yes) s[r][k] = -INFINITY;
                    seen[r][k] = __ballot_sync(0xffffffffu, yes);
                }
                top[r] = fmaxf(top[r], s[r][k]);
            }
        }
#pragma unroll
        for (int x = 16; x >= F::kSame; x /= 2)
#pragma unroll
            for (int r = 0; r < R; ++r) top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], x));
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float mn = fmaxf(m[r], top[r]), safe = mn == -INFINITY ? 0.f : mn;
            const float keep = exp2_approx(m[r] - safe);
            m[r] = mn;
            l[r] *= keep;
#pragma unroll
            for (int e = 0; e < E / 2; ++e) o[r][e] = make_float2(o[r][e].x * keep, o[r][e].y * keep);
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                s[r][k] = exp2_approx(s[r][k] - safe);
                l[r] += s[r][k];
                if constexpr (F::kScaled) s[r][k] *= vs[k];
            }
        }
        // a value that a row does not see does not meet its weight of zero: it may
        // be an infinity or a NaN
        auto weighted = [&](auto masked) {
#pragma unroll
            for (int i = 0; i < I; ++i) {
                const int from = grp * LPR + i / NV * F::kSame;
                float2 x[E / 2];
                widen<KIND, E>(vr[i], x);
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float p = __shfl_sync(0xffffffffu, s[r][i % NV], from);
                    if (!decltype(masked)::value || (seen[r][i % NV] >> from & 1)) {
#pragma unroll
                        for (int e = 0; e < E / 2; ++e) o[r][e] = fma2(make_float2(p, p), x[e], o[r][e]);
                    }
                }
            }
        };
        if (tail) weighted(std::true_type());
        else weighted(std::false_type());
    }

    // ---- join the warp's rows of the cache, the warps, the cluster ----
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
        for (int x = 16; x >= F::kSame; x /= 2) l[r] += __shfl_xor_sync(0xffffffffu, l[r], x);
#pragma unroll
        for (int x = 16; x >= LPR; x /= 2)
#pragma unroll
            for (int e = 0; e < E / 2; ++e) {
                o[r][e].x += __shfl_xor_sync(0xffffffffu, o[r][e].x, x);
                o[r][e].y += __shfl_xor_sync(0xffffffffu, o[r][e].y, x);
            }
        if (lane == 0) {
            sm_m[warp][r] = m[r];
            sm_l[warp][r] = l[r];
        }
    }
    if (tid == 0) sm_bad = 0;
    __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r) {
        float top = sm_m[0][r];
#pragma unroll
        for (int w = 1; w < kNW; ++w) top = fmaxf(top, sm_m[w][r]);
        const float f = top == -INFINITY ? 0.f : exp2_approx(m[r] - top);
        if (lane < LPR) {
#pragma unroll
            for (int e = 0; e < E; e += 4)
                *reinterpret_cast<float4 *>(so + (warp * R + r) * D + c * E + e) =
                    make_float4(o[r][e / 2].x * f, o[r][e / 2].y * f, o[r][e / 2 + 1].x * f, o[r][e / 2 + 1].y * f);
        }
    }
    __syncthreads();
    join<KIND, D, R>(a, so, sm_m, sm_l, sm_f, &sm_bad, false, rank, Unit{row_base, f0, row0, kvh, rows, pre, total, total});
}

template <int KIND, int D>
cudaError_t few_rows(const TreeArgs &a, int r, cudaStream_t s)
{
    if (r == 1) return launch_tree(k_tree_few<KIND, D, 1>, a, 0, s);
    if (r == 2) return launch_tree(k_tree_few<KIND, D, 2>, a, 0, s);
    if constexpr (KIND == GPT2_F32) return launch_tree(k_tree_few<KIND, D, 4>, a, 0, s);
    else return cudaErrorInvalidValue;
}

template <int KIND>
cudaError_t few_dims(const TreeArgs &a, int r, cudaStream_t s)
{
    switch (a.kv.head_dim) {
    case 32: return few_rows<KIND, 32>(a, r, s);
    case 64: return few_rows<KIND, 64>(a, r, s);
    default: return few_rows<KIND, 128>(a, r, s);
    }
}

}  // namespace
}  // namespace tree

cudaError_t tree_attn_few(const TreeArgs &a, int r, cudaStream_t s)
{
    switch (a.kv.dtype) {
    case GPT2_F32: return tree::few_dims<GPT2_F32>(a, r, s);
    case GPT2_F16: return tree::few_dims<GPT2_F16>(a, r, s);
    case GPT2_BF16: return tree::few_dims<GPT2_BF16>(a, r, s);
    case GPT2_INT8: return tree::few_dims<GPT2_INT8>(a, r, s);
    default: return tree::few_dims<GPT2_E4M3>(a, r, s);
    }
}

}  // namespace gpt2
