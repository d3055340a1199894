// Attention over a paged cache on the CUDA cores in fp32, for one to four query
// heads on a cache head: the layout of tree_attn_few.cu's kernel (a cache row in
// neighbouring lanes, 16 bytes in each, scores summed over them by halving), over
// the list of paged.cuh.  Lane l looks up the place of the tile's row l in the
// block table, so that pages may have any size and end anywhere in a tile; the
// next tile's places are looked up, and its keys are on their way, while this
// tile's weights are formed.
#pragma once

#include "paged.cuh"

namespace gpt2 {
namespace paged {
namespace {

template <int KIND, int D, int R>
__global__ void __launch_bounds__(kThreads, R == 1 ? 4 : R == 2 ? 3 : 2) k_paged_few(const __grid_constant__ PagedArgs a)
{
    using F = Few<KIND, D>;
    constexpr int E = F::kE, I = F::kLoads, NV = F::kNV, KS = F::KS, LPR = F::kLPR, RPL = F::kRPL;
    constexpr uint32_t kAll = KS == 32 ? 0xffffffffu : (1u << KS) - 1;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, c = lane % LPR, grp = lane / LPR;
    const uint32_t w = warp * gridDim.x + blockIdx.x;    // (so that fewer shares than warps spread over the SMs)
    pdl_wait();
    pdl_launch_dependents();
    Shares sh(1, 1);
    uint32_t x0 = 0, x1 = 0;
    Place<KS> at;
    if (!find_share<KS, D>(a, w, sh, x0, x1, at)) {
        if (lane == 0) a.heads[w] = make_int4(0, 0, 0, 0);
        return;
    }
    const uint8_t *kbase = static_cast<const uint8_t *>(a.kv.k) + c * 16;
    const uint8_t *vbase = static_cast<const uint8_t *>(a.kv.v) + c * 16;
    // access i of a tile holds cache rows i * RPL + grp; after the halving this
    // lane holds the scores of accesses i0 .. i0 + NV - 1
    const int i0 = c / F::kSame * NV;
    uint32_t kr[I][4], vr[I][4];
    auto load = [&](uint32_t (&x)[I][4], const uint8_t *base, uint32_t rows) {
#pragma unroll
        for (int i = 0; i < I; ++i) {
            const uint32_t r = __shfl_sync(0xffffffffu, rows, i * RPL + grp);
            load_piece<16>(x[i], base + size_t(r) * F::kRowB, r != kNone);
        }
    };
    float2 q[R][E / 2], o[R][E / 2];
    float m[R], l[R];
    int heads = 0;
    uint32_t from = 0;                                   // the first of the unit's tiles that are this warp's
    auto begin_unit = [&]() {
        heads = heads_of<R>(a, at.unit);
        from = at.tile;
        const size_t q0 = row_at<D, R>(a, at.row, at.unit, a.q_stride) + c * E;
#pragma unroll
        for (int r = 0; r < R; ++r) {
#pragma unroll
            for (int e = 0; e < E; e += 4) {
                const float4 v = load_row4(a.q, q0 + size_t(r < heads ? r : 0) * D + e, a.q_dtype);
                q[r][e / 2] = make_float2(v.x * a.scale_log2, v.y * a.scale_log2);
                q[r][e / 2 + 1] = make_float2(v.z * a.scale_log2, v.w * a.scale_log2);
            }
#pragma unroll
            for (int e = 0; e < E / 2; ++e) o[r][e] = make_float2(0.f, 0.f);
            m[r] = -INFINITY;
            l[r] = 0.f;
        }
    };
    uint32_t rows = at.at(a, lane);
    load(kr, kbase, rows);
    begin_unit();
    int4 head = make_int4(0, 0, 0, 0);

    for (uint32_t x = x0; x < x1; ++x) {
        load(vr, vbase, rows);
        float ks = 0.f, vs = 0.f;                        // of the tile's row `lane`
        if constexpr (F::kScaled) {
            ks = load_scale(a.kv.k_scale + rows, rows != kNone);
            vs = load_scale(a.kv.v_scale + rows, rows != kNone);
        }
        const bool more = x + 1 < x1;
        Place<KS> then = at;
        uint32_t rows_then = kNone;
        if (more) {
            then.next(a);
            rows_then = then.at(a, lane);
        }
        float s[R][I];
#pragma unroll
        for (int i = 0; i < I; ++i) {
            float2 k[E / 2];
            widen<KIND, E>(kr[i], k);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                float2 y = make_float2(k[0].x * q[r][0].x, k[0].y * q[r][0].y);
#pragma unroll
                for (int e = 1; e < E / 2; ++e) y = fma2(k[e], q[r][e], y);
                s[r][i] = y.x + y.y;
            }
        }
        if (more) load(kr, kbase, rows_then);
        // sums over a cache row's lanes (a step of every query row before the next
        // step: the shuffles' latencies overlap)
        int n = I;
#pragma unroll
        for (int d = LPR / 2; d > 0; d /= 2) {
            const bool halve = n > NV, up = c & d;
            if (halve) n /= 2;
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int i = 0; i < I; ++i)
                    if (i < n) {
                        if (halve) {
                            const float mine = up ? s[r][i + n] : s[r][i], other = up ? s[r][i] : s[r][i + n];
                            s[r][i] = mine + __shfl_xor_sync(0xffffffffu, other, d);
                        } else {
                            s[r][i] += __shfl_xor_sync(0xffffffffu, s[r][i], d);
                        }
                    }
        }
        const uint32_t there = __ballot_sync(0xffffffffu, rows != kNone) & kAll;
        float kf[NV], vf[NV];
        if constexpr (F::kScaled) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                kf[k] = __shfl_sync(0xffffffffu, ks, (i0 + k) * RPL + grp);
                vf[k] = __shfl_sync(0xffffffffu, vs, (i0 + k) * RPL + grp);
            }
        }
        float top[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            top[r] = -INFINITY;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                if constexpr (F::kScaled) s[r][k] *= kf[k];
                if (there != kAll && !(there >> ((i0 + k) * RPL + grp) & 1)) s[r][k] = -INFINITY;
                top[r] = fmaxf(top[r], s[r][k]);
            }
        }
#pragma unroll
        for (int d = 16; d >= F::kSame; d /= 2)
#pragma unroll
            for (int r = 0; r < R; ++r) top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], d));
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
                if constexpr (F::kScaled) s[r][k] *= vf[k];
            }
        }
        // (a row that is not there is not read: its zeros meet weights of zero)
#pragma unroll
        for (int i = 0; i < I; ++i) {
            const int src = grp * LPR + i / NV * F::kSame;
            float2 v[E / 2];
            widen<KIND, E>(vr[i], v);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float p = __shfl_sync(0xffffffffu, s[r][i % NV], src);
#pragma unroll
                for (int e = 0; e < E / 2; ++e) o[r][e] = fma2(make_float2(p, p), v[e], o[r][e]);
            }
        }

        const bool ends = at.tile + 1 == at.tiles;
        if (ends || !more) {                             // the unit's result, or this warp's part of it
            const bool whole = ends && from == 0;
            const uint32_t part = w * 2 + (from == 0);
#pragma unroll
            for (int r = 0; r < R; ++r) {
#pragma unroll
                for (int d = 16; d >= F::kSame; d /= 2) l[r] += __shfl_xor_sync(0xffffffffu, l[r], d);
#pragma unroll
                for (int d = 16; d >= LPR; d /= 2)
#pragma unroll
                    for (int e = 0; e < E / 2; ++e) {
                        o[r][e].x += __shfl_xor_sync(0xffffffffu, o[r][e].x, d);
                        o[r][e].y += __shfl_xor_sync(0xffffffffu, o[r][e].y, d);
                    }
                if (r >= heads || lane >= LPR) continue;
                if (whole) {
                    const float inv = l[r] == 0.f ? 0.f : 1.f / l[r];
                    const size_t to = row_at<D, R>(a, at.row, at.unit, a.out_stride) + size_t(r) * D + c * E;
#pragma unroll
                    for (int e = 0; e < E; e += 4)
                        put4(a, to + e, o[r][e / 2].x * inv, o[r][e / 2].y * inv, o[r][e / 2 + 1].x * inv,
                             o[r][e / 2 + 1].y * inv);
                } else {
                    float *to = a.sums + (size_t(part) * R + r) * D + c * E;
#pragma unroll
                    for (int e = 0; e < E; e += 4)
                        *reinterpret_cast<float4 *>(to + e) =
                            make_float4(o[r][e / 2].x, o[r][e / 2].y, o[r][e / 2 + 1].x, o[r][e / 2 + 1].y);
                    if (lane == 0) a.ml[size_t(part) * R + r] = make_float2(m[r], l[r]);
                }
            }
            if (!whole && from == 0)
                head = make_int4(at.row, at.unit, int(sh.of(x + at.tiles - 1 - at.tile) - w) + 1, 0);
            if (more) {
                at = then;
                begin_unit();
            }
        }
        at = then;
        rows = rows_then;
    }
    if (lane == 0) a.heads[w] = head;
}

template <int KIND, int D>
cudaError_t few_rows(const PagedArgs &a, int r, int ctas, cudaStream_t s)
{
    if (r == 1) return spec_launch(k_paged_few<KIND, D, 1>, dim3(ctas), kThreads, 0, 1, s, a);
    if (r == 2) return spec_launch(k_paged_few<KIND, D, 2>, dim3(ctas), kThreads, 0, 1, s, a);
    return spec_launch(k_paged_few<KIND, D, 4>, dim3(ctas), kThreads, 0, 1, s, a);
}

template <int KIND>
cudaError_t few_dims(const PagedArgs &a, int r, int ctas, cudaStream_t s)
{
    switch (a.kv.head_dim) {
    case 32: return few_rows<KIND, 32>(a, r, ctas, s);
    case 64: return few_rows<KIND, 64>(a, r, ctas, s);
    default: return few_rows<KIND, 128>(a, r, ctas, s);
    }
}

}  // namespace
}  // namespace paged
}  // namespace gpt2
