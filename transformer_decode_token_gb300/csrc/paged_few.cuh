// Attention over a paged cache on the CUDA cores in fp32, for one to four query
// heads on a cache head, over the list and the rings of paged.cuh.
//
// A row of the cache lies in a few neighbouring lanes (four for one query head):
// the more of a row a lane holds, the fewer steps across lanes a tile takes, and
// those steps, one waiting for the other, are what a warp's time goes to.  A lane
// multiplies its pieces of T keys with its pieces of q; the products are summed over
// the row's lanes by halving, after which every lane holds keys of its own, and the
// weighted sum takes the weights from the lanes that hold them.  The weights are
// taken relative to a maximum that is only raised when a score passes it by more
// than kSlack (a vote instead of a reduction per tile; fp32 holds 2^kSlack as well as
// 1, but for values near its largest: row_anew).  Lane l looks up the place of the tile's row l in the block table, so that pages
// may have any size and end anywhere in a tile.
//
// Long caches run at the memory's rate (64 sequences of 2,000 to 4,000 rows, 12 heads
// of 64: fp32 175 us, 0.99 of the copy rate, bf16 92, 0.94; int8 58.2, 0.8, where the
// conversion of the codes takes as long as they take to arrive).
#pragma once

#include "paged.cuh"

namespace gpt2 {
namespace paged {
namespace {

constexpr float kSlack = 8.f;

template <int KIND, int D, int R>
struct Few {
    static constexpr int kES = KIND == GPT2_F32 ? 4 : KIND == GPT2_INT8 || KIND == GPT2_E4M3 ? 1 : 2;
    static constexpr bool kScaled = kES == 1;
    static constexpr int kRowB = D * kES, kPieces = kRowB / 16;
    static constexpr int kWant = kES == 1 && (R == 1 || D <= 64) ? 4 : 8;
    static constexpr int LPR = kPieces < kWant ? kPieces : kWant;    // lanes of a cache row
    static constexpr int P = kPieces / LPR;                          // 16-byte pieces of a lane: c, c + LPR, ..
    static constexpr int EP = 16 / kES, E = P * EP;                  // elements of a piece, of a lane
    static constexpr int RPL = 32 / LPR;                             // rows that a warp holds side by side
    static constexpr int KS = tile_rows(R, kES, kRowB);              // rows of a tile
    static constexpr int T = KS / RPL < 1 ? 1 : KS / RPL;            // of which a lane has this many
    static constexpr int kSplit = LPR < T ? LPR : T;                 // lanes that a row's T scores are spread over
    static constexpr int NV = T / kSplit, kSame = LPR / kSplit;      // scores of a lane; lanes with the same ones
    static constexpr int kBytes = 2 * T * P * 512;                   // keys and values of a tile
    static constexpr int kStage = kBytes + (kScaled ? 256 : 0);      // and their scales
    static constexpr int kCtas = ring_ctas(R, kES, kRowB), S = ring_stages(R, kES, kRowB);
    static constexpr size_t kSmem = size_t(kNW) * S * kStage;
};

template <int KIND, int D, int R>
__global__ void __launch_bounds__(kThreads, Few<KIND, D, R>::kCtas) k_paged_few(const __grid_constant__ PagedArgs a)
{
    using F = Few<KIND, D, R>;
    constexpr int E = F::E, EP = F::EP, P = F::P, T = F::T, NV = F::NV, KS = F::KS, LPR = F::LPR, RPL = F::RPL, S = F::S;
    constexpr uint32_t kAll = KS == 32 ? 0xffffffffu : (1u << KS) - 1;
    static_assert(RPL * T == KS && E >= RPL, "every lane has rows, and dimensions of the result");
    extern __shared__ __align__(16) uint8_t dyn[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, c = lane % LPR, grp = lane / LPR;
    pdl_wait();                                          // (the joining kernel is placed when this one's CTAs leave)
    Share<KS> sh;
    find_share<KS, D>(a, sh);
    Place<KS> at = sh.at;
    __shared__ int began[kNW][2];                        // where the warp's share begins: row, unit
    __shared__ uint32_t began_tile[kNW];
    if (lane == 0) began[warp][0] = at.row, began[warp][1] = at.unit, began_tile[warp] = at.tile;
    float sane = 0.f;                                    // NaN once something that was written is not finite
    const uint32_t w = sh.w, x0 = sh.x0, x1 = sh.x1;
    int4 head = make_int4(0, 0, 0, 0);                   // the unit whose parts begin with this warp's: row, unit, parts
    uint8_t *ring = dyn + warp * (S * F::kStage) + lane * 16;
    const uint8_t *kbase = static_cast<const uint8_t *>(a.kv.k) + c * 16;
    const uint8_t *vbase = static_cast<const uint8_t *>(a.kv.v) + c * 16;
    // rows t * RPL + grp of a tile are this lane's; after the halving it holds the
    // scores of t0 .. t0 + NV - 1
    const int t0 = c / F::kSame * NV;
    uint32_t there[S];                                   // which of their rows the ring's tiles have, oldest first
    Place<KS> far = at;                                  // the tile whose copies begin next
    Lookup look;
    uint32_t to_come = x1 - x0;                          // tiles whose copies have not begun
    auto copy = [&](uint32_t stage) {
        uint32_t yes = 0;
        if (to_come) {
            const uint32_t rows = look.rows(a, far, lane), base = smem_addr(ring) + stage * F::kStage;
#pragma unroll
            for (int t = 0; t < T; ++t) {
                const uint32_t r = __shfl_sync(0xffffffffu, rows, t * RPL + grp);
                const bool ok = r != kNone;
                const size_t off = ok ? size_t(r) * F::kRowB : 0;
#pragma unroll
                for (int p = 0; p < P; ++p) {
                    copy_async<16>(base + (t * P + p) * 512, kbase + off + p * LPR * 16, ok);
                    copy_async<16>(base + ((T + t) * P + p) * 512, vbase + off + p * LPR * 16, ok);
                }
            }
            if constexpr (F::kScaled) {
                const bool ok = rows != kNone;
                copy_async<4>(base - lane * 12 + F::kBytes, a.kv.k_scale + (ok ? rows : 0), ok);
                copy_async<4>(base - lane * 12 + F::kBytes + 128, a.kv.v_scale + (ok ? rows : 0), ok);
            }
            yes = __ballot_sync(0xffffffffu, rows != kNone) & kAll;
            if (--to_come) far.next(a);
        }
        copies_commit();
#pragma unroll
        for (int i = 0; i + 1 < S; ++i) there[i] = there[i + 1];
        there[S - 1] = yes;
    };
    float2 q[R][E / 2], o[R][E / 2];
    float m[R], l[R];
    int heads = 0;
    uint32_t from = 0;                                   // the first of the unit's tiles that are this warp's
    auto begin_unit = [&]() {
        heads = heads_of<R>(a, at.unit);
        from = at.tile;
        const size_t q0 = row_at<D, R>(a, at.row, at.unit, a.q_stride) + c * EP;
#pragma unroll
        for (int r = 0; r < R; ++r) {
#pragma unroll
            for (int e = 0; e < E; e += 4) {
                const float4 v = load_row4(a.q, q0 + size_t(r < heads ? r : 0) * D + e / EP * (LPR * EP) + e % EP, a.q_dtype);
                q[r][e / 2] = make_float2(v.x * a.scale_log2, v.y * a.scale_log2);
                q[r][e / 2 + 1] = make_float2(v.z * a.scale_log2, v.w * a.scale_log2);
            }
#pragma unroll
            for (int e = 0; e < E / 2; ++e) o[r][e] = make_float2(0.f, 0.f);
            m[r] = -INFINITY;
            l[r] = 0.f;
        }
    };
#pragma unroll
    for (int i = 0; i < S; ++i) there[i] = 0;
    for (int i = 0; i < S - 1; ++i) copy(i);
    if (x0 < x1) begin_unit();

    uint32_t stage = 0;
    for (uint32_t x = x0; x < x1; ++x) {
        copies_wait<S - 2>();
        copy(stage == 0 ? S - 1 : stage - 1);
        const uint8_t *tile = ring + stage * F::kStage;
        const uint32_t got = there[0];
        stage = stage == S - 1 ? 0 : stage + 1;
        const bool more = x + 1 < x1;
        float s[R][T];
#pragma unroll
        for (int t = 0; t < T; ++t) {
            float2 y[R];
#pragma unroll
            for (int p = 0; p < P; ++p) {
                const uint4 raw = *reinterpret_cast<const uint4 *>(tile + (t * P + p) * 512);
                const uint32_t word[4] = {raw.x, raw.y, raw.z, raw.w};
                float2 k[EP / 2];
                widen<KIND, EP>(word, k);
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int e = 0; e < EP / 2; ++e) {
                        const float2 qe = q[r][p * (EP / 2) + e];
                        y[r] = p == 0 && e == 0 ? make_float2(k[e].x * qe.x, k[e].y * qe.y) : fma2(k[e], qe, y[r]);
                    }
            }
#pragma unroll
            for (int r = 0; r < R; ++r) s[r][t] = y[r].x + y[r].y;
        }
        // sums over a cache row's lanes (a step of every query row before the next
        // step: the shuffles' latencies overlap)
        int n = T;
#pragma unroll
        for (int d = LPR / 2; d > 0; d /= 2) {
            const bool halve = n > NV, up = c & d;
            if (halve) n /= 2;
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int i = 0; i < T; ++i)
                    if (i < n) {
                        if (halve) {
                            const float mine = up ? s[r][i + n] : s[r][i], other = up ? s[r][i] : s[r][i + n];
                            s[r][i] = mine + __shfl_xor_sync(0xffffffffu, other, d);
                        } else {
                            s[r][i] += __shfl_xor_sync(0xffffffffu, s[r][i], d);
                        }
                    }
        }
        float kf[NV], vf[NV];
        if constexpr (F::kScaled) {
            const float ks = *reinterpret_cast<const float *>(tile - lane * 12 + F::kBytes);   // of the tile's row `lane`
            const float vs = *reinterpret_cast<const float *>(tile - lane * 12 + F::kBytes + 128);
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                kf[k] = __shfl_sync(0xffffffffu, ks, (t0 + k) * RPL + grp);
                vf[k] = __shfl_sync(0xffffffffu, vs, (t0 + k) * RPL + grp);
            }
        }
        bool above = false;
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                if constexpr (F::kScaled) s[r][k] *= kf[k];
                if (got != kAll && !(got >> ((t0 + k) * RPL + grp) & 1)) s[r][k] = -INFINITY;
                above = above || s[r][k] > m[r] + kSlack;
            }
        if (__any_sync(0xffffffffu, above)) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                float top = m[r];
#pragma unroll
                for (int k = 0; k < NV; ++k) top = fmaxf(top, s[r][k]);
                top = warp_max(top);
                const float keep = exp2_approx(m[r] - (top == -INFINITY ? 0.f : top));
                m[r] = top;
                l[r] *= keep;
#pragma unroll
                for (int e = 0; e < E / 2; ++e) o[r][e] = make_float2(o[r][e].x * keep, o[r][e].y * keep);
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float safe = m[r] == -INFINITY ? 0.f : m[r];
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                s[r][k] = exp2_approx(s[r][k] - safe);
                l[r] += s[r][k];
                if constexpr (F::kScaled) s[r][k] *= vf[k];
            }
        }
        // (a row that is not there is not read: its zeros meet weights of zero)
#pragma unroll
        for (int t = 0; t < T; ++t) {
            float w8[R];
#pragma unroll
            for (int r = 0; r < R; ++r) w8[r] = __shfl_sync(0xffffffffu, s[r][t % NV], grp * LPR + t / NV * F::kSame);
#pragma unroll
            for (int p = 0; p < P; ++p) {
                const uint4 raw = *reinterpret_cast<const uint4 *>(tile + ((T + t) * P + p) * 512);
                const uint32_t word[4] = {raw.x, raw.y, raw.z, raw.w};
                float2 v[EP / 2];
                widen<KIND, EP>(word, v);
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int e = 0; e < EP / 2; ++e) {
                        float2 &y = o[r][p * (EP / 2) + e];
                        y = fma2(make_float2(w8[r], w8[r]), v[e], y);
                    }
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
                // the rows side by side are added by halving: each lane ends with N of its E elements
                constexpr int N = E / RPL;
                float v[E];
#pragma unroll
                for (int e = 0; e < E / 2; ++e) v[2 * e] = o[r][e].x, v[2 * e + 1] = o[r][e].y;
                int first = 0, k = E;
#pragma unroll
                for (int d = 16; d >= LPR; d /= 2) {
                    k /= 2;
                    const bool up = lane & d;
                    if (up) first += k;
#pragma unroll
                    for (int i = 0; i < E / 2; ++i)
                        if (i < k) {
                            const float mine = up ? v[i + k] : v[i], other = up ? v[i] : v[i + k];
                            v[i] = mine + __shfl_xor_sync(0xffffffffu, other, d);
                        }
                }
                if (r < heads) {
                    const int dim = (c + first / EP * LPR) * EP + first % EP;
                    const float inv = l[r] == 0.f ? 0.f : 1.f / l[r];
#pragma unroll
                    for (int i = 0; i < N; ++i) sane = fmaf(v[i] * inv, 0.f, sane);
                    if (whole) {
                        put<N>(a, row_at<D, R>(a, at.row, at.unit, a.out_stride) + size_t(r) * D + dim, v, inv);
                    } else {
                        float *to = a.sums + (size_t(part) * R + r) * D + dim;
#pragma unroll
                        for (int i = 0; i < N; ++i) to[i] = v[i] * inv;
                        if (lane == 0) a.ml[size_t(part) * R + r] = make_float2(m[r], l[r]);
                    }
                }
            }
            if (!whole && from == 0)
                head = make_int4(at.row, at.unit, int(sh.all.of(x + at.tiles - 1 - at.tile) - w) + 1, 0);
        }
        if (more) {
            at.next(a);
            if (ends) begin_unit();
        }
    }
    if (lane == 0) a.heads[w] = head;
    // (here and not where it is written: a call from the loop takes registers of the loop's)
    if (__any_sync(0xffffffffu, sane != 0.f)) {
        __syncwarp();
        share_anew<KIND, D, R, KS>(a, w, began[warp][0], began[warp][1], began_tile[warp], at.row, at.unit, at.tile);
    }
}

template <int KIND, int D, int R>
cudaError_t few_launch(const PagedArgs &a, int ctas, cudaStream_t s)
{
    const size_t smem = Few<KIND, D, R>::kSmem;
    const cudaError_t e = allow<k_paged_few<KIND, D, R>>(smem);
    return e != cudaSuccess ? e : spec_launch(k_paged_few<KIND, D, R>, dim3(ctas), kThreads, smem, 1, s, a);
}

template <int KIND, int D>
cudaError_t few_rows(const PagedArgs &a, int r, int ctas, cudaStream_t s)
{
    if (r == 1) return few_launch<KIND, D, 1>(a, ctas, s);
    if (r == 2) return few_launch<KIND, D, 2>(a, ctas, s);
    return few_launch<KIND, D, 4>(a, ctas, s);
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
