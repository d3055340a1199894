// Attention over a paged cache on the matrix instructions, for 16-bit rows and
// three or more query heads on a cache head, over the list of paged.cuh.
//
// The weights meet the values in two parts, p = hi + lo.  For up to 8 query heads
// the 16 rows of an instruction's A side are the heads twice (HALVES = 1): the upper
// half takes the second part of what the lower half is the first part of, so that both
// parts cost one instruction and meet in one thread, which adds the two halves of the
// accumulators.  For up to 16 heads (HALVES = 2) each part has its own instruction.
// Cache rows reach the operand registers in the order of tree_attn.cuh: keys by
// 16-byte pieces c, c + 4, .., values by pieces g, g + 8, .. of the rows whose weights
// the thread holds.
//
// What bounds the kernel over 8-bit caches is the conversion of their codes, two
// thirds of its instructions.  As keys they become fp16, which takes five
// instructions for four int8 codes where bf16 takes eight, and holds e4m3 as it is;
// bf16 queries meet them as fp16 too, each head's times a power of two that brings its
// largest to 2^14 .. 2^15, so that what fp16 cannot hold of the others is below 2^-39
// of that.  The values' weights include the rows' scales, whose range only bf16 has.
#include "paged.cuh"

namespace gpt2 {
namespace paged {
namespace {

// Two 8-bit codes (bytes 0, 1 of x for HIGH = 0, else 2, 3) as a bf16 pair.
// int8: 0x43uu with the code's low seven bits is 128 + those, and 128 or, for a
// negative code, 256 is taken off.
template <int KIND, int HIGH>
__device__ __forceinline__ uint32_t codes_to_bf162(uint32_t x)
{
    if constexpr (KIND == GPT2_INT8) {
        const uint32_t y = __byte_perm(x, 0x43434343u, HIGH ? 0x4342u : 0x4140u);
        const uint32_t u = y & 0xff7fff7fu, v = y & 0xff80ff80u;
        const __nv_bfloat162 d =
            __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&u), *reinterpret_cast<const __nv_bfloat162 *>(&v));
        return *reinterpret_cast<const uint32_t *>(&d);
    } else {
        const uint32_t h = codes_to_half2<true>(x, HIGH ? 0x4342u : 0x4140u);
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
        const __nv_bfloat162 d = __floats2bfloat162_rn(f.x, f.y);
        return *reinterpret_cast<const uint32_t *>(&d);
    }
}

template <int KIND, int D>
struct Shape {
    static constexpr int kES = KIND == GPT2_INT8 || KIND == GPT2_E4M3 ? 1 : 2;
    static constexpr bool kScaled = kES == 1, kHalf = KIND == GPT2_F16;
    static constexpr int kRowB = D * kES;
    static constexpr int kKLd = kRowB / 4 < 16 ? kRowB / 4 : 16, kNK = kRowB / (4 * kKLd);
    static constexpr int kVLd = kRowB / 8 < 16 ? kRowB / 8 : 16, kNV = kRowB / (8 * kVLd);
    static constexpr int kEK = kKLd / kES, kEV = kVLd / kES;   // elements of an access
    static constexpr int KS = tile_rows(8, kES, kRowB);
    static constexpr int kT8 = KS / 8, kSteps = D / 16, kNT = D / 8;
};

template <int KIND, int D>
struct MmaRing {
    using S = Shape<KIND, D>;
    static constexpr int kKeys = S::KS * S::kRowB;
    static constexpr int kStage = 2 * kKeys + (S::kScaled ? 256 : 0);
    static constexpr int kCtas = ring_ctas(8, S::kES, S::kRowB), kStages = ring_stages(8, S::kES, S::kRowB);
    static constexpr size_t kSmem = size_t(kNW) * kStages * kStage;
};

template <int KIND, int D, bool QF16, int HALVES>
__global__ void __launch_bounds__(kThreads, MmaRing<KIND, D>::kCtas) k_paged_mma(const __grid_constant__ PagedArgs a)
{
    using S = Shape<KIND, D>;
    using G = MmaRing<KIND, D>;
    constexpr int R = 8 * HALVES, KS = S::KS, T8 = S::kT8, N = G::kStages;
    constexpr float kRaise = S::kHalf ? 2.f : 8.f;
    constexpr bool kBf = !S::kHalf;
    constexpr uint32_t kAll = KS == 32 ? 0xffffffffu : (1u << KS) - 1;
    extern __shared__ __align__(16) uint8_t dyn[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
    pdl_wait();                                          // (the joining kernel is placed when this one's CTAs leave)
    Share<KS> sh;
    find_share<KS, D>(a, sh);
    Place<KS> at = sh.at;
    const uint32_t w = sh.w, x0 = sh.x0, x1 = sh.x1;
    int4 head = make_int4(0, 0, 0, 0);                   // the unit whose parts begin with this warp's: row, unit, parts
    uint8_t *ring = dyn + warp * (N * G::kStage);
    const uint8_t *kbase = static_cast<const uint8_t *>(a.kv.k) + c * S::kKLd;
    const uint8_t *vbase = static_cast<const uint8_t *>(a.kv.v) + g * S::kVLd;
    uint32_t there[N];                                   // which of their rows the ring's tiles have, oldest first
    Place<KS> far = at;                                  // the tile whose copies begin next
    Lookup look;
    uint32_t to_come = x1 - x0;                          // tiles whose copies have not begun
    auto copy = [&](uint32_t stage) {
        uint32_t yes = 0;
        if (to_come) {
            const uint32_t rows = look.rows(a, far, lane), base = smem_addr(ring) + stage * G::kStage;
#pragma unroll
            for (int t = 0; t < T8; ++t) {
                const uint32_t r = __shfl_sync(0xffffffffu, rows, t * 8 + g);
                const size_t off = r != kNone ? size_t(r) * S::kRowB : 0;
#pragma unroll
                for (int p = 0; p < S::kNK; ++p)
                    copy_async<S::kKLd>(base + ((t * S::kNK + p) * 32 + lane) * S::kKLd, kbase + off + p * 4 * S::kKLd,
                                        r != kNone);
            }
#pragma unroll
            for (int t = 0; t < T8; ++t)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t r = __shfl_sync(0xffffffffu, rows, t * 8 + 2 * c + i);
                    const size_t off = r != kNone ? size_t(r) * S::kRowB : 0;
#pragma unroll
                    for (int p = 0; p < S::kNV; ++p)
                        copy_async<S::kVLd>(base + G::kKeys + (((t * 2 + i) * S::kNV + p) * 32 + lane) * S::kVLd,
                                            vbase + off + p * 8 * S::kVLd, r != kNone);
                }
            if constexpr (S::kScaled) {
                const bool ok = rows != kNone;
                copy_async<4>(base + 2 * G::kKeys + lane * 4, a.kv.k_scale + (ok ? rows : 0), ok);
                copy_async<4>(base + 2 * G::kKeys + 128 + lane * 4, a.kv.v_scale + (ok ? rows : 0), ok);
            }
            yes = __ballot_sync(0xffffffffu, rows != kNone) & kAll;
            if (--to_come) far.next(a);
        }
        copies_commit();
#pragma unroll
        for (int i = 0; i + 1 < N; ++i) there[i] = there[i + 1];
        there[N - 1] = yes;
    };
    uint32_t qa[S::kSteps][HALVES][2];                   // the queries' operands, of heads g and g + 8
    float qs[HALVES];                                    // what their scores are times
    float o[S::kNT][4], m[HALVES], l[HALVES];            // m, l: of query heads g and g + 8
    int heads = 0;
    uint32_t from = 0;
    auto begin_unit = [&]() {
        heads = heads_of<R>(a, at.unit);
        from = at.tile;
#pragma unroll
        for (int h = 0; h < HALVES; ++h) {
            const uint16_t *q = static_cast<const uint16_t *>(a.q) + row_at<D, R>(a, at.row, at.unit, a.q_stride) +
                                size_t(g + 8 * h < heads ? g + 8 * h : 0) * D;
#pragma unroll
            for (int s = 0; s < S::kSteps; ++s) {
                constexpr int kPer = S::kEK / 4;         // steps of an access
                const uint2 v = *reinterpret_cast<const uint2 *>(q + (s / kPer * 4 + c) * S::kEK + s % kPer * 4);
                qa[s][h][0] = v.x, qa[s][h][1] = v.y;
            }
            qs[h] = a.scale_log2;
            if constexpr (S::kScaled && !QF16) {
                uint32_t top = 0;                        // the largest magnitude's bits
#pragma unroll
                for (int s = 0; s < S::kSteps; ++s)
                    top = __vmaxu2(top, __vmaxu2(qa[s][h][0] & 0x7fff7fffu, qa[s][h][1] & 0x7fff7fffu));
                top = max(top & 0xffffu, top >> 16);
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const uint32_t e = top >> 7, f = e == 255 ? 127 : min(268 - e, 253u);   // (infinities and NaN: as they are)
                const float up = __uint_as_float(f << 23);
#pragma unroll
                for (int s = 0; s < S::kSteps; ++s)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t x = qa[s][h][i];
                        const __half2 y = __floats2half2_rn(__uint_as_float(x << 16) * up,
                                                            __uint_as_float(x & 0xffff0000u) * up);
                        qa[s][h][i] = *reinterpret_cast<const uint32_t *>(&y);
                    }
                qs[h] *= __uint_as_float((254 - f) << 23);
            }
            m[h] = -INFINITY;
            l[h] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < S::kNT; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[j][i] = 0.f;
    };
#pragma unroll
    for (int i = 0; i < N; ++i) there[i] = 0;
    for (int i = 0; i < N - 1; ++i) copy(i);
    if (x0 < x1) begin_unit();

    uint32_t stage = 0;
    for (uint32_t x = x0; x < x1; ++x) {
        copies_wait<N - 2>();
        copy(stage == 0 ? N - 1 : stage - 1);
        const uint8_t *tile = ring + stage * G::kStage;
        const uint32_t got = there[0];
        stage = stage == N - 1 ? 0 : stage + 1;
        const bool more = x + 1 < x1;
        uint32_t ks = 0, vs = 0;                         // scales of the tile's row `lane`
        if constexpr (S::kScaled) {
            fetch<4>(&ks, tile + 2 * G::kKeys + lane * 4);
            fetch<4>(&vs, tile + 2 * G::kKeys + 128 + lane * 4);
        }
        float s[T8][4];
#pragma unroll
        for (int t = 0; t < T8; ++t) {
            uint32_t kr[S::kRowB / 16];
#pragma unroll
            for (int p = 0; p < S::kNK; ++p)
                fetch<S::kKLd>(kr + p * S::kKLd / 4, tile + ((t * S::kNK + p) * 32 + lane) * S::kKLd);
#pragma unroll
            for (int i = 0; i < 4; ++i) s[t][i] = 0.f;
#pragma unroll
            for (int k = 0; k < S::kSteps; ++k) {
                uint32_t b0, b1;
                if constexpr (S::kScaled) {
                    const uint32_t z = KIND == GPT2_INT8 ? kr[k] ^ 0x80808080u : kr[k];
                    b0 = codes_to_half2<KIND == GPT2_E4M3>(z, 0x4140u);
                    b1 = codes_to_half2<KIND == GPT2_E4M3>(z, 0x4342u);
                } else {
                    b0 = kr[2 * k];
                    b1 = kr[2 * k + 1];
                }
                const uint32_t A[4] = {qa[k][0][0], HALVES == 1 ? 0u : qa[k][HALVES - 1][0], qa[k][0][1],
                                       HALVES == 1 ? 0u : qa[k][HALVES - 1][1]};
                mma16816(s[t], A, b0, b1, kBf && !S::kScaled);
            }
        }
        bool above = false;
#pragma unroll
        for (int t = 0; t < T8; ++t)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int key = t * 8 + 2 * c + i;
                const float f = S::kScaled ? __uint_as_float(__shfl_sync(0xffffffffu, ks, key)) : 1.f;
                const bool no = got != kAll && !(got >> key & 1);
#pragma unroll
                for (int h = 0; h < HALVES; ++h) {
                    float y = s[t][i + 2 * h] * (S::kScaled ? qs[h] * f : qs[h]);
                    if (no) y = -INFINITY;
                    s[t][i + 2 * h] = y;
                    above = above || y > m[h] + kRaise;
                }
            }
        // (the maximum is raised only when a score passes it by more than fp16's weights,
        // 2^13 of the largest, or fp32's sums have room for)
        if (__any_sync(0xffffffffu, above)) {
            float keep[HALVES];
#pragma unroll
            for (int h = 0; h < HALVES; ++h) {
                float top = m[h];
#pragma unroll
                for (int t = 0; t < T8; ++t) top = fmaxf(top, fmaxf(s[t][2 * h], s[t][2 * h + 1]));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                keep[h] = exp2_approx(m[h] - (top == -INFINITY ? 0.f : top));
                m[h] = top;
                l[h] *= keep[h];
            }
#pragma unroll
            for (int j = 0; j < S::kNT; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[j][i] *= keep[i / 2 % HALVES];
        }
        uint32_t hi[T8][HALVES], lo[T8][HALVES];         // weights of keys 2c, 2c + 1 of each eight, in two parts
#pragma unroll
        for (int t = 0; t < T8; ++t) {
            float f[2] = {1.f, 1.f};
            if constexpr (S::kScaled)
#pragma unroll
                for (int i = 0; i < 2; ++i) f[i] = __uint_as_float(__shfl_sync(0xffffffffu, vs, t * 8 + 2 * c + i));
#pragma unroll
            for (int h = 0; h < HALVES; ++h) {
                const float base = (m[h] == -INFINITY ? 0.f : m[h]) - (S::kHalf ? kShift : 0.f);
                float p[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    p[i] = exp2_approx(s[t][i + 2 * h] - base);
                    l[h] += p[i];
                    p[i] *= f[i];
                }
                uint32_t part[2];
                split16<S::kHalf ? kF16 : kBf16, 2>(p[0], p[1], part);
                hi[t][h] = part[0], lo[t][h] = part[1];
            }
        }
#pragma unroll
        for (int t = 0; t < T8; t += 2) {
            uint32_t vr[4][S::kRowB / 32];               // rows 2c, 2c + 1, 2c + 8, 2c + 9
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int p = 0; p < S::kNV; ++p)
                    fetch<S::kVLd>(vr[i] + p * S::kVLd / 4,
                                   tile + G::kKeys + (((t * 2 + i) * S::kNV + p) * 32 + lane) * S::kVLd);
#pragma unroll
            for (int j = 0; j < S::kNT; ++j) {
                constexpr int EV = S::kEV;
                const int at4 = j / EV * (S::kVLd / 4), e = j % EV;
                uint32_t b[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t *r0 = vr[2 * h] + at4, *r1 = vr[2 * h + 1] + at4;
                    if constexpr (S::kScaled) {
                        const uint32_t z = __byte_perm(r0[e / 4], r1[e / 4], e % 4 < 2 ? 0x5140u : 0x7362u);   // a0 b0 a1 b1
                        b[h] = e % 2 == 0 ? codes_to_bf162<KIND, 0>(z) : codes_to_bf162<KIND, 1>(z);
                    } else {
                        b[h] = __byte_perm(r0[e / 2], r1[e / 2], e % 2 == 0 ? 0x5410u : 0x7632u);
                    }
                }
                if constexpr (HALVES == 1) {
                    const uint32_t A[4] = {hi[t][0], lo[t][0], hi[t + 1][0], lo[t + 1][0]};
                    mma16816(o[j], A, b[0], b[1], kBf);
                } else {
                    const uint32_t A[4] = {hi[t][0], hi[t][HALVES - 1], hi[t + 1][0], hi[t + 1][HALVES - 1]};
                    const uint32_t B[4] = {lo[t][0], lo[t][HALVES - 1], lo[t + 1][0], lo[t + 1][HALVES - 1]};
                    mma16816(o[j], A, b[0], b[1], kBf);
                    mma16816(o[j], B, b[0], b[1], kBf);
                }
            }
        }

        const bool ends = at.tile + 1 == at.tiles;
        if (ends || !more) {                             // the unit's result, or this warp's part of it
            const bool whole = ends && from == 0;
            const uint32_t part = w * 2 + (from == 0);
#pragma unroll
            for (int h = 0; h < HALVES; ++h) {
                l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
                l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
                const int r = g + 8 * h;
                const float inv = l[h] == 0.f ? 0.f : 1.f / l[h];
                float sane = 0.f;                        // NaN once a result is not finite
                if (r < heads) {
                    const size_t to = row_at<D, R>(a, at.row, at.unit, a.out_stride) + size_t(r) * D;
                    float *sum = a.sums + (size_t(part) * R + r) * D;
#pragma unroll
                    for (int p = 0; p < S::kNV; ++p)
#pragma unroll
                        for (int i = 0; i < 2; ++i)      // dimensions of columns 2c and 2c + 1
#pragma unroll
                            for (int e = 0; e < S::kEV; e += 4) {
                                float v[4];
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    const float *y = o[p * S::kEV + e + k];
                                    v[k] = (HALVES == 1 ? y[i] + y[i + 2] : y[i + 2 * h]) * inv;
                                    sane = fmaf(v[k], 0.f, sane);
                                }
                                const int d = (8 * p + 2 * c + i) * S::kEV + e;
                                if (whole) put4(a, to + d, v[0], v[1], v[2], v[3]);
                                else *reinterpret_cast<float4 *>(sum + d) = make_float4(v[0], v[1], v[2], v[3]);
                            }
                    if (!whole && c == 0) a.ml[size_t(part) * R + r] = make_float2(m[h], l[h]);
                }
                if (whole) {
                    uint32_t odd = __ballot_sync(0xffffffffu, sane != 0.f);
                    while (odd) {
                        const int k = (__ffs(odd) - 1) >> 2;
                        row_anew<KIND, D, R>(a, at.row, at.unit, k + 8 * h, 0, at.len, nullptr);
                        odd &= ~(0xfu << (k * 4));
                    }
                }
            }
            if (!whole && from == 0) {
                head = make_int4(at.row, at.unit, int(sh.all.of(x + at.tiles - 1 - at.tile) - w) + 1, 0);
            }
        }
        if (more) {
            at.next(a);
            if (ends) begin_unit();
        }
    }
    if (lane == 0) a.heads[w] = head;
}

template <int KIND, int D, bool QF16>
cudaError_t mma_launch(const PagedArgs &a, int r, int ctas, cudaStream_t s)
{
    const size_t smem = MmaRing<KIND, D>::kSmem;
    const cudaError_t e = r == 8 ? allow<k_paged_mma<KIND, D, QF16, 1>>(smem) : allow<k_paged_mma<KIND, D, QF16, 2>>(smem);
    if (e != cudaSuccess) return e;
    if (r == 8) return spec_launch(k_paged_mma<KIND, D, QF16, 1>, dim3(ctas), kThreads, smem, 1, s, a);
    return spec_launch(k_paged_mma<KIND, D, QF16, 2>, dim3(ctas), kThreads, smem, 1, s, a);
}

template <int KIND, bool QF16>
cudaError_t mma_dims(const PagedArgs &a, int r, int ctas, cudaStream_t s)
{
    switch (a.kv.head_dim) {
    case 32: return mma_launch<KIND, 32, QF16>(a, r, ctas, s);
    case 64: return mma_launch<KIND, 64, QF16>(a, r, ctas, s);
    default: return mma_launch<KIND, 128, QF16>(a, r, ctas, s);
    }
}

}  // namespace
}  // namespace paged

cudaError_t paged_mma(const PagedArgs &a, int r, int ctas, cudaStream_t s)
{
    const bool f16 = a.q_dtype == GPT2_F16;
    switch (a.kv.dtype) {
    case GPT2_F16: return paged::mma_dims<GPT2_F16, true>(a, r, ctas, s);
    case GPT2_BF16: return paged::mma_dims<GPT2_BF16, false>(a, r, ctas, s);
    case GPT2_INT8: return f16 ? paged::mma_dims<GPT2_INT8, true>(a, r, ctas, s) : paged::mma_dims<GPT2_INT8, false>(a, r, ctas, s);
    default: return f16 ? paged::mma_dims<GPT2_E4M3, true>(a, r, ctas, s) : paged::mma_dims<GPT2_E4M3, false>(a, r, ctas, s);
    }
}

}  // namespace gpt2
