// Attention of a tree of drafted tokens over a cache: the kernel.
//
// For a sequence's nodes i and the cache rows j that node i sees (the cached
// prefix, and the nodes of its mask),
//   s_ij = scale * q_i . k_j,   o_i = sum_j 2^(s'_ij - m_i) v_j / sum_j 2^(s'_ij - m_i),
// s' = s log2(e), m_i the maximum so far, in one pass over the cache rows: a
// new maximum scales what has been summed.
//
// Work split.  The rows of a (sequence, cache head) are its nodes times the
// query heads that share the head; 16 * MT of them are the M side of the
// matrix instructions, so every cache row is read once for all of them.  A
// warp takes tiles of KS cache rows; the kNW warps of a CTA and the CTAs of a
// cluster take different tiles (long caches and few sequences still fill the
// GPU) and join their (m, sum, o) in shared memory, then over the cluster's
// distributed shared memory, in a fixed order: one launch, no workspace, and
// every run gives the same bits.
//
// Cache rows go straight from global memory to registers, in the order the
// matrix instructions want them.  In mma.m16n8k* the thread with g = lane / 4,
// c = lane % 4 supplies B's column g at the k indices of c.  Which head
// dimension (or cache row) a k index stands for is free as long as A agrees,
// so for the scores thread (g, c) loads 16-byte pieces c, c + 4, .. of cache
// row g of eight, and for the weighted sum pieces g, g + 8, .. of the values
// of the rows 2c, 2c + 1, whose weights it holds already.  Every access of a
// warp covers whole lines, nothing is staged or transposed in shared memory,
// and the next tile's keys are loaded while this one's weights are formed.
//
// Types (struct Tr): the fp32 cache uses tf32 products with q, k, p and v as
// two parts each (three products, all but the two second parts'); 16-bit caches
// the products of their own type; 8-bit codes are exact in fp16.  q and the
// weights p are split into kNQ and kNP parts, so that results keep about 22 bits
// for fp32 rows, and for 16-bit rows at least 16 bits of every weight: only the
// final rounding to the row type is visible.
//
// What bounds it: 16 trees of 16 bf16 nodes over 100 to 1,000 int8 positions, 12
// heads of 64: 12.9 us (1.2 TB/s) where the bytes take 2.3: a chain of dependent
// steps (lengths, keys, scores, maxima, weights, sums, the joins of warps and
// cluster) with one to three tiles per warp, of which only the next one's keys are
// on their way (over bf16 13.9 us, 2.0 TB/s); with more sequences or rows the matrix
// instructions and what is done per weight (64 trees of 24 over 50 to 500 bf16
// positions 35.7 us; 8 trees of 64 fp32 rows over 100 to 1,000 positions: bf16 27.5,
// fp32 44.8), and every tile of 32 rows reads the cache again (4 trees of 64 nodes,
// 32 / 8 heads of 128 over 2,000 to 4,000 int8 positions: 118 us where the bytes take
// 4.4).  Tiles of 4 KB, 4 warps and 3 CTAs per SM
// were the best of 2 to 8 KB, 2 to 8 warps and 2 to 4 CTAs.
#pragma once

#include <cooperative_groups.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "spec.h"

namespace gpt2 {

struct TreeArgs {
    gpt2_kv kv;
    const void *q;
    void *out;
    int64_t q_stride, out_stride;
    const int32_t *slot, *cached, *first;
    const uint64_t *mask;
    int32_t n_seqs, n_rows, max_nodes, group, row_tiles, splits, q_dtype;
    float scale_log2;               // scale * log2(e)
};

cudaError_t tree_attn_f32(const TreeArgs &a, int mt, cudaStream_t s);
cudaError_t tree_attn_16(const TreeArgs &a, int mt, cudaStream_t s);
cudaError_t tree_attn_8(const TreeArgs &a, int mt, cudaStream_t s);
// r: query rows of a tile, 1, 2, or 4 over an fp32 cache
cudaError_t tree_attn_few(const TreeArgs &a, int r, cudaStream_t s);
// n: query rows of a tile, 32 or 64
cudaError_t tree_attn_tc(const TreeArgs &a, int n, int sms, void *workspace, cudaStream_t s);
size_t tree_attn_tc_workspace(int head_dim, int n, int sms);

namespace tree {

constexpr int kNW = 4;              // warps of a CTA
constexpr int kMaxSplits = 16;      // CTAs of a cluster
constexpr float kShift = 13.f;      // fp16 weights are 2^(s' - m + 13): small ones stay normal numbers

enum Mma { kTf32, kF16, kBf16 };

template <Mma M, int ES, int NQ, int NP, bool E4M3 = false>
struct Traits {
    static constexpr Mma kMma = M;
    static constexpr int kES = ES;          // bytes of a cache element
    static constexpr int kNQ = NQ, kNP = NP;
    static constexpr bool kE4M3 = E4M3;
    static constexpr bool kScaled = ES == 1;
    static constexpr int kKind = ES == 4 ? GPT2_F32 : ES == 1 ? (E4M3 ? GPT2_E4M3 : GPT2_INT8) : M == kBf16 ? GPT2_BF16 : GPT2_F16;
    static constexpr bool kNorm = M == kF16 && (NQ > 1 || ES == 1);   // q brought into fp16's range by a power of two
};

// Shape of a warp's tile.
template <class Tr, int D, int MT>
struct Tile {
    static constexpr int kRowB = D * Tr::kES;
    static constexpr int kKLd = kRowB / 4 < 16 ? kRowB / 4 : 16;     // bytes per key access of a thread
    static constexpr int kNK = kRowB / (4 * kKLd);                   // key accesses per row
    static constexpr int kVLd = kRowB / 8 < 16 ? kRowB / 8 : 16;     // bytes per value access
    static constexpr int kNV = kRowB / (8 * kVLd);
    static constexpr int kEK = kKLd / Tr::kES, kEV = kVLd / Tr::kES; // elements of an access
    static constexpr int kMost = MT * D >= 256 ? 16 : 32;
    static constexpr int KS = 4096 / kRowB > kMost ? kMost : 4096 / kRowB;   // cache rows per tile: 4 KB of keys, or fewer
    static constexpr int kT8 = KS / 8;                               // score tiles of 8 cache rows
    static constexpr int kSteps = Tr::kMma == kTf32 ? D / 8 : D / 16;   // k steps of the score product
    static constexpr int kKR = kT8 * kRowB / 16;                     // 32-bit registers of the keys
    static constexpr int kVR = kT8 * 2 * kRowB / 32;                 // ... of the values
    static constexpr int kNT = D / 8;                                // output tiles of 8 dimensions
};

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, bool bf)
{
    if (bf)
        asm(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma1688(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm(
        "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// x as a tf32 number (rounded to nearest) and what that leaves, up to 12 bits, of
// which the product takes the first 11.  (An infinity leaves a NaN, and so do
// numbers that round to one: unit_anew.)
__device__ __forceinline__ void split_tf32(uint32_t x, uint32_t &hi, uint32_t &lo)
{
    hi = (x + 0x1000u) & 0xffffe000u;
    lo = __float_as_uint(__uint_as_float(x) - __uint_as_float(hi));
}

__device__ __forceinline__ float exp2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two fp32 values at once (IEEE operations).
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(reinterpret_cast<uint64_t &>(d))
        : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)), "l"(reinterpret_cast<uint64_t &>(c)));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    float2 d;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<uint64_t &>(d))
        : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)));
    return d;
}
// B bytes at p (zeros where !there) into B / 4 registers.
template <int B>
__device__ __forceinline__ void load_piece(uint32_t *r, const uint8_t *p, bool there)
{
    const int t = there;
    if constexpr (B == 16)
        asm volatile(
            "{.reg .pred p;\n\tsetp.ne.s32 p, %5, 0;\n\tmov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\t"
            "mov.b32 %3, 0;\n\t@p ld.global.nc.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];}"
            : "=&r"(r[0]), "=&r"(r[1]), "=&r"(r[2]), "=&r"(r[3])
            : "l"(p), "r"(t));
    else if constexpr (B == 8)
        asm volatile(
            "{.reg .pred p;\n\tsetp.ne.s32 p, %3, 0;\n\tmov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\t"
            "@p ld.global.nc.L1::no_allocate.v2.b32 {%0,%1}, [%2];}"
            : "=&r"(r[0]), "=&r"(r[1])
            : "l"(p), "r"(t));
    else
        asm volatile(
            "{.reg .pred p;\n\tsetp.ne.s32 p, %2, 0;\n\tmov.b32 %0, 0;\n\t"
            "@p ld.global.nc.L1::no_allocate.b32 %0, [%1];}"
            : "=&r"(r[0])
            : "l"(p), "r"(t));
}
__device__ __forceinline__ float load_scale(const float *p, bool there)
{
    float v;
    const int t = there;
    asm volatile("{.reg .pred p;\n\tsetp.ne.s32 p, %2, 0;\n\tmov.f32 %0, 0f00000000;\n\t@p ld.global.nc.f32 %0, [%1];}"
                 : "=&f"(v)
                 : "l"(p), "r"(t));
    return v;
}

// Two codes in the low half of `x` (one per byte) as an fp16 pair.
// int8 (already offset by 128): 0x64uu is 1024 + u, minus 1152 is the code.
template <bool E4M3>
__device__ __forceinline__ uint32_t codes_to_half2(uint32_t x, uint32_t sel)
{
    if constexpr (E4M3) {
        const uint16_t two = uint16_t(sel == 0x4140u ? x & 0xffffu : x >> 16);
        uint32_t r;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(two));
        return r;
    } else {
        uint32_t h = __byte_perm(x, 0x64646464u, sel);
        const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
        __half2 v = __hsub2(*reinterpret_cast<__half2 *>(&h), off);
        return *reinterpret_cast<uint32_t *>(&v);
    }
}

// B operands of the score product, k step s, from a row's registers.
template <class Tr>
__device__ __forceinline__ void key_operand(const uint32_t *r, int s, uint32_t &b0, uint32_t &b1)
{
    if constexpr (Tr::kES == 1) {
        const uint32_t x = Tr::kE4M3 ? r[s] : r[s] ^ 0x80808080u;
        b0 = codes_to_half2<Tr::kE4M3>(x, 0x4140u);
        b1 = codes_to_half2<Tr::kE4M3>(x, 0x4342u);
    } else {
        b0 = r[2 * s];
        b1 = r[2 * s + 1];
    }
}

// B operand of the weighted sum: the values of element j of two rows (registers
// a, b of the rows' accesses) as a 16-bit pair.
template <class Tr>
__device__ __forceinline__ uint32_t value_pair(const uint32_t *a, const uint32_t *b, int j)
{
    if constexpr (Tr::kES == 1) {
        uint32_t x = a[j / 4], y = b[j / 4];
        if (!Tr::kE4M3) {
            x ^= 0x80808080u;
            y ^= 0x80808080u;
        }
        const uint32_t z = __byte_perm(x, y, j % 4 < 2 ? 0x5140u : 0x7362u);   // a0 b0 a1 b1
        return codes_to_half2<Tr::kE4M3>(z, j % 2 == 0 ? 0x4140u : 0x4342u);
    } else {
        return __byte_perm(a[j / 2], b[j / 2], j % 2 == 0 ? 0x5410u : 0x7632u);
    }
}

// x as NP parts of the 16-bit type, each the rounding of what the parts before
// it leave (pairs: x0 in the low half).
template <Mma M, int N>
__device__ __forceinline__ void split16(float x0, float x1, uint32_t (&part)[N])
{
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if constexpr (M == kBf16) {
            __nv_bfloat162 h = __floats2bfloat162_rn(x0, x1);
            part[i] = *reinterpret_cast<uint32_t *>(&h);
            x0 -= __uint_as_float(part[i] << 16);
            x1 -= __uint_as_float(part[i] & 0xffff0000u);
        } else {
            __half2 h = __floats2half2_rn(x0, x1);
            part[i] = *reinterpret_cast<uint32_t *>(&h);
            const float2 f = __half22float2(h);
            x0 -= f.x;
            x1 -= f.y;
        }
    }
}

// Which halves of a 16-bit pair are not finite, as a mask of whole halves.
template <Mma M>
__device__ __forceinline__ uint32_t not_finite(uint32_t x)
{
    constexpr uint32_t e = M == kBf16 ? 0x7f80u : 0x7c00u;
    return ((x & e) == e ? 0xffffu : 0u) | ((x >> 16 & e) == e ? 0xffff0000u : 0u);
}

// Four elements of a query row (aligned to their size) as fp32.
__device__ __forceinline__ float4 load_row4(const void *p, size_t i, int dtype)
{
    if (dtype == GPT2_F32) return *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i);
    const uint2 u = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p) + i);
    if (dtype == GPT2_BF16)
        return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                           __uint_as_float(u.y & 0xffff0000u));
    const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&u.x));
    const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&u.y));
    return make_float4(a.x, a.y, b.x, b.y);
}

template <class Tr, int D, int MT>
struct Smem {
    static constexpr int kRows = 16 * MT;
    static constexpr int kParts = Tr::kMma == kTf32 ? 2 : Tr::kNQ;
    static constexpr size_t kQ = size_t(MT) * Tile<Tr, D, MT>::kSteps * kParts * 32 * 16;
    static constexpr size_t kO = size_t(kNW) * kRows * D * 4;
    static constexpr size_t kBytes = kQ > kO ? kQ : kO;   // q's operands, then the warps' sums
};

// Element i of rows or of a cache (a code without its scale) as fp32.
template <int KIND>
__device__ __forceinline__ float value_at(const void *p, size_t i)
{
    if constexpr (KIND == GPT2_F32) return static_cast<const float *>(p)[i];
    else if constexpr (KIND == GPT2_F16) return __half2float(static_cast<const __half *>(p)[i]);
    else if constexpr (KIND == GPT2_BF16) return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
    else if constexpr (KIND == GPT2_INT8) return float(static_cast<const int8_t *>(p)[i]);
    else {
        const uint32_t h = codes_to_half2<true>(static_cast<const uint8_t *>(p)[i], 0x4140u);
        return __half2float(__ushort_as_half(uint16_t(h)));
    }
}
__device__ __forceinline__ float row_value(const void *p, size_t i, int dtype)
{
    return dtype == GPT2_F32 ? value_at<GPT2_F32>(p, i) : dtype == GPT2_F16 ? value_at<GPT2_F16>(p, i) : value_at<GPT2_BF16>(p, i);
}

__device__ __forceinline__ bool is_finite(float x) { return fabsf(x) <= 3.402823466e38f; }

// A query row's inputs: the cache rows of its head, its place in q, its mask.
struct RowOf {
    gpt2_kv kv;
    const void *q;
    size_t q_at, row_base;
    uint64_t mask;
    int32_t q_dtype, pre, total;
    float scale_log2;
};

// The sum of what is not finite among the values of dimension d that the row sees
// in cache rows from .. to - 1: 0 where all of them are finite.
template <int KIND, int D>
__device__ __noinline__ float seen_not_finite(const RowOf r, int d, int from, int to)
{
    constexpr bool kScaled = KIND == GPT2_INT8 || KIND == GPT2_E4M3;
    float sum = 0.f;
#pragma unroll 8
    for (int j = from; j < to; ++j) {
        const size_t row = r.row_base + j;
        float v = value_at<KIND>(r.kv.v, row * D + d);
        if constexpr (kScaled) v *= r.kv.v_scale[row];
        if (!is_finite(v) && (j < r.pre || (r.mask >> (j - r.pre) & 1))) sum += v;
    }
    return sum;
}

// What becomes of results that are not finite.  The kernels' products of several
// parts make a NaN of a seen infinity (infinity times a second part of zero,
// infinity minus infinity), and so they do of an infinite key whose weight is
// zero.  Where the sum of the weights is sound and there are values that are not
// finite, the result is the sum of those; else the row is computed by its
// definition, below.
//
// Dimensions dim .. dim + N - 1 (each lane its own) of one row's result, by a warp
// in fp32: the maximum and the sum of the weights, a key per lane, then the
// weighted values.  Slow beside the kernels, but a row with a score that is NaN or
// +infinity is NaN as soon as that has been met.
template <int KIND, int D, int N>
__device__ __noinline__ void row_by_definition(const RowOf r, int dim, float (&out)[N])
{
    constexpr bool kScaled = KIND == GPT2_INT8 || KIND == GPT2_E4M3;
    const int lane = threadIdx.x & 31;
    auto sees = [&](int j) { return j < r.pre || (j < r.total && (r.mask >> (j - r.pre) & 1)); };
    auto score = [&](int j) {                        // -infinity where it is not seen
        if (!sees(j)) return -INFINITY;
        const size_t row = r.row_base + j;
        const float s = kScaled ? r.kv.k_scale[row] : 1.f;
        float x = 0.f;
#pragma unroll 4
        for (int d = 0; d < D; d += 4) {
            const float4 q = load_row4(r.q, r.q_at + d, r.q_dtype);
            const float y[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) x = fmaf(y[i] * r.scale_log2, value_at<KIND>(r.kv.k, row * D + d + i) * s, x);
        }
        return x;
    };
    float m = -INFINITY, l = 0.f;
    bool nan = false;
    for (int j0 = 0; j0 < r.total && !nan; j0 += 32) {
        const float s = score(j0 + lane), top = fmaxf(m, s), safe = top == -INFINITY ? 0.f : top;
        nan = __any_sync(0xffffffffu, s != s || s == INFINITY);
        l = l * exp2_approx(m - safe) + exp2_approx(s - safe);
        m = top;
    }
    const float top = warp_max(m);
#pragma unroll
    for (int i = 0; i < N; ++i) out[i] = nan ? __int_as_float(0x7fc00000) : 0.f;
    if (nan || top == -INFINITY) return;
    l = warp_sum(l * exp2_approx(m - top));
    for (int j0 = 0; j0 < r.total; j0 += 32) {
        const float p = exp2_approx(score(j0 + lane) - top) / l;
        const uint32_t seen = __ballot_sync(0xffffffffu, sees(j0 + lane));
#pragma unroll 8
        for (int t = 0; t < 32; ++t) {
            const size_t row = r.row_base + j0 + t;
            const bool yes = seen >> t & 1;
            const float w = __shfl_sync(0xffffffffu, p, t), s = !kScaled ? 1.f : yes ? r.kv.v_scale[row] : 0.f;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float v = yes ? value_at<KIND>(r.kv.v, row * D + dim + i) : 0.f;
                out[i] = fmaf(w, v * s, out[i]);
            }
        }
    }
}

// The query rows and the cache rows of a CTA.
struct Unit {
    size_t row_base;                 // its head's first cache row
    int f0, row0, kvh, rows, pre, total;
    int cut;                         // values from this cache row on were taken out where they are not finite
};

// Element of q and out (of row stride `stride`) where row r begins.
template <int D>
__device__ __forceinline__ size_t begins(const TreeArgs &a, const Unit &u, int r, int64_t stride)
{
    return size_t(u.f0 + (u.row0 + r) / a.group) * stride + size_t(u.kvh * a.group + (u.row0 + r) % a.group) * D;
}

// Four elements of a result row, from element e = row * D + dim on.
template <int D>
__device__ __forceinline__ void store4(const TreeArgs &a, const Unit &u, int e, const float (&v)[4])
{
    const size_t at = begins<D>(a, u, e / D, a.out_stride) + e % D;
    if (a.q_dtype == GPT2_F32) {
        *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + at) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
        uint32_t w[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
            const __nv_bfloat162 x = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = a.q_dtype == GPT2_F16 ? *reinterpret_cast<const uint32_t *>(&h)
                                         : *reinterpret_cast<const uint32_t *>(&x);
        }
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + at) = make_uint2(w[0], w[1]);
    }
}

template <int D>
__device__ __forceinline__ RowOf row_of(const TreeArgs &a, const Unit &u, int r)
{
    return RowOf{a.kv,      a.q,   begins<D>(a, u, r, a.q_stride), u.row_base, a.mask[u.f0 + (u.row0 + r) / a.group],
                 a.q_dtype, u.pre, u.total, a.scale_log2};
}

// Adds what was taken out, and they see, to the four elements from e on.
template <int KIND, int D>
__device__ __noinline__ float4 with_taken_out(const TreeArgs &a, const Unit u, int e, float4 v)
{
    const RowOf of = row_of<D>(a, u, e / D);
    v.x += seen_not_finite<KIND, D>(of, e % D, u.cut, u.total);
    v.y += seen_not_finite<KIND, D>(of, e % D + 1, u.cut, u.total);
    v.z += seen_not_finite<KIND, D>(of, e % D + 2, u.cut, u.total);
    v.w += seen_not_finite<KIND, D>(of, e % D + 3, u.cut, u.total);
    return v;
}

// Results that are not finite, by whole warps, whose elements follow one another:
// first, the warp's first; step between its turns (a multiple of D, so that a
// lane's dimensions stay).  sums [n][R]: the rows' sums of weights, or shares of
// them that add up to a number above zero where the sum is one.
template <int KIND, int D, int R>
__device__ __noinline__ void unit_anew(const TreeArgs &a, const Unit u, const float (*sums)[R], int n, int first, int step)
{
    float prefix[4];                                 // what is not finite in the prefix, in this lane's dimensions
    bool have = false;
    for (int e0 = first; e0 < u.rows * D; e0 += step) {
        const int e = e0 + (threadIdx.x & 31) * 4, d = e % D;
        float v[4] = {0.f, 0.f, 0.f, 0.f};
        if (e < u.rows * D)
            for (int i = 0; i < 4; ++i) v[i] = row_value(a.out, begins<D>(a, u, e / D, a.out_stride) + d + i, a.q_dtype);
        const bool odd = !(is_finite(v[0]) && is_finite(v[1]) && is_finite(v[2]) && is_finite(v[3]));
        for (uint32_t left = __ballot_sync(0xffffffffu, odd); left;) {   // a row at a time
            const int r = __shfl_sync(0xffffffffu, e / D, __ffs(left) - 1);
            const bool mine = odd && e / D == r;
            const RowOf of = row_of<D>(a, u, r);
            float sum = 0.f;
            for (int k = 0; k < n; ++k) sum += sums[k][r];
            bool search = !(sum > 0.f && is_finite(sum));
            float x[4] = {0.f, 0.f, 0.f, 0.f};
            if (!search) {
                for (int i = 0; i < 4; ++i) {
                    if (!have) prefix[i] = seen_not_finite<KIND, D>(of, d + i, 0, u.pre);
                    x[i] = prefix[i] + seen_not_finite<KIND, D>(of, d + i, u.pre, u.total);
                    search = search || (mine && !is_finite(v[i]) && x[i] == 0.f);
                }
                have = true;
            }
            if (__any_sync(0xffffffffu, search)) row_by_definition<KIND, D, 4>(of, d, x);
            if (mine) {
                for (int i = 0; i < 4; ++i)
                    if (!is_finite(v[i])) v[i] = x[i];
                store4<D>(a, u, e, v);
            }
            left &= ~__ballot_sync(0xffffffffu, mine);
        }
    }
}

// The warps' sums so [kNW][R][D] (in units of 2^(the CTA's maximum)), with their
// maxima and sums of weights, to results: over the warps, then over the CTAs of
// the cluster.  cta_bad: values that are not finite were taken out.  What
// is not finite in the end is computed anew (seen_not_finite, row_by_definition).
template <int KIND, int D, int R>
__device__ __forceinline__ void join(const TreeArgs &a, float *so, float (*sm_m)[R], float (*sm_l)[R],
                                     float (*sm_f)[R], int *sm_bad, bool cta_bad, int rank, const Unit u)
{
    const int tid = threadIdx.x, rows = u.rows;
    float cta_m = 0.f, cta_l = 0.f;
    if (tid < R) {
        float top = sm_m[0][tid];
        for (int w = 1; w < kNW; ++w) top = fmaxf(top, sm_m[w][tid]);
        for (int w = 0; w < kNW; ++w)
            cta_l += top == -INFINITY ? 0.f : sm_l[w][tid] * exp2_approx(sm_m[w][tid] - top);
        cta_m = top;
    }
    for (int e = tid * 4; e < rows * D; e += kNW * 32 * 4) {
        float4 v = *reinterpret_cast<const float4 *>(so + e);
#pragma unroll
        for (int w = 1; w < kNW; ++w) {
            const float4 x = *reinterpret_cast<const float4 *>(so + w * R * D + e);
            v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
        }
        *reinterpret_cast<float4 *>(so + e) = v;
    }
    __syncthreads();
    if (tid < R) {
        sm_m[0][tid] = cta_m;
        sm_l[0][tid] = cta_l;
    }
    float sane = 0.f;                                // NaN once a result is not finite
    auto finish4 = [&](int e, bool any_bad, float4 v) {
        if (any_bad) v = with_taken_out<KIND, D>(a, u, e, v);
        const float w[4] = {v.x, v.y, v.z, v.w};
        store4<D>(a, u, e, w);
#pragma unroll
        for (int i = 0; i < 4; ++i) sane = fmaf(w[i], 0.f, sane);
    };
    if (a.splits == 1) {
        __syncthreads();
        for (int e = tid * 4; e < rows * D; e += kNW * 32 * 4) {
            const float sum = sm_l[0][e / D], inv = sum == 0.f ? 0.f : 1.f / sum;
            const float4 o4 = *reinterpret_cast<const float4 *>(so + e);
            finish4(e, cta_bad, make_float4(o4.x * inv, o4.y * inv, o4.z * inv, o4.w * inv));
        }
        if (__any_sync(0xffffffffu, sane != 0.f)) unit_anew<KIND, D, R>(a, u, sm_l, 1, (tid & ~31) * 4, kNW * 32 * 4);
    } else {
        namespace cg = cooperative_groups;
        cg::cluster_group cl = cg::this_cluster();
        cl.sync();
        // every CTA finishes its share of the elements from all CTAs' sums: first
        // each CTA's factor for each row (2^(its m - the largest) / the sum)
        for (int r = tid; r < rows; r += kNW * 32) {
            float mk[kMaxSplits], lk[kMaxSplits], top = -INFINITY, sum = 0.f;
#pragma unroll
            for (int k = 0; k < kMaxSplits; ++k) {
                mk[k] = k < a.splits ? *cl.map_shared_rank(&sm_m[0][r], k) : -INFINITY;
                lk[k] = k < a.splits ? *cl.map_shared_rank(&sm_l[0][r], k) : 0.f;
            }
#pragma unroll
            for (int k = 0; k < kMaxSplits; ++k) top = fmaxf(top, mk[k]);
#pragma unroll
            for (int k = 0; k < kMaxSplits; ++k) {
                mk[k] = mk[k] == -INFINITY ? 0.f : exp2_approx(mk[k] - top);
                sum += lk[k] * mk[k];
            }
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
            for (int k = 0; k < kMaxSplits; ++k) sm_f[k][r] = mk[k] * inv;
        }
        const bool any_bad = __syncthreads_or(tid < a.splits ? *cl.map_shared_rank(sm_bad, tid) : 0);
        for (int e = (rank * kNW * 32 + tid) * 4; e < rows * D; e += a.splits * kNW * 32 * 4) {
            float4 x[kMaxSplits];
            float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < kMaxSplits; ++i)
                x[i] = i < a.splits ? *reinterpret_cast<const float4 *>(cl.map_shared_rank(so + e, i))
                                    : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int i = 0; i < kMaxSplits; ++i) {
                const float f = sm_f[i][e / D];
                v[0] = fmaf(x[i].x, f, v[0]), v[1] = fmaf(x[i].y, f, v[1]);
                v[2] = fmaf(x[i].z, f, v[2]), v[3] = fmaf(x[i].w, f, v[3]);
            }
            finish4(e, any_bad, make_float4(v[0], v[1], v[2], v[3]));
        }
        if (__any_sync(0xffffffffu, sane != 0.f))
            unit_anew<KIND, D, R>(a, u, sm_f, kMaxSplits, (rank * kNW * 32 + (tid & ~31)) * 4, a.splits * kNW * 32 * 4);
        cl.sync();          // nobody leaves while its sums are read
    }
}

template <class Tr, int D, int MT>
__global__ void __launch_bounds__(kNW * 32, MT == 1 && D <= 64 ? 3 : 2) k_tree_attn(const __grid_constant__ TreeArgs a)
{
    using T = Tile<Tr, D, MT>;
    using S = Smem<Tr, D, MT>;
    constexpr int KS = T::KS, R = S::kRows, kQP = S::kParts;
    extern __shared__ __align__(16) uint8_t dyn[];
    __shared__ float sm_m[kNW][R], sm_l[kNW][R];   // [0] then holds the CTA's
    __shared__ float sm_rs[R];                     // score factor of each row
    __shared__ int sm_bad;
    __shared__ float sm_f[kMaxSplits][R];

    const int rank = blockIdx.x % a.splits, unit = blockIdx.x / a.splits;
    const int rt = unit % a.row_tiles, bh = unit / a.row_tiles;
    const int kvh = bh % a.kv.n_head, b = bh / a.kv.n_head;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
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
    const uint8_t *kbase = static_cast<const uint8_t *>(a.kv.k) + row_base * T::kRowB;
    const uint8_t *vbase = static_cast<const uint8_t *>(a.kv.v) + row_base * T::kRowB;
    const float *kscale = Tr::kScaled ? a.kv.k_scale + row_base : nullptr;
    const float *vscale = Tr::kScaled ? a.kv.v_scale + row_base : nullptr;

    // this warp's tiles: t0, t0 + kNW, ... < t1
    const int tiles = (total + KS - 1) / KS, per = (tiles + a.splits - 1) / a.splits;
    const int t0 = rank * per + warp, t1 = min(tiles, (rank + 1) * per);

    uint32_t kr[T::kKR];
    auto load_keys = [&](int t) {
#pragma unroll
        for (int u = 0; u < T::kT8; ++u) {
            const int j = t * KS + u * 8 + g;
            const uint8_t *p = kbase + size_t(j) * T::kRowB + c * T::kKLd;
#pragma unroll
            for (int i = 0; i < T::kNK; ++i)
                load_piece<T::kKLd>(kr + (u * T::kNK + i) * (T::kKLd / 4), p + i * 4 * T::kKLd, j < total);
        }
    };
    // values (and scales) of rows 2c, 2c + 1 of each eight
    uint32_t vr[T::kVR];
    float ks[T::kT8][2], vs[T::kT8][2];
    auto load_values = [&](int t) {
#pragma unroll
        for (int u = 0; u < T::kT8; ++u)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int j = t * KS + u * 8 + 2 * c + e;
                const uint8_t *p = vbase + size_t(j) * T::kRowB + g * T::kVLd;
#pragma unroll
                for (int i = 0; i < T::kNV; ++i)
                    load_piece<T::kVLd>(vr + ((u * 2 + e) * T::kNV + i) * (T::kVLd / 4), p + i * 8 * T::kVLd,
                                        j < total);
                if constexpr (Tr::kScaled) {
                    ks[u][e] = load_scale(kscale + j, j < total);
                    vs[u][e] = load_scale(vscale + j, j < total);
                }
            }
    };
    // what the first tile needs is on its way while q is made ready
    if (t0 < t1) {
        load_keys(t0);
        load_values(t0);
    }
    // masks of this thread's rows (g and g + 8 of each 16)
    uint64_t see[MT][2], all = ~0ull;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int r = mt * 16 + half * 8 + g;
            see[mt][half] = r < rows ? a.mask[f0 + (row0 + r) / G] : ~0ull;
            all &= see[mt][half];
        }

    // ---- q as the A operand, in the order the threads take it ----
    uint32_t *qop = reinterpret_cast<uint32_t *>(dyn);   // [MT][kSteps][kQP][32][4]
    for (int mt = warp; mt < MT; mt += kNW) {
        constexpr int kE = Tr::kMma == kTf32 ? 2 : 4;    // elements of a thread per k step
        float x[2][T::kSteps * kE];
        float top[2] = {0.f, 0.f};
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int r = mt * 16 + half * 8 + g;
            const bool ok = r < rows;
            const int node = (row0 + (ok ? r : 0)) / G, h = kvh * G + (row0 + (ok ? r : 0)) % G;
            const size_t base = size_t(f0 + node) * a.q_stride + size_t(h) * D;
#pragma unroll
            for (int e = 0; e < T::kSteps * kE; e += 4) {
                const int d = (4 * (e / T::kEK) + c) * T::kEK + e % T::kEK;
                const float4 v = ok ? load_row4(a.q, base + d, a.q_dtype) : make_float4(0.f, 0.f, 0.f, 0.f);
                x[half][e] = v.x, x[half][e + 1] = v.y, x[half][e + 2] = v.z, x[half][e + 3] = v.w;
            }
#pragma unroll
            for (int e = 0; e < T::kSteps * kE; ++e) top[half] = fmaxf(top[half], fabsf(x[half][e]));
            float f = 1.f;
            if constexpr (Tr::kNorm) {
                // bring the row's largest value into [2^13, 2^14)
                top[half] = fmaxf(top[half], __shfl_xor_sync(0xffffffffu, top[half], 1));
                top[half] = fmaxf(top[half], __shfl_xor_sync(0xffffffffu, top[half], 2));
                const int ex = int(__float_as_uint(top[half]) >> 23);           // biased exponent
                const int up = min(max(127 + 13 - ex, -100), 100);
                f = __uint_as_float(uint32_t(127 + up) << 23);
#pragma unroll
                for (int e = 0; e < T::kSteps * kE; ++e) x[half][e] *= f;
            }
            if (c == 0) sm_rs[r] = a.scale_log2 / f;     // (f is a power of two)
        }
#pragma unroll
        for (int s = 0; s < T::kSteps; ++s) {
            uint32_t w[kQP][4];
            if constexpr (Tr::kMma == kTf32) {
#pragma unroll
                for (int half = 0; half < 2; ++half)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float v = x[half][2 * s + e];
                        uint32_t hi, lo;
                        split_tf32(__float_as_uint(v), hi, lo);
                        w[0][e * 2 + half] = hi;
                        w[1][e * 2 + half] = lo;
                    }
            } else {
#pragma unroll
                for (int half = 0; half < 2; ++half)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        uint32_t part[kQP];
                        split16<Tr::kMma, kQP>(x[half][4 * s + 2 * e], x[half][4 * s + 2 * e + 1], part);
#pragma unroll
                        for (int i = 0; i < kQP; ++i) w[i][e * 2 + half] = part[i];
                    }
            }
#pragma unroll
            for (int i = 0; i < kQP; ++i)
                reinterpret_cast<uint4 *>(qop)[((mt * T::kSteps + s) * kQP + i) * 32 + lane] =
                    make_uint4(w[i][0], w[i][1], w[i][2], w[i][3]);
        }
    }
    __syncthreads();

    // this thread's rows: factors, softmax state
    float rs[MT][2], m[MT][2], l[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            rs[mt][half] = sm_rs[mt * 16 + half * 8 + g];
            m[mt][half] = -INFINITY;
            l[mt][half] = 0.f;
        }
    // some row does not see some node: a value that is not finite must not
    // reach it through a weight of zero
    const uint64_t present = nodes >= 64 ? ~0ull : (1ull << nodes) - 1;
    const bool partial = __any_sync(0xffffffffu, (all & present) != present);

    float o[MT][T::kNT][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int j = 0; j < T::kNT; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[mt][j][i] = 0.f;
    float gv = 0x1p-126f;            // scaled caches: o counts in units of gv, a power of two >= the value scales so far

    auto visible = [&](int mt, int half, int j) {
        return j < pre || (j < total && (see[mt][half] >> (j - pre) & 1));
    };

    bool bad = false;                // a value that some row does not see is not finite
    for (int t = t0; t < t1; t += kNW) {
        const bool tail = (t + 1) * KS > pre;      // the tile holds nodes, or ends inside
        if (t > t0) load_values(t);
        // scores
        float sc[MT][T::kT8][4], lo[kQP > 1 ? MT : 1][T::kT8][4];   // the first parts' products, the others'
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int u = 0; u < T::kT8; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    sc[mt][u][i] = 0.f;
                    if (kQP > 1) lo[mt][u][i] = 0.f;
                }
#pragma unroll
        for (int s = 0; s < T::kSteps; ++s) {
            uint32_t qa[MT][kQP][4];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int i = 0; i < kQP; ++i) {
                    const uint4 w = reinterpret_cast<const uint4 *>(qop)[((mt * T::kSteps + s) * kQP + i) * 32 + lane];
                    qa[mt][i][0] = w.x, qa[mt][i][1] = w.y, qa[mt][i][2] = w.z, qa[mt][i][3] = w.w;
                }
#pragma unroll
            for (int u = 0; u < T::kT8; ++u) {
                const uint32_t *r = kr + u * T::kNK * (T::kKLd / 4);
                if constexpr (Tr::kMma == kTf32) {
                    uint32_t h0, h1, l0, l1;
                    split_tf32(r[2 * s], h0, l0);
                    split_tf32(r[2 * s + 1], h1, l1);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        mma1688(lo[mt][u], qa[mt][0], l0, l1);
                        mma1688(lo[mt][u], qa[mt][1], h0, h1);
                        mma1688(sc[mt][u], qa[mt][0], h0, h1);
                    }
                } else {
                    uint32_t b0, b1;
                    key_operand<Tr>(r, s, b0, b1);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                        for (int i = kQP - 1; i >= 0; --i)
                            mma16816(i ? lo[mt][u] : sc[mt][u], qa[mt][i], b0, b1, Tr::kMma == kBf16);
                }
            }
        }
        if (t + kNW < t1) load_keys(t + kNW);

#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int u = 0; u < T::kT8; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (kQP > 1) sc[mt][u][i] += lo[mt][u][i];
                    sc[mt][u][i] *= rs[mt][i >> 1];
                    if constexpr (Tr::kScaled) sc[mt][u][i] *= ks[u][i & 1];
                }
        if (tail) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int u = 0; u < T::kT8; ++u)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (!visible(mt, i >> 1, t * KS + u * 8 + 2 * c + (i & 1))) sc[mt][u][i] = -INFINITY;
            if (partial) {
                // a value that is not finite must not meet the weight zero of a
                // row that does not see it: it is taken out here and added at the end
                // (with those of the prefix's last rows, if they are in this tile: to tell
                // them apart here cost 4 % of 8 trees of 16 nodes)
                if constexpr (Tr::kScaled) {
#pragma unroll
                    for (int u = 0; u < T::kT8; ++u)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int j = t * KS + u * 8 + 2 * c + e;
                            if (j >= pre && !is_finite(vs[u][e])) vs[u][e] = 0.f, bad = true;
                        }
                }
#pragma unroll
                for (int i = 0; i < T::kVR; ++i) {
                    const uint32_t x = vr[i];
                    uint32_t gone = 0;
                    if constexpr (Tr::kMma == kTf32) gone = (x & 0x7f800000u) == 0x7f800000u ? ~0u : 0u;
                    else if constexpr (Tr::kES == 2) gone = not_finite<Tr::kMma>(x);
                    else if constexpr (Tr::kE4M3) gone = __vcmpeq4(x & 0x7f7f7f7fu, 0x7f7f7f7fu);
                    vr[i] = x & ~gone;
                    bad = bad || gone != 0;
                }
            }
        }

        // weights, in place of the scores
        float inv_gv = 1.f;
        if constexpr (Tr::kScaled) {
            float top = 0.f;
#pragma unroll
            for (int u = 0; u < T::kT8; ++u) top = fmaxf(top, fmaxf(fabsf(vs[u][0]), fabsf(vs[u][1])));   // (of either sign)
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            if (top > gv) {      // (the same in every thread: rows 2c, 2c + 1 of all c)
                const uint32_t up = min((__float_as_uint(top) + 0x7fffffu) & 0x7f800000u, 253u << 23);
                const float f = gv * __uint_as_float((254u << 23) - up);
                gv = __uint_as_float(up);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int j = 0; j < T::kNT; ++j)
#pragma unroll
                        for (int i = 0; i < 4; ++i) o[mt][j][i] *= f;
            }
            inv_gv = __uint_as_float((254u << 23) - __float_as_uint(gv));
#pragma unroll
            for (int u = 0; u < T::kT8; ++u) vs[u][0] *= inv_gv, vs[u][1] *= inv_gv;
        }
        float keep[MT][2];           // what a new maximum leaves of the sums so far
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                float top = -INFINITY;
#pragma unroll
                for (int u = 0; u < T::kT8; ++u)
                    top = fmaxf(top, fmaxf(sc[mt][u][half * 2], sc[mt][u][half * 2 + 1]));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const float mn = fmaxf(m[mt][half], top), safe = mn == -INFINITY ? 0.f : mn;
                const float ref = safe - (Tr::kMma == kF16 ? kShift : 0.f);
                const float old = exp2_approx(m[mt][half] - safe);
                m[mt][half] = mn;
                float sum = 0.f;
#pragma unroll
                for (int u = 0; u < T::kT8; ++u)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float &x = sc[mt][u][half * 2 + e];
                        x = exp2_approx(x - ref);
                        sum += x;
                        if constexpr (Tr::kScaled) x *= vs[u][e];
                    }
                l[mt][half] = l[mt][half] * old + sum;
                keep[mt][half] = old;
            }

        // weighted sum: the tile's own in fresh accumulators (the matrix units
        // cut each sum off, so the running sums are kept by fp32 additions),
        // the small parts first
        uint32_t pw[MT][Tr::kMma == kTf32 ? T::kT8 : T::kT8 / 2][Tr::kNP][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
            if constexpr (Tr::kMma == kTf32) {
                // a0 (g, row 2c), a1 (g + 8, 2c), a2 (g, 2c + 1), a3 (g + 8, 2c + 1)
#pragma unroll
                for (int u = 0; u < T::kT8; ++u)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        split_tf32(__float_as_uint(sc[mt][u][(i & 1) * 2 + (i >> 1)]), pw[mt][u][0][i], pw[mt][u][1][i]);
            } else {
                // a0 (g, rows 2c, 2c + 1), a1 (g + 8), a2 (g, the next eight's), a3 (g + 8)
#pragma unroll
                for (int u = 0; u < T::kT8; u += 2)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int uu = u + (k >> 1), half = k & 1;
                        uint32_t part[Tr::kNP];
                        split16<Tr::kMma, Tr::kNP>(sc[mt][uu][half * 2], sc[mt][uu][half * 2 + 1], part);
#pragma unroll
                        for (int i = 0; i < Tr::kNP; ++i) pw[mt][u / 2][i][k] = part[i];
                    }
            }
        auto value = [&](int row, int j) {   // registers of a row's access (row: 0 .. 2 kT8 - 1) that holds element j
            return vr + (row * T::kNV + j / T::kEV) * (T::kVLd / 4);
        };
#pragma unroll
        for (int j = 0; j < T::kNT; ++j) {
            float sum[MT][4];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int i = 0; i < 4; ++i) sum[mt][i] = 0.f;
            if constexpr (Tr::kMma == kTf32) {
                uint32_t h[T::kT8][2], l_[T::kT8][2];
#pragma unroll
                for (int u = 0; u < T::kT8; ++u)
#pragma unroll
                    for (int e = 0; e < 2; ++e) split_tf32(value(2 * u + e, j)[j % T::kEV], h[u][e], l_[u][e]);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
                    for (int u = 0; u < T::kT8; ++u) {
                        mma1688(sum[mt], pw[mt][u][0], l_[u][0], l_[u][1]);
                        mma1688(sum[mt], pw[mt][u][1], h[u][0], h[u][1]);
                    }
#pragma unroll
                    for (int u = 0; u < T::kT8; ++u) mma1688(sum[mt], pw[mt][u][0], h[u][0], h[u][1]);
                }
            } else {
                uint32_t b[T::kT8 / 2][2];
#pragma unroll
                for (int u = 0; u < T::kT8 / 2; ++u)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        b[u][e] = value_pair<Tr>(value(4 * u + 2 * e, j), value(4 * u + 2 * e + 1, j), j % T::kEV);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int i = Tr::kNP - 1; i >= 0; --i)
#pragma unroll
                        for (int u = 0; u < T::kT8 / 2; ++u)
                            mma16816(sum[mt], pw[mt][u][i], b[u][0], b[u][1], Tr::kMma == kBf16);
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[mt][j][i] = fmaf(o[mt][j][i], keep[mt][i >> 1], sum[mt][i]);
        }
    }

    // ---- join the warps, then the cluster ----
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            float &x = l[mt][half];
            x += __shfl_xor_sync(0xffffffffu, x, 1);
            x += __shfl_xor_sync(0xffffffffu, x, 2);
            if (c == 0) {
                sm_m[warp][mt * 16 + half * 8 + g] = m[mt][half];
                sm_l[warp][mt * 16 + half * 8 + g] = x;
            }
        }
    const bool cta_bad = __syncthreads_or(bad);   // (also: every warp is done with q's operands)
    if (tid == 0) sm_bad = cta_bad;
    float *so = reinterpret_cast<float *>(dyn);          // [kNW][R][D]
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int r = mt * 16 + half * 8 + g;
            float top = sm_m[0][r];
#pragma unroll
            for (int w = 1; w < kNW; ++w) top = fmaxf(top, sm_m[w][r]);
            const float f = (top == -INFINITY ? 0.f : exp2_approx(m[mt][half] - top)) * (Tr::kScaled ? gv : 1.f);
            float *dst = so + (size_t(warp) * R + r) * D;
            if (r < rows)
#pragma unroll
            for (int j = 0; j < T::kNT; ++j) {
                const int piece = j / T::kEV, w = j % T::kEV;
                dst[(8 * piece + 2 * c) * T::kEV + w] = o[mt][j][half * 2] * f;
                dst[(8 * piece + 2 * c + 1) * T::kEV + w] = o[mt][j][half * 2 + 1] * f;
            }
        }
    __syncthreads();
    join<Tr::kKind, D, R>(a, so, sm_m, sm_l, sm_f, &sm_bad, cta_bad, rank, Unit{row_base, f0, row0, kvh, rows, pre, total, pre - pre % KS});
}

template <typename K>
cudaError_t launch_tree(K fn, const TreeArgs &a, size_t smem, cudaStream_t s)
{
    cudaError_t e = cudaSuccess;
    if (smem > 40 * 1024)
        e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    if (e == cudaSuccess && a.splits > 8) e = cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    return spec_launch(fn, dim3(unsigned(a.n_seqs) * a.kv.n_head * a.row_tiles * a.splits), kNW * 32, smem, a.splits, s, a);
}

template <class Tr, int D, int MT>
cudaError_t launch(const TreeArgs &a, cudaStream_t s)
{
    return launch_tree(k_tree_attn<Tr, D, MT>, a, Smem<Tr, D, MT>::kBytes, s);
}

template <class Tr>
cudaError_t launch_shape(const TreeArgs &a, int mt, cudaStream_t s)
{
    switch (a.kv.head_dim) {
    case 32: return mt == 1 ? launch<Tr, 32, 1>(a, s) : launch<Tr, 32, 2>(a, s);
    case 64: return mt == 1 ? launch<Tr, 64, 1>(a, s) : launch<Tr, 64, 2>(a, s);
    default: return mt == 1 ? launch<Tr, 128, 1>(a, s) : launch<Tr, 128, 2>(a, s);
    }
}

}  // namespace tree
}  // namespace gpt2
