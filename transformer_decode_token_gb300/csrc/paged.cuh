// Attention over a paged cache: what its kernels share.
//
// A unit is one (query row, cache head, tile of up to R of the query heads that
// share the head).  Its cache rows come in tiles of KS; the tiles of all units,
// one unit after another, are one list, and every warp takes an equal share of
// it, whatever the lengths: no warp waits for a longer row, none meets a barrier.
// A unit that lies in one warp's share is written by that warp.  Of a unit that is
// cut, each warp writes its part (maximum, sum of the weights, weighted mean, in
// fp32) to the workspace, and a second kernel joins the parts in the order of the
// list, so every call gives the same bits.  (It costs 2 to 3 us.  Joins by the warp
// that comes last, through tickets, took 10 us more for one request's 63 parts, and
// clusters of 16 CTAs that share out whole units and join behind their barrier 1.4
// us more; joins of a CTA's four warps behind its barrier 1.3 to 3 us more.)
//
// What bounds such kernels is how much of the cache is on its way to an SM at a
// time, so every warp has a ring of tiles in shared memory that asynchronous
// copies fill: each thread copies the pieces that it will read itself, in the order
// of its registers, so that no barrier is needed and no access has a bank conflict.
#pragma once

#include "tree_attn.cuh"

namespace gpt2 {

struct PagedArgs {
    gpt2_kv kv;
    const void *q;
    void *out;
    int64_t q_stride, out_stride;
    const int32_t *table, *seq, *position;
    int4 *heads;                    // workspace: [warps] the unit whose parts begin with this warp's
    float2 *ml;                     // [warps][2][R]
    float *sums;                    // [warps][2][R][D]
    int32_t n_seqs, n_rows, max_blocks, group, row_tiles, q_dtype, warps;
    int32_t per_block;              // 65536 / block size, rounded up (blocks of fewer than 32 rows)
    float scale_log2;               // scale * log2(e)
};

// R: 1, 2 or 4 query heads of a tile, on the CUDA cores
cudaError_t paged_few_f32(const PagedArgs &a, int r, int ctas, cudaStream_t s);
cudaError_t paged_few_16(const PagedArgs &a, int r, int ctas, cudaStream_t s);
cudaError_t paged_few_8(const PagedArgs &a, int r, int ctas, cudaStream_t s);
// R: 8 or 16 query heads of a tile, on the matrix instructions (16-bit rows)
cudaError_t paged_mma(const PagedArgs &a, int r, int ctas, cudaStream_t s);
// the second kernel
cudaError_t paged_join(const PagedArgs &a, int r, cudaStream_t s);

namespace paged {

using namespace tree;

constexpr int kThreads = kNW * 32;
constexpr uint32_t kNone = 0xffffffffu;      // no cache row

// Cache rows that query row i sees, below 2^31 (counts and places of rows and tiles are
// unsigned: rounded up to whole tiles they may pass it).
__device__ __forceinline__ uint32_t seen(const PagedArgs &a, int i)
{
    const long long cap = (long long)a.max_blocks * a.kv.n_positions;
    const long long n = (long long)a.position[i] + 1;
    if (n <= 0) return 0;
    if (a.seq) {
        const int b = a.seq[i];
        if (b < 0 || b >= a.n_seqs) return 0;
    }
    return uint32_t(n < cap ? n : cap);
}
__device__ __forceinline__ const int32_t *table_of(const PagedArgs &a, int i)
{
    return a.table + size_t(a.seq ? a.seq[i] : i) * a.max_blocks;
}

// The cache row of a sequence's row j for head h (kNone where its block is none).
__device__ __forceinline__ uint32_t cache_row(const PagedArgs &a, const int32_t *table, uint32_t j, int h)
{
    const uint32_t bs = uint32_t(a.kv.n_positions), k = j / bs;
    const int32_t block = table[k];
    if (block < 0 || block >= a.kv.n_slots) return kNone;
    return (uint32_t(block) * uint32_t(a.kv.n_head) + uint32_t(h)) * bs + (j - k * bs);
}

// Equal shares of n tiles: share w begins at w * q + min(w, rest).
struct Shares {
    uint32_t q, rest;
    __device__ __forceinline__ Shares(uint32_t n, uint32_t parts) : q(n / parts), rest(n % parts) {}
    __device__ __forceinline__ uint32_t begin(uint32_t w) const { return w * q + min(w, rest); }
    __device__ __forceinline__ uint32_t of(uint32_t x) const      // the share of tile x
    {
        const uint32_t big = rest * (q + 1);
        return x < big ? x / (q + 1) : rest + (x - big) / q;
    }
};

// x / block size for x < block size + 32: a comparison, or, for blocks of fewer than
// 32 rows, a product (65536 / size rounded up is near enough for x < 64).
__device__ __forceinline__ uint32_t blocks_in(const PagedArgs &a, uint32_t x)
{
    const uint32_t bs = uint32_t(a.kv.n_positions);
    return bs >= 32 ? (x >= bs ? 1u : 0u) : x * uint32_t(a.per_block) >> 16;
}

// A place in the list: a tile of a unit.
template <int KS>
struct Place {
    const int32_t *table;           // of the row's sequence
    int row, unit;                  // unit of the row: cache head * row_tiles + tile of query heads
    uint32_t tile, tiles, len;
    uint32_t block, offset;         // where the tile's first key lies: entry of the table, row of the block

    __device__ __forceinline__ void enter(const PagedArgs &a, int i)
    {
        row = i;
        len = seen(a, i);
        tiles = (len + KS - 1) / KS;
        table = len ? table_of(a, i) : nullptr;
    }
    __device__ __forceinline__ void next(const PagedArgs &a)
    {
        if (++tile < tiles) {
            const uint32_t k = blocks_in(a, offset + KS);
            block += k;
            offset += KS - k * uint32_t(a.kv.n_positions);
            return;
        }
        tile = block = offset = 0;
        if (++unit < a.kv.n_head * a.row_tiles) return;
        unit = 0;
        do enter(a, row + 1);
        while (tiles == 0);         // (there is a next tile)
    }
};

// The cache rows of a tile, one per lane.  32 entries of the table, from the tile's
// first block on, are held one per lane until a tile passes them (or another
// row begins), so that most tiles need no load.
struct Lookup {
    int row = -1;
    uint32_t from = 0;
    int32_t entry = -1;
    template <int KS>
    __device__ __forceinline__ uint32_t rows(const PagedArgs &a, const Place<KS> &at, int lane)
    {
        const uint32_t bs = uint32_t(a.kv.n_positions), x = at.offset + lane, k = blocks_in(a, x);
        const uint32_t most = blocks_in(a, at.offset + KS - 1);
        if (row != at.row || at.block < from || at.block + most >= from + 32) {
            row = at.row;
            from = at.block;
            // (the last block that the row sees: its length is above the tile's first key)
            const uint32_t left = at.len - at.tile * KS + at.offset;   // rows from the block's first on
            entry = uint64_t(lane) * bs < left ? at.table[from + lane] : -1;
        }
        const int32_t e = __shfl_sync(0xffffffffu, entry, (at.block - from + k) & 31);
        const bool yes = lane < KS && at.tile * KS + lane < at.len && e >= 0 && e < a.kv.n_slots;
        return yes ? (uint32_t(e) * uint32_t(a.kv.n_head) + uint32_t(at.unit / a.row_tiles)) * bs + (x - k * bs) : kNone;
    }
};

// B bytes from global to shared memory, asynchronously (zeros where !there).  Through
// L1: past it (.cg) the same kernel fetched every sector from L2 twice (64 requests of
// 2,000 to 4,000 fp32 rows, 12 heads of 64: 215 us instead of 178).
template <int B>
__device__ __forceinline__ void copy_async(uint32_t dst, const void *src, bool there)
{
    const int n = there ? B : 0;
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(B), "r"(n) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait()       // until at most the last N groups are on their way
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// B bytes of shared memory into registers.
template <int B>
__device__ __forceinline__ void fetch(uint32_t *r, const uint8_t *p)
{
    if constexpr (B == 16) {
        const uint4 v = *reinterpret_cast<const uint4 *>(p);
        r[0] = v.x, r[1] = v.y, r[2] = v.z, r[3] = v.w;
    } else if constexpr (B == 8) {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        r[0] = v.x, r[1] = v.y;
    } else {
        r[0] = *reinterpret_cast<const uint32_t *>(p);
    }
}

// The shape of the rings, for r query heads of a tile, cache elements of `size` bytes
// and rows of `row` bytes.  The copies pass through L1, which takes what shared memory
// leaves: a ring that is too large costs more than its depth gives.  Measured, us:
//   8-bit codes, whose conversion takes the most instructions per byte: 4 CTAs of an SM
//     with 2 stages of 4 KB 52.7, 4 stages with 3 CTAs 67.7, 3 with 4 66 (32 requests of
//     3,000 to 8,000 int8 rows of 64); rows of 128: 64.7, stages of 8 KB with 3 CTAs 83
//   16-bit and fp32 rows: 3 CTAs with 2 stages of 8 KB 92, with 4 of 4 KB 94.5, 2 CTAs 101
//     (64 requests of 2,000 to 4,000 bf16 rows of 64); 4 CTAs with 3 of 4 KB 116
//   the matrix instructions, 128 dimensions: 2 CTAs with 3 stages 54, with 2 55, 3 with 2
//     58 (bf16); over int8 2 stages 35, 3 41
constexpr int tile_rows(int r, int size, int row)        // cache rows of a tile, at most 32
{
    const int n = (r == 1 && size == 1 ? 2048 : 4096) / row;
    return n > 32 ? 32 : n;
}
constexpr int ring_ctas(int r, int size, int row)        // CTAs of an SM
{
    return r >= 8 ? (row / size == 128 ? 2 : 3) : r == 1 && size == 1 ? 4 : r <= 2 ? 3 : 2;
}
constexpr int ring_stages(int r, int size, int row)
{
    if (size == 1) return 2;
    const int n = (ring_ctas(r, size, row) == 2 ? 24 : 16) * 1024 / (2 * tile_rows(r, size, row) * row);
    return n > 6 ? 6 : n;
}

// Lets a kernel use so much dynamic shared memory (once per device and kernel).
template <auto FN>
cudaError_t allow(size_t bytes)
{
    static uint64_t done = 0;       // a bit per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (__atomic_load_n(&done, __ATOMIC_RELAXED) >> (dev & 63) & 1)) return e;
    e = cudaFuncSetAttribute(FN, cudaFuncAttributeMaxDynamicSharedMemorySize, int(bytes));
    if (e == cudaSuccess) __atomic_fetch_or(&done, 1ull << (dev & 63), __ATOMIC_RELAXED);
    return e;
}

// A warp's tiles x0 .. x1 - 1 of the list, and the place where they begin.
template <int KS>
struct Share {
    Shares all;
    uint32_t w, x0, x1;
    Place<KS> at;
    __device__ __forceinline__ Share() : all(1, 1), w(0), x0(0), x1(0) {}
};

// This warp's share.  Called by all threads of the CTA; also writes the zeros of
// rows that see nothing.
template <int KS, int D>
__device__ __forceinline__ void find_share(const PagedArgs &a, Share<KS> &sh)
{
    __shared__ uint32_t sums[kNW], base[kNW];
    __shared__ int rows[kNW];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int per = (a.n_rows + kThreads - 1) / kThreads, r0 = min(tid * per, a.n_rows), r1 = min(r0 + per, a.n_rows);
    uint32_t mine = 0;
    for (int r = r0; r < r1; ++r) mine += (seen(a, r) + KS - 1) / KS;
    uint32_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    uint32_t total = 0;
#pragma unroll
    for (int i = 0; i < kNW; ++i) {
        if (i < warp) incl += sums[i];
        total += sums[i];
    }
    const uint32_t units = uint32_t(a.kv.n_head) * a.row_tiles;
    const uint32_t n = total * units, parts = max(1u, min(uint32_t(a.warps), n));
    sh.all = Shares(n, parts);
    sh.w = warp * gridDim.x + blockIdx.x;        // (so that fewer shares than warps spread over the SMs)
#pragma unroll
    for (int i = 0; i < kNW; ++i) {              // the rows where this CTA's warps begin, and the tiles before them
        const uint32_t wi = i * gridDim.x + blockIdx.x;
        if (wi >= parts || n == 0) continue;
        const uint32_t y = sh.all.begin(wi) / units;
        if (y < incl - mine || y >= incl) continue;
        uint32_t t = incl - mine;
        int r = r0;
        for (;; ++r) {
            const uint32_t k = (seen(a, r) + KS - 1) / KS;
            if (y < t + k) break;
            t += k;
        }
        rows[i] = r;
        base[i] = t * units;
    }
    for (int r = blockIdx.x; r < a.n_rows; r += gridDim.x) {
        if (seen(a, r) != 0) continue;
        const int cols = a.kv.n_head * a.group * D;
        for (int e = tid * 4; e < cols; e += kThreads * 4) {
            const size_t o = size_t(r) * a.out_stride + e;
            if (a.q_dtype == GPT2_F32) *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + o) = make_float4(0.f, 0.f, 0.f, 0.f);
            else *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + o) = make_uint2(0u, 0u);
        }
    }
    __syncthreads();
    if (sh.w >= parts || n == 0) return;         // (x0 == x1)
    sh.x0 = sh.all.begin(sh.w);
    sh.x1 = sh.all.begin(sh.w + 1);
    Place<KS> &at = sh.at;
    at.enter(a, rows[warp]);
    const uint32_t off = sh.x0 - base[warp];
    at.unit = int(off / at.tiles);
    at.tile = off % at.tiles;
    at.block = at.tile * KS / uint32_t(a.kv.n_positions);
    at.offset = at.tile * KS - at.block * uint32_t(a.kv.n_positions);
}

// Query heads of a unit, and where its first one's row of q (or out) begins.
template <int R>
__device__ __forceinline__ int heads_of(const PagedArgs &a, int unit)
{
    return min(R, a.group - unit % a.row_tiles * R);
}
template <int D, int R>
__device__ __forceinline__ size_t row_at(const PagedArgs &a, int row, int unit, int64_t stride)
{
    return size_t(row) * stride + size_t(unit / a.row_tiles * a.group + unit % a.row_tiles * R) * D;
}

// Four elements of a result.
__device__ __forceinline__ void put4(const PagedArgs &a, size_t at, float x, float y, float z, float w)
{
    if (a.q_dtype == GPT2_F32) {
        *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + at) = make_float4(x, y, z, w);
    } else {
        uint2 v;
        if (a.q_dtype == GPT2_F16) {
            const __half2 p = __floats2half2_rn(x, y), r = __floats2half2_rn(z, w);
            v = make_uint2(*reinterpret_cast<const uint32_t *>(&p), *reinterpret_cast<const uint32_t *>(&r));
        } else {
            const __nv_bfloat162 p = __floats2bfloat162_rn(x, y), r = __floats2bfloat162_rn(z, w);
            v = make_uint2(*reinterpret_cast<const uint32_t *>(&p), *reinterpret_cast<const uint32_t *>(&r));
        }
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + at) = v;
    }
}

// N elements of a result, v times f.
template <int N>
__device__ __forceinline__ void put(const PagedArgs &a, size_t at, const float *v, float f)
{
    if constexpr (N >= 4) {
#pragma unroll
        for (int i = 0; i < N; i += 4) put4(a, at + i, v[i] * f, v[i + 1] * f, v[i + 2] * f, v[i + 3] * f);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float x = v[i] * f;
            if (a.q_dtype == GPT2_F32) static_cast<float *>(a.out)[at + i] = x;
            else if (a.q_dtype == GPT2_F16) static_cast<__half *>(a.out)[at + i] = __float2half_rn(x);
            else static_cast<__nv_bfloat16 *>(a.out)[at + i] = __float2bfloat16_rn(x);
        }
    }
}

// One result row (query head h of the unit's tile), or a part of it (keys j_from .. j_to - 1,
// to `part`), by its definition, by a warp in fp32: the maximum and the sum of the
// weights, a key per lane, then the weighted values, D / 32 dimensions per lane.  For
// what is not finite: the kernels sum values times weights of up to 2^8 and divide in
// the end (and the matrix instructions' products in parts make a NaN of an infinity), so
// that large values can pass fp32's range where those of the formula, whose weights
// add up to one, do not.
template <int KIND, int D, int R>
__device__ __noinline__ void row_anew(const PagedArgs &a, int row, int unit, int h, uint32_t j_from, uint32_t j_to,
                                      float *part)
{
    constexpr bool kScaled = KIND == GPT2_INT8 || KIND == GPT2_E4M3;
    constexpr int N = D / 32;
    const int lane = threadIdx.x & 31, head = unit / a.row_tiles;
    const int32_t *table = table_of(a, row);
    const size_t q_at = row_at<D, R>(a, row, unit, a.q_stride) + size_t(h) * D;
    auto score = [&](uint32_t j, uint32_t r) {       // -infinity where it is not seen
        if (r == kNone) return -INFINITY;
        const float s = kScaled ? a.kv.k_scale[r] : 1.f;
        float x = 0.f;
#pragma unroll 4
        for (int d = 0; d < D; d += 4) {
            const float4 q = load_row4(a.q, q_at + d, a.q_dtype);
            const float y[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) x = fmaf(y[i] * a.scale_log2, value_at<KIND>(a.kv.k, size_t(r) * D + d + i) * s, x);
        }
        return x;
    };
    auto at = [&](uint32_t j) { return j < j_to ? cache_row(a, table, j, head) : kNone; };
    float m = -INFINITY, l = 0.f, out[N];
    bool nan = false;
    for (uint32_t j0 = j_from; j0 < j_to && !nan; j0 += 32) {
        const float s = score(j0 + lane, at(j0 + lane)), top = fmaxf(m, s), safe = top == -INFINITY ? 0.f : top;
        nan = __any_sync(0xffffffffu, s != s || s == INFINITY);
        l = l * exp2_approx(m - safe) + exp2_approx(s - safe);
        m = top;
    }
    const float top = warp_max(m);
#pragma unroll
    for (int i = 0; i < N; ++i) out[i] = nan ? __int_as_float(0x7fc00000) : 0.f;
    if (!nan && top != -INFINITY) {
        l = warp_sum(l * exp2_approx(m - top));
        for (uint32_t j0 = j_from; j0 < j_to; j0 += 32) {
            const uint32_t r = at(j0 + lane);
            const float p = exp2_approx(score(j0 + lane, r) - top) / l;
            for (int t = 0; t < 32; ++t) {
                const uint32_t rt = __shfl_sync(0xffffffffu, r, t);
                const float w = __shfl_sync(0xffffffffu, p, t);
                if (rt == kNone) continue;
                const float s = kScaled ? a.kv.v_scale[rt] : 1.f;
#pragma unroll
                for (int i = 0; i < N; ++i) out[i] = fmaf(w, value_at<KIND>(a.kv.v, size_t(rt) * D + lane * N + i) * s, out[i]);
            }
        }
    }
    const size_t o = row_at<D, R>(a, row, unit, a.out_stride) + size_t(h) * D + lane * N;
    __syncwarp();                                        // (what other lanes have written there comes first)
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (part) part[lane * N + i] = out[i];
        else if (a.q_dtype == GPT2_F32) static_cast<float *>(a.out)[o + i] = out[i];
        else if (a.q_dtype == GPT2_F16) static_cast<__half *>(a.out)[o + i] = __float2half_rn(out[i]);
        else static_cast<__nv_bfloat16 *>(a.out)[o + i] = __float2bfloat16_rn(out[i]);
    }
}

// What a warp has written of its share and is not finite, computed anew: its share w goes
// from tile `tile` of the unit (row, unit) to tile last_tile of (last_row, last_unit).
template <int KIND, int D, int R, int KS>
__device__ __noinline__ void share_anew(const PagedArgs &a, uint32_t w, int row, int unit, uint32_t tile, int last_row,
                                        int last_unit, uint32_t last_tile)
{
    const int lane = threadIdx.x & 31, units = a.kv.n_head * a.row_tiles;
    for (; row <= last_row; ++row, unit = 0) {
        const uint32_t len = seen(a, row), tiles = (len + KS - 1) / KS;
        if (len == 0) continue;
        for (const int end = row == last_row ? last_unit + 1 : units; unit < end; ++unit, tile = 0) {
            const bool last = row == last_row && unit == last_unit;
            const bool whole = tile == 0 && (!last || last_tile + 1 == tiles);
            const uint32_t to = last && last_tile + 1 < tiles ? (last_tile + 1) * KS : len;
            for (int r = 0; r < heads_of<R>(a, unit); ++r) {
                float *part = a.sums + ((size_t(w) * 2 + (tile == 0)) * R + r) * D;
                const size_t at = row_at<D, R>(a, row, unit, a.out_stride) + size_t(r) * D + lane;
                bool odd = false;
#pragma unroll
                for (int i = 0; i < D; i += 32)
                    odd = odd || !is_finite(whole ? row_value(a.out, at + i, a.q_dtype) : part[lane + i]);
                if (__any_sync(0xffffffffu, odd)) row_anew<KIND, D, R>(a, row, unit, r, tile * KS, to, whole ? nullptr : part);
            }
        }
    }
}

// Part i of a unit whose parts begin with warp w: the end of that one's share, then
// the beginnings of the others'.
__device__ __forceinline__ size_t part_of(uint32_t w, uint32_t i) { return i == 0 ? size_t(w) * 2 + 1 : size_t(w + i) * 2; }

// Joins the n parts (from warp w on) of query head r of a unit, by a warp: their means,
// each times its share of the weights, so that nothing grows past the largest mean.
// KIND: the cache's type where the parts come from the matrix instructions, whose results
// that are not finite are computed anew here; -1 where that has been done for the parts.
template <int KIND, int D, int R>
__device__ __forceinline__ void join_row(const PagedArgs &a, int row, int unit, uint32_t w, uint32_t n, int r)
{
    constexpr int kLanes = D / 4, kSide = 32 / kLanes, kBatch = 16;   // lanes of a part, parts side by side
    const int lane = threadIdx.x & 31, e = lane % kLanes * 4, side = lane / kLanes;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    float top = -INFINITY, l = 0.f;
    for (uint32_t i0 = 0; i0 < n; i0 += 32) {        // 32 parts' (m, l), one per lane, and their sums
        float2 ml = make_float2(-INFINITY, 0.f);
        if (i0 + lane < n) ml = __ldcg(a.ml + part_of(w, i0 + lane) * R + r);
        const uint32_t here = min(32u, n - i0);
        float4 x[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const uint32_t i = k * kSide + side;
            x[k] = i < here ? __ldcg(reinterpret_cast<const float4 *>(a.sums + (part_of(w, i0 + i) * R + r) * D + e))
                            : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        const float mn = fmaxf(top, warp_max(ml.x)), safe = mn == -INFINITY ? 0.f : mn;
        float keep = exp2_approx(top - safe), f = ml.y * exp2_approx(ml.x - safe);
        top = mn;
        keep *= l;
        l = keep + warp_sum(f);
        const float inv = l == 0.f ? 0.f : 1.f / l;
        keep *= inv, f *= inv;
        v.x *= keep, v.y *= keep, v.z *= keep, v.w *= keep;
        for (uint32_t j = 0; j < here; j += kBatch * kSide) {
            if (j)
#pragma unroll
                for (int k = 0; k < kBatch; ++k) {
                    const uint32_t i = j + k * kSide + side;
                    x[k] = i < here ? __ldcg(reinterpret_cast<const float4 *>(a.sums + (part_of(w, i0 + i) * R + r) * D + e))
                                    : make_float4(0.f, 0.f, 0.f, 0.f);
                }
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const uint32_t i = j + k * kSide + side;
                const float g = __shfl_sync(0xffffffffu, f, i & 31);
                if (i >= here) continue;
                v.x = fmaf(x[k].x, g, v.x), v.y = fmaf(x[k].y, g, v.y), v.z = fmaf(x[k].z, g, v.z), v.w = fmaf(x[k].w, g, v.w);
            }
        }
    }
#pragma unroll
    for (int d = kLanes; d < 32; d *= 2) {
        v.x += __shfl_xor_sync(0xffffffffu, v.x, d), v.y += __shfl_xor_sync(0xffffffffu, v.y, d);
        v.z += __shfl_xor_sync(0xffffffffu, v.z, d), v.w += __shfl_xor_sync(0xffffffffu, v.w, d);
    }
    if (side == 0) put4(a, row_at<D, R>(a, row, unit, a.out_stride) + size_t(r) * D + e, v.x, v.y, v.z, v.w);
    if constexpr (KIND >= 0)
        if (__any_sync(0xffffffffu, !(is_finite(v.x) && is_finite(v.y) && is_finite(v.z) && is_finite(v.w))))
            row_anew<KIND, D, R>(a, row, unit, r, 0, seen(a, row), nullptr);
}

}  // namespace paged
}  // namespace gpt2
