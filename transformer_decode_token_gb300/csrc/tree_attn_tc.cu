// Tree attention over a 16-bit cache on the 5th-generation tensor cores, for
// many rows (drafted nodes times the query heads that share a cache head).
//
// The scores of a tile of 128 cache rows against N = 32 or 64 query rows are
// computed transposed, S^T [128][N] = K_tile . Q^T, and so is the weighted sum,
// O^T [dims][N] += V_tile^T . P: the cache is the A operand in both, so the 128
// rows of an MMA are always full and the query rows cost their own number only
// (N), whatever it is.  V's tile is used as it lies in memory ([row][dim], the
// dimension contiguous: an MN-major A operand).
//   a warp     one lane: TMA loads of K and V tiles (128 rows, 64 dimensions
//              per box, 128-byte swizzle) into two rings
//   one or two tcgen05.mma of the scores (ready a tile ahead) and of the weighted
//   warps      sums (the weights' two parts as 2 N columns of one MMA)
//   the others a thread owns one cache row of the tile (its TMEM lane) and kC
//              of the query rows: p = 2^(s - m), split in two 16-bit parts
//              (hi + lo: 16 bits and more of every weight), written to shared
//              memory as the B operand (MN-major, without swizzle: a thread's
//              8 query rows are one 16-byte store, a warp's stores are
//              contiguous).
// The maxima m are those of the tiles so far (less a lift in fp16, kLift), and are
// only raised when a score exceeds its row's by more than 2^8 in weight (a vote;
// the sums then rescaled in TMEM): weights stay below 2^8 (2^15), and most tiles
// need no reduction over their cache rows at all.
// Work split.  The tiles of all (sequence, cache head, query row tile) units form
// one list; each CTA of a grid that fills the GPU once takes an equal run of it,
// so ragged lengths and odd numbers of units leave no SM idle (with a CTA per
// unit, 384 units on 304 places took two rounds, 1.6 times as long; splitting
// units over clusters left SMs without a place for a whole cluster).  The producer runs ahead into the next
// unit.  A unit that lies within one run is written at once; of one that several
// runs share, each leaves (m, sum, O) in the workspace and k_tree_join adds them
// up in the runs' order, so every call gives the same bits.
//
// What bounds it: 32 f16 trees of 64 nodes over 2,000 to 4,000 positions, 12 heads
// of 64: 87.5 us, 3.5 TB/s, 214 TFLOP/s, where reading the cache takes 45.  An SM's
// share of HBM brings a tile of 128 rows (32 KB) in 1,400 cycles and its MMAs take
// 800, but the softmax of 64 query rows keeps the SM 1,700 (of 16 exponentials and
// two conversions per thread and 16 columns, and the barriers between the
// warps), and every change from one unit to the next costs a CTA some 15,000
// cycles of empty pipeline.  With 32 query rows of 128 dimensions (8 sequences, 4,000
// to 16,000 bf16 positions, 8 heads) the softmax is a quarter of that per byte:
// 62.9 us, 5.2 TB/s.  Not kept: one part of the weights only (the error is 1.4
// times the plain form's), a pair of tiles per step (registers spill: 170 us), 16
// softmax warps in one CTA per SM (127 us).
#include <cuda.h>

#include "tree_attn.cuh"

namespace gpt2 {
namespace {

using tree::add2;
using tree::fma2;

constexpr int kRowsT = 128;                      // cache rows of a tile
constexpr uint32_t kBoxB = kRowsT * 128;         // one TMA box: 128 rows of 64 16-bit dimensions
constexpr float kRaise = 8.f;                    // log2 of the weight, over the maximum's, that raises a maximum
// fp16 weights are 2^(s - m + 7): at most 2^15, and those down to 2^-32 of the
// maximum's are not lost below fp16's smallest number
template <bool BF>
constexpr float kLift = BF ? 0.f : 7.f;
constexpr float kNone = -3.402823466e38f;        // the maximum of a row that has seen nothing: no score is below it

// 64 dimensions: two CTAs per SM, which overlap one another's softmax, products
// and changes of unit (one CTA of 16 softmax warps took 2,400 cycles a tile, two
// of 8 take about 1,700 together); the sums of the weights come from the matrix
// units as well (see kOnes).  128 dimensions: one CTA, a tile's loads are twice
// as long.
template <int D, int N>
struct Shape {
    static constexpr int kPerSM = D == 64 ? 2 : 1;
    static constexpr int kC = D == 64 ? N / 2 : 16;              // query rows of a softmax thread
    static constexpr int kSoft = 4 * N / kC;                     // softmax warps: 128 cache rows x N / kC
    static constexpr int kMmaWarps = D == 64 ? 1 : 2;
    static constexpr int kThreads = (kSoft + 1 + kMmaWarps) * 32;
    static constexpr int kBoxes = D / 64;
    static constexpr uint32_t kTileB = kBoxes * kBoxB;           // K or V of a tile
    static constexpr int kPBufs = D == 128 && N == 32 ? 2 : 1;   // buffers of weights
    static constexpr int kQBufs = D == 64 ? 1 : 2;               // of query rows: the next unit's come early
    // 64 dimensions leave half of the weighted sum's 128 rows free: there V's tile
    // is followed by a block of ones, and those rows are the sums of the weights.
    static constexpr bool kOnes = D == 64;
    // Rings of K and of V tiles.  Two, because a barrier may only be waited on by
    // who has seen its every phase (a wait names a phase by its parity): in one
    // ring of an odd size a place holds K and V in turn, and the warp that runs
    // ahead mistakes the phase before last for its own.
    static constexpr int kKRing = 2, kVRing = N == 64 ? 2 : 3;
    static constexpr int kStages = kKRing + kVRing;
    static_assert(kVRing >= kPBufs, "the softmax warps wait for V too");
    static constexpr uint32_t kPB = kRowsT * N * 2;              // one part of the weights
    static constexpr uint32_t kQB = N * 128 * kBoxes;
    static constexpr uint32_t kOffP = kStages * kTileB, kOffQ = kOffP + kPBufs * 2 * kPB;
    static constexpr uint32_t kOffOnes = kOffQ + kQBufs * kQB;   // 16 rows of 64 ones
    static constexpr uint32_t kBytes = kOffOnes + (kOnes ? 2048 : 0) + 1024;   // + alignment
    static constexpr uint32_t kCols = 4 * N;                     // TMEM: S twice, O of the first parts, of the second
    static_assert(kBytes <= (kPerSM == 2 ? 108 : 220) * 1024, "shared memory of an SM");
};

__device__ __forceinline__ bool wait_phase(uint64_t *bar, uint32_t parity)
{
    return mbar_test_wait(bar, parity & 1u) || mbar_wait_bounded(bar, parity & 1u);
}
__device__ __forceinline__ void arrive(uint64_t *bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void commit(uint64_t *bar, bool leader)
{
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_addr(bar)),
        "r"(uint32_t(leader))
        : "memory");
}
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap *map, int x, int y, uint64_t *bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_addr(bar))
        : "memory");
}
// One MMA by the lane with `leader`; the whole warp takes part, so that the
// operands' addresses are uniform values (computed by one lane alone they cost
// more than the MMA: 120 cycles an instruction).  a, b: low words of the
// descriptors.
__device__ __forceinline__ void mma(uint32_t d, uint32_t a, uint32_t a_hi, uint32_t b, uint32_t b_hi, uint32_t idesc,
                                    bool add, bool leader)
{
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 x, y;\n\tsetp.ne.b32 p, %6, 0;\n\tsetp.ne.b32 q, %7, 0;\n\t"
        "mov.b64 x, {%1, %2};\n\tmov.b64 y, {%3, %4};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %5, p;\n\t}" ::"r"(d),
        "r"(a), "r"(a_hi), "r"(b), "r"(b_hi), "r"(idesc), "r"(uint32_t(add)), "r"(uint32_t(leader))
        : "memory");
}
// Shared-memory matrix descriptor: start, leading and stride byte offsets (in
// 16-byte units), version 1, swizzle (2: 128 bytes, 0: none).
//   K-major, 128-byte swizzle: rows of 128 bytes; stride = 8 rows.
//   MN-major, 128-byte swizzle: a row holds 64 values of the MN index for one k;
//     stride = 8 k, leading = the next 64 values of the MN index.
//   MN-major, no swizzle: 8 values of the MN index (16 bytes) for one k, 8 k
//     contiguous; leading = the next 8 k, stride = the next 8 values.
// Low word: the start and the leading offset; high word: the rest.
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t leading)
{
    return ((addr & 0x3FFFFu) >> 4) | ((leading >> 4) << 16);
}
__host__ __device__ constexpr uint32_t desc_hi(uint32_t stride, uint32_t swizzle)
{
    return (stride >> 4) | (1u << 14) | (swizzle << 29);
}
// D fp32; A and B fp16 (0) or bf16 (1); A, B MN-major (1); N, M = 128.
__host__ __device__ constexpr uint32_t instruction(int n, bool bf, bool mn)
{
    return (1u << 4) | (bf ? (1u << 7) | (1u << 10) : 0u) | (mn ? (1u << 15) | (1u << 16) : 0u) |
           (uint32_t(n >> 3) << 17) | (uint32_t(128 >> 4) << 24);
}

// 16 columns of this thread's lane; the wait is part of the statement, so that
// no use of the values can come before it.
__device__ __forceinline__ void tmem_load16(uint32_t addr, float *v)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];\n\ttcgen05.wait::ld.sync.aligned;"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
          "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
        : "r"(addr)
        : "memory");
}
// The sum of 16 columns of SUMS accumulators N columns apart.
template <int SUMS, int N>
__device__ __forceinline__ void tmem_sum16(uint32_t addr, float *v)
{
    tmem_load16(addr, v);
#pragma unroll
    for (int k = 1; k < SUMS; ++k) {
        float x[16];
        tmem_load16(addr + k * N, x);
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] += x[i];
    }
}
__device__ __forceinline__ void tmem_store16(uint32_t addr, const float (&v)[16])
{
    uint32_t r[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(v[i]);
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_store() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// p as two parts of the 16-bit type, the second the rounding of what the first
// leaves.
template <bool BF>
__device__ __forceinline__ void split_pair(float2 p, uint32_t &hi, uint32_t &lo)
{
    float2 f;
    if constexpr (BF) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(p.x, p.y);
        hi = reinterpret_cast<const uint32_t &>(h);
        f = make_float2(__uint_as_float(hi << 16), __uint_as_float(hi & 0xffff0000u));
    } else {
        const __half2 h = __floats2half2_rn(p.x, p.y);
        hi = reinterpret_cast<const uint32_t &>(h);
        f = __half22float2(h);
    }
    p = fma2(f, make_float2(-1.f, -1.f), p);
    if constexpr (BF) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(p.x, p.y);
        lo = reinterpret_cast<const uint32_t &>(h);
    } else {
        const __half2 h = __floats2half2_rn(p.x, p.y);
        lo = reinterpret_cast<const uint32_t &>(h);
    }
}

// Asynchronous copies into shared memory; bytes past `have` are zero.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, uint32_t have)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(have) : "memory");
}
__device__ __forceinline__ void copy8(uint32_t dst, const void *src, uint32_t have)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(have) : "memory");
}
__device__ __forceinline__ void copies_landed() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Barrier of the softmax warps, alone (1) and with a vote (2).
template <int THREADS>
__device__ __forceinline__ void soft_sync()
{
    asm volatile("barrier.cta.sync 1, %0;" ::"n"(THREADS) : "memory");
}
template <int THREADS>
__device__ __forceinline__ bool soft_any(bool x)
{
    uint32_t y;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, 2, %2, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(y)
        : "r"(uint32_t(x)), "n"(THREADS)
        : "memory");
    return y != 0;
}

// Reduces v[0..C) over the warp's lanes by halving: the result for index
// lane / (32 / C) ends up in that lane (C a power of two, at most 32).
template <int C, typename F>
__device__ __forceinline__ float warp_columns(float (&v)[C], int lane, F f)
{
    int o = 16;
#pragma unroll
    for (int n = C / 2; n > 0; n /= 2, o /= 2) {
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float mine = up ? v[i + n] : v[i], other = up ? v[i] : v[i + n];
            v[i] = f(mine, __shfl_xor_sync(0xffffffffu, other, o));
        }
    }
    for (; o > 0; o /= 2) v[0] = f(v[0], __shfl_xor_sync(0xffffffffu, v[0], o));
    return v[0];
}

// The list of tiles.  Sequence b has units (cache head, query row tile) of
// tiles(b) tiles each: at least one where it has nodes, so that every query
// row is written.
struct Sequence {
    int f0, nodes, rows, pre, total, tiles, units;
    int64_t row_base;                            // the slot's first cache row
    __device__ Sequence(const TreeArgs &a, int b, int n)
    {
        f0 = min(max(a.first[b], 0), a.n_rows);
        const int f1 = min(max(a.first[b + 1], f0), a.n_rows);
        nodes = min(f1 - f0, a.max_nodes);
        rows = nodes * a.group;
        const int slot = a.slot[b], P = a.kv.n_positions;
        const bool there = slot >= 0 && slot < a.kv.n_slots;
        pre = there ? min(max(a.cached[b], 0), P) : 0;
        total = there ? min(pre + nodes, P) : 0;
        tiles = max(1, (total + kRowsT - 1) / kRowsT);
        units = a.kv.n_head * ((rows + n - 1) / n);
        row_base = int64_t(there ? slot : 0) * a.kv.n_head * P;
    }
    __device__ long long count() const { return (long long)units * tiles; }
};

// Sum over the sequences before `end` of their tiles, by a whole CTA.
__device__ __forceinline__ long long tiles_before(const TreeArgs &a, int end, int n, long long *red)
{
    long long x = 0;
    for (int b = threadIdx.x; b < end; b += blockDim.x) x += Sequence(a, b, n).count();
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
    __syncthreads();
    x = 0;
    for (int w = 0; w < int(blockDim.x >> 5); ++w) x += red[w];
    return x;
}

// First tile of run i of `runs` over `all` tiles.  Runs have two tiles or more
// (kLeast), so that few tiles do not leave many parts to add up.
constexpr int kLeast = 2;
__device__ __forceinline__ long long run_begin(long long all, int i, int runs)
{
    const long long n = min((long long)runs, max(1ll, all / kLeast));
    return i >= n ? all : all * i / n;
}

// The units of a run in order: unit u of sequence s from tile t0, n tiles.
struct Walk {
    Sequence s;
    int b, u, t0, n;
    long long left;                              // tiles of the run behind these
    __device__ Walk(const TreeArgs &a, int b_, int u_, int t_, long long run, int rows)
        : s(a, b_, rows), b(b_), u(u_), t0(t_)
    {
        n = int(min((long long)(s.tiles - t0), run));
        left = run - n;
    }
    // false at the end of the run
    __device__ bool next(const TreeArgs &a, int rows)
    {
        if (left <= 0) return false;
        t0 = 0;
        if (++u >= s.units) {
            u = 0;
            do {
                if (++b >= a.n_seqs) return false;
                s = Sequence(a, b, rows);
            } while (s.units == 0);
        }
        n = int(min((long long)s.tiles, left));
        left -= n;
        return true;
    }
};

// Where a run leaves its parts of shared units: two places per run, the first
// for the unit that its first tile belongs to, the second for its last.
struct Head {
    int b, u, t0, n, tiles, bad;                 // n 0: no part
};
template <int D, int N>
struct Part {
    float o[N][D], m[N], l[N];                   // m: minus the maxima (less the lift)
};

// Element of q or `out` where query row r (of a cache head's) begins.
__device__ __forceinline__ int64_t row_at(const TreeArgs &a, const Sequence &s, int64_t stride, int D, int kvh, int r)
{
    return int64_t(s.f0 + r / a.group) * stride + int64_t(kvh * a.group + r % a.group) * D;
}

// What row_by_definition needs of query row r.
__device__ __forceinline__ tree::RowOf row_of(const TreeArgs &a, const Sequence &s, int D, int kvh, int r)
{
    return tree::RowOf{a.kv, a.q, size_t(row_at(a, s, a.q_stride, D, kvh, r)),
                       size_t(s.row_base + int64_t(kvh) * a.kv.n_positions), a.mask[s.f0 + r / a.group], a.q_dtype, s.pre,
                       s.total, a.scale_log2};
}

// This lane's result of a row that has come out not finite in some of the warp's
// dimensions (odd: in this one); sound: the sum of its weights is a number above
// zero.  have, prefix: what is not finite in the prefix, once looked up.
template <int KIND, int D>
__device__ __noinline__ float anew(const tree::RowOf of, int dim, bool odd, bool sound, bool &have, float &prefix)
{
    if (sound) {
        if (!have) prefix = tree::seen_not_finite<KIND, D>(of, dim, 0, of.pre);
        have = true;
        const float x = prefix + tree::seen_not_finite<KIND, D>(of, dim, of.pre, of.total);
        if (!__any_sync(0xffffffffu, odd && x == 0.f)) return x;
    }
    float x[1];
    tree::row_by_definition<KIND, D, 1>(of, dim, x);
    return x[0];
}

template <bool BF, int D, int N>
__global__ void __launch_bounds__(Shape<D, N>::kThreads, Shape<D, N>::kPerSM)
    k_tree_tc(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
              const __grid_constant__ TreeArgs a, Part<D, N> *parts, Head *heads)
{
    using S = Shape<D, N>;
    using T16 = typename std::conditional<BF, __nv_bfloat16, __half>::type;
    constexpr int kKind = BF ? GPT2_BF16 : GPT2_F16;
    constexpr int kSt = S::kStages, kKR = S::kKRing, kVR = S::kVRing, kPB = S::kPBufs, kSoft = S::kSoft, kSync = kSoft * 32, C = S::kC;
    extern __shared__ uint8_t raw[];
    __shared__ __align__(8) uint64_t full[kSt], empty[kSt], sfull[2], sfree[2], pfull[kPB], pfree[kPB], qfull, odone;
    __shared__ uint32_t tmem_slot;
    __shared__ __align__(16) float sm_m[N], sm_alpha[N];   // minus the maxima (log2); what a raise leaves of the sums
    __shared__ float sm_inv[N], sm_part[4][N];
    __shared__ int64_t sm_out[N];
    __shared__ uint64_t sm_mask[2][N];           // the unit's query rows' masks, and the next unit's
    __shared__ uint64_t sm_see[GPT2_MAX_NODES];  // which query rows see a node
    __shared__ long long red[S::kThreads / 32];
    __shared__ int start_b, start_u, start_t;
    __shared__ int sm_bad, sm_fail;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t base = (smem_addr(raw) + 1023u) & ~1023u;
    uint8_t *sm = raw + (base - smem_addr(raw));
    if (warp == kSoft && lane == 0) {
        for (int i = 0; i < kSt; ++i) mbar_init(&full[i], 1), mbar_init(&empty[i], 1);
        for (int i = 0; i < 2; ++i) mbar_init(&sfull[i], 1), mbar_init(&sfree[i], kSoft);
        for (int i = 0; i < kPB; ++i) mbar_init(&pfull[i], kSoft), mbar_init(&pfree[i], 1);
        mbar_init(&qfull, kSoft);
        mbar_init(&odone, S::kMmaWarps);
        mbar_init_fence();
        sm_bad = 0;
        sm_fail = 0;
    }
    if (warp == kSoft + 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&tmem_slot)),
                     "r"(S::kCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if constexpr (S::kOnes) {
        constexpr uint32_t one = BF ? 0x3f803f80u : 0x3c003c00u;
        for (int i = tid; i < 2048 / 16; i += S::kThreads)
            *reinterpret_cast<uint4 *>(sm + S::kOffOnes + i * 16) = make_uint4(one, one, one, one);
        fence_async();
    }
    pdl_wait();
    pdl_launch_dependents();                     // (k_tree_join waits for this kernel's end)
    // this CTA's run of the list
    const long long all = tiles_before(a, a.n_seqs, N, red);
    const long long begin = run_begin(all, blockIdx.x, gridDim.x), end = run_begin(all, blockIdx.x + 1, gridDim.x);
    {
        // the sequence that holds tile `begin`: whole CTA steps, then one warp
        long long before = 0;
        int b0 = 0;
        for (; b0 + int(blockDim.x) < a.n_seqs; b0 += blockDim.x) {   // (more sequences than threads)
            const long long x = tiles_before(a, b0 + blockDim.x, N, red);
            if (x > begin) break;
            before = x;
        }
        if (warp == 0) {
            bool found = begin >= end;
            for (int b1 = b0; b1 < a.n_seqs && !found; b1 += 32) {
                const int b = b1 + lane;
                long long x = 0;
                int tiles = 1;
                if (b < a.n_seqs) {
                    const Sequence s(a, b, N);
                    x = s.count();
                    tiles = s.tiles;
                }
                long long upto = x;
                for (int o = 1; o < 32; o <<= 1) {
                    const long long y = __shfl_up_sync(0xffffffffu, upto, o);
                    if (lane >= o) upto += y;
                }
                const bool mine = before + upto > begin && before + upto - x <= begin;
                if (mine) {
                    const long long off = begin - (before + upto - x);
                    start_b = b, start_u = int(off / tiles), start_t = int(off % tiles);
                }
                found = __any_sync(0xffffffffu, mine);
                before += __shfl_sync(0xffffffffu, upto, 31);
            }
        }
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = tmem_slot, t_o = tmem + 2 * N;
    bool ok = true;
    int g = 0;                                   // tiles of the run so far (ring and buffer phases)
    const bool some = begin < end;
    // (a role walks the run on its own: the producer runs ahead)
    Walk w(a, some ? start_b : 0, some ? start_u : 0, some ? start_t : 0, end - begin, N);

    if (warp == kSoft) {
        if (lane == 0) {
            // tile t's K is at place t % kKR, its V at kKR + t % kVR
            int t = 0;
            auto put = [&](bool v, int64_t row) {
                const int r = v ? kVR : kKR, st = t % r + (v ? kKR : 0);
                if (t >= r) ok = wait_phase(&empty[st], uint32_t(t / r - 1));
                if (!ok) return;
                mbar_arrive_expect_tx(&full[st], S::kTileB);
                for (int x = 0; x < S::kBoxes; ++x)
                    load_box(base + st * S::kTileB + x * kBoxB, v ? &v_map : &k_map, x * 64, int(row), &full[st]);
            };
            bool half = false;                   // tile t's K is on its way, its V is not
            if (some) do {
                const int64_t row = w.s.row_base + int64_t(w.u % a.kv.n_head) * a.kv.n_positions;   // (below 2^31, checked on the host)
                for (int k = 0; k < w.n && ok; ++k) {
                    put(false, row + (w.t0 + k) * kRowsT);
                    half = ok;
                    if (ok) put(true, row + (w.t0 + k) * kRowsT);
                    if (ok) ++t, half = false;
                }
            } while (ok && w.next(a, N));
            if (!ok) {                           // what is in flight lands before the CTA leaves
                sm_fail = 1;
                const int k1 = t + (half ? 1 : 0);
                for (int k = max(0, k1 - kKR); k < k1; ++k) wait_phase(&full[k % kKR], uint32_t(k / kKR));
                for (int k = max(0, t - kVR); k < t; ++k) wait_phase(&full[kKR + k % kVR], uint32_t(k / kVR));
            }
        }
    } else if (warp > kSoft) {
        // A warp issues an MMA in about 85 cycles and tests a barrier in 100 to
        // 200, whatever the MMA's size: with a tile in 1,400 cycles or more, one
        // warp per CTA of two, or one for the scores and one for the weighted sums.
        const bool leader = lane == 0;
        constexpr uint32_t kIS = instruction(N, BF, false), kIO = instruction(2 * N, BF, true);
        constexpr uint32_t kHiK = desc_hi(1024, 2), kHiP = desc_hi(kRowsT * 16, 0);
        auto wait = [&](uint64_t *bar, uint32_t phase) {
            if (ok) ok = __all_sync(0xffffffffu, wait_phase(bar, phase));
        };
        int kst = 0, vst = kKR;                  // ring places of the next K and V, and how often they were used
        uint32_t kuse = 0, vuse = 0, unit = 0;
        auto scores = [&](int g) {
            wait(&full[kst], kuse);
            if (g >= 2) wait(&sfree[g & 1], uint32_t(g / 2 - 1));
            if (!ok) return;
            fence_after();
            const uint32_t k = desc_lo(base + kst * S::kTileB, 16);
            const uint32_t qd = desc_lo(base + S::kOffQ + ((unit - 1) % S::kQBufs) * S::kQB, 16);
#pragma unroll
            for (int s = 0; s < D / 16; ++s)
                mma(tmem + (g & 1) * N, k + (s / 4) * (kBoxB >> 4) + (s % 4) * 2, kHiK,
                    qd + (s / 4) * (N * 128 >> 4) + (s % 4) * 2, kHiK, kIS, s > 0, leader);
            commit(&empty[kst], leader);
            commit(&sfull[g & 1], leader);
            if (++kst == kKR) kst = 0, ++kuse;
        };
        auto weighted = [&](int g, bool first) {   // (the first of a unit starts O anew)
            const int pb = g % kPB;
            wait(&full[vst], vuse);
            wait(&pfull[pb], uint32_t(g / kPB));
            if (!ok) return;
            fence_after();
            const uint32_t at = base + vst * S::kTileB, v = desc_lo(at, S::kOnes ? base + S::kOffOnes - at : kBoxB);
            const uint32_t p = desc_lo(base + S::kOffP + pb * 2 * S::kPB, 128);
            // (the second parts follow the first, as further columns; the block of
            // ones stays where it is: its distance shrinks with every step)
#pragma unroll
            for (int s = 0; s < kRowsT / 16; ++s)
                mma(t_o, v + s * (2048 >> 4) - (S::kOnes ? uint32_t(s * (2048 >> 4)) << 16 : 0u), kHiK,
                    p + s * (256 >> 4), kHiP, kIO, !first || s > 0, leader);
            commit(&empty[vst], leader);
            commit(&pfree[pb], leader);
            if (++vst == kSt) vst = kKR, ++vuse;
        };
        const bool do_scores = S::kMmaWarps == 1 || warp == kSoft + 1;
        if (some) do {
            const int n = __shfl_sync(0xffffffffu, w.n, 0);
            if (do_scores) wait(&qfull, unit);
            ++unit;
            if constexpr (S::kMmaWarps == 1) {
                for (int t = 0; t < n && ok; ++t, ++g) {
                    scores(g);
                    if (t > 0) weighted(g - 1, t == 1);
                }
                weighted(g - 1, n == 1);
            } else {
                for (int t = 0; t < n && ok; ++t, ++g) {
                    if (do_scores) scores(g);
                    else weighted(g, t == 0);
                }
            }
        } while (ok && w.next(a, N));
        if (!ok && leader) sm_fail = 1;
        commit(&odone, leader);
    } else {
        const int q = warp & 3, c0 = (warp >> 2) * C, key = q * 32 + lane;   // TMEM lane, first query row
        const uint32_t lanes = uint32_t(q * 32) << 16;
        const float2 scale = make_float2(a.scale_log2, a.scale_log2);
        // A wait that runs out makes the result NaN; the warp goes on without
        // waiting, since the others meet it at the barriers.
        auto wait = [&](uint64_t *bar, int phase) {
            if (ok) ok = __all_sync(0xffffffffu, wait_phase(bar, uint32_t(phase)));
        };
        // a unit's query rows as the B operand (K-major, 128-byte swizzle; rows
        // past the last are zero) and their masks, on their way
        auto fetch_q = [&](const Walk &w, int buf) {
            const int kvh = w.u % a.kv.n_head, row0 = w.u / a.kv.n_head * N;
            for (int i = tid; i < N * (D / 8); i += kSync) {
                const int r = i / (D / 8), piece = i % (D / 8);
                const bool ok = row0 + r < w.s.rows;
                const int rr = ok ? row0 + r : 0, node = rr / a.group, h = kvh * a.group + rr % a.group;
                copy16(base + S::kOffQ + buf * S::kQB + (piece / 8) * (N * 128) + r * 128 + ((piece % 8) ^ (r & 7)) * 16,
                       static_cast<const T16 *>(a.q) + size_t(w.s.f0 + node) * a.q_stride + size_t(h) * D + piece * 8,
                       ok ? 16 : 0);
            }
            if (tid < N) {
                const bool ok = row0 + tid < w.s.rows;
                copy8(smem_addr(&sm_mask[buf][tid]), a.mask + w.s.f0 + (ok ? (row0 + tid) / a.group : 0), ok ? 8 : 0);
            }
        };
        auto have_q = [&]() {                    // fetched rows are there: the scores may begin
            copies_landed();
            fence_async();
            __syncwarp();
            if (lane == 0) arrive(&qfull);
        };
        if (tid < 2) heads[2 * blockIdx.x + tid].n = 0;
        bool more = some, first_unit = true;
        int buf = 0;
        if (some) {
            fetch_q(w, 0);
            have_q();
        }
        for (; more; buf = (buf + 1) % S::kQBufs) {
            const Sequence sq = w.s;
            const int unit = w.u, t0 = w.t0, n = w.n, w_b = w.b;
            const int kvh = unit % a.kv.n_head, row0 = unit / a.kv.n_head * N, rows = min(sq.rows - row0, N);
            // who sees node j: a lane per query row
            const uint64_t valid = rows >= 64 ? ~0ull : (1ull << rows) - 1;
            bool partial = false;
            soft_sync<kSync>();                  // masks are there; the last unit's maxima and sums are no longer read
            if ((t0 + n) * kRowsT > sq.pre) {
                uint64_t mask[N / 32];
#pragma unroll
                for (int k = 0; k < N / 32; ++k) mask[k] = sm_mask[buf][k * 32 + lane];
                for (int j = warp; j < sq.nodes; j += kSoft) {
                    uint64_t see = 0;
#pragma unroll
                    for (int k = 0; k < N / 32; ++k)
                        see |= uint64_t(__ballot_sync(0xffffffffu, (mask[k] >> j & 1) != 0)) << (32 * k);
                    partial = partial || (see & valid) != valid;   // some query row does not see some node
                    if (lane == 0) sm_see[j] = see;
                }
            }
            if (tid < N) sm_m[tid] = -kNone;
            if (tid == 0) sm_bad = 0;
            partial = soft_any<kSync>(partial);
            float2 l[C / 2];                     // (not where the matrix units sum the weights)
#pragma unroll
            for (int i = 0; i < C / 2; ++i) l[i] = make_float2(0.f, 0.f);

            for (int t = 0; t < n; ++t, ++g) {
                // this thread's cache row, and which of its query rows see it
                const int j = (t0 + t) * kRowsT + key;
                const uint32_t see = j < sq.pre ? ~0u : j < sq.total ? uint32_t(sm_see[j - sq.pre] >> c0) : 0u;
                const bool tail = (t0 + t + 1) * kRowsT > sq.pre;
                const uint32_t t_s = tmem + (g & 1) * N + lanes + c0;
                wait(&sfull[g & 1], g / 2);
                fence_after();
                float d[C];                                            // scores less their rows' maxima, in log2
                auto distances = [&]() {
                    float most = -INFINITY;
#pragma unroll
                    for (int i = 0; i < C; i += 16) tmem_load16(t_s + i, d + i);
#pragma unroll
                    for (int i = 0; i < C; i += 4) {
                        const float4 m = *reinterpret_cast<const float4 *>(&sm_m[c0 + i]);
                        const float2 x = fma2(make_float2(d[i], d[i + 1]), scale, make_float2(m.x, m.y));
                        const float2 y = fma2(make_float2(d[i + 2], d[i + 3]), scale, make_float2(m.z, m.w));
                        d[i] = x.x, d[i + 1] = x.y, d[i + 2] = y.x, d[i + 3] = y.y;
                    }
                    if (see != ~0u) {
#pragma unroll
                        for (int i = 0; i < C; ++i)
                            if (!(see >> i & 1)) d[i] = -INFINITY;
                    }
#pragma unroll
                    for (int i = 0; i < C; ++i) most = fmaxf(most, d[i]);
                    return most;
                };
                if (soft_any<kSync>(distances() > kRaise + kLift<BF>)) {
                    // raise the maxima: this tile's per query row, over the warp's
                    // cache rows and then the warps
#pragma unroll
                    for (int i = 0; i < C; i += 16) tmem_load16(t_s + i, d + i);
#pragma unroll
                    for (int i = 0; i < C; ++i) d[i] = see >> i & 1 ? d[i] * a.scale_log2 : -INFINITY;
                    const float mx = warp_columns(d, lane, [](float x, float y) { return fmaxf(x, y); });
                    if (lane % (32 / C) == 0) sm_part[q][c0 + lane / (32 / C)] = mx;
                    soft_sync<kSync>();
                    if (tid < N) {
                        const float old = -sm_m[tid];
                        float m = old;
                        for (int k = 0; k < 4; ++k) m = fmaxf(m, sm_part[k][tid] - kLift<BF>);
                        sm_m[tid] = -m;
                        sm_alpha[tid] = tree::exp2_approx(old - m);
                    }
                    if (t > 0) wait(&pfree[(g - 1) % kPB], (g - 1) / kPB);   // the sums so far are complete
                    soft_sync<kSync>();
                    fence_after();
#pragma unroll
                    for (int i = 0; i < (S::kOnes ? 0 : C / 2); ++i) l[i].x *= sm_alpha[c0 + 2 * i], l[i].y *= sm_alpha[c0 + 2 * i + 1];
                    if (t > 0) {
#pragma unroll 1
                        for (int i = 0; i < 2 * C; i += 16) {
                            const int col = i % C;
                            const uint32_t at = t_o + (i / C) * N + lanes + c0 + col;
                            float x[16];
                            tmem_load16(at, x);
#pragma unroll
                            for (int e = 0; e < 16; ++e) x[e] *= sm_alpha[c0 + col + e];
                            tmem_store16(at, x);
                        }
                        tmem_wait_store();
                    }
                    distances();
                }
                fence_before();
                __syncwarp();
                if (lane == 0) arrive(&sfree[g & 1]);
                if (g >= kPB) wait(&pfree[g % kPB], g / kPB - 1);
                uint8_t *ph = sm + S::kOffP + (g % kPB) * 2 * S::kPB + key * 16 + c0 / 8 * (kRowsT * 16);
#pragma unroll
                for (int i = 0; i < C; i += 8) {
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float2 p =
                            make_float2(tree::exp2_approx(d[i + 2 * k]), tree::exp2_approx(d[i + 2 * k + 1]));
                        if constexpr (!S::kOnes) l[i / 2 + k] = add2(l[i / 2 + k], p);
                        split_pair<BF>(p, hi[k], lo[k]);
                    }
                    *reinterpret_cast<uint4 *>(ph + i / 8 * (kRowsT * 16)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *reinterpret_cast<uint4 *>(ph + S::kPB + i / 8 * (kRowsT * 16)) =
                        make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
                // rows past the end hold anything, and a value that is not finite must
                // not meet the weight zero of a row that does not see it: taken out
                // here (by the first warps), the latter added at the end
                if (tail && warp < 4 && (partial || (t0 + t + 1) * kRowsT > sq.total)) {
                    const int st = kKR + g % kVR;
                    wait(&full[st], g / kVR);
                    if (j >= sq.total || (partial && j >= sq.pre)) {
                        bool bad = false;
                        for (int y = 0; y < S::kBoxes; ++y) {
                            uint4 *v = reinterpret_cast<uint4 *>(sm + st * S::kTileB + y * kBoxB + key * 128);
                            for (int k = 0; k < 8; ++k) {
                                uint32_t w4[4] = {v[k].x, v[k].y, v[k].z, v[k].w}, gone = 0;
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const uint32_t x16 =
                                        j >= sq.total ? ~0u : tree::not_finite<BF ? tree::kBf16 : tree::kF16>(w4[e]);
                                    gone |= x16;
                                    w4[e] &= ~x16;
                                }
                                if (gone) v[k] = make_uint4(w4[0], w4[1], w4[2], w4[3]);
                                bad = bad || (gone && j < sq.total);
                            }
                        }
                        if (bad) sm_bad = 1;
                    }
                }
                fence_async();
                fence_before();
                __syncwarp();
                if (lane == 0) arrive(&pfull[g % kPB]);
                // the next unit's query rows are fetched during this one, and its
                // scores begin as soon as this one's have been computed
                if (S::kQBufs == 2 && t == 0) {
                    more = w.next(a, N);
                    if (more) fetch_q(w, buf ^ 1);
                } else if (S::kQBufs == 2 && t == 1 && more) {
                    have_q();
                }
            }
            if (S::kQBufs == 1) {                // (every product that reads this unit's is complete)
                more = w.next(a, N);
                if (more) fetch_q(w, 0);
            } else if (n == 1 && more) {
                have_q();
            }

            // ---- the unit's sums: of the weights (over the tile's rows, or from the
            // rows of O that the ones gave), then O from TMEM
            if (!ok) sm_fail = 1;
            if constexpr (S::kOnes) {
                wait(&pfree[(g - 1) % kPB], (g - 1) / kPB);
                fence_after();
                if (q == 2) {
                    float x[C];
#pragma unroll
                    for (int i = 0; i < C; i += 16) tmem_sum16<2, N>(t_o + lanes + c0 + i, x + i);
#pragma unroll
                    for (int i = 0; i < C; ++i)
                        if (lane == i) sm_part[0][c0 + i] = x[i];   // (every lane holds the same)
                }
            } else {
                float sum[C];
#pragma unroll
                for (int i = 0; i < C / 2; ++i) sum[2 * i] = l[i].x, sum[2 * i + 1] = l[i].y;
                const float x = warp_columns(sum, lane, [](float p, float y) { return p + y; });
                if (lane % (32 / C) == 0) sm_part[q][c0 + lane / (32 / C)] = x;
            }
            soft_sync<kSync>();
            const bool whole = n == sq.tiles, bad = sm_bad != 0;
            const int place = 2 * blockIdx.x + (first_unit ? 0 : 1);
            const float nan = __int_as_float(0x7fc00000);
            if (tid < N) {
                float sum = sm_part[0][tid];
                if constexpr (!S::kOnes) sum += sm_part[1][tid] + sm_part[2][tid] + sm_part[3][tid];
                // (what a wait that ran out leaves is NaN; so is, for now, a row without a
                // weight: it sees nothing, or scores of 2^30 and more, whose rounding
                // alone passes the exponent's range)
                sm_inv[tid] = sm_fail || sum == 0.f ? nan : 1.f / sum;
                if (tid < rows) sm_out[tid] = row_at(a, sq, a.out_stride, D, kvh, row0 + tid);
                if (!whole) parts[place].m[tid] = sm_m[tid], parts[place].l[tid] = sm_fail ? nan : sum;
                if (!whole && tid == 0) heads[place] = Head{w_b, unit, t0, n, sq.tiles, bad};
            }
            if constexpr (!S::kOnes) {
                wait(&pfree[(g - 1) % kPB], (g - 1) / kPB);
                fence_after();
            }
            soft_sync<kSync>();
            if (q * 32 < D) {
                const int dim = q * 32 + lane;
                T16 *out = static_cast<T16 *>(a.out) + dim;
                float sane = 0.f;                // NaN once a result is not finite
                // (in a loop: what is run once per unit should be short, its
                // instructions come from memory)
#pragma unroll 1
                for (int i0 = 0; i0 < C; i0 += 16) {
                    float o[16];
                    tmem_sum16<2, N>(t_o + lanes + c0 + i0, o);
                    const int r0 = c0 + i0;
                    if (whole) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const float x = o[i] * sm_inv[r0 + i];
                            sane = fmaf(x, 0.f, sane);
                            if (r0 + i < rows) out[sm_out[r0 + i]] = T16(x);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (r0 + i < rows) parts[place].o[r0 + i][dim] = o[i];
                    }
                }
                // what is not finite, or should not be, is computed anew (what a wait that ran
                // out left stays NaN)
                if (__any_sync(0xffffffffu, sane != 0.f || (bad && whole)) && !sm_fail) {
                    float prefix = 0.f;
                    bool have = false;
                    for (int r = c0; r < min(c0 + C, rows); ++r) {
                        const tree::RowOf of = row_of(a, sq, D, kvh, row0 + r);
                        const float nodes = bad ? tree::seen_not_finite<kKind, D>(of, dim, of.pre, of.total) : 0.f;
                        const bool odd = !tree::is_finite(float(out[sm_out[r]])) || nodes != 0.f;
                        if (!__any_sync(0xffffffffu, odd)) continue;
                        const float x = anew<kKind, D>(of, dim, odd, tree::is_finite(sm_inv[r]), have, prefix);
                        if (odd) out[sm_out[r]] = T16(x);
                    }
                }
                fence_before();
            }
            if (S::kQBufs == 1 && more) have_q();
            first_unit = false;
        }
        if (!ok) sm_fail = 1;
    }
    if ((warp < kSoft || lane == 0) && !wait_phase(&odone, 0)) sm_fail = 1;
    __syncwarp();
    __syncthreads();
    fence_after();
    if (warp == kSoft + 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(S::kCols) : "memory");
}

constexpr int kJoinThreads = 256, kJoinCut = 8, kJoinAhead = 8;

// Computes the results of a joined unit that are not finite anew (those of this
// thread's turns; a warp's elements are 32 dimensions of one row, the same in
// every turn).
template <bool BF, int D, int N>
__device__ __noinline__ void join_anew(const TreeArgs &a, const Part<D, N> *parts, const Head *heads, int first, int last)
{
    using T16 = typename std::conditional<BF, __nv_bfloat16, __half>::type;
    constexpr int kKind = BF ? GPT2_BF16 : GPT2_F16;
    const Head h = heads[first];
    const Sequence s(a, h.b, N);
    const int kvh = h.u % a.kv.n_head, row0 = h.u / a.kv.n_head * N, rows = min(s.rows - row0, N);
    float prefix = 0.f;
    bool have = false;
    static_assert(kJoinCut * kJoinThreads % D == 0, "a lane's dimension stays");
    for (int e = blockIdx.y * kJoinThreads + threadIdx.x; e < rows * D; e += kJoinCut * kJoinThreads) {
        const int r = e / D, d = e % D;
        T16 *out = static_cast<T16 *>(a.out) + row_at(a, s, a.out_stride, D, kvh, row0 + r) + d;
        const bool odd = !tree::is_finite(float(*out));
        if (!__any_sync(0xffffffffu, odd)) continue;
        float sum = parts[first].l[r];               // (only whether it is a number, and not zero)
        for (int i = blockIdx.x + 1; i <= last; ++i) sum += parts[2 * i].l[r];
        const float x = anew<kKind, D>(row_of(a, s, D, kvh, row0 + r), d, odd, tree::is_finite(sum) && sum != 0.f, have, prefix);
        if (odd) *out = T16(x);
    }
}

// Adds up the parts of a unit that several runs share, in the runs' order: a
// row of CTAs for the run that holds the unit's first tile.
template <bool BF, int D, int N>
__global__ void __launch_bounds__(kJoinThreads) k_tree_join(const __grid_constant__ TreeArgs a, const Part<D, N> *parts, const Head *heads)
{
    using T16 = typename std::conditional<BF, __nv_bfloat16, __half>::type;
    const int runs = gridDim.x;
    pdl_wait();                                   // k_tree_tc's parts
    pdl_launch_dependents();
    Head h;
    int first = -1;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const Head x = heads[2 * blockIdx.x + k];
        if (x.n > 0 && x.t0 == 0) h = x, first = 2 * blockIdx.x + k;
    }
    if (first < 0) return;
    // the following runs' first places, up to the unit's last tile
    int last = blockIdx.x, got = h.n;
    bool bad = h.bad != 0;
    while (got < h.tiles && ++last < runs) {
        const Head x = heads[2 * last];
        got += x.n;
        bad = bad || (x.n > 0 && x.bad != 0);
    }
    const Sequence s(a, h.b, N);
    const int kvh = h.u % a.kv.n_head, row0 = h.u / a.kv.n_head * N, rows = min(s.rows - row0, N);
    float sane = 0.f;                             // NaN once a result is not finite
    for (int e = blockIdx.y * kJoinThreads + threadIdx.x; e < rows * D; e += kJoinCut * kJoinThreads) {
        const int r = e / D, d = e % D;
        float m = -parts[first].m[r], sum = parts[first].l[r], v = parts[first].o[r][d];
        // (the runs between hold one unit each, in their first place)
        for (int i0 = blockIdx.x + 1; i0 <= last; i0 += kJoinAhead) {
            float mi[kJoinAhead], li[kJoinAhead], vi[kJoinAhead];
#pragma unroll
            for (int k = 0; k < kJoinAhead; ++k) {
                const Part<D, N> &p = parts[2 * min(i0 + k, last)];
                mi[k] = -p.m[r];
                li[k] = p.l[r];
                vi[k] = p.o[r][d];
            }
#pragma unroll
            for (int k = 0; k < kJoinAhead; ++k)
                if (i0 + k <= last) {
                    const float top = fmaxf(m, mi[k]), f = tree::exp2_approx(m - top), fi = tree::exp2_approx(mi[k] - top);
                    sum = sum * f + li[k] * fi;
                    v = v * f + vi[k] * fi;
                    m = top;
                }
        }
        v = sum == 0.f ? __int_as_float(0x7fc00000) : v / sum;   // (no weight: computed anew)
        if (bad) v += tree::seen_not_finite<(BF ? GPT2_BF16 : GPT2_F16), D>(row_of(a, s, D, kvh, row0 + r), d, s.pre, s.total);
        static_cast<T16 *>(a.out)[row_at(a, s, a.out_stride, D, kvh, row0 + r) + d] = T16(v);
        sane = fmaf(v, 0.f, sane);
    }
    if (__any_sync(0xffffffffu, sane != 0.f)) join_anew<BF, D, N>(a, parts, heads, first, last);
}

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                 const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encoder()
{
    static EncodeTiled fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeTiled>(p);
    }();
    return fn;
}

// The cache as a matrix [slots * heads * positions][head_dim], boxes of 128 rows
// x 64 dimensions, 128-byte swizzle; rows past its end read as zero.
bool cache_map(CUtensorMap *map, const void *p, const gpt2_kv &kv)
{
    const cuuint64_t dims[2] = {cuuint64_t(kv.head_dim),
                                cuuint64_t(kv.n_slots) * cuuint64_t(kv.n_head) * cuuint64_t(kv.n_positions)};
    const cuuint64_t strides[1] = {cuuint64_t(kv.head_dim) * 2};
    const cuuint32_t box[2] = {64, kRowsT}, one[2] = {1, 1};
    return encoder()(map, kv.dtype == GPT2_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
                     const_cast<void *>(p), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool BF, int D, int N>
cudaError_t launch_tc(const TreeArgs &a, int sms, void *workspace, cudaStream_t s)
{
    auto fn = k_tree_tc<BF, D, N>;
    CUtensorMap km, vm;
    if (!encoder() || !cache_map(&km, a.kv.k, a.kv) || !cache_map(&vm, a.kv.v, a.kv)) return cudaErrorUnknown;
    cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, int(Shape<D, N>::kBytes));
    if (e != cudaSuccess) return e;
    const int runs = sms * Shape<D, N>::kPerSM;
    Part<D, N> *parts = static_cast<Part<D, N> *>(workspace);
    Head *heads = reinterpret_cast<Head *>(parts + 2 * runs);
    e = spec_launch(fn, dim3(runs), Shape<D, N>::kThreads, Shape<D, N>::kBytes, 1, s, km, vm, a, parts, heads);
    if (e != cudaSuccess) return e;
    return spec_launch(k_tree_join<BF, D, N>, dim3(runs, kJoinCut), kJoinThreads, 0, 1, s, a, parts, heads);
}

template <int D, int N>
constexpr size_t parts_bytes(int sms)
{
    return size_t(2) * sms * Shape<D, N>::kPerSM * (sizeof(Part<D, N>) + sizeof(Head));
}

}  // namespace

size_t tree_attn_tc_workspace(int head_dim, int n, int sms)
{
    if (n == 32) return head_dim == 64 ? parts_bytes<64, 32>(sms) : parts_bytes<128, 32>(sms);
    return head_dim == 64 ? parts_bytes<64, 64>(sms) : parts_bytes<128, 64>(sms);
}

cudaError_t tree_attn_tc(const TreeArgs &a, int n, int sms, void *ws, cudaStream_t s)
{
    const bool bf = a.kv.dtype == GPT2_BF16, d64 = a.kv.head_dim == 64;
    if (n == 32) {
        if (bf) return d64 ? launch_tc<true, 64, 32>(a, sms, ws, s) : launch_tc<true, 128, 32>(a, sms, ws, s);
        return d64 ? launch_tc<false, 64, 32>(a, sms, ws, s) : launch_tc<false, 128, 32>(a, sms, ws, s);
    }
    if (bf) return d64 ? launch_tc<true, 64, 64>(a, sms, ws, s) : launch_tc<true, 128, 64>(a, sms, ws, s);
    return d64 ? launch_tc<false, 64, 64>(a, sms, ws, s) : launch_tc<false, 128, 64>(a, sms, ws, s);
}

}  // namespace gpt2
