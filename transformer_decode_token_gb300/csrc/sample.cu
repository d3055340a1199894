// gpt2_op_sample: the next token of each row of logits, by temperature, top-k,
// top-p and min-p, from given random numbers.
//
// A row belongs to a cluster of CTAs, each with a share of it in shared memory in
// the row's own type, so that the logits are read once.  With w = exp((l - max) /
// T) and the ids ordered by logit (highest first, ties to the lowest id), every
// cut keeps a beginning of that order, so all that is needed is where the kept
// ids end.
//   - Nothing cut: one pass, the race argmax w / -log u and the sum of w; one
//     exchange in the cluster.
//   - Else the cluster first bounds what can be kept: the top_k highest lie above
//     the k-th highest of its threads' own maxima (to a bin), and with top-p alone
//     every id whose weight is at most (1 - top_p) z / V, z the sum of all, lies
//     behind the cut.  What is left, usually dozens to a few hundred ids, goes to a list.
//   - A list of up to kList ids is settled by one CTA: sorted, the masses before
//     each id from a prefix sum, the race over what is kept.
//   - A longer one is narrowed by histograms over the cluster, of counts and
//     masses, by digits of (weight, logit, id), until the digit where the cut
//     lies holds at most kList ids, which are then sorted as above.
// Masses are summed as integers (in units of 2^-40 of the largest weight; a few weights
// of one thread at a time in fp32), so that the order in which CTAs and threads come does
// not show and every call gives the same bits.
//
// What bounds it is latency: the load of a share, two or three exchanges over the
// cluster, and barriers around the list, its order and the race, most of them the same
// for one row (8.8 us with top-p) as for 64 (12.8 with top-k and top-p, 11.5 uncut; the
// logits alone would take 1.9, with the random numbers 3.8).  A flat row, whose cut lies
// among thousands of ids, takes 56 us: two passes of two shared-memory atomics per id,
// two of lists, and the race.
//
// Rounding: a weight is off by some 2^-22 of itself (the exponent's integer part is
// taken off exactly before the exponential), those of a row's or a long list's sum, whose
// exponents are rounded as a whole, by up to 1e-6 of the sum together, and up to eight of a
// thread are added in fp32.  So a cut by mass can differ from the exact one where it
// falls within 2e-6 of its border (usually 1e-7), and a race where its two best are
// within 1e-6 of each other; probabilities are off by at most 4e-6 (lists of up to 512
// ids: 6e-7).
#include <cooperative_groups.h>

#include <cfloat>
#include <cmath>

#include "common.cuh"
#include "spec.h"

namespace gpt2 {
namespace {

namespace cg = cooperative_groups;
typedef unsigned long long u64;

constexpr int kST = 512;                  // threads of a CTA, and bins of a histogram
constexpr int kSW = kST / 32;
constexpr int kList = 512;                // ids that one CTA sorts: one per thread
constexpr int kCand = 4096;               // ids of a CTA's share that it lists
constexpr int kMaxSplit = 16;
constexpr int kShareBytes = 160 * 1024;   // a CTA's share of a row, at most
constexpr int kShareIds = 65535;          // (mass sums: see find_cut)
constexpr float kUnit = 1099511627776.f;  // 2^40: units of mass

struct SampleArgs {
    const void *logits;
    const float *temperature, *top_p, *min_p, *u;
    const int32_t *top_k;
    int32_t *token;
    float *prob, *dist;
    int64_t stride;
    int32_t V, per, split;                // ids of a row, of a CTA's share; CTAs of a row
};

// 1 / (T ln 2) in two parts, and the row's largest logit; with a temperature near fp32's
// largest the logits are taken in units of 2^8 (pre = 2^-8), so that their differences,
// which it makes ordinary, stay in fp32's range.
struct Scale {
    float hi, lo, m, pre;                 // (m in these units, hi and lo per unit)
    __device__ __forceinline__ float t(float l) const { return fmaf(-l, pre, m) * hi; }   // -log2 of the weight (monotone)
    // exp((l - m) / T) for t(l) < 126
    __device__ __forceinline__ float weight(float l) const
    {
        l *= pre;
        const float d = m - l, v = d - m, rest = (m - (d - v)) - (l + v);
        const float n = rintf(d * hi), f = fmaf(d, hi, -n) + fmaf(rest, hi, d * lo);
        float y;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(-f));
        return y * __int_as_float((127 - int(n)) << 23);
    }
    // the same for any t
    __device__ __forceinline__ float weight_or_0(float l) const { return t(l) < 125.f ? weight(l) : 0.f; }
    // the same for any t, the exponent rounded as a whole: off by 2^-24 t ln 2 more, for sums (where t is
    // large enough to show, there are many of them or they weigh nothing)
    static __device__ __forceinline__ float rough(float t)
    {
        float y;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(-t));
        return y;
    }
};

// Place in the order: smaller is earlier (the logit, then the id).
__device__ __forceinline__ uint32_t order_bits(float l)
{
    const uint32_t b = __float_as_uint(l + 0.f);   // (-0 as 0: they tie)
    return ~((b & 0x80000000u) ? ~b : (b | 0x80000000u));
}
__device__ __forceinline__ u64 place(float l, uint32_t id) { return u64(order_bits(l)) << 32 | id; }

__device__ __forceinline__ float logit_at(u64 place)
{
    const uint32_t b = ~uint32_t(place >> 32);
    return __uint_as_float((b & 0x80000000u) ? b & 0x7fffffffu : ~b);
}

// t as a 32-bit number in units of 2^-26 (the weights below 2^-64 are one)
__device__ __forceinline__ uint32_t fixed(float t) { return t < 63.9f ? uint32_t(t * 67108864.f) : 0xffffffffu; }

__device__ __forceinline__ u64 mass_of(float w) { return u64(w * kUnit); }

struct Range {                            // ids whose leading digits are these
    uint32_t t, t_mask, bits, bits_mask, id, id_mask;
};

struct Border {                           // the digit where a cut lies, and what lies before it
    u64 before;
    uint32_t digit, inside;
    int found;
};

struct Exchange {                         // what the CTAs of a row tell one another
    u64 best;                             // highest logit (argmax key); then the race's winner
    u64 z;                                // mass
    float m, w;
    int bad;
};

struct Shared {
    Exchange ex[3];
    u64 red[kSW];
    uint32_t count[2][kST], lo[2][kST], hi[2][kST];
    uint32_t scan[kSW];
    u64 mscan[kSW];
    Border border;
    u64 list[kList];                      // places of the row's ids that are left, in the first CTA of the cluster
    u64 sort[kList], mass_before[kList];
    uint32_t list_n;
    u64 cut, cut_mass;
    uint32_t n_cand;
    float bound;
    uint32_t cand[kCand];
};

__device__ __forceinline__ u64 warp_sum64(u64 v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sums (or maxima) over the CTA; all threads get the result.
__device__ __forceinline__ u64 block_sum(Shared &s, u64 v)
{
    v = warp_sum64(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s.red[threadIdx.x >> 5] = v;
    __syncthreads();
    u64 r = 0;
#pragma unroll
    for (int i = 0; i < kSW; ++i) r += s.red[i];
    return r;
}
__device__ __forceinline__ u64 block_max(Shared &s, u64 v)
{
    v = warp_max_u64(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s.red[threadIdx.x >> 5] = v;
    __syncthreads();
    u64 r = 0;
#pragma unroll
    for (int i = 0; i < kSW; ++i) r = s.red[i] > r ? s.red[i] : r;
    return r;
}

// What CTA `lane` of the cluster has to tell, in lane `lane` of every warp (lanes
// behind the last CTA: nothing), so that the reads from all of them overlap.
__device__ __forceinline__ Exchange told(Exchange &x, int split)
{
    const int lane = threadIdx.x & 31;
    Exchange y{0, 0, -INFINITY, 0.f, 0};
    if (lane < split) y = *cg::this_cluster().map_shared_rank(&x, lane);
    return y;
}

// The sum of every CTA's *p.
__device__ __forceinline__ uint32_t cluster_sum(uint32_t *p, int split)
{
    uint32_t v[kMaxSplit], sum = 0;
#pragma unroll
    for (int i = 0; i < kMaxSplit; ++i) v[i] = i < split ? *cg::this_cluster().map_shared_rank(p, i) : 0;
#pragma unroll
    for (int i = 0; i < kMaxSplit; ++i) sum += v[i];
    return sum;
}
__device__ __forceinline__ u64 cluster_sum_wide(uint32_t *p, int split)
{
    uint32_t v[kMaxSplit];
    u64 sum = 0;
#pragma unroll
    for (int i = 0; i < kMaxSplit; ++i) v[i] = i < split ? *cg::this_cluster().map_shared_rank(p, i) : 0;
#pragma unroll
    for (int i = 0; i < kMaxSplit; ++i) sum += v[i];
    return sum;
}

__device__ __forceinline__ uint32_t block_max(Shared &s, uint32_t v)
{
    v = __reduce_max_sync(0xffffffffu, v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s.scan[threadIdx.x >> 5] = v;
    __syncthreads();
    uint32_t r = 0;
#pragma unroll
    for (int i = 0; i < kSW; ++i) r = max(r, s.scan[i]);
    return r;
}

// Inclusive sums over the threads of the CTA.
__device__ __forceinline__ void block_scan(Shared &s, uint32_t &n, u64 &mass)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const uint32_t a = __shfl_up_sync(0xffffffffu, n, o);
        const u64 b = __shfl_up_sync(0xffffffffu, mass, o);
        if (lane >= o) n += a, mass += b;
    }
    __syncthreads();
    if (lane == 31) s.scan[warp] = n, s.mscan[warp] = mass;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kSW; ++i)
        if (i < warp) n += s.scan[i], mass += s.mscan[i];
}

template <typename T>
struct Row {
    const SampleArgs &a;
    Shared &s;
    const T *share;                       // this CTA's ids lo .. lo + n - 1
    int lo, n, rank;
    Scale c;
    float t_max, l_min;                   // ids with t above are not kept; those with logits below are not looked at
    bool listed;                          // the others are in s.cand, else the whole share is looked at
    int round = 0;                        // histograms so far
    float t_lo = 0.f, t_hi = INFINITY;    // only ids with t in this range are looked at

    // f(logit, id) for each id that can be kept and is in the range
    template <typename F>
    __device__ __forceinline__ void each(F f) const
    {
        const int count = listed ? int(s.n_cand) : n;
        for (int i0 = threadIdx.x; i0 < count; i0 += 4 * kST) {
            float l[4];
            uint32_t j[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int i = i0 + k * kST;
                j[k] = i < count ? (listed ? s.cand[i] : uint32_t(i)) : 0;
                l[k] = i < count ? float(share[j[k]]) : -INFINITY;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (const float t = c.t(l[k]); l[k] >= l_min && t >= t_lo && t < t_hi) f(l[k], uint32_t(lo) + j[k]);
        }
    }
};

// A digit of an id: `width` bits from `shift` on of its weight (word 0), its logit
// (1) or itself (2).
struct Digit {
    int word, shift, width;
    __device__ __forceinline__ uint32_t of(uint32_t t, uint32_t bits, uint32_t id) const
    {
        return (word == 0 ? t : word == 1 ? bits : id) >> shift & ((1u << width) - 1);
    }
    __device__ __forceinline__ bool last() const { return word == 2 && shift == 0; }
    __device__ __forceinline__ void next()
    {
        if (shift == 0) ++word, shift = 32;
        width = min(8, shift);
        shift -= width;
    }
    __device__ __forceinline__ void narrow(Range &r, uint32_t digit) const
    {
        const uint32_t v = digit << shift, mask = ((1u << width) - 1) << shift;
        if (word == 0) r.t |= v, r.t_mask |= mask;
        else if (word == 1) r.bits |= v, r.bits_mask |= mask;
        else r.id |= v, r.id_mask |= mask;
    }
};
__device__ __forceinline__ bool within(const Range &r, uint32_t t, uint32_t bits, uint32_t id)
{
    return (((t ^ r.t) & r.t_mask) | ((bits ^ r.bits) & r.bits_mask) | ((id ^ r.id) & r.id_mask)) == 0;
}

// The first CTA's list of n places in order, one per thread (~0 behind them).
__device__ u64 sorted(Shared &s, int n)
{
    const int tid = threadIdx.x;
    u64 key = tid < n ? s.list[tid] : ~0ull;
    int size = 32;
    while (size < n) size *= 2;
    for (int k = 2; k <= size; k *= 2)
        for (int j = k / 2; j > 0; j /= 2) {
            u64 other;
            if (j >= 32) {
                __syncthreads();
                s.sort[tid] = key;
                __syncthreads();
                other = s.sort[tid ^ j];
            } else {
                other = __shfl_xor_sync(0xffffffffu, key, j);
            }
            const bool low = ((tid & j) == 0) == ((tid & k) == 0);   // this thread takes the smaller one
            key = (other < key) == low ? other : key;
        }
    return key;
}

// For the id `my` of mass `own` of this thread, one of n in the list: how many come
// before it and with what mass; sum_k: the mass of the first top_k (where that is
// not 0).  Short lists by comparing each with each (four threads per id: 128 ids
// take 32 steps), longer ones by sorting.
__device__ void settle(Shared &s, int n, u64 my, u64 own, int top_k, uint32_t &ahead, u64 &before, u64 &sum_k)
{
    const int tid = threadIdx.x;
    if (n <= kST / 4) {
        if (tid < n) s.sort[tid] = own;
        __syncthreads();
        const int i = tid >> 2;
        const u64 key = i < n ? s.list[i] : 0;
        uint32_t c = 0;
        u64 b = 0;
        for (int j = tid & 3; j < n; j += 4)
            if (s.list[j] < key) ++c, b += s.sort[j];
        c += __shfl_xor_sync(0xffffffffu, c, 1), b += __shfl_xor_sync(0xffffffffu, b, 1);
        c += __shfl_xor_sync(0xffffffffu, c, 2), b += __shfl_xor_sync(0xffffffffu, b, 2);
        if (i < n && (tid & 3) == 0) s.count[0][i] = c, s.mass_before[i] = b;
        __syncthreads();
        if (tid < n) ahead = s.count[0][tid], before = s.mass_before[tid];
    } else {
        const u64 at = sorted(s, n);
        __syncthreads();
        s.sort[tid] = at;
        __syncthreads();
        // every thread finds its own id in the order
        int lo = 0, hi = n;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (s.sort[mid] < my) lo = mid + 1;
            else hi = mid;
        }
        ahead = uint32_t(lo);
        // masses in order, and their sums
        __syncthreads();
        if (tid < n) s.sort[lo] = own;
        __syncthreads();
        u64 to = tid < n ? s.sort[tid] : 0;
        const u64 mass = to;
        uint32_t none = 0;
        block_scan(s, none, to);
        if (tid < n) s.mass_before[tid] = to - mass;
        __syncthreads();
        if (tid < n) before = s.mass_before[lo];
    }
    sum_k = top_k > 0 ? block_sum(s, tid < n && ahead < uint32_t(top_k) ? own : 0) : 0;
}

// The place of the last kept id: of the `want` first of the order (by_mass false),
// or of the ids before which less than `want` mass lies; only ids up to `last`
// count.  ~0 where all of them are kept.
template <typename T>
__device__ u64 find_cut(Row<T> &r, bool by_mass, u64 want, u64 last)
{
    Shared &s = r.s;
    const cg::cluster_group cl = cg::this_cluster();
    const int tid = threadIdx.x;
    Range range{};
    u64 before = 0;                       // ids, or mass, before the range
    r.t_lo = 0.f, r.t_hi = INFINITY;
    // the first digit: 256 to 512 bins up to the largest t that is left, which is l_min's (t is
    // monotone) and not t_max, since l_min is rounded to the logits' spacing
    const int top = 32 - __clz(fixed(r.c.t(r.l_min)) | 1);
    for (Digit digit{0, max(top - 9, 0), min(top, 9)};; digit.next()) {
        const int k = r.round++ & 1;
        s.count[k][tid] = s.lo[k][tid] = s.hi[k][tid] = 0;
        __syncthreads();
        r.each([&](float l, uint32_t id) {
            const float tf = r.c.t(l);
            const uint32_t t = fixed(tf);
            uint32_t d = t >> digit.shift;
            if (range.t_mask != 0 || last != ~0ull) {
                const uint32_t bits = order_bits(l);
                if ((u64(bits) << 32 | id) > last || !within(range, t, bits, id)) return;
                d = digit.of(t, bits, id);
            }
            if (!by_mass) {
                atomicAdd(&s.count[k][d], 1u);
            } else {
                // in units of 2^-31 of the largest weight of an octave, so that every weight
                // is whole; 15 and 16 bits of it apart, so that a share's sums fit
                const int octave = int(t >> 26);
                const uint32_t x = uint32_t(fminf(Scale::rough(tf - float(octave + 31)), 2147483648.f));
                atomicAdd(&s.lo[k][d], x & 0x7fffu);
                atomicAdd(&s.hi[k][d], x >> 15);
            }
        });
        cl.sync();
        u64 own;
        if (by_mass) {
            own = (cluster_sum_wide(&s.hi[k][tid], r.a.split) << 15) + cluster_sum_wide(&s.lo[k][tid], r.a.split);
            // to units of 2^-40 of the largest weight
            const int octave = int((range.t_mask == 0 ? uint32_t(tid) << digit.shift : range.t) >> 26);
            own = octave <= 9 ? own << (9 - octave) : own >> (octave - 9);
        } else {
            own = cluster_sum(&s.count[k][tid], r.a.split);
        }
        if (tid == 0) s.border.found = 0;
        u64 at = own, none_wide = 0;
        uint32_t none = 0;
        block_scan(s, none, at);
        at += before;
        u64 goal = want;
        if (by_mass && range.t_mask != 0) {
            // (within a digit that the cut is known to lie in, its bins' masses, rounded one by
            // one, may end before it)
            if (tid == kST - 1) s.border.before = at;
            __syncthreads();
            goal = min(want, s.border.before);
            __syncthreads();
        }
        if (own && at - own < goal && at >= goal) {
            s.border.found = 1;
            s.border.digit = tid;
            s.border.before = at - own;
            s.border.inside = uint32_t(own);
        }
        __syncthreads();
        const bool found = s.border.found;
        before = s.border.before;
        uint32_t inside = s.border.inside;         // (of counts)
        if (found) digit.narrow(range, s.border.digit);
        if (digit.word == 0 && digit.shift >= 8) {       // (fp32 holds the range's ends; see fixed)
            const u64 end = u64(range.t) + (1ull << digit.shift);
            r.t_lo = fminf(float(range.t) * (1.f / 67108864.f), 63.9f);
            r.t_hi = end >> 32 ? INFINITY : float(end) * (1.f / 67108864.f);
        }
        __syncthreads();
        if (!found) return ~0ull;

        // the first CTA sorts these, if they are few enough
        if (!by_mass && inside > kList && !digit.last()) continue;
        Shared *first = cl.map_shared_rank(&s, 0);
        if (r.rank == 0 && tid == 0) s.list_n = 0;
        auto in_range = [&](float l, uint32_t id, u64 &at) {
            const uint32_t t = fixed(r.c.t(l));
            if ((t ^ range.t) & range.t_mask) return false;
            const uint32_t bits = order_bits(l);
            at = u64(bits) << 32 | id;
            return at <= last && within(range, t, bits, id);
        };
        uint32_t mine = 0;
        r.each([&](float l, uint32_t id) {
            u64 at;
            mine += in_range(l, id, at);
        });
        uint32_t to = mine;
        block_scan(s, to, none_wide);
        cl.sync();
        if (tid == kST - 1) {
            s.scan[0] = atomicAdd(&first->list_n, to);
            s.scan[1] = to;
        }
        __syncthreads();
        if (s.scan[0] + s.scan[1] <= kList) {
            uint32_t i = s.scan[0] + to - mine;
            r.each([&](float l, uint32_t id) {
                u64 at;
                if (in_range(l, id, at)) first->list[i++] = at;
            });
        }
        cl.sync();
        inside = first->list_n;
        if (inside > kList && !digit.last()) {
            cl.sync();                    // (before the first CTA clears it)
            continue;
        }
        if (r.rank == 0) {
            const int m = int(min(inside, uint32_t(kList)));
            const u64 key = sorted(s, m);
            u64 own = tid < m ? (by_mass ? mass_of(r.c.weight_or_0(logit_at(key))) : 1) : 0, to = own;
            uint32_t none = 0;
            block_scan(s, none, to);
            // kept are those with fewer ids, or less mass, before them than wanted
            const int kept = __syncthreads_count(tid < m && before + to - own < want);
            if (tid == kept - 1) s.cut = key;
        }
        cl.sync();
        const u64 cut = first->cut;
        cl.sync();                        // (before the first CTA writes another)
        return cut;
    }
}

template <typename T>
__global__ void __launch_bounds__(kST, 2) k_sample(const __grid_constant__ SampleArgs a)
{
    extern __shared__ __align__(16) uint8_t dyn[];
    __shared__ Shared s;
    const cg::cluster_group cl = cg::this_cluster();
    const int row = blockIdx.x / a.split, rank = blockIdx.x % a.split, tid = threadIdx.x;
    pdl_wait();
    pdl_launch_dependents();
    const int lo = min(rank * a.per, a.V), n = min(a.per, a.V - lo);
    const T *p = static_cast<const T *>(a.logits) + size_t(row) * a.stride + lo;
    const float temperature = a.temperature ? a.temperature[row] : 0.f;
    int top_k = a.top_k ? a.top_k[row] : 0;
    float top_p = a.top_p ? a.top_p[row] : 1.f, min_p = a.min_p ? a.min_p[row] : 0.f;
    const bool greedy = !(temperature > 0.f);
    if (top_k <= 0 || top_k >= a.V) top_k = 0;
    top_p = top_p < 1.f ? fmaxf(top_p, 0.f) : 1.f;
    if (!(min_p > 0.f)) min_p = 0.f;
    min_p = fminf(min_p, 1.f);
    const bool cut = top_k > 0 || top_p < 1.f || min_p > 0.f;
    const float *u = a.u + size_t(row) * a.V;
    if (tid == 0) s.list_n = s.n_cand = 0, s.bound = 0.f;

    // ---- the share into shared memory (16-byte pieces as they lie in the row), its highest logit ----
    constexpr int E = 16 / sizeof(T), U = 4;
    const int front = min(n, int((16 - reinterpret_cast<uintptr_t>(p) % 16) % 16 / sizeof(T)));
    T *share = reinterpret_cast<T *>(dyn) + (E - front) % E;
    float thread_top = -INFINITY;
    bool bad = false;
    auto take = [&](T v) {
        const float x = float(v);
        thread_top = fmaxf(thread_top, x);        // (a NaN is never above)
        bad = bad || !(x < INFINITY);
    };
    const int nv = (n - front) / E, rest = front + nv * E;
    uint4 *sv = reinterpret_cast<uint4 *>(share + front);
    const int edges = front + n - rest, edge = tid < front ? tid : rest + tid - front;   // the ids around the pieces
    {
        const uint4 *pv = reinterpret_cast<const uint4 *>(p + front);
        if (!greedy && !cut)                       // the random numbers follow the logits from memory
            for (int j = tid * 32; j < n; j += kST * 32) asm volatile("prefetch.global.L2 [%0];" ::"l"(u + lo + j));
        for (int i0 = tid; i0 < nv; i0 += U * kST) {
            uint4 v[U];
#pragma unroll
            for (int k = 0; k < U; ++k)
                if (i0 + k * kST < nv) v[k] = __ldcs(pv + i0 + k * kST);
#pragma unroll
            for (int k = 0; k < U; ++k)
                if (i0 + k * kST < nv) {
                    sv[i0 + k * kST] = v[k];
                    const T *e = reinterpret_cast<const T *>(&v[k]);
#pragma unroll
                    for (int j = 0; j < E; ++j) take(e[j]);
                }
        }
        if (tid < edges) take(share[edge] = p[edge]);
    }
    constexpr int B = 8;
    float e_first = 0.5f, e[B];           // the first random numbers, where nothing is cut, on their way before the maximum
    auto load_u = [&](int j0) {
#pragma unroll
        for (int k = 0; k < B; ++k) {
            const int j = j0 + k * kST + tid;
            e[k] = j < n ? __ldcs(u + lo + j) : 0.5f;
        }
    };
    if (!greedy && !cut) {
        if (tid < n) e_first = __ldcs(u + lo + tid);
        load_u(kST);
    }
    // (the order of the keys is the logits'; a logit that makes the row's choice none is above all)
    constexpr uint32_t kBad = 0xffffffffu;
    const uint32_t cta_key = block_max(s, bad && !greedy ? kBad : ~order_bits(thread_top));
    bad = cta_key == kBad;
    const float cta_top = logit_at(u64(~cta_key) << 32);
    auto logit_of = [](u64 key) {         // of an argmax key
        const uint32_t b = uint32_t(key >> 32);
        return __uint_as_float((b & 0x80000000u) ? b & 0x7fffffffu : ~b);
    };
    Row<T> r{a, s, share, lo, n, rank};
    {
        const float unit = temperature >= 0x1p100f ? 256.f : 1.f, c = 1.4426950408889634f * unit / temperature;
        r.c.pre = 1.f / unit;
        r.c.hi = fminf(fmaxf(c, FLT_TRUE_MIN), FLT_MAX);   // (above 0: a logit of -infinity has t = infinity)
        r.c.lo = 0.f;
        if (c > 0.f && c <= FLT_MAX)
            r.c.lo = (fmaf(-c, temperature, 1.4426950216293335f * unit) + 1.9259629911e-8f * unit) / temperature;
    }
    int32_t token = -1;
    float prob = 0.f;
    u64 last = ~0ull;                     // the place of the last kept id
    u64 z = 0;                            // the mass of the kept ids

    if (!greedy && !cut) {
        // ---- the race over all ids, by this CTA's own maximum ----
        r.c.m = cta_top * r.c.pre;
        float won = 0.f, won_w = 0.f;
        int who = -1;
        u64 mass = 0;
        // an id's weight, and its part in the race unless `bound` rules it out, which
        // needs no logarithm: -log u >= 1 - u
        auto take_part = [&](float l, float e, int j, float bound, float &sum) {
            const float t = r.c.t(l);
            float w = Scale::rough(t);
            sum += w;
            if (w > bound * (1.f - e)) {
                if (t < 125.f) w = r.c.weight(l);
                const float y = __fdividef(w, -logf(e));
                if (y > won) won = y, won_w = w, who = j;
            }
        };
        // the first id of every thread gives all of them a bound; the others raise it
        float sum = 0.f;
        if (tid < n) take_part(float(share[tid]), e_first, tid, 0.f, sum);
        if (tid == 0) s.bound = 0.f;
        const float first_best = __uint_as_float(block_max(s, __float_as_uint(won)));
        if (tid == 0) s.bound = first_best * 0.999f;
        __syncthreads();
        for (int j0 = kST; j0 < n; j0 += B * kST) {
            if (j0 > kST) load_u(j0);
            const float bound = fmaxf(*static_cast<volatile float *>(&s.bound), won * 0.999f);
#pragma unroll
            for (int k = 0; k < B; ++k) {
                const int j = j0 + k * kST + tid;
                if (j < n) take_part(float(share[j]), e[k], j, bound, sum);
            }
            if (won * 0.999f > bound) atomicMax(reinterpret_cast<int *>(&s.bound), __float_as_int(won * 0.999f));
            mass += mass_of(sum);
            sum = 0.f;
        }
        mass += mass_of(sum);
        const u64 key = who >= 0 ? argmax_key(won, uint32_t(lo + who)) : 0, high = block_max(s, key);
        if (key && key == high) s.ex[0].w = won_w;
        mass = block_sum(s, mass);
        if (tid == 0) {
            s.ex[0].best = high;
            s.ex[0].z = mass;
            s.ex[0].m = cta_top;
            s.ex[0].bad = bad;
        }
        cl.sync();
        const Exchange x = told(s.ex[0], a.split);
        const bool any_bad = __any_sync(0xffffffffu, x.bad);
        r.c.m = warp_max(x.m) * r.c.pre;
        const float f = x.best ? r.c.weight_or_0(x.m) : 0.f;
        const float total = warp_sum(f * (float(x.z) * (1.f / kUnit)));
        const u64 mine = f > 0.f ? argmax_key(f * logit_of(x.best), uint32_t(argmax_key_index(x.best))) : 0;
        const u64 win = warp_max_u64(mine);
        const float w = __shfl_sync(0xffffffffu, f * x.w, win ? __ffs(__ballot_sync(0xffffffffu, mine == win)) - 1 : 0);
        if (win && !any_bad) token = argmax_key_index(win), prob = w / total;
        r.listed = false;
        r.t_max = 124.9f;
        z = token >= 0 ? u64(double(total) * double(kUnit)) : 0;
    } else {
        // ---- the row's highest logit ----
        if (greedy && cta_top > -INFINITY) {       // the lowest id that has the CTA's
            int id = n;
            for (int j = tid; j < n; j += kST)
                if (float(share[j]) == cta_top) {
                    id = j;
                    break;
                }
            const u64 key = block_max(s, id < n ? argmax_key(cta_top + 0.f, uint32_t(lo + id)) : 0);
            if (tid == 0) s.ex[0].best = key;
        }
        if (tid == 0) {
            s.ex[0].m = cta_top;
            s.ex[0].bad = bad;
        }
        cl.sync();
        const Exchange x = told(s.ex[0], a.split);
        const bool any_bad = __any_sync(0xffffffffu, x.bad);
        const float row_top = warp_max(x.m);
        if (greedy) {
            const u64 best = warp_max_u64(x.m > -INFINITY ? x.best : 0);
            if (best) token = argmax_key_index(best), prob = 1.f;
        } else if (row_top > -INFINITY && !any_bad) {
            r.c.m = row_top * r.c.pre;
            // ---- what can be kept ----
            r.t_max = 124.9f;
            u64 all = 0;                  // the row's mass (top-p alone)
            // (top-p of the top_k needs all of these, those below min_p too)
            if (min_p > 0.f && !(top_k > 0 && top_p < 1.f)) r.t_max = fminf(r.t_max, -log2f(min_p) + 0.01f);
            if (top_k > 0) {
                // the k-th highest of the cluster's threads' maxima, to a bin
                s.count[0][tid] = 0;
                __syncthreads();
                const float t = r.c.t(thread_top);
                if (t < 63.f) atomicAdd(&s.count[0][fixed(t) >> 23], 1u);
                cl.sync();
                ++r.round;
                const uint32_t own = cluster_sum(&s.count[0][tid], a.split);
                uint32_t k = own;
                u64 none = 0;
                if (tid == 0) s.border.found = 0;
                block_scan(s, k, none);
                if (own && k >= uint32_t(top_k) && k - own < uint32_t(top_k)) {
                    s.border.found = 1;
                    s.border.digit = tid;
                }
                __syncthreads();
                if (s.border.found) r.t_max = fminf(r.t_max, float(s.border.digit + 1) * 0.125f + 1e-5f);
            } else if (top_p < 1.f) {
                u64 mass = 0;
                for (int q = tid; q < nv; q += kST) {
                    alignas(16) T e16[E];
                    *reinterpret_cast<uint4 *>(e16) = sv[q];
                    float sum = 0.f;
#pragma unroll
                    for (int j = 0; j < E; ++j) sum += Scale::rough(r.c.t(float(e16[j])));
                    mass += mass_of(sum);
                }
                if (tid < edges) mass += mass_of(Scale::rough(r.c.t(float(share[edge]))));
                mass = block_sum(s, mass);
                if (tid == 0) s.ex[1].z = mass;
                cl.sync();
                all = warp_sum64(told(s.ex[1], a.split).z);
                const float least = (1.f - top_p) * (float(all) * (1.f / kUnit)) / float(a.V);
                if (least > 0.f) r.t_max = fminf(r.t_max, -log2f(least) + 0.01f);
            }
            // ---- their list, and a common one in the first CTA, as far as it goes ----
            // (by the logits, a little below the bound, and above those of no weight)
            r.l_min = fmaxf((r.c.m - r.t_max / r.c.hi * 1.00001f) * (1.f / r.c.pre), -FLT_MAX);
            Shared *first = cl.map_shared_rank(&s, 0);
            const int lane = tid & 31;
            bool at_edge = tid < edges && float(share[edge]) >= r.l_min;   // an id before or behind the whole pieces
            for (int q0 = 0; q0 == 0 || q0 < nv; q0 += 32 / E * kST) {
                uint32_t mask = 0;
#pragma unroll
                for (int k = 0; k < 32 / E; ++k) {
                    const int q = q0 + k * kST + tid;
                    if (q >= nv) continue;
                    alignas(16) T e16[E];
                    *reinterpret_cast<uint4 *>(e16) = sv[q];
#pragma unroll
                    for (int j = 0; j < E; ++j)
                        if (float(e16[j]) >= r.l_min) mask |= 1u << (k * E + j);
                }
                const uint32_t own = __popc(mask) + at_edge;
                uint32_t to = own;
#pragma unroll
                for (int o = 1; o < 32; o *= 2) {
                    const uint32_t x = __shfl_up_sync(0xffffffffu, to, o);
                    if (lane >= o) to += x;
                }
                uint32_t here = 0, there = 0;
                if (lane == 31 && to) there = atomicAdd(&first->list_n, to), here = atomicAdd(&s.n_cand, to);
                here = __shfl_sync(0xffffffffu, here, 31) + to - own;
                there = __shfl_sync(0xffffffffu, there, 31) + to - own;
                auto keep = [&](int j) {
                    if (here < kCand) s.cand[here] = uint32_t(j);
                    if (there < kList) first->list[there] = place(float(share[j]), uint32_t(lo + j));
                    ++here, ++there;
                };
                if (at_edge) keep(edge);
                at_edge = false;
                for (; mask; mask &= mask - 1) {
                    const int i = __ffs(mask) - 1;
                    keep(front + (q0 + i / E * kST + tid) * E + i % E);
                }
            }
            cl.sync();
            r.listed = s.n_cand <= kCand;
            const uint32_t m = first->list_n;
            const u64 want = u64(double(top_p) * double(all));
            if (m <= kList) {
                if (rank == 0) {
                    // this thread's id in the race, and the number of ids and the mass before it
                    const bool mine = tid < int(m);
                    const u64 my = mine ? s.list[tid] : ~0ull;
                    // (l_min may let some of no weight through)
                    const float e = mine ? u[uint32_t(my)] : 0.5f, w = mine ? r.c.weight_or_0(logit_at(my)) : 0.f;
                    const u64 own = mine ? mass_of(w) : 0;
                    uint32_t ahead = 0;
                    u64 before = 0, sum_k = 0;
                    settle(s, int(m), my, own, top_k, ahead, before, sum_k);
                    const u64 up_to = top_k > 0 ? u64(double(top_p) * double(sum_k)) : want;
                    const bool keep = w > 0.f && (top_k == 0 || ahead < uint32_t(top_k)) && w >= min_p &&
                                      (top_p >= 1.f || before < up_to || ahead == 0);
                    z = block_sum(s, keep ? own : 0);
                    const u64 key = keep ? argmax_key(__fdividef(w, -logf(e)), uint32_t(my)) : 0, high = block_max(s, key);
                    if (key && key == high) s.ex[2].w = w;
                    if (a.dist) {
                        const u64 worst = block_max(s, keep ? my : 0);
                        if (tid == 0) s.cut = worst, s.cut_mass = z;
                    }
                    __syncthreads();
                    token = argmax_key_index(high);
                    prob = s.ex[2].w / (float(z) * (1.f / kUnit));
                }
                if (a.dist) {
                    cl.sync();
                    last = first->cut;
                    z = first->cut_mass;
                }
            } else {
                u64 mass = 0;
                if (top_k > 0) last = find_cut(r, false, u64(top_k), ~0ull);
                if (top_p < 1.f) {
                    u64 up_to = want;
                    if (top_k > 0) {      // of the mass of these
                        r.t_lo = 0.f, r.t_hi = INFINITY;
                        r.each([&](float l, uint32_t id) {
                            if (place(l, id) <= last) mass += mass_of(Scale::rough(r.c.t(l)));
                        });
                        mass = block_sum(s, mass);
                        if (tid == 0) s.ex[1].z = mass;
                        cl.sync();
                        up_to = u64(double(top_p) * double(warp_sum64(told(s.ex[1], a.split).z)));
                    }
                    const u64 p_last = find_cut(r, true, up_to > 0 ? up_to : 1, last);
                    last = p_last < last ? p_last : last;
                }
                // the race over the kept ids
                float won = 0.f, won_w = 0.f;
                int who = -1;
                mass = 0;
                const int count = r.listed ? int(s.n_cand) : n;
                const float l_last = last == ~0ull ? r.l_min : logit_at(last);
                const int id_last = last == ~0ull ? a.V : int(uint32_t(last));
                for (int i0 = 0; i0 < count; i0 += B * kST) {
                    float l[B];
                    int id[B];
                    const float bound = fmaxf(*static_cast<volatile float *>(&s.bound), won * 0.999f);
#pragma unroll
                    for (int k = 0; k < B; ++k) {          // (the random numbers' loads overlap)
                        const int i = i0 + k * kST + tid;
                        id[k] = -1;
                        e[k] = 0.5f;
                        if (i >= count) continue;
                        const int j = r.listed ? int(s.cand[i]) : i;
                        l[k] = float(share[j]);
                        if (l[k] > l_last || (l[k] == l_last && lo + j <= id_last)) {
                            id[k] = lo + j;
                            e[k] = __ldcs(u + lo + j);
                        }
                    }
#pragma unroll
                    for (int k = 0; k < B; ++k) {
                        if (id[k] < 0) continue;
                        const float t = r.c.t(l[k]);
                        float w = Scale::rough(t);
                        // (next to min_p by the exact weight, as the distribution has it)
                        if (w < min_p * 1.0001f && r.c.weight_or_0(l[k]) < min_p) continue;
                        mass += mass_of(w);
                        if (!(w > bound * (1.f - e[k]))) continue;
                        w = r.c.weight(l[k]);
                        const float y = __fdividef(w, -logf(e[k]));
                        if (y > won || (y == won && id[k] < who)) won = y, won_w = w, who = id[k];
                    }
                    if (won * 0.999f > bound) atomicMax(reinterpret_cast<int *>(&s.bound), __float_as_int(won * 0.999f));
                }
                const u64 key = who >= 0 ? argmax_key(won, uint32_t(who)) : 0, high = block_max(s, key);
                if (key && key == high) s.ex[2].w = won_w;
                mass = block_sum(s, mass);
                if (tid == 0) s.ex[2].best = high, s.ex[2].z = mass;
                cl.sync();
                const Exchange y = told(s.ex[2], a.split);
                z = warp_sum64(y.z);
                const u64 win = warp_max_u64(y.best);
                const float ww = __shfl_sync(0xffffffffu, y.w, __ffs(__ballot_sync(0xffffffffu, y.best == win)) - 1);
                token = argmax_key_index(win);
                prob = ww / (float(z) * (1.f / kUnit));
            }
        }
    }
    if (rank == 0 && tid == 0) {
        a.token[row] = token;
        if (a.prob) a.prob[row] = prob;
    }
    if (a.dist) {
        float *d = a.dist + size_t(row) * a.V + lo;
        const float inv = 1.f / (float(z) * (1.f / kUnit));
        for (int j = tid; j < n; j += kST) {
            float y = 0.f;
            if (greedy) {
                y = lo + j == token ? 1.f : 0.f;
            } else if (z > 0) {
                const float l = float(share[j]), t = r.c.t(l);
                if (t < 125.f && place(l, uint32_t(lo + j)) <= last) {
                    const float w = r.c.weight(l);
                    if (w >= min_p) y = w * inv;
                }
            }
            d[j] = y;
        }
    }
    cl.sync();                            // nobody leaves while its shares are read
}

template <typename T>
cudaError_t run(const SampleArgs &a, int rows, cudaStream_t s)
{
    const size_t smem = (size_t(a.per) * sizeof(T) + 15) / 16 * 16 + 16;
    cudaError_t e = cudaFuncSetAttribute(k_sample<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kShareBytes + 32);
    if (e == cudaSuccess && a.split > 8)
        e = cudaFuncSetAttribute(k_sample<T>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    return spec_launch(k_sample<T>, dim3(unsigned(rows) * a.split), kST, smem, a.split, s, a);
}

}  // namespace
}  // namespace gpt2

using namespace gpt2;

extern "C" int gpt2_op_sample(const void *logits, int32_t dtype, int64_t row_stride, int32_t n_rows, int32_t vocab,
                              const float *temperature, const int32_t *top_k, const float *top_p, const float *min_p,
                              const float *u, int32_t *token, float *prob, float *dist, void *stream)
{
    if (!logits || !token || !is_row_type(dtype) || n_rows < 0 || vocab < 1 || row_stride < vocab)
        return GPT2_ERR_INVALID_ARG;
    if (temperature && !u) return GPT2_ERR_INVALID_ARG;
    if (!aligned4(temperature, top_k, top_p, min_p, u, token, prob, dist)) return GPT2_ERR_INVALID_ARG;
    const int size = elem_size(dtype);
    if (reinterpret_cast<uintptr_t>(logits) % size) return GPT2_ERR_INVALID_ARG;
    if (vocab > GPT2_SAMPLE_MAX_VOCAB || (long long)n_rows * kMaxSplit >= (1ll << 31)) return GPT2_ERR_INVALID_ARG;
    if (n_rows == 0) return GPT2_OK;
    int rc;
    const int sms = spec_sms(&rc);
    if (!sms) return rc;
    SampleArgs a{logits, temperature, top_p, min_p, u, top_k, token, prob, dist, row_stride, vocab, 0, 1};
    // As many CTAs as a share needs, and twice as many while every row's cluster still
    // runs at once and a share has 2048 ids or more; for more rows than that, enough for
    // two CTAs of an SM, so that one computes while the other loads.
    int split = 1;
    auto per = [&](int n) { return (vocab + n - 1) / n; };
    auto held = [&](int n) { return (long long)per(n) * size + int(sizeof(Shared)) <= 112 * 1024 ? 2 : 1; };
    while ((long long)per(split) * size > kShareBytes || per(split) > kShareIds) split *= 2;
    for (int i = 0; i < 3; ++i)          // (16: one row 10.9 us instead of 8.8, eight rows 17.3 instead of 9.3)
        if (split == 1 << i && vocab >= 4096 * split && (n_rows <= kClustersFit[i] * held(2 * split) || held(split) < 2))
            split *= 2;
    a.split = split;
    a.per = per(split);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    switch (dtype) {
    case GPT2_F32: return spec_rc(run<float>(a, n_rows, s));
    case GPT2_F16: return spec_rc(run<__half>(a, n_rows, s));
    default: return spec_rc(run<__nv_bfloat16>(a, n_rows, s));
    }
}
