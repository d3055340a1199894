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
//   - Else each CTA first bounds what can be kept: the top_k highest lie above
//     the k-th highest of its threads' own maxima (to a bin), and with top-p alone
//     every id whose weight is at most (1 - top_p) z / V lies behind the cut, z a
//     part of the sum.  What is left, usually dozens to a few hundred ids, goes to a list.
//   - A list of up to kList ids is settled by one CTA: an id's rank and the mass
//     before it are counted over the list, and the race is run over what is kept.
//   - A longer one is narrowed by histograms over the cluster, of counts and
//     masses, by digits of (weight, logit, id), until the digit where the cut
//     lies holds at most kList ids, which are then ranked as above.
// Masses are summed as integers (a weight in units of 2^-40 of the largest), so that
// neither order nor shape of a sum shows and every call gives the same bits.
//
// Rounding: a weight is off by some 2^-22 of itself (the exponent's integer part
// is taken off exactly before the exponential), so a cut by mass can differ from
// the exact one where it falls within about 1e-7 of its border, and a race where
// its two best are within 1e-6 of each other.
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
constexpr int kList = 256;                // ids that one CTA ranks
constexpr int kCand = 4096;               // ids of a CTA's share that it lists
constexpr int kMaxSplit = 16;
constexpr int kShareBytes = 160 * 1024;   // a CTA's share of a row
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

// 1 / (T ln 2) in two parts, and the row's largest logit.
struct Scale {
    float hi, lo, m;
    __device__ __forceinline__ float t(float l) const { return (m - l) * hi; }   // -log2 of the weight (monotone)
    // exp((l - m) / T) for t(l) < 126
    __device__ __forceinline__ float weight(float l) const
    {
        const float d = m - l, v = d - m, rest = (m - (d - v)) - (l + v);
        const float n = rintf(d * hi), f = fmaf(d, hi, -n) + fmaf(rest, hi, d * lo);
        float y;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(-f));
        return y * __int_as_float((127 - int(n)) << 23);
    }
};

// Place in the order: smaller is earlier (the logit, then the id).
__device__ __forceinline__ uint32_t order_bits(float l)
{
    const uint32_t b = __float_as_uint(l + 0.f);   // (-0 as 0: they tie)
    return ~((b & 0x80000000u) ? ~b : (b | 0x80000000u));
}
__device__ __forceinline__ u64 place(float l, uint32_t id) { return u64(order_bits(l)) << 32 | id; }

// t as a 32-bit number in units of 2^-26 (the weights below 2^-64 are one)
__device__ __forceinline__ uint32_t fixed(float t) { return t < 63.9f ? uint32_t(t * 67108864.f) : 0xffffffffu; }

__device__ __forceinline__ u64 mass_of(float w) { return u64(w * kUnit); }

struct Range {                            // ids whose leading digits are these
    uint32_t t, t_mask, bits, bits_mask, id, id_mask;
};

struct Border {                           // where a cut lies: in a digit, or at an id
    u64 before_mass;
    uint32_t before, inside, digit;
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
    float fred[kSW];
    uint32_t count[2][kST], lo[2][kST], hi[2][kST];
    uint32_t scan[kSW];
    u64 mscan[kSW], total;
    Border border;
    // the row's list, in the first CTA of the cluster
    float list_l[kList];
    uint32_t list_id[kList];
    u64 list_mass[kList];
    uint32_t list_n;
    u64 cut, cut_mass;
    uint32_t n_cand;
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
    float t_max;                          // ids with t above it are not kept
    bool listed;                          // they are in s.cand, else the whole share is looked at
    int round = 0;                        // histograms so far

    // f(logit, id) for each id that can be kept
    template <typename F>
    __device__ __forceinline__ void each(F f) const
    {
        if (listed) {
            const int k = int(s.n_cand);
            for (int i = threadIdx.x; i < k; i += kST) {
                const uint32_t j = s.cand[i];
                f(float(share[j]), uint32_t(lo) + j);
            }
        } else {
            for (int j = threadIdx.x; j < n; j += kST) {
                const float l = float(share[j]);
                if (c.t(l) <= t_max) f(l, uint32_t(lo + j));
            }
        }
    }
};

// The digit of level 0..11 of an id: of the weight (9, 8, 8 and 7 bits), of the
// logit (8 each), of the id (8 each).
__device__ __forceinline__ uint32_t digit_of(int level, uint32_t t, uint32_t bits, uint32_t id)
{
    switch (level) {
    case 0: return t >> 23;
    case 1: return t >> 15 & 255;
    case 2: return t >> 7 & 255;
    case 3: return t & 127;
    default: break;
    }
    const uint32_t v = level < 8 ? bits : id;
    return v >> (8 * (3 - (level & 3))) & 255;
}
__device__ __forceinline__ void narrow(Range &r, int level, uint32_t digit)
{
    switch (level) {
    case 0: r.t = digit << 23, r.t_mask = 0xff800000u; return;
    case 1: r.t |= digit << 15, r.t_mask |= 0x007f8000u; return;
    case 2: r.t |= digit << 7, r.t_mask |= 0x00007f80u; return;
    case 3: r.t |= digit, r.t_mask |= 0x7fu; return;
    default: break;
    }
    const int shift = 8 * (3 - (level & 3));
    if (level < 8) r.bits |= digit << shift, r.bits_mask |= 255u << shift;
    else r.id |= digit << shift, r.id_mask |= 255u << shift;
}
__device__ __forceinline__ bool within(const Range &r, uint32_t t, uint32_t bits, uint32_t id)
{
    return (((t ^ r.t) & r.t_mask) | ((bits ^ r.bits) & r.bits_mask) | ((id ^ r.id) & r.id_mask)) == 0;
}

// The place of the last kept id: of the `want` first of the order (by_mass false),
// or of the ids before which less than `want` mass lies; only ids up to `last`
// count.  ~0 where all of them are kept.  mass: of the ids up to that place.
template <typename T>
__device__ u64 find_cut(Row<T> &r, bool by_mass, u64 want, u64 last, u64 &mass)
{
    Shared &s = r.s;
    const cg::cluster_group cl = cg::this_cluster();
    const int tid = threadIdx.x;
    Range range{};
    u64 before_mass = 0;
    uint32_t before = 0;
    for (int level = 0;; ++level) {
        const int k = r.round++ & 1;
        s.count[k][tid] = s.lo[k][tid] = s.hi[k][tid] = 0;
        __syncthreads();
        r.each([&](float l, uint32_t id) {
            const uint32_t t = fixed(r.c.t(l)), bits = order_bits(l);
            if ((u64(bits) << 32 | id) > last || !within(range, t, bits, id)) return;
            const uint32_t d = digit_of(level, t, bits, id);
            // in units of 2^-31 of the largest weight of an octave, so that every weight is whole
            const uint32_t x = uint32_t(r.c.weight(l) * __int_as_float((158 + int(t >> 26)) << 23));
            atomicAdd(&s.count[k][d], 1u);
            const uint32_t old = atomicAdd(&s.lo[k][d], x);
            if (old + x < old) atomicAdd(&s.hi[k][d], 1u);
        });
        cl.sync();
        uint32_t n = 0;
        u64 sum = 0;
        for (int i = 0; i < r.a.split; ++i) {
            n += *cl.map_shared_rank(&s.count[k][tid], i);
            sum += (u64(*cl.map_shared_rank(&s.hi[k][tid], i)) << 32) + *cl.map_shared_rank(&s.lo[k][tid], i);
        }
        // to units of 2^-40 of the largest weight
        const int octave = int((level == 0 ? uint32_t(tid) << 23 : range.t) >> 26);
        sum = octave <= 9 ? sum << (9 - octave) : sum >> (octave - 9);
        uint32_t n_to = n;
        u64 sum_to = sum;
        if (tid == 0) s.border.found = 0;
        block_scan(s, n_to, sum_to);
        const u64 at = by_mass ? before_mass + sum_to : before + n_to, was = at - (by_mass ? sum : u64(n));
        if (n && was < want && at >= want) {
            s.border.found = 1;
            s.border.digit = tid;
            s.border.inside = n;
            s.border.before = before + n_to - n;
            s.border.before_mass = before_mass + sum_to - sum;
        }
        if (tid == kST - 1) s.total = before_mass + sum_to;
        __syncthreads();
        if (!s.border.found) {
            mass = s.total;
            __syncthreads();
            return ~0ull;
        }
        before = s.border.before;
        before_mass = s.border.before_mass;
        const uint32_t inside = s.border.inside;
        narrow(range, level, s.border.digit);
        __syncthreads();
        if (inside > kList && level < 11) continue;

        // the first CTA ranks these
        Shared *first = cl.map_shared_rank(&s, 0);
        if (r.rank == 0 && tid == 0) s.list_n = 0;
        cl.sync();
        r.each([&](float l, uint32_t id) {
            const uint32_t bits = order_bits(l);
            if ((u64(bits) << 32 | id) > last || !within(range, fixed(r.c.t(l)), bits, id)) return;
            const uint32_t i = atomicAdd(&first->list_n, 1u);
            if (i < kList) {
                first->list_l[i] = l;
                first->list_id[i] = id;
                first->list_mass[i] = mass_of(r.c.weight(l));
            }
        });
        cl.sync();
        if (r.rank == 0) {
            const int m = int(inside < kList ? inside : kList), i = tid >> 1;
            uint32_t rank = 0;
            u64 sums = 0, own = 0, my = ~0ull;
            if (i < m) {
                my = place(s.list_l[i], s.list_id[i]);
                own = s.list_mass[i];
                for (int j = tid & 1; j < m; j += 2)
                    if (place(s.list_l[j], s.list_id[j]) < my) ++rank, sums += s.list_mass[j];
            }
            rank += __shfl_xor_sync(0xffffffffu, rank, 1);
            sums += __shfl_xor_sync(0xffffffffu, sums, 1);
            // kept are those with a rank, or a mass before them, below what is wanted
            const bool keep = i < m && (by_mass ? before_mass + sums < want : before + rank < want);
            const u64 worst = block_max(s, keep ? my : 0);
            const u64 total = block_sum(s, keep && !(tid & 1) ? own : 0);
            if (tid == 0) s.cut = worst, s.cut_mass = before_mass + total;
        }
        cl.sync();
        const u64 cut = first->cut;
        mass = first->cut_mass;
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
    T *share = reinterpret_cast<T *>(dyn);
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
    if (tid == 0) s.list_n = s.n_cand = 0;

    // ---- the share into shared memory, its highest logit ----
    float top = -INFINITY;
    int id = -1;
    bool bad = false;
    auto take = [&](T v, int j) {
        share[j] = v;
        const float x = float(v);
        if (x > top) top = x, id = j;     // (a NaN or -infinity is never above)
        bad = bad || x != x || x == INFINITY;
    };
    {
        constexpr int E = 16 / sizeof(T), U = 4;
        const int head = min(n, int((16 - reinterpret_cast<uintptr_t>(p) % 16) % 16 / sizeof(T)));
        const int nv = (n - head) / E, rest = head + nv * E;
        const uint4 *pv = reinterpret_cast<const uint4 *>(p + head);
        if (tid < head) take(p[tid], tid);
        for (int i0 = tid; i0 < nv; i0 += U * kST) {
            uint4 v[U];
#pragma unroll
            for (int k = 0; k < U; ++k)
                if (i0 + k * kST < nv) v[k] = __ldcs(pv + i0 + k * kST);
#pragma unroll
            for (int k = 0; k < U; ++k)
                if (i0 + k * kST < nv) {
                    const T *e = reinterpret_cast<const T *>(&v[k]);
#pragma unroll
                    for (int j = 0; j < E; ++j) take(e[j], head + (i0 + k * kST) * E + j);
                }
        }
        if (tid < n - rest) take(p[rest + tid], rest + tid);
    }
    const float thread_top = top;
    u64 best = block_max(s, id >= 0 ? argmax_key(top + 0.f, uint32_t(lo + id)) : 0);
    bad = __syncthreads_or(bad);
    auto logit_of = [](u64 key) {         // of an argmax key
        const uint32_t b = uint32_t(key >> 32);
        return __uint_as_float((b & 0x80000000u) ? b & 0x7fffffffu : ~b);
    };
    Row<T> r{a, s, share, lo, n, rank};
    {
        const float c = 1.4426950408889634f / temperature;
        r.c.hi = fminf(c, FLT_MAX);
        r.c.lo = 0.f;
        if (c > 0.f && c <= FLT_MAX)
            r.c.lo = (fmaf(-c, temperature, 1.4426950216293335f) + 1.9259629911e-8f) / temperature;
    }
    int32_t token = -1;
    float prob = 0.f;
    u64 last = ~0ull;                     // the place of the last kept id
    u64 z = 0;                            // the mass of the kept ids

    if (!greedy && !cut) {
        // ---- the race over all ids, by this CTA's own maximum ----
        r.c.m = best ? logit_of(best) : 0.f;
        float won = -1.f, won_w = 0.f, bound = 0.f;
        int who = -1;
        u64 mass = 0;
        for (int j0 = 0; j0 < n; j0 += 4 * kST) {
            float e[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int j = j0 + k * kST + tid;
                e[k] = j < n ? u[lo + j] : 0.5f;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int j = j0 + k * kST + tid;
                const float l = j < n ? float(share[j]) : -INFINITY;
                if (!(r.c.t(l) < 125.f)) continue;
                const float w = r.c.weight(l);
                mass += mass_of(w);
                // (what the warp's best rules out needs no logarithm: -log u >= 1 - u)
                if (w > bound * (1.f - e[k])) {
                    const float y = __fdividef(w, -logf(e[k]));
                    if (y > won) won = y, won_w = w, who = j;
                }
            }
            bound = warp_max(won) * 0.999f;
        }
        const u64 key = who >= 0 ? argmax_key(won, uint32_t(lo + who)) : 0, high = block_max(s, key);
        if (key && key == high) s.ex[0].w = won_w;
        mass = block_sum(s, mass);
        if (tid == 0) {
            s.ex[0].best = high;
            s.ex[0].z = mass;
            s.ex[0].m = best ? r.c.m : -INFINITY;
            s.ex[0].bad = bad;
        }
        cl.sync();
        float m = -INFINITY, mw = 0.f;
        int any_bad = 0;
        for (int i = 0; i < a.split; ++i) {
            const Exchange *x = cl.map_shared_rank(&s.ex[0], i);
            m = fmaxf(m, x->m);
            any_bad |= x->bad;
        }
        float score = -1.f, total = 0.f;
        for (int i = 0; i < a.split && !any_bad; ++i) {
            const Exchange *x = cl.map_shared_rank(&s.ex[0], i);
            if (x->best == 0) continue;
            const float t = (m - x->m) * r.c.hi, f = t < 125.f ? Scale{r.c.hi, r.c.lo, m}.weight(x->m) : 0.f;
            total += f * (float(x->z) * (1.f / kUnit));
            const float y = f * logit_of(x->best);
            if (y > score) score = y, token = argmax_key_index(x->best), mw = f * x->w;
        }
        if (token >= 0) prob = mw / total;
        r.c.m = m;
        r.listed = false;
        r.t_max = 124.9f;
        z = u64(double(total) * double(kUnit));
        if (any_bad) token = -1;
    } else {
        // ---- the row's highest logit ----
        if (tid == 0) {
            s.ex[0].best = best;
            s.ex[0].bad = bad;
        }
        cl.sync();
        int any_bad = 0;
        best = 0;
        for (int i = 0; i < a.split; ++i) {
            const Exchange *x = cl.map_shared_rank(&s.ex[0], i);
            best = x->best > best ? x->best : best;
            any_bad |= x->bad;
        }
        if (greedy) {
            if (best) token = argmax_key_index(best), prob = 1.f;
        } else if (best && !any_bad) {
            r.c.m = logit_of(best);
            // ---- what can be kept ----
            r.t_max = 124.9f;
            u64 all = 0;                  // this CTA's mass, then the row's
            // (top-p of the top_k needs all of these, those below min_p too)
            if (min_p > 0.f && !(top_k > 0 && top_p < 1.f)) r.t_max = fminf(r.t_max, -log2f(min_p) + 0.01f);
            if (top_k > 0) {
                // the k-th highest of the threads' maxima, to a bin
                s.count[0][tid] = 0;
                __syncthreads();
                const float t = r.c.t(thread_top);
                if (t < 63.f) atomicAdd(&s.count[0][fixed(t) >> 23], 1u);
                __syncthreads();
                uint32_t k = s.count[0][tid];
                const uint32_t own = k;
                u64 none = 0;
                block_scan(s, k, none);
                if (tid == 0) s.border.found = 0;
                __syncthreads();
                if (own && k >= uint32_t(top_k) && k - own < uint32_t(top_k)) {
                    s.border.found = 1;
                    s.border.digit = tid;
                }
                __syncthreads();
                if (s.border.found) r.t_max = fminf(r.t_max, float(s.border.digit + 1) * 0.125f + 1e-5f);
            } else if (top_p < 1.f) {
                u64 mass = 0;
                for (int j = tid; j < n; j += kST) {
                    const float l = float(share[j]);
                    if (r.c.t(l) < 125.f) mass += mass_of(r.c.weight(l));
                }
                all = block_sum(s, mass);
                const float least = (1.f - top_p) * (float(all) * (1.f / kUnit)) / float(a.V);
                if (least > 0.f) r.t_max = fminf(r.t_max, -log2f(least) + 0.01f);
            }
            // ---- their list ----
            for (int j0 = 0; j0 < n; j0 += kST) {
                const int j = j0 + tid;
                const bool yes = j < n && r.c.t(float(share[j])) <= r.t_max;
                const uint32_t who = __ballot_sync(0xffffffffu, yes);
                if (!who) continue;
                uint32_t at = 0;
                if ((tid & 31) == 0) at = atomicAdd(&s.n_cand, uint32_t(__popc(who)));
                at = __shfl_sync(0xffffffffu, at, 0) + __popc(who & ((1u << (tid & 31)) - 1));
                if (yes && at < kCand) s.cand[at] = uint32_t(j);
            }
            __syncthreads();
            r.listed = s.n_cand <= kCand;
            // the lists to the first CTA, where they fit
            Shared *first = cl.map_shared_rank(&s, 0);
            if (tid == 0) {
                s.scan[0] = atomicAdd(&first->list_n, s.n_cand);
                s.ex[1].z = all;
            }
            __syncthreads();
            const uint32_t base = s.scan[0];
            if (base + s.n_cand <= kList)
                for (int i = tid; i < int(s.n_cand); i += kST) {
                    const uint32_t j = s.cand[i];
                    const float l = float(share[j]);
                    first->list_l[base + i] = l;
                    first->list_id[base + i] = uint32_t(lo) + j;
                    first->list_mass[base + i] = mass_of(r.c.weight(l));
                }
            cl.sync();
            all = 0;
            for (int i = 0; i < a.split; ++i) all += cl.map_shared_rank(&s.ex[1], i)->z;
            const uint32_t m = first->list_n;
            const u64 want = u64(double(top_p) * double(all));
            if (m <= kList) {
                if (rank == 0) {
                    // two threads per id: its rank, and the mass before it
                    const int i = tid >> 1;
                    const bool mine = i < int(m);
                    const uint32_t my_id = mine ? s.list_id[i] : 0;
                    const float e = mine ? u[my_id] : 0.5f, w = mine ? r.c.weight(s.list_l[i]) : 0.f;
                    const u64 my = mine ? place(s.list_l[i], my_id) : ~0ull;
                    uint32_t before = 0;
                    u64 mass = 0;
                    for (int j = tid & 1; j < int(m); j += 2)
                        if (place(s.list_l[j], s.list_id[j]) < my) ++before, mass += s.list_mass[j];
                    before += __shfl_xor_sync(0xffffffffu, before, 1);
                    mass += __shfl_xor_sync(0xffffffffu, mass, 1);
                    bool keep = mine && (top_k == 0 || before < uint32_t(top_k)) && w >= min_p;
                    if (top_p < 1.f) {
                        u64 bound = want;
                        if (top_k > 0)
                            bound = u64(double(top_p) *
                                        double(block_sum(s, mine && !(tid & 1) && before < uint32_t(top_k) ? s.list_mass[i] : 0)));
                        keep = keep && (mass < bound || before == 0);
                    }
                    const bool one = keep && !(tid & 1);
                    z = block_sum(s, one ? s.list_mass[i] : 0);
                    const u64 key = one ? argmax_key(__fdividef(w, -logf(e)), my_id) : 0, high = block_max(s, key);
                    if (key && key == high) s.ex[0].w = w;
                    if (a.dist) {
                        const u64 worst = block_max(s, keep ? my : 0);
                        if (tid == 0) s.cut = worst, s.cut_mass = z;
                    }
                    __syncthreads();
                    token = argmax_key_index(high);
                    prob = s.ex[0].w / (float(z) * (1.f / kUnit));
                }
                if (a.dist) {
                    cl.sync();
                    last = first->cut;
                    z = first->cut_mass;
                }
            } else {
                u64 mass = all;
                if (top_k > 0) last = find_cut(r, false, u64(top_k), ~0ull, mass);
                if (top_p < 1.f) {
                    const u64 up_to = top_k > 0 ? u64(double(top_p) * double(mass)) : want;
                    u64 none;
                    const u64 p_last = find_cut(r, true, up_to > 0 ? up_to : 1, last, none);
                    last = p_last < last ? p_last : last;
                }
                // the race over the kept ids
                float won = -1.f, won_w = 0.f;
                int who = -1;
                mass = 0;
                r.each([&](float l, uint32_t v) {
                    if (place(l, v) > last) return;
                    const float w = r.c.weight(l);
                    if (w < min_p) return;
                    mass += mass_of(w);
                    const float y = __fdividef(w, -logf(u[v]));
                    if (y > won || (y == won && int(v) < who)) won = y, won_w = w, who = int(v);
                });
                const u64 key = who >= 0 ? argmax_key(won, uint32_t(who)) : 0, high = block_max(s, key);
                if (key && key == high) s.ex[2].w = won_w;
                mass = block_sum(s, mass);
                if (tid == 0) s.ex[2].best = high, s.ex[2].z = mass;
                cl.sync();
                u64 win = 0;
                float ww = 0.f;
                for (int i = 0; i < a.split; ++i) {
                    const Exchange *x = cl.map_shared_rank(&s.ex[2], i);
                    z += x->z;
                    if (x->best > win) win = x->best, ww = x->w;
                }
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
    const size_t smem = (size_t(a.per) * sizeof(T) + 15) / 16 * 16;
    cudaError_t e = cudaFuncSetAttribute(k_sample<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kShareBytes);
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
    // as many CTAs as a share needs; more while every row's cluster runs at once and a
    // share has 2048 ids or more
    int split = 1;
    auto per = [&](int n) { return (vocab + n - 1) / n; };
    while ((long long)per(split) * size > kShareBytes) split *= 2;
    for (int i = 0; i < 4; ++i)
        if (split == 1 << i && vocab >= 4096 * split && n_rows <= kClustersFit[i]) split *= 2;
    a.split = split;
    a.per = per(split);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    switch (dtype) {
    case GPT2_F32: return spec_rc(run<float>(a, n_rows, s));
    case GPT2_F16: return spec_rc(run<__half>(a, n_rows, s));
    default: return spec_rc(run<__nv_bfloat16>(a, n_rows, s));
    }
}
