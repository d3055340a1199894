// gpt2_op_verify_tree: which drafted nodes the target accepts, and the token
// after them.
//
// Two kernels.  k_row_stats reads every logit once and leaves, per chunk of a
// row, the maximum and the sum of exp((l - max) / temperature) (or the argmax
// key): it is bound by HBM.  k_verify, one cluster of CTAs per sequence, joins
// the chunks, looks up every node's probability at its parent, walks the tree
// in one thread, and draws the next token with all threads: of the rows, only
// the last node's is read again (and its draft distribution and the sequence's
// random numbers once).  A rejected child that has a sibling behind it costs
// one more pass over the row, for the sum that makes the rest a distribution.
//
// What bounds it, at a vocabulary of 50,257: 64 chains of 8 nodes 28.7 us (4.0
// TB/s; greedy 18.1): 18 for the rows (90 MB at 5.0 TB/s) and the walks, 10 for the
// draws, whose loads begin where a walk ends and whose logarithms and keys cost half
// of it, and none of which begins before every sequence's rows have been read;
// one chain of 6 nodes 7.8 to 8.4 us, 8 trees of 8 10.5 to 11.5 (greedy chains of 8:
// 4.9, 5.6): two launches and a chain of dependent steps (first, tokens, logits;
// sums; walk; row and random numbers; the cluster's join).
//
// Rounding: everything is fp32 (a few units in the last place; the sums over
// the vocabulary are of a few dozen terms per thread, then pairwise or in 64
// bits), so a decision can differ from the exact one where a random number
// falls within about 1e-6 of its border.  After a rejected child of probability
// r, what is left, 1 - r or the sum of max(p - q, 0), has cancelled: it is off by some
// 3e-7 / (1 - r) relatively, and so are its siblings' borders (3e-5 for r = 0.99);
// the distribution of the tokens, in which that child's r weighs as much, moves by
// 1e-6 at most.
#include <cooperative_groups.h>

#include <algorithm>
#include <cfloat>
#include <cmath>

#include "common.cuh"
#include "spec.h"

namespace gpt2 {
namespace {

// (64 chains of 8 rows of 50,257: 28.4 us in all; 256 threads 29.1, 512 31.6; half the chunk 28.5)
constexpr int kChunk = 8192;       // logits per CTA of k_row_stats
constexpr int kStatThreads = 128;
constexpr int kVec = kChunk / 4 / kStatThreads;   // 16-byte loads in flight per thread
constexpr int kVThreads = 512;
constexpr int kMaxCluster = 16;
constexpr int kBatch = 8;          // ids whose loads a thread has in flight together

struct Stat {
    float m, z;                    // maximum, sum of exp((l - m) / T)
    unsigned long long key;        // temperature 0: argmax key
};

struct VerifyArgs {
    const float *logits, *draft, *u_accept, *u_draw;
    const int32_t *tokens, *parents, *first;
    int32_t *path, *n_path, *next_token;
    Stat *stats;                   // [n_rows][chunks]
    int32_t V, n_seqs, n_rows, max_nodes, chunks, cluster;
    float c_hi, c_lo;              // log2(e) / temperature as two fp32 parts; 0: greedy
};

// exp(d / temperature) for d <= 0, 0 for -infinity (the two parts, both
// positive, keep the exponent's scale to 47 bits; the exponent itself is
// rounded once).
__device__ __forceinline__ float weight(const VerifyArgs &a, float d)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(fmaf(d, a.c_hi, d * a.c_lo)));
    return y;
}
__device__ __forceinline__ float weight(const VerifyArgs &a, float d, float rest)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(fmaf(d, a.c_hi, fmaf(rest, a.c_hi, d * a.c_lo))));
    return y;
}

__global__ void __launch_bounds__(kStatThreads) k_row_stats(const VerifyArgs a)
{
    __shared__ float red[kStatThreads / 32];
    __shared__ unsigned long long keys[kStatThreads / 32];
    pdl_wait();
    pdl_launch_dependents();                       // (k_verify reads the call's inputs from then on)
    const int row = blockIdx.x, chunk = blockIdx.y, tid = threadIdx.x;
    if (row >= min(max(a.first[a.n_seqs], 0), a.n_rows)) return;
    // chunks of a row: equal shares, a multiple of 4
    const int per = ((a.V + a.chunks - 1) / a.chunks + 3) / 4 * 4;
    const int lo = min(chunk * per, a.V), hi = min(lo + per, a.V);
    const float *p = a.logits + size_t(row) * a.V + lo;
    const int n = hi - lo;
    // up to three values before a 16-byte boundary, then whole vectors, then the rest
    const int head = min(n, int((16 - reinterpret_cast<uintptr_t>(p) % 16) / 4 % 4));
    const int n4 = (n - head) / 4, rest = head + n4 * 4;
    const float4 *p4 = reinterpret_cast<const float4 *>(p + head);
    float v[kVec + 1][4];
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        const int k = tid + i * kStatThreads;
        float4 x = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        if (k < n4) x = __ldcs(p4 + k);
        v[i][0] = x.x, v[i][1] = x.y, v[i][2] = x.z, v[i][3] = x.w;
    }
    v[kVec][0] = tid < head ? p[tid] : -INFINITY;
    v[kVec][1] = tid < n - rest ? p[rest + tid] : -INFINITY;
    v[kVec][2] = v[kVec][3] = -INFINITY;
    Stat *out = a.stats + size_t(row) * a.chunks + chunk;
    if (a.c_hi == 0.f) {
        // in order of the ids, so that the lowest of equals stays (a NaN or
        // -infinity is never above)
        float top = -INFINITY;
        int id = -1;
        auto take = [&](float x, int i) {
            if (x > top) top = x, id = i;
        };
        take(v[kVec][0], tid);
#pragma unroll
        for (int i = 0; i < kVec; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) take(v[i][j], head + (tid + i * kStatThreads) * 4 + j);
        take(v[kVec][1], rest + tid);
        unsigned long long best = id >= 0 ? argmax_key(top + 0.f, uint32_t(lo + id)) : 0;   // (-0 as 0: they tie)
        best = warp_max_u64(best);
        if ((tid & 31) == 0) keys[tid >> 5] = best;
        __syncthreads();
        if (tid == 0) {
            for (int w = 1; w < kStatThreads / 32; ++w) best = keys[w] > best ? keys[w] : best;
            *out = Stat{0.f, 0.f, best};
        }
        return;
    }
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i <= kVec; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) m = fmaxf(m, v[i][j]);
    m = warp_max(m);
    if ((tid & 31) == 0) red[tid >> 5] = m;
    __syncthreads();
    for (int w = 0; w < kStatThreads / 32; ++w) m = fmaxf(m, red[w]);
    __syncthreads();
    float z = 0.f;
    const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int i = 0; i <= kVec; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) z += weight(a, v[i][j] - ref);   // (NaN and +infinity leave a NaN)
    z = warp_sum(z);
    if ((tid & 31) == 0) red[tid >> 5] = z;
    __syncthreads();
    if (tid == 0) {
        for (int w = 1; w < kStatThreads / 32; ++w) z += red[w];
        *out = Stat{m, z, 0};
    }
}

// What the walk of a sequence has come to; thread 0 of every CTA of the
// cluster computes the same.
struct Walk {
    unsigned long long children[GPT2_MAX_NODES];
    float prob[GPT2_MAX_NODES];        // p(token) at the parent
    float q[GPT2_MAX_NODES], u[GPT2_MAX_NODES];
    float m[GPT2_MAX_NODES], inv_z[GPT2_MAX_NODES];
    int choice[GPT2_MAX_NODES];        // temperature 0
    int token[GPT2_MAX_NODES];
    bool valid[GPT2_MAX_NODES];
    // nodes that can be tried (token and parent's logits are sound), and those
    // of them that are accepted if no sibling was rejected before
    unsigned long long usable, first_ok;
    // children of `cur` rejected so far: their tokens (draft on one token), or
    // 1 / the sums that bring what is left back to a distribution
    int rejected[GPT2_MAX_NODES];
    float inv_mass[GPT2_MAX_NODES];    // (0 where nothing is left)
    int n_rejected, cur, length, path[GPT2_MAX_NODES];
    float scale;                       // draft on one token: 1 / what is left
    unsigned long long left;           // children of cur not tried yet
    bool need_mass, dead;
};

// Goes on until the walk ends (need_mass false) or a sum over the vocabulary
// is needed (need_mass true; inv_mass[n_rejected - 1] is then to be set).
__device__ void walk_on(const VerifyArgs &a, Walk &w)
{
    w.need_mass = false;
    const unsigned long long usable = w.usable, first_ok = w.first_ok;
    unsigned long long left = w.left;
    while (left &= usable) {
        const int i = __ffsll((long long)left) - 1;
        left &= left - 1;
        bool yes;
        float r = 0.f;
        if (w.n_rejected == 0) {
            yes = first_ok >> i & 1;
            r = w.prob[i];
        } else {
            const int x = w.token[i];
            r = w.prob[i];
            if (a.draft) {
                for (int k = 0; k < w.n_rejected; ++k) r = fmaxf(r - w.q[i], 0.f) * w.inv_mass[k];
            } else {
                r = w.dead ? 0.f : r * w.scale;
                for (int k = 0; k < w.n_rejected; ++k)
                    if (w.rejected[k] == x) r = 0.f;
            }
            yes = w.u[i] * w.q[i] < r;
        }
        if (yes) {
            w.path[w.length++] = i;
            w.cur = i;
            left = w.children[i];
            w.n_rejected = 0;
            w.scale = 1.f;
            w.dead = false;
        } else if (a.c_hi != 0.f) {
            w.rejected[w.n_rejected] = w.token[i];
            w.inv_mass[w.n_rejected++] = 1.f;
            if (!a.draft) {
                const float rest = 1.f - r;
                if (rest > 0.f) w.scale *= __frcp_rn(rest);
                else w.dead = true;
            } else if (left & usable) {
                w.need_mass = true;
                break;
            }
        }
    }
    w.left = left;
}

__global__ void __launch_bounds__(kVThreads) k_verify(const VerifyArgs a)
{
    namespace cg = cooperative_groups;
    __shared__ Walk w;
    __shared__ double red[kVThreads / 32];
    __shared__ unsigned long long keys[kVThreads / 32];
    __shared__ double part_sum[2];                 // this CTA's share, for the cluster (two rounds in flight)
    __shared__ unsigned long long part_key[2];
    const int b = blockIdx.x / a.cluster, rank = blockIdx.x % a.cluster;
    const int tid = threadIdx.x;
    const int f0 = min(max(a.first[b], 0), a.n_rows), f1 = min(max(a.first[b + 1], f0), a.n_rows);
    const int nodes = min(f1 - f0, a.max_nodes);
    int parent = -1;
    if (tid < GPT2_MAX_NODES) {
        w.children[tid] = 0;
        if (tid > 0 && tid < nodes) parent = a.parents[f0 + tid];
        if (tid < nodes) w.token[tid] = a.tokens[f0 + tid];
        if (tid == 0) w.usable = w.first_ok = 0;
    }
    __syncthreads();
    // What is read before the wait are the call's inputs, which k_row_stats does not
    // write.  They are complete: this kernel is launched right behind k_row_stats, and
    // can start only when all of that one's CTAs have passed their own wait for
    // whatever was before.
    float lx = 0.f, qx = 1.f, ux = 0.f;            // of this thread's node: target's logit at its parent, draft's, random number
    if (parent >= 0 && parent < tid) {
        atomicOr(&w.children[parent], 1ull << tid);
        const int x = w.token[tid];
        if (a.c_hi != 0.f && x >= 0 && x < a.V) {
            const size_t at = size_t(f0 + parent) * a.V + x;
            lx = a.logits[at];
            ux = a.u_accept[f0 + tid];
            if (a.draft) qx = a.draft[at];
        }
    }
    if (a.c_hi != 0.f) {                           // the random numbers of the final draw, into L2
        const int share = (a.V + a.cluster - 1) / a.cluster, to = min(a.V, (rank + 1) * share);
        for (int v = rank * share + tid * 32; v < to; v += kVThreads * 32)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(a.u_draw + size_t(b) * a.V + v));
    }
    pdl_wait();                                    // k_row_stats' sums
    // eight threads per node join its chunks
    for (int i0 = 0; i0 < nodes; i0 += kVThreads / 8) {
        const int i = i0 + tid / 8, l = tid % 8;
        const Stat *st = a.stats + size_t(f0 + min(i, nodes - 1)) * a.chunks;
        float m = -INFINITY;
        unsigned long long key = 0;
        float z = 0.f;
        for (int k0 = 0; k0 < a.chunks; k0 += 8) {
            const Stat v = k0 + l < a.chunks ? st[k0 + l] : Stat{-INFINITY, 0.f, 0};
            float mk = v.m;
            key = v.key > key ? v.key : key;
            for (int o = 4; o > 0; o >>= 1) mk = fmaxf(mk, __shfl_xor_sync(0xffffffffu, mk, o));
            const float mn = fmaxf(m, mk);         // the same in all eight threads
            if (mn > -INFINITY) {
                if (m > -INFINITY) z *= weight(a, m - mn);
                if (v.z != 0.f) z += v.z * weight(a, v.m - mn);
            } else {
                z += v.z;                          // (0, or the NaN of a chunk without a number)
            }
            m = mn;
        }
        for (int o = 4; o > 0; o >>= 1) {
            z += __shfl_xor_sync(0xffffffffu, z, o);
            const unsigned long long other = __shfl_xor_sync(0xffffffffu, key, o);
            key = other > key ? other : key;
        }
        if (l == 0 && i < nodes) {
            if (a.c_hi == 0.f) {
                w.valid[i] = key != 0;
                w.choice[i] = key != 0 ? argmax_key_index(key) : -1;
            } else {
                w.m[i] = m;
                w.inv_z[i] = __frcp_rn(z);
                w.valid[i] = z > 0.f && fabsf(m) <= FLT_MAX;   // (false for NaN sums)
            }
        }
    }
    __syncthreads();
    if (parent >= 0 && parent < tid && w.valid[parent] && w.token[tid] >= 0 && w.token[tid] < a.V) {
        w.u[tid] = ux;
        w.q[tid] = qx;
        bool ok;
        if (a.c_hi == 0.f) {
            ok = w.choice[parent] == w.token[tid];
        } else {
            // lx - m in two parts, so that its rounding does not show (no second part
            // where the first is -infinity: a logit of -infinity, or a difference past fp32's range)
            const float m = w.m[parent], d = lx - m, t = d + m, rest = (lx - t) + (m - (t - d));
            w.prob[tid] = d >= -FLT_MAX ? weight(a, d, rest) * w.inv_z[parent] : 0.f;
            ok = ux * qx < w.prob[tid];
        }
        atomicOr(&w.usable, 1ull << tid);
        if (ok) atomicOr(&w.first_ok, 1ull << tid);
    }
    if (tid == 0) {
        w.cur = 0;
        w.length = nodes > 0 ? 1 : 0;
        w.path[0] = 0;
        w.left = nodes > 0 ? w.children[0] : 0;
        w.n_rejected = 0;
        w.scale = 1.f;
        w.dead = false;
    }
    __syncthreads();

    const cg::cluster_group cl = cg::this_cluster();
    const int per = (a.V + a.cluster - 1) / a.cluster, v0 = rank * per, v1 = min(a.V, v0 + per);
    int round = 0;
    // what is left of p at ids v, v + kVThreads, .. after n rejected children
    // (scaled by any factor)
    auto residual = [&](float (&p)[kBatch], const float (&q)[kBatch], int v, int n) {
        for (int k = 0; k < n; ++k) {
            const float inv = a.draft ? w.inv_mass[k] : w.dead ? 0.f : 1.f;
            const int x = w.rejected[k];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                if (a.draft) p[i] = fmaxf(p[i] - q[i], 0.f) * inv;
                else p[i] = x == v + i * kVThreads ? 0.f : p[i] * inv;
            }
        }
    };
    for (;;) {
        if (tid == 0) walk_on(a, w);
        __syncthreads();
        if (!w.need_mass) break;                   // (the same in every CTA of the cluster)
        const size_t row = size_t(f0 + w.cur) * a.V;
        const float m = w.m[w.cur], iz = w.inv_z[w.cur];
        const int n = w.n_rejected;
        float s = 0.f;
        for (int b0 = v0 + tid; b0 < v1; b0 += kBatch * kVThreads) {
            float x[kBatch], q[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int v = b0 + i * kVThreads;
                x[i] = v < v1 ? a.logits[row + v] : -INFINITY;
                q[i] = v < v1 ? a.draft[row + v] : 0.f;
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) x[i] = weight(a, x[i] - m) * iz;
            residual(x, q, b0, n);
#pragma unroll
            for (int i = 0; i < kBatch; ++i) s += x[i];
        }
        s = warp_sum(s);
        if ((tid & 31) == 0) red[tid >> 5] = double(s);
        __syncthreads();
        if (tid == 0) {
            double t = 0.0;
            for (int k = 0; k < kVThreads / 32; ++k) t += red[k];
            part_sum[round & 1] = t;
        }
        cl.sync();
        if (tid == 0) {
            double t = 0.0;
            for (int k = 0; k < a.cluster; ++k) t += *cl.map_shared_rank(&part_sum[round & 1], k);
            w.inv_mass[n - 1] = t > 0.0 ? __frcp_rn(float(t)) : 0.f;
        }
        ++round;
        __syncthreads();
    }

    int token = -1;
    if (nodes > 0 && w.valid[w.cur]) {             // (the same in every CTA of the cluster)
        if (a.c_hi == 0.f) {
            token = w.choice[w.cur];
        } else {
            const size_t row = size_t(f0 + w.cur) * a.V;
            const float m = w.m[w.cur], iz = w.inv_z[w.cur];
            const float *u = a.u_draw + size_t(b) * a.V;
            // the race over what is left; where nothing is, over the node's own distribution
            for (int pass = 0; pass < 2; ++pass) {
                const int n = pass == 0 ? w.n_rejected : 0;
                const bool dense = a.draft && n > 0;
                // the best value and its id; what the warp's best rules out needs no
                // logarithm (-log u >= 1 - u; the margin is far above its rounding)
                float top = -1.f, bound = -1.f;
                int id = -1;
                for (int w0 = v0; w0 < v1; w0 += kBatch * kVThreads) {
                    const int b0 = w0 + tid;
                    float x[kBatch], q[kBatch], e[kBatch];
#pragma unroll
                    for (int i = 0; i < kBatch; ++i) {
                        const int v = b0 + i * kVThreads;
                        x[i] = v < v1 ? a.logits[row + v] : -INFINITY;
                        e[i] = v < v1 ? u[v] : 0.5f;
                        q[i] = dense && v < v1 ? a.draft[row + v] : 0.f;
                    }
#pragma unroll
                    for (int i = 0; i < kBatch; ++i) x[i] = weight(a, x[i] - m) * iz;
                    residual(x, q, b0, n);
                    if (bound < 0.f) {             // (the first ones: side by side)
                        float y[kBatch];
#pragma unroll
                        for (int i = 0; i < kBatch; ++i) y[i] = __fdividef(x[i], -logf(e[i]));
#pragma unroll
                        for (int i = 0; i < kBatch; ++i)
                            if (x[i] > 0.f && y[i] > top) top = y[i], id = b0 + i * kVThreads;
                    } else {
#pragma unroll
                        for (int i = 0; i < kBatch; ++i)
                            if (x[i] > 0.f && x[i] > bound * (1.f - e[i])) {
                                const float y = __fdividef(x[i], -logf(e[i]));
                                if (y > top) top = y, id = b0 + i * kVThreads;
                            }
                    }
                    bound = warp_max(top) * 0.999f;
                }
                unsigned long long best = id >= 0 ? argmax_key(top, uint32_t(id)) : 0;
                best = warp_max_u64(best);
                if ((tid & 31) == 0) keys[tid >> 5] = best;
                __syncthreads();
                if (tid == 0) {
                    for (int k = 0; k < kVThreads / 32; ++k) best = keys[k] > best ? keys[k] : best;
                    part_key[round & 1] = best;
                }
                cl.sync();
                best = 0;
                for (int k = 0; k < a.cluster; ++k) {
                    const unsigned long long o = *cl.map_shared_rank(&part_key[round & 1], k);
                    best = o > best ? o : best;
                }
                ++round;
                if (best != 0) {
                    token = argmax_key_index(best);
                    break;
                }
                if (n == 0) break;
            }
        }
    }
    if (rank == 0) {
        if (tid < a.max_nodes) a.path[size_t(b) * a.max_nodes + tid] = tid < w.length ? w.path[tid] : -1;
        if (tid == 0) {
            a.n_path[b] = w.length;
            a.next_token[b] = token;
        }
    }
    cl.sync();                                     // nobody leaves while its shares are read
}

int chunks_of(int32_t vocab) { return (vocab + kChunk - 1) / kChunk; }

}  // namespace
}  // namespace gpt2

using namespace gpt2;

extern "C" {

size_t gpt2_op_verify_tree_workspace(int32_t n_rows, int32_t vocab)
{
    if (n_rows < 1 || vocab < 1) return 16;
    return size_t(n_rows) * chunks_of(vocab) * sizeof(Stat);
}

int gpt2_op_verify_tree(const float *logits, int32_t vocab, const int32_t *tokens, const int32_t *parents,
                        const int32_t *first, int32_t n_seqs, int32_t n_rows, int32_t max_nodes, float temperature,
                        const float *draft_probs, const float *u_accept, const float *u_draw, int32_t *path,
                        int32_t *n_path, int32_t *next_token, void *workspace, size_t workspace_bytes, void *stream)
{
    if (!logits || !tokens || !parents || !first || !path || !n_path || !next_token || !workspace)
        return GPT2_ERR_INVALID_ARG;
    if (vocab < 1 || n_seqs < 0 || n_rows < 0 || max_nodes < 1 || max_nodes > GPT2_MAX_NODES)
        return GPT2_ERR_INVALID_ARG;
    if (!(temperature >= 0.f) || !std::isfinite(temperature)) return GPT2_ERR_INVALID_ARG;
    const double c = temperature > 0.f ? 1.4426950408889634 / double(temperature) : 0.0;
    if (c > double(FLT_MAX)) return GPT2_ERR_INVALID_ARG;
    if (temperature > 0.f && (!u_accept || !u_draw)) return GPT2_ERR_INVALID_ARG;
    if (!aligned4(logits, tokens, parents, first, path, n_path, next_token) || !aligned16(workspace))
        return GPT2_ERR_INVALID_ARG;
    if (temperature > 0.f && !aligned4(draft_probs, u_accept, u_draw)) return GPT2_ERR_INVALID_ARG;
    if (workspace_bytes < gpt2_op_verify_tree_workspace(n_rows, vocab)) return GPT2_ERR_INVALID_ARG;
    if (chunks_of(vocab) > 65535 || (long long)n_seqs * kMaxCluster >= (1ll << 31)) return GPT2_ERR_INVALID_ARG;
    if (n_seqs == 0) return GPT2_OK;
    int rc;
    const int sms = spec_sms(&rc);
    if (!sms) return rc;
    VerifyArgs a{};
    a.logits = logits;
    a.tokens = tokens;
    a.parents = parents;
    a.first = first;
    a.path = path;
    a.n_path = n_path;
    a.next_token = next_token;
    a.stats = static_cast<Stat *>(workspace);
    a.V = vocab;
    a.n_seqs = n_seqs;
    a.n_rows = n_rows;
    a.max_nodes = max_nodes;
    a.chunks = chunks_of(vocab);
    a.cluster = 1;
    if (temperature > 0.f) {
        a.draft = draft_probs;
        a.u_accept = u_accept;
        a.u_draw = u_draw;
        a.c_hi = std::nextafterf(float(c), 0.f);    // below c, so that the rest is positive
        a.c_lo = std::max(float(c - double(a.c_hi)), FLT_TRUE_MIN);   // (and not zero, for the largest temperatures)
        // the final draw reads a row with the CTAs of a cluster: as many as
        // keep 2048 ids or more each, while all sequences' clusters run at once (of
        // 16 CTAs one per SM: 8 trees of 8 took 11.5 us with 16, 10.5 with 8, on one GPU in turn)
        for (int i = 0; i < 4 && vocab >= 4096 * a.cluster && n_seqs <= kClustersFit[i] * (i == 3 ? 1 : 2); ++i) a.cluster *= 2;
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (n_rows > 0) {
        rc = spec_rc(spec_launch(k_row_stats, dim3(n_rows, a.chunks), kStatThreads, 0, 1, s, a));
        if (rc != GPT2_OK) return rc;
    }
    if (a.cluster > 8) {
        rc = spec_rc(cudaFuncSetAttribute(k_verify, cudaFuncAttributeNonPortableClusterSizeAllowed, 1));
        if (rc != GPT2_OK) return rc;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(n_seqs) * a.cluster);
    cfg.blockDim = dim3(kVThreads);
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = unsigned(a.cluster);
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = n_rows > 0 ? 1 : 0;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return spec_rc(cudaLaunchKernelEx(&cfg, k_verify, a));
}

}  // extern "C"
