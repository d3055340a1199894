// gpt2_op_page_map: the block tables and the slot map of a step's tokens, from
// the requests' lengths.
//
// All of it is prefix sums over the sequences: of the tokens (where a
// sequence's rows begin), of the blocks that they need (which free block each
// gets, and who still gets one), and of the blocks that leaving sequences give
// back.  Every CTA makes the same sums in shared memory, which costs less than
// sharing them, and the CTAs then split the rows, the new table entries and the
// returned blocks; a row finds its sequence by binary search.  Where the lengths are
// updated in place the CTAs are one cluster, whose barrier lies between the last
// read of them and the first write; blocks are taken from one end of the ring and given
// back at the other, and tables grow behind what is read, so nothing else is
// both read and written.  What bounds it is latency: a launch, one load of the
// lengths, three scans, a search and one dependent load per row (64 rows 4.5 us, 16,384 rows 5.5,
// whose bytes would take 0.04).
#include <cooperative_groups.h>

#include "common.cuh"
#include "spec.h"

namespace gpt2 {
namespace {

constexpr int kMapThreads = 512;      // (1024: 64 rows 7.2 us instead of 4.3)
constexpr int kMapCluster = 8;        // CTAs at most, in place
constexpr int kMapCtas = 128;         // ... otherwise
constexpr int kRowsPerCta = 256;      // rows that are worth another CTA (of 1024: 16,384 rows 6.2 us instead of 5.4)

struct MapArgs {
    const int32_t *cached, *grow, *free_state;
    int32_t *table, *ring, *cached_out, *free_state_out, *first, *seq, *slot, *offset, *position;
    int32_t n_seqs, block, max_blocks, n_blocks, n_rows, in_place;
};

typedef unsigned long long u64;

// Inclusive prefix sums of one value per thread, and their total.
__device__ __forceinline__ u64 block_scan(u64 v, u64 *warp_sums, u64 &total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const u64 w = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += w;
    }
    if (lane == 31) warp_sums[warp] = v;
    __syncthreads();
    u64 before = 0, all = 0;
#pragma unroll
    for (int i = 0; i < kMapThreads / 32; ++i) {
        if (i < warp) before += warp_sums[i];
        all += warp_sums[i];
    }
    total = all;
    __syncthreads();                  // (warp_sums may be written again)
    return v + before;
}

// The first index whose inclusive sum is above x (n: none).
__device__ __forceinline__ int above(const uint32_t *sums, int n, uint32_t x)
{
    int lo = 0, hi = n;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (sums[mid] > x) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

__global__ void __launch_bounds__(kMapThreads) k_page_map(const MapArgs a)
{
    namespace cg = cooperative_groups;
    // per sequence: inclusive sums of tokens, blocks taken and blocks given back (cut
    // off just above what there is room for), and the cached length, with the
    // top bit where the sequence's tokens are not served
    extern __shared__ uint32_t dyn[];
    __shared__ u64 warp_sums[kMapThreads / 32];
    __shared__ uint32_t s_used;
    const int n = a.n_seqs, tid = threadIdx.x;
    uint32_t *end = dyn, *taken = dyn + n, *given = dyn + 2 * n, *len = dyn + 3 * n;
    const uint32_t bs = a.block, cap = uint32_t(a.max_blocks) * bs;
    pdl_wait();
    pdl_launch_dependents();

    const int32_t nb = a.n_blocks;
    const uint32_t count = uint32_t(min(max(a.free_state[1], 0), nb));
    const int32_t h = a.free_state[0] % nb;
    const uint32_t head = uint32_t(h < 0 ? h + nb : h), room = uint32_t(nb) - count;
    if (tid == 0) s_used = 0;

    const int per = (n + kMapThreads - 1) / kMapThreads, b0 = min(tid * per, n), b1 = min(b0 + per, n);
    u64 tokens = 0, back = 0, total;
    for (int b = b0; b < b1; ++b) {
        const int32_t g = a.grow[b];
        const uint32_t c = min(uint32_t(max(a.cached[b], 0)), cap);
        len[b] = c;
        tokens += uint32_t(max(g, 0));
        back += g < 0 ? (c + bs - 1) / bs : 0;
        end[b] = uint32_t(g);         // (until its sum replaces it)
    }
    u64 t_at = block_scan(tokens, warp_sums, total) - tokens;
    u64 g_at = block_scan(back, warp_sums, total) - back;
    const uint32_t released = uint32_t(min(total, u64(room)));
    u64 need = 0;
    for (int b = b0; b < b1; ++b) {
        const int32_t g = int32_t(end[b]);
        const uint32_t c = len[b], more = uint32_t(max(g, 0)), have = (c + bs - 1) / bs;
        t_at += more;
        g_at += g < 0 ? have : 0;
        end[b] = uint32_t(min(t_at, u64(a.n_rows) + 1));
        given[b] = uint32_t(min(g_at, u64(released)));
        // (c + more <= cap keeps the sum in 32 bits)
        const bool fits = g >= 0 && t_at <= u64(a.n_rows) && more <= cap - c;
        const uint32_t want = fits ? (c + more + bs - 1) / bs - have : 0;
        need += want;
        taken[b] = want;
        if (!fits) len[b] |= 0x80000000u;
        if (g < 0) len[b] |= 0x40000000u;
    }
    u64 n_at = block_scan(need, warp_sums, total) - need;
    uint32_t used = 0;
    for (int b = b0; b < b1; ++b) {
        const uint32_t want = taken[b];
        n_at += want;
        if (n_at <= count) used = uint32_t(n_at);
        else if (want) len[b] |= 0x80000000u;
        taken[b] = uint32_t(min(n_at, u64(count) + 1));
    }
    if (used) atomicMax(&s_used, used);
    if (a.in_place) cg::this_cluster().sync();   // the lengths have been read, and these sums are there
    else __syncthreads();
    used = s_used;

    const int rank = blockIdx.x, at = rank * kMapThreads + tid, step = gridDim.x * kMapThreads;
    constexpr uint32_t kLen = 0x3fffffffu, kUnserved = 0x80000000u, kLeaves = 0x40000000u;
    for (int b = at; b < n; b += step) {
        const uint32_t l = len[b], rows = end[b] - (b ? end[b - 1] : 0);
        a.cached_out[b] = l & kLeaves ? 0 : int32_t((l & kLen) + (l & kUnserved ? 0 : rows));
        a.first[b + 1] = int32_t(min(end[b], uint32_t(a.n_rows)));
    }
    if (at == 0) {
        a.first[0] = 0;
        a.free_state_out[0] = int32_t((u64(head) + used) % uint32_t(nb));
        a.free_state_out[1] = int32_t(count - used + released);
    }
    auto ring_at = [&](uint32_t j) { return uint32_t((u64(head) + j) % uint32_t(nb)); };
    for (uint32_t j = at; j < used; j += step) {
        const int b = above(taken, n, j);
        const uint32_t have = ((len[b] & kLen) + bs - 1) / bs, k = have + j - (b ? taken[b - 1] : 0);
        a.table[size_t(b) * a.max_blocks + k] = a.ring[ring_at(j)];
    }
    for (uint32_t j = at; j < released; j += step) {
        const int b = above(given, n, j);
        a.ring[ring_at(count + j)] = a.table[size_t(b) * a.max_blocks + j - (b ? given[b - 1] : 0)];
    }
    const uint32_t last = n ? end[n - 1] : 0;
    for (uint32_t i = at; i < uint32_t(a.n_rows); i += step) {
        int32_t seq = -1, slot = -1, offset = -1, position = -1;
        if (i < last) {
            seq = above(end, n, i);
            const uint32_t l = len[seq];
            if (!(l & kUnserved)) {
                const uint32_t c = l & kLen, p = c + i - (seq ? end[seq - 1] : 0), k = p / bs, have = (c + bs - 1) / bs;
                slot = k < have ? a.table[size_t(seq) * a.max_blocks + k]
                                : a.ring[ring_at((seq ? taken[seq - 1] : 0) + k - have)];
                offset = int32_t(p - k * bs);
                position = int32_t(p);
            }
        }
        a.seq[i] = seq;
        a.slot[i] = slot;
        a.offset[i] = offset;
        a.position[i] = position;
    }
}

}  // namespace
}  // namespace gpt2

using namespace gpt2;

extern "C" int gpt2_op_page_map(const int32_t *cached, const int32_t *grow, int32_t n_seqs, int32_t block_size,
                                int32_t *table, int32_t max_blocks, int32_t *free_blocks, int32_t n_blocks,
                                const int32_t *free_state, int32_t *cached_out, int32_t *free_state_out, int32_t *first,
                                int32_t *seq, int32_t *slot, int32_t *offset, int32_t *position, int32_t n_rows,
                                void *stream)
{
    if (!cached || !grow || !table || !free_blocks || !free_state || !cached_out || !free_state_out || !first)
        return GPT2_ERR_INVALID_ARG;
    if (n_seqs < 0 || n_seqs > GPT2_MAX_PAGED_SEQS || n_rows < 0 || block_size < 1 || max_blocks < 1 || n_blocks < 1)
        return GPT2_ERR_INVALID_ARG;
    if (n_rows > 0 && (!seq || !slot || !offset || !position)) return GPT2_ERR_INVALID_ARG;
    if ((long long)block_size * max_blocks >= (1ll << 30)) return GPT2_ERR_INVALID_ARG;
    if (!aligned4(cached, grow, table, free_blocks, free_state, cached_out, free_state_out, first, seq, slot, offset,
                  position))
        return GPT2_ERR_INVALID_ARG;
    int rc;
    if (!spec_sms(&rc)) return rc;
    const bool in_place = cached_out == cached || free_state_out == free_state;
    const MapArgs a{cached, grow,   free_state, table,  free_blocks, cached_out, free_state_out, first,     seq,
                    slot,   offset, position,   n_seqs, block_size,  max_blocks, n_blocks,       n_rows,
                    in_place};
    int ctas = 1;
    while (ctas < (in_place ? kMapCluster : kMapCtas) && (long long)ctas * kRowsPerCta < n_rows) ctas *= 2;
    const size_t smem = size_t(n_seqs) * 16;
    if (smem > 48 * 1024) {
        rc = spec_rc(cudaFuncSetAttribute(k_page_map, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                          GPT2_MAX_PAGED_SEQS * 16));
        if (rc != GPT2_OK) return rc;
    }
    return spec_rc(spec_launch(k_page_map, dim3(ctas), kMapThreads, smem, in_place ? ctas : 1,
                              static_cast<cudaStream_t>(stream), a));
}
