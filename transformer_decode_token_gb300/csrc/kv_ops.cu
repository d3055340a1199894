// The quantised key/value cache: rows written into it, read back, and the
// accepted path of a tree of drafted tokens moved into place.  All three only
// move data (a few operations per value), so HBM bounds them at prompt sizes
// and the launch at decode sizes.
#include <cfloat>
#include <type_traits>

#include <cuda_fp8.h>

#include "common.cuh"
#include "spec.h"

namespace gpt2 {

int spec_sms(int *rc)
{
    constexpr int kMaxDevices = 64;
    static int sms[kMaxDevices];   // 0: not looked up; written with the same value by every thread
    int dev = 0;
    *rc = spec_rc(cudaGetDevice(&dev));
    if (*rc != GPT2_OK) return 0;
    if (dev < 0 || dev >= kMaxDevices) {
        *rc = GPT2_ERR_UNSUPPORTED_DEVICE;
        return 0;
    }
    int n = __atomic_load_n(&sms[dev], __ATOMIC_RELAXED);
    if (n == 0) {
        int major = 0, minor = 0;
        cudaError_t e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
        if (e == cudaSuccess) e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
        if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
        *rc = spec_rc(e);
        if (*rc == GPT2_OK && !(major == 10 && minor == 3)) *rc = GPT2_ERR_UNSUPPORTED_DEVICE;
        if (*rc != GPT2_OK) return 0;
        __atomic_store_n(&sms[dev], n, __ATOMIC_RELAXED);
    }
    return n;
}

namespace {

constexpr int kVals = 8;   // values of a row per thread: 32, 16 or 8 bytes in one or two accesses

struct RowArgs {
    gpt2_kv kv;
    const void *src_k, *src_v; // store: rows
    void *dst_k, *dst_v;       // load: rows
    int64_t stride;
    const int32_t *slot, *pos;
    int32_t n_rows;
};

// A thread's kVals values of a row are two pieces of four.  Where the rows or
// the cache are fp32 the pieces lie half a row apart, so that the 16-byte
// accesses of neighbouring threads follow one another and fill whole sectors
// (8 consecutive fp32 values per thread wrote half sectors: 1.7 times as long for
// 17,408 rows of 12 x 64 int8 read back as fp32); else they are
// neighbours.
template <typename T, typename CT>
constexpr bool kApart = sizeof(T) == 4 || sizeof(CT) == 4;

// The row's first element of thread l, and the distance of its pieces.
template <bool APART>
__device__ __forceinline__ uint32_t piece_at(uint32_t l)
{
    return l * (APART ? 4 : kVals);
}
template <bool APART>
__device__ __forceinline__ uint32_t piece_step(uint32_t D)
{
    return APART ? D / 2 : 4;
}

// The bits of a thread's values of type T at p (and p + step), in words.
template <typename T>
union Words {
    uint32_t w[kVals * sizeof(T) / 4];
    T t[kVals];
    __device__ Words() {}
};

template <typename T, bool APART, bool STREAM>
__device__ __forceinline__ void get_words(const T *p, uint32_t step, Words<T> &x)
{
    auto get = [](const auto *q) {
        if constexpr (STREAM) return __ldcs(q);
        else return *q;
    };
    if constexpr (!APART && sizeof(T) == 2) {
        const uint4 a = get(reinterpret_cast<const uint4 *>(p));
        x.w[0] = a.x, x.w[1] = a.y, x.w[2] = a.z, x.w[3] = a.w;
    } else if constexpr (!APART && sizeof(T) == 1) {
        const uint2 a = get(reinterpret_cast<const uint2 *>(p));
        x.w[0] = a.x, x.w[1] = a.y;
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const T *q = p + h * step;
            if constexpr (sizeof(T) == 4) {
                const uint4 a = get(reinterpret_cast<const uint4 *>(q));
                x.w[4 * h] = a.x, x.w[4 * h + 1] = a.y, x.w[4 * h + 2] = a.z, x.w[4 * h + 3] = a.w;
            } else if constexpr (sizeof(T) == 2) {
                const uint2 a = get(reinterpret_cast<const uint2 *>(q));
                x.w[2 * h] = a.x, x.w[2 * h + 1] = a.y;
            } else {
                x.w[h] = get(reinterpret_cast<const uint32_t *>(q));
            }
        }
    }
}

template <typename T, bool APART>
__device__ __forceinline__ void put_words(T *p, uint32_t step, const Words<T> &x)
{
    if constexpr (!APART && sizeof(T) == 2) {
        *reinterpret_cast<uint4 *>(p) = make_uint4(x.w[0], x.w[1], x.w[2], x.w[3]);
    } else if constexpr (!APART && sizeof(T) == 1) {
        *reinterpret_cast<uint2 *>(p) = make_uint2(x.w[0], x.w[1]);
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            T *q = p + h * step;
            if constexpr (sizeof(T) == 4)
                *reinterpret_cast<uint4 *>(q) = make_uint4(x.w[4 * h], x.w[4 * h + 1], x.w[4 * h + 2], x.w[4 * h + 3]);
            else if constexpr (sizeof(T) == 2)
                *reinterpret_cast<uint2 *>(q) = make_uint2(x.w[2 * h], x.w[2 * h + 1]);
            else
                *reinterpret_cast<uint32_t *>(q) = x.w[h];
        }
    }
}

// A row's values as fp32, and back (rounded to nearest even); VEC: the accesses
// above are aligned.
template <typename T, bool APART, bool VEC>
__device__ __forceinline__ void get_vals(const T *p, uint32_t step, float (&x)[kVals])
{
    Words<T> w;
    if constexpr (VEC) {
        get_words<T, APART, true>(p, step, w);
    } else {
#pragma unroll
        for (int j = 0; j < kVals; ++j) w.t[j] = p[j / 4 * step + j % 4];
    }
#pragma unroll
    for (int j = 0; j < kVals; ++j) x[j] = float(w.t[j]);
}

template <typename T, bool APART, bool VEC>
__device__ __forceinline__ void put_vals(T *p, uint32_t step, const float (&x)[kVals])
{
    Words<T> w;
#pragma unroll
    for (int j = 0; j < kVals; ++j) w.t[j] = T(x[j]);
    if constexpr (VEC) {
        put_words<T, APART>(p, step, w);
    } else {
#pragma unroll
        for (int j = 0; j < kVals; ++j) p[j / 4 * step + j % 4] = w.t[j];
    }
}

// Codes of kVals values, the integers nearest x / s (|x| <= 127 s (1 + 2^-22)),
// ties to even, of the exact quotient and not of a rounded one.  Adding 1.5 *
// 2^23 to x * (1/s) rounds it to an integer q, whose two's complement is then
// the low byte of the sum; q is at most one off.  The remainder x - q s is
// exact in one fused multiply-add (a multiple of half an ulp of s, and no
// larger than about s/2), so q is right where twice its size is below s; the
// few values near a tie (about 1 in 10^5) are looked at one by one.
__device__ __forceinline__ void quant_int8(const float (&x)[kVals], float s, float inv, uint32_t (&code)[2])
{
    constexpr float kMagic = 12582912.f;
    uint32_t t[kVals];
    float worst = 0.f;
#pragma unroll
    for (int j = 0; j < kVals; ++j) {
        const float y = fmaf(x[j], inv, kMagic);
        t[j] = __float_as_uint(y);
        worst = fmaxf(worst, fabsf(fmaf(kMagic - y, s, x[j])));
    }
    if (2.f * worst >= s) {
#pragma unroll
        for (int j = 0; j < kVals; ++j) {
            const float q = __uint_as_float(t[j]) - kMagic, r = fmaf(-q, s, x[j]), r2 = 2.f * fabsf(r);
            if (r2 > s || (r2 == s && (t[j] & 1u))) t[j] += r > 0.f ? 1u : ~0u;
        }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j)
        code[j] = __byte_perm(__byte_perm(t[4 * j], t[4 * j + 1], 0x0040), __byte_perm(t[4 * j + 2], t[4 * j + 3], 0x0040),
                              0x5410);
}

// e4m3 codes of kVals values times inv (|x inv| <= 448), rounded to nearest even.
__device__ __forceinline__ void quant_e4m3(const float (&x)[kVals], float inv, uint32_t (&code)[2])
{
    uint32_t two[kVals / 2];
#pragma unroll
    for (int j = 0; j < kVals / 2; ++j)
        two[j] = __nv_cvt_float2_to_fp8x2(make_float2(x[2 * j] * inv, x[2 * j + 1] * inv), __NV_SATFINITE, __NV_E4M3);
    code[0] = two[0] | two[1] << 16;
    code[1] = two[2] | two[3] << 16;
}

// The smallest power of two s >= 2^-126 with top / s <= 448 = 1.75 * 2^8.
__device__ __forceinline__ float e4m3_scale(float top)
{
    const uint32_t b = __float_as_uint(top);
    const int e = int(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
    return __uint_as_float(uint32_t(max(e, -126) + 127) << 23);
}

// One thread per kVals values of U (row, part, head) units; a unit's head_dim /
// kVals threads are neighbours in a warp and find the largest value by
// shuffles.  A block's units follow one another, so its accesses do.  With U
// units a thread has U units' loads in flight; measured for 17,408 rows of 12 x
// 64 fp32 into int8 and back (two launches): U = 2 and 4 (store, load) 46 us, 5.9
// TB/s, 0.87 of the measured copy's rate; 1 and 2 0.7 us more, 4 and 8 6 us, 8
// and 16 36 us (registers).  U is the same for 16-bit rows, of which a thread then
// has half the bytes in flight: 8,191 rows of 8 x 128 bf16 into e4m3 and back 25.2
// us, 4.0 TB/s, eight times as many 184 us, 4.4 TB/s; into bf16 24.5, 5.5 TB/s (fp32
// into fp32, 17,408 rows of 12 x 64: 67.0, 6.4 TB/s).  64 rows, a decode step's: 3.0
// us for both, the launches.
// CT: the cache's element type (int8_t and __nv_fp8_e4m3 with scales).
struct Unit {
    int i, part, h;                // row, 0: k / 1: v, head
    __device__ __forceinline__ Unit(uint32_t unit, uint32_t H)
    {
        const uint32_t hd = unit / H;
        h = int(unit - hd * H);
        part = int(hd & 1);
        i = int(hd >> 1);
    }
};

template <typename ST, typename CT, bool VEC, int U>
__global__ void __launch_bounds__(256) k_kv_store(const RowArgs a)
{
    constexpr bool kA = kApart<ST, CT>;
    pdl_wait();
    pdl_launch_dependents();
    const uint32_t D = a.kv.head_dim, H = a.kv.n_head, lanes = D / kVals, step = piece_step<kA>(D);
    const uint32_t per = 256 / lanes, l = threadIdx.x % lanes;
    const uint32_t unit0 = blockIdx.x * (U * per) + threadIdx.x / lanes;
    float x[U][kVals];
    int slot[U], pos[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const Unit n(unit0 + u * per, H);
        const bool ok = n.i < a.n_rows;
        slot[u] = ok ? a.slot[n.i] : -1;
        pos[u] = ok ? a.pos[n.i] : -1;
#pragma unroll
        for (int j = 0; j < kVals; ++j) x[u][j] = 0.f;
        if (ok)
            get_vals<ST, kA, VEC>(static_cast<const ST *>(n.part ? a.src_v : a.src_k) + n.i * a.stride + n.h * D + piece_at<kA>(l),
                                  step, x[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const Unit n(unit0 + u * per, H);
        const bool there = slot[u] >= 0 && slot[u] < a.kv.n_slots && pos[u] >= 0 && pos[u] < a.kv.n_positions;
        const size_t row = (size_t(there ? slot[u] : 0) * H + n.h) * a.kv.n_positions + (there ? pos[u] : 0);
        CT *c = static_cast<CT *>(n.part ? a.kv.v : a.kv.k) + row * D + piece_at<kA>(l);
        if constexpr (sizeof(CT) > 1) {
            if (there) put_vals<CT, kA, true>(c, step, x[u]);
        } else {
            // (times zero, an infinity or a NaN leaves a NaN)
            float top = 0.f, nan = 0.f;
#pragma unroll
            for (int j = 0; j < kVals; ++j) {
                top = fmaxf(top, fabsf(x[u][j]));
                nan = fmaf(x[u][j], 0.f, nan);
            }
            for (uint32_t o = lanes / 2; o > 0; o >>= 1) {
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                nan += __shfl_xor_sync(0xffffffffu, nan, o);
            }
            const bool bad = nan != 0.f;
            float s;
            Words<CT> codes;
            if constexpr (std::is_same<CT, int8_t>::value) {
                s = fmaxf(top * (1.f / 127.f), FLT_MIN);
                quant_int8(x[u], s, __frcp_rn(s), codes.w);
            } else {
                s = e4m3_scale(top);
                quant_e4m3(x[u], __uint_as_float((254u << 23) - __float_as_uint(s)), codes.w);   // exact: a power of two
            }
            if (bad) {
                codes.w[0] = codes.w[1] = 0;
                s = __int_as_float(0x7fc00000);
            }
            if (there) {
                put_words<CT, kA>(c, step, codes);
                if (l == 0) (n.part ? a.kv.v_scale : a.kv.k_scale)[row] = s;
            }
        }
    }
}

// (the cache's values stay as they are in memory until they are written, so
// that a thread has 32 bytes in flight)
template <typename CT, typename DT, bool VEC, int U>
__global__ void __launch_bounds__(256) k_kv_load(const RowArgs a)
{
    constexpr bool kA = kApart<DT, CT>;
    pdl_wait();
    pdl_launch_dependents();
    const uint32_t D = a.kv.head_dim, H = a.kv.n_head, lanes = D / kVals, step = piece_step<kA>(D);
    const uint32_t per = 256 / lanes, l = threadIdx.x % lanes;
    const uint32_t unit0 = blockIdx.x * (U * per) + threadIdx.x / lanes;
    Words<CT> raw[U];
    float s[U];
    size_t row[U];
    bool there[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const Unit n(unit0 + u * per, H);
        const int slot = n.i < a.n_rows ? a.slot[n.i] : -1, pos = n.i < a.n_rows ? a.pos[n.i] : -1;
        there[u] = slot >= 0 && slot < a.kv.n_slots && pos >= 0 && pos < a.kv.n_positions;
        row[u] = (size_t(there[u] ? slot : 0) * H + n.h) * a.kv.n_positions + (there[u] ? pos : 0);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const Unit n(unit0 + u * per, H);
        const CT *c = static_cast<const CT *>(n.part ? a.kv.v : a.kv.k) + row[u] * D + piece_at<kA>(l);
#pragma unroll
        for (int j = 0; j < int(kVals * sizeof(CT) / 4); ++j) raw[u].w[j] = 0;
        s[u] = 1.f;
        if (there[u]) {
            get_words<CT, kA, false>(c, step, raw[u]);
            if constexpr (sizeof(CT) == 1) s[u] = (n.part ? a.kv.v_scale : a.kv.k_scale)[row[u]];
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const Unit n(unit0 + u * per, H);
        float x[kVals];
#pragma unroll
        for (int j = 0; j < kVals; ++j) {
            if constexpr (sizeof(CT) > 1) {
                x[j] = float(raw[u].t[j]);
            } else if constexpr (std::is_same<CT, int8_t>::value) {
                x[j] = float(raw[u].t[j]) * s[u];
            } else if (j % 2 == 0) {
                const __half2_raw h =
                    __nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(raw[u].w[j / 4] >> (j % 4 * 8)), __NV_E4M3);
                const float2 f = __half22float2(__half2(h));
                x[j] = f.x * s[u];
                x[j + 1] = f.y * s[u];
            }
        }
        if (n.i < a.n_rows)
            put_vals<DT, kA, VEC>(static_cast<DT *>(n.part ? a.dst_v : a.dst_k) + n.i * a.stride + n.h * D + piece_at<kA>(l), step, x);
    }
}

// Accepted rows into place.  One block per (layer, sequence) and share of the
// columns: a thread owns 16 bytes of a (part, head) row (or one scale) and
// moves them for every accepted node, so no other thread touches them.  A
// source row is never one that an earlier move has written (path[j] >= j), so
// kAhead loads go out before their stores.
struct CommitArgs {
    gpt2_kv kv;
    const int32_t *slot, *cached, *path, *n_path;
    int32_t n_seqs, max_nodes, row16;   // row16: 16-byte columns of a head's row
};

constexpr int kAhead = 8;

template <typename T>
__device__ __forceinline__ void move_rows(T *base, size_t ld, const int *path, int n)
{
    for (int i0 = 1; i0 < n; i0 += kAhead) {
        T v[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            if (i0 + j < n && path[i0 + j] != i0 + j) v[j] = base[path[i0 + j] * ld];
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            if (i0 + j < n && path[i0 + j] != i0 + j) base[(i0 + j) * ld] = v[j];
    }
}

__global__ void __launch_bounds__(256) k_kv_commit(const CommitArgs a)
{
    __shared__ int path[GPT2_MAX_NODES];
    __shared__ int n_ok;
    const int b = blockIdx.x % a.n_seqs, layer = blockIdx.x / a.n_seqs;
    pdl_wait();
    pdl_launch_dependents();
    const int H = a.kv.n_head, P = a.kv.n_positions;
    const int slot = a.slot[b], cached = a.cached[b];
    const bool there = slot >= 0 && slot < a.kv.n_slots && cached >= 0;
    const int n = there ? min(a.n_path[b], a.max_nodes) : 0;
    if (threadIdx.x < GPT2_MAX_NODES && int(threadIdx.x) < n) path[threadIdx.x] = a.path[size_t(b) * a.max_nodes + threadIdx.x];
    __syncthreads();
    if (threadIdx.x == 0) {
        int k = 0;
        while (k < n && path[k] >= k && path[k] < a.max_nodes && (k == 0 || path[k] > path[k - 1]) &&
               cached < P - path[k])
            ++k;
        n_ok = n > 0 && path[0] == 0 ? k : 0;
    }
    __syncthreads();
    const int m = n_ok;
    const int cols = 2 * H * a.row16, scales = (a.kv.dtype == GPT2_INT8 || a.kv.dtype == GPT2_E4M3) ? 2 * H : 0;
    for (int c = blockIdx.y * 256 + threadIdx.x; c < cols + scales; c += gridDim.y * 256) {
        const bool sc = c >= cols;
        const int u = sc ? c - cols : c / a.row16;   // (part, head)
        const int part = u / H, h = u % H;
        const size_t row = ((size_t(layer) * a.kv.n_slots + slot) * H + h) * P + cached;
        if (m <= 1) break;
        if (sc)
            move_rows((part ? a.kv.v_scale : a.kv.k_scale) + row, 1, path, m);
        else
            move_rows(static_cast<uint4 *>(part ? a.kv.v : a.kv.k) + row * a.row16 + c % a.row16, size_t(a.row16),
                      path, m);
    }
}

template <typename F>
int by_row_type(int t, F f)
{
    if (t == GPT2_F32) return f(float());
    if (t == GPT2_F16) return f(__half());
    return f(__nv_bfloat16());
}

int rows_ok(const gpt2_kv *kv, const void *k, const void *v, int32_t dtype, int64_t stride, const int32_t *slot,
            const int32_t *pos, int32_t n_rows)
{
    if (!kv_ok(kv) || !k || !v || !slot || !pos || !is_row_type(dtype) || n_rows < 0) return GPT2_ERR_INVALID_ARG;
    const int E = kv->n_head * kv->head_dim, es = elem_size(dtype);
    if ((long long)kv->n_head * kv->head_dim > (1ll << 24) || stride < E) return GPT2_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(k) % es || reinterpret_cast<uintptr_t>(v) % es) return GPT2_ERR_INVALID_ARG;
    if (!aligned4(slot, pos)) return GPT2_ERR_INVALID_ARG;
    // (row, part, head) units, and a block's last ones past the end, are counted in 32 bits
    if (((long long)n_rows + 1) * 2 * kv->n_head + 4096 >= (1ll << 31)) return GPT2_ERR_INVALID_ARG;
    return GPT2_OK;
}

// Several units per thread once that still gives every SM four blocks.
bool many_rows(const gpt2_kv *kv, int32_t n_rows, int sms)
{
    return (long long)n_rows * 2 * kv->n_head * (kv->head_dim / kVals) >= 4ll * 256 * 4 * sms;
}

unsigned row_blocks(const gpt2_kv *kv, int32_t n_rows, int units)
{
    const long long per = (long long)units * (256 / (kv->head_dim / kVals));
    return unsigned(((long long)n_rows * 2 * kv->n_head + per - 1) / per);
}

bool vec_ok(const void *k, const void *v, int32_t dtype, int64_t stride)
{
    return aligned16(k) && aligned16(v) && stride * elem_size(dtype) % 16 == 0;
}

}  // namespace
}  // namespace gpt2

using namespace gpt2;

extern "C" {

int gpt2_op_kv_store(const gpt2_kv *kv, const void *k, const void *v, int32_t src_dtype, int64_t row_stride,
                     const int32_t *slot, const int32_t *pos, int32_t n_rows, void *stream)
{
    int rc = rows_ok(kv, k, v, src_dtype, row_stride, slot, pos, n_rows);
    if (rc != GPT2_OK || n_rows == 0) return rc;
    const int sms = spec_sms(&rc);
    if (!sms) return rc;
    const bool many = many_rows(kv, n_rows, sms);
    const RowArgs a{*kv, k, v, nullptr, nullptr, row_stride, slot, pos, n_rows};
    const bool vec = vec_ok(k, v, src_dtype, row_stride);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return by_row_type(src_dtype, [&](auto st) {
        using ST = decltype(st);
        auto go = [&](auto ct) {
            using CT = decltype(ct);
            if (!vec) return spec_rc(spec_launch(k_kv_store<ST, CT, false, 1>, dim3(row_blocks(kv, n_rows, 1)), 256, 0, 1, s, a));
            if (many) return spec_rc(spec_launch(k_kv_store<ST, CT, true, 2>, dim3(row_blocks(kv, n_rows, 2)), 256, 0, 1, s, a));
            return spec_rc(spec_launch(k_kv_store<ST, CT, true, 1>, dim3(row_blocks(kv, n_rows, 1)), 256, 0, 1, s, a));
        };
        if (kv->dtype == GPT2_INT8) return go(int8_t());
        if (kv->dtype == GPT2_E4M3) return go(__nv_fp8_e4m3());
        return by_row_type(kv->dtype, go);
    });
}

int gpt2_op_kv_load(const gpt2_kv *kv, const int32_t *slot, const int32_t *pos, int32_t n_rows, void *k, void *v,
                    int32_t dst_dtype, int64_t row_stride, void *stream)
{
    int rc = rows_ok(kv, k, v, dst_dtype, row_stride, slot, pos, n_rows);
    if (rc != GPT2_OK || n_rows == 0) return rc;
    const int sms = spec_sms(&rc);
    if (!sms) return rc;
    const bool many = many_rows(kv, n_rows, sms);
    const RowArgs a{*kv, nullptr, nullptr, k, v, row_stride, slot, pos, n_rows};
    const bool vec = vec_ok(k, v, dst_dtype, row_stride);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return by_row_type(dst_dtype, [&](auto dt) {
        using DT = decltype(dt);
        auto go = [&](auto ct) {
            using CT = decltype(ct);
            if (!vec) return spec_rc(spec_launch(k_kv_load<CT, DT, false, 1>, dim3(row_blocks(kv, n_rows, 1)), 256, 0, 1, s, a));
            if (many) {
                constexpr int U = 4 / int(sizeof(CT));
                return spec_rc(spec_launch(k_kv_load<CT, DT, true, U>, dim3(row_blocks(kv, n_rows, U)), 256, 0, 1, s, a));
            }
            return spec_rc(spec_launch(k_kv_load<CT, DT, true, 1>, dim3(row_blocks(kv, n_rows, 1)), 256, 0, 1, s, a));
        };
        if (kv->dtype == GPT2_INT8) return go(int8_t());
        if (kv->dtype == GPT2_E4M3) return go(__nv_fp8_e4m3());
        return by_row_type(kv->dtype, go);
    });
}

int gpt2_op_kv_commit(const gpt2_kv *kv, int32_t n_layer, const int32_t *slot, const int32_t *cached,
                      const int32_t *path, const int32_t *n_path, int32_t n_seqs, int32_t max_nodes, void *stream)
{
    if (!kv_ok(kv) || n_layer < 1 || !slot || !cached || !path || !n_path || n_seqs < 0) return GPT2_ERR_INVALID_ARG;
    if (max_nodes < 1 || max_nodes > GPT2_MAX_NODES || (long long)n_layer * n_seqs >= (1ll << 31) - 1)
        return GPT2_ERR_INVALID_ARG;
    if ((long long)kv->n_head * kv->head_dim > (1ll << 24)) return GPT2_ERR_INVALID_ARG;
    if (!aligned4(slot, cached, path, n_path)) return GPT2_ERR_INVALID_ARG;
    if (n_seqs == 0) return GPT2_OK;
    int rc;
    if (!spec_sms(&rc)) return rc;
    const CommitArgs a{*kv, slot, cached, path, n_path, n_seqs, max_nodes,
                       kv->head_dim * elem_size(kv->dtype) / 16};
    const int cols = 2 * kv->n_head * (a.row16 + 1);
    const dim3 grid(unsigned(n_layer) * n_seqs, (cols + 255) / 256);
    return spec_rc(spec_launch(k_kv_commit, grid, 256, 0, 1, static_cast<cudaStream_t>(stream), a));
}

}  // extern "C"
