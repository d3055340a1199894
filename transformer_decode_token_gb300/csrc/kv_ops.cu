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
    const void *src[2];        // store: k, v rows
    void *dst[2];              // load: k, v rows
    int64_t stride;
    const int32_t *slot, *pos;
    int32_t n_rows;
};

// kVals values of a row of type T, as fp32; VEC: 16-byte accesses are aligned.
template <typename T, bool VEC>
__device__ __forceinline__ void get_vals(const T *p, float (&x)[kVals])
{
    if constexpr (!VEC) {
#pragma unroll
        for (int i = 0; i < kVals; ++i) x[i] = float(p[i]);
    } else if constexpr (sizeof(T) == 4) {
        const float4 a = __ldcs(reinterpret_cast<const float4 *>(p)), b = __ldcs(reinterpret_cast<const float4 *>(p) + 1);
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    } else {
        union {
            uint4 u;
            T t[kVals];
        } w;
        w.u = __ldcs(reinterpret_cast<const uint4 *>(p));
#pragma unroll
        for (int i = 0; i < kVals; ++i) x[i] = float(w.t[i]);
    }
}

template <typename T>
__device__ __forceinline__ T round_to(float x)
{
    if constexpr (sizeof(T) == 4) return x;
    else return T(x);   // round to nearest even
}

template <typename T, bool VEC>
__device__ __forceinline__ void put_vals(T *p, const float (&x)[kVals])
{
    if constexpr (!VEC) {
#pragma unroll
        for (int i = 0; i < kVals; ++i) p[i] = round_to<T>(x[i]);
    } else if constexpr (sizeof(T) == 4) {
        reinterpret_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
        reinterpret_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
        union {
            uint4 u;
            T t[kVals];
        } w;
#pragma unroll
        for (int i = 0; i < kVals; ++i) w.t[i] = round_to<T>(x[i]);
        *reinterpret_cast<uint4 *>(p) = w.u;
    }
}

// The integer nearest x / s (|x| <= 127 s (1 + 2^-23)), ties to even, of the exact quotient
// and not of a rounded one: q = rint(x * (1/s)) is at most one off, and the
// remainder x - q s is exact in one fused multiply-add (it is a multiple of
// half an ulp of s and no larger than about s/2), so comparing twice its size
// with s says whether q has to move.
__device__ __forceinline__ int quant_int8(float x, float s, float inv)
{
    float q = rintf(x * inv);
    const float r = fmaf(-q, s, x), r2 = 2.f * fabsf(r);
    const bool odd = (int(q) & 1) != 0;
    if (r2 > s || (r2 == s && odd)) q += r > 0.f ? 1.f : -1.f;
    return max(-127, min(127, int(q)));
}

// The smallest power of two s >= 2^-126 with top / s <= 448 = 1.75 * 2^8.
__device__ __forceinline__ float e4m3_scale(float top)
{
    const uint32_t b = __float_as_uint(top);
    const int e = int(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
    return __uint_as_float(uint32_t(max(e, -126) + 127) << 23);
}

// One thread per kVals values; the head_dim / kVals threads of a (row, part,
// head) are neighbours in a warp and find the largest value by shuffles.
// CT: the cache's element type (int8_t and __nv_fp8_e4m3 with scales).
template <typename ST, typename CT, bool VEC>
__global__ void __launch_bounds__(256) k_kv_store(const RowArgs a)
{
    const int D = a.kv.head_dim, H = a.kv.n_head, lanes = D / kVals;
    const long long unit = (blockIdx.x * 256ll + threadIdx.x) / lanes;
    const int l = threadIdx.x % lanes;
    const long long hd = unit / H;
    const int h = int(unit - hd * H), part = int(hd & 1);
    const long long i = hd >> 1;
    const int slot = i < a.n_rows ? a.slot[i] : -1, pos = i < a.n_rows ? a.pos[i] : -1;
    const bool there = slot >= 0 && slot < a.kv.n_slots && pos >= 0 && pos < a.kv.n_positions;
    float x[kVals] = {};
    if (there) get_vals<ST, VEC>(static_cast<const ST *>(a.src[part]) + i * a.stride + h * D + l * kVals, x);
    const size_t row = (size_t(there ? slot : 0) * H + h) * a.kv.n_positions + (there ? pos : 0);
    CT *c = static_cast<CT *>(part ? a.kv.v : a.kv.k) + row * D + l * kVals;
    if constexpr (sizeof(CT) > 1) {
        if (there) put_vals<CT, true>(c, x);
    } else {
        float top = 0.f;
        bool fine = true;
#pragma unroll
        for (int j = 0; j < kVals; ++j) {
            top = fmaxf(top, fabsf(x[j]));
            fine = fine && fabsf(x[j]) <= FLT_MAX;
        }
        uint32_t bad = fine ? 0u : 1u;
        for (int o = lanes / 2; o > 0; o >>= 1) {
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            bad |= __shfl_xor_sync(0xffffffffu, bad, o);
        }
        union {
            uint2 u;
            uint8_t b[kVals];
        } w;
        float s;
        if constexpr (std::is_same<CT, int8_t>::value) {
            s = fmaxf(__fdiv_rn(top, 127.f), FLT_MIN);
            const float inv = __frcp_rn(s);
#pragma unroll
            for (int j = 0; j < kVals; ++j) w.b[j] = bad ? 0 : uint8_t(int8_t(quant_int8(x[j], s, inv)));
        } else {
            s = e4m3_scale(top);
            const float inv = __uint_as_float((254u << 23) - __float_as_uint(s));   // exact: a power of two
#pragma unroll
            for (int j = 0; j < kVals; ++j)
                w.b[j] = bad ? 0 : uint8_t(__nv_cvt_float_to_fp8(x[j] * inv, __NV_SATFINITE, __NV_E4M3));
        }
        if (there) {
            *reinterpret_cast<uint2 *>(c) = w.u;
            if (l == 0) (part ? a.kv.v_scale : a.kv.k_scale)[row] = bad ? __int_as_float(0x7fc00000) : s;
        }
    }
}

template <typename CT, typename DT, bool VEC>
__global__ void __launch_bounds__(256) k_kv_load(const RowArgs a)
{
    const int D = a.kv.head_dim, H = a.kv.n_head, lanes = D / kVals;
    const long long unit = (blockIdx.x * 256ll + threadIdx.x) / lanes;
    const int l = threadIdx.x % lanes;
    const long long hd = unit / H;
    const int h = int(unit - hd * H), part = int(hd & 1);
    const long long i = hd >> 1;
    if (i >= a.n_rows) return;
    const int slot = a.slot[i], pos = a.pos[i];
    float x[kVals] = {};
    if (slot >= 0 && slot < a.kv.n_slots && pos >= 0 && pos < a.kv.n_positions) {
        const size_t row = (size_t(slot) * H + h) * a.kv.n_positions + pos;
        const CT *c = static_cast<const CT *>(part ? a.kv.v : a.kv.k) + row * D + l * kVals;
        if constexpr (sizeof(CT) > 1) {
            get_vals<CT, true>(c, x);
        } else {
            union {
                uint2 u;
                CT t[kVals];
            } w;
            w.u = *reinterpret_cast<const uint2 *>(c);
            const float s = (part ? a.kv.v_scale : a.kv.k_scale)[row];
#pragma unroll
            for (int j = 0; j < kVals; ++j) x[j] = float(w.t[j]) * s;
        }
    }
    put_vals<DT, VEC>(static_cast<DT *>(a.dst[part]) + i * a.stride + h * D + l * kVals, x);
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
    if ((long long)n_rows * 2 * E / kVals / 256 >= (1ll << 31) - 1) return GPT2_ERR_INVALID_ARG;
    return GPT2_OK;
}

unsigned row_blocks(const gpt2_kv *kv, int32_t n_rows)
{
    return unsigned(((long long)n_rows * 2 * kv->n_head * (kv->head_dim / kVals) + 255) / 256);
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
    if (!spec_sms(&rc)) return rc;
    const RowArgs a{*kv, {k, v}, {}, row_stride, slot, pos, n_rows};
    const unsigned grid = row_blocks(kv, n_rows);
    const bool vec = vec_ok(k, v, src_dtype, row_stride);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return by_row_type(src_dtype, [&](auto st) {
        using ST = decltype(st);
        auto go = [&](auto ct) {
            using CT = decltype(ct);
            if (vec) k_kv_store<ST, CT, true><<<grid, 256, 0, s>>>(a);
            else k_kv_store<ST, CT, false><<<grid, 256, 0, s>>>(a);
            return spec_rc(cudaGetLastError());
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
    if (!spec_sms(&rc)) return rc;
    const RowArgs a{*kv, {}, {k, v}, row_stride, slot, pos, n_rows};
    const unsigned grid = row_blocks(kv, n_rows);
    const bool vec = vec_ok(k, v, dst_dtype, row_stride);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return by_row_type(dst_dtype, [&](auto dt) {
        using DT = decltype(dt);
        auto go = [&](auto ct) {
            using CT = decltype(ct);
            if (vec) k_kv_load<CT, DT, true><<<grid, 256, 0, s>>>(a);
            else k_kv_load<CT, DT, false><<<grid, 256, 0, s>>>(a);
            return spec_rc(cudaGetLastError());
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
    if (n_seqs == 0) return GPT2_OK;
    int rc;
    if (!spec_sms(&rc)) return rc;
    const CommitArgs a{*kv, slot, cached, path, n_path, n_seqs, max_nodes,
                       kv->head_dim * elem_size(kv->dtype) / 16};
    const int cols = 2 * kv->n_head * (a.row16 + 1);
    const dim3 grid(unsigned(n_layer) * n_seqs, (cols + 255) / 256);
    k_kv_commit<<<grid, 256, 0, static_cast<cudaStream_t>(stream)>>>(a);
    return spec_rc(cudaGetLastError());
}

}  // extern "C"
