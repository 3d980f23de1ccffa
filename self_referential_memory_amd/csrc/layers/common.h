// common.h -- what the layers' translation units share: argument
// checks, and device helpers for fp32 and bf16 rows of any alignment.
#ifndef SRNL_LAYERS_COMMON_H
#define SRNL_LAYERS_COMMON_H

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstdio>
#include <type_traits>

#include "error.h"

namespace srnl_i {

inline srnl_status fail(srnl_status s, const char *msg) { return srnl_set_error(s, msg); }

inline srnl_status launched(const char *what)
{
    const hipError_t e = hipGetLastError();
    if (e == hipSuccess)
        return SRNL_OK;
    char buf[160];
    snprintf(buf, sizeof buf, "%s: %s", what, hipGetErrorString(e));
    return fail(SRNL_ERR_HIP, buf);
}

inline bool valid_dtype(srnl_dtype t) { return t == SRNL_F32 || t == SRNL_BF16; }
inline size_t dtype_size(srnl_dtype t) { return t == SRNL_F32 ? 4 : 2; }

// One named pointer argument. Optional ones may be NULL.
struct PtrArg {
    const void *p;
    const char *name;
    bool optional;
};

// Every pointer must be 16-byte aligned memory of the device that is current,
// on which the kernels are launched.
inline srnl_status check_ptrs(const PtrArg *a, int n)
{
    int cur = -1;
    char buf[160];
    for (int i = 0; i < n; ++i) {
        if (!a[i].p) {
            if (a[i].optional)
                continue;
            snprintf(buf, sizeof buf, "%s is NULL", a[i].name);
            return fail(SRNL_ERR_PTR, buf);
        }
        if (reinterpret_cast<uintptr_t>(a[i].p) & 15u) {
            snprintf(buf, sizeof buf, "%s must be 16-byte aligned", a[i].name);
            return fail(SRNL_ERR_PTR, buf);
        }
        hipPointerAttribute_t at;
        if (hipPointerGetAttributes(&at, a[i].p) != hipSuccess) {
            (void)hipGetLastError();
            snprintf(buf, sizeof buf, "%s must be device memory", a[i].name);
            return fail(SRNL_ERR_PTR, buf);
        }
        if (at.type == hipMemoryTypeManaged)
            continue;
        if (at.type != hipMemoryTypeDevice) {
            snprintf(buf, sizeof buf, "%s must be device memory", a[i].name);
            return fail(SRNL_ERR_PTR, buf);
        }
        if (cur < 0 && hipGetDevice(&cur) != hipSuccess) {
            (void)hipGetLastError();
            return fail(SRNL_ERR_HIP, "hipGetDevice failed");
        }
        if (at.device != cur) {
            snprintf(buf, sizeof buf, "%s is memory of device %d, but device %d is current",
                     a[i].name, at.device, cur);
            return fail(SRNL_ERR_PTR, buf);
        }
    }
    return SRNL_OK;
}

// ------------------------------------------------------------ device helpers

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// two floats to two bf16 words, round to nearest even (v_cvt_pk_bf16_f32)
__device__ __forceinline__ uint32_t pack_bf16(float a, float b)
{
    const f32x2 v = {a, b};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ float bf16_one(uint16_t w)
{
    return __uint_as_float(static_cast<uint32_t>(w) << 16);
}
__device__ __forceinline__ uint16_t to_bf16(float a)
{
    return static_cast<uint16_t>(pack_bf16(a, 0.0f));
}

// N consecutive elements (4 or 8) from element offset o of a row array of
// fp32 or bf16 words; ALIGNED: the address is a multiple of the piece's size
// (or 16 bytes), else of one element (the card takes such wide loads too).
template <int N, bool ALIGNED>
__device__ __forceinline__ void load_f32(const float *p, float (&v)[N])
{
    f32x4 w[N / 4];
    if (ALIGNED) {
#pragma unroll
        for (int k = 0; k < N / 4; ++k)
            w[k] = *reinterpret_cast<const f32x4 *>(p + 4 * k);
    } else {
        __builtin_memcpy(w, p, sizeof w);
    }
#pragma unroll
    for (int k = 0; k < N; ++k)
        v[k] = w[k / 4][k % 4];
}
template <int N, bool ALIGNED>
__device__ __forceinline__ void load_bf16(const uint16_t *p, float (&v)[N])
{
    uint32_t w[N / 2];
    if (ALIGNED && N == 8) {
        const u32x4 t = *reinterpret_cast<const u32x4 *>(p);
#pragma unroll
        for (int k = 0; k < N / 2; ++k)
            w[k] = t[k];
    } else if (ALIGNED) {
        const u32x2 t = *reinterpret_cast<const u32x2 *>(p);
        w[0] = t[0];
        w[1] = t[1];
    } else {
        __builtin_memcpy(w, p, sizeof w);
    }
#pragma unroll
    for (int k = 0; k < N / 2; ++k) {
        v[2 * k] = bf16_lo(w[k]);
        v[2 * k + 1] = bf16_hi(w[k]);
    }
}
// n of the N elements are inside the row; the others read as 0 without an
// access. ALIGNED also says that rows are whole pieces (n >= N or n <= 0).
template <int N, bool ALIGNED>
__device__ __forceinline__ void load_row(const void *p, bool bf, long long o, int n, float (&v)[N])
{
    if (ALIGNED ? n > 0 : n >= N) {
        if (bf)
            load_bf16<N, ALIGNED>(static_cast<const uint16_t *>(p) + o, v);
        else
            load_f32<N, ALIGNED>(static_cast<const float *>(p) + o, v);
        return;
    }
#pragma unroll
    for (int k = 0; k < N; ++k)
        v[k] = 0.0f;
    if (ALIGNED)
        return;
#pragma unroll
    for (int k = 0; k < N; ++k)
        if (k < n)
            v[k] = bf ? bf16_one(static_cast<const uint16_t *>(p)[o + k])
                      : static_cast<const float *>(p)[o + k];
}
template <int N, bool ALIGNED>
__device__ __forceinline__ void store_row(void *p, bool bf, long long o, int n, const float (&v)[N])
{
    if (ALIGNED ? n > 0 : n >= N) {
        if (bf) {
            uint16_t *q = static_cast<uint16_t *>(p) + o;
            uint32_t w[N / 2];
#pragma unroll
            for (int k = 0; k < N / 2; ++k)
                w[k] = pack_bf16(v[2 * k], v[2 * k + 1]);
            if (ALIGNED && N == 8) {
                const u32x4 t = {w[0], w[1], w[N / 2 - 2], w[N / 2 - 1]};
                *reinterpret_cast<u32x4 *>(q) = t;
            } else if (ALIGNED) {
                const u32x2 t = {w[0], w[1]};
                *reinterpret_cast<u32x2 *>(q) = t;
            } else {
                __builtin_memcpy(q, w, sizeof w);
            }
        } else {
            float *q = static_cast<float *>(p) + o;
            f32x4 w[N / 4];
#pragma unroll
            for (int k = 0; k < N; ++k)
                w[k / 4][k % 4] = v[k];
            if (ALIGNED) {
#pragma unroll
                for (int k = 0; k < N / 4; ++k)
                    *reinterpret_cast<f32x4 *>(q + 4 * k) = w[k];
            } else {
                __builtin_memcpy(q, w, sizeof w);
            }
        }
        return;
    }
    if (ALIGNED)
        return;
#pragma unroll
    for (int k = 0; k < N; ++k)
        if (k < n) {
            if (bf)
                static_cast<uint16_t *>(p)[o + k] = to_bf16(v[k]);
            else
                static_cast<float *>(p)[o + k] = v[k];
        }
}

// Sums over partial rows: out[c] = sum over p, in order of slices, of
// part[p * ld + c] (c < n0 to out0, the rest to out1). 32 columns by 32
// slices of the rows per block; a slice's rows and then the slices add in a
// fixed order, so the result repeats bit for bit.
__global__ __launch_bounds__(1024) static void sum_rows_kernel(const float *__restrict__ part, int rows, long long ld,
                                                        long long cols, long long n0,
                                                        float *__restrict__ out0, float *__restrict__ out1)
{
    __shared__ float s[32][33];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    for (long long c0 = 32LL * blockIdx.x; c0 < cols; c0 += 32LL * gridDim.x) {
        const long long c = c0 + tx;
        float a = 0.0f;
        if (c < cols) {
#pragma unroll 8
            for (int p = ty; p < rows; p += 32)
                a += part[p * ld + c];
        }
        s[ty][tx] = a;
        __syncthreads();
        // the thread's column is its row of the transposed read
        float v = s[tx][ty];
#pragma unroll
        for (int off = 16; off > 0; off >>= 1)
            v += __shfl_xor(v, off);
        const long long cc = c0 + ty;
        if (tx == 0 && cc < cols) {
            if (cc < n0) {
                if (out0)
                    out0[cc] = v;
            } else if (out1) {
                out1[cc - n0] = v;
            }
        }
        __syncthreads();
    }
}

__global__ __launch_bounds__(256) static void zero_kernel(float *__restrict__ p, long long n)
{
    for (long long i = blockIdx.x * 256LL + threadIdx.x; i < n; i += 256LL * gridDim.x)
        p[i] = 0.0f;
}

inline srnl_status zero_fill(float *p, long long n, hipStream_t st)
{
    if (!p || n <= 0)
        return SRNL_OK;
    const long long g = (n + 255) / 256;
    hipLaunchKernelGGL(zero_kernel, dim3(static_cast<unsigned>(g < 4096 ? g : 4096)), dim3(256), 0, st, p, n);
    return launched("zero_kernel");
}

inline srnl_status sum_rows(const float *part, int rows, long long ld, long long cols, long long n0,
                            float *out0, float *out1, hipStream_t st)
{
    const long long blocks = (cols + 31) / 32;
    hipLaunchKernelGGL(sum_rows_kernel, dim3(static_cast<unsigned>(blocks < 65536 ? blocks : 65536)), dim3(1024), 0, st,
                       part, rows, ld, cols, n0, out0, out1);
    return launched("sum_rows_kernel");
}

}  // namespace srnl_i

#endif
