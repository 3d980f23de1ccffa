// linear.h -- what the linear layer's translation units share: activations,
// the split of fp32 values into bf16 parts, operands, the epilogue.
#ifndef SRNL_LAYERS_LINEAR_H
#define SRNL_LAYERS_LINEAR_H

#include "common.h"
#include "plan.h"

namespace srnl_i {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

// ------------------------------------------------------------ activations

// 1 - Phi(|z|) of the standard normal as exp(-z^2 / 2) P(s), s = |z| / (|z| + 3):
// P is the degree-7 polynomial of least weighted relative error (weighted least
// squares on a Chebyshev basis, its weight moved to the largest errors, the
// constant then set to 1/2), which keeps the lower tail's digits: P is right to
// 1.7e-7 of itself up to |z| = 3 and 4e-6 beyond, the whole in fp32 to 4.3e-7 up to
// 2, 2.2e-6 up to 5 and 1.2e-5 at 13, where it leaves fp32's range. ex returns
// exp(-z^2 / 2).
// A polynomial in z alone takes six issue slots fewer (19, not 25; 200704 x 64 ->
// 256 gelu 69.6 us, not 73.0), but Phi is then right to 1.9e-7 in absolute
// terms only: gelu(-4.5) to two digits.
__device__ __forceinline__ float normal_tail(float z, float &ex)
{
    // an infinity would be infinity x 0 in s; ex is 0 there, and NaN for NaN
    const float a = __builtin_amdgcn_fmed3f(fabsf(z), 0.0f, 1e30f), s = a * __builtin_amdgcn_rcpf(a + 3.0f);
    float p = fmaf(s, -0.0477076843f, 0.108733349f);
    p = fmaf(s, p, 0.0186278392f);
    p = fmaf(s, p, -0.14763853f);
    p = fmaf(s, p, -0.288549364f);
    p = fmaf(s, p, 1.05326533f);
    p = fmaf(s, p, -1.19682932f);
    p = fmaf(s, p, 0.5f);
    ex = __builtin_amdgcn_exp2f(z * (z * -0.721347520f));
    return p * ex;
}
__device__ __forceinline__ float gelu(float z)
{
    float ex;
    const float q = normal_tail(z, ex);
    return z * (z >= 0.0f ? 1.0f - q : q);
}
__device__ __forceinline__ float gelu_slope(float z)
{
    float ex;
    const float q = normal_tail(z, ex);
    return fmaf(z * 0.39894228040143268f, ex, z >= 0.0f ? 1.0f - q : q);
}
__device__ __forceinline__ float logistic(float z)
{
    return __builtin_amdgcn_rcpf(1.0f + __expf(-z));
}
__device__ __forceinline__ void act_values(float (&v)[8], int act)
{
    if (act == SRNL_ACT_GELU) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] = gelu(v[e]);
    } else if (act == SRNL_ACT_SILU) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] *= logistic(v[e]);
    }
}
// d *= act'(z)
__device__ __forceinline__ void act_slopes(const float (&z)[8], int act, float (&d)[8])
{
    if (act == SRNL_ACT_GELU) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            d[e] *= gelu_slope(z[e]);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float s = logistic(z[e]);
            d[e] *= s * fmaf(z[e], 1.0f - s, 1.0f);
        }
    }
}

// ------------------------------------------------------------ operands

// 8 fp32 values to PARTS planes of bf16 words
__device__ __forceinline__ void split_parts(const float (&v)[8], u32x4 (&w)[3])
{
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float a = v[2 * k], b = v[2 * k + 1];
        const uint32_t h = pack_bf16(a, b);
        const float ra = a - bf16_lo(h), rb = b - bf16_hi(h);
        const uint32_t m = pack_bf16(ra, rb);
        w[0][k] = h;
        w[1][k] = m;
        w[2][k] = pack_bf16(ra - bf16_lo(m), rb - bf16_hi(m));
    }
}

// One operand as memory: element (row, r) is at row * ld + r (reduction
// contiguous, RC) or r * ld + row.
struct Operand {
    const void *p;
    long long ld;
    long long rows;       // output rows (or columns) of this operand
    const float *z;       // SLOPE: pre-activations laid out like p
    int act;
};

// Barrier for LDS alone: __syncthreads() would also wait for every load from
// memory that is in flight, prefetched registers among them.
__device__ __forceinline__ void lds_barrier()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// ------------------------------------------------------------ epilogue

struct Epilogue {
    void *out;             // [I][J]
    bool obf;
    const float *bias;     // [J] or NULL
    int act;
    const void *add;       // [I][J] or NULL: added after the activation
    bool abf;
    float *pre;            // [I][J] or NULL: z before the activation
};

// Eight neighbouring outputs from their sums z, o their place; n are inside.
// WHOLE: the rows are whole pieces, so that n is 8 or nothing. The bias is in
// registers: a load between the stores of two pieces would wait for the first
// piece's stores.
template <bool WHOLE>
__device__ __forceinline__ void finish_piece(const Epilogue &e, long long o, int n, float (&v)[8],
                                             const float (&bias)[8])
{
    if (n <= 0)
        return;
#pragma unroll
    for (int k = 0; k < 8; ++k)
        v[k] += bias[k];
    if (e.pre)
        store_row<8, WHOLE>(e.pre, false, o, n, v);
    act_values(v, e.act);
    if (e.add) {
        float a[8];
        load_row<8, WHOLE>(e.add, e.abf, o, n, a);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            v[k] += a[k];
    }
    store_row<8, WHOLE>(e.out, e.obf, o, n, v);
}
// the bias of outputs j .. j + 7, zeros without one
template <bool WHOLE>
__device__ __forceinline__ void load_bias(const Epilogue &e, int j, int n, float (&b)[8])
{
#pragma unroll
    for (int k = 0; k < 8; ++k)
        b[k] = 0.0f;
    if (e.bias)
        load_row<8, WHOLE>(e.bias, false, j, n, b);
}
// the two together, for a thread with one piece
__device__ __forceinline__ void finish8(const Epilogue &e, long long o, int j, int n, float (&v)[8])
{
    float b[8];
    load_bias<false>(e, j, n, b);
    finish_piece<false>(e, o, n, v, b);
}

}  // namespace srnl_i

#endif
