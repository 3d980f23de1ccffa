// delta_mma.h -- matrix operands of the gated delta rule's chunks.
//
// A 16 x 16 x 32 product: lane l holds, of an operand, 8 consecutive reduction
// elements from 8 (l >> 4) of row (or column) l & 15; of the result, column
// l & 15 in rows 4 (l >> 4) .. + 3. fp32 products run as eight 16 x 16 x 4 ones
// whose reduction order is the same for both operands.
//
// Inputs (In) are bf16 words or fp32 values. What the kernels form between
// (Mid) is fp32, or with bf16 inputs the sum of two bf16 words, right to 2^-17:
// one word would round states and errors to 2^-9 at every chunk. The product of
// two such pairs leaves out the low words' (2^-18). A row of split values takes 4
// bytes a value either way, 8 high words followed by their 8 low ones.
#ifndef SRNL_LAYERS_DELTA_MMA_H
#define SRNL_LAYERS_DELTA_MMA_H

#include "delta.h"
#include "linear.h"

namespace srnl_i {

template <bool BF> struct In { bf16x8 v; };
template <> struct In<false> { float v[8]; };
template <bool BF> struct Mid { bf16x8 hi, lo; };
template <> struct Mid<false> { float v[8]; };

__device__ __forceinline__ v4f mma16(bf16x8 a, bf16x8 b, v4f c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ v4f mma16(const float (&a)[8], const float (&b)[8], v4f c)
{
#pragma unroll
    for (int j = 0; j < 8; ++j)
        c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[j], b[j], c, 0, 0, 0);
    return c;
}
// smallest parts first
__device__ __forceinline__ v4f mma(const In<true> &a, const In<true> &b, v4f c) { return mma16(a.v, b.v, c); }
__device__ __forceinline__ v4f mma(const In<true> &a, const Mid<true> &b, v4f c)
{
    return mma16(a.v, b.hi, mma16(a.v, b.lo, c));
}
__device__ __forceinline__ v4f mma(const Mid<true> &a, const In<true> &b, v4f c)
{
    return mma16(a.hi, b.v, mma16(a.lo, b.v, c));
}
__device__ __forceinline__ v4f mma(const Mid<true> &a, const Mid<true> &b, v4f c)
{
    return mma16(a.hi, b.hi, mma16(a.hi, b.lo, mma16(a.lo, b.hi, c)));
}
__device__ __forceinline__ v4f mma(const In<false> &a, const In<false> &b, v4f c) { return mma16(a.v, b.v, c); }
__device__ __forceinline__ v4f mma(const In<false> &a, const Mid<false> &b, v4f c) { return mma16(a.v, b.v, c); }
__device__ __forceinline__ v4f mma(const Mid<false> &a, const In<false> &b, v4f c) { return mma16(a.v, b.v, c); }
__device__ __forceinline__ v4f mma(const Mid<false> &a, const Mid<false> &b, v4f c) { return mma16(a.v, b.v, c); }

__device__ __forceinline__ v4f v4f_zero() { return v4f{0.0f, 0.0f, 0.0f, 0.0f}; }

// ---- values

template <bool BF> __device__ __forceinline__ float value(const void *p, long long o)
{
    if constexpr (BF)
        return bf16_one(static_cast<const uint16_t *>(p)[o]);
    else
        return static_cast<const float *>(p)[o];
}
template <bool BF> __device__ __forceinline__ void put_value(void *p, long long o, float v)
{
    if constexpr (BF)
        static_cast<uint16_t *>(p)[o] = to_bf16(v);
    else
        static_cast<float *>(p)[o] = v;
}

// ---- inputs

template <bool BF> __device__ __forceinline__ In<BF> in_zero()
{
    In<BF> f;
    __builtin_memset(&f, 0, sizeof f);
    return f;
}
// 8 elements from element o (a multiple of 8) on, zeros where not live
template <bool BF> __device__ __forceinline__ In<BF> in_load(const void *p, long long o, bool live)
{
    In<BF> f = in_zero<BF>();
    if (live)
        __builtin_memcpy(&f, static_cast<const char *>(p) + o * (BF ? 2 : 4), sizeof f);
    return f;
}
__device__ __forceinline__ float in_squares(const In<true> &f)
{
    u32x4 w;
    __builtin_memcpy(&w, &f, 16);
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        s = fmaf(bf16_lo(w[j]), bf16_lo(w[j]), fmaf(bf16_hi(w[j]), bf16_hi(w[j]), s));
    return s;
}
__device__ __forceinline__ float in_squares(const In<false> &f)
{
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        s = fmaf(f.v[j], f.v[j], s);
    return s;
}

// ---- split values

template <bool BF> __device__ __forceinline__ Mid<BF> mid_zero()
{
    Mid<BF> f;
    __builtin_memset(&f, 0, sizeof f);
    return f;
}
// 8 values at p (LDS or memory; 32 bytes, 16-byte aligned)
template <bool BF> __device__ __forceinline__ Mid<BF> mid_load(const char *p)
{
    Mid<BF> f;
    const u32x4 *w = reinterpret_cast<const u32x4 *>(p);
    const u32x4 t[2] = {w[0], w[1]};
    __builtin_memcpy(&f, t, 32);
    return f;
}
__device__ __forceinline__ void split_pair(float a, float b, uint32_t &hi, uint32_t &lo)
{
    hi = pack_bf16(a, b);
    lo = pack_bf16(a - bf16_lo(hi), b - bf16_hi(hi));
}
// 8 fp32 values to p
template <bool BF> __device__ __forceinline__ void mid_store8(char *p, const float (&v)[8])
{
    u32x4 t[2];
    if constexpr (BF) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t hi, lo;
            split_pair(v[2 * j], v[2 * j + 1], hi, lo);
            t[0][j] = hi;
            t[1][j] = lo;
        }
    } else {
        __builtin_memcpy(t, v, 32);
    }
    reinterpret_cast<u32x4 *>(p)[0] = t[0];
    reinterpret_cast<u32x4 *>(p)[1] = t[1];
}
// a result tile's column as a row of its transpose: 4 values at place k (a
// multiple of 4) of the row at p
template <bool BF> __device__ __forceinline__ void mid_store4(char *p, int k, v4f v)
{
    char *q = p + (k & ~7) * 4;
    if constexpr (BF) {
        u32x2 hi, lo;
        uint32_t h, l;
        split_pair(v[0], v[1], h, l);
        hi[0] = h;
        lo[0] = l;
        split_pair(v[2], v[3], h, l);
        hi[1] = h;
        lo[1] = l;
        *reinterpret_cast<u32x2 *>(q + (k & 4) * 2) = hi;
        *reinterpret_cast<u32x2 *>(q + 16 + (k & 4) * 2) = lo;
    } else {
        *reinterpret_cast<v4f *>(q + (k & 4) * 4) = v;
    }
}
// a result tile as it lies: this lane's 4 rows, `stride` bytes apart from the row
// at p, at column col. Two neighbouring lanes pair up, one writes both high
// words, the other both low ones. All lanes of a pair call it; live alike.
template <bool BF> __device__ __forceinline__ void mid_store_rows(char *p, long long stride, int col, v4f v, bool live)
{
    if constexpr (BF) {
        const int odd = col & 1;
        char *q = p + (col & ~7) * 4 + (col & 6) * 2 + 16 * odd;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t hi, lo;
            split_pair(v[i], 0.0f, hi, lo);
            const uint32_t both = (hi & 0xFFFFu) | (lo << 16);
            const uint32_t other = __shfl_xor(both, 1);
            const uint32_t w = odd ? (other >> 16) | (both & 0xFFFF0000u) : (both & 0xFFFFu) | (other << 16);
            if (live)
                *reinterpret_cast<uint32_t *>(q + i * stride) = w;
        }
    } else {
        if (live)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                *reinterpret_cast<float *>(p + i * stride + col * 4) = v[i];
    }
}
// sum of the products of two operands' values
__device__ __forceinline__ float mid_dot(const Mid<true> &a, const Mid<true> &b)
{
    u32x4 ah, al, bh, bl;
    __builtin_memcpy(&ah, &a.hi, 16);
    __builtin_memcpy(&al, &a.lo, 16);
    __builtin_memcpy(&bh, &b.hi, 16);
    __builtin_memcpy(&bl, &b.lo, 16);
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        s = fmaf(bf16_lo(ah[j]) + bf16_lo(al[j]), bf16_lo(bh[j]) + bf16_lo(bl[j]), s);
        s = fmaf(bf16_hi(ah[j]) + bf16_hi(al[j]), bf16_hi(bh[j]) + bf16_hi(bl[j]), s);
    }
    return s;
}
__device__ __forceinline__ float mid_dot(const Mid<false> &a, const Mid<false> &b)
{
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        s = fmaf(a.v[j], b.v[j], s);
    return s;
}

// ---- a chunk's rows of q or k in LDS, read down the tokens

// Elements of a row: KD and a pad that spreads a transposing read's four rows
// over the banks.
template <bool BF, int KD> struct Rows {
    static constexpr int LD = BF ? KD + 24 : KD + 4;
    typename std::conditional<BF, uint16_t, float>::type e[64][LD];

    // this lane's 8 elements of row r from element k on
    __device__ __forceinline__ void put(int r, int k, const In<BF> &f)
    {
        __builtin_memcpy(__builtin_assume_aligned(&e[r][k], 16), &f, sizeof f);
    }
    // operand: columns col0 .. + 15, reduction over tokens tok0 .. + 31
    __device__ __forceinline__ In<BF> down(int tok0, int col0) const
    {
        const int l = threadIdx.x & 63, quad = l >> 4, l15 = l & 15;
        In<BF> f;
        if constexpr (BF) {
            s16x4 t[2];
#pragma unroll
            for (int h = 0; h < 2; ++h)
                t[h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (__attribute__((address_space(3))) s16x4 *)(const_cast<uint16_t *>(
                        &e[tok0 + 8 * quad + 4 * h + (l15 >> 2)][col0 + 4 * (l15 & 3)])));
            __builtin_memcpy(&f, t, 16);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                f.v[j] = e[tok0 + 8 * quad + j][col0 + l15];
        }
        return f;
    }
};

// e^(G_i - G_j) of sums kept as two floats
__device__ __forceinline__ float decay(float ihi, float ilo, float jhi, float jlo)
{
    return __expf((ihi - jhi) + (ilo - jlo));
}

}  // namespace srnl_i

#endif
