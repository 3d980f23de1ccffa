// delta_mma.h -- matrix operands of the gated delta rule's chunks.
//
// A 16 x 16 x 32 product: lane l holds, of an operand, 8 consecutive reduction
// elements from 8 (l >> 4) of row (or column) l & 15; of the result, column
// l & 15 in rows 4 (l >> 4) .. + 3. fp32 products run as eight 16 x 16 x 4 ones
// whose reduction order is the same for both operands.
//
// Inputs (In) are bf16 words or fp32 values. What the kernels form between (Mid) is
// fp32, or with bf16 inputs a sum of PL bf16 words: three, right to 2^-27, so that
// results are off by what fp32 sums lose. With two (2^-18) states and gradients were
// off by 2e-6 to 7e-6, and a bf16 output in 400 rounded to the other side. A product
// of two leaves out the pairs of words below its smallest kept one.
#ifndef SRNL_LAYERS_DELTA_MMA_H
#define SRNL_LAYERS_DELTA_MMA_H

#include "delta.h"
#include "linear.h"

namespace srnl_i {

template <bool BF> struct In { bf16x8 v; };
template <> struct In<false> { float v[8]; };
template <bool BF, int PL> struct Mid { bf16x8 p[PL]; };
template <int PL> struct Mid<false, PL> { float v[8]; };
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
template <int PL> __device__ __forceinline__ v4f mma(const In<true> &a, const Mid<true, PL> &b, v4f c)
{
#pragma unroll
    for (int j = PL - 1; j >= 0; --j)
        c = mma16(a.v, b.p[j], c);
    return c;
}
template <int PL> __device__ __forceinline__ v4f mma(const Mid<true, PL> &a, const In<true> &b, v4f c)
{
#pragma unroll
    for (int j = PL - 1; j >= 0; --j)
        c = mma16(a.p[j], b.v, c);
    return c;
}
template <int PL> __device__ __forceinline__ v4f mma(const Mid<true, PL> &a, const Mid<true, PL> &b, v4f c)
{
#pragma unroll
    for (int s = PL - 1; s >= 0; --s)
#pragma unroll
        for (int i = 0; i <= s; ++i)
            c = mma16(a.p[i], b.p[s - i], c);
    return c;
}
__device__ __forceinline__ v4f mma(const In<false> &a, const In<false> &b, v4f c) { return mma16(a.v, b.v, c); }
template <int PL> __device__ __forceinline__ v4f mma(const In<false> &a, const Mid<false, PL> &b, v4f c)
{
    return mma16(a.v, b.v, c);
}
template <int PL> __device__ __forceinline__ v4f mma(const Mid<false, PL> &a, const In<false> &b, v4f c)
{
    return mma16(a.v, b.v, c);
}
template <int PL> __device__ __forceinline__ v4f mma(const Mid<false, PL> &a, const Mid<false, PL> &b, v4f c)
{
    return mma16(a.v, b.v, c);
}

// A result in parts: products of equal significance have a sum of their own, so
// that no product waits for the one before it.
template <bool BF, int PL> struct Sum {
    v4f part[BF ? PL : 1];
    __device__ __forceinline__ Sum()
    {
#pragma unroll
        for (int j = 0; j < (BF ? PL : 1); ++j)
            part[j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    }
    __device__ __forceinline__ void add(const In<BF> &a, const Mid<BF, PL> &b)
    {
        if constexpr (BF) {
#pragma unroll
            for (int j = PL - 1; j >= 0; --j)
                part[j] = mma16(a.v, b.p[j], part[j]);
        } else {
            part[0] = mma16(a.v, b.v, part[0]);
        }
    }
    __device__ __forceinline__ void add(const Mid<BF, PL> &a, const Mid<BF, PL> &b)
    {
        if constexpr (BF) {
#pragma unroll
            for (int i = 0; i < PL; ++i)
#pragma unroll
                for (int s = PL - 1; s >= i; --s)
                    part[s] = mma16(a.p[i], b.p[s - i], part[s]);
        } else {
            part[0] = mma16(a.v, b.v, part[0]);
        }
    }
    __device__ __forceinline__ v4f value() const
    {
        v4f v = part[BF ? PL - 1 : 0];
        if constexpr (BF)
#pragma unroll
            for (int j = PL - 2; j >= 0; --j)
                v += part[j];
        return v;
    }
};

// the value of the lane beside (lane ^ 1), and sums over the 16 lanes of a row
__device__ __forceinline__ float beside(float v)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0xB1, 0xF, 0xF, true));
}
__device__ __forceinline__ uint32_t beside(uint32_t v)
{
    return __builtin_amdgcn_mov_dpp(static_cast<int>(v), 0xB1, 0xF, 0xF, true);
}
template <int CTRL> __device__ __forceinline__ float turned(float v)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
}
__device__ __forceinline__ float sum16(float v)
{
    v += turned<0x128>(v);            // row_ror 8, 4, 2, 1
    v += turned<0x124>(v);
    v += turned<0x122>(v);
    v += turned<0x121>(v);
    return v;
}
__device__ __forceinline__ v4f sum16(v4f v)
{
#pragma unroll
    for (int e = 0; e < 4; ++e)
        v[e] = sum16(v[e]);
    return v;
}

__device__ __forceinline__ v4f v4f_zero() { return v4f{0.0f, 0.0f, 0.0f, 0.0f}; }

// ---- memory
//
// Loads and stores go through buffer descriptors over 2 GB from a base that the
// whole wave shares: a lane that has nothing there gives an offset past the end,
// reads 0 and writes nothing. No branch parts the loads, so that none is waited for
// before its value is used.

constexpr unsigned NOWHERE = 0x80000000u;
// a && b without the branch
__device__ __forceinline__ bool both(bool a, bool b) { return (static_cast<int>(a) & static_cast<int>(b)) != 0; }
struct Buf {
    __amdgpu_buffer_rsrc_t r;
    __device__ __forceinline__ Buf(const void *base, long long byte)
        : r(__builtin_amdgcn_make_buffer_rsrc(const_cast<char *>(static_cast<const char *>(base)) + byte, 0, 0x7FFFFFF0,
                                              0x00020000))
    {
    }
};
__device__ __forceinline__ u32x4 buf16(const Buf &b, unsigned o)
{
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(b.r, o, 0, 0));
}

// a value at element o
template <bool BF> __device__ __forceinline__ void put_value(const Buf &b, int o, bool live, float v)
{
    if constexpr (BF)
        __builtin_amdgcn_raw_buffer_store_b16(to_bf16(v), b.r, live ? 2u * o : NOWHERE, 0, 0);
    else
        __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, v), b.r, live ? 4u * o : NOWHERE, 0, 0);
}
// The states and errors that forward records, and their gradients, lie in panels of 8
// columns: element of a row and column, of rows rows.
__device__ __forceinline__ int record_at(int row, int col, int rows) { return ((col >> 3) * rows + row) * 8 + (col & 7); }
// They are stored past the caches (the nt bit): written as others are, they put q, k, X
// and P, which a head's blocks share, out of the L2, and the chain takes 167 us forward
// and 192 back at 4 x 4096 x 8 heads of 128, not 145 and 172.
constexpr int NT_STORE = 2;
// four or eight fp32 values from o on, a multiple of 4
__device__ __forceinline__ void put4(const Buf &b, int o, bool live, v4f v)
{
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), b.r, live ? 4u * o : NOWHERE, 0, NT_STORE);
}
__device__ __forceinline__ void put8(const Buf &b, int o, bool live, const float (&v)[8])
{
    put4(b, o, live, v4f{v[0], v[1], v[2], v[3]});
    put4(b, o + 4, live, v4f{v[4], v[5], v[6], v[7]});
}
// a value by its address, for what no loop waits for
template <bool BF> __device__ __forceinline__ void put_at(void *p, long long o, float v)
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
template <bool BF> __device__ __forceinline__ In<BF> in_load(const Buf &b, int o, bool live)
{
    In<BF> f;
    const unsigned at = live ? static_cast<unsigned>(o) * (BF ? 2u : 4u) : NOWHERE;
    u32x4 t[BF ? 1 : 2];
    t[0] = buf16(b, at);
    if constexpr (!BF)
        t[1] = buf16(b, at + 16);
    __builtin_memcpy(&f, t, sizeof f);
    return f;
}
// ---- split values

// An operand of X or P in memory lies as a wave reads it, 16 bytes a lane after
// 16 bytes a lane: rows of 64 values would have every lane of a load on a cache line
// of its own, and the loads, not the products, set the chain's pace.
template <bool BF, int PL> constexpr int frag_bytes = (BF ? PL : 2) * 1024;
template <bool BF, int PL> __device__ __forceinline__ Mid<BF, PL> frag_load(const Buf &b, int frag)
{
    Mid<BF, PL> f;
    u32x4 t[BF ? PL : 2];
    const unsigned at = frag * frag_bytes<BF, PL> + 16u * (threadIdx.x & 63);
#pragma unroll
    for (int j = 0; j < (BF ? PL : 2); ++j)
        t[j] = buf16(b, at + 1024 * j);
    __builtin_memcpy(&f, t, sizeof f);
    return f;
}
// the PL words of two values, from the largest
template <int PL> __device__ __forceinline__ void split_pair(float a, float b, uint32_t (&w)[PL])
{
#pragma unroll
    for (int j = 0; j < PL; ++j) {
        w[j] = pack_bf16(a, b);
        if (j + 1 < PL) {
            a -= bf16_lo(w[j]);
            b -= bf16_hi(w[j]);
        }
    }
}
template <bool BF, int PL> __device__ __forceinline__ Mid<BF, PL> mid_split(const float (&v)[8])
{
    Mid<BF, PL> f;
    if constexpr (BF) {
        u32x4 t[PL];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t w[PL];
            split_pair<PL>(v[2 * j], v[2 * j + 1], w);
#pragma unroll
            for (int k = 0; k < PL; ++k)
                t[k][j] = w[k];
        }
        __builtin_memcpy(&f, t, sizeof f);
    } else {
        __builtin_memcpy(&f, v, sizeof f);
    }
    return f;
}
// past: past the caches
template <bool BF, int PL> __device__ __forceinline__ void frag_store(const Buf &b, int frag, const float (&v)[8], bool past)
{
    const Mid<BF, PL> f = mid_split<BF, PL>(v);
    u32x4 t[sizeof f / 16];
    __builtin_memcpy(t, &f, sizeof f);
    const unsigned at = frag * frag_bytes<BF, PL> + 16u * (threadIdx.x & 63);
#pragma unroll
    for (unsigned j = 0; j < sizeof f / 16; ++j)
        if (past)
            __builtin_amdgcn_raw_buffer_store_b128(t[j], b.r, at + 1024 * j, 0, NT_STORE);
        else
            __builtin_amdgcn_raw_buffer_store_b128(t[j], b.r, at + 1024 * j, 0, 0);
}
// ROWS rows of K split values in LDS, a plane for each word. Rows are 32 bytes longer
// than their values, so that 16 rows' reads of one piece of 16 bytes meet no bank
// twice (16 bytes suit writes of 8 bytes a lane better, 73 cycles and not 82, but the
// kernels read more: the gradient kernel takes as long with either).
template <bool BF, int PL, int ROWS, int K> struct Split {
    static constexpr int PLANES = BF ? PL : 1, ROW = K * (BF ? 2 : 4) + 32;
    __attribute__((aligned(16))) char b[PLANES][ROWS][ROW];

    // 8 values of row r from piece g on
    __device__ __forceinline__ Mid<BF, PL> get(int r, int g) const
    {
        Mid<BF, PL> f;
        u32x4 t[BF ? PL : 2];
        if constexpr (BF) {
#pragma unroll
            for (int p = 0; p < PL; ++p)
                t[p] = *reinterpret_cast<const u32x4 *>(&b[p][r][16 * g]);
        } else {
            t[0] = *reinterpret_cast<const u32x4 *>(&b[0][r][32 * g]);
            t[1] = *reinterpret_cast<const u32x4 *>(&b[0][r][32 * g + 16]);
        }
        __builtin_memcpy(&f, t, sizeof f);
        return f;
    }
    // 8 rows from r0 on of element k0 + (lane & 15), as fp32: three words hold all bits
    // of a normal fp32 value. Lanes of a quad have r0 and k0 in common.
    __device__ __forceinline__ void down(int r0, int k0, float (&v)[8]) const
    {
        const int l15 = threadIdx.x & 15;
        if constexpr (BF) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                u32x2 w[PL];
#pragma unroll
                for (int p = 0; p < PL; ++p)
                    w[p] = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                        (__attribute__((address_space(3))) s16x4 *)(const_cast<char *>(
                            &b[p][r0 + 4 * h + (l15 >> 2)][2 * (k0 + 4 * (l15 & 3))]))));
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float lo = bf16_lo(w[PL - 1][j]), hi = bf16_hi(w[PL - 1][j]);
#pragma unroll
                    for (int p = PL - 2; p >= 0; --p) {
                        lo += bf16_lo(w[p][j]);
                        hi += bf16_hi(w[p][j]);
                    }
                    v[4 * h + 2 * j] = lo;
                    v[4 * h + 2 * j + 1] = hi;
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] = *reinterpret_cast<const float *>(&b[0][r0 + j][4 * (k0 + l15)]);
        }
    }
    // one-word values: inputs
    __device__ __forceinline__ In<BF> get_in(int r, int g) const
    {
        In<BF> f;
        __builtin_memcpy(&f, __builtin_assume_aligned(&b[0][r][(BF ? 16 : 32) * g], 16), sizeof f);
        return f;
    }
    __device__ __forceinline__ void put_in(int r, int g, const In<BF> &f)
    {
        __builtin_memcpy(__builtin_assume_aligned(&b[0][r][(BF ? 16 : 32) * g], 16), &f, sizeof f);
    }
    // 8 fp32 values to piece g of row r
    __device__ __forceinline__ void put8(int r, int g, const float (&v)[8])
    {
        const Mid<BF, PL> f = mid_split<BF, PL>(v);
        u32x4 t[sizeof f / 16];
        __builtin_memcpy(t, &f, sizeof f);
        if constexpr (BF) {
#pragma unroll
            for (int p = 0; p < PL; ++p)
                *reinterpret_cast<u32x4 *>(&b[p][r][16 * g]) = t[p];
        } else {
            *reinterpret_cast<u32x4 *>(&b[0][r][32 * g]) = t[0];
            *reinterpret_cast<u32x4 *>(&b[0][r][32 * g + 16]) = t[1];
        }
    }
    // a result tile's column as a row of its transpose: 4 values of row r at place k,
    // a multiple of 4
    __device__ __forceinline__ void put4(int r, int k, v4f v)
    {
        if constexpr (BF) {
            uint32_t x[PL], y[PL];
            split_pair<PL>(v[0], v[1], x);
            split_pair<PL>(v[2], v[3], y);
#pragma unroll
            for (int p = 0; p < PL; ++p)
                *reinterpret_cast<u32x2 *>(&b[p][r][2 * k]) = u32x2{x[p], y[p]};
        } else {
            *reinterpret_cast<v4f *>(&b[0][r][4 * k]) = v;
        }
    }
    // a result tile as it lies: this lane's rows r .. r + 3 at column k. Lanes of
    // neighbouring columns exchange, so that each writes whole words: two rows of
    // both columns. All lanes of a pair call it.
    __device__ __forceinline__ void put_rows(int r, int k, v4f v)
    {
        if constexpr (BF) {
            const int odd = k & 1;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float mine = odd ? v[2 + i] : v[i], give = odd ? v[i] : v[2 + i];
                const float got = beside(give);
                uint32_t w[PL];
                split_pair<PL>(odd ? got : mine, odd ? mine : got, w);
#pragma unroll
                for (int p = 0; p < PL; ++p)
                    *reinterpret_cast<uint32_t *>(&b[p][r + 2 * odd + i][2 * (k - odd)]) = w[p];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                *reinterpret_cast<float *>(&b[0][r + i][4 * k]) = v[i];
        }
    }
};
// 8 fp32 values from memory, o in values, zeros where not live
__device__ __forceinline__ void load8(const Buf &b, int o, bool live, float (&v)[8])
{
    const unsigned at = live ? 4u * o : NOWHERE;
    const u32x4 t[2] = {buf16(b, at), buf16(b, at + 16)};
    __builtin_memcpy(v, t, 32);
}

// ---- a chunk's rows of q or k in LDS, read down the tokens

// Elements of a row: KD and a pad that spreads over the banks the four rows of a
// transposing read and the 16 of a plain one.
template <bool BF, int KD> struct Rows {
    static constexpr int LD = BF ? KD + 16 : KD + 4;
    typename std::conditional<BF, uint16_t, float>::type e[64][LD];

    // this lane's 8 elements of row r from element k on
    __device__ __forceinline__ void put(int r, int k, const In<BF> &f)
    {
        __builtin_memcpy(__builtin_assume_aligned(&e[r][k], 16), &f, sizeof f);
    }
    // operand: row r, reduction along it from element k on
    __device__ __forceinline__ In<BF> across(int r, int k) const
    {
        In<BF> f;
        __builtin_memcpy(&f, __builtin_assume_aligned(&e[r][k], 16), sizeof f);
        return f;
    }
    // as a result tile lies: rows row0 + 4 quad .. + 3 of column col0 + (lane & 15)
    __device__ __forceinline__ v4f tile(int row0, int col0) const
    {
        const int l = threadIdx.x & 63, quad = l >> 4, l15 = l & 15;
        v4f v;
        if constexpr (BF) {
            const s16x4 t = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (__attribute__((address_space(3))) s16x4 *)(const_cast<uint16_t *>(
                    &e[row0 + 4 * quad + (l15 >> 2)][col0 + 4 * (l15 & 3)])));
            const u32x2 w = __builtin_bit_cast(u32x2, t);
            v = v4f{bf16_lo(w[0]), bf16_hi(w[0]), bf16_lo(w[1]), bf16_hi(w[1])};
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] = e[row0 + 4 * quad + i][col0 + l15];
        }
        return v;
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

// e^(G_i - G_j) of sums kept as two floats. The fast exponential is off by |x| 2^-24 of
// e^x besides its last place: at most 0.4 2^-24 of 1, what a term is rounded by.
__device__ __forceinline__ float decay(float ihi, float ilo, float jhi, float jlo)
{
    return __expf((ihi - jhi) + (ilo - jlo));
}

}  // namespace srnl_i

#endif
