// linear.hip -- the linear layer with bias, activation and residual in
// its epilogue, forward and backward. Entry points as declared in
// include/srnl.h.
//
//   z = x W^T + b,  y = act(z) + residual
//   dz = dy act'(z);  dx = dz W [+ add],  dW = dz^T x,  db = sum over rows of dz
//
// All three products run on v_mfma_f32_32x32x16_bf16 with fp32 accumulators
// in one tiled kernel (linear_tile_kernel). A bf16 operand is its own MFMA
// operand. An fp32 operand is split while it is staged into three bf16 parts,
// x = h + m + l with h = bf16(x), m = bf16(x - h), l = x - h - m, all exact
// in round to nearest (8 significant bits each, |m| <= 2^-9 |x|,
// |l| <= 2^-18 |x|), so a product with a bf16 operand takes three MFMAs and
// is exact, and a product of two fp32 operands takes the six with
// part indices p + q <= 2: what is left out (m l, l m, l l) is below
// 2^-26 |x w|, a quarter of an fp32 rounding. Six bf16 MFMAs are 2.7 times
// faster than one fp32 MFMA of the same shape.
//
// A few rows (or few output tiles) go to linear_few_kernel, which splits the
// reduction over the waves of a block and joins them in LDS.
#include "common.h"

namespace {

using namespace srnl_i;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

// ------------------------------------------------------------ activations

// 1 - Phi(|z|) of the standard normal, from formula 7.1.26 of Abramowitz and
// Stegun (Handbook of Mathematical Functions), |error| <= 0.75e-7:
// erfc(x) = t (a1 + t (a2 + t (a3 + t (a4 + t a5)))) exp(-x^2),
// t = 1 / (1 + p x), x = |z| / sqrt 2. ex returns exp(-z^2 / 2).
__device__ __forceinline__ float normal_tail(float z, float &ex)
{
    const float x = fabsf(z) * 0.70710678118654752f;
    const float t = __builtin_amdgcn_rcpf(fmaf(0.3275911f, x, 1.0f));
    float p = fmaf(t, 1.061405429f, -1.453152027f);
    p = fmaf(t, p, 1.421413741f);
    p = fmaf(t, p, -0.284496736f);
    p = fmaf(t, p, 0.254829592f);
    ex = __expf(-0.5f * z * z);
    return 0.5f * t * p * ex;
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

// dz = dy act'(z), the pre-pass of the backward products
__global__ __launch_bounds__(256) void act_slope_kernel(const void *__restrict__ dy, bool dybf,
                                                        const float *__restrict__ z, int act,
                                                        long long n, float *__restrict__ dz)
{
    for (long long o = 8 * (blockIdx.x * 256LL + threadIdx.x); o < n; o += 8 * 256LL * gridDim.x) {
        const int m = n - o < 8 ? static_cast<int>(n - o) : 8;
        float a[8], b[8];
        load_row<8, false>(dy, dybf, o, m, a);
        load_row<8, false>(z, false, o, m, b);
        act_slopes(b, act, a);
        store_row<8, false>(dz, false, o, m, a);
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

// 16 bytes that lanes read in place of pieces outside an operand
__device__ __align__(16) const uint32_t zero_piece[4] = {0, 0, 0, 0};

// One operand as memory: element (row, r) is at row * ld + r (reduction
// contiguous, RC) or r * ld + row.
struct Operand {
    const void *p;
    long long ld;
    long long rows;       // output rows (or columns) of this operand
};

// A tile of ROWS x BK of an operand, staged in LDS as PARTS planes of bf16.
// RC: plane[row][BK], 16-byte pieces of a row permuted so that 16 consecutive
// rows' reads of one piece fall on all 64 banks. Not RC: plane[r][ROWS] as
// in memory, the 64-byte blocks of a row permuted by r, read through the
// transposing LDS read (ds_read_b64_tr_b16: of the 4 x 16 block that 16
// lanes address, each lane gets a column).
template <bool F32, bool RC, int ROWS, int BK, bool ALIGNED> struct Tile {
    static constexpr int PARTS = F32 ? 3 : 1;
    static constexpr bool ASYNC = ALIGNED && !F32;        // straight from memory into LDS
    static constexpr int PLANE = ROWS * BK;               // words
    static constexpr int PIECES = PLANE / 8 / 256;        // 8-element pieces per thread
    static_assert(PIECES >= 1 && PIECES * 256 * 8 == PLANE, "pieces divide evenly");
    static constexpr int PER = RC ? BK / 8 : ROWS / 8;    // pieces per stored row

    float v[F32 ? PIECES : 1][8];
    u32x4 raw[F32 ? 1 : PIECES];

    static __device__ __forceinline__ int place(int major, int c)
    {
        if (RC) {
            constexpr int RP = 16 / PER;                  // rows per 256 bytes
            return c ^ ((major / RP) & (PER - 1));
        }
        constexpr int NB = ROWS / 32, RPB = 4 / NB;       // 64-byte blocks a row, rows per 256 bytes
        return c ^ (4 * ((major / RPB) & (NB - 1)));
    }

    // start fetching the tile at (row0, r0); ASYNC: into buf
    __device__ __forceinline__ void fetch(const Operand &o, long long row0, long long r0, long long rend,
                                          uint16_t *buf)
    {
        const int tid = threadIdx.x;
#pragma unroll
        for (int q = 0; q < PIECES; ++q) {
            const int s = tid + 256 * q;
            const int major = s / PER, c = ASYNC ? place(major, s % PER) : s % PER;
            const long long row = row0 + (RC ? major : 8 * c), r = r0 + (RC ? 8 * c : major);
            if constexpr (ASYNC) {
                const uint16_t *src = reinterpret_cast<const uint16_t *>(zero_piece);
                if (row < o.rows && r < rend)
                    src = static_cast<const uint16_t *>(o.p) + (RC ? row * o.ld + r : r * o.ld + row);
                // lane l of the wave writes base + 16 l
                uint16_t *dst = buf + 8 * (256 * q + (tid & ~63));
                __builtin_amdgcn_global_load_lds(
                    reinterpret_cast<const __attribute__((address_space(1))) void *>(
                        reinterpret_cast<uintptr_t>(src)),
                    (__attribute__((address_space(3))) void *)dst, 16, 0, 0);
            } else {
                const long long left = RC ? rend - r : o.rows - row;
                const bool in = RC ? row < o.rows : r < rend;
                const int n = !in || left <= 0 ? 0 : left < 8 ? static_cast<int>(left) : 8;
                const long long at = RC ? row * o.ld + r : r * o.ld + row;
                if constexpr (F32) {
                    load_row<8, ALIGNED>(o.p, false, at, n, v[q]);
                } else {
                    raw[q] = u32x4{0, 0, 0, 0};
                    const uint16_t *src = static_cast<const uint16_t *>(o.p) + at;
                    if (n == 8) {
                        __builtin_memcpy(&raw[q], src, 16);
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (e < n)
                                raw[q][e / 2] |= static_cast<uint32_t>(src[e]) << (16 * (e & 1));
                    }
                }
            }
        }
    }
    // write what fetch holds in registers to buf
    __device__ __forceinline__ void commit(uint16_t *buf) const
    {
        if constexpr (!ASYNC) {
#pragma unroll
            for (int q = 0; q < PIECES; ++q) {
                const int s = threadIdx.x + 256 * q;
                const int major = s / PER;
                uint16_t *dst = buf + 8 * (major * PER + place(major, s % PER));
                if constexpr (F32) {
                    u32x4 w[3];
                    split_parts(v[q], w);
#pragma unroll
                    for (int p = 0; p < 3; ++p)
                        *reinterpret_cast<u32x4 *>(dst + p * PLANE) = w[p];
                } else {
                    *reinterpret_cast<u32x4 *>(dst) = raw[q];
                }
            }
        }
    }
    // MFMA operand: rows row0 .. row0 + 31 (row0 a multiple of 32), reduction
    // indices 16 kk + (0..15) of plane p: lane l holds row l % 32, indices
    // 8 (l / 32) + e
    static __device__ __forceinline__ bf16x8 frag(const uint16_t *buf, int p, int row0, int kk)
    {
        const int l = threadIdx.x & 63;
        const uint16_t *b = buf + p * PLANE;
        if constexpr (RC) {
            const int row = row0 + (l & 31);
            return *reinterpret_cast<const bf16x8 *>(b + 8 * (row * PER + place(row, 2 * kk + (l >> 5))));
        } else {
            const int r = 16 * kk + 8 * (l >> 5) + ((l & 15) >> 2);
            const int at = r * ROWS + 8 * place(r, row0 / 8) + 16 * ((l >> 4) & 1) + 4 * (l & 3);
            s16x4 t[2];
#pragma unroll
            for (int h = 0; h < 2; ++h)     // r + 4: same permutation
                t[h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (__attribute__((address_space(3))) s16x4 *)(const_cast<uint16_t *>(b) + at + 4 * h * ROWS));
            bf16x8 f;
            __builtin_memcpy(&f, t, 16);
            return f;
        }
    }
};

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

// eight neighbouring outputs (i, j .. j + 7) from their sums; n are inside
template <bool ALIGNED>
__device__ __forceinline__ void finish8(const Epilogue &e, long long o, int j, int n, float (&v)[8])
{
    if (n <= 0)
        return;
    if (e.bias) {
        float b[8];
        load_row<8, ALIGNED>(e.bias, false, j, n, b);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            v[k] += b[k];
    }
    if (e.pre)
        store_row<8, ALIGNED>(e.pre, false, o, n, v);
    act_values(v, e.act);
    if (e.add) {
        float a[8];
        load_row<8, ALIGNED>(e.add, e.abf, o, n, a);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            v[k] += a[k];
    }
    store_row<8, ALIGNED>(e.out, e.obf, o, n, v);
}

// ------------------------------------------------------------ tiled product

struct TileArgs {
    Operand a, b;          // out[i][j] = sum over r of a(i, r) b(j, r)
    long long R;           // reduction length
    long long slice;       // reduction length per split, a multiple of BK
    int splits;
    int ti, tj;            // output tiles
    float *part;           // [splits][I][J] partial sums instead of the epilogue, or NULL
    float *rowsum;         // [splits][I]: sums of a's rows over r (the bias gradient), or NULL
    Epilogue e;
};

// Block order: consecutive blocks go to the card's eight dies in turn, so die
// d takes the d-th eighth of the tiles; neighbouring tiles, which share an
// operand's rows, then share a die's L2 cache.
__device__ __forceinline__ unsigned die_order(unsigned id, unsigned n)
{
    const unsigned q = n / 8, rem = n % 8, d = id % 8, k = id / 8;
    return d * q + (d < rem ? d : rem) + k;
}

// Barrier after staging; a direct load into LDS counts as a vector load, which
// the barrier alone does not wait for.
template <bool DIRECT> __device__ __forceinline__ void tile_barrier()
{
    if (DIRECT)
        __builtin_amdgcn_s_waitcnt(0x0F70);      // vmcnt(0)
    __syncthreads();
}

// BI x BJ output tile per block of four waves (2 x 2), BI / 2 x BJ / 2 each,
// in 32 x 32 MFMA tiles. An operand that goes straight to LDS is fetched one
// step ahead into the other buffer; one that is converted waits in registers.
template <bool AF, bool BF, bool RCA, bool RCB, int BI, int BJ, bool ALIGNED, bool SUMS>
__global__ __launch_bounds__(256) void linear_tile_kernel(TileArgs g)
{
    constexpr int BK = (AF || BF) ? 32 : 64;
    using TA = Tile<AF, RCA, BI, BK, ALIGNED>;
    using TB = Tile<BF, RCB, BJ, BK, ALIGNED>;
    constexpr int NBUF = (TA::ASYNC || TB::ASYNC) ? 2 : 1;
    constexpr int PA = TA::PARTS, PB = TB::PARTS;
    constexpr int FI = BI / 64, FJ = BJ / 64;                   // 32 x 32 tiles per wave
    constexpr int WORDS = NBUF * (PA * TA::PLANE + PB * TB::PLANE);
    constexpr int OUTP = 32 * FJ + 4;                           // floats per staged output row
    constexpr int OUT_WORDS = 4 * 32 * OUTP * 2;
    __shared__ __align__(16) uint16_t lds[WORDS > OUT_WORDS ? WORDS : OUT_WORDS];
    uint16_t *const la = lds, *const lb = lds + NBUF * PA * TA::PLANE;

    const unsigned t = die_order(blockIdx.x, gridDim.x);
    const int tj = t % g.tj, ti = (t / g.tj) % g.ti, sp = t / (g.tj * g.ti);
    const long long i0 = static_cast<long long>(ti) * BI, j0 = static_cast<long long>(tj) * BJ;
    const long long rb = sp * g.slice, re = rb + g.slice < g.R ? rb + g.slice : g.R;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int wi = (wave >> 1) * 32 * FI, wj = (wave & 1) * 32 * FJ;
    const bool sums = SUMS && g.rowsum && tj == 0 && wj == 0;

    TA ta;
    TB tb;
    v16f acc[FI][FJ], rs[SUMS ? FI : 1];
#pragma unroll
    for (int i = 0; i < FI; ++i)
#pragma unroll
        for (int j = 0; j < FJ; ++j)
#pragma unroll
            for (int k = 0; k < 16; ++k)
                acc[i][j][k] = 0.0f;
#pragma unroll
    for (int i = 0; i < (SUMS ? FI : 1); ++i)
#pragma unroll
        for (int k = 0; k < 16; ++k)
            rs[i][k] = 0.0f;
    bf16x8 ones;
    {
        const u32x4 w = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
        ones = __builtin_bit_cast(bf16x8, w);
    }

    ta.fetch(g.a, i0, rb, re, la);
    tb.fetch(g.b, j0, rb, re, lb);
    ta.commit(la);
    tb.commit(lb);
    int cur = 0;
    tile_barrier<NBUF == 2>();
    for (long long r = rb; r < re; r += BK) {
        uint16_t *const ca = la + cur * PA * TA::PLANE, *const cb = lb + cur * PB * TB::PLANE;
        const int nxt = NBUF == 2 ? cur ^ 1 : 0;
        uint16_t *const na = la + nxt * PA * TA::PLANE, *const nb = lb + nxt * PB * TB::PLANE;
        const bool more = r + BK < re;
        if (more) {
            ta.fetch(g.a, i0, r + BK, re, na);
            tb.fetch(g.b, j0, r + BK, re, nb);
        }
#pragma unroll
        for (int kk = 0; kk < BK / 16; ++kk) {
            bf16x8 fa[FI][PA], fb[FJ][PB];
#pragma unroll
            for (int i = 0; i < FI; ++i)
#pragma unroll
                for (int p = 0; p < PA; ++p)
                    fa[i][p] = TA::frag(ca, p, wi + 32 * i, kk);
#pragma unroll
            for (int j = 0; j < FJ; ++j)
#pragma unroll
                for (int p = 0; p < PB; ++p)
                    fb[j][p] = TB::frag(cb, p, wj + 32 * j, kk);
            // smallest parts first
#pragma unroll
            for (int s = 2; s >= 0; --s)
#pragma unroll
                for (int p = 0; p < PA; ++p) {
                    const int q = s - p;
                    if (q < 0 || q >= PB)
                        continue;
#pragma unroll
                    for (int i = 0; i < FI; ++i)
#pragma unroll
                        for (int j = 0; j < FJ; ++j)
                            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[i][p], fb[j][q],
                                                                                acc[i][j], 0, 0, 0);
                }
            if (SUMS && sums) {
#pragma unroll
                for (int i = 0; i < (SUMS ? FI : 1); ++i)
#pragma unroll
                    for (int p = PA - 1; p >= 0; --p)
                        rs[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[i][p], ones, rs[i], 0, 0, 0);
            }
        }
        if (NBUF == 1)
            __syncthreads();                 // everyone has read the only buffer
        if (more) {
            ta.commit(na);
            tb.commit(nb);
        }
        cur = nxt;
        tile_barrier<NBUF == 2>();
    }

    if (SUMS && sums && (lane & 31) == 0) {  // every column of rs holds the sums
#pragma unroll
        for (int i = 0; i < (SUMS ? FI : 1); ++i)
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const long long row = i0 + wi + 32 * i + 8 * (k / 4) + 4 * (lane >> 5) + k % 4;
                if (row < g.a.rows)
                    g.rowsum[sp * g.a.rows + row] = rs[i][k];
            }
    }

    // each wave turns its 32-row slabs through its own part of LDS, so that a
    // lane finishes eight neighbouring outputs with 16-byte accesses
    float *const st = reinterpret_cast<float *>(lds) + wave * 32 * OUTP;
    Epilogue e = g.e;
    if (g.part) {
        e = Epilogue{};
        e.out = g.part + sp * g.a.rows * g.b.rows;
    }
#pragma unroll
    for (int i = 0; i < FI; ++i) {
#pragma unroll
        for (int j = 0; j < FJ; ++j)
#pragma unroll
            for (int k = 0; k < 16; ++k)
                st[(8 * (k / 4) + 4 * (lane >> 5) + k % 4) * OUTP + 32 * j + (lane & 31)] = acc[i][j][k];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        constexpr int LPR = 4 * FJ;                             // lanes per row
#pragma unroll 2
        for (int q = 0; q < 32 * LPR / 64; ++q) {
            const int row = q * (64 / LPR) + lane / LPR, c = 8 * (lane % LPR);
            float v[8];
            load_f32<8, true>(st + row * OUTP + c, v);
            const long long oi = i0 + wi + 32 * i + row;
            const long long oj = j0 + wj + c;
            const long long left = g.b.rows - oj;
            if (oi < g.a.rows)
                finish8<ALIGNED>(e, oi * g.b.rows + oj, static_cast<int>(oj),
                                 left < 8 ? static_cast<int>(left) : 8, v);
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
}

// out = sum of the splits' partial products through the epilogue, in order
__global__ __launch_bounds__(256) void join_kernel(const float *__restrict__ part, int splits, long long n,
                                                   Epilogue e)
{
    for (long long o = 8 * (blockIdx.x * 256LL + threadIdx.x); o < n; o += 8 * 256LL * gridDim.x) {
        const int m = n - o < 8 ? static_cast<int>(n - o) : 8;
        float v[8];
        load_row<8, false>(part, false, o, m, v);
#pragma unroll 4
        for (int s = 1; s < splits; ++s) {
            float w[8];
            load_row<8, false>(part, false, s * n + o, m, w);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                v[k] += w[k];
        }
        finish8<false>(e, o, 0, m, v);
    }
}

// ------------------------------------------------------------ few rows

// 16 MI rows by 16 columns of the output per block; its eight waves take the
// reduction in turns of 64 or 128 indices, straight from memory into MFMA operands
// (v_mfma_f32_16x16x32_bf16), and join through LDS in wave order.
constexpr int kFewWaves = 8;

template <bool F32, bool ALIGNED>
__device__ __forceinline__ void few_load(const Operand &o, long long row, long long r, long long R,
                                         u32x4 (&w)[3])
{
    const long long left = R - r;
    const int n = row >= o.rows || left <= 0 ? 0 : left < 8 ? static_cast<int>(left) : 8;
    const long long at = row * o.ld + r;
    if constexpr (F32) {
        float v[8];
        load_row<8, ALIGNED>(o.p, false, at, n, v);
        split_parts(v, w);
    } else {
        w[0] = u32x4{0, 0, 0, 0};
        const uint16_t *src = static_cast<const uint16_t *>(o.p) + at;
        if (ALIGNED ? n > 0 : n == 8) {
            if (ALIGNED)
                w[0] = *reinterpret_cast<const u32x4 *>(src);
            else
                __builtin_memcpy(&w[0], src, 16);
        } else if (!ALIGNED) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < n)
                    w[0][e / 2] |= static_cast<uint32_t>(src[e]) << (16 * (e & 1));
        }
    }
}

template <bool AF, bool BF, int MI, bool ALIGNED>
__global__ __launch_bounds__(64 * kFewWaves) void linear_few_kernel(TileArgs g)
{
    constexpr int PA = AF ? 3 : 1, PB = BF ? 3 : 1;
    constexpr int P = 20;                                       // floats per staged row of 16
    __shared__ __align__(16) float red[kFewWaves][16 * MI * P];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, rl = lane & 15, g8 = 8 * (lane >> 4);
    const int tj = blockIdx.x % g.tj;
    const long long i0 = static_cast<long long>(blockIdx.x / g.tj) * 16 * MI, j0 = 16LL * tj;
    v4f acc[MI];
#pragma unroll
    for (int i = 0; i < MI; ++i)
        acc[i] = v4f{0.f, 0.f, 0.f, 0.f};
    constexpr int U = MI == 1 ? 4 : 2;                          // pieces in flight
    for (long long r = 32LL * U * wave; r < g.R; r += 32LL * U * kFewWaves) {
        u32x4 wb[U][3], wa[U][MI][3];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            few_load<BF, ALIGNED>(g.b, j0 + rl, r + 32 * u + g8, g.R, wb[u]);
#pragma unroll
            for (int i = 0; i < MI; ++i)
                few_load<AF, ALIGNED>(g.a, i0 + 16 * i + rl, r + 32 * u + g8, g.R, wa[u][i]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int s = 2; s >= 0; --s)
#pragma unroll
                    for (int p = 0; p < PA; ++p) {
                        const int q = s - p;
                        if (q < 0 || q >= PB)
                            continue;
                        acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            __builtin_bit_cast(bf16x8, wa[u][i][p]), __builtin_bit_cast(bf16x8, wb[u][q]),
                            acc[i], 0, 0, 0);
                    }
    }
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k)
            red[wave][(16 * i + 4 * (lane >> 4) + k) * P + rl] = acc[i][k];
    __syncthreads();
    const int row = threadIdx.x >> 1, c = 8 * (threadIdx.x & 1);
    if (row >= 16 * MI || i0 + row >= g.a.rows)
        return;
    float v[8];
    load_f32<8, true>(&red[0][row * P + c], v);
#pragma unroll
    for (int w = 1; w < kFewWaves; ++w) {
        float t[8];
        load_f32<8, true>(&red[w][row * P + c], t);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            v[k] += t[k];
    }
    const long long left = g.b.rows - (j0 + c);
    finish8<ALIGNED>(g.e, (i0 + row) * g.b.rows + j0 + c, static_cast<int>(j0 + c),
                     left < 8 ? static_cast<int>(left) : 8, v);
}

// ------------------------------------------------------------ host

long long cdiv(long long a, long long b) { return (a + b - 1) / b; }

enum Form { FORWARD, GRAD_X, GRAD_W };     // which operands have the reduction contiguous

struct Plan {
    bool aligned;
    int bi;                // tile side
    int splits;
    long long slice;
    long long ti, tj;
};

// Tile and split of out[I][J] over R. 128 x 128 tiles where they give every CU
// one, else 64 x 64. The reduction is split where the tiles leave CUs idle
// (the weight gradient over many tokens; an input gradient of few rows), as
// long as a split keeps at least four staged steps.
Plan plan_tile(Form f, long long I, long long J, long long R, bool af, bool bf, bool aligned)
{
    Plan p;
    p.aligned = aligned;
    const int bk = af || bf ? 32 : 64;
    const long long big = cdiv(I, 128) * cdiv(J, 128);
    p.bi = aligned && (big >= 256 || (f == GRAD_W && big * cdiv(R, 8 * bk) >= 256 && I >= 96 && J >= 96)) ? 128 : 64;
    p.ti = cdiv(I, p.bi);
    p.tj = cdiv(J, p.bi);
    const long long tiles = p.ti * p.tj;
    long long s = f == FORWARD ? 1 : tiles >= 256 ? 1 : 256 / tiles;
    const long long most = cdiv(R, 4 * bk);
    s = s < most ? s : most;
    s = s < 1 ? 1 : s;
    p.slice = cdiv(cdiv(R, s), bk) * bk;
    p.splits = static_cast<int>(cdiv(R, p.slice));
    return p;
}

template <bool AF, bool BF, Form F>
void launch_tile(const TileArgs &g, const Plan &p, hipStream_t st)
{
    constexpr bool RCA = F != GRAD_W, RCB = F == FORWARD, SUMS = F == GRAD_W;
    const dim3 grid(static_cast<unsigned>(p.ti * p.tj * p.splits)), block(256);
    if (!p.aligned)
        hipLaunchKernelGGL((linear_tile_kernel<AF, BF, RCA, RCB, 64, 64, false, SUMS>), grid, block, 0, st, g);
    else if (p.bi == 128)
        hipLaunchKernelGGL((linear_tile_kernel<AF, BF, RCA, RCB, 128, 128, true, SUMS>), grid, block, 0, st, g);
    else
        hipLaunchKernelGGL((linear_tile_kernel<AF, BF, RCA, RCB, 64, 64, true, SUMS>), grid, block, 0, st, g);
}

template <Form F>
srnl_status run_tile(TileArgs g, const Plan &p, bool af, bool bf, hipStream_t st)
{
    g.slice = p.slice;
    g.splits = p.splits;
    g.ti = static_cast<int>(p.ti);
    g.tj = static_cast<int>(p.tj);
    if (af && bf) launch_tile<true, true, F>(g, p, st);
    else if (af) launch_tile<true, false, F>(g, p, st);
    else if (bf) launch_tile<false, true, F>(g, p, st);
    else launch_tile<false, false, F>(g, p, st);
    return launched("linear_tile_kernel");
}

template <bool AF, bool BF>
void launch_few(const TileArgs &g, bool aligned, int mi, unsigned grid, hipStream_t st)
{
#define FEW(MI, AL) hipLaunchKernelGGL((linear_few_kernel<AF, BF, MI, AL>), dim3(grid), dim3(64 * kFewWaves), 0, st, g)
    if (aligned) {
        if (mi == 1) FEW(1, true);
        else if (mi == 2) FEW(2, true);
        else FEW(4, true);
    } else {
        if (mi == 1) FEW(1, false);
        else if (mi == 2) FEW(2, false);
        else FEW(4, false);
    }
#undef FEW
}

// Workspace of the backward pass (floats, 64-float aligned parts): dz where an
// activation makes it, then the larger of the input gradient's and the weight
// gradient's partial products, then the partial bias gradient.
struct BwdLayout {
    Plan px, pw;
    long long o_part = 0, o_sum = 0, total = 0;
};
long long up64(long long n) { return (n + 63) & ~63LL; }

bool pieces_ok(long long a, long long b) { return a % 8 == 0 && b % 8 == 0; }

BwdLayout bwd_layout(long long M, int K, int N, const srnl_linear_params *p, bool dx, bool dw)
{
    BwdLayout l;
    const bool zf = p->act != SRNL_ACT_NONE || p->out_dtype == SRNL_F32;     // dz is fp32
    const bool al = pieces_ok(K, N);
    l.px = plan_tile(GRAD_X, M, K, N, zf, p->w_dtype == SRNL_F32, al);
    l.pw = plan_tile(GRAD_W, N, K, M, zf, p->x_dtype == SRNL_F32, al);
    l.o_part = p->act != SRNL_ACT_NONE ? up64(M * N) : 0;
    long long part = dx && l.px.splits > 1 ? l.px.splits * M * K : 0;
    const long long pw = dw && l.pw.splits > 1 ? static_cast<long long>(l.pw.splits) * N * K : 0;
    part = part > pw ? part : pw;
    l.o_sum = l.o_part + up64(part);
    l.total = l.o_sum + (dw && l.pw.splits > 1 ? up64(static_cast<long long>(l.pw.splits) * N) : 0);
    return l;
}

srnl_status check_linear(long long M, int K, int N, const srnl_linear_params *p)
{
    if (!p)
        return fail(SRNL_ERR_PTR, "params is NULL");
    if (M < 0)
        return fail(SRNL_ERR_ARG, "M must be >= 0");
    if (K < 1 || N < 1)
        return fail(SRNL_ERR_ARG, "K and N must be >= 1");
    if (p->act != SRNL_ACT_NONE && p->act != SRNL_ACT_GELU && p->act != SRNL_ACT_SILU)
        return fail(SRNL_ERR_ARG, "unknown activation");
    const long long wide = K > N ? K : N;
    if (static_cast<__int128>(M) * wide >= (static_cast<__int128>(1) << 58) ||
        cdiv(M, 16) * cdiv(wide, 16) > 0x7FFFFFFF || cdiv(K, 16) * cdiv(N, 16) > 0xFFFFFF)
        return fail(SRNL_ERR_ARG, "sizes too large");
    if (!valid_dtype(p->x_dtype) || !valid_dtype(p->w_dtype) || !valid_dtype(p->out_dtype) ||
        (p->residual && !valid_dtype(p->residual_dtype)))
        return fail(SRNL_ERR_DTYPE, "dtype must be SRNL_F32 or SRNL_BF16");
    return SRNL_OK;
}

}  // namespace

extern "C" {

srnl_status srnl_linear_fwd(const void *x, long long M, int K, int N, const srnl_linear_params *p,
                            void *out, float *pre)
{
    srnl_set_error(SRNL_OK, "");
    srnl_status s = check_linear(M, K, N, p);
    if (s != SRNL_OK)
        return s;
    if (M == 0)
        return SRNL_OK;
    const PtrArg ptrs[] = {{x, "x", false},          {p->w, "w", false},
                           {out, "out", false},      {p->bias, "bias", true},
                           {p->residual, "residual", true}, {pre, "pre", true}};
    s = check_ptrs(ptrs, 6);
    if (s != SRNL_OK)
        return s;
    hipStream_t st = static_cast<hipStream_t>(p->stream);
    TileArgs g = {};
    g.a = {x, K, M};
    g.b = {p->w, K, N};
    g.R = K;
    g.e = {out, p->out_dtype == SRNL_BF16, p->bias, p->act, p->residual,
           p->residual_dtype == SRNL_BF16, pre};
    const bool af = p->x_dtype == SRNL_F32, bf = p->w_dtype == SRNL_F32;
    const bool al = pieces_ok(K, N);
    // few rows, or fewer 64 x 64 tiles than half the CUs
    if (M <= 64 || cdiv(M, 64) * cdiv(N, 64) < 128) {
        g.tj = static_cast<int>(cdiv(N, 16));
        const int mi = M <= 16 || cdiv(M, 16) * g.tj <= 512 ? 1 : cdiv(M, 32) * g.tj <= 512 ? 2 : 4;
        const unsigned grid = static_cast<unsigned>(cdiv(M, 16 * mi) * g.tj);
        if (af && bf) launch_few<true, true>(g, al, mi, grid, st);
        else if (af) launch_few<true, false>(g, al, mi, grid, st);
        else if (bf) launch_few<false, true>(g, al, mi, grid, st);
        else launch_few<false, false>(g, al, mi, grid, st);
        return launched("linear_few_kernel");
    }
    return run_tile<FORWARD>(g, plan_tile(FORWARD, M, N, K, af, bf, al), af, bf, st);
}

size_t srnl_linear_bwd_workspace_bytes(long long M, int K, int N, const srnl_linear_params *p)
{
    if (check_linear(M, K, N, p) != SRNL_OK || M == 0)
        return 0;
    return static_cast<size_t>(bwd_layout(M, K, N, p, true, true).total) * sizeof(float);
}

srnl_status srnl_linear_bwd(const void *dout, const void *x, long long M, int K, int N,
                            const srnl_linear_params *p, const float *pre, const void *dx_add,
                            void *dx, float *dw, float *db, void *workspace, size_t workspace_bytes)
{
    srnl_set_error(SRNL_OK, "");
    srnl_status s = check_linear(M, K, N, p);
    if (s != SRNL_OK)
        return s;
    hipStream_t st = static_cast<hipStream_t>(p->stream);
    if (M == 0) {                         // the sums over no rows
        const PtrArg ptrs[] = {{dw, "dw", true}, {db, "db", true}};
        s = check_ptrs(ptrs, 2);
        if (s == SRNL_OK)
            s = zero_fill(dw, static_cast<long long>(N) * K, st);
        return s == SRNL_OK ? zero_fill(db, N, st) : s;
    }
    if (!dx && !dw && !db)
        return SRNL_OK;
    if (db && !dw)
        return fail(SRNL_ERR_PTR, "db without dw: the bias gradient is formed with the weight gradient");
    const size_t need = srnl_linear_bwd_workspace_bytes(M, K, N, p);
    if (need && (!workspace || workspace_bytes < need))
        return fail(SRNL_ERR_WORKSPACE, "workspace smaller than srnl_linear_bwd_workspace_bytes");
    const bool act = p->act != SRNL_ACT_NONE;
    const PtrArg ptrs[] = {{dout, "dout", false}, {x, "x", !dw},  {p->w, "w", !dx},
                           {pre, "pre", !act},    {dx, "dx", true}, {dx_add, "dx_add", true},
                           {dw, "dw", true},      {db, "db", true}, {need ? workspace : nullptr, "workspace", true}};
    s = check_ptrs(ptrs, 9);
    if (s != SRNL_OK)
        return s;
    const BwdLayout l = bwd_layout(M, K, N, p, true, true);
    float *const ws = static_cast<float *>(workspace);
    const void *dz = dout;
    bool zf = p->out_dtype == SRNL_F32;
    if (act) {
        const long long n = M * N, blocks = cdiv(n, 2048);
        hipLaunchKernelGGL(act_slope_kernel, dim3(static_cast<unsigned>(blocks < 16384 ? blocks : 16384)),
                           dim3(256), 0, st, dout, p->out_dtype == SRNL_BF16, pre, p->act, n, ws);
        s = launched("act_slope_kernel");
        if (s != SRNL_OK)
            return s;
        dz = ws;
        zf = true;
    }
    float *const part = ws + l.o_part;
    if (dx) {
        TileArgs g = {};
        g.a = {dz, N, M};
        g.b = {p->w, K, K};
        g.R = N;
        g.e.out = dx;
        g.e.obf = p->x_dtype == SRNL_BF16;
        g.e.add = dx_add;
        g.e.abf = g.e.obf;
        g.part = l.px.splits > 1 ? part : nullptr;
        s = run_tile<GRAD_X>(g, l.px, zf, p->w_dtype == SRNL_F32, st);
        if (s != SRNL_OK)
            return s;
        if (g.part) {
            const long long n = M * K, blocks = cdiv(n, 2048);
            hipLaunchKernelGGL(join_kernel, dim3(static_cast<unsigned>(blocks < 16384 ? blocks : 16384)),
                               dim3(256), 0, st, part, l.px.splits, n, g.e);
            s = launched("join_kernel");
            if (s != SRNL_OK)
                return s;
        }
    }
    if (dw) {
        TileArgs g = {};
        g.a = {dz, N, N};
        g.b = {x, K, K};
        g.R = M;
        g.e.out = dw;
        const bool split = l.pw.splits > 1;
        g.part = split ? part : nullptr;
        g.rowsum = db ? (split ? ws + l.o_sum : db) : nullptr;
        s = run_tile<GRAD_W>(g, l.pw, zf, p->x_dtype == SRNL_F32, st);
        if (s != SRNL_OK || !split)
            return s;
        const long long n = static_cast<long long>(N) * K;
        if (l.pw.splits >= 16) {
            s = sum_rows(part, l.pw.splits, n, n, n, dw, nullptr, st);
        } else {
            const long long blocks = cdiv(n, 2048);
            hipLaunchKernelGGL(join_kernel, dim3(static_cast<unsigned>(blocks < 16384 ? blocks : 16384)),
                               dim3(256), 0, st, part, l.pw.splits, n, g.e);
            s = launched("join_kernel");
        }
        if (s == SRNL_OK && db)
            s = sum_rows(g.rowsum, l.pw.splits, N, N, N, db, nullptr, st);
        return s;
    }
    return SRNL_OK;
}

}  // extern "C"
