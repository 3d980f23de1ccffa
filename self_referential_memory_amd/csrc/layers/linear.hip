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
// 2^-26 |x w|, a quarter of an fp32 rounding. Below 2^-108 the parts reach
// bf16's smallest numbers and x is held to 2^-134. Six bf16 MFMAs are 2.7 times
// faster than one fp32 MFMA of the same shape.
//
// A few rows (or few output tiles) go to linear_few_kernel, which splits the
// reduction over the waves of a block and joins them in LDS. Which kernel takes
// which sizes and types is in plan.h.
#include "narrow.h"

namespace {

using namespace srnl_i;

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

// What lanes read in place of pieces outside an operand: 16 bytes in the tiled
// kernels, the 32 of eight fp32 values in the few-rows kernel.
__device__ __align__(16) const uint32_t zero_piece[8] = {0, 0, 0, 0, 0, 0, 0, 0};

// A tile of ROWS x BK of an operand, staged in LDS as PARTS planes of bf16.
// RC: plane[row][BK], 16-byte pieces of a row permuted so that 16 consecutive
// rows' reads of one piece fall on all 64 banks. Not RC: plane[r][ROWS] as
// in memory, the 64-byte blocks of a row permuted by r, read through the
// transposing LDS read (ds_read_b64_tr_b16: of the 4 x 16 block that 16
// lanes address, each lane gets a column).
template <Source SRC, bool RC, int ROWS, int BK, int NT = 256> struct Tile {
    static constexpr bool F32 = !is_bf16(SRC), SLOPE = SRC == SLOPE_BF16 || SRC == SLOPE_FP32;
    static constexpr bool VALUES = SRC == FP32 || SRC == SLOPE_FP32;
    static constexpr int PARTS = F32 ? 3 : 1;
    static constexpr bool ASYNC = SRC == BF16;            // straight from memory into LDS
    static constexpr int PLANE = ROWS * BK;               // words
    static constexpr int PIECES = PLANE / 8 / NT;         // 8-element pieces per thread
    static_assert(PIECES >= 1 && PIECES * NT * 8 == PLANE, "pieces divide evenly");
    static constexpr int PER = RC ? BK / 8 : ROWS / 8;    // pieces per stored row

    float v[VALUES ? PIECES : 1][8];
    u32x4 raw[VALUES ? 1 : PIECES];
    float z[SLOPE ? PIECES : 1][8];
    const uint16_t *next[ASYNC ? PIECES : 1];             // ASYNC: where the next step's pieces are
    long long off;                                        // otherwise: the first one's offset
    long long total;                                      // elements of the operand

    static __device__ __forceinline__ int place(int major, int c)
    {
        if (RC) {
            constexpr int RP = 16 / PER;                  // rows per 256 bytes
            return c ^ ((major / RP) & (PER - 1));
        }
        constexpr int NB = ROWS < 128 ? ROWS / 32 : 4, RPB = 4 / NB;    // 64-byte blocks of 256 bytes, rows in them
        return c ^ (4 * ((major / RPB) & (NB - 1)));
    }

    // before the first fetch, at (row0, r0) of an operand with R reduction
    // indices. ASYNC: pieces of rows outside the operand take the last row's (or
    // first columns'), whose products are not stored.
    __device__ __forceinline__ void start(const Operand &o, long long row0, long long r0, long long R)
    {
        if constexpr (ASYNC) {
#pragma unroll
            for (int q = 0; q < PIECES; ++q) {
                const int s = threadIdx.x + NT * q, major = s / PER, c = place(major, s % PER);
                const long long row = row0 + (RC ? major : 8 * c), r = r0 + (RC ? 8 * c : major);
                const long long in = row < o.rows ? row : RC ? o.rows - 1 : 0;
                next[q] = static_cast<const uint16_t *>(o.p) + (RC ? in * o.ld + r : r * o.ld + in);
            }
        } else {
            total = RC ? o.rows * o.ld : R * o.ld;
            off = offset(o, row0, r0, 0);
        }
    }
    static __device__ __forceinline__ long long offset(const Operand &o, long long row0, long long r0, int q)
    {
        const int s = threadIdx.x + NT * q, major = s / PER, c = s % PER;
        return RC ? (row0 + major) * o.ld + r0 + 8 * c : (r0 + major) * o.ld + row0 + 8 * c;
    }
    // start fetching the tile at r0, step by step from where start() was; ASYNC:
    // into buf
    __device__ __forceinline__ void fetch(const Operand &o, long long r0, long long rend, uint16_t *buf)
    {
        const int tid = threadIdx.x;
        if constexpr (ASYNC) {
            const bool tail = r0 + BK > rend;
            const long long stride = RC ? BK : BK * o.ld;
#pragma unroll
            for (int q = 0; q < PIECES; ++q) {
                const uint16_t *src = next[q];
                if (tail) {
                    const int s = tid + NT * q, major = s / PER;
                    if (r0 + (RC ? 8 * place(major, s % PER) : major) >= rend)
                        src = reinterpret_cast<const uint16_t *>(zero_piece);
                }
                next[q] += stride;
                // lane l of the wave writes base + 16 l
                uint16_t *dst = buf + 8 * (NT * q + (tid & ~63));
                __builtin_amdgcn_global_load_lds(
                    reinterpret_cast<const __attribute__((address_space(1))) void *>(
                        reinterpret_cast<uintptr_t>(src)),
                    (__attribute__((address_space(3))) void *)dst, 16, 0, 0);
            }
            return;
        }
        // Every piece is one wide load without a condition, so that nothing waits
        // for it here: what lies past the reduction, or past the operand's last
        // eight elements, is put right by commit(). Rows (columns) past the last
        // hold whatever is there; their products are not stored.
        const long long last = total - 8;
        if (last >= 0) {
#pragma unroll
            for (int q = 0; q < PIECES; ++q) {
                static_assert(NT % PER == 0, "a thread's pieces are alike but for their row");
                const long long my = off + q * (NT / PER) * o.ld, at = my < last ? my : last;
                if constexpr (SLOPE)
                    load_f32<8, false>(o.z + at, z[q]);
                if constexpr (VALUES)
                    load_f32<8, false>(static_cast<const float *>(o.p) + at, v[q]);
                else
                    __builtin_memcpy(&raw[q], static_cast<const uint16_t *>(o.p) + at, 16);
            }
            off += RC ? BK : BK * o.ld;
        }
    }
    // the tile at (row0, r0) as fetched, where it reaches the operand's end:
    // zeros past the reduction, and the last elements one by one
    __device__ __forceinline__ void mend(const Operand &o, long long row0, long long r0, long long rend)
    {
        const long long wide = row0 + ROWS < o.rows ? row0 + ROWS : (o.rows + 7) & ~7LL;
        if (r0 + BK <= rend && (RC || (r0 + BK - 1) * o.ld + wide <= total))
            return;
#pragma unroll
        for (int q = 0; q < PIECES; ++q) {
            const int s = threadIdx.x + NT * q, major = s / PER, c = s % PER;
            const long long left = RC ? rend - r0 - 8 * c : r0 + major < rend ? 8 : 0;
            const int n = left < 0 ? 0 : left < 8 ? static_cast<int>(left) : 8;
            const long long at = offset(o, row0, r0, q);
            const bool single = n > 0 && at > total - 8;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const bool in = e < n;
                if constexpr (SLOPE)
                    z[q][e] = in ? z[q][e] : 0.0f;
                if constexpr (VALUES)
                    v[q][e] = in ? v[q][e] : 0.0f;
                else
                    raw[q][e / 2] = in ? raw[q][e / 2] : raw[q][e / 2] & (e & 1 ? 0xFFFFu : 0xFFFF0000u);
            }
            if (single) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const bool in = e < n && at + e < total;
                    const long long x = in ? at + e : 0;
                    if constexpr (SLOPE)
                        z[q][e] = in ? o.z[x] : 0.0f;
                    if constexpr (VALUES) {
                        v[q][e] = in ? static_cast<const float *>(o.p)[x] : 0.0f;
                    } else {
                        const uint32_t w = in ? static_cast<const uint16_t *>(o.p)[x] : 0u;
                        raw[q][e / 2] = e & 1 ? raw[q][e / 2] | w << 16 : w;
                    }
                }
            }
        }
    }
    // write what fetch holds in registers to buf
    __device__ __forceinline__ void commit(const Operand &o, long long row0, long long r0, long long rend, uint16_t *buf)
    {
        if constexpr (!ASYNC) {
            mend(o, row0, r0, rend);
#pragma unroll
            for (int q = 0; q < PIECES; ++q) {
                const int s = threadIdx.x + NT * q;
                const int major = s / PER;
                uint16_t *dst = buf + 8 * (major * PER + place(major, s % PER));
                if constexpr (F32) {
                    u32x4 w[3];
                    float d[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        d[e] = VALUES ? v[VALUES ? q : 0][e]
                                      : e & 1 ? bf16_hi(raw[VALUES ? 0 : q][e / 2]) : bf16_lo(raw[VALUES ? 0 : q][e / 2]);
                    if constexpr (SLOPE)
                        act_slopes(z[q], o.act, d);
                    split_parts(d, w);
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

// ------------------------------------------------------------ tiled product

struct TileArgs {
    Operand a, b;          // out[i][j] = sum over r of a(i, r) b(j, r)
    long long R;           // reduction length
    long long slice;       // reduction length per split, a multiple of a step's
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
// Tiles of 64 are for small products, where a step is mostly the wait for its
// loads: they take twice the reduction a step.
constexpr int tile_waves(int bi) { return bi == 256 ? 8 : 4; }

template <Source SA, Source SB, bool RCA, bool RCB, int BI, int BJ> struct TileCfg {
    static constexpr int BK = (is_bf16(SA) && is_bf16(SB) ? 64 : 32) * (BI == 64 ? 2 : 1);
    static constexpr int NW = tile_waves(BI), WI = 2, WJ = NW / WI;      // waves, down and across
    using TA = Tile<SA, RCA, BI, BK, 64 * NW>;
    using TB = Tile<SB, RCB, BJ, BK, 64 * NW>;
    static constexpr int NA = TA::ASYNC ? 2 : 1, NB = TB::ASYNC ? 2 : 1;    // buffers
    static constexpr int PA = TA::PARTS, PB = TB::PARTS;
    static constexpr int FI = BI / 32 / WI, FJ = BJ / 32 / WJ;  // 32 x 32 tiles per wave
    static constexpr int OUTP = 32 * FJ + 4;                    // floats per staged output row
    static constexpr int WORDS = NA * PA * TA::PLANE + NB * PB * TB::PLANE;
    static constexpr int OUT_WORDS = NW * 32 * OUTP * 2;
    static constexpr int LDS = WORDS > OUT_WORDS ? WORDS : OUT_WORDS;
    // Blocks a CU that the registers are held to: as many as fit in LDS where
    // that costs no spill (132 registers become 128, three blocks four:
    // 200704 x 64 -> 256 fp32 with bf16 weights 78 -> 73 us).
    static constexpr int BLOCKS = RCA && RCB && BI == 128 && SA == FP32 && SB != BF16_ANY ? 160 * 1024 / (2 * LDS) : 1;
};

// tile t of g, in lds of TileCfg::LDS words. Long reductions are bound by the
// LDS reads behind the MFMAs (16384 x 2048 -> 2048 bf16: 147 us, 0.94 PFLOP/s),
// short ones by memory and the epilogue's arithmetic (200704 x 64 -> 256 fp32,
// gelu: 73 us, 3.5 TB/s; 24 of a value's 39 vector issue slots are gelu's),
// small ones by the latency of their steps (1003 x 333 -> 777 fp32: 17 us for
// six steps).
template <Source SA, Source SB, bool RCA, bool RCB, int BI, int BJ, bool SUMS>
__device__ __forceinline__ void tile_product(const TileArgs &g, unsigned t, uint16_t *lds)
{
    using Cfg = TileCfg<SA, SB, RCA, RCB, BI, BJ>;
    using TA = typename Cfg::TA;
    using TB = typename Cfg::TB;
    constexpr int BK = Cfg::BK, NA = Cfg::NA, NB = Cfg::NB, PA = Cfg::PA, PB = Cfg::PB, OUTP = Cfg::OUTP;
    constexpr int FI = Cfg::FI, FJ = Cfg::FJ;
    uint16_t *const la = lds, *const lb = lds + NA * PA * TA::PLANE;

    const int tj = t % g.tj, ti = (t / g.tj) % g.ti, sp = t / (g.tj * g.ti);
    const long long i0 = static_cast<long long>(ti) * BI, j0 = static_cast<long long>(tj) * BJ;
    const long long rb = sp * g.slice, re = rb + g.slice < g.R ? rb + g.slice : g.R;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int wi = (wave / Cfg::WJ) * 32 * FI, wj = (wave % Cfg::WJ) * 32 * FJ;
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

    ta.start(g.a, i0, rb, g.R);
    tb.start(g.b, j0, rb, g.R);
    ta.fetch(g.a, rb, re, la);
    tb.fetch(g.b, rb, re, lb);
    ta.commit(g.a, i0, rb, re, la);
    tb.commit(g.b, j0, rb, re, lb);
    int cur = 0;
    tile_barrier<NA == 2 || NB == 2>();
    for (long long r = rb; r < re; r += BK) {
        const int nxt = cur ^ 1;
        uint16_t *const ca = la + (NA == 2 ? cur : 0) * PA * TA::PLANE, *const na = la + (NA == 2 ? nxt : 0) * PA * TA::PLANE;
        uint16_t *const cb = lb + (NB == 2 ? cur : 0) * PB * TB::PLANE, *const nb = lb + (NB == 2 ? nxt : 0) * PB * TB::PLANE;
        const bool more = r + BK < re;
        if (more) {
            ta.fetch(g.a, r + BK, re, na);
            tb.fetch(g.b, r + BK, re, nb);
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
        if (NA == 1 || NB == 1)
            __syncthreads();                 // everyone has read the only buffer
        if (more) {
            ta.commit(g.a, i0, r + BK, re, na);
            tb.commit(g.b, j0, r + BK, re, nb);
        }
        cur = nxt;
        tile_barrier<NA == 2 || NB == 2>();
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
    constexpr int LPR = 4 * FJ, RPQ = 64 / LPR, NQ = 32 / RPQ;  // lanes per row; rows a pass, passes
    const long long oj = j0 + wj + 8 * (lane % LPR), left = g.b.rows - oj;
    const int cols = left < 0 ? 0 : left < 8 ? static_cast<int>(left) : 8;
    const bool whole = g.b.rows % 8 == 0;
    float bias[8];
    if (whole)
        load_bias<true>(e, static_cast<int>(oj), cols, bias);
    else
        load_bias<false>(e, static_cast<int>(oj), cols, bias);
    const long long oi0 = i0 + wi + lane / LPR;
#pragma unroll
    for (int i = 0; i < FI; ++i) {
#pragma unroll
        for (int j = 0; j < FJ; ++j)
#pragma unroll
            for (int k = 0; k < 16; ++k)
                st[(8 * (k / 4) + 4 * (lane >> 5) + k % 4) * OUTP + 32 * j + (lane & 31)] = acc[i][j][k];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
#pragma unroll 2
        for (int q = 0; q < NQ; ++q) {
            float v[8];
            load_f32<8, true>(st + (RPQ * q + lane / LPR) * OUTP + 8 * (lane % LPR), v);
            const long long oi = oi0 + 32 * i + RPQ * q, o = oi * g.b.rows + oj;
            const int n = oi < g.a.rows ? cols : 0;
            if (whole) {
                finish_piece<true>(e, o, n, v, bias);
            } else {
                finish_piece<false>(e, o, n, v, bias);
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
}

template <Source SA, Source SB, bool RCA, bool RCB, int BI, int BJ, bool SUMS>
__global__ __launch_bounds__(64 * tile_waves(BI), (TileCfg<SA, SB, RCA, RCB, BI, BJ>::BLOCKS))
void linear_tile_kernel(TileArgs g)
{
    __shared__ __align__(16) uint16_t lds[TileCfg<SA, SB, RCA, RCB, BI, BJ>::LDS];
    tile_product<SA, SB, RCA, RCB, BI, BJ, SUMS>(g, die_order(blockIdx.x, gridDim.x), lds);
}

// Both gradients of a small layer in one launch: the first nx blocks take the
// input gradient's tiles, the others the weight gradient's, so that neither
// waits for the other's last tiles. SZ, SW, SX: what dz, w and x are.
template <Source SZ, Source SW, Source SX>
__global__ __launch_bounds__(256) void linear_grads_kernel(TileArgs gx, TileArgs gw, unsigned nx)
{
    constexpr int LX = TileCfg<SZ, SW, true, false, 64, 64>::LDS;
    constexpr int LW = TileCfg<SZ, SX, false, false, 64, 64>::LDS;
    __shared__ __align__(16) uint16_t lds[LX > LW ? LX : LW];
    if (blockIdx.x < nx)
        tile_product<SZ, SW, true, false, 64, 64, false>(gx, die_order(blockIdx.x, nx), lds);
    else
        tile_product<SZ, SX, false, false, 64, 64, true>(
            gw, die_order(blockIdx.x - nx, gridDim.x - nx), lds);
}

// out = sum of the splits' partial products through the epilogue, in a fixed
// order: `group` threads a piece of eight outputs, each with every group-th
// split, joined through LDS. Bound by the latency of its loads, so many splits
// take many threads: the 256 parts of 256 x 64 sums (16.8 MB) take
// 7.8 us (11.9 with eight threads a piece).
struct Join {
    const float *part;
    int splits, group;      // group: 1, 8 or 32
    long long n;            // outputs; 0: nothing to join
    long long blocks;
    Epilogue e;
};

__device__ __forceinline__ void join_block(const Join &j, long long block)
{
    __shared__ __align__(16) float red[2048], top[256];
    const int tid = threadIdx.x, pieces = 256 / j.group, outs = 8 * pieces;
    const int piece = tid & (pieces - 1), sub = tid / pieces;
    const long long o = block * outs + 8 * piece;
    const int m = o >= j.n ? 0 : j.n - o < 8 ? static_cast<int>(j.n - o) : 8;
    const float *p = j.part + o;
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
        v[k] = 0.0f;
    if (m == 8) {
#pragma unroll 8
        for (int s = sub; s < j.splits; s += j.group) {
            float w[8];
            load_f32<8, false>(p + s * j.n, w);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                v[k] += w[k];
        }
    } else if (m) {
        for (int s = sub; s < j.splits; s += j.group) {
            float w[8];
            load_row<8, false>(p, false, s * j.n, m, w);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                v[k] += w[k];
        }
    }
    if (j.group > 1) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            red[tid * 8 + k] = v[k];             // [sub][output]
        __syncthreads();
        // a thread adds eight subs of an output, the piece's first the eights
        const int out = tid & (outs - 1), eight = tid / outs;
        float t = 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k)
            t += red[(8 * eight + k) * outs + out];
        top[tid] = t;
        __syncthreads();
        if (sub)
            return;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            v[k] = top[8 * piece + k];
            for (int e = 1; e < j.group / 8; ++e)
                v[k] += top[e * outs + 8 * piece + k];
        }
    }
    finish8(j.e, o, 0, m, v);
}

// the input gradient's, the weight gradient's and the bias gradient's partial
// sums in one launch
__global__ __launch_bounds__(256) void join_kernel(Join a, Join b, Join c)
{
    long long k = blockIdx.x;
    if (k < a.blocks)
        return join_block(a, k);
    k -= a.blocks;
    if (k < b.blocks)
        return join_block(b, k);
    join_block(c, k - b.blocks);
}

Join make_join(const float *part, int splits, long long n, const Epilogue &e)
{
    Join j = {};
    if (splits > 1 && n > 0) {
        j.group = splits >= 64 ? 32 : splits >= 16 ? 8 : 1;
        const long long per = 2048 / j.group;
        j.part = part;
        j.splits = splits;
        j.n = n;
        j.blocks = (n + per - 1) / per;
        j.e = e;
    }
    return j;
}

srnl_status join(const Join &a, const Join &b, const Join &c, hipStream_t st)
{
    const long long blocks = a.blocks + b.blocks + c.blocks;
    if (blocks == 0)
        return SRNL_OK;
    hipLaunchKernelGGL(join_kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, st, a, b, c);
    return launched("join_kernel");
}

// ------------------------------------------------------------ few rows

// 16 MI x 16 MJ outputs per block; its eight waves take the reduction 32 indices
// at a time in turn, straight from memory into MFMA operands
// (v_mfma_f32_16x16x32_bf16), and join through LDS in wave order. Bound by the
// latency of its rounds of loads, 512 indices each, one after the other (1 x 512
// -> 2048 bf16 gelu, one round, 4.0 us; 49 x 2048 -> 512, four rounds on 128 CUs,
// 6.7 us; an empty launch takes 3), for wide weights by memory (1 x 4096 -> 16384
// bf16 24 us, 5.6 TB/s).
constexpr int kFewWaves = 8;

// Eight reduction indices from k on of an operand's row, as they lie in memory.
template <bool F32> struct FewPiece {
    u32x4 w[F32 ? 2 : 1];
    // Without a condition, so that a round's loads leave together: rows past the
    // last take the last (their outputs are not stored), and what lies past the
    // operand's last eight elements is loaded by mend().
    __device__ __forceinline__ void load(const Operand &o, long long row, long long k, long long total)
    {
        static_assert(sizeof w <= sizeof zero_piece, "a whole piece is read in place of a short operand");
        row = row < o.rows ? row : o.rows - 1;
        const long long at = row * o.ld + k, last = total < 8 ? 0 : total - 8;
        const uintptr_t p = total < 8 ? reinterpret_cast<uintptr_t>(zero_piece) : reinterpret_cast<uintptr_t>(o.p);
        const __attribute__((address_space(1))) char *src = reinterpret_cast<const __attribute__((address_space(1))) char *>(p);
        __builtin_memcpy(w, src + (at < last ? at : last) * (F32 ? 4 : 2), sizeof w);
    }
    // where the piece may reach past the reduction's end R
    __device__ __forceinline__ void mend(const Operand &o, long long row, long long k, long long R, long long total)
    {
        row = row < o.rows ? row : o.rows - 1;
        const int n = R - k < 8 ? static_cast<int>(R - k < 0 ? 0 : R - k) : 8;
        const long long at = row * o.ld + k;
        uint32_t e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            e[i] = F32 ? w[F32 ? i / 4 : 0][i % 4] : w[0][i / 2] >> (16 * (i & 1)) & 0xFFFFu;
        if (n > 0 && at > total - 8) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const long long x = i < n ? at + i : at;
                e[i] = F32 ? static_cast<const uint32_t *>(o.p)[x] : static_cast<const uint16_t *>(o.p)[x];
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            e[i] = i < n ? e[i] : 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (F32) {
                w[0][i] = e[i];
                w[1][i] = e[4 + i];
            } else {
                w[0][i] = e[2 * i] | e[2 * i + 1] << 16;
            }
        }
    }
    __device__ __forceinline__ void parts(u32x4 (&p)[3]) const
    {
        if constexpr (F32) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = __uint_as_float(w[i / 4][i % 4]);
            split_parts(v, p);
        } else {
            p[0] = w[0];
        }
    }
};

template <bool AF, bool BF, int MI, int MJ>
__global__ __launch_bounds__(64 * kFewWaves) void linear_few_kernel(TileArgs g)
{
    constexpr int PA = AF ? 3 : 1, PB = BF ? 3 : 1;
    constexpr int P = 16 * MJ + 4;                              // floats per staged row
    __shared__ __align__(16) float red[kFewWaves][16 * MI * P];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63, rl = lane & 15, g8 = 8 * (lane >> 4);
    const int tj = blockIdx.x % g.tj;
    const long long i0 = static_cast<long long>(blockIdx.x / g.tj) * 16 * MI, j0 = 16LL * MJ * tj;
    const long long na = g.a.rows * g.R, nb = g.b.rows * g.R;
    v4f acc[MI][MJ];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < MJ; ++j)
            acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
    constexpr int U = 2;                                        // pieces in flight
    constexpr long long ROUND = 32LL * U * kFewWaves;
    for (long long r = 32LL * wave; r < g.R; r += ROUND) {
        FewPiece<BF> wb[U][MJ];
        FewPiece<AF> wa[U][MI];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const long long k = r + 32LL * kFewWaves * u + g8;
#pragma unroll
            for (int j = 0; j < MJ; ++j)
                wb[u][j].load(g.b, j0 + 16 * j + rl, k, nb);
#pragma unroll
            for (int i = 0; i < MI; ++i)
                wa[u][i].load(g.a, i0 + 16 * i + rl, k, na);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const long long k0 = r + 32LL * kFewWaves * u, k = k0 + g8;
            if (k0 >= g.R)
                break;
            if (k0 + 32 > g.R) {
#pragma unroll
                for (int j = 0; j < MJ; ++j)
                    wb[u][j].mend(g.b, j0 + 16 * j + rl, k, g.R, nb);
#pragma unroll
                for (int i = 0; i < MI; ++i)
                    wa[u][i].mend(g.a, i0 + 16 * i + rl, k, g.R, na);
            }
            u32x4 pb[MJ][3];
#pragma unroll
            for (int j = 0; j < MJ; ++j)
                wb[u][j].parts(pb[j]);
#pragma unroll
            for (int i = 0; i < MI; ++i) {
                u32x4 pa[3];
                wa[u][i].parts(pa);
#pragma unroll
                for (int s = 2; s >= 0; --s)
#pragma unroll
                    for (int p = 0; p < PA; ++p) {
                        const int q = s - p;
                        if (q < 0 || q >= PB)
                            continue;
#pragma unroll
                        for (int j = 0; j < MJ; ++j)
                            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                __builtin_bit_cast(bf16x8, pa[p]), __builtin_bit_cast(bf16x8, pb[j][q]),
                                acc[i][j], 0, 0, 0);
                    }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < MJ; ++j)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                red[wave][(16 * i + 4 * (lane >> 4) + k) * P + 16 * j + rl] = acc[i][j][k];
    __syncthreads();
    const int row = threadIdx.x / (2 * MJ), c = 8 * (threadIdx.x % (2 * MJ));
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
    finish8(g.e, (i0 + row) * g.b.rows + j0 + c, static_cast<int>(j0 + c),
            left < 8 ? static_cast<int>(left) : 8, v);
}

// ------------------------------------------------------------ host

unsigned blocks_of(const Plan &p) { return static_cast<unsigned>(p.ti * p.tj * p.splits); }

void take_plan(TileArgs &g, const Plan &p)
{
    g.slice = p.slice;
    g.splits = p.splits;
    g.ti = static_cast<int>(p.ti);
    g.tj = static_cast<int>(p.tj);
}

// the forward pass, and the gradients' products of 128 x 128 tiles
template <Source SA, Source SB, Form F>
void launch_tile(const TileArgs &g, const Plan &p, hipStream_t st)
{
    constexpr bool RCA = F != GRAD_W, RCB = F == FORWARD, SUMS = F == GRAD_W;
    const dim3 grid(blocks_of(p)), block(256);
    if (p.bi == 256) {
        if constexpr (SA == BF16 && SB == BF16 && F != GRAD_W)
            hipLaunchKernelGGL((linear_tile_kernel<SA, SB, RCA, RCB, 256, 256, SUMS>), grid, dim3(512), 0, st, g);
    } else if (p.bi == 128) {
        hipLaunchKernelGGL((linear_tile_kernel<SA, SB, RCA, RCB, 128, 128, SUMS>), grid, block, 0, st, g);
    } else if constexpr (F == FORWARD) {
        hipLaunchKernelGGL((linear_tile_kernel<SA, SB, RCA, RCB, 64, 64, SUMS>), grid, block, 0, st, g);
    }
}

template <Source SA, Form F> void launch_tile_of(const TileArgs &g, const Plan &p, Source sb, hipStream_t st)
{
    // forward: both operands' rows are K long, so of one kind
    if (sb == FP32) {
        launch_tile<SA, FP32, F>(g, p, st);
    } else if (sb == BF16) {
        if constexpr (F != FORWARD || SA != BF16_ANY)
            launch_tile<SA, BF16, F>(g, p, st);
    } else {
        if constexpr (F != FORWARD || SA != BF16)
            launch_tile<SA, BF16_ANY, F>(g, p, st);
    }
}

template <Form F> srnl_status run_tile(const TileArgs &g, const Plan &p, Source sa, Source sb, hipStream_t st)
{
    if (sa == FP32) launch_tile_of<FP32, F>(g, p, sb, st);
    else if (sa == BF16) launch_tile_of<BF16, F>(g, p, sb, st);
    else launch_tile_of<BF16_ANY, F>(g, p, sb, st);
    return launched("linear_tile_kernel");
}

struct GradsLaunch {
    TileArgs gx, gw;
    unsigned nx, nw;
    Source sz, sw, sx;
};

template <Source SZ, Source SW, Source SX> void launch_grads(const GradsLaunch &l, hipStream_t st)
{
    hipLaunchKernelGGL((linear_grads_kernel<SZ, SW, SX>), dim3(l.nx + l.nw), dim3(256), 0, st, l.gx, l.gw, l.nx);
}

template <Source SZ> void launch_grads_of(const GradsLaunch &l, hipStream_t st)
{
    if (l.sw == FP32 && l.sx == FP32) launch_grads<SZ, FP32, FP32>(l, st);
    else if (l.sw == FP32 && l.sx == BF16) launch_grads<SZ, FP32, BF16>(l, st);
    else if (l.sw == FP32) launch_grads<SZ, FP32, BF16_ANY>(l, st);
    else if (l.sx == FP32 && l.sw == BF16) launch_grads<SZ, BF16, FP32>(l, st);
    else if (l.sx == FP32) launch_grads<SZ, BF16_ANY, FP32>(l, st);
    else if (l.sw == BF16) launch_grads<SZ, BF16, BF16>(l, st);     // both have rows of K
    else launch_grads<SZ, BF16_ANY, BF16_ANY>(l, st);
}

srnl_status run_grads(const GradsLaunch &l, hipStream_t st)
{
    switch (l.sz) {
    case BF16: launch_grads_of<BF16>(l, st); break;
    case BF16_ANY: launch_grads_of<BF16_ANY>(l, st); break;
    case FP32: launch_grads_of<FP32>(l, st); break;
    case SLOPE_BF16: launch_grads_of<SLOPE_BF16>(l, st); break;
    case SLOPE_FP32: launch_grads_of<SLOPE_FP32>(l, st); break;
    }
    return launched("linear_grads_kernel");
}

template <bool AF, bool BF> void launch_few(TileArgs g, FewShape f, hipStream_t st)
{
    g.tj = static_cast<int>(cdiv(g.b.rows, 16 * f.mj));
    const dim3 grid(static_cast<unsigned>(cdiv(g.a.rows, 16 * f.mi) * g.tj)), block(64 * kFewWaves);
#define FEW(MI, MJ) hipLaunchKernelGGL((linear_few_kernel<AF, BF, MI, MJ>), grid, block, 0, st, g)
    if (f.mi == 1 && f.mj == 1)
        FEW(1, 1);
    else if (f.mi == 1)
        FEW(1, 2);
    else if (f.mj == 1)
        FEW(2, 1);
    else if (f.mi == 2 && f.mj == 2)
        FEW(2, 2);
    else if constexpr (AF && !BF)
        FEW(2, 4);
    else if constexpr (BF)
        FEW(4, 2);
#undef FEW
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
        cdiv(M, 128) * cdiv(wide, 128) > 0xFFFFFF || cdiv(K, 16) * cdiv(N, 16) > 0xFFFFFF)    // launches of 2^32 threads
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
    g.a = {x, K, M, nullptr, 0};
    g.b = {p->w, K, N, nullptr, 0};
    g.R = K;
    g.e = {out, p->out_dtype == SRNL_BF16, p->bias, p->act, p->residual,
           p->residual_dtype == SRNL_BF16, pre};
    const Source sx = source_of(p->x_dtype, K), sw = source_of(p->w_dtype, K);
    if (const FewShape f = few_shape(M, N, K, sx == FP32, sw == FP32); f.mi) {
        if (sx == FP32 && sw == FP32) launch_few<true, true>(g, f, st);
        else if (sx == FP32) launch_few<true, false>(g, f, st);
        else if (sw == FP32) launch_few<false, true>(g, f, st);
        else launch_few<false, false>(g, f, st);
        return launched("linear_few_kernel");
    }
    const Plan plan = plan_tile(FORWARD, M, N, K, sx, sw);
    take_plan(g, plan);
    return run_tile<FORWARD>(g, plan, sx, sw, st);
}

size_t srnl_linear_bwd_workspace_bytes(long long M, int K, int N, const srnl_linear_params *p)
{
    if (check_linear(M, K, N, p) != SRNL_OK || M == 0)
        return 0;
    return static_cast<size_t>(bwd_layout(M, K, N, p).total) * sizeof(float);
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
    const BwdLayout l = bwd_layout(M, K, N, p);
    float *const ws = static_cast<float *>(workspace);
    Epilogue ew = {}, eb = {};
    ew.out = dw;
    eb.out = db;
    if (dx && dw && l.narrow) {
        const Operand oz = {dout, N, M, pre, p->act}, ow = {p->w, K, N, nullptr, 0}, ox = {x, K, M, nullptr, 0};
        const bool xb = p->x_dtype == SRNL_BF16;
        const Epilogue ex = {dx, xb, nullptr, SRNL_ACT_NONE, dx_add, xb, nullptr};
        float *const nb = db ? ws + l.o_nb : nullptr;
        const NarrowArgs g = {oz, ow, ox, M, K, N, ex, ws, nb};
        // rows of N in whole pieces, so dz is never BF16_ANY here
        if (l.narrow_z == FP32) s = narrow_launch<FP32>(g, l.narrow, l.sw, l.sx, st);
        else if (l.narrow_z == SLOPE_BF16) s = narrow_launch<SLOPE_BF16>(g, l.narrow, l.sw, l.sx, st);
        else if (l.narrow_z == SLOPE_FP32) s = narrow_launch<SLOPE_FP32>(g, l.narrow, l.sw, l.sx, st);
        else s = narrow_launch<BF16>(g, l.narrow, l.sw, l.sx, st);
        return s == SRNL_OK ? join({}, make_join(ws, l.narrow, static_cast<long long>(N) * K, ew),
                                   make_join(nb, db ? l.narrow : 1, N, eb), st) : s;
    }
    const void *dz = dout;
    if (act && !l.fused) {
        const long long n = M * N, blocks = cdiv(n, 2048);
        hipLaunchKernelGGL(act_slope_kernel, dim3(static_cast<unsigned>(blocks < 16384 ? blocks : 16384)),
                           dim3(256), 0, st, dout, p->out_dtype == SRNL_BF16, pre, p->act, n, ws);
        s = launched("act_slope_kernel");
        if (s != SRNL_OK)
            return s;
        dz = ws;
    }
    const bool xb = p->x_dtype == SRNL_BF16;
    TileArgs gx = {}, gw = {};
    gx.a = {dz, N, M, pre, p->act};
    gx.b = {p->w, K, K, nullptr, 0};
    gx.R = N;
    gx.e.out = dx;
    gx.e.obf = xb;
    gx.e.add = dx_add;
    gx.e.abf = xb;
    gx.part = l.px.splits > 1 ? ws + l.o_x : nullptr;
    take_plan(gx, l.px);
    gw.a = {dz, N, N, pre, p->act};
    gw.b = {x, K, K, nullptr, 0};
    gw.R = M;
    gw.e = ew;
    const bool split = l.pw.splits > 1;
    gw.part = split ? ws + l.o_w : nullptr;
    gw.rowsum = db ? (split ? ws + l.o_b : db) : nullptr;
    take_plan(gw, l.pw);
    const bool bigx = dx && l.px.bi >= 128, bigw = dw && l.pw.bi >= 128;
    const unsigned nx = dx && !bigx ? blocks_of(l.px) : 0, nw = dw && !bigw ? blocks_of(l.pw) : 0;
    if (bigx)
        s = run_tile<GRAD_X>(gx, l.px, l.sz, l.sw, st);
    if (s == SRNL_OK && bigw)
        s = run_tile<GRAD_W>(gw, l.pw, l.sz, l.sx, st);
    if (s == SRNL_OK && nx + nw)
        s = run_grads({gx, gw, nx, nw, l.sz, l.sw, l.sx}, st);
    if (s != SRNL_OK)
        return s;
    return join(make_join(gx.part, dx ? l.px.splits : 1, M * K, gx.e),
                make_join(gw.part, dw ? l.pw.splits : 1, static_cast<long long>(N) * K, ew),
                make_join(gw.rowsum, db ? l.pw.splits : 1, N, eb), st);
}

}  // extern "C"
