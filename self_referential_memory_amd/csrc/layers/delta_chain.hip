// delta_chain.hip -- the gated delta rule's states from chunk to chunk, with the
// outputs, and their gradients from the last chunk back (formulas in delta.h).
//
// The state's columns are independent: a block takes NV of them for one item and
// head, keeps them in registers in fp32 and walks the chunks. What one chunk
// waits for from the one before is a chain of three products, K^ S, X R and K^T W.
// Four of the block's waves do only those, each 16 of the chunk's rows (or its
// share of the state's); four more do what the chain need not wait for, in the
// slots it leaves: forward the outputs, backward the parts P^T dO and Q^T dO of the
// chunk before, and what is recorded. States, errors and their scaled copies pass
// from wave to wave through LDS, transposed; operands that are rows of q, k, X and P
// come straight from memory in the layout the matrix units want, a chunk ahead. Three
// barriers a chunk.
//
// Measured: 16384 tokens, 16 heads of 128, 1.75 us a chunk (450 us, 128 blocks); 4 x
// 4096 x 8 heads 120 us, with the record 145 us (201 MB of it) and back 155 to 172 us.
// The steps' latency bounds it: a barrier, reads of LDS, 12 dependent products, a split,
// three times a chunk. Four waves that shared a state's rows and added partial products
// instead of reading the whole state took 20 % longer, k and v through the helpers 10 %,
// U formed by the helpers from E's tiles 18 %.
#include "delta_mma.h"

namespace {

using namespace srnl_i;

// A block's slab of the state: KD x NV in 16 x 16 tiles, a wave's tiles one
// after the other.
template <int KD, int NV> struct Slab {
    static constexpr int NT = NV / 16, TILES = KD / 16 * NT, MINE = (TILES + 3) / 4;
    static constexpr int COLS = MINE < NT ? MINE : NT;      // columns of tiles a wave has
    int wave, quad, l15;
    __device__ __forceinline__ bool live(int i) const { return TILES % 4 == 0 || wave * MINE + i < TILES; }
    __device__ __forceinline__ int row16(int i) const { return 16 * ((wave * MINE + i) / NT); }
    __device__ __forceinline__ int row(int i) const { return row16(i) + 4 * quad; }
    __device__ __forceinline__ int col(int i) const { return 16 * ((wave * MINE + i) % NT) + l15; }
    __device__ __forceinline__ int col0() const { return COLS < NT ? 16 * (wave * MINE % NT) : 0; }
    // k or q down the chunk's tokens, for every tile
    template <bool BF> __device__ __forceinline__ void down(const Rows<BF, KD> &r, In<BF> (&f)[2][MINE]) const
    {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < MINE; ++i)
                f[h][i] = i % COLS ? f[h][i - 1] : live(i) ? r.down(32 * h, row16(i)) : in_zero<BF>();
    }
};

// The operands that a wave reads of a transposed array in LDS: N reductions of 32
// for each of NT columns of tiles, all at once, so that the products do not wait
// for them one by one.
template <bool BF, int PL, int ROWS, int K, int N, int NT>
__device__ __forceinline__ void read_columns(const Split<BF, PL, ROWS, K> &p, int col0, int quad, int l15, Mid<BF, PL> (&f)[N][NT])
{
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
            f[i][j] = p.get(col0 + 16 * j + l15, 4 * i + quad);
}
// (A chunk's loads are issued without a condition, the last chunk's again at the end:
// behind a branch that may have issued loads, a wait for earlier ones waits for all.
// They go between the operands' reads and the products, in the time that the reads
// take: behind the products they cost a chunk 8 % more.)
__device__ __forceinline__ void hold() { __builtin_amdgcn_sched_barrier(0); }

// What every wave of a block knows.
template <int NV> struct Place {
    int bh, b, h, hk, v0, wave, quad, l15, n, chunks, row, rows;
    bool helper;
    __device__ __forceinline__ explicit Place(const DeltaArgs &a)
    {
        // A head's slabs read the same q, k, X and P: of every eight heads each goes
        // to one XCD (blocks go round the eight), whose L2 then serves all its slabs.
        const int slabs = (a.Dv + NV - 1) / NV, full = a.B * a.H / 8 * 8;
        const int i = blockIdx.x, rest = i - full * slabs;
        bh = rest < 0 ? i % 8 + i / (8 * slabs) * 8 : full + rest / slabs;
        v0 = (rest < 0 ? i / 8 % slabs : rest % slabs) * NV;
        b = bh / a.H;
        h = bh - b * a.H;
        hk = h / (a.H / a.Hk);
        const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        wave = w & 3;
        helper = w >= 4;
        quad = (threadIdx.x & 63) >> 4;
        l15 = threadIdx.x & 15;
        n = delta_tokens(a, b);
        chunks = (n + DELTA_CHUNK - 1) / DELTA_CHUNK;
        row = 16 * wave + l15;            // as an operand
        rows = 16 * wave + 4 * quad;      // in a result
    }
    __device__ __forceinline__ long long at(const DeltaArgs &a, int c) const
    {
        return static_cast<long long>(bh) * a.N + c;
    }
    __device__ __forceinline__ long long token(const DeltaArgs &a, int c) const
    {
        return static_cast<long long>(b) * a.T + DELTA_CHUNK * c;
    }
};

// this wave's 16 rows of a chunk's q or k
template <bool BF, int KF, class P>
__device__ __forceinline__ void load_rows(const DeltaArgs &a, const P &pl, const void *p, long long stride, int c,
                                          In<BF> (&f)[KF])
{
    const Buf b(p, (pl.token(a, c) * stride + static_cast<long long>(pl.hk) * a.Dk) * (BF ? 2 : 4));
    const bool live = pl.row < pl.n - DELTA_CHUNK * c;
    const int o = pl.row * static_cast<int>(stride) + 8 * pl.quad;
#pragma unroll
    for (int i = 0; i < KF; ++i)
        f[i] = in_load<BF>(b, o + 32 * i, both(live, 32 * i + 8 * pl.quad < a.Dk));
}
// this wave's 16 rows of X or P, lower triangular (UPPER: of their transposes): the
// waves whose half of 32 is zero leave it out, here and in the products
template <bool UPPER> __device__ __forceinline__ bool half_live(int wave, int i) { return i == UPPER || (UPPER ? wave < 2 : wave >= 2); }
template <bool BF, int PL, bool UPPER, class P>
__device__ __forceinline__ void load_square(const DeltaArgs &a, const P &pl, const char *p, int c, Mid<BF, PL> (&f)[2])
{
    const Buf b(p, pl.at(a, c) * DELTA_SQUARE);
    if (half_live<UPPER>(pl.wave, !UPPER))
        f[!UPPER] = frag_load<BF, PL>(b, 2 * pl.wave + !UPPER);
    f[UPPER] = frag_load<BF, PL>(b, 2 * pl.wave + UPPER);
}
// This wave's rows of a [tokens][H][Dv] array, as result tiles. Of bf16 ones a lane
// loads two neighbouring columns in two of its four rows, and has the rest from the
// lane beside it: half the loads.
template <bool BF> struct Column { uint32_t w[2]; };
template <> struct Column<false> { float v[4]; };
template <bool BF, int NT, class P>
__device__ __forceinline__ void load_values(const DeltaArgs &a, const P &pl, const void *p, long long stride, int c,
                                            Column<BF> (&v)[NT])
{
    const Buf b(p, (pl.token(a, c) * stride + static_cast<long long>(pl.h) * a.Dv + pl.v0) * (BF ? 2 : 4));
    const int left = pl.n - DELTA_CHUNK * c;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const int col = 16 * j + pl.l15;
        if constexpr (BF) {
            const int odd = pl.l15 & 1;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = pl.rows + 2 * odd + i;
                const bool live = both(r < left, pl.v0 + col < a.Dv);
                v[j].w[i] = __builtin_amdgcn_raw_buffer_load_b32(
                    b.r, live ? 2u * (r * static_cast<int>(stride) + col - odd) : NOWHERE, 0, 0);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const bool live = both(pl.rows + e < left, pl.v0 + col < a.Dv);
                v[j].v[e] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(
                    b.r, live ? 4u * ((pl.rows + e) * static_cast<int>(stride) + col) : NOWHERE, 0, 0));
            }
        }
    }
}
__device__ __forceinline__ v4f values(const Column<true> &c)
{
    const int odd = threadIdx.x & 1;
    v4f v;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t other = beside(c.w[i]);
        // even: this lane's rows 0 and 1, the other's rows 2 and 3, low halves
        v[i] = odd ? bf16_hi(other) : bf16_lo(c.w[i]);
        v[2 + i] = odd ? bf16_hi(c.w[i]) : bf16_lo(other);
    }
    return v;
}
__device__ __forceinline__ v4f values(const Column<false> &c) { return v4f{c.v[0], c.v[1], c.v[2], c.v[3]}; }
// ... and its outputs; tokens past the item's length get zeros. bf16 ones pass the
// caches, as what is recorded does (4 x 4096 x 8 heads with the record: 145 us, 153 not
// so; alone no difference).
template <bool BF, class P>
__device__ __forceinline__ void store_values(const DeltaArgs &a, const P &pl, void *p, int c, int j, v4f v)
{
    const Buf b(p, ((pl.token(a, c) * a.H + pl.h) * a.Dv + pl.v0) * (BF ? 2 : 4));
    const int left = pl.n - DELTA_CHUNK * c, inside = a.T - DELTA_CHUNK * c;
    const int col = 16 * j + pl.l15;
    if constexpr (BF) {
        // lanes of neighbouring columns exchange: each writes two rows of both
        const int odd = pl.l15 & 1;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float mine = odd ? v[2 + i] : v[i], give = odd ? v[i] : v[2 + i];
            const float got = beside(give);
            const int r = pl.rows + 2 * odd + i;
            const uint32_t w = odd ? pack_bf16(got, mine) : pack_bf16(mine, got);
            const bool live = both(r < inside, pl.v0 + col < a.Dv);
            __builtin_amdgcn_raw_buffer_store_b32(r < left ? w : 0u, b.r,
                                                  live ? 2u * (r * a.H * a.Dv + col - odd) : NOWHERE, 0, NT_STORE);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            put_value<false>(b, (pl.rows + e) * a.H * a.Dv + col, both(pl.rows + e < inside, pl.v0 + col < a.Dv),
                             pl.rows + e < left ? v[e] : 0.0f);
    }
}
template <bool BF, int NV> __device__ __forceinline__ void zero_values(const DeltaArgs &a, const Place<NV> &pl, void *p)
{
    const long long past = a.T - static_cast<long long>(DELTA_CHUNK) * pl.chunks;
    for (long long i = threadIdx.x; i < past * NV; i += 512) {
        const int col = pl.v0 + static_cast<int>(i % NV);
        if (col < a.Dv)
            put_at<BF>(p, ((pl.token(a, pl.chunks) + i / NV) * a.H + pl.h) * a.Dv + col, 0.0f);
    }
}
// A chunk's row factors go through LDS: two helpers load them for the whole block
// (a load costs the same for 16 bytes a lane as for the 64 bytes that four rows'
// factors are), two buffers taking turns.
struct Factors {
    __attribute__((aligned(16))) float row[256];     // from VEC_READK on
    float last;                                      // e^(G_63)
    __device__ __forceinline__ v4f rows(int which, int r) const { return *reinterpret_cast<const v4f *>(&row[which + r]); }
};
struct Vec {
    u32x4 w;
    template <class P> __device__ __forceinline__ void load(const DeltaArgs &a, const P &pl, int c)
    {
        const Buf b(a.vec, pl.at(a, c) * VEC_FLOATS * 4);
        w = buf16(b, pl.wave == 0 ? 16 * (threadIdx.x & 63) : pl.wave == 1 ? 4 * (VEC_GAM + 63) : NOWHERE);
    }
    __device__ __forceinline__ void store(Factors &f, int wave) const
    {
        if (wave == 0)
            *reinterpret_cast<u32x4 *>(&f.row[4 * (threadIdx.x & 63)]) = w;
        else if (wave == 1)
            f.last = __builtin_bit_cast(float, w[0]);
    }
};
// the state's slab from memory, and back
template <int KD, int NV>
__device__ __forceinline__ void load_state(const DeltaArgs &a, const Place<NV> &pl, const Slab<KD, NV> &sl, const float *p,
                                           v4f (&S)[Slab<KD, NV>::MINE])
{
#pragma unroll
    for (int i = 0; i < Slab<KD, NV>::MINE; ++i) {
        S[i] = v4f_zero();
        const int col = pl.v0 + sl.col(i);
        if (p && sl.live(i) && col < a.Dv)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (sl.row(i) + e < a.Dk)
                    S[i][e] = p[(static_cast<long long>(pl.bh) * a.Dk + sl.row(i) + e) * a.Dv + col];
    }
}
template <int KD, int NV>
__device__ __forceinline__ void store_state(const DeltaArgs &a, const Place<NV> &pl, const Slab<KD, NV> &sl, float *p,
                                            long long at, const v4f (&S)[Slab<KD, NV>::MINE])
{
    const Buf b(p, (at * a.Dk * a.Dv + pl.v0) * 4);
#pragma unroll
    for (int i = 0; i < Slab<KD, NV>::MINE; ++i) {
        // rows go in fours, Dk in eights
        const bool live = both(both(sl.live(i), sl.row(i) < a.Dk), pl.v0 + sl.col(i) < a.Dv);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            put_value<false>(b, (sl.row(i) + e) * a.Dv + sl.col(i), live, S[i][e]);
    }
}
// What is recorded, by the helpers, 16 bytes a lane, in panels of 8 columns (record_at),
// so that a wave writes 512 bytes side by side. The state's slab comes from its words
// in LDS, which hold all its 24 bits: a lane has 8 columns of a row.
template <bool BF, int KD, int NV>
__device__ __forceinline__ void store_words(const DeltaArgs &a, const Place<NV> &pl, const Split<BF, 3, NV, KD> &s, float *p,
                                            long long at)
{
    constexpr int PER = 512 / NV, ALL = KD / PER;      // rows a wave has at once; times
    const Buf b(p, at * a.Dk * a.Dv * 4);
    const int g = pl.quad % (NV / 8), tile = 16 * (pl.quad / (NV / 8));
#pragma unroll
    for (int i = 0; i < (ALL + 3) / 4; ++i) {
        const int u = pl.wave + 4 * i;
        if (ALL % 4 && u >= ALL)
            break;
        float v[8];
        s.down(8 * g, PER * u + tile, v);
        const int row = PER * u + tile + pl.l15;
        put8(b, record_at(row, pl.v0 + 8 * g, a.Dk), both(row < a.Dk, pl.v0 + 8 * g < a.Dv), v);
    }
}
// this wave's 16 rows of a [64][Dv] fp32 array, from its result tile in LDS
template <class P> __device__ __forceinline__ void store_rows(const DeltaArgs &a, const P &pl, float *p, int c, int j, const v4f (&t)[64])
{
    const Buf b(p, pl.at(a, c) * DELTA_CHUNK * a.Dv * 4);
    const int lane = threadIdx.x & 63, r = lane >> 2, col = 16 * j + 4 * (lane & 3);
    v4f v;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] = reinterpret_cast<const float *>(&t[16 * (r >> 2) + (col & 15) + i])[r & 3];
    put4(b, record_at(16 * pl.wave + r, pl.v0 + col, DELTA_CHUNK), pl.v0 + col < a.Dv, v);
}

// ------------------------------------------------------------------- forward

template <bool BF, int KD, int NV, bool RECORD> struct FwdShared {
    __attribute__((aligned(16))) Rows<BF, KD> k;
    Split<BF, 3, NV, KD> S;                            // the state, transposed
    Split<BF, 3, NV, 64> R, W, U;
    v4f e[RECORD ? 4 : 1][NV / 16][64];                // E as result tiles, for the helpers to record
    Factors w[2];
};

// What the chain reads of a chunk, in two parts, so that its loads and the helpers'
// take turns.
template <bool BF, int KF, int NT, bool BACK> struct ChainIn {
    In<BF> k[KF];
    Mid<BF, 3> x[2];                  // of X, backward of its transpose
    Column<BF> v[NT];                 // forward
    template <class P> __device__ __forceinline__ void load(const DeltaArgs &a, const P &pl, int c)
    {
        load_rows<BF, KF>(a, pl, a.k, a.ks, c, k);
        if (!BACK)
            load_values<BF, NT>(a, pl, a.v, a.vs, c, v);
    }
    template <class P> __device__ __forceinline__ void load_x(const DeltaArgs &a, const P &pl, int c)
    {
        load_square<BF, 3, BACK>(a, pl, a.X, c, x);
    }
};
template <bool BF, int KF> struct OutIn {
    In<BF> q[KF];
    Mid<BF, 3> p[2];
    Vec vec;                          // the next chunk's
    template <class P> __device__ __forceinline__ void load(const DeltaArgs &a, const P &pl, int c)
    {
        const int last = pl.chunks - 1;
        load_rows<BF, KF>(a, pl, a.q, a.qs, c < last ? c : last, q);
        load_square<BF, 3, false>(a, pl, a.P, c < last ? c : last, p);
        vec.load(a, pl, c + 1 < last ? c + 1 : last);
    }
};

template <bool BF, int KD, int NV, bool RECORD> __global__ __launch_bounds__(512) void delta_chain_kernel(DeltaArgs a)
{
    constexpr int KF = KD / 32, NT = NV / 16;
    using Sl = Slab<KD, NV>;
    __shared__ FwdShared<BF, KD, NV, RECORD> sh;
    const Place<NV> pl(a);
    const int lane = threadIdx.x & 63;
    if (!pl.helper) {
        const Sl sl{pl.wave, pl.quad, pl.l15};
        v4f S[Sl::MINE];
        load_state<KD, NV>(a, pl, sl, a.state, S);
#pragma unroll
        for (int i = 0; i < Sl::MINE; ++i)
            if (sl.live(i))
                sh.S.put4(sl.col(i), sl.row(i), S[i]);
        __builtin_amdgcn_s_setprio(2);
        const auto chunk = [&](const ChainIn<BF, KF, NT, false> &in, ChainIn<BF, KF, NT, false> &next, int c) __attribute__((always_inline)) {
            Mid<BF, 3> op[KF][NT];
            read_columns(sh.S, 0, pl.quad, pl.l15, op);
            const int after = c + 1 < pl.chunks ? c + 1 : c;
            next.load(a, pl, after);
            hold();
            Sum<BF, 3> kS[NT];
#pragma unroll
            for (int f = 0; f < KF; ++f)
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    kS[j].add(in.k[f], op[f][j]);
            const Factors &w = sh.w[c & 1];
            const v4f read = w.rows(VEC_READK, pl.rows);
#pragma unroll
            for (int f = 0; f < KF; ++f)
                sh.k.put(pl.row, 32 * f + 8 * pl.quad, in.k[f]);
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                sh.R.put4(16 * j + pl.l15, pl.rows, values(in.v[j]) - read * kS[j].value());
            }
            lds_barrier();
            const v4f write = w.rows(VEC_WRITE, pl.rows), beta = w.rows(VEC_BETA, pl.rows);
            Mid<BF, 3> rs[2][NT];
            read_columns(sh.R, 0, pl.quad, pl.l15, rs);
            next.load_x(a, pl, after);
            hold();
            Sum<BF, 3> err[NT];
#pragma unroll
            for (int f = 0; f < 2; ++f)
                if (half_live<false>(pl.wave, f))
#pragma unroll
                    for (int j = 0; j < NT; ++j)
                        err[j].add(in.x[f], rs[f][j]);
            In<BF> kd[2][Sl::MINE];
            sl.template down<BF>(sh.k, kd);
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const v4f e = err[j].value();
                sh.W.put4(16 * j + pl.l15, pl.rows, write * e);
                sh.U.put4(16 * j + pl.l15, pl.rows, beta * e);
                if (RECORD)
                    sh.e[pl.wave][j][lane] = e;
            }
            lds_barrier();
            const float last = w.last;
            Mid<BF, 3> ws[2][Sl::COLS];
            read_columns(sh.W, sl.col0(), pl.quad, pl.l15, ws);
            hold();
            Sum<BF, 3> dS[Sl::MINE];
#pragma unroll
            for (int f = 0; f < 2; ++f)
#pragma unroll
                for (int i = 0; i < Sl::MINE; ++i)
                    dS[i].add(kd[f][i], ws[f][i % Sl::COLS]);
#pragma unroll
            for (int i = 0; i < Sl::MINE; ++i) {
                S[i] = S[i] * last + dS[i].value();
                if (sl.live(i))
                    sh.S.put4(sl.col(i), sl.row(i), S[i]);
            }
            lds_barrier();
        };
        ChainIn<BF, KF, NT, false> in[2];
        if (pl.chunks) {
            in[0].load(a, pl, 0);
            in[0].load_x(a, pl, 0);
        }
        lds_barrier();
        for (int c = 0; c < pl.chunks; c += 2) {
            chunk(in[0], in[1], c);
            if (c + 1 < pl.chunks)
                chunk(in[1], in[0], c + 1);
        }
        if (a.state_out)
            store_state<KD, NV>(a, pl, sl, a.state_out, pl.bh, S);
    } else {
        const auto chunk = [&](const OutIn<BF, KF> &in, OutIn<BF, KF> &next, int c) __attribute__((always_inline)) {
            Sum<BF, 3> qS[NT];
#pragma unroll
            for (int f = 0; f < KF; ++f)
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    qS[j].add(in.q[f], sh.S.get(16 * j + pl.l15, 4 * f + pl.quad));
            const v4f read = sh.w[c & 1].rows(VEC_READQ, pl.rows);
            lds_barrier();
            next.load(a, pl, c + 1);
            if (RECORD)
                store_words<BF, KD, NV>(a, pl, sh.S, a.S0, pl.at(a, c));
            lds_barrier();
            in.vec.store(sh.w[(c + 1) & 1], pl.wave);
            Mid<BF, 3> us[2][NT];
            read_columns(sh.U, 0, pl.quad, pl.l15, us);
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                Sum<BF, 3> pU;
#pragma unroll
                for (int f = 0; f < 2; ++f)
                    if (half_live<false>(pl.wave, f))
                        pU.add(in.p[f], us[f][j]);
                store_values<BF>(a, pl, a.out, c, j, read * qS[j].value() + pU.value());
                if (RECORD)
                    store_rows(a, pl, a.E, c, j, sh.e[pl.wave][j]);
            }
            lds_barrier();
        };
        OutIn<BF, KF> in[2];
        if (pl.chunks) {
            Vec first;
            first.load(a, pl, 0);
            in[0].load(a, pl, 0);
            first.store(sh.w[0], pl.wave);
        }
        lds_barrier();
        for (int c = 0; c < pl.chunks; c += 2) {
            chunk(in[0], in[1], c);
            if (c + 1 < pl.chunks)
                chunk(in[1], in[0], c + 1);
        }
    }
    zero_values<BF, NV>(a, pl, a.out);
}

// ------------------------------------------------------------------ backward

template <bool BF, int KD, int NV> struct BwdShared {
    using Sl = Slab<KD, NV>;
    __attribute__((aligned(16))) Rows<BF, KD> k, q;
    Split<BF, 3, NV, KD> D;                            // the state's gradient, transposed
    Split<BF, 3, NV, 64> W, V, Os;                     // Os: dO times scale e^G / |q|
    Split<BF, 1, NV, 64> O;                            // dO, transposed
    // what the helpers hand to the chain, as result tiles: P^T dO and Q^T dO
    v4f po[4][NV / 16][64], qo[4][Sl::MINE][64];
    v4f dv[4][NV / 16][64];                            // and the chain to them: dV
    Factors w[2];
};

template <bool BF, int KF, int NT> struct HelpBack {
    In<BF> q[KF];
    Mid<BF, 3> p[2];                  // of P's transpose
    Column<BF> o[NT];
    v4f read;                         // scale e^G / |q|
    Vec vec;
    template <class P> __device__ __forceinline__ void load(const DeltaArgs &a, const P &pl, int c)
    {
        load_rows<BF, KF>(a, pl, a.q, a.qs, c, q);
        load_square<BF, 3, true>(a, pl, a.P, c, p);
        load_values<BF, NT>(a, pl, a.dout, static_cast<long long>(a.H) * a.Dv, c, o);
        const Buf b(a.vec, pl.at(a, c) * VEC_FLOATS * 4);
        read = __builtin_bit_cast(v4f, buf16(b, 4 * (VEC_READQ + pl.rows)));
        vec.load(a, pl, c);
    }
};

template <bool BF, int KD, int NV> __global__ __launch_bounds__(512) void delta_chain_bwd_kernel(DeltaArgs a)
{
    constexpr int KF = KD / 32, NT = NV / 16;
    using Sl = Slab<KD, NV>;
    __shared__ BwdShared<BF, KD, NV> sh;
    const Place<NV> pl(a);
    const Sl sl{pl.wave, pl.quad, pl.l15};
    const int lane = threadIdx.x & 63;
    if (!pl.helper) {
        v4f D[Sl::MINE];
        load_state<KD, NV>(a, pl, sl, a.dstate_out, D);
#pragma unroll
        for (int i = 0; i < Sl::MINE; ++i)
            if (sl.live(i))
                sh.D.put4(sl.col(i), sl.row(i), D[i]);
        __builtin_amdgcn_s_setprio(2);
        const auto chunk = [&](const ChainIn<BF, KF, NT, true> &in, ChainIn<BF, KF, NT, true> &next, int c) __attribute__((always_inline)) {
            Mid<BF, 3> op[KF][NT];
            read_columns(sh.D, 0, pl.quad, pl.l15, op);
            const int after = c > 0 ? c - 1 : 0;
            next.load(a, pl, after);
            hold();
            Sum<BF, 3> kD[NT];
#pragma unroll
            for (int f = 0; f < KF; ++f)
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    kD[j].add(in.k[f], op[f][j]);
            const Factors &w = sh.w[c & 1];
            const v4f write = w.rows(VEC_WRITE, pl.rows), beta = w.rows(VEC_BETA, pl.rows);
#pragma unroll
            for (int f = 0; f < KF; ++f)
                sh.k.put(pl.row, 32 * f + 8 * pl.quad, in.k[f]);
#pragma unroll
            for (int j = 0; j < NT; ++j)
                sh.W.put4(16 * j + pl.l15, pl.rows,
                                  write * kD[j].value() + beta * sh.po[pl.wave][j][lane]);
            lds_barrier();
            const v4f read = w.rows(VEC_READK, pl.rows);
            Mid<BF, 3> ws[2][NT];
            read_columns(sh.W, 0, pl.quad, pl.l15, ws);
            next.load_x(a, pl, after);
            hold();
            Sum<BF, 3> dv[NT];
#pragma unroll
            for (int f = 0; f < 2; ++f)
                if (half_live<true>(pl.wave, f))
#pragma unroll
                    for (int j = 0; j < NT; ++j)
                        dv[j].add(in.x[f], ws[f][j]);
            In<BF> kd[2][Sl::MINE];
            sl.template down<BF>(sh.k, kd);
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const v4f d = dv[j].value();
                sh.V.put4(16 * j + pl.l15, pl.rows, -read * d);
                sh.dv[pl.wave][j][lane] = d;
            }
            lds_barrier();
            const float last = w.last;
            Mid<BF, 3> vs[2][Sl::COLS];
            read_columns(sh.V, sl.col0(), pl.quad, pl.l15, vs);
            hold();
            Sum<BF, 3> dD[Sl::MINE];
#pragma unroll
            for (int f = 0; f < 2; ++f)
#pragma unroll
                for (int i = 0; i < Sl::MINE; ++i)
                    dD[i].add(kd[f][i], vs[f][i % Sl::COLS]);
#pragma unroll
            for (int i = 0; i < Sl::MINE; ++i) {
                D[i] = (D[i] * last + sh.qo[pl.wave][i][lane]) + dD[i].value();
                if (sl.live(i))
                    sh.D.put4(sl.col(i), sl.row(i), D[i]);
            }
            lds_barrier();
        };
        ChainIn<BF, KF, NT, true> in[2];
        if (pl.chunks) {
            in[0].load(a, pl, pl.chunks - 1);
            in[0].load_x(a, pl, pl.chunks - 1);
        }
        lds_barrier();
        lds_barrier();
        for (int c = pl.chunks - 1; c >= 0; c -= 2) {
            chunk(in[0], in[1], c);
            if (c > 0)
                chunk(in[1], in[0], c - 1);
        }
        if (a.dstate)
            store_state<KD, NV>(a, pl, sl, a.dstate, pl.bh, D);
    } else {
        v4f qo[Sl::MINE];
        // q, dO and the factors of a chunk to LDS
        const auto spread = [&](const HelpBack<BF, KF, NT> &in, int c) __attribute__((always_inline)) {
            in.vec.store(sh.w[c & 1], pl.wave);
#pragma unroll
            for (int f = 0; f < KF; ++f)
                sh.q.put(pl.row, 32 * f + 8 * pl.quad, in.q[f]);
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const v4f o = values(in.o[j]);
                sh.O.put4(16 * j + pl.l15, pl.rows, o);
                sh.Os.put4(16 * j + pl.l15, pl.rows, in.read * o);
            }
        };
        // its parts P^T dO, to LDS, and Q^T dO, kept
        const auto parts = [&](const HelpBack<BF, KF, NT> &in) __attribute__((always_inline)) {
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                v4f o = v4f_zero();
#pragma unroll
                for (int f = 0; f < 2; ++f) {
                    if (!half_live<true>(pl.wave, f))
                        continue;
                    o = mma(in.p[f], sh.O.get_in(16 * j + pl.l15, 4 * f + pl.quad), o);
                }
                sh.po[pl.wave][j][lane] = o;
            }
#pragma unroll
            for (int i = 0; i < Sl::MINE; ++i) {
                qo[i] = v4f_zero();
                if (sl.live(i))
#pragma unroll
                    for (int f = 0; f < 2; ++f)
                        qo[i] = mma(sh.q.down(32 * f, sl.row16(i)), sh.Os.get(sl.col(i), 4 * f + pl.quad), qo[i]);
            }
        };
        HelpBack<BF, KF, NT> in;
        if (pl.chunks) {
            in.load(a, pl, pl.chunks - 1);
            spread(in, pl.chunks - 1);
        }
        lds_barrier();
        if (pl.chunks) {
            parts(in);
            in.load(a, pl, pl.chunks > 1 ? pl.chunks - 2 : 0);
        }
        lds_barrier();
        for (int c = pl.chunks - 1; c >= 0; --c) {
            // the chain reads Q^T dO of chunk c behind its second barrier from here
#pragma unroll
            for (int i = 0; i < Sl::MINE; ++i)
                sh.qo[pl.wave][i][lane] = qo[i];
            if (c > 0)
                spread(in, c - 1);
            store_words<BF, KD, NV>(a, pl, sh.D, a.D1, pl.at(a, c));
            lds_barrier();
            if (c > 0) {
                parts(in);
                in.load(a, pl, c > 1 ? c - 2 : 0);
            }
            lds_barrier();
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                store_rows(a, pl, a.dV, c, j, sh.dv[pl.wave][j]);
                if (a.dv)
                    store_values<BF>(a, pl, a.dv, c, j, sh.dv[pl.wave][j][lane]);
            }
            lds_barrier();
        }
    }
    if (a.dv)
        zero_values<BF, NV>(a, pl, a.dv);
}

template <bool BF, int KD, int NV> void launch_chain(const DeltaArgs &a, bool backward, hipStream_t st)
{
    const dim3 grid(static_cast<unsigned>(static_cast<long long>(a.B) * a.H * ((a.Dv + NV - 1) / NV))), block(512);
    if (backward)
        hipLaunchKernelGGL((delta_chain_bwd_kernel<BF, KD, NV>), grid, block, 0, st, a);
    else if (a.E)
        hipLaunchKernelGGL((delta_chain_kernel<BF, KD, NV, true>), grid, block, 0, st, a);
    else
        hipLaunchKernelGGL((delta_chain_kernel<BF, KD, NV, false>), grid, block, 0, st, a);
}

}  // namespace

namespace srnl_i {

srnl_status launch_delta_chain(const DeltaArgs &a, bool backward, hipStream_t st)
{
    // 32 columns a block; 16 where that leaves compute units idle: 16 chunks of 128 with
    // the record take 64 us with 256 blocks of 32 (16: 79), 58 with 128 of 32 (16: 39)
    const bool narrow = a.Dv <= 16 || static_cast<long long>(a.B) * a.H * ((a.Dv + 31) / 32) < 256;
#define SRNL_DELTA_CHAIN(BF, KD)                   \
    if (narrow)                                    \
        launch_chain<BF, KD, 16>(a, backward, st); \
    else                                           \
        launch_chain<BF, KD, 32>(a, backward, st)
    SRNL_DELTA_DISPATCH(a, SRNL_DELTA_CHAIN);
    return launched(backward ? "delta_chain_bwd_kernel" : "delta_chain_kernel");
}

}  // namespace srnl_i
