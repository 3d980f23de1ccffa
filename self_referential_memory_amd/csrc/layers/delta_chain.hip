// delta_chain.hip -- the gated delta rule's states from chunk to chunk, with the
// outputs, and their gradients from the last chunk back (formulas in delta.h).
//
// The state's columns are independent: a block takes NV of them for one item and
// head, keeps them in registers in fp32 and walks the chunks. What one chunk
// waits for from the one before is a chain of three products, K^ S, X R and K^T W.
// Four of the block's waves do only those, each 16 of the chunk's rows (or its
// share of the state's); four more do what the chain need not wait for, in the
// slots it leaves: forward the outputs, backward the parts P^T dO and Q^T dO of the
// chunk before. States, errors and their scaled copies pass from wave to wave
// through LDS, transposed; operands that are rows of q, k, X and P come straight
// from memory in the layout the matrix units want, a chunk ahead. Three barriers a
// chunk.
#include "delta_mma.h"

namespace {

using namespace srnl_i;

// A block's slab of the state: KD x NV in 16 x 16 tiles, a wave's tiles one
// after the other.
template <int KD, int NV> struct Slab {
    static constexpr int NT = NV / 16, TILES = KD / 16 * NT, MINE = (TILES + 3) / 4;
    int wave, quad, l15;
    __device__ __forceinline__ bool live(int i) const { return TILES % 4 == 0 || wave * MINE + i < TILES; }
    __device__ __forceinline__ int row16(int i) const { return 16 * ((wave * MINE + i) / NT); }
    __device__ __forceinline__ int row(int i) const { return row16(i) + 4 * quad; }
    __device__ __forceinline__ int col(int i) const { return 16 * ((wave * MINE + i) % NT) + l15; }
};

// What every wave of a block knows.
template <int NV> struct Place {
    int bh, b, h, hk, v0, wave, quad, l15, n, chunks, row, rows;
    bool helper;
    __device__ __forceinline__ explicit Place(const DeltaArgs &a)
    {
        const int slabs = (a.Dv + NV - 1) / NV;
        bh = blockIdx.x / slabs;
        v0 = (blockIdx.x - bh * slabs) * NV;
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
        f[i] = in_load<BF>(b, o + 32 * i, live && 32 * i + 8 * pl.quad < a.Dk);
}
// this wave's 16 rows of X or P
template <bool BF, int PL, class P>
__device__ __forceinline__ void load_square(const DeltaArgs &a, const P &pl, const char *p, int c, Mid<BF, PL> (&f)[2])
{
    const Buf b(p, pl.at(a, c) * DELTA_SQUARE);
#pragma unroll
    for (int i = 0; i < 2; ++i)
        f[i] = mid_load<BF, PL>(b, (pl.row * 8 + pl.quad + 4 * i) * mid8<BF, PL>);
}
// this wave's rows of a [tokens][H][Dv] array, as a result tile
template <bool BF, int NT, class P>
__device__ __forceinline__ void load_values(const DeltaArgs &a, const P &pl, const void *p, long long stride, int c,
                                            Raw<BF> (&v)[NT][4])
{
    const Buf b(p, (pl.token(a, c) * stride + static_cast<long long>(pl.h) * a.Dv + pl.v0) * (BF ? 2 : 4));
    const int left = pl.n - DELTA_CHUNK * c;
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            v[j][e] = raw_load<BF>(b, (pl.rows + e) * static_cast<int>(stride) + 16 * j + pl.l15,
                                   pl.rows + e < left && pl.v0 + 16 * j + pl.l15 < a.Dv);
}
// ... and its outputs; tokens past the item's length get zeros
template <bool BF, class P>
__device__ __forceinline__ void store_values(const DeltaArgs &a, const P &pl, void *p, int c, int j, v4f v)
{
    const Buf b(p, ((pl.token(a, c) * a.H + pl.h) * a.Dv + pl.v0) * (BF ? 2 : 4));
    const int left = pl.n - DELTA_CHUNK * c, inside = a.T - DELTA_CHUNK * c;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        put_value<BF>(b, (pl.rows + e) * a.H * a.Dv + 16 * j + pl.l15,
                      pl.rows + e < inside && pl.v0 + 16 * j + pl.l15 < a.Dv, pl.rows + e < left ? v[e] : 0.0f);
}
// this wave's rows of a [64][Dv] fp32 array
template <class P> __device__ __forceinline__ void store_rows(const DeltaArgs &a, const P &pl, float *p, int c, int j, v4f v)
{
    const Buf b(p, (pl.at(a, c) * DELTA_CHUNK * a.Dv + pl.v0) * 4);
#pragma unroll
    for (int e = 0; e < 4; ++e)
        put_value<false>(b, (pl.rows + e) * a.Dv + 16 * j + pl.l15, pl.v0 + 16 * j + pl.l15 < a.Dv, v[e]);
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
// this wave's rows of a chunk's factors, and the chunk's whole decay
struct Factors {
    v4f gam, end, beta, rk, rq;
    float last;
};
template <class P> __device__ __forceinline__ Factors load_factors(const DeltaArgs &a, const P &pl, int c)
{
    const Buf b(a.vec, pl.at(a, c) * VEC_FLOATS * 4);
    const auto four = [&](int which) { return __builtin_bit_cast(v4f, buf16(b, 4 * (which + pl.rows))); };
    Factors f = {four(VEC_GAM), four(VEC_END), four(VEC_BETA), four(VEC_RK), four(VEC_RQ), 0.0f};
    f.last = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(b.r, 4 * (VEC_GAM + 63), 0, 0));
    return f;
}
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
        const bool live = sl.live(i) && sl.row(i) < a.Dk && pl.v0 + sl.col(i) < a.Dv;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            put_value<false>(b, (sl.row(i) + e) * a.Dv + sl.col(i), live, S[i][e]);
    }
}

// ------------------------------------------------------------------- forward

template <bool BF, int KD, int NV> struct FwdShared {
    __attribute__((aligned(16))) Rows<BF, KD> k;
    __attribute__((aligned(16))) char S[NV][mid_row<BF, 3>(KD)];       // the state, transposed
    __attribute__((aligned(16))) char R[NV][mid_row<BF, 3>(64)], U[NV][mid_row<BF, 2>(64)], W[NV][mid_row<BF, 3>(64)];
};

template <bool BF, int KF, int NT> struct ChainIn {
    In<BF> k[KF];
    Mid<BF, 3> x[2];
    Raw<BF> v[NT][4];
    Factors w;
    template <class P> __device__ __forceinline__ void load(const DeltaArgs &a, const P &pl, int c)
    {
        load_rows<BF, KF>(a, pl, a.k, a.ks, c, k);
        load_square<BF, 3>(a, pl, a.X, c, x);
        load_values<BF, NT>(a, pl, a.v, a.vs, c, v);
        w = load_factors(a, pl, c);
    }
};
template <bool BF, int KF> struct OutIn {
    In<BF> q[KF];
    Mid<BF, 2> p[2];
    Factors w;
    template <class P> __device__ __forceinline__ void load(const DeltaArgs &a, const P &pl, int c)
    {
        load_rows<BF, KF>(a, pl, a.q, a.qs, c, q);
        load_square<BF, 2>(a, pl, a.P, c, p);
        w = load_factors(a, pl, c);
    }
};

template <bool BF, int KD, int NV, bool RECORD> __global__ __launch_bounds__(512) void delta_chain_kernel(DeltaArgs a)
{
    constexpr int KF = KD / 32, NT = NV / 16, S8 = mid8<BF, 3>;
    using Sl = Slab<KD, NV>;
    __shared__ FwdShared<BF, KD, NV> sh;
    const Place<NV> pl(a);
    if (!pl.helper) {
        const Sl sl{pl.wave, pl.quad, pl.l15};
        v4f S[Sl::MINE];
        load_state<KD, NV>(a, pl, sl, a.state, S);
#pragma unroll
        for (int i = 0; i < Sl::MINE; ++i)
            if (sl.live(i))
                mid_store4<BF, 3>(sh.S[sl.col(i)], sl.row(i), S[i]);
        __builtin_amdgcn_s_setprio(2);
        const auto chunk = [&](const ChainIn<BF, KF, NT> &in, ChainIn<BF, KF, NT> &next, int c) __attribute__((always_inline)) {
            if (c + 1 < pl.chunks)
                next.load(a, pl, c + 1);
#pragma unroll
            for (int f = 0; f < KF; ++f)
                sh.k.put(pl.row, 32 * f + 8 * pl.quad, in.k[f]);
            const v4f read = in.w.gam * in.w.rk, write = in.w.end * in.w.rk;
            v4f kS[NT];
#pragma unroll
            for (int j = 0; j < NT; ++j)
                kS[j] = v4f_zero();
#pragma unroll
            for (int f = 0; f < KF; ++f)
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    kS[j] = mma(in.k[f], mid_load<BF, 3>(sh.S[16 * j + pl.l15] + (4 * f + pl.quad) * S8), kS[j]);
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                v4f r;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    r[e] = value(in.v[j][e]) - read[e] * kS[j][e];
                mid_store4<BF, 3>(sh.R[16 * j + pl.l15], pl.rows, r);
            }
            if (RECORD)
                store_state<KD, NV>(a, pl, sl, a.S0, pl.at(a, c), S);
            lds_barrier();
            v4f err[NT];
#pragma unroll
            for (int j = 0; j < NT; ++j)
                err[j] = v4f_zero();
#pragma unroll
            for (int f = 0; f < 2; ++f)
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    err[j] = mma(in.x[f], mid_load<BF, 3>(sh.R[16 * j + pl.l15] + (4 * f + pl.quad) * S8), err[j]);
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const v4f u = in.w.beta * err[j];
                mid_store4<BF, 3>(sh.W[16 * j + pl.l15], pl.rows, write * u);
                mid_store4<BF, 2>(sh.U[16 * j + pl.l15], pl.rows, u);
            }
            if (RECORD) {
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    store_rows(a, pl, a.E, c, j, err[j]);
            }
            lds_barrier();
#pragma unroll
            for (int i = 0; i < Sl::MINE; ++i) {
                if (!sl.live(i))
                    continue;
                S[i] *= in.w.last;
#pragma unroll
                for (int f = 0; f < 2; ++f)
                    S[i] = mma(sh.k.down(32 * f, sl.row16(i)), mid_load<BF, 3>(sh.W[sl.col(i)] + (4 * f + pl.quad) * S8), S[i]);
                mid_store4<BF, 3>(sh.S[sl.col(i)], sl.row(i), S[i]);
            }
            lds_barrier();
        };
        ChainIn<BF, KF, NT> in[2];
        if (pl.chunks)
            in[0].load(a, pl, 0);
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
            if (c + 1 < pl.chunks)
                next.load(a, pl, c + 1);
            v4f o[NT];
#pragma unroll
            for (int j = 0; j < NT; ++j)
                o[j] = v4f_zero();
#pragma unroll
            for (int f = 0; f < KF; ++f)
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    o[j] = mma(in.q[f], mid_load<BF, 2>(sh.S[16 * j + pl.l15] + (4 * f + pl.quad) * S8), o[j]);
            lds_barrier();
            lds_barrier();
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                o[j] *= in.w.gam * in.w.rq * a.scale;
#pragma unroll
                for (int f = 0; f < 2; ++f)
                    o[j] = mma(in.p[f], mid_load<BF, 2>(sh.U[16 * j + pl.l15] + (4 * f + pl.quad) * mid8<BF, 2>), o[j]);
                store_values<BF>(a, pl, a.out, c, j, o[j]);
            }
            lds_barrier();
        };
        OutIn<BF, KF> in[2];
        if (pl.chunks)
            in[0].load(a, pl, 0);
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
    __attribute__((aligned(16))) char D[NV][mid_row<BF, 3>(KD)];       // the state's gradient, transposed
    __attribute__((aligned(16))) char W[NV][mid_row<BF, 3>(64)], V[NV][mid_row<BF, 3>(64)];
    __attribute__((aligned(16))) char Os[NV][mid_row<BF, 3>(64)];      // dO times scale e^G / |q|, transposed
    __attribute__((aligned(16))) char O[NV][mid_row<BF, 1>(64)];       // dO, transposed
    // what the helpers hand to the chain, as result tiles: P^T dO and Q^T dO
    v4f po[4][NV / 16][64], qo[4][Sl::MINE][64];
};

template <bool BF, int KF> struct ChainBack {
    In<BF> k[KF];
    Mid<BF, 3> x[2];                  // of X's transpose
    Factors w;
    template <class P> __device__ __forceinline__ void load(const DeltaArgs &a, const P &pl, int c)
    {
        load_rows<BF, KF>(a, pl, a.k, a.ks, c, k);
        load_square<BF, 3>(a, pl, a.X, c, x);
        w = load_factors(a, pl, c);
    }
};
template <bool BF, int KF, int NT> struct HelpBack {
    In<BF> q[KF];
    Mid<BF, 3> p[2];                  // of P's transpose
    Raw<BF> o[NT][4];
    Factors w;
    template <class P> __device__ __forceinline__ void load(const DeltaArgs &a, const P &pl, int c)
    {
        load_rows<BF, KF>(a, pl, a.q, a.qs, c, q);
        load_square<BF, 3>(a, pl, a.P, c, p);
        load_values<BF, NT>(a, pl, a.dout, static_cast<long long>(a.H) * a.Dv, c, o);
        w = load_factors(a, pl, c);
    }
};

template <bool BF, int KD, int NV> __global__ __launch_bounds__(512) void delta_chain_bwd_kernel(DeltaArgs a)
{
    constexpr int KF = KD / 32, NT = NV / 16, S8 = mid8<BF, 3>;
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
                mid_store4<BF, 3>(sh.D[sl.col(i)], sl.row(i), D[i]);
        __builtin_amdgcn_s_setprio(2);
        const auto chunk = [&](const ChainBack<BF, KF> &in, ChainBack<BF, KF> &next, int c) __attribute__((always_inline)) {
            if (c > 0)
                next.load(a, pl, c - 1);
#pragma unroll
            for (int f = 0; f < KF; ++f)
                sh.k.put(pl.row, 32 * f + 8 * pl.quad, in.k[f]);
            const v4f read = in.w.gam * in.w.rk, write = in.w.end * in.w.rk;
            v4f kD[NT];
#pragma unroll
            for (int j = 0; j < NT; ++j)
                kD[j] = v4f_zero();
#pragma unroll
            for (int f = 0; f < KF; ++f)
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    kD[j] = mma(in.k[f], mid_load<BF, 3>(sh.D[16 * j + pl.l15] + (4 * f + pl.quad) * S8), kD[j]);
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const v4f du = write * kD[j] + sh.po[pl.wave][j][lane];
                mid_store4<BF, 3>(sh.W[16 * j + pl.l15], pl.rows, in.w.beta * du);
            }
            store_state<KD, NV>(a, pl, sl, a.D1, pl.at(a, c), D);
            lds_barrier();
            v4f dv[NT];
#pragma unroll
            for (int j = 0; j < NT; ++j)
                dv[j] = v4f_zero();
#pragma unroll
            for (int f = 0; f < 2; ++f)
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    dv[j] = mma(in.x[f], mid_load<BF, 3>(sh.W[16 * j + pl.l15] + (4 * f + pl.quad) * S8), dv[j]);
#pragma unroll
            for (int j = 0; j < NT; ++j)
                mid_store4<BF, 3>(sh.V[16 * j + pl.l15], pl.rows, -read * dv[j]);
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                store_rows(a, pl, a.dV, c, j, dv[j]);
                if (a.dv)
                    store_values<BF>(a, pl, a.dv, c, j, dv[j]);
            }
            lds_barrier();
#pragma unroll
            for (int i = 0; i < Sl::MINE; ++i) {
                if (!sl.live(i))
                    continue;
                D[i] = D[i] * in.w.last + sh.qo[pl.wave][i][lane];
#pragma unroll
                for (int f = 0; f < 2; ++f)
                    D[i] = mma(sh.k.down(32 * f, sl.row16(i)), mid_load<BF, 3>(sh.V[sl.col(i)] + (4 * f + pl.quad) * S8), D[i]);
                mid_store4<BF, 3>(sh.D[sl.col(i)], sl.row(i), D[i]);
            }
            lds_barrier();
        };
        ChainBack<BF, KF> in[2];
        if (pl.chunks)
            in[0].load(a, pl, pl.chunks - 1);
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
        // q and dO of a chunk to LDS
        const auto spread = [&](const HelpBack<BF, KF, NT> &in) __attribute__((always_inline)) {
#pragma unroll
            for (int f = 0; f < KF; ++f)
                sh.q.put(pl.row, 32 * f + 8 * pl.quad, in.q[f]);
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const v4f o = {value(in.o[j][0]), value(in.o[j][1]), value(in.o[j][2]), value(in.o[j][3])};
                mid_store4<BF, 1>(sh.O[16 * j + pl.l15], pl.rows, o);
                mid_store4<BF, 3>(sh.Os[16 * j + pl.l15], pl.rows, in.w.gam * in.w.rq * a.scale * o);
            }
        };
        // its parts P^T dO, to LDS, and Q^T dO, kept
        const auto parts = [&](const HelpBack<BF, KF, NT> &in) __attribute__((always_inline)) {
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                v4f o = v4f_zero();
#pragma unroll
                for (int f = 0; f < 2; ++f) {
                    In<BF> d;
                    __builtin_memcpy(&d, __builtin_assume_aligned(sh.O[16 * j + pl.l15] + (4 * f + pl.quad) * mid8<BF, 1>, 16), sizeof d);
                    o = mma(in.p[f], d, o);
                }
                sh.po[pl.wave][j][lane] = o;
            }
#pragma unroll
            for (int i = 0; i < Sl::MINE; ++i) {
                qo[i] = v4f_zero();
                if (sl.live(i))
#pragma unroll
                    for (int f = 0; f < 2; ++f)
                        qo[i] = mma(sh.q.down(32 * f, sl.row16(i)), mid_load<BF, 3>(sh.Os[sl.col(i)] + (4 * f + pl.quad) * S8), qo[i]);
            }
        };
        HelpBack<BF, KF, NT> in;
        if (pl.chunks) {
            in.load(a, pl, pl.chunks - 1);
            spread(in);
        }
        lds_barrier();
        if (pl.chunks) {
            parts(in);
            if (pl.chunks > 1)
                in.load(a, pl, pl.chunks - 2);
        }
        lds_barrier();
        for (int c = pl.chunks - 1; c >= 0; --c) {
            // the chain reads Q^T dO of chunk c behind its second barrier from here
#pragma unroll
            for (int i = 0; i < Sl::MINE; ++i)
                sh.qo[pl.wave][i][lane] = qo[i];
            if (c > 0)
                spread(in);
            lds_barrier();
            if (c > 0) {
                parts(in);
                if (c > 1)
                    in.load(a, pl, c - 2);
            }
            lds_barrier();
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
    // 32 columns a block; 16 where that leaves compute units idle
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
