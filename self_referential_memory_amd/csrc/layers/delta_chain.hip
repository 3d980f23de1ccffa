// delta_chain.hip -- the gated delta rule's states from chunk to chunk, with the
// outputs, and their gradients from the last chunk back (formulas in delta.h).
//
// The state's columns are independent: a block takes NV of them for one item and
// head, keeps them in registers in fp32 and walks the chunks. Its four waves hold
// 16 of a chunk's rows each for the products with q, k, X and P, whose operands
// they read straight from memory in the layout the matrix units want; the state,
// the errors and their scaled copies pass from wave to wave through LDS,
// transposed. Three barriers a chunk.
#include "delta_mma.h"

namespace {

using namespace srnl_i;

// A block's slab of the state: KD x NV in 16 x 16 tiles, a wave's tiles one
// after the other.
template <int KD, int NV> struct Slab {
    static constexpr int NT = NV / 16, TILES = KD / 16 * NT, MINE = (TILES + 3) / 4;
    __device__ __forceinline__ static bool live(int t) { return TILES >= 4 || t < TILES; }
    __device__ __forceinline__ static int first() { return (threadIdx.x >> 6) * MINE; }
    __device__ __forceinline__ static int row(int t) { return 16 * (t / NT) + 4 * ((threadIdx.x & 63) >> 4); }
    __device__ __forceinline__ static int col(int t) { return 16 * (t % NT) + (threadIdx.x & 15); }
};

template <bool BF, int KD, int NV> struct FwdShared {
    __attribute__((aligned(16))) Rows<BF, KD> k;
    __attribute__((aligned(16))) char S[NV][KD * 4 + 16];        // the state, transposed
    __attribute__((aligned(16))) char R[NV][272], U[NV][272], W[NV][272];
};

template <bool BF, int KD, int NV, bool RECORD>
__global__ __launch_bounds__(256) void delta_chain_kernel(DeltaArgs a)
{
    constexpr int KF = KD / 32, NT = NV / 16;
    using Sl = Slab<KD, NV>;
    __shared__ FwdShared<BF, KD, NV> sh;
    const int slabs = (a.Dv + NV - 1) / NV;
    const int bh = blockIdx.x / slabs, v0 = (blockIdx.x - bh * slabs) * NV;
    const int b = bh / a.H, h = bh - b * a.H, hk = h / (a.H / a.Hk);
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, quad = lane >> 4, l15 = lane & 15;
    const int n = delta_tokens(a, b), chunks = (n + DELTA_CHUNK - 1) / DELTA_CHUNK;
    const int row = 16 * wave + l15, rows = 16 * wave + 4 * quad;    // as an operand, in a result

    v4f S[Sl::MINE];
#pragma unroll
    for (int i = 0; i < Sl::MINE; ++i) {
        const int t = Sl::first() + i, r = Sl::row(t), cl = Sl::col(t);
        S[i] = v4f_zero();
        if (a.state && Sl::live(t) && v0 + cl < a.Dv)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (r + e < a.Dk)
                    S[i][e] = a.state[(static_cast<long long>(bh) * a.Dk + r + e) * a.Dv + v0 + cl];
        if (Sl::live(t))
            mid_store4<BF>(sh.S[cl], r, S[i]);
    }

    for (int c = 0; c < chunks; ++c) {
        const long long at = static_cast<long long>(bh) * a.N + c;
        const long long tok = static_cast<long long>(b) * a.T + DELTA_CHUNK * c;
        const int left = n - DELTA_CHUNK * c;
        const float *vec = a.vec + at * VEC_FLOATS;
        In<BF> kf[KF], qf[KF];
#pragma unroll
        for (int f = 0; f < KF; ++f) {
            const int k = 32 * f + 8 * quad;
            const bool live = row < left && k < a.Dk;
            kf[f] = in_load<BF>(a.k, (tok + row) * a.ks + static_cast<long long>(hk) * a.Dk + k, live);
            qf[f] = in_load<BF>(a.q, (tok + row) * a.qs + static_cast<long long>(hk) * a.Dk + k, live);
            sh.k.put(row, k, kf[f]);
        }
        Mid<BF> xf[2], pf[2];
#pragma unroll
        for (int f = 0; f < 2; ++f) {
            const long long o = at * DELTA_SQUARE + row * 256 + 4 * (32 * f + 8 * quad);
            xf[f] = mid_load<BF>(a.X + o);
            pf[f] = mid_load<BF>(a.P + o);
        }
        float v[NT][4];
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                v[j][e] = rows + e < left && v0 + 16 * j + l15 < a.Dv
                              ? value<BF>(a.v, (tok + rows + e) * a.vs + static_cast<long long>(h) * a.Dv + v0 +
                                                   16 * j + l15)
                              : 0.0f;
        const v4f gam = *reinterpret_cast<const v4f *>(vec + VEC_GAM + rows);
        const v4f end = *reinterpret_cast<const v4f *>(vec + VEC_END + rows);
        const v4f bet = *reinterpret_cast<const v4f *>(vec + VEC_BETA + rows);
        const v4f rk = *reinterpret_cast<const v4f *>(vec + VEC_RK + rows);
        const v4f rq = *reinterpret_cast<const v4f *>(vec + VEC_RQ + rows);
        const float last = vec[VEC_GAM + 63];
        if (RECORD)
#pragma unroll
            for (int i = 0; i < Sl::MINE; ++i) {
                const int t = Sl::first() + i, r = Sl::row(t), cl = v0 + Sl::col(t);
                // rows go in fours, Dk in eights
                if (Sl::live(t))
                    mid_store_rows<BF>(a.S0 + (at * a.Dk + r) * a.Dv * 4, a.Dv * 4LL, cl, S[i], r < a.Dk && cl < a.Dv);
            }
        lds_barrier();           // the state is in LDS

        v4f kS[NT], qS[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            kS[j] = qS[j] = v4f_zero();
#pragma unroll
            for (int f = 0; f < KF; ++f) {
                const Mid<BF> s = mid_load<BF>(sh.S[16 * j + l15] + 4 * (32 * f + 8 * quad));
                kS[j] = mma(kf[f], s, kS[j]);
                qS[j] = mma(qf[f], s, qS[j]);
            }
            v4f r;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                r[e] = v[j][e] - gam[e] * rk[e] * kS[j][e];
            mid_store4<BF>(sh.R[16 * j + l15], rows, r);
        }
        lds_barrier();

#pragma unroll
        for (int j = 0; j < NT; ++j) {
            v4f err = v4f_zero();
#pragma unroll
            for (int f = 0; f < 2; ++f)
                err = mma(xf[f], mid_load<BF>(sh.R[16 * j + l15] + 4 * (32 * f + 8 * quad)), err);
            if (RECORD) {
                const int cl = v0 + 16 * j + l15;
                mid_store_rows<BF>(a.E + (at * DELTA_CHUNK + rows) * a.Dv * 4, a.Dv * 4LL, cl, err, cl < a.Dv);
            }
            v4f u, w;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                u[e] = bet[e] * err[e];
                w[e] = end[e] * rk[e] * u[e];
            }
            mid_store4<BF>(sh.U[16 * j + l15], rows, u);
            mid_store4<BF>(sh.W[16 * j + l15], rows, w);
        }
        lds_barrier();

#pragma unroll
        for (int i = 0; i < Sl::MINE; ++i) {
            const int t = Sl::first() + i, r = Sl::row(t), cl = Sl::col(t);
            if (!Sl::live(t))
                continue;
            S[i] *= last;
#pragma unroll
            for (int f = 0; f < 2; ++f)
                S[i] = mma(sh.k.down(32 * f, r & ~15), mid_load<BF>(sh.W[cl] + 4 * (32 * f + 8 * quad)), S[i]);
            mid_store4<BF>(sh.S[cl], r, S[i]);
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            v4f o;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                o[e] = a.scale * gam[e] * rq[e] * qS[j][e];
#pragma unroll
            for (int f = 0; f < 2; ++f)
                o = mma(pf[f], mid_load<BF>(sh.U[16 * j + l15] + 4 * (32 * f + 8 * quad)), o);
            const int cl = v0 + 16 * j + l15;
            if (cl < a.Dv)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (DELTA_CHUNK * c + rows + e < a.T)
                        put_value<BF>(a.out, ((tok + rows + e) * a.H + h) * a.Dv + cl, rows + e < left ? o[e] : 0.0f);
        }
        lds_barrier();           // the chunk's k is free
    }
    // what lies past the last chunk
    for (long long i = threadIdx.x; i < (a.T - static_cast<long long>(DELTA_CHUNK) * chunks) * NV; i += 256) {
        const int cl = v0 + static_cast<int>(i % NV);
        const long long t = static_cast<long long>(b) * a.T + DELTA_CHUNK * chunks + i / NV;
        if (cl < a.Dv)
            put_value<BF>(a.out, (t * a.H + h) * a.Dv + cl, 0.0f);
    }
    if (a.state_out)
#pragma unroll
        for (int i = 0; i < Sl::MINE; ++i) {
            const int t = Sl::first() + i, r = Sl::row(t), cl = v0 + Sl::col(t);
            if (Sl::live(t) && cl < a.Dv)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (r + e < a.Dk)
                        a.state_out[(static_cast<long long>(bh) * a.Dk + r + e) * a.Dv + cl] = S[i][e];
        }
}

template <bool BF, int KD, int NV> struct BwdShared {
    __attribute__((aligned(16))) Rows<BF, KD> k, q;
    __attribute__((aligned(16))) char D[NV][KD * 4 + 16];        // the state's gradient, transposed
    __attribute__((aligned(16))) char O[NV][272], Os[NV][272], W[NV][272], V[NV][272];
};

template <bool BF, int KD, int NV> __global__ __launch_bounds__(256) void delta_chain_bwd_kernel(DeltaArgs a)
{
    constexpr int KF = KD / 32, NT = NV / 16;
    using Sl = Slab<KD, NV>;
    __shared__ BwdShared<BF, KD, NV> sh;
    const int slabs = (a.Dv + NV - 1) / NV;
    const int bh = blockIdx.x / slabs, v0 = (blockIdx.x - bh * slabs) * NV;
    const int b = bh / a.H, h = bh - b * a.H, hk = h / (a.H / a.Hk);
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, quad = lane >> 4, l15 = lane & 15;
    const int n = delta_tokens(a, b), chunks = (n + DELTA_CHUNK - 1) / DELTA_CHUNK;
    const int row = 16 * wave + l15, rows = 16 * wave + 4 * quad;

    v4f D[Sl::MINE];
#pragma unroll
    for (int i = 0; i < Sl::MINE; ++i) {
        const int t = Sl::first() + i, r = Sl::row(t), cl = Sl::col(t);
        D[i] = v4f_zero();
        if (a.dstate_out && Sl::live(t) && v0 + cl < a.Dv)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (r + e < a.Dk)
                    D[i][e] = a.dstate_out[(static_cast<long long>(bh) * a.Dk + r + e) * a.Dv + v0 + cl];
        if (Sl::live(t))
            mid_store4<BF>(sh.D[cl], r, D[i]);
    }

    for (int c = chunks - 1; c >= 0; --c) {
        const long long at = static_cast<long long>(bh) * a.N + c;
        const long long tok = static_cast<long long>(b) * a.T + DELTA_CHUNK * c;
        const int left = n - DELTA_CHUNK * c;
        const float *vec = a.vec + at * VEC_FLOATS;
        In<BF> kf[KF];
#pragma unroll
        for (int f = 0; f < KF; ++f) {
            const int k = 32 * f + 8 * quad;
            const bool live = row < left && k < a.Dk;
            kf[f] = in_load<BF>(a.k, (tok + row) * a.ks + static_cast<long long>(hk) * a.Dk + k, live);
            sh.k.put(row, k, kf[f]);
            sh.q.put(row, k, in_load<BF>(a.q, (tok + row) * a.qs + static_cast<long long>(hk) * a.Dk + k, live));
        }
        Mid<BF> xf[2], pf[2];                          // transposed
#pragma unroll
        for (int f = 0; f < 2; ++f) {
            const long long o = at * DELTA_SQUARE + row * 256 + 4 * (32 * f + 8 * quad);
            xf[f] = mid_load<BF>(a.X + o);
            pf[f] = mid_load<BF>(a.P + o);
        }
        const v4f gam = *reinterpret_cast<const v4f *>(vec + VEC_GAM + rows);
        const v4f end = *reinterpret_cast<const v4f *>(vec + VEC_END + rows);
        const v4f bet = *reinterpret_cast<const v4f *>(vec + VEC_BETA + rows);
        const v4f rk = *reinterpret_cast<const v4f *>(vec + VEC_RK + rows);
        const v4f rq = *reinterpret_cast<const v4f *>(vec + VEC_RQ + rows);
        const float last = vec[VEC_GAM + 63];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            v4f o, os;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                o[e] = rows + e < left && v0 + 16 * j + l15 < a.Dv
                           ? value<BF>(a.dout, ((tok + rows + e) * a.H + h) * a.Dv + v0 + 16 * j + l15)
                           : 0.0f;
                os[e] = a.scale * gam[e] * rq[e] * o[e];
            }
            mid_store4<BF>(sh.O[16 * j + l15], rows, o);
            mid_store4<BF>(sh.Os[16 * j + l15], rows, os);
        }
#pragma unroll
        for (int i = 0; i < Sl::MINE; ++i) {
            const int t = Sl::first() + i, r = Sl::row(t), cl = v0 + Sl::col(t);
            if (Sl::live(t))
                mid_store_rows<BF>(a.D1 + (at * a.Dk + r) * a.Dv * 4, a.Dv * 4LL, cl, D[i], r < a.Dk && cl < a.Dv);
        }
        lds_barrier();

#pragma unroll
        for (int j = 0; j < NT; ++j) {
            v4f kD = v4f_zero();
#pragma unroll
            for (int f = 0; f < KF; ++f)
                kD = mma(kf[f], mid_load<BF>(sh.D[16 * j + l15] + 4 * (32 * f + 8 * quad)), kD);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                kD[e] *= end[e] * rk[e];
#pragma unroll
            for (int f = 0; f < 2; ++f)
                kD = mma(pf[f], mid_load<BF>(sh.O[16 * j + l15] + 4 * (32 * f + 8 * quad)), kD);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                kD[e] *= bet[e];
            mid_store4<BF>(sh.W[16 * j + l15], rows, kD);
        }
        lds_barrier();

#pragma unroll
        for (int j = 0; j < NT; ++j) {
            v4f dv = v4f_zero();
#pragma unroll
            for (int f = 0; f < 2; ++f)
                dv = mma(xf[f], mid_load<BF>(sh.W[16 * j + l15] + 4 * (32 * f + 8 * quad)), dv);
            const int cl = v0 + 16 * j + l15;
            mid_store_rows<BF>(a.dV + (at * DELTA_CHUNK + rows) * a.Dv * 4, a.Dv * 4LL, cl, dv, cl < a.Dv);
            if (a.dv && cl < a.Dv)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (DELTA_CHUNK * c + rows + e < a.T)
                        put_value<BF>(a.dv, ((tok + rows + e) * a.H + h) * a.Dv + cl, rows + e < left ? dv[e] : 0.0f);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                dv[e] *= -gam[e] * rk[e];
            mid_store4<BF>(sh.V[16 * j + l15], rows, dv);
        }
        lds_barrier();

#pragma unroll
        for (int i = 0; i < Sl::MINE; ++i) {
            const int t = Sl::first() + i, r = Sl::row(t), cl = Sl::col(t);
            if (!Sl::live(t))
                continue;
            D[i] *= last;
#pragma unroll
            for (int f = 0; f < 2; ++f) {
                const In<BF> kd = sh.k.down(32 * f, r & ~15), qd = sh.q.down(32 * f, r & ~15);
                D[i] = mma(qd, mid_load<BF>(sh.Os[cl] + 4 * (32 * f + 8 * quad)), D[i]);
                D[i] = mma(kd, mid_load<BF>(sh.V[cl] + 4 * (32 * f + 8 * quad)), D[i]);
            }
            mid_store4<BF>(sh.D[cl], r, D[i]);
        }
        lds_barrier();
    }
    if (a.dv)
        for (long long i = threadIdx.x; i < (a.T - static_cast<long long>(DELTA_CHUNK) * chunks) * NV; i += 256) {
            const int cl = v0 + static_cast<int>(i % NV);
            const long long t = static_cast<long long>(b) * a.T + DELTA_CHUNK * chunks + i / NV;
            if (cl < a.Dv)
                put_value<BF>(a.dv, (t * a.H + h) * a.Dv + cl, 0.0f);
        }
    if (a.dstate)
#pragma unroll
        for (int i = 0; i < Sl::MINE; ++i) {
            const int t = Sl::first() + i, r = Sl::row(t), cl = v0 + Sl::col(t);
            if (Sl::live(t) && cl < a.Dv)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (r + e < a.Dk)
                        a.dstate[(static_cast<long long>(bh) * a.Dk + r + e) * a.Dv + cl] = D[i][e];
        }
}

}  // namespace

namespace srnl_i {

srnl_status launch_delta_chain(const DeltaArgs &a, hipStream_t st)
{
#define SRNL_DELTA_CHAIN(BF, KD)                                                                               \
    do {                                                                                                       \
        constexpr int NV = 32;                                                                                 \
        const dim3 grid(static_cast<unsigned>(static_cast<long long>(a.B) * a.H * ((a.Dv + NV - 1) / NV)));    \
        if (a.E)                                                                                               \
            hipLaunchKernelGGL((delta_chain_kernel<BF, KD, NV, true>), grid, dim3(256), 0, st, a);             \
        else                                                                                                   \
            hipLaunchKernelGGL((delta_chain_kernel<BF, KD, NV, false>), grid, dim3(256), 0, st, a);            \
    } while (0)
    SRNL_DELTA_DISPATCH(a, SRNL_DELTA_CHAIN);
    return launched("delta_chain_kernel");
}

srnl_status launch_delta_chain_bwd(const DeltaArgs &a, hipStream_t st)
{
#define SRNL_DELTA_CHAIN_BWD(BF, KD)                                                                           \
    do {                                                                                                       \
        constexpr int NV = 32;                                                                                 \
        const dim3 grid(static_cast<unsigned>(static_cast<long long>(a.B) * a.H * ((a.Dv + NV - 1) / NV)));    \
        hipLaunchKernelGGL((delta_chain_bwd_kernel<BF, KD, NV>), grid, dim3(256), 0, st, a);                   \
    } while (0)
    SRNL_DELTA_DISPATCH(a, SRNL_DELTA_CHAIN_BWD);
    return launched("delta_chain_bwd_kernel");
}

}  // namespace srnl_i
