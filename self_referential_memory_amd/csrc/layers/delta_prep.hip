// delta_prep.hip -- per chunk and head of the gated delta rule: the row factors,
// X = (I + M b)^-1 and P (see delta.h), every chunk at once.
//
// A block takes one chunk, a wave 16 of its rows. X is inverted in fp32: the four
// 16 x 16 blocks on the diagonal by substitution, a column a lane; then the blocks
// below, one diagonal after the other, X_ij = -X_ii sum L_ik X_kj, with fp32
// matrix products whose result is the next one's operand without a move (its rows
// 4 quad + s serve as the reduction elements of step s).
//
// 2048 chunks of 128 take 32 to 34 us: 67 MB of q and k in, 81 MB out, 4.5 TB/s. Four
// blocks a CU; one chunk alone takes 8 us, a chain of loads, sums, substitution and
// blocks, so that 6272 chunks of 32 (61 us) are bound by their latency as much.
#include "delta_mma.h"

namespace {

using namespace srnl_i;

template <bool BF, int KD> struct PrepShared {
    union {
        Rows<BF, KD> k;                // until the products are formed
        struct {
            __attribute__((aligned(16))) float L[64][68], X[64][68];
        } m;
    };
    float ghi[64], glo[64], beta[64], rk[64], rq[64], gam[64], end[64];
};

template <bool BF, int KD, bool TRANSPOSED>
__global__ __launch_bounds__(256) void delta_prep_kernel(DeltaArgs a, bool past)
{
    constexpr int KF = KD / 32;
    __shared__ PrepShared<BF, KD> sh;
    auto &L = sh.m.L, &X = sh.m.X;
    const int c = blockIdx.x % a.N, bh = blockIdx.x / a.N;
    const int b = bh / a.H, h = bh - b * a.H, hk = h / (a.H / a.Hk);
    const int n = delta_tokens(a, b), tok0 = DELTA_CHUNK * c;
    if (tok0 >= n)
        return;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63, quad = lane >> 4, l15 = lane & 15;
    const long long tok = static_cast<long long>(b) * a.T + tok0;
    const int row = 16 * wave + l15;

    In<BF> kf[KF], qf[KF];
    {
        const Buf bk(a.k, (tok * a.ks + static_cast<long long>(hk) * a.Dk) * (BF ? 2 : 4));
        const Buf bq(a.q, (tok * a.qs + static_cast<long long>(hk) * a.Dk) * (BF ? 2 : 4));
#pragma unroll
        for (int f = 0; f < KF; ++f) {
            const int k = 32 * f + 8 * quad;
            const bool live = both(tok0 + row < n, k < a.Dk);
            kf[f] = in_load<BF>(bk, row * static_cast<int>(a.ks) + k, live);
            qf[f] = in_load<BF>(bq, row * static_cast<int>(a.qs) + k, live);
        }
    }
    if (wave == 0) {
        // sums in 64 bits: what matters later is their differences. Below -1000 a
        // factor is 0 either way; -infinity would make NaN of a difference.
        const bool live = tok0 + lane < n;
        const long long at = (tok + lane) * a.H + h;
        const float g = live ? a.g[at] : 0.0f;
        double G = g < -1000.0f ? -1000.0 : static_cast<double>(g);
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const double o = __shfl_up(G, off);
            if (lane >= off)
                G += o;
        }
        const float hi = static_cast<float>(G), lo = static_cast<float>(G - hi);
        const double left = __shfl(G, 63) - G;
        const float lhi = static_cast<float>(left);
        sh.ghi[lane] = hi;
        sh.glo[lane] = lo;
        sh.beta[lane] = live ? a.beta[at] : 0.0f;
        sh.gam[lane] = expf(hi) * (1.0f + lo);
        sh.end[lane] = expf(lhi) * (1.0f + static_cast<float>(left - lhi));
    }
#pragma unroll
    for (int f = 0; f < KF; ++f)
        sh.k.put(row, 32 * f + 8 * quad, kf[f]);
    __syncthreads();

    // k_i.k_j and q_i.k_j of this wave's rows, and q_i.q_i: the norms are diagonals
    v4f m[4], p[4], qq = v4f_zero();
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        m[j] = p[j] = v4f_zero();
        if (j <= wave)
#pragma unroll
            for (int f = 0; f < KF; ++f) {
                const In<BF> o = sh.k.across(16 * j + l15, 32 * f + 8 * quad);
                m[j] = mma(kf[f], o, m[j]);
                p[j] = mma(qf[f], o, p[j]);
            }
    }
    if (a.eps > 0.0f) {
#pragma unroll
        for (int f = 0; f < KF; ++f)
            qq = mma(qf[f], qf[f], qq);
    }
    if (quad == l15 >> 2) {
        // a row past the end has no direction: its factor is 0, not 1 / sqrt(eps)
        const v4f kk = wave == 0 ? m[0] : wave == 1 ? m[1] : wave == 2 ? m[2] : m[3];
        const int e = l15 & 3;
        const float k2 = e == 0 ? kk[0] : e == 1 ? kk[1] : e == 2 ? kk[2] : kk[3];
        const float q2 = e == 0 ? qq[0] : e == 1 ? qq[1] : e == 2 ? qq[2] : qq[3];
        const bool live = tok0 + row < n;
        sh.rk[row] = !live ? 0.0f : a.eps > 0.0f ? 1.0f / sqrtf(k2 + a.eps) : 1.0f;
        sh.rq[row] = !live ? 0.0f : a.eps > 0.0f ? 1.0f / sqrtf(q2 + a.eps) : 1.0f;
    }
    __syncthreads();
    if (wave == 0) {
        float *vec = a.vec + static_cast<long long>(blockIdx.x) * VEC_FLOATS;
        const float ga = sh.gam[lane], en = sh.end[lane], be = sh.beta[lane], rk = sh.rk[lane], rq = sh.rq[lane];
        vec[VEC_GAM + lane] = ga;
        vec[VEC_END + lane] = en;
        vec[VEC_BETA + lane] = be;
        vec[VEC_RK + lane] = rk;
        vec[VEC_RQ + lane] = rq;
        vec[VEC_GHI + lane] = sh.ghi[lane];
        vec[VEC_GLO + lane] = sh.glo[lane];
        vec[VEC_READK + lane] = ga * rk;
        vec[VEC_WRITE + lane] = en * be * rk;
        vec[VEC_READQ + lane] = a.scale * ga * rq;
    }
    {
        const int i0 = 16 * wave + 4 * quad;
        const v4f ihi = *reinterpret_cast<const v4f *>(&sh.ghi[i0]), ilo = *reinterpret_cast<const v4f *>(&sh.glo[i0]);
        const v4f ri = *reinterpret_cast<const v4f *>(&sh.rk[i0]);
        const v4f qi = *reinterpret_cast<const v4f *>(&sh.rq[i0]) * a.scale;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int col = 16 * j + l15;
            if (j > wave) {
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    X[i0 + r][col] = 0.0f;
                continue;
            }
            const float jhi = sh.ghi[col], jlo = sh.glo[col], rj = sh.rk[col], bj = sh.beta[col];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float d = decay(ihi[r], ilo[r], jhi, jlo) * rj;
                const float x = m[j][r] * ri[r] * (d * bj), y = p[j][r] * qi[r] * d;
                L[i0 + r][col] = j < wave || col < i0 + r ? x : 0.0f;
                p[j][r] = j < wave || col <= i0 + r ? y : 0.0f;
            }
        }
    }
    __syncthreads();

    // blocks on the diagonal
    {
        float x[16];
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            float s = r == l15 ? 1.0f : 0.0f;
#pragma unroll
            for (int k = 0; k < r; ++k)
                s = fmaf(-L[16 * wave + r][16 * wave + k], x[k], s);
            x[r] = s;
        }
        if (quad == 0)
#pragma unroll
            for (int r = 0; r < 16; ++r)
                X[16 * wave + r][16 * wave + l15] = x[r];
    }
#pragma unroll
    for (int d = 1; d < 4; ++d) {
        __syncthreads();
        if (wave < d)
            continue;
        const int j = wave - d;
        v4f y = v4f_zero();
        for (int k = j; k < wave; ++k) {
            const v4f l = *reinterpret_cast<const v4f *>(&L[16 * wave + l15][16 * k + 4 * quad]);
#pragma unroll
            for (int s = 0; s < 4; ++s)
                y = __builtin_amdgcn_mfma_f32_16x16x4f32(l[s], X[16 * k + 4 * quad + s][16 * j + l15], y, 0, 0, 0);
        }
        const v4f xi = *reinterpret_cast<const v4f *>(&X[16 * wave + l15][16 * wave + 4 * quad]);
        v4f z = v4f_zero();
#pragma unroll
        for (int s = 0; s < 4; ++s)
            z = __builtin_amdgcn_mfma_f32_16x16x4f32(xi[s], y[s], z, 0, 0, 0);
#pragma unroll
        for (int r = 0; r < 4; ++r)
            X[16 * wave + 4 * quad + r][16 * j + l15] = -z[r];
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            L[16 * wave + 4 * quad + r][16 * j + l15] = p[j][r];
    __syncthreads();
    // The half of a row that is zero is not written: nobody reads it.
    const long long square = static_cast<long long>(blockIdx.x) * DELTA_SQUARE;
    const Buf xo(a.X, square), po(a.P, square);
#pragma unroll
    for (int f = 0; f < 2; ++f) {
        if (f == (TRANSPOSED ? 0 : 1) && (TRANSPOSED ? wave >= 2 : wave < 2))
            continue;
        const int k = 32 * f + 8 * quad;
        float x[8], y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            x[e] = TRANSPOSED ? X[k + e][row] : X[row][k + e];
            y[e] = TRANSPOSED ? L[k + e][row] : L[row][k + e];
        }
        frag_store<BF, 3>(xo, 2 * wave + f, x, past);
        frag_store<BF, 3>(po, 2 * wave + f, y, past);
    }
}

}  // namespace

namespace srnl_i {

srnl_status launch_delta_prep(const DeltaArgs &a, bool transposed, hipStream_t st)
{
    const long long chunks = static_cast<long long>(a.B) * a.H * a.N;
    const dim3 grid(static_cast<unsigned>(chunks));
    // X and P stay in the caches for the chain only while they fit. Written past them,
    // this kernel and the chain take 197 us for 2048 chunks of a record with k and v of
    // 128 (180 not so), 292 for 3584 without (310) and 135 for 6272 with 32 (165).
    const bool past = chunks * 2 * DELTA_SQUARE > 128ll << 20;
#define SRNL_DELTA_PREP(BF, KD)                                                                    \
    if (transposed)                                                                                \
        hipLaunchKernelGGL((delta_prep_kernel<BF, KD, true>), grid, dim3(256), 0, st, a, past);    \
    else                                                                                           \
        hipLaunchKernelGGL((delta_prep_kernel<BF, KD, false>), grid, dim3(256), 0, st, a, past)
    SRNL_DELTA_DISPATCH(a, SRNL_DELTA_PREP);
    return launched("delta_prep_kernel");
}

}  // namespace srnl_i
