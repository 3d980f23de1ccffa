// delta_grads.hip -- the gradients of q, k, g and beta of the gated delta rule,
// every chunk at once, from the states (S0), the errors (E), the gradients of v
// (dV) and of the states after each chunk (D1). With the hats and factors of
// delta.h and for j < i unless said otherwise:
//   A_ij = dO_i.E_j (j <= i),  Y_ij = dV_i.E_j,  F_ij = P_ij A_ij - M_ij Y_ij
//   dq^_i = scale e^G_i S0 dO_i + sum_{j <= i} scale e^(G_i - G_j) beta_j A_ij k^_j
//   dk^_j = beta_j w_j + sum_{i >= j} scale e^(G_i - G_j) beta_j A_ij q^_i
//           - e^G_j S0 dV_j - sum_i of the two halves of e^(..) beta Y with k^
//   w_j = e^(G_63 - G_j) D1 E_j
//   dbeta_j = k^_j.w_j + sum_{i >= j} F_ij
//   dg_t = sum_{i >= t} (r_i - c_i + s_i) + sum_{j < t} beta_j k^_j.w_j + e^G_63 <S0, D1>
//   with r and c the row and column sums of F_ij beta_j and s_i = q^_i.(first term of
//   dq^_i) - k^_i.(e^G_i S0 dV_i).
// dg sums what depends on g_t alone: taken as q.dq - k.dk summed over later tokens,
// large terms would cancel. dk = (dk^ - k^ (k^.dk^)) / |k| at the end, likewise q.
//
// A block of eight waves takes a chunk of one q/k head and the v heads that share
// it, one after the other. It walks the columns of v, 32 at a time: dO, E and dV go
// to LDS, the next 32 columns on their way meanwhile; of the 64 x 64 parts a wave
// forms 16 rows by 32 columns, of the products with the states 16 of the head's
// columns (narrow heads: fewer rows), so that the states, the largest operands, are
// read once, straight into registers. A, Y and the row factors then make the
// matrices that multiply q and k, in the LDS that dO, E and dV leave.
#include "delta_mma.h"

namespace {

using namespace srnl_i;

template <bool BF, int KD> struct GradShared {
    __attribute__((aligned(16))) Rows<BF, KD> k, q;
    union {
        struct {
            __attribute__((aligned(16))) char O[64][mid_row<BF, 1>(32)], E[64][mid_row<BF, 3>(32)], V[64][mid_row<BF, 3>(32)];
        } in[2];
        struct {
            __attribute__((aligned(16))) char A[64][mid_row<BF, 2>(64)], At[64][mid_row<BF, 2>(64)], Z[64][mid_row<BF, 2>(64)];
        } out;
    };
    float gam[64], end[64], beta[64], rk[64], rq[64], ghi[64], glo[64];
    float colF[4][64], rowF[2][64], diag[64], dot[2][8][64], sd[8];
};

template <bool BF, int KD> struct Columns {
    static constexpr int CW = KD / 16, RW = 8 / CW;      // waves along columns, rows
    static constexpr int RT = 4 / RW;                    // a wave's tiles: rows, in one column
};

__device__ __forceinline__ float sum16(float v)
{
#pragma unroll
    for (int off = 8; off > 0; off >>= 1)
        v += __shfl_xor(v, off);
    return v;
}

template <bool BF, int KD> __global__ __launch_bounds__(512) void delta_grads_kernel(DeltaArgs a)
{
    constexpr int KF = KD / 32;
    using Sh = GradShared<BF, KD>;
    using Co = Columns<BF, KD>;
    constexpr int RT = Co::RT;
    __shared__ Sh sh;
    const int c = blockIdx.x % a.N, bk = blockIdx.x / a.N;
    const int b = bk / a.Hk, hk = bk - b * a.Hk, per = a.H / a.Hk;
    const int n = delta_tokens(a, b), left = n - DELTA_CHUNK * c;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, quad = lane >> 4, l15 = lane & 15;
    const int band = wave & 3, half = wave >> 2;                        // of the 64 x 64 parts
    const int row = 16 * band + l15, rows = 16 * band + 4 * quad;
    const long long tok = static_cast<long long>(b) * a.T + DELTA_CHUNK * c;
    const int rt0 = wave / Co::CW * RT, col0 = 16 * (wave % Co::CW), mycol = col0 + l15;
    const int inside = a.T - DELTA_CHUNK * c < DELTA_CHUNK ? a.T - DELTA_CHUNK * c : DELTA_CHUNK;

    if (left <= 0) {                   // past the end: zeros
        for (int i = threadIdx.x; i < inside * a.Dk; i += 512) {
            const long long o = ((tok + i / a.Dk) * a.Hk + hk) * a.Dk + i % a.Dk;
            if (a.dq)
                put_at<BF>(a.dq, o, 0.0f);
            if (a.dk)
                put_at<BF>(a.dk, o, 0.0f);
        }
        for (int i = threadIdx.x; i < inside * per; i += 512) {
            const long long o = (tok + i / per) * a.H + hk * per + i % per;
            if (a.dg)
                a.dg[o] = 0.0f;
            if (a.dbeta)
                a.dbeta[o] = 0.0f;
        }
        return;
    }

    const long long head = static_cast<long long>(hk) * a.Dk;
    const Buf rowsK(a.k, (tok * a.ks + head) * (BF ? 2 : 4)), rowsQ(a.q, (tok * a.qs + head) * (BF ? 2 : 4));
#pragma unroll
    for (int x = 0; x < KD / 64 + (KD < 64); ++x) {
        // a thread's pieces of 8: every row, KD / 8 pieces
        const int i = threadIdx.x + 512 * x, r = i / (KD / 8), k = i % (KD / 8) * 8;
        if (r < 64) {
            sh.k.put(r, k, in_load<BF>(rowsK, r * static_cast<int>(a.ks) + k, r < left && k < a.Dk));
            sh.q.put(r, k, in_load<BF>(rowsQ, r * static_cast<int>(a.qs) + k, r < left && k < a.Dk));
        }
    }

    v4f dq[RT], dk[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i)
        dq[i] = dk[i] = v4f_zero();

    for (int g = 0; g < per; ++g) {
        const int h = hk * per + g;
        const long long at = (static_cast<long long>(b) * a.H + h) * a.N + c;
        const Buf bS(a.S0, at * a.Dk * a.Dv * 4), bD(a.D1, at * a.Dk * a.Dv * 4);
        const float *vec = a.vec + at * VEC_FLOATS;
        // this thread's piece of 8 of E or dV, and of dO
        const int pr = (threadIdx.x & 255) >> 2, pc = (threadIdx.x & 3) * 8;
        const bool ofE = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) < 4;
        const Buf bEV(ofE ? a.E : a.dV, at * DELTA_CHUNK * a.Dv * 4);
        const Buf bO(a.dout, (tok * a.H + h) * a.Dv * (BF ? 2 : 4));
        struct { float ev[8], s[8], d[8]; In<BF> o; } next;
        const auto fetch = [&](int v) __attribute__((always_inline)) {
            load8(bEV, pr * a.Dv + pc + v, v + pc < a.Dv, next.ev);
            next.o = in_load<BF>(bO, pr * a.H * a.Dv + pc + v, ofE && v + pc < a.Dv && pr < left);
            load8(bS, mycol * a.Dv + 8 * quad + v, mycol < a.Dk && v + 8 * quad < a.Dv, next.s);
            load8(bD, mycol * a.Dv + 8 * quad + v, mycol < a.Dk && v + 8 * quad < a.Dv, next.d);
        };
        const auto spread = [&](int buf) __attribute__((always_inline)) {
            mid_store8<BF, 3>((ofE ? sh.in[buf].E[pr] : sh.in[buf].V[pr]) + pc / 8 * mid8<BF, 3>, next.ev);
            if (ofE)
                __builtin_memcpy(__builtin_assume_aligned(sh.in[buf].O[pr] + pc / 8 * mid8<BF, 1>, 16), &next.o, sizeof next.o);
        };
        fetch(0);
        __syncthreads();               // the head before is done with the shared arrays
        if (threadIdx.x < 64) {
            sh.gam[lane] = vec[VEC_GAM + lane];
            sh.end[lane] = vec[VEC_END + lane];
            sh.beta[lane] = vec[VEC_BETA + lane];
            sh.rk[lane] = vec[VEC_RK + lane];
            sh.rq[lane] = vec[VEC_RQ + lane];
            sh.ghi[lane] = vec[VEC_GHI + lane];
            sh.glo[lane] = vec[VEC_GLO + lane];
        }
        spread(0);

        v4f A[2], Y[2], oS[RT], vS[RT], eD[RT];
#pragma unroll
        for (int x = 0; x < 2; ++x)
            A[x] = Y[x] = v4f_zero();
#pragma unroll
        for (int ri = 0; ri < RT; ++ri)
            oS[ri] = vS[ri] = eD[ri] = v4f_zero();
        float sd = 0.0f;
        int buf = 0;
#pragma unroll 1
        for (int v = 0; v < a.Dv; v += 32, buf ^= 1) {
            const Mid<BF, 3> s = mid_split<BF, 3>(next.s), d = mid_split<BF, 3>(next.d);
            if (rt0 == 0)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    sd = fmaf(next.s[e], next.d[e], sd);
            if (v + 32 < a.Dv)
                fetch(v + 32);
            lds_barrier();
            const auto rowO = [&](int r) __attribute__((always_inline)) {
                In<BF> f;
                __builtin_memcpy(&f, __builtin_assume_aligned(sh.in[buf].O[r] + quad * mid8<BF, 1>, 16), sizeof f);
                return f;
            };
            {
                const In<BF> o = rowO(row);
                const Mid<BF, 3> y = mid_load<BF, 3>(sh.in[buf].V[row] + quad * mid8<BF, 3>);
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int j = 2 * half + x;
                    if (j > band)
                        continue;
                    const Mid<BF, 3> e = mid_load<BF, 3>(sh.in[buf].E[16 * j + l15] + quad * mid8<BF, 3>);
                    A[x] = mma(o, e, A[x]);
                    Y[x] = mma(y, e, Y[x]);
                }
            }
#pragma unroll
            for (int ri = 0; ri < RT; ++ri) {
                const int r = 16 * (rt0 + ri) + l15;
                oS[ri] = mma(rowO(r), s, oS[ri]);
                vS[ri] = mma(mid_load<BF, 3>(sh.in[buf].V[r] + quad * mid8<BF, 3>), s, vS[ri]);
                eD[ri] = mma(mid_load<BF, 3>(sh.in[buf].E[r] + quad * mid8<BF, 3>), d, eD[ri]);
            }
            if (v + 32 < a.Dv)
                spread(buf ^ 1);
        }
        __syncthreads();               // dO, E and dV are read

        // ---- 64 x 64 parts: this wave's rows i against its columns j
        float rowF[4] = {0, 0, 0, 0};
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const int j = 2 * half + p, col = 16 * j + l15;
            v4f wa = v4f_zero(), wat = v4f_zero(), zl = v4f_zero(), zu = v4f_zero();
            float colF = 0.0f;
            if (j <= band) {
                v4f kk = v4f_zero(), qk = v4f_zero();
#pragma unroll
                for (int f = 0; f < KF; ++f) {
                    const int k = 32 * f + 8 * quad;
                    const In<BF> o = sh.k.across(col, k);
                    kk = mma(sh.k.across(row, k), o, kk);
                    qk = mma(sh.q.across(row, k), o, qk);
                }
                const float bj = sh.beta[col], rj = sh.rk[col];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int i = rows + e;
                    const float d = decay(sh.ghi[i], sh.glo[i], sh.ghi[col], sh.glo[col]);
                    const float ri = sh.rk[i], qi = sh.rq[i];
                    const bool on = col <= i, below = col < i;
                    const float x = on ? a.scale * d * A[p][e] : 0.0f;          // dP before beta
                    const float y = below ? d * Y[p][e] : 0.0f;
                    const float F = on ? x * qi * rj * qk[e] - (below ? y * ri * rj * kk[e] : 0.0f) : 0.0f;
                    wa[e] = x * bj * rj;
                    wat[e] = x * bj * qi;
                    zl[e] = -y * bj * rj;
                    zu[e] = -y * bj * ri;
                    colF += F;
                    // the diagonal is no decay's
                    rowF[e] += below ? bj * F : 0.0f;
                    if (on && !below)
                        sh.diag[i] = F;
                }
            }
            mid_store_rows<BF, 2>(sh.out.A[rows], sizeof sh.out.A[0], col, wa);
            mid_store4<BF, 2>(sh.out.At[col], rows, wat);
            // Z's two triangles: rows i > j from here, its mirror from the same values
            if (j < band) {
                mid_store_rows<BF, 2>(sh.out.Z[rows], sizeof sh.out.Z[0], col, zl);
                mid_store4<BF, 2>(sh.out.Z[col], rows, zu);
            }
            colF += __shfl_xor(colF, 16);
            colF += __shfl_xor(colF, 32);
            if (quad == 0)
                sh.colF[band][col] = colF;
            if (j == band) {
                // the diagonal tile is both: its upper half comes from the lanes across
                v4f z;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    // element (4 quad + e, l15) above the diagonal is zu of (l15, 4 quad + e)
                    const int src = (l15 >> 2) * 16 + 4 * quad + e;
                    const float u0 = __shfl(zu[0], src), u1 = __shfl(zu[1], src), u2 = __shfl(zu[2], src),
                                u3 = __shfl(zu[3], src);
                    const float up = (l15 & 2) ? ((l15 & 1) ? u3 : u2) : ((l15 & 1) ? u1 : u0);
                    z[e] = l15 < 4 * quad + e ? zl[e] : l15 > 4 * quad + e ? up : 0.0f;
                }
                mid_store_rows<BF, 2>(sh.out.Z[rows], sizeof sh.out.Z[0], col, z);
            }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float s = sum16(rowF[e]);
            if (l15 == 0)
                sh.rowF[half][rows + e] = s;
        }
        __syncthreads();
        // ---- products with the head's width: this wave's columns
#pragma unroll
        for (int f = 0; f < 2; ++f) {
            const int o = (4 * f + quad) * mid8<BF, 2>;
            const In<BF> kd = sh.k.down(32 * f, col0), qd = sh.q.down(32 * f, col0);
#pragma unroll
            for (int ri = 0; ri < RT; ++ri) {
                const int r = 16 * (rt0 + ri) + l15;
                dq[ri] = mma(mid_load<BF, 2>(sh.out.A[r] + o), kd, dq[ri]);
                dk[ri] = mma(mid_load<BF, 2>(sh.out.At[r] + o), qd, dk[ri]);
                dk[ri] = mma(mid_load<BF, 2>(sh.out.Z[r] + o), kd, dk[ri]);
            }
        }
#pragma unroll
        for (int ri = 0; ri < RT; ++ri)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = 16 * (rt0 + ri) + 4 * quad + e;
                const float x = a.scale * sh.gam[i] * oS[ri][e];
                const float y = -sh.gam[i] * vS[ri][e];
                const float w = sh.end[i] * eD[ri][e];
                const float kh = sh.rk[i] * sh.k.at(i, mycol), qh = sh.rq[i] * sh.q.at(i, mycol);
                const float s = sum16(fmaf(qh, x, kh * y)), t = sum16(kh * w);
                if (l15 == 0) {
                    sh.dot[0][wave % Co::CW][i] = s;
                    sh.dot[1][wave % Co::CW][i] = t;
                }
                dq[ri][e] += x;
                dk[ri][e] += fmaf(sh.beta[i], w, y);
            }
#pragma unroll
        for (int off = 32; off > 0; off >>= 1)
            sd += __shfl_xor(sd, off);
        if (lane == 0)
            sh.sd[wave] = sd;
        __syncthreads();
        if (wave == 0) {
            float s = 0.0f, w = 0.0f, col = 0.0f;
#pragma unroll
            for (int x = 0; x < Co::CW; ++x) {
                s += sh.dot[0][x][lane];
                w += sh.dot[1][x][lane];
            }
#pragma unroll
            for (int x = 0; x < 4; ++x)
                col += x >= lane / 16 ? sh.colF[x][lane] : 0.0f;
            const float beta = sh.beta[lane];
            const float dbeta = w + col;
            w *= beta;
            // tokens after this one and itself; tokens before this one
            float after = (sh.rowF[0][lane] + sh.rowF[1][lane]) - beta * (col - sh.diag[lane]) + s, before = w;
#pragma unroll
            for (int off = 1; off < 64; off <<= 1) {
                const float x = __shfl_down(after, off), y = __shfl_up(before, off);
                after += lane + off < 64 ? x : 0.0f;
                before += lane >= off ? y : 0.0f;
            }
            float inner = 0.0f;
#pragma unroll
            for (int x = 0; x < 8; ++x)
                inner += sh.sd[x];
            const float dg = after + (before - w) + sh.gam[63] * inner;
            if (lane < inside) {
                const long long o = (tok + lane) * a.H + h;
                if (a.dg)
                    a.dg[o] = lane < left ? dg : 0.0f;
                if (a.dbeta)
                    a.dbeta[o] = lane < left ? dbeta : 0.0f;
            }
        }
    }

    // ---- through the normalisation, and out
    if (a.eps > 0.0f) {
        __syncthreads();               // the last head's sums are read
#pragma unroll
        for (int ri = 0; ri < RT; ++ri)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = 16 * (rt0 + ri) + 4 * quad + e;
                const float x = sum16(sh.q.at(i, mycol) * dq[ri][e]);
                const float y = sum16(sh.k.at(i, mycol) * dk[ri][e]);
                if (l15 == 0) {
                    sh.dot[0][wave % Co::CW][i] = x;
                    sh.dot[1][wave % Co::CW][i] = y;
                }
            }
        __syncthreads();
    }
#pragma unroll
    for (int ri = 0; ri < RT; ++ri)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = 16 * (rt0 + ri) + 4 * quad + e;
            float x = dq[ri][e], y = dk[ri][e];
            if (a.eps > 0.0f) {
                const float rq = sh.rq[i], rk = sh.rk[i];
                float xs = 0.0f, ys = 0.0f;
#pragma unroll
                for (int w = 0; w < Co::CW; ++w) {
                    xs += sh.dot[0][w][i];
                    ys += sh.dot[1][w][i];
                }
                x = rq * (x - rq * sh.q.at(i, mycol) * (rq * xs));
                y = rk * (y - rk * sh.k.at(i, mycol) * (rk * ys));
            }
            if (i >= inside || mycol >= a.Dk)
                continue;
            const long long o = ((tok + i) * a.Hk + hk) * a.Dk + mycol;
            if (a.dq)
                put_at<BF>(a.dq, o, i < left ? x : 0.0f);
            if (a.dk)
                put_at<BF>(a.dk, o, i < left ? y : 0.0f);
        }
}

}  // namespace

namespace srnl_i {

srnl_status launch_delta_grads(const DeltaArgs &a, hipStream_t st)
{
    const dim3 grid(static_cast<unsigned>(static_cast<long long>(a.B) * a.Hk * a.N));
#define SRNL_DELTA_GRADS(BF, KD) hipLaunchKernelGGL((delta_grads_kernel<BF, KD>), grid, dim3(512), 0, st, a)
    SRNL_DELTA_DISPATCH(a, SRNL_DELTA_GRADS);
    return launched("delta_grads_kernel");
}

}  // namespace srnl_i
