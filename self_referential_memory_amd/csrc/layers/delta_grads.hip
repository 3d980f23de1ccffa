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
// A block of eight waves takes a chunk of one head. It walks the columns of v, 32 at
// a time: dO, E and dV go to LDS, the next 32 columns on their way meanwhile; of the
// 64 x 64 parts a wave forms 16 rows by 32 columns, of the products with the states
// 16 of the head's columns (narrow heads: fewer rows), so that the states, the
// largest operands, are read once, straight into registers. A, Y and the row factors
// then make the matrices that multiply q and k, in the LDS that dO, E and dV leave.
// Heads that share q and k write their parts in fp32, and a second kernel adds them
// in order.
//
// 2048 chunks of 128 x 128 take 202 us, eight rounds of one block a CU: of a block's 25
// us half goes to the walk, where a step's products (2500 cycles) and LDS reads (2400)
// only partly overlap with two waves a SIMD, 2 us each to the first loads, the 64 x 64
// parts, the states' terms and the norms, 1 us to the last products and the stores.
#include "delta_mma.h"

namespace {

using namespace srnl_i;

template <bool BF, int KD> struct GradShared {
    Rows<BF, KD> k, q;
    union {
        struct {
            Split<BF, 1, 64, 32> O;
            Split<BF, 3, 64, 32> E, V;
        } in[2];
        struct {
            Split<BF, 3, 64, 64> A, At, Z;
        } out;
    };
    // a chunk's row factors, as they lie in memory from VEC_BETA on
    __attribute__((aligned(16))) float vec[VEC_FLOATS - VEC_BETA];
    __attribute__((aligned(16))) float norm[2][64];
    float colF[4][64], diag[64], sd[8];
    __attribute__((aligned(16))) float rowF[2][64], dot[2][8][64];
    __device__ __forceinline__ float at(int which, int r) const { return vec[which - VEC_BETA + r]; }
    __device__ __forceinline__ v4f four(int which, int r) const
    {
        return *reinterpret_cast<const v4f *>(&vec[which - VEC_BETA + r]);
    }
};

template <bool BF, int KD> __global__ __launch_bounds__(512) void delta_grads_kernel(DeltaArgs a)
{
    constexpr int KF = KD / 32;
    constexpr int CW = KD / 16, RW = 8 / CW;             // waves along columns, rows
    constexpr int RT = 4 / RW;                           // a wave's tiles: rows, in one column
    __shared__ GradShared<BF, KD> sh;
    const int c = blockIdx.x % a.N, bh = blockIdx.x / a.N;
    const int b = bh / a.H, h = bh - b * a.H, per = a.H / a.Hk, hk = h / per;
    const int n = delta_tokens(a, b), left = n - DELTA_CHUNK * c;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63, quad = lane >> 4, l15 = lane & 15;
    const int band = wave & 3, half = wave >> 2;                        // of the 64 x 64 parts
    const int row = 16 * band + l15, rows = 16 * band + 4 * quad;
    const int rt0 = wave / CW * RT, col0 = 16 * (wave % CW), mycol = col0 + l15;
    const long long tok = static_cast<long long>(b) * a.T + DELTA_CHUNK * c;
    const int inside = a.T - DELTA_CHUNK * c < DELTA_CHUNK ? a.T - DELTA_CHUNK * c : DELTA_CHUNK;
    // dq and dk: in place, or this head's part
    const bool parts = per > 1;
    const long long oqk = parts ? (tok * a.H + h) * a.Dk : (tok * a.Hk + hk) * a.Dk;
    const int sqk = (parts ? a.H : a.Hk) * a.Dk;
    const long long ogb = tok * a.H + h;

    if (left <= 0) {                   // past the end: zeros
        for (int i = threadIdx.x; i < inside * a.Dk; i += 512) {
            const long long o = oqk + static_cast<long long>(i / a.Dk) * sqk + i % a.Dk;
            if (parts) {
                a.dq_part[o] = 0.0f;
                a.dk_part[o] = 0.0f;
            } else {
                if (a.dq)
                    put_at<BF>(a.dq, o, 0.0f);
                if (a.dk)
                    put_at<BF>(a.dk, o, 0.0f);
            }
        }
        if (static_cast<int>(threadIdx.x) < inside) {
            if (a.dg)
                a.dg[ogb + static_cast<long long>(threadIdx.x) * a.H] = 0.0f;
            if (a.dbeta)
                a.dbeta[ogb + static_cast<long long>(threadIdx.x) * a.H] = 0.0f;
        }
        return;
    }

    const long long at = static_cast<long long>(bh) * a.N + c;
    const Buf bS(a.S0, at * a.Dk * a.Dv * 4), bD(a.D1, at * a.Dk * a.Dv * 4);
    // this thread's piece of 8 of E or dV, and of dO
    const int pr = (threadIdx.x & 255) >> 2, pg = threadIdx.x & 3;
    const bool ofE = wave < 4;
    const Buf bEV(ofE ? a.E : a.dV, at * DELTA_CHUNK * a.Dv * 4);
    const Buf bO(a.dout, (tok * a.H + h) * a.Dv * (BF ? 2 : 4));
    struct Next {
        float ev[8], s[8], d[8];
        In<BF> o;
    } next;
    const auto fetch = [&](int v) __attribute__((always_inline)) {
        const bool mine = v + 8 * pg < a.Dv, states = both(mycol < a.Dk, v + 8 * quad < a.Dv);
        load8(bEV, record_at(pr, 8 * pg + v, DELTA_CHUNK), mine, next.ev);
        next.o = in_load<BF>(bO, pr * a.H * a.Dv + 8 * pg + v, both(both(ofE, mine), pr < left));
        load8(bS, record_at(mycol, 8 * quad + v, a.Dk), states, next.s);
        load8(bD, record_at(mycol, 8 * quad + v, a.Dk), states, next.d);
    };
    const auto spread = [&](int buf) __attribute__((always_inline)) {
        if (ofE) {
            sh.in[buf].E.put8(pr, pg, next.ev);
            sh.in[buf].O.put_in(pr, pg, next.o);
        } else {
            sh.in[buf].V.put8(pr, pg, next.ev);
        }
    };
    fetch(0);
    {
        const long long head = static_cast<long long>(hk) * a.Dk;
        const Buf rowsK(a.k, (tok * a.ks + head) * (BF ? 2 : 4)), rowsQ(a.q, (tok * a.qs + head) * (BF ? 2 : 4));
#pragma unroll
        for (int x = 0; x < KD / 64 + (KD < 64); ++x) {
            // a thread's pieces of 8: every row, KD / 8 pieces
            const int i = threadIdx.x + 512 * x, r = i / (KD / 8), k = i % (KD / 8) * 8;
            const bool live = both(r < left, k < a.Dk);
            const In<BF> fk = in_load<BF>(rowsK, r * static_cast<int>(a.ks) + k, live);
            const In<BF> fq = in_load<BF>(rowsQ, r * static_cast<int>(a.qs) + k, live);
            if (r < 64) {
                sh.k.put(r, k, fk);
                sh.q.put(r, k, fq);
            }
        }
        if (threadIdx.x < (VEC_FLOATS - VEC_BETA) / 4)
            *reinterpret_cast<v4f *>(&sh.vec[4 * threadIdx.x]) =
                *reinterpret_cast<const v4f *>(a.vec + at * VEC_FLOATS + VEC_BETA + 4 * threadIdx.x);
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
        fetch(v + 32 < a.Dv ? v + 32 : v);
        lds_barrier();
        const auto &in = sh.in[buf];
        {
            const In<BF> o = in.O.get_in(row, quad);
            const Mid<BF, 3> y = in.V.get(row, quad);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int j = 2 * half + x;
                if (j > band)
                    continue;
                const Mid<BF, 3> e = in.E.get(16 * j + l15, quad);
                A[x] = mma(o, e, A[x]);
                Y[x] = mma(y, e, Y[x]);
            }
        }
        // a tile's operands are read while the one before is multiplied (with matrices of
        // two words below 200 us, 205 without; with three no difference is left)
        In<BF> ro[2];
        Mid<BF, 3> rv[2], re[2];
        ro[0] = in.O.get_in(16 * rt0 + l15, quad), rv[0] = in.V.get(16 * rt0 + l15, quad), re[0] = in.E.get(16 * rt0 + l15, quad);
#pragma unroll
        for (int ri = 0; ri < RT; ++ri) {
            if (ri + 1 < RT) {
                const int r = 16 * (rt0 + ri + 1) + l15, n = (ri + 1) & 1;
                ro[n] = in.O.get_in(r, quad), rv[n] = in.V.get(r, quad), re[n] = in.E.get(r, quad);
            }
            __builtin_amdgcn_sched_barrier(0);
            oS[ri] = mma(ro[ri & 1], s, oS[ri]);
            vS[ri] = mma(rv[ri & 1], s, vS[ri]);
            eD[ri] = mma(re[ri & 1], d, eD[ri]);
        }
        if (v + 32 < a.Dv)
            spread(buf ^ 1);
    }
    lds_barrier();                     // dO, E and dV are read

    // ---- 64 x 64 parts: this wave's rows i against its columns j
    v4f rowF = v4f_zero();
    const v4f ihi = sh.four(VEC_GHI, rows), ilo = sh.four(VEC_GLO, rows);
    const v4f ri = sh.four(VEC_RK, rows), qi = sh.four(VEC_RQ, rows);
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        const int j = 2 * half + p, col = 16 * j + l15;
        v4f wa = v4f_zero(), wat = v4f_zero();
        float colF = 0.0f;
        if (j <= band) {
            v4f kk = v4f_zero(), qk = v4f_zero(), zl, zu;
#pragma unroll
            for (int f = 0; f < KF; ++f) {
                const int k = 32 * f + 8 * quad;
                const In<BF> o = sh.k.across(col, k);
                kk = mma(sh.k.across(row, k), o, kk);
                qk = mma(sh.q.across(row, k), o, qk);
            }
            const float bj = sh.at(VEC_BETA, col), rj = sh.at(VEC_RK, col);
            const float jhi = sh.at(VEC_GHI, col), jlo = sh.at(VEC_GLO, col);
            v4f F;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const bool on = j < band || col <= rows + e, below = j < band || col < rows + e;
                const float d = decay(ihi[e], ilo[e], jhi, jlo);
                const float x = on ? a.scale * d * A[p][e] : 0.0f;          // dP before beta
                const float y = below ? d * Y[p][e] : 0.0f;
                const float xf = x * qi[e] * rj * qk[e], yf = y * ri[e] * rj * kk[e];
                F[e] = (on ? xf : 0.0f) - (below ? yf : 0.0f);
                const float xb = x * bj, yb = -y * bj;
                wa[e] = xb * rj;
                wat[e] = xb * qi[e];
                zl[e] = yb * rj;
                zu[e] = yb * ri[e];
                // the diagonal is no decay's
                rowF[e] += below ? bj * F[e] : 0.0f;
            }
            colF = (F[0] + F[1]) + (F[2] + F[3]);
            if (j == band && quad == l15 >> 2)
                sh.diag[col] = (l15 & 2) ? ((l15 & 1) ? F[3] : F[2]) : ((l15 & 1) ? F[1] : F[0]);
            // Z's two triangles: rows i > j from here, its mirror from the same values
            if (j < band) {
                sh.out.Z.put_rows(rows, col, zl);
                sh.out.Z.put4(col, rows, zu);
            } else {
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
                sh.out.Z.put_rows(rows, col, z);
            }
        }
        sh.out.A.put_rows(rows, col, wa);
        sh.out.At.put4(col, rows, wat);
        colF += __shfl_xor(colF, 16);
        colF += __shfl_xor(colF, 32);
        if (quad == 0)
            sh.colF[band][col] = colF;
    }
    rowF = sum16(rowF);
    if (l15 == 0)
        *reinterpret_cast<v4f *>(&sh.rowF[half][rows]) = rowF;
    // ---- the states' terms, while the matrices come together
    v4f dq[RT], dk[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        const int r0 = 16 * (rt0 + t), r = r0 + 4 * quad;
        const v4f gam = sh.four(VEC_GAM, r);
        const v4f x = a.scale * gam * oS[t], y = -gam * vS[t], w = sh.four(VEC_END, r) * eD[t];
        const v4f kh = sh.four(VEC_RK, r) * sh.k.tile(r0, col0), qh = sh.four(VEC_RQ, r) * sh.q.tile(r0, col0);
        const v4f s = sum16(qh * x + kh * y), v = sum16(kh * w);
        if (l15 == 0) {
            *reinterpret_cast<v4f *>(&sh.dot[0][wave % CW][r]) = s;
            *reinterpret_cast<v4f *>(&sh.dot[1][wave % CW][r]) = v;
        }
        dq[t] = x;
        dk[t] = sh.four(VEC_BETA, r) * w + y;
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1)
        sd += __shfl_xor(sd, off);
    if (lane == 0)
        sh.sd[wave] = sd;
    lds_barrier();

    // ---- products with the head's width: this wave's columns
#pragma unroll
    for (int f = 0; f < 2; ++f) {
        const In<BF> kd = sh.k.down(32 * f, col0), qd = sh.q.down(32 * f, col0);
#pragma unroll
        for (int ri = 0; ri < RT; ++ri) {
            const int r = 16 * (rt0 + ri) + l15;
            dq[ri] = mma(sh.out.A.get(r, 4 * f + quad), kd, dq[ri]);
            dk[ri] = mma(sh.out.At.get(r, 4 * f + quad), qd, dk[ri]);
            dk[ri] = mma(sh.out.Z.get(r, 4 * f + quad), kd, dk[ri]);
        }
    }
    if (wave == 0) {
        float s = 0.0f, w = 0.0f, col = 0.0f, inner = 0.0f;
#pragma unroll
        for (int x = 0; x < CW; ++x) {
            s += sh.dot[0][x][lane];
            w += sh.dot[1][x][lane];
        }
#pragma unroll
        for (int x = 0; x < 4; ++x)
            col += x >= lane / 16 ? sh.colF[x][lane] : 0.0f;
#pragma unroll
        for (int x = 0; x < 8; ++x)
            inner += sh.sd[x];
        const float beta = sh.at(VEC_BETA, lane);
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
        const float dg = after + (before - w) + sh.at(VEC_GAM, 63) * inner;
        if (lane < inside) {
            const long long o = ogb + static_cast<long long>(lane) * a.H;
            if (a.dg)
                a.dg[o] = lane < left ? dg : 0.0f;
            if (a.dbeta)
                a.dbeta[o] = lane < left ? dbeta : 0.0f;
        }
    }

    // ---- through the normalisation, and out
    if (a.eps > 0.0f) {
        lds_barrier();                 // the sums for dg are read
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            const int r0 = 16 * (rt0 + t), r = r0 + 4 * quad;
            const v4f x = sum16(sh.q.tile(r0, col0) * dq[t]), y = sum16(sh.k.tile(r0, col0) * dk[t]);
            if (l15 == 0) {
                *reinterpret_cast<v4f *>(&sh.dot[0][wave % CW][r]) = x;
                *reinterpret_cast<v4f *>(&sh.dot[1][wave % CW][r]) = y;
            }
        }
        lds_barrier();
        if (threadIdx.x < 128) {
            const int which = threadIdx.x >> 6;
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < CW; ++w)
                s += sh.dot[which][w][lane];
            const float r = sh.at(which ? VEC_RK : VEC_RQ, lane);
            sh.norm[which][lane] = r * r * s;          // r q^.dq^, likewise k
        }
        lds_barrier();
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            const int r0 = 16 * (rt0 + t), r = r0 + 4 * quad;
            dq[t] = sh.four(VEC_RQ, r) * (dq[t] - sh.q.tile(r0, col0) * *reinterpret_cast<const v4f *>(&sh.norm[0][r]));
            dk[t] = sh.four(VEC_RK, r) * (dk[t] - sh.k.tile(r0, col0) * *reinterpret_cast<const v4f *>(&sh.norm[1][r]));
        }
    }
    const Buf oq(parts ? a.dq_part : a.dq, oqk * (parts || !BF ? 4 : 2));
    const Buf ok(parts ? a.dk_part : a.dk, oqk * (parts || !BF ? 4 : 2));
#pragma unroll
    for (int ri = 0; ri < RT; ++ri)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = 16 * (rt0 + ri) + 4 * quad + e, o = i * sqk + mycol;
            const bool live = both(i < inside, mycol < a.Dk);
            const float x = i < left ? dq[ri][e] : 0.0f, y = i < left ? dk[ri][e] : 0.0f;
            if (parts) {
                put_value<false>(oq, o, live, x);
                put_value<false>(ok, o, live, y);
            } else {
                put_value<BF>(oq, o, both(live, a.dq != nullptr), x);
                put_value<BF>(ok, o, both(live, a.dk != nullptr), y);
            }
        }
}

// dq and dk over the heads that share them, from fp32 parts [B][T][H][Dk]: 8 values a
// thread, the heads in order.
template <bool BF> __global__ __launch_bounds__(256) void delta_heads_kernel(DeltaArgs a)
{
    const int per = a.H / a.Hk, pieces = a.Dk / 8;
    const long long total = static_cast<long long>(a.B) * a.T * a.Hk * pieces;
    for (long long i = blockIdx.x * 256LL + threadIdx.x; i < 2 * total; i += 256LL * gridDim.x) {
        const bool ofK = i >= total;
        const long long x = ofK ? i - total : i, row = x / pieces;       // token and q/k head
        void *out = ofK ? a.dk : a.dq;
        if (!out)
            continue;
        const float *part = (ofK ? a.dk_part : a.dq_part) + row * per * a.Dk + x % pieces * 8;
        float s[8];
        load_f32<8, true>(part, s);
        for (int g = 1; g < per; ++g) {
            float v[8];
            load_f32<8, true>(part + static_cast<long long>(g) * a.Dk, v);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                s[e] += v[e];
        }
        store_row<8, true>(out, BF, row * a.Dk + x % pieces * 8, 8, s);
    }
}

}  // namespace

namespace srnl_i {

srnl_status launch_delta_grads(const DeltaArgs &a, hipStream_t st)
{
    const dim3 grid(static_cast<unsigned>(static_cast<long long>(a.B) * a.H * a.N));
#define SRNL_DELTA_GRADS(BF, KD) hipLaunchKernelGGL((delta_grads_kernel<BF, KD>), grid, dim3(512), 0, st, a)
    SRNL_DELTA_DISPATCH(a, SRNL_DELTA_GRADS);
    if (a.H > a.Hk && (a.dq || a.dk)) {
        const long long blocks = (static_cast<long long>(a.B) * a.T * a.Hk * (a.Dk / 8) * 2 + 255) / 256;
        const dim3 heads(static_cast<unsigned>(blocks < 1 << 16 ? blocks : 1 << 16));
        if (a.bf)
            hipLaunchKernelGGL(delta_heads_kernel<true>, heads, dim3(256), 0, st, a);
        else
            hipLaunchKernelGGL(delta_heads_kernel<false>, heads, dim3(256), 0, st, a);
    }
    return launched("delta_grads_kernel");
}

}  // namespace srnl_i
