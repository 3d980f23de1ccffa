// delta_step.hip -- the gated delta rule token by token, for a few tokens per
// sequence: the form a server appends tokens with.
//
// With a = exp(g), r_q = 1/|q| and r_k = 1/|k| (1 without normalisation) and
// the state S before the token,
//   u = beta (v - a r_k S^T k),  o = scale (a r_q S^T q + r_q r_k (q.k) u),
//   S <- a S + r_k k u^T,
// so one pass over S gives S^T k and S^T q together, and one reduction over
// the rows serves both, the norms and q.k.
//
// The call is bound by the state: 2 x 4 bytes per entry, read once and written
// once; a block keeps a 64-column slab of it in registers over all its tokens.
#include "delta.h"

namespace {

using namespace srnl_i;

__device__ __forceinline__ float element(const void *p, bool bf, long long o)
{
    return bf ? bf16_one(static_cast<const uint16_t *>(p)[o]) : static_cast<const float *>(p)[o];
}

// 256 threads: 16 row groups x 16 lanes of 4 columns; a thread holds rows
// group, group + 16, ... (R of them).
template <int R>
__global__ __launch_bounds__(256) void delta_step_kernel(DeltaArgs a)
{
    __shared__ float part[2][4][16][8];
    __shared__ float dots[2][4][3];
    const int tiles = (a.Dv + 63) / 64;
    const int bh = blockIdx.x / tiles, tile = blockIdx.x - bh * tiles;
    const int b = bh / a.H, h = bh - b * a.H, hk = h / (a.H / a.Hk);
    const int lane = threadIdx.x & 15, grp = threadIdx.x >> 4, wave = threadIdx.x >> 6;
    const int col = 64 * tile + 4 * lane;
    const bool mine = col < a.Dv;                       // Dv is a multiple of 8
    const long long base = static_cast<long long>(bh) * a.Dk * a.Dv + col;
    const int n = delta_tokens(a, b);

    f32x4 S[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int row = grp + 16 * i;
        S[i] = f32x4{0, 0, 0, 0};
        if (a.state && mine && row < a.Dk)
            S[i] = *reinterpret_cast<const f32x4 *>(a.state + base + static_cast<long long>(row) * a.Dv);
    }
    for (int t = 0; t < n; ++t) {
        const long long tok = static_cast<long long>(b) * a.T + t;
        float kr[R], qr[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int row = grp + 16 * i;
            kr[i] = qr[i] = 0.0f;
            if (row < a.Dk) {
                kr[i] = element(a.k, a.bf, tok * a.ks + hk * a.Dk + row);
                qr[i] = element(a.q, a.bf, tok * a.qs + hk * a.Dk + row);
            }
        }
        float v[4] = {0, 0, 0, 0};
        if (mine)
            load_row<4, true>(a.v, a.bf, tok * a.vs + static_cast<long long>(h) * a.Dv + col, 4, v);
        const float dec = expf(a.g[tok * a.H + h]), beta = a.beta[tok * a.H + h];
        f32x4 sk = {0, 0, 0, 0}, sq = {0, 0, 0, 0};
        float kk = 0.0f, qq = 0.0f, kq = 0.0f;
#pragma unroll
        for (int i = 0; i < R; ++i) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                sk[c] = fmaf(S[i][c], kr[i], sk[c]);
                sq[c] = fmaf(S[i][c], qr[i], sq[c]);
            }
            kk = fmaf(kr[i], kr[i], kk);
            qq = fmaf(qr[i], qr[i], qq);
            kq = fmaf(kr[i], qr[i], kq);
        }
        // over the wave's 4 row groups, then over the 4 waves; two buffers, so
        // one barrier per token is enough
        float red[11] = {sk[0], sk[1], sk[2], sk[3], sq[0], sq[1], sq[2], sq[3], kk, qq, kq};
#pragma unroll
        for (int j = 0; j < 11; ++j) {
            red[j] += __shfl_xor(red[j], 16);
            red[j] += __shfl_xor(red[j], 32);
        }
        const int buf = t & 1;
        if ((threadIdx.x & 63) < 16) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                part[buf][wave][lane][j] = red[j];
            if (lane < 3)
                dots[buf][wave][lane] = lane == 0 ? red[8] : lane == 1 ? red[9] : red[10];
        }
        __syncthreads();
        float sum[8], dot[3];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            sum[j] = (part[buf][0][lane][j] + part[buf][1][lane][j]) + (part[buf][2][lane][j] + part[buf][3][lane][j]);
#pragma unroll
        for (int j = 0; j < 3; ++j)
            dot[j] = (dots[buf][0][j] + dots[buf][1][j]) + (dots[buf][2][j] + dots[buf][3][j]);
        const float rk = a.eps > 0.0f ? 1.0f / sqrtf(dot[0] + a.eps) : 1.0f;
        const float rq = a.eps > 0.0f ? 1.0f / sqrtf(dot[1] + a.eps) : 1.0f;
        float u[4], o[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            u[c] = beta * (v[c] - dec * rk * sum[c]);
            o[c] = a.scale * rq * (dec * sum[4 + c] + rk * dot[2] * u[c]);
        }
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c)
                S[i][c] = fmaf(rk * kr[i], u[c], dec * S[i][c]);
        if (grp == 0 && mine)
            store_row<4, true>(a.out, a.bf, (tok * a.H + h) * a.Dv + col, 4, o);
    }
    if (mine && grp == 0) {
        const float zero[4] = {0, 0, 0, 0};
        for (int t = n; t < a.T; ++t)
            store_row<4, true>(a.out, a.bf, ((static_cast<long long>(b) * a.T + t) * a.H + h) * a.Dv + col, 4, zero);
    }
    if (a.state_out && mine) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int row = grp + 16 * i;
            if (row < a.Dk)
                *reinterpret_cast<f32x4 *>(a.state_out + base + static_cast<long long>(row) * a.Dv) = S[i];
        }
    }
}

}  // namespace

namespace srnl_i {

srnl_status launch_delta_step(const DeltaArgs &a, hipStream_t st)
{
    const dim3 grid(static_cast<unsigned>(static_cast<long long>(a.B) * a.H * ((a.Dv + 63) / 64)));
    if (a.Dk <= 32)
        hipLaunchKernelGGL(delta_step_kernel<2>, grid, dim3(256), 0, st, a);
    else if (a.Dk <= 64)
        hipLaunchKernelGGL(delta_step_kernel<4>, grid, dim3(256), 0, st, a);
    else
        hipLaunchKernelGGL(delta_step_kernel<8>, grid, dim3(256), 0, st, a);
    return launched("delta_step_kernel");
}

}  // namespace srnl_i
