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
// once; a block keeps a slab of its columns in registers over all its tokens. q and
// k of a token go through LDS: read from memory by every thread that needs them,
// their loads, one per row, would outnumber the state's (256 sequences, 16 heads of
// 128 x 128: 198 us, 101 us so, as fast as a copy).
#include "delta.h"
#include "linear.h"

namespace {

using namespace srnl_i;

// 256 threads: 256 / LANES row groups x LANES lanes of 4 columns; a thread holds R
// rows one after the other.
template <int R, int LANES> __global__ __launch_bounds__(256, 4) void delta_step_kernel(DeltaArgs a)
{
    constexpr int GROUPS = 256 / LANES, WIDTH = 4 * LANES;
    __shared__ float part[2][4][LANES][8];
    __shared__ float dots[2][4][3];
    __shared__ __attribute__((aligned(16))) float kq[2][2][GROUPS * R];
    const int tiles = (a.Dv + WIDTH - 1) / WIDTH;
    const int bh = blockIdx.x / tiles, tile = blockIdx.x - bh * tiles;
    const int b = bh / a.H, h = bh - b * a.H, hk = h / (a.H / a.Hk);
    const int lane = threadIdx.x % LANES, grp = threadIdx.x / LANES, wave = threadIdx.x >> 6;
    const int col = WIDTH * tile + 4 * lane, row0 = grp * R;
    const bool mine = col < a.Dv;                       // Dv is a multiple of 8
    const long long base = static_cast<long long>(bh) * a.Dk * a.Dv + col;
    const int n = delta_tokens(a, b);

    // a token's k (threads 0 ..) and q (threads 128 ..), 4 values a thread
    const int half = threadIdx.x >> 7, piece = 4 * (threadIdx.x & 127);
    const bool fetches = piece < GROUPS * R;
    float ahead[4] = {0, 0, 0, 0};
    const auto fetch = [&](int t) __attribute__((always_inline)) {
        const long long tok = static_cast<long long>(b) * a.T + t;
        if (piece < a.Dk) {
            if (half == 0)
                load_row<4, true>(a.k, a.bf, tok * a.ks + hk * a.Dk + piece, 4, ahead);
            else
                load_row<4, true>(a.q, a.bf, tok * a.qs + hk * a.Dk + piece, 4, ahead);
        }
    };
    if (n > 0)
        fetch(0);
    f32x4 S[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        S[i] = f32x4{0, 0, 0, 0};
        if (a.state && mine && row0 + i < a.Dk)
            S[i] = *reinterpret_cast<const f32x4 *>(a.state + base + static_cast<long long>(row0 + i) * a.Dv);
    }
    for (int t = 0; t < n; ++t) {
        const long long tok = static_cast<long long>(b) * a.T + t;
        const int buf = t & 1;
        if (fetches)
            *reinterpret_cast<f32x4 *>(&kq[buf][half][piece]) = f32x4{ahead[0], ahead[1], ahead[2], ahead[3]};
        float v[4] = {0, 0, 0, 0};
        if (mine)
            load_row<4, true>(a.v, a.bf, tok * a.vs + static_cast<long long>(h) * a.Dv + col, 4, v);
        const float dec = expf(a.g[tok * a.H + h]), beta = a.beta[tok * a.H + h];
        if (t + 1 < n)
            fetch(t + 1);
        lds_barrier();
        float kr[R], qr[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            kr[i] = kq[buf][0][row0 + i];
            qr[i] = kq[buf][1][row0 + i];
        }
        f32x4 sk = {0, 0, 0, 0}, sq = {0, 0, 0, 0};
        float kk = 0.0f, qq = 0.0f, kq1 = 0.0f;
#pragma unroll
        for (int i = 0; i < R; ++i) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                sk[c] = fmaf(S[i][c], kr[i], sk[c]);
                sq[c] = fmaf(S[i][c], qr[i], sq[c]);
            }
            kk = fmaf(kr[i], kr[i], kk);
            qq = fmaf(qr[i], qr[i], qq);
            kq1 = fmaf(kr[i], qr[i], kq1);
        }
        // over the wave's row groups, then over the 4 waves; two buffers, so that two
        // barriers per token are enough
        float red[11] = {sk[0], sk[1], sk[2], sk[3], sq[0], sq[1], sq[2], sq[3], kk, qq, kq1};
#pragma unroll
        for (int j = 0; j < 11; ++j)
#pragma unroll
            for (int off = LANES; off < 64; off <<= 1)
                red[j] += __shfl_xor(red[j], off);
        if ((threadIdx.x & 63) < LANES) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                part[buf][wave][lane][j] = red[j];
            if (lane < 3)
                dots[buf][wave][lane] = lane == 0 ? red[8] : lane == 1 ? red[9] : red[10];
        }
        lds_barrier();
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
        for (int i = 0; i < R; ++i)
            if (row0 + i < a.Dk)
                *reinterpret_cast<f32x4 *>(a.state_out + base + static_cast<long long>(row0 + i) * a.Dv) = S[i];
    }
}

template <int LANES> void launch_step(const DeltaArgs &a, hipStream_t st)
{
    constexpr int GROUPS = 256 / LANES;
    const long long tiles = (a.Dv + 4 * LANES - 1) / (4 * LANES);
    const dim3 grid(static_cast<unsigned>(static_cast<long long>(a.B) * a.H * tiles));
    if (a.Dk <= 32)
        hipLaunchKernelGGL((delta_step_kernel<32 / GROUPS, LANES>), grid, dim3(256), 0, st, a);
    else if (a.Dk <= 64)
        hipLaunchKernelGGL((delta_step_kernel<64 / GROUPS, LANES>), grid, dim3(256), 0, st, a);
    else
        hipLaunchKernelGGL((delta_step_kernel<128 / GROUPS, LANES>), grid, dim3(256), 0, st, a);
}

}  // namespace

namespace srnl_i {

srnl_status launch_delta_step(const DeltaArgs &a, hipStream_t st)
{
    // 64 columns a block, 32 where v has no more: 256 x 16 heads of 128 x 32 take 25 us
    // with 32, 27 with 64; 64 x 16 of 128 x 128, 5 tokens, 68 and 44
    if (a.Dv <= 32)
        launch_step<8>(a, st);
    else
        launch_step<16>(a, st);
    return launched("delta_step_kernel");
}

}  // namespace srnl_i
