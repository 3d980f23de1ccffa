// group_norm.hip -- group norm with an activation over channels-last maps,
// forward and backward. Entry points as declared in include/srnl.h.
//
//   n = (x - mean) rstd, z = n gain + bias, y = act(z); mean and the biased
//   variance over the cells and channels of one item's group
//   dz = dout act'(z), d = dz gain:
//   dx = rstd (d - mean(d) - n mean(d n)) [+ add]
//   dgain = sum of dz n,  dbias = sum of dz, over items and cells
//
// An item's map is cut into slabs of cells. A thread keeps a column of V
// channels and walks the slab's cells, a block of 256 threads side by side, so
// every access is a wide piece of a row.
#include "linear.h"

namespace {

using namespace srnl_i;

struct GnArgs {
    const void *x;          // [B][S][C]
    int B, C, G;
    long long S;
    bool xbf;
    const float *gain, *bias;
    float eps;
    int act;
    void *out;              // forward: y; backward: dx
    bool obf;
    float *mean, *rstd;     // [B][G]
    const void *dout, *add; // backward
    bool dbf;
    float *part;            // [B][slabs][2 C]
    float *means;           // backward: [B][G][2], mean(d) and mean(d n)
    int slabs;
    long long rows;         // cells of a slab
    int tiles;              // blocks side by side along the channels
};

template <int V> __device__ __forceinline__ void load_piece(const void *p, bool bf, long long o, float (&v)[V])
{
    if constexpr (V >= 4) {
        load_row<V, true>(p, bf, o, V, v);
    } else if constexpr (V == 2) {
        if (bf) {
            const uint32_t w = *reinterpret_cast<const uint32_t *>(static_cast<const uint16_t *>(p) + o);
            v[0] = bf16_lo(w);
            v[1] = bf16_hi(w);
        } else {
            const f32x2 w = *reinterpret_cast<const f32x2 *>(static_cast<const float *>(p) + o);
            v[0] = w[0];
            v[1] = w[1];
        }
    } else {
        v[0] = bf ? bf16_one(static_cast<const uint16_t *>(p)[o]) : static_cast<const float *>(p)[o];
    }
}
template <int V> __device__ __forceinline__ void store_piece(void *p, bool bf, long long o, const float (&v)[V])
{
    if constexpr (V >= 4) {
        store_row<V, true>(p, bf, o, V, v);
    } else if constexpr (V == 2) {
        if (bf)
            *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(p) + o) = pack_bf16(v[0], v[1]);
        else
            *reinterpret_cast<f32x2 *>(static_cast<float *>(p) + o) = f32x2{v[0], v[1]};
    } else {
        if (bf)
            static_cast<uint16_t *>(p)[o] = to_bf16(v[0]);
        else
            static_cast<float *>(p)[o] = v[0];
    }
}

// A thread's place: its channels, and the cells it walks.
template <int V> struct Place {
    int b, c, lanes, lane;          // channel c .. c + V - 1; every lanes-th cell from lane
    long long first, last;          // the slab's cells
    bool live;
    __device__ __forceinline__ explicit Place(const GnArgs &a)
    {
        const int pieces = a.C / V;
        const int tile = blockIdx.x % a.tiles;
        const int rest = blockIdx.x / a.tiles;
        const int slab = rest % a.slabs;
        b = rest / a.slabs;
        const int wide = pieces < 256 ? pieces : 256;
        lanes = 256 / wide;
        lane = threadIdx.x / wide;
        const int piece = tile * 256 + threadIdx.x % wide;
        live = lane < lanes && piece < pieces;
        c = V * piece;
        first = slab * a.rows;
        last = first + a.rows < a.S ? first + a.rows : a.S;
    }
    __device__ __forceinline__ long long at(const GnArgs &a, long long s) const
    {
        return (b * a.S + s) * a.C + c;
    }
    __device__ __forceinline__ int wide(const GnArgs &a) const { return a.C / V < 256 ? a.C / V : 256; }
};

// Cells that lane l of `lanes` walks between first and last.
__device__ __forceinline__ long long cells_of(long long cells, int lanes, int l)
{
    return cells > l ? (cells - l + lanes - 1) / lanes : 0;
}

// Mean and sum of squares about it, per channel of a slab. A thread sums
// distances from its first cell, so an offset costs no digits: what is lost is
// at most its number of cells times the rounding of the sum.
template <int V> __global__ __launch_bounds__(256) void gn_stats_kernel(GnArgs a)
{
    __shared__ float lds[256][2 * V];
    const Place<V> pl(a);
    const long long cells = pl.last - pl.first;
    if (pl.live) {
        const long long mine = cells_of(cells, pl.lanes, pl.lane);
        float from[V], s1[V], s2[V];
#pragma unroll
        for (int e = 0; e < V; ++e)
            from[e] = s1[e] = s2[e] = 0.0f;
        if (mine)
            load_piece<V>(a.x, a.xbf, pl.at(a, pl.first + pl.lane), from);
#pragma unroll 4
        for (long long i = 1; i < mine; ++i) {
            float v[V];
            load_piece<V>(a.x, a.xbf, pl.at(a, pl.first + pl.lane + i * pl.lanes), v);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float d = v[e] - from[e];
                s1[e] += d;
                s2[e] = fmaf(d, d, s2[e]);
            }
        }
        const float n = static_cast<float>(mine);
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float m = mine ? s1[e] / n : 0.0f;
            lds[threadIdx.x][e] = from[e] + m;
            lds[threadIdx.x][V + e] = fmaxf(s2[e] - n * m * m, s2[e] * 0.0f);
        }
    }
    __syncthreads();
    const int wide = pl.wide(a);
    float *part = a.part + (static_cast<long long>(pl.b) * a.slabs + blockIdx.x / a.tiles % a.slabs) * 2 * a.C;
    const int c0 = blockIdx.x % a.tiles * 256 * V;
    for (int j = threadIdx.x; j < wide * V && c0 + j < a.C; j += 256) {
        const int piece = j / V, e = j % V;
        // about the first lane's mean, so that a constant map's mean is exact
        const float ref = lds[piece][e];
        float mean = 0.0f, m2 = 0.0f;
        for (int l = 1; l < pl.lanes; ++l) {
            const float n = static_cast<float>(cells_of(cells, pl.lanes, l));
            mean = n > 0.0f ? fmaf(lds[l * wide + piece][e] - ref, n / static_cast<float>(cells), mean) : mean;
        }
        mean += ref;
        for (int l = 0; l < pl.lanes; ++l) {
            const float d = lds[l * wide + piece][e] - mean;
            const float n = static_cast<float>(cells_of(cells, pl.lanes, l));
            m2 += n > 0.0f ? fmaf(n * d, d, lds[l * wide + piece][V + e]) : 0.0f;
        }
        part[c0 + j] = mean;
        part[a.C + c0 + j] = m2;
    }
}

__device__ __forceinline__ float wave_sum(float v)
{
#pragma unroll
    for (int off = 32; off > 0; off >>= 1)
        v += __shfl_xor(v, off);
    return v;
}

// A wave joins one group's channels and slabs.
__global__ __launch_bounds__(256) void gn_join_kernel(GnArgs a)
{
    const long long group = blockIdx.x * 4LL + (threadIdx.x >> 6);
    if (group >= static_cast<long long>(a.B) * a.G)
        return;
    const int b = static_cast<int>(group / a.G), cpg = a.C / a.G, c0 = static_cast<int>(group % a.G) * cpg;
    const int lane = threadIdx.x & 63;
    const float *part = a.part + static_cast<long long>(b) * a.slabs * 2 * a.C;
    const long long entries = static_cast<long long>(a.slabs) * cpg;
    const float total = static_cast<float>(a.S) * static_cast<float>(cpg);
    const float ref = part[c0];
    float mean = 0.0f;
    for (long long i = lane; i < entries; i += 64) {
        const long long slab = i / cpg;
        const long long cells = slab + 1 < a.slabs ? a.rows : a.S - slab * a.rows;
        mean = fmaf(part[slab * 2 * a.C + c0 + i % cpg] - ref, static_cast<float>(cells) / total, mean);
    }
    mean = ref + wave_sum(mean);
    float m2 = 0.0f;
    for (long long i = lane; i < entries; i += 64) {
        const long long slab = i / cpg;
        const long long cells = slab + 1 < a.slabs ? a.rows : a.S - slab * a.rows;
        const float d = part[slab * 2 * a.C + c0 + i % cpg] - mean;
        m2 += fmaf(static_cast<float>(cells) * d, d, part[slab * 2 * a.C + a.C + c0 + i % cpg]);
    }
    m2 = wave_sum(m2);
    if (lane == 0) {
        a.mean[group] = mean;
        a.rstd[group] = 1.0f / sqrtf(m2 / total + a.eps);
    }
}

// What a thread keeps of its channels: n = (x - mean) rstd, z = n gain + bias.
template <int V> struct Channels {
    float mean[V], rstd[V], gain[V], bias[V];
    __device__ __forceinline__ Channels(const GnArgs &a, const Place<V> &pl)
    {
        const int cpg = a.C / a.G;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const long long group = static_cast<long long>(pl.b) * a.G + (pl.c + e) / cpg;
            mean[e] = a.mean[group];
            rstd[e] = a.rstd[group];
            gain[e] = a.gain ? a.gain[pl.c + e] : 1.0f;
            bias[e] = a.bias ? a.bias[pl.c + e] : 0.0f;
        }
    }
};

template <int V> __device__ __forceinline__ void act_piece(float (&v)[V], int act)
{
    if (act == SRNL_ACT_GELU) {
#pragma unroll
        for (int e = 0; e < V; ++e)
            v[e] = gelu(v[e]);
    } else if (act == SRNL_ACT_SILU) {
#pragma unroll
        for (int e = 0; e < V; ++e)
            v[e] *= logistic(v[e]);
    }
}
template <int V> __device__ __forceinline__ void slope_piece(const float (&z)[V], int act, float (&d)[V])
{
    if (act == SRNL_ACT_GELU) {
#pragma unroll
        for (int e = 0; e < V; ++e)
            d[e] *= gelu_slope(z[e]);
    } else if (act == SRNL_ACT_SILU) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float s = logistic(z[e]);
            d[e] *= s * fmaf(z[e], 1.0f - s, 1.0f);
        }
    }
}

template <int V> __global__ __launch_bounds__(256) void gn_apply_kernel(GnArgs a)
{
    const Place<V> pl(a);
    if (!pl.live)
        return;
    const Channels<V> ch(a, pl);
#pragma unroll 4
    for (long long s = pl.first + pl.lane; s < pl.last; s += pl.lanes) {
        float v[V];
        load_piece<V>(a.x, a.xbf, pl.at(a, s), v);
#pragma unroll
        for (int e = 0; e < V; ++e)
            v[e] = fmaf((v[e] - ch.mean[e]) * ch.rstd[e], ch.gain[e], ch.bias[e]);
        act_piece<V>(v, a.act);
        store_piece<V>(a.out, a.obf, pl.at(a, s), v);
    }
}

// Sums of dz n and of dz, per channel of a slab.
template <int V> __global__ __launch_bounds__(256) void gn_bwd_sums_kernel(GnArgs a)
{
    __shared__ float lds[256][2 * V];
    const Place<V> pl(a);
    if (pl.live) {
        const Channels<V> ch(a, pl);
        float s0[V], s1[V];
#pragma unroll
        for (int e = 0; e < V; ++e)
            s0[e] = s1[e] = 0.0f;
#pragma unroll 4
        for (long long s = pl.first + pl.lane; s < pl.last; s += pl.lanes) {
            float v[V], d[V], z[V];
            load_piece<V>(a.x, a.xbf, pl.at(a, s), v);
            load_piece<V>(a.dout, a.dbf, pl.at(a, s), d);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                v[e] = (v[e] - ch.mean[e]) * ch.rstd[e];
                z[e] = fmaf(v[e], ch.gain[e], ch.bias[e]);
            }
            slope_piece<V>(z, a.act, d);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                s0[e] = fmaf(d[e], v[e], s0[e]);
                s1[e] += d[e];
            }
        }
#pragma unroll
        for (int e = 0; e < V; ++e) {
            lds[threadIdx.x][e] = s0[e];
            lds[threadIdx.x][V + e] = s1[e];
        }
    }
    __syncthreads();
    const int wide = pl.wide(a);
    float *part = a.part + (static_cast<long long>(pl.b) * a.slabs + blockIdx.x / a.tiles % a.slabs) * 2 * a.C;
    const int c0 = blockIdx.x % a.tiles * 256 * V;
    for (int j = threadIdx.x; j < wide * V && c0 + j < a.C; j += 256) {
        float s0 = 0.0f, s1 = 0.0f;
        for (int l = 0; l < pl.lanes; ++l) {
            s0 += lds[l * wide + j / V][j % V];
            s1 += lds[l * wide + j / V][V + j % V];
        }
        part[c0 + j] = s0;
        part[a.C + c0 + j] = s1;
    }
}

__global__ __launch_bounds__(256) void gn_bwd_join_kernel(GnArgs a)
{
    const long long group = blockIdx.x * 4LL + (threadIdx.x >> 6);
    if (group >= static_cast<long long>(a.B) * a.G)
        return;
    const int b = static_cast<int>(group / a.G), cpg = a.C / a.G, c0 = static_cast<int>(group % a.G) * cpg;
    const int lane = threadIdx.x & 63;
    const float *part = a.part + static_cast<long long>(b) * a.slabs * 2 * a.C;
    const long long entries = static_cast<long long>(a.slabs) * cpg;
    float sn = 0.0f, sd = 0.0f;
    for (long long i = lane; i < entries; i += 64) {
        const int c = c0 + static_cast<int>(i % cpg);
        const float *p = part + i / cpg * 2 * a.C;
        const float gain = a.gain ? a.gain[c] : 1.0f;
        sn = fmaf(p[c], gain, sn);
        sd = fmaf(p[a.C + c], gain, sd);
    }
    sn = wave_sum(sn);
    sd = wave_sum(sd);
    if (lane == 0) {
        const float total = static_cast<float>(a.S) * static_cast<float>(cpg);
        a.means[2 * group] = sd / total;
        a.means[2 * group + 1] = sn / total;
    }
}

template <int V> __global__ __launch_bounds__(256) void gn_bwd_apply_kernel(GnArgs a)
{
    const Place<V> pl(a);
    if (!pl.live)
        return;
    const Channels<V> ch(a, pl);
    float md[V], mn[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
        const long long group = static_cast<long long>(pl.b) * a.G + (pl.c + e) / (a.C / a.G);
        md[e] = a.means[2 * group];
        mn[e] = a.means[2 * group + 1];
    }
#pragma unroll 4
    for (long long s = pl.first + pl.lane; s < pl.last; s += pl.lanes) {
        float v[V], d[V], z[V], w[V];
        load_piece<V>(a.x, a.xbf, pl.at(a, s), v);
        load_piece<V>(a.dout, a.dbf, pl.at(a, s), d);
        if (a.add)
            load_piece<V>(a.add, a.xbf, pl.at(a, s), w);
#pragma unroll
        for (int e = 0; e < V; ++e) {
            v[e] = (v[e] - ch.mean[e]) * ch.rstd[e];
            z[e] = fmaf(v[e], ch.gain[e], ch.bias[e]);
        }
        slope_piece<V>(z, a.act, d);
#pragma unroll
        for (int e = 0; e < V; ++e) {
            v[e] = ch.rstd[e] * (d[e] * ch.gain[e] - md[e] - v[e] * mn[e]);
            if (a.add)
                v[e] += w[e];
        }
        store_piece<V>(a.out, a.obf, pl.at(a, s), v);
    }
}

// ------------------------------------------------------------------ launches

// The widest piece that divides a row.
int piece_of(int C) { return C % 8 == 0 ? 8 : C % 4 == 0 ? 4 : C % 2 == 0 ? 2 : 1; }

// Slabs of at least 8 cells a lane, as many as make about 4 blocks per CU.
void cut_map(GnArgs &a)
{
    const int pieces = a.C / piece_of(a.C);
    a.tiles = (pieces + 255) / 256;
    const int lanes = pieces < 256 ? 256 / pieces : 1;
    const long long most = (a.S + 8LL * lanes - 1) / (8LL * lanes);
    const long long items = static_cast<long long>(a.B) * a.tiles;
    long long slabs = (1024 + items - 1) / items;
    slabs = slabs < most ? slabs : most;
    a.rows = (a.S + slabs - 1) / slabs;
    a.slabs = static_cast<int>((a.S + a.rows - 1) / a.rows);
}

size_t part_floats(const GnArgs &a) { return static_cast<size_t>(a.B) * a.slabs * 2 * a.C; }
size_t group_floats(const GnArgs &a) { return 2 * static_cast<size_t>(a.B) * a.G; }

#define SRNL_GN_LAUNCH(kernel, a, st)                                                                  \
    do {                                                                                               \
        const dim3 grid(static_cast<unsigned>(static_cast<long long>((a).B) * (a).slabs * (a).tiles)); \
        switch (piece_of((a).C)) {                                                                     \
        case 8: hipLaunchKernelGGL(kernel<8>, grid, dim3(256), 0, st, a); break;                       \
        case 4: hipLaunchKernelGGL(kernel<4>, grid, dim3(256), 0, st, a); break;                       \
        case 2: hipLaunchKernelGGL(kernel<2>, grid, dim3(256), 0, st, a); break;                       \
        default: hipLaunchKernelGGL(kernel<1>, grid, dim3(256), 0, st, a); break;                      \
        }                                                                                              \
    } while (0)

dim3 join_grid(const GnArgs &a)
{
    return dim3(static_cast<unsigned>((static_cast<long long>(a.B) * a.G + 3) / 4));
}

srnl_status check_gn(int B, long long S, int C, int G, srnl_dtype x, srnl_dtype out, float eps, int act)
{
    if (B < 0 || S < 0)
        return fail(SRNL_ERR_ARG, "B and S must be >= 0");
    if (C < 1 || G < 1 || C % G)
        return fail(SRNL_ERR_ARG, "C must be >= 1 and a multiple of groups");
    if (C > 1 << 20 || static_cast<__int128>(B) * S * C >= (static_cast<__int128>(1) << 60) || S >= 1LL << 40)
        return fail(SRNL_ERR_ARG, "map too large");
    // an item and tile of channels is a block, a group a wave
    if (static_cast<__int128>(B) * C > 1 << 23)
        return fail(SRNL_ERR_ARG, "B x C is too large");
    if (!valid_dtype(x) || !valid_dtype(out))
        return fail(SRNL_ERR_DTYPE, "dtype must be SRNL_F32 or SRNL_BF16");
    if (!(eps > 0.0f) || !std::isfinite(eps))
        return fail(SRNL_ERR_ARG, "eps must be positive and finite");
    if (act != SRNL_ACT_NONE && act != SRNL_ACT_GELU && act != SRNL_ACT_SILU)
        return fail(SRNL_ERR_ARG, "unknown activation");
    return SRNL_OK;
}

GnArgs gn_args(const void *x, int B, long long S, int C, int G, srnl_dtype x_dtype, const float *gain,
               const float *bias, float eps, int act)
{
    GnArgs a = {};
    a.x = x;
    a.B = B;
    a.S = S;
    a.C = C;
    a.G = G;
    a.xbf = x_dtype == SRNL_BF16;
    a.gain = gain;
    a.bias = bias;
    a.eps = eps;
    a.act = act;
    cut_map(a);
    return a;
}

}  // namespace

extern "C" {

size_t srnl_group_norm_fwd_workspace_bytes(int B, long long S, int C, int groups)
{
    if (check_gn(B, S, C, groups, SRNL_F32, SRNL_F32, 1.0f, 0) != SRNL_OK || B == 0 || S == 0)
        return 0;
    const GnArgs a = gn_args(nullptr, B, S, C, groups, SRNL_F32, nullptr, nullptr, 1.0f, 0);
    return (part_floats(a) + group_floats(a)) * sizeof(float);
}

srnl_status srnl_group_norm_fwd(const void *x, int B, long long S, int C, int groups, srnl_dtype in_dtype,
                                const float *gain, const float *bias, float eps, srnl_act act,
                                srnl_dtype out_dtype, void *out, float *mean, float *rstd, void *workspace,
                                size_t workspace_bytes, void *stream)
{
    srnl_set_error(SRNL_OK, "");
    srnl_status s = check_gn(B, S, C, groups, in_dtype, out_dtype, eps, act);
    if (s != SRNL_OK)
        return s;
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (B == 0 || S == 0) {
        const PtrArg ptrs[] = {{mean, "mean", true}, {rstd, "rstd", true}};
        s = check_ptrs(ptrs, 2);
        if (s == SRNL_OK)
            s = zero_fill(mean, static_cast<long long>(B) * groups, st);
        return s == SRNL_OK ? zero_fill(rstd, static_cast<long long>(B) * groups, st) : s;
    }
    if (!workspace || workspace_bytes < srnl_group_norm_fwd_workspace_bytes(B, S, C, groups))
        return fail(SRNL_ERR_WORKSPACE, "workspace smaller than srnl_group_norm_fwd_workspace_bytes");
    const PtrArg ptrs[] = {{x, "x", false},       {out, "out", false},  {gain, "gain", true},
                           {bias, "bias", true},  {mean, "mean", true}, {rstd, "rstd", true},
                           {workspace, "workspace", false}};
    s = check_ptrs(ptrs, 7);
    if (s != SRNL_OK)
        return s;
    GnArgs a = gn_args(x, B, S, C, groups, in_dtype, gain, bias, eps, act);
    a.part = static_cast<float *>(workspace);
    float *own = a.part + part_floats(a);
    a.mean = mean ? mean : own;
    a.rstd = rstd ? rstd : own + static_cast<long long>(B) * groups;
    a.out = out;
    a.obf = out_dtype == SRNL_BF16;
    SRNL_GN_LAUNCH(gn_stats_kernel, a, st);
    hipLaunchKernelGGL(gn_join_kernel, join_grid(a), dim3(256), 0, st, a);
    SRNL_GN_LAUNCH(gn_apply_kernel, a, st);
    return launched("group norm kernels");
}

size_t srnl_group_norm_bwd_workspace_bytes(int B, long long S, int C, int groups)
{
    return srnl_group_norm_fwd_workspace_bytes(B, S, C, groups);
}

srnl_status srnl_group_norm_bwd(const void *dout, srnl_dtype out_dtype, const void *x, int B, long long S, int C,
                                int groups, srnl_dtype in_dtype, const float *gain, const float *bias,
                                const float *mean, const float *rstd, srnl_act act, const void *dx_add, void *dx,
                                float *dgain, float *dbias, void *workspace, size_t workspace_bytes, void *stream)
{
    srnl_set_error(SRNL_OK, "");
    srnl_status s = check_gn(B, S, C, groups, in_dtype, out_dtype, 1.0f, act);
    if (s != SRNL_OK)
        return s;
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (B == 0 || S == 0) {              // the sums over no cells
        const PtrArg ptrs[] = {{dgain, "dgain", true}, {dbias, "dbias", true}};
        s = check_ptrs(ptrs, 2);
        if (s == SRNL_OK)
            s = zero_fill(dgain, C, st);
        return s == SRNL_OK ? zero_fill(dbias, C, st) : s;
    }
    if (!workspace || workspace_bytes < srnl_group_norm_bwd_workspace_bytes(B, S, C, groups))
        return fail(SRNL_ERR_WORKSPACE, "workspace smaller than srnl_group_norm_bwd_workspace_bytes");
    const PtrArg ptrs[] = {{dout, "dout", false},   {x, "x", false},        {dx, "dx", true},
                           {gain, "gain", true},    {bias, "bias", true},   {mean, "mean", false},
                           {rstd, "rstd", false},   {dx_add, "dx_add", true}, {dgain, "dgain", true},
                           {dbias, "dbias", true},  {workspace, "workspace", false}};
    s = check_ptrs(ptrs, 11);
    if (s != SRNL_OK)
        return s;
    GnArgs a = gn_args(x, B, S, C, groups, in_dtype, gain, bias, 1.0f, act);
    a.part = static_cast<float *>(workspace);
    a.means = a.part + part_floats(a);
    a.mean = const_cast<float *>(mean);
    a.rstd = const_cast<float *>(rstd);
    a.dout = dout;
    a.dbf = out_dtype == SRNL_BF16;
    a.add = dx_add;
    a.out = dx;
    a.obf = a.xbf;
    SRNL_GN_LAUNCH(gn_bwd_sums_kernel, a, st);
    if (dx) {
        hipLaunchKernelGGL(gn_bwd_join_kernel, join_grid(a), dim3(256), 0, st, a);
        SRNL_GN_LAUNCH(gn_bwd_apply_kernel, a, st);
    }
    s = launched("group norm backward kernels");
    if (s != SRNL_OK || (!dgain && !dbias))
        return s;
    return sum_rows(a.part, a.B * a.slabs, 2LL * C, 2LL * C, C, dgain, dbias, st);
}

}  // extern "C"
