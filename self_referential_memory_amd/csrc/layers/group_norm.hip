// group_norm.hip -- group norm with an activation over channels-last maps,
// forward and backward. Entry points as declared in include/srnl.h.
//
//   n = (x - mean) rstd, z = n gain + bias, y = act(z); mean and the biased
//   variance over the cells and channels of one item's group
//   dz = dout act'(z), d = dz gain:
//   dx = rstd (d - mean(d) - n mean(d n)) [+ add]
//   dgain = sum of dz n,  dbias = sum of dz, over items and cells
//
// Two ways. Where items and groups make enough blocks, a block takes all the cells of
// a slice of whole groups: one kernel each way, which holds the slice in registers if
// it fits and otherwise reads it again, from the L2 as far as that holds the eight items
// an XCD works on, else from the cache behind it. Else an item's map is cut into slabs of
// cells whose sums a second kernel joins and a third applies. A thread keeps a column of
// V channels and walks the cells, threads side by side along the channels, so every
// access is a wide piece of a row.
//
// 64 x 3136 x 64 bf16, slices: forward 25 us (51 MB, 2.1 TB/s), back 31 (77 MB read and
// written once, 2.5 TB/s): a slice's accesses are 16 or 32 bytes of each row. 5 x 1551 x
// 210 fp32, slabs: 5 + 7 + 6 us and 7 + 5 + 7 + 5, seven short kernels.
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
    int slice;              // channels of a slice, 0: slabs
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

// A piece as it lies in memory, at most 16 bytes: 8 channels are bf16 words, fewer
// either type's. Loads and conversions are apart, so that many loads are in flight.
template <int V> struct Held {
    uint32_t w[V == 8 ? 4 : V];
    __device__ __forceinline__ void load(const void *p, bool bf, long long o)
    {
        if (V == 8 || bf) {
            const uint16_t *q = static_cast<const uint16_t *>(p) + o;
            if constexpr (V == 8) {
                const u32x4 t = *reinterpret_cast<const u32x4 *>(q);
                w[0] = t[0], w[1] = t[1], w[2] = t[2], w[3] = t[3];
            } else if constexpr (V == 4) {
                const u32x2 t = *reinterpret_cast<const u32x2 *>(q);
                w[0] = t[0], w[1] = t[1];
            } else if constexpr (V == 2) {
                w[0] = *reinterpret_cast<const uint32_t *>(q);
            } else {
                w[0] = *q;
            }
        } else if constexpr (V < 8) {
            float v[V];
            load_piece<V>(p, false, o, v);
#pragma unroll
            for (int e = 0; e < V; ++e)
                w[e] = __float_as_uint(v[e]);
        }
    }
    __device__ __forceinline__ void get(bool bf, float (&v)[V]) const
    {
        if (V == 8 || bf) {
#pragma unroll
            for (int e = 0; e < V; ++e)
                v[e] = e & 1 ? bf16_hi(w[e / 2]) : bf16_lo(w[e / 2]);
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e)
                v[e] = __uint_as_float(w[V == 8 ? 0 : e]);
        }
    }
};
// f(k, s) for s = first, first + step and so on below last, U at a time (k = 0 .. U - 1),
// after load(k, s) of all U: in a loop over single cells the branches on type and
// activation keep each one's load behind the one before (2 x 12544 x 128 bf16 19 us
// forward and 25 back, 17 and 21 so; 64 x 3136 x 64 fp32 forward 40, 34 so).
template <int U, class L, class F>
__device__ __forceinline__ void in_batches(long long first, long long step, long long last, L load, F f)
{
    for (long long s0 = first; s0 < last; s0 += U * step) {
#pragma unroll
        for (int k = 0; k < U; ++k)
            load(k, s0 + k * step < last ? s0 + k * step : s0);
#pragma unroll
        for (int k = 0; k < U; ++k)
            if (s0 + k * step < last)
                f(k, s0 + k * step);
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

// Cells of a slab that lane l walks.
struct Shares {
    long long each;
    int more;               // the first lanes have one more
    __device__ __forceinline__ Shares(long long cells, int lanes)
        : each(cells / lanes), more(static_cast<int>(cells - each * lanes))
    {
    }
    __device__ __forceinline__ long long of(int l) const { return each + (l < more); }
    __device__ __forceinline__ float part(int l, float cells) const { return static_cast<float>(of(l)) / cells; }
};

// Mean and sum of squares about it, per channel of a slab. A thread takes four cells
// at a time: their mean and their squares about it, from distances to the first of them;
// then joins them (m cells) to what it has (n cells): with d the distance of the means,
// the mean moves by d m / (n + m) and the squares grow by d^2 n m / (n + m). The mean is
// two floats. So neither an offset nor a cell far out costs digits: what is lost is a
// rounding a batch of the squares. (Sums about the first cell, less their mean's square,
// lose 2e-3 of 1400 cells' squares where that one lies 1000 deviations out.)
template <int V> __global__ __launch_bounds__(256) void gn_stats_kernel(GnArgs a)
{
    __shared__ float lds[256][2 * V];
    const Place<V> pl(a);
    const long long cells = pl.last - pl.first;
    const Shares shares(cells, pl.lanes);
    if (pl.live) {
        float hi[V], lo[V], m2[V], n = 0.0f;
#pragma unroll
        for (int e = 0; e < V; ++e)
            hi[e] = lo[e] = m2[e] = 0.0f;
        for (long long s0 = pl.first + pl.lane; s0 < pl.last; s0 += 4 * pl.lanes) {
            Held<V> x[4];
            float v[4][V], m = 0.0f;
            bool on[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const long long s = s0 + k * pl.lanes;
                on[k] = s < pl.last;
                x[k].load(a.x, a.xbf, pl.at(a, on[k] ? s : s0));
                m += on[k] ? 1.0f : 0.0f;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
                x[k].get(a.xbf, v[k]);
            const float each = 1.0f / m, w = m / (n + m), both = n * w;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                float d[4], of = 0.0f, b2 = 0.0f;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    d[k] = v[k][e] - v[0][e];
                    of += on[k] ? d[k] : 0.0f;
                }
                of *= each;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float y = on[k] ? d[k] - of : 0.0f;
                    b2 = fmaf(y, y, b2);
                }
                const float from = n > 0.0f ? hi[e] : v[0][e];
                const float y = ((v[0][e] - from) - lo[e]) + of, step = y * w, to = from + step;
                lo[e] += (from - to) + step;
                hi[e] = to;
                m2[e] += fmaf(y * both, y, b2);
            }
            n += m;
        }
#pragma unroll
        for (int e = 0; e < V; ++e) {
            lds[threadIdx.x][e] = hi[e] + lo[e];
            lds[threadIdx.x][V + e] = m2[e];
        }
    }
    __syncthreads();
    const int wide = pl.wide(a);
    float *part = a.part + (static_cast<long long>(pl.b) * a.slabs + blockIdx.x / a.tiles % a.slabs) * 2 * a.C;
    const int c0 = blockIdx.x % a.tiles * 256 * V;
    for (int j = threadIdx.x; j < wide * V && c0 + j < a.C; j += 256) {
        const int piece = j / V, e = j % V;
        // about the first lane's mean, so that a constant map's mean is exact; lanes
        // are full (or one cell short) but where the slab has fewer cells than lanes
        const float ref = lds[piece][e], all = static_cast<float>(cells);
        const float w0 = shares.part(pl.lanes - 1, all), w1 = shares.part(0, all);
        const float n0 = static_cast<float>(shares.of(pl.lanes - 1)), n1 = static_cast<float>(shares.of(0));
        const int used = shares.each ? pl.lanes : shares.more;
        float mean = 0.0f, m2 = 0.0f;
#pragma unroll 8
        for (int l = 0; l < used; ++l)
            mean = fmaf(lds[l * wide + piece][e] - ref, l < shares.more ? w1 : w0, mean);
        mean += ref;
#pragma unroll 8
        for (int l = 0; l < used; ++l) {
            const float d = lds[l * wide + piece][e] - mean;
            m2 += fmaf((l < shares.more ? n1 : n0) * d, d, lds[l * wide + piece][V + e]);
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

// f(row, channel) over rows x channels by the threads i of n side by side along the
// channels (no division inside, loads in flight together)
template <class F> __device__ __forceinline__ void each_of_group(int i, int n, int rows, int channels, F f)
{
    const int wide = channels < n ? channels : n, high = n / wide;
    const int r0 = i / wide, c0 = i - r0 * wide;
    if (r0 < high)
        for (int c = c0; c < channels; c += wide)
#pragma unroll 8
            for (int r = r0; r < rows; r += high)
                f(r, c);
}
// A block joins one group's channels and slabs. There may be few groups and much of
// each: with 256 threads 3 x 2 groups of 268 slabs x 183 channels take 37 us, with
// 1024 20 (5 x 7 of 97 x 30: 7.3 and 6.8).
constexpr int JOIN_THREADS = 1024;
// the sum over such a block
__device__ __forceinline__ float block_sum(float v, float (&red)[JOIN_THREADS / 64])
{
    v = wave_sum(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0)
        red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int w = 0; w < JOIN_THREADS / 64; ++w)
        v += red[w];
    return v;
}

__global__ __launch_bounds__(JOIN_THREADS) void gn_join_kernel(GnArgs a)
{
    __shared__ float red[JOIN_THREADS / 64];
    const int group = blockIdx.x, b = group / a.G, cpg = a.C / a.G, c0 = group % a.G * cpg;
    const float *part = a.part + static_cast<long long>(b) * a.slabs * 2 * a.C;
    const float total = static_cast<float>(a.S) * static_cast<float>(cpg);
    const float ref = part[c0];
    const float whole = static_cast<float>(a.rows), rest = static_cast<float>(a.S - (a.slabs - 1) * a.rows);
    float mean = 0.0f;
    each_of_group(threadIdx.x, JOIN_THREADS, a.slabs, cpg, [&](int r, int c) {
        mean = fmaf(part[r * 2LL * a.C + c0 + c] - ref, (r + 1 < a.slabs ? whole : rest) / total, mean);
    });
    mean = ref + block_sum(mean, red);
    float m2 = 0.0f;
    each_of_group(threadIdx.x, JOIN_THREADS, a.slabs, cpg, [&](int r, int c) {
        const float d = part[r * 2LL * a.C + c0 + c] - mean;
        m2 += fmaf((r + 1 < a.slabs ? whole : rest) * d, d, part[r * 2LL * a.C + a.C + c0 + c]);
    });
    m2 = block_sum(m2, red);
    if (threadIdx.x == 0) {
        a.mean[group] = mean;
        a.rstd[group] = 1.0f / sqrtf(m2 / total + a.eps);
    }
}

// The groups of V channels from c on, counted from channel 0 (one division).
template <int V> struct Groups {
    int g[V];
    __device__ __forceinline__ Groups(int c, int cpg)
    {
        int of = c / cpg, in = c - of * cpg;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            g[e] = of;
            if (++in == cpg) {
                in = 0;
                ++of;
            }
        }
    }
};
// V channels' parameters, `other` without any
template <int V> __device__ __forceinline__ void load_channels(const float *p, int c, float other, float (&v)[V])
{
    if (p) {
        load_piece<V>(p, false, c, v);
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e)
            v[e] = other;
    }
}

// What a thread keeps of its channels: n = (x - mean) rstd, z = n gain + bias.
template <int V> struct Channels {
    float mean[V], rstd[V], gain[V], bias[V];
    __device__ __forceinline__ Channels(const GnArgs &a, const Place<V> &pl)
    {
        const Groups<V> gr(pl.c, a.C / a.G);
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const long long group = static_cast<long long>(pl.b) * a.G + gr.g[e];
            mean[e] = a.mean[group];
            rstd[e] = a.rstd[group];
        }
        load_channels<V>(a.gain, pl.c, 1.0f, gain);
        load_channels<V>(a.bias, pl.c, 0.0f, bias);
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
    Held<V> x[4];
    in_batches<4>(
        pl.first + pl.lane, pl.lanes, pl.last,
        [&](int k, long long s) __attribute__((always_inline)) { x[k].load(a.x, a.xbf, pl.at(a, s)); },
        [&](int k, long long s) __attribute__((always_inline)) {
            float v[V];
            x[k].get(a.xbf, v);
#pragma unroll
            for (int e = 0; e < V; ++e)
                v[e] = fmaf((v[e] - ch.mean[e]) * ch.rstd[e], ch.gain[e], ch.bias[e]);
            act_piece<V>(v, a.act);
            store_piece<V>(a.out, a.obf, pl.at(a, s), v);
        });
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
        Held<V> x[4], dy[4];
        in_batches<4>(
            pl.first + pl.lane, pl.lanes, pl.last,
            [&](int k, long long s) __attribute__((always_inline)) {
                x[k].load(a.x, a.xbf, pl.at(a, s));
                dy[k].load(a.dout, a.dbf, pl.at(a, s));
            },
            [&](int k, long long) __attribute__((always_inline)) {
                float v[V], d[V], z[V];
                x[k].get(a.xbf, v);
                dy[k].get(a.dbf, d);
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
            });
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

__global__ __launch_bounds__(JOIN_THREADS) void gn_bwd_join_kernel(GnArgs a)
{
    __shared__ float red[JOIN_THREADS / 64];
    const int group = blockIdx.x, b = group / a.G, cpg = a.C / a.G, c0 = group % a.G * cpg;
    const float *part = a.part + static_cast<long long>(b) * a.slabs * 2 * a.C;
    float sn = 0.0f, sd = 0.0f;
    each_of_group(threadIdx.x, JOIN_THREADS, a.slabs, cpg, [&](int r, int c) {
        const float *p = part + r * 2LL * a.C + c0 + c;
        const float gain = a.gain ? a.gain[c0 + c] : 1.0f;
        sn = fmaf(p[0], gain, sn);
        sd = fmaf(p[a.C], gain, sd);
    });
    sn = block_sum(sn, red);
    sd = block_sum(sd, red);
    if (threadIdx.x == 0) {
        const float total = static_cast<float>(a.S) * static_cast<float>(cpg);
        a.means[2LL * group] = sd / total;
        a.means[2LL * group + 1] = sn / total;
    }
}

template <int V> __global__ __launch_bounds__(256) void gn_bwd_apply_kernel(GnArgs a)
{
    const Place<V> pl(a);
    if (!pl.live)
        return;
    const Channels<V> ch(a, pl);
    float md[V], mn[V];
    const Groups<V> gr(pl.c, a.C / a.G);
#pragma unroll
    for (int e = 0; e < V; ++e) {
        const long long group = static_cast<long long>(pl.b) * a.G + gr.g[e];
        md[e] = a.means[2LL * group];
        mn[e] = a.means[2LL * group + 1];
    }
    Held<V> x[4], dy[4], add[4];
    in_batches<4>(
        pl.first + pl.lane, pl.lanes, pl.last,
        [&](int k, long long s) __attribute__((always_inline)) {
            x[k].load(a.x, a.xbf, pl.at(a, s));
            dy[k].load(a.dout, a.dbf, pl.at(a, s));
            if (a.add)
                add[k].load(a.add, a.xbf, pl.at(a, s));
        },
        [&](int k, long long s) __attribute__((always_inline)) {
            float v[V], d[V], z[V], w[V];
            x[k].get(a.xbf, v);
            dy[k].get(a.dbf, d);
            if (a.add)
                add[k].get(a.xbf, w);
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
        });
}

// ------------------------------------------------------------------ slices

constexpr int SLICE_THREADS = 512;

// A block's slice: all cells of `slice` channels of one item. Of every eight items
// each goes to one XCD (blocks go round the eight), so that slices that share cache
// lines share an L2.
template <int V> struct Slice {
    int b, c0, c, lanes, lane, used;
    bool live;
    __device__ __forceinline__ explicit Slice(const GnArgs &a)
    {
        const int slices = a.C / a.slice, full = a.B / 8 * 8;
        const int i = blockIdx.x, rest = i - full * slices;
        b = rest < 0 ? i % 8 + i / (8 * slices) * 8 : full + rest / slices;
        c0 = (rest < 0 ? i / 8 % slices : rest % slices) * a.slice;
        const int wide = a.slice / V;
        lanes = SLICE_THREADS / wide;
        lane = threadIdx.x / wide;
        c = c0 + V * (threadIdx.x % wide);
        used = a.S < lanes ? static_cast<int>(a.S) : lanes;      // lanes that have cells
        live = lane < used;
    }
    __device__ __forceinline__ long long at(const GnArgs &a, long long s) const { return (b * a.S + s) * a.C + c; }
};

// The slice's cells as a thread walks them: its NV pieces are held, or (NV = 0) each
// is read whenever it is wanted.
template <int V, int NV> struct Cells {
    Held<V> v[NV > 0 ? NV : 1];
    __device__ __forceinline__ void load(const GnArgs &a, const Slice<V> &sl, const void *p, bool bf)
    {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const long long s = sl.lane + static_cast<long long>(k) * sl.lanes;
            if (sl.live && s < a.S)
                v[k].load(p, bf, sl.at(a, s));
        }
    }
};
// f(piece, cell) for every cell of this thread
template <int V, int NV, class F>
__device__ __forceinline__ void each_cell(const GnArgs &a, const Slice<V> &sl, const Cells<V, NV> &x, F f)
{
    float v[V];
    if constexpr (NV > 0) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const long long s = sl.lane + static_cast<long long>(k) * sl.lanes;
            if (sl.live && s < a.S) {
                x.v[k].get(a.xbf, v);
                f(v, s);
            }
        }
    } else if (sl.live) {
        Held<V> h[4];
        in_batches<4>(
            sl.lane, sl.lanes, a.S,
            [&](int k, long long s) __attribute__((always_inline)) { h[k].load(a.x, a.xbf, sl.at(a, s)); },
            [&](int k, long long s) __attribute__((always_inline)) {
                h[k].get(a.xbf, v);
                f(v, s);
            });
    }
}
template <int V, int NV, class F>
__device__ __forceinline__ void each_cell(const GnArgs &a, const Slice<V> &sl, const Cells<V, NV> &x,
                                          const Cells<V, NV> &d, F f)
{
    float v[V], w[V];
    if constexpr (NV > 0) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const long long s = sl.lane + static_cast<long long>(k) * sl.lanes;
            if (sl.live && s < a.S) {
                x.v[k].get(a.xbf, v);
                d.v[k].get(a.dbf, w);
                f(v, w, s);
            }
        }
    } else if (sl.live) {
        Held<V> h[2], g[2];
        in_batches<2>(
            sl.lane, sl.lanes, a.S,
            [&](int k, long long s) __attribute__((always_inline)) {
                h[k].load(a.x, a.xbf, sl.at(a, s));
                g[k].load(a.dout, a.dbf, sl.at(a, s));
            },
            [&](int k, long long s) __attribute__((always_inline)) {
                h[k].get(a.xbf, v);
                g[k].get(a.dbf, w);
                f(v, w, s);
            });
    }
}

// Sums over a block, per group of its slice: every thread's V channels' terms go to
// buf [used lanes][slice]; a wave adds up a group's.
template <int V>
__device__ __forceinline__ void group_totals(const GnArgs &a, const Slice<V> &sl, const float (&t)[V], float *buf,
                                             float *totals)
{
    __syncthreads();
    if (sl.live)
#pragma unroll
        for (int e = 0; e < V; ++e)
            buf[sl.lane * a.slice + sl.c - sl.c0 + e] = t[e];
    __syncthreads();
    const int cpg = a.C / a.G, wave = threadIdx.x >> 6;
    for (int g = wave; g < a.slice / cpg; g += SLICE_THREADS / 64) {
        float s = 0.0f;
        each_of_group(threadIdx.x & 63, 64, sl.used, cpg, [&](int r, int c) { s += buf[r * a.slice + g * cpg + c]; });
        s = wave_sum(s);
        if ((threadIdx.x & 63) == 0)
            totals[g] = s;
    }
    __syncthreads();
}

__device__ __forceinline__ long long b_first(const GnArgs &a, int b, int c) { return b * a.S * a.C + c; }

template <int V, int NV> __global__ __launch_bounds__(SLICE_THREADS) void gn_slice_kernel(GnArgs a)
{
    __shared__ float buf[SLICE_THREADS * V], totals[SLICE_THREADS * V], firsts[SLICE_THREADS * V];
    const Slice<V> sl(a);
    const int cpg = a.C / a.G, groups = a.slice / cpg;
    const Groups<V> gr(sl.c - sl.c0, cpg);
    Cells<V, NV> x;
    x.load(a, sl, a.x, a.xbf);
    // Distances from the group's first value, so that a constant group's mean is
    // exact and an offset costs no digits; then squares of distances from the mean.
    for (int g = threadIdx.x; g < groups; g += SLICE_THREADS) {
        float v[1];
        load_piece<1>(a.x, a.xbf, b_first(a, sl.b, sl.c0 + g * cpg), v);
        firsts[g] = v[0];
    }
    __syncthreads();
    const float n = static_cast<float>(a.S) * static_cast<float>(cpg);
    float mean[V], rstd[V], t[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
        t[e] = 0.0f;
        mean[e] = sl.live ? firsts[gr.g[e]] : 0.0f;
    }
    each_cell<V, NV>(a, sl, x, [&](const float (&v)[V], long long) __attribute__((always_inline)) {
#pragma unroll
        for (int e = 0; e < V; ++e)
            t[e] += v[e] - mean[e];
    });
    group_totals<V>(a, sl, t, buf, totals);
#pragma unroll
    for (int e = 0; e < V; ++e) {
        t[e] = 0.0f;
        if (sl.live)
            mean[e] += totals[gr.g[e]] / n;
    }
    if (threadIdx.x < static_cast<unsigned>(groups) && a.mean)
        a.mean[static_cast<long long>(sl.b) * a.G + sl.c0 / cpg + threadIdx.x] = firsts[threadIdx.x] + totals[threadIdx.x] / n;
    each_cell<V, NV>(a, sl, x, [&](const float (&v)[V], long long) __attribute__((always_inline)) {
#pragma unroll
        for (int e = 0; e < V; ++e)
            t[e] = fmaf(v[e] - mean[e], v[e] - mean[e], t[e]);
    });
    group_totals<V>(a, sl, t, buf, totals);
    if (threadIdx.x < static_cast<unsigned>(groups) && a.rstd)
        a.rstd[static_cast<long long>(sl.b) * a.G + sl.c0 / cpg + threadIdx.x] = 1.0f / sqrtf(totals[threadIdx.x] / n + a.eps);
    if (!sl.live)
        return;
    float gain[V], bias[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
        rstd[e] = 1.0f / sqrtf(totals[gr.g[e]] / n + a.eps);
    }
    load_channels<V>(a.gain, sl.c, 1.0f, gain);
    load_channels<V>(a.bias, sl.c, 0.0f, bias);
    each_cell<V, NV>(a, sl, x, [&](const float (&v)[V], long long s) __attribute__((always_inline)) {
        float y[V];
#pragma unroll
        for (int e = 0; e < V; ++e)
            y[e] = fmaf((v[e] - mean[e]) * rstd[e], gain[e], bias[e]);
        act_piece<V>(y, a.act);
        store_piece<V>(a.out, a.obf, sl.at(a, s), y);
    });
}

template <int V, int NV> __global__ __launch_bounds__(SLICE_THREADS) void gn_slice_bwd_kernel(GnArgs a)
{
    __shared__ float buf[2][SLICE_THREADS * V], sums[2][SLICE_THREADS * V];
    const Slice<V> sl(a);
    const int cpg = a.C / a.G;
    Cells<V, NV> x, d;
    x.load(a, sl, a.x, a.xbf);
    d.load(a, sl, a.dout, a.dbf);
    const Groups<V> gr(sl.c - sl.c0, cpg);
    float mean[V], rstd[V], gain[V], bias[V], tn[V], td[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
        tn[e] = td[e] = 0.0f;
        mean[e] = rstd[e] = gain[e] = bias[e] = 0.0f;
        if (sl.live) {
            const long long group = static_cast<long long>(sl.b) * a.G + sl.c0 / cpg + gr.g[e];
            mean[e] = a.mean[group];
            rstd[e] = a.rstd[group];
        }
    }
    if (sl.live) {
        load_channels<V>(a.gain, sl.c, 1.0f, gain);
        load_channels<V>(a.bias, sl.c, 0.0f, bias);
    }
    // n and dz of a cell
    const auto form = [&](const float (&v)[V], const float (&w)[V], float (&n)[V], float (&dz)[V]) __attribute__((always_inline)) {
        float z[V];
#pragma unroll
        for (int e = 0; e < V; ++e) {
            n[e] = (v[e] - mean[e]) * rstd[e];
            z[e] = fmaf(n[e], gain[e], bias[e]);
            dz[e] = w[e];
        }
        slope_piece<V>(z, a.act, dz);
    };
    each_cell<V, NV>(a, sl, x, d, [&](const float (&v)[V], const float (&w)[V], long long) __attribute__((always_inline)) {
        float n[V], dz[V];
        form(v, w, n, dz);
#pragma unroll
        for (int e = 0; e < V; ++e) {
            tn[e] = fmaf(dz[e], n[e], tn[e]);
            td[e] += dz[e];
        }
    });
    if (sl.live)
#pragma unroll
        for (int e = 0; e < V; ++e) {
            buf[0][sl.lane * a.slice + sl.c - sl.c0 + e] = tn[e];
            buf[1][sl.lane * a.slice + sl.c - sl.c0 + e] = td[e];
        }
    __syncthreads();
    // a channel's sums: a wave each
    for (int i = threadIdx.x >> 6; i < 2 * a.slice; i += SLICE_THREADS / 64) {
        const int which = i >= a.slice, c = i - which * a.slice;
        float s = 0.0f;
        for (int l = threadIdx.x & 63; l < sl.used; l += 64)
            s += buf[which][l * a.slice + c];
        s = wave_sum(s);
        if ((threadIdx.x & 63) == 0) {
            sums[which][c] = s;
            if (a.part)
                a.part[static_cast<long long>(sl.b) * 2 * a.C + which * a.C + sl.c0 + c] = s;
        }
    }
    __syncthreads();
    if (!a.out)
        return;
    // a group's means: its channels' sums times their gains
    for (int g = threadIdx.x; g < a.slice / cpg; g += SLICE_THREADS) {
        float sn = 0.0f, sd = 0.0f;
        for (int c = g * cpg; c < (g + 1) * cpg; ++c) {
            const float w = a.gain ? a.gain[sl.c0 + c] : 1.0f;
            sn = fmaf(sums[0][c], w, sn);
            sd = fmaf(sums[1][c], w, sd);
        }
        const float n = static_cast<float>(a.S) * static_cast<float>(cpg);
        buf[0][g] = sn / n;
        buf[1][g] = sd / n;
    }
    __syncthreads();
    if (!sl.live)
        return;
    float mn[V], md[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
        mn[e] = buf[0][gr.g[e]];
        md[e] = buf[1][gr.g[e]];
    }
    each_cell<V, NV>(a, sl, x, d, [&](const float (&v)[V], const float (&w)[V], long long s) __attribute__((always_inline)) {
        float n[V], dz[V];
        form(v, w, n, dz);
#pragma unroll
        for (int e = 0; e < V; ++e)
            n[e] = rstd[e] * (dz[e] * gain[e] - md[e] - n[e] * mn[e]);
        if (a.add) {
            float add[V];
            load_piece<V>(a.add, a.xbf, sl.at(a, s), add);
#pragma unroll
            for (int e = 0; e < V; ++e)
                n[e] += add[e];
        }
        store_piece<V>(a.out, a.obf, sl.at(a, s), n);
    });
}

// ------------------------------------------------------------------ launches

// The widest piece that divides a row.
int piece_of(int C) { return C % 8 == 0 ? 8 : C % 4 == 0 ? 4 : C % 2 == 0 ? 2 : 1; }

// The kernels' pieces are 16 bytes at most of the wider type that they read.
int read_piece(const GnArgs &a)
{
    const int v = piece_of(a.C);
    return v == 8 && !(a.xbf && (!a.dout || a.dbf)) ? 4 : v;
}
// The pieces of V channels that a thread holds of a slice of w, 0: it reads them again.
// Backward there are two arrays to hold: eight pieces of each are slower than reading
// again in slices of 8 channels (64 x 3136 x 64 bf16 39.8 us, 30.9), and as fast in the
// wider ones chosen (64 x 1568 x 64 18.5 and 18.6, 64 x 784 x 128 21.2 and 20.6).
int held(long long S, int w, int v, bool backward = false)
{
    const int lanes = SLICE_THREADS / (w / v);
    return S <= 2LL * lanes ? 2 : S <= 8LL * lanes && !backward ? 8 : 0;
}
// The slice: whole groups and pieces. None (slabs instead) where it is wider than a block's
// threads, or where the slices are too few to fill the card and long: forward and
// back, 32 slices of 2048 cells of 8 take 26 us (slabs 36), 16 of 3136 32 us (45), but
// 32 of 4096 in fp32 68 us (38) and 35 of 1551 cells of 30 102 us (40). The same for
// every type: pieces of 4 at most are counted.
void cut_slices(GnArgs &a)
{
    const int v = piece_of(a.C), v4 = v < 4 ? v : 4, cpg = a.C / a.G;
    int w = cpg;
    while (w % v)
        w += cpg;
    a.slice = 0;
    if (w / v4 > SLICE_THREADS)
        return;
    if (static_cast<long long>(a.B) * (a.C / w) < 128 && a.S > 14LL * (SLICE_THREADS / (w / v4)))
        return;
    a.slice = w;
}
// ... made wider, for longer pieces of a row, while that leaves a block for every CU
// and forward the cells in registers: 64 x 196 x 256 bf16 in slices of 16 takes 19 us
// forward and 25 back, of 64 11 and 21; but 64 x 784 x 128 fp32 of 16, held, 15 us
// forward, of 32 20.
void widen_slices(GnArgs &a)
{
    const int v = read_piece(a);
    while (a.C % (2 * a.slice) == 0 && static_cast<long long>(a.B) * (a.C / (2 * a.slice)) >= 256 &&
           2 * a.slice <= 64 && (a.dout || held(a.S, 2 * a.slice, v) || !held(a.S, a.slice, v)))
        a.slice *= 2;
}

// Slabs of at least 8 cells a lane, as many as make about 4 blocks per CU.
void cut_map(GnArgs &a)
{
    const int pieces = a.C / piece_of(a.C);
    const int lanes = pieces < 256 ? 256 / pieces : 1;
    const long long most = (a.S + 8LL * lanes - 1) / (8LL * lanes);
    const long long items = static_cast<long long>(a.B) * ((pieces + 255) / 256);
    long long slabs = (1024 + items - 1) / items;
    slabs = slabs < most ? slabs : most;
    a.rows = (a.S + slabs - 1) / slabs;
    a.slabs = static_cast<int>((a.S + a.rows - 1) / a.rows);
}

// slices take none forward; backward a sum of every item's channels
size_t part_floats(const GnArgs &a) { return static_cast<size_t>(a.B) * (a.slice ? 1 : a.slabs) * 2 * a.C; }
size_t group_floats(const GnArgs &a) { return 2 * static_cast<size_t>(a.B) * a.G; }

#define SRNL_GN_LAUNCH(kernel, a, st)                                                                  \
    do {                                                                                               \
        (a).tiles = ((a).C / read_piece(a) + 255) / 256;                                               \
        const dim3 grid(static_cast<unsigned>(static_cast<long long>((a).B) * (a).slabs * (a).tiles)); \
        switch (read_piece(a)) {                                                                       \
        case 8: hipLaunchKernelGGL(kernel<8>, grid, dim3(256), 0, st, a); break;                       \
        case 4: hipLaunchKernelGGL(kernel<4>, grid, dim3(256), 0, st, a); break;                       \
        case 2: hipLaunchKernelGGL(kernel<2>, grid, dim3(256), 0, st, a); break;                       \
        default: hipLaunchKernelGGL(kernel<1>, grid, dim3(256), 0, st, a); break;                      \
        }                                                                                              \
    } while (0)

#define SRNL_GN_SLICE_NV(kernel, V, MORE, a, st)                                                       \
    do {                                                                                               \
        const dim3 grid(static_cast<unsigned>(static_cast<long long>((a).B) * ((a).C / (a).slice)));   \
        const int nv = held((a).S, (a).slice, V, (a).dout != nullptr);                                 \
        if (nv == 2)                                                                                   \
            hipLaunchKernelGGL((kernel<V, 2>), grid, dim3(SLICE_THREADS), 0, st, a);                   \
        else if (nv == MORE)                                                                           \
            hipLaunchKernelGGL((kernel<V, MORE>), grid, dim3(SLICE_THREADS), 0, st, a);                \
        else                                                                                           \
            hipLaunchKernelGGL((kernel<V, 0>), grid, dim3(SLICE_THREADS), 0, st, a);                   \
    } while (0)
#define SRNL_GN_SLICE(kernel, MORE, a, st)                    \
    switch (read_piece(a)) {                                 \
    case 8: SRNL_GN_SLICE_NV(kernel, 8, MORE, a, st); break;  \
    case 4: SRNL_GN_SLICE_NV(kernel, 4, MORE, a, st); break;  \
    case 2: SRNL_GN_SLICE_NV(kernel, 2, MORE, a, st); break;  \
    default: SRNL_GN_SLICE_NV(kernel, 1, MORE, a, st); break; \
    }

dim3 join_grid(const GnArgs &a)
{
    return dim3(static_cast<unsigned>(a.B * a.G));
}

srnl_status check_gn(int B, long long S, int C, int G, srnl_dtype x, srnl_dtype out, float eps, int act)
{
    if (B < 0 || S < 0)
        return fail(SRNL_ERR_ARG, "B and S must be >= 0");
    if (C < 1 || G < 1 || C % G)
        return fail(SRNL_ERR_ARG, "C must be >= 1 and a multiple of groups");
    if (C > 1 << 20 || static_cast<__int128>(B) * S * C >= (static_cast<__int128>(1) << 60) || S >= 1LL << 40)
        return fail(SRNL_ERR_ARG, "map too large");
    // an item and tile of channels is a block, and so is a group; a slice is one of 512
    // threads, of which a launch takes 2^32 - 1: maps of one channel have 2^23 slices
    if (static_cast<__int128>(B) * C > (C == 1 ? (1 << 23) - 1 : 1 << 23))
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
    cut_slices(a);
    if (!a.slice)
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
    return a.slice ? 0 : (part_floats(a) + group_floats(a)) * sizeof(float);
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
    GnArgs a = gn_args(x, B, S, C, groups, in_dtype, gain, bias, eps, act);
    if (!a.slice && (!workspace || workspace_bytes < srnl_group_norm_fwd_workspace_bytes(B, S, C, groups)))
        return fail(SRNL_ERR_WORKSPACE, "workspace smaller than srnl_group_norm_fwd_workspace_bytes");
    const PtrArg ptrs[] = {{x, "x", false},       {out, "out", false},  {gain, "gain", true},
                           {bias, "bias", true},  {mean, "mean", true}, {rstd, "rstd", true},
                           {a.slice ? nullptr : workspace, "workspace", true}};
    s = check_ptrs(ptrs, 7);
    if (s != SRNL_OK)
        return s;
    a.out = out;
    a.obf = out_dtype == SRNL_BF16;
    if (a.slice) {
        a.mean = mean;
        a.rstd = rstd;
        widen_slices(a);
        SRNL_GN_SLICE(gn_slice_kernel, 8, a, st);
        return launched("gn_slice_kernel");
    }
    a.part = static_cast<float *>(workspace);
    float *own = a.part + part_floats(a);
    a.mean = mean ? mean : own;
    a.rstd = rstd ? rstd : own + static_cast<long long>(B) * groups;
    SRNL_GN_LAUNCH(gn_stats_kernel, a, st);
    hipLaunchKernelGGL(gn_join_kernel, join_grid(a), dim3(JOIN_THREADS), 0, st, a);
    SRNL_GN_LAUNCH(gn_apply_kernel, a, st);
    return launched("group norm kernels");
}

size_t srnl_group_norm_bwd_workspace_bytes(int B, long long S, int C, int groups)
{
    if (check_gn(B, S, C, groups, SRNL_F32, SRNL_F32, 1.0f, 0) != SRNL_OK || B == 0 || S == 0)
        return 0;
    const GnArgs a = gn_args(nullptr, B, S, C, groups, SRNL_F32, nullptr, nullptr, 1.0f, 0);
    return (part_floats(a) + (a.slice ? 0 : group_floats(a))) * sizeof(float);
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
    if (a.slice) {
        widen_slices(a);
        SRNL_GN_SLICE(gn_slice_bwd_kernel, 2, a, st);
        s = launched("gn_slice_bwd_kernel");
        if (s != SRNL_OK || (!dgain && !dbias))
            return s;
        return sum_rows(a.part, a.B, 2LL * C, 2LL * C, C, dgain, dbias, st);
    }
    SRNL_GN_LAUNCH(gn_bwd_sums_kernel, a, st);
    if (dx) {
        hipLaunchKernelGGL(gn_bwd_join_kernel, join_grid(a), dim3(JOIN_THREADS), 0, st, a);
        SRNL_GN_LAUNCH(gn_bwd_apply_kernel, a, st);
    }
    s = launched("group norm backward kernels");
    if (s != SRNL_OK || (!dgain && !dbias))
        return s;
    return sum_rows(a.part, a.B * a.slabs, 2LL * C, 2LL * C, C, dgain, dbias, st);
}

}  // extern "C"
