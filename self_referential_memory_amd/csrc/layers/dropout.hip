// dropout.hip -- dropout whose mask is a function of the seed, the offset and
// the element's place, so that neither pass stores it. Entry points as
// declared in include/srnl.h.
//
// Element n takes 16 of the 128 bits of block n / 8 of Philox4x32-10: one
// block, 20 wide multiplications, serves the 8 elements that a thread moves.
// With 32 bits an element the multiplications, a quarter of the card's rate
// each, would take as long as bf16 elements take to move. 200704 x 64 bf16 with a
// residual takes 14.5 us (5.3 TB/s), its gradient 11.2 (4.6).
#include "common.h"

namespace {

using namespace srnl_i;

struct DropArgs {
    const void *x, *add;
    void *out;
    long long n;
    bool xbf, abf, obf;
    unsigned cut;             // dropped below this, of 65536
    float up;                 // 65536 / (65536 - cut)
    unsigned long long seed, offset;
    const unsigned long long *counter;
};

__device__ __forceinline__ u32x4 philox(unsigned long long block, unsigned long long offset,
                                        unsigned long long seed)
{
    uint32_t c0 = static_cast<uint32_t>(block), c1 = static_cast<uint32_t>(block >> 32);
    uint32_t c2 = static_cast<uint32_t>(offset), c3 = static_cast<uint32_t>(offset >> 32);
    uint32_t k0 = static_cast<uint32_t>(seed), k1 = static_cast<uint32_t>(seed >> 32);
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t p0 = static_cast<uint64_t>(c0) * 0xD2511F53u, p1 = static_cast<uint64_t>(c2) * 0xCD9E8D57u;
        c0 = static_cast<uint32_t>(p1 >> 32) ^ c1 ^ k0;
        c1 = static_cast<uint32_t>(p1);
        c2 = static_cast<uint32_t>(p0 >> 32) ^ c3 ^ k1;
        c3 = static_cast<uint32_t>(p0);
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return u32x4{c0, c1, c2, c3};
}

__global__ __launch_bounds__(256) void dropout_kernel(DropArgs a)
{
    const unsigned long long offset = a.offset + (a.counter ? *a.counter : 0);
    const long long pieces = (a.n + 7) / 8;
    for (long long i = blockIdx.x * 256LL + threadIdx.x; i < pieces; i += 256LL * gridDim.x) {
        const long long o = 8 * i;
        const int live = a.n - o < 8 ? static_cast<int>(a.n - o) : 8;
        float v[8], w[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        // whole pieces are aligned; the last one may be short
        if (live == 8) {
            load_row<8, true>(a.x, a.xbf, o, 8, v);
            if (a.add)
                load_row<8, true>(a.add, a.abf, o, 8, w);
        } else {
            load_row<8, false>(a.x, a.xbf, o, live, v);
            if (a.add)
                load_row<8, false>(a.add, a.abf, o, live, w);
        }
        const u32x4 r = philox(i, offset, a.seed);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t bits = e & 1 ? r[e / 2] >> 16 : r[e / 2] & 0xFFFFu;
            // chosen, not multiplied: what is dropped may be infinite
            const float y = bits >= a.cut ? v[e] * a.up : 0.0f;
            v[e] = a.add ? y + w[e] : y;
        }
        if (live == 8)
            store_row<8, true>(a.out, a.obf, o, 8, v);
        else
            store_row<8, false>(a.out, a.obf, o, live, v);
    }
}

srnl_status run_dropout(const void *x, srnl_dtype in_dtype, long long n, double p, unsigned long long seed,
                        unsigned long long offset, const unsigned long long *counter, const void *add,
                        srnl_dtype add_dtype, srnl_dtype out_dtype, void *out, const char *names[3], void *stream)
{
    srnl_set_error(SRNL_OK, "");
    if (n < 0 || n >= 1LL << 60)
        return fail(SRNL_ERR_ARG, "n must be >= 0 and below 2^60");
    if (!(p >= 0.0f && p < 1.0f))
        return fail(SRNL_ERR_ARG, "p must be in [0, 1)");
    if (!valid_dtype(in_dtype) || !valid_dtype(out_dtype) || (add && !valid_dtype(add_dtype)))
        return fail(SRNL_ERR_DTYPE, "dtype must be SRNL_F32 or SRNL_BF16");
    if (n == 0)
        return SRNL_OK;
    const PtrArg ptrs[] = {{x, names[0], false}, {out, names[1], false}, {add, names[2], true},
                           {counter, "counter", true}};
    const srnl_status s = check_ptrs(ptrs, 4);
    if (s != SRNL_OK)
        return s;
    DropArgs a = {};
    a.x = x;
    a.add = add;
    a.out = out;
    a.n = n;
    a.xbf = in_dtype == SRNL_BF16;
    a.abf = add_dtype == SRNL_BF16;
    a.obf = out_dtype == SRNL_BF16;
    const unsigned cut = static_cast<unsigned>(std::floor(p * 65536.0 + 0.5));
    a.cut = cut < 65535u ? cut : 65535u;
    a.up = 65536.0f / static_cast<float>(65536u - a.cut);
    a.seed = seed;
    a.offset = offset;
    a.counter = counter;
    const long long blocks = ((n + 7) / 8 + 255) / 256;
    hipLaunchKernelGGL(dropout_kernel, dim3(static_cast<unsigned>(blocks < 1 << 20 ? blocks : 1 << 20)), dim3(256), 0,
                       static_cast<hipStream_t>(stream), a);
    return launched("dropout_kernel");
}

}  // namespace

extern "C" {

srnl_status srnl_dropout_fwd(const void *x, srnl_dtype in_dtype, long long n, double p, unsigned long long seed,
                             unsigned long long offset, const unsigned long long *counter, const void *residual,
                             srnl_dtype residual_dtype, srnl_dtype out_dtype, void *out, void *stream)
{
    const char *names[] = {"x", "out", "residual"};
    return run_dropout(x, in_dtype, n, p, seed, offset, counter, residual, residual_dtype, out_dtype, out, names,
                       stream);
}

srnl_status srnl_dropout_bwd(const void *dout, srnl_dtype out_dtype, long long n, double p, unsigned long long seed,
                             unsigned long long offset, const unsigned long long *counter, const void *dx_add,
                             srnl_dtype in_dtype, void *dx, void *stream)
{
    const char *names[] = {"dout", "dx", "dx_add"};
    return run_dropout(dout, out_dtype, n, p, seed, offset, counter, dx_add, in_dtype, in_dtype, dx, names, stream);
}

}  // extern "C"
