// plan.h -- which kernel takes a linear layer of given sizes and types: tiles and
// splits, the few-rows and the narrow form, the backward pass's workspace. Host
// arithmetic alone, so that tests can ask it without a GPU.
#ifndef SRNL_LAYERS_PLAN_H
#define SRNL_LAYERS_PLAN_H

#include "srnl.h"

namespace srnl_i {

constexpr long long cdiv(long long a, long long b) { return (a + b - 1) / b; }

// What an operand is made of: bf16 words (in rows of whole 16-byte pieces, or
// in rows of any length), fp32 values, or dy act'(z) formed while it is staged,
// with dy in bf16 or fp32. The card takes wide loads at any element's address;
// only the direct loads into LDS ask for whole pieces.
enum Source { BF16, BF16_ANY, FP32, SLOPE_BF16, SLOPE_FP32 };
constexpr bool is_bf16(Source s) { return s == BF16 || s == BF16_ANY; }

enum Form { FORWARD, GRAD_X, GRAD_W };     // which operands have the reduction contiguous

struct Plan {
    int bi;                // tile side
    int splits;
    long long slice;
    long long ti, tj;
};

// Tile and split of out[I][J] over R. 256 x 256 (bf16 operands) or 128 x 128
// tiles where they give every CU one, else 64 x 64: 16384 x 2048 -> 2048 bf16
// takes 147 us in the largest and 182 us in 128 x 128, whose waves read twice
// the LDS bytes a product (31 and 23 bytes a cycle and wave). An input gradient
// of a short reduction shares a launch with the weight gradient in tiles of 64,
// which is worth more than the larger tiles up to one and a half a CU (backward
// of 6272 x 768 -> 256 bf16, 294 tiles, 25.3 us in tiles of 64 and 29.2 in 128;
// 12544 x 768 -> 192, 588 tiles, 45.3 and 41.6). A weight
// gradient's reduction is long enough to fill the card with parts of 128 x 128
// tiles; where these are a quarter empty, at twice the parts (backward, fp32:
// 14560 x 1776 -> 74, 797 parts, with bf16 weights 111 us in tiles of 64 and 92
// in 128; 4626 x 93 -> 1863, 285 parts, 60 and 67).
//
// A gradient's reduction is split where the tiles leave CUs idle (the weight
// gradient over many tokens; an input gradient of few rows):
// - to two blocks a CU for tiles of 128 (backward of 10496 x 1472 -> 440 fp32
//   240 us at one block, 214 at two, 227 at three) of at least four steps;
// - to one block a CU for tiles of 64, of at least two steps, and to two where
//   each keeps eight steps, since one block mostly waits for its loads (backward
//   of 14560 x 1776 -> 74, fp32 with bf16 weights: 145 and 106 us; but 1003 x
//   333 -> 777 fp32, 13 steps: 23.5 and 27);
// - not at all where the whole reduction takes about as long as the launch that
//   joins the parts: three steps of converted operands (640 x 16 -> 50 fp32 split
//   19.5, whole 10.7 us), ten of bf16 ones (439 x 854 -> 707 split 14.5, whole 11.8).
inline Plan plan_tile(Form f, long long I, long long J, long long R, Source sa, Source sb)
{
    Plan p;
    const int bk = is_bf16(sa) && is_bf16(sb) ? 64 : 32;
    const long long big = cdiv(I, 128) * cdiv(J, 128);
    const long long side = I < J ? I : J, parts = big * cdiv(R, 8 * bk);
    p.bi = big >= (f == GRAD_X && R <= 256 ? 384 : 256) || (f == GRAD_W && side > 64 && parts >= (side >= 96 ? 256 : 512)) ? 128 : 64;
    if (sa == BF16 && sb == BF16 && f != GRAD_W && cdiv(I, 256) * cdiv(J, 256) >= 256 && R >= 256)
        p.bi = 256;
    p.ti = cdiv(I, p.bi);
    p.tj = cdiv(J, p.bi);
    const int step = p.bi >= 128 ? bk : 2 * bk;
    const long long tiles = p.ti * p.tj;
    auto split = [&](long long blocks, long long steps) {
        const long long s = blocks / tiles, most = cdiv(R, steps * step);
        return s < most ? s : most;
    };
    long long s = 1;
    if (f != FORWARD && R > (bk == 64 ? 10 : 3) * step) {
        const long long one = split(256, 2), two = split(512, 8);
        s = p.bi >= 128 ? split(512, 4) : one > two ? one : two;
    }
    s = s < 1 ? 1 : s;
    p.slice = cdiv(cdiv(R, s), step) * step;
    p.splits = static_cast<int>(cdiv(R, p.slice));
    return p;
}

struct FewShape {
    int mi, mj;            // 16 mi x 16 mj outputs a block; 0: not for the few-rows kernel
};

// The few-rows kernel takes a product of which every CU gets at most one block,
// in the smallest blocks for which that holds. Its blocks are longer along the
// bf16 operand, so that less of an fp32 one is split twice; the largest only
// pay where an operand is split and the reduction is no short one. A product of
// up to 32 rows goes there whatever its columns. Measured (us, few rows / tiles;
// x, w fp32, then bf16): 49 x 2048 -> 512 10.0 / 51 and 6.3 / 12.4; 512 x 512 ->
// 512 7.2 / 15.3 and 4.8 / 5.6; 672 x 864 -> 512 14.3 / 24.4, with bf16 w 8.9 /
// 16.8, but all bf16 6.3 / 7.7; 128 x 1024 -> 4096 16.0 / 30.3, all bf16 8.9 /
// 8.3; 300 x 64 -> 1024 5.5 / 4.8; 1 x 1024 -> 8192 7.4 / 28.9 and 5.1 / 7.6;
// past it 1003 x 333 -> 777 15.5 / 13.6 and 16.9 / 8.8.
inline FewShape few_shape(long long M, long long N, long long R, bool xf, bool wf)
{
    const bool wide = (xf && !wf) || M <= 16;
    auto fits = [&](int mi, int mj) { return cdiv(M, 16 * mi) * cdiv(N, 16 * mj) <= 256; };
    if (fits(1, 1))
        return {1, 1};
    if (wide ? fits(1, 2) : fits(2, 1))
        return wide ? FewShape{1, 2} : FewShape{2, 1};
    const bool few = M <= 32 && N <= 1 << 26;                  // and a launch below 2^32 threads
    if (fits(2, 2) || (few && M > 16))
        return {2, 2};
    if (few)
        return {1, 2};
    if ((xf || wf) && R >= 256 && (wide ? fits(2, 4) : fits(4, 2)))
        return wide ? FewShape{2, 4} : FewShape{4, 2};
    return {0, 0};
}

// ------------------------------------------------------------ narrow backward

constexpr int kThreads = 512;                 // eight waves
constexpr int kLdsWords = 81920;              // all 160 KB: one block a CU
constexpr int kMaxPieces = 4;                 // 8-element pieces of dz, or of x, per thread and slice (6 of both)

constexpr int narrow_parts(Source s) { return s == BF16 ? 1 : 3; }
constexpr int narrow_width(int n) { return n <= 64 ? 64 : n <= 128 ? 128 : 256; }

// Rows per slice for widths rounded up: the most that LDS, the pieces a thread
// holds in flight and two dx tiles a wave allow; 0 where not even 32 fit.
constexpr int narrow_rows(int kp, int np, Source sz, Source sw, Source sx)
{
    if (kp * np > 16384)
        return 0;
    for (int bm = 128; bm >= 32; bm /= 2) {
        const int words = narrow_parts(sz) * bm * np + narrow_parts(sx) * bm * kp + narrow_parts(sw) * np * kp;
        const int most = 8 * kThreads * kMaxPieces;
        if (words <= kLdsWords && bm * np <= most && bm * kp <= most && bm * (np + kp) <= most * 3 / 2 &&
            (bm / 32) * (kp / 32) <= 16 &&
            bm * np >= 8 * kThreads && bm * kp >= 8 * kThreads)
            return bm;
    }
    return 0;
}

// Partial weight (and bias) gradients that narrow_launch leaves for the caller
// to join, one a block; 0 where it does not take the layer. Every block should
// have a few slices.
inline int narrow_bwd_parts(long long M, int K, int N, Source sz, Source sw, Source sx)
{
    if (K % 8 || N % 8 || K > 256 || N > 256)
        return 0;
    const int bm = narrow_rows(narrow_width(K), narrow_width(N), sz, sw, sx);
    return bm && M >= 512LL * bm ? 256 : 0;
}

// ------------------------------------------------------------ backward pass

// what an operand with rows of n elements is, for the tiled kernels
inline Source source_of(srnl_dtype t, long long n) { return t == SRNL_F32 ? FP32 : n % 8 == 0 ? BF16 : BF16_ANY; }

// Workspace of the backward pass (floats, 64-float aligned parts): dz where a
// pass of its own makes it, then the partial products of the input gradient and of
// the weight gradient, and the partial bias gradient, where they are split.
struct BwdLayout {
    Plan px, pw;
    bool fused = false;    // the activation's slope is applied while dz is staged
    int narrow = 0;        // partial gradients of the narrow form (both gradients wanted), or 0
    Source sz = BF16, sw = BF16, sx = BF16;      // what the tiled kernels stage
    Source narrow_z = BF16;
    long long o_x = 0, o_w = 0, o_b = 0, o_nb = 0, total = 0;
};
inline long long up64(long long n) { return (n + 63) & ~63LL; }

inline BwdLayout bwd_layout(long long M, int K, int N, const srnl_linear_params *p)
{
    BwdLayout l;
    const bool act = p->act != SRNL_ACT_NONE;
    l.sw = source_of(p->w_dtype, K);
    l.sx = source_of(p->x_dtype, K);
    const Source sy = source_of(p->out_dtype, N), sz = act ? FP32 : sy;      // dz as a pass leaves it
    l.px = plan_tile(GRAD_X, M, K, N, sz, l.sw);
    l.pw = plan_tile(GRAD_W, N, K, M, sz, l.sx);
    const Source slope = p->out_dtype == SRNL_F32 ? SLOPE_FP32 : SLOPE_BF16;
    // dz = dy act'(z) is formed anew for every 64 columns of either product:
    // up to 2 M values that costs less than a pass of its own (backward kernels
    // with gelu less those without, fp32: 500 x 200 -> 300, 0.6 M values, 2 us;
    // 1000 x 512 -> 512, 4 M, 5 us; the pass takes 4.6 us and a launch)
    l.fused = act && l.px.bi == 64 && l.pw.bi == 64 && M * N * cdiv(K, 64) <= (2LL << 20);
    l.sz = l.fused ? slope : sz;
    l.o_x = act && !l.fused ? up64(M * N) : 0;
    l.o_w = l.o_x + (l.px.splits > 1 ? up64(l.px.splits * M * K) : 0);
    const bool split = l.pw.splits > 1;
    l.o_b = l.o_w + (split ? up64(static_cast<long long>(l.pw.splits) * N * K) : 0);
    l.total = l.o_b + (split ? up64(static_cast<long long>(l.pw.splits) * N) : 0);
    l.narrow_z = act ? slope : sy;
    l.narrow = narrow_bwd_parts(M, K, N, l.narrow_z, l.sw, l.sx);
    if (l.narrow) {
        l.o_nb = up64(static_cast<long long>(l.narrow) * N * K);
        const long long all = l.o_nb + up64(static_cast<long long>(l.narrow) * N);
        l.total = l.total > all ? l.total : all;
    }
    return l;
}

}  // namespace srnl_i

#endif
