// layers.hip -- the layers around the operator with their backward
// passes: layer norm and the depthwise 3x3 branch (the linear layer is in
// linear.hip). Entry points as declared in include/srnl.h.
#include "common.h"

namespace {

using namespace srnl_i;

#include "norm.inc"
#include "dwconv.inc"

// rows x C elements of at most 4 bytes within the address range, a row's (and
// its two gradients') channels within an int
bool norm_sizes_ok(long long rows, int C)
{
    return C <= 1 << 30 && static_cast<__int128>(rows) * C < (static_cast<__int128>(1) << 60);
}

srnl_status check_norm(long long rows, int C, srnl_dtype a, srnl_dtype b)
{
    if (rows < 0)
        return fail(SRNL_ERR_ARG, "rows must be >= 0");
    if (C < 1)
        return fail(SRNL_ERR_ARG, "C must be >= 1");
    if (!norm_sizes_ok(rows, C))
        return fail(SRNL_ERR_ARG, "rows x C is too large");
    if (!valid_dtype(a) || !valid_dtype(b))
        return fail(SRNL_ERR_DTYPE, "dtype must be SRNL_F32 or SRNL_BF16");
    return SRNL_OK;
}

srnl_status check_dwconv(int B, int H, int W, int C)
{
    if (B < 0 || H < 0 || W < 0)
        return fail(SRNL_ERR_ARG, "B, H and W must be >= 0");
    if (C < 1)
        return fail(SRNL_ERR_ARG, "C must be >= 1");
    if (static_cast<__int128>(B) * H * W * C >= (static_cast<__int128>(1) << 60))
        return fail(SRNL_ERR_ARG, "grid too large");
    // a grid's columns and channels are launch dimensions
    if (static_cast<long long>(W) * C > (1LL << 30))
        return fail(SRNL_ERR_ARG, "W x C is too large");
    return SRNL_OK;
}

}  // namespace

extern "C" {

srnl_status srnl_layer_norm_fwd(const void *x, long long rows, int C, srnl_dtype in_dtype,
                                const float *gain, const float *bias, float eps,
                                srnl_dtype out_dtype, void *out, float *mean, float *rstd,
                                void *stream)
{
    srnl_set_error(SRNL_OK, "");
    srnl_status s = check_norm(rows, C, in_dtype, out_dtype);
    if (s != SRNL_OK)
        return s;
    if (!(eps > 0.0f) || !std::isfinite(eps))
        return fail(SRNL_ERR_ARG, "eps must be positive and finite");
    if (rows == 0)
        return SRNL_OK;
    const PtrArg ptrs[] = {{x, "x", false},       {out, "out", false},  {gain, "gain", true},
                           {bias, "bias", true},  {mean, "mean", true}, {rstd, "rstd", true}};
    s = check_ptrs(ptrs, 6);
    if (s != SRNL_OK)
        return s;
    NormArgs a = {};
    a.x = x;
    a.rows = rows;
    a.C = C;
    a.xbf = in_dtype == SRNL_BF16;
    a.gain = gain;
    a.bias = bias;
    a.eps = eps;
    a.out = out;
    a.obf = out_dtype == SRNL_BF16;
    a.mean = mean;
    a.rstd = rstd;
    return launch_norm(a, false, static_cast<hipStream_t>(stream));
}

size_t srnl_layer_norm_bwd_workspace_bytes(long long rows, int C)
{
    if (rows <= 0 || C < 1 || !norm_sizes_ok(rows, C))
        return 0;
    const int blocks = norm_bwd_blocks(rows, C);
    return norm_direct(blocks, C) ? 0 : static_cast<size_t>(blocks) * 2 * C * sizeof(float);
}

srnl_status srnl_layer_norm_bwd(const void *dout, srnl_dtype out_dtype, const void *x,
                                long long rows, int C, srnl_dtype in_dtype, const float *gain,
                                const float *mean, const float *rstd, const void *dx_add,
                                srnl_dtype add_dtype, void *dx, float *dgain, float *dbias,
                                void *workspace, size_t workspace_bytes, void *stream)
{
    srnl_set_error(SRNL_OK, "");
    srnl_status s = check_norm(rows, C, in_dtype, out_dtype);
    if (s != SRNL_OK)
        return s;
    if (dx_add && !valid_dtype(add_dtype))
        return fail(SRNL_ERR_DTYPE, "add_dtype must be SRNL_F32 or SRNL_BF16");
    hipStream_t st = static_cast<hipStream_t>(stream);
    const bool params = dgain || dbias;
    if (rows == 0) {                     // the sums over no rows
        const PtrArg ptrs[] = {{dgain, "dgain", true}, {dbias, "dbias", true}};
        s = check_ptrs(ptrs, 2);
        if (s == SRNL_OK)
            s = zero_fill(dgain, C, st);
        return s == SRNL_OK ? zero_fill(dbias, C, st) : s;
    }
    const bool join = params && !norm_direct(norm_bwd_blocks(rows, C), C);
    if (join && (!workspace || workspace_bytes < srnl_layer_norm_bwd_workspace_bytes(rows, C)))
        return fail(SRNL_ERR_WORKSPACE, "workspace smaller than srnl_layer_norm_bwd_workspace_bytes");
    const PtrArg ptrs[] = {{dout, "dout", false},     {x, "x", false},         {dx, "dx", false},
                           {mean, "mean", false},     {rstd, "rstd", false},   {gain, "gain", true},
                           {dx_add, "dx_add", true},  {dgain, "dgain", true},  {dbias, "dbias", true},
                           {join ? workspace : nullptr, "workspace", true}};
    s = check_ptrs(ptrs, 10);
    if (s != SRNL_OK)
        return s;
    NormArgs a = {};
    a.x = x;
    a.rows = rows;
    a.C = C;
    a.xbf = in_dtype == SRNL_BF16;
    a.gain = gain;
    a.out = dx;
    a.mean = const_cast<float *>(mean);
    a.rstd = const_cast<float *>(rstd);
    a.dout = dout;
    a.dbf = out_dtype == SRNL_BF16;
    a.add = dx_add;
    a.abf = add_dtype == SRNL_BF16;
    a.part = join ? static_cast<float *>(workspace) : nullptr;
    a.dgain = dgain;
    a.dbias = dbias;
    s = launch_norm(a, true, st);
    if (s != SRNL_OK || !join)
        return s;
    return sum_rows(a.part, norm_bwd_blocks(rows, C), 2LL * C, 2LL * C, C, dgain, dbias, st);
}

srnl_status srnl_dwconv_fwd(const void *u, int B, int H, int W, int C, srnl_dtype in_dtype,
                            const float *w, const float *bias, const void *add1,
                            srnl_dtype add1_dtype, const void *add2, srnl_dtype add2_dtype,
                            srnl_dtype out_dtype, void *out, void *stream)
{
    srnl_set_error(SRNL_OK, "");
    srnl_status s = check_dwconv(B, H, W, C);
    if (s != SRNL_OK)
        return s;
    if (!valid_dtype(in_dtype) || !valid_dtype(out_dtype) || (add1 && !valid_dtype(add1_dtype)) ||
        (add2 && !valid_dtype(add2_dtype)))
        return fail(SRNL_ERR_DTYPE, "dtype must be SRNL_F32 or SRNL_BF16");
    if (B == 0 || H == 0 || W == 0)
        return SRNL_OK;
    const PtrArg ptrs[] = {{u, "u", false},       {w, "w", false},       {out, "out", false},
                           {bias, "bias", true},  {add1, "add1", true},  {add2, "add2", true}};
    s = check_ptrs(ptrs, 6);
    if (s != SRNL_OK)
        return s;
    DwArgs a = {};
    a.B = B;
    a.H = H;
    a.W = W;
    a.C = C;
    a.src = u;
    a.sbf = in_dtype == SRNL_BF16;
    a.w = w;
    a.bias = bias;
    a.add1 = add1;
    a.a1bf = add1_dtype == SRNL_BF16;
    a.add2 = add2;
    a.a2bf = add2_dtype == SRNL_BF16;
    a.out = out;
    a.obf = out_dtype == SRNL_BF16;
    return launch_dwconv(a, false, static_cast<hipStream_t>(stream));
}

size_t srnl_dwconv_bwd_workspace_bytes(int B, int H, int W, int C)
{
    if (check_dwconv(B, H, W, C) != SRNL_OK || B == 0 || H == 0 || W == 0)
        return 0;
    const DwShape d = dw_shape(B, H, W, C);
    return static_cast<size_t>(d.gy) * d.jgroups * 10 * C * sizeof(float);
}

srnl_status srnl_dwconv_bwd(const void *dout, srnl_dtype out_dtype, const void *u, int B, int H,
                            int W, int C, srnl_dtype in_dtype, const float *w, const void *du_add,
                            void *du, float *dw, float *db, void *workspace,
                            size_t workspace_bytes, void *stream)
{
    srnl_set_error(SRNL_OK, "");
    srnl_status s = check_dwconv(B, H, W, C);
    if (s != SRNL_OK)
        return s;
    if (!valid_dtype(in_dtype) || !valid_dtype(out_dtype))
        return fail(SRNL_ERR_DTYPE, "dtype must be SRNL_F32 or SRNL_BF16");
    hipStream_t st = static_cast<hipStream_t>(stream);
    const bool params = dw || db;
    if (B == 0 || H == 0 || W == 0) {    // the sums over no cells
        const PtrArg ptrs[] = {{dw, "dw", true}, {db, "db", true}};
        s = check_ptrs(ptrs, 2);
        if (s == SRNL_OK)
            s = zero_fill(dw, 9LL * C, st);
        return s == SRNL_OK ? zero_fill(db, C, st) : s;
    }
    if (params && (!workspace || workspace_bytes < srnl_dwconv_bwd_workspace_bytes(B, H, W, C)))
        return fail(SRNL_ERR_WORKSPACE, "workspace smaller than srnl_dwconv_bwd_workspace_bytes");
    const PtrArg ptrs[] = {{dout, "dout", false}, {u, "u", !params}, {w, "w", false}, {du, "du", true},
                           {dw, "dw", true},      {db, "db", true},         {du_add, "du_add", true},
                           {params ? workspace : nullptr, "workspace", true}};
    s = check_ptrs(ptrs, 8);
    if (s != SRNL_OK)
        return s;
    if (!params && !du)
        return SRNL_OK;
    DwArgs a = {};
    a.B = B;
    a.H = H;
    a.W = W;
    a.C = C;
    a.src = dout;
    a.sbf = out_dtype == SRNL_BF16;
    a.w = w;
    a.u = u;
    a.ubf = in_dtype == SRNL_BF16;
    a.add1 = du_add;
    a.a1bf = a.ubf;
    a.out = du;
    a.obf = in_dtype == SRNL_BF16;
    a.part = params ? static_cast<float *>(workspace) : nullptr;
    s = launch_dwconv(a, true, st);
    if (s != SRNL_OK || !params)
        return s;
    const DwShape d = dw_shape(B, H, W, C);
    return sum_rows(a.part, d.gy * d.jgroups, 10LL * C, 10LL * C, 9LL * C, dw, db, st);
}

}  // extern "C"
