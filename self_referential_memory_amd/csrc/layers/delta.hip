// delta.hip -- the gated delta rule's entry points (declared in
// include/srnl.h): argument checks and the choice of kernels.
#include "delta.h"

namespace {

using namespace srnl_i;

constexpr long long MAX_BLOCKS = 1 << 23;       // of 256 threads, per launch

srnl_status check_delta(const srnl_gated_delta_params *p)
{
    if (!p)
        return fail(SRNL_ERR_PTR, "params is NULL");
    if (p->B < 0 || p->T < 0)
        return fail(SRNL_ERR_ARG, "B and T must be >= 0");
    if (p->Hk < 1 || p->H < 1 || p->H % p->Hk)
        return fail(SRNL_ERR_ARG, "heads must be >= 1 and H a multiple of Hk");
    if (p->Dk < 8 || p->Dk > 256 || p->Dk % 8 || p->Dv < 8 || p->Dv > 256 || p->Dv % 8)
        return fail(SRNL_ERR_ARG, "Dk and Dv must be multiples of 8 from 8 to 256");
    if (p->H > 1 << 20)
        return fail(SRNL_ERR_ARG, "too many heads");
    if (!valid_dtype(p->dtype))
        return fail(SRNL_ERR_DTYPE, "dtype must be SRNL_F32 or SRNL_BF16");
    if (!std::isfinite(p->scale))
        return fail(SRNL_ERR_ARG, "scale must be finite");
    if (!(p->norm_eps >= 0.0f) || !std::isfinite(p->norm_eps))
        return fail(SRNL_ERR_ARG, "norm_eps must be >= 0 and finite");
    const long long rows[3] = {static_cast<long long>(p->Hk) * p->Dk, static_cast<long long>(p->Hk) * p->Dk,
                               static_cast<long long>(p->H) * p->Dv};
    const long long strides[3] = {p->q_stride, p->k_stride, p->v_stride};
    for (int i = 0; i < 3; ++i) {
        if (strides[i] && (strides[i] < rows[i] || strides[i] % 8))
            return fail(SRNL_ERR_ARG, "a token stride must be 0, or a multiple of 8 and at least heads x head size");
        const long long s = strides[i] ? strides[i] : rows[i];
        if (static_cast<__int128>(p->B) * p->T * s >= (static_cast<__int128>(1) << 60))
            return fail(SRNL_ERR_ARG, "tensors too large");
    }
    // a block per 16 columns or per 64 tokens of a head
    const __int128 bh = static_cast<__int128>(p->B) * p->H;
    if (bh * ((p->Dv + 15) / 16) > MAX_BLOCKS || bh * ((p->T + 63LL) / 64) > MAX_BLOCKS)
        return fail(SRNL_ERR_ARG, "too many heads x tokens");
    return SRNL_OK;
}

DeltaArgs delta_args(const srnl_gated_delta_params &p)
{
    DeltaArgs a = {};
    a.q = p.q;
    a.k = p.k;
    a.v = p.v;
    a.g = p.g;
    a.beta = p.beta;
    a.state = p.state;
    a.lengths = p.lengths;
    a.B = p.B;
    a.T = p.T;
    a.Hk = p.Hk;
    a.H = p.H;
    a.Dk = p.Dk;
    a.Dv = p.Dv;
    a.qs = p.q_stride ? p.q_stride : static_cast<long long>(p.Hk) * p.Dk;
    a.ks = p.k_stride ? p.k_stride : static_cast<long long>(p.Hk) * p.Dk;
    a.vs = p.v_stride ? p.v_stride : static_cast<long long>(p.H) * p.Dv;
    a.bf = p.dtype == SRNL_BF16;
    a.scale = p.scale;
    a.eps = p.norm_eps;
    return a;
}

srnl_status check_inputs(const srnl_gated_delta_params &p)
{
    const bool tokens = p.T > 0;
    const PtrArg ptrs[] = {{p.q, "q", !tokens},       {p.k, "k", !tokens},         {p.v, "v", !tokens},
                           {p.g, "g", !tokens},       {p.beta, "beta", !tokens},   {p.state, "state", true},
                           {p.lengths, "lengths", true}};
    return check_ptrs(ptrs, 7);
}

}  // namespace

extern "C" {

srnl_status srnl_gated_delta_step(const srnl_gated_delta_params *p, void *out, float *state_out)
{
    srnl_set_error(SRNL_OK, "");
    srnl_status s = check_delta(p);
    if (s != SRNL_OK || p->B == 0)
        return s;
    s = check_inputs(*p);
    const PtrArg outs[] = {{out, "out", p->T == 0}, {state_out, "state_out", true}};
    if (s == SRNL_OK)
        s = check_ptrs(outs, 2);
    if (s != SRNL_OK)
        return s;
    DeltaArgs a = delta_args(*p);
    a.out = out;
    a.state_out = state_out;
    return launch_delta_step(a, static_cast<hipStream_t>(p->stream));
}

}  // extern "C"
