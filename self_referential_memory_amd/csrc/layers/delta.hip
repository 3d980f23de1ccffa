// delta.hip -- the gated delta rule's entry points (declared in
// include/srnl.h): argument checks and the choice of kernels.
#include "delta.h"

namespace {

using namespace srnl_i;

constexpr long long MAX_BLOCKS = (1 << 23) - 1;  // of 512 threads, per launch

srnl_status check_delta(const srnl_gated_delta_params *p)
{
    if (!p)
        return fail(SRNL_ERR_PTR, "params is NULL");
    if (p->B < 0 || p->T < 0)
        return fail(SRNL_ERR_ARG, "B and T must be >= 0");
    if (p->Hk < 1 || p->H < 1 || p->H % p->Hk)
        return fail(SRNL_ERR_ARG, "heads must be >= 1 and H a multiple of Hk");
    if (p->Dk < 8 || p->Dk > 128 || p->Dk % 8 || p->Dv < 8 || p->Dv > 256 || p->Dv % 8)
        return fail(SRNL_ERR_ARG, "Dk and Dv must be multiples of 8, up to 128 and 256");
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
        // 64 tokens' offsets are 31 bits
        if (s > 1 << 22)
            return fail(SRNL_ERR_ARG, "a token's heads, or a token stride, exceed 2^22 elements");
        if (static_cast<__int128>(p->B) * p->T * s >= (static_cast<__int128>(1) << 60))
            return fail(SRNL_ERR_ARG, "tensors too large");
    }
    // so are those of the parts of dq and dk that heads which share them write
    if (static_cast<long long>(p->H) * p->Dk > 1 << 22)
        return fail(SRNL_ERR_ARG, "a token's heads exceed 2^22 elements");
    // a block (of 512 threads at most) per 16 columns or per 64 tokens of a head
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
    a.N = (p.T + DELTA_CHUNK - 1) / DELTA_CHUNK;
    return a;
}

size_t chunks_of(const DeltaArgs &a) { return static_cast<size_t>(a.B) * a.H * a.N; }

// workspace: X, P and the row factors of every chunk; the record: errors and states
size_t square_bytes(const DeltaArgs &a) { return chunks_of(a) * DELTA_SQUARE; }
size_t vec_bytes(const DeltaArgs &a) { return chunks_of(a) * VEC_FLOATS * sizeof(float); }
size_t rows_bytes(const DeltaArgs &a) { return chunks_of(a) * DELTA_CHUNK * a.Dv * 4; }
size_t state_bytes(const DeltaArgs &a) { return chunks_of(a) * a.Dk * a.Dv * 4; }

size_t fwd_bytes(const DeltaArgs &a) { return 2 * square_bytes(a) + vec_bytes(a); }
size_t record_bytes_of(const DeltaArgs &a) { return rows_bytes(a) + state_bytes(a); }
// the parts of dq (or dk) of heads that share them
size_t part_bytes(const DeltaArgs &a)
{
    return a.H > a.Hk ? static_cast<size_t>(a.B) * a.T * a.H * a.Dk * 4 : 0;
}
size_t bwd_bytes(const DeltaArgs &a) { return fwd_bytes(a) + rows_bytes(a) + state_bytes(a) + 2 * part_bytes(a); }

char *place_squares(DeltaArgs &a, void *workspace)
{
    a.X = static_cast<char *>(workspace);
    a.P = a.X + square_bytes(a);
    a.vec = reinterpret_cast<float *>(a.P + square_bytes(a));
    return reinterpret_cast<char *>(a.vec) + vec_bytes(a);
}

void place_record(DeltaArgs &a, const void *record)
{
    a.E = static_cast<float *>(const_cast<void *>(record));
    a.S0 = a.E + rows_bytes(a) / 4;
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

size_t srnl_gated_delta_record_bytes(const srnl_gated_delta_params *p)
{
    return check_delta(p) == SRNL_OK ? record_bytes_of(delta_args(*p)) : 0;
}

size_t srnl_gated_delta_fwd_workspace_bytes(const srnl_gated_delta_params *p)
{
    return check_delta(p) == SRNL_OK ? fwd_bytes(delta_args(*p)) : 0;
}

size_t srnl_gated_delta_bwd_workspace_bytes(const srnl_gated_delta_params *p)
{
    return check_delta(p) == SRNL_OK ? bwd_bytes(delta_args(*p)) : 0;
}

srnl_status srnl_gated_delta_fwd(const srnl_gated_delta_params *p, void *out, float *state_out, void *record,
                                 size_t record_bytes, void *workspace, size_t workspace_bytes)
{
    srnl_set_error(SRNL_OK, "");
    srnl_status s = check_delta(p);
    if (s != SRNL_OK || p->B == 0)
        return s;
    DeltaArgs a = delta_args(*p);
    if (a.N && (!workspace || workspace_bytes < fwd_bytes(a)))
        return fail(SRNL_ERR_WORKSPACE, "workspace smaller than srnl_gated_delta_fwd_workspace_bytes");
    if (record && record_bytes < record_bytes_of(a))
        return fail(SRNL_ERR_WORKSPACE, "record smaller than srnl_gated_delta_record_bytes");
    s = check_inputs(*p);
    const PtrArg outs[] = {{out, "out", a.N == 0},
                           {state_out, "state_out", true},
                           {a.N ? record : nullptr, "record", true},
                           {a.N ? workspace : nullptr, "workspace", true}};
    if (s == SRNL_OK)
        s = check_ptrs(outs, 4);
    if (s != SRNL_OK)
        return s;
    hipStream_t st = static_cast<hipStream_t>(p->stream);
    a.out = out;
    a.state_out = state_out;
    if (a.N) {
        place_squares(a, workspace);
        if (record)
            place_record(a, record);
        s = launch_delta_prep(a, false, st);
        if (s != SRNL_OK)
            return s;
    }
    return launch_delta_chain(a, false, st);
}

srnl_status srnl_gated_delta_bwd(const srnl_gated_delta_params *p, const void *dout, const float *dstate_out,
                                 const void *record, size_t record_bytes, void *dq, void *dk, void *dv, float *dg,
                                 float *dbeta, float *dstate, void *workspace, size_t workspace_bytes)
{
    srnl_set_error(SRNL_OK, "");
    srnl_status s = check_delta(p);
    if (s != SRNL_OK || p->B == 0)
        return s;
    DeltaArgs a = delta_args(*p);
    if (a.N && (!workspace || workspace_bytes < bwd_bytes(a)))
        return fail(SRNL_ERR_WORKSPACE, "workspace smaller than srnl_gated_delta_bwd_workspace_bytes");
    if (a.N && (!record || record_bytes < record_bytes_of(a)))
        return fail(SRNL_ERR_WORKSPACE, "record smaller than srnl_gated_delta_record_bytes");
    s = check_inputs(*p);
    const PtrArg more[] = {{dout, "dout", a.N == 0},
                           {dstate_out, "dstate_out", true},
                           {a.N ? record : nullptr, "record", true},
                           {dq, "dq", true},
                           {dk, "dk", true},
                           {dv, "dv", true},
                           {dg, "dg", true},
                           {dbeta, "dbeta", true},
                           {dstate, "dstate", true},
                           {a.N ? workspace : nullptr, "workspace", true}};
    if (s == SRNL_OK)
        s = check_ptrs(more, 10);
    if (s != SRNL_OK)
        return s;
    hipStream_t st = static_cast<hipStream_t>(p->stream);
    a.dout = dout;
    a.dstate_out = dstate_out;
    a.dq = dq;
    a.dk = dk;
    a.dv = dv;
    a.dg = dg;
    a.dbeta = dbeta;
    a.dstate = dstate;
    if (a.N) {
        a.dV = reinterpret_cast<float *>(place_squares(a, workspace));
        a.D1 = a.dV + rows_bytes(a) / 4;
        a.dq_part = a.D1 + state_bytes(a) / 4;
        a.dk_part = a.dq_part + part_bytes(a) / 4;
        place_record(a, record);
        s = launch_delta_prep(a, true, st);
        if (s != SRNL_OK)
            return s;
    }
    s = launch_delta_chain(a, true, st);
    if (s == SRNL_OK && a.N && (dq || dk || dg || dbeta))
        s = launch_delta_grads(a, st);
    return s;
}

}  // extern "C"
