// Which kernels a linear layer takes (csrc/layers/plan.h), one layer a line on
// the standard input: M K N, then 0 (fp32) or 1 (bf16) for x, w and the output,
// then the activation (srnl_act). Prints the instantiations that its forward
// pass and its backward pass with every gradient launch.
#include <cstdio>

#include "plan.h"

using namespace srnl_i;

int main()
{
    static const char *const name[] = {"BF16", "BF16_ANY", "FP32", "SLOPE_BF16", "SLOPE_FP32"};
    long long M;
    int K, N, xt, wt, yt, act;
    while (scanf("%lld %d %d %d %d %d %d", &M, &K, &N, &xt, &wt, &yt, &act) == 7) {
        srnl_linear_params p = {};
        p.x_dtype = static_cast<srnl_dtype>(xt);
        p.w_dtype = static_cast<srnl_dtype>(wt);
        p.out_dtype = static_cast<srnl_dtype>(yt);
        p.act = static_cast<srnl_act>(act);
        const Source sx = source_of(p.x_dtype, K), sw = source_of(p.w_dtype, K);
        const FewShape f = few_shape(M, N, K, sx == FP32, sw == FP32);
        if (f.mi)
            printf("few_%s_%s_%dx%d", sx == FP32 ? "FP32" : "BF16", sw == FP32 ? "FP32" : "BF16", f.mi, f.mj);
        else
            printf("fwd_%s_%s_%d", name[sx], name[sw], plan_tile(FORWARD, M, N, K, sx, sw).bi);
        const BwdLayout l = bwd_layout(M, K, N, &p);
        if (l.narrow) {
            printf(" narrow_%s_%s_%s_%dx%d\n", name[l.narrow_z], name[l.sw], name[l.sx], narrow_width(N), narrow_width(K));
            continue;
        }
        if (l.px.bi >= 128)
            printf(" gradx_%s_%s_%d", name[l.sz], name[l.sw], l.px.bi);
        if (l.pw.bi >= 128)
            printf(" gradw_%s_%s_%d", name[l.sz], name[l.sx], l.pw.bi);
        if (l.px.bi < 128 || l.pw.bi < 128)
            printf(" grads_%s_%s_%s", name[l.sz], name[l.sw], name[l.sx]);
        if (act && !l.fused)
            printf(" slope");
        if (l.px.splits > 1)
            printf(" splitx_%d", l.px.bi);
        if (l.pw.splits > 1)
            printf(" splitw_%d", l.pw.bi);
        printf("\n");
    }
    return 0;
}
