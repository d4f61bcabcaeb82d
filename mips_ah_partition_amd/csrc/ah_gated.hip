// Gated feed-forward by leaf: the products of ah_tiles.hpp whose epilogues activate, multiply and drop, and, back, turn
// the hidden values' gradient into the two projections'.  Neither the projections' sums nor the hidden values' gradient (of
// 16,384 rows and 4,096 columns 0.5 and 0.27 GB in float32) leave the registers they are made in.
#include "ah_tiles.hpp"

namespace ah {

static ProdArgs gated_args(const GatedProblem& g, const Dropout& d, int32_t act) {
    ProdArgs a{};
    a.q = static_cast<const char*>(g.q);
    a.qs = g.q_stride * 2;
    a.p = static_cast<const char*>(g.w);
    a.off = g.offsets;
    a.order = g.order;
    a.T = a.I = g.slots;
    a.L = g.L;
    a.J = g.n;
    a.red = g.k;
    a.act = act;
    a.drop = d;
    return a;
}

hipError_t launch_gated(const GatedProblem& g, const Dropout& d, int32_t act, void* pre, void* out, int32_t out_dtype,
                        hipStream_t stream) {
    ProdArgs a = gated_args(g, d, act);
    a.ps = (int64_t)g.k * 2;
    a.pg = (int64_t)g.n * 2 * a.ps;
    a.pre = static_cast<char*>(pre);
    a.out = out;
    a.out_f32 = out_dtype == AH_F32;
    return launch_prod<kGate>(a, g.fan, stream);
}

hipError_t launch_gated_grad(const GatedProblem& g, const Dropout& d, int32_t act, const void* pre, void* dpre,
                             void* hidden, hipStream_t stream) {
    ProdArgs a = gated_args(g, d, act);
    a.ps = (int64_t)g.n * 2;
    a.pg = (int64_t)g.k * a.ps;
    a.pre = static_cast<char*>(const_cast<void*>(pre));  // read only
    a.out = dpre;
    a.hidden = static_cast<char*>(hidden);
    return launch_prod<kGrad>(a, 1, stream);
}

}  // namespace ah
