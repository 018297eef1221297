// gla_resnorm_bwd_bf16.cu — the residual norm's gradient in bf16, a translation unit of its own for the compiler's sake.
#include "gla_common.cuh"

GLA_DEFINE_STATUS(resnorm_bwd_bf16)

#include "gla_resnorm_bwd.cuh"

namespace gla {
namespace resnorm {

int bwd_bf16(const void *dr, const void *dout, const void *r, const void *y, const void *gate, const float *scale,
              const float *post_weight, const float *post_bias, const float *weight, int kind, int post, int act, float eps,
              void *dx, void *dy, void *dgate, float *part, int64_t rows, int D, cudaStream_t st) {
    return launch_bwd<__nv_bfloat16, __nv_bfloat16>(dr, dout, r, y, gate, {scale, post_weight, post_bias, weight, nullptr}, kind, post, act, eps,
                                 dx, dy, dgate, part, rows, D, st);
}

int64_t bwd_units(int64_t rows, int D) {
    const Plan pl = make_plan(D, kBwdVecs, kWidest);
    return units(pl, rows, per_sm(pl, kBwdThreads));
}

}  // namespace resnorm
}  // namespace gla
