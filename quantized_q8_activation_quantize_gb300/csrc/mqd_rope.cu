// mqd_rope.cu -- rotary positions of dense heads.
#include "mqd_rope.cuh"

namespace mq {
namespace {

// Bound by HBM: 20000 tokens of 28 heads of 128, bf16, 47 us (6.1 TB/s); 8000 f32 38 us (6.1 TB/s).  Six blocks an SM hold 40 registers a thread.
template <typename T, int W>
__global__ void __launch_bounds__(kRopeThreads, 6) rope_kernel(RopePlan plan, RopeRows r, const int32_t *__restrict__ pos) {
    __shared__ __align__(16) float s_cos[kRopePairs], s_sin[kRopePairs];
    grid_dep_launch();
    grid_dep_wait();
    const int64_t t0 = (int64_t)blockIdx.x * r.per_block;
    rope_block<T, W>(plan, r, t0, (int)min((int64_t)r.per_block, r.n_tokens - t0), s_cos, s_sin, [&](int t) { return pos[t0 + t]; },
                     [](int) { return 1; }, false);
}

}  // namespace

int launch_rope(const RopePlan &plan, RopeRows r, int dtype, const int32_t *pos, cudaStream_t s) {
    r.per_block = rope_tokens(plan, r);
    const dim3 grid((unsigned)((r.n_tokens + r.per_block - 1) / r.per_block)), block(kRopeThreads);
    const bool wide = rope_wide(plan, r);
    cudaError_t e = dtype == MQD_F32   ? launch_pdl(rope_kernel<float, 4>, grid, block, 0, s, plan, r, pos)
                    : dtype == MQD_F16 ? launch_pdl(wide ? rope_kernel<__half, 8> : rope_kernel<__half, 4>, grid, block, 0, s, plan, r, pos)
                                       : launch_pdl(wide ? rope_kernel<__nv_bfloat16, 8> : rope_kernel<__nv_bfloat16, 4>, grid, block, 0, s, plan, r, pos);
    return cuda_error(e, "mqd_rope launch");
}

}  // namespace mq
