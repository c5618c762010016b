// gemm_tc_f32.cu -- the tensor-core GEMM (gemm_tc_kernel.cuh) with FP32 output, for a kernel that adds
// to the layer's output before it is rounded.
#include "gemm_tc_kernel.cuh"
#include "routed.cuh"

namespace w4a16 {

int launch_gemm_tc_f32(const void* A, int a_dtype, int M, int K, const void* tiled, int N, int group, int sym,
                       float* y, void* workspace, int* dev_status, cudaStream_t stream) {
    const TcPlan pl = plan_gemm_tc(M, N, K, group, sym, gemv_stream_sm_count());
    if (!pl.ok) return W4A16_EUNSUPPORTED;
    const bool bf16 = a_dtype == W4A16_BF16;
    CUtensorMap map;
    if (!make_act_map(&map, A, M, K, pl.bn, bf16)) return W4A16_ECUDA;
    TcParams prm = tc_params(pl, tiled, M, N, K, group, sym, bf16, workspace, dev_status);
    prm.C32 = y;
    if (bf16) return launch_tc_bn<__nv_bfloat16, kTcF32>(pl.bn, map, prm, pl.smem, stream);
    return launch_tc_bn<__half, kTcF32>(pl.bn, map, prm, pl.smem, stream);
}

}  // namespace w4a16
