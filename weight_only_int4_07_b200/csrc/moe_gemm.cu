// moe_gemm.cu -- the experts' INT4 products on sorted rows, tensor-core form (gemm_tc_kernel.cuh).
//
// C[i] = A[i] . dequant(W_e) for offsets[e] <= i < offsets[e + 1]; the offsets are read on the device.
// Tiles are 128 channels x up to BN rows of one expert, their unit steps cut evenly over the SMs as
// in the dense launch, so experts with few rows, many rows or none share the machine without a host
// decision.
#include "gemm_tc_kernel.cuh"
#include "routed.cuh"

namespace w4a16 {
namespace {

// Rows per tile from the mean rows of an expert (the host knows no more).
int moe_block_rows(int R, int E) {
    const int mean = (R + E - 1) / E;
    if (mean <= 12) return 16;
    if (mean <= 24) return 32;
    if (mean <= 48) return 64;
    if (mean <= 96) return 128;
    return 256;
}

TcPlan plan_moe_tc(int R, int E, int N, int K, int group, int sym) {
    const int n_sm = gemv_stream_sm_count();
    if (R < 1 || E < 1 || K % 128 != 0 || N % 128 != 0 || K < 128 || N < 128 || n_sm <= 0) return TcPlan{};
    return plan_tc_rows(moe_block_rows(R, E), N, K, group, sym, n_sm, (size_t)E * 12 + 4);
}

}  // namespace

size_t moe_gemm_partial_bytes(int R, int E, int N, int K, int group) {
    (void)N;
    (void)K;
    (void)group;
    int n_sm = gemv_stream_sm_count();
    if (n_sm <= 0) n_sm = 148;
    return (size_t)n_sm * moe_block_rows(R, E) * 128 * sizeof(float);
}

int launch_moe_gemm(const void* A, int a_dtype, int R, int K, const void* tiled, int E, const int32_t* offsets, int N,
                    int group, int sym, void* C, void* workspace, int kernel, int* dev_status, cudaStream_t stream) {
    if (kernel == W4A16_KERNEL_GEMV) return W4A16_EUNSUPPORTED;
    const TcPlan pl = plan_moe_tc(R, E, N, K, group, sym);
    if (!pl.ok) return W4A16_EUNSUPPORTED;
    const bool bf16 = a_dtype == W4A16_BF16;
    CUtensorMap map;
    if (!make_act_map(&map, A, R, K, pl.bn, bf16)) return W4A16_ECUDA;
    TcParams prm = tc_params(pl, tiled, R, N, K, group, sym, bf16, workspace, dev_status);
    prm.C = C;
    prm.offsets = offsets;
    prm.E = E;
    prm.off_grp = pl.off_bar + 1024;
    if (bf16) return launch_tc_bn<__nv_bfloat16, kTcGrouped>(pl.bn, map, prm, pl.smem, stream);
    return launch_tc_bn<__half, kTcGrouped>(pl.bn, map, prm, pl.smem, stream);
}

}  // namespace w4a16
