// moe_gemm.cu -- the experts' INT4 products on sorted rows: the choice between the decode kernel
// (moe_gemv.cu) and the tensor-core form (gemm_tc_kernel.cuh), and the latter's launch.
//
// C[i] = A[i] . dequant(W_e) for offsets[e] <= i < offsets[e + 1]; the offsets are read on the device.
// Tiles are 128 channels x up to BN rows of one expert, their unit steps cut evenly over the SMs as
// in the dense launch, so experts with few rows, many rows or none share the machine without a host
// decision.
#include "gemm_tc_kernel.cuh"
#include "routed.cuh"

namespace w4a16 {
namespace {

// Rows per tile from the mean rows of an expert (the host knows no more). A tile's cost goes mostly by its
// weights (dequantized once per tile) and little by its rows, so it should hold most experts' rows at
// once. Measured, us at tiles of 16 / 32 / 64 / 128 / 256 rows, 16 experts of 4096 x 4096 (bf16, group 128;
// even routing): mean 6: 69 / 71 / 81 / 92 / 96, 16: 96 / 72 / 82 / 92 / 97, 40: 186 / 129 / 84 / 94 / 100, 100:
// 399 / 232 / 141 / 102 / 108, 256: 961 / 518 / 303 / 215 / 181; uneven routing moves the best up: mean 10: 75 / 66 /
// 74, 24: 127 / 93 / 85 / 94, 160: 613 / 335 / 212 / 165 / 151.
int moe_block_rows(int R, int E) {
    const int mean = (R + E - 1) / E;
    if (mean <= 4) return 16;
    if (mean <= 20) return 32;
    if (mean <= 48) return 64;
    if (mean <= 128) return 128;
    return 256;
}

// The decode kernel takes blocks of 8 rows; it lays the rows' activations out in the workspace, which
// bounds the mean rows of an expert that it accepts.
int moe_gemv_max_rows(int E) { return 8 * E; }

// Few rows per expert: the decode kernel. Measured with even routing and weights that come from HBM, us, decode against
// tensor cores, by the mean rows of an expert.
// Experts whose weights keep every SM busy: 64 of 2048 x 1408, group 128 (bf16) 21.3 / 25.9 at 0.5, 39.6 / 46.6 at 2,
// 45.3 / 49.6 at 4, 50.5 / 51.0 at 6; group 32 (fp16), where every weight takes a scale multiply in both, 21.0 / 22.5
// at 0.5, 42.6 / 42.9 at 3, 44.6 / 44.2 at 4; 8 of 4096 x 4096 34.0 / 38.4 at 4 (group 128), 32.6 / 35.9 at 3 (32).
// Below 32 unit records per SM (all experts') the tensor cores' whole tiles end sooner from about 3/8 on, where there
// are more than 8 rows: 16 of 1024 x 768 9.3 / 10.0 at 0.5, 10.9 / 10.4 at 1; 32 of 768 x 768 9.2 / 9.2 at 0.38,
// 10.0 / 9.3 at 0.5; 64 of 1024 x 384 10.5 / 10.5 at 0.38, 11.2 / 10.7 at 0.5; 8 of 1024 x 1024 9.8 / 10.0 at 1, 10.5 /
// 10.1 at 1.5; 8 of 2048 x 2048 13.8 / 14.8 at 1; 4 of 768 x 1280 8.3 / 8.7 at 1, 9.2 / 8.7 at 1.5.
// (Not every size follows: 16 of 2048 x 1408, 19 records per SM, would gain from the decode kernel up to 4, 15.3 / 19.0
// at 1. And the host knows R alone: padded choices count, an expert with most of the rows is not seen.)
bool moe_few_rows(int R, int E, int N, int K, int group) {
    int n_sm = gemv_stream_sm_count();
    if (n_sm <= 0) n_sm = 148;
    if ((long long)E * (N / 128) * (K / 128) < 32ll * n_sm) return R <= (E < 8 ? E : 8) || 8ll * R <= 3ll * E;
    return R <= 8 || (long long)R <= (group == 128 ? 4ll * E : 3ll * E);
}

TcPlan plan_moe_tc(int R, int E, int N, int K, int group, int sym) {
    const int n_sm = gemv_stream_sm_count();
    if (R < 1 || E < 1 || K % 128 != 0 || N % 128 != 0 || K < 128 || N < 128 || n_sm <= 0) return TcPlan{};
    return plan_tc_rows(moe_block_rows(R, E), N, K, group, sym, n_sm, 32 + (size_t)E * 12 + 4);
}

}  // namespace

// Room for R rows and for any fewer: the decode kernel's records count up to the most rows that it accepts, also
// where R itself is beyond them. (Both terms grow with R.)
size_t moe_gemm_partial_bytes(int R, int E, int K) {
    int n_sm = gemv_stream_sm_count();
    if (n_sm <= 0) n_sm = 148;
    const size_t tc = (size_t)2 * n_sm * moe_block_rows(R, E) * 128 * sizeof(float);
    const size_t gemv = moe_gemv_partial_bytes(R < moe_gemv_max_rows(E) ? R : moe_gemv_max_rows(E), K);
    return tc > gemv ? tc : gemv;
}

int moe_select_kernel(int R, int E, int N, int K, int group, int sym, int forced) {
    const bool want = forced == W4A16_KERNEL_AUTO ? moe_few_rows(R, E, N, K, group) : forced == W4A16_KERNEL_GEMV;
    return want && R <= moe_gemv_max_rows(E) && moe_gemv_fits(R, E, N, K, group, sym)
               ? W4A16_KERNEL_GEMV
               : W4A16_KERNEL_TC;
}

int launch_moe_gemm(const void* A, int a_dtype, int R, int K, const void* tiled, int E, const int32_t* offsets, int N,
                    int group, int sym, void* C, void* workspace, int kernel, int* dev_status, cudaStream_t stream) {
    if (kernel == W4A16_KERNEL_GEMV) {
        if (R > moe_gemv_max_rows(E)) return W4A16_EUNSUPPORTED;
        return launch_moe_gemv(A, a_dtype, R, K, tiled, E, offsets, N, group, sym, C, workspace, dev_status, stream);
    }
    const TcPlan pl = plan_moe_tc(R, E, N, K, group, sym);
    if (!pl.ok) return W4A16_EUNSUPPORTED;
    const bool bf16 = a_dtype == W4A16_BF16;
    CUtensorMap map;
    if (!make_act_map(&map, A, R, K, tc_box_rows(pl.bn), bf16)) return W4A16_ECUDA;
    TcParams prm = tc_params(pl, tiled, R, N, K, group, sym, bf16, workspace, dev_status);
    prm.C = C;
    prm.offsets = offsets;
    prm.E = E;
    prm.off_grp = pl.off_bar + 1024;
    if (bf16) return launch_tc_bn<__nv_bfloat16, kTcGrouped>(pl.bn, map, map, prm, pl.smem, stream);
    return launch_tc_bn<__half, kTcGrouped>(pl.bn, map, map, prm, pl.smem, stream);
}

}  // namespace w4a16
