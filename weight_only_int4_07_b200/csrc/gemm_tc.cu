// gemm_tc.cu -- the dense launches of the tensor-core GEMM (gemm_tc_kernel.cuh) and its host side:
// tensor maps, shared-memory layout, dispatch on the rows of A.
#include <cudaTypedefs.h>

#include <mutex>

#include "gemm_tc_kernel.cuh"
#include "routed.cuh"

namespace w4a16 {

// ------------------------------------------------------------------------------ host side
static PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* q = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &q, cudaEnableDefault, &r) == cudaSuccess &&
            r == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(q);
    });
    return fn;
}

// Activations A [M, K] (16-bit, row-major) as a 2-D tensor map: box 64 (K) x box_rows,
// 128-byte swizzle; rows past M read as zero.
bool make_act_map(CUtensorMap* map, const void* A, int M, int K, int box_rows, bool bf16) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)M};
    cuuint64_t strides[1] = {(cuuint64_t)K * 2};
    cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
    cuuint32_t estr[2] = {1, 1};
    CUresult r = fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
                    const_cast<void*>(A), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

// An 8-bit matrix [rows, K] (row-major, K bytes per row) as a 2-D tensor map: box 128 (K) x
// box_rows, 128-byte swizzle; rows past the end read as zero.
bool make_u8_map(CUtensorMap* map, const void* base, int rows, int K, int box_rows) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)K};
    cuuint32_t box[2] = {128, (cuuint32_t)box_rows};
    cuuint32_t estr[2] = {1, 1};
    CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

int tc_block_rows(int M) {
    if (M <= 16) return 16;
    if (M <= 32) return 32;
    if (M <= 64) return 64;
    if (M <= 128) return 128;
    return 256;   // more rows: blocks of 256 (one accumulator of 256 columns in TMEM, one MMA of
                  // N = 256 per K step, each weight unit dequantized once per 256 rows)
}

TcPlan plan_gemm_tc(int M, int N, int K, int group, int sym, int n_sm) {
    TcPlan pl = {};
    if (M < 1 || K % 128 != 0 || N % 128 != 0 || K < 128 || N < 128 || n_sm <= 0) return pl;
    const int bn = tc_block_rows(M);
    const int mblocks = (M + bn - 1) / bn;
    const long long tiles = (long long)(N / 128) * mblocks;
    if (tiles > kGemvStreamMaxTiles) return pl;
    const long long units = tiles * (K / 128);
    pl = plan_tc_rows(bn, N, K, group, sym, (int)(units < n_sm ? units : n_sm), 0);
    pl.mblocks = mblocks;
    return pl;
}

// The shared-memory layout and the partial sums of a launch with tiles of bn rows on `ctas` CTAs;
// `table` bytes follow the barriers (the grouped launch's runs).
TcPlan plan_tc_rows(int bn, int N, int K, int group, int sym, int ctas, size_t table) {
    TcPlan pl = {};
    const TiledLayout L = tiled_layout(K, N, group, sym);
    pl.bn = bn;
    pl.ctas = ctas;
    pl.slot_w = (uint32_t)((tc_units_per_load(pl.bn) * L.record + 127) & ~127u);
    pl.nd = tc_steps(pl.bn);   // steps in flight: activation tiles in shared memory, weights in TMEM
    pl.na = pl.nd;
    const uint32_t slot_a = (uint32_t)pl.bn * 256u;
    const size_t bars = 1024 + ((table + 127) & ~(size_t)127);   // barriers, tensor-memory slot, abort flag; table
    const size_t avail = (size_t)kTcSmemMax - 1024 /* alignment */ - bars;
    if ((size_t)pl.na * slot_a + 2 * (size_t)pl.slot_w > avail) return TcPlan{};
    size_t nr = (avail - (size_t)pl.na * slot_a) / pl.slot_w;
    if (nr > kTcMaxRing) nr = kTcMaxRing;
    pl.nr = (int)nr;
    pl.off_a = 0;
    pl.off_w = (uint32_t)pl.na * slot_a;
    pl.off_bar = pl.off_w + (uint32_t)pl.nr * pl.slot_w;
    pl.off_bar = (pl.off_bar + 127u) & ~127u;
    pl.smem = 1024 + pl.off_bar + bars;
    pl.partial_bytes = (size_t)pl.ctas * pl.bn * 128 * sizeof(float);
    pl.ok = pl.smem <= (size_t)kTcSmemMax;
    return pl;
}

int launch_gemm_tc(const void* A, int a_dtype, int M, int K, const void* tiled, int N, int group, int sym,
                   void* C, void* workspace, int* dev_status, cudaStream_t stream) {
    const TcPlan pl = plan_gemm_tc(M, N, K, group, sym, gemv_stream_sm_count());
    if (!pl.ok) return W4A16_EUNSUPPORTED;
    if (!workspace) return W4A16_EWORKSPACE;
    const bool bf16 = a_dtype == W4A16_BF16;
    CUtensorMap map;
    if (!make_act_map(&map, A, M, K, pl.bn, bf16)) return W4A16_ECUDA;
    TcParams prm = tc_params(pl, tiled, M, N, K, group, sym, bf16, workspace, dev_status);
    prm.C = C;
    if (bf16) return launch_tc_bn<__nv_bfloat16, kTcDense>(pl.bn, map, map, prm, pl.smem, stream);
    return launch_tc_bn<__half, kTcDense>(pl.bn, map, map, prm, pl.smem, stream);
}

}  // namespace w4a16
