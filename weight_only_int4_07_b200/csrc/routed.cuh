// routed.cuh -- host-side launchers of the routed layers (rows that pick an expert or an adapter).
#pragma once

#include <cuda.h>

#include "common.cuh"

namespace w4a16 {

constexpr int kRouteMaxBins = 1024;      // experts, or adapters
constexpr int kRouteMaxChoices = 32;     // choices per token
constexpr int kRouteDirectIds = 8192;    // ids that every CTA counts by itself
constexpr int kRouteHistIds = 2048;      // ids of one histogram block above that

// Counting sort of n = T k ids into E bins, stable in the flat index: offsets[E + 1], rows (sorted
// row -> flat index), slots (flat index -> sorted row, -1 without one) and, with X, the gathered rows.
struct RouteSort {
    const int32_t* ids;
    int T, k, E;
    const void* X;       // [T, H] 16-bit, or null
    int H;
    int32_t* offsets;
    int32_t* rows;
    int32_t* slots;
    void* Xs;
    int32_t* hist;       // route_sort_workspace_bytes
};
size_t route_sort_workspace_bytes(int T, int k, int E);
int launch_route_sort(const RouteSort& p, cudaStream_t stream);

int launch_moe_combine(const void* Ys, int dtype, int T, int k, int H, const int32_t* slots, const float* weights,
                       void* Y, cudaStream_t stream);
int launch_moe_combine_grad(const void* dY, const void* Ys, int dtype, int T, int k, int H, const int32_t* slots,
                            const float* weights, void* dYs, float* dweights, cudaStream_t stream);

// Shared with the dense tensor-core GEMM (gemm_tc.cu).
bool make_act_map(CUtensorMap* map, const void* A, int M, int K, int box_rows, bool bf16);
TcPlan plan_tc_rows(int bn, int N, int K, int group, int sym, int ctas, size_t table);

// The experts' products on R sorted rows: workspace after the counters, and the launch.
size_t moe_gemm_partial_bytes(int R, int E, int K);
size_t moe_gemv_partial_bytes(int R, int K);
int launch_moe_gemv(const void* A, int a_dtype, int R, int K, const void* tiled, int E, const int32_t* offsets, int N,
                    int group, int sym, void* C, void* workspace, int* dev_status, cudaStream_t stream);
bool moe_gemv_fits(int R, int E, int N, int K, int group, int sym);
// What AUTO takes, W4A16_KERNEL_GEMV or _TC; forced: the environment's choice, if any (where it can serve the call).
int moe_select_kernel(int R, int E, int N, int K, int group, int sym, int forced);
int launch_moe_gemm(const void* A, int a_dtype, int R, int K, const void* tiled, int E, const int32_t* offsets, int N,
                    int group, int sym, void* C, void* workspace, int kernel, int* dev_status, cudaStream_t stream);

// The dense decode kernel with low-rank terms added to its FP32 sums (gemv_stream.cu).
struct GemvLora {
    const void* b;              // Lb [adapters][N][rank]
    const float* scale;         // [adapters]
    const int32_t* row_adapter; // [M]
    const float* part;          // [slices][M][rank]: A . La^T over slices of K
    int slices, rank, adapters;
};
GemvStreamPlan plan_gemv_lora(int M, int N, int K, int group, int sym, int n_sm, int rank);
int launch_gemv_lora(const void* A, int a_dtype, int M, int K, const void* tiled, int N, int group, int sym, void* C,
                     const GemvLora& lora, void* workspace, int* dev_status, cudaStream_t stream);

// The layer with low-rank adapters.
constexpr int kLoraMaxRank = 256;
size_t lora_workspace_bytes(int M, int N, int K, int group, int rank, int adapters);
int lora_select_kernel(int M, int N, int K, int group, int rank);   // W4A16_KERNEL_GEMV or _TC
int launch_lora_gemm(const void* A, int a_dtype, int M, int K, const void* tiled, int N, int group, int sym,
                     const void* La, const void* Lb, const float* scale, int adapters, int rank,
                     const int32_t* row_adapter, void* C, void* workspace, int* dev_status, cudaStream_t stream);

}  // namespace w4a16
