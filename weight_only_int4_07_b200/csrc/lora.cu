// lora.cu -- low-rank adapters of many requests at once beside the INT4 layer (sm_100a).
//
// C[m] = A[m] . dequant(W) + s_a (A[m] . La_a^T) . Lb_a^T,  a = row m's adapter (none: the first term).
// Three kernels after one another, joined by programmatic dependent launch:
//   shrink  T[m, j] = sum_k A[m, k] La_a[j, k] over slices of K (FP32 partial sums per slice);
//   base    the layer's own kernel with FP32 output (gemv_stream.cu or gemm_tc_kernel.cuh);
//   expand  C = base + 2^e (T 2^-e s_a) . Lb_a^T, rounded once.
// Rows of one adapter are taken together, so an adapter's matrices come from memory once however many
// requests use it: up to 16 rows each CTA groups them itself, above a counting sort (moe_route.cu)
// lists runs of up to 32 rows.
// Both products are m16n8k16 warp MMAs on operands read straight from global memory: a lane reads 16
// (or 8) consecutive bytes of a row and the same permutation of K (or of the ranks) stands on both
// sides of the product, so no shared-memory staging is needed. The work is small beside the
// layer's (2 r (K + N) of 2 K N operations per row); what counts is that it streams at full width.
// T stays at FP32 accuracy: it enters the second product as the sum of two 16-bit values, hi and lo,
// after a power of two per row that puts its largest value near 2^14 (fp16 then keeps everything
// down to 2^-38 of it).
#include "pdl.cuh"
#include "dequant.cuh"
#include "routed.cuh"

namespace w4a16 {
namespace {

constexpr int kLoraThreads = 256, kLoraWarps = kLoraThreads / 32;
constexpr int kLoraSmallRows = 16;          // up to here CTAs group the rows themselves
constexpr int kShrinkRanks = 64;            // ranks of one pass over K
constexpr size_t kLoraChunkBytes = (size_t)64 << 20;   // FP32 base outputs held at a time

struct LoraParams {
    const void* A;              // [M, K]
    const void* La;             // [L, r, K]
    const void* Lb;             // [L, N, r]
    const float* scale;         // [L]
    const int32_t* row_adapter; // [M]
    const RouteTile* tiles;     // M > 16: runs of sorted rows
    const int* ntiles;
    const int32_t* rows;        // sorted row -> row
    float* part;                // [S][M][r]
    const float* base;          // [slices][M][N]
    void* C;
    int M, K, N, r, L, S, slices, passes;
};

// The rows of one work item: those of tile `i`, or (up to 16 rows) the rows that share row i's
// adapter when i is the first of them. `list` (shared) gets their indices; returns how many, 0 for
// none. All threads of the CTA call it.
__device__ __forceinline__ int lora_rows(const LoraParams& p, int i, int* list, int& adapter) {
    if (p.tiles) {
        if (i >= *p.ntiles) return 0;
        const RouteTile t = p.tiles[i];
        adapter = t.bin;
        if (threadIdx.x < t.count) list[threadIdx.x] = p.rows[t.begin + threadIdx.x];
        __syncthreads();
        return t.count;
    }
    const int lane = threadIdx.x & 31;
    int a = -1;
    if (lane < p.M) {
        a = p.row_adapter[lane];
        if ((unsigned)a >= (unsigned)p.L) a = p.L;
    }
    adapter = __shfl_sync(0xffffffffu, a, i);
    const unsigned same = __ballot_sync(0xffffffffu, lane < p.M && a == adapter);
    if (__ffs(same) - 1 != i) return 0;
    if (threadIdx.x < 32 && (same >> lane) & 1u) list[__popc(same & ((1u << lane) - 1u))] = lane;
    __syncthreads();
    return __popc(same);
}

// T's partial sums over one slice of K. NB: 8-row blocks (2: up to 16 rows, 4: up to 32). Warp w takes
// every eighth 32-K step of the slice; MMA rows are ranks, MMA columns rows of A.
template <int NB, typename T>
__global__ void __launch_bounds__(kLoraThreads) lora_shrink_kernel(const LoraParams p) {
    constexpr int RB = kShrinkRanks / 16;
    __shared__ float red[4][kShrinkRanks * NB * 8];
    __shared__ int list[32];
    using Ops = GsOps<T>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    pdl_wait();
    pdl_trigger();
    int adapter;
    const int n = lora_rows(p, blockIdx.y, list, adapter);
    if (n == 0 || adapter >= p.L) return;
    const T* A = static_cast<const T*>(p.A);
    const T* La = static_cast<const T*>(p.La) + (size_t)adapter * p.r * p.K;
    const int steps = p.K / 32, S = p.S, sl = blockIdx.x;
    const int s0 = (int)((long long)steps * sl / S), s1 = (int)((long long)steps * (sl + 1) / S);
    const T* x[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) x[b] = 8 * b + g < n ? A + (size_t)list[8 * b + g] * p.K + 8 * t : nullptr;
    for (int r0 = 0; r0 < p.r; r0 += kShrinkRanks) {
        float acc[RB][NB][4];
#pragma unroll
        for (int q = 0; q < RB; ++q)
#pragma unroll
            for (int b = 0; b < NB; ++b) acc[q][b][0] = acc[q][b][1] = acc[q][b][2] = acc[q][b][3] = 0.0f;
        const int nq = min(RB, (p.r - r0 + 15) / 16);
#pragma unroll 2
        for (int s = s0 + warp; s < s1; s += kLoraWarps) {
            uint4 xv[NB], lo[RB], hi[RB];
            const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int b = 0; b < NB; ++b) xv[b] = x[b] ? __ldg(reinterpret_cast<const uint4*>(x[b] + 32 * s)) : zero;
#pragma unroll
            for (int q = 0; q < RB; ++q)
                if (q < nq) {
                    const int j = r0 + 16 * q + g;
                    const T* a = La + (size_t)j * p.K + 32 * s + 8 * t;
                    lo[q] = j < p.r ? __ldg(reinterpret_cast<const uint4*>(a)) : zero;
                    hi[q] = j + 8 < p.r ? __ldg(reinterpret_cast<const uint4*>(a + (size_t)8 * p.K)) : zero;
                }
#pragma unroll
            for (int q = 0; q < RB; ++q)
                if (q < nq)
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        Ops::mma(acc[q][b], lo[q].x, hi[q].x, lo[q].y, hi[q].y, xv[b].x, xv[b].y);
                        Ops::mma(acc[q][b], lo[q].z, hi[q].z, lo[q].w, hi[q].w, xv[b].z, xv[b].w);
                    }
        }
        // the warps' sums, halves onto halves (a fixed order)
        auto each = [&](auto f) {
#pragma unroll
            for (int q = 0; q < RB; ++q)
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int e = 0; e < 4; ++e) f(acc[q][b][e], ((q * NB + b) * 4 + e) * 32 + lane);
        };
#pragma unroll
        for (int half = kLoraWarps / 2; half >= 1; half >>= 1) {
            if (warp >= half && warp < 2 * half) each([&](float& v, int at) { red[warp - half][at] = v; });
            __syncthreads();
            if (warp < half) each([&](float& v, int at) { v += red[warp][at]; });
            __syncthreads();
        }
        if (warp == 0) {
            float* out = p.part + (size_t)sl * p.M * p.r;
#pragma unroll
            for (int q = 0; q < RB; ++q)
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int j = r0 + 16 * q + g + 8 * (e >> 1), m = 8 * b + 2 * t + (e & 1);
                        if (j < p.r && m < n) out[(size_t)list[m] * p.r + j] = acc[q][b][e];
                    }
        }
    }
}

__host__ __device__ inline int lora_t_stride(int r) {   // elements between rows of T's hi (or lo) tile
    const int bytes = ((r + 15) / 16) * 32;
    return (bytes % 64 == 0 ? bytes + 32 : bytes) / 2;    // 32 mod 64: the lanes' 8-byte reads miss no bank
}

// C's rows of one item and `passes` blocks of 256 channels. NB: 16-row blocks. MMA rows are rows of C,
// MMA columns channels: column c of tile j is channel 8 (c / 2) + 2 j + c % 2 of the warp's 32, so a
// lane's four tiles are eight consecutive channels of C.
template <int NB, typename T>
__global__ void __launch_bounds__(kLoraThreads) lora_expand_kernel(const LoraParams p) {
    extern __shared__ __align__(16) uint8_t lora_smem[];
    __shared__ int list[32];
    __shared__ float up[16 * NB];
    using Ops = GsOps<T>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int ts = lora_t_stride(p.r), r16 = (p.r + 15) / 16;
    T* thi = reinterpret_cast<T*>(lora_smem);
    T* tlo = thi + (size_t)16 * NB * ts;
    pdl_wait();
    pdl_trigger();
    int adapter;
    const int n = lora_rows(p, blockIdx.y, list, adapter);
    if (n == 0) return;
    const bool low = adapter < p.L;
    if (low) {
        // row m of T: the slices' sums in order, times the adapter's scale; a warp per row
        const float sc = __ldg(p.scale + adapter);
        for (int m = warp; m < 16 * NB; m += kLoraWarps) {
            float big = 0.0f, v[8];   // r <= 256
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const int j = lane + 32 * q;
                v[q] = 0.0f;
                if (m < n && j < p.r) {
                    const float* at = p.part + (size_t)list[m] * p.r + j;
                    float s = 0.0f;
#pragma unroll 4
                    for (int k = 0; k < p.S; ++k) s += __ldcg(at + (size_t)k * p.M * p.r);
                    v[q] = s * sc;
                    big = fmaxf(big, fabsf(v[q]));
                }
            }
            const unsigned top = __reduce_max_sync(0xffffffffu, __float_as_uint(big));
            const int e = top ? min(max((int)(top >> 23) - 127 - 14, -100), 100) : 0;
            const float down = __int_as_float((127 - e) << 23);
            if (lane == 0) up[m] = __int_as_float((127 + e) << 23);
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const int j = lane + 32 * q;
                if (j < 16 * r16) {
                    const float x = v[q] * down;
                    const T h = Act<T>::from_f32(x);
                    thi[m * ts + j] = h;
                    tlo[m * ts + j] = Act<T>::from_f32(x - Act<T>::to_f32(h));
                }
            }
        }
        __syncthreads();
    }
    const T* Lb = static_cast<const T*>(p.Lb) + (low ? (size_t)adapter * p.N * p.r : 0);
    T* C = static_cast<T*>(p.C);
    for (int pass = 0; pass < p.passes; ++pass) {
        const int n0 = (blockIdx.x * p.passes + pass) * 256 + 32 * warp;
        if (n0 >= p.N) break;   // (N is a multiple of 128: a warp's 32 channels are all there or none)
        float acc[NB][4][4];
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[b][j][0] = acc[b][j][1] = acc[b][j][2] = acc[b][j][3] = 0.0f;
        if (low) {
            const T* brow = Lb + (size_t)(n0 + 8 * (g >> 1) + (g & 1)) * p.r + 4 * t;
#pragma unroll 4
            for (int q = 0; q < r16; ++q) {
                uint2 bv[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    bv[j] = 16 * q + 4 * t < p.r ? __ldg(reinterpret_cast<const uint2*>(brow + (size_t)(2 * j) * p.r + 16 * q))
                                                 : make_uint2(0, 0);
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const T* th = thi + (16 * b + g) * ts + 16 * q + 4 * t;
                    const T* tl = tlo + (16 * b + g) * ts + 16 * q + 4 * t;
                    const uint2 h0 = *reinterpret_cast<const uint2*>(th), h1 = *reinterpret_cast<const uint2*>(th + 8 * ts);
                    const uint2 l0 = *reinterpret_cast<const uint2*>(tl), l1 = *reinterpret_cast<const uint2*>(tl + 8 * ts);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        Ops::mma(acc[b][j], h0.x, h1.x, h0.y, h1.y, bv[j].x, bv[j].y);
                        Ops::mma(acc[b][j], l0.x, l1.x, l0.y, l1.y, bv[j].x, bv[j].y);
                    }
                }
            }
        }
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int h = 0; h < 2; ++h) {   // rows 16 b + g and 16 b + g + 8
                const int m = 16 * b + 8 * h + g;
                if (m >= n) continue;
                const size_t at = (size_t)list[m] * p.N + n0 + 8 * t;
                float y[8] = {0, 0, 0, 0, 0, 0, 0, 0};
                for (int s = 0; s < p.slices; ++s) {
                    const float4* q = reinterpret_cast<const float4*>(p.base + (size_t)s * p.M * p.N + at);
                    const float4 u = __ldcg(q), v = __ldcg(q + 1);
                    y[0] += u.x; y[1] += u.y; y[2] += u.z; y[3] += u.w;
                    y[4] += v.x; y[5] += v.y; y[6] += v.z; y[7] += v.w;
                }
                if (low) {
                    const float f = up[m];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        y[2 * j] = fmaf(acc[b][j][2 * h], f, y[2 * j]);
                        y[2 * j + 1] = fmaf(acc[b][j][2 * h + 1], f, y[2 * j + 1]);
                    }
                }
                uint4 o;
                T* oh = reinterpret_cast<T*>(&o);
#pragma unroll
                for (int i = 0; i < 8; ++i) oh[i] = Act<T>::from_f32(y[i]);
                *reinterpret_cast<uint4*>(C + at) = o;
            }
    }
}

// ------------------------------------------------------------------------------ host side
struct LoraPlan {
    int rows;       // rows of A taken at a time
    int S;          // slices of K of the shrink kernel
    int tiles;      // work items of a chunk (an upper bound above 16 rows)
    int slices;     // FP32 outputs of the base kernel to add up
    size_t base_ws; // workspace of the base kernel
    size_t off_y, off_part, off_tiles, off_ntiles, off_rows, off_hist, total;
};

int lora_chunk_rows(int M, int N) {
    size_t rows = kLoraChunkBytes / ((size_t)N * 4) / 256 * 256;
    if (rows < 256) rows = 256;
    return (size_t)M < rows ? M : (int)rows;
}

LoraPlan plan_lora(int M, int N, int K, int group, int rank, int adapters) {
    LoraPlan pl = {};
    pl.rows = lora_chunk_rows(M, N);
    const int m = pl.rows;
    pl.slices = 1;
    int n_sm = gemv_stream_sm_count();
    if (n_sm <= 0) n_sm = 148;
    if (m <= kLoraSmallRows) {
        const GemvStreamPlan q = plan_gemv_stream(m, N, K, group, 0, n_sm);
        if (q.ok) pl.slices = q.slices;
        pl.tiles = m;
        pl.S = 16;
    } else {
        const int most = m / 32 + adapters + 1;
        pl.tiles = m < most ? m : most;
        pl.S = 2 * n_sm / ((m + 31) / 32);   // two CTAs per SM when rows share adapters
        if (pl.S > 16) pl.S = 16;
    }
    if (pl.S > K / 256) pl.S = K / 256;   // a 32-K step per warp
    if (pl.S < 1) pl.S = 1;
    auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
    pl.base_ws = up(w4a16_workspace_bytes(m, N, K, group));
    pl.off_y = pl.base_ws;
    pl.off_part = pl.off_y + up((size_t)pl.slices * m * N * 4);
    pl.off_tiles = pl.off_part + up((size_t)pl.S * m * rank * 4);
    pl.off_ntiles = pl.off_tiles + up((size_t)pl.tiles * sizeof(RouteTile));
    pl.off_rows = pl.off_ntiles + 256;
    pl.off_hist = pl.off_rows + up((size_t)m * 4);
    pl.total = pl.off_hist + up(route_sort_workspace_bytes(m, 1, adapters, 1));
    return pl;
}

template <typename T>
int launch_lora_chunk(LoraParams p, const LoraPlan& pl, uint8_t* ws, const void* tiled, int group, int sym, int dtype,
                      int* dev_status, cudaStream_t stream) {
    const bool small = p.M <= kLoraSmallRows;
    float* y = reinterpret_cast<float*>(ws + pl.off_y);
    p.S = pl.S;
    p.part = reinterpret_cast<float*>(ws + pl.off_part);
    p.base = y;
    int items = p.M;
    if (!small) {
        RouteSort q = {};
        q.ids = p.row_adapter;
        q.T = p.M;
        q.k = 1;
        q.E = p.L;
        q.H = 8;
        q.spare = 1;
        q.rows = reinterpret_cast<int32_t*>(ws + pl.off_rows);
        q.hist = reinterpret_cast<int32_t*>(ws + pl.off_hist);
        q.tiles = reinterpret_cast<RouteTile*>(ws + pl.off_tiles);
        q.ntiles = reinterpret_cast<int*>(ws + pl.off_ntiles);
        q.tile_rows = 32;
        const int st = launch_route_sort(q, stream);
        if (st != W4A16_OK) return st;
        p.tiles = q.tiles;
        p.ntiles = q.ntiles;
        p.rows = q.rows;
        const int most = p.M / 32 + p.L + 1;
        items = p.M < most ? p.M : most;
    }
    const dim3 block(kLoraThreads), sgrid(p.S, items);
    cudaError_t e = small ? launch_pdl(lora_shrink_kernel<2, T>, sgrid, block, 0, stream, p)
                          : launch_pdl(lora_shrink_kernel<4, T>, sgrid, block, 0, stream, p);
    if (e != cudaSuccess) return W4A16_ECUDA;
    int slices = 1;
    const int st = launch_gemm_f32(p.A, dtype, p.M, p.K, tiled, p.N, group, sym, y, &slices, ws, dev_status, stream);
    if (st != W4A16_OK) return st;
    p.slices = slices;
    const int blocks = (p.N + 255) / 256;
    int n_sm = gemv_stream_sm_count();
    if (n_sm <= 0) n_sm = 148;
    // at least four CTAs per SM, then as many channel blocks per CTA as divide the rest (T's tile is
    // made once per CTA)
    const int busy = small ? 1 : (p.M + 31) / 32;
    p.passes = blocks * busy / (4 * n_sm);
    if (p.passes < 1) p.passes = 1;
    if (p.passes > 8) p.passes = 8;
    const dim3 egrid((blocks + p.passes - 1) / p.passes, items);
    const int nb = small ? 1 : 2;
    const size_t smem = (size_t)2 * 16 * nb * lora_t_stride(p.r) * 2;
    e = small ? launch_pdl(lora_expand_kernel<1, T>, egrid, block, smem, stream, p)
              : launch_pdl(lora_expand_kernel<2, T>, egrid, block, smem, stream, p);
    return e == cudaSuccess ? W4A16_OK : W4A16_ECUDA;
}

}  // namespace

size_t lora_workspace_bytes(int M, int N, int K, int group, int rank, int adapters) {
    // the last chunk may be short enough for the small-row kernels, whose plan differs
    const LoraPlan a = plan_lora(M, N, K, group, rank, adapters);
    size_t need = a.total;
    const int rest = M % a.rows;
    if (rest) {
        const LoraPlan b = plan_lora(rest, N, K, group, rank, adapters);
        if (b.total > need) need = b.total;
    }
    return need;
}

int launch_lora_gemm(const void* A, int a_dtype, int M, int K, const void* tiled, int N, int group, int sym,
                     const void* La, const void* Lb, const float* scale, int adapters, int rank,
                     const int32_t* row_adapter, void* C, void* workspace, int* dev_status, cudaStream_t stream) {
    const int chunk = lora_chunk_rows(M, N);
    for (int m0 = 0; m0 < M; m0 += chunk) {
        const int m = M - m0 < chunk ? M - m0 : chunk;
        const LoraPlan pl = plan_lora(m, N, K, group, rank, adapters);
        LoraParams p = {};
        p.A = static_cast<const uint8_t*>(A) + (size_t)m0 * K * 2;
        p.La = La;
        p.Lb = Lb;
        p.scale = scale;
        p.row_adapter = row_adapter + m0;
        p.C = static_cast<uint8_t*>(C) + (size_t)m0 * N * 2;
        p.M = m;
        p.K = K;
        p.N = N;
        p.r = rank;
        p.L = adapters;
        uint8_t* ws = static_cast<uint8_t*>(workspace);
        const int st = a_dtype == W4A16_BF16
                           ? launch_lora_chunk<__nv_bfloat16>(p, pl, ws, tiled, group, sym, a_dtype, dev_status, stream)
                           : launch_lora_chunk<__half>(p, pl, ws, tiled, group, sym, a_dtype, dev_status, stream);
        if (st != W4A16_OK) return st;
    }
    return W4A16_OK;
}

}  // namespace w4a16
