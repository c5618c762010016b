// lora.cu -- low-rank adapters of many requests at once beside the INT4 layer (sm_100a).
//
// C[m] = A[m] . dequant(W) + s_a (A[m] . La_a^T) . Lb_a^T,  a = row m's adapter (none: the first term).
//   shrink  T[m, j] = s_a sum_k A[m, k] La_a[j, k], FP32 partial sums over slices of K. Both operands of
//           its warp MMAs (m16n8k16) come straight from global memory: a lane reads 16 consecutive
//           bytes of a row and the same permutation of K stands on both sides. Rows of one adapter
//           within a block of 8 or 32 rows are taken together.
// Then, where the layer runs on the tensor cores (launch_lora_tc):
//   place   per block of BN rows, T as a matrix with one run of columns per adapter of the block, its
//           rows' values there (as bf16 hi + lo) and zeros in the other rows;
//   layer   the tensor-core GEMM (kTcLora), whose tiles go on over those columns: the second product is
//           a few more steps of the same accumulation. One rounding, no intermediate of C's size. (A
//           kernel that added T . Lb^T to FP32 outputs of the layer took 93 us of every 512 rows
//           of the 4096 x 28672 layer, beside the layer's 117.)
// and for few rows, where the decode kernel streams the layer (launch_lora_gemv):
//   layer   that kernel (gemv_stream.cu), whose compute warps add a tile's T . Lb^T to their sums by a few
//           more MMAs.
// The kernels follow each other by programmatic dependent launch.
#include <type_traits>

#include "gemm_tc_kernel.cuh"
#include "pdl.cuh"
#include "routed.cuh"

namespace w4a16 {
namespace {

constexpr int kLoraThreads = 256, kLoraWarps = kLoraThreads / 32;
constexpr size_t kLoraPlaceBytes = (size_t)64 << 20;   // T as placed, held at a time (or 256 rows of it)
constexpr int kLoraMaxChunk = 16384;

struct LoraParams {
    const void* A;              // [M, K]
    const void* La;             // [L, r, K]
    const void* Lb;             // [L, N, r]
    const float* scale;         // [L]
    const int32_t* row_adapter; // [M]
    float* part;                // [S][M][r]
    int* units;                 // tensor cores: the row blocks' low-rank units and pieces (null: none wanted)
    int* pieces;
    int* place;                 // [M] a row's adapter's place among those of its row block (-1: none)
    int* bad;
    int* slices;                // the slices that the shrink kernel took, of at most S (null: S)
    int bn, max_units, per, lists;
    void* C;
    int M, K, N, r, L, S;
};

// Row `lane` of a block of up to 32 rows from row m0: its adapter (-1: none), the lanes that share it,
// and one bit per adapter of the block, at its first row.
struct LoraBlock {
    int adapter;
    unsigned peers, firsts;
    __device__ __forceinline__ LoraBlock(const LoraParams& p, int m0, int rows) {
        const int lane = threadIdx.x & 31;
        adapter = lane < rows && m0 + lane < p.M ? p.row_adapter[m0 + lane] : -1;
        if ((unsigned)adapter >= (unsigned)p.L) adapter = -1;
        peers = __match_any_sync(0xffffffffu, adapter);
        firsts = __ballot_sync(0xffffffffu, adapter >= 0 && __ffs(peers) - 1 == lane);
    }
};

// slot[a]: place of adapter a among the adapters of the bn rows from m0, for those that are there. Four
// adapters per thread: f, their flags, and `before`, the first one's place. Returns how many there are.
__device__ __forceinline__ int lora_slots(const LoraParams& p, int m0, int bn, int* slot, int* wsum, int (&f)[4], int& before) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    for (int a = tid; a < p.L; a += kLoraThreads) slot[a] = 0;
    __syncthreads();
    for (int i = tid; i < bn && m0 + i < p.M; i += kLoraThreads) {
        const int a = p.row_adapter[m0 + i];
        if ((unsigned)a < (unsigned)p.L) slot[a] = 1;
    }
    __syncthreads();
    int c = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        f[q] = 4 * tid + q < p.L ? slot[4 * tid + q] : 0;
        c += f[q];
    }
    int x = c;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
    }
    if (lane == 31) wsum[warp] = x;
    __syncthreads();
    before = x - c;
    int total = 0;
#pragma unroll
    for (int w = 0; w < kLoraWarps; ++w) {
        if (w < warp) before += wsum[w];
        total += wsum[w];
    }
    int at = before;
#pragma unroll
    for (int q = 0; q < 4; ++q)
        if (4 * tid + q < p.L) {
            slot[4 * tid + q] = at;
            at += f[q];
        }
    __syncthreads();
    return total;
}

// The low-rank units, pieces and places of row block mb, and the flag of values that are not finite.
__device__ __forceinline__ void lora_list(const LoraParams& p, int mb) {
    __shared__ int slot[kRouteMaxBins];
    __shared__ int wsum[kLoraWarps];
    int f[4], before;
    const int total = lora_slots(p, mb * p.bn, p.bn, slot, wsum, f, before);
    const int pr = (p.r + 15) / 16, lu = (total * pr + p.per - 1) / p.per;
    int* pieces = p.pieces + (size_t)mb * p.max_units * p.per;
#pragma unroll
    for (int q = 0; q < 4; ++q)
        if (f[q]) {
            for (int j = 0; j < pr; ++j) pieces[before * pr + j] = 256 * (4 * threadIdx.x + q) + j;
            ++before;
        }
    for (int j = total * pr + threadIdx.x; j < lu * p.per; j += kLoraThreads) pieces[j] = -1;
    for (int m = mb * p.bn + threadIdx.x; m < min((mb + 1) * p.bn, p.M); m += kLoraThreads) {
        const int a = p.row_adapter[m];
        p.place[m] = (unsigned)a < (unsigned)p.L ? slot[a] : -1;
    }
    if (threadIdx.x == 0) {
        p.units[mb] = lu;
        if (mb == 0) *p.bad = 0;
    }
}

// T's partial sums. An item is one adapter's rows within a block of 8 NB rows, 16 RB ranks of it and one
// slice of K; the items are dealt out to the CTAs. How many slices there are goes by the number of
// items (p.slices: at most p.S, and the kernel says how many it took): 154 rows of 49 adapters have ten
// times the items of 154 rows of one. Warp w takes every eighth 32-K step of the slice; MMA rows are ranks,
// MMA columns the adapter's rows. With p.units, the first p.lists CTAs list the row blocks' units instead.
// RB: 16-rank blocks of one item.
template <int NB, int RB, typename T>
__global__ void __launch_bounds__(kLoraThreads, 2) lora_shrink_kernel(const LoraParams p) {
    __shared__ float red[4][RB * NB * 128];
    __shared__ int list[32];
    __shared__ int before[NB == 1 ? 1 : kLoraMaxChunk / 32 + 1];   // adapters of the blocks before each
    using Ops = GsOps<T>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    pdl_wait();
    pdl_trigger();   // (after the wait: the decode layer reads before its own, pdl.cuh)
    if ((int)blockIdx.x < p.lists) {
        lora_list(p, blockIdx.x);
        return;
    }
    const int cta = blockIdx.x - p.lists, ctas = gridDim.x - p.lists;
    const int blocks = (p.M + 8 * NB - 1) / (8 * NB), chunks = (p.r + 16 * RB - 1) / (16 * RB);
    int S = p.S, pairs;
    if constexpr (NB == 1) {   // (one block)
        pairs = __popc(LoraBlock(p, 0, 8).firsts);
    } else {
        for (int b0 = warp; b0 < blocks; b0 += 4 * kLoraWarps) {
            int a[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int m = 32 * (b0 + q * kLoraWarps) + lane;
                a[q] = m < p.M ? p.row_adapter[m] : -1;
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if ((unsigned)a[q] >= (unsigned)p.L) a[q] = -1;
                const unsigned peers = __match_any_sync(0xffffffffu, a[q]);
                const int n = __popc(__ballot_sync(0xffffffffu, a[q] >= 0 && __ffs(peers) - 1 == lane));
                if (lane == 0 && b0 + q * kLoraWarps < blocks) before[b0 + q * kLoraWarps] = n;
            }
        }
        __syncthreads();
        if (warp == 0) {
            int base = 0;
            for (int b = lane; b - lane < blocks; b += 32) {
                const int n = b < blocks ? before[b] : 0;
                int x = n;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, x, d);
                    if (lane >= d) x += y;
                }
                if (b < blocks) before[b] = base + x - n;
                base += __shfl_sync(0xffffffffu, x, 31);
            }
            if (lane == 0) before[blocks] = base;
        }
        __syncthreads();
        pairs = before[blocks];
        if (p.slices) {
            // the fewest rounds: a CTA's items one after another, each a step per 256 K of its slice and
            // about four steps' time besides (lane s: s + 1 slices; the fewest slices among equals)
            const int rounds = (pairs * chunks * (lane + 1) + ctas - 1) / ctas;
            const int cost = rounds * (4 + (p.K + 256 * (lane + 1) - 1) / (256 * (lane + 1)));
            const unsigned best = __reduce_min_sync(0xffffffffu, lane < p.S ? (unsigned)cost : 0xffffffffu);
            S = __ffs(__ballot_sync(0xffffffffu, lane < p.S && (unsigned)cost == best));
            if (cta == 0 && threadIdx.x == 0) *p.slices = S;
        }
    }
    const int items = pairs * chunks * S;
    for (int item = cta; item < items; item += ctas) {
    const int sl = item % S, pc = item / S, r0 = pc % chunks * 16 * RB;
    int nth = pc / chunks, block = 0;
    if constexpr (NB > 1) {
        int hi = blocks - 1;   // the last block with no more than nth adapters before it
        while (block < hi) {
            const int m = (block + hi + 1) >> 1;
            if (before[m] <= nth) block = m;
            else hi = m - 1;
        }
        nth -= before[block];
    }
    const LoraBlock blk(p, block * 8 * NB, 8 * NB);
    unsigned left = blk.firsts;
    for (int q = 0; q < nth; ++q) left &= left - 1;
    const int first = __ffs(left) - 1;
    const int adapter = __shfl_sync(0xffffffffu, blk.adapter, first);
    const unsigned same = __shfl_sync(0xffffffffu, blk.peers, first);
    const int n = __popc(same);
    __syncthreads();   // (the last item's rows have been used)
    if (threadIdx.x < 32 && ((same >> lane) & 1u)) list[__popc(same & ((1u << lane) - 1u))] = block * 8 * NB + lane;
    __syncthreads();
    const T* A = static_cast<const T*>(p.A);
    const T* La = static_cast<const T*>(p.La) + (size_t)adapter * p.r * p.K;
    const int steps = p.K / 32;
    const int s0 = (int)((long long)steps * sl / S), s1 = (int)((long long)steps * (sl + 1) / S);
    const T* x[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) x[b] = 8 * b + g < n ? A + (size_t)list[8 * b + g] * p.K + 8 * t : nullptr;
    {
        float acc[RB][NB][4];
#pragma unroll
        for (int q = 0; q < RB; ++q)
#pragma unroll
            for (int b = 0; b < NB; ++b) acc[q][b][0] = acc[q][b][1] = acc[q][b][2] = acc[q][b][3] = 0.0f;
        const int nq = min(RB, (p.r - r0 + 15) / 16);
#pragma unroll(RB == 1 ? 4 : RB == 2 ? 2 : 1)
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
                        if (8 * b >= n) break;   // no row of the adapter in this block of columns
                        Ops::mma(acc[q][b], lo[q].x, hi[q].x, lo[q].y, hi[q].y, xv[b].x, xv[b].y);
                        Ops::mma(acc[q][b], lo[q].z, hi[q].z, lo[q].w, hi[q].w, xv[b].z, xv[b].w);
                    }
        }
        // the warps' sums in a fixed order: 4..7 onto 0..3 through shared memory, then one thread per
        // output adds the four
        auto each = [&](auto f) {
#pragma unroll
            for (int q = 0; q < RB; ++q)
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (q < nq && 8 * b < n) f(acc[q][b][e], ((q * NB + b) * 4 + e) * 32 + lane);
        };
        if (warp >= 4) each([&](float& v, int at) { red[warp - 4][at] = v; });
        __syncthreads();
        if (warp < 4) each([&](float& v, int at) { red[warp][at] += v; });
        __syncthreads();
        float* out = p.part + (size_t)sl * p.M * p.r;
        for (int o = threadIdx.x; o < n * RB * 16; o += kLoraThreads) {
            const int m = o / (RB * 16), j = o % (RB * 16);   // the adapter's row m, rank r0 + j
            const int at = (((j >> 4) * NB + (m >> 3)) * 4 + (m & 1) + ((j >> 2) & 2)) * 32 + (j & 7) * 4 + ((m & 7) >> 1);
            if (r0 + j < p.r) out[(size_t)list[m] * p.r + r0 + j] = (red[0][at] + red[1][at]) + (red[2][at] + red[3][at]);
        }
    }
    }
}

// T as the tensor-core layer takes it. A row block (bn rows) has its adapters in order, each with
// pr = ceil(r / 16) pieces of 16 ranks, `per` pieces (4 in a bf16 layer, 2 in an fp16 one) to a low-rank
// unit of 128 columns: per piece [hi | lo] (bf16), or [hi | lo | hi | 0] (fp16, whose Lb is split into hi and
// lo too). `warps` (1, 2, 4 or 8) warps write one row, all units of its block.
template <typename T>
__global__ void __launch_bounds__(kLoraThreads) lora_place_kernel(const LoraParams p, __nv_bfloat16* __restrict__ placed,
                                                                  int warps) {
    constexpr int kPer = std::is_same<T, __nv_bfloat16>::value ? 4 : 2;
    __shared__ __align__(16) __nv_bfloat16 hi[kLoraWarps][kLoraMaxRank], lo[kLoraWarps][kLoraMaxRank];
    const int warp = threadIdx.x >> 5, local = warp / warps, at = threadIdx.x - local * warps * 32, step = 32 * warps;
    const int row = blockIdx.x * (kLoraWarps / warps) + local;
    const int pr = (p.r + 15) / 16;
    pdl_wait();
    pdl_trigger();   // (after the wait: the layer reads and writes before its own, pdl.cuh)
    const int mine = row < p.M ? __ldcg(p.place + row) : -1;
    const int columns = row < p.M ? 16 * __ldcg(p.units + row / p.bn) : 0;   // of 8 values
    if (mine >= 0) {
        const float sc = __ldg(p.scale + p.row_adapter[row]);
        const int S = __ldcg(p.slices);
        for (int j = at; j < 16 * pr; j += step) {
            float s = 0.0f;
            if (j < p.r)
#pragma unroll 16
                for (int k = 0; k < S; ++k) s += __ldcg(p.part + ((size_t)k * p.M + row) * p.r + j);
            s *= sc;
            const __nv_bfloat16 h = __float2bfloat16_rn(s);
            hi[local][j] = h;
            lo[local][j] = __float2bfloat16_rn(s - __bfloat162float(h));
        }
    }
    __syncthreads();
    uint4* out = reinterpret_cast<uint4*>(placed + (size_t)row * p.max_units * 128);
    for (int q = at; q < columns; q += step) {   // unit q / 16, block (q / 4) % 4, part q % 4
        const int b = (q >> 2) & 3, part = q & 3;
        const int piece = (q >> 4) * kPer + (kPer == 4 ? b : b >> 1) - mine * pr;   // of the row's adapter
        uint4 v = make_uint4(0, 0, 0, 0);
        if (mine >= 0 && (unsigned)piece < (unsigned)pr && !(kPer == 2 && (b & 1) && part >= 2)) {
            const __nv_bfloat16* src = part < 2 ? hi[local] : lo[local];
            v = *reinterpret_cast<const uint4*>(src + 16 * piece + 8 * (part & 1));
        }
        out[q] = v;
    }
}

// ------------------------------------------------------------------------------ host side
// K slices of the shrink kernel at most: about two CTAs per SM when rows share adapters, a 32-K step per warp.
int shrink_slices(int M, int K, int rows, int n_sm) {
    int S = 2 * n_sm / ((M + rows - 1) / rows);
    if (S > 32) S = 32;
    if (S > K / 256) S = K / 256;
    return S < 1 ? 1 : S;
}

int lora_sm_count() {
    const int n = gemv_stream_sm_count();
    return n > 0 ? n : 148;
}

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

struct LoraGemvPlan {
    int S;
    size_t off_part, total;
};

LoraGemvPlan plan_lora_gemv(int M, int N, int K, int group, int rank) {
    LoraGemvPlan pl = {};
    const GemvStreamPlan q = plan_gemv_lora(M, N, K, group, 0, lora_sm_count(), rank);
    if (!q.ok) return pl;
    pl.S = shrink_slices(M, K, 8, lora_sm_count());
    pl.off_part = up256(kGemvStreamCounterBytes + q.partial_bytes);
    pl.total = pl.off_part + up256((size_t)pl.S * M * rank * 4);
    return pl;
}

// The decode kernel takes up to 8 rows, and two values of t per thread.
bool lora_gemv_fits(int M, int rank) { return M <= 8 && M * rank <= 1024; }

struct LoraTcPlan {
    int rows;        // rows of A taken at a time
    int bn, mblocks; // of a piece of `rows` rows
    int S, per, max_units;
    size_t off_part, off_placed, off_units, off_pieces, off_place, off_bad, total;
};

LoraTcPlan plan_lora_tc(int M, int K, int rank, int adapters, int per) {
    LoraTcPlan pl = {};
    pl.per = per;
    pl.bn = M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : M <= 128 ? 128 : 256;
    const int most = adapters < pl.bn ? adapters : pl.bn;   // adapters of a row block
    pl.max_units = (most * ((rank + 15) / 16) + per - 1) / per;
    size_t rows = kLoraPlaceBytes / ((size_t)pl.max_units * 256) / 256 * 256;
    if (rows < 256) rows = 256;
    if (rows > (size_t)kLoraMaxChunk) rows = kLoraMaxChunk;
    pl.rows = (size_t)M < rows ? M : (int)rows;
    pl.mblocks = (pl.rows + pl.bn - 1) / pl.bn;
    pl.S = shrink_slices(pl.rows, K, 32, lora_sm_count());
    pl.off_part = up256(kGemvStreamCounterBytes + (size_t)2 * lora_sm_count() * pl.bn * 128 * sizeof(float));
    // S M of any piece: one slice of up to `rows` rows, or at most two CTAs per SM of 32 rows each
    size_t sm = (size_t)64 * lora_sm_count();
    if (sm > (size_t)32 * pl.rows) sm = (size_t)32 * pl.rows;
    if (sm < (size_t)pl.rows) sm = (size_t)pl.rows;
    pl.off_placed = pl.off_part + up256(sm * rank * 4);
    pl.off_units = pl.off_placed + up256((size_t)pl.rows * pl.max_units * 256);
    pl.off_pieces = pl.off_units + up256((size_t)pl.mblocks * 4);
    pl.off_place = pl.off_pieces + up256((size_t)pl.mblocks * pl.max_units * per * 4);
    pl.off_bad = pl.off_place + up256((size_t)pl.rows * 4);
    pl.total = pl.off_bad + 256;
    return pl;
}

// ctas: for the items, beside the lists.
template <int NB, typename T>
cudaError_t launch_shrink(const LoraParams& p, int ctas, cudaStream_t stream) {
    const dim3 grid(ctas + p.lists), block(kLoraThreads);
    if (p.r <= 16) return launch_pdl(lora_shrink_kernel<NB, 1, T>, grid, block, 0, stream, p);
    if (NB > 1 || p.r <= 32) return launch_pdl(lora_shrink_kernel<NB, 2, T>, grid, block, 0, stream, p);
    return launch_pdl(lora_shrink_kernel<NB, NB == 1 ? 4 : 2, T>, grid, block, 0, stream, p);
}

template <typename T>
int launch_lora_gemv(LoraParams p, const LoraGemvPlan& pl, uint8_t* ws, const void* tiled, int group, int sym, int dtype,
                     int* dev_status, cudaStream_t stream) {
    p.S = pl.S;
    p.part = reinterpret_cast<float*>(ws + pl.off_part);
    const int chunks = p.r <= 32 ? 1 : (p.r + 63) / 64;
    if (launch_shrink<1, T>(p, p.S * p.M * chunks, stream) != cudaSuccess) return W4A16_ECUDA;
    GemvLora lora = {};
    lora.b = p.Lb;
    lora.scale = p.scale;
    lora.row_adapter = p.row_adapter;
    lora.part = p.part;
    lora.slices = pl.S;
    lora.rank = p.r;
    lora.adapters = p.L;
    return launch_gemv_lora(p.A, dtype, p.M, p.K, tiled, p.N, group, sym, p.C, lora, ws, dev_status, stream);
}

// One piece of rows on the tensor cores. `pl` is the whole batch's plan: its offsets, bn and widths
// hold for every piece.
template <typename T>
int launch_lora_tc(LoraParams p, const LoraTcPlan& pl, uint8_t* ws, const void* tiled, int group, int sym, int dtype,
                   int* dev_status, cudaStream_t stream) {
    const int mblocks = (p.M + pl.bn - 1) / pl.bn, n_sm = lora_sm_count();
    const long long least = (long long)(p.N / 128) * mblocks * (p.K / 128);   // units without the low-rank ones
    const TcPlan tp = plan_tc_rows(pl.bn, p.N, p.K, group, sym, (int)(least < n_sm ? least : n_sm), 32 + (size_t)(mblocks + 1) * 4);
    if (!tp.ok) return W4A16_EUNSUPPORTED;
    p.S = shrink_slices(p.M, p.K, 32, n_sm);
    p.part = reinterpret_cast<float*>(ws + pl.off_part);
    __nv_bfloat16* placed = reinterpret_cast<__nv_bfloat16*>(ws + pl.off_placed);
    p.units = reinterpret_cast<int*>(ws + pl.off_units);
    p.pieces = reinterpret_cast<int*>(ws + pl.off_pieces);
    p.place = reinterpret_cast<int*>(ws + pl.off_place);
    p.bad = reinterpret_cast<int*>(ws + pl.off_bad);
    p.slices = p.bad + 1;
    p.lists = mblocks;
    p.bn = pl.bn;
    p.max_units = pl.max_units;
    p.per = pl.per;
    if (launch_shrink<4, T>(p, 2 * n_sm, stream) != cudaSuccess) return W4A16_ECUDA;
    int warps = 1;   // of one row: up to four CTAs per SM in all
    while (warps < kLoraWarps && (long long)p.M * warps * 2 <= (long long)4 * n_sm * kLoraWarps) warps *= 2;
    if (launch_pdl(lora_place_kernel<T>, dim3((p.M * warps + kLoraWarps - 1) / kLoraWarps), dim3(kLoraThreads), 0, stream, p,
                   placed, warps) != cudaSuccess)
        return W4A16_ECUDA;
    CUtensorMap map, map_t;
    if (!make_act_map(&map, p.A, p.M, p.K, pl.bn, dtype == W4A16_BF16) ||
        !make_act_map(&map_t, placed, p.M, pl.max_units * 128, pl.bn, true))
        return W4A16_ECUDA;
    TcParams prm = tc_params(tp, tiled, p.M, p.N, p.K, group, sym, dtype == W4A16_BF16, ws, dev_status);
    prm.mblocks = mblocks;
    prm.C = p.C;
    prm.off_grp = tp.off_bar + 1024;
    prm.lora_units = p.units;
    prm.lora_pieces = p.pieces;
    prm.lora_b = p.Lb;
    prm.row_adapter = p.row_adapter;
    prm.lora_bad = p.bad;
    prm.max_pieces = pl.max_units * pl.per;
    prm.rank = p.r;
    prm.adapters = p.L;
    return launch_tc_bn<T, kTcLora>(pl.bn, map, map_t, prm, tp.smem, stream);
}

}  // namespace

size_t lora_workspace_bytes(int M, int N, int K, int group, int rank, int adapters) {
    // the largest need over both types and both forms, so that a forced kernel also fits, and over all batches
    // of up to M rows (the tensor cores' grows with M)
    const size_t a = plan_lora_tc(M, K, rank, adapters, 2).total, b = plan_lora_tc(M, K, rank, adapters, 4).total;
    size_t most = a > b ? a : b;
    for (int m = 1; m <= M && lora_gemv_fits(m, rank); ++m) {
        const size_t gemv = plan_lora_gemv(m, N, K, group, rank).total;
        if (gemv > most) most = gemv;
    }
    return most;
}

int lora_select_kernel(int M, int N, int K, int group, int rank) {
    return lora_gemv_fits(M, rank) && w4a16_select_kernel(M, N, K, group) == W4A16_KERNEL_GEMV &&
                   plan_lora_gemv(M, N, K, group, rank).total
               ? W4A16_KERNEL_GEMV
               : W4A16_KERNEL_TC;
}

int launch_lora_gemm(const void* A, int a_dtype, int M, int K, const void* tiled, int N, int group, int sym,
                     const void* La, const void* Lb, const float* scale, int adapters, int rank,
                     const int32_t* row_adapter, void* C, void* workspace, int* dev_status, cudaStream_t stream) {
    const bool bf16 = a_dtype == W4A16_BF16;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    LoraParams p = {};
    p.A = A;
    p.La = La;
    p.Lb = Lb;
    p.scale = scale;
    p.row_adapter = row_adapter;
    p.C = C;
    p.M = M;
    p.K = K;
    p.N = N;
    p.r = rank;
    p.L = adapters;
    if (lora_select_kernel(M, N, K, group, rank) == W4A16_KERNEL_GEMV) {
        const LoraGemvPlan pl = plan_lora_gemv(M, N, K, group, rank);
        return bf16 ? launch_lora_gemv<__nv_bfloat16>(p, pl, ws, tiled, group, sym, a_dtype, dev_status, stream)
                    : launch_lora_gemv<__half>(p, pl, ws, tiled, group, sym, a_dtype, dev_status, stream);
    }
    const LoraTcPlan pl = plan_lora_tc(M, K, rank, adapters, bf16 ? 4 : 2);
    for (int m0 = 0; m0 < M; m0 += pl.rows) {
        p.M = M - m0 < pl.rows ? M - m0 : pl.rows;
        p.A = static_cast<const uint8_t*>(A) + (size_t)m0 * K * 2;
        p.C = static_cast<uint8_t*>(C) + (size_t)m0 * N * 2;
        p.row_adapter = row_adapter + m0;
        const int st = bf16 ? launch_lora_tc<__nv_bfloat16>(p, pl, ws, tiled, group, sym, a_dtype, dev_status, stream)
                            : launch_lora_tc<__half>(p, pl, ws, tiled, group, sym, a_dtype, dev_status, stream);
        if (st != W4A16_OK) return st;
    }
    return W4A16_OK;
}

}  // namespace w4a16
