// gemm_tc_kernel.cuh -- persistent stream-K tcgen05 tensor-core W4A16 GEMM for sm_100a: the larger-M
// path of the dense layer, and the experts' products on sorted rows (runs of rows with a weight each).
//
// C[M, N] = A[M, K] . dequant(W)[K, N], FP32 accumulation in tensor memory.
// "4.3 Weight-only INT4", section 4: read, unpack, dequantize and multiply in one pipeline, each
// weight byte crossing HBM once, data movement overlapped with on-chip compute; section 1: codes
// dequantized on chip to FP16/BF16, multiply inputs stay 16-bit. "INT8 vs INT4 Quantization, in
// depth", "Two regimes": for tens of rows the layer still waits for memory, so every SM streams
// weights; for hundreds it waits for the tensor cores.
//
// Mapping. The MMA computes D[n, m] = sum_k W^T[n, k] A^T[k, m] (swap-AB): the dequantized weight
// tile (128 output channels x 64 K) is operand A (M_mma = 128), the activation tile (BN rows of
// A x 64 K, 128-byte swizzle, loaded by TMA) is operand B (N_mma = BN), D (128 x BN, FP32) lives
// in tensor memory, lane = output channel, column = row of A.
//
// Work split (stream-K). A tile is 128 output channels x one block of BN rows of A, the whole K;
// tiles are ordered channel-major (the row blocks of one channel tile are neighbours, so their
// weights are read from HBM once and from L2 after). The U = tiles x K/128 unit steps (one unit
// record of the tiled buffer each) are cut into P contiguous ranges, one per SM, so every SM
// streams the same number of weight bytes whatever the shape. A tile cut between CTAs cf < ... <
// cl is the last of cf's range and the first of every later one: each later CTA publishes its
// FP32 sums to the workspace and counts them (release, no wait); cf, after its own last unit,
// waits for the count (acquire, bounded), adds the sums in CTA order, writes C and resets the
// counter. The result does not depend on timing.
// (Launches with adapters or experts, from 64 rows per tile: every CTA of a cut tile publishes, and
// all of them add up a share of its rows once their ranges are done; tc_share.)
// (They also choose, from the number and length of their tiles, between this cut, ranges of whole tiles, and ranges
// that each lie within one tile; kTcCutOne.)
//
// Warp roles (768 threads):
//   warp 0      : weight loader -- one bulk copy per two unit records (codes, scales and zeros
//                 of 2 x 128 K, contiguous in the tiled buffer) into a ring of record slots.
//   warp 1      : activation loader -- per 128-K step (one unit), two TMA boxes of BN rows x
//                 64 K into the step's slot of a ring (4-7 slots: the tiles come from L2, and a
//                 slot stays busy until its MMAs complete); owns the tensor memory.
//   warps 2, 3  : MMA issuers (two below BN = 128, one at 128) -- lane 0 of warp 2 + j takes the
//                 units j, j + 2, .. of the range:
//                 the eight tcgen05.mma (K = 16 each) of a step, operand A (the weights) from
//                 tensor memory and B (the activations) from shared memory, into issuer j's own
//                 accumulator of the tile, and one commit that frees the step's activation and
//                 weight tiles together; after a tile's last step a commit to the tile's barrier
//                 (one arrival per issuer). The epilogue adds the accumulators.
//   warps 4..7  : epilogue -- tcgen05.ld of the accumulator (warp w reads lanes 32 (w % 4) ..),
//                 then C (or the published partial sums of a cut tile); two accumulators, so one
//                 tile's epilogue runs under the next tile's MMAs.
//   warps 8..23 : dequantize -- thread (n, b) turns the 32 codes of channel n in 32-K block b
//                 of a unit into 16-bit weights (u - z) s (one rounding) and stores them with
//                 tcgen05.st into a ring of weight tiles in tensor memory (lane n = channel n, 64
//                 columns of K pairs per 128-K step); warp w writes the lanes 32 (w % 4) .. its
//                 channels occupy.
// Unit-scaled mode (BN = 16, group 128, where one group spans a unit): the dequant warps store
// u - z only (exact in 16 bits), each unit's MMAs go to a fresh accumulator (two per issuer), and
// the epilogue warps add s times the unit's sums into registers as each unit completes, saving the
// dequant warps the scale multiply (two instructions per register with bf16).
// Tensor memory (512 columns): two tiles in flight (one at BN = 256), each with one accumulator per
// issuer (BN columns), then the weight tiles of the step ring (64 columns per step). A has at
// most 256 rows per tile (one MMA of N = 256 per K step); more rows of A are more tiles (row
// blocks), whose weights are dequantized again but read from L2.
// Record slots are freed by the dequant warps, activation and weight-tile slots by the MMA
// commits, so the weight stream runs several units ahead of the tensor cores, and the shared
// memory holds only copies in flight (weight records and activation tiles).
// Every wait on an mbarrier or a tile counter is bounded; on expiry the kernel records
// W4A16_ETIMEOUT in dev_status, every role stops, the loaders wait for their copies in flight,
// the MMA thread waits for its last MMAs, and the CTA frees its tensor memory and returns.
#pragma once

#include <type_traits>

#include "common.cuh"
#include "dequant.cuh"
#include "moe_walk.cuh"
#include "pdl.cuh"
#include "sm100_ptx.cuh"
#include "tiled_layout.cuh"

namespace w4a16 {

namespace {

using namespace sm100;

// Rows of one activation box of a grouped launch: a tile loads as many boxes as its rows need.
__host__ __device__ constexpr int tc_box_rows(int bn) { return bn < 64 ? bn : 64; }

// What the tiles are and where the sums go.
constexpr int kTcDense = 0;     // rows [0, M) of A, C in the type of A
constexpr int kTcLora = 1;      // the same, each tile with the low-rank units of its row block (lora.cu)
constexpr int kTcGrouped = 2;   // runs of rows with a weight of their own each (experts): offsets on the device

// Whether the CTAs of a cut tile share the sum of its rows at the end, or the one that opened it adds the
// others' sums in its epilogue. Measured (us, shared against not): 256-row tiles, 295 x 4224 x 1920 with
// adapters 44 / 71, 844 x 768 x 896 38 / 72; 16-row tiles, 64 experts of 2048 x 1408 44.9 / 40.1.
__host__ __device__ constexpr bool tc_share(int bn, int mode) { return mode != kTcDense && bn >= 64; }

// Units that the exchange of a cut tile's sums costs, beside half a unit for every CTA of the tile: where the
// CTAs of a tile have no other, and where a range may end one cut tile and open the next. They decide how
// launches with adapters or experts are cut. Measured (us, cut evenly whatever the sizes against so): 144 rows of 4
// experts of 768 x 1280 16.0 / 9.9, 3000 of 16 of 1024 x 512 27.3 / 14.9, 11264 of 3 of 6144 x 384 74 / 51; 500 of
// 4 of 5120 x 640, whose tiles are cut either way, 22.7 / 19.0.
constexpr int kTcCutOne = 4;
__host__ __device__ constexpr int tc_cut_two(bool share) { return share ? 14 : 10; }

constexpr int kTcThreads = 768;
constexpr int kTcWarpLoadW = 0, kTcWarpLoadA = 1, kTcWarpMma = 2, kTcWarpEpi = 4, kTcWarpDeq = 8;
constexpr int kTcDeqWarps = 16;
// unit records per record slot (one bulk copy): two, one at BN = 256 (whose activation tiles take
// most of the shared memory)
__host__ __device__ constexpr int tc_units_per_load(int bn) { return bn >= 256 ? 1 : 2; }
constexpr int kTcSmemMax = 227 * 1024;
constexpr int kTcMaxRing = 16;
constexpr int kTcTmemCols = 512;
constexpr int kTcStepCols = 64;        // tensor-memory columns of one 128-K weight tile (K pairs)

// MMA threads: two below BN = 128 (issuer j takes the units j, j + 2, .. of the range; at small N
// one thread's issue rate, not the tensor pipe, sets the time), one from BN = 128. Tensor memory:
// two tiles in flight below BN = 256 (one tile's epilogue runs under the next tile's MMAs), one
// at 256, each with one accumulator per issuer (BN columns, at least 32), then the step ring's
// weight tiles: as many as fit, at most 8; at BN = 256 three (the shared memory holds three
// activation tiles of 64 KiB).
__host__ __device__ constexpr int tc_issuers(int bn) { return bn >= 128 ? 1 : 2; }
__host__ __device__ constexpr int tc_acc_bufs(int bn) { return bn >= 256 ? 1 : 2; }
__host__ __device__ constexpr int tc_acc_cols(int bn) { return bn < 32 ? 32 : bn; }
__host__ __device__ constexpr int tc_steps(int bn) {
    return bn >= 256 ? 3
                     : ((kTcTmemCols - 2 * tc_issuers(bn) * tc_acc_cols(bn)) / kTcStepCols > 8
                            ? 8
                            : (kTcTmemCols - 2 * tc_issuers(bn) * tc_acc_cols(bn)) / kTcStepCols);
}
constexpr uint64_t kTcDrainNs = 2000000000ull;

struct TcParams {
    const uint8_t* tiled;
    void* C;
    int* counters;      // one int per tile, zero between calls
    float* partials;    // [P][BN][128]: sums a CTA publishes for the tile that opens its range; kTcLora,
                        // kTcGrouped: [P][2][BN][128], for the cut tiles that open and that end its range
    int* dev_status;
    const int32_t* offsets;   // kTcGrouped: rows offsets[e] .. offsets[e + 1] - 1 meet weight e < E
    int E;
    uint32_t off_grp;         // kTcGrouped, kTcLora: shared-memory offset of the runs' (units') table
    const int* lora_units;    // kTcLora: [mblocks] low-rank units of a row block,
    const int* lora_pieces;   //   [mblocks][max_pieces] 256 a + p: ranks 16 p .. of adapter a, or -1
    const void* lora_b;       //   [adapters][N][rank]
    const int32_t* row_adapter;
    int* lora_bad;            //   set to 1 when some value of a used Lb is not finite
    int max_pieces, rank, adapters;
    int M, K, N, sym, group;
    uint32_t record, scales_off, zeros_off, slot_w;
    int P, mblocks, nr;
    uint32_t off_w, off_bar;   // shared-memory offsets; the activation tiles start at 0
    uint64_t wait_ns;
    GsMasks km;
};

__device__ __forceinline__ long long tc_unit_begin(int c, long long U, int P) { return ((long long)c * U) / P; }
__device__ __forceinline__ int tc_unit_owner(long long u, long long U, int P) {
    return (int)(((u + 1) * P - 1) / U);
}

__device__ __forceinline__ void tc_named_bar(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Two values rounded to T, the first in the low half.
template <typename T>
__device__ __forceinline__ uint32_t tc_pack2(float a, float b) {
    if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    } else {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
}

// The thread's tensor-memory loads have arrived; `v` is named so that no use of it moves ahead.
__device__ __forceinline__ void tc_ld_wait16(uint32_t (&v)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                   "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15])
                 :
                 : "memory");
}

// Warp-uniform bounded wait.
__device__ __forceinline__ bool tc_wait(uint64_t* bar, uint32_t parity, volatile int* abort, int* dev_status,
                                        uint64_t ns) {
    if (__all_sync(0xffffffffu, mbar_test_wait(bar, parity))) return true;
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, dev_status, ns));
}

// kTcLora: a role's place among the units. A tile (channel tile nt, row block mb) has UT = K / 128 weight
// units, then the row block's low-rank units: 128 K of the products T . Lb^T, where T (bf16, written by
// lora_place_kernel) holds, for every adapter of the row block, its rows' rank products as hi + lo and
// zeros in the other rows. cum: low-rank units before each row block.
struct TcLoraWalk {
    const int* cum = nullptr;
    int UT = 0, mblocks = 0, nt = 0, mb = 0, ku = 0, len = 0;
    __device__ __forceinline__ void init(const int* c, int units, int blocks, long long u) {
        cum = c;
        UT = units;
        mblocks = blocks;
        const long long S = (long long)mblocks * UT + cum[mblocks];
        nt = (int)(u / S);
        const int r = (int)(u - (long long)nt * S);
        int lo = 0, hi = mblocks - 1;
        while (lo < hi) {
            const int m = (lo + hi + 1) >> 1;
            if (m * UT + cum[m] <= r) lo = m;
            else hi = m - 1;
        }
        mb = lo;
        ku = r - (mb * UT + cum[mb]);
        len = UT + cum[mb + 1] - cum[mb];
    }
    // n units further, within the tile or to the start of the next one
    __device__ __forceinline__ void step(int n) {
        if ((ku += n) < len) return;
        ku = 0;
        if (++mb == mblocks) {
            mb = 0;
            ++nt;
        }
        len = UT + cum[mb + 1] - cum[mb];
    }
    __device__ __forceinline__ bool low() const { return ku >= UT; }
};

// US (unit-scaled, run at BN = 16 with group 128): every unit's MMAs go to an accumulator of
// their own, the dequant warps store the exact integers u - z, and the epilogue warps add s times
// each unit's sums into registers (the unit's scale s of channel n read from its record).
// Otherwise the dequant warps store (u - z) s and the MMAs accumulate a whole tile segment.
template <int BN, typename T, bool US, int MODE>
__global__ void __launch_bounds__(kTcThreads, 1)
tc_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmT, const TcParams p) {
    static_assert(!US || BN <= 32, "unit-scaled accumulation keeps BN sums per thread in registers");
    using Ops = GsOps<T>;
    constexpr int kCols = tc_acc_cols(BN);       // tensor-memory columns of one accumulator
    constexpr int kIss = tc_issuers(BN);         // MMA threads
    constexpr int kBufs = tc_acc_bufs(BN);       // tiles in flight
    constexpr int kUPL = tc_units_per_load(BN);  // unit records per record slot
    constexpr int NS = tc_steps(BN);             // steps in flight (activation + weight tiles)
    constexpr uint32_t kSlotA = (uint32_t)BN * 256u;   // 128 K of BN rows: two 64-K TMA boxes
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    // 1024-byte aligned base, kept a shared-memory pointer (no integer round trip)
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const int nr = p.nr;
    uint8_t* ring_a = smem;
    uint8_t* ring_w = smem + p.off_w;
    uint64_t* full_r = reinterpret_cast<uint64_t*>(smem + p.off_bar);
    uint64_t* empty_r = full_r + nr;
    uint64_t* full_a = empty_r + nr;     // [NS] the step's activation tile landed
    uint64_t* full_d = full_a + NS;      // [NS] the step's weight tile is in tensor memory
    uint64_t* free_s = full_d + NS;      // [NS] the step's MMAs completed: both tiles free
    constexpr int kAccBars = US ? 2 * kIss : 2;   // per tile buffer, or per accumulator (US)
    uint64_t* accfull = free_s + NS;              // [kAccBars]
    uint64_t* accempty = accfull + kAccBars;      // [kAccBars]
    uint64_t* lastmma = accempty + kAccBars;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(lastmma + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int UT = p.K / 128;                              // unit steps per tile
    constexpr bool kGrp = MODE == kTcGrouped, kLora = MODE == kTcLora;
    constexpr bool kShare = tc_share(BN, MODE);  // cut tiles are summed at the end, by all their CTAs
    long long* range = reinterpret_cast<long long*>(smem + p.off_grp);       // kShare, kTcLora: u0, u1, U, P and pieces
    const int2* run_tab = reinterpret_cast<const int2*>(range + 4);          // kTcGrouped
    const int* blk_tab = reinterpret_cast<const int*>(run_tab + p.E);
    int* cum_tab = reinterpret_cast<int*>(range + 4);                        // kTcLora
    const int cta = blockIdx.x;
    const uint32_t R = p.record;
    const uint64_t wait_ns = p.wait_ns;

    if (threadIdx.x == 0) {
        for (int i = 0; i < nr; ++i) {
            mbar_init(&full_r[i], 1);
            mbar_init(&empty_r[i], kTcDeqWarps);
        }
        for (int i = 0; i < NS; ++i) {
            mbar_init(&full_a[i], 1);
            mbar_init(&full_d[i], kTcDeqWarps);
            mbar_init(&free_s[i], 1);
        }
        for (int i = 0; i < kAccBars; ++i) {
            mbar_init(&accfull[i], US ? 1 : kIss);
            mbar_init(&accempty[i], 4);
        }
        mbar_init(lastmma, kIss);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kTcWarpLoadA) {
        tmem_alloc(tmem_slot, kTcTmemCols);
        tmem_relinquish();
    }
    if constexpr (MODE != kTcDense) {
        // (launched as a programmatic dependent: what it reads may be the previous kernel's. kTcLora: that one
        // only places T, which the activation loader waits for by itself; it lets this one start after
        // everything before it has completed.)
        if (!kLora) pdl_wait();
        pdl_trigger();
    }
    if constexpr (kGrp) {
        moe_table(p.offsets, p.E, p.M, BN, const_cast<int2*>(run_tab), const_cast<int*>(blk_tab), [] { cta_sync(); });
    }
    if constexpr (kLora) {
        if (warp == kTcWarpEpi) {
            int base = 0;
            for (int b0 = 0; b0 < p.mblocks; b0 += 32) {
                const int n = b0 + lane < p.mblocks ? __ldcg(p.lora_units + b0 + lane) : 0;
                int x = n;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, x, d);
                    if (lane >= d) x += y;
                }
                if (b0 + lane < p.mblocks) cum_tab[b0 + lane] = base + x - n;
                base += __shfl_sync(0xffffffffu, x, 31);
            }
            if (lane == 0) cum_tab[p.mblocks] = base;
        }
    }
    tc_fence_before();
    cta_sync();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const long long tiles = (long long)(p.N / 128) * (kGrp ? blk_tab[p.E] : p.mblocks);
    const long long U = tiles * UT + (kLora ? (long long)(p.N / 128) * cum_tab[p.mblocks] : 0);
    // no more ranges than units (the dense launch's host saw to it): none of a tile's ranges is empty
    int P = kGrp && U < p.P ? (int)U : p.P;
    // How the units are cut (launches of tiles of one length; not the dense ones): ranges of whole tiles
    // (pieces = 1), each tile into `pieces` ranges of its own, or evenly (0).
    long long u0 = 0, u1 = 0;
    int pieces = 0;
    if constexpr (MODE != kTcDense) {
        const int len = kLora ? UT + cum_tab[p.mblocks] : UT;
        if (U > 0 && (kGrp || p.mblocks == 1)) {
            const long long each = (tiles + P - 1) / P;
            const long long least = (U + P - 1) / P;
            const int most = tiles < P ? min((int)(P / tiles), 255) : 1;
            const long long even = least + tc_cut_two(kShare) + most / 2;
            int cost = 0x7fffffff;   // in units; lane i: the best of i + 2, i + 34, .. pieces
            if (each * len > least + kTcCutOne + 1) {
                for (int n = lane + 2; n <= most && n <= len; n += 32)
                    cost = min(cost, ((len + n - 1) / n + kTcCutOne + n / 2) * 256 + n);
                cost = __reduce_min_sync(0xffffffffu, cost);
            }
            if (each * len <= min(even, (long long)(cost >> 8))) {
                pieces = 1;
                P = (int)((tiles + each - 1) / each);
                if (cta < P) {
                    u0 = tc_unit_begin(cta, tiles, P) * len;
                    u1 = tc_unit_begin(cta + 1, tiles, P) * len;
                }
            } else if (cost != 0x7fffffff && (cost >> 8) <= even) {
                pieces = cost & 255;
                P = (int)tiles * pieces;
                if (cta < P) {
                    const int tile = cta / pieces, q = cta - tile * pieces;
                    u0 = (long long)tile * len + q * len / pieces;
                    u1 = (long long)tile * len + (q + 1) * len / pieces;
                }
            }
        }
    }
    if (pieces == 0 && cta < P) {
        u0 = tc_unit_begin(cta, U, P);
        u1 = tc_unit_begin(cta + 1, U, P);
    }
    // the CTAs of a tile [t0u, t1u) that this one has units of
    auto first_of = [&](long long t0u) { return pieces ? cta - cta % pieces : tc_unit_owner(t0u, U, P); };
    auto last_of = [&](long long t1u) { return pieces ? cta - cta % pieces + pieces - 1 : tc_unit_owner(t1u - 1, U, P); };
    if constexpr (kShare || kLora)
        if (threadIdx.x == 0) {
            range[0] = u0;
            range[1] = u1;
            range[2] = U;
            range[3] = ((long long)pieces << 32) + P;
        }
    const uint32_t tmem_w = tmem + (uint32_t)(kBufs * kIss * kCols);   // the step ring's weight tiles

    if (warp == kTcWarpLoadW) {
        // ------------------------------------------------------------ weight records
        if (lane == 0) {
            int rs = 0, issued[kTcMaxRing];
            uint32_t rph = 0;
            for (int i = 0; i < nr; ++i) issued[i] = 0;
            // unit i = tile tau (channel tile nt, row block mb), step ku (kept by increments)
            const long long tau0 = u0 / UT;
            int ku = (int)(u0 - tau0 * UT), mb = kGrp ? 0 : (int)(tau0 % p.mblocks);
            long long nt = kGrp ? 0 : tau0 / p.mblocks;
            MoeWalk gw;
            TcLoraWalk lw;
            if constexpr (kGrp) gw.init(run_tab, blk_tab, p.E, p.N / 128, tau0);
            if constexpr (kLora) lw.init(cum_tab, UT, p.mblocks, u0);
            for (long long i = u0; i < u1;) {
                if constexpr (kLora) {
                    if (lw.low()) {   // the dequantizing warps read Lb themselves
                        const int skip = u1 - i < lw.len - lw.ku ? (int)(u1 - i) : lw.len - lw.ku;
                        lw.step(skip);
                        i += skip;
                        continue;
                    }
                    ku = lw.ku;
                }
                const int n = UT - ku < kUPL ? (u1 - i < UT - ku ? (int)(u1 - i) : UT - ku)
                                              : (u1 - i < kUPL ? (int)(u1 - i) : kUPL);
                if (!mbar_wait(&empty_r[rs], rph ^ 1u, abort_flag, p.dev_status, wait_ns)) break;
                const long long rec = (kGrp ? gw.rec0(UT) : (kLora ? (long long)lw.nt : nt) * UT) + ku;
                mbar_arrive_expect_tx(&full_r[rs], (uint32_t)n * R);
                bulk_g2s(ring_w + (size_t)rs * p.slot_w, p.tiled + (size_t)rec * R, (uint32_t)n * R, &full_r[rs]);
                ++issued[rs];
                i += n;
                if constexpr (kLora) {
                    lw.step(n);
                } else if ((ku += n) == UT) {
                    ku = 0;
                    if constexpr (kGrp) {
                        if (i < u1) gw.next();
                    } else if (++mb == p.mblocks) {
                        mb = 0;
                        ++nt;
                    }
                }
                if (++rs == nr) {
                    rs = 0;
                    rph ^= 1u;
                }
            }
            // every copy issued lands before the CTA may exit
            volatile int keep = 0;
            for (int s = 0; s < nr; ++s)
                if (issued[s] > 0) mbar_wait(&full_r[s], (uint32_t)(issued[s] - 1) & 1u, &keep, nullptr, kTcDrainNs);
        }
    } else if (warp == kTcWarpLoadA) {
        // ------------------------------------------------------------ activation tiles
        if (lane == 0) {
            prefetch_tensormap(&tmA);
            int issued[8];
            for (int i = 0; i < NS; ++i) issued[i] = 0;
            int s = 0;
            uint32_t ph = 0;
            // unit i = tile tau, step ku; row block mb = tau mod mblocks (kept by increments)
            long long tau0 = u0 / UT;
            int ku = (int)(u0 - tau0 * UT), mb = kGrp ? 0 : (int)(tau0 % p.mblocks);
            MoeWalk gw;
            TcLoraWalk lw;
            bool placed = false;
            if constexpr (kGrp) gw.init(run_tab, blk_tab, p.E, p.N / 128, tau0);
            if constexpr (kLora) lw.init(cum_tab, UT, p.mblocks, u0);
            for (long long i = u0; i < u1; ++i) {
                if constexpr (kLora) {
                    if (i > u0) lw.step(1);
                } else if (i > u0 && ++ku == UT) {
                    ku = 0;
                    if constexpr (kGrp) gw.next();
                    else if (++mb == p.mblocks) mb = 0;
                }
                // (a grouped tile may run into the next expert's rows: those columns are not stored)
                const int row = kGrp ? gw.row0(BN) : (kLora ? lw.mb : mb) * BN;
                const bool low = kLora && lw.low();
                if (low && !placed) {
                    pdl_wait();
                    placed = true;
                }
                const CUtensorMap* map = low ? &tmT : &tmA;
                const int kx = kLora ? (low ? lw.ku - UT : lw.ku) : ku;
                if (!mbar_wait(&free_s[s], ph ^ 1u, abort_flag, p.dev_status, wait_ns)) break;
                uint8_t* dst = ring_a + (size_t)s * kSlotA;
                if constexpr (kGrp) {
                    constexpr int kBox = tc_box_rows(BN);
                    const int left = gw.row_end() - row, boxes = left >= BN ? BN / kBox : (left + kBox - 1) / kBox;
                    mbar_arrive_expect_tx(&full_a[s], (uint32_t)(boxes * kBox) * 256u);
                    for (int b = 0; b < boxes; ++b) {
                        tma_2d_g2s(dst + b * kBox * 128, map, kx * 128, row + b * kBox, &full_a[s]);
                        tma_2d_g2s(dst + kSlotA / 2 + b * kBox * 128, map, kx * 128 + 64, row + b * kBox, &full_a[s]);
                    }
                } else {
                    mbar_arrive_expect_tx(&full_a[s], kSlotA);
                    tma_2d_g2s(dst, map, kx * 128, row, &full_a[s]);
                    tma_2d_g2s(dst + kSlotA / 2, map, kx * 128 + 64, row, &full_a[s]);
                }
                ++issued[s];
                if (++s == NS) {
                    s = 0;
                    ph ^= 1u;
                }
            }
            volatile int keep = 0;
            for (int q = 0; q < NS; ++q)
                if (issued[q] > 0) mbar_wait(&full_a[q], (uint32_t)(issued[q] - 1) & 1u, &keep, nullptr, kTcDrainNs);
            if (kLora) pdl_wait();   // this kernel does not complete before the one that it overtook
        }
    } else if (warp >= kTcWarpMma && warp < kTcWarpMma + kIss) {
        // ------------------------------------------------------------ MMA issuers
        // Issuer j (lane 0 of warp kTcWarpMma + j) takes the units j, j + kIss, .. of the range into
        // its own accumulator of the tile; the epilogue adds them. (One thread issuing all the
        // MMAs measured about 1.1k cycles per unit at N = 16, the tensor pipe mostly idle.)
        if (lane == 0) {
            const int j = warp - kTcWarpMma;
            constexpr uint32_t idesc = idesc_f16(BN, std::is_same<T, __nv_bfloat16>::value);
            constexpr uint32_t idesc_low = idesc_f16(BN, true);   // low-rank units: bf16 on both sides
            int s = 0, use[2] = {0, 0}, ab = 0;
            uint32_t ph = 0;
            bool ok = true;
            TcLoraWalk lw;
            if constexpr (kLora) lw.init(cum_tab, UT, p.mblocks, u0);
            MoeWalk gw;
            if constexpr (kGrp)
                if (u0 < u1) gw.init(run_tab, blk_tab, p.E, p.N / 128, u0 / UT);
            if constexpr (US) {
                // each own unit into accumulator ab * kIss + j (two per issuer, alternating)
                long long low_from = kLora ? u0 - lw.ku + UT : 0, tile_to = kLora ? u0 - lw.ku + lw.len : 0;
                for (long long i = u0; i < u1; ++i) {
                    if (kLora && i == tile_to) {
                        lw.step(lw.len - lw.ku);
                        low_from = i + UT;
                        tile_to = i + lw.len;
                    }
                    if (kIss == 1 || (int)((i - u0) & 1) == j) {
                        const int slot = ab * kIss + j;
                        if (!mbar_wait(&accempty[slot], ((uint32_t)use[ab] & 1u) ^ 1u, abort_flag, p.dev_status,
                                       wait_ns) ||
                            !mbar_wait(&full_d[s], ph, abort_flag, p.dev_status, wait_ns) ||
                            !mbar_wait(&full_a[s], ph, abort_flag, p.dev_status, wait_ns))
                            break;
                        tc_fence_after();
                        const uint32_t d_tmem = tmem + (uint32_t)(slot * kCols);
                        const uint32_t a_tm = tmem_w + (uint32_t)(s * kTcStepCols);
                        const uint32_t b_sm = smem_u32(ring_a + (size_t)s * kSlotA);
                        const uint32_t ids = kLora && i >= low_from ? idesc_low : idesc;
                        mma4_f16_ts(d_tmem, a_tm, smem_desc_sw128(b_sm), ids, 0u);
                        mma4_f16_ts(d_tmem, a_tm + 32u, smem_desc_sw128(b_sm + kSlotA / 2), ids, 1u);
                        mma_commit(&free_s[s]);
                        mma_commit(&accfull[slot]);
                        ++use[ab];
                        ab ^= 1;
                    }
                    if (++s == NS) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
                ok = false;   // (the tile loop below is not run)
            }
            for (long long i = u0; i < u1 && ok;) {
                const long long tau = kLora ? 0 : i / UT;
                const long long tile_end = kLora ? i + (lw.len - lw.ku) : (tau + 1) * UT;
                const long long seg_end = u1 < tile_end ? u1 : tile_end;
                const long long low_from = kLora ? i - lw.ku + UT : 0;
                if constexpr (kLora) lw.step((int)(seg_end - i));
                uint32_t idesc_t = idesc;
                if constexpr (kGrp && BN > 64) {   // as many columns as the tile has rows, in boxes
                    if (i > u0) gw.next();
                    constexpr int kBox = tc_box_rows(BN);
                    const int left = gw.row_end() - gw.row0(BN);
                    idesc_t = idesc_f16(left >= BN ? BN : (left + kBox - 1) / kBox * kBox, std::is_same<T, __nv_bfloat16>::value);
                }
                if (!mbar_wait(&accempty[ab], ((uint32_t)use[ab] & 1u) ^ 1u, abort_flag, p.dev_status, wait_ns)) break;
                tc_fence_after();
                const uint32_t d_tmem = tmem + (uint32_t)((ab * kIss + j) * kCols);
                bool first = true;
                for (; i < seg_end; ++i) {
                    if (kIss == 1 || (int)((i - u0) & 1) == j) {
                        if (!mbar_wait(&full_d[s], ph, abort_flag, p.dev_status, wait_ns) ||
                            !mbar_wait(&full_a[s], ph, abort_flag, p.dev_status, wait_ns)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        // the unit's eight K-steps of 16: weights from tensor memory, activations
                        // from the two 64-K boxes of the step's tile; one commit frees both tiles
                        const uint32_t a_tm = tmem_w + (uint32_t)(s * kTcStepCols);
                        const uint32_t b_sm = smem_u32(ring_a + (size_t)s * kSlotA);
                        const uint32_t ids = kLora && i >= low_from ? idesc_low : idesc_t;
                        mma4_f16_ts(d_tmem, a_tm, smem_desc_sw128(b_sm), ids, first ? 0u : 1u);
                        mma4_f16_ts(d_tmem, a_tm + 32u, smem_desc_sw128(b_sm + kSlotA / 2), ids, 1u);
                        mma_commit(&free_s[s]);
                        first = false;
                    }
                    if (++s == NS) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
                if (!ok) break;
                // (with no unit of this tile, the commit arrives at once)
                mma_commit(&accfull[ab]);
                ++use[ab];
                if (kBufs == 2) ab ^= 1;
            }
            // the CTA exits only after the last MMAs of every issuer completed
            mma_commit(lastmma);
            volatile int keep = 0;
            mbar_wait(lastmma, 0, &keep, nullptr, kTcDrainNs);
        }
    } else if (warp >= kTcWarpEpi && warp < kTcWarpEpi + 4) {
        // ------------------------------------------------------------ epilogue
        const int q = warp & 3;                   // tensor-memory lane quarter
        const int n = 32 * q + lane;              // channel within the tile
        const bool leader = warp == kTcWarpEpi && lane == 0;
        T* C = static_cast<T*>(p.C);
        int use[2] = {0, 0}, ab = 0;
        bool ok = true;
        MoeWalk gw;
        if constexpr (kGrp)
            if (u0 < u1) gw.init(run_tab, blk_tab, p.E, p.N / 128, u0 / UT);
        TcLoraWalk lw;
        if constexpr (kLora) lw.init(cum_tab, UT, p.mblocks, u0);
        // the counter of a cut tile: one per tile (dense), or one per CTA, of the one cut tile that
        // opens in the CTA's range
        auto counter = [&](long long tau, int cf) { return p.counters + (MODE == kTcDense ? tau : (long long)cf); };
        // where this CTA publishes its sums of a cut tile that CTA cf opened
        auto own_slot = [&](int cf) { return kShare ? 2 * cta + (cta == cf ? 1 : 0) : cta; };
        // 16 rows from m of the warp's 32 channels, rounded. A lane holds one channel of every row; two
        // exchanges (with lanes 1 and 2 away) give it four channels of every fourth row, so the rows go
        // out in 8-byte stores of 64 bytes per row: a store of 2 bytes per lane and row kept the
        // single accumulator of a 256-row tile for 5k cycles, a fifth of the tile.
        auto put16 = [&](int m, int mend, size_t n0, const float (&y)[16]) {
            uint32_t v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {   // rows 2 j, 2 j + 1
                const uint32_t u = tc_pack2<T>(y[2 * j], y[2 * j + 1]);
                const uint32_t o = __shfl_xor_sync(0xffffffffu, u, 1);
                v[j] = lane & 1 ? __byte_perm(o, u, 0x7632) : __byte_perm(u, o, 0x5410);   // row 2 j + (lane & 1)
            }
            T* c = C + (size_t)(m + (lane & 3)) * p.N + n0 + 32 * q + 4 * (lane >> 2);
#pragma unroll
            for (int i = 0; i < 4; ++i) {   // row 4 i + (lane & 3)
                const uint32_t o = __shfl_xor_sync(0xffffffffu, lane & 2 ? v[2 * i] : v[2 * i + 1], 2);
                const uint2 w = lane & 2 ? make_uint2(o, v[2 * i + 1]) : make_uint2(v[2 * i], o);
                if (m + 4 * i + (lane & 3) < mend) *reinterpret_cast<uint2*>(c + (size_t)(4 * i) * p.N) = w;
            }
        };
        // kTcLora: the tile's rows of every Lb it takes, on their way to L2 while the weight units run (a
        // fetch by the dequantizing warps that finds them in HBM waits behind the weight stream: 3.6 us
        // per low-rank unit at 16 rows of 14 adapters)
        auto ahead = [&](int tile_nt, int mb, int low_units) {
            if constexpr (kLora) {
                constexpr int kPer = std::is_same<T, __nv_bfloat16>::value ? 4 : 2;
                const int pr = (p.rank + 15) / 16;
                for (int j = n; j * pr < low_units * kPer; j += 128) {
                    const int piece = __ldg(p.lora_pieces + (size_t)mb * p.max_pieces + j * pr);
                    if (piece >= 0)
                        bulk_prefetch_l2(static_cast<const T*>(p.lora_b) +
                                             ((size_t)(piece >> 8) * p.N + (size_t)tile_nt * 128) * p.rank,
                                         256u * (uint32_t)p.rank);
                }
            }
        };
        if constexpr (US) {
            // per unit: s times the unit's sums into run[] (row m0 + r of channel n); per tile
            // segment: run[] to C, or to the published sums of a cut tile
            float run[BN];
#pragma unroll
            for (int r = 0; r < BN; ++r) run[r] = 0.0f;
            int abj[2] = {0, 0}, uses[2 * kIss];
#pragma unroll
            for (int k = 0; k < 2 * kIss; ++k) uses[k] = 0;
            const uint16_t* scl = reinterpret_cast<const uint16_t*>(p.tiled + p.scales_off) + n;
            for (long long i = u0; i < u1;) {
                const long long tau = kLora ? 0 : i / UT;
                const long long t0u = kLora ? i - lw.ku : tau * UT, t1u = t0u + (kLora ? lw.len : UT);   // the tile's units
                const long long seg_end = u1 < t1u ? u1 : t1u;
                if constexpr (kGrp)
                    if (i > u0) gw.next();
                const int nt = kGrp ? gw.nt : kLora ? lw.nt : (int)(tau / p.mblocks);
                const int mb = kGrp ? 0 : kLora ? lw.mb : (int)(tau % p.mblocks);
                const size_t n0 = (size_t)nt * 128;
                const int m0 = kGrp ? gw.row0(BN) : mb * BN, mend = kGrp ? gw.row_end() : p.M;
                const int cf = first_of(t0u), cl = last_of(t1u);
                if (kLora && seg_end > t0u + UT) ahead(nt, mb, lw.len - UT);
                for (; i < seg_end; ++i) {
                    const int j = kIss == 1 ? 0 : (int)((i - u0) & 1);
                    const int slot = abj[j] * kIss + j;
                    // the unit's record is nt K/128 + its K-step; its scale of channel n (group 128)
                    const long long rec = (kGrp ? gw.rec0(UT) : (long long)nt * UT) + (i - t0u);
                    // (a low-rank unit's sums count as they are: 1 in fp16)
                    const uint16_t sb = kLora && lw.low() ? (uint16_t)0x3C00u : __ldg(scl + (size_t)rec * (R / 2));
                    ok = ok && tc_wait(&accfull[slot], (uint32_t)uses[slot] & 1u, abort_flag, p.dev_status, wait_ns);
                    tc_fence_after();
                    if (ok) {
                        const float sf = __half2float(__ushort_as_half(sb));
                        const uint32_t lb = tmem + (uint32_t)(slot * kCols) + ((uint32_t)(32 * q) << 16);
#pragma unroll
                        for (int c = 0; c < BN / 16; ++c) {
                            uint32_t v[16];
                            tmem_ld16(lb + (uint32_t)(c * 16), v);
                            tmem_ld_wait();
#pragma unroll
                            for (int jj = 0; jj < 16; ++jj) run[c * 16 + jj] = fmaf(sf, __uint_as_float(v[jj]), run[c * 16 + jj]);
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&accempty[slot]);
                    ++uses[slot];
                    abj[j] ^= 1;
                    if constexpr (kLora) lw.step(1);
                }
                if (cf == cl || (!kShare && cta == cf)) {
                    if (cf != cl) {
                        if (leader) {
                            const uint64_t t0 = globaltimer_ns();
                            for (;;) {
                                int c;
                                asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(c) : "l"(counter(tau, cf))
                                             : "memory");
                                if (c >= cl - cf) break;
                                if (*abort_flag || globaltimer_ns() - t0 > wait_ns) {
                                    *abort_flag = 1;
                                    report_status(p.dev_status, W4A16_ETIMEOUT);
                                    break;
                                }
                            }
                            *counter(tau, cf) = 0;
                        }
                        tc_named_bar(1, 128);
                    }
                    if (__all_sync(0xffffffffu, ok && !*abort_flag)) {
#pragma unroll
                        for (int c = 0; c < BN / 16; ++c) {
                            float y[16];
#pragma unroll
                            for (int jj = 0; jj < 16; ++jj) y[jj] = run[c * 16 + jj];
#pragma unroll 1
                            for (int cc = cf + 1; cc <= cl; ++cc) {   // (!kShare)
                                const float* part = p.partials + ((size_t)cc * BN + c * 16) * 128 + n;
                                float pv[16];
#pragma unroll
                                for (int jj = 0; jj < 16; ++jj)
                                    pv[jj] = m0 + c * 16 + jj < mend ? __ldcg(part + jj * 128) : 0.0f;
#pragma unroll
                                for (int jj = 0; jj < 16; ++jj) y[jj] += pv[jj];
                            }
                            put16(m0 + c * 16, mend, n0, y);
                        }
                    }
                } else {
                    if (__all_sync(0xffffffffu, ok && !*abort_flag)) {
                        float* part = p.partials + (size_t)own_slot(cf) * BN * 128;
#pragma unroll
                        for (int r = 0; r < BN; ++r)
                            if (m0 + r < mend) __stcg(part + (size_t)r * 128 + n, run[r]);
                    }
                    __threadfence();
                    tc_named_bar(1, 128);
                    if (leader) asm volatile("red.release.gpu.global.add.s32 [%0], 1;" ::"l"(counter(tau, cf)) : "memory");
                }
#pragma unroll
                for (int r = 0; r < BN; ++r) run[r] = 0.0f;
            }
            ok = false;   // (the tile loop below is not run)
        }
        for (long long i = u0; i < u1 && (!US || ok);) {
            const long long tau = kLora ? 0 : i / UT;
            const long long t0u = kLora ? i - lw.ku : tau * UT, t1u = t0u + (kLora ? lw.len : UT);   // the tile's units
            const long long seg_end = u1 < t1u ? u1 : t1u;
            if (kLora && seg_end > t0u + UT) ahead(lw.nt, lw.mb, lw.len - UT);
            // the issuers that hold units of this tile segment (issuer j: units j, j + 2, ..)
            const long long seg_lo = i;
            const bool has0 = kIss == 1 || seg_end - seg_lo >= 2 || ((seg_lo - u0) & 1) == 0;
            const bool has1 = kIss == 2 && (seg_end - seg_lo >= 2 || ((seg_lo - u0) & 1) == 1);
            ok = ok && tc_wait(&accfull[ab], (uint32_t)use[ab] & 1u, abort_flag, p.dev_status, wait_ns);
            tc_fence_after();
            if constexpr (kGrp)
                if (i > u0) gw.next();
            const int nt = kGrp ? gw.nt : kLora ? lw.nt : (int)(tau / p.mblocks);
            const int mb = kGrp ? 0 : kLora ? lw.mb : (int)(tau % p.mblocks);
            const size_t n0 = (size_t)nt * 128;
            const int m0 = kGrp ? gw.row0(BN) : mb * BN, mend = kGrp ? gw.row_end() : p.M;
            const int cf = first_of(t0u), cl = last_of(t1u);
            if constexpr (kLora) lw.step((int)(seg_end - i));
            i = seg_end;
            const uint32_t lane_base = tmem + (uint32_t)(ab * kIss * kCols) + ((uint32_t)(32 * q) << 16);
            // the accumulator is free for the next tile's MMAs
            auto release = [&]() {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&accempty[ab]);
            };
            // the tile's FP32 sums, 16 columns at a time, to f(c, y): the issuers' accumulators added. The
            // accumulator is released with the last ones read. (Loading the next 16 columns ahead, and
            // releasing a 256-row tile's accumulator in halves, measured 5% slower and the same.)
            auto sums = [&](auto f) {
                const int nc = kGrp && mend - m0 < BN ? (mend - m0 + 15) / 16 : BN / 16;
                uint32_t v[16];
#pragma unroll 1
                for (int c = 0; c < nc; ++c) {
                    float y[16];
#pragma unroll
                    for (int jj = 0; jj < 16; ++jj) y[jj] = 0.0f;
                    if (has0) {
                        tmem_ld16(lane_base + (uint32_t)(c * 16), v);
                        tc_ld_wait16(v);
#pragma unroll
                        for (int jj = 0; jj < 16; ++jj) y[jj] = __uint_as_float(v[jj]);
                    }
                    if (has1) {
                        tmem_ld16(lane_base + (uint32_t)(kCols + c * 16), v);
                        tc_ld_wait16(v);
#pragma unroll
                        for (int jj = 0; jj < 16; ++jj) y[jj] += __uint_as_float(v[jj]);
                    }
                    if (c + 1 == nc) release();
                    f(c, y);
                }
            };
            if (cf == cl || (!kShare && cta == cf)) {
                if (cf != cl) {
                    // the tile is cut between CTAs cf .. cl and this is cf: wait until every later
                    // CTA of the tile has published its sums (the tile opens their ranges)
                    if (leader) {
                        const uint64_t t0 = globaltimer_ns();
                        for (;;) {
                            int c;
                            asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(c) : "l"(counter(tau, cf))
                                         : "memory");
                            if (c >= cl - cf) break;
                            if (*abort_flag || globaltimer_ns() - t0 > wait_ns) {
                                *abort_flag = 1;
                                report_status(p.dev_status, W4A16_ETIMEOUT);
                                break;
                            }
                        }
                        *counter(tau, cf) = 0;
                    }
                    tc_named_bar(1, 128);
                }
                if (__all_sync(0xffffffffu, ok && !*abort_flag)) {
                    sums([&](int c, float (&y)[16]) {
                        // the other CTAs' sums, in CTA order; the 16 loads of one CTA in flight together
#pragma unroll 1
                        for (int cc = cf + 1; cc <= cl; ++cc) {
                            const float* part = p.partials + ((size_t)cc * BN + c * 16) * 128 + n;
                            float pv[16];
#pragma unroll
                            for (int j = 0; j < 16; ++j) pv[j] = m0 + c * 16 + j < mend ? __ldcg(part + j * 128) : 0.0f;
#pragma unroll
                            for (int j = 0; j < 16; ++j) y[j] += pv[j];
                        }
                        put16(m0 + c * 16, mend, n0, y);
                    });
                } else {
                    release();
                }
            } else {
                // a later CTA of a cut tile (the tile opens its range), or (kShare) any CTA of it: publish the
                // sums and count them, without waiting
                if (__all_sync(0xffffffffu, ok && !*abort_flag)) {
                    float* part = p.partials + (size_t)own_slot(cf) * BN * 128;
                    sums([&](int c, float (&y)[16]) {
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const int mr = c * 16 + j;
                            if (m0 + mr < mend) __stcg(part + (size_t)mr * 128 + n, y[j]);
                        }
                    });
                } else {
                    release();
                }
                __threadfence();
                tc_named_bar(1, 128);
                if (leader) asm volatile("red.release.gpu.global.add.s32 [%0], 1;" ::"l"(counter(tau, cf)) : "memory");
            }
            ++use[ab];
            if (kBufs == 2) ab ^= 1;
        }
    } else if (warp >= kTcWarpDeq) {
        // ------------------------------------------------------------ dequantize
        const int dt = threadIdx.x - 32 * kTcWarpDeq;
        const int n = dt & 127, blk = dt >> 7;   // channel, and the unit's 32-K block (0..3)
        const int sym = p.sym;
        const GsMasks km = p.km;
        const int lg = (32 * blk) / p.group;     // the block's group within the unit
        const uint32_t coff = 2048u * (uint32_t)blk + 16u * (uint32_t)(n ^ (2 * blk));
        const uint32_t soff = p.scales_off + 256u * (uint32_t)lg + 2u * (uint32_t)n;
        const uint32_t zoff = p.zeros_off + 64u * (uint32_t)lg + 4u * (uint32_t)(n >> 3);
        const int zsh = 4 * (n & 7);
        // this warp's lanes of tensor memory (its 32 channels), columns [16 blk, 16 blk + 16) of the
        // step's tile
        const uint32_t d_lane = tmem_w + ((uint32_t)(32 * (warp & 3)) << 16) + (uint32_t)(16 * blk);
        int rs = 0, s = 0;
        uint32_t rph = 0, ph = 0;
        bool ok = true;
        long long tend = (u0 / UT + 1) * UT;   // end of the current tile's units
        // kTcLora: block blk's 16 ranks of Lb, fetched a unit ahead, and the piece after them
        [[maybe_unused]] TcLoraWalk lw;
        [[maybe_unused]] uint4 b0 = make_uint4(0, 0, 0, 0), b1 = b0;
        [[maybe_unused]] int piece = -1;
        auto piece_of = [&](int unit) {   // low-rank unit of the walk's row block
            constexpr int kPer = std::is_same<T, __nv_bfloat16>::value ? 4 : 2;   // pieces per unit
            return __ldg(p.lora_pieces + (size_t)lw.mb * p.max_pieces + unit * kPer + (kPer == 4 ? blk : blk >> 1));
        };
        auto fetch = [&]() {
            b0 = b1 = make_uint4(0, 0, 0, 0);
            if (piece < 0) return;
            const int j = 16 * (piece & 255);
            const uint4* src = reinterpret_cast<const uint4*>(
                static_cast<const T*>(p.lora_b) + ((size_t)(piece >> 8) * p.N + (size_t)lw.nt * 128 + n) * p.rank + j);
            b0 = __ldg(src);
            if (j + 8 < p.rank) b1 = __ldg(src + 1);
        };
        // (a tile's weight units run to `tend` by the dense loop; the walk moves per tile and low-rank unit)
        if constexpr (kLora) {
            lw.init(cum_tab, UT, p.mblocks, u0);
            tend = lw.low() ? u0 : u0 + (UT - lw.ku);
            if (u0 < u1 && lw.len > UT) {
                piece = piece_of(lw.low() ? lw.ku - UT : 0);
                if (lw.low()) {
                    fetch();
                    if (lw.ku + 1 < lw.len) piece = piece_of(lw.ku + 1 - UT);
                } else {
                    lw.ku = UT;
                }
            } else {
                lw.ku = UT;
            }
        }
        for (long long i = u0; i < u1 && ok;) {
            if constexpr (kLora) {
                if (i == tend) {
                    if (lw.ku == lw.len) {   // the next tile's weight units
                        lw.step(0);
                        lw.ku = UT;
                        tend = i + UT;
                        if (lw.len > UT) piece = piece_of(0);
                        continue;
                    }
                    // bf16 layer: [Lb | Lb] beside T's [hi | lo]; fp16 layer: Lb = hi + lo exactly (8 + 3
                    // bits), blocks [hi | hi], [lo | 0] beside T's [hi | lo], [hi | 0]
                    if (!tc_wait(&free_s[s], ph ^ 1u, abort_flag, p.dev_status, wait_ns)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    uint32_t w8[8] = {b0.x, b0.y, b0.z, b0.w, b1.x, b1.y, b1.z, b1.w};
                    uint32_t out[16];
                    {
                        constexpr uint32_t kExp = std::is_same<T, __nv_bfloat16>::value ? 0x7F80u : 0x7C00u;
                        bool bad = false;
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            const bool bl = (w8[c] & kExp) == kExp, bh = (w8[c] & (kExp << 16)) == (kExp << 16);
                            w8[c] &= (bl ? 0u : 0xFFFFu) | (bh ? 0u : 0xFFFF0000u);
                            bad = bad || bl || bh;
                        }
                        if (bad) {
                            *static_cast<volatile int*>(p.lora_bad) = 1;
                            __threadfence();
                        }
                    }
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        if constexpr (std::is_same<T, __nv_bfloat16>::value) {
                            out[c] = out[8 + c] = w8[c];
                        } else {
                            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w8[c]));
                            const uint32_t hx = __float_as_uint(f.x) & 0xFFFF0000u, hy = __float_as_uint(f.y) & 0xFFFF0000u;
                            const uint32_t lx = __float_as_uint(f.x - __uint_as_float(hx));
                            const uint32_t ly = __float_as_uint(f.y - __uint_as_float(hy));
                            const uint32_t hi = (hx >> 16) | hy, lo = (lx >> 16) | (ly & 0xFFFF0000u);
                            out[c] = blk & 1 ? lo : hi;
                            out[8 + c] = blk & 1 ? 0u : hi;
                        }
                    }
                    tend = ++i;
                    if (++lw.ku < lw.len) {
                        fetch();
                        if (lw.ku + 1 < lw.len) piece = piece_of(lw.ku + 1 - UT);
                    }
                    tmem_st16(d_lane + (uint32_t)(s * kTcStepCols), out);
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&full_d[s]);
                    if (++s == NS) {
                        s = 0;
                        ph ^= 1u;
                    }
                    continue;
                }
            }
            const long long seg_end = u1 < tend ? u1 : tend;
            const int nu = (int)(seg_end - i < kUPL ? seg_end - i : kUPL);
            i += nu;
            if constexpr (kLora) {
                if (i == tend && lw.len > UT) {   // the tile's low-rank units come next
                    fetch();
                    if (lw.len > UT + 1) piece = piece_of(1);
                }
            } else if (i == tend) {
                tend += UT;
            }
            if (!tc_wait(&full_r[rs], rph, abort_flag, p.dev_status, wait_ns)) {
                ok = false;
                break;
            }
            for (int uu = 0; uu < nu; ++uu) {
                const uint8_t* rec = ring_w + (size_t)rs * p.slot_w + (size_t)uu * R;
                const uint4 cw = *reinterpret_cast<const uint4*>(rec + coff);
                const uint16_t sb = US ? (uint16_t)0 : *reinterpret_cast<const uint16_t*>(rec + soff);
                const uint32_t zv = sym ? 8u : (*reinterpret_cast<const uint32_t*>(rec + zoff) >> zsh) & 0xFu;
                if (!tc_wait(&free_s[s], ph ^ 1u, abort_flag, p.dev_status, wait_ns)) {
                    ok = false;
                    break;
                }
                tc_fence_after();   // the MMAs that read this tile completed before the stores
                const uint32_t za = Ops::zz_a(zv), zb = Ops::zz_b(zv);
                typename Ops::Scale sc;
                if constexpr (!US) sc.set(sb);
                const uint32_t words[4] = {cw.x, cw.y, cw.z, cw.w};
                uint32_t out[16];   // column c: K pair (2 c, 2 c + 1) of the block
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    uint32_t r[4];
                    Ops::unpack(words[w], km, r);
                    if constexpr (US) {   // u - z, exact; the scale multiplies the unit's sums
                        out[4 * w + 0] = Ops::sub_a(r[0], za);
                        out[4 * w + 1] = Ops::sub_b(r[1], zb);
                        out[4 * w + 2] = Ops::sub_a(r[2], za);
                        out[4 * w + 3] = Ops::sub_b(r[3], zb);
                    } else {
                        out[4 * w + 0] = sc.apply(Ops::sub_a(r[0], za));
                        out[4 * w + 1] = sc.apply(Ops::sub_b(r[1], zb));
                        out[4 * w + 2] = sc.apply(Ops::sub_a(r[2], za));
                        out[4 * w + 3] = sc.apply(Ops::sub_b(r[3], zb));
                    }
                }
                tmem_st16(d_lane + (uint32_t)(s * kTcStepCols), out);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&full_d[s]);
                if (++s == NS) {
                    s = 0;
                    ph ^= 1u;
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty_r[rs]);
            if (++rs == nr) {
                rs = 0;
                rph ^= 1u;
            }
        }
    }

    tc_fence_before();
    cta_sync();
    if constexpr (kShare || kLora) {
        // The cut tiles (kShare). All CTAs cf .. cl of a tile have published their sums (or do so soon: none waits
        // before it has); each adds up, in CTA order, every (cl - cf + 1)-th row of it with all its threads
        // and writes those rows of C. The counter counts the publishing CTAs, then the finished ones; the
        // last resets it. (With one CTA's four epilogue warps adding the others' sums, a 256-row tile cut
        // between six CTAs took 32 us: one L2 round trip per 16 rows and CTA.)
        // kTcLora: values of Lb that are not finite entered the products as 0, or they would have reached
        // the other rows of the block (0 times them); the rows of their adapter get NaN here. Kept out of the
        // epilogue's loop, where its mere presence cost 5 us per tile. (The flag is seen: it was set before
        // the unit's weights were handed over, here or by the CTAs of a cut tile.)
        // (The range comes from shared memory: kept in registers since the start it spilled the roles.)
        const volatile long long* rg = range;
        const long long b0 = rg[0], b1 = rg[1], U_ = rg[2];
        const int P_ = (int)rg[3], pieces_ = (int)(rg[3] >> 32), me = blockIdx.x, UT_ = p.K / 128;
        auto not_finite = [&](int m, size_t ch) {   // some value of Lb[row m's adapter][ch]
            const int a = p.row_adapter[m];
            if ((unsigned)a >= (unsigned)p.adapters) return false;
            const T* b = static_cast<const T*>(p.lora_b) + ((size_t)a * p.N + ch) * p.rank;
            bool bad = false;
            for (int j = 0; j < p.rank; ++j) bad = bad || !isfinite(Act<T>::to_f32(b[j]));
            return bad;
        };
        for (int which = 0; kShare && which < 2 && b0 < b1 && pieces_ != 1; ++which) {   // the range's first tile, its last
            const long long u = which == 0 ? b0 : b1 - 1;
            long long t0u, t1u;
            int nt, m0, mend;
            if constexpr (kLora) {
                TcLoraWalk w;
                w.init(cum_tab, UT_, p.mblocks, u);
                t0u = u - w.ku;
                t1u = t0u + w.len;
                nt = w.nt;
                m0 = w.mb * BN;
                mend = p.M;
            } else {
                MoeWalk w;
                w.init(run_tab, blk_tab, p.E, p.N / 128, u / UT_);
                t0u = u / UT_ * UT_;
                t1u = t0u + UT_;
                nt = w.nt;
                m0 = w.row0(BN);
                mend = w.row_end();
            }
            const int cf = pieces_ ? me - me % pieces_ : tc_unit_owner(t0u, U_, P_);
            const int cl = pieces_ ? cf + pieces_ - 1 : tc_unit_owner(t1u - 1, U_, P_), n = cl - cf + 1;
            if (n == 1 || (which == 0) == (cf == me)) continue;
            if (threadIdx.x == 0) {
                const uint64_t t0 = globaltimer_ns();
                for (;;) {
                    int c;
                    asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(c) : "l"(p.counters + cf) : "memory");
                    if (c >= n) break;
                    if (*abort_flag || globaltimer_ns() - t0 > wait_ns) {
                        *abort_flag = 1;
                        report_status(p.dev_status, W4A16_ETIMEOUT);
                        break;
                    }
                }
            }
            cta_sync();
            if (!*abort_flag) {
                const int rows = mend - m0 < BN ? mend - m0 : BN, mine = (rows - (me - cf) + n - 1) / n;
                const bool bad = kLora && *static_cast<volatile int*>(p.lora_bad) != 0;
                for (int o = threadIdx.x; o < mine * 32; o += kTcThreads) {
                    const int r = (me - cf) + (o >> 5) * n, c4 = 4 * (o & 31);
                    const float* part = p.partials + (size_t)r * 128 + c4;
                    float4 y = __ldcg(reinterpret_cast<const float4*>(part + (size_t)(2 * cf + 1) * BN * 128));
#pragma unroll 4
                    for (int cc = cf + 1; cc <= cl; ++cc) {
                        const float4 v = __ldcg(reinterpret_cast<const float4*>(part + (size_t)(2 * cc) * BN * 128));
                        y.x += v.x;
                        y.y += v.y;
                        y.z += v.z;
                        y.w += v.w;
                    }
                    const size_t ch = (size_t)nt * 128 + c4;
                    if (bad) {
                        float* f = &y.x;
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (not_finite(m0 + r, ch + e)) f[e] = __int_as_float(0x7FC00000);
                    }
                    *reinterpret_cast<uint2*>(static_cast<T*>(p.C) + (size_t)(m0 + r) * p.N + ch) =
                        make_uint2(tc_pack2<T>(y.x, y.y), tc_pack2<T>(y.z, y.w));
                }
            }
            if (threadIdx.x == 0 && atomicAdd(p.counters + cf, 1) == 2 * n - 1) p.counters[cf] = 0;
        }
        if constexpr (kLora)
            if (*static_cast<volatile int*>(p.lora_bad) != 0) {   // the other tiles that this CTA has written
                TcLoraWalk w;
                w.init(cum_tab, UT_, p.mblocks, b0);
                for (long long i = b0; i < b1;) {
                    const long long t1u = i - w.ku + w.len, to = b1 < t1u ? b1 : t1u;
                    const int m0 = w.mb * BN, rows = p.M - m0 < BN ? p.M - m0 : BN;
                    if (w.ku == 0 && (!kShare || to == t1u))
                        for (int o = threadIdx.x; o < rows * 128; o += kTcThreads) {
                            const int m = m0 + (o >> 7);
                            const size_t ch = (size_t)w.nt * 128 + (o & 127);
                            if (not_finite(m, ch))
                                static_cast<T*>(p.C)[(size_t)m * p.N + ch] = Act<T>::from_f32(__int_as_float(0x7FC00000));
                        }
                    w.step((int)(to - i));
                    i = to;
                }
            }
    }
    if (warp == kTcWarpLoadA) {
        tc_fence_after();
        tmem_dealloc(tmem, kTcTmemCols);
    }
}

}  // namespace

namespace {

// The parameters that every mode shares.
inline TcParams tc_params(const TcPlan& pl, const void* tiled, int M, int N, int K, int group, int sym, bool bf16,
                          void* workspace, int* dev_status) {
    const TiledLayout L = tiled_layout(K, N, group, sym);
    TcParams prm = {};
    prm.tiled = static_cast<const uint8_t*>(tiled);
    prm.counters = static_cast<int*>(workspace);
    prm.partials = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kGemvStreamCounterBytes);
    prm.dev_status = dev_status;
    prm.M = M;
    prm.K = K;
    prm.N = N;
    prm.sym = sym;
    prm.group = group;
    prm.record = L.record;
    prm.scales_off = L.scales;
    prm.zeros_off = L.zeros;
    prm.slot_w = pl.slot_w;
    prm.P = pl.ctas;
    prm.mblocks = pl.mblocks;
    prm.nr = pl.nr;
    prm.off_w = pl.off_w;
    prm.off_bar = pl.off_bar;
    prm.wait_ns = wait_limit_ns();
    prm.km.lo = 0x000F000Fu;
    prm.km.hi = bf16 ? 0x000F000Fu : 0x00F000F0u;
    prm.km.magic = bf16 ? 0x43004300u : 0x64006400u;
    prm.km.m4 = 1u << 28;
    prm.km.m8 = 1u << 24;
    prm.km.m12 = 1u << 20;
    return prm;
}

template <int BN, typename T, bool US, int MODE>
int launch_tc_typed(const CUtensorMap& map, const CUtensorMap& map_t, const TcParams& prm, size_t smem, cudaStream_t stream) {
    static std::atomic<uint64_t> done{0};
    if (!allow_smem(tc_gemm_kernel<BN, T, US, MODE>, kTcSmemMax, done)) return W4A16_ECUDA;
    if constexpr (MODE != kTcDense)
        return launch_pdl(tc_gemm_kernel<BN, T, US, MODE>, dim3(prm.P), dim3(kTcThreads), smem, stream, map, map_t, prm) ==
                       cudaSuccess
                   ? W4A16_OK
                   : W4A16_ECUDA;
    tc_gemm_kernel<BN, T, US, MODE><<<prm.P, kTcThreads, smem, stream>>>(map, map_t, prm);
    return launch_status();
}

template <typename T, int MODE>
int launch_tc_bn(int bn, const CUtensorMap& map, const CUtensorMap& map_t, const TcParams& prm, size_t smem, cudaStream_t stream) {
    switch (bn) {
        // unit-scaled accumulation where one group spans a unit, at BN = 16 (measured on the
        // (8192, 28672) layer: 71.2 -> 67.8 us at M = 16; at BN = 32 it was slower, 74.4 -> 76.6)
        case 16: return prm.group == 128 ? launch_tc_typed<16, T, true, MODE>(map, map_t, prm, smem, stream)
                                         : launch_tc_typed<16, T, false, MODE>(map, map_t, prm, smem, stream);
        case 32: return launch_tc_typed<32, T, false, MODE>(map, map_t, prm, smem, stream);
        case 64: return launch_tc_typed<64, T, false, MODE>(map, map_t, prm, smem, stream);
        case 128: return launch_tc_typed<128, T, false, MODE>(map, map_t, prm, smem, stream);
        case 256: return launch_tc_typed<256, T, false, MODE>(map, map_t, prm, smem, stream);
        default: return W4A16_EUNSUPPORTED;
    }
}

}  // namespace

}  // namespace w4a16
