// moe_gemv.cu -- the experts' INT4 products on sorted rows when experts have few rows (decode).
//
// C[i, n] = sum_k A[i, k] (u[k, n] - z[g, n]) s[g, n] with the weight of row i's expert, FP32 sums. Bound
// by the weight stream of the experts that have rows. One CTA per SM; the tiles (128 channels x up
// to `rows` rows of one expert, moe_walk.cuh) times K / 128 unit records are cut into one contiguous
// range per CTA, as in the dense decode kernel (gemv_stream.cu), with its stages of four records, its
// compute warps' roles, MMA forms and cut-tile sums. What differs: a range may pass from expert to
// expert, so the activations are not staged per CTA but travel with the weights, per unit. A first
// kernel (moe_acts_kernel) lays them out once, [K / 128][R] records of 320 bytes: the 128 values of one
// row as the MMAs take them and, in the padding that keeps their reads free of bank conflicts, the
// record's sum (group 128 takes the zero point off the FP32 sums) and, for bf16 rows at group 128, the
// power of two under which they were converted to fp16 exactly (a record whose values span more than
// 31 binades stays bf16). Then per stage
//   producer warp    : the four units' weight records (one bulk copy per run of consecutive ones) and
//                      activation records (one copy per unit: the tile's rows are neighbours);
//   16 compute warps : group q takes unit q of every stage, warp w of it channels 32 w ..;
//   epilogue warp    : the four groups' sums, then C or the cut-tile protocol (one counter per CTA, of
//                      the one cut tile that opens in its range).
// The second kernel reads the offsets and streams weights while the first still runs: that one lets
// it start only after everything before it has completed.
// Converting inside the second kernel, by two warps per CTA, held it to 1.4 TB/s on the 4096 x 14336
// experts at one token: every channel tile converted its expert's rows again.
// Columns of an MMA past the tile's rows hold whatever the shared memory held; columns are
// independent and those are not stored.
// Every wait is bounded as in gemv_stream.cu.
#include <type_traits>

#include "dequant.cuh"
#include "moe_walk.cuh"
#include "pdl.cuh"
#include "routed.cuh"
#include "sm100_ptx.cuh"
#include "tiled_layout.cuh"

namespace w4a16 {
namespace {

using namespace sm100;

constexpr int kMgGroups = 4, kMgWarps = 16;   // compute warps, four to a group
constexpr int kMgWarpProducer = 16, kMgWarpEpilogue = 17;
constexpr int kMgThreads = 32 * 18;
constexpr int kMgMaxRows = 8, kMgMaxStages = 12, kMgMinStages = 3;
constexpr int kMgSmemMax = 227 * 1024;
constexpr int kMgRowBytes = 320;              // 128 K of one row: four 32-K blocks of 64 + 16 bytes
constexpr uint64_t kMgDrainNs = 2000000000ull;

// In the padding of an activation record's first 32-K block.
struct __align__(16) MgNote {
    float sum;   // 2^-24 sum_k of the (converted) values
    float up;    // the power of two that takes the products back
    int wide;    // kept in bf16
    int pad;
};

struct MgParams {
    const uint8_t* acts;   // [K / 128][R] records
    const uint8_t* tiled;
    void* C;
    int* counters;
    float* partials;    // [P][rows][128]
    int* dev_status;
    const int32_t* offsets;
    int E, R, K, N, sym, ns, P, rows;
    uint32_t record, scales_off, zeros_off, stage_bytes;
    uint32_t off_acts, off_red, off_bar, off_grp;
    GsMasks km, km_native;
    uint64_t wait_ns;
};

__device__ __forceinline__ long long mg_begin(int c, long long U, int P) { return ((long long)c * U) / P; }
__device__ __forceinline__ int mg_owner(long long u, long long U, int P) { return (int)(((u + 1) * P - 1) / U); }

__device__ __forceinline__ bool mg_wait(uint64_t* bar, uint32_t parity, volatile int* abort, int* dev_status,
                                        uint64_t ns) {
    if (__all_sync(0xffffffffu, mbar_test_wait(bar, parity))) return true;
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, dev_status, ns));
}

// The MMAs of one unit for a warp's 32 channels (two 16-row tiles) and 8 rows: operands (u - z) or
// (u - z) s in 16 bits, as O forms them; kPost scales the unit's FP32 sums.
template <typename O, bool kPost>
__device__ __forceinline__ void mg_unit(const GsMasks& km, const uint4 (&cw)[4], const uint16_t (&sb)[4], const uint4& zw,
                                        const uint4 (&v)[4], int zsh, float (&tot)[2][4]) {
    const uint32_t zws[4] = {zw.x, zw.y, zw.z, zw.w};
#pragma unroll
    for (int rt = 0; rt < 2; ++rt) {
        const uint4 c0 = cw[2 * rt], c1 = cw[2 * rt + 1];
        const uint32_t w0[4] = {c0.x, c0.y, c0.z, c0.w}, w1[4] = {c1.x, c1.y, c1.z, c1.w};
        const uint32_t z0 = (zws[2 * rt] >> zsh) & 0xFu, z1 = (zws[2 * rt + 1] >> zsh) & 0xFu;
        const uint32_t za0 = O::zz_a(z0), za1 = O::zz_a(z1), zb0 = O::zz_b(z0), zb1 = O::zz_b(z1);
        typename O::Scale sc0, sc1;
        if constexpr (!kPost) {
            sc0.set(sb[2 * rt]);
            sc1.set(sb[2 * rt + 1]);
        }
        float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        float (&d)[4] = kPost ? acc : tot[rt];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t q0[4], q1[4];
            O::unpack(w0[i], km, q0);
            O::unpack(w1[i], km, q1);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                q0[x] = x & 1 ? O::sub_b(q0[x], zb0) : O::sub_a(q0[x], za0);
                q1[x] = x & 1 ? O::sub_b(q1[x], zb1) : O::sub_a(q1[x], za1);
                if constexpr (!kPost) {
                    q0[x] = sc0.apply(q0[x]);
                    q1[x] = sc1.apply(q1[x]);
                }
            }
            O::mma(d, q0[0], q1[0], q0[2], q1[2], v[i].x, v[i].y);
            O::mma(d, q0[1], q1[1], q0[3], q1[3], v[i].z, v[i].w);
        }
        if constexpr (kPost) {
            const float s0 = __half2float(__ushort_as_half(sb[2 * rt])), s1 = __half2float(__ushort_as_half(sb[2 * rt + 1]));
            tot[rt][0] = fmaf(s0, acc[0], tot[rt][0]);
            tot[rt][1] = fmaf(s0, acc[1], tot[rt][1]);
            tot[rt][2] = fmaf(s1, acc[2], tot[rt][2]);
            tot[rt][3] = fmaf(s1, acc[3], tot[rt][3]);
        }
    }
}

// Group 128 on fp16 operands: one AND per register leaves a code pair as fp16 subnormals, u 2^-24 or
// 16 u 2^-24 (a second chain, times 1/16 in FP32), multiplied exactly; per unit the zero point comes
// off the FP32 sum, lo + hi / 16 - z sum_k a_k, and the scale (times 2^24 and the rows' powers of two)
// multiplies it.
template <bool kConv>
__device__ __forceinline__ void mg_unit_sub(uint32_t m8, const uint4 (&cw)[4], const uint16_t (&sb)[4], const uint4& zw,
                                            const uint4 (&v)[4], int zsh, float2 su, float2 up, float (&tot)[2][4]) {
    using O = GsOps<__half>;
    const uint32_t zws[4] = {zw.x, zw.y, zw.z, zw.w};
#pragma unroll
    for (int rt = 0; rt < 2; ++rt) {
        const uint4 c0 = cw[2 * rt], c1 = cw[2 * rt + 1];
        const uint32_t w0[4] = {c0.x, c0.y, c0.z, c0.w}, w1[4] = {c1.x, c1.y, c1.z, c1.w};
        float alo[4], ahi[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t h0 = mulhi(w0[i], m8), h1 = mulhi(w1[i], m8);
            const uint32_t a0 = w0[i] & 0x000F000Fu, a1 = w1[i] & 0x000F000Fu;
            const uint32_t a2 = h0 & 0x000F000Fu, a3 = h1 & 0x000F000Fu;
            const uint32_t b0 = w0[i] & 0x00F000F0u, b1 = w1[i] & 0x00F000F0u;
            const uint32_t b2 = h0 & 0x00F000F0u, b3 = h1 & 0x00F000F0u;
            if (i == 0) {
                O::mma_z(alo, a0, a1, a2, a3, v[i].x, v[i].y);
                O::mma_z(ahi, b0, b1, b2, b3, v[i].z, v[i].w);
            } else {
                O::mma(alo, a0, a1, a2, a3, v[i].x, v[i].y);
                O::mma(ahi, b0, b1, b2, b3, v[i].z, v[i].w);
            }
        }
        const float z0 = (float)((zws[2 * rt] >> zsh) & 0xFu), z1 = (float)((zws[2 * rt + 1] >> zsh) & 0xFu);
        const float s0 = __half2float(__ushort_as_half(sb[2 * rt])) * 16777216.0f;
        const float s1 = __half2float(__ushort_as_half(sb[2 * rt + 1])) * 16777216.0f;
        auto term = [](float z, float su1, float hi, float lo) { return fmaf(-z, su1, fmaf(hi, 0.0625f, lo)); };
        const float s0x = kConv ? s0 * up.x : s0, s0y = kConv ? s0 * up.y : s0;
        const float s1x = kConv ? s1 * up.x : s1, s1y = kConv ? s1 * up.y : s1;
        tot[rt][0] = fmaf(s0x, term(z0, su.x, ahi[0], alo[0]), tot[rt][0]);
        tot[rt][1] = fmaf(s0y, term(z0, su.y, ahi[1], alo[1]), tot[rt][1]);
        tot[rt][2] = fmaf(s1x, term(z1, su.x, ahi[2], alo[2]), tot[rt][2]);
        tot[rt][3] = fmaf(s1y, term(z1, su.y, ahi[3], alo[3]), tot[rt][3]);
    }
}

// The activation records. Half a warp takes one row's 128 K of a unit: lane c holds chunk c (8 K), whose
// pairs are stored (p0, p2, p1, p3). CONV: bf16 to fp16 (group 128); SUM: the record's sum (group 128).
constexpr int kMgActThreads = 256;
template <typename T, bool POST>
__global__ void __launch_bounds__(kMgActThreads) moe_acts_kernel(const T* __restrict__ A, int R, int K,
                                                                 uint8_t* __restrict__ acts) {
    constexpr bool kConv = POST && std::is_same<T, __nv_bfloat16>::value;
    pdl_wait();
    pdl_trigger();   // (after the wait: moe_gemv_kernel reads and writes before its own, pdl.cuh)
    const int c = threadIdx.x & 15;
    const long long item = (long long)blockIdx.x * (kMgActThreads / 16) + (threadIdx.x >> 4);
    const long long items = (long long)R * (K / 128);
    const long long at = item < items ? item : items - 1;   // (a whole warp stays for the shuffles)
    const int ku = (int)(at / R), row = (int)(at - (long long)ku * R);
    uint4 x = __ldg(reinterpret_cast<const uint4*>(A + (size_t)row * K + ku * 128 + 8 * c));
    uint32_t* xw = reinterpret_cast<uint32_t*>(&x);
    int k = 0;
    bool wide = false;
    float sum = 0.0f;
    if constexpr (kConv) {
        uint32_t emax = 0, emin = 255;   // largest and smallest nonzero biased exponent
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const uint32_t e0 = (xw[q] >> 7) & 0xFFu, e1 = (xw[q] >> 23) & 0xFFu;
            emax = max(emax, max(e0, e1));
            if (xw[q] & 0x7FFFu) emin = min(emin, e0);
            if (xw[q] & 0x7FFF0000u) emin = min(emin, e1);
        }
        uint32_t ee = (emax << 16) | (255u - emin);   // two 16-bit maxima at once
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) ee = __vmaxu2(ee, __shfl_xor_sync(0xffffffffu, ee, d));
        const int top = (int)(ee >> 16);
        wide = top - (255 - (int)(ee & 0xFFFFu)) > 31;
        k = half_shift(top);
        if (!wide) {
            const float down = pow2_f32(-k);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const __half2 y = __floats2half2_rn(__uint_as_float(xw[q] << 16) * down,
                                                    __uint_as_float(xw[q] & 0xFFFF0000u) * down);
                xw[q] = *reinterpret_cast<const uint32_t*>(&y);
            }
        }
    }
    if constexpr (POST) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const __half2 y = *reinterpret_cast<const __half2*>(&xw[q]);
            sum += __low2float(y) + __high2float(y);
        }
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    }
    if (item >= items) return;
    uint8_t* dst = acts + (size_t)at * kMgRowBytes;
    *reinterpret_cast<uint4*>(dst + (c >> 2) * 80 + (c & 3) * 16) = make_uint4(x.x, x.z, x.y, x.w);
    if (POST && c == 0) {
        MgNote n;
        n.sum = sum * 5.9604644775390625e-08f;   // 2^-24
        n.up = pow2_f32(k);
        n.wide = wide;
        n.pad = 0;
        *reinterpret_cast<MgNote*>(dst + 64) = n;
    }
}

template <typename T, int GROUP>
__global__ void __launch_bounds__(kMgThreads, 1) moe_gemv_kernel(const MgParams p) {
    extern __shared__ __align__(128) uint8_t smem[];
    constexpr bool kPost = GROUP == 128;
    constexpr bool kConv = kPost && std::is_same<T, __nv_bfloat16>::value;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int steps = p.K / 128, ns = p.ns, MR = p.rows, N = p.N;
    const uint32_t R = p.record;
    uint8_t* stages = smem;
    uint8_t* acts = smem + p.off_acts;                                 // [ns][4][MR][320]
    float* red = reinterpret_cast<float*>(smem + p.off_red);           // [2][4][MR][128]
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + p.off_bar);    // [ns] the stage's records landed
    uint64_t* empty = full + ns;                                       // [ns] the compute warps left it
    uint64_t* tfull = empty + ns;                                      // [2] the groups' sums are in `red`
    uint64_t* tempty = tfull + 2;                                      // [2] the epilogue warp has read them
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tempty + 2);
    int2* run_tab = reinterpret_cast<int2*>(smem + p.off_grp);
    int* blk_tab = reinterpret_cast<int*>(run_tab + p.E);

    if (threadIdx.x == 0) {
        for (int i = 0; i < ns; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], kMgWarps);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&tfull[i], kMgWarps);
            mbar_init(&tempty[i], 1);
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    // no row of a fresh slot reads as wide
    for (int i = threadIdx.x; i < ns * 4 * MR; i += kMgThreads)
        *reinterpret_cast<uint4*>(acts + (size_t)i * kMgRowBytes + 64) = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();   // (the slots are refilled by bulk copies)
    pdl_trigger();
    moe_table(p.offsets, p.E, p.R, MR, run_tab, blk_tab, [] { cta_sync(); });
    cta_sync();

    const long long U = (long long)blk_tab[p.E] * (N / 128) * steps;
    const int P = U < p.P ? (int)U : p.P, cta = blockIdx.x;
    if (cta >= P) {
        pdl_wait();   // this kernel does not complete before the one that it overtook
        return;
    }
    const long long u0 = mg_begin(cta, U, P), u1 = mg_begin(cta + 1, U, P);
    const int nunits = (int)(u1 - u0);   // (the host keeps the units of one range below 2^31)
    const int nst = (nunits + 3) / 4;
    const long long tau0 = u0 / steps;
    const int ku0 = (int)(u0 - tau0 * steps);

    if (warp == kMgWarpProducer) {
        // ------------------------------------------------------------ weight and activation records
        if (lane == 0) {
            MoeWalk w, wa;
            w.init(run_tab, blk_tab, p.E, N / 128, tau0);
            wa = w;
            int ku = ku0, kua = ku0, issued = 0;
            for (int st = 0; st < nst; ++st) {
                const int s = st % ns, n = min(4, nunits - 4 * st);
                if (st >= ns && !mbar_wait(&empty[s], (uint32_t)(st / ns - 1) & 1u, abort_flag, p.dev_status, p.wait_ns))
                    break;
                // the stage's bytes: its records, and every unit's rows
                uint32_t bytes = (uint32_t)n * R;
                int arow[4], am[4], ak[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (j < n) {
                        arow[j] = wa.row0(MR);
                        am[j] = min(MR, wa.row_end() - arow[j]);
                        ak[j] = kua;
                        bytes += (uint32_t)am[j] * kMgRowBytes;
                        if (++kua == steps && 4 * st + j + 1 < nunits) {
                            kua = 0;
                            wa.next();
                        }
                    }
                mbar_arrive_expect_tx(&full[s], bytes);
                uint8_t* dst = stages + (size_t)s * p.stage_bytes;
                for (int j = 0; j < n;) {   // runs of consecutive weight records
                    const long long rec = w.rec0(steps) + ku;
                    int c = min(n - j, steps - ku);
                    ku += c;
                    while (ku == steps) {
                        if (4 * st + j + c == nunits) break;
                        w.next();
                        ku = 0;
                        if (j + c < n && w.rec0(steps) == rec + c) {
                            const int more = min(n - j - c, steps);
                            c += more;
                            ku = more;
                        }
                    }
                    bulk_g2s(dst + (size_t)j * R, p.tiled + (size_t)rec * R, (uint32_t)c * R, &full[s]);
                    j += c;
                }
                if (st == 0) pdl_wait();   // the activation records are the previous kernel's
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (j < n)
                        bulk_g2s(acts + (size_t)(s * 4 + j) * MR * kMgRowBytes,
                                 p.acts + ((size_t)ak[j] * p.R + arow[j]) * kMgRowBytes, (uint32_t)am[j] * kMgRowBytes,
                                 &full[s]);
                ++issued;
            }
            // every copy issued lands before the CTA may exit
            volatile int keep = 0;
            for (int st = max(0, issued - ns); st < issued; ++st)
                mbar_wait(&full[st % ns], (uint32_t)(st / ns) & 1u, &keep, nullptr, kMgDrainNs);
        }
    } else if (warp == kMgWarpEpilogue) {
        // ------------------------------------------------------------ sums of a tile
        T* C = static_cast<T*>(p.C);
        MoeWalk w;
        w.init(run_tab, blk_tab, p.E, N / 128, tau0);
        int lo = 0, hi = min(steps - ku0, nunits);
        for (int et = 0; lo < nunits; ++et) {
            if (et > 0) w.next();
            const int bsel = et & 1;
            const long long tau = tau0 + et;
            const int cf = mg_owner(tau * steps, U, P), cl = mg_owner(tau * steps + steps - 1, U, P);
            const int r0 = w.row0(MR), m = min(MR, w.row_end() - r0);
            const size_t n0 = (size_t)w.nt * 128;
            const bool gather = cf != cl && cta == cf;
            float* pre = red + (size_t)(bsel ^ 1) * kMgGroups * MR * 128;
            if (gather) {
                // this tile is the range's last: the later CTAs' sums, added in CTA order into the other
                // buffer while the compute warps are still on the tile
                if (lane == 0) {
                    const uint64_t t0 = globaltimer_ns();
                    for (;;) {
                        int n;
                        asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(n) : "l"(p.counters + cta) : "memory");
                        if (n >= cl - cf) break;
                        if (*abort_flag || globaltimer_ns() - t0 > p.wait_ns) {
                            *abort_flag = 1;
                            report_status(p.dev_status, W4A16_ETIMEOUT);
                            break;
                        }
                    }
                    p.counters[cta] = 0;
                }
                __syncwarp();
                for (int r = 0; r < m; ++r) {
                    float y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                    for (int c0 = cf + 1; c0 <= cl; c0 += 4) {
                        float ld[4][4];
#pragma unroll
                        for (int q = 0; q < 4; ++q)
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                ld[q][j] = c0 + q <= cl ? __ldcg(p.partials + ((size_t)(c0 + q) * MR + r) * 128 + lane + 32 * j) : 0.0f;
#pragma unroll
                        for (int q = 0; q < 4; ++q)
#pragma unroll
                            for (int j = 0; j < 4; ++j) y[j] += ld[q][j];
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) pre[r * 128 + lane + 32 * j] = y[j];
                }
            }
            const bool ok = mg_wait(&tfull[bsel], (uint32_t)(et >> 1) & 1u, abort_flag, p.dev_status, p.wait_ns);
            const float* rb = red + (size_t)bsel * kMgGroups * MR * 128;
            float* part = p.partials + (size_t)cta * MR * 128;
            const bool mine = cf == cl || cta == cf;
            if (ok && !*abort_flag)
                for (int r = 0; r < m; ++r)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int ch = lane + 32 * j;
                        float o = (rb[(0 * MR + r) * 128 + ch] + rb[(1 * MR + r) * 128 + ch]) +
                                  (rb[(2 * MR + r) * 128 + ch] + rb[(3 * MR + r) * 128 + ch]);
                        if (!mine) part[r * 128 + ch] = o;
                        else C[(size_t)(r0 + r) * N + n0 + ch] = Act<T>::from_f32(gather ? o + pre[r * 128 + ch] : o);
                    }
            if (!mine) {
                __threadfence();
                __syncwarp();
                if (lane == 0) asm volatile("red.release.gpu.global.add.s32 [%0], 1;" ::"l"(p.counters + cf) : "memory");
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&tempty[bsel]);
            lo = hi;
            hi = min(lo + steps, nunits);
        }
    } else {
        // ------------------------------------------------------------ compute warps
        const int grp = warp >> 2, wg = warp & 3, g = lane >> 2, t = lane & 3;
        const int ch0 = 32 * wg + g;                                                   // channels ch0 + 8 r
        const int lg = kPost ? 0 : (32 * t) / GROUP;
        const uint32_t coff = (uint32_t)t * 2048u + (uint32_t)(ch0 ^ (2 * t)) * 16u;
        const uint32_t soff = p.scales_off + 256u * (uint32_t)lg + 2u * (uint32_t)ch0;
        const uint32_t zoff = p.zeros_off + 64u * (uint32_t)lg + 16u * (uint32_t)wg;
        const int zsh = 4 * g, sym = p.sym;
        // rows at or past MR read row MR - 1 (their sums are not stored)
        const uint32_t aoff = (uint32_t)min(g, MR - 1) * kMgRowBytes + (uint32_t)t * 80u;
        const uint32_t note0 = (uint32_t)min(2 * t, MR - 1) * kMgRowBytes + 64u;
        const uint32_t note1 = (uint32_t)min(2 * t + 1, MR - 1) * kMgRowBytes + 64u;
        float tot[2][4] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
        bool aborted = false;
        int s = -1, n_tile = 0;
        uint32_t ph = 0;
        int lo = 0, hi = min(steps - ku0, nunits);
        for (;;) {
            for (int li = lo + ((grp - lo) & 3); li < hi; li += 4) {
                if (++s == ns) {
                    s = 0;
                    ph ^= 1u;
                }
                if (!aborted && !mg_wait(&full[s], ph, abort_flag, p.dev_status, p.wait_ns)) aborted = true;
                if (!aborted) {
                    const uint8_t* rec = stages + (size_t)s * p.stage_bytes + (uint32_t)grp * R;
                    const uint8_t* au = acts + (size_t)(s * 4 + grp) * MR * kMgRowBytes;
                    const uint8_t* a = au + aoff;
                    uint4 cw[4], v[4];
                    uint16_t sb[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        cw[r] = *reinterpret_cast<const uint4*>(rec + coff + 128 * r);
                        sb[r] = *reinterpret_cast<const uint16_t*>(rec + soff + 16 * r);
                        v[r] = *reinterpret_cast<const uint4*>(a + 16 * r);
                    }
                    uint4 zw = make_uint4(0x88888888u, 0x88888888u, 0x88888888u, 0x88888888u);   // symmetric: z = 8
                    if (!sym) zw = *reinterpret_cast<const uint4*>(rec + zoff);
                    if constexpr (kPost) {
                        // the notes of this lane's columns, rows 2 t and 2 t + 1
                        const MgNote n0 = *reinterpret_cast<const MgNote*>(au + note0);
                        const MgNote n1 = *reinterpret_cast<const MgNote*>(au + note1);
                        const bool mix = kConv && __any_sync(0xffffffffu, n0.wide | n1.wide);
                        float nat[2][4];
                        if (mix) {   // some row of the unit is kept in bf16: both forms, then each column's own
#pragma unroll
                            for (int e = 0; e < 8; ++e) nat[e >> 2][e & 3] = tot[e >> 2][e & 3];
                            mg_unit<GsOps<__nv_bfloat16>, true>(p.km_native, cw, sb, zw, v, zsh, nat);
                        }
                        mg_unit_sub<kConv>(p.km.m8, cw, sb, zw, v, zsh, make_float2(n0.sum, n1.sum),
                                           make_float2(n0.up, n1.up), tot);
                        if (mix) {
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                if (e & 1 ? n1.wide : n0.wide) tot[e >> 2][e & 3] = nat[e >> 2][e & 3];
                        }
                    } else {
                        mg_unit<GsOps<T>, false>(p.km, cw, sb, zw, v, zsh, tot);
                    }
                }
                __syncwarp();
                if (lane == 0 && !aborted) mbar_arrive(&empty[s]);
            }
            // the group's sums of the tile segment, to one of two buffers
            const int bsel = n_tile & 1;
            (void)mg_wait(&tempty[bsel], ((uint32_t)(n_tile >> 1) & 1u) ^ 1u, abort_flag, p.dev_status, p.wait_ns);
            float* rb = red + ((size_t)bsel * kMgGroups + grp) * MR * 128;
#pragma unroll
            for (int rt = 0; rt < 2; ++rt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int r = 2 * t + (e & 1);
                    if (r < MR) rb[r * 128 + ch0 + 16 * rt + 8 * (e >> 1)] = tot[rt][e];
                    tot[rt][e] = 0.0f;
                }
            __syncwarp();
            if (lane == 0) mbar_arrive(&tfull[bsel]);
            ++n_tile;
            lo = hi;
            if (lo >= nunits) break;
            hi = min(lo + steps, nunits);
        }
    }
    cta_sync();
}

struct MgPlan {
    bool ok;
    int rows, ns, ctas;
    uint32_t stage_bytes, off_acts, off_red, off_bar, off_grp;
    size_t smem;
};

MgPlan plan_moe_gemv(int R, int E, int N, int K, int group, int sym, int n_sm) {
    MgPlan pl = {};
    if (R < 1 || E < 1 || K % 128 != 0 || N % 128 != 0 || K < 128 || N < 128 || n_sm <= 0) return pl;
    const TiledLayout L = tiled_layout(K, N, group, sym);
    pl.rows = R < kMgMaxRows ? R : kMgMaxRows;
    pl.ctas = n_sm;
    pl.stage_bytes = (4u * L.record + 127u) & ~127u;
    auto up = [](size_t x) { return (x + 127) & ~(size_t)127; };
    const size_t red = up((size_t)2 * kMgGroups * pl.rows * 128 * 4);
    const size_t bars = up((size_t)2 * kMgMaxStages * 8 + 32 + 16), grp = up((size_t)E * 12 + 4);
    const size_t per = pl.stage_bytes + up((size_t)4 * pl.rows * kMgRowBytes);
    size_t ns = ((size_t)kMgSmemMax - red - bars - grp - 256) / per;
    if (ns > kMgMaxStages) ns = kMgMaxStages;
    if (ns < kMgMinStages) return pl;
    pl.ns = (int)ns;
    size_t at = ns * pl.stage_bytes;
    pl.off_acts = (uint32_t)at;
    at = up(at + ns * 4 * pl.rows * kMgRowBytes);
    pl.off_red = (uint32_t)at;
    at += red;
    pl.off_bar = (uint32_t)at;
    at += bars;
    pl.off_grp = (uint32_t)at;
    at += grp;
    pl.smem = at;
    // the units of one CTA's range fit an int
    const long long most = ((long long)R / pl.rows + E) * (N / 128) * (K / 128) / n_sm;
    pl.ok = at <= (size_t)kMgSmemMax && most < (1ll << 30);
    return pl;
}

template <typename T, int GROUP>
int launch_mg(const MgParams& prm, size_t smem, cudaStream_t stream) {
    static std::atomic<uint64_t> done{0};
    if (!allow_smem(moe_gemv_kernel<T, GROUP>, kMgSmemMax, done)) return W4A16_ECUDA;
    return launch_pdl(moe_gemv_kernel<T, GROUP>, dim3(prm.P), dim3(kMgThreads), smem, stream, prm) == cudaSuccess
               ? W4A16_OK
               : W4A16_ECUDA;
}

template <typename T>
int launch_acts(const void* A, int R, int K, int group, const uint8_t* acts, cudaStream_t stream) {
    const long long items = (long long)R * (K / 128);
    const dim3 grid((unsigned)((items + kMgActThreads / 16 - 1) / (kMgActThreads / 16))), block(kMgActThreads);
    const cudaError_t e = group == 128 ? launch_pdl(moe_acts_kernel<T, true>, grid, block, 0, stream, static_cast<const T*>(A), R, K,
                                                    const_cast<uint8_t*>(acts))
                                       : launch_pdl(moe_acts_kernel<T, false>, grid, block, 0, stream, static_cast<const T*>(A), R, K,
                                                    const_cast<uint8_t*>(acts));
    return e == cudaSuccess ? W4A16_OK : W4A16_ECUDA;
}

template <typename T>
int launch_mg_group(const MgParams& prm, int group, size_t smem, cudaStream_t stream) {
    switch (group) {
        case 32: return launch_mg<T, 32>(prm, smem, stream);
        case 64: return launch_mg<T, 64>(prm, smem, stream);
        default: return launch_mg<T, 128>(prm, smem, stream);
    }
}

}  // namespace

// Workspace after the counters: the cut tiles' sums, then the activation records.
static size_t moe_gemv_sum_bytes(int R) {
    int n_sm = gemv_stream_sm_count();
    if (n_sm <= 0) n_sm = 148;
    return (size_t)n_sm * (R < kMgMaxRows ? R : kMgMaxRows) * 128 * sizeof(float);
}

// (without a device to ask, as where it has 148 SMs)
bool moe_gemv_fits(int R, int E, int N, int K, int group, int sym) {
    const int n_sm = gemv_stream_sm_count();
    return plan_moe_gemv(R, E, N, K, group, sym, n_sm > 0 ? n_sm : 148).ok;
}

size_t moe_gemv_partial_bytes(int R, int K) { return moe_gemv_sum_bytes(R) + (size_t)R * (K / 128) * kMgRowBytes; }

int launch_moe_gemv(const void* A, int a_dtype, int R, int K, const void* tiled, int E, const int32_t* offsets, int N,
                    int group, int sym, void* C, void* workspace, int* dev_status, cudaStream_t stream) {
    const MgPlan pl = plan_moe_gemv(R, E, N, K, group, sym, gemv_stream_sm_count());
    if (!pl.ok) return W4A16_EUNSUPPORTED;
    const TiledLayout L = tiled_layout(K, N, group, sym);
    const bool bf16 = a_dtype == W4A16_BF16;
    MgParams prm = {};
    prm.acts = static_cast<uint8_t*>(workspace) + kGemvStreamCounterBytes + moe_gemv_sum_bytes(R);
    prm.tiled = static_cast<const uint8_t*>(tiled);
    prm.C = C;
    prm.counters = static_cast<int*>(workspace);
    prm.partials = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kGemvStreamCounterBytes);
    prm.dev_status = dev_status;
    prm.offsets = offsets;
    prm.E = E;
    prm.R = R;
    prm.K = K;
    prm.N = N;
    prm.sym = sym;
    prm.ns = pl.ns;
    prm.P = pl.ctas;
    prm.rows = pl.rows;
    prm.record = L.record;
    prm.scales_off = L.scales;
    prm.zeros_off = L.zeros;
    prm.stage_bytes = pl.stage_bytes;
    prm.off_acts = pl.off_acts;
    prm.off_red = pl.off_red;
    prm.off_bar = pl.off_bar;
    prm.off_grp = pl.off_grp;
    const bool bf16_math = bf16 && group != 128;   // bf16 at group 128 runs the fp16 arithmetic
    prm.km.lo = 0x000F000Fu;
    prm.km.hi = bf16_math ? 0x000F000Fu : 0x00F000F0u;
    prm.km.magic = bf16_math ? 0x43004300u : 0x64006400u;
    prm.km.m4 = 1u << 28;
    prm.km.m8 = 1u << 24;
    prm.km.m12 = 1u << 20;
    prm.km_native = prm.km;
    prm.km_native.hi = 0x000F000Fu;
    prm.km_native.magic = 0x43004300u;
    prm.wait_ns = wait_limit_ns();
    const int st = bf16 ? launch_acts<__nv_bfloat16>(A, R, K, group, prm.acts, stream)
                        : launch_acts<__half>(A, R, K, group, prm.acts, stream);
    if (st != W4A16_OK) return st;
    return bf16 ? launch_mg_group<__nv_bfloat16>(prm, group, pl.smem, stream)
                : launch_mg_group<__half>(prm, group, pl.smem, stream);
}

}  // namespace w4a16
