// moe_route.cu -- tokens sorted by expert, back with weights applied, and the gradients (sm_100a).
//
// A router gives token t the experts ids[t, j], j < k. With the flat index i = t k + j and e_i its id,
//   slot_i = #{i' : e_i' < e_i} + #{i' < i : e_i' = e_i},  rows[slot_i] = i,  Xs[slot_i] = X[t]
// (a stable counting sort), offsets[e] = #{i : e_i < e}; an id outside [0, E) has no row (slot -1).
//   combine:  Y[t] = sum_j w[t, j] Ys[slot[t, j]]   (FP32 sums in the order of j, rounded once)
//   gradient: dYs[slot] = w dY[t],  dw[t, j] = <dY[t], Ys[slot]>,  dX[t] = sum_j dXs[slot[t, j]]
// With rows to move, all of it is bound by memory: they go once in and once out. The maps are small beside them up to
// some 10^5 ids; beyond, the histograms set the time, blocks x E counts that every CTA adds up by itself (maps alone, us:
// 131072 ids 20.4 at 128 bins, 31.4 at 1024; 1048576 ids 91.8 and 166; 8388608 ids at 1024 bins 1790).
#include "pdl.cuh"
#include "routed.cuh"

namespace w4a16 {
namespace {

constexpr int kSortThreads = 256;
constexpr int kSortList = 1024;   // slots of own ids kept in shared memory at a time

// One count per distinct bin of the warp: the lanes that share a bin add once.
__device__ __forceinline__ void count_bin(int* bins, int e, bool live) {
    const unsigned active = __ballot_sync(0xffffffffu, live);
    if (!live) return;
    const unsigned peers = __match_any_sync(active, e);
    if ((threadIdx.x & 31) == __ffs(peers) - 1) atomicAdd(&bins[e], __popc(peers));
}

__device__ __forceinline__ int bin_of(int id, int E) { return (unsigned)id < (unsigned)E ? id : -1; }

// hist[b][e]: ids of block b (kRouteHistIds consecutive ids) in bin e.
__global__ void __launch_bounds__(kSortThreads) route_hist_kernel(const int32_t* __restrict__ ids, int n, int E,
                                                                  int32_t* __restrict__ hist) {
    __shared__ int bins[kRouteMaxBins];
    for (int e = threadIdx.x; e < E; e += kSortThreads) bins[e] = 0;
    __syncthreads();
    pdl_wait();
    pdl_trigger();
    const int lo = blockIdx.x * kRouteHistIds;
    int e[kRouteHistIds / kSortThreads];
#pragma unroll
    for (int q = 0; q < kRouteHistIds / kSortThreads; ++q) {
        const int i = lo + q * kSortThreads + threadIdx.x;
        e[q] = i < n ? bin_of(ids[i], E) : -1;
    }
#pragma unroll
    for (int q = 0; q < kRouteHistIds / kSortThreads; ++q) count_bin(bins, e[q], e[q] >= 0);
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kSortThreads) hist[(size_t)blockIdx.x * E + e] = bins[e];
}

// The sort and the gather in one launch. Every CTA (blockIdx.x) owns tokens_per_cta consecutive
// tokens and finds their slots by itself: it counts all ids (up to kRouteDirectIds of them, a few
// KB from L2) or adds up the blocks' histograms, so no CTA waits for another. blockIdx.y cuts the
// row length when there are fewer tokens than SMs. Measured on the decode batch (64 ids): one
// launch instead of count, scan, scatter and gather.
__global__ void __launch_bounds__(kSortThreads) route_sort_kernel(const RouteSort p, int tokens_per_cta, int chunks) {
    __shared__ int lower[kRouteMaxBins];   // ids of the bin before the CTA's own, then the next slot
    __shared__ int upper[kRouteMaxBins];   // ids of the bin from the CTA's own on
    __shared__ int list[kSortList];
    __shared__ int wsum[kSortThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n = p.T * p.k, E = p.E;
    const int t0 = blockIdx.x * tokens_per_cta;
    const int t1 = min(t0 + tokens_per_cta, p.T);
    const int lo = t0 * p.k;
    for (int e = tid; e < E; e += kSortThreads) lower[e] = upper[e] = 0;
    __syncthreads();
    pdl_wait();
    pdl_trigger();

    // counts of every bin, before the CTA's first id and from it on
    if (p.hist) {
        const int blocks = (n + kRouteHistIds - 1) / kRouteHistIds, own = lo / kRouteHistIds;
        for (int e = tid; e < E; e += kSortThreads) {
            int a = 0, b = 0;
#pragma unroll 8
            for (int q = 0; q < blocks; ++q) {
                const int c = __ldcg(p.hist + (size_t)q * E + e);
                if (q < own) a += c;
                else b += c;
            }
            lower[e] = a;
            upper[e] = b;
        }
        __syncthreads();
        for (int i0 = own * kRouteHistIds; i0 < lo; i0 += 8 * kSortThreads) {   // (once)
            int e[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const int i = i0 + q * kSortThreads + tid;
                e[q] = i < lo ? bin_of(p.ids[i], E) : -1;
            }
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const unsigned active = __ballot_sync(0xffffffffu, e[q] >= 0);
                if (e[q] >= 0) {
                    const unsigned peers = __match_any_sync(active, e[q]);
                    if (lane == __ffs(peers) - 1) {
                        atomicAdd(&lower[e[q]], __popc(peers));
                        atomicSub(&upper[e[q]], __popc(peers));
                    }
                }
            }
        }
    } else {
        for (int i0 = 0; i0 < n; i0 += 4 * kSortThreads) {
            int e[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int i = i0 + q * kSortThreads + tid;
                e[q] = i < n ? bin_of(p.ids[i], E) : -1;
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int i = i0 + q * kSortThreads + tid;
                count_bin(lower, e[q], e[q] >= 0 && i < lo);
                count_bin(upper, e[q], e[q] >= 0 && i >= lo);
            }
        }
    }
    __syncthreads();

    // exclusive scan over the bins: `per` consecutive bins per thread. lower[e] becomes the slot of
    // the CTA's next id of bin e. The first CTA writes the offsets.
    const bool first = blockIdx.x == 0 && blockIdx.y == 0;
    {
        const int per = (E + kSortThreads - 1) / kSortThreads;
        const int e0 = tid * per, e1 = min(e0 + per, E);
        int s = 0;
        for (int e = e0; e < e1; ++e) s += lower[e] + upper[e];
        int x = s;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, d);
            if (lane >= d) x += y;
        }
        if (lane == 31) wsum[warp] = x;
        __syncthreads();
        int base = x - s;
        for (int w = 0; w < warp; ++w) base += wsum[w];
        for (int e = e0; e < e1; ++e) {
            const int c = lower[e] + upper[e];
            if (first) {
                p.offsets[e] = base;
                if (e == E - 1) p.offsets[E] = base + c;
            }
            lower[e] += base;
            base += c;
        }
    }
    __syncthreads();

    // the CTA's ids in order, by one warp, kSortList of them at a time; then their rows
    const int H8 = p.H / 8;
    const int c0 = (int)((long long)H8 * blockIdx.y / chunks), c1 = (int)((long long)H8 * (blockIdx.y + 1) / chunks);
    const int batch = kSortList / p.k;
    for (int ta = t0; ta < t1; ta += batch) {
        const int tb = min(ta + batch, t1);
        const int own = (tb - ta) * p.k;
        if (warp == 0) {
            for (int q = 0; q < own; q += 32) {
                const int i = ta * p.k + q + lane;
                const int e = q + lane < own ? bin_of(p.ids[i], E) : -1;
                const unsigned active = __ballot_sync(0xffffffffu, e >= 0);
                int slot = -1;
                if (e >= 0) {
                    const unsigned peers = __match_any_sync(active, e);
                    slot = lower[e] + __popc(peers & ((1u << lane) - 1u));
                    __syncwarp(active);
                    if (lane == __ffs(peers) - 1) lower[e] += __popc(peers);
                }
                __syncwarp();
                if (q + lane < own) {
                    list[q + lane] = slot;
                    if (blockIdx.y == 0) {
                        p.slots[i] = slot;
                        if (slot >= 0) p.rows[slot] = i;
                    }
                }
            }
        }
        __syncthreads();
        if (p.X) {
            const uint4* X = static_cast<const uint4*>(p.X);
            uint4* Xs = static_cast<uint4*>(p.Xs);
            const int w = c1 - c0;
            // two (token, chunk) items per thread in flight
            const int items = (tb - ta) * w;
            for (int it = tid; it < items; it += 2 * kSortThreads) {
                const int it2 = it + kSortThreads;
                const int ra = it / w, ca = it - ra * w;
                const int rb = it2 / w, cb = it2 - rb * w;
                const uint4 va = __ldcs(X + (size_t)(ta + ra) * H8 + c0 + ca);
                uint4 vb = make_uint4(0, 0, 0, 0);
                if (it2 < items) vb = __ldcs(X + (size_t)(ta + rb) * H8 + c0 + cb);
                for (int j = 0; j < p.k; ++j) {
                    const int sa = list[ra * p.k + j];
                    if (sa >= 0) Xs[(size_t)sa * H8 + c0 + ca] = va;
                    if (it2 < items) {
                        const int sb = list[rb * p.k + j];
                        if (sb >= 0) Xs[(size_t)sb * H8 + c0 + cb] = vb;
                    }
                }
            }
        }
        __syncthreads();
    }
}

// ------------------------------------------------------------------------------ combine
constexpr int kCombThreads = 256;

template <typename T>
__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
    const T* h = reinterpret_cast<const T*>(&v);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = Act<T>::to_f32(h[i]);
}

template <typename T>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    uint4 v;
    T* h = reinterpret_cast<T*>(&v);
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = Act<T>::from_f32(f[i]);
    return v;
}

// One thread per 8 columns of one token: up to eight choices' rows in flight, FP32 sums in the
// order of j. A choice without a row (slot outside [0, T k)) is neither read nor multiplied.
template <typename T, bool W>
__global__ void __launch_bounds__(kCombThreads) moe_combine_kernel(const uint4* __restrict__ Ys, int tokens, int k,
                                                                   int H8, const int32_t* __restrict__ slots,
                                                                   const float* __restrict__ weights,
                                                                   uint4* __restrict__ Y) {
    pdl_wait();
    pdl_trigger();
    const long long i0 = (long long)blockIdx.x * kCombThreads;
    const long long tb = i0 / H8;
    const int local = (int)(i0 - tb * H8) + threadIdx.x;
    const long long t = tb + local / H8;
    const int c = local % H8;
    if (t >= tokens) return;
    const unsigned n = (unsigned)(tokens * k);
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = 0.0f;
    for (int j0 = 0; j0 < k; j0 += 8) {
        uint4 v[8];
        float w[8];
        bool has[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            has[j] = false;
            if (j0 + j < k) {
                const int s = __ldg(slots + t * k + j0 + j);
                has[j] = (unsigned)s < n;
                if (has[j]) {
                    v[j] = __ldcs(Ys + (size_t)s * H8 + c);
                    w[j] = W ? __ldg(weights + t * k + j0 + j) : 1.0f;
                }
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (has[j]) {
                float f[8];
                unpack8<T>(v[j], f);
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = W ? fmaf(w[j], f[i], y[i]) : y[i] + f[i];
            }
    }
    Y[(size_t)t * H8 + c] = pack8<T>(y);
}

// ------------------------------------------------------------------------------ combine's gradient
// One warp per choice (t, j): dY[t] (from L1 or L2 after the token's first warp) times w to the sorted
// row, and its product with Ys[slot] summed per lane, then over the lanes in a fixed order.
template <typename T, bool W>
__global__ void __launch_bounds__(kCombThreads) moe_combine_grad_kernel(const uint4* __restrict__ dY,
                                                                        const uint4* __restrict__ Ys, int n, int k,
                                                                        int H8, const int32_t* __restrict__ slots,
                                                                        const float* __restrict__ weights,
                                                                        uint4* __restrict__ dYs,
                                                                        float* __restrict__ dw) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int i = blockIdx.x * (kCombThreads / 32) + (threadIdx.x >> 5);
    if (i >= n) return;
    const int s = __ldg(slots + i);
    if ((unsigned)s >= (unsigned)n) {
        if (dw && lane == 0) dw[i] = 0.0f;
        return;
    }
    const float w = W ? __ldg(weights + i) : 1.0f;
    const uint4* g = dY + (size_t)(i / k) * H8;
    const uint4* y = Ys + (size_t)s * H8;
    uint4* o = dYs + (size_t)s * H8;
    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int c0 = lane; c0 < H8; c0 += 128) {
        uint4 gv[4], yv[4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (c0 + 32 * q < H8) {
                gv[q] = __ldg(g + c0 + 32 * q);
                if (dw) yv[q] = __ldcs(y + c0 + 32 * q);
            }
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (c0 + 32 * q < H8) {
                float f[8], h[8];
                unpack8<T>(gv[q], f);
                if (dw) {
                    unpack8<T>(yv[q], h);
#pragma unroll
                    for (int e = 0; e < 8; ++e) acc[q] = fmaf(f[e], h[e], acc[q]);
                }
                if (W) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) f[e] *= w;
                    o[c0 + 32 * q] = pack8<T>(f);
                } else {
                    o[c0 + 32 * q] = gv[q];
                }
            }
    }
    if (dw) {
        float a = (acc[0] + acc[1]) + (acc[2] + acc[3]);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) a += __shfl_xor_sync(0xffffffffu, a, d);
        if (lane == 0) dw[i] = a;
    }
}

}  // namespace

size_t route_sort_workspace_bytes(int T, int k, int E) {
    const long long n = (long long)T * k;
    if (n <= kRouteDirectIds) return 0;
    return (size_t)((n + kRouteHistIds - 1) / kRouteHistIds) * (size_t)E * sizeof(int32_t);
}

int launch_route_sort(const RouteSort& q, cudaStream_t stream) {
    RouteSort p = q;
    const int n = p.T * p.k;
    if (n <= kRouteDirectIds) {
        p.hist = nullptr;
    } else {
        const unsigned blocks = (unsigned)((n + kRouteHistIds - 1) / kRouteHistIds);
        if (launch_pdl(route_hist_kernel, dim3(blocks), dim3(kSortThreads), 0, stream, p.ids, n, p.E, p.hist) !=
            cudaSuccess)
            return W4A16_ECUDA;
    }
    int n_sm = gemv_stream_sm_count();
    if (n_sm <= 0) n_sm = 148;
    int ctas, chunks = 1;
    if (p.X) {
        // four CTAs per SM; with fewer tokens than SMs, the rows cut into pieces of at least 256
        // 16-byte chunks
        ctas = p.T < 4 * n_sm ? p.T : 4 * n_sm;
        while (ctas * chunks * 2 <= 2 * n_sm && p.H / 8 / (chunks * 2) >= kSortThreads) chunks *= 2;
    } else {
        ctas = (n + kSortThreads - 1) / kSortThreads;
        if (ctas > 2 * n_sm) ctas = 2 * n_sm;
        if (ctas > p.T) ctas = p.T;
    }
    const int per = (p.T + ctas - 1) / ctas;
    ctas = (p.T + per - 1) / per;
    const cudaError_t e =
        launch_pdl(route_sort_kernel, dim3(ctas, chunks), dim3(kSortThreads), 0, stream, p, per, chunks);
    return e == cudaSuccess ? W4A16_OK : W4A16_ECUDA;
}

int launch_moe_combine(const void* Ys, int dtype, int T, int k, int H, const int32_t* slots, const float* weights,
                       void* Y, cudaStream_t stream) {
    const int H8 = H / 8;
    const long long threads = (long long)T * H8;
    const dim3 grid((unsigned)((threads + kCombThreads - 1) / kCombThreads)), block(kCombThreads);
    auto go = [&](auto kernel) {
        return launch_pdl(kernel, grid, block, 0, stream, static_cast<const uint4*>(Ys), T, k, H8, slots, weights,
                          static_cast<uint4*>(Y)) == cudaSuccess
                   ? W4A16_OK
                   : W4A16_ECUDA;
    };
    if (dtype == W4A16_BF16)
        return weights ? go(moe_combine_kernel<__nv_bfloat16, true>) : go(moe_combine_kernel<__nv_bfloat16, false>);
    return weights ? go(moe_combine_kernel<__half, true>) : go(moe_combine_kernel<__half, false>);
}

int launch_moe_combine_grad(const void* dY, const void* Ys, int dtype, int T, int k, int H, const int32_t* slots,
                            const float* weights, void* dYs, float* dweights, cudaStream_t stream) {
    const int n = T * k;
    const dim3 grid((unsigned)((n + kCombThreads / 32 - 1) / (kCombThreads / 32))), block(kCombThreads);
    auto go = [&](auto kernel) {
        return launch_pdl(kernel, grid, block, 0, stream, static_cast<const uint4*>(dY), static_cast<const uint4*>(Ys), n,
                          k, H / 8, slots, weights, static_cast<uint4*>(dYs), dweights) == cudaSuccess
                   ? W4A16_OK
                   : W4A16_ECUDA;
    };
    if (dtype == W4A16_BF16)
        return weights ? go(moe_combine_grad_kernel<__nv_bfloat16, true>)
                       : go(moe_combine_grad_kernel<__nv_bfloat16, false>);
    return weights ? go(moe_combine_grad_kernel<__half, true>) : go(moe_combine_grad_kernel<__half, false>);
}

}  // namespace w4a16
