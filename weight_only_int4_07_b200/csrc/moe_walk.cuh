// moe_walk.cuh -- the tiles of a launch over runs of sorted rows (experts), found on the device.
//
// A tile is 128 channels x one block of up to `bn` rows of one expert. Tiles are ordered expert-major,
// then by channel tile, then by row block (the row blocks of one channel tile are neighbours, so their
// weights come from HBM once and from L2 after); an expert without rows has none.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace w4a16 {
namespace {

// The runs' table in shared memory: first and past-the-last row of every expert, and blk[e], the row
// blocks before expert e (blk[E]: all). Offsets outside [0, rows] are clamped to it and a run that
// ends before it begins is empty, so no offset reads or writes outside the buffers. Called by all
// threads; the table may be read after the block's next barrier.
template <typename Sync>
__device__ __forceinline__ void moe_table(const int32_t* offsets, int E, int rows, int bn, int2* run, int* blk, Sync sync) {
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
        const int lo = min(max(__ldcg(offsets + e), 0), rows), hi = min(max(__ldcg(offsets + e + 1), 0), rows);
        run[e] = make_int2(lo, max(lo, hi));
    }
    sync();
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        int base = 0;
        for (int e0 = 0; e0 < E; e0 += 32) {
            const int e = e0 + lane;
            const int nb = e < E ? (run[e].y - run[e].x + bn - 1) / bn : 0;
            int x = nb;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, d);
                if (lane >= d) x += y;
            }
            if (e < E) blk[e] = base + x - nb;
            base += __shfl_sync(0xffffffffu, x, 31);
        }
        if (lane == 0) blk[E] = base;
    }
}

// A role's place among the tiles.
struct MoeWalk {
    const int2* run;
    const int* blk;
    int e, nt, mb, NT;
    __device__ __forceinline__ void init(const int2* r, const int* b, int E, int channel_tiles, long long tau) {
        run = r;
        blk = b;
        NT = channel_tiles;
        int lo = 0, hi = E - 1;   // the last expert whose first tile is at or before tau (one with rows)
        while (lo < hi) {
            const int m = (lo + hi + 1) >> 1;
            if ((long long)blk[m] * NT <= tau) lo = m;
            else hi = m - 1;
        }
        e = lo;
        const int nb = blk[e + 1] - blk[e];
        const int q = (int)(tau - (long long)blk[e] * NT);
        nt = nb > 0 ? q / nb : 0;
        mb = nb > 0 ? q - nt * nb : 0;
    }
    // the next tile (the caller knows that there is one)
    __device__ __forceinline__ void next() {
        if (++mb < blk[e + 1] - blk[e]) return;
        mb = 0;
        if (++nt < NT) return;
        nt = 0;
        do ++e;
        while (blk[e + 1] == blk[e]);
    }
    // record index of the tile's first unit in the experts' buffers, its first row, past the run's last
    __device__ __forceinline__ long long rec0(int steps) const { return ((long long)e * NT + nt) * steps; }
    __device__ __forceinline__ int row0(int bn) const { return run[e].x + mb * bn; }
    __device__ __forceinline__ int row_end() const { return run[e].y; }
};

}  // namespace
}  // namespace w4a16
