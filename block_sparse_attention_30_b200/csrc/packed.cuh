// packed.cuh -- where a tile of packed sequences lies.  The borders `cu` are
// device data, so the host only knows an upper bound of the number of tiles;
// every warp finds its tile by a scan over the sequences' tile counts.
#pragma once
#include <cstdint>

#include "common.cuh"

namespace vsa {

struct SeqRange {
    int begin, len;
};

// Sequence i's rows.  Borders that do not ascend within [0, total] are
// reported, and the sequence is taken as empty: no row outside the tensors
// is ever addressed.
__device__ __forceinline__ SeqRange seq_range(const int32_t* __restrict__ cu, int i, int total, int* status) {
    const int a = __ldg(cu + i), b = __ldg(cu + i + 1);
    if (a < 0 || b < a || b > total) {
        report(status, kStatusBadIndex);
        return {0, 0};
    }
    return {a, b - a};
}

// Keys that query token i of the sequence sees.
__device__ __forceinline__ int seen_keys(int i, int nq, int nk, int causal) {
    return causal ? max(0, min(nk, i + 1 + nk - nq)) : nk;
}

struct SeqTile {
    int seq;     // -1: past the last tile
    int tile;    // tile within the sequence
};

// Tile t of the tiles of `len` rows that the sequences are cut into (`least`
// for an empty one), sequence after sequence (whole warp; every lane gets the
// result).  Four sequences per lane and step: one round trip to L2 covers 128
// sequences.
__device__ __forceinline__ SeqTile find_tile(const int32_t* __restrict__ cu, int n_seq, int total, int len, int t,
                                             int* status, int least = 0) {
    const int lane = threadIdx.x & 31;
    long long base = 0;            // 64 bits: borders that overlap can sum to more than the rows
    for (int s0 = 0; s0 < n_seq; s0 += 128) {
        int cnt[4];
        long long sum = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int s = s0 + 4 * lane + e;
            cnt[e] = 0;
            if (s < n_seq) cnt[e] = max(least, (seq_range(cu, s, total, status).len + len - 1) / len);
            sum += cnt[e];
        }
        long long incl = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += y;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, base + incl > t);
        if (hit) {
            const int src = __ffs(hit) - 1;
            SeqTile r{-1, 0};
            long long at = base + incl - sum;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (r.seq < 0 && t < at + cnt[e]) { r.seq = s0 + 4 * lane + e; r.tile = (int)(t - at); }
                at += cnt[e];
            }
            r.seq = __shfl_sync(0xffffffffu, r.seq, src);
            r.tile = __shfl_sync(0xffffffffu, r.tile, src);
            return r;
        }
        base += __shfl_sync(0xffffffffu, incl, 31);
    }
    return {-1, 0};
}

}  // namespace vsa
