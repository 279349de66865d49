// packed.cuh -- where a tile of packed sequences lies.  The borders `cu` are
// device data, so the host only knows an upper bound of the number of tiles;
// every warp finds its tile by a search over the borders.
#pragma once
#include <cstdint>

#include "common.cuh"
#include "packed.h"
#include "sm100.cuh"

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
    int seq;     // -1: none
    int tile;    // tile within the sequence
    SeqRange a, b;
};

// The last of the sequences 0 .. n_seq - 1 for which left(s), which descends, is
// not below 0, or -1 (whole warp): 32 parts at a time.
template <typename F>
__device__ __forceinline__ int find_last(int n_seq, F left) {
    const int lane = threadIdx.x & 31;
    int lo = 0, step = 1;
    while (32 * step < n_seq) step *= 32;
    for (;; step /= 32) {
        const int s = lo + lane * step;
        const unsigned hit = __ballot_sync(0xffffffffu, s < n_seq && left(s) >= 0);
        if (!hit) return -1;
        lo += (31 - __clz(hit)) * step;
        if (step == 1) return lo;
    }
}

// A border that is within the rows, whatever the memory holds.
__device__ __forceinline__ int border(const int32_t* __restrict__ cu, int s, int total) { return max(0, min(total, __ldg(cu + s))); }

// What is at place t when each sequence is cut into tiles of `len` rows (an
// empty one into `least`, 0 or 1), with the sequence's rows by `cu` and by `cu_b`
// (may be null).  Sequence s takes the places from cu[s] / len + s on: that is
// total / len + n_seq places at most, and never two sequences' (n rows have
// n / len + 1 tiles at most, divided as those are); the places between are
// empty.  So the whole warp finds a place's sequence by a search, one round trip
// for 32 sequences and two for 1024, where adding up the tiles before it (dense
// places) reads all borders before it: 4096 sequences of 16 tokens, 8 heads,
// d 64: 3860 against 1000 us for the softmax branch, 7490 against 1280 for the
// one with decays; 16 of 300 tokens: 26.6 and 24.6, 25.6 and 23.8 us.
// Borders that do not ascend mislead the search; every place checks the borders
// of its own number, so that they are always reported.
__device__ __forceinline__ SeqTile find_tile(const int32_t* __restrict__ cu, int n_seq, int total, const Divisor& len, int t,
                                             int* status, int least = 0, const int32_t* __restrict__ cu_b = nullptr,
                                             int total_b = 0) {
    SeqTile r{-1, 0, {0, 0}, {0, 0}};
    if (t < n_seq) {
        seq_range(cu, t, total, status);
        if (cu_b) seq_range(cu_b, t, total_b, status);
    }
    auto tile = [&](int s) { return t - s - border(cu, s, total) / len; };
    const int s = find_last(n_seq, tile);
    if (s < 0) return r;
    r.tile = tile(s);
    r.a = seq_range(cu, s, total, status);
    if (cu_b) r.b = seq_range(cu_b, s, total_b, status);
    if (r.tile < least || (long long)r.tile * len.n < r.a.len) r.seq = s;
    return r;
}

// Four lanes with four 16-byte units of a row each -> unit (lane & 3) of each
// of the four rows, so that their stores fill 64 bytes of a row together.
__device__ __forceinline__ void transpose_units(uint4 (&u)[4], int lane) {
    uint32_t* x = reinterpret_cast<uint32_t*>(u);
#pragma unroll
    for (int m = 2; m > 0; m >>= 1) {
        const bool up = lane & m;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i & m) continue;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                uint32_t &a = x[4 * i + e], &b = x[4 * (i + m) + e];
                const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? a : b, m);
                if (up) a = got;
                else b = got;
            }
        }
    }
}

// Where four lanes' rows start (elements), -1 for a row that is not stored; for
// a warp whose lanes hold one row each.
struct QuadRows {
    long long at[4];
    __device__ __forceinline__ QuadRows(long long own) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int e = 0; e < 4; ++e) at[e] = __shfl_sync(0xffffffffu, own, (lane & ~3) + e);
    }
};

// 32 columns of every lane's row, as bf16 or fp32, 64 bytes of a row at a time
// (a lane that stores 16 bytes of its own row touches 32 lines per warp; eight
// such warps keep the load/store unit busy for 4000 cycles).
__device__ __forceinline__ void store_rows(__nv_bfloat16* p, const QuadRows& rows, const float (&v)[32]) {
    const int lane = threadIdx.x & 31;
    uint4 u[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
        u[e] = make_uint4(pack_bf16x2(v[8 * e], v[8 * e + 1]), pack_bf16x2(v[8 * e + 2], v[8 * e + 3]),
                          pack_bf16x2(v[8 * e + 4], v[8 * e + 5]), pack_bf16x2(v[8 * e + 6], v[8 * e + 7]));
    transpose_units(u, lane);
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (rows.at[e] >= 0) *reinterpret_cast<uint4*>(p + rows.at[e] + (lane & 3) * 8) = u[e];
}
__device__ __forceinline__ void store_rows(float* p, const QuadRows& rows, const float (&v)[32]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int h = 0; h < 32; h += 16) {
        uint4 u[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            u[e] = make_uint4(__float_as_uint(v[h + 4 * e]), __float_as_uint(v[h + 4 * e + 1]), __float_as_uint(v[h + 4 * e + 2]),
                              __float_as_uint(v[h + 4 * e + 3]));
        transpose_units(u, lane);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (rows.at[e] >= 0) *reinterpret_cast<uint4*>(p + rows.at[e] + h + (lane & 3) * 4) = u[e];
    }
}

// 32 columns of every lane's row of fp32, read as store_rows writes them.
__device__ __forceinline__ void load_rows(const float* __restrict__ p, const QuadRows& rows, float (&v)[32]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int h = 0; h < 32; h += 16) {
        uint4 u[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            u[e] = rows.at[e] >= 0 ? __ldg(reinterpret_cast<const uint4*>(p + rows.at[e] + h + (lane & 3) * 4)) : make_uint4(0, 0, 0, 0);
        transpose_units(u, lane);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[h + 4 * e] = __uint_as_float(u[e].x); v[h + 4 * e + 1] = __uint_as_float(u[e].y);
            v[h + 4 * e + 2] = __uint_as_float(u[e].z); v[h + 4 * e + 3] = __uint_as_float(u[e].w);
        }
    }
}

// A CTA's queue of work: one warp finds what the CTA is to do and hands it to
// the other warps.  Where a CTA has an SM to itself it then takes over CTAs that
// have not started yet from the grid (cluster launch control): the latency of
// its start and end overlaps with the pieces around it, and the hardware's own
// queue still balances long and short ones (the next piece is asked for when
// the last loads of this one are on their way: one asked for earlier would wait
// here while another SM runs dry).  Two CTAs on an SM hide each other's latency
// instead.
// W is a plain struct with an int `seq`, -1 for the end.
//
// A warp may wait here for as long as a piece takes, so that these waits give
// up later than those within a piece.
constexpr unsigned long long kQueueWait = 16ull * VSA_WAIT_LIMIT_CYCLES;
template <typename W>
struct WorkQueue {
    uint4 answer;
    W slot[2];
    uint64_t full[2], empty[2], asked, ending;
};

template <typename W>
__device__ __forceinline__ void queue_init(WorkQueue<W>* q, int consumer_warps) {
    for (int x = 0; x < 2; ++x) { sm100::mbar_init(&q->full[x], 1); sm100::mbar_init(&q->empty[x], consumer_warps); }
    sm100::mbar_init(&q->asked, 1);
    sm100::mbar_init(&q->ending, 1);
}

// By one thread, once for each piece that was not the end: its last loads are
// on their way.
template <typename W>
__device__ __forceinline__ void queue_ending(WorkQueue<W>* q) {
    sm100::mbar_arrive(&q->ending);
}

// The producing warp's whole run; make(id) (whole warp) gives the work of CTA
// `id`, which is left out if its seq is below 0.  False: a wait gave up.
template <bool TAKE_OVER, typename W, typename F>
__device__ __forceinline__ bool queue_produce(WorkQueue<W>* q, const volatile int* abort, F make) {
    const int lane = threadIdx.x & 31;
    int k = 0;
    auto put = [&](const W& w) {
        if (k >= 2 && !__all_sync(0xffffffffu, sm100::mbar_wait_for(&q->empty[k & 1], (k / 2 - 1) & 1, abort, kQueueWait))) return false;
        if (lane == 0) {
            q->slot[k & 1] = w;
            sm100::mbar_arrive(&q->full[k & 1]);
        }
        __syncwarp();
        ++k;
        return true;
    };
    int id = blockIdx.x;
    for (int asked = 0; id >= 0; ++asked) {
        const W w = make(id);
        if (w.seq >= 0) {
            if (!put(w)) return false;
            if (TAKE_OVER && !__all_sync(0xffffffffu, sm100::mbar_wait_for(&q->ending, (k - 1) & 1, abort, kQueueWait))) return false;
        }
        if (!TAKE_OVER) break;
        if (lane == 0) {
            sm100::mbar_arrive_expect_tx(&q->asked, 16);
            sm100::try_cancel(&q->answer, &q->asked);
        }
        __syncwarp();
        // (not given up early: the answer has to arrive before the CTA leaves)
        if (!__all_sync(0xffffffffu, sm100::wait_noabort(&q->asked, asked & 1))) return false;
        id = sm100::cancelled_ctaid(&q->answer);
        __syncwarp();
        sm100::fence_proxy_async_smem();                 // read before the next answer is written
    }
    W end{};
    end.seq = -1;
    return put(end);
}

// Piece k of the queue (whole warp); false: a wait gave up.
template <typename W>
__device__ __forceinline__ bool queue_get(WorkQueue<W>* q, int k, const volatile int* abort, W& w) {
    if (!__all_sync(0xffffffffu, sm100::mbar_wait_for(&q->full[k & 1], (k / 2) & 1, abort, kQueueWait))) return false;
    w = q->slot[k & 1];
    __syncwarp();
    if ((threadIdx.x & 31) == 0) sm100::mbar_arrive(&q->empty[k & 1]);
    return true;
}

}  // namespace vsa
