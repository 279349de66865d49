// decay_attn.cu -- linear attention with a decay per head over packed
// sequences, chunked form and its gradient, on sm_100a (the causal counterpart
// of the linear branch, whose state sums over the whole grid: here token t
// only sees the tokens before it, and less of them the further back they lie).
//
// Per sequence and head, with lam = exp(log_decay) and an outer product per token:
//     S_t = lam S_(t-1) + k_t^T v_t,     o_t = scale q_t S_t.
// One general pass serves the forward and the three gradients:
//     out_i = sum_j lam^|i-j| (a_i.b_j) c_j    (j <= i, or j >= i walking
//             backwards in time)  + lam^(..) a_i X,   X the state before the
//             chunk, b^T c summed with its decays:
//     out: a, b, c = q, k, v;   dq: dout, v, k (the same state, transposed);
//     dv:  k, q, dout and dk: v, dout, q backwards in time (state: the
//          gradient of S, transposed for dk).
//
// Tokens go in chunks of 128.  A sequence is cut into segments, and these into
// parts (a rule on the sizes, see decay_shape); three launches compute
//   decay_state_kernel  each part's own contribution to the state at its
//                       border: (b w)^T c with w = lam^(tokens to the border),
//                       one GEMM with the tokens as its inner dimension;
//   decay_scan_kernel   the states at the borders, border after border;
//   decay_out_kernel    one CTA per segment and head walks its chunks with the
//                       state in registers: per chunk
//                         scores A B^T, times lam^|i-j|, as bf16 P;
//                         O1 = P C, O2 = A X, out = O1 + lam^(..) O2;
//                         U = (B w)^T C, X = lam^128 X + U.
// Sequences of one segment need the last launch alone.
//
// The state is fp32 throughout.  In the walk its update's weighted operand is
// split into bf16 hi + lo (2^-17 relative) and the state is rounded to bf16 as
// the operand of A X, as P is as the operand of P C (2^-8 relative at most, as
// much as the rounding of the output).  A final state that the caller asks for
// comes from the state and scan kernels, with three parts (2^-25) and sums of
// 8 chunks' steps at a time in registers: the tensor cores' own sums drop the
// bits below their accumulator's last one, always towards zero, which would add
// up over a long sequence.
//
// At d = 64 hi and lo are the two halves of one M = 128 operand of the walk's
// update: X's hi part belongs to TMEM lanes 0-63 and its lo part to lanes
// 64-127, and A X runs over both.
//
// Measured, forward of 23296 tokens (one sequence), 12 heads, d 128: state 38 us
// (138 MB read), scan 8, walk 63 (273 MB); backward: state 64, scan 8, walk 162
// (665 MB).  DRAM is half busy in all of them: the operands pass shared memory
// several times (loads, weighted copies written and read, products' operands),
// and that and the chain from one chunk's state to the next bound the walk.
#include <algorithm>
#include <cmath>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "packed.cuh"
#include "packed.h"
#include "sm100.cuh"

namespace vsa {
using namespace sm100;

// One scan over the sequences: a kind of output.
struct DecayPass {
    CUtensorMap a, b, c;
    __nv_bfloat16* out;
    long long out_stride;
    const float* first;          // [n_seq][heads][d][d]: the state the walk starts with, or null (zeros)
    const float* border;         // [slots][heads][d][d]: the states between segments
    int back;                    // walk backwards in time
    int trans;                   // the states in memory are c^T b
    float w_scale, p_scale, s_scale;   // factors of b^T c in the state, of P, and of A X
};

struct DecayPasses {
    DecayPass p[3];
};

struct DecayShape {
    int n_seq, total, heads;
    Divisor seg, part;           // tokens of a segment and of a part of it (multiples of 128)
    Divisor n_heads;
    int per;                     // parts of a segment
};

// log2(lam); below 2^-1024 a decay is a plain 0 (and lam^0 stays 1)
__device__ __forceinline__ float decay_log2(const float* __restrict__ log_decay, int head) {
    const float x = __ldg(log_decay + head) * 1.4426950408889634f;
    return x < -1024.f ? -1024.f : x;
}

// A piece (segment or part) of a sequence.  The border behind a part that is
// not the sequence's last has its place in the scratch at (the part's first
// row) / part: these parts are full, so no two start within one multiple.
struct Piece {
    int seq, begin, len;         // first row and rows
    int off, rest;               // tokens of the sequence before it and from its first on
};

__device__ __forceinline__ Piece find_piece(const int32_t* __restrict__ cu, const DecayShape& s, const Divisor& len, int t, int* status) {
    Piece g{-1, 0, 0, 0, 0};
    const SeqTile at = find_tile(cu, s.n_seq, s.total, len, t, status, 1);
    if (at.seq < 0) return g;
    const SeqRange r = at.a;
    g.seq = at.seq;
    g.off = at.tile * len.n;
    g.rest = r.len - g.off;
    g.begin = r.begin + g.off;
    g.len = min(len.n, g.rest);
    return g;
}

// The sequence that has the last of the rows len j .. len j + len - 1 (whole
// warp; -1 if none).  Whatever piece of len rows starts among them has that row.
__device__ __forceinline__ int find_row(const int32_t* __restrict__ cu, const DecayShape& s, int len, int j, SeqRange& r, int* status) {
    const int row = len * j + len - 1;
    const int seq = find_last(s.n_seq, [&](int i) { return row - border(cu, i, s.total); });
    if (seq < 0) return -1;
    r = seq_range(cu, seq, s.total, status);
    return row - r.begin < r.len ? seq : -1;
}

// The part before border j (or behind it) of a sequence that has one there.
__device__ __forceinline__ Piece find_border(const int32_t* __restrict__ cu, const DecayShape& s, int j, bool behind, int* status) {
    Piece g{-1, 0, 0, 0, 0};
    SeqRange r;
    const int seq = find_row(cu, s, s.part.n, j, r, status);
    if (seq < 0) return g;
    const int off = (s.part.n * j + s.part.n - 1 - r.begin) / s.part * s.part.n;
    if (off + s.part.n >= r.len) return g;               // no border: the sequence ends first
    g.seq = seq;
    g.off = behind ? off + s.part.n : off;
    g.rest = r.len - g.off;
    g.begin = r.begin + g.off;
    g.len = min(s.part.n, g.rest);
    return g;
}

// bf16 pairs x times w as hi + lo.
__device__ __forceinline__ void split_pair(uint32_t x, float w, uint32_t& hi, uint32_t& lo) {
    const uint64_t p = mul_f32x2(f32x2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u)), f32x2(w, w));
    float x0, x1;
    unf32x2(p, x0, x1);
    hi = pack_bf16x2(x0, x1);
    // p - hi, exactly
    unf32x2(fma_f32x2(f32x2(__uint_as_float(hi << 16), __uint_as_float(hi & 0xffff0000u)), f32x2(-1.f, -1.f), p), x0, x1);
    lo = pack_bf16x2(x0, x1);
}

// ... as hi + mid + lo.
__device__ __forceinline__ void split_pair3(uint32_t x, float w, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
    const uint64_t p = mul_f32x2(f32x2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u)), f32x2(w, w));
    const uint64_t neg = f32x2(-1.f, -1.f);
    float x0, x1;
    unf32x2(p, x0, x1);
    hi = pack_bf16x2(x0, x1);
    // what hi leaves, exactly
    const uint64_t r = fma_f32x2(f32x2(__uint_as_float(hi << 16), __uint_as_float(hi & 0xffff0000u)), neg, p);
    unf32x2(r, x0, x1);
    mid = pack_bf16x2(x0, x1);
    unf32x2(fma_f32x2(f32x2(__uint_as_float(mid << 16), __uint_as_float(mid & 0xffff0000u)), neg, r), x0, x1);
    lo = pack_bf16x2(x0, x1);
}

__device__ __forceinline__ void split8(uint4& x, float w, uint4& mid, uint4& lo) {
    split_pair3(x.x, w, x.x, mid.x, lo.x);
    split_pair3(x.y, w, x.y, mid.y, lo.y);
    split_pair3(x.z, w, x.z, mid.z, lo.z);
    split_pair3(x.w, w, x.w, mid.w, lo.w);
}

__device__ __forceinline__ void split8(uint4& x, float w, uint4& lo) {
    split_pair(x.x, w, x.x, lo.x);
    split_pair(x.y, w, x.y, lo.y);
    split_pair(x.z, w, x.z, lo.z);
    split_pair(x.w, w, x.w, lo.w);
}

// ---------------------------------------------------------------- border sums
template <int D>
struct DecStateCfg {
    static constexpr int NCH = D / 64;
    static constexpr int CHUNK = 64 * 128;               // 64 tokens of one 64-feature chunk
    static constexpr int TILE = NCH * CHUNK;
    static constexpr int NST = D == 128 ? 5 : 8;         // stages of b (hi in its place) and c
    static constexpr int ZERO_OFF = NST * 2 * TILE;      // d = 64: a tile of zeros
    static constexpr int LO_OFF = ZERO_OFF + (D == 64 ? TILE : 0);   // mid and lo of even and odd steps
    static constexpr int BAR_OFF = LO_OFF + 4 * TILE;
    static constexpr int SMEM = BAR_OFF + 512;
    static constexpr int GROUP = 8;                      // steps that one TMEM accumulator sums
    static constexpr int THREADS = 512;                  // warpgroups: 2 split, sums, loads and MMAs and queue; 128 registers a thread
    static constexpr int REG_SPLIT = 104, REG_SUM = 208, REG_LOAD = 96;      // 2 * 104 + 208 + 96 = 4 * 128
};
static_assert(DecStateCfg<128>::SMEM <= 232448, "shared memory");

struct DecayPart {
    int seq, head, kind;
    int begin, len;
    int ends;                    // the walk's last part
    bool alone;                  // the sequence is this part
};

template <int D>
struct DecStateBars {
    WorkQueue<DecayPart> queue;
    uint64_t full[DecStateCfg<D>::NST], done[DecStateCfg<D>::NST];
    uint64_t ready[2], sum_full[2], sum_free[2], half_full, half_free;
    uint32_t tmem_base;
    int abort;
};
static_assert(sizeof(DecStateBars<64>) <= 512, "barrier block");

struct DecayStateArgs {
    CUtensorMap b[2], c[2];
    float* border[2];
    float* last[2];              // [n_seq][heads][d][d]: the walk's last part, for the scan to finish (of a sequence of one
                                 // part: the state after it); or null
    const float* first[2];       // the states the walks start with, or null (zeros)
    int back[2];
    float w_scale[2];
    int ends;                    // some `last` is wanted
};

// grid (kinds of state x parts x heads), from a queue per CTA.  Forward in time
// the sum of part p goes to the border behind it, backwards that of part p + 1;
// the walk's last part's to `last`, and without that the parts of its last
// segment are not needed, and the places are the borders' (total / part, however
// many sequences are too short to have one).  Steps of 64 tokens are counted on from part to part.
//
// Where states leave the library (`last`) the sums are good to fp32: the
// weighted operand is split into three bf16 parts (all 24 bits) instead of two,
// and the products of the small ones have an accumulator of their own.  The
// tensor cores' accumulation cuts off (a sum over 88 products of 16 tokens came
// out 1.4e-6 off), so that one accumulator sums 8 steps and fp32 registers sum
// those, one of two accumulators being read while the other is filled.
template <int D>
__global__ void __launch_bounds__(DecStateCfg<D>::THREADS, 1)
decay_state_kernel(const __grid_constant__ DecayStateArgs args, const Divisor kinds, const DecayShape sh,
                   const int32_t* __restrict__ cu, const float* __restrict__ log_decay, int* status) {
    using C = DecStateCfg<D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    if (smem_u32(smem) & 1023) {
        if (threadIdx.x == 0) report(status, kStatusMisaligned);
        return;
    }
    const int tid = threadIdx.x, warp = warp_uniform(tid >> 5), lane = tid & 31;
    DecStateBars<D>* bars = reinterpret_cast<DecStateBars<D>*>(smem + C::BAR_OFF);
    volatile int* abort_flag = &bars->abort;
    if (tid == 0) {
        bars->abort = 0;
        queue_init(&bars->queue, 14);
        for (int x = 0; x < C::NST; ++x) { mbar_init(&bars->full[x], 1); mbar_init(&bars->done[x], 1); }
        for (int x = 0; x < 2; ++x) mbar_init(&bars->ready[x], 256);
        for (int x = 0; x < 2; ++x) { mbar_init(&bars->sum_full[x], 1); mbar_init(&bars->sum_free[x], 128); }
        mbar_init(&bars->half_full, 64);
        mbar_init(&bars->half_free, 64);
        fence_barrier_init();
    }
    if (warp == 13) { tmem_alloc(&bars->tmem_base, 512); tmem_relinquish(); }
    if (D == 64) {
        for (int u = tid; u < C::TILE / 16; u += C::THREADS) *reinterpret_cast<uint4*>(smem + C::ZERO_OFF + u * 16) = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = warp_uniform(bars->tmem_base);
    auto fail = [&]() { *abort_flag = 1; report(status, kStatusTimeout); };
    auto full_wait = [&](int t) { return mbar_wait(&bars->full[t % C::NST], (t / C::NST) & 1, abort_flag); };
    auto done_wait = [&](int t) { return mbar_wait(&bars->done[t % C::NST], (t / C::NST) & 1, abort_flag); };
    auto steps = [](const DecayPart& w) { return (w.len + 63) / 64; };
    // against the direction of decay_out_kernel's walk: what that reads first
    // is what this one read last, and still in L2
    auto token = [&](const DecayPart& w, int t) { return 64 * (args.back[w.kind] ? t : (w.len + 63) / 64 - 1 - t); };

    if (warp >= 12) {
      reg_dec<C::REG_LOAD>();
      if (warp == 14) {
        const bool ok = queue_produce<true>(&bars->queue, abort_flag, [&](int id) {
            DecayPart w{};
            w.kind = id % kinds;
            id = id / kinds;
            w.head = id % sh.n_heads;
            id = id / sh.n_heads;
            const bool back = args.back[w.kind];
            const Piece g = args.ends ? find_piece(cu, sh, sh.part, id, status) : find_border(cu, sh, id, back, status);
            const bool needed = args.last[w.kind] ? true : back ? g.off >= sh.seg.n : g.rest > sh.seg.n - g.off % sh.seg;
            w.seq = needed ? g.seq : -1;
            w.begin = g.begin; w.len = g.len;
            w.alone = g.off == 0 && g.rest <= sh.part.n;
            w.ends = back ? g.off == 0 : g.rest <= sh.part.n;
            return w;
        });
        if (!ok) fail();
      } else if (warp == 12) {
        // -------------------------------------------------------------- loads
        int s0 = 0, issued = 0;
        bool ok = true;
        for (int k = 0; ok; ++k) {
            DecayPart w;
            if (!(ok = queue_get(&bars->queue, k, abort_flag, w)) || w.seq < 0) break;
            const int n = steps(w);
            if (lane == 0) {
                for (int t = 0; t < n; ++t) {
                    const int st = (s0 + t) % C::NST, row = w.begin + token(w, t);
                    if (s0 + t >= C::NST && !(ok = done_wait(s0 + t - C::NST))) break;
                    uint8_t* p = smem + st * 2 * C::TILE;
                    mbar_arrive_expect_tx(&bars->full[st], 2 * C::TILE);
                    for (int c = 0; c < C::NCH; ++c) {
                        tma_load_3d(p + c * C::CHUNK, &args.b[w.kind], &bars->full[st], 64 * c, w.head, row);
                        tma_load_3d(p + C::TILE + c * C::CHUNK, &args.c[w.kind], &bars->full[st], 64 * c, w.head, row);
                    }
                    ++issued;
                }
                queue_ending(&bars->queue);
            }
            __syncwarp();
            ok = __all_sync(0xffffffffu, ok);
            s0 += n;
        }
        if (!ok) fail();
        if (lane == 0 && *abort_flag)                    // every load must land before the shared memory is given up
            for (int i = max(0, issued - C::NST); i < issued; ++i) wait_noabort(&bars->full[i % C::NST], (i / C::NST) & 1);
      } else if (warp == 13) {
        // --------------------------------------------------------------- MMAs
        constexpr uint32_t id_x = idesc_bf16_f32(128, D, true, true);
        const uint32_t base = smem_u32(smem);
        const uint64_t mn_major = smem_desc_sw128(base, C::CHUNK, 1024);
        auto wait = [&](uint64_t* bar, int parity) { return __all_sync(0xffffffffu, mma_wait(bar, parity, abort_flag)) != 0; };
        int s0 = 0, group = -1, last_step = -1;
        bool ok = true;
        for (int k = 0; ok; ++k) {
            DecayPart w;
            if (!(ok = queue_get(&bars->queue, k, abort_flag, w)) || w.seq < 0) break;
            const int n = warp_uniform(steps(w));
            const bool three = args.last[warp_uniform(w.kind)] != nullptr;
            for (int t = 0; t < n; ++t) {
                const bool fresh = t % C::GROUP == 0;
                if (fresh && ++group >= 2 && !(ok = wait(&bars->sum_free[group & 1], (group / 2 - 1) & 1))) break;
                const uint32_t acc = tbase + 128 * (group & 1);
                const int step = s0 + t, at = (step % C::NST) * 2 * C::TILE, mid_at = C::LO_OFF + (step & 1) * 2 * C::TILE;
                const int lo_at = mid_at + C::TILE;
                const uint64_t c = desc_add(mn_major, at + C::TILE);
                // d = 64: hi and mid, and zeros and lo, are the two 64-feature chunks of one operand
                const uint64_t hi = D == 128 ? desc_add(mn_major, at) : smem_desc_sw128(base + at, mid_at - at, 1024);
                const uint64_t mid = desc_add(mn_major, mid_at);
                const uint64_t lo = D == 128 ? desc_add(mn_major, lo_at) : smem_desc_sw128(base + C::ZERO_OFF, lo_at - C::ZERO_OFF, 1024);
                if (!(ok = wait(&bars->ready[step & 1], (step >> 1) & 1))) break;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {     // 16 tokens per MMA
                        const uint64_t cd = desc_add(c, kk * 2048);
                        mma_bf16_ss(acc, desc_add(hi, kk * 2048), cd, id_x, !fresh || kk > 0);
                        if (D == 128) mma_bf16_ss(acc + 256, desc_add(mid, kk * 2048), cd, id_x, !fresh || kk > 0);
                        if (three) mma_bf16_ss(D == 128 ? acc + 256 : acc, desc_add(lo, kk * 2048), cd, id_x, 1);
                    }
                    mma_commit(&bars->done[step % C::NST]);
                    if (t == n - 1 || t % C::GROUP == C::GROUP - 1) mma_commit(&bars->sum_full[group & 1]);
                }
                __syncwarp();
                last_step = step;
            }
            s0 += n;
        }
        if (!ok) fail();
        // products in flight have to finish before the CTA leaves
        if (last_step >= 0) wait_noabort(&bars->done[last_step % C::NST], (last_step / C::NST) & 1);
      }
    } else if (warp < 8) {
        reg_dec<C::REG_SPLIT>();
        // -------------------------------------------------------------- split
        int s0 = 0;
        bool ok = true;
        for (int k = 0; ok; ++k) {
            DecayPart w;
            if (!(ok = queue_get(&bars->queue, k, abort_flag, w)) || w.seq < 0) break;
            const float l2 = decay_log2(log_decay, w.head), w0 = args.w_scale[w.kind];
            const bool back = args.back[w.kind], three = args.last[w.kind] != nullptr;
            const int n = steps(w);
            for (int t = 0; t < n; ++t) {
                const int step = s0 + t, tok = token(w, t);
                // mid's and lo's place is free with the products of two steps before
                if (!__all_sync(0xffffffffu, full_wait(step) && (step < 2 || done_wait(step - 2)))) { ok = false; break; }
                uint8_t* st = smem + (step % C::NST) * 2 * C::TILE;
                uint8_t* sl = smem + C::LO_OFF + (step & 1) * 2 * C::TILE;
#pragma unroll
                for (int u = tid; u < C::TILE / 16; u += 256) {
                    const int r = tok + (u & 511) / 8;   // token of the part
                    uint4 x = *reinterpret_cast<const uint4*>(st + u * 16), mid, lo;
                    const float wr = w0 * ex2((float)(back ? r + 1 : w.len - 1 - r) * l2);
                    if (three) split8(x, wr, mid, lo);
                    else split8(x, wr, mid);
                    if (r >= w.len) {                    // another sequence's rows
                        x = mid = lo = make_uint4(0, 0, 0, 0);
                        *reinterpret_cast<uint4*>(st + C::TILE + u * 16) = x;
                    }
                    *reinterpret_cast<uint4*>(st + u * 16) = x;
                    *reinterpret_cast<uint4*>(sl + u * 16) = mid;
                    if (three) *reinterpret_cast<uint4*>(sl + C::TILE + u * 16) = lo;
                }
                fence_proxy_async_smem();
                mbar_arrive(&bars->ready[step & 1]);
            }
            s0 += n;
        }
        if (!ok) fail();
    } else {
        reg_inc<C::REG_SUM>();
        // --------------------------------------------------------------- sums
        // a TMEM lane per thread: a feature of b (d = 64: of hi, and of mid and
        // lo, whose sums meet in shared memory)
        const int row = 32 * (warp & 3) + lane, feat = row & (D - 1);
        __shared__ float half[D == 64 ? 32 * 64 : 1];
        int group = 0, exchanges = 0;
        bool ok = true;
        for (int k = 0; ok; ++k) {
            DecayPart w;
            if (!(ok = queue_get(&bars->queue, k, abort_flag, w)) || w.seq < 0) break;
            float x[D];
#pragma unroll
            for (int c = 0; c < D; ++c) x[c] = 0.f;
            const int n = steps(w);
            for (int t = 0; t < n; t += C::GROUP, ++group) {
                if (!(ok = __all_sync(0xffffffffu, mbar_wait(&bars->sum_full[group & 1], (group / 2) & 1, abort_flag)))) break;
                tc_fence_after();
                const uint32_t acc = tbase + 128 * (group & 1) + ((uint32_t)(32 * (warp & 3)) << 16);
#pragma unroll
                for (int c = 0; c < D; c += 32) {
                    float y[32];
                    tmem_ld_32x32b_x32(acc + c, y);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; ++e) x[c + e] += y[e];
                    if (D == 128) {
                        tmem_ld_32x32b_x32(acc + 256 + c, y);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) x[c + e] += y[e];
                    }
                }
                tc_fence_before();
                mbar_arrive(&bars->sum_free[group & 1]);
            }
            if (!ok) break;
            const long long slot = (args.back[w.kind] ? w.begin - sh.part.n : w.begin) / sh.part;
            float* dst = w.ends ? args.last[w.kind] + ((long long)w.seq * sh.heads + w.head) * D * D
                                : args.border[w.kind] + (slot * sh.heads + w.head) * D * D;
            const QuadRows at((long long)feat * D);
            const float* const first = w.ends && w.alone && args.first[w.kind] ? args.first[w.kind] + ((long long)w.seq * sh.heads + w.head) * D * D : nullptr;
            const float f_first = ex2((float)w.len * decay_log2(log_decay, w.head));
#pragma unroll
            for (int c = 0; c < D; c += 32) {
                float(&v)[32] = *reinterpret_cast<float(*)[32]>(&x[c]);
                if (D == 64) {
                    if (!ok) break;
                    if (row >= 64) {
                        if (exchanges > 0 && !(ok = __all_sync(0xffffffffu, mbar_wait(&bars->half_free, (exchanges - 1) & 1, abort_flag)))) break;
#pragma unroll
                        for (int e = 0; e < 32; ++e) half[e * 64 + feat] = v[e];
                        mbar_arrive(&bars->half_full);
                    } else {
                        if (!(ok = __all_sync(0xffffffffu, mbar_wait(&bars->half_full, exchanges & 1, abort_flag)))) break;
#pragma unroll
                        for (int e = 0; e < 32; ++e) v[e] += half[e * 64 + feat];
                        mbar_arrive(&bars->half_free);
                    }
                    ++exchanges;
                }
                if (row >= D) continue;                  // (whole warps)
                if (first) {
                    float y[32];
                    load_rows(first + c, at, y);
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = fmaf(f_first, y[e], v[e]);
                }
                store_rows(dst + c, at, v);
            }
        }
        if (!ok) fail();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 13) tmem_dealloc(tbase, 512);
}

struct DecayScanArgs {
    float* border[2];
    const float* first[2];
    float* last[2];              // or null
    int back[2];
};

// Border sums -> states at the borders, in place, and the last part's sum in
// `last` -> the state that the walk ends with.  grid (sequences x heads,
// D^2 / 1024, kinds of state), 4 elements per thread.  Sequences without a border
// (of one segment; where `last` is wanted, of one part) have nothing to do here;
// where there are more sequences than total / that length, the grid has so many
// places instead, and a sequence that is longer has the one where it starts.
template <int D>
__global__ void __launch_bounds__(256)
decay_scan_kernel(const __grid_constant__ DecayScanArgs args, const int by_seq, const Divisor longer, const DecayShape sh, const int32_t* __restrict__ cu,
                  const float* __restrict__ log_decay, int* status) {
    grid_dependents_launch();                            // decay_out_kernel may start: it waits for the borders itself
    const int id = blockIdx.x, head = id % sh.n_heads, kind = blockIdx.z;
    int seq = id / sh.n_heads;
    SeqRange r{0, 0};
    if (by_seq) {
        r = seq_range(cu, seq, sh.total, status);
    } else {
        const int j = seq;
        seq = find_row(cu, sh, longer.n, j, r, status);
        if (seq < 0 || r.begin / longer != j) r.len = 0;
    }
    const int per = sh.per, parts = (r.len + sh.part.n - 1) / sh.part, full_segs = max(0, r.len - 1) / sh.seg;
    const int slot0 = r.begin / sh.part;
    grid_dependency_wait();                              // (by every CTA: so decay_out_kernel's wait covers the sums' launch too)
    float* last = args.last[kind];
    if (r.len <= (last ? sh.part.n : sh.seg.n)) return;
    const int back = args.back[kind];
    // border b lies behind part b; without `last`, forward those up to the last
    // segment's, backwards from the last one down to the first segment's
    const int n = last ? parts - 1 : back ? parts - per : full_segs * per, b0 = back ? parts - 2 : 0;
    const int e = (blockIdx.y * 256 + threadIdx.x) * 4;
    const float l2 = decay_log2(log_decay, head);
    const float full = ex2((float)sh.part.n * l2);
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (args.first[kind]) s = __ldg(reinterpret_cast<const float4*>(args.first[kind] + ((long long)seq * sh.heads + head) * D * D + e));
    const int tail = r.len - (parts - 1) * sh.part.n;      // tokens of the last part
    const long long step = (long long)sh.heads * D * D;
    float* base = args.border[kind] + slot0 * step + (long long)head * D * D + e;   // border 0
    constexpr int AHEAD = 12;
    for (int i0 = 0; i0 < n; i0 += AHEAD) {
        float4 u[AHEAD];
#pragma unroll
        for (int j = 0; j < AHEAD; ++j)
            if (i0 + j < n) u[j] = __ldcg(reinterpret_cast<const float4*>(base + (back ? b0 - i0 - j : i0 + j) * step));
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
            if (i0 + j >= n) break;
            const float f = back && i0 + j == 0 ? ex2((float)tail * l2) : full;
            s.x = fmaf(f, s.x, u[j].x); s.y = fmaf(f, s.y, u[j].y); s.z = fmaf(f, s.z, u[j].z); s.w = fmaf(f, s.w, u[j].w);
            *reinterpret_cast<float4*>(base + (back ? b0 - i0 - j : i0 + j) * step) = s;
        }
    }
    if (last) {
        float4* p = reinterpret_cast<float4*>(last + ((long long)seq * sh.heads + head) * D * D + e);
        // the walk's last part: forward the sequence's last, backwards its first, a full one
        const float f = back ? full : ex2((float)tail * l2);
        const float4 u = __ldcg(p);
        s.x = fmaf(f, s.x, u.x); s.y = fmaf(f, s.y, u.y); s.z = fmaf(f, s.z, u.z); s.w = fmaf(f, s.w, u.w);
        *p = s;
    }
}

// --------------------------------------------------------------------- outputs
template <int D>
struct DecOutCfg {
    static constexpr int NCH = D / 64;
    static constexpr int CHUNK = 128 * 128;              // 128 tokens of one 64-feature chunk
    static constexpr int TILE = NCH * CHUNK;
    static constexpr int NB = D == 128 ? 2 : 3;          // slots of the ring of B tiles
    static constexpr int NAC = D == 128 ? 3 : 6;         // of the ring of A and C tiles, in turn
    static constexpr int AC_OFF = NB * TILE;
    static constexpr int LO_OFF = (NB + NAC) * TILE;     // lo part of the weighted operand (hi in its tile's place)
    static constexpr int X_OFF = LO_OFF + TILE;          // the state as bf16: 128 rows (d = 64: hi rows, lo rows) x D
    static constexpr int UNITS = 4 * NCH;                // 16-byte units of the weighted operand per thread pair,
    static constexpr int UNITS_P = D == 128 ? 5 : 2;     // of which the score warps split so many
    static constexpr int POW_OFF = X_OFF + TILE;         // powers of lam, see the weights: 64 floats, and again one float on; of two walks
    static constexpr int POW_FLOATS = 132;
    static constexpr int BAR_OFF = POW_OFF + 2 * POW_FLOATS * 4;
    static constexpr int SMEM = BAR_OFF + 512;
    static constexpr int THREADS = 768;                  // warpgroups: 2 scores, 2 state, outputs, loads and MMAs; 80 registers a thread
    static constexpr int REG_SCORE = 72, REG_STATE = 104, REG_OUT = 80, REG_LOAD = 48;   // 2 * 72 + 2 * 104 + 80 + 48 = 6 * 80
    // TMEM; at d = 64 the scores have two places, so that those of the next step
    // are formed before the weights of this one are used up
    static constexpr int NS = D == 128 ? 1 : 2;
    static constexpr int U_COL = 0, S_COL = D == 128 ? 128 : 64, O1_COL = D == 128 ? 256 : 320, O2_COL = 384;
};
static_assert(DecOutCfg<128>::SMEM <= 232448 && DecOutCfg<64>::SMEM <= 232448, "shared memory");

// What decay_out_kernel walks: one segment of one head for one pass.
struct DecayWork {
    int seq, pass, head;
    int begin, len;              // first row and rows
    int off, rest;               // tokens of the sequence before it and from its first on
};

template <int D>
struct DecOutBars {
    WorkQueue<DecayWork> queue;
    uint64_t b_full[DecOutCfg<D>::NB], ac_full[DecOutCfg<D>::NAC];
    uint64_t u_done[DecOutCfg<D>::NB];   // every product of a step in this slot of B
    uint64_t s_full[2], p_ready[2], x_ready, w_ready, o_full, o_free, mma_done;
    uint64_t pow_ready[2];               // of even and odd walks, as the tables
    uint32_t tmem_base;
    int abort;
};
static_assert(sizeof(DecOutBars<64>) <= 512 && sizeof(DecOutBars<128>) <= 512, "barrier block");

// grid (passes x segments x heads: the passes over one segment run side by
// side and share its tiles in L2).  Every role takes walk after walk from the
// CTA's queue; steps (chunks), items and phases are counted on from walk to walk.
template <int D>
__global__ void __launch_bounds__(DecOutCfg<D>::THREADS, 1)
decay_out_kernel(const __grid_constant__ DecayPasses passes, const Divisor n_passes, const DecayShape sh,
                 const int32_t* __restrict__ cu, const float* __restrict__ log_decay, int* status) {
    using C = DecOutCfg<D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    if (smem_u32(smem) & 1023) {
        if (threadIdx.x == 0) report(status, kStatusMisaligned);
        return;
    }
    const int tid = threadIdx.x, warp = warp_uniform(tid >> 5), lane = tid & 31;
    uint8_t* sLo = smem + C::LO_OFF;
    uint8_t* sX = smem + C::X_OFF;
    DecOutBars<D>* bars = reinterpret_cast<DecOutBars<D>*>(smem + C::BAR_OFF);
    volatile int* abort_flag = &bars->abort;
    if (tid == 0) {
        bars->abort = 0;
        queue_init(&bars->queue, 22);
        for (int x = 0; x < C::NB; ++x) { mbar_init(&bars->b_full[x], 1); mbar_init(&bars->u_done[x], 1); }
        for (int x = 0; x < C::NAC; ++x) mbar_init(&bars->ac_full[x], 1);
        for (int x = 0; x < 2; ++x) mbar_init(&bars->s_full[x], 1);
        for (int x = 0; x < 2; ++x) mbar_init(&bars->p_ready[x], 256);
        mbar_init(&bars->x_ready, 256);
        mbar_init(&bars->w_ready, 512);
        mbar_init(&bars->o_full, 1);
        mbar_init(&bars->o_free, 128);
        mbar_init(&bars->mma_done, 1);
        for (int x = 0; x < 2; ++x) mbar_init(&bars->pow_ready[x], 64);
        fence_barrier_init();
    }
    if (warp == 21) { tmem_alloc(&bars->tmem_base, 512); tmem_relinquish(); }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = warp_uniform(bars->tmem_base);
    auto fail = [&]() { *abort_flag = 1; report(status, kStatusTimeout); };
    // B of step t, and item i of the A and C tiles (A of step t at 2 t, C at 2 t + 1)
    auto b_slot = [&](int t) { return (t % C::NB) * C::TILE; };
    auto b_wait = [&](int t) { return mma_wait(&bars->b_full[t % C::NB], (t / C::NB) & 1, abort_flag); };
    auto ac_slot = [&](int i) { return C::AC_OFF + (i % C::NAC) * C::TILE; };
    auto ac_wait = [&](int i) { return mma_wait(&bars->ac_full[i % C::NAC], (i / C::NAC) & 1, abort_flag); };
    auto u_wait = [&](int t) { return mbar_wait(&bars->u_done[t % C::NB], (t / C::NB) & 1, abort_flag); };
    auto s_wait = [&](int t) { return mbar_wait(&bars->s_full[t % C::NS], (t / C::NS) & 1, abort_flag); };
    // the walk's chunks: step t is chunk t, or chunks - 1 - t backwards; the
    // state is updated after each but the last
    auto chunks = [](const DecayWork& w) { return (w.len + 127) / 128; };
    auto token = [](const DecayWork& w, bool back, int t) { return 128 * (back ? (w.len + 127) / 128 - 1 - t : t); };

    // hi and lo of B w for the units [i0, i1) of this one of 256 threads
    auto split_units = [&](int t, int id, int i0, int i1, int rows, bool back, float w_scale, float l2) {
        if (!__all_sync(0xffffffffu, b_wait(t))) return false;     // (long done: the scores are)
        uint8_t* b = smem + b_slot(t);
#pragma unroll
        for (int i = i0; i < i1; ++i) {
            const int r = id / 8 + 32 * (i & 3);         // token of the chunk
            uint4 y = *reinterpret_cast<const uint4*>(b + id * 16 + 4096 * i), lo;
            split8(y, w_scale * ex2((float)(back ? r + 1 : rows - 1 - r) * l2), lo);
            if (r >= rows) y = lo = make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4*>(b + id * 16 + 4096 * i) = y;
            *reinterpret_cast<uint4*>(sLo + id * 16 + 4096 * i) = lo;
        }
        fence_proxy_async_smem();
        mbar_arrive(&bars->w_ready);
        return true;
    };

    if (warp >= 20) {
      reg_dec<C::REG_LOAD>();
      if (warp == 22) {
        const bool ok = queue_produce<true>(&bars->queue, abort_flag, [&](int id) {
            DecayWork w{};
            w.pass = id % n_passes;
            id = id / n_passes;
            w.head = id % sh.n_heads;
            const Piece g = find_piece(cu, sh, sh.seg, id / sh.n_heads, status);
            w.seq = g.len > 0 ? g.seq : -1;
            w.begin = g.begin; w.len = g.len; w.off = g.off; w.rest = g.rest;
            return w;
        });
        if (!ok) fail();
      } else if (warp == 20) {
        // -------------------------------------------------------------- loads
        // When step t - NB has finished, so has what was in the slots of B and
        // A (d = 64: and C) of step t; at d = 128 C takes the slot of A of
        // step t - 1, free with that step's outputs.
        static_assert(D == 128 ? C::NB == 2 && C::NAC == 3 : C::NAC == 2 * C::NB, "which products free a slot");
        int s0 = 0, nb = 0, nac = 0;
        bool ok = true;
        for (int k = 0; ok; ++k) {
            DecayWork w;
            if (!(ok = queue_get(&bars->queue, k, abort_flag, w)) || w.seq < 0) break;
            const DecayPass& ps = passes.p[w.pass];
            const int n = chunks(w);
            if (lane == 0) {
                auto load = [&](int dst, const CUtensorMap* map, uint64_t* full, int t) {
                    const int row = w.begin + token(w, ps.back, t);
                    mbar_arrive_expect_tx(full, C::TILE);
                    for (int c = 0; c < C::NCH; ++c) tma_load_3d(smem + dst + c * C::CHUNK, map, full, 64 * c, w.head, row);
                };
                auto load_ac = [&](const CUtensorMap* map, int t) {
                    load(ac_slot(nac), map, &bars->ac_full[nac % C::NAC], t);
                    ++nac;
                };
                for (int t = 0; t < n; ++t) {
                    const int step = s0 + t;
                    if (step >= C::NB && !(ok = u_wait(step - C::NB))) break;
                    load(b_slot(step), &ps.b, &bars->b_full[step % C::NB], t);
                    ++nb;
                    load_ac(&ps.a, t);
                    if (D == 128 && step > 0 && !(ok = mbar_wait(&bars->o_full, (step - 1) & 1, abort_flag))) break;
                    load_ac(&ps.c, t);
                }
                queue_ending(&bars->queue);
            }
            __syncwarp();
            ok = __all_sync(0xffffffffu, ok);
            s0 += n;
        }
        if (!ok) fail();
        if (lane == 0 && *abort_flag) {
            // drain: every load must land before the CTA's shared memory is given up
            for (int i = max(0, nb - C::NB); i < nb; ++i) wait_noabort(&bars->b_full[i % C::NB], (i / C::NB) & 1);
            for (int i = max(0, nac - C::NAC); i < nac; ++i) wait_noabort(&bars->ac_full[i % C::NAC], (i / C::NAC) & 1);
        }
      } else if (warp == 21) {
        // --------------------------------------------------------------- MMAs
        // (the whole warp walks the loop, so that every branch and value is
        // uniform; one elected lane issues)
        constexpr uint32_t id_s = idesc_bf16_f32(128, 128, false, false);
        constexpr uint32_t id_o = idesc_bf16_f32(128, D, false, true);
        constexpr uint32_t id_x = idesc_bf16_f32(128, D, true, true);
        const uint32_t base = smem_u32(smem);
        const uint64_t k_major = smem_desc_sw128(base, 16, 1024), mn_major = smem_desc_sw128(base, C::CHUNK, 1024);
        auto all = [](bool x) { return __all_sync(0xffffffffu, x) != 0; };
        auto issue_s = [&](int t) {
            const uint64_t b = desc_add(k_major, b_slot(t)), a = desc_add(k_major, ac_slot(2 * t));
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t o = (kk >> 2) * C::CHUNK + (kk & 3) * 32;
                    mma_bf16_ss(tbase + C::S_COL + 128 * (t % C::NS), desc_add(a, o), desc_add(b, o), id_s, kk > 0);
                }
                mma_commit(&bars->s_full[t % C::NS]);
            }
            __syncwarp();
        };
        int s0 = 0, w0 = 0;
        bool ok = true;
        for (int k = 0; ok; ++k) {
            DecayWork w;
            if (!(ok = queue_get(&bars->queue, k, abort_flag, w)) || w.seq < 0) break;
            const int n = warp_uniform(chunks(w));
            if (!(ok = all(b_wait(s0) && ac_wait(2 * s0)))) break;
            issue_s(s0);
            for (int t = 0; t < n && ok; ++t) {
                const int step = s0 + t;
                const uint64_t a = desc_add(k_major, ac_slot(2 * step)), c = desc_add(mn_major, ac_slot(2 * step + 1));
                if (C::NS == 2 && t + 1 < n) {
                    if (!(ok = all(b_wait(step + 1) && ac_wait(2 * step + 2)))) break;
                    issue_s(step + 1);
                }
                // O1 = P C
                if (!(ok = all((step == 0 || mma_wait(&bars->o_free, (step - 1) & 1, abort_flag)) && ac_wait(2 * step + 1) &&
                               mma_wait(&bars->p_ready[step % C::NS], (step / C::NS) & 1, abort_flag))))
                    break;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)       // P: 64 tokens in 32 columns, each half where its scores were
                        mma_bf16_ts(tbase + C::O1_COL, tbase + C::S_COL + 128 * (step % C::NS) + (kk >> 2) * 64 + (kk & 3) * 8,
                                    desc_add(c, kk * 2048), id_o, kk > 0);
                }
                __syncwarp();
                // O2 = A X
                if (!(ok = all(mma_wait(&bars->x_ready, step & 1, abort_flag)))) break;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk) {     // d = 64: the features twice, over hi and lo rows
                        const int f = kk % (D / 16);
                        mma_bf16_ss(tbase + C::O2_COL, desc_add(a, (f >> 2) * C::CHUNK + (f & 3) * 32),
                                    desc_add(mn_major, C::X_OFF + kk * 2048), id_o, kk > 0);
                    }
                    mma_commit(&bars->o_full);
                    if (t == n - 1) mma_commit(&bars->u_done[step % C::NB]);
                }
                __syncwarp();
                // the scores of the next step and U of this one, as their inputs arrive
                bool s_next = C::NS == 1 && t + 1 < n, u_next = t + 1 < n;
                const unsigned long long t0 = clock64();
                while (s_next || u_next) {
                    if (s_next && all(mbar_test_wait(&bars->b_full[(step + 1) % C::NB], ((step + 1) / C::NB) & 1) &&
                                      mbar_test_wait(&bars->ac_full[(2 * step + 2) % C::NAC], ((2 * step + 2) / C::NAC) & 1))) {
                        issue_s(step + 1);
                        s_next = false;
                    } else if (u_next && all(mbar_test_wait(&bars->w_ready, (w0 + t) & 1))) {
                        // U = (B w)^T C
                        const uint64_t lo = desc_add(mn_major, C::LO_OFF);
                        // d = 64: hi and lo are the two 64-feature chunks of one operand
                        const uint64_t b = D == 128 ? desc_add(mn_major, b_slot(step))
                                                    : smem_desc_sw128(base + b_slot(step), C::LO_OFF - b_slot(step), 1024);
                        tc_fence_after();
                        if (elect_one()) {
#pragma unroll
                            for (int kk = 0; kk < 8; ++kk) {
                                const uint64_t cd = desc_add(c, kk * 2048);
                                mma_bf16_ss(tbase + C::U_COL, desc_add(b, kk * 2048), cd, id_x, kk > 0);
                                if (D == 128) mma_bf16_ss(tbase + C::U_COL, desc_add(lo, kk * 2048), cd, id_x, 1);
                            }
                            mma_commit(&bars->u_done[step % C::NB]);
                        }
                        __syncwarp();
                        u_next = false;
                    } else if (!all(!*abort_flag && clock64() - t0 <= VSA_WAIT_LIMIT_CYCLES)) {
                        ok = false;
                        break;
                    }
                }
            }
            s0 += n;
            w0 += n - 1;
        }
        if (!ok) fail();
        if (elect_one()) mma_commit(&bars->mma_done);
        __syncwarp();
        wait_noabort(&bars->mma_done, 0);
      }
    } else if (warp < 8) {
        reg_dec<C::REG_SCORE>();
        // -------------------------------------------------------- the weights
        const int quarter = warp & 3, hf = warp >> 2;    // 32 tokens; half of the columns
        const int r = 32 * quarter + lane;               // token of the chunk
        const uint32_t tS = tbase + ((uint32_t)(32 * quarter) << 16) + C::S_COL + 64 * hf;
        // lam^|i-j| is lam^(to the near end of j's block of 32) times
        // lam^(within the block), both factors at most 1; in the diagonal block
        // it is a table's entry at j - i, 0 on the masked side.
        int s0 = 0;
        bool ok = true;
        for (int k = 0; ok; ++k) {
            DecayWork w;
            if (!(ok = queue_get(&bars->queue, k, abort_flag, w)) || w.seq < 0) break;
            const DecayPass& ps = passes.p[w.pass];
            const bool back = ps.back;
            const float l2 = decay_log2(log_decay, w.head);
            // forward lam^31 .. lam^0 and zeros, backwards zeros and lam^0 .. lam^31
            float* sPow = reinterpret_cast<float*>(smem + C::POW_OFF) + (k & 1) * C::POW_FLOATS;
            if (tid < 64) {
                const float y = (back ? tid >= 32 : tid < 32) ? ex2((float)(back ? tid - 32 : 31 - tid) * l2) : 0.f;
                sPow[tid] = y;
                sPow[64 + 1 + tid] = y;                  // for pairs that start at an odd place
                mbar_arrive(&bars->pow_ready[k & 1]);
            }
            // (Two warps complete a phase and eight wait for it, so that those two
            // may be a walk ahead of the others here, which one barrier would let
            // them leave behind; not two, as the scores of the next walk follow
            // the weights of all eight in this one.)
            if (!(ok = __all_sync(0xffffffffu, mbar_wait(&bars->pow_ready[k & 1], (k >> 1) & 1, abort_flag)))) break;
            const int n = chunks(w);
            for (int t = 0; t < n; ++t) {
                const int step = s0 + t, rows = min(128, w.len - token(w, back, t));
                if (rows < 128) {
                    // C's rows behind the sequence are another one's: zeros
                    if (!__all_sync(0xffffffffu, ac_wait(2 * step + 1))) { ok = false; break; }
                    uint8_t* c = smem + ac_slot(2 * step + 1);
                    for (int u = tid; u < (128 - rows) * 8 * C::NCH; u += 256)
                        *reinterpret_cast<uint4*>(c + (u % C::NCH) * C::CHUNK + rows * 128 + (u / C::NCH) * 16) = make_uint4(0, 0, 0, 0);
                    fence_proxy_async_smem();
                }
                if (!__all_sync(0xffffffffu, s_wait(step))) { ok = false; break; }
                tc_fence_after();
                const uint32_t tP = tS + 128 * (step % C::NS);
                // P over the scores, 32 columns at a time (a loop: the kernel's
                // roles have to share the instruction cache)
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    const int blk = 2 * hf + h;
                    uint32_t pk[16];
                    if (back ? blk >= quarter : blk <= quarter) {
                        const int far = blk == quarter ? 0 : back ? 32 * blk - r : r - 32 * blk - 31;
                        const int at = blk == quarter ? (back ? 32 : 31) - lane : back ? 32 : 0;
                        const uint64_t* y = reinterpret_cast<const uint64_t*>(sPow + (at & 1 ? 64 + 1 + at : at));
                        const float f = ps.p_scale * ex2((float)far * l2);
                        float s[32];
                        tmem_ld_32x32b_x32(tP + 32 * h, s);
                        tmem_wait_ld();
                        const uint64_t f2 = f32x2(f, f);
#pragma unroll
                        for (int e = 0; e < 32; e += 2)
                            unf32x2(mul_f32x2(f32x2(s[e], s[e + 1]), mul_f32x2(f2, y[e / 2])), s[e], s[e + 1]);
                        if (rows < 128) {                // scores of rows behind the sequence may be anything
                            const int lo = back && blk == quarter ? lane : 0;
                            const int hi = min(rows - 32 * blk, !back && blk == quarter ? lane + 1 : 32);
#pragma unroll
                            for (int e = 0; e < 32; ++e) s[e] = e >= lo && e < hi ? s[e] : 0.f;
                        }
#pragma unroll
                        for (int e = 0; e < 16; ++e) pk[e] = pack_bf16x2(s[2 * e], s[2 * e + 1]);
                    } else {
#pragma unroll
                        for (int e = 0; e < 16; ++e) pk[e] = 0;
                    }
                    tmem_st_32x32b_x16(tP + 16 * h, pk); // (over scores of this thread's that are read or masked)
                }
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(&bars->p_ready[step % C::NS]);
                if (t + 1 < n) {
                    // the products that read the last step's lo part have finished
                    if (step > 0 && !__all_sync(0xffffffffu, u_wait(step - 1))) { ok = false; break; }
                    if (!split_units(step, tid, 0, C::UNITS_P, rows, back, ps.w_scale, l2)) { ok = false; break; }
                }
            }
            s0 += n;
        }
        if (!ok) fail();
    } else if (warp >= 16) {
        // -------------------------------------------------------- the outputs
        const int quarter = warp & 3, r = 32 * quarter + lane;
        const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
        int s0 = 0;
        bool ok = true;
        for (int k = 0; ok; ++k) {
            DecayWork w;
            if (!(ok = queue_get(&bars->queue, k, abort_flag, w)) || w.seq < 0) break;
            const DecayPass& ps = passes.p[w.pass];
            const bool back = ps.back;
            const float l2 = decay_log2(log_decay, w.head), f_full = ps.s_scale * ex2((float)(back ? 127 - r : r + 1) * l2);
            const int n = chunks(w);
            for (int t = 0; t < n; ++t) {
                const int tok = token(w, back, t), rows = min(128, w.len - tok);
                const float f = back && rows < 128 ? ps.s_scale * ex2((float)(rows - 1 - r) * l2) : f_full;
                const QuadRows at(r < rows ? (long long)(w.begin + tok + r) * ps.out_stride + (long long)w.head * D : -1);
                if (!__all_sync(0xffffffffu, mbar_wait(&bars->o_full, (s0 + t) & 1, abort_flag))) { ok = false; break; }
                tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    float o[32];
                    {
                        float x[32];
                        tmem_ld_32x32b_x32(tbase + lanes + C::O1_COL + c, o);
                        tmem_ld_32x32b_x32(tbase + lanes + C::O2_COL + c, x);
                        tmem_wait_ld();
                        const uint64_t f2 = f32x2(f, f);
#pragma unroll
                        for (int e = 0; e < 32; e += 2) unf32x2(fma_f32x2(f2, f32x2(x[e], x[e + 1]), f32x2(o[e], o[e + 1])), o[e], o[e + 1]);
                    }
                    if (c + 32 == D) {
                        tc_fence_before();
                        mbar_arrive(&bars->o_free);
                    }
                    store_rows(ps.out + c, at, o);
                }
            }
            s0 += n;
        }
        if (!ok) fail();
    } else {
        reg_inc<C::REG_STATE>();
        // ---------------------------------------------------------- the state
        grid_dependency_wait();                          // the borders; nothing else here depends on the launches before
        // in registers: a row (TMEM lane) and half of its columns
        const int id = tid - 256, hf = id >> 7, row = id & 127, feat = row & (D - 1);
        const uint32_t tU = tbase + ((uint32_t)(32 * (warp & 3)) << 16) + C::U_COL + hf * (D / 2);
        int s0 = 0;
        bool ok = true;
        for (int k = 0; ok; ++k) {
            DecayWork w;
            if (!(ok = queue_get(&bars->queue, k, abort_flag, w)) || w.seq < 0) break;
            const DecayPass& ps = passes.p[w.pass];
            const bool back = ps.back;
            const float l2 = decay_log2(log_decay, w.head);
            const int n = chunks(w);
            const float* x0;                             // the state before step 0, or null: zeros
            if (back ? w.rest <= sh.seg.n : w.off == 0) x0 = ps.first ? ps.first + ((long long)w.seq * sh.heads + w.head) * D * D : nullptr;
            else x0 = ps.border + ((long long)(((back ? w.begin + sh.seg.n : w.begin) - sh.part.n) / sh.part) * sh.heads + w.head) * D * D;
            float x[D / 2];
#pragma unroll
            for (int c = 0; c < D / 2; ++c) x[c] = 0.f;
            if (x0 && row < D) {                         // (whole warps; from L2: the scan may have run beside this kernel's start)
                if (ps.trans) {
#pragma unroll
                    for (int c = 0; c < D / 2; ++c) x[c] = __ldcg(x0 + (long long)(hf * (D / 2) + c) * D + feat);
                } else {
#pragma unroll
                    for (int c = 0; c < D / 2; c += 16) {
                        uint4 u[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            u[e] = __ldcg(reinterpret_cast<const uint4*>(x0 + (long long)((feat & ~3) + e) * D + hf * (D / 2) + c + (lane & 3) * 4));
                        transpose_units(u, lane);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            x[c + 4 * e] = __uint_as_float(u[e].x); x[c + 4 * e + 1] = __uint_as_float(u[e].y);
                            x[c + 4 * e + 2] = __uint_as_float(u[e].z); x[c + 4 * e + 3] = __uint_as_float(u[e].w);
                        }
                    }
                }
            }
            // X = lam^tokens X + U, once the products of step t have finished
            auto update = [&](int t) {
                if (!__all_sync(0xffffffffu, u_wait(s0 + t))) return false;
                tc_fence_after();
                const float f = ex2((float)min(128, w.len - token(w, back, t)) * l2);
#pragma unroll
                for (int c = 0; c < D / 2; c += 32) {
                    float u[32];
                    tmem_ld_32x32b_x32(tU + c, u);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; ++e) x[c + e] = fmaf(f, x[c + e], u[e]);
                }
                tc_fence_before();
                return true;
            };
            for (int t = 0; t < n; ++t) {
                const int step = s0 + t, rows = min(128, w.len - token(w, back, t));
                if (t > 0) {
                    if (!update(t - 1)) { ok = false; break; }
                } else {
                    // the walk before has left the bf16 state's place
                    if (step > 0 && !__all_sync(0xffffffffu, u_wait(step - 1))) { ok = false; break; }
                }
                uint8_t* xr = sX + row * 128;
#pragma unroll
                for (int c = 0; c < D / 2; c += 8) {
                    const int col = hf * (D / 2) + c;
                    *reinterpret_cast<uint4*>(xr + (col >> 6) * C::CHUNK + ((((col & 63) >> 3) ^ (row & 7)) << 4)) =
                        make_uint4(pack_bf16x2(x[c], x[c + 1]), pack_bf16x2(x[c + 2], x[c + 3]), pack_bf16x2(x[c + 4], x[c + 5]),
                                   pack_bf16x2(x[c + 6], x[c + 7]));
                }
                // (before x_ready: the scores that would follow in the same place wait for that, so this phase cannot be missed)
                if (!__all_sync(0xffffffffu, s_wait(step))) { ok = false; break; }
                fence_proxy_async_smem();
                mbar_arrive(&bars->x_ready);
                if (t + 1 < n && !split_units(step, id, C::UNITS_P, C::UNITS, rows, back, ps.w_scale, l2)) { ok = false; break; }
            }
            s0 += n;
        }
        if (!ok) fail();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 21) tmem_dealloc(tbase, 512);
}

// --------------------------------------------------------------------- launch

// How the sequences are cut, whose lengths only the device knows: m chunks to
// a segment.  Estimated times in units of one chunk of decay_out_kernel (2.6 us
// at d = 128, 1.9 us at d = 64), each constant from a sweep over m:
//   outputs  one sequence: rounds of 148 CTAs of m chunks and two more for
//            their start and end; several: their mean share, half a longest
//            piece of imbalance, the starts.  The memory bounds them too: at
//            d = 128 a round of 148 chunks reads and writes 1.1 units' worth
//            (passes over the same tensors meet in L2).
//   borders  0.6 units a round of chunks whose sums are needed (half of the
//            tensors are read), and 3.5 for the two further launches.
// A sequence is taken to be 2.5 times the average at most; a longer one is cut
// in pieces of that (8000 tokens among 15 sequences of 20, 12 heads, d 128: 69 us
// forward and 114 backwards, alone 50 and 99).
static DecayShape decay_shape(int n_seq, int total, int heads, int d, int passes) {
    const long long chunks = std::max(1ll, ((long long)total + 127) / 128);
    const long long longest = n_seq == 1 ? chunks : std::min(chunks, (5 * chunks + 2ll * n_seq - 1) / (2ll * n_seq));
    const double walks = (double)heads * passes, sums = (double)heads * (passes > 1 ? 2 : 1);
    const double work = chunks * walks / 148;
    const double memory = work * (d == 128 ? 1.1 : 0.8) * (passes > 1 ? 7.0 / 12 : 1.0);
    long long best = longest;
    double best_cost = 1e300;
    auto consider = [&](long long pieces) {
        if (pieces < 1 || pieces > longest) return;
        const long long m = (longest + pieces - 1) / pieces;
        const bool cut = m < longest;
        double cost;
        if (n_seq == 1)
            cost = std::ceil((double)((chunks + m - 1) / m) * walks / 148) * (m + 2.0);
        else
            cost = std::max(m + 2.0, work + 0.5 * m + 2.0 * std::max(1.0, (cut ? (double)chunks / m + 0.5 * n_seq : n_seq) * walks / 148));
        cost = std::max(cost, memory);
        if (cut) cost += 0.6 * chunks * sums / 148 * (1.0 - (double)m / longest) + 3.5;
        if (cost < best_cost) { best_cost = cost; best = m; }
    };
    for (int pieces = 1; pieces <= 12; ++pieces) consider(pieces);
    for (int rounds = 1; rounds <= 4; ++rounds) consider((long long)(148 * rounds / walks));
    // parts of a segment: rounds of CTAs, one chunk for a start and end
    const double cuts = std::max(1.0, (double)chunks / best);
    long long part = best, k = 1;
    best_cost = 1e300;
    for (long long i = 1; i <= 4 && i <= best; ++i) {
        const long long len = (best + i - 1) / i;
        const double cost = std::ceil(cuts * i * sums / 148) * (len + 1.0);
        if (cost < best_cost) { best_cost = cost; part = len; k = i; }
    }
    return {n_seq, total, heads, divisor(128 * part * k), divisor(128 * part), divisor(heads), (int)k};
}

static size_t border_bytes(const DecayShape& s, int d) { return (size_t)(s.total / s.part.n) * s.heads * d * d * sizeof(float); }

long long decay_work_items(int n_seq, int total, int heads) { return 3 * ((long long)total / 128 + n_seq) * heads; }

size_t decay_scratch_bytes(int n_seq, int total, int heads, int d) {
    return std::max(border_bytes(decay_shape(n_seq, total, heads, d, 1), d), 2 * border_bytes(decay_shape(n_seq, total, heads, d, 3), d));
}

static bool decay_map(CUtensorMap* m, const PackedTensor& t, const DecayArgs& a, int box_rows) {
    return a.total == 0 || encode_packed_map(m, t, a.total, a.heads, a.d, 1, box_rows, a.enc);
}

template <int D>
static cudaError_t launch_decay(const DecayArgs& a, const DecayShape& sh, const DecayPasses& passes, int n_passes,
                                const DecayStateArgs& st, const DecayScanArgs& sc, int kinds, cudaStream_t stream) {
    const unsigned segs = (unsigned)(((long long)sh.total / sh.seg.n + sh.n_seq) * a.heads);
    // places of the sums and of the scan: every part and sequence, or those with borders
    const unsigned parts = (unsigned)(((long long)sh.total / sh.part.n + (st.ends ? sh.n_seq : 0)) * a.heads);
    const Divisor longer = st.ends ? sh.part : sh.seg;
    const bool by_seq = sh.n_seq <= sh.total / longer.n;
    const unsigned scans = (unsigned)((long long)(by_seq ? sh.n_seq : sh.total / longer.n) * a.heads);
    cudaError_t e = cudaFuncSetAttribute(decay_out_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, DecOutCfg<D>::SMEM);
    if (e != cudaSuccess) return e;
    if (a.total > sh.seg.n || st.ends) {  // some sequence may have several segments, or states are wanted
        e = cudaFuncSetAttribute(decay_state_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, DecStateCfg<D>::SMEM);
        if (e != cudaSuccess) return e;
        decay_state_kernel<D><<<parts * kinds, DecStateCfg<D>::THREADS, DecStateCfg<D>::SMEM, stream>>>(st, divisor(kinds), sh, a.cu, a.log_decay, a.status);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        if (scans)
            e = launch_overlapped(decay_scan_kernel<D>, dim3(scans, D * D / 1024, kinds), 256, 0, stream, sc, by_seq, longer, sh, a.cu, a.log_decay, a.status);
        if (e != cudaSuccess) return e;
        return launch_overlapped(decay_out_kernel<D>, dim3(segs * n_passes), DecOutCfg<D>::THREADS, DecOutCfg<D>::SMEM, stream, passes,
                                 divisor(n_passes), sh, a.cu, a.log_decay, a.status);
    }
    decay_out_kernel<D><<<segs * n_passes, DecOutCfg<D>::THREADS, DecOutCfg<D>::SMEM, stream>>>(passes, divisor(n_passes), sh, a.cu, a.log_decay, a.status);
    return cudaGetLastError();
}

cudaError_t launch_decay_fwd(const DecayArgs& a, cudaStream_t stream) {
    const DecayShape sh = decay_shape(a.n_seq, a.total, a.heads, a.d, 1);
    float* border = reinterpret_cast<float*>(a.scratch);
    DecayPasses ps{};
    DecayStateArgs st{};
    DecayPass& p = ps.p[0];
    if (!decay_map(&p.a, a.q, a, 128) || !decay_map(&p.b, a.k, a, 128) || !decay_map(&p.c, a.v, a, 128) ||
        !decay_map(&st.b[0], a.k, a, 64) || !decay_map(&st.c[0], a.v, a, 64))
        return cudaErrorInvalidValue;
    p.out = static_cast<__nv_bfloat16*>(a.out.p);
    p.out_stride = a.out.stride;
    p.first = a.state_in;
    p.border = border;
    p.w_scale = 1.f;
    p.p_scale = p.s_scale = a.scale;
    st.border[0] = border;
    st.last[0] = a.state_out;
    st.first[0] = a.state_in;
    st.w_scale[0] = 1.f;
    DecayScanArgs sc{};
    sc.border[0] = border;
    sc.last[0] = a.state_out;
    st.ends = a.state_out != nullptr;
    sc.first[0] = a.state_in;
    return a.d == 128 ? launch_decay<128>(a, sh, ps, 1, st, sc, 1, stream) : launch_decay<64>(a, sh, ps, 1, st, sc, 1, stream);
}

cudaError_t launch_decay_bwd(const DecayArgs& a, cudaStream_t stream) {
    const DecayShape sh = decay_shape(a.n_seq, a.total, a.heads, a.d, 3);
    float* border[2] = {reinterpret_cast<float*>(a.scratch), reinterpret_cast<float*>(a.scratch + border_bytes(sh, a.d))};
    CUtensorMap mq, mk, mv, mg;
    DecayStateArgs st{};
    if (!decay_map(&mq, a.q, a, 128) || !decay_map(&mk, a.k, a, 128) || !decay_map(&mv, a.v, a, 128) || !decay_map(&mg, a.dout, a, 128) ||
        !decay_map(&st.b[0], a.k, a, 64) || !decay_map(&st.c[0], a.v, a, 64) || !decay_map(&st.b[1], a.q, a, 64) ||
        !decay_map(&st.c[1], a.dout, a, 64))
        return cudaErrorInvalidValue;
    auto pass = [&](const CUtensorMap& ma, const CUtensorMap& mb, const CUtensorMap& mc, const PackedTensor& out, bool back, bool trans) {
        DecayPass p{};
        p.a = ma; p.b = mb; p.c = mc;
        p.out = static_cast<__nv_bfloat16*>(out.p);
        p.out_stride = out.stride;
        p.first = back ? a.dstate_out : a.state_in;
        p.border = border[back];
        p.back = back;
        p.trans = trans;
        // backwards the state is the gradient of S, which has the scale in it
        p.w_scale = back ? a.scale : 1.f;
        p.p_scale = a.scale;
        p.s_scale = back ? 1.f : a.scale;
        return p;
    };
    DecayPasses ps{};
    ps.p[0] = pass(mg, mv, mk, a.dq, false, true);
    ps.p[1] = pass(mv, mg, mq, a.dk, true, true);
    ps.p[2] = pass(mk, mq, mg, a.dv, true, false);
    st.w_scale[0] = 1.f;
    st.w_scale[1] = a.scale;
    DecayScanArgs sc{};
    sc.first[0] = a.state_in;
    sc.first[1] = a.dstate_out;
    for (int i = 0; i < 2; ++i) st.first[i] = sc.first[i];
    st.last[1] = sc.last[1] = a.dstate_in;
    st.ends = a.dstate_in != nullptr;
    for (int i = 0; i < 2; ++i) st.border[i] = sc.border[i] = border[i], st.back[i] = sc.back[i] = i;
    return a.d == 128 ? launch_decay<128>(a, sh, ps, 3, st, sc, 2, stream) : launch_decay<64>(a, sh, ps, 3, st, sc, 2, stream);
}

}  // namespace vsa
