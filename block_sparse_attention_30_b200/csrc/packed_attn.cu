// packed_attn.cu -- causal softmax attention over packed sequences with
// grouped heads on sm_100a (no counterpart on the pages, whose attention is
// bidirectional over one grid; this is the dense, causal form that a model
// generating clip after clip, or conditioned on prompts of different lengths,
// needs next to the block-sparse pass).
//
// Per query token i of a sequence with nq queries and nk keys, and query head
// h of the group that shares kv head h / G:
//     O_i = sum_j p_ij v_j,   p_ij = softmax over j <= i + nk - nq of
//     q_i.k_j / sqrt(d)      (j < nk without the causal mask);
// a row that sees no key gives O = 0 and lse = -inf.
//
// A CTA works on NT = 2 tiles of 128 rows of one kv head (one where sequences
// are shorter); a row is a (token, head of the group) pair, token-major, so the
// group's heads share every K and V tile that is loaded, and a single new token
// fills G rows of a tile instead of one.  Per block of 128 keys:
//   * warp 4 NT brings Q once and the K and V blocks through one ring of TMA
//     stages, last block first (the masked ones come first, the rest of the
//     walk needs no mask);
//   * warp 4 NT + 1 issues S = Q K^T (M = 128, N = 128) for each tile into
//     TMEM and, once the softmax has written P as bf16 over S, O += P V
//     (A = P from TMEM): the tensor cores work on one tile while the other is
//     in its softmax;
//   * 4 warps per tile (one row per thread) do the online softmax in the exp2
//     domain with fp32 statistics; O is rescaled in TMEM only when a row
//     maximum grows by more than 2^8 (P stays below 256, far from overflow).
//     P is rounded to bf16 for the tensor cores (2^-8 relative at most per
//     weight, as much as the rounding of the output); the row sum adds the
//     fp32 weights, so lse is good to fp32.
// With NT = 2 a CTA fills the SM, and warp 4 NT + 2 takes over CTAs of the grid
// that have not started (cluster launch control), so that the set-up is paid
// once and the next work's loads and products run under this one's last softmax
// and its epilogue.  With the causal mask the works with the most keys of a
// sequence come first; from sequence to sequence the order is the batch's, the
// last one first.
// Few and long sequences (single tokens over a cache): the key axis is split
// and packed_combine_kernel joins the shares, as many for every sequence: the
// host knows the average length only (one cache of 100000 keys among 23 of 100,
// 40 heads on 8, d 128: 450 us, where alone it takes 105).
//
// Measured: one sequence of 8192 tokens, 12 heads, d 128: 203 us, tensor pipe
// and the exponentials' unit busy 60 % of the time each (at d 128 a block of 128
// x 128 scores takes 1024 tensor cycles, 16 products of 64, and its 16384
// exponentials as long at 16 a cycle; the two tiles' turns overlap in part);
// 23296 tokens: 1460 us, 1.14 PFLOP/s, 0.70 of a large library product's rate,
// with the power cap active.  At d 64 the products are half of that and the
// exponentials as many: 163 us and 1046 us (d 128 in the same runs, one call at a
// time: 214 and 1257).  One token
// on each of 24 caches, 40 heads on 8 (394 MB): 85 us, 0.71 of the copy rate.
// The rows of a K/V tile behind the sequence's last key belong to another
// sequence.  Scores there are masked by selection, whatever they are; V rows
// there are overwritten with zeros before P V (0 x NaN would not be 0).
#include <algorithm>
#include <cmath>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include "common.cuh"
#include "packed.cuh"
#include "packed.h"
#include "sm100.cuh"
#include "softmax_step.cuh"

namespace vsa {
using namespace sm100;

// NT tiles of 128 rows per CTA: two, or one where most sequences have no
// rows for a second (single tokens; two such CTAs share an SM instead).
template <int D, int NT>
struct PackCfg {
    static constexpr int NCH = D / 64;                   // 64-feature chunks
    static constexpr int CHUNK = 128 * 128;              // 128 rows of one chunk (bf16)
    static constexpr int TILE = NCH * CHUNK;             // 128 rows of one tensor
    static constexpr int NST = (NT == 2 ? 5 : 2) * 128 / D;   // K/V ring stages
    static constexpr int BAR_OFF = (NT + NST) * TILE;
    static constexpr int SMEM = BAR_OFF + 1024;
    static constexpr int THREADS = 128 * (NT + 1);       // softmax warpgroups and the loads' and MMAs'
    // registers a thread: 168 at launch, 72 + 2 * 216 = 3 * 168; 128 at launch, 56 + 200 = 2 * 128
    static constexpr int REG_LOAD = NT == 2 ? 72 : 56, REG_SOFT = NT == 2 ? 216 : 200;
    static constexpr int TMEM_COLS = 256 * NT;
    static constexpr int S_COL = 0;                      // S / P of tile w at 128 w
    static constexpr int O_COL = 128 * NT;               // O of tile w at O_COL + D w
};
static_assert(PackCfg<128, 2>::SMEM <= 232448 && PackCfg<64, 2>::SMEM <= 232448, "shared memory");
static_assert(PackCfg<128, 1>::SMEM <= 115712 && PackCfg<64, 1>::SMEM <= 115712, "shared memory of two CTAs");

// What a CTA works on: the rows of its tiles and their key blocks.
struct PackWork {
    int seq;             // -1: nothing
    int q0, nq;          // the sequence's first query row and query count
    int k0, nk;
    int tok[2];          // first token (within the sequence) of each tile
    int nb[2];           // key blocks each tile needs (0: none visible)
    int lo, hi;          // its share of the blocks [lo, hi)
    int kvh, split;
};

template <int D, int NT>
struct PackBars {
    WorkQueue<PackWork> queue;
    uint64_t q_full[2], q_empty;
    uint64_t full[PackCfg<D, NT>::NST], empty[PackCfg<D, NT>::NST];
    uint64_t s_full[2], p_half[2], p_full[2], o_full[2], o_free[2];
    uint64_t mma_done;                   // every MMA of the CTA finished
    uint32_t tmem_base;
    int abort;
};
static_assert(sizeof(PackBars<64, 2>) <= 1024, "barrier block");

__device__ __forceinline__ PackWork pack_work(const int32_t* __restrict__ cu_q, const int32_t* __restrict__ cu_k,
                                              const PackedShape& s, int nt, const PackedCut& cut, int tiles, int id,
                                              int causal, int* status) {
    PackWork w{};
    // the shares of a tile start together, so that long sequences come first as a whole
    w.split = id % cut.shares;
    id = id / cut.shares;
    w.kvh = id % cut.heads;
    const int tok_per_tile = cut.tok.n;
    const SeqTile at = find_tile(cu_q, s.n_seq, s.total_q, cut.cta, tiles - 1 - id / cut.heads, status, 0, cu_k, s.total_k);
    w.seq = at.seq;
    if (at.seq < 0) return w;
    const SeqRange q = at.a, k = at.b;
    w.q0 = q.begin; w.nq = q.len; w.k0 = k.begin; w.nk = k.len;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        w.tok[x] = (nt * at.tile + x) * tok_per_tile;
        // the tile's last token sees the most keys
        const int last = min(w.tok[x] + tok_per_tile, w.nq) - 1;
        w.nb[x] = x < nt && w.tok[x] < w.nq ? (seen_keys(last, w.nq, w.nk, causal) + 127) / 128 : 0;
    }
    const int nb = max(w.nb[0], w.nb[1]);
    const int per = (nb + cut.shares.n - 1) / cut.shares;
    w.lo = min(nb, w.split * per);
    w.hi = min(nb, w.lo + per);
    return w;
}

template <int D, int NT>
__global__ void __launch_bounds__(PackCfg<D, NT>::THREADS, 3 - NT)
packed_fwd_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                  const __grid_constant__ CUtensorMap mv, const PackedShape sh, const PackedCut cut,
                  const int tiles, const int32_t* __restrict__ cu_q, const int32_t* __restrict__ cu_k,
                  const int causal, const float scale_log2, __nv_bfloat16* __restrict__ out,
                  const long long out_stride, float* __restrict__ out32, float* __restrict__ lse,
                  float* __restrict__ part_o, float* __restrict__ part_lse, int* status) {
    using C = PackCfg<D, NT>;
    extern __shared__ __align__(1024) uint8_t smem[];
    if (smem_u32(smem) & 1023) {
        if (threadIdx.x == 0) report(status, kStatusMisaligned);
        return;
    }
    const int tid = threadIdx.x, warp = warp_uniform(tid >> 5), lane = tid & 31;
    const int group = cut.group.n, tok_per_tile = cut.tok.n, n_splits = cut.shares.n;
    uint8_t* sQ = smem;
    uint8_t* ring = smem + NT * C::TILE;
    PackBars<D, NT>* bars = reinterpret_cast<PackBars<D, NT>*>(smem + C::BAR_OFF);
    volatile int* abort_flag = &bars->abort;
    if (NT == 1 && n_splits > 1) grid_dependents_launch();   // the joining kernel may start: it waits for the shares itself
    if (tid == 32) { tma_prefetch_desc(&mq); tma_prefetch_desc(&mk); tma_prefetch_desc(&mv); }
    if (tid == 0) {
        bars->abort = 0;
        queue_init(&bars->queue, 4 * NT + 2);
        for (int x = 0; x < NT; ++x) {
            mbar_init(&bars->q_full[x], 1);
            mbar_init(&bars->s_full[x], 1);
            mbar_init(&bars->p_half[x], 128);
            mbar_init(&bars->p_full[x], 128);
            mbar_init(&bars->o_full[x], 1);
            mbar_init(&bars->o_free[x], 128);
        }
        for (int x = 0; x < C::NST; ++x) { mbar_init(&bars->full[x], 1); mbar_init(&bars->empty[x], 1); }
        mbar_init(&bars->q_empty, 1);
        mbar_init(&bars->mma_done, 1);
        fence_barrier_init();
    }
    if (warp == 4 * NT + 1) { tmem_alloc(&bars->tmem_base, C::TMEM_COLS); tmem_relinquish(); }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = warp_uniform(bars->tmem_base);
    auto fail = [&]() { *abort_flag = 1; report(status, kStatusTimeout); };
    // Every role walks the queue.  Of work with n = hi - lo > 0 blocks, step t
    // is block hi - 1 - t, and tile x takes part from step first(x) on (with
    // fewer steps than that, not at all).  Phases and ring items are counted
    // on from work to work.
    auto first_step = [](const PackWork& w, int x) { return max(0, w.hi - w.nb[x]); };

    if (warp >= 4 * NT) {
      reg_dec<C::REG_LOAD>();
      if (warp == 4 * NT + 2) {
        if (!queue_produce<NT == 2>(&bars->queue, abort_flag, [&](int id) {
                return pack_work(cu_q, cu_k, sh, NT, cut, tiles, id, causal, status);
            }))
            fail();
      } else if (warp == 4 * NT) {
        // ---------------------------------------------------------- loads
        // ring item r0 + 2 t is K of step t, r0 + 2 t + 1 its V
        int r0 = 0, works = 0, issued = 0, q_count[2] = {0, 0};
        bool ok = true;
        for (int k = 0; ok; ++k) {
            PackWork w;
            if (!(ok = queue_get(&bars->queue, k, abort_flag, w)) || w.seq < 0) break;
            const int n = w.hi - w.lo;
            if (n == 0) {
                if (lane == 0) queue_ending(&bars->queue);
                continue;
            }
            // Q's place is free once the last scores of the work before are finished
            if (works > 0 && !(ok = __all_sync(0xffffffffu, mbar_wait(&bars->q_empty, (works - 1) & 1, abort_flag)))) break;
            ++works;
            if (lane == 0) {
                for (int x = 0; x < NT; ++x) {
                    if (first_step(w, x) >= n) continue;
                    mbar_arrive_expect_tx(&bars->q_full[x], C::NCH * tok_per_tile * group * 128);
                    for (int c = 0; c < C::NCH; ++c)
                        tma_load_3d(sQ + x * C::TILE + c * C::CHUNK, &mq, &bars->q_full[x], 64 * c, w.kvh * group, w.q0 + w.tok[x]);
                    ++q_count[x];
                }
                for (int i = 0; i < 2 * n; ++i) {
                    const int r = r0 + i, st = r % C::NST;
                    if (r >= C::NST && !(ok = mbar_wait(&bars->empty[st], ((r / C::NST) - 1) & 1, abort_flag))) break;
                    mbar_arrive_expect_tx(&bars->full[st], C::TILE);
                    for (int c = 0; c < C::NCH; ++c)
                        tma_load_3d(ring + st * C::TILE + c * C::CHUNK, (i & 1) ? &mv : &mk, &bars->full[st], 64 * c, w.kvh,
                                    w.k0 + 128 * (w.hi - 1 - (i >> 1)));
                    ++issued;
                }
                queue_ending(&bars->queue);
            }
            __syncwarp();
            ok = __all_sync(0xffffffffu, ok);
            r0 += 2 * n;
        }
        if (!ok) fail();
        if (lane == 0 && *abort_flag) {
            // drain: every load must land before the CTA's shared memory is given up
            for (int x = 0; x < NT; ++x)
                if (q_count[x]) wait_noabort(&bars->q_full[x], (q_count[x] - 1) & 1);
            for (int i = max(0, issued - C::NST); i < issued; ++i) wait_noabort(&bars->full[i % C::NST], (i / C::NST) & 1);
        }
      } else if (warp == 4 * NT + 1) {
        // ----------------------------------------------------------- MMAs
        // (the whole warp walks the loop, so that every branch and value is
        // uniform; one elected lane issues)
        const uint32_t id_s = idesc_bf16_f32(128, 128, false, false);
        const uint32_t id_o = idesc_bf16_f32(128, D, false, true);
        const uint64_t q_desc = smem_desc_sw128(smem_u32(sQ), 16, 1024);
        const uint64_t k_desc = smem_desc_sw128(smem_u32(ring), 16, 1024), v_desc = smem_desc_sw128(smem_u32(ring), C::CHUNK, 1024);
        auto wait = [&](uint64_t* bar, int parity) { return __all_sync(0xffffffffu, mma_wait(bar, parity, abort_flag)) != 0; };
        int r0 = 0, steps[2] = {0, 0}, parts[2] = {0, 0};
        bool ok = true;
        for (int k = 0; ok; ++k) {
            PackWork w;
            if (!(ok = queue_get(&bars->queue, k, abort_flag, w)) || w.seq < 0) break;
            const int n = warp_uniform(w.hi - w.lo);
            if (n == 0) continue;
            const int first[2] = {warp_uniform(first_step(w, 0)), warp_uniform(first_step(w, 1))};
            auto item = [&](int i) { return wait(&bars->full[(r0 + i) % C::NST], ((r0 + i) / C::NST) & 1); };
            auto issue_s = [&](int x, int t) {
                const uint64_t a0 = desc_add(q_desc, x * C::TILE), b0 = desc_add(k_desc, ((r0 + 2 * t) % C::NST) * C::TILE);
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t o = (kk >> 2) * C::CHUNK + (kk & 3) * 32;
                        mma_bf16_ss(tbase + C::S_COL + 128 * x, desc_add(a0, o), desc_add(b0, o), id_s, kk > 0);
                    }
                    mma_commit(&bars->s_full[x]);
                }
                __syncwarp();
            };
            auto issue_o = [&](int x, int t, int half) {     // 64 keys
                const uint64_t b0 = desc_add(v_desc, ((r0 + 2 * t + 1) % C::NST) * C::TILE);
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)           // 16 keys per MMA
                        mma_bf16_ts(tbase + C::O_COL + D * x, tbase + C::S_COL + 128 * x + 32 * half + kk * 8,
                                    desc_add(b0, 8192 * half + kk * 2048), id_o, t > first[x] || half || kk > 0);
                    if (half && t == n - 1) mma_commit(&bars->o_full[x]);
                }
                __syncwarp();
            };
            for (int x = 0; x < NT && ok; ++x)
                if (first[x] < n) ok = wait(&bars->q_full[x], parts[x] & 1);
            // step t: P V of step t, then S of step t + 1 over the same columns
            // (MMAs of one thread run in issue order); step -1 has only the S
            for (int t = -1; t < n && ok; ++t) {
                bool have_k = false, have_v = false;
#pragma unroll
                for (int x = 0; x < NT; ++x) {
                    if (t >= first[x] && t >= 0) {
                        if (!have_v) { ok = item(2 * t + 1); have_v = true; }
                        // the work before has left O
                        if (ok && t == first[x] && parts[x] > 0) ok = wait(&bars->o_free[x], (parts[x] - 1) & 1);
                        const int parity = (steps[x] + t - first[x]) & 1;
                        if (!ok || !(ok = wait(&bars->p_half[x], parity))) break;
                        tc_fence_after();
                        issue_o(x, t, 0);
                        if (!(ok = wait(&bars->p_full[x], parity))) break;
                        tc_fence_after();
                        issue_o(x, t, 1);
                    }
                    if (t + 1 >= first[x] && t + 1 < n) {
                        if (!have_k) { ok = item(2 * t + 2); have_k = true; }
                        if (!ok) break;
                        tc_fence_after();
                        issue_s(x, t + 1);
                    }
                }
                if (!ok) break;
                if (elect_one()) {
                    if (t >= 0) mma_commit(&bars->empty[(r0 + 2 * t + 1) % C::NST]);
                    if (t + 1 < n) mma_commit(&bars->empty[(r0 + 2 * t + 2) % C::NST]);
                    if (t + 2 == n) mma_commit(&bars->q_empty);
                }
                __syncwarp();
            }
            r0 += 2 * n;
#pragma unroll
            for (int x = 0; x < NT; ++x)
                if (first[x] < n) { steps[x] += n - first[x]; ++parts[x]; }
        }
        if (!ok) fail();
        if (elect_one()) mma_commit(&bars->mma_done);
        __syncwarp();
        wait_noabort(&bars->mma_done, 0);
      }
    } else {
        reg_inc<C::REG_SOFT>();
        // ------------------------------------------------------- softmax
        const int x = warp >> 2;                         // tile
        const int r = tid & 127;                         // row of the tile
        const uint32_t lane_base = tbase + ((uint32_t)(32 * (warp & 3)) << 16);
        const uint32_t tS = lane_base + C::S_COL + 128 * x, tO = lane_base + C::O_COL + D * x;
        int r0 = 0, steps = 0, parts = 0;
        bool ok = true;
        for (int k = 0; ok; ++k) {
            PackWork w;
            if (!(ok = queue_get(&bars->queue, k, abort_flag, w)) || w.seq < 0) break;
            const int n = w.hi - w.lo, f = first_step(w, x);
            const int tok = w.tok[x] + r / cut.group;    // token within the sequence
            const bool valid = r < tok_per_tile * group && tok < w.nq;
            const int head = w.kvh * group + r % cut.group;
            const int lim = valid ? seen_keys(tok, w.nq, w.nk, causal) : 0;
            const int lim_min = seen_keys(w.tok[x], w.nq, w.nk, causal);   // of the tile's first token: the smallest
            float m_run = -CUDART_INF_F, l_run = 0.f;
            // a warp without rows has nothing to compute: what it leaves in its
            // rows of P only reaches its own rows of O, which are not stored
            const bool idle = !__any_sync(0xffffffffu, valid);
            for (int t = f; t < n; ++t) {
                const int key0 = 128 * (w.hi - 1 - t);
                if (!__all_sync(0xffffffffu, mbar_wait(&bars->s_full[x], (steps + t - f) & 1, abort_flag))) { ok = false; break; }
                if (key0 + 128 > w.nk) {
                    // the sequence's last, partial block (step 0): zero V's rows behind it.
                    // (After its scores: a tile that sat out the work before may be a
                    // round of the ring ahead, where the phase would be another one's.)
                    const int i = r0 + 2 * t + 1;
                    if (!__all_sync(0xffffffffu, mbar_wait(&bars->full[i % C::NST], (i / C::NST) & 1, abort_flag))) { ok = false; break; }
                    uint8_t* v = ring + (i % C::NST) * C::TILE;
                    const int z0 = w.nk - key0;
                    for (int u = r; u < (128 - z0) * 8 * C::NCH; u += 128)
                        *reinterpret_cast<uint4*>(v + (u % C::NCH) * C::CHUNK + z0 * 128 + (u / C::NCH) * 16) = make_uint4(0, 0, 0, 0);
                    fence_proxy_async_smem();
                }
                if (idle) {
                    mbar_arrive(&bars->p_half[x]);
                    mbar_arrive(&bars->p_full[x]);
                    continue;
                }
                tc_fence_after();
                float s[128];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld_32x32b_x32(tS + 32 * c, *reinterpret_cast<float(*)[32]>(&s[32 * c]));
                tmem_wait_ld();
                if (key0 + 128 > lim_min) {              // uniform over the tile
                    const int seen = lim - key0;
#pragma unroll
                    for (int e = 0; e < 128; ++e)
                        if (e >= seen) s[e] = -CUDART_INF_F;
                }
                float m0 = s[0], m1 = s[1], m2 = s[2], m3 = s[3];
#pragma unroll
                for (int e = 4; e < 124; e += 8) {
                    m0 = max3f(m0, s[e], s[e + 1]);
                    m1 = max3f(m1, s[e + 2], s[e + 3]);
                    m2 = max3f(m2, s[e + 4], s[e + 5]);
                    m3 = max3f(m3, s[e + 6], s[e + 7]);
                }
                m0 = max3f(m0, s[124], s[125]);
                m1 = max3f(m1, s[126], s[127]);
                const float mx = fmaxf(max3f(m0, m1, m2), m3) * scale_log2;
                const bool raise = mx > m_run + 8.f;
                const float alpha = raise ? ex2(m_run - mx) : 1.f;   // 0 from -inf
                if (raise) m_run = mx;
                l_run *= alpha;
                // P V of the step before is finished (s_full was committed behind
                // it), so O can be rescaled here; step f has no O yet
                if (t > f && __any_sync(0xffffffffu, raise)) {
#pragma unroll
                    for (int c = 0; c < D; c += 32) {
                        float o[32];
                        tmem_ld_32x32b_x32(tO + c, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] *= alpha;
                        tmem_st_32x32b_x32f(tO + c, o);
                    }
                }
                const float m_sub = m_run == -CUDART_INF_F ? 0.f : m_run;
                const uint64_t sc2 = f32x2(scale_log2, scale_log2), nm2 = f32x2(-m_sub, -m_sub);
                uint64_t acc0 = 0, acc1 = 0;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t pk[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        float t0, t1;
                        unf32x2(fma_f32x2(f32x2(s[32 * c + 2 * e], s[32 * c + 2 * e + 1]), sc2, nm2), t0, t1);
                        const float p0 = ex2(t0), p1 = ex2(t1);
                        pk[e] = pack_bf16x2(p0, p1);
                        if (e & 1) acc1 = add_f32x2(acc1, f32x2(p0, p1));
                        else acc0 = add_f32x2(acc0, f32x2(p0, p1));
                    }
                    tmem_st_32x32b_x16(tS + 16 * c, pk);
                    if (c == 1) {                        // P V starts on the first half of the keys
                        tmem_wait_st();
                        tc_fence_before();
                        mbar_arrive(&bars->p_half[x]);
                    }
                }
                float a0, a1, b0, b1;
                unf32x2(acc0, a0, a1);
                unf32x2(acc1, b0, b1);
                l_run += (a0 + a1) + (b0 + b1);
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(&bars->p_full[x]);
            }
            if (!ok) break;
            const bool took = f < n;                     // uniform over the tile
            if (took) {
                if (!(ok = __all_sync(0xffffffffu, mbar_wait(&bars->o_full[x], parts & 1, abort_flag)))) break;
                tc_fence_after();
                steps += n - f;
                ++parts;
            }
            r0 += 2 * n;
            const bool none = l_run == 0.f;               // the row saw no key (of this share)
            const float inv = none ? 0.f : 1.f / l_run;
            const float row_lse = none ? -CUDART_INF_F : m_run + log2f(l_run);
            const long long row = (long long)w.q0 + tok;
            if (n_splits > 1) {
                // partial result of this share, joined by combine_kernel
                if (valid) part_lse[((long long)w.split * sh.heads_q + head) * sh.total_q + row] = row_lse;
            } else {
                if (valid && lse) lse[(long long)head * sh.total_q + row] = row_lse;
            }
            // where this row goes: 16-bit and 32-bit output, or the share's partial one
            const long long dense = (row * sh.heads_q + head) * D;
            const QuadRows rows_b(valid && n_splits == 1 ? row * out_stride + (long long)head * D : -1);
            const QuadRows rows_f(n_splits > 1 ? (valid && !none ? (long long)w.split * sh.total_q * sh.heads_q * D + dense : -1)
                                               : (valid && out32 ? dense : -1));
            float* pf = n_splits > 1 ? part_o : out32;
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                float o[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = 0.f;
                if (took) { tmem_ld_32x32b_x32(tO + c, o); tmem_wait_ld(); }
                if (took && c + 32 == D) {
                    tc_fence_before();
                    mbar_arrive(&bars->o_free[x]);
                }
                if (idle) continue;
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = none ? 0.f : o[e] * inv;
                if (n_splits == 1) store_rows(out + c, rows_b, o);
                if (pf) store_rows(pf + c, rows_f, o);
            }
        }
        if (!ok) fail();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 4 * NT + 1) tmem_dealloc(tbase, C::TMEM_COLS);
}

// Joins the shares of a split key axis: out = sum_s 2^(lse_s - m) O_s / sum_s 2^(lse_s - m), m the largest lse_s.
// One CTA per `tok_per_cta` tokens and kv head as in the kernel before it, D / 4 threads per row.
template <int D>
__global__ void __launch_bounds__(256)
packed_combine_kernel(const PackedShape sh, const PackedCut cut, const int tiles, const int32_t* __restrict__ cu_q,
                      const float* part_o, const float* part_lse, __nv_bfloat16* __restrict__ out,
                      const long long out_stride, float* __restrict__ out32, float* __restrict__ lse, int* status) {
    constexpr int TPR = D / 4;
    const int group = cut.group.n, tok_per_cta = cut.cta.n, n_splits = cut.shares.n, id = blockIdx.x;
    const int kvh = id % cut.heads;
    const SeqTile at = find_tile(cu_q, sh.n_seq, sh.total_q, cut.cta, tiles - 1 - id / cut.heads, status);
    if (at.seq < 0) {
        grid_dependency_wait();                          // (by every CTA, so that what follows in the stream follows both launches)
        return;
    }
    const SeqRange q = at.a;
    const int tok0 = at.tile * tok_per_cta;
    const int rows = min(tok_per_cta, q.len - tok0) * group;
    grid_dependency_wait();                              // (and from L2: the shares may have been written beside this kernel's start)
    const int f = threadIdx.x % TPR * 4;
    for (int r = threadIdx.x / TPR + blockIdx.y * (256 / TPR); r < rows; r += 256 / TPR * gridDim.y) {
        const long long row = (long long)q.begin + tok0 + r / cut.group;
        const int head = kvh * group + r % cut.group;
        float m = -CUDART_INF_F;
        for (int s = 0; s < n_splits; ++s) m = fmaxf(m, __ldcg(part_lse + ((long long)s * sh.heads_q + head) * sh.total_q + row));
        float sum = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int s = 0; s < n_splits; ++s) {
            const float l = __ldcg(part_lse + ((long long)s * sh.heads_q + head) * sh.total_q + row);
            if (l == -CUDART_INF_F) continue;            // the share saw no key: its O was not written
            const float w = ex2(l - m);
            const float4 p = __ldcg(reinterpret_cast<const float4*>(part_o + (((long long)s * sh.total_q + row) * sh.heads_q + head) * D + f));
            sum += w;
            o.x = fmaf(w, p.x, o.x); o.y = fmaf(w, p.y, o.y); o.z = fmaf(w, p.z, o.z); o.w = fmaf(w, p.w, o.w);
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        o.x *= inv; o.y *= inv; o.z *= inv; o.w *= inv;
        *reinterpret_cast<uint2*>(out + row * out_stride + (long long)head * D + f) = make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
        if (out32) *reinterpret_cast<float4*>(out32 + (row * sh.heads_q + head) * D + f) = o;
        if (lse && f == 0) lse[(long long)head * sh.total_q + row] = sum == 0.f ? -CUDART_INF_F : m + log2f(sum);
    }
}

bool encode_packed_map(CUtensorMap* m, const PackedTensor& t, int rows, int heads, int d, int box_heads,
                       int box_rows, PFN_cuTensorMapEncodeTiled_v12000 enc) {
    cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)rows};
    cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)t.stride * 2};
    cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_rows};
    cuuint32_t es[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, t.p, dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// One tile per CTA where the average sequence does not fill it.
static int tiles_per_cta(const PackedShape& s) { return (long long)s.total_q * s.group() <= 128ll * s.n_seq ? 1 : 2; }

// Upper bound of the CTAs' worth of tokens that the sequences are cut into
// (their lengths are device data).
static long long cta_bound(const PackedShape& s) {
    return (long long)s.total_q / (tiles_per_cta(s) * (128 / s.group())) + s.n_seq;
}

long long packed_work_items(const PackedShape& s) { return cta_bound(s) * s.heads_kv; }

// Shares the key axis is split into, by the time of the rounds of CTAs in
// units of one block of 128 keys (1.6 us): a CTA takes two more for its start
// and end, and joining n shares takes two for its launch and n times the
// partial rows at 3 TB/s.  The host knows the average lengths only.
int packed_splits(const PackedShape& s) {
    const long long items = packed_work_items(s);
    const double slots = tiles_per_cta(s) == 1 ? 296 : 148;
    const double blocks = std::max(1.0, (double)s.total_k / s.n_seq / 128);
    const double rows = (double)s.total_q * s.heads_q * s.d * 4 / 3e12 / 1.6e-6;
    if (items >= 2 * slots) return 1;                    // enough to balance by themselves
    int best = 1;
    double best_cost = 1e300;
    for (int n = 1; n <= 64 && n <= blocks / 2 + 1; ++n) {
        const double cost = std::ceil(items * n / slots) * (blocks / n + 2) + (n > 1 ? 2 + n * rows : 0);
        if (cost < best_cost) { best_cost = cost; best = n; }
    }
    return best;
}

size_t packed_fwd_scratch_bytes(const PackedShape& s) {
    const int n = packed_splits(s);
    return n > 1 ? (size_t)n * s.total_q * s.heads_q * (s.d + 1) * sizeof(float) : 0;
}

template <int D, int NT>
static cudaError_t launch_packed_fwd_impl(const PackedArgs& a, cudaStream_t stream) {
    using C = PackCfg<D, NT>;
    // set on every call: a cache by device would need a lock to be re-entrant
    cudaError_t e = cudaFuncSetAttribute(packed_fwd_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    const int group = a.s.group(), tok = 128 / group;
    const long long tiles = cta_bound(a.s);
    // without keys nothing is read from k and v: any valid address will do for their maps
    const PackedTensor kk = a.s.total_k ? a.k : a.q, vv = a.s.total_k ? a.v : a.q;
    CUtensorMap mq, mk, mv;
    if (!encode_packed_map(&mq, a.q, a.s.total_q, a.s.heads_q, D, group, tok, a.enc) ||
        !encode_packed_map(&mk, kk, std::max(1, a.s.total_k), a.s.heads_kv, D, 1, 128, a.enc) ||
        !encode_packed_map(&mv, vv, std::max(1, a.s.total_k), a.s.heads_kv, D, 1, 128, a.enc))
        return cudaErrorInvalidValue;
    const int n = packed_splits(a.s);
    const PackedCut cut{divisor(group), divisor(tok), divisor(NT * tok), divisor(a.s.heads_kv), divisor(n)};
    float* part_o = reinterpret_cast<float*>(a.scratch);
    float* part_lse = part_o + (size_t)n * a.s.total_q * a.s.heads_q * D;
    const float scale_log2 = 1.4426950408889634f / sqrtf((float)D);
    packed_fwd_kernel<D, NT><<<(unsigned)(tiles * a.s.heads_kv * n), C::THREADS, C::SMEM, stream>>>(
        mq, mk, mv, a.s, cut, (int)tiles, a.cu_q, a.cu_k, a.causal, scale_log2,
        static_cast<__nv_bfloat16*>(a.out.p), a.out.stride, a.out32, a.lse, part_o, part_lse, a.status);
    if (n > 1) {
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        // rows of an average sequence's share of a CTA
        const long long rows = std::min<long long>(NT * tok, (a.s.total_q + a.s.n_seq - 1) / a.s.n_seq) * group, per = 256 / (D / 4);
        const int gy = (int)std::min((rows + per - 1) / per, 8ll);
        return launch_overlapped(packed_combine_kernel<D>, dim3((unsigned)(tiles * a.s.heads_kv), gy), 256, 0, stream, a.s, cut,
                                 (int)tiles, a.cu_q, part_o, part_lse, static_cast<__nv_bfloat16*>(a.out.p), a.out.stride, a.out32,
                                 a.lse, a.status);
    }
    return cudaGetLastError();
}

cudaError_t launch_packed_fwd(const PackedArgs& a, cudaStream_t stream) {
    if (tiles_per_cta(a.s) == 1)
        return a.s.d == 128 ? launch_packed_fwd_impl<128, 1>(a, stream) : launch_packed_fwd_impl<64, 1>(a, stream);
    return a.s.d == 128 ? launch_packed_fwd_impl<128, 2>(a, stream) : launch_packed_fwd_impl<64, 2>(a, stream);
}

}  // namespace vsa
