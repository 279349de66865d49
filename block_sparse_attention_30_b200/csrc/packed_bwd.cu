// packed_bwd.cu -- gradients of the softmax attention over packed sequences
// (packed_attn.cu) on sm_100a.
//
// With P_ij = 2^(q_i.k_j log2(e)/sqrt(d) - lse_i) recomputed from the
// forward's lse, and the output gradient dO:
//     dV_j = sum_i P_ij dO_i,      dP_ij = dO_i.v_j,   D_i = dO_i.O_i,
//     dS_ij = P_ij (dP_ij - D_i),  dQ_i = sum_j dS_ij k_j / sqrt(d),
//     dK_j = sum_i dS_ij q_i / sqrt(d),
// the sums over i running over every query head of the group as well.
//
// Three launches, no atomics (the same call gives the same bits); each may
// start while the last CTAs of the one before end, and waits for it before the
// terms are read:
//   row_terms_kernel  (lse, D) of every packed row, D from the forward's fp32
//                  output (the bf16 one's rounding would enter dQ as
//                  -dD sum_j P_j k_j, which does not shrink with dQ when the
//                  keys share a large common component); rows whose keys are
//                  all in one block get a better D in the next kernel;
//   dq_kernel      one CTA per 128 rows of one kv head ((token, head of the
//                  group) pairs, as in the forward), walking its key blocks:
//                  S = Q K^T, dP = dO V^T, dQ += dS K;
//   dkdv_kernel    one CTA, or a cluster of them that share the walk and add
//                  their sums at its end (key_shares), per 128 keys of one kv
//                  head, walking the blocks of 128 rows that see them:
//                  S^T = K Q^T, dP^T = V dO^T, dV += P^T dO, dK += dS^T Q.  The
//                  rows of a block include the group's heads, so the sum over
//                  shared heads is part of the products.
// 7 products instead of the 5 of a single kernel, which would have to add dQ
// with atomics.  P and dS are rounded to bf16 for the products (2^-8 relative
// at most per weight); everything else, sums included, is fp32.
//
// TMEM holds S twice (dQ) or once (dK/dV), dP once (dK/dV at d = 64: twice) and
// the accumulators: 512 columns.  The tensor cores always have a product that
// does not wait for the softmax of the current block: dQ alternates dP of block
// j+1, dQ of block j and S of block j+2; dK/dV runs dV of block j and S^T of
// block j+1 while dS is formed, and dK of block j and dP^T of block j+1 while
// the next weights are.  Eight warps do the elementwise part, each row shared
// by two threads (64 columns each); warp 8 loads, warp 9 issues the products.
//
// 8192 tokens of one sequence, 12 heads, d 128, causal: 16 us for the terms
// (0.54 of the copy rate), 285 us for dQ (tensor pipe busy 58 % of the time) and
// 331 us for dK and dV (67 %).  The 7 products alone would take 440 us at the
// rate of a large library product; the rest is the start and end of a CTA's
// walk (it holds the whole SM: nothing covers its first loads and its epilogue)
// and, at d = 128, where TMEM has room for one dP, the wait for the elementwise
// part.
// Rows of a tile behind the sequence's end are masked by selection in the
// scores and overwritten with zeros in shared memory before they enter a
// product as its inner dimension (0 x NaN would not be 0).
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

namespace vsa {
using namespace sm100;

// ------------------------------------------------------------------ row terms
// terms[kv head][token][head of the group] = (lse, D), lse = +inf where the
// row saw no key (its weights are then 2^-inf = 0).  D/8 threads per row.
template <int D>
__global__ void __launch_bounds__(256)
row_terms_kernel(const float* __restrict__ o, const __nv_bfloat16* __restrict__ dout, const long long dout_stride,
                 const float* __restrict__ lse, const int total, const int heads, const int group,
                 float2* __restrict__ terms) {
    grid_dependents_launch();                            // the next kernel may start: it waits for the terms itself
    constexpr int TPR = D / 8;
    const long long id = (long long)blockIdx.x * (256 / TPR) + threadIdx.x / TPR;
    const int f = threadIdx.x % TPR * 8;
    const bool in = id < (long long)total * heads;
    const long long tok = in ? id / heads : 0;
    const int h = in ? (int)(id % heads) : 0;
    float acc = 0.f;
    if (in) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(o + (tok * heads + h) * D + f));
        const float4 b = __ldg(reinterpret_cast<const float4*>(o + (tok * heads + h) * D + f + 4));
        const uint4 g = __ldg(reinterpret_cast<const uint4*>(dout + tok * dout_stride + (long long)h * D + f));
        const float x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        const uint32_t y[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            acc = fmaf(x[2 * e], __uint_as_float(y[e] << 16), acc);
            acc = fmaf(x[2 * e + 1], __uint_as_float(y[e] & 0xffff0000u), acc);
        }
    }
#pragma unroll
    for (int m = TPR / 2; m > 0; m >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, m);
    if (in && f == 0) {
        const float l = __ldg(lse + (long long)h * total + tok);
        terms[((long long)(h / group) * total + tok) * group + h % group] = make_float2(l == -CUDART_INF_F ? CUDART_INF_F : l, acc);
    }
}

template <int D>
struct PackBwdCfg {
    static constexpr int NCH = D / 64;
    static constexpr int CHUNK = 128 * 128;
    static constexpr int TILE = NCH * CHUNK;
    static constexpr int BAR_OFF = 7 * TILE;             // (dK/dV uses 6 tiles; its row terms lie in the 7th)
    static constexpr int DELTA_OFF = BAR_OFF + 512;      // dQ: D of 128 rows, one half of the columns each
    static constexpr int SMEM = DELTA_OFF + 1024;
    static constexpr int THREADS = 320;                  // 8 elementwise warps, loads, MMAs
};
static_assert(PackBwdCfg<128>::SMEM <= 232448, "shared memory");

// (lse, D, last key seen) of a block's 128 rows, each kind in a row of its own:
// the keys' threads read four rows at a time, the same ones in every thread.
struct RowTerms {
    float lse[128], delta[128];
    int last[128];
};

struct PackBwdBars {
    uint64_t own_full;                   // the CTA's own tiles
    uint64_t x_full[3], x_empty[3];      // K blocks | Q blocks (2)
    uint64_t y_full[2], y_empty[2];      // V blocks | dO blocks
    uint64_t s_full[2], dp_full[2], p_ready, ds_ready, mma_done, delta_ready;
    uint32_t tmem_base;
    int abort;
};

__device__ __forceinline__ void bwd_bars_init(PackBwdBars* b) {
    b->abort = 0;
    mbar_init(&b->own_full, 1);
    for (int x = 0; x < 3; ++x) { mbar_init(&b->x_full[x], 1); mbar_init(&b->x_empty[x], 1); }
    for (int x = 0; x < 2; ++x) { mbar_init(&b->y_full[x], 1); mbar_init(&b->y_empty[x], 1); mbar_init(&b->s_full[x], 1); mbar_init(&b->dp_full[x], 1); }
    mbar_init(&b->p_ready, 256);
    mbar_init(&b->ds_ready, 256);
    mbar_init(&b->mma_done, 1);
    mbar_init(&b->delta_ready, 256);
    fence_barrier_init();
}

// acc = A B^T, both tiles of 128 rows in shared memory (K-major descriptors).
// Here and below the whole warp calls, one elected lane issues, and its
// completion is committed to the given barriers.
template <int D>
__device__ __forceinline__ void mma_scores(uint32_t acc, uint64_t a, uint64_t b, uint64_t* bar, uint64_t* bar2 = nullptr) {
    constexpr uint32_t id = idesc_bf16_f32(128, 128, false, false);
    if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t o = (kk >> 2) * PackBwdCfg<D>::CHUNK + (kk & 3) * 32;
            mma_bf16_ss(acc, desc_add(a, o), desc_add(b, o), id, kk > 0);
        }
        mma_commit(bar);
        if (bar2) mma_commit(bar2);
    }
    __syncwarp();
}

// acc (+)= T X: T 128 x 128 bf16 in TMEM (columns 0-63 of its inner dimension
// at t, 64-127 at t + 64), X a tile of 128 rows x D in shared memory (MN-major
// descriptor).
template <int D>
__device__ __forceinline__ void mma_weighted(uint32_t acc, uint32_t t, uint64_t x, bool accumulate, uint64_t* bar) {
    constexpr uint32_t id = idesc_bf16_f32(128, D, false, true);
    if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
            mma_bf16_ts(acc, t + (kk >> 2) * 64 + (kk & 3) * 8, desc_add(x, kk * 2048), id, accumulate || kk > 0);
        if (bar) mma_commit(bar);
    }
    __syncwarp();
}

// Rows [from, 128) of a tile become zeros (256 threads).
template <int D>
__device__ __forceinline__ void zero_rows(uint8_t* tile, int from, int tid) {
    constexpr int NCH = PackBwdCfg<D>::NCH;
    for (int u = tid; u < (128 - from) * 8 * NCH; u += 256)
        *reinterpret_cast<uint4*>(tile + (u % NCH) * PackBwdCfg<D>::CHUNK + from * 128 + (u / NCH) * 16) = make_uint4(0, 0, 0, 0);
}

// Half a row (D/2 features) of an accumulator, times `scale`, as bf16; zeros
// where the accumulator was never written.  `rows`: where the quad's rows start.
template <int D>
__device__ __forceinline__ void store_grad(uint32_t acc, bool written, float scale, __nv_bfloat16* dst, const QuadRows& rows) {
#pragma unroll
    for (int c = 0; c < D / 2; c += 32) {
        float o[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = 0.f;
        if (written) { tmem_ld_32x32b_x32(acc + c, o); tmem_wait_ld(); }
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] *= scale;
        store_rows(dst + c, rows, o);
    }
}

// A cluster's CTAs sum the blocks' shares of one accumulator each; this puts
// half a row of one (fp32, 16-byte units swizzled against bank conflicts) into
// the CTA's own shared memory for the others.
template <int D>
__device__ __forceinline__ void share_grad(uint32_t acc, bool written, float* image, int row, int hf) {
#pragma unroll
    for (int c = 0; c < D / 2; c += 32) {
        float o[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = 0.f;
        if (written) { tmem_ld_32x32b_x32(acc + c, o); tmem_wait_ld(); }
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
            const int unit = (hf * (D / 2) + c + e) / 4;
            *reinterpret_cast<float4*>(image + row * D + (unit ^ (row & 7)) * 4) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
        }
    }
}

// ------------------------------------------------------------------------ dQ
template <int D>
__global__ void __launch_bounds__(PackBwdCfg<D>::THREADS, 1)
packed_dq_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                 const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mg, const PackedShape sh,
                 const PackedCut cut, const int tiles, const int32_t* __restrict__ cu_q,
                 const int32_t* __restrict__ cu_k, const int causal, const float scale_log2, const float scale,
                 float2* terms, __nv_bfloat16* __restrict__ dq, const long long dq_stride,
                 int* status) {
    using C = PackBwdCfg<D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    if (smem_u32(smem) & 1023) {
        if (threadIdx.x == 0) report(status, kStatusMisaligned);
        return;
    }
    const int tid = threadIdx.x, warp = warp_uniform(tid >> 5), lane = tid & 31;
    PackBwdBars* bars = reinterpret_cast<PackBwdBars*>(smem + C::BAR_OFF);
    volatile int* abort_flag = &bars->abort;
    grid_dependents_launch();
    if (tid == 0) bwd_bars_init(bars);
    if (tid == 32) { tma_prefetch_desc(&mq); tma_prefetch_desc(&mk); tma_prefetch_desc(&mv); tma_prefetch_desc(&mg); }
    if (warp == 9) { tmem_alloc(&bars->tmem_base, 512); tmem_relinquish(); }
    const int group = cut.group.n, tok_per_tile = cut.tok.n, id = blockIdx.x;
    const int kvh = id % cut.heads;
    // the last tiles of a sequence see the most keys: they start first
    const SeqTile tile = find_tile(cu_q, sh.n_seq, sh.total_q, cut.cta, tiles - 1 - id / cut.heads, status, 0, cu_k, sh.total_k);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = warp_uniform(bars->tmem_base);
    if (tile.seq < 0) {
        grid_dependency_wait();                          // (by every CTA, so that the next launch's wait covers the one before this)
        if (warp == 9) tmem_dealloc(tbase, 512);
        return;
    }
    const SeqRange qr = tile.a, kr = tile.b;
    const int tok0 = tile.tile * tok_per_tile;
    const int n = warp_uniform((seen_keys(min(tok0 + tok_per_tile, qr.len) - 1, qr.len, kr.len, causal) + 127) / 128);   // key blocks
    uint8_t* sQ = smem;
    uint8_t* sG = smem + C::TILE;
    uint8_t* sK = smem + 2 * C::TILE;                    // 3 slots: a K block is read by S and, two steps later, by dQ
    uint8_t* sV = smem + 5 * C::TILE;                    // 2 slots
    const uint32_t tDP = tbase + 256, tAcc = tbase + 384;     // S of block j at 128 (j & 1)
    auto fail = [&]() { *abort_flag = 1; report(status, kStatusTimeout); };

    if (warp == 8) {
        if (n > 0 && elect_one()) {
            mbar_arrive_expect_tx(&bars->own_full, 2 * C::NCH * tok_per_tile * group * 128);
            for (int c = 0; c < C::NCH; ++c) {
                tma_load_3d(sQ + c * C::CHUNK, &mq, &bars->own_full, 64 * c, kvh * group, qr.begin + tok0);
                tma_load_3d(sG + c * C::CHUNK, &mg, &bars->own_full, 64 * c, kvh * group, qr.begin + tok0);
            }
            int done = 0;
            for (int t = 0; t < n; ++t) {
                const int x = t % 3, y = t & 1;
                if (t >= 3 && !mbar_wait(&bars->x_empty[x], (t / 3 - 1) & 1, abort_flag)) { fail(); break; }
                mbar_arrive_expect_tx(&bars->x_full[x], C::TILE);
                for (int c = 0; c < C::NCH; ++c)
                    tma_load_3d(sK + x * C::TILE + c * C::CHUNK, &mk, &bars->x_full[x], 64 * c, kvh, kr.begin + 128 * t);
                if (t >= 2 && !mbar_wait(&bars->y_empty[y], (t / 2 - 1) & 1, abort_flag)) {
                    wait_noabort(&bars->x_full[x], (t / 3) & 1);
                    fail();
                    break;
                }
                mbar_arrive_expect_tx(&bars->y_full[y], C::TILE);
                for (int c = 0; c < C::NCH; ++c)
                    tma_load_3d(sV + y * C::TILE + c * C::CHUNK, &mv, &bars->y_full[y], 64 * c, kvh, kr.begin + 128 * t);
                ++done;
            }
            if (*abort_flag) {
                // drain: every load must land before the shared memory is given up
                wait_noabort(&bars->own_full, 0);
                for (int t = max(0, done - 3); t < done; ++t) wait_noabort(&bars->x_full[t % 3], (t / 3) & 1);
                for (int t = max(0, done - 2); t < done; ++t) wait_noabort(&bars->y_full[t & 1], (t / 2) & 1);
            }
        }
    } else if (warp == 9) {
        if (n > 0) {
            const uint64_t q = smem_desc_sw128(smem_u32(sQ), 16, 1024), g = smem_desc_sw128(smem_u32(sG), 16, 1024);
            const uint64_t k = smem_desc_sw128(smem_u32(sK), 16, 1024), v = smem_desc_sw128(smem_u32(sV), 16, 1024);
            const uint64_t k_mn = smem_desc_sw128(smem_u32(sK), C::CHUNK, 1024);
            auto wait = [&](uint64_t* bar, int parity) {
                const bool done = __all_sync(0xffffffffu, mma_wait(bar, parity, abort_flag));
                tc_fence_after();
                return done;
            };
            auto issue_s = [&](int t) {
                if (!wait(&bars->x_full[t % 3], (t / 3) & 1)) return false;
                mma_scores<D>(tbase + 128 * (t & 1), q, desc_add(k, (t % 3) * C::TILE), &bars->s_full[t & 1]);
                return true;
            };
            auto issue_dp = [&](int t) {
                if (!wait(&bars->y_full[t & 1], (t / 2) & 1)) return false;
                mma_scores<D>(tDP, g, desc_add(v, (t & 1) * C::TILE), &bars->dp_full[0], &bars->y_empty[t & 1]);
                return true;
            };
            bool ok = wait(&bars->own_full, 0) && issue_s(0) && issue_dp(0) && (n < 2 || issue_s(1));
            for (int t = 0; t < n && ok; ++t) {
                if (!(ok = wait(&bars->ds_ready, t & 1))) break;
                if (t + 1 < n && !(ok = issue_dp(t + 1))) break;
                mma_weighted<D>(tAcc, tbase + 128 * (t & 1), desc_add(k_mn, (t % 3) * C::TILE), t > 0, &bars->x_empty[t % 3]);
                if (t + 2 < n) ok = issue_s(t + 2);
            }
            if (!ok) fail();
            if (elect_one()) mma_commit(&bars->mma_done);
            __syncwarp();
            wait_noabort(&bars->mma_done, 0);
        }
    } else {
        const int r = 32 * (warp & 3) + lane, hf = warp >> 2;     // row, half of the columns
        const int tok = tok0 + r / cut.group;
        const bool valid = r < tok_per_tile * group && tok < qr.len;
        const int lim = valid ? seen_keys(tok, qr.len, kr.len, causal) : 0;
        const int lim_min = seen_keys(tok0, qr.len, kr.len, causal);
        const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
        float2 ld = make_float2(0.f, 0.f);
        float2* term = terms + ((long long)kvh * sh.total_q + qr.begin + tok) * group + r % cut.group;
        grid_dependency_wait();
        if (valid) ld = __ldcg(term);
        bool ok = true;
        for (int t = 0; t < n; ++t) {
            if (128 * t + 128 > kr.len) {                // the last, partial block: K's rows behind the sequence
                if (!__all_sync(0xffffffffu, mbar_wait(&bars->x_full[t % 3], (t / 3) & 1, abort_flag))) { ok = false; break; }
                zero_rows<D>(sK + (t % 3) * C::TILE, kr.len - 128 * t, tid);
                fence_proxy_async_smem();
            }
            const uint32_t tS = tbase + lane_base + 128 * (t & 1) + 64 * hf;
            if (!__all_sync(0xffffffffu, mbar_wait(&bars->s_full[t & 1], (t >> 1) & 1, abort_flag))) { ok = false; break; }
            tc_fence_after();
            float p[64];
            tmem_ld_32x32b_x32(tS, *reinterpret_cast<float(*)[32]>(&p[0]));
            tmem_ld_32x32b_x32(tS + 32, *reinterpret_cast<float(*)[32]>(&p[32]));
            tmem_wait_ld();
            if (128 * t + 128 > lim_min) {
                const int seen = lim - 128 * t - 64 * hf;
#pragma unroll
                for (int e = 0; e < 64; ++e) p[e] = e < seen ? ex2(fmaf(p[e], scale_log2, -ld.x)) : 0.f;
            } else {
#pragma unroll
                for (int e = 0; e < 64; ++e) p[e] = ex2(fmaf(p[e], scale_log2, -ld.x));
            }
            if (!__all_sync(0xffffffffu, mbar_wait(&bars->dp_full[0], t & 1, abort_flag))) { ok = false; break; }
            tc_fence_after();
            const bool masked = 128 * t + 128 > lim_min;
            if (n == 1) {
                // all keys of these rows are here: D = sum_j P_j dP_j from the
                // fp32 weights.  (The forward's output, with its weights rounded
                // to bf16, is as good where rows see many keys; where they see
                // few, its error is felt in every dS of the row.)
                float part = 0.f;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float dp[32];
                    tmem_ld_32x32b_x32(tDP + lane_base + 64 * hf + 32 * c, dp);
                    tmem_wait_ld();
                    const int seen = lim - 64 * hf - 32 * c;
#pragma unroll
                    for (int e = 0; e < 32; ++e) part = fmaf(p[32 * c + e], e < seen ? dp[e] : 0.f, part);
                }
                float* half = reinterpret_cast<float*>(smem + C::DELTA_OFF);
                half[128 * hf + r] = part;
                mbar_arrive(&bars->delta_ready);
                if (!__all_sync(0xffffffffu, mbar_wait(&bars->delta_ready, 0, abort_flag))) { ok = false; break; }
                ld.y = half[r] + half[128 + r];
                if (valid && hf == 0) term->y = ld.y;    // for dK and dV
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float dp[32];
                tmem_ld_32x32b_x32(tDP + lane_base + 64 * hf + 32 * c, dp);
                tmem_wait_ld();
                uint32_t pk[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    float d0 = p[32 * c + 2 * e] * (dp[2 * e] - ld.y), d1 = p[32 * c + 2 * e + 1] * (dp[2 * e + 1] - ld.y);
                    if (masked) {                        // dP of a masked place may be anything
                        const int seen = lim - 128 * t - 64 * hf - 32 * c;
                        d0 = 2 * e < seen ? d0 : 0.f;
                        d1 = 2 * e + 1 < seen ? d1 : 0.f;
                    }
                    pk[e] = pack_bf16x2(d0, d1);
                }
                tmem_st_32x32b_x16(tS + 16 * c, pk);     // dS over S: this thread's 64 columns in 32
            }
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&bars->ds_ready);
        }
        if (ok && n > 0 && !__all_sync(0xffffffffu, mbar_wait(&bars->mma_done, 0, abort_flag))) ok = false;
        if (!ok) fail();
        if (ok) {
            tc_fence_after();
            const QuadRows at(valid ? ((long long)qr.begin + tok) * dq_stride + (long long)(kvh * group + r % cut.group) * D : -1);
            store_grad<D>(tAcc + lane_base + hf * (D / 2), n > 0, scale, dq + hf * (D / 2), at);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 9) tmem_dealloc(tbase, 512);
}

// --------------------------------------------------------------------- dK, dV
template <int D>
__global__ void __launch_bounds__(PackBwdCfg<D>::THREADS, 1)
packed_dkdv_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                   const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mg, const PackedShape sh,
                   const PackedCut cut, const int32_t* __restrict__ cu_q, const int32_t* __restrict__ cu_k,
                   const int causal, const float scale_log2, const float scale, const float2* terms,
                   __nv_bfloat16* __restrict__ dk, const long long dk_stride, __nv_bfloat16* __restrict__ dv,
                   const long long dv_stride, int* status) {
    using C = PackBwdCfg<D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    if (smem_u32(smem) & 1023) {
        if (threadIdx.x == 0) report(status, kStatusMisaligned);
        return;
    }
    const int tid = threadIdx.x, warp = warp_uniform(tid >> 5), lane = tid & 31;
    PackBwdBars* bars = reinterpret_cast<PackBwdBars*>(smem + C::BAR_OFF);
    volatile int* abort_flag = &bars->abort;
    if (tid == 0) bwd_bars_init(bars);
    if (tid == 32) { tma_prefetch_desc(&mq); tma_prefetch_desc(&mk); tma_prefetch_desc(&mv); tma_prefetch_desc(&mg); }
    if (warp == 9) { tmem_alloc(&bars->tmem_base, 512); tmem_relinquish(); }
    const int group = cut.group.n, tok_per_tile = cut.tok.n, shares = cut.shares.n, rows = tok_per_tile * group;   // rows of a block in use
    uint8_t* sQ = smem + 2 * C::TILE;                    // 2 slots
    uint8_t* sG = smem + 4 * C::TILE;                    // 2 slots
    if (rows < 128 && tid < 256) {
        // rows that no load writes (a group that does not divide 128): zeros
        for (int x = 0; x < 4; ++x) zero_rows<D>(sQ + x * C::TILE, rows, tid);
        fence_proxy_async_smem();
    }
    // a cluster of `shares` CTAs per tile of keys, each with its share of the row blocks
    const int id = blockIdx.x, share = id % cut.shares, item = id / cut.shares;
    const int kvh = item % cut.heads;
    // the first tiles of a sequence are seen by the most queries: they start first
    const SeqTile tile = find_tile(cu_k, sh.n_seq, sh.total_k, cut.cta, item / cut.heads, status, 0, cu_q, sh.total_q);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = warp_uniform(bars->tmem_base);
    if (tile.seq < 0) {                                  // the whole cluster
        grid_dependency_wait();
        if (warp == 9) tmem_dealloc(tbase, 512);
        return;
    }
    const SeqRange qr = tile.b, kr = tile.a;
    const int key0 = 128 * tile.tile;
    // first query token that sees key0, and the blocks from its on
    const int tok_first = causal ? max(0, key0 + qr.len - kr.len) : 0;
    const int all = max(0, (qr.len + tok_per_tile - 1) / cut.tok - tok_first / cut.tok);
    const int per = (all + shares - 1) / cut.shares;
    const int b0 = tok_first / cut.tok + min(all, share * per);
    const int n = warp_uniform(min(per, all - min(all, share * per)));
    uint8_t* sK = smem;
    uint8_t* sV = smem + C::TILE;
    RowTerms* sT = reinterpret_cast<RowTerms*>(smem + 6 * C::TILE);   // of the even and the odd blocks
    // at d = 64 there is room for two dP, so that the next block's does not
    // wait for this one's dS to be used up
    constexpr int NDP = D == 64 ? 2 : 1;
    const uint32_t tS = tbase, tDV = tbase + 256, tDK = tbase + 256 + D;
    auto tDP = [&](int t) { return tbase + 128 + (t % NDP) * 256; };
    auto fail = [&]() { *abort_flag = 1; report(status, kStatusTimeout); };

    if (warp == 8) {
        if (n > 0 && elect_one()) {
            mbar_arrive_expect_tx(&bars->own_full, 2 * C::TILE);
            for (int c = 0; c < C::NCH; ++c) {
                tma_load_3d(sK + c * C::CHUNK, &mk, &bars->own_full, 64 * c, kvh, kr.begin + key0);
                tma_load_3d(sV + c * C::CHUNK, &mv, &bars->own_full, 64 * c, kvh, kr.begin + key0);
            }
            int done = 0;
            for (int t = 0; t < n; ++t) {
                const int x = t & 1;
                // one barrier frees a slot's Q and dO: dK of step t - 2, the last product to read them
                if (t >= 2 && !mbar_wait(&bars->x_empty[x], (t / 2 - 1) & 1, abort_flag)) { fail(); break; }
                const int row = qr.begin + (b0 + t) * tok_per_tile;
                mbar_arrive_expect_tx(&bars->x_full[x], C::NCH * rows * 128);
                for (int c = 0; c < C::NCH; ++c)
                    tma_load_3d(sQ + x * C::TILE + c * C::CHUNK, &mq, &bars->x_full[x], 64 * c, kvh * group, row);
                mbar_arrive_expect_tx(&bars->y_full[x], C::NCH * rows * 128);
                for (int c = 0; c < C::NCH; ++c)
                    tma_load_3d(sG + x * C::TILE + c * C::CHUNK, &mg, &bars->y_full[x], 64 * c, kvh * group, row);
                ++done;
            }
            if (*abort_flag) {
                wait_noabort(&bars->own_full, 0);
                for (int t = max(0, done - 2); t < done; ++t) {
                    wait_noabort(&bars->x_full[t & 1], (t / 2) & 1);
                    wait_noabort(&bars->y_full[t & 1], (t / 2) & 1);
                }
            }
        }
    } else if (warp == 9) {
        if (n > 0) {
            const uint64_t k = smem_desc_sw128(smem_u32(sK), 16, 1024), v = smem_desc_sw128(smem_u32(sV), 16, 1024);
            const uint64_t q = smem_desc_sw128(smem_u32(sQ), 16, 1024), g = smem_desc_sw128(smem_u32(sG), 16, 1024);
            const uint64_t q_mn = smem_desc_sw128(smem_u32(sQ), C::CHUNK, 1024), g_mn = smem_desc_sw128(smem_u32(sG), C::CHUNK, 1024);
            auto wait = [&](uint64_t* bar, int parity) {
                const bool done = __all_sync(0xffffffffu, mma_wait(bar, parity, abort_flag));
                tc_fence_after();
                return done;
            };
            auto issue_s = [&](int t) {
                if (!wait(&bars->x_full[t & 1], (t / 2) & 1)) return false;
                mma_scores<D>(tS, k, desc_add(q, (t & 1) * C::TILE), &bars->s_full[0]);
                return true;
            };
            auto issue_dp = [&](int t) {
                if (!wait(&bars->y_full[t & 1], (t / 2) & 1)) return false;
                mma_scores<D>(tDP(t), v, desc_add(g, (t & 1) * C::TILE), &bars->dp_full[t % NDP]);
                return true;
            };
            bool ok = wait(&bars->own_full, 0) && issue_s(0) && issue_dp(0);
            for (int t = 0; t < n && ok; ++t) {
                if (!(ok = wait(&bars->p_ready, t & 1))) break;
                mma_weighted<D>(tDV, tS, desc_add(g_mn, (t & 1) * C::TILE), t > 0, nullptr);
                if (t + 1 < n && !(ok = issue_s(t + 1) && (NDP == 1 || issue_dp(t + 1)))) break;
                if (!(ok = wait(&bars->ds_ready, t & 1))) break;
                mma_weighted<D>(tDK, tDP(t), desc_add(q_mn, (t & 1) * C::TILE), t > 0, &bars->x_empty[t & 1]);
                if (NDP == 1 && t + 1 < n) ok = issue_dp(t + 1);
            }
            if (!ok) fail();
            if (elect_one()) mma_commit(&bars->mma_done);
            __syncwarp();
            wait_noabort(&bars->mma_done, 0);
        }
    } else {
        const int r = 32 * (warp & 3) + lane, hf = warp >> 2;     // key of the tile, half of the query rows
        const int key = key0 + r;
        const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
        // weights of a row that is not there are 2^-inf = 0
        float row_lse = CUDART_INF_F, row_delta = 0.f;
        int row_last = -1;
        auto fetch = [&](int t) {
            const int tok = (b0 + t) * tok_per_tile + tid / cut.group;
            row_lse = CUDART_INF_F; row_delta = 0.f; row_last = -1;
            if (tid < rows && tok < qr.len) {
                const float2 ld = __ldcg(terms + ((long long)kvh * sh.total_q + qr.begin + tok) * group + tid % cut.group);
                row_lse = ld.x;
                row_delta = ld.y;
                row_last = seen_keys(tok, qr.len, kr.len, causal) - 1;
            }
        };
        grid_dependency_wait();                          // for the terms; the operands were there before
        if (tid < 128 && n > 0) fetch(0);
        bool ok = true;
        // A wait that gave up leaves `ok` false in its warp, which then walks on
        // through the barriers below without working.
        for (int t = 0; t < n; ++t) {
            RowTerms& tr = sT[t & 1];
            if (tid < 128) {
                tr.lse[tid] = row_lse; tr.delta[tid] = row_delta; tr.last[tid] = row_last;
                if (t + 1 < n) fetch(t + 1);
            }
            asm volatile("bar.sync 1, 256;" ::: "memory");
            if (!ok) continue;
            const int tok0 = (b0 + t) * tok_per_tile;
            const bool tail = tok0 + tok_per_tile > qr.len;
            // keys hidden from the block's first token, or rows behind the sequence
            const bool masked = tail || seen_keys(tok0, qr.len, kr.len, causal) < min(key0 + 128, kr.len);
            if (tail) {
                bool here = mbar_wait(&bars->x_full[t & 1], (t / 2) & 1, abort_flag);
                here = here && mbar_wait(&bars->y_full[t & 1], (t / 2) & 1, abort_flag);
                if (!__all_sync(0xffffffffu, here)) { ok = false; continue; }
                zero_rows<D>(sQ + (t & 1) * C::TILE, (qr.len - tok0) * group, tid);
                zero_rows<D>(sG + (t & 1) * C::TILE, (qr.len - tok0) * group, tid);
                fence_proxy_async_smem();
            }
            if (!__all_sync(0xffffffffu, mbar_wait(&bars->s_full[0], t & 1, abort_flag))) { ok = false; continue; }
            tc_fence_after();
            float p[64];
            tmem_ld_32x32b_x32(tS + lane_base + 64 * hf, *reinterpret_cast<float(*)[32]>(&p[0]));
            tmem_ld_32x32b_x32(tS + lane_base + 64 * hf + 32, *reinterpret_cast<float(*)[32]>(&p[32]));
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 64; e += 4) {
                const float4 l = *reinterpret_cast<const float4*>(&tr.lse[64 * hf + e]);
                p[e] = ex2(fmaf(p[e], scale_log2, -l.x));
                p[e + 1] = ex2(fmaf(p[e + 1], scale_log2, -l.y));
                p[e + 2] = ex2(fmaf(p[e + 2], scale_log2, -l.z));
                p[e + 3] = ex2(fmaf(p[e + 3], scale_log2, -l.w));
            }
            if (masked) {
#pragma unroll
                for (int e = 0; e < 64; ++e) p[e] = key <= tr.last[64 * hf + e] ? p[e] : 0.f;
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                uint32_t pk[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) pk[e] = pack_bf16x2(p[32 * c + 2 * e], p[32 * c + 2 * e + 1]);
                tmem_st_32x32b_x16(tS + lane_base + 64 * hf + 16 * c, pk);
            }
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&bars->p_ready);
            if (!__all_sync(0xffffffffu, mbar_wait(&bars->dp_full[t % NDP], (t / NDP) & 1, abort_flag))) { ok = false; continue; }
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float dp[32];
                tmem_ld_32x32b_x32(tDP(t) + lane_base + 64 * hf + 32 * c, dp);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; e += 4) {
                    const float4 x = *reinterpret_cast<const float4*>(&tr.delta[64 * hf + 32 * c + e]);
                    dp[e] = p[32 * c + e] * (dp[e] - x.x);
                    dp[e + 1] = p[32 * c + e + 1] * (dp[e + 1] - x.y);
                    dp[e + 2] = p[32 * c + e + 2] * (dp[e + 2] - x.z);
                    dp[e + 3] = p[32 * c + e + 3] * (dp[e + 3] - x.w);
                }
                if (masked) {                            // dP of a masked place may be anything
#pragma unroll
                    for (int e = 0; e < 32; ++e) dp[e] = key <= tr.last[64 * hf + 32 * c + e] ? dp[e] : 0.f;
                }
                uint32_t pk[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) pk[e] = pack_bf16x2(dp[2 * e], dp[2 * e + 1]);
                tmem_st_32x32b_x16(tDP(t) + lane_base + 64 * hf + 16 * c, pk);
            }
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&bars->ds_ready);
        }
        if (ok && n > 0 && !__all_sync(0xffffffffu, mbar_wait(&bars->mma_done, 0, abort_flag))) ok = false;
        if (!ok) fail();
        if (ok) {
            tc_fence_after();
            if (shares == 1) {
                const long long row = (long long)kr.begin + key;
                const QuadRows at_v(key < kr.len ? row * dv_stride + (long long)kvh * D : -1);
                const QuadRows at_k(key < kr.len ? row * dk_stride + (long long)kvh * D : -1);
                store_grad<D>(tDV + lane_base + hf * (D / 2), n > 0, 1.f, dv + hf * (D / 2), at_v);
                store_grad<D>(tDK + lane_base + hf * (D / 2), n > 0, scale, dk + hf * (D / 2), at_k);
            } else {
                // every product has finished: the operands' places hold the CTA's sums for the cluster
                share_grad<D>(tDV + lane_base + hf * (D / 2), n > 0, reinterpret_cast<float*>(smem), r, hf);
                share_grad<D>(tDK + lane_base + hf * (D / 2), n > 0, reinterpret_cast<float*>(smem) + 128 * D, r, hf);
            }
        }
    }
    if (shares > 1) {
        // each CTA adds up its part of the rows, share after share (a fixed order)
        __syncwarp();
        cluster_sync();
        const int count = 128 / shares, row0 = share * count;
        constexpr int PER = C::THREADS / (D / 4);        // rows per pass
        const int unit = tid % (D / 4);
        for (int at = tid / (D / 4); at < 2 * count; at += 2 * PER) {
            float4 sum[2], y[2];
            for (int x = 0; x < shares; ++x) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int u = min(at + i * PER, 2 * count - 1), which = u >= count, row = row0 + u - which * count;
                    y[i] = cluster_load(reinterpret_cast<const float*>(smem) + which * 128 * D + row * D + (unit ^ (row & 7)) * 4, x);
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (x == 0) sum[i] = y[i];
                    else { sum[i].x += y[i].x; sum[i].y += y[i].y; sum[i].z += y[i].z; sum[i].w += y[i].w; }
                }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int u = at + i * PER, which = u >= count, row = row0 + u - which * count;
                if (u >= 2 * count || key0 + row >= kr.len) continue;
                const float f = which ? scale : 1.f;
                __nv_bfloat16* dst = (which ? dk + ((long long)kr.begin + key0 + row) * dk_stride : dv + ((long long)kr.begin + key0 + row) * dv_stride) +
                                     (long long)kvh * D + unit * 4;
                *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(sum[i].x * f, sum[i].y * f), pack_bf16x2(sum[i].z * f, sum[i].w * f));
            }
        }
        cluster_sync();                                  // the others have read this CTA's sums
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 9) tmem_dealloc(tbase, 512);
}

// --------------------------------------------------------------------- launch
static long long key_items(const PackedShape& s) { return ((long long)s.total_k / 128 + s.n_seq) * s.heads_kv; }

// CTAs that share a tile of keys in dK/dV: as many as make its rounds shortest,
// in units of one row block (1.5 us), 10 of them for a CTA's start and end and
// 0.75 for each share to add up.  A tile's longest chain of blocks (all rows of a sequence, taken to
// be 2.5 times the average one: the lengths are device data, and a longer one makes the estimate
// worse, not the result) bounds the time from below: few kv heads and a
// large group make long chains and few of them.  Packed training batch (4128
// tokens, 16 heads on 4, d 64): 1 share 94 us, 2 shares 66 us, 4 shares 80 us; 4000 tokens, 5
// heads on 1, d 128, with dQ: 304 and 129 us.  One sequence of 8000 tokens among 15 of 20, 12 heads
// on 4, d 128: 585 us, as long as alone.
static int key_shares(const PackedShape& s, int causal) {
    const double per_seq = (double)s.total_q / s.n_seq / (128 / s.group());
    const double longest = std::min(s.n_seq == 1 ? 1.0 : 2.5, (double)s.n_seq) * per_seq, mean = causal ? 0.5 * per_seq : per_seq;
    const double items = (double)key_items(s);
    int best = 1;
    double best_cost = 1e300;
    for (int n = 1; n <= 8; n *= 2) {
        const double cost = std::max(std::ceil(items * n / 148) * (mean / n + 10), longest / n + 10) + (n > 1 ? 0.75 * n : 0);
        if (cost < best_cost) { best_cost = cost; best = n; }
    }
    return best;
}

long long packed_bwd_work_items(const PackedShape& s) {
    const long long q = (long long)s.total_q / (128 / s.group()) + s.n_seq;
    return std::max(std::max(q * s.heads_kv, 8 * key_items(s)), ((long long)s.total_q * s.heads_q * s.d + 2047) / 2048);
}

size_t packed_bwd_scratch_bytes(const PackedShape& s) {
    return (size_t)s.total_q * s.heads_q * sizeof(float2);
}

template <int D>
static cudaError_t launch_packed_bwd_impl(const PackedArgs& a, cudaStream_t stream) {
    using C = PackBwdCfg<D>;
    const PackedShape& s = a.s;
    const int group = s.group(), tok = 128 / group;
    cudaError_t e = cudaFuncSetAttribute(packed_dq_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(packed_dkdv_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    float2* terms = reinterpret_cast<float2*>(a.scratch);
    // a side without rows is never loaded: any valid address will do for its maps
    void* any = s.total_q ? a.q.p : a.k.p;
    const PackedTensor none_q{any, (long long)s.heads_q * D}, none_k{any, (long long)s.heads_kv * D};
    const int rq = std::max(1, s.total_q), rk = std::max(1, s.total_k);
    CUtensorMap mq, mk, mv, mg;
    if (!encode_packed_map(&mq, s.total_q ? a.q : none_q, rq, s.heads_q, D, group, tok, a.enc) ||
        !encode_packed_map(&mg, s.total_q ? a.dout : none_q, rq, s.heads_q, D, group, tok, a.enc) ||
        !encode_packed_map(&mk, s.total_k ? a.k : none_k, rk, s.heads_kv, D, 1, 128, a.enc) ||
        !encode_packed_map(&mv, s.total_k ? a.v : none_k, rk, s.heads_kv, D, 1, 128, a.enc))
        return cudaErrorInvalidValue;
    const float scale = 1.f / sqrtf((float)D), scale_log2 = 1.4426950408889634f * scale;
    if (s.total_q) {
        const long long rows = (long long)s.total_q * s.heads_q;
        row_terms_kernel<D><<<(unsigned)((rows + 2048 / D - 1) / (2048 / D)), 256, 0, stream>>>(
            a.out32, static_cast<const __nv_bfloat16*>(a.dout.p), a.dout.stride, a.lse, s.total_q, s.heads_q, group, terms);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        const int tiles = s.total_q / tok + s.n_seq;
        const PackedCut cut{divisor(group), divisor(tok), divisor(tok), divisor(s.heads_kv), divisor(1)};
        e = launch_overlapped(packed_dq_kernel<D>, dim3((unsigned)(tiles * s.heads_kv)), C::THREADS, C::SMEM, stream, mq, mk, mv, mg, s,
                              cut, tiles, a.cu_q, a.cu_k, a.causal, scale_log2, scale, terms, static_cast<__nv_bfloat16*>(a.dq.p),
                              a.dq.stride, a.status);
        if (e != cudaSuccess) return e;
    }
    if (s.total_k) {
        const int shares = key_shares(s, a.causal);
        const PackedCut cut{divisor(group), divisor(tok), divisor(128), divisor(s.heads_kv), divisor(shares)};
        // after dQ (without queries there is none: then nothing to overlap with)
        e = launch_with(packed_dkdv_kernel<D>, shares, s.total_q > 0, dim3((unsigned)(key_items(s) * shares)), C::THREADS, C::SMEM, stream,
                        mq, mk, mv, mg, s, cut, a.cu_q, a.cu_k, a.causal, scale_log2, scale, terms,
                        static_cast<__nv_bfloat16*>(a.dk.p), a.dk.stride, static_cast<__nv_bfloat16*>(a.dv.p), a.dv.stride, a.status);
    }
    return e;
}

cudaError_t launch_packed_bwd(const PackedArgs& a, cudaStream_t stream) {
    return a.s.d == 128 ? launch_packed_bwd_impl<128>(a, stream) : launch_packed_bwd_impl<64>(a, stream);
}

}  // namespace vsa
