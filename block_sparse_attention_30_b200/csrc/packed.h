// packed.h -- internal launch interface of the operators over packed
// sequences: causal softmax attention with grouped heads (packed_attn.cu,
// packed_bwd.cu) and linear attention with a decay per head (decay_attn.cu,
// decay_step.cu).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <cstdint>

namespace vsa {

// Launch a kernel in clusters of n CTAs (n divides the grid).  `overlapped`: it
// may start before the one before it in the stream has ended; it waits
// (grid_dependency_wait) before it touches what that writes.
template <typename... P, typename... A>
cudaError_t launch_with(void (*kernel)(P...), unsigned n, bool overlapped, dim3 grid, unsigned threads, size_t smem,
                        cudaStream_t stream, A&&... args) {
    cudaLaunchAttribute at[2] = {};
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = n;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c{};
    c.gridDim = grid;
    c.blockDim = dim3(threads);
    c.dynamicSmemBytes = smem;
    c.stream = stream;
    c.attrs = n > 1 ? at : at + 1;
    c.numAttrs = (n > 1 ? 1 : 0) + (overlapped ? 1 : 0);
    return cudaLaunchKernelEx(&c, kernel, static_cast<P>(args)...);
}

template <typename... P, typename... A>
cudaError_t launch_overlapped(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t stream, A&&... args) {
    return launch_with(kernel, 1, true, grid, threads, smem, stream, static_cast<A&&>(args)...);
}

// Division by a number that the host knows, of 0 <= x < 2^31: one high product
// and a correction (magic = floor((2^32 - 1) / n), so the quotient is at most 1
// too small) instead of some 100 cycles; finding a piece of work takes several
// in a row.
struct Divisor {
    int n;
    unsigned magic;
};
inline Divisor divisor(long long n) { return {(int)n, 0xffffffffu / (unsigned)n}; }
__device__ __forceinline__ int operator/(int x, const Divisor& d) {
    const unsigned q = __umulhi((unsigned)x, d.magic);
    return (int)(q + ((unsigned)x - q * (unsigned)d.n >= (unsigned)d.n));
}
__device__ __forceinline__ int operator%(int x, const Divisor& d) { return x - x / d * d.n; }

// One bf16 tensor [rows][heads][d]: heads and features contiguous, rows
// `stride` elements apart.
struct PackedTensor {
    void* p;
    long long stride;
};

struct PackedShape {
    int n_seq, total_q, total_k, heads_q, heads_kv, d;
    int group() const { return heads_q / heads_kv; }
};

// How the rows of the packed tensors are handed to CTAs.
struct PackedCut {
    Divisor group;               // query heads per kv head
    Divisor tok;                 // tokens of a tile of 128 rows
    Divisor cta;                 // tokens of a CTA
    Divisor heads;               // kv heads
    Divisor shares;              // of the other axis
};

struct PackedArgs {
    PackedShape s;
    PackedTensor q, k, v, out, dout, dq, dk, dv;
    const int32_t* cu_q;         // [n_seq + 1]
    const int32_t* cu_k;
    float* out32;                // [total_q][heads_q][d] or null
    float* lse;                  // [heads_q][total_q] or null
    int causal;
    uint8_t* scratch;            // behind the workspace's status block
    int* status;
    PFN_cuTensorMapEncodeTiled_v12000 enc;
};

// 3-D map {d, heads, rows} of a packed tensor; box {64, box_heads, box_rows},
// 128-byte swizzle; rows past the end read as zeros.
bool encode_packed_map(CUtensorMap* m, const PackedTensor& t, int rows, int heads, int d, int box_heads,
                       int box_rows, PFN_cuTensorMapEncodeTiled_v12000 enc);

long long packed_work_items(const PackedShape& s);   // CTAs of one share, at most 2^31 - 1
long long packed_bwd_work_items(const PackedShape& s);   // of the backward's largest launch
int packed_splits(const PackedShape& s);
size_t packed_fwd_scratch_bytes(const PackedShape& s);
size_t packed_bwd_scratch_bytes(const PackedShape& s);
cudaError_t launch_packed_fwd(const PackedArgs& a, cudaStream_t stream);
cudaError_t launch_packed_bwd(const PackedArgs& a, cudaStream_t stream);

struct DecayArgs {
    int n_seq, total, heads, d;
    PackedTensor q, k, v, out, dout, dq, dk, dv;
    const float* log_decay;      // [heads]
    const int32_t* cu;           // [n_seq + 1]
    const float* state_in;       // [n_seq][heads][d][d] or null
    float* state_out;            // or null
    const float* dstate_out;     // or null
    float* dstate_in;            // or null
    float scale;
    uint8_t* scratch;            // behind the workspace's status block
    int* status;
    PFN_cuTensorMapEncodeTiled_v12000 enc;
};

long long decay_work_items(int n_seq, int total, int heads);   // CTAs of the largest launch, at most 2^31 - 1
size_t decay_scratch_bytes(int n_seq, int total, int heads, int d);
cudaError_t launch_decay_fwd(const DecayArgs& a, cudaStream_t stream);
cudaError_t launch_decay_bwd(const DecayArgs& a, cudaStream_t stream);

// One token per sequence: q, k, v, out [batch][heads][d], states [batch][heads][d][d].
struct DecayStepArgs {
    int batch, heads, d;
    PackedTensor q, k, v, out;
    const float* log_decay;
    const float* state;
    float* state_out;            // may be `state`
    float scale;
};

cudaError_t launch_decay_step(const DecayStepArgs& a, cudaStream_t stream);

}  // namespace vsa
