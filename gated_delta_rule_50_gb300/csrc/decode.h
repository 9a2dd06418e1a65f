// decode.h -- arguments and launchers of the decoding kernels (decode_api.cu checks, the other files launch).
#pragma once
#include <cuda_runtime.h>

#include <atomic>

#include "common.cuh"

namespace gdn {

// A checked gdn_decode_problem with its pointers; passed to the kernels by value.
struct DecodeArgs {
    const void *q, *k, *v;
    const float *g, *beta;
    gdn_strides sq, sk, sv, sg, sb;
    float *state;
    float *out_state;  // nullptr: in place
    void *o;           // nullptr: the states only
    const int32_t *state_indices, *cu, *token_indices, *parents;
    int64_t n_slots, slot_stride;
    int T, Hq, Hv, G, V;
    int n_seqs, n_steps;
    float scale;
};

// Allows a kernel `bytes` of dynamic shared memory, once per device and kernel (the setting stays with the context, and
// setting it again costs about as much as a launch).
template <typename Kernel> cudaError_t allow_smem(Kernel kernel, int bytes, std::atomic<uint64_t> &done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// The decoding kernels follow each other closely: each is launched so that its CTAs may take their places while the
// stream's previous kernel ends, and waits on the GPU for that end (and for its writes) before it touches memory.
__device__ __forceinline__ void wait_for_previous() {
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
}
template <typename... Params>
cudaError_t launch_clusters(void (*kernel)(Params...), int cluster, dim3 grid, int block, size_t smem, cudaStream_t st, Params... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[2] = {};
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)cluster, at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}
template <typename... Params>
cudaError_t launch_behind(void (*kernel)(Params...), dim3 grid, int block, size_t smem, cudaStream_t st, Params... args) {
    return launch_clusters(kernel, 1, grid, block, smem, st, args...);
}

cudaError_t launch_recurrent(const DecodeArgs &a, int K, gdn_dtype io, cudaStream_t st);
cudaError_t launch_linear_recurrent(const DecodeArgs &a, int K, gdn_dtype io, cudaStream_t st);  // without beta; g may be null
cudaError_t launch_tree(const DecodeArgs &a, int K, gdn_dtype io, cudaStream_t st);

cudaError_t launch_tree_tc(const DecodeArgs &a, int K, cudaStream_t st);  // bf16 io

struct BeamArgs {
    const void *logits;
    const float *scores;
    const uint8_t *finished, *mask;
    int64_t logits_batch, logits_beam, mask_batch, mask_beam;
    int B, W, vocab, n;
    int chunk, n_chunks;  // elements of a row that one CTA takes, CTAs per row
    float2 *stats;        // [B * W][n_chunks] running maximum and sum
    uint64_t *keys;       // [B * W][n_chunks][n] best logits of the chunk, 0 where there are fewer
    float *out_scores;
    int32_t *out_tokens, *out_parents;
};
int beam_chunk(int64_t rows, int64_t vocab, int64_t n, gdn_dtype io);
cudaError_t launch_beam(const BeamArgs &a, gdn_dtype io, cudaStream_t st);

struct SampleArgs {
    const void *logits;
    const float *u;
    const uint8_t *mask;
    int64_t logits_row, mask_row;
    int B, vocab;
    const float *temperatures, *top_ps, *min_ps;  // nullptr: the one number for all rows
    const int32_t *top_ks;
    float temperature, top_p, min_p;
    int top_k;
    int32_t *tokens;
    float *logprobs;
    bool cached;  // a CTA's slice of a row stays in shared memory
};
cudaError_t launch_sample(const SampleArgs &a, gdn_dtype io, cudaStream_t st);

constexpr int kMaxViews = 32;
struct ReorderArgs {
    struct {
        unsigned char *data;
        int64_t stride, bytes;
    } view[kMaxViews];
    int n_views;
    int64_t n_slots;
    int B, W;
    const int32_t *parents, *state_indices;
};
cudaError_t launch_reorder(const ReorderArgs &a, cudaStream_t st);

}  // namespace gdn
