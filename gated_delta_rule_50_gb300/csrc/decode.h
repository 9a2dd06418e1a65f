// decode.h -- arguments and launchers of the decoding kernels (decode_api.cu checks, the other files launch).
#pragma once
#include <cuda_runtime.h>

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

cudaError_t launch_recurrent(const DecodeArgs &a, int K, gdn_dtype io, cudaStream_t st);
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
int beam_chunk(int64_t rows, int64_t vocab, gdn_dtype io);
cudaError_t launch_beam(const BeamArgs &a, gdn_dtype io, cudaStream_t st);

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
