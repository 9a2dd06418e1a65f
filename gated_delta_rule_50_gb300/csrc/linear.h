// linear.h -- one run of linear attention over sequences, and its launchers (linear_api.cu checks and plans).
//
// With l = e^g of the head, tokens j = 0 .. n - 1 of a sequence and a state X that enters it, a run computes
//     out_j = o_scale l^(j + e) X^T a_j + p_scale sum_{i <= j} l^(j - i) (a_j . b_i) c_i
//     X    <- l^n X + s_scale sum_i l^(n - i - e) b_i c_i^T
// The forward is the run (q, k, v) with e = 1.  Its gradients are three more: with S the forward's states and D the
// state's gradient, which runs from the last token to the first,
//     dq_j = scale S_j do_j      the run (do, v, k), whose state is S^T, e = 1
//     dk_i = D_i v_i             the run (v, do, q) over the tokens in reverse, whose state is D^T, e = 0
//     dv_i = D_i^T k_i           the run (k, q, do) in reverse, whose state is D, e = 0
// so that one kernel serves them all.
#pragma once
#include <cuda_runtime.h>

#include "common.cuh"

namespace gdn {

enum { LIN_WHOLE = 0, LIN_SEG = 1, LIN_MAIN = 2 };

struct LinearRun {
    const void *a, *b, *c;
    gdn_strides sa, sb, sc;
    int ga, gb, gc;     // value head h reads head h / g? of a, b, c
    int da, dc;         // width of a and b, of c and out: 64 or 128
    const float *g;     // [Hv] or nullptr: 0
    const float *init;  // [n_seqs][Hv] states or nullptr: 0
    float *fin;         // the same, or nullptr
    bool transposed;    // the states of init and fin are [dc][da], not [da][dc]
    void *out;          // [B T][Hv][dc], io type, or fp32
    bool out_f32;
    float p_scale, s_scale, o_scale;
    int e;
    bool reverse;
    const int32_t *cu;  // device [n_seqs + 1] or nullptr
    int B, T, Hv, n_seqs;
    // Sequences are cut into n_seg segments of whole chunks where there are few of them.  LIN_SEG: the state that each
    // segment but the last adds, from 0, into seg; launch_linear_join makes the segments' first states of them; LIN_MAIN:
    // the segments from their first states.
    int n_seg, mode;
    float *seg;         // [n_seqs][Hv][n_seg][da][dc]
};

// First token (of all B T), tokens and chunks of sequence s; offsets that fall or leave the T tokens: an empty one
struct LinearSpan {
    int64_t first;
    int tokens, chunks, per_seg;  // per_seg: chunks of a segment
};
__device__ __forceinline__ LinearSpan linear_span(const LinearRun &r, int s) {
    LinearSpan x;
    x.first = (int64_t)s * r.T, x.tokens = r.T;
    if (r.cu) {
        const int lo = r.cu[s], hi = r.cu[s + 1];
        const bool valid = lo >= 0 && hi >= lo && hi <= r.T;
        x.first = valid ? lo : 0, x.tokens = valid ? hi - lo : 0;
    }
    x.chunks = (x.tokens + C - 1) / C;
    x.per_seg = (x.chunks + r.n_seg - 1) / r.n_seg;
    return x;
}

// The sequence that the CTAs of place `slot` take: where packed sequences are few they go longest first, so that a long one
// does not begin when the others are done.  A whole warp
__device__ __forceinline__ int linear_seq(const LinearRun &r, int slot) {
    if (!r.cu || r.n_seqs > 32 || r.n_seqs == 1) return slot;
    const int lane = threadIdx.x & 31;
    const int mine = lane < r.n_seqs ? r.cu[lane + 1] - r.cu[lane] : 0;
    int rank = 0;
    for (int s = 0; s < r.n_seqs; ++s) {
        const int other = __shfl_sync(~0u, mine, s);
        rank += other > mine || (other == mine && s < lane);
    }
    return __ffs(__ballot_sync(~0u, lane < r.n_seqs && rank == slot)) - 1;
}

// The tensor cores' kernel: bf16, rows on 16-byte boundaries.  What it does not take, the CUDA cores' does
bool linear_tc_supported(const LinearRun &r, gdn_dtype io);
cudaError_t launch_linear_tc(const LinearRun &r, cudaStream_t st);
cudaError_t launch_linear_simt(const LinearRun &r, gdn_dtype io, cudaStream_t st);
cudaError_t launch_linear_join(const LinearRun &r, cudaStream_t st);
// out[tokens][heads][d] (io type) = sum over each group of x[tokens][heads G][d] (fp32)
cudaError_t launch_group_sum(const float *x, void *out, int64_t tokens, int heads, int G, int d, gdn_dtype io, cudaStream_t st);
// Rows of x [T][row_bytes] that no sequence claims become 0
cudaError_t launch_unclaimed(void *x, int T, int64_t row_bytes, const int32_t *cu, int n_seqs, cudaStream_t st);

}  // namespace gdn
