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
    // Of packed sequences (2 to 32) only those are cut that are longer than seg_chunks, if that is not 0.
    // Segments have numbers, their slots, 0 .. slots - 1 at most.
    int n_seg, seg_chunks, slots, mode;
    float *seg;         // [slots][Hv][da][dc]
    int drop_chunk;     // test aid (gdn_debug_set_wait): a chunk that the tensor cores' kernel does not load, -1: none
};

// A sequence's first token (of its row of the batch), its tokens and chunks (offsets that fall or leave the T tokens: none),
// the chunks of its segments, and the slot of its first segment
struct LinearSpan {
    int first, tokens, chunks, per_seg, slot, segs;
};
__device__ __forceinline__ LinearSpan linear_span(const LinearRun &r, int s) {
    LinearSpan x;
    x.first = 0, x.tokens = r.T;
    if (r.cu) {
        const int lo = r.cu[s], hi = r.cu[s + 1];
        const bool valid = lo >= 0 && hi >= lo && hi <= r.T;
        x.first = valid ? lo : 0, x.tokens = valid ? hi - lo : 0;
    }
    x.chunks = (x.tokens + C - 1) / C;
    x.per_seg = (x.chunks + r.n_seg - 1) / r.n_seg;
    x.slot = s * r.n_seg, x.segs = x.per_seg ? (x.chunks + x.per_seg - 1) / x.per_seg : 1;
    return x;
}
// The tokens [from, to) of a sequence that its segment `part` takes: whole chunks, the last one's rest, none behind it.  By
// chunks, for (part + 1) per_seg C passes 2^31 where a sequence nearly has as many tokens
struct LinearPart {
    int from, to;
};
__host__ __device__ inline LinearPart linear_part(int tokens, int chunks, int per_seg, int part) {
    const int first = part * per_seg, c0 = first < chunks ? first : chunks, c1 = per_seg < chunks - c0 ? c0 + per_seg : chunks;
    return {c0 < chunks ? c0 * C : tokens, c1 < chunks ? c1 * C : tokens};
}
// Packed sequences: lane s has the s-th one's, and their slots follow each other by the segments' lengths, the longest first,
// so that a long one does not begin when the others are done.  A whole warp
__device__ __forceinline__ bool linear_packed(const LinearRun &r) { return r.cu && r.n_seqs > 1 && r.n_seqs <= 32; }
__device__ __forceinline__ LinearSpan linear_table(const LinearRun &r) {
    const int lane = threadIdx.x & 31;
    LinearSpan x = {0, 0, 0, 0, 0, 0};
    if (lane < r.n_seqs) {
        x = linear_span(r, lane);
        if (r.seg_chunks) {
            const int cuts = x.chunks > r.seg_chunks + r.seg_chunks / 4 ? (x.chunks + r.seg_chunks - 1) / r.seg_chunks : 1;
            x.per_seg = (x.chunks + cuts - 1) / cuts, x.segs = x.per_seg ? (x.chunks + x.per_seg - 1) / x.per_seg : 1;
        }
    }
    if (__reduce_add_sync(~0u, x.segs) > r.slots && lane < r.n_seqs) x.per_seg = x.chunks, x.segs = 1;  // overlapping ones
    for (int s = 0; s < r.n_seqs; ++s) {
        const int per = __shfl_sync(~0u, x.per_seg, s), segs = __shfl_sync(~0u, x.segs, s);
        if (s == 0) x.slot = 0;
        if (per > x.per_seg || (per == x.per_seg && s < lane)) x.slot += segs;
    }
    return x;
}
// What the CTAs of a slot take: segment `part` of sequence seq, which is -1 where there is none
__device__ __forceinline__ LinearSpan linear_place(const LinearRun &r, int slot, int &seq, int &part) {
    if (!linear_packed(r)) {
        seq = slot / r.n_seg, part = slot % r.n_seg;
        return linear_span(r, seq);
    }
    LinearSpan x = linear_table(r);
    seq = __ffs(__ballot_sync(~0u, slot >= x.slot && slot < x.slot + x.segs)) - 1;
    const int from = seq < 0 ? 0 : seq;
    x.first = __shfl_sync(~0u, x.first, from), x.tokens = __shfl_sync(~0u, x.tokens, from), x.chunks = __shfl_sync(~0u, x.chunks, from);
    x.per_seg = __shfl_sync(~0u, x.per_seg, from), x.slot = __shfl_sync(~0u, x.slot, from), x.segs = __shfl_sync(~0u, x.segs, from);
    part = slot - x.slot;
    return x;
}

// What a state is moved on by, again and again, over n tokens: X <- f X + U with f = l^n, at = g n.  One product and one sum:
// X + (l^n - 1) X would leave, where l^n is small, what X was rounded by, which may be more than all of U.  Where l is all but
// 1, f rounded would be off by up to 2^-25 every time, and always to the same side: 1e-5 after 300 chunks.  So each f is one
// of the two fp32 numbers around l^n, and `owed`, which is what the ones before it left out, says which: their product stays
// within 2^-23 of what it should be, however many there are.
struct LinearDecay {
    float f, left, owed;  // l^n = f + left
    __device__ __forceinline__ explicit LinearDecay(float at) {
        const float less = expm1f(at);
        const bool near = fabsf(less) < 0.5f;  // else states are soon gone, or grow: f as it is
        f = near ? 1.f + less : expf(at);
        left = near ? less - (f - 1.f) : 0.f;
        owed = 0.f;
    }
    __device__ __forceinline__ float next() {
        owed += left;
        const float now = f + owed;
        owed -= now - f;
        return now;
    }
};

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
