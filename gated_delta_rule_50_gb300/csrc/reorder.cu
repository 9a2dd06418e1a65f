// reorder.cu -- states follow the beams, in place.
//
// A thread owns one vector of bytes at the same offset of all W slots of a search: it loads every slot that has a
// follower, once, then stores to the followers, so no other thread's reads can meet its writes and nothing is
// staged in memory.  Slots that stay are not written, slots without followers are not read.
//
// Bound by memory: two layers of 8 x 16 states of 32 heads, 128 x 128, with a short tail each, 824 MB read and
// written, take 121 us, 6.8 TB/s (the rate of a plain copy is 6.7).  4 states of one layer take 2.7 us, a launch and
// three dependent reads.
#include "decode.h"

namespace gdn {
namespace {

template <typename Vec> __device__ __forceinline__ Vec filled();
template <> __device__ __forceinline__ uint4 filled<uint4>() { return make_uint4(~0u, ~0u, ~0u, ~0u); }
template <> __device__ __forceinline__ uint2 filled<uint2>() { return make_uint2(~0u, ~0u); }
template <> __device__ __forceinline__ uint32_t filled<uint32_t>() { return ~0u; }
template <> __device__ __forceinline__ uint8_t filled<uint8_t>() { return 0xFF; }

// grid: (offsets, searches, views); MAXW slots at once in registers
template <int MAXW, typename Vec> __global__ void __launch_bounds__(256) k_reorder(const __grid_constant__ ReorderArgs a) {
    __shared__ unsigned char *s_from[MAXW], *s_to[MAXW], *s_fill[MAXW];  // slots; followers by source; slots to fill
    __shared__ uint64_t s_followers[MAXW];
    __shared__ int s_begin[MAXW], s_count[MAXW], s_listed, s_fills;
    const int b = blockIdx.y, tid = threadIdx.x, W = a.W;
    const auto &view = a.view[blockIdx.z];
    const int64_t n = view.bytes / (int64_t)sizeof(Vec), first = blockIdx.x * (int64_t)blockDim.x + tid;
    if (first - tid >= n) return;
    wait_for_previous();
    unsigned char *slot = nullptr;
    int p = -1;
    if (tid < W) {
        p = a.parents[(int64_t)b * W + tid];
        const int64_t i = a.state_indices ? a.state_indices[(int64_t)b * W + tid] : (int64_t)b * W + tid;
        if (i >= 0 && i < a.n_slots) slot = view.data + i * view.stride;
    }
    if (tid < MAXW) s_from[tid] = slot, s_followers[tid] = 0;
    if (tid == 0) s_listed = s_fills = 0;
    __syncthreads();
    const bool moves = tid < W && slot && p >= 0 && p != tid, follows = moves && p < W && s_from[p];
    if (follows) atomicOr(reinterpret_cast<unsigned long long *>(&s_followers[p]), 1ull << tid);
    if (moves && !follows) s_fill[atomicAdd(&s_fills, 1)] = slot;
    __syncthreads();
    if (tid < MAXW) {
        s_count[tid] = __popcll(s_followers[tid]);
        s_begin[tid] = atomicAdd(&s_listed, s_count[tid]);
    }
    __syncthreads();
    if (follows) s_to[s_begin[p] + __popcll(s_followers[p] & ((1ull << tid) - 1))] = slot;
    __syncthreads();
    const int fills = s_fills;
    for (int64_t e = first; e < n; e += (int64_t)gridDim.x * blockDim.x) {
        Vec x[MAXW];
#pragma unroll
        for (int j = 0; j < MAXW; ++j)
            if (s_count[j]) x[j] = reinterpret_cast<const Vec *>(s_from[j])[e];
#pragma unroll
        for (int j = 0; j < MAXW; ++j)
            for (int k = 0, at = s_begin[j]; k < s_count[j]; ++k) reinterpret_cast<Vec *>(s_to[at + k])[e] = x[j];
        for (int k = 0; k < fills; ++k) reinterpret_cast<Vec *>(s_fill[k])[e] = filled<Vec>();
    }
}

// Vectors of W slots in at most 128 registers.  The widths are a loop's bounds: 8 slots in a loop over 32 take 245 us
// instead of 131.
template <int MAXW, typename Vec> cudaError_t launch_width(const ReorderArgs &a, dim3 grid, cudaStream_t st) {
    if constexpr (MAXW * sizeof(Vec) <= 512) return launch_behind(k_reorder<MAXW, Vec>, grid, 256, 0, st, a);
    return cudaErrorInvalidValue;
}

template <typename Vec> cudaError_t launch(const ReorderArgs &a, cudaStream_t st) {
    int64_t most = 0;
    for (int i = 0; i < a.n_views; ++i) most = a.view[i].bytes > most ? a.view[i].bytes : most;
    // A vector per thread, or as many as leave 48 CTAs for every SM: a CTA sets out with a chain of small reads.  8 x 16
    // states of 32 heads in two layers, moved in 130 us with 16 of them, 123 with 32, 121 with 48, 119 with 64 and 150
    // with a vector per thread; 4 x 4 states of one layer in 16.7, 15.8, 16.3 and 16.6 us.
    const int64_t blocks = (most / (int64_t)sizeof(Vec) + 255) / 256, share = 152 * 48 / ((int64_t)a.B * a.n_views);
    const int64_t x = blocks < share ? blocks : share;
    const dim3 grid((unsigned)(x < 1 ? 1 : x), (unsigned)a.B, (unsigned)a.n_views);
    if (a.W <= 4) return launch_width<4, Vec>(a, grid, st);
    if (a.W <= 8) return launch_width<8, Vec>(a, grid, st);
    if (a.W <= 16) return launch_width<16, Vec>(a, grid, st);
    if (a.W <= 32) return launch_width<32, Vec>(a, grid, st);
    return launch_width<64, Vec>(a, grid, st);
}

}  // namespace

cudaError_t launch_reorder(const ReorderArgs &a, cudaStream_t st) {
    uint64_t mix = 0;
    for (int i = 0; i < a.n_views; ++i)
        mix |= reinterpret_cast<uint64_t>(a.view[i].data) | (uint64_t)a.view[i].stride | (uint64_t)a.view[i].bytes;
    // The widest vector that all views' places and sizes allow.  The large case above takes 121 us with 16 bytes, 123.5 with
    // 8 and 132.5 with 4; one slot of an odd number of 16-bit values (tails of 3 x 12289) takes all views to single
    // bytes and the call to 425.
    if (!(mix & 15) && a.W <= 32) return launch<uint4>(a, st);
    if (!(mix & 7)) return launch<uint2>(a, st);
    if (!(mix & 3)) return launch<uint32_t>(a, st);
    return launch<uint8_t>(a, st);
}

}  // namespace gdn
