// reorder.cu -- states follow the beams, in place.
//
// A thread owns one vector of bytes at the same offset of all W slots of a search: it loads every slot that has a
// follower, once, then stores to the followers, so no other thread's reads can meet its writes and nothing is
// staged in memory.  Slots that stay are not written, slots without followers are not read.
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
    __shared__ int64_t s_slot[MAXW];
    __shared__ uint64_t s_followers[MAXW], s_fill;
    const int b = blockIdx.y, tid = threadIdx.x, W = a.W;
    const auto &view = a.view[blockIdx.z];
    wait_for_previous();
    int64_t slot = -1;
    int p = -1;
    if (tid < W) {
        p = a.parents[(int64_t)b * W + tid];
        slot = a.state_indices ? a.state_indices[(int64_t)b * W + tid] : (int64_t)b * W + tid;
        if (slot >= a.n_slots) slot = -1;
    }
    if (tid < MAXW) s_slot[tid] = slot, s_followers[tid] = 0;
    if (tid == 0) s_fill = 0;
    __syncthreads();
    if (tid < W && slot >= 0 && p >= 0 && p != tid) {
        const bool none = p >= W || s_slot[p] < 0;
        atomicOr(reinterpret_cast<unsigned long long *>(none ? &s_fill : &s_followers[p]), 1ull << tid);
    }
    __syncthreads();
    const int64_t n = view.bytes / (int64_t)sizeof(Vec);
    for (int64_t e = blockIdx.x * (int64_t)blockDim.x + tid; e < n; e += (int64_t)gridDim.x * blockDim.x) {
        Vec x[MAXW];
#pragma unroll
        for (int j = 0; j < MAXW; ++j)
            if (s_followers[j]) x[j] = reinterpret_cast<const Vec *>(view.data + s_slot[j] * view.stride)[e];
#pragma unroll
        for (int j = 0; j < MAXW; ++j)
            for (uint64_t f = s_followers[j]; f; f &= f - 1)
                reinterpret_cast<Vec *>(view.data + s_slot[__ffsll(f) - 1] * view.stride)[e] = x[j];
        for (uint64_t f = s_fill; f; f &= f - 1)
            reinterpret_cast<Vec *>(view.data + s_slot[__ffsll(f) - 1] * view.stride)[e] = filled<Vec>();
    }
}

// Vectors of W slots in at most 128 registers
template <int MAXW, typename Vec> cudaError_t launch_width(const ReorderArgs &a, dim3 grid, cudaStream_t st) {
    if constexpr (MAXW * sizeof(Vec) <= 512) return launch_behind(k_reorder<MAXW, Vec>, grid, 256, 0, st, a);
    return cudaErrorInvalidValue;
}

template <typename Vec> cudaError_t launch(const ReorderArgs &a, cudaStream_t st) {
    int64_t most = 0;
    for (int i = 0; i < a.n_views; ++i) most = a.view[i].bytes > most ? a.view[i].bytes : most;
    const int64_t blocks = (most / (int64_t)sizeof(Vec) + 255) / 256;
    const dim3 grid((unsigned)(blocks < 1024 ? blocks : 1024), (unsigned)a.B, (unsigned)a.n_views);
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
    if (!(mix & 15) && a.W <= 32) return launch<uint4>(a, st);
    if (!(mix & 7)) return launch<uint2>(a, st);
    if (!(mix & 3)) return launch<uint32_t>(a, st);
    return launch<uint8_t>(a, st);
}

}  // namespace gdn
