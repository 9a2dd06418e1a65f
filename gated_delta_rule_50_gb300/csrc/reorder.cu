// reorder.cu -- states follow the beams, in place.
//
// A thread owns one vector of bytes at the same offset of all W slots of a search: it loads what every slot
// gets, then stores, so no other thread's reads can meet its writes and nothing is staged in memory.  Slots
// that stay are neither read nor written; a source with several followers comes from the caches after its
// first read.
#include "decode.h"

namespace gdn {
namespace {

template <typename Vec> __device__ __forceinline__ Vec filled();
template <> __device__ __forceinline__ uint4 filled<uint4>() { return make_uint4(~0u, ~0u, ~0u, ~0u); }
template <> __device__ __forceinline__ uint32_t filled<uint32_t>() { return ~0u; }
template <> __device__ __forceinline__ uint8_t filled<uint8_t>() { return 0xFF; }

// grid: (offsets, searches, views); MAXW slots at once in registers
template <int MAXW, typename Vec> __global__ void __launch_bounds__(256) k_reorder(const ReorderArgs a) {
    __shared__ int64_t s_src[MAXW], s_dst[MAXW];
    const int b = blockIdx.y, tid = threadIdx.x, W = a.W;
    const auto &view = a.view[blockIdx.z];
    if (tid < MAXW) {  // -1: nothing to do at this place; source -2: fill
        int64_t src = -1, dst = -1;
        if (tid < W) {
            const int p = a.parents[(int64_t)b * W + tid];
            dst = a.state_indices ? a.state_indices[(int64_t)b * W + tid] : (int64_t)b * W + tid;
            if (dst >= a.n_slots || dst < 0 || p < 0 || p == tid) dst = -1;
            if (dst >= 0) {
                src = p >= W ? -2 : a.state_indices ? a.state_indices[(int64_t)b * W + p] : (int64_t)b * W + p;
                if (src < 0 || src >= a.n_slots) src = -2;
            }
        }
        s_src[tid] = src, s_dst[tid] = dst;
    }
    __syncthreads();
    const int64_t n = view.bytes / (int64_t)sizeof(Vec);
    for (int64_t e = blockIdx.x * (int64_t)blockDim.x + tid; e < n; e += (int64_t)gridDim.x * blockDim.x) {
        Vec x[MAXW];
#pragma unroll
        for (int i = 0; i < MAXW; ++i) {
            x[i] = filled<Vec>();
            if (s_dst[i] >= 0 && s_src[i] >= 0) x[i] = reinterpret_cast<const Vec *>(view.data + s_src[i] * view.stride)[e];
        }
#pragma unroll
        for (int i = 0; i < MAXW; ++i)
            if (s_dst[i] >= 0) reinterpret_cast<Vec *>(view.data + s_dst[i] * view.stride)[e] = x[i];
    }
}

template <typename Vec> cudaError_t launch(const ReorderArgs &a, cudaStream_t st) {
    int64_t most = 0;
    for (int i = 0; i < a.n_views; ++i) most = a.view[i].bytes > most ? a.view[i].bytes : most;
    const int64_t blocks = (most / (int64_t)sizeof(Vec) + 255) / 256;
    const dim3 grid((unsigned)(blocks < 1024 ? blocks : 1024), (unsigned)a.B, (unsigned)a.n_views);
    if (a.W <= 4) k_reorder<4, Vec><<<grid, 256, 0, st>>>(a);
    else if (a.W <= 8) k_reorder<8, Vec><<<grid, 256, 0, st>>>(a);
    else if (a.W <= 16) k_reorder<16, Vec><<<grid, 256, 0, st>>>(a);
    else if (a.W <= 32) k_reorder<32, Vec><<<grid, 256, 0, st>>>(a);
    else k_reorder<64, Vec><<<grid, 256, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_reorder(const ReorderArgs &a, cudaStream_t st) {
    uint64_t mix = 0;
    for (int i = 0; i < a.n_views; ++i)
        mix |= reinterpret_cast<uint64_t>(a.view[i].data) | (uint64_t)a.view[i].stride | (uint64_t)a.view[i].bytes;
    if (!(mix & 15) && a.W <= 32) return launch<uint4>(a, st);
    if (!(mix & 3)) return launch<uint32_t>(a, st);
    return launch<uint8_t>(a, st);
}

}  // namespace gdn
