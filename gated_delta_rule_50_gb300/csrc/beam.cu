// beam.cu -- one selection of a beam search over beams and vocabulary.
//
// k_beam_scan: a CTA takes a chunk of one beam's logits, once through memory: the running maximum and sum of
// the softmax, and the chunk's n best logits.  A logit and its place make one whole number (a key: ordered
// bits of the value above, complement of the index below), so all keys differ and "the n best" needs no rule
// for ties.  The n-th largest of the threads' own maxima bounds the n-th best key from below, and at most n
// threads hold anything above it; those read their elements again (from the caches) and what is left, at
// most n times a thread's elements whatever the order of the input, is ranked by counting.
// k_beam_pick: a CTA per search joins the chunks' sums into the beams' normalisers, turns the keys into
// scores and selects in the same way, by the heads of the sorted lists.
// No result depends on the order in which threads arrive: places of collected keys do, their ranks do not.
#include <cuda_bf16.h>

#include "common.cuh"
#include "decode.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxPer = 128;  // elements of a chunk per thread, at most

__device__ __forceinline__ uint32_t ordered(float x) {  // larger for larger x; +0 and -0 alike
    const uint32_t u = __float_as_uint(x + 0.f);
    return u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t u) {
    return __uint_as_float(u ^ ((u >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}
// 0 for what can never be chosen: -inf and NaN
__device__ __forceinline__ uint64_t make_key(float x, uint32_t index) {
    return x > -INFINITY ? (uint64_t)ordered(x) << 32 | (0xFFFFFFFFu - index) : 0;
}
__device__ __forceinline__ uint32_t key_index(uint64_t key) { return 0xFFFFFFFFu - (uint32_t)key; }
__device__ __forceinline__ float key_value(uint64_t key) { return unordered((uint32_t)(key >> 32)); }

__device__ __forceinline__ float exp_of(float x) {  // e^x for x <= 0
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.4426950408889634f));
    return y;
}

// Joins (m, s) with (m2, s2): sums of e^(x - m).  An empty side has m = -inf, s = 0.
__device__ __forceinline__ void join(float &m, float &s, float m2, float s2) {
    const float top = fmaxf(m, m2);
    s = (m == -INFINITY ? s : s * expf(m - top)) + (m2 == -INFINITY ? s2 : s2 * expf(m2 - top));
    m = top;
}

// The n-th largest (n <= 256) of the 256 threads' keys, to all threads: each warp sorts its 32, then a key's
// rank is its place there plus, by bisection, the number of larger ones in the other warps' lists.  Keys that
// are equal (only 0 can be) take the ranks of their warps.
__device__ uint64_t nth_largest(uint64_t key, int n, uint64_t *s_sorted, uint64_t *s_answer) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint64_t x = key;
#pragma unroll
    for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
        for (int step = size >> 1; step; step >>= 1) {
            const uint64_t y = __shfl_xor_sync(~0u, x, step);
            const bool larger = ((lane & step) == 0) == ((lane & size) == 0);  // descending
            x = larger ? (x > y ? x : y) : (x > y ? y : x);
        }
    __syncthreads();  // the arrays may still be read from an earlier use
    s_sorted[threadIdx.x] = x;
    __syncthreads();
    int rank = lane;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        const uint64_t *list = s_sorted + 32 * w;
        int at = 0;  // entries of the list that come before x
#pragma unroll
        for (int step = 16; step; step >>= 1)
            if (w < warp ? list[at + step - 1] >= x : list[at + step - 1] > x) at += step;
        if (at == 31 && (w < warp ? list[31] >= x : list[31] > x)) at = 32;
        if (w != warp) rank += at;
    }
    if (rank == n - 1) *s_answer = x;
    __syncthreads();
    return *s_answer;
}

template <typename IO> struct Pack;
template <> struct Pack<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void unpack(uint4 u, float (&x)[8]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) x[2 * i] = __uint_as_float(w[i] << 16), x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
};
template <> struct Pack<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void unpack(uint4 u, float (&x)[4]) {
        x[0] = __uint_as_float(u.x), x[1] = __uint_as_float(u.y), x[2] = __uint_as_float(u.z), x[3] = __uint_as_float(u.w);
    }
};

// Elements [at, at + N) of a row (at may begin before it); what is outside or masked is -inf.
template <typename IO>
__device__ __forceinline__ void load(const IO *row, const uint8_t *mask, bool mask_whole, int at, int vocab, float (&x)[Pack<IO>::N]) {
    constexpr int N = Pack<IO>::N;
    if (at >= 0 && at + N <= vocab) {
        Pack<IO>::unpack(*reinterpret_cast<const uint4 *>(row + at), x);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = at + i >= 0 && at + i < vocab ? to_f<IO>(row[at + i]) : -INFINITY;
    }
    if (mask) {
        if (mask_whole && at >= 0 && at + N <= vocab) {
            uint32_t u[2] = {0, 0};
            if (N == 8) {
                const uint2 p = *reinterpret_cast<const uint2 *>(mask + at);
                u[0] = p.x, u[1] = p.y;
            } else {
                u[0] = *reinterpret_cast<const uint32_t *>(mask + at);
            }
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (!(u[i >> 2] >> (8 * (i & 3)) & 0xFF)) x[i] = -INFINITY;
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (at + i >= 0 && at + i < vocab && !mask[at + i]) x[i] = -INFINITY;
        }
    }
}

template <typename IO> __global__ void __launch_bounds__(kThreads) k_beam_scan(const BeamArgs a) {
    constexpr int N = Pack<IO>::N;
    extern __shared__ uint64_t s_got[];  // n * (elements per thread)
    __shared__ uint64_t s_sorted[kThreads], s_nth;
    __shared__ float2 s_stat[kThreads / 32];
    __shared__ int s_count;
    const int tid = threadIdx.x, n = a.n;
    const int64_t unit = blockIdx.x;  // (row, chunk)
    const int row = (int)(unit / a.n_chunks), chunk = (int)(unit - (int64_t)row * a.n_chunks);
    if (a.finished && a.finished[row]) return;
    const int b = row / a.W, w = row - b * a.W;
    const IO *x_row = static_cast<const IO *>(a.logits) + b * a.logits_batch + w * a.logits_beam;
    const uint8_t *mask = a.mask ? a.mask + b * a.mask_batch + w * a.mask_beam : nullptr;
    // vectors lie on 16-byte boundaries: the first one may begin before the row
    const int shift = (int)((reinterpret_cast<uintptr_t>(x_row) & 15) / sizeof(IO));
    const bool mask_whole = mask && ((reinterpret_cast<uintptr_t>(mask) - shift) & (N - 1)) == 0;
    const int begin = chunk * a.chunk - shift + tid * N, end = min((chunk + 1) * a.chunk - shift, a.vocab);

    float m = -INFINITY, s = 0.f, best = -INFINITY;
    int best_at = begin;
#pragma unroll 4
    for (int at = begin; at < end; at += kThreads * N) {
        float x[N];
        load<IO>(x_row, mask, mask_whole, at, a.vocab, x);
        float top = x[0];
#pragma unroll
        for (int i = 1; i < N; ++i) top = fmaxf(top, x[i]);
        if (top > best) best = top, best_at = at;
        if (top > m) {
            s = m == -INFINITY ? s : s * exp_of(m - top);
            m = top;
        }
        float add = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) add += m == -INFINITY ? (x[i] == -INFINITY ? 0.f : x[i]) : exp_of(x[i] - m);
        s += add;
    }
    uint64_t mine = 0;
    if (best > -INFINITY) {
        float x[N];
        load<IO>(x_row, mask, mask_whole, best_at, a.vocab, x);
#pragma unroll
        for (int i = N - 1; i >= 0; --i)
            if (x[i] == best) mine = make_key(best, best_at + i);
    }
#pragma unroll
    for (int step = 16; step; step >>= 1) {
        const float m2 = __shfl_xor_sync(~0u, m, step), s2 = __shfl_xor_sync(~0u, s, step);
        join(m, s, m2, s2);
    }
    if (tid == 0) s_count = 0;
    if ((tid & 31) == 0) s_stat[tid >> 5] = make_float2(m, s);
    const uint64_t low = nth_largest(mine, n, s_sorted, &s_nth);
    if (tid == 0) {
        for (int i = 1; i < kThreads / 32; ++i) join(m, s, s_stat[i].x, s_stat[i].y);
        a.stats[unit] = make_float2(m, s);
    }
    if (mine && mine >= low)
        for (int at = begin; at < end; at += kThreads * N) {
            float x[N];
            load<IO>(x_row, mask, mask_whole, at, a.vocab, x);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const uint64_t key = make_key(x[i], at + i);
                if (key && key >= low) s_got[atomicAdd(&s_count, 1)] = key;
            }
        }
    __syncthreads();
    const int count = s_count;
    uint64_t *out = a.keys + unit * n;
    for (int e = tid; e < count; e += kThreads) {
        const uint64_t key = s_got[e];
        int rank = 0;
        for (int i = 0; i < count; ++i) rank += s_got[i] > key;
        if (rank < n) out[rank] = key;
    }
    for (int e = count + tid; e < n; e += kThreads) out[e] = 0;
}

__global__ void __launch_bounds__(kThreads) k_beam_pick(const BeamArgs a) {
    extern __shared__ uint64_t s_got[];  // n * n, or n times a thread's heads where that is more
    __shared__ uint64_t s_sorted[kThreads], s_nth;
    __shared__ float s_norm[GDN_BEAM_MAX], s_score[GDN_BEAM_MAX];
    __shared__ uint8_t s_done[GDN_BEAM_MAX];
    __shared__ int s_count;
    const int tid = threadIdx.x, lane = tid & 31, n = a.n, W = a.W, b = blockIdx.x;
    const int lists = W * a.n_chunks;
    const uint64_t *keys = a.keys + (int64_t)b * lists * n;
    for (int w = tid >> 5; w < W; w += kThreads / 32) {
        const bool done = a.finished && a.finished[b * W + w];
        float m = -INFINITY, s = 0.f;
        if (!done)
            for (int i = lane; i < a.n_chunks; i += 32) {
                const float2 st = a.stats[(int64_t)(b * W + w) * a.n_chunks + i];
                join(m, s, st.x, st.y);
            }
#pragma unroll
        for (int step = 16; step; step >>= 1) {
            const float m2 = __shfl_xor_sync(~0u, m, step), s2 = __shfl_xor_sync(~0u, s, step);
            join(m, s, m2, s2);
        }
        if (lane == 0) s_norm[w] = m + logf(s), s_score[w] = a.scores[b * W + w], s_done[w] = done;
    }
    if (tid == 0) s_count = 0;
    __syncthreads();

    // entry j of a list, as a key of its score and its place in the search
    auto entry = [&](int list, int j) -> uint64_t {
        const int w = list / a.n_chunks;
        if (s_done[w]) return j == 0 && list == w * a.n_chunks ? make_key(s_score[w], (uint32_t)w * a.vocab) : 0;
        const uint64_t key = keys[(int64_t)list * n + j];
        if (!key) return 0;
        return make_key(s_score[w] + (key_value(key) - s_norm[w]), (uint32_t)w * a.vocab + key_index(key));
    };
    uint64_t mine = 0;
    for (int l = tid; l < lists; l += kThreads) {
        const uint64_t head = entry(l, 0);
        mine = head > mine ? head : mine;
    }
    uint64_t low = nth_largest(mine, n, s_sorted, &s_nth);
    if (lists > kThreads) {  // the n-th largest head itself, so that no more than n lists are opened
        if (mine && mine >= low)
            for (int l = tid; l < lists; l += kThreads) {
                const uint64_t head = entry(l, 0);
                if (head && head >= low) s_got[atomicAdd(&s_count, 1)] = head;
            }
        __syncthreads();
        const int count = s_count;
        for (int e = tid; e < count; e += kThreads) {
            int rank = 0;
            for (int i = 0; i < count; ++i) rank += s_got[i] > s_got[e];
            if (rank == n - 1) s_nth = s_got[e];
        }
        __syncthreads();
        low = count >= n ? s_nth : 0;
        if (tid == 0) s_count = 0;
        __syncthreads();
    }
    for (int l = tid; l < lists; l += kThreads) {
        const uint64_t head = entry(l, 0);
        if (!head || head < low) continue;
        for (int j = 0; j < n; ++j) {
            const uint64_t key = entry(l, j);
            if (key && key >= low) s_got[atomicAdd(&s_count, 1)] = key;
        }
    }
    __syncthreads();
    const int count = s_count;
    for (int e = tid; e < count; e += kThreads) {
        const uint64_t key = s_got[e];
        int rank = 0;
        for (int i = 0; i < count; ++i) rank += s_got[i] > key;
        if (rank < n) {
            const uint32_t flat = key_index(key);
            const int w = (int)(flat / (uint32_t)a.vocab);
            const int64_t at = (int64_t)b * n + rank;
            a.out_scores[at] = key_value(key);
            a.out_tokens[at] = s_done[w] ? -1 : (int)(flat - (uint32_t)w * a.vocab);
            a.out_parents[at] = w;
        }
    }
    for (int e = count + tid; e < n; e += kThreads) {
        const int64_t at = (int64_t)b * n + e;
        a.out_scores[at] = -INFINITY;
        a.out_tokens[at] = -1;
        a.out_parents[at] = e % W;
    }
}

template <typename IO> cudaError_t launch(const BeamArgs &a, cudaStream_t st) {
    const int per = (a.W * a.n_chunks + kThreads - 1) / kThreads;  // heads per thread
    const int scan = a.n * (a.chunk / kThreads) * 8, pick = a.n * (a.n > per ? a.n : per) * 8;
    cudaError_t e = cudaFuncSetAttribute(k_beam_scan<IO>, cudaFuncAttributeMaxDynamicSharedMemorySize, GDN_BEAM_MAX * kMaxPer * 8);
    if (e != cudaSuccess) return e;
    k_beam_scan<IO><<<(unsigned)((int64_t)a.B * a.W * a.n_chunks), kThreads, scan, st>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    k_beam_pick<<<(unsigned)a.B, kThreads, pick, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

// Elements of a row that one CTA takes: enough CTAs for four on every SM where the rows allow it, a vector per
// thread at least, kMaxPer elements per thread at most.
int beam_chunk(int64_t rows, int64_t vocab, gdn_dtype io) {
    const int64_t least = kThreads * (io == GDN_BF16 ? 8 : 4), most = (int64_t)kThreads * kMaxPer;
    const int64_t per_row = rows >= 152 * 4 ? 1 : rows < 1 ? 1 : (152 * 4 + rows - 1) / rows;
    int64_t c = (vocab + per_row - 1) / per_row;
    c = (c + least - 1) / least * least;
    return (int)(c < least ? least : c > most ? most : c);
}

cudaError_t launch_beam(const BeamArgs &a, gdn_dtype io, cudaStream_t st) {
    return io == GDN_BF16 ? launch<__nv_bfloat16>(a, st) : launch<float>(a, st);
}

}  // namespace gdn
