// beam.cu -- one selection of a beam search over beams and vocabulary.
//
// k_beam_scan: a CTA takes a chunk of one beam's logits, once through memory: the running maximum and sum of
// the softmax, and the chunk's n best logits.  A logit and its place make one whole number (a key: ordered
// bits of the value above, complement of the index below), so all keys differ and "the n best" needs no rule
// for ties.  The n-th largest of the threads' own maxima bounds the n-th best key from below, and at most n
// threads hold anything above it; a warp reads each of those threads' elements again (from the caches) and what
// is left, at most n times a thread's elements whatever the order of the input, is ranked by counting.
// k_beam_pick: a CTA per search joins the chunks' sums into the beams' normalisers, turns the keys into
// scores and selects in the same way.
// No result depends on the order in which threads arrive: places of collected keys do, their ranks do not.
//
// The sum is one of 2^(c (x - m)) with c = log2 e: a subtraction, a product and an exp2 per logit.  m is itself one of the
// logits, so that x - m is exact near 0 whatever the logits' size (c x - c m in one multiply-add is not: past 3e9, as
// where forbidden tokens hold -1e30, the rounding of c m alone is hundreds).  m follows the maximum only where that has
// grown by kSlack, so that the sums are hardly ever rescaled.  The normaliser is kept as a pair, its rounding beside it:
// where it is large, that is more than the scores' differences.
//
// The logits' way through memory is the floor, two bytes or four each.  64 searches of 8 beams over 131072 bf16
// logits (a seventh of them finished, 114 MB) take 31 us: about 18 of streaming, the rest the first
// reads, the selection at the end of every CTA (all come to it together) and the joining kernel.  One search of 4
// beams over 32000 takes 8.5 us, 8 of 5 over 50021 masked fp32 logits 14.6: two kernels of dependent steps.
// Asking for a row's next 16 to 128 KB ahead in L2 made none of them faster.
#include <cuda_bf16.h>

#include "common.cuh"
#include "decode.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxGot = 8192;  // n times the elements per thread, at most: keys in shared memory
constexpr int kPickKeys = 8;   // keys per thread that k_beam_pick holds in registers
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSlack = 28.f;

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

__device__ __forceinline__ float exp2_of(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// A sum of 2^(c (x - m)) and its m; an empty one is (-inf, 0).  A logit of NaN or +inf leaves s = NaN.
__device__ __forceinline__ void join(float &m, float &s, float m2, float s2) {
    const float top = fmaxf(m, m2);
    s = (m == -INFINITY ? s : s * exp2f(kLog2e * (m - top))) + (m2 == -INFINITY ? s2 : s2 * exp2f(kLog2e * (m2 - top)));
    m = top;
}
__device__ __forceinline__ void join_warp(float &m, float &s) {
    float top = m;
#pragma unroll
    for (int step = 16; step; step >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, step));
    if (m != -INFINITY) s *= exp2f(kLog2e * (m - top));
#pragma unroll
    for (int step = 16; step; step >>= 1) s += __shfl_xor_sync(~0u, s, step);
    m = top;
}

// The logarithm of the sum, m + ln s, as a rounded value and what the rounding left.  ln s = (e + f) ln 2 with the
// exponent e of s apart, so that log2f sees a number near 1.
__device__ __forceinline__ float2 normaliser(float m, float s) {
    if (!(s > 0.f)) return make_float2(s == 0.f ? -INFINITY : s, 0.f);
    // s is at least 1, up to rounding, and at most 2^61: the elements of a row times 2^(c kSlack)
    const float e = (float)((int)(__float_as_uint(s) >> 23) - 127);
    const float f = log2f(__uint_as_float((__float_as_uint(s) & 0x007FFFFFu) | 0x3F800000u));
    constexpr double ln2 = 0.69314718055994530942;
    constexpr float hi = (float)ln2, lo = (float)(ln2 - (double)hi);
    const float p = e * hi, rest = fmaf(e, hi, -p) + fmaf(e, lo, f * hi);  // p + rest = ln s
    const float a = m + p, v = a - m, r = (m - (a - v)) + (p - v) + rest;  // a + r = m + ln s
    const float sum = a + r;
    return make_float2(sum, r - (sum - a));
}

struct Nth {  // shared memory of nth_largest
    uint32_t warp[kThreads / 32];
    uint64_t heads[kThreads], answer;
    int count;
};
// The n-th largest of the 256 threads' keys (all different, but for 0) to all threads; 0 if there are fewer.
// `value` is the upper half of this thread's key, key() the whole of it, asked for where it can matter: the least of
// the maxima of n groups or more bounds the n-th largest from below, and what reaches it is ranked by counting.
template <typename Key>
__device__ __forceinline__ uint64_t nth_largest(uint32_t value, Key key, int n, Nth &sh) {
    const int groups = n <= 8 ? 1 : n <= 16 ? 2 : n <= 32 ? 4 : 8;  // of a warp
    uint32_t v = value;
#pragma unroll
    for (int step = 1; step < 32; step <<= 1) {
        const uint32_t y = __shfl_xor_sync(~0u, v, step);
        v = step * groups < 32 ? max(v, y) : min(v, y);
    }
    if ((threadIdx.x & 31) == 0) sh.warp[threadIdx.x >> 5] = v;
    if (threadIdx.x == 0) sh.answer = 0, sh.count = 0;
    __syncthreads();
    uint32_t low = ~0u;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) low = min(low, sh.warp[w]);
    if (value && value >= low) sh.heads[atomicAdd(&sh.count, 1)] = key();
    __syncthreads();
    const int count = sh.count;
    if ((int)threadIdx.x < count) {
        const uint64_t mine = sh.heads[threadIdx.x];
        int rank = 0;
        for (int i = 0; i < count; ++i) rank += sh.heads[i] > mine;
        if (rank == n - 1) sh.answer = mine;
    }
    __syncthreads();
    return sh.answer;
}
// Two fp32 operations at once, on a pair of registers
__device__ __forceinline__ uint64_t pair_of(float lo, float hi) {
    uint64_t p;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(lo), "f"(hi));
    return p;
}
__device__ __forceinline__ void halves(uint64_t p, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(p));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

template <typename IO> struct Pack;
template <> struct Pack<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ float get(const uint4 &u, int i) {
        const uint32_t w = i < 2 ? u.x : i < 4 ? u.y : i < 6 ? u.z : u.w;
        return __uint_as_float(i & 1 ? w & 0xFFFF0000u : w << 16);
    }
    static __device__ __forceinline__ float max(const uint4 &u) {  // NaN counts as nothing
        const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&u);
        const __nv_bfloat162 t = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
        return fmaxf(__low2float(t), __high2float(t));
    }
    // the words of four elements' mask bytes, a pair each
    static __device__ __forceinline__ void apply(uint32_t &lo, uint32_t &hi, uint32_t m) {
        if (!(m & 0x000000FFu)) lo = (lo & 0xFFFF0000u) | 0xFF80u;
        if (!(m & 0x0000FF00u)) lo = (lo & 0x0000FFFFu) | 0xFF800000u;
        if (!(m & 0x00FF0000u)) hi = (hi & 0xFFFF0000u) | 0xFF80u;
        if (!(m & 0xFF000000u)) hi = (hi & 0x0000FFFFu) | 0xFF800000u;
    }
    static __device__ __forceinline__ void apply(uint4 &u, const uint8_t *mask) {  // mask: 8 bytes, aligned
        const uint2 m = *reinterpret_cast<const uint2 *>(mask);
        apply(u.x, u.y, m.x);
        apply(u.z, u.w, m.y);
    }
};
template <> struct Pack<float> {
    static constexpr int N = 4;
    static constexpr uint32_t kNone = 0xFF800000u;
    static __device__ __forceinline__ float get(const uint4 &u, int i) {
        return __uint_as_float(i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w);
    }
    static __device__ __forceinline__ float max(const uint4 &u) {
        return fmaxf(fmaxf(get(u, 0), get(u, 1)), fmaxf(get(u, 2), get(u, 3)));
    }
    static __device__ __forceinline__ void apply(uint4 &u, const uint8_t *mask) {
        const uint32_t m = *reinterpret_cast<const uint32_t *>(mask);
        if (!(m & 0x000000FFu)) u.x = kNone;
        if (!(m & 0x0000FF00u)) u.y = kNone;
        if (!(m & 0x00FF0000u)) u.z = kNone;
        if (!(m & 0xFF000000u)) u.w = kNone;
    }
};

// One beam's logits as vectors on 16-byte boundaries: the first may begin before the row, the last end after it
template <typename IO, bool MASK> struct Row {
    static constexpr int N = Pack<IO>::N;
    const IO *x;
    const uint8_t *mask;
    bool mask_whole;  // a vector's mask bytes are aligned too
    int vocab;

    // elements [at, at + N), all in the row; what is masked is -inf
    __device__ __forceinline__ uint4 inside(int at) const {
        uint4 u = *reinterpret_cast<const uint4 *>(x + at);
        if (MASK) {
            if (mask_whole) {
                Pack<IO>::apply(u, mask + at);
            } else {
                alignas(8) uint32_t m[2] = {0, 0};
#pragma unroll
                for (int i = 0; i < N; ++i) m[i >> 2] |= (uint32_t)mask[at + i] << (8 * (i & 3));
                Pack<IO>::apply(u, reinterpret_cast<const uint8_t *>(m));
            }
        }
        return u;
    }
    // elements [at, at + N); what is outside too is -inf
    __device__ __forceinline__ uint4 load(int at) const { return at >= 0 && at + N <= vocab ? inside(at) : edge(at); }
    __device__ __noinline__ uint4 edge(int at) const {
        IO v[N];
#pragma unroll
        for (int i = 0; i < N; ++i)
            v[i] = at + i >= 0 && at + i < vocab && (!MASK || mask[at + i]) ? x[at + i] : from_f<IO>(-INFINITY);
        uint4 u;
        memcpy(&u, v, 16);
        return u;
    }
};

// Eight CTAs per SM with three vectors on the way per thread, or six with four where a mask takes registers too: 512
// rows of 131072 bf16 logits in two chunks each take 32 us (31.7 before x - m was formed first), in six CTAs per SM
// 37.7, because 1024 do not fit at once; masked with eight 16.4 instead of 14.4 for 40 rows of 50021.
template <typename IO, bool MASK> __global__ void __launch_bounds__(kThreads, MASK ? 6 : 8) k_beam_scan(const BeamArgs a) {
    constexpr int N = Pack<IO>::N, STEP = kThreads * N, DEEP = MASK ? 4 : 3;
    extern __shared__ uint64_t s_got[];  // n times the elements per thread
    __shared__ Nth sh;
    __shared__ float2 s_stat[kThreads / 32];
    __shared__ int s_count, s_list[GDN_BEAM_MAX], s_listed;
    const int tid = threadIdx.x, lane = tid & 31, n = a.n;
    const int row = blockIdx.x / a.n_chunks, chunk = blockIdx.x - row * a.n_chunks;
    wait_for_previous();
    if (a.finished && a.finished[row]) return;
    const int b = row / a.W, w = row - b * a.W;
    Row<IO, MASK> x;
    x.x = static_cast<const IO *>(a.logits) + b * a.logits_batch + w * a.logits_beam;
    x.mask = MASK ? a.mask + b * a.mask_batch + w * a.mask_beam : nullptr;
    x.vocab = a.vocab;
    const int shift = (int)((reinterpret_cast<uintptr_t>(x.x) & 15) / sizeof(IO));
    x.mask_whole = ((reinterpret_cast<uintptr_t>(x.mask) - shift) & (N - 1)) == 0;
    const int first = chunk * a.chunk - shift, begin = first + tid * N;
    const int end = min(first + a.chunk, a.vocab);

    float best = -INFINITY, m = 0.f;  // m: at most best, 0 before there is one
    uint64_t sum = 0, neg_m = 0;      // pairs: the even and the odd elements' sums; -m twice
    const uint64_t c2 = pair_of(kLog2e, kLog2e);
    int best_at = begin;
    auto take = [&](const uint4 &u, int at) {
        const float top = Pack<IO>::max(u);
        if (top > best) {
            if (best == -INFINITY || top - m > kSlack) {
                const float f = best == -INFINITY ? 1.f : exp2_of(kLog2e * (m - top));
                sum = mul2(sum, pair_of(f, f));
                m = top, neg_m = pair_of(-m, -m);
            }
            best = top, best_at = at;
        }
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            float e0, e1;
            halves(mul2(add2(pair_of(Pack<IO>::get(u, i), Pack<IO>::get(u, i + 1)), neg_m), c2), e0, e1);
            sum = add2(sum, pair_of(exp2_of(e0), exp2_of(e1)));
        }
    };
    // a row's first vector may begin before it and its last one end after it: all others are read as they are
    int at = begin;
    if (at < 0) take(x.edge(at), at), at += STEP;
    const int whole = min(end, a.vocab - N + 1);
    for (; at + (DEEP - 1) * STEP < whole; at += DEEP * STEP) {
        uint4 u[DEEP];
#pragma unroll
        for (int j = 0; j < DEEP; ++j) u[j] = x.inside(at + j * STEP);
#pragma unroll
        for (int j = 0; j < DEEP; ++j) take(u[j], at + j * STEP);
    }
#pragma unroll 1  // its code, unrolled, costs one search of 4 beams 0.7 us
    for (; at < whole; at += STEP) take(x.inside(at), at);
    if (at < end) take(x.edge(at), at);
    float s, s_odd, ms = best == -INFINITY ? -INFINITY : m;
    halves(sum, s, s_odd);
    s += s_odd;
    join_warp(ms, s);
    if (tid == 0) s_count = 0, s_listed = 0;
    if (lane == 0) s_stat[tid >> 5] = make_float2(ms, s);
    uint64_t mine = 0;
    const uint64_t low = nth_largest(
        best > -INFINITY ? ordered(best) : 0u,
        [&] {
            const uint4 u = x.load(best_at);
#pragma unroll
            for (int i = N - 1; i >= 0; --i)
                if (Pack<IO>::get(u, i) == best) mine = make_key(best, best_at + i);
            return mine;
        },
        n, sh);
    const int64_t unit = blockIdx.x;
    if (tid < 32) {
        const float2 st = lane < kThreads / 32 ? s_stat[lane] : make_float2(-INFINITY, 0.f);
        ms = st.x, s = st.y;
        join_warp(ms, s);
        if (lane == 0) a.stats[unit] = make_float2(ms, s);
    }
    if (mine && mine >= low) s_list[atomicAdd(&s_listed, 1)] = tid;
    const float low_value = low ? key_value(low) : -INFINITY;
    __syncthreads();
    for (int e = tid >> 5; e < s_listed; e += kThreads / 32)
        for (int v = first + s_list[e] * N + lane * STEP; v < end; v += 32 * STEP) {
            const uint4 u = x.load(v);
            if (Pack<IO>::max(u) < low_value) continue;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const uint64_t key = make_key(Pack<IO>::get(u, i), v + i);
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
    extern __shared__ uint64_t s_got[];
    __shared__ Nth sh;
    __shared__ float2 s_norm[GDN_BEAM_MAX];
    __shared__ float s_score[GDN_BEAM_MAX];
    __shared__ uint8_t s_done[GDN_BEAM_MAX];
    __shared__ int s_count;
    const int tid = threadIdx.x, lane = tid & 31, n = a.n, W = a.W, b = blockIdx.x;
    const int lists = W * a.n_chunks, total = lists * n;
    // quotients by n and n_chunks as products: exact below 2^20 over the divisor, and few keys are far below that
    const uint32_t by_n = (1u << 20) / (uint32_t)n + 1, by_chunks = (1u << 20) / (uint32_t)a.n_chunks + 1;
    wait_for_previous();
    const uint64_t *keys = a.keys + (int64_t)b * total;
    if (tid == 0) s_count = 0;
    // Few keys are read once, by whom they will be held: 14.5 us against 16.4 by the heads of the lists for 8 searches
    // of 5 beams with 10 wanted, 29.9 against 31.9 for 64 of 8; more would take registers that few searches pay for.
    const bool few = total <= kPickKeys * kThreads;
    uint64_t held[kPickKeys];
    if (few) {  // all reads before anything waits for one
#pragma unroll
        for (int i = 0; i < kPickKeys; ++i) held[i] = tid + i * kThreads < total ? __ldcg(keys + tid + i * kThreads) : 0;
    }
    const int mine_w = kThreads - 1 - tid;  // not the warps that begin with the beams' sums
    const float score = mine_w < W ? a.scores[b * W + mine_w] : 0.f;
    const uint8_t done = mine_w < W && a.finished ? a.finished[b * W + mine_w] : 0;
    for (int w = tid >> 5; w < W; w += kThreads / 32) {  // what a finished beam left there is not used
        float m = -INFINITY, s = 0.f;
        for (int i = lane; i < a.n_chunks; i += 32) {
            const float2 st = __ldcg(a.stats + (int64_t)(b * W + w) * a.n_chunks + i);
            join(m, s, st.x, st.y);
        }
        join_warp(m, s);
        if (lane == 0) s_norm[w] = normaliser(m, s);
    }
    if (mine_w < W) s_score[mine_w] = score, s_done[mine_w] = done != 0;
    __syncthreads();

    // key j of a list, as a key of its score and its place in the search
    auto entry = [&](int w, int list, int j, uint64_t key) -> uint64_t {
        if (s_done[w]) return j == 0 && list == w * a.n_chunks ? make_key(s_score[w], (uint32_t)w * a.vocab) : 0;
        if (!key) return 0;
        return make_key(s_score[w] + ((key_value(key) - s_norm[w].x) - s_norm[w].y), (uint32_t)w * a.vocab + key_index(key));
    };
    auto read = [&](int list, int j) { return entry(list / a.n_chunks, list, j, __ldcg(keys + (int64_t)list * n + j)); };
    uint64_t mine = 0;
    if (few) {
#pragma unroll
        for (int i = 0; i < kPickKeys; ++i) {
            const uint32_t e = tid + i * kThreads, list = e * by_n >> 20, w = list * by_chunks >> 20;
            if ((int)e < total) held[i] = entry(w, list, e - list * n, held[i]);
            mine = held[i] > mine ? held[i] : mine;
        }
        const uint64_t low = nth_largest((uint32_t)(mine >> 32), [&] { return mine; }, n, sh);
        if (mine >= low)
#pragma unroll
            for (int i = 0; i < kPickKeys; ++i)
                if (held[i] && held[i] >= low) s_got[atomicAdd(&s_count, 1)] = held[i];
    } else {  // by the heads of the sorted lists
        for (int l = tid; l < lists; l += kThreads) {
            const uint64_t head = read(l, 0);
            mine = head > mine ? head : mine;
        }
        uint64_t low = nth_largest((uint32_t)(mine >> 32), [&] { return mine; }, n, sh);
        if (lists > kThreads) {  // the n-th largest head itself, so that no more than n lists are opened
            if (mine && mine >= low)
                for (int l = tid; l < lists; l += kThreads) {
                    const uint64_t head = read(l, 0);
                    if (head && head >= low) s_got[atomicAdd(&s_count, 1)] = head;
                }
            __syncthreads();  // all have the first bound
            if (tid == 0) sh.answer = 0;
            __syncthreads();
            const int count = s_count;
            for (int e = tid; e < count; e += kThreads) {
                int rank = 0;
                for (int i = 0; i < count; ++i) rank += s_got[i] > s_got[e];
                if (rank == n - 1) sh.answer = s_got[e];
            }
            __syncthreads();
            low = sh.answer;
            if (tid == 0) s_count = 0;
            __syncthreads();
        }
        for (int l = tid; l < lists; l += kThreads) {
            const uint64_t head = read(l, 0);
            if (!head || head < low) continue;
            for (int j = 0; j < n; ++j) {
                const uint64_t key = read(l, j);
                if (key && key >= low) s_got[atomicAdd(&s_count, 1)] = key;
            }
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

template <typename IO, bool MASK> cudaError_t scan(const BeamArgs &a, int lists, cudaStream_t st) {
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(k_beam_scan<IO, MASK>, kMaxGot * 8, done);
    if (e != cudaSuccess) return e;
    return launch_behind(k_beam_scan<IO, MASK>, dim3((unsigned)(a.B * lists)), kThreads, (size_t)a.n * (a.chunk / kThreads) * 8, st, a);
}

template <typename IO> cudaError_t launch(const BeamArgs &a, cudaStream_t st) {
    const int lists = a.W * a.n_chunks;
    cudaError_t e = a.mask ? scan<IO, true>(a, lists, st) : scan<IO, false>(a, lists, st);
    if (e != cudaSuccess) return e;
    // keys collected at once: n threads' or n lists', or the heads of n threads' lists
    const int per = lists * a.n <= kPickKeys * kThreads ? kPickKeys : a.n, heads = (lists + kThreads - 1) / kThreads;
    return launch_behind(k_beam_pick, dim3((unsigned)a.B), kThreads, (size_t)a.n * (per > heads ? per : heads) * 8, st, a);
}

}  // namespace

// Elements of a row that one CTA takes: enough CTAs for six on every SM where the rows allow it (64 searches of 8
// beams over 131072 take 31 us with four or six wanted, 35 with eight and 34 to 41 with more: each CTA selects), a vector per thread at least, and no more than the keys in shared memory allow.  Equal chunks: up to seven
// elements are added for a row that begins inside a vector.
int beam_chunk(int64_t rows, int64_t vocab, int64_t n, gdn_dtype io) {
    const int64_t wanted = 152 * 6, least = kThreads * (io == GDN_BF16 ? 8 : 4), per = kMaxGot / n < 512 ? kMaxGot / n : 512;
    const int64_t most = kThreads * per / least * least;
    int64_t chunks = rows < 1 ? 1 : (wanted + rows - 1) / rows;
    const int64_t fewest = (vocab + 7 + most - 1) / most;
    if (chunks < fewest) chunks = fewest;
    return (int)(((vocab + 7 + chunks - 1) / chunks + least - 1) / least * least);
}

cudaError_t launch_beam(const BeamArgs &a, gdn_dtype io, cudaStream_t st) {
    return io == GDN_BF16 ? launch<__nv_bfloat16>(a, st) : launch<float>(a, st);
}

}  // namespace gdn
