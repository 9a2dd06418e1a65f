// sample.cu -- one token for each row of logits, by temperature, top-k, top-p and min-p, from a given random number.
//
// A row's candidates in order, best first and equal ones by the lower token, are its keys in descending order (ordered
// bits of the logit above, complement of the token below: all keys differ).  Each filter keeps a beginning of that order,
// so that what is kept is {key >= cut} for one cut, and the token is found by running through the vocabulary.
//
// Shares are whole numbers, w = 2^(42 + t) with t = (x - m) log2(e) / temperature and m the largest logit: their sums are
// the same in every order, by atomics too, and a cut lies where it lies.  t is a pair of fp32 (x - m with what its
// rounding leaves, times the constant as a pair), 2^t a table of 64 steps an octave times 1 + e with e in fp32: off by
// 2^-31 of itself, a border is mistaken about once in 10^9 / (tokens of that size).
//
// The CTAs of a cluster share a row; each reads its slice once and keeps it in shared memory, -inf for what the mask
// forbids.  A cut is found by bins of 1/8 octave of t, whose running sum (of w, or of tokens for top-k) says in which bin
// it lies.  For top-k they take at first the best of every thread's elements alone: what these reach, all reach, so that
// the true cut lies in that bin or before it.  If no more than kList tokens do, those are collected and sorted, and the
// rest of the work is done on that list.  If they are too many, what lies in the cut's bin (or in one of kSub parts of
// it) is collected and sorted to find the cut; where even that is too much for the list (many equal logits), the cut is
// searched for by bisection, over the logit and then over the tokens that share it.
//
// Waiting bounds it, not memory: the steps are separated by barriers.  A list of up to 64 tokens takes 23 of a CTA and four of a
// cluster, one of 256 tokens 43, of which its two sorts by one CTA (best first, then by token) have 8 and 28; the rest of the
// row's CTAs wait.  One row of 32000 bf16 logits with top-k and top-p 12 us; 8 masked rows of 50021
// fp32, top-p and min-p, 31 us (top-p over all of the vocabulary is found by bins, a list and a second pass); 64 rows of
// 131072, all filters, 21 us, 0.8 TB/s, of which reading takes some 5.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include "common.cuh"
#include "decode.h"

namespace gdn {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kOctave = 8, kBins = 44 * kOctave;  // w = 0 from t = -43 on
constexpr int kSub = kThreads;
constexpr int kList = 1024;
constexpr int kSlice = 1 << 17;  // elements of a CTA for which the next cluster size is taken
// A slice has a few more where the longest row begins off a 16-byte boundary: a bin's sum of 14-bit parts, and of what w has
// from bit 28 on, 2^14 at most, stays within 32 bits all the same
static_assert((int64_t)kMaxCluster * kSlice >= GDN_SAMPLE_VOCAB_MAX && ((int64_t)(kSlice + 32) << 14) <= INT64_C(1) << 32, "sums of parts");
constexpr int kCache = 96 << 10; // bytes of shared memory for the slice; larger ones are read again in every pass
static_assert(kBins <= kThreads, "a thread per bin");
constexpr int kShift = 42;

__device__ __forceinline__ uint32_t ordered(float x) {  // larger for larger x; +0 and -0 alike
    const uint32_t u = __float_as_uint(x + 0.f);
    return u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t u) {
    return __uint_as_float(u ^ ((u >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}
__device__ __forceinline__ uint64_t make_key(float x, uint32_t token) { return (uint64_t)ordered(x) << 32 | (0xFFFFFFFFu - token); }
__device__ __forceinline__ uint32_t key_token(uint64_t key) { return 0xFFFFFFFFu - (uint32_t)key; }

// 2^(42 + j / 64), j = -32 .. 32, by the series of the exponential
struct Powers {
    uint64_t of[65];
};
constexpr Powers powers() {
    Powers p = {};
    for (int j = -32; j <= 32; ++j) {
        const double x = j / 64. * 0.69314718055994530942;
        double term = 1., sum = 1.;
        for (int i = 1; i < 24; ++i) term *= x / i, sum += term;
        p.of[j + 32] = (uint64_t)(sum * (double)(1ull << kShift) + 0.5);
    }
    return p;
}
__constant__ constexpr Powers kPowers = powers();

struct Sums {
    uint64_t w;
    uint32_t n;
};
__device__ __forceinline__ Sums operator+(Sums a, Sums b) { return {a.w + b.w, a.n + b.n}; }
__device__ __forceinline__ uint64_t shfl_up64(uint64_t x, int d) { return __shfl_up_sync(~0u, (unsigned long long)x, d); }
__device__ __forceinline__ uint64_t shfl_xor64(uint64_t x, int d) { return __shfl_xor_sync(~0u, (unsigned long long)x, d); }

struct Shared {
    uint32_t part[3][kSub];  // sums of w by bins, in parts: bits 0 .. 13, 14 .. 27, 28 ..
    uint32_t count[kSub];
    uint64_t total[kSub];    // of either, as whole numbers
    uint64_t key[kList], w[kList];
    uint64_t table[65];  // 2^(42 + j / 64), j = -32 .. 32
    uint64_t warp_w[kWarps];
    uint32_t warp_n[kWarps];
    uint64_t best;       // of the CTA's slice; all ones where there is what must not be
    Sums sum[2];         // what the CTA adds to a sum over the cluster
    uint64_t warp_kept[kWarps];
    uint32_t listed;     // entries of the list (the first CTA's)
    uint64_t cut;        // found by the first CTA
    int at_bin;
    uint64_t before, here;  // what lies in the bins before it, and in it
    float warp_f[kWarps], most;  // how many tokens these and that bin have at most, where w was summed
};
// floor or ceil of f x for an f from [0, 1]
__device__ __forceinline__ uint64_t part_of(float f, uint64_t x, bool up) {
    const uint32_t u = __float_as_uint(f);
    const int e = max((int)(u >> 23), 1);  // f = c 2^(e - 150)
    const uint64_t c = (u & 0x7FFFFFu) | (u >> 23 ? 0x800000u : 0u);
    const uint64_t lo = c * x, hi = __umul64hi(c, x);
    const int down = 150 - e;  // 23 .. 149
    uint64_t whole, rest;
    if (down < 64) whole = hi << (64 - down) | lo >> down, rest = lo << (64 - down);
    else if (down < 128) whole = down == 64 ? hi : hi >> (down - 64), rest = lo | (down == 64 ? 0 : hi << (128 - down));
    else whole = 0, rest = lo | hi;
    return whole + (up && rest ? 1 : 0);
}


template <typename IO> struct Sampler {
    static constexpr int VEC = 16 / (int)sizeof(IO);
    Shared &s;
    const cg::cluster_group cluster;
    const IO *x;          // the row
    const uint8_t *mask;  // the row's, or nullptr
    uint4 *cache;         // the slice, or nullptr where it does not fit
    int vocab, v0, v1;    // this CTA's vectors; vector v has the elements VEC v - skew ..
    int skew;             // elements by which the row begins behind a 16-byte boundary
    bool mask16;          // the mask's bytes of a vector can be read at once
    float m, c_hi, c_lo;
    int turn;

    // Vector v as it lies in memory, -inf in place of what the mask forbids and of what lies outside the row
    __device__ __forceinline__ uint4 fetch(int v) const {
        const int at = v * VEC - skew;
        uint4 raw;
        IO *e = reinterpret_cast<IO *>(&raw);
        if (at >= 0 && at + VEC <= vocab) {
            raw = __ldg(reinterpret_cast<const uint4 *>(x + at));
            if (mask) {
                uint8_t ok[VEC];
                if (mask16) {
                    if constexpr (VEC == 8) *reinterpret_cast<uint2 *>(ok) = __ldg(reinterpret_cast<const uint2 *>(mask + at));
                    else *reinterpret_cast<uint32_t *>(ok) = __ldg(reinterpret_cast<const uint32_t *>(mask + at));
                } else {
#pragma unroll
                    for (int i = 0; i < VEC; ++i) ok[i] = mask[at + i];
                }
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    if (!ok[i]) e[i] = from_f<IO>(-INFINITY);
            }
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                e[i] = at + i >= 0 && at + i < vocab && (!mask || mask[at + i]) ? x[at + i] : from_f<IO>(-INFINITY);
        }
        return raw;
    }
    // f(x, token) for the elements of a vector; those that are forbidden or outside the row have x = -inf
    template <typename F> __device__ __forceinline__ void elements(uint4 raw, int v, F f) const {
        const IO *e = reinterpret_cast<const IO *>(&raw);
#pragma unroll
        for (int i = 0; i < VEC; ++i) f(to_f<IO>(e[i]), v * VEC - skew + i);
    }
    template <typename F> __device__ __forceinline__ void vector(int v, F f) const { elements(cache ? cache[v - v0] : fetch(v), v, f); }
    // Warps have consecutive parts of the slice
    __device__ __forceinline__ void warp_part(int warp, int &a, int &b) const {
        const int each = (v1 - v0 + kWarps - 1) / kWarps;
        a = min(v1, v0 + warp * each), b = min(v1, a + each);
    }
    template <typename F> __device__ __forceinline__ void each(F f) const {
        int a, b;
        warp_part(threadIdx.x >> 5, a, b);
        a += threadIdx.x & 31;
        if (cache) {
#pragma unroll 1
            for (int v = a; v < b; v += 32) elements(cache[v - v0], v, f);
        } else {
#pragma unroll 1
            for (int v = a; v < b; v += 64) {  // two vectors on their way
                const uint4 first = fetch(v);
                uint4 second;
                if (v + 32 < b) second = fetch(v + 32);
                elements(first, v, f);
                if (v + 32 < b) elements(second, v + 32, f);
            }
        }
    }
    // The first pass: into the cache too
    template <typename F> __device__ __forceinline__ void each_first(F f) const {
        int a, b;
        warp_part(threadIdx.x >> 5, a, b);
        a += threadIdx.x & 31;
#pragma unroll 1
        for (int v = a; v < b; v += 128) {
            uint4 raw[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (v + 32 * i < b) raw[i] = fetch(v + 32 * i);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (v + 32 * i < b) {
                    if (cache) cache[v + 32 * i - v0] = raw[i];
                    elements(raw[i], v + 32 * i, f);
                }
        }
    }

    __device__ __forceinline__ float t_of(float y) const { return (y - m) * c_hi; }
    // In which bin; not less for a smaller logit.  kBins: w is 0
    __device__ __forceinline__ int bin_of(float y) const {
        const float t = -t_of(y) * kOctave;
        return t < (float)(43 * kOctave + 1) ? (int)t : kBins;
    }
    __device__ __forceinline__ int sub_of(float y, int bin) const {
        return min(kSub - 1, (int)((-t_of(y) * kOctave - (float)bin) * kSub));
    }
    // t as a pair
    __device__ __forceinline__ float t_pair(float y, float &low) const {
        const float d = y - m, z = d - y, rest = (y - (d - z)) - (m + z);
        const float t = d * c_hi;
        low = fmaf(d, c_hi, -t) + fmaf(d, c_lo, rest * c_hi);
        return t;
    }
    __device__ __forceinline__ uint64_t weight(float y) const {
        float low;
        const float t = t_pair(y, low);
        if (!(t > -43.5f)) return 0;
        const float n = rintf(t), f = t - n;
        const float j = rintf(f * 64.f), g = fmaf(j, -1.f / 64.f, f) + low;
        // 2^g - 1, |g| < 1/127
        const float e = g * fmaf(g, fmaf(g, fmaf(g, 0.009618129f, 0.055504109f), 0.240226507f), 0.693147181f);
        const uint64_t base = s.table[(int)j + 32];
        const int64_t w = (int64_t)base + (((int64_t)(uint32_t)(base >> 11) * (int64_t)__float2int_rn(e * (float)(1ull << 38))) >> 27);
        const int down = -(int)n;
        return down < 64 ? (uint64_t)w >> down : 0;
    }

    __device__ __forceinline__ Sums block_sum(Sums a) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
        for (int d = 16; d; d >>= 1) a.w += shfl_xor64(a.w, d), a.n += __shfl_xor_sync(~0u, a.n, d);
        __syncthreads();
        if (lane == 0) s.warp_w[warp] = a.w, s.warp_n[warp] = a.n;
        __syncthreads();
        Sums all = {0, 0};
        for (int i = 0; i < kWarps; ++i) all = all + Sums{s.warp_w[i], s.warp_n[i]};
        return all;
    }
    // Sums over the cluster, to all threads; two turns' parts are apart, so that one sync serves each
    __device__ __forceinline__ Sums row_sum(Sums a) {
        a = block_sum(a);
        if (threadIdx.x == 0) s.sum[turn] = a;
        cluster.sync();
        return read_sum();
    }
    __device__ __forceinline__ Sums read_sum() {  // of what lies in sum[turn]
        const unsigned r = threadIdx.x & 31;
        Sums all = {0, 0};
        if (r < cluster.num_blocks()) all = *cluster.map_shared_rank(&s.sum[turn], r);
#pragma unroll
        for (int d = kMaxCluster / 2; d; d >>= 1) all.w += shfl_xor64(all.w, d), all.n += __shfl_xor_sync(~0u, all.n, d);
        all.w = __shfl_sync(~0u, (unsigned long long)all.w, 0), all.n = __shfl_sync(~0u, all.n, 0);
        turn ^= 1;
        return all;
    }

    // The CTA's bins as whole numbers, for locate() behind the next sync
    __device__ __forceinline__ void close_bins(bool by_count) {
        __syncthreads();
        const int i = threadIdx.x;
        s.total[i] = by_count ? s.count[i] : ((uint64_t)s.part[2][i] << 28) + ((uint64_t)s.part[1][i] << 14) + s.part[0][i];
    }
    // Where in the bins (over the cluster; a thread for each) the running sum reaches `need`, of w or of tokens: at_bin
    // (kThreads: nowhere), what lies before it and in it, and how many tokens that are at most.  Bins of t only, where w was
    // summed: a token of bin i has 2^(42 - (i + 1) / kOctave) at least.
    __device__ __forceinline__ void locate(bool by_count, uint64_t need) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        uint64_t part[kMaxCluster], mine = 0;
        const unsigned ranks = cluster.num_blocks();
#pragma unroll
        for (unsigned r = 0; r < kMaxCluster; ++r) part[r] = r < ranks ? cluster.map_shared_rank(&s, r)->total[threadIdx.x] : 0;
#pragma unroll
        for (unsigned r = 0; r < kMaxCluster; ++r) mine += part[r];
        const float most = by_count ? 0.f : (float)mine * exp2f((float)(threadIdx.x + 1) * (1.f / kOctave) - (float)kShift) * 1.001f;
        uint64_t run = mine;
        float tokens = most;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint64_t y = shfl_up64(run, d);
            const float f = __shfl_up_sync(~0u, tokens, d);
            if (lane >= d) run += y, tokens += f;
        }
        __syncthreads();
        if (lane == 31) s.warp_w[warp] = run, s.warp_f[warp] = tokens;
        if (threadIdx.x == 0) s.at_bin = kThreads;
        __syncthreads();
        for (int i = 0; i < warp; ++i) run += s.warp_w[i], tokens += s.warp_f[i];
        if (run - mine < need && run >= need) s.at_bin = threadIdx.x, s.before = run - mine, s.here = mine, s.most = by_count ? (float)run : tokens;
        __syncthreads();
    }
    __device__ __forceinline__ void clear_bins() {
        s.count[threadIdx.x] = s.part[0][threadIdx.x] = s.part[1][threadIdx.x] = s.part[2][threadIdx.x] = 0;
        __syncthreads();
    }
    __device__ __forceinline__ void add(int bin, uint64_t w) {
        atomicAdd(&s.part[0][bin], (uint32_t)w & 0x3FFFu);
        atomicAdd(&s.part[1][bin], (uint32_t)(w >> 14) & 0x3FFFu);
        if (w >> 28) atomicAdd(&s.part[2][bin], (uint32_t)(w >> 28));
    }
    // Into the first CTA's list
    __device__ __forceinline__ void collect(uint64_t key) {
        Shared *first = cluster.map_shared_rank(&s, 0);
        const uint32_t at = atomicAdd(&first->listed, 1u);
        if (at < kList) first->key[at] = key;
    }
    // Sorts the first n entries of the list: descending keys.  E entries a thread, those of tid + 512 e; partners less than
    // a warp apart meet by shuffles.  Warps without entries stay out of it.
    template <int E> __device__ __forceinline__ void sort_entries(int n, int size) {
        uint64_t k[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int i = threadIdx.x + e * kThreads;
            k[e] = i < n ? s.key[i] : 0;
        }
        const int threads = min(size, kThreads);
        if ((int)threadIdx.x >= threads) {
            __syncthreads();
            return;
        }
        auto meet = [&] { asm volatile("bar.sync 1, %0;" ::"r"(threads) : "memory"); };
        meet();
        for (int g = 2; g <= size; g <<= 1)
            for (int j = g >> 1; j; j >>= 1) {
                if (E == 2 && j == kThreads) {
                    if (k[0] < k[E - 1]) {  // the last merge: descending
                        const uint64_t y = k[0];
                        k[0] = k[E - 1], k[E - 1] = y;
                    }
                    continue;
                }
                if (j >= 32) {
#pragma unroll
                    for (int e = 0; e < E; ++e) s.key[threadIdx.x + e * kThreads] = k[e];
                    meet();
                }
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const int i = threadIdx.x + e * kThreads;
                    const uint64_t y = j >= 32 ? s.key[i ^ j] : shfl_xor64(k[e], j);
                    const bool keep_larger = ((i & g) == 0) == ((i & j) == 0);
                    k[e] = keep_larger ? max(k[e], y) : min(k[e], y);
                }
                if (j >= 32) meet();
            }
#pragma unroll
        for (int e = 0; e < E; ++e) s.key[threadIdx.x + e * kThreads] = k[e];
        __syncthreads();
    }
    __device__ __forceinline__ void sort_list(int n) {
        int size = 32;
        while (size < n) size <<= 1;
        if (size <= kThreads) sort_entries<1>(n, size);
        else sort_entries<2>(n, size);
    }
    // w[i] of the list's n entries becomes the running sum of its tokens' shares
    __device__ __forceinline__ void scan_list(int n) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        uint64_t base = 0;
        for (int from = 0; from < n; from += kThreads) {
            const int i = from + threadIdx.x;
            uint64_t run = i < n ? weight(unordered((uint32_t)(s.key[i] >> 32))) : 0;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const uint64_t y = shfl_up64(run, d);
                if (lane >= d) run += y;
            }
            __syncthreads();
            if (lane == 31) s.warp_w[warp] = run;
            __syncthreads();
            run += base;
            for (int j = 0; j < kWarps; ++j) {
                if (j < warp) run += s.warp_w[j];
                base += s.warp_w[j];
            }
            if (i < n) s.w[i] = run;
        }
        __syncthreads();
    }
    // The first place of the list where the running sum reaches need, n where there is none
    __device__ __forceinline__ int place(int n, uint64_t need) const {
        int lo = 0, hi = n;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (s.w[mid] >= need) hi = mid;
            else lo = mid + 1;
        }
        return lo;
    }

    // The cut in a bin, as locate() left it: the key at which, among the keys from `floor` on, the running sum reaches need
    __device__ __forceinline__ uint64_t cut_in(bool by_count, uint64_t need, uint64_t floor) {
        const int bin = s.at_bin;
        need -= s.before;
        const float most = by_count ? (float)s.here : (float)s.here * exp2f((float)(bin + 1) * (1.f / kOctave) - (float)kShift) * 1.001f;
        int sub = -1;  // all of the bin
        cluster.sync();  // all have read the bins
        if (threadIdx.x == 0) s.listed = 0;
        if (most > (float)kList) {
            clear_bins();
            each([&](float y, int token) {
                if (bin_of(y) != bin || make_key(y, token) < floor) return;
                if (by_count) atomicAdd(&s.count[sub_of(y, bin)], 1u);
                else add(sub_of(y, bin), weight(y));
            });
            close_bins(by_count);
            cluster.sync();
            locate(by_count, need);
            sub = s.at_bin;
            if (sub == kThreads) return floor;  // all of it
            need -= s.before;
        } else {
            cluster.sync();
        }
        uint32_t n = 0;
        each([&](float y, int token) {
            const uint64_t key = make_key(y, token);
            if (bin_of(y) == bin && key >= floor && (sub < 0 || sub_of(y, bin) == sub)) collect(key), ++n;
        });
        n = row_sum({0, n}).n;
        if (n <= kList) {
            if (cluster.block_rank() == 0) {
                sort_list((int)n);
                if (!by_count) scan_list((int)n);
                if (threadIdx.x == 0) s.cut = s.key[by_count ? min((int)need, (int)n) - 1 : min(place((int)n, need), (int)n - 1)];
            }
            cluster.sync();
            return cluster.map_shared_rank(&s, 0)->cut;
        }
        // the largest logit from which on the sum reaches need
        uint32_t lo = 0, hi = 0xFFFFFFFFu;
        Sums above = {0, 0};  // of what is larger than the logit
        while (lo < hi) {
            const uint32_t mid = lo + (hi - lo) / 2 + 1;
            Sums a = {0, 0};
            each([&](float y, int token) {
                if (ordered(y) >= mid && bin_of(y) == bin && make_key(y, token) >= floor && (sub < 0 || sub_of(y, bin) == sub))
                    a.w += weight(y), ++a.n;
            });
            a = row_sum(a);
            if ((by_count ? a.n : a.w) >= need) lo = mid;
            else hi = mid - 1, above = a;
        }
        const float value = unordered(lo);
        const uint64_t w = by_count ? 1 : weight(value);
        const uint64_t left = need - (by_count ? above.n : above.w);
        const uint64_t ties = w ? (left + w - 1) / w : 1;
        uint32_t first = 0, last = (uint32_t)vocab - 1;  // the token with which there are so many
        while (first < last) {
            const uint32_t mid = first + (last - first) / 2;
            Sums a = {0, 0};
            each([&](float y, int token) {
                if (ordered(y) == lo && (uint32_t)token <= mid && make_key(y, token) >= floor) ++a.n;
            });
            a = row_sum(a);
            if (a.n >= ties) last = mid;
            else first = mid + 1;
        }
        return max(floor, make_key(value, first));
    }
};

template <typename IO> __global__ void __launch_bounds__(kThreads, 2) k_sample(const __grid_constant__ SampleArgs a) {
    extern __shared__ uint4 sample_cache[];
    __shared__ Shared s;
    const cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
    const int row = blockIdx.x / ranks, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    Sampler<IO> z{s, cluster};
    z.x = static_cast<const IO *>(a.logits) + row * a.logits_row;
    z.mask = a.mask ? a.mask + row * a.mask_row : nullptr;
    z.vocab = a.vocab, z.turn = 0;
    z.skew = (int)((reinterpret_cast<uintptr_t>(z.x) & 15) / sizeof(IO));
    z.mask16 = z.mask && ((reinterpret_cast<uintptr_t>(z.mask) - z.skew) & (Sampler<IO>::VEC - 1)) == 0;
    const int vectors = (a.vocab + z.skew + Sampler<IO>::VEC - 1) / Sampler<IO>::VEC;
    const int slice = (vectors + ranks - 1) / ranks;
    z.v0 = min(vectors, rank * slice), z.v1 = min(vectors, z.v0 + slice);
    z.cache = a.cached ? sample_cache : nullptr;
    wait_for_previous();
    const float heat = a.temperatures ? a.temperatures[row] : a.temperature;
    const int top_k = a.top_ks ? a.top_ks[row] : a.top_k;
    const float top_p = a.top_ps ? a.top_ps[row] : a.top_p;
    const float given_min_p = a.min_ps ? a.min_ps[row] : a.min_p, min_p = fminf(given_min_p, 1.f);
    const bool none = !(heat >= 0.f) || heat == INFINITY || isnan(top_p) || isnan(given_min_p);
    float u = a.u[row];
    u = u >= 0.f ? fminf(u, 0.99999994f) : 0.f;
    if (tid == 0) s.listed = 0;
    if (tid < 65) s.table[tid] = kPowers.of[tid];
    {  // log2(e) / temperature as a pair
        constexpr double c = 1.4426950408889634;
        constexpr float hi = (float)c, lo = (float)(c - (double)hi);
        z.c_hi = fminf(hi / heat, 3e38f);
        const float rest = fmaf(-z.c_hi, heat, hi) + lo;
        z.c_lo = z.c_hi < 3e38f ? rest / heat : 0.f;
    }
    // the best logit, of this thread's elements and of the row
    float mine = -INFINITY;
    {
        float best = -INFINITY;
        int at = 0;
        bool bad = false;
        z.each_first([&](float y, int token) {
            bad |= !(y < INFINITY);
            if (y > best) best = y, at = token;
        });
        mine = best;
        uint64_t key = best > -INFINITY ? make_key(best, at) : 0;
#pragma unroll
        for (int d = 16; d; d >>= 1) key = max(key, shfl_xor64(key, d));
        if (lane == 0) s.warp_w[warp] = key;
        z.clear_bins();
        const int anywhere = __syncthreads_or(bad);
        if (warp == 0) {
            key = lane < kWarps ? s.warp_w[lane] : 0;
#pragma unroll
            for (int d = 16; d; d >>= 1) key = max(key, shfl_xor64(key, d));
            if (lane == 0) s.best = anywhere ? ~0ull : key;
        }
        cluster.sync();
    }
    uint64_t best = lane < ranks ? cluster.map_shared_rank(&s, lane)->best : 0;
#pragma unroll
    for (int d = kMaxCluster / 2; d; d >>= 1) best = max(best, shfl_xor64(best, d));
    best = __shfl_sync(~0u, (unsigned long long)best, 0);
    const bool bad = none || best == ~0ull;
    auto answer = [&](int token, float logprob) {
        a.tokens[row] = token;
        if (a.logprobs) a.logprobs[row] = logprob;
    };
    if (bad || best == 0 || heat == 0.f) {
        if (rank == 0 && tid == 0) {
            const bool no = bad || best == 0;
            answer(no ? -1 : (int)key_token(best), no ? -INFINITY : 0.f);
        }
        cluster.sync();  // nobody's shared memory is read any more
        return;
    }
    z.m = unordered((uint32_t)(best >> 32));
    auto logprob = [&](float y, uint64_t w, uint64_t total) {  // near 1 by what is left of it
        if (w > total / 2) return log1pf(-((float)(total - w) / (float)total));
        float low;
        const float t = z.t_pair(y, low);
        return (t + low) * 0.693147181f - logf((float)total * (1.f / (float)(1ull << kShift)));
    };
    uint64_t cut = 0;
    const uint64_t least = min_p > 0.f ? part_of(min_p, 1ull << kShift, true) : 0;  // share that min-p asks for
    const bool by_k = top_k > 0 && top_k < a.vocab, by_p = top_p < 1.f;
    if (by_k || by_p) {
        auto share = [&](uint64_t of) { return max((uint64_t)1, part_of(fmaxf(top_p, 0.f), of, true)); };
        Sums all = {0, 0};
        const bool by_best = by_k && top_k <= kList / 2;
        auto fill = [&](bool by_count, uint64_t floor) {  // the bins, of every element from a key on; what their w sum to
            Sums sum = {0, 0};
            z.each([&](float y, int token) {
                const int bin = z.bin_of(y);
                if (bin >= kBins || make_key(y, token) < floor) return;
                if (by_count) {
                    atomicAdd(&s.count[bin], 1u);
                } else {
                    const uint64_t w = z.weight(y);
                    z.add(bin, w);
                    sum.w += w;
                }
            });
            z.close_bins(by_count);
            return z.row_sum(sum);
        };
        if (by_best) {
            const int own = z.bin_of(mine);
            if (own < kBins) atomicAdd(&s.count[own], 1u);
            z.close_bins(true);
            cluster.sync();
        } else {
            all = fill(by_k, 0);
        }
        z.locate(by_k, by_k ? (uint64_t)top_k : share(all.w));
        // All up to this bin into the list, if they may fit.  (Where the best ones do not reach so far, they do only if the
        // row itself is no longer.)
        const int reach = min(s.at_bin, kBins);
        uint32_t n = kList + 1;
        if (reach < kBins ? by_best || s.most <= (float)kList : a.vocab <= kList) {
            // by a logit that is below all of these bins': what is listed is a beginning of the order all the same
            const float low = reach < kBins ? z.m - (float)(reach + 1) / (z.c_hi * kOctave) * 1.0001f - fabsf(z.m) * 1e-6f : -INFINITY;
            z.each([&](float y, int token) {
                if (y >= low && y > -INFINITY) z.collect(make_key(y, token));
            });
            cluster.sync();
            n = cluster.map_shared_rank(&s, 0)->listed;
        }
        if (n <= kList) {
            if (rank == 0) {
                z.sort_list((int)n);
                z.scan_list((int)n);
                int kept = by_k ? min((int)n, top_k) : (int)n;
                if (by_p) kept = min(kept, z.place(kept, share(by_k ? s.w[kept - 1] : all.w)) + 1);
                {  // min-p: entries before the first below it; the best one is none of these
                    int lo = 1, hi = kept;
                    while (lo < hi) {
                        const int mid = (lo + hi) >> 1;
                        if (s.w[mid] - s.w[mid - 1] < least) hi = mid;
                        else lo = mid + 1;
                    }
                    kept = lo;
                }
                const uint64_t total = s.w[kept - 1];
                __syncthreads();
                // by the tokens' numbers: entries with their halves exchanged
                for (int i = tid; i < kept; i += kThreads) s.key[i] = s.key[i] << 32 | s.key[i] >> 32;
                __syncthreads();
                z.sort_list(kept);
                for (int i = tid; i < kept; i += kThreads) s.key[i] = s.key[i] << 32 | s.key[i] >> 32;
                __syncthreads();
                z.scan_list(kept);
                if (tid == 0) {
                    const int i = min(z.place(kept, part_of(u, total, false) + 1), kept - 1);
                    const float y = unordered((uint32_t)(s.key[i] >> 32));
                    answer((int)key_token(s.key[i]), logprob(y, s.w[i] - (i ? s.w[i - 1] : 0), total));
                }
            }
            cluster.sync();
            return;
        }
        // the cut of top-k, then that of top-p behind it
        uint64_t floor = 0;
        if (by_k) {
            if (by_best) {
                cluster.sync();
                z.clear_bins();
                fill(true, 0);
                z.locate(true, (uint64_t)top_k);
            }
            if (s.at_bin < kBins) floor = z.cut_in(true, (uint64_t)top_k, 0);
        }
        if (by_p) {
            if (by_k) {
                cluster.sync();
                z.clear_bins();
                all = fill(false, floor);
                z.locate(false, share(all.w));
            }
            if (s.at_bin < kBins) floor = z.cut_in(false, share(all.w), floor);
        }
        cut = floor;
    }
    // the token in the order of the vocabulary: sums of the warps' parts, then the part that has it
    Sums kept = {0, 0};
    auto kept_weight = [&](float y, int token) {
        const uint64_t w = make_key(y, token) >= cut ? z.weight(y) : 0;
        return w >= least ? w : 0;
    };
    z.each([&](float y, int token) { kept.w += kept_weight(y, token); });
    const Sums total = z.row_sum(kept);
    uint64_t warp_sum = kept.w;
#pragma unroll
    for (int d = 16; d; d >>= 1) warp_sum += shfl_xor64(warp_sum, d);
    uint64_t before = 0;
    if (lane < rank) before = cluster.map_shared_rank(&s.sum[z.turn ^ 1], lane)->w;
#pragma unroll
    for (int d = kMaxCluster / 2; d; d >>= 1) before += shfl_xor64(before, d);
    before = __shfl_sync(~0u, (unsigned long long)before, 0);
    __syncthreads();
    if (lane == 0) s.warp_kept[warp] = warp_sum;
    __syncthreads();
    for (int i = 0; i < warp; ++i) before += s.warp_kept[i];
    const uint64_t need = part_of(u, total.w, false) + 1;
    if (before < need && before + warp_sum >= need) {  // one warp of the row
        int lo, hi;
        z.warp_part(warp, lo, hi);
        for (int v = lo; v < hi; v += 32) {
            uint64_t run = 0;
            if (v + lane < hi)
                z.vector(v + lane, [&](float y, int token) { run += kept_weight(y, token); });
            const uint64_t own = run;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const uint64_t y = shfl_up64(run, d);
                if (lane >= d) run += y;
            }
            const uint64_t all = __shfl_sync(~0u, (unsigned long long)run, 31);
            uint64_t at = before + run - own;
            if (before + all >= need) {
                if (at < need && at + own >= need)
                    z.vector(v + lane, [&](float y, int token) {
                        const uint64_t w = kept_weight(y, token);
                        if (at < need && at + w >= need) answer(token, logprob(y, w, total.w));
                        at += w;
                    });
                break;
            }
            before += all;
        }
    }
    cluster.sync();
}

template <typename IO> cudaError_t launch(SampleArgs a, cudaStream_t st) {
    // CTAs per row: up to 8 while the rows leave SMs free and each has 2048 tokens at least, and as many as a slice's
    // limit needs
    int ranks = 1;
    while (ranks < kMaxCluster && (((int64_t)a.B * ranks * 2 <= 2 * 152 && a.vocab / (ranks * 2) >= 2048) || a.vocab + 16 > ranks * kSlice))
        ranks *= 2;
    constexpr int VEC = 16 / (int)sizeof(IO);
    const int bytes = ((a.vocab + 2 * VEC - 1) / VEC + ranks - 1) / ranks * 16;  // of a slice, whatever the row's alignment
    a.cached = bytes <= kCache;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(k_sample<IO>, kCache, done);
    if (e != cudaSuccess) return e;
    return launch_clusters(k_sample<IO>, ranks, dim3((unsigned)(a.B * ranks)), kThreads, a.cached ? (size_t)bytes : 0, st, a);
}

}  // namespace

cudaError_t launch_sample(const SampleArgs &a, gdn_dtype io, cudaStream_t st) {
    return io == GDN_BF16 ? launch<__nv_bfloat16>(a, st) : launch<float>(a, st);
}

}  // namespace gdn
