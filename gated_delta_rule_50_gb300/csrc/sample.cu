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
// A cut is found by counting.  Bins of 1/32 octave of t (kBins of them; below the last every w is 0 and a token counts
// for nothing) get their sums of w, or for top-k their number of tokens; the running sum over them says in which bin the
// cut lies.  If all up to there fit a list (kList), they are collected and sorted, and the rest of the work is done on
// the list.  If not, that bin is cut into kSub further ones and what lies in one of those is collected and sorted to find
// the cut; where even that is too much for the list (many equal logits), the cut is searched for by bisection, over the
// logit and then over the tokens that share it.
//
// The CTAs of a cluster share a row: slices of it, read again in each pass (they come from L2).
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include "common.cuh"
#include "decode.h"

namespace gdn {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kOctave = 32, kBins = 44 * kOctave;  // w = 0 from t = -43 on
constexpr int kSub = 1024;
constexpr int kList = 1024;
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
    uint32_t lo[kBins], hi[kBins];  // sums of w, in two halves
    uint32_t count[kBins];
    uint64_t key[kList], w[kList];
    uint64_t table[65];  // 2^(42 + j / 64), j = -32 .. 32
    uint64_t warp_w[kWarps];
    uint32_t warp_n[kWarps];
    uint64_t best;       // of the CTA's slice
    int bad;
    Sums part[2];        // what the CTA adds to a sum over the cluster
    uint64_t warp_kept[kWarps];
    uint32_t listed;     // entries of the list (the first CTA's)
    uint64_t cut;        // found by the first CTA
    int at_bin;
    Sums before;         // what lies in the bins before it
    float c_hi, c_lo;
    double min_p;        // temperature ln(min_p)
    int found;
};

template <typename IO> struct Sampler {
    static constexpr int VEC = 16 / (int)sizeof(IO);
    Shared &s;
    const cg::cluster_group cluster;
    const IO *x;          // the row
    const uint8_t *mask;  // the row's, or nullptr
    int vocab, v0, v1;    // this CTA's vectors; vector v has the elements VEC v - skew ..
    int skew;             // elements by which the row begins behind a 16-byte boundary
    bool mask8;           // the mask's bytes of a vector can be read at once
    float m, c_hi, c_lo;
    int turn;

    // f(x, token) for every allowed element of this warp's part of the slice, in ascending vectors by lane
    template <typename F> __device__ __forceinline__ void vector(int v, F f) const {
        const int at = v * VEC - skew;
        IO e[VEC];
        uint8_t ok[VEC];
        if (at >= 0 && at + VEC <= vocab) {
            *reinterpret_cast<uint4 *>(e) = __ldg(reinterpret_cast<const uint4 *>(x + at));
            if (mask) {
                if (mask8) {
                    if constexpr (VEC == 8) *reinterpret_cast<uint2 *>(ok) = __ldg(reinterpret_cast<const uint2 *>(mask + at));
                    else *reinterpret_cast<uint32_t *>(ok) = __ldg(reinterpret_cast<const uint32_t *>(mask + at));
                } else {
#pragma unroll
                    for (int i = 0; i < VEC; ++i) ok[i] = mask[at + i];
                }
            }
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                if (!mask || ok[i]) f(to_f<IO>(e[i]), at + i);
        } else {
            for (int i = 0; i < VEC; ++i)
                if (at + i >= 0 && at + i < vocab && (!mask || mask[at + i])) f(to_f<IO>(x[at + i]), at + i);
        }
    }
    __device__ __forceinline__ void warp_part(int warp, int &a, int &b) const {
        const int each = (v1 - v0 + kWarps - 1) / kWarps;
        a = min(v1, v0 + warp * each), b = min(v1, a + each);
    }
    template <typename F> __device__ __forceinline__ void each(F f) const {
        int a, b;
        warp_part(threadIdx.x >> 5, a, b);
        for (int v = a + (threadIdx.x & 31); v < b; v += 32) vector(v, f);
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
        if (threadIdx.x == 0) s.part[turn] = a;
        cluster.sync();
        Sums all = {0, 0};
        for (unsigned r = 0; r < cluster.num_blocks(); ++r) all = all + *cluster.map_shared_rank(&s.part[turn], r);
        turn ^= 1;
        return all;
    }

    // Where in bins 0 .. n - 1 (over the cluster) the running sum reaches `need` (of w, or of tokens): at_bin (n: nowhere)
    // and what lies before it.  The bins stay as they are until the next sync.
    __device__ __forceinline__ void locate(int n, bool by_count, uint64_t need) {
        const int per = (n + kThreads - 1) / kThreads, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        constexpr int MOST = (kBins + kThreads - 1) / kThreads;
        uint64_t v[MOST];
        uint64_t mine = 0;
#pragma unroll
        for (int i = 0; i < MOST; ++i) {
            v[i] = 0;
            const int bin = threadIdx.x * per + i;
            if (i < per && bin < n)
                for (unsigned r = 0; r < cluster.num_blocks(); ++r) {
                    const Shared *o = cluster.map_shared_rank(&s, r);
                    v[i] += by_count ? o->count[bin] : ((uint64_t)o->hi[bin] << 32) + o->lo[bin];
                }
            mine += v[i];
        }
        uint64_t run = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint64_t y = shfl_up64(run, d);
            if (lane >= d) run += y;
        }
        __syncthreads();
        if (lane == 31) s.warp_w[warp] = run;
        if (threadIdx.x == 0) s.at_bin = n;
        __syncthreads();
        for (int i = 0; i < warp; ++i) run += s.warp_w[i];
        uint64_t before = run - mine;
        if (before < need && run >= need) {
#pragma unroll
            for (int i = 0; i < MOST; ++i) {
                if (before < need && before + v[i] >= need) s.at_bin = threadIdx.x * per + i, s.before = {before, (uint32_t)before};
                before += v[i];
            }
        }
        __syncthreads();
    }
    __device__ __forceinline__ void clear_bins() {
        for (int i = threadIdx.x; i < kBins; i += kThreads) s.lo[i] = s.hi[i] = s.count[i] = 0;
        __syncthreads();
    }
    __device__ __forceinline__ void add(int bin, bool by_count, float y) {
        if (by_count) {
            atomicAdd(&s.count[bin], 1u);
        } else {
            const uint64_t w = weight(y);
            const uint32_t low = (uint32_t)w, old = atomicAdd(&s.lo[bin], low);
            const uint32_t high = (uint32_t)(w >> 32) + (old + low < old ? 1u : 0u);
            if (high) atomicAdd(&s.hi[bin], high);
        }
    }
    // Into the first CTA's list
    __device__ __forceinline__ void collect(uint64_t key) {
        Shared *first = cluster.map_shared_rank(&s, 0);
        const uint32_t at = atomicAdd(&first->listed, 1u);
        if (at < kList) first->key[at] = key;
    }
    // Sorts the first n entries of the list (the rest of a power of two filled up): descending keys
    __device__ __forceinline__ int sort_list(int n) {
        int size = 32;
        while (size < n) size <<= 1;
        for (int i = n + threadIdx.x; i < size; i += kThreads) s.key[i] = 0;
        __syncthreads();
        for (int k = 2; k <= size; k <<= 1)
            for (int j = k >> 1; j; j >>= 1) {
                for (int i = threadIdx.x; i < size / 2; i += kThreads) {
                    const int a = (i / j) * 2 * j + i % j, b = a + j;
                    const bool down = (a & k) == 0;
                    const uint64_t x0 = s.key[a], x1 = s.key[b];
                    if ((x0 < x1) == down) s.key[a] = x1, s.key[b] = x0;
                }
                __syncthreads();
            }
        return size;
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

    // The cut in a bin: the key at which, among the keys from `floor` on, the running sum over the bin reaches need
    __device__ __forceinline__ uint64_t cut_in(int bin, bool by_count, uint64_t need, uint64_t floor) {
        cluster.sync();  // all have read the bins
        clear_bins();
        if (threadIdx.x == 0) s.listed = 0;
        each([&](float y, int token) {
            if (bin_of(y) == bin && make_key(y, token) >= floor) add(sub_of(y, bin), by_count, y);
        });
        cluster.sync();
        locate(kSub, by_count, need);
        const int sub = s.at_bin;
        if (sub == kSub) return floor;  // all of it
        need -= s.before.w;
        uint32_t n = 0;
        each([&](float y, int token) {
            const uint64_t key = make_key(y, token);
            if (bin_of(y) == bin && key >= floor && sub_of(y, bin) == sub) collect(key), ++n;
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
                if (ordered(y) >= mid && bin_of(y) == bin && make_key(y, token) >= floor && sub_of(y, bin) == sub)
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

template <typename IO> __global__ void __launch_bounds__(kThreads) k_sample(const __grid_constant__ SampleArgs a) {
    __shared__ Shared s;
    const cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
    const int row = blockIdx.x / ranks, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    Sampler<IO> z{s, cluster};
    z.x = static_cast<const IO *>(a.logits) + row * a.logits_row;
    z.mask = a.mask ? a.mask + row * a.mask_row : nullptr;
    z.vocab = a.vocab, z.turn = 0;
    z.skew = (int)((reinterpret_cast<uintptr_t>(z.x) & 15) / sizeof(IO));
    z.mask8 = z.mask && ((reinterpret_cast<uintptr_t>(z.mask) - z.skew) & (Sampler<IO>::VEC - 1)) == 0;
    const int vectors = (a.vocab + z.skew + Sampler<IO>::VEC - 1) / Sampler<IO>::VEC;
    const int slice = (vectors + ranks - 1) / ranks;
    z.v0 = min(vectors, rank * slice), z.v1 = min(vectors, z.v0 + slice);
    wait_for_previous();
    const float heat = a.temperatures ? a.temperatures[row] : a.temperature;
    const int top_k = a.top_ks ? a.top_ks[row] : a.top_k;
    const float top_p = a.top_ps ? a.top_ps[row] : a.top_p;
    const float given_min_p = a.min_ps ? a.min_ps[row] : a.min_p, min_p = fminf(given_min_p, 1.f);
    const bool none = !(heat >= 0.f) || heat == INFINITY || isnan(top_p) || isnan(given_min_p);
    float u = a.u[row];
    u = u >= 0.f ? fminf(u, 0.99999994f) : 0.f;
    if (tid == 0) s.bad = 0, s.listed = 0;
    if (tid == 32) {
        const double c = 1.4426950408889634 / (double)heat;
        s.c_hi = c < 3e38 ? (float)c : 3e38f;
        s.c_lo = c < 3e38 ? (float)(c - (double)s.c_hi) : 0.f;
    }
    if (tid == 64) s.min_p = min_p > 0.f ? (double)heat * log((double)min_p) : 0.;
    if (tid >= 128 && tid < 128 + 65) s.table[tid - 128] = kPowers.of[tid - 128];
    __syncthreads();
    // the best logit
    {
        float best = -INFINITY;
        int at = 0;
        bool bad = false;
        z.each([&](float y, int token) {
            bad |= !(y < INFINITY);
            if (y > best) best = y, at = token;
        });
        uint64_t key = best > -INFINITY ? make_key(best, at) : 0;
#pragma unroll
        for (int d = 16; d; d >>= 1) key = max(key, shfl_xor64(key, d));
        if (lane == 0) s.warp_w[warp] = key;
        if (bad) s.bad = 1;
        __syncthreads();
        if (tid == 0) {
            for (int i = 1; i < kWarps; ++i) key = max(key, s.warp_w[i]);
            s.best = key;
        }
        cluster.sync();
    }
    uint64_t best = 0;
    bool bad = none;
    for (int r = 0; r < ranks; ++r) {
        const Shared *o = cluster.map_shared_rank(&s, r);
        best = max(best, o->best);
        bad |= o->bad != 0;
    }
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
    z.c_hi = s.c_hi, z.c_lo = s.c_lo;
    auto logprob = [&](float y, uint64_t w, uint64_t total) {  // near 1 by what is left of it
        if (w > total / 2) return log1pf(-((float)(total - w) / (float)total));
        float low;
        const float t = z.t_pair(y, low);
        return (t + low) * 0.693147181f - logf((float)total * (1.f / (float)(1ull << kShift)));
    };
    uint64_t cut = 0;
    if (min_p > 0.f) cut = (uint64_t)ordered(__double2float_ru((double)z.m + s.min_p)) << 32;
    const bool by_k = top_k > 0 && top_k < a.vocab, by_p = top_p < 1.f;
    if (by_k || by_p) {
        // bins of what can be drawn: tokens for top-k, else shares
        z.clear_bins();
        Sums all = {0, 0};
        z.each([&](float y, int) {
            const int bin = z.bin_of(y);
            if (bin < kBins) z.add(bin, by_k, y);
            if (!by_k) all.w += z.weight(y);
        });
        auto share = [&](uint64_t of) { return max((uint64_t)1, (uint64_t)ceil((double)fmaxf(top_p, 0.f) * (double)of)); };
        if (!by_k) all = z.row_sum(all);
        else cluster.sync();
        z.locate(kBins, by_k, by_k ? (uint64_t)top_k : share(all.w));
        const int bin = s.at_bin;
        const Sums before = s.before;
        // do all up to this bin fit the list?
        Sums listed = {0, 0};
        z.each([&](float y, int) { listed.n += z.bin_of(y) <= bin; });
        listed = z.row_sum(listed);
        if (listed.n <= kList) {
            z.each([&](float y, int token) {
                if (z.bin_of(y) <= bin) z.collect(make_key(y, token));
            });
            cluster.sync();
            if (rank == 0) {
                int n = (int)listed.n;
                z.sort_list(n);
                z.scan_list(n);
                if (by_k) n = min(n, top_k);
                if (by_p) n = min(n, z.place(n, share(by_k ? s.w[n - 1] : all.w)) + 1);
                {  // min-p: entries before the first below it
                    int lo = 1, hi = n;
                    while (lo < hi) {
                        const int mid = (lo + hi) >> 1;
                        if (s.key[mid] < cut) hi = mid;
                        else lo = mid + 1;
                    }
                    n = lo;
                }
                const uint64_t total = s.w[n - 1];
                __syncthreads();
                // by the tokens' numbers: entries with their halves exchanged
                for (int i = tid; i < n; i += kThreads) s.key[i] = s.key[i] << 32 | s.key[i] >> 32;
                z.sort_list(n);
                for (int i = tid; i < n; i += kThreads) s.key[i] = s.key[i] << 32 | s.key[i] >> 32;
                __syncthreads();
                z.scan_list(n);
                if (tid == 0) {
                    const int i = min(z.place(n, (uint64_t)((double)u * (double)total) + 1), n - 1);
                    const float y = unordered((uint32_t)(s.key[i] >> 32));
                    answer((int)key_token(s.key[i]), logprob(y, s.w[i] - (i ? s.w[i - 1] : 0), total));
                }
            }
            cluster.sync();
            return;
        }
        uint64_t floor = 0;
        if (by_k && bin < kBins) floor = z.cut_in(bin, true, (uint64_t)top_k - before.w, 0);
        if (by_p) {
            if (by_k) {
                cluster.sync();
                z.clear_bins();
                all = {0, 0};
                z.each([&](float y, int token) {
                    const int b = z.bin_of(y);
                    if (b < kBins && make_key(y, token) >= floor) z.add(b, false, y), all.w += z.weight(y);
                });
                all = z.row_sum(all);
                z.locate(kBins, false, share(all.w));
            }
            const int at = s.at_bin;
            const uint64_t need = share(all.w) - s.before.w;
            if (at < kBins) floor = z.cut_in(at, false, need, floor);
        }
        cut = max(cut, floor);
    }
    // the token in the order of the vocabulary: sums of the warps' parts, then the part that has it
    Sums kept = {0, 0};
    z.each([&](float y, int token) {
        if (make_key(y, token) >= cut) kept.w += z.weight(y);
    });
    const Sums total = z.row_sum(kept);
    uint64_t mine = kept.w;
#pragma unroll
    for (int d = 16; d; d >>= 1) mine += shfl_xor64(mine, d);
    uint64_t before = 0;
    for (int r = 0; r < rank; ++r) before += cluster.map_shared_rank(&s.part[z.turn ^ 1], r)->w;
    __syncthreads();
    if (lane == 0) s.warp_kept[warp] = mine;
    __syncthreads();
    for (int i = 0; i < warp; ++i) before += s.warp_kept[i];
    const uint64_t need = (uint64_t)((double)u * (double)total.w) + 1;
    if (before < need && before + mine >= need) {  // one warp of the row
        int lo, hi;
        z.warp_part(warp, lo, hi);
        for (int v = lo; v < hi; v += 32) {
            uint64_t run = 0;
            if (v + lane < hi)
                z.vector(v + lane, [&](float y, int token) {
                    if (make_key(y, token) >= cut) run += z.weight(y);
                });
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
                        if (make_key(y, token) < cut) return;
                        const uint64_t w = z.weight(y);
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

template <typename IO> cudaError_t launch(const SampleArgs &a, cudaStream_t st) {
    // CTAs per row: up to 8 while the rows leave SMs free and each has 2048 tokens at least
    int ranks = 1;
    while (ranks < kMaxCluster && (int64_t)a.B * ranks * 2 <= 2 * 152 && a.vocab / (ranks * 2) >= 2048) ranks *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.B * ranks));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute at[2] = {};
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)ranks, at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, k_sample<IO>, a);
}

}  // namespace

cudaError_t launch_sample(const SampleArgs &a, gdn_dtype io, cudaStream_t st) {
    return io == GDN_BF16 ? launch<__nv_bfloat16>(a, st) : launch<float>(a, st);
}

}  // namespace gdn
