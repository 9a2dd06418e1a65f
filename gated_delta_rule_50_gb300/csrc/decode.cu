// decode.cu -- the gated delta rule token by token, on a pool of states.
//
// Per row and value head, with a = e^g:  d = beta (v - a S^T k),  S' = a S + k d^T,  o = scale S'^T q.
// Both products are taken from the state before the update, o = scale (a S^T q + (q.k) d), so one pass over
// the state's registers serves k and q and a second one updates it.
//
// A warp holds a [K][32] tile of the state in registers: lane = (r, c) with c = 0..7 has the four columns
// 4c .. 4c+3 of the rows 16 i + 4 r + j (K values of 32 bits per lane, K/4 accesses of 16 bytes, each a full
// 128-byte line per row across the lanes).  The value columns are independent, so nothing crosses warps;
// the four r lanes of a column group meet through shuffles.
//
// For one token the states' way through memory bounds the step (each is read and written once): 64 rows of 32 heads,
// 128 x 128, bf16, take 45 us, 6.0 TB/s; one row 3.0 us, where reads, sums and writes wait for each other.  More tokens
// on the same states take 53 us (3) and 74 us (6), where memory would take 41 and 42: each costs three multiply-adds per
// element of the state and two reads of k, with seven or eight warps on an SM.  Two kernels share the arithmetic: k_recurrent, a warp per CTA and 32 columns, and k_recurrent_flow for
// lists of tokens on many heads (see launch()).
#include <cuda_bf16.h>

#include "common.cuh"
#include "decode.h"
#include "tc.cuh"

namespace gdn {
namespace {

using namespace tc;

template <typename IO> constexpr int kTok = 16 / (int)sizeof(IO);  // tokens staged in shared memory at a time
constexpr int kTile = 32;  // state columns per warp
constexpr int kSMs = 152;

// Sums x[0..3] (the lane's four columns) over the four r lanes; lane (r, c) gets column 4c + r.
__device__ __forceinline__ float reduce_columns(const float (&x)[4], int r) {
    const bool r0 = r & 1, r1 = r & 2;
    float a = r0 ? x[1] : x[0], b = r0 ? x[3] : x[2];
    a += __shfl_xor_sync(~0u, r0 ? x[0] : x[1], 8);
    b += __shfl_xor_sync(~0u, r0 ? x[2] : x[3], 8);
    return (r1 ? b : a) + __shfl_xor_sync(~0u, r1 ? a : b, 16);
}

// What one row runs through: tokens [bos, bos + len) of batch row b, or a list of len tokens at most
struct Run {
    int64_t bos, out_row, slot;
    int b, len;
    bool valid;  // the row's offsets lie in the tensor
};
__device__ __forceinline__ Run run_of(const DecodeArgs &a, int n) {
    Run u;
    u.valid = true, u.bos = 0, u.b = n;
    u.len = a.token_indices ? a.n_steps : a.T;
    u.out_row = (int64_t)n * u.len;
    if (a.cu) {
        const int lo = a.cu[n], hi = a.cu[n + 1];
        u.valid = lo >= 0 && hi >= lo && hi <= a.T;
        u.b = 0, u.bos = u.out_row = lo, u.len = hi - lo;
    }
    u.slot = a.state_indices ? a.state_indices[n] : n;
    return u;
}

__device__ __forceinline__ void cp_async16(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

// Up to kTok tokens for COLS threads, one state column each
template <int K, int COLS, typename IO> struct Stage {
    alignas(16) IO k[kTok<IO>][K], q[kTok<IO>][K], v[kTok<IO>][COLS];
    float a[kTok<IO>], b[kTok<IO>];
    int tok[kTok<IO>];
};
__device__ __forceinline__ float4 load4(const float *x) { return *reinterpret_cast<const float4 *>(x); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16 *x) {
    const uint2 u = *reinterpret_cast<const uint2 *>(x);
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                       __uint_as_float(u.y & 0xFFFF0000u));
}

// The threads of one head (tid = 0 .. COLS - 1, columns col0 + tid) and, for more than a warp, their barrier
template <int K, int COLS, typename IO> struct Head {
    static constexpr int NR = K / 4;
    const DecodeArgs &a;
    Stage<K, COLS, IO> &s;
    const Run u;
    const IO *q, *k, *v;
    const float *g, *beta;
    IO *o;  // row out_row of this head, this thread's column
    int n, tid, bar;
    bool rows16;  // rows of q, k and v begin on 16-byte boundaries

    __device__ __forceinline__ Head(const DecodeArgs &a, Stage<K, COLS, IO> &s, const Run &u, int n, int h, int hq, int col0, int tid, int bar,
                                    bool rows16)
        : a(a), s(s), u(u), n(n), tid(tid), bar(bar), rows16(rows16) {
        q = static_cast<const IO *>(a.q) + u.b * a.sq.batch + hq * a.sq.head;
        k = static_cast<const IO *>(a.k) + u.b * a.sk.batch + hq * a.sk.head;
        v = static_cast<const IO *>(a.v) + u.b * a.sv.batch + h * a.sv.head + col0 + tid;
        g = a.g + u.b * a.sg.batch + h * a.sg.head;
        beta = a.beta + u.b * a.sb.batch + h * a.sb.head;
        o = a.o ? static_cast<IO *>(a.o) + (u.out_row * a.Hv + h) * a.V + col0 : nullptr;
    }
    __device__ __forceinline__ void sync() const {
        if constexpr (COLS == 32) __syncwarp();
        else named_bar(bar, COLS);
    }
    __device__ __forceinline__ int64_t o_tok() const { return (int64_t)a.Hv * a.V; }
    // o of tokens [from, len): 0, or NaN where an index was none
    __device__ __forceinline__ void fill(int from, bool bad) const {
        if (!o) return;
        for (int t = from; t < u.len; ++t) o[t * o_tok() + tid] = from_f<IO>(bad ? __int_as_float(0x7fffffff) : 0.f);
    }
    // Tokens t0 .. t0 + kTok - 1 into the stage; how many there are, and whether the row ends in them
    __device__ __forceinline__ int stage(int t0, bool &more, bool &bad) const {
        int m = min(kTok<IO>, u.len - t0);
        if (a.token_indices) {
            if (tid < m) s.tok[tid] = a.token_indices[(int64_t)n * a.n_steps + t0 + tid];
            sync();
            for (int t = 0; t < m; ++t) {
                const int at = s.tok[t];
                if (at >= 0 && at < a.T) continue;
                bad = at >= 0;
                m = t, more = false;
                break;
            }
        }
        auto token = [&](int t) -> int64_t { return a.token_indices ? s.tok[t] : u.bos + t0 + t; };
        if (rows16) {
            constexpr int PIECE = 16 / (int)sizeof(IO), PIECES = K / PIECE;
            for (int e = tid; e < m * PIECES; e += COLS) {
                const int t = e / PIECES, x = e % PIECES * PIECE;
                cp_async16(&s.k[t][x], k + token(t) * a.sk.token + x);
                if (o) cp_async16(&s.q[t][x], q + token(t) * a.sq.token + x);
            }
            constexpr int pieces = COLS / PIECE;
            for (int e = tid; e < m * pieces; e += COLS) {
                const int t = e / pieces, x = (e - t * pieces) * PIECE;
                cp_async16(&s.v[t][x], v - tid + token(t) * a.sv.token + x);
            }
        } else {
#pragma unroll 4
            for (int e = tid; e < m * K; e += COLS) {
                const int t = e / K, x = e % K;
                s.k[t][x] = k[token(t) * a.sk.token + x];
                if (o) s.q[t][x] = q[token(t) * a.sq.token + x];
            }
#pragma unroll 4
            for (int t = 0; t < m; ++t) s.v[t][tid] = v[token(t) * a.sv.token];
        }
        if (tid < m) s.a[tid] = expf(g[token(tid) * a.sg.token]), s.b[tid] = beta[token(tid) * a.sb.token];
        asm volatile("cp.async.wait_all;" ::: "memory");
        return m;
    }
    // m staged tokens, the first of them the t0-th of the row
    __device__ __forceinline__ void advance(float4 (&S)[NR], int t0, int m) const {
        const int lane = tid & 31, c = lane & 7, r = lane >> 3;
        const int col = (tid & ~31) + 4 * c + r;  // the column whose sums this lane gets
#pragma unroll 1
        for (int t = 0; t < m; ++t) {
            float ks[4] = {0.f, 0.f, 0.f, 0.f}, qs[4] = {0.f, 0.f, 0.f, 0.f}, qk = 0.f;
#pragma unroll
            for (int i = 0; i < K / 16; ++i) {
                const float4 kk = load4(s.k[t] + 16 * i + 4 * r);
                const float kj[4] = {kk.x, kk.y, kk.z, kk.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float4 x = S[4 * i + j];
                    ks[0] = fmaf(kj[j], x.x, ks[0]);
                    ks[1] = fmaf(kj[j], x.y, ks[1]);
                    ks[2] = fmaf(kj[j], x.z, ks[2]);
                    ks[3] = fmaf(kj[j], x.w, ks[3]);
                }
                if (o) {
                    const float4 qq = load4(s.q[t] + 16 * i + 4 * r);
                    const float qj[4] = {qq.x, qq.y, qq.z, qq.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float4 x = S[4 * i + j];
                        qs[0] = fmaf(qj[j], x.x, qs[0]);
                        qs[1] = fmaf(qj[j], x.y, qs[1]);
                        qs[2] = fmaf(qj[j], x.z, qs[2]);
                        qs[3] = fmaf(qj[j], x.w, qs[3]);
                        qk = fmaf(qj[j], kj[j], qk);
                    }
                }
            }
            const float al = s.a[t];
            const float d = s.b[t] * (to_f<IO>(s.v[t][col]) - al * reduce_columns(ks, r));
            if (o) {
                qk += __shfl_xor_sync(~0u, qk, 8);
                qk += __shfl_xor_sync(~0u, qk, 16);
                o[(t0 + t) * o_tok() + col] = from_f<IO>(a.scale * fmaf(qk, d, al * reduce_columns(qs, r)));
            }
            float dj[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) dj[j] = __shfl_sync(~0u, d, c + 8 * j);
#pragma unroll
            for (int i = 0; i < K / 16; ++i) {
                const float4 kk = load4(s.k[t] + 16 * i + 4 * r);
                const float kj[4] = {kk.x, kk.y, kk.z, kk.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float4 &x = S[4 * i + j];
                    x.x = fmaf(kj[j], dj[0], al * x.x);
                    x.y = fmaf(kj[j], dj[1], al * x.y);
                    x.z = fmaf(kj[j], dj[2], al * x.z);
                    x.w = fmaf(kj[j], dj[3], al * x.w);
                }
            }
        }
    }
    // The row from its first m tokens, which all threads see in the stage, to its end; whether the new state is to be
    // kept
    __device__ __forceinline__ bool run(float4 (&S)[NR], int m, bool more, bool bad) const {
        int t0 = 0;
        for (;;) {
            advance(S, t0, m);
            t0 += m;
            if (!more || t0 >= u.len) break;
            sync();
            m = stage(t0, more, bad);
            sync();
            if (m == 0) break;
        }
        if (t0 < u.len) fill(t0, bad);
        return !bad;
    }
    __device__ __forceinline__ float *out(int h) const {
        return a.out_state ? a.out_state + ((int64_t)n * a.Hv + h) * K * a.V
                           : a.state + u.slot * a.slot_stride + (int64_t)h * K * a.V;
    }
};

// One warp, 32 columns of a state.  Warps of their own begin and end as they come, so that one's reads run under
// another's arithmetic; a CTA of four for a whole state takes 3.9 us instead of 3.3 for one row of 32 heads (1 token),
// 25.8 instead of 24.7 for 32 rows, 53 instead of 45 for 64.  16-byte copies of the tokens' rows, where they are
// aligned, against reads of single elements: 3.3 and 3.6 us for that one row, 5.4 and 6.4 us for 37 rows of 8 fp32
// heads, 64 x 64, 3 tokens.
// grid (rows, q/k heads, value heads of one * parts of the columns)
template <int K, typename IO> __global__ void __launch_bounds__(kTile) k_recurrent(const __grid_constant__ DecodeArgs a, bool rows16) {
    constexpr int NR = K / 4;
    __shared__ Stage<K, kTile, IO> s;
    const int tid = threadIdx.x;
    const int n = blockIdx.x, hq = blockIdx.y, h = hq * a.G + blockIdx.z % a.G, col0 = blockIdx.z / a.G * kTile;
    wait_for_previous();
    const Run u = run_of(a, n);
    if (!u.valid) return;
    const Head<K, kTile, IO> head(a, s, u, n, h, hq, col0, tid, 0, rows16);
    if (u.slot < 0 || u.slot >= a.n_slots) {
        head.fill(0, u.slot >= 0);
        return;
    }
    const int c = tid & 7, r = (tid & 31) >> 3;
    const int at = 4 * r * a.V + col0 + (tid & ~31) + 4 * c;
    const float *src = a.state + u.slot * a.slot_stride + (int64_t)h * K * a.V + at;
    float4 S[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) S[i] = *reinterpret_cast<const float4 *>(src + (16 * (i >> 2) + (i & 3)) * a.V);
    bool more = true, bad = false;
    const int m = head.stage(0, more, bad);
    __syncwarp();
    if (!head.run(S, m, more, bad)) return;
    float *dst = head.out(h) + at;
#pragma unroll
    for (int i = 0; i < NR; ++i) *reinterpret_cast<float4 *>(dst + (16 * (i >> 2) + (i & 3)) * a.V) = S[i];
}

// Shared memory of k_recurrent_flow: a ring of slots, each a state and the first tokens of its row (k, q, v as they
// are), what there is to know of the slots, a stage per group, barriers
constexpr int kMaxSlots = 8, kGroup = 128;
struct SlotInfo {
    float a[8], b[8];
    int m, more, bad;
};
template <typename IO> struct Flow {
    static constexpr int K = 128, V = kGroup, groups = 2, state_bytes = K * V * 4;
    static constexpr int slot_bytes = state_bytes + kTok<IO> * (2 * K + V) * (int)sizeof(IO);
    static constexpr int stage_bytes = (int)sizeof(Stage<K, V, IO>);
    static constexpr int rest = 128 + groups * stage_bytes + kMaxSlots * (int)sizeof(SlotInfo) + 256;
    static constexpr int room = (232448 - rest) / slot_bytes;  // 227 KB
    static constexpr int slots = room < kMaxSlots ? room : kMaxSlots, bytes = rest + slots * slot_bytes;
};

// Lists of tokens (128 x 128 states).  There a warp on its own waits for its list, then for the rows that it names, and
// only then works.  One CTA per SM: two groups of 128 threads take this CTA's heads in order, whichever is free, each
// from the ring into registers, ask at once for what comes next into the slot, run theirs and write it back from the
// registers.  What a fetch itself depends on (slot, list, gates) is read while the group waits for its state.
//
// A slot's turns: its i-th use is asked for (`armed` ends its i-th phase, after `full` has been armed for its own), then
// arrives (`full` ends its i-th phase), then is taken and asked for again.  A phase is waited for by its parity, which
// says nothing while an earlier phase of the same slot is open: hence `armed` first, which the group that took the
// slot's previous use may be late with, since that can be the other group.  Late by a copy, not by a list: between
// taking a head and asking for the next one into its slot a group waits for nothing else, so that the limits of the
// waits hold whatever the lengths of the lists.  The parity of `armed` always tells: the slot's use before this one was
// taken by this group, which waited for its `armed`, or by the other one, which took it after asking for it or waits
// for a head that this group asked for.
// 96 rows of 64 heads, up to 6 tokens each: 134 us, 6.0 TB/s.
template <typename IO>
__global__ void __launch_bounds__(2 * kGroup, 1) k_recurrent_flow(const __grid_constant__ DecodeArgs a, int heads) {
    using F = Flow<IO>;
    constexpr int K = F::K, V = F::V, NR = K / 4, AHEAD = kTok<IO>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *sm = smem_raw + ((128u - (smem_u32(smem_raw) & 127u)) & 127u);
    unsigned char *stages = sm + F::slots * F::slot_bytes;
    SlotInfo *info = reinterpret_cast<SlotInfo *>(stages + F::groups * F::stage_bytes);
    unsigned char *bars = reinterpret_cast<unsigned char *>(info + kMaxSlots);
    static_assert(F::groups == 2 && 8 * kMaxSlots <= 64, "see above; the places of the barriers");
    const uint32_t full = smem_u32(bars), armed = full + 64;
    volatile int *issued = reinterpret_cast<volatile int *>(bars + 128), *abort_flag = issued + kMaxSlots;
    int *counter = reinterpret_cast<int *>(bars + 128) + kMaxSlots + 1, *taken = counter + 1;  // taken: one per group
    const int group = threadIdx.x / V, tid = threadIdx.x - group * V, bar = 1 + group, lane = tid & 31;

    struct Ahead {  // of a head that is to be fetched; lane t has its t-th token
        Run u;
        int64_t tok;
        float g, beta;
        int m, more, bad, h;
    };
    auto look = [&](int item) {  // a whole warp
        Ahead x;
        const int n = item / a.Hv;
        x.h = item - n * a.Hv;
        x.u = run_of(a, n);
        const bool live = x.u.valid && x.u.slot >= 0 && x.u.slot < a.n_slots;
        x.m = live ? min(AHEAD, x.u.len) : 0;
        x.more = 1, x.bad = 0;
        const int at = lane < x.m ? a.token_indices[(int64_t)n * a.n_steps + lane] : 0;
        const uint32_t none = __ballot_sync(~0u, at < 0 || at >= a.T) & ((1u << x.m) - 1u);
        if (none) {
            x.m = __ffs(none) - 1;
            x.more = 0, x.bad = __shfl_sync(~0u, at, x.m) >= 0;
        }
        x.tok = at;
        x.g = x.beta = 0.f;
        if (lane < x.m) {
            x.g = a.g[x.u.b * a.sg.batch + x.h * a.sg.head + x.tok * a.sg.token];
            x.beta = a.beta[x.u.b * a.sb.batch + x.h * a.sb.head + x.tok * a.sb.token];
        }
        return x;
    };
    auto fetch = [&](int i, const Ahead &x) {  // a whole warp: the i-th head of this CTA into its slot
        const int slot = i % F::slots, hq = x.h / a.G;
        const uint32_t at = smem_u32(sm) + slot * F::slot_bytes, bar_f = full + 8 * slot;
        const bool live = x.u.valid && x.u.slot >= 0 && x.u.slot < a.n_slots;
        if (lane < x.m) info[slot].a[lane] = expf(x.g), info[slot].b[lane] = x.beta;
        __syncwarp();
        if (lane == 0) {
            info[slot].m = x.m, info[slot].more = x.more, info[slot].bad = x.bad;
            issued[slot] = i / F::slots + 1;
            const uint32_t row = (uint32_t)((a.o ? 2 : 1) * K + V) * (uint32_t)sizeof(IO);
            if (live) {
                mbar_arrive_expect_tx(bar_f, (uint32_t)F::state_bytes + x.m * row);
                bulk_load(at, a.state + x.u.slot * a.slot_stride + (int64_t)x.h * K * V, (uint32_t)F::state_bytes, bar_f);
            } else {
                mbar_arrive(bar_f);
            }
            mbar_arrive(armed + 8 * slot);
        }
        __syncwarp();
        if (lane < x.m) {
            const IO *k = static_cast<const IO *>(a.k) + x.u.b * a.sk.batch + hq * a.sk.head + x.tok * a.sk.token;
            const IO *v = static_cast<const IO *>(a.v) + x.u.b * a.sv.batch + x.h * a.sv.head + x.tok * a.sv.token;
            const uint32_t kb = K * sizeof(IO), vb = V * sizeof(IO), to = at + F::state_bytes;
            bulk_load(to + lane * kb, k, kb, bar_f);
            bulk_load(to + 2 * AHEAD * kb + lane * vb, v, vb, bar_f);
            if (a.o) {
                const IO *q = static_cast<const IO *>(a.q) + x.u.b * a.sq.batch + hq * a.sq.head + x.tok * a.sq.token;
                bulk_load(to + (AHEAD + lane) * kb, q, kb, bar_f);
            }
        }
    };
    if (threadIdx.x < 32) {
        if (lane == 0) {
            for (int i = 0; i < F::slots; ++i) mbar_init(full + 8 * i, 1), mbar_init(armed + 8 * i, 1), issued[i] = 0;
            *abort_flag = 0, *counter = 0;
            fence_mbar_init();
        }
        __syncwarp();
        wait_for_previous();
        for (int i = 0, item = blockIdx.x; i < F::slots && item < heads; ++i, item += gridDim.x) fetch(i, look(item));
    }
    if (threadIdx.x >= 32) wait_for_previous();
    __syncthreads();
    const int c = tid & 7, r = lane >> 3, at = 4 * r * V + (tid & ~31) + 4 * c;
    Stage<K, V, IO> &s = *reinterpret_cast<Stage<K, V, IO> *>(stages + group * F::stage_bytes);
    bool alive = true;  // no wait of this group has run out
    for (;;) {
        if (tid == 0) taken[group] = atomicAdd(counter, 1);
        named_bar(bar, V);  // the stage is free too
        const int i = taken[group], item = blockIdx.x + i * (int)gridDim.x;
        if (item >= heads) break;
        const int slot = i % F::slots, n = item / a.Hv, h = item - n * a.Hv;
        const int next = item + F::slots * gridDim.x;
        const Run u = run_of(a, n);
        const Head<K, V, IO> head(a, s, u, n, h, h / a.G, 0, tid, bar, true);
        const bool live = u.valid && u.slot >= 0 && u.slot < a.n_slots;
        int m = 0;
        bool more = false, bad = false;
        float4 S[NR];
        if (alive) {
            Ahead ahead;
            if (tid < 32 && next < heads) ahead = look(next);
            const uint32_t parity = (i / F::slots) & 1;
            const bool ok = mbar_wait_warp(armed + 8 * slot, parity, abort_flag) && mbar_wait_warp(full + 8 * slot, parity, abort_flag);
            const unsigned char *from = sm + slot * F::slot_bytes;
            m = ok ? info[slot].m : 0;
            more = info[slot].more, bad = info[slot].bad;
            const float *src = reinterpret_cast<const float *>(from) + at;
#pragma unroll
            for (int j = 0; j < NR; ++j) S[j] = *reinterpret_cast<const float4 *>(src + (16 * (j >> 2) + (j & 3)) * V);
            const uint4 *raw = reinterpret_cast<const uint4 *>(from + F::state_bytes);
            constexpr int ROW = K * (int)sizeof(IO) / 16;
            uint4 *sk = reinterpret_cast<uint4 *>(s.k), *sq = reinterpret_cast<uint4 *>(s.q);
            for (int e = tid; e < m * ROW; e += V) {
                sk[e] = raw[e];
                if (a.o) sq[e] = raw[AHEAD * ROW + e];
            }
            const IO *raw_v = reinterpret_cast<const IO *>(raw + 2 * AHEAD * ROW) + tid;
            for (int t = 0; t < m; ++t) s.v[t][tid] = raw_v[t * V];
            if (tid < m) s.a[tid] = info[slot].a[tid], s.b[tid] = info[slot].b[tid];
            alive = named_bar_and(bar, V, ok);
            if (alive && tid < 32 && next < heads) fetch(i + F::slots, ahead);
        }
        if (!live) {
            if (u.valid) head.fill(0, u.slot >= 0);
            continue;
        }
        if (!alive) {  // a copy did not arrive in a second: this head and all that follow show it
            head.fill(0, true);
            const float nan = __int_as_float(0x7fffffff);
#pragma unroll
            for (int j = 0; j < NR; ++j) S[j] = make_float4(nan, nan, nan, nan);
        } else if (!head.run(S, m, more, bad)) {
            continue;
        }
        float *dst = head.out(h) + at;
#pragma unroll
        for (int j = 0; j < NR; ++j) *reinterpret_cast<float4 *>(dst + (16 * (j >> 2) + (j & 3)) * V) = S[j];
    }
    __syncthreads();
    if (threadIdx.x == 0 && *abort_flag)  // no copy is left in flight
        for (int j = 0; j < F::slots; ++j)
            if (issued[j]) mbar_drain(full + 8 * j, (issued[j] - 1) & 1);
}

template <int K, typename IO> cudaError_t launch(const DecodeArgs &a, cudaStream_t st) {
    const int64_t heads = (int64_t)a.n_seqs * a.Hv;
    // rows that a bulk copy, or 16-byte ones, can take: multiples of 16 bytes apart
    const int64_t strides = a.sk.batch | a.sk.token | a.sk.head | a.sv.batch | a.sv.token | a.sv.head |
                            (a.o ? a.sq.batch | a.sq.token | a.sq.head : 0);
    const uintptr_t at = reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v) |
                         (a.o ? reinterpret_cast<uintptr_t>(a.q) : 0);
    const bool rows16 = !((strides * (int64_t)sizeof(IO)) & 15) && !(at & 15);
    // The ring pays for lists of tokens from about twelve states per SM on: 52.4 us against 52.8 of single warps at 2048
    // heads, 92 against 99 at 4096, 134 against 148 at 6144 (6 tokens at most; fp32: 148 against 156; 2 tokens: 129.5
    // against 126.4), but 31.8 against 30.0 at 1024.  Without lists warps are faster at every size (64 rows of 32 heads
    // with 1, 3 and 6 tokens: 44.7, 53.2 and 73.8 us against 46.0, 53.6 and 75.8; 16 rows: 13.4 against 14.2), for narrow
    // heads too (96 rows of 64 heads, 64 x 64, lists: 23 against 35).
    if constexpr (K == 128)
        if (a.token_indices && a.V == kGroup && heads >= 12 * kSMs && rows16) {
            static std::atomic<uint64_t> done{0};
            const cudaError_t e = allow_smem(k_recurrent_flow<IO>, Flow<IO>::bytes, done);
            if (e != cudaSuccess) return e;
            return launch_behind(k_recurrent_flow<IO>, dim3(kSMs), 2 * kGroup, Flow<IO>::bytes, st, a, (int)heads);
        }
    return launch_behind(k_recurrent<K, IO>, dim3((unsigned)a.n_seqs, (unsigned)a.Hq, (unsigned)(a.G * (a.V / kTile))), kTile, 0, st, a, rows16);
}

}  // namespace

cudaError_t launch_recurrent(const DecodeArgs &a, int K, gdn_dtype io, cudaStream_t st) {
    if (io == GDN_BF16) return K == 128 ? launch<128, __nv_bfloat16>(a, st) : launch<64, __nv_bfloat16>(a, st);
    return K == 128 ? launch<128, float>(a, st) : launch<64, float>(a, st);
}

}  // namespace gdn
