// tree_tc.cu -- the drafted-tree operator on the tensor cores (bf16 io).  The mathematics is in tree.cu, here as
//
//   o_t = scale Gam_t S^T q_t + sum_i W_ti R_i,  R_i = v_i - Gam_i S^T k_i,  W = scale P (I + L)^-1 diag(beta)
//
// because W needs no state: it is made while the state is on its way.  With L = diag(beta) N the blocks of W are
// W_b = (scale P_b - sum_{c > b} W_c N_cb) (I + L_bb)^-1 diag(beta_b).  One CTA computes a (row, value head):
//
//   all warps     rows of k and q into shared memory
//   group B       G = [K; Q] K^T (lane r: row r of K K^T, then of Q K^T); the products of e^g down the tree; N and
//                 P; W by blocks of 16 columns from the last on, 16 rows per warp on fragments that stay in registers
//   group A       S^T from its bulk copy to TMEM; D1 = S^T [K; Q]^T (lane v: S^T k_t, then S^T q_t, of column v);
//                 (I + L_bb)^-1 diag(beta_b); R^T to TMEM
//   all warps     D2 = R^T W^T (lane v: sum_i W_ti R_i of column v); o
//
// q and k are bf16 as given; S, R, L, P and W enter products as hi + lo bf16 pairs (16 bits; one bf16 rounding of
// them would cost as much as the rounding of o) and are kept in fp32 between them.
// A head with an output that is not finite is done again along its paths (along_paths; tree.cu says why).
// S arrives by one bulk copy (a head's state is contiguous); its place in shared memory then holds L, P, W and o, or,
// where these have a place of their own, the next head's state.
// Two CTAs stay on each SM (up to 110 KB, 256 TMEM columns each) and take head after head, so that one's copies run under
// the other's arithmetic; k, q and the gates of a CTA's next head come while group B finishes W.
//
// The states' way from memory is the floor.  64 rows of 64 heads, 64 nodes, 128 x 128, take 106 us where that is 66:
// a head's steps wait for each other (state, products, inverses, W, products, o), and two heads per SM do not fill
// the gaps (tensor pipe 18 %, instruction issue 36 %).  Before: CTAs that ended with their head 122 us, W by
// substitution on CUDA cores behind the state 247.  16 rows of 32 heads, 33 nodes: 15.5 us; one row, 7 nodes: 4.7 us.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>

#include "common.cuh"
#include "decode.h"
#include "tc.cuh"

namespace gdn {
namespace {

using namespace tc;

constexpr int GROUP = 128, NT = 2 * GROUP, kSMs = 152;
constexpr uint32_t kCols = 256;     // TMEM: S^T hi, lo (K columns), later R^T hi, lo and D2 | G, later D1
constexpr uint32_t kRlo = 32, kD2 = 64, kD1 = 128;
enum { BAR_S = 0, BAR_G = 8, BAR_D = 16, BAR_O = 24, BAR_K = 32, BAR_V = 40, BARS = 6 };  // state, G, D1, D2, k and q, v
enum { NB_STATE = 1, NB_B = 2, NB_FREE = 3, NB_A = 4, NB_DIAG = 5, NB_INV = 6, NB_OUT = 7, NB_WALK = 8 };  // named barriers

// q, k, v and o as [columns of all heads][token][batch]
struct RowMaps {
    CUtensorMap q, k, v, o;
    // the maps of q, k and v describe them (see rows_map); otherwise their rows are copied in pieces, by all threads:
    // 104 us with maps, 122 without for 64 rows of 64 heads, 64 nodes, 4.6 and 5.0 for one row, 7 nodes
    bool mapped;
    bool rows16;  // pieces of 16 bytes are aligned
};

template <int K, int V, int TP, bool APART> struct Map {
    // [K; Q] in blocks of 64 columns (as the 128 rows of an operand a block goes on into what follows, for rows of the
    // product that nobody reads), then the state
    static constexpr uint32_t KQ = 0, KQ_BLOCK = 2 * TP * 128, STATE = K / 64 * KQ_BLOCK, state = K * V * 4;
    // scratch: P in fp32, then row by row W (eight rows of hi, then of lo, in the place of eight of P), then o; L hi and
    // lo (halves of the same rows where 32 columns do); the blocks of L on the diagonal in fp32, by columns; their
    // inverses as hi, then lo, in rows of 48 bytes; v
    static constexpr uint32_t L_BYTES = TP * (TP <= 32 ? 128 : 256), DS = 20, DIAG_BYTES = TP * DS * 4, INV_BLOCK = 16 * 48;
    static constexpr uint32_t INV_BYTES = TP / 16 * 2 * INV_BLOCK, scratch = TP * 256 + L_BYTES + DIAG_BYTES + INV_BYTES + TP * V * 2;
    // the products of e^g from node i to node t >= i: rows t and TP - 1 - t share one (see table_row); the stride
    // puts eight neighbouring rows on different banks
    static constexpr uint32_t LS = TP + 4, TABLE_BYTES = TP / 2 * LS * 4;
    // (a, parent), the same of the parent, beta, Gam, scale Gam: TP each; gates and parents of the next head
    static constexpr uint32_t rest = TABLE_BYTES + 10 * TP * 4 + 8 * BARS + 32 + 1024;
    // APART: the scratch has a place of its own, and the next head's state comes while this one's products run.
    // Otherwise it lies over the state, once that is in TMEM.
    static constexpr uint32_t PW = STATE + (APART ? state : 0), LHI = PW + TP * 256, LLO = TP <= 32 ? LHI : LHI + TP * 128;
    static constexpr int L_LO = TP <= 32 ? 4 : 0;  // first 16-byte piece of lo in its rows
    static constexpr uint32_t DIAG = LHI + L_BYTES, INV = DIAG + DIAG_BYTES, VAL = INV + INV_BYTES;
    static constexpr uint32_t END = PW + scratch, TABLE = ((END > STATE + state ? END : STATE + state) + 15) / 16 * 16;
    static constexpr uint32_t VEC = TABLE + TABLE_BYTES, NEXT = VEC + 7 * TP * 4, BAR = NEXT + 3 * TP * 4, MISC = BAR + 8 * BARS;
    static constexpr uint32_t bytes = MISC + 32 + 1024;
    static_assert(TP * TP * 8 <= scratch, "L and P of along_paths");
};

// Where row t of the table begins: the first half of the rows at 0, with entries up to t at most; the others
// behind those of their partner TP - 1 - t, on a 16-byte boundary.
template <int TP> __host__ __device__ constexpr int table_row(int t) {
    return t < TP / 2 ? t * (TP + 4) : (TP - 1 - t) * (TP + 4) + ((TP - 1 - t + 4) & ~3);
}

__device__ __forceinline__ uint64_t kdesc(uint32_t a) { return sdesc_sw128(a, 16, 1024); }

__device__ __forceinline__ void bar_arrive(uint32_t id, uint32_t threads) {
    asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// Rows of all tokens of batch row n, from column x on
__device__ __forceinline__ void load_rows(uint32_t dst, const CUtensorMap *map, uint32_t bar, int x, int n) {
    tma_load_3d(dst, map, bar, x, 0, n);
}
__device__ __forceinline__ void store_rows(const CUtensorMap *map, uint32_t src, int x, int n) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(0), "r"(n), "r"(src)
                 : "memory");
}
// 16 bytes of a row, 0 where there is no such row; asynchronously where they are aligned
__device__ __forceinline__ void copy_piece(uint32_t dst, const __nv_bfloat16 *src, bool in, bool rows16) {
    if (in && rows16) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
        return;
    }
    uint32_t w[4] = {0, 0, 0, 0};
    if (in)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = (uint32_t)__bfloat16_as_ushort(src[2 * i]) | (uint32_t)__bfloat16_as_ushort(src[2 * i + 1]) << 16;
    st_shared_v4(dst, w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void copy_word(void *dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// Two fp32 products at once, on a pair of registers
__device__ __forceinline__ uint64_t pair_of(float lo, float hi) {
    uint64_t p;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(lo), "f"(hi));
    return p;
}
__device__ __forceinline__ void halves(uint64_t p, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(p));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
// split_pair with its two differences at once
__device__ __forceinline__ void split2(float x0, float x1, uint32_t &hi, uint32_t &lo) {
    hi = pack_bf16(x0, x1);
    uint64_t d;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(pair_of(x0, x1)), "l"(pair_of(__uint_as_float(hi << 16), __uint_as_float(hi & 0xFFFF0000u))));
    float d0, d1;
    halves(d, d0, d1);
    lo = pack_bf16(d0, d1);
}
// Fragments of 16 x 16 blocks: C as two 16 x 8 accumulators, A as hi and lo of four registers each.
struct Frag {
    uint32_t hi[4], lo[4];
};
__device__ __forceinline__ Frag split_frag(const float (&c)[8]) {  // C of a product -> A of the next
    Frag f;
#pragma unroll
    for (int i = 0; i < 4; ++i) split2(c[2 * i], c[2 * i + 1], f.hi[i], f.lo[i]);
    return f;
}
__device__ __forceinline__ void mma16816(float *c, const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// c += a B for a 16 x 16 block B [k][n] of bf16 hi and lo in shared memory; each lane gives the address of its row.
// The small products have sums of their own, so that no more than two follow each other.
__device__ __forceinline__ void block_product(float (&c)[8], const Frag &a, uint32_t b_hi, uint32_t b_lo) {
    uint32_t h[4], l[4];
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
                 : "r"(b_hi)
                 : "memory");
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(l[0]), "=r"(l[1]), "=r"(l[2]), "=r"(l[3])
                 : "r"(b_lo)
                 : "memory");
    float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        mma16816(c + 4 * j, a.hi, h[2 * j], h[2 * j + 1]);
        mma16816(x + 4 * j, a.lo, h[2 * j], h[2 * j + 1]);
        mma16816(x + 4 * j, a.hi, l[2 * j], l[2 * j + 1]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] += x[i];
}

// All outputs of a head, each sum over the nodes of a path alone, from the inputs in memory and what the head has left
// in shared memory: the products of e^g, beta (0 for nodes of no use), Gam, parents.  All threads; L and P in `scratch`.
// 0.06, 0.3 and 0.7 ms for 7, 33 and 64 nodes.  Looking for what is not finite costs 2 % of the heads' time elsewhere (64
// rows of 64 heads, 64 nodes: 103.4 -> 105.7 us); keeping it out of every operand as it came up took 128 us.
template <int K, int V, int TP>
__device__ __noinline__ void along_paths(const DecodeArgs &a, int head, int64_t slot, const float *table, const int4 *s_up, const float *s_b,
                                         const float *s_gam, uint64_t absent, uint64_t bad, float *scratch) {
    const int n = head / a.Hv, h = head - n * a.Hv, hq = h / a.G, T = a.T, tid = threadIdx.x;
    const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(a.q) + n * a.sq.batch + hq * a.sq.head;
    const __nv_bfloat16 *k = static_cast<const __nv_bfloat16 *>(a.k) + n * a.sk.batch + hq * a.sk.head;
    const __nv_bfloat16 *v = static_cast<const __nv_bfloat16 *>(a.v) + n * a.sv.batch + h * a.sv.head + tid;
    const float *S = a.state + slot * a.slot_stride + (int64_t)h * K * V + tid;
    __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(a.o) + ((int64_t)n * T * a.Hv + h) * V + tid;
    const uint64_t none = absent | bad;
    float2 *lp = reinterpret_cast<float2 *>(scratch);  // (L, P) of node t and i <= t, t TP + i
    for (int e = tid; e < T * TP; e += NT) {
        const int t = e / TP, i = e % TP;
        if (i > t || (none >> t & 1)) continue;
        float kk = 0.f, qk = 0.f;
#pragma unroll 4
        for (int j = 0; j < K; ++j) {
            const float x = __bfloat162float(k[i * a.sk.token + j]);
            kk = fmaf(__bfloat162float(k[t * a.sk.token + j]), x, kk);
            qk = fmaf(__bfloat162float(q[t * a.sq.token + j]), x, qk);
        }
        const float D = table[table_row<TP>(t) + i];
        lp[e] = make_float2(s_b[t] * D * kk, D * qk);
    }
    __syncthreads();
    if (tid < V) {
        float d[TP];
        for (int t = 0; t < T; ++t) {
            float ks = 0.f, qs = 0.f;
            if (!(none >> t & 1)) {
#pragma unroll 4
                for (int j = 0; j < K; ++j) {
                    ks = fmaf(__bfloat162float(k[t * a.sk.token + j]), S[j * V], ks);
                    qs = fmaf(__bfloat162float(q[t * a.sq.token + j]), S[j * V], qs);
                }
                float x = s_b[t] * (__bfloat162float(v[t * a.sv.token]) - s_gam[t] * ks), y = s_gam[t] * qs;
                for (int p = s_up[t].y; p >= 0; p = s_up[p].y) x = fmaf(-lp[t * TP + p].x, d[p], x);
                d[t] = x;
                for (int p = t; p >= 0; p = s_up[p].y) y = fmaf(lp[t * TP + p].y, d[p], y);
                qs = a.scale * y;
            }
            o[(int64_t)t * a.Hv * V] = __float2bfloat16_rn(bad >> t & 1 ? __int_as_float(0x7fffffff) : qs);
        }
    }
}

template <int K, int V, int TP, bool APART>
__global__ void __launch_bounds__(NT, 2) k_tree_tc(const __grid_constant__ DecodeArgs a, const __grid_constant__ RowMaps maps, int heads) {
    using M = Map<K, V, TP, APART>;
    constexpr uint32_t ID_1 = idesc_bf16(128, TP, 0, 0), ID_2 = idesc_bf16(128, 2 * TP, 0, 0);
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *sm = smem_align1024(smem_raw);
    const uint32_t sb = smem_u32(sm), bars = sb + M::BAR;
    const int t = threadIdx.x, warp = t >> 5, T = a.T, lane_row = t & (GROUP - 1);
    const float nan = __int_as_float(0x7fffffff);
    constexpr int SETUP = 7;  // the warp that sets up, copies the state and issues G
    constexpr int INVERTERS = (TP + 31) / 32 * 32;  // threads of group A's warps 1 and 2 that invert, rounded up to warps
    const bool group_b = t >= GROUP, column = lane_row < V;  // the same for a whole warp
    const int64_t o_tok = (int64_t)a.Hv * V;
    int4 *s_up = reinterpret_cast<int4 *>(sm + M::VEC);  // e^g (its bits) and the parent, then the parent's
    float *s_b = reinterpret_cast<float *>(s_up + TP), *s_gam = s_b + TP, *s_sg = s_gam + TP;
    float *table = reinterpret_cast<float *>(sm + M::TABLE);
    uint32_t *misc = reinterpret_cast<uint32_t *>(sm + M::MISC);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(misc + 1);
    uint32_t *s_absent = misc + 2, *s_bad = misc + 4, *s_found = misc + 6;  // nodes of each kind, a bit each; an output is not finite
    if (t == 32 * SETUP) {
        for (int i = 0; i < BARS; ++i) mbar_init(bars + 8 * i, 1);
        misc[1] = 0;
        fence_mbar_init();
    }
    __syncthreads();  // thread 0 uses BAR_K at once
    wait_for_previous();
    // What a head's turn begins with: rows of k and q on the way to shared memory (one copy each per 64 columns; what
    // is past the last node comes as 0), gates and parent of this thread's node too (in registers the compiler would
    // wait for them where it runs out of registers); returns the slot
    float *next_g = reinterpret_cast<float *>(sm + M::NEXT), *next_b = next_g + TP;
    int *next_up = reinterpret_cast<int *>(next_b + TP);
    auto look = [&](int head) -> int {
        const int n = head / a.Hv, h = head - n * a.Hv, hq = h / a.G;
        const int slot = a.state_indices ? a.state_indices[n] : n;
        if (t < T) {
            copy_word(next_g + t, a.g + n * a.sg.batch + h * a.sg.head + t * a.sg.token);
            copy_word(next_b + t, a.beta + n * a.sb.batch + h * a.sb.head + t * a.sb.token);
            copy_word(next_up + t, a.parents + (int64_t)n * T + t);
        }
        if (maps.mapped) {
            if (t == 0) {
                mbar_arrive_expect_tx(bars + BAR_K, 2 * TP * K * 2);
                for (int kb = 0; kb < K / 64; ++kb) {
                    load_rows(sb + M::KQ + kb * M::KQ_BLOCK, &maps.k, bars + BAR_K, hq * (int)a.sk.head + 64 * kb, n);
                    load_rows(sb + M::KQ + kb * M::KQ_BLOCK + TP * 128, &maps.q, bars + BAR_K, hq * (int)a.sq.head + 64 * kb, n);
                }
            }
        } else if (!group_b) {
            constexpr int PIECES = K / 8, ROWS = GROUP / PIECES;
            const int x = t % PIECES, r0 = t / PIECES;
            const __nv_bfloat16 *k = static_cast<const __nv_bfloat16 *>(a.k) + n * a.sk.batch + hq * a.sk.head + 8 * x;
            const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(a.q) + n * a.sq.batch + hq * a.sq.head + 8 * x;
            const uint32_t dst = sw128_addr(sb + M::KQ + (x >> 3) * M::KQ_BLOCK, r0, x & 7);
#pragma unroll 1
            for (int r = 0; r < TP; r += ROWS) {  // a multiple of eight rows at a time
                copy_piece(dst + r * 128, k + (r0 + r) * a.sk.token, r0 + r < T, maps.rows16);
                copy_piece(dst + (TP + r) * 128, q + (r0 + r) * a.sq.token, r0 + r < T, maps.rows16);
            }
        }
        return slot;
    };
    auto load_state = [&](int slot, int h) {  // one thread
        mbar_arrive_expect_tx(bars + BAR_S, M::state);
        bulk_load(sb + M::STATE, a.state + slot * a.slot_stride + (int64_t)h * K * V, M::state, bars + BAR_S);
    };
    int next_slot = look(blockIdx.x);
    bool ok = true, first = true, coming = false, asked = false;  // the next head's state is on its way; by this thread
    uint32_t phase = 0, phase_k = 0;  // of the mbarriers: each is used once per head, that of k and q for idle ones too
    for (int head = blockIdx.x; head < heads; head += gridDim.x) {
        const int n = head / a.Hv, h = head - n * a.Hv;
        __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(a.o) + ((int64_t)n * T * a.Hv + h) * V;
        const int slot = next_slot;
        const bool more = head + gridDim.x < heads, here = coming;
        int ahead = -1;  // the slot whose state is asked for before this head is done
        if (APART && more) ahead = a.state_indices ? a.state_indices[(head + gridDim.x) / a.Hv] : (head + gridDim.x) / a.Hv;
        coming = asked = false;
        if (slot < 0 || slot >= a.n_slots || !ok) {  // an idle row, no such slot, or a wait that ran out before
            if (t < V)
                for (int i = 0; i < T; ++i) o[i * o_tok + t] = __float2bfloat16_rn(slot < 0 ? 0.f : nan);
            copies_done();
            if (maps.mapped && t == 0) mbar_drain(bars + BAR_K, phase_k);  // their place is wanted again
            phase_k ^= 1;
            if (more) next_slot = look(head + gridDim.x);
            continue;
        }
        if (t == 32 * SETUP) {
            if (!here) load_state(slot, h);
            for (int i = 2; i < 7; ++i) misc[i] = 0;
        }
        if (warp == SETUP && first) {
            __syncwarp();
            tmem_alloc(sb + M::MISC, kCols);
        }
        first = false;
        for (int e = t; e < TP / 2 * (int)M::LS / 4; e += NT) reinterpret_cast<float4 *>(table)[e] = make_float4(0.f, 0.f, 0.f, 0.f);
        copies_done();
        if (t < TP) {  // what this thread copied
            const bool in = t < T;
            *reinterpret_cast<int2 *>(s_up + t) = make_int2(__float_as_int(in ? expf(next_g[t]) : 0.f), in ? next_up[t] : -1);
            s_b[t] = in ? next_b[t] : 0.f;
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        const uint32_t tmem = misc[0], lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        if (group_b) {
            if (warp == SETUP) {
                if (maps.mapped) ok = mbar_wait_warp(bars + BAR_K, phase_k, abort_flag);
                if (t == 32 * SETUP) {
                    for (int kb = 0; kb < K / 64; ++kb)
                        mma_chain<4, 2, 2>(tmem + kD1, kdesc(sb + M::KQ + kb * M::KQ_BLOCK), kdesc(sb + M::KQ + kb * M::KQ_BLOCK), ID_1, kb);
                    mma_commit(bars + BAR_G);
                }
                __syncwarp();
            }
            const int row = lane_row, node = row < TP ? row : row - TP;
            const bool has_row = row < 2 * TP, is_p = row >= TP;
            float *mine = table + table_row<TP>(has_row ? node : 0);
            constexpr int WALKERS = (TP + 31) / 32 * 32;  // the first warps of the group
            if (row < WALKERS) {  // each node's parent beside it: two steps for one access
                if (row < TP) {
                    const int up = s_up[node].y;
                    if (up >= 0 && up < node) reinterpret_cast<int2 *>(s_up + node)[1] = *reinterpret_cast<const int2 *>(s_up + up);
                }
                named_bar(NB_WALK, WALKERS);
            }
            if (row < TP) {  // from the node up to the state, leaving the products of e^g on the way
                float prod = 1.f;
                int p = node, kind = 0;
                auto step = [&](int a_bits, int up) {  // whether there is another node above p
                    mine[p] = prod;
                    if (up >= p || up < -1) kind = up < -1 ? 1 : 2;
                    prod *= kind ? 1.f : __int_as_float(a_bits);
                    p = up;
                    return !kind && up >= 0;
                };
                for (;;) {
                    const int4 up = s_up[p];
                    if (!step(up.x, up.y) || !step(up.z, up.w)) break;
                }
                if (kind) {  // nothing of such a node is used, whatever it holds
                    for (int i = 0; i <= node; ++i) mine[i] = 0.f;
                    atomicOr(&(kind == 1 ? s_absent : s_bad)[node >> 5], 1u << (node & 31));
                }
                const float b = kind ? 0.f : s_b[node];
                s_b[node] = b;
                s_gam[node] = kind ? 0.f : prod;
                s_sg[node] = kind ? 0.f : a.scale * prod;
            }
            ok = mbar_wait_warp(bars + BAR_G, phase, abort_flag) && ok;
            tc_fence_after();
            float x[TP];
#pragma unroll
            for (int c = 0; c < TP / 16; ++c) {
                uint32_t r[16];
                tmem_ld16(lanes + kD1 + 16 * c, r);
#pragma unroll
                for (int i = 0; i < 16; ++i) x[16 * c + i] = __uint_as_float(r[i]);
            }
            tc_fence_before();
            bar_arrive(NB_STATE, NT);
            named_bar(NB_B, GROUP);  // the products are there
            const bool dead = s_absent[0] | s_absent[1] | s_bad[0] | s_bad[1];
            if (has_row) {
                const float b = is_p ? a.scale : 1.f;
                const uint64_t bb = pair_of(b, b);
#pragma unroll
                for (int c = 0; c < TP / 4; ++c) {
                    const ulonglong2 d = reinterpret_cast<const ulonglong2 *>(mine)[c];
                    const uint64_t lo = mul2(mul2(bb, d.x), pair_of(x[4 * c], x[4 * c + 1]));
                    const uint64_t hi = mul2(mul2(bb, d.y), pair_of(x[4 * c + 2], x[4 * c + 3]));
                    // four entries past the node's are another row's; those of its own four are 0, and the diagonal of L,
                    // which nothing reads, may stay
                    const bool own = 4 * c <= node;
                    halves(own ? lo : 0, x[4 * c], x[4 * c + 1]);
                    halves(own ? hi : 0, x[4 * c + 2], x[4 * c + 3]);
                    if (dead) {
                        float f[4];
                        halves(d.x, f[0], f[1]);
                        halves(d.y, f[2], f[3]);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (f[i] == 0.f) x[4 * c + i] = 0.f;
                    }
                }
            }
            named_bar(NB_FREE, NT);  // the state's place is free
            if (has_row && is_p) {
                float4 *p = reinterpret_cast<float4 *>(sm + M::PW + node * 256);
#pragma unroll
                for (int c = 0; c < TP / 4; ++c)
                    p[c ^ (node & 15)] = make_float4(x[4 * c], x[4 * c + 1], x[4 * c + 2], x[4 * c + 3]);
            } else if (has_row) {
#pragma unroll
                for (int c = 0; c < TP / 8; ++c)
                    if ((node >> 4) == (c >> 1)) {
                        float *diag = reinterpret_cast<float *>(sm + M::DIAG) + ((node & ~15) + 8 * (c & 1)) * M::DS + (node & 15);
#pragma unroll
                        for (int i = 0; i < 8; ++i) diag[i * M::DS] = s_b[node] * x[8 * c + i];
                    }
            }
            bar_arrive(NB_DIAG, GROUP + INVERTERS);  // group A makes the inverses of the blocks on the diagonal
            if (has_row && !is_p)
#pragma unroll
                for (int c = 0; c < TP / 8; ++c) {
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) split_pair(x[8 * c + 2 * i], x[8 * c + 2 * i + 1], hi[i], lo[i]);
                    st_shared_v4(sw128_addr(sb + M::LHI, node, c), hi[0], hi[1], hi[2], hi[3]);
                    st_shared_v4(sw128_addr(sb + M::LLO, node, c + M::L_LO), lo[0], lo[1], lo[2], lo[3]);
                }
            named_bar(NB_INV, GROUP + INVERTERS);
            const int w = warp - 4, lane = t & 31;
            if (16 * w < TP) {  // rows 16 w .. 16 w + 15 of W: blocks beyond the w-th are 0
                const int g = lane >> 2, q2 = lane & 3;
                float c[TP / 16][8];
#pragma unroll
                for (int b = 0; b < TP / 16; ++b)
                    if (b <= w)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {  // (rows g, g + 8) x (columns 2 q2, 2 q2 + 1 of each half)
                            const int r = 16 * w + g + 8 * (i & 1), col = 16 * b + 8 * (i >> 1) + 2 * q2;
                            const float2 f = *reinterpret_cast<const float2 *>(sm + M::PW + r * 256 + ((col >> 2) ^ (r & 15)) * 16 +
                                                                               (col & 2) * 4);
                            c[b][4 * (i >> 1) + 2 * (i & 1)] = f.x;
                            c[b][4 * (i >> 1) + 2 * (i & 1) + 1] = f.y;
                        }
                __syncwarp();  // W takes the place of P's rows
                // the row of a 16 x 16 block whose address this lane gives, and the half
                const int br = (lane & 7) + (lane & 8), bh = lane >> 4;
#pragma unroll
                for (int b = TP / 16 - 1; b >= 0; --b) {
                    Frag f;
                    if (b <= w) {
                        float y[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                        const uint32_t inv = sb + M::INV + b * 2 * M::INV_BLOCK + br * 48 + bh * 16;
                        block_product(y, split_frag(c[b]), inv, inv + M::INV_BLOCK);
                        f = split_frag(y);
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i) f.hi[i] = f.lo[i] = 0u;
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r = 16 * w + g + 8 * (i & 1);
                        const uint32_t at = sb + M::PW + (r >> 3) * 2048 + (r & 7) * 128 + (((2 * b + (i >> 1)) ^ (r & 7)) << 4) + 4 * q2;
                        asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(f.hi[i]) : "memory");
                        asm volatile("st.shared.b32 [%0], %1;" ::"r"(at + 1024), "r"(f.lo[i]) : "memory");
                    }
                    if (b <= w) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) f.hi[i] ^= 0x80008000u, f.lo[i] ^= 0x80008000u;
#pragma unroll
                        for (int e = 0; e < b; ++e)
                            block_product(c[e], f, sw128_addr(sb + M::LHI, 16 * b + br, 2 * e + bh),
                                          sw128_addr(sb + M::LLO, 16 * b + br, M::L_LO + 2 * e + bh));
                    }
                }
                fence_proxy_async_smem();
            }
        } else {
            ok = mbar_wait_warp(bars + BAR_S, phase, abort_flag);
            if (column) {
                const float *s = reinterpret_cast<const float *>(sm + M::STATE) + t;
#pragma unroll 1
                for (int c = 0; c < K / 32; ++c) {
                    float y[32];
                    uint32_t hi[16], lo[16];
#pragma unroll
                    for (int i = 0; i < 32; ++i) y[i] = s[i * V];
                    s += 32 * V;
#pragma unroll
                    for (int i = 0; i < 16; ++i) split2(y[2 * i], y[2 * i + 1], hi[i], lo[i]);
                    tmem_st16x2(lanes + 16 * c, hi, lanes + K / 2 + 16 * c, lo);
                }
            }
            tc_fence_before();
            bar_arrive(NB_FREE, NT);
            named_bar(NB_STATE, NT);  // the state is in TMEM, G has been read
            if (warp == 0) {
                tc_fence_after();
                if (t == 0) {
                    if (maps.mapped) {  // v has its place now that the state has left it
                        mbar_arrive_expect_tx(bars + BAR_V, TP * V * 2);
                        load_rows(sb + M::VAL, &maps.v, bars + BAR_V, h * (int)a.sv.head, n);
                    }
                    for (int part = 0; part < 2; ++part)
                        for (int kb = 0; kb < K / 64; ++kb)
                            mma_chain_ta<4, 2>(tmem + kD1, tmem + part * (K / 2) + 32 * kb, kdesc(sb + M::KQ + kb * M::KQ_BLOCK), ID_2,
                                               part + kb);
                    mma_commit(bars + BAR_D);
                    asked = ahead >= 0 && ahead < a.n_slots && ok;  // this warp has seen the state arrive, all have taken it
                    if (asked) load_state(ahead, (head + gridDim.x) % a.Hv);
                }
                __syncwarp();
            } else if (t < 32 + INVERTERS) {
                named_bar(NB_DIAG, GROUP + INVERTERS);
                if (t >= 32 && t < 32 + TP) {  // a column of an inverse per thread: a finished y_i at once into all rows below it
                    const int u = t - 32, j0 = u & 15;
                    const float *diag = reinterpret_cast<const float *>(sm + M::DIAG) + (u & ~15) * M::DS;
                    float y[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) y[j] = j == j0 ? s_b[u] : 0.f;
#pragma unroll
                    for (int i = 0; i < 15; ++i) {
                        float l[16];
#pragma unroll
                        for (int j = (i + 1) / 4 * 4; j < 16; j += 4) {
                            const float4 f = *reinterpret_cast<const float4 *>(diag + i * M::DS + j);
                            l[j] = f.x, l[j + 1] = f.y, l[j + 2] = f.z, l[j + 3] = f.w;
                        }
#pragma unroll
                        for (int j = i + 1; j < 16; ++j) y[j] = fmaf(-l[j], y[i], y[j]);
                    }
                    unsigned char *inv = sm + M::INV + (u >> 4) * 2 * M::INV_BLOCK + 2 * j0;
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const __nv_bfloat16 hi = __float2bfloat16_rn(y[j]);
                        *reinterpret_cast<__nv_bfloat16 *>(inv + j * 48) = hi;
                        *reinterpret_cast<__nv_bfloat16 *>(inv + M::INV_BLOCK + j * 48) = __float2bfloat16_rn(y[j] - __bfloat162float(hi));
                    }
                }
                bar_arrive(NB_INV, GROUP + INVERTERS);
            }
            ok = mbar_wait_warp(bars + BAR_D, phase, abort_flag) && ok;
            tc_fence_after();
            if (maps.mapped) {
                ok = mbar_wait_warp(bars + BAR_V, phase, abort_flag) && ok;
            } else {
                const __nv_bfloat16 *v = static_cast<const __nv_bfloat16 *>(a.v) + n * a.sv.batch + h * a.sv.head;
                for (int e = t; e < TP * (V / 8); e += GROUP) {
                    const int r = e / (V / 8), c = e % (V / 8);
                    copy_piece(sb + M::VAL + 16 * e, v + r * a.sv.token + 8 * c, r < T, maps.rows16);
                }
                copies_done();
                named_bar(NB_A, GROUP);
            }
            const bool dead = s_absent[0] | s_absent[1] | s_bad[0] | s_bad[1];
            const __nv_bfloat16 *vs = reinterpret_cast<const __nv_bfloat16 *>(sm + M::VAL) + t;
            if (column)
#pragma unroll 1
                for (int c = 0; c < TP / 16; ++c) {
                    uint32_t ks[16], hi[8], lo[8];
                    float gam[16], y[16];
                    tmem_ld16(lanes + kD1 + 16 * c, ks);
                    lds16f(s_gam + 16 * c, gam);
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        y[j] = fmaf(-gam[j], __uint_as_float(ks[j]), __bfloat162float(vs[(16 * c + j) * V]));
                    if (dead) {
                        const uint32_t gone = (s_absent[c >> 1] | s_bad[c >> 1]) >> (16 * (c & 1));
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            if (gone >> j & 1) y[j] = 0.f;
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) split2(y[2 * i], y[2 * i + 1], hi[i], lo[i]);
                    tmem_st8x2(lanes + 8 * c, hi, lanes + kRlo + 8 * c, lo);
                }
        }
        if (more) next_slot = look(head + gridDim.x);  // the products have read k and q
        coming = ahead >= 0 && ahead < a.n_slots;
        tc_fence_before();
        ok = __syncthreads_and(ok) != 0;
        tc_fence_after();
        if (ok) {
            if (t == 0) {
                const uint64_t hi = sdesc_sw128(sb + M::PW, 16, 2048), lo = sdesc_sw128(sb + M::PW + 1024, 16, 2048);
                mma_chain_ta<TP / 16, 2>(tmem + kD2, tmem, hi, ID_1, 0);
                mma_chain_ta<TP / 16, 2>(tmem + kD2, tmem + kRlo, hi, ID_1, 1);
                mma_chain_ta<TP / 16, 2>(tmem + kD2, tmem, lo, ID_1, 1);
                mma_commit(bars + BAR_O);
            }
            __syncwarp();
            ok = mbar_wait_warp(bars + BAR_O, phase, abort_flag);
            tc_fence_after();
            // o by way of shared memory (the place of W, whose products are done), all rows in one copy
            __nv_bfloat16 *s_o = reinterpret_cast<__nv_bfloat16 *>(sm + M::PW);
            if (column)
#pragma unroll 1
                for (int c = t / GROUP; 16 * c < T; c += 2) {
                    uint32_t sq[16], d2[16];
                    float sg[16];
                    tmem_ld16x2(lanes + kD1 + TP + 16 * c, sq, lanes + kD2 + 16 * c, d2);
                    lds16f(s_sg + 16 * c, sg);
                    uint64_t zeros = 0;
#pragma unroll
                    for (int i = 0; i < 16; i += 2) {
                        const float y0 = fmaf(sg[i], __uint_as_float(sq[i]), __uint_as_float(d2[i]));
                        const float y1 = fmaf(sg[i + 1], __uint_as_float(sq[i + 1]), __uint_as_float(d2[i + 1]));
                        s_o[(16 * c + i) * V + lane_row] = __float2bfloat16_rn(y0);
                        s_o[(16 * c + i + 1) * V + lane_row] = __float2bfloat16_rn(y1);
                        zeros = fma2(pair_of(y0, y1), 0, zeros);
                    }
                    float z0, z1;
                    halves(zeros, z0, z1);
                    if (z0 + z1 != 0.f) {  // whatever nodes hold that give no output, it is none of this
                        const uint32_t none = (s_absent[c >> 1] | s_bad[c >> 1]) >> (16 * (c & 1));
                        for (int i = 0; i < 16; ++i)
                            if (!(none >> i & 1) && !(fabsf(__bfloat162float(s_o[(16 * c + i) * V + lane_row])) < INFINITY)) *s_found = 1;
                    }
                }
            fence_proxy_async_smem();
            named_bar(NB_OUT, NT);
            const bool dead = s_absent[0] | s_absent[1] | s_bad[0] | s_bad[1], again = *s_found;
            if (again) {
                along_paths<K, V, TP>(a, head, slot, table, s_up, s_b, s_gam, s_absent[0] | (uint64_t)s_absent[1] << 32,
                                      s_bad[0] | (uint64_t)s_bad[1] << 32, reinterpret_cast<float *>(sm + M::PW));
            } else if (dead) {
                for (int i = t / GROUP; i < T && column; i += 2) {
                    if (s_absent[i >> 5] >> (i & 31) & 1) s_o[i * V + lane_row] = __float2bfloat16_rn(0.f);
                    if (s_bad[i >> 5] >> (i & 31) & 1) s_o[i * V + lane_row] = __float2bfloat16_rn(nan);
                }
                fence_proxy_async_smem();
                named_bar(NB_OUT, NT);
            }
            if (t == 0 && !again) {  // rows past the last node are not written
                store_rows(&maps.o, sb + M::PW, h * V, n);
                bulk_commit();
                bulk_wait_read_all();
            }
        }
        fence_proxy_async_smem();  // the next state comes over what has been written here
        tc_fence_before();
        ok = __syncthreads_and(ok) != 0;
        if (!ok) {  // a wait ran out (its limit is a second): no copy of a state is left in flight, and the rows show it
            if (t == 0) mbar_drain(bars + BAR_S, phase);
            if (asked) mbar_drain(bars + BAR_S, phase ^ 1);
            if (t < V)
                for (int i = 0; i < T; ++i) o[i * o_tok + t] = __float2bfloat16_rn(nan);
        }
        phase ^= 1, phase_k ^= 1;
    }
    copies_done();
    if (t == 0) bulk_wait_all();
    __syncthreads();
    if (warp == SETUP && !first) {
        tc_fence_after();
        tmem_dealloc(misc[0], kCols);
    }
}

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult found;
        const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found);
        const bool ok = e == cudaSuccess && found == cudaDriverEntryPointSuccess;
        return ok ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p) : nullptr;
    }();
    return fn;
}

// A map of [B][T] rows that hold all heads, boxes of `columns` of all tokens (`rows`, zeros past the last).  False
// where the layout is another: strides that are no multiples of 16 bytes, heads outside the tokens, rows that overlap.
bool rows_map(CUtensorMap *m, const void *p, int width, int heads, int T, int B, const gdn_strides &s, int columns, int rows,
              CUtensorMapSwizzle swizzle) {
    const int64_t across = heads > 1 ? (heads - 1) * s.head + width : width;  // elements of a row
    if ((heads > 1 && (s.head < width || s.head % 8)) || across > INT32_MAX) return false;
    const int64_t batch = B > 1 ? s.batch : 0, token = T > 1 ? s.token : B > 1 ? batch : across;
    if (token < across || token % 8 || token > (1ll << 38)) return false;
    if (B > 1 && (batch < T * token || batch % token || batch > (1ll << 38))) return false;
    const auto fn = encoder();
    if (!fn || (reinterpret_cast<uintptr_t>(p) & 15)) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)across, (cuuint64_t)T, (cuuint64_t)B};
    const cuuint64_t strides[2] = {(cuuint64_t)token * 2, (cuuint64_t)(B > 1 ? batch : T * token) * 2};
    const cuuint32_t box[3] = {(cuuint32_t)columns, (cuuint32_t)rows, 1}, step[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(p), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
              swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int K, int V, int TP, bool APART = false> cudaError_t launch(const DecodeArgs &a, cudaStream_t st) {
    constexpr int bytes = (int)Map<K, V, TP, APART>::bytes;
    static_assert(2 * (bytes + 1024) <= 233472, "two CTAs per SM");
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(k_tree_tc<K, V, TP, APART>, bytes, done);
    if (e != cudaSuccess) return e;
    RowMaps maps;
    const gdn_strides so = {(int64_t)a.T * a.Hv * V, (int64_t)a.Hv * V, V};
    if (!rows_map(&maps.o, a.o, V, a.Hv, a.T, a.n_seqs, so, V, TP, CU_TENSOR_MAP_SWIZZLE_NONE)) return cudaErrorInvalidValue;
    maps.mapped = rows_map(&maps.q, a.q, K, a.Hq, a.T, a.n_seqs, a.sq, 64, TP, CU_TENSOR_MAP_SWIZZLE_128B) &&
                  rows_map(&maps.k, a.k, K, a.Hq, a.T, a.n_seqs, a.sk, 64, TP, CU_TENSOR_MAP_SWIZZLE_128B) &&
                  rows_map(&maps.v, a.v, V, a.Hv, a.T, a.n_seqs, a.sv, V, TP, CU_TENSOR_MAP_SWIZZLE_NONE);
    const int64_t steps = a.sq.batch | a.sq.token | a.sq.head | a.sk.batch | a.sk.token | a.sk.head | a.sv.batch | a.sv.token |
                          a.sv.head;
    const uintptr_t at = reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v);
    maps.rows16 = !(steps & 7) && !(at & 15);
    const int heads = a.n_seqs * a.Hv;
    return launch_behind(k_tree_tc<K, V, TP, APART>, dim3((unsigned)(heads < 2 * kSMs ? heads : 2 * kSMs)), NT, bytes, st, a, maps, heads);
}

// Products, tables and W are as wide as the nodes, rounded up to blocks of 16: 16 rows of 32 heads with 16, 32 and 48
// nodes take 11.5, 13.9 and 16.0 us and with 64 as the only width 16.2, 17.0 and 17.6; one row of 7 nodes 4.8 and 6.7.
template <int K, int V> cudaError_t launch_nodes(const DecodeArgs &a, cudaStream_t st) {
    // The scratch apart from the state, and the state asked for ahead, from more than two turns of the CTAs on: 64 rows
    // of 64 heads with 16 nodes 62.2 us against 73.6, with 32 75.3 against 83.7; 768 heads with 7 nodes 16.4 and 16.5,
    // but 512 12.0 and 11.0.  Narrower states lose by it at every size (64 x 64, 64 rows of 64 heads, 32 nodes: 65.8
    // and 61.3 us), and with more nodes two CTAs do not fit on an SM.
    if constexpr (K == 128 && V == 128)
        if (a.T <= 32 && (int64_t)a.n_seqs * a.Hv >= 4 * kSMs) return a.T <= 16 ? launch<K, V, 16, true>(a, st) : launch<K, V, 32, true>(a, st);
    if (a.T <= 16) return launch<K, V, 16>(a, st);
    if (a.T <= 32) return launch<K, V, 32>(a, st);
    if (a.T <= 48) return launch<K, V, 48>(a, st);
    return launch<K, V, 64>(a, st);
}
template <int K> cudaError_t launch_width(const DecodeArgs &a, cudaStream_t st) {
    return a.V == 128 ? launch_nodes<K, 128>(a, st) : launch_nodes<K, 64>(a, st);
}

}  // namespace

cudaError_t launch_tree_tc(const DecodeArgs &a, int K, cudaStream_t st) {
    return K == 128 ? launch_width<128>(a, st) : launch_width<64>(a, st);
}

}  // namespace gdn
