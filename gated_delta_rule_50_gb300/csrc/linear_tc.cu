// linear_tc.cu -- runs of linear attention (linear.h) on the tensor cores: bf16 inputs, chunks of 64 tokens.
//
// One CTA takes a head of a sequence (or of one of its segments) from chunk to chunk.  All products are tcgen05 with
// M = 128, in the form whose rows are the columns of c, so that TMEM lane y holds column y of c, out and the state; two
// threads keep X^T[y][:], the state, in registers (fp32), half a row each.  Per chunk, with a, b, c its rows:
//
//   P      = a b^T                          (rows of b below a's in the operand: M = 128, the lower half unused)
//   P~     = p_scale l^|r - i| P, r >= i    (CUDA cores; hi + lo bf16 into shared memory)
//   I^T    = X^T a^T                        (X hi + lo, from TMEM)
//   O^T    = c^T P~^T                       (c as it lies, hi + lo of P~)
//   out_r  = o_scale l^(j + e) I_r + O_r    (CUDA cores)
//   U^T    = (w c)^T b                      (w c as hi + lo from TMEM, and a third part where the final state is wanted)
//   X     <- l^n X + U
//
// Operands made here (X, P~, w c) enter as hi + lo bf16 pairs, which keeps about 16 bits: one rounding of any of them
// would cost as much as the rounding of out.  A final state is fp32, so that w c then gets a third part (24 bits): with
// two it is off by 3e-6 of itself.
//
// Tokens past the end of a sequence in its last chunk belong to its neighbour, and may hold anything: the producer clears
// them in shared memory before anyone reads them.
//
// Roles (512 threads): warps 0 and 1 make P~, warp 2 loads (TMA, three stages), warp 3 issues the products, warps 4 .. 11
// keep the state and write out, warps 12 .. 15 make w c.  Per chunk the tensor cores are asked for, in this order,
//     U(j), P(j + 1), I(j), O(j)
// and the others follow them: w c while I(j - 1) and O(j - 1) run, U, X and out from I(j - 1)'s end on, P~(j + 1) until O(j + 1).
//
// 4 sequences of 4096 tokens, 32 heads of 128 x 128 on 16 of q and k, with their final states: 123 us (112 without them),
// 3.3 TB/s; 1.9 us a chunk, 1.4 where only the state is wanted.  What bounds it is the products in their order: without any
// conversion and without out 100 us are left, of which the 44 products of a chunk (40 without a third part of w c) take 2600 to
// 2900 of 3000 cycles at the rates that they have alone (w c with b across rows 89 cycles, the others 46 to 77, where 32 would be full rate); the tensor
// pipe counts 50 % as active.  The conversions read and write the shared memory from which the operands come, and slow them
// down to 3800 cycles a chunk.  Chunks of 64: half of P's rows and of P~ are not used, at 128 it would be as much of O; and
// three stages of 128 tokens are 288 KB, where two of 64 already cost a third of the speed.
// Two stages instead of three: 241 -> 330 us (2 x 8192 tokens, 64 heads).  28 warps instead of 16, products issued by two
// warps, out and I in one accumulator: within 3 % of this.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "common.cuh"
#include "decode.h"
#include "linear.h"
#include "tc.cuh"

namespace gdn {
namespace {

using namespace tc;

constexpr int kThreads = 512, kStages = 3;
constexpr int W_TMA = 2, W_MMA = 3, W_MAIN0 = 4, W_W0 = 12;  // warps 0 and 1: P~
constexpr uint32_t kMainWarps = 8, kWWarps = 4;

// shared memory (bytes from a 1024-aligned base)
constexpr uint32_t STAGE = 49152, BOX = 8192;  // a stage: {a, b} of columns 0 .. 63, {a, b} of 64 .. 127, c of both
constexpr uint32_t B_OFF = BOX, KB = 2 * BOX, C_OFF = 4 * BOX;
constexpr uint32_t SM_P = kStages * STAGE;   // P~ {hi, lo} [64 r][64 i], two buffers
constexpr uint32_t SM_W3 = SM_P + 4 * BOX;   // third part of (w c)^T [128 y][64 i], two buffers
constexpr uint32_t SM_OUT = SM_W3 + 4 * BOX; // out on its way, 2 KB per warp
constexpr uint32_t SM_TAB = SM_OUT + kMainWarps * 2048;
struct Tables {
    float mask[128];               // p_scale l^d, d = r - i in the order of the scan, at 64 + r - i of the tile's rows; 0 for d < 0
    float into[2][64], up[2][64];  // weights of I's and of c's rows; [1]: of the last chunk
};
constexpr uint32_t SM_BAR = SM_TAB + (uint32_t)sizeof(Tables);
enum {
    FULL0 = 0, EMPTY0 = FULL0 + kStages, TAIL = EMPTY0 + kStages, PDONE, PREAD, PREADY0, PREADY1, WREADY0, WREADY1, UDONE0, UDONE1, XREADY, IDONE, ODONE, FINAL, BARRIERS
};
constexpr uint32_t SM_MISC = SM_BAR + 8 * 32;
constexpr uint32_t SMEM_BYTES = SM_MISC + 64 + 1024;
static_assert(BARRIERS <= 32 && SMEM_BYTES <= 232448, "shared memory");

// TMEM columns
constexpr uint32_t TM_XH = 0, TM_XL = 64, TM_U = 128, TM_P = 256, TM_I = 320, TM_O = 384, TM_W = 448, TM_WL = 32;
// Where only the state is wanted, P, I, O and X are not there, and U and W have second buffers in their place
constexpr uint32_t TM_U1 = 256, TM_W1 = 0;

constexpr uint32_t ID_N64 = idesc_bf16(128, 64, 0, 0), ID_N64_AMN = idesc_bf16(128, 64, 1, 0);

// Two loads of 16 lanes x 32 columns, waited: thread t has, of every eight columns, 2 (t % 4) and the next one of lane t / 4
// (two registers) and of lane t / 4 + 8 (two more), as a matrix fragment has them
#define GDN_R8(r, o) "=r"(r[o]), "=r"(r[o + 1]), "=r"(r[o + 2]), "=r"(r[o + 3]), "=r"(r[o + 4]), "=r"(r[o + 5]), "=r"(r[o + 6]), "=r"(r[o + 7])
__device__ __forceinline__ void tmem_ld_fragments(uint32_t ta, uint32_t (&a)[16], uint32_t tb, uint32_t (&b)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%32];\n\t"
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, "
        "[%33];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : GDN_R8(a, 0), GDN_R8(a, 8), GDN_R8(b, 0), GDN_R8(b, 8)
        : "r"(ta), "r"(tb)
        : "memory");
}
#undef GDN_R8
// Two stores of 16 lanes x 32 columns, waited: thread t gives, of every four columns, t % 4 of lane t / 4 and of lane t / 4 + 8
#define GDN_S8(r, o) "r"(r[o]), "r"(r[o + 1]), "r"(r[o + 2]), "r"(r[o + 3]), "r"(r[o + 4]), "r"(r[o + 5]), "r"(r[o + 6]), "r"(r[o + 7])
__device__ __forceinline__ void tmem_st_fragments(uint32_t ta, const uint32_t (&a)[16], uint32_t tb, const uint32_t (&b)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x128b.x8.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};\n\t"
        "tcgen05.st.sync.aligned.16x128b.x8.b32 [%33], {%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};\n\t"
        "tcgen05.wait::st.sync.aligned;" ::GDN_S8(a, 0), GDN_S8(a, 8), GDN_S8(b, 0), GDN_S8(b, 8), "r"(ta), "r"(tb)
        : "memory");
}
#undef GDN_S8
// Four 8 x 8 matrices of 16-bit values; lane l gives row l % 8 of matrix l / 8.  Loaded with rows and columns exchanged, and
// stored as they are
__device__ __forceinline__ void load_transposed(uint32_t addr, uint32_t (&x)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];" : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void store_rows(uint32_t addr, const uint32_t (&x)[4]) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]) : "memory");
}
// Four 8 x 8 matrices of bf16 fragments, stored with rows and columns exchanged; lane l gives row l % 8 of matrix l / 8
__device__ __forceinline__ void store_transposed(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

struct Maps {
    CUtensorMap a, b, c;
};

// A try at a wait that may last kHold ns: warps that wait then issue nothing (tries without it end after some 80 cycles, and
// their loops took a third of all issue slots)
constexpr uint32_t kHold = 100000;
__device__ __forceinline__ bool try_for(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(kHold)
        : "memory");
    return ok != 0;
}
// Waits of one thread and of a whole warp, with one answer: false, and *abort set, after WAIT_NS, or once another has given up
__device__ __forceinline__ bool wait_alone(uint32_t bar, uint32_t parity, volatile int *abort) {
    if (try_for(bar, parity)) return true;
    const uint64_t t0 = global_ns();
    while (!try_for(bar, parity)) {
        if (!*abort && global_ns() - t0 < WAIT_NS) continue;
        *abort = 1;
        return false;
    }
    return true;
}
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, volatile int *abort) {
    return __all_sync(~0u, wait_alone(bar, parity, abort));
}
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
// Rounds a pair to bf16; what is left of it
__device__ __forceinline__ uint32_t take_bf16(uint64_t &x) {
    float x0, x1;
    halves(x, x0, x1);
    const uint32_t hi = pack_bf16(x0, x1);
    uint64_t d;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(x), "l"(pair_of(__uint_as_float(hi << 16), __uint_as_float(hi & 0xFFFF0000u))));
    x = d;
    return hi;
}
__device__ __forceinline__ uint32_t last_bf16(uint64_t x) {
    float x0, x1;
    halves(x, x0, x1);
    return pack_bf16(x0, x1);
}
// Products are issued by one elected thread, unrolled: the compiler then keeps addresses in uniform registers, and an issue
// takes about 30 cycles (52 by a thread that it cannot tell for one, 65 and 90 in loops; the product itself takes 32 at
// N = 64).  Descriptors (sdesc_sw128) as their lower words: the upper one is the same for all, groups of eight rows are
// 1024 bytes apart.
__device__ __forceinline__ bool elected() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(r));
    return r != 0;
}
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc(uint32_t addr, uint32_t lbo) { return ((addr & 0x3FFFFu) >> 4) | (lbo >> 4 << 16); }
template <uint32_t IDESC, bool ADD> __device__ __forceinline__ void product(uint32_t d, uint32_t a, uint32_t b) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tsetp.ne.b32 p, %3, 0;\n\tmov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "n"((int)ADD), "n"(IDESC), "n"(kDescHigh)
        : "memory");
}
template <uint32_t IDESC, bool ADD> __device__ __forceinline__ void product_ta(uint32_t d, uint32_t a, uint32_t b) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\tsetp.ne.b32 p, %3, 0;\n\tmov.b64 y, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "n"((int)ADD), "n"(IDESC), "n"(kDescHigh)
        : "memory");
}
// Four steps of 16 along the contraction: descriptors advance by ASTEP and BSTEP (16 bytes), A in TMEM by 8 columns
template <uint32_t IDESC, bool ADD, int ASTEP, int BSTEP> __device__ __forceinline__ void products(uint32_t d, uint32_t a, uint32_t b) {
    product<IDESC, ADD>(d, a, b);
#pragma unroll
    for (int i = 1; i < 4; ++i) product<IDESC, true>(d, a + i * ASTEP, b + i * BSTEP);
}
template <uint32_t IDESC, bool ADD, int BSTEP> __device__ __forceinline__ void products_ta(uint32_t d, uint32_t a, uint32_t b) {
    product_ta<IDESC, ADD>(d, a, b);
#pragma unroll
    for (int i = 1; i < 4; ++i) product_ta<IDESC, true>(d, a + 8 * i, b + i * BSTEP);
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, uint32_t bar, int x, int y, int z, int w) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
        : "memory");
}

enum { NO_OUT, BF16_OUT, F32_OUT };
template <int DA, int OUT, bool THIRD>
__global__ void __launch_bounds__(kThreads, 1) k_linear_tc(const __grid_constant__ Maps maps, const __grid_constant__ LinearRun r) {
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *sm = smem_align1024(smem_raw);
    const uint32_t sb = smem_u32(sm);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t *misc = reinterpret_cast<uint32_t *>(sm + SM_MISC);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(misc + 1);
    Tables &tab = *reinterpret_cast<Tables *>(sm + SM_TAB);
    auto bar = [&](int i) { return sb + SM_BAR + 8u * (uint32_t)i; };
    const int h = blockIdx.x % r.Hv, slot = blockIdx.x / r.Hv;
    int seq, part;
    LinearSpan span;
    if (r.seg_chunks) {  // many slots may have nothing to do: they leave at once
        wait_for_previous();
        span = linear_place(r, slot, seq, part);
        if (seq < 0 || (r.mode == LIN_SEG && part + 1 >= span.segs)) return;
    }

    if (threadIdx.x == 0) {
        // of 64 columns only half of these warps have any
        const uint32_t x = r.dc == 128 ? kMainWarps : kMainWarps / 2, w = x + (r.dc == 128 ? kWWarps : kWWarps / 2);
        const uint32_t counts[BARRIERS] = {1, 1, 1, 1, 1, 1, 1, 1, 2, 2, 2, w, w, 1, 1, x, 1, 1, 1};
        for (int i = 0; i < BARRIERS; ++i) mbar_init(bar(i), counts[i]);
        misc[1] = 0;
        fence_mbar_init();
    }
    if (warp == W_MMA) tmem_alloc(sb + SM_MISC, 512);
    if (warp == W_TMA && lane == 0) prefetch_tmap(&maps.a), prefetch_tmap(&maps.b), prefetch_tmap(&maps.c);
    if (!r.seg_chunks) {
        wait_for_previous();
        span = linear_place(r, slot, seq, part);
    }

    const int c0 = min(span.chunks, part * span.per_seg), c1 = min(span.chunks, c0 + span.per_seg);
    const int64_t unit = (int64_t)seq * r.Hv + h, words = (int64_t)DA * r.dc;
    bool init_t = r.transposed, fin_t = r.transposed, live = seq >= 0;
    const float *init = live && r.init ? r.init + unit * words : nullptr;
    float *fin = live && r.fin ? r.fin + unit * words : nullptr, *seg = r.seg + ((int64_t)slot * r.Hv + h) * words;
    constexpr bool outs = OUT != NO_OUT, F32OUT = OUT == F32_OUT;
    // The buffer of U(j) and w c(j), how often it has been used before, and the chunk that takes it next
    auto buffer = [](int j) { return outs ? 0 : j & 1; };
    auto turn = [](int j) { return outs ? j : j >> 1; };
    constexpr int kNext = outs ? 1 : 2;
    if (r.mode == LIN_SEG) {  // the last segment feeds no other
        live = live && c1 < span.chunks && c0 < c1;
        init = nullptr, fin = seg, fin_t = false;
    } else {
        if (part > 0) {
            live = live && c0 < c1;
            init = seg, init_t = false;
        }
    }
    if (!live || (r.mode != LIN_SEG && c1 < span.chunks)) fin = nullptr;
    const int nck = live ? c1 - c0 : 0, updates = fin ? nck : nck - 1;  // chunks whose part in the state is wanted
    const int first = span.first, batch = r.cu ? 0 : seq;
    // chunk j of this CTA: its lowest token in the row, and its tokens
    auto tokens = [&](int j) { return min(C, span.tokens - (c0 + j) * C); };
    auto token0 = [&](int j) {
        const int at = (c0 + j) * C;
        return first + (r.reverse ? span.tokens - at - tokens(j) : at);
    };
    const float g = r.g ? r.g[h] : 0.f;
    {  // tables: powers of l by the rows of the tile
        auto power = [&](int d) { return d <= 0 ? (d == 0 ? 1.f : 0.f) : expf(g * (float)d); };
        const int t = threadIdx.x, n = nck > 0 ? tokens(nck - 1) : C;
        if (t < 128) {
            const int d = r.reverse ? 64 - t : t - 64;
            tab.mask[t] = d < 0 ? 0.f : r.p_scale * power(d);
        } else if (t < 384) {
            const int k = t - 128, i = k & 63, which = k >> 6 & 1, m = which ? n : C;
            const int j = r.reverse ? m - 1 - i : i;
            if (k < 128) tab.into[which][i] = i < m ? r.o_scale * power(j + r.e) : 0.f;
            else tab.up[which][i] = i < m ? r.s_scale * power(m - j - r.e) : 0.f;
        }
        // what the order of the scan forbids stays 0: rows 0 .. 31 with columns 32 .. 63, or the reverse
        for (int i = t; i < 4 * 32 * 4; i += kThreads) {  // buffer and half, row, 16 bytes
            const int row = (i >> 2 & 31) + (r.reverse ? 32 : 0), chunk = (i & 3) + (r.reverse ? 0 : 4);
            st_shared_v4(sw128_addr(sb + SM_P + (uint32_t)(i >> 7) * BOX, row, chunk), 0, 0, 0, 0);
        }
        fence_proxy_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = misc[0];
    const uint32_t boxes_a = DA / 64, boxes_c = (uint32_t)r.dc / 64;
    auto stage = [&](int j) { return sb + (uint32_t)(j % kStages) * STAGE; };

    if (warp == W_TMA) {
        const uint32_t bytes = BOX * ((outs ? 2 : 1) * boxes_a + boxes_c);
        const int ha = h / r.ga, hb = h / r.gb, hc = h / r.gc;
        int issued = 0;
        bool tail = false;
#pragma unroll 1
        for (int j = 0; j < nck; ++j) {
            const int st = j % kStages;
            if (j >= kStages && !wait_for(bar(EMPTY0 + st), (j / kStages - 1) & 1, abort_flag)) break;
            tail = tokens(j) < C;
            const uint32_t to = tail ? bar(TAIL) : bar(FULL0 + st), at = stage(j);
            if (lane == 0 && j != r.drop_chunk) {
                const int tok = token0(j);
                mbar_arrive_expect_tx(to, bytes);
                for (uint32_t x = 0; x < boxes_a; ++x) {
                    if (outs) tma_load_4d(at + x * KB, &maps.a, to, 64 * x, ha, tok, batch);
                    tma_load_4d(at + x * KB + B_OFF, &maps.b, to, 64 * x, hb, tok, batch);
                }
                for (uint32_t x = 0; x < boxes_c; ++x) tma_load_4d(at + C_OFF + x * BOX, &maps.c, to, 64 * x, hc, tok, batch);
            }
            issued = j + 1;
            if (tail) {  // the last chunk: clears what is not this sequence's
                const bool ok = wait_for(to, 0, abort_flag);
                if (!ok) break;
                const int n = tokens(j);
                for (uint32_t x = 0; x < 4 + boxes_c; ++x) {
                    if (x < 4 && x >= 2 * boxes_a) continue;
                    for (int i = lane; i < (C - n) * 8; i += 32) st_shared_v4(at + x * BOX + (uint32_t)(n * 128 + i * 16), 0, 0, 0, 0);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(FULL0 + st));
            }
        }
        // never leave with copies in flight
        if (lane == 0) {
            for (int j = max(0, issued - kStages); j < issued; ++j) {
                if (j == r.drop_chunk) continue;
                if (j == nck - 1 && tail) mbar_drain(bar(TAIL), 0);
                else mbar_drain(bar(FULL0 + j % kStages), (j / kStages) & 1);
            }
        }
        __syncwarp();
    } else if (warp == W_MMA) {
        if (nck > 0 && elected()) {
            const uint32_t tm = tmem;
            auto wait = [&](int id, uint32_t parity) { return wait_alone(bar(id), parity, abort_flag); };
            auto full = [&](int j) { return wait(FULL0 + j % kStages, (j / kStages) & 1); };
            auto product_p = [&](uint32_t at) {
                products<ID_N64, false, 2, 2>(tm + TM_P, desc(at, 16), desc(at + B_OFF, 16));
                if (DA == 128) products<ID_N64, true, 2, 2>(tm + TM_P, desc(at + KB, 16), desc(at + KB + B_OFF, 16));
                mma_commit(bar(PDONE));
            };
            bool ok = full(0);
            tc_fence_after();
            if (ok && outs) product_p(stage(0));
#pragma unroll 1
            for (int j = 0; ok && j < nck; ++j) {
                const uint32_t ph = j & 1, at = stage(j);
                if (j < updates) {
                    if (!(ok = wait(WREADY0 + buffer(j), turn(j) & 1))) break;
                    tc_fence_after();
                    constexpr uint32_t ID_U = idesc_bf16(128, DA, 0, 1);
                    const uint32_t b = desc(at + B_OFF, KB), u = tm + (buffer(j) ? TM_U1 : TM_U), w = tm + (buffer(j) ? TM_W1 : TM_W);
                    products_ta<ID_U, false, 128>(u, w, b);
                    products_ta<ID_U, true, 128>(u, w + TM_WL, b);
                    if (THIRD) products<ID_U, true, 2, 128>(u, desc(sb + SM_W3 + ph * 2 * BOX, 16), b);
                    mma_commit(bar(UDONE0 + buffer(j)));
                }
                if (j + 1 < nck) {
                    if (!(ok = full(j + 1)) || (outs && !(ok = wait(PREAD, ph)))) break;
                    tc_fence_after();
                    if (outs) product_p(stage(j + 1));
                }
                if (outs) {
                    if (!(ok = wait(XREADY, ph))) break;
                    tc_fence_after();
                    products_ta<ID_N64, false, 2>(tm + TM_I, tm + TM_XH, desc(at, 16));
                    if (DA == 128) products_ta<ID_N64, true, 2>(tm + TM_I, tm + TM_XH + 32, desc(at + KB, 16));
                    products_ta<ID_N64, true, 2>(tm + TM_I, tm + TM_XL, desc(at, 16));
                    if (DA == 128) products_ta<ID_N64, true, 2>(tm + TM_I, tm + TM_XL + 32, desc(at + KB, 16));
                    mma_commit(bar(IDONE));
                    if (!(ok = wait(PREADY0 + ph, (j >> 1) & 1))) break;  // P~(j + 1) may be ready before it is looked for: a barrier for each buffer
                    tc_fence_after();
                    products<ID_N64_AMN, false, 128, 2>(tm + TM_O, desc(at + C_OFF, BOX), desc(sb + SM_P + ph * 2 * BOX, 16));
                    products<ID_N64_AMN, true, 128, 2>(tm + TM_O, desc(at + C_OFF, BOX), desc(sb + SM_P + ph * 2 * BOX + BOX, 16));
                    mma_commit(bar(ODONE));
                }
                mma_commit(bar(EMPTY0 + j % kStages));
            }
            mma_commit(bar(FINAL));  // every product completes before TMEM is released
            mbar_drain(bar(FINAL), 0);
        }
        __syncwarp();
    } else if (warp >= W_MAIN0 && warp < W_W0) {
        // column y of c; half hh of the state's row (HALF columns of a) and of out's tokens (32)
        const int quarter = warp & 3, y = 32 * quarter + lane, hh = (warp - W_MAIN0) >> 2;
        auto wait = [&](int id, int use) { return wait_for(bar(id), use & 1, abort_flag); };
        if (32 * quarter < r.dc) {
            constexpr int HALF = DA / 2;
            const uint32_t trow = tmem + ((uint32_t)(32 * quarter) << 16), t_x = trow + TM_XH + HALF / 2 * hh, t_u = trow + HALF * hh,
                           t_io = trow + TM_I + 32 * hh;
            unsigned char *staged = sm + SM_OUT + 2048 * (warp - W_MAIN0);
            uint64_t X[HALF / 2];
#pragma unroll
            for (int i = 0; i < HALF / 2; ++i) {
                const int x = HALF * hh + 2 * i;
                float v0 = 0.f, v1 = 0.f;
                if (init && live) {
                    v0 = init[init_t ? y * DA + x : x * r.dc + y];
                    v1 = init[init_t ? y * DA + x + 1 : (x + 1) * r.dc + y];
                }
                X[i] = pair_of(v0, v1);
            }
            LinearDecay whole(g * (float)C);  // of any chunk but the last
            // X takes U(i), if i is not -1 (and says that the buffer is free), and goes to TMEM as hi and lo
            auto advance = [&](int i, float f, bool store) {
                const bool update = i >= 0;
                const uint64_t f2 = pair_of(f, f);
                const uint32_t from = t_u + (buffer(i) ? TM_U1 : TM_U);
#pragma unroll
                for (int q = 0; q < HALF / 32; ++q) {
                    if (update) {
                        uint32_t u[32];
                        tmem_ld32(from + 32 * q, u);
                        if (q + 1 == HALF / 32 && i + kNext < updates) {
                            tc_fence_before();
                            mbar_arrive_warp(bar(WREADY0 + buffer(i + kNext)));
                        }
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            X[16 * q + i] = fma2(f2, X[16 * q + i], pair_of(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1])));
                    }
                    if (store) {
                        uint32_t xh[16], xl[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            uint64_t x = X[16 * q + i];
                            xh[i] = take_bf16(x), xl[i] = last_bf16(x);
                        }
                        tmem_st16x2(t_x + 16 * q, xh, t_x + (TM_XL - TM_XH) + 16 * q, xl);
                    }
                }
            };
            // 32 tokens of out of a chunk, staged as bf16 (or held as fp32), and their way to memory
            const int64_t row = (int64_t)r.Hv * r.dc;
            const int64_t low = first + (r.reverse ? (int64_t)span.tokens - (c0 + 1) * C : c0 * C);  // of chunk 0, were it whole
            const int64_t at0 = ((int64_t)batch * r.T + low + 32 * hh) * row + h * r.dc + 32 * quarter;
            const int64_t step = r.reverse ? -C * row : C * row;
            // Fragments: columns (tokens) 8 n + 2 (lane % 4) and the next one, weighted by into[], 16 lanes at a time.  Staged rows
            // of 64 bytes have their 16-byte pieces exchanged by pairs of rows, so that eight rows meet no bank twice
            const uint32_t stage_at = smem_u32(staged);
            auto piece = [&](int t, int c) { return (uint32_t)(t * 64 + ((c ^ (t >> 1 & 3)) << 4)); };
            auto write_out = [&](int j) {  // reads I and O, says so, and goes on
                const bool last = j + 1 == nck;
                const float *into = tab.into[last ? 1 : 0] + 32 * hh;
                // in the order of the scan the last chunk is the only short one; in reverse it is cut at its lower end
                int64_t at = at0 + j * step;
                int n = 32;
                if (last) {
                    n = tokens(j) - 32 * hh;
                    if (r.reverse) at += (C - tokens(j)) * row;
                }
                if constexpr (F32OUT) {  // a lane's column, token by token: whole lines
                    float *to = static_cast<float *>(r.out) + at + lane;
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        uint32_t in[16], o[16];
                        float w[16];
                        lds16f(into + 16 * q, w);
                        tmem_ld16x2(t_io + 16 * q, in, t_io + (TM_O - TM_I) + 16 * q, o);
                        if (q == 1) {
                            tc_fence_before();
                            mbar_arrive_warp(bar(XREADY));
                        }
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (16 * q + i < n) to[(16 * q + i) * row] = fmaf(w[i], __uint_as_float(in[i]), __uint_as_float(o[i]));
                    }
                    return;
                }
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t in[16], o[16];
                    const uint32_t t16 = t_io + ((uint32_t)(16 * half) << 16);
                    tmem_ld_fragments(t16, in, t16 + (TM_O - TM_I), o);
                    if (half == 1) {
                        tc_fence_before();
                        mbar_arrive_warp(bar(XREADY));
                    }
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        uint32_t b[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {  // tokens 8 (2 m + i / 2) .., lanes 16 half + 8 (i % 2) ..
                            const int e = 4 * (2 * m + i / 2) + 2 * (i & 1);
                            const uint64_t w = *reinterpret_cast<const uint64_t *>(into + 8 * (2 * m + i / 2) + 2 * (lane & 3));
                            b[i] = last_bf16(fma2(w, pair_of(__uint_as_float(in[e]), __uint_as_float(in[e + 1])),
                                                  pair_of(__uint_as_float(o[e]), __uint_as_float(o[e + 1]))));
                        }
                        const int i = lane >> 3, t = 8 * (2 * m + (i >> 1)) + (lane & 7);
                        store_transposed(stage_at + piece(t, 2 * half + (i & 1)), b[0], b[1], b[2], b[3]);
                    }
                }
                {  // 64-byte pieces of the rows by 16-byte stores
                    __syncwarp();
                    __nv_bfloat16 *ob = static_cast<__nv_bfloat16 *>(r.out) + at + (lane >> 2) * row + 8 * (lane & 3);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int t = 8 * i + (lane >> 2);
                        const uint4 x = *reinterpret_cast<const uint4 *>(staged + piece(t, lane & 3));
                        if (t < n) __stcs(reinterpret_cast<uint4 *>(ob + i * 8 * row), x);
                    }
                    __syncwarp();
                }
            };
            bool ok = true;
#pragma unroll 1
            for (int j = 0; j < nck; ++j) {
                const float f = j > 0 ? whole.next() : 0.f;
                if (j > 0) {  // I(j - 1) ends after U(j - 1)
                    if (!(ok = outs ? wait(IDONE, j - 1) : wait(UDONE0 + buffer(j - 1), turn(j - 1)))) break;
                    tc_fence_after();
                } else {
                    for (int i = 0; i < kNext && i < updates; ++i) mbar_arrive_warp(bar(WREADY0 + buffer(i)));
                }
                advance(j - 1, f, outs);
                if (!outs) continue;
                if (j > 0) {
                    if (!(ok = wait(ODONE, j - 1))) break;
                    tc_fence_after();
                    write_out(j - 1);
                } else {
                    tc_fence_before();
                    mbar_arrive_warp(bar(XREADY));
                }
            }
            if (ok && nck > 0 && updates == nck && (ok = wait(UDONE0 + buffer(nck - 1), turn(nck - 1)))) {
                tc_fence_after();
                advance(nck - 1, LinearDecay(g * (float)tokens(nck - 1)).f, false);
            }
            if (ok && nck > 0 && outs && wait(ODONE, nck - 1)) {
                tc_fence_after();
                write_out(nck - 1);
            }
            if (fin) {
                const bool bad = *abort_flag != 0;
#pragma unroll
                for (int i = 0; i < HALF / 2; ++i) {
                    const int x = HALF * hh + 2 * i;
                    float v0, v1;
                    halves(X[i], v0, v1);
                    if (bad) v0 = v1 = __int_as_float(0x7fffffff);
                    fin[fin_t ? y * DA + x : x * r.dc + y] = v0;
                    fin[fin_t ? y * DA + x + 1 : (x + 1) * r.dc + y] = v1;
                }
            }
        }
    } else if (warp >= W_W0) {
        // w c: columns 32 quarter .. of c, as matrix fragments: a lane has, of eight tokens and each of four times eight columns,
        // tokens 2 (lane % 4) and the next one of column lane / 4, which is how 16 lanes of TMEM take 128 bits each
        const int quarter = warp & 3, row = lane & 7;
        const uint32_t t_w = tmem + ((uint32_t)(32 * quarter) << 16);
        const uint32_t c_at = sb + C_OFF + (uint32_t)(quarter >> 1) * BOX + (uint32_t)(row * 128 + ((((quarter & 1) * 4 + (lane >> 3)) ^ row) << 4));
        const uint32_t w3_at = sb + SM_W3 + (uint32_t)((32 * quarter + lane) * 128);
#pragma unroll 1
        for (int j = 0; 32 * quarter < r.dc && j < updates; ++j) {
            if (!wait_for(bar(FULL0 + j % kStages), (j / kStages) & 1, abort_flag)) break;
            // the buffer's last reader is U(j - 1), or U(j - 2)
            auto readable = [&] { return j < kNext || wait_for(bar(UDONE0 + buffer(j)), turn(j - kNext) & 1, abort_flag); };
            if (!outs && !readable()) break;
            const uint32_t c = c_at + (uint32_t)(j % kStages) * STAGE, w3 = w3_at + (j & 1) * 2 * BOX;
            const uint64_t *up = reinterpret_cast<const uint64_t *>(tab.up[j + 1 < nck ? 0 : 1]) + (lane & 3);
            uint32_t hi[2][16], lo[2][16];  // of columns 0 .. 15 and 16 .. 31
#pragma unroll
            for (int m = 0; m < 8; ++m) {  // eight tokens
                uint32_t x[4], rest[4];
                load_transposed(c + m * 1024, x);
                const uint64_t w = up[4 * m];
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    uint64_t v = mul2(pair_of(__uint_as_float(x[n] << 16), __uint_as_float(x[n] & 0xFFFF0000u)), w);
                    uint32_t &h = hi[n >> 1][2 * m + (n & 1)], &l = lo[n >> 1][2 * m + (n & 1)];
                    h = take_bf16(v);
                    if (THIRD) l = take_bf16(v), rest[n] = last_bf16(v);
                    else l = last_bf16(v);
                }
                // into the buffer whose reader, U(j - 2), is done: it was waited for before the last W was stored
                if (THIRD) store_rows(w3 + ((uint32_t)(m ^ row) << 4), rest);
            }
            if (THIRD) fence_proxy_async_smem();
            if (outs && !readable()) break;
            tc_fence_after();
            const uint32_t to = t_w + (buffer(j) ? TM_W1 : TM_W);
            tmem_st_fragments(to, hi[0], to + TM_WL, lo[0]);
            tmem_st_fragments(to + (16u << 16), hi[1], to + (16u << 16) + TM_WL, lo[1]);
            tc_fence_before();
            mbar_arrive_warp(bar(WREADY0 + buffer(j)));
        }
    } else {
        // P~: row y of the chunk, 32 columns that its own row cuts off and, for one of the two warps, 32 before them
        const int y = 32 * warp + lane;
        const bool two = r.reverse ? warp == 0 : warp == 1;
        const int other = r.reverse ? 1 : 0;
        const uint32_t trow = tmem + ((uint32_t)(32 * warp) << 16) + TM_P;
        auto convert = [&](const uint32_t (&p)[32], int x, uint32_t to) {
            const float *w = tab.mask + 64 + y - 32 * x;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int k = 8 * q + 2 * i;
                    uint64_t v = mul2(pair_of(__uint_as_float(p[k]), __uint_as_float(p[k + 1])), pair_of(w[-k], w[-k - 1]));
                    hi[i] = take_bf16(v), lo[i] = last_bf16(v);
                }
                st_shared_v4(sw128_addr(to, y, 4 * x + q), hi[0], hi[1], hi[2], hi[3]);
                st_shared_v4(sw128_addr(to + BOX, y, 4 * x + q), lo[0], lo[1], lo[2], lo[3]);
            }
        };
#pragma unroll 1
        for (int j = 0; outs && j < nck; ++j) {
            if (!wait_for(bar(PDONE), j & 1, abort_flag)) break;
            tc_fence_after();
            uint32_t p0[32], p1[32];
            tmem_ld32(trow + 32 * warp, p0);
            if (two) tmem_ld32(trow + 32 * other, p1);
            tc_fence_before();
            mbar_arrive_warp(bar(PREAD));
            // products end in the order of their issue: with P(j), O(j - 2), the buffer's last reader, is done
            const uint32_t to = sb + SM_P + (j & 1) * 2 * BOX;
            convert(p0, warp, to);
            if (two) convert(p1, other, to);
            fence_proxy_async_smem();
            mbar_arrive_warp(bar(PREADY0 + (j & 1)));
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == W_MMA) tmem_dealloc(tmem, 512);
    if (outs && *abort_flag) {  // a wait ran out: all that this CTA answers for shows it
        const int from = token0(r.reverse ? nck - 1 : 0), n = min(span.tokens - c0 * C, nck * C);
        const float nan = __int_as_float(0x7fffffff);
#pragma unroll 1
        for (int64_t i = threadIdx.x; i < (int64_t)n * r.dc; i += kThreads) {
            const int64_t at = (((int64_t)batch * r.T + from + i / r.dc) * r.Hv + h) * r.dc + i % r.dc;
            if (F32OUT) static_cast<float *>(r.out)[at] = nan;
            else static_cast<__nv_bfloat16 *>(r.out)[at] = __float2bfloat16_rn(nan);
        }
    }
}

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        cudaDriverEntryPointQueryResult q;
        void *p = nullptr;
        const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q);
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(e == cudaSuccess && q == cudaDriverEntryPointSuccess ? p : nullptr);
    }();
    return fn;
}

// [B][T][heads][d] bf16 as {column, head, token, row of the batch}, boxes of 64 columns x 64 tokens
bool make_map(CUtensorMap *m, const void *x, const gdn_strides &s, int d, int heads, int T, int B) {
    const auto fn = encoder();
    if (!fn) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)T, (cuuint64_t)B};
    const cuuint64_t strides[3] = {(cuuint64_t)(heads > 1 ? 2 * s.head : 16), (cuuint64_t)(T > 1 ? 2 * s.token : 16),
                                   (cuuint64_t)(B > 1 ? 2 * s.batch : 16)};
    const cuuint32_t box[4] = {64, 1, C, 1}, steps[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(x), dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DA, int OUT, bool THIRD> cudaError_t launch(const Maps &maps, const LinearRun &r, cudaStream_t st) {
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(k_linear_tc<DA, OUT, THIRD>, (int)SMEM_BYTES, done);
    if (e != cudaSuccess) return e;
    return launch_behind(k_linear_tc<DA, OUT, THIRD>, dim3((unsigned)(r.slots * r.Hv)), kThreads, SMEM_BYTES, st, maps, r);
}

// A dimension that is stepped over needs a positive stride of a multiple of 16 bytes
bool mappable(const void *x, const gdn_strides &s, int heads, int64_t T, int64_t B) {
    auto steps = [](int64_t stride, int64_t n) { return n <= 1 || (stride > 0 && stride % 8 == 0 && stride < (int64_t)1 << 38); };
    return (reinterpret_cast<uintptr_t>(x) & 15) == 0 && steps(s.head, heads) && steps(s.token, T) && steps(s.batch, B);
}

template <int DA> cudaError_t launch(const Maps &maps, const LinearRun &r, int out, cudaStream_t st) {
    const bool third = r.fin != nullptr;  // segments' states are parts of it
    if (out == NO_OUT) return third ? launch<DA, NO_OUT, true>(maps, r, st) : launch<DA, NO_OUT, false>(maps, r, st);
    if (out == BF16_OUT) return third ? launch<DA, BF16_OUT, true>(maps, r, st) : launch<DA, BF16_OUT, false>(maps, r, st);
    return third ? launch<DA, F32_OUT, true>(maps, r, st) : launch<DA, F32_OUT, false>(maps, r, st);
}

}  // namespace

bool linear_tc_supported(const LinearRun &r, gdn_dtype io) {
    return io == GDN_BF16 && r.B > 0 && r.T > 0 && mappable(r.a, r.sa, r.Hv / r.ga, r.T, r.B) &&
           mappable(r.b, r.sb, r.Hv / r.gb, r.T, r.B) && mappable(r.c, r.sc, r.Hv / r.gc, r.T, r.B);
}

cudaError_t launch_linear_tc(const LinearRun &r, cudaStream_t st) {
    Maps maps;
    if (!make_map(&maps.a, r.a, r.sa, r.da, r.Hv / r.ga, r.T, r.B) || !make_map(&maps.b, r.b, r.sb, r.da, r.Hv / r.gb, r.T, r.B) ||
        !make_map(&maps.c, r.c, r.sc, r.dc, r.Hv / r.gc, r.T, r.B))
        return cudaErrorInvalidValue;
    const int out = r.mode == LIN_SEG || !r.out ? NO_OUT : r.out_f32 ? F32_OUT : BF16_OUT;
    return r.da == 128 ? launch<128>(maps, r, out, st) : launch<64>(maps, r, out, st);
}

}  // namespace gdn
