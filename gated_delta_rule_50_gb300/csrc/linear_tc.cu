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
// keep the state, warps 12 .. 15 make w c and write out.  Per chunk the tensor cores are asked for, in this order,
//     U(j), I(j), O(j), P(j + 1)
// so that the state's conversion runs under the products of the chunk before and the next one's w c under I, O and P.
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
constexpr int W_TMA = 2, W_MMA = 3, W_STATE0 = 4, W_AUX0 = 12;  // warps 0 and 1: P~
constexpr uint32_t kStateWarps = 8, kAuxWarps = 4;

// shared memory (bytes from a 1024-aligned base)
constexpr uint32_t STAGE = 49152, BOX = 8192;  // a stage: {a, b} of columns 0 .. 63, {a, b} of 64 .. 127, c of both
constexpr uint32_t B_OFF = BOX, KB = 2 * BOX, C_OFF = 4 * BOX;
constexpr uint32_t SM_P = kStages * STAGE;   // P~ {hi, lo} [64 r][64 i]
constexpr uint32_t SM_W3 = SM_P + 2 * BOX;   // third part of (w c)^T [128 y][64 i]
constexpr uint32_t SM_OUT = SM_W3 + 2 * BOX; // out on its way, 4 KB per warp
constexpr uint32_t SM_TAB = SM_OUT + kAuxWarps * 4096;
struct Tables {
    float mask[128];               // p_scale l^d, d = r - i in the order of the scan, at 64 + r - i of the tile's rows; 0 for d < 0
    float into[2][64], up[2][64];  // weights of I's and of c's rows; [1]: of the last chunk
};
constexpr uint32_t SM_BAR = SM_TAB + (uint32_t)sizeof(Tables);
enum {
    FULL0 = 0, EMPTY0 = FULL0 + kStages, TAIL = EMPTY0 + kStages, PDONE, PREADY, WREADY, UDONE, UFREE, XREADY, IDONE, ODONE,
    OFREE, FINAL, BARRIERS
};
constexpr uint32_t SM_MISC = SM_BAR + 8 * 32;
constexpr uint32_t SMEM_BYTES = SM_MISC + 64 + 1024;
static_assert(BARRIERS <= 32 && SMEM_BYTES <= 232448, "shared memory");

// TMEM columns
constexpr uint32_t TM_XH = 0, TM_XL = 64, TM_U = 128, TM_P = 256, TM_I = 320, TM_O = 384, TM_WH = 448, TM_WL = 480;

constexpr uint32_t ID_N64 = idesc_bf16(128, 64, 0, 0), ID_N64_AMN = idesc_bf16(128, 64, 1, 0);

struct Maps {
    CUtensorMap a, b, c;
};

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
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
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
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, uint32_t bar, int x, int y, int z, int w) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
        : "memory");
}

template <int DA, bool F32OUT>
__global__ void __launch_bounds__(kThreads, 1) k_linear_tc(const __grid_constant__ Maps maps, const __grid_constant__ LinearRun r) {
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *sm = smem_align1024(smem_raw);
    const uint32_t sb = smem_u32(sm);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t *misc = reinterpret_cast<uint32_t *>(sm + SM_MISC);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(misc + 1);
    Tables &tab = *reinterpret_cast<Tables *>(sm + SM_TAB);
    auto bar = [&](int i) { return sb + SM_BAR + 8u * (uint32_t)i; };

    if (threadIdx.x == 0) {
        const uint32_t w = kStateWarps, x = kAuxWarps;
        const uint32_t counts[BARRIERS] = {1, 1, 1, 1, 1, 1, 1, 1, 2, x, 1, w, w, 1, 1, x, 1};
        for (int i = 0; i < BARRIERS; ++i) mbar_init(bar(i), counts[i]);
        misc[1] = 0;
        fence_mbar_init();
    }
    if (warp == W_MMA) tmem_alloc(sb + SM_MISC, 512);
    if (warp == W_TMA && lane == 0) prefetch_tmap(&maps.a), prefetch_tmap(&maps.b), prefetch_tmap(&maps.c);
    wait_for_previous();

    const int h = blockIdx.y, seq = blockIdx.x / r.n_seg, part = blockIdx.x % r.n_seg;
    const LinearSpan span = linear_span(r, seq);
    const int c0 = min(span.chunks, part * span.per_seg), c1 = min(span.chunks, c0 + span.per_seg);
    const int64_t unit = (int64_t)seq * r.Hv + h, words = (int64_t)DA * r.dc;
    const float *init = r.init ? r.init + unit * words : nullptr;
    float *fin = r.fin ? r.fin + unit * words : nullptr;
    bool init_t = r.transposed, fin_t = r.transposed, outs = r.out != nullptr, live = true;
    if (r.mode == LIN_SEG) {  // the last segment feeds no other
        live = c1 < span.chunks && c0 < c1, outs = false;
        init = nullptr, fin = r.seg + (unit * r.n_seg + part) * words, fin_t = false;
    } else {
        if (part > 0) {
            live = c0 < c1;
            init = r.seg + (unit * r.n_seg + part) * words, init_t = false;
        }
        if (c1 < span.chunks || !live) fin = nullptr;
    }
    const int nck = live ? c1 - c0 : 0, updates = fin ? nck : nck - 1;  // chunks whose part in the state is wanted
    const bool third = r.fin != nullptr && fin != nullptr;
    const int first = r.cu ? (int)span.first : 0, batch = r.cu ? 0 : seq;
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
        for (int i = t; i < 2 * 32 * 4; i += kThreads) {  // half, row, 16 bytes
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
        for (int j = 0; j < nck; ++j) {
            const int st = j % kStages;
            if (j >= kStages && !mbar_wait_warp(bar(EMPTY0 + st), (j / kStages - 1) & 1, abort_flag)) break;
            tail = tokens(j) < C;
            const uint32_t to = tail ? bar(TAIL) : bar(FULL0 + st), at = stage(j);
            if (lane == 0) {
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
                const bool ok = mbar_wait_warp(to, 0, abort_flag);
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
                if (j == nck - 1 && tail) mbar_drain(bar(TAIL), 0);
                else mbar_drain(bar(FULL0 + j % kStages), (j / kStages) & 1);
            }
        }
        __syncwarp();
    } else if (warp == W_MMA) {
        if (lane == 0 && nck > 0) {
            auto wait = [&](int id, uint32_t parity) { return mbar_wait(bar(id), parity, abort_flag); };
            auto full = [&](int j) { return wait(FULL0 + j % kStages, (j / kStages) & 1); };
            auto product_p = [&](int j) {
                for (int x = 0; x < DA / 64; ++x)
                    mma_chain<4, 2, 2>(tmem + TM_P, sdesc_sw128(stage(j) + x * KB, 16, 1024),
                                       sdesc_sw128(stage(j) + x * KB + B_OFF, 16, 1024), ID_N64, x);
                mma_commit(bar(PDONE));
            };
            bool ok = full(0);
            tc_fence_after();
            if (ok && outs) product_p(0);
            for (int j = 0; ok && j < nck; ++j) {
                const uint32_t ph = j & 1, at = stage(j);
                if (j < updates) {
                    if (!(ok = wait(WREADY, ph)) || (j > 0 && !(ok = wait(UFREE, (j - 1) & 1)))) break;
                    tc_fence_after();
                    constexpr uint32_t ID_U = idesc_bf16(128, DA, 0, 1);
                    const uint64_t b = sdesc_sw128(at + B_OFF, KB, 1024);
                    for (int x = 0; x < 2; ++x) mma_chain_ta<4, 128>(tmem + TM_U, tmem + (x ? TM_WL : TM_WH), b, ID_U, x);
                    if (third) mma_chain<4, 2, 128>(tmem + TM_U, sdesc_sw128(sb + SM_W3, 16, 1024), b, ID_U, 1);
                    mma_commit(bar(UDONE));
                }
                if (outs) {
                    if (!(ok = wait(XREADY, ph)) || (j > 0 && !(ok = wait(OFREE, (j - 1) & 1)))) break;
                    tc_fence_after();
                    for (int x = 0; x < 2; ++x)
                        for (int y = 0; y < DA / 64; ++y)
                            mma_chain_ta<4, 2>(tmem + TM_I, tmem + (x ? TM_XL : TM_XH) + 32 * y, sdesc_sw128(at + y * KB, 16, 1024),
                                               ID_N64, x | y);
                    mma_commit(bar(IDONE));
                    if (!(ok = wait(PREADY, ph))) break;
                    tc_fence_after();
                    for (int x = 0; x < 2; ++x)
                        mma_chain<4, 128, 2>(tmem + TM_O, sdesc_sw128(at + C_OFF, BOX, 1024),
                                             sdesc_sw128(sb + SM_P + x * BOX, 16, 1024), ID_N64_AMN, x);
                    mma_commit(bar(ODONE));
                }
                mma_commit(bar(EMPTY0 + j % kStages));
                if (j + 1 < nck) {
                    if (!(ok = full(j + 1))) break;
                    tc_fence_after();
                    if (outs) product_p(j + 1);
                }
            }
            mma_commit(bar(FINAL));  // every product completes before TMEM is released
            mbar_drain(bar(FINAL), 0);
        }
        __syncwarp();
    } else if (warp >= W_STATE0 && warp < W_AUX0) {
        // the state: column y of c, half hh of its row
        const int quarter = warp & 3, y = 32 * quarter + lane, hh = (warp - W_STATE0) >> 2;
        const bool mine = 32 * quarter < r.dc;
        constexpr int HALF = DA / 2;
        const uint32_t trow = tmem + ((uint32_t)(32 * quarter) << 16);
        uint64_t X[HALF / 2];
#pragma unroll
        for (int i = 0; i < HALF / 2; ++i) {
            const int x = HALF * hh + 2 * i;
            float v0 = 0.f, v1 = 0.f;
            if (init && live && mine) {
                v0 = init[init_t ? y * DA + x : x * r.dc + y];
                v1 = init[init_t ? y * DA + x + 1 : (x + 1) * r.dc + y];
            }
            X[i] = pair_of(v0, v1);
        }
        bool ok = true;
        for (int j = 0; j < nck && ok; ++j) {
            if (outs) {
                if (j > 0 && !(ok = mbar_wait_warp(bar(IDONE), (j - 1) & 1, abort_flag))) break;
                tc_fence_after();
                if (mine) {
#pragma unroll
                    for (int q = 0; q < HALF / 16; ++q) {
                        uint32_t hi[8], lo[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            uint64_t x = X[8 * q + i];
                            hi[i] = take_bf16(x), lo[i] = last_bf16(x);
                        }
                        const uint32_t to = HALF / 2 * hh + 8 * q;
                        tmem_st8x2(trow + TM_XH + to, hi, trow + TM_XL + to, lo);
                    }
                }
                tc_fence_before();
                mbar_arrive_warp(bar(XREADY));
            }
            if (j >= updates) break;
            const float l1 = expm1f(g * (float)tokens(j));  // X l^n as X + l1 X: nothing is lost where l is all but 1
            const uint64_t l2 = pair_of(l1, l1);
            if (!(ok = mbar_wait_warp(bar(UDONE), j & 1, abort_flag))) break;
            tc_fence_after();
            if (mine) {
#pragma unroll
                for (int q = 0; q < HALF / 16; ++q) {
                    uint32_t u[16];
                    tmem_ld16(trow + TM_U + HALF * hh + 16 * q, u);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        uint64_t &x = X[8 * q + i];
                        x = add2(x, fma2(l2, x, pair_of(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1]))));
                    }
                }
            }
            tc_fence_before();
            mbar_arrive_warp(bar(UFREE));
        }
        if (fin && mine) {
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
    } else if (warp >= W_AUX0) {
        // w c, and out: column y of c
        const int quarter = warp & 3, y = 32 * quarter + lane;
        const bool mine = 32 * quarter < r.dc;
        const uint32_t trow = tmem + ((uint32_t)(32 * quarter) << 16);
        unsigned char *staged = sm + SM_OUT + 4096 * (warp - W_AUX0);
        auto write_out = [&](int j) {
            if (!mbar_wait_warp(bar(ODONE), j & 1, abort_flag)) return false;
            tc_fence_after();
            const int n = tokens(j);
            const float *w = tab.into[n < C ? 1 : 0];
            const int64_t at = (((int64_t)batch * r.T + token0(j)) * r.Hv + h) * r.dc + 32 * quarter;  // of out
#pragma unroll
            for (int q = 0; q < 4; ++q) {  // 16 tokens
                uint32_t in[16], o[16];
                float ww[16];
                lds16f(w + 16 * q, ww);
                if (mine) tmem_ld16x2(trow + TM_I + 16 * q, in, trow + TM_O + 16 * q, o);
                if (q == 3) {
                    tc_fence_before();
                    mbar_arrive_warp(bar(OFREE));
                }
                if (!mine) continue;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float v = fmaf(ww[i], __uint_as_float(in[i]), __uint_as_float(o[i]));
                    if (F32OUT) {
                        if (16 * q + i < n) static_cast<float *>(r.out)[at + (int64_t)(16 * q + i) * r.Hv * r.dc + lane] = v;
                    } else {
                        reinterpret_cast<__nv_bfloat16 *>(staged)[(16 * q + i) * 32 + lane] = __float2bfloat16_rn(v);
                    }
                }
            }
            if (!F32OUT && mine) {
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int row = 8 * i + (lane >> 2);
                    const uint4 v = *reinterpret_cast<const uint4 *>(staged + row * 64 + (lane & 3) * 16);
                    if (row < n)
                        __stcs(reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(r.out) + at + (int64_t)row * r.Hv * r.dc + 8 * (lane & 3)), v);
                }
                __syncwarp();
            }
            return true;
        };
        bool ok = true;
        for (int j = 0; j < nck && ok; ++j) {
            if (j < updates) {
                if (!(ok = mbar_wait_warp(bar(FULL0 + j % kStages), (j / kStages) & 1, abort_flag))) break;
                if (j > 0 && !(ok = mbar_wait_warp(bar(UDONE), (j - 1) & 1, abort_flag))) break;
                tc_fence_after();
                if (mine) {
                    const unsigned char *c = sm + (j % kStages) * STAGE + C_OFF + (y >> 6) * BOX + (y & 7) * 2;
                    const float *up = tab.up[tokens(j) < C ? 1 : 0];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {  // 16 tokens
                        float w[16];
                        lds16f(up + 16 * q, w);
                        uint32_t hi[8], lo[8], rest[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            float v[2];
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const int t = 16 * q + 2 * i + k;
                                v[k] = __bfloat162float(*reinterpret_cast<const __nv_bfloat16 *>(
                                    c + t * 128 + ((((y & 63) >> 3) ^ (t & 7)) << 4)));
                            }
                            uint64_t x = mul2(pair_of(v[0], v[1]), pair_of(w[2 * i], w[2 * i + 1]));
                            hi[i] = take_bf16(x), lo[i] = take_bf16(x), rest[i] = last_bf16(x);
                        }
                        tmem_st8x2(trow + TM_WH + 8 * q, hi, trow + TM_WL + 8 * q, lo);
                        if (third) {
#pragma unroll
                            for (int k = 0; k < 2; ++k)
                                st_shared_v4(sw128_addr(sb + SM_W3, y, 2 * q + k), rest[4 * k], rest[4 * k + 1], rest[4 * k + 2],
                                             rest[4 * k + 3]);
                        }
                    }
                    if (third) fence_proxy_async_smem();
                }
                tc_fence_before();
                mbar_arrive_warp(bar(WREADY));
            }
            if (outs && j > 0) ok = write_out(j - 1);
        }
        if (ok && outs && nck > 0) write_out(nck - 1);
    } else {
        // P~: row y of the chunk.  The products are issued in order, so that with P(j) the one that read P~(j - 1) is done
        const int y = 32 * warp + lane;
        const uint32_t trow = tmem + ((uint32_t)(32 * warp) << 16) + TM_P;
        for (int j = 0; outs && j < nck; ++j) {
            if (!mbar_wait_warp(bar(PDONE), j & 1, abort_flag)) break;
            tc_fence_after();
#pragma unroll
            for (int x = 0; x < 2; ++x) {  // columns 32 x ..
                if (r.reverse ? x < warp : x > warp) continue;
                uint32_t p[32];
                tmem_ld32(trow + 32 * x, p);
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
                    st_shared_v4(sw128_addr(sb + SM_P, y, 4 * x + q), hi[0], hi[1], hi[2], hi[3]);
                    st_shared_v4(sw128_addr(sb + SM_P + BOX, y, 4 * x + q), lo[0], lo[1], lo[2], lo[3]);
                }
            }
            fence_proxy_async_smem();
            tc_fence_before();
            mbar_arrive_warp(bar(PREADY));
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == W_MMA) tmem_dealloc(tmem, 512);
    if (*abort_flag && outs) {  // a wait ran out: all that this CTA answers for shows it
        const int from = token0(r.reverse ? nck - 1 : 0), n = min(span.tokens - c0 * C, nck * C);
        const float nan = __int_as_float(0x7fffffff);
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

template <int DA, bool F32OUT> cudaError_t launch(const Maps &maps, const LinearRun &r, cudaStream_t st) {
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(k_linear_tc<DA, F32OUT>, (int)SMEM_BYTES, done);
    if (e != cudaSuccess) return e;
    return launch_behind(k_linear_tc<DA, F32OUT>, dim3((unsigned)(r.n_seqs * r.n_seg), (unsigned)r.Hv), kThreads, SMEM_BYTES, st, maps, r);
}

// A dimension that is stepped over needs a positive stride of a multiple of 16 bytes
bool mappable(const void *x, const gdn_strides &s, int heads, int64_t T, int64_t B) {
    auto steps = [](int64_t stride, int64_t n) { return n <= 1 || (stride > 0 && stride % 8 == 0 && stride < (int64_t)1 << 38); };
    return (reinterpret_cast<uintptr_t>(x) & 15) == 0 && steps(s.head, heads) && steps(s.token, T) && steps(s.batch, B);
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
    if (r.da == 128) return r.out_f32 ? launch<128, true>(maps, r, st) : launch<128, false>(maps, r, st);
    return r.out_f32 ? launch<64, true>(maps, r, st) : launch<64, false>(maps, r, st);
}

}  // namespace gdn
