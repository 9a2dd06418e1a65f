// tree_tc.cu -- the drafted-tree operator on the tensor cores (bf16 io).  The mathematics is in tree.cu; here
// one CTA of 128 threads computes a (row, value head) with thread v = TMEM lane v = value column v:
//
//   G  = [K; Q] K^T                (operands in shared memory)       lane r: row r of K K^T, then of Q K^T
//   D1 = S^T [K; Q]^T              (S^T from TMEM, hi + lo)          lane v: S^T k_t, then S^T q_t, of column v
//   d  = (I + L)^-1 R              forward substitution, a column per thread, all of it in registers
//   D2 = d^T P^T                   (d^T from TMEM, hi + lo)          lane v: sum_i P_ti d_i of column v
//   o_t = scale (Gam_t D1_q + D2)
//
// q and k are bf16 as given; S, P and d enter as hi + lo bf16 pairs (16 bits; one bf16 rounding of them would
// cost as much as the rounding of o).  L stays in fp32: the substitution multiplies it by unrounded d.
// S arrives by one bulk copy (a head's state is contiguous) while q, k and G are made, and goes to TMEM; its
// place in shared memory then holds L and P.  Two CTAs fit on an SM (100 KB, 256 TMEM columns), so that one's
// copies run under the other's arithmetic.
#include <cuda_bf16.h>

#include "common.cuh"
#include "decode.h"
#include "tc.cuh"

namespace gdn {
namespace {

using namespace tc;

constexpr int NT = 128;
constexpr uint32_t kBlock = 16384;  // 128 rows of 64 bf16: one K block of [K; Q]
constexpr uint32_t kCols = 256;     // TMEM: S^T hi, lo (K columns; later d^T hi, lo and D2) | D1 from column 128
constexpr uint32_t kD1 = 128, kD2 = 64, kDlo = 32;

template <int K, int TP> struct Map {
    static constexpr uint32_t LS = TP + 4;  // L begins at 0, its row stride: 16-byte rows, eight neighbours on different banks
    static constexpr uint32_t PHI = (2 * TP * LS * 4 + 1023) / 1024 * 1024, PLO = PHI + TP * 128;
    static constexpr uint32_t scratch = PLO + TP * 128, state = K * 128 * 4;
    static constexpr uint32_t KQ = ((scratch > state ? scratch : state) + 1023) / 1024 * 1024;
    static constexpr uint32_t VEC = KQ + K / 64 * kBlock;  // a, beta, Gam, parent, what the node is: TP each
    static constexpr uint32_t BAR = VEC + 5 * TP * 4;
    static constexpr uint32_t bytes = BAR + 32 + 1024;
};

__device__ __forceinline__ uint64_t kdesc(uint32_t a) { return sdesc_sw128(a, 16, 1024); }

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

template <int K, int TP>
__global__ void __launch_bounds__(NT, 2) k_tree_tc(const DecodeArgs a, bool vec) {
    using M = Map<K, TP>;
    constexpr int LS = M::LS;
    constexpr uint32_t ID_G = idesc_bf16(128, TP, 0, 0), ID_S = idesc_bf16(128, 2 * TP, 0, 0);
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *sm = smem_align1024(smem_raw);
    const uint32_t sb = smem_u32(sm);
    const int t = threadIdx.x, warp = t >> 5, T = a.T, V = a.V;
    const int n = blockIdx.x / a.Hv, h = blockIdx.x - n * a.Hv, hq = h / a.G;
    const float nan = __int_as_float(0x7fffffff);
    const bool mine = t < V;  // this thread has a value column (the same for a whole warp)
    __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(a.o) + ((int64_t)n * T * a.Hv + h) * V + t;
    const int64_t o_tok = (int64_t)a.Hv * V;

    const int64_t slot = a.state_indices ? a.state_indices[n] : n;
    if (slot < 0 || slot >= a.n_slots) {
        if (mine)
            for (int i = 0; i < T; ++i) o[i * o_tok] = __float2bfloat16_rn(slot < 0 ? 0.f : nan);
        return;
    }
    float *s_a = reinterpret_cast<float *>(sm + M::VEC), *s_b = s_a + TP, *s_gam = s_b + TP;
    int *s_par = reinterpret_cast<int *>(s_gam + TP), *s_kind = s_par + TP;  // kind: 0 a node, 1 absent, 2 no such parent
    uint32_t *misc = reinterpret_cast<uint32_t *>(sm + M::BAR + 16);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(misc + 1);
    const uint32_t bar_s = sb + M::BAR, bar_m = bar_s + 8;
    if (t == 0) {
        mbar_init(bar_s, 1);
        mbar_init(bar_m, 1);
        misc[1] = 0;
        fence_mbar_init();
        const uint32_t bytes = (uint32_t)(K * V * 4);
        mbar_arrive_expect_tx(bar_s, bytes);
        bulk_load(sb, a.state + slot * a.slot_stride + (int64_t)h * K * V, bytes, bar_s);
    }
    if (warp == 0) tmem_alloc(sb + M::BAR + 16, kCols);

    const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(a.q) + n * a.sq.batch + hq * a.sq.head;
    const __nv_bfloat16 *k = static_cast<const __nv_bfloat16 *>(a.k) + n * a.sk.batch + hq * a.sk.head;
    const __nv_bfloat16 *v = static_cast<const __nv_bfloat16 *>(a.v) + n * a.sv.batch + h * a.sv.head + t;
    for (int e = t; e < 2 * T * (K / 8); e += NT) {  // 16-byte pieces of the rows of k, then of q
        const int row = e / (K / 8), x = e % (K / 8);
        const bool is_q = row >= T;
        const int tok = is_q ? row - T : row;
        const __nv_bfloat16 *src = is_q ? q + tok * a.sq.token : k + tok * a.sk.token;
        const uint32_t dst = sw128_addr(sb + M::KQ + (x >> 3) * kBlock, is_q ? TP + tok : tok, x & 7);
        if (vec) {
            cp_async16(dst, src + 8 * x);
        } else {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = (uint32_t)__bfloat16_as_ushort(src[8 * x + 2 * i]) | (uint32_t)__bfloat16_as_ushort(src[8 * x + 2 * i + 1]) << 16;
            st_shared_v4(dst, w[0], w[1], w[2], w[3]);
        }
    }
    if (t < TP) {
        const bool in = t < T;
        s_a[t] = in ? expf(a.g[n * a.sg.batch + h * a.sg.head + t * a.sg.token]) : 0.f;
        s_b[t] = in ? a.beta[n * a.sb.batch + h * a.sb.head + t * a.sb.token] : 0.f;
        s_par[t] = in ? a.parents[(int64_t)n * T + t] : -2;
    }
    __nv_bfloat16 vr[TP];
#pragma unroll
    for (int i = 0; i < TP; ++i) vr[i] = mine && i < T ? v[i * a.sv.token] : __float2bfloat16_rn(0.f);
    asm volatile("cp.async.wait_all;" ::: "memory");
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = misc[0], lanes = (uint32_t)(32 * warp) << 16;
    bool ok = true;

    if (t == 0) {
        for (int kb = 0; kb < K / 64; ++kb)
            mma_chain<4, 2, 2>(tmem + kD1, kdesc(sb + M::KQ + kb * kBlock), kdesc(sb + M::KQ + kb * kBlock), ID_G, kb);
        mma_commit(bar_m);
    }
    ok = mbar_wait_warp(bar_m, 0, abort_flag) && ok;
    tc_fence_after();
    uint32_t gram[TP];  // row t of K K^T, or row t - TP of Q K^T
#pragma unroll
    for (int c = 0; c < TP / 16; ++c) {
        uint32_t r[16];
        tmem_ld16(tmem + lanes + kD1 + 16 * c, r);
#pragma unroll
        for (int i = 0; i < 16; ++i) gram[16 * c + i] = r[i];
    }
    ok = mbar_wait_warp(bar_s, 0, abort_flag) && ok;
    if (mine) {
        const float *s = reinterpret_cast<const float *>(sm) + t;
#pragma unroll
        for (int c = 0; c < K / 32; ++c) {
            float x[32];
            uint32_t hi[16], lo[16];
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = s[(32 * c + i) * V];
            split_pack16(x, hi, lo);
            tmem_st16x2(tmem + lanes + 16 * c, hi, tmem + lanes + K / 2 + 16 * c, lo);
        }
    }
    tc_fence_before();
    ok = __syncthreads_and(ok) != 0;
    if (ok) {
        tc_fence_after();
        if (t == 0) {
            for (int part = 0; part < 2; ++part)
                for (int kb = 0; kb < K / 64; ++kb)
                    mma_chain_ta<4, 2>(tmem + kD1, tmem + part * (K / 2) + 32 * kb, kdesc(sb + M::KQ + kb * kBlock), ID_S,
                                       part + kb);
            mma_commit(bar_m);
        }
        // Meanwhile L and P, over the state's place: thread t walks from node t (or t - TP) up to the state and
        // leaves the products of e^g on the way in its row.
        float *row = reinterpret_cast<float *>(sm) + t * LS;
        const int node = t < TP ? t : t - TP;
        if (t < 2 * TP) {
#pragma unroll
            for (int i = 0; i < TP / 4; ++i) reinterpret_cast<float4 *>(row)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            float prod = 1.f;
            int p = node, kind = 0;
            while (p >= 0) {
                row[p] = prod;
                const int up = s_par[p];
                if (up >= p || up < -1) {
                    kind = up < -1 ? 1 : 2;
                    break;
                }
                prod *= s_a[p];
                p = up;
            }
            if (t < TP) s_gam[t] = prod, s_kind[t] = kind;
            const float b = t < TP ? s_b[node] : 1.f;
#pragma unroll
            for (int c = 0; c < TP / 8; ++c) {
                float x[8];
                lds8f(row + 8 * c, x);
#pragma unroll
                for (int i = 0; i < 8; ++i) {  // what is not above the node may hold anything: selected, not multiplied
                    const float w = __uint_as_float(gram[8 * c + i]);
                    const bool above = x[i] != 0.f && kind == 0 && (t >= TP || 8 * c + i < node);
                    x[i] = above ? b * x[i] * w : 0.f;
                }
                if (t < TP) {
                    reinterpret_cast<float4 *>(row)[2 * c] = make_float4(x[0], x[1], x[2], x[3]);
                    reinterpret_cast<float4 *>(row)[2 * c + 1] = make_float4(x[4], x[5], x[6], x[7]);
                } else {
                    st_split_chunk(sb + M::PHI, sb + M::PLO, node, c, x);
                }
            }
        }
        fence_proxy_async_smem();
        ok = mbar_wait_warp(bar_m, 1, abort_flag);
        tc_fence_after();
        ok = __syncthreads_and(ok) != 0;
    }
    float x[TP];
    if (ok) {
        if (mine) {
#pragma unroll
            for (int c = 0; c < TP / 16; ++c) {
                uint32_t r[16];
                tmem_ld16(tmem + lanes + kD1 + 16 * c, r);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int j = 16 * c + i;
                    x[j] = s_kind[j] ? 0.f : s_b[j] * (__bfloat162float(vr[j]) - s_gam[j] * __uint_as_float(r[i]));
                }
            }
            // four rows at a time: what the rows before them give, then the triangle between the four
            const float *L = reinterpret_cast<const float *>(sm);
#pragma unroll
            for (int j = 0; j < TP; j += 4) {
                float acc[4] = {x[j], x[j + 1], x[j + 2], x[j + 3]};
#pragma unroll
                for (int i = 0; i < j; i += 4)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float4 l = *reinterpret_cast<const float4 *>(L + (j + r) * LS + i);
                        acc[r] = fmaf(-l.x, x[i], acc[r]);
                        acc[r] = fmaf(-l.y, x[i + 1], acc[r]);
                        acc[r] = fmaf(-l.z, x[i + 2], acc[r]);
                        acc[r] = fmaf(-l.w, x[i + 3], acc[r]);
                    }
                const float4 l1 = *reinterpret_cast<const float4 *>(L + (j + 1) * LS + j);
                const float4 l2 = *reinterpret_cast<const float4 *>(L + (j + 2) * LS + j);
                const float4 l3 = *reinterpret_cast<const float4 *>(L + (j + 3) * LS + j);
                acc[1] = fmaf(-l1.x, acc[0], acc[1]);
                acc[2] = fmaf(-l2.y, acc[1], fmaf(-l2.x, acc[0], acc[2]));
                acc[3] = fmaf(-l3.z, acc[2], fmaf(-l3.y, acc[1], fmaf(-l3.x, acc[0], acc[3])));
#pragma unroll
                for (int r = 0; r < 4; ++r) x[j + r] = acc[r];
            }
#pragma unroll
            for (int c = 0; c < TP / 16; ++c) {
                uint32_t hi[8], lo[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) split_pair(x[16 * c + 2 * i], x[16 * c + 2 * i + 1], hi[i], lo[i]);
                tmem_st8x2(tmem + lanes + 8 * c, hi, tmem + lanes + kDlo + 8 * c, lo);
            }
        }
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        if (t == 0) {
            mma_chain_ta<TP / 16, 2>(tmem + kD2, tmem, kdesc(sb + M::PHI), ID_G, 0);
            mma_chain_ta<TP / 16, 2>(tmem + kD2, tmem + kDlo, kdesc(sb + M::PHI), ID_G, 1);
            mma_chain_ta<TP / 16, 2>(tmem + kD2, tmem, kdesc(sb + M::PLO), ID_G, 1);
            mma_commit(bar_m);
        }
        ok = mbar_wait_warp(bar_m, 0, abort_flag);
        tc_fence_after();
        if (mine && ok) {
#pragma unroll
            for (int c = 0; c < TP / 16; ++c) {
                uint32_t sq[16], d2[16];
                tmem_ld16x2(tmem + lanes + kD1 + TP + 16 * c, sq, tmem + lanes + kD2 + 16 * c, d2);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int j = 16 * c + i;
                    const float y = a.scale * fmaf(s_gam[j], __uint_as_float(sq[i]), __uint_as_float(d2[i]));
                    if (j < T) o[j * o_tok] = __float2bfloat16_rn(s_kind[j] == 0 ? y : s_kind[j] == 1 ? 0.f : nan);
                }
            }
        }
    }
    // A wait that ran out (its limit is a second): nothing in flight is left behind, and the row shows it.
    ok = __syncthreads_and(ok) != 0;
    if (!ok) {
        if (t == 0) mbar_drain(bar_s, 0);
        if (mine)
            for (int i = 0; i < T; ++i) o[i * o_tok] = __float2bfloat16_rn(nan);
        __syncthreads();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, kCols);
    }
}

template <int K, int TP> cudaError_t launch(const DecodeArgs &a, bool vec, cudaStream_t st) {
    constexpr int bytes = (int)Map<K, TP>::bytes;
    static_assert(2 * (bytes + 1024) <= 233472, "two CTAs per SM");
    const cudaError_t e = cudaFuncSetAttribute(k_tree_tc<K, TP>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    k_tree_tc<K, TP><<<(unsigned)(a.n_seqs * a.Hv), NT, bytes, st>>>(a, vec);
    return cudaGetLastError();
}

template <int K> cudaError_t launch_width(const DecodeArgs &a, bool vec, cudaStream_t st) {
    if (a.T <= 16) return launch<K, 16>(a, vec, st);
    if (a.T <= 32) return launch<K, 32>(a, vec, st);
    if (a.T <= 48) return launch<K, 48>(a, vec, st);
    return launch<K, 64>(a, vec, st);
}

}  // namespace

cudaError_t launch_tree_tc(const DecodeArgs &a, int K, cudaStream_t st) {
    // 16-byte copies of the rows of q and k where every row begins on such a boundary
    const int64_t s = a.sq.batch | a.sq.token | a.sq.head | a.sk.batch | a.sk.token | a.sk.head;
    const bool vec = !(s & 7) && !((reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.k)) & 15);
    return K == 128 ? launch_width<128>(a, vec, st) : launch_width<64>(a, vec, st);
}

}  // namespace gdn
