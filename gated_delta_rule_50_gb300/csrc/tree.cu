// tree.cu -- a tree of drafted tokens answered from a state, which is only read.
//
// With S the state, anc(t) the nodes on the path down to t (t included) and, for i in anc(t), D_ti the product
// of e^g over the path's nodes after i, Gam_t the product over the whole path:
//     d_t = beta_t (v_t - Gam_t S^T k_t) - sum_{i in anc(t), i != t} L_ti d_i,   L_ti = beta_t D_ti (k_t . k_i)
//     o_t = scale (Gam_t S^T q_t + sum_{i in anc(t)} P_ti d_i),                  P_ti = D_ti (q_t . k_i)
// which is the recurrence along every path at once: no node needs a state of its own.  D is built by products
// down the tree (D_ti = e^{g_t} D_parent(t),i), so a gate of -inf stays 0 and nothing is a difference of sums.
// The fast sums run over all nodes, with zeros in L and P where i is not above t, and 0 times a NaN is one.  Such a sum
// cannot be finite again, so it is enough to look at the results: where one is not, the sums are taken again over the
// paths alone (from node to parent), and a NaN or an infinity reaches what its path reaches and nothing else.
// This file holds the CUDA-core kernel, for fp32 io; tree_tc.cu has the tensor-core kernel for bf16.
//
// One CTA computes a (row, value head), two threads per value column.  Both have the state in registers as in
// decode.cu and take S^T k_t and S^T q_t of every other node; then one makes the column's corrections d, and both
// the outputs, with L and P read as broadcast vectors.  64 rows of 32 heads, 64 nodes, 128 x 128, take 830 us; 16 rows of
// 32 heads 35 us with 7 nodes, 98 with 32.  Neither memory (5 %) nor the multiply-adds (2 T K V for the state, T^2 (K + V)
// for the rest: 7.7 T a second, a fifth of what the SMs could) bound it, but the chain: an SM holds one such CTA, whose
// loads, products, substitution and outputs follow each other (1.5 instructions a cycle, barriers first among the stalls).
// One thread per column and rows staged element by element took 1265 us, but 98 instead of 114 for 16 rows of 32 heads
// with 33 nodes.
#include "common.cuh"
#include "decode.h"

namespace gdn {
namespace {

constexpr int kTile = 32;  // state columns per warp

__device__ __forceinline__ float reduce_columns(const float (&x)[4], int r) {
    const bool r0 = r & 1, r1 = r & 2;
    float a = r0 ? x[1] : x[0], b = r0 ? x[3] : x[2];
    a += __shfl_xor_sync(~0u, r0 ? x[0] : x[1], 8);
    b += __shfl_xor_sync(~0u, r0 ? x[2] : x[3], 8);
    return (r1 ? b : a) + __shfl_xor_sync(~0u, r1 ? a : b, 16);
}

// Shared memory of a CTA for T nodes, TP with padding, in floats: rows of k and q (padded by 4, so that float4 reads of neighbouring rows fall on
// different banks), L (before that the products D) and P, R and Gam S^T q, e^g, Gam, beta
template <int K, int TP> __host__ __device__ constexpr int tree_floats(int T, int V) {
    return T * (2 * (K + 4) + 2 * V) + TP * (2 * (TP + 4) + 3);
}

__device__ __forceinline__ uint32_t shared(const void *p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

template <int K, int TP> __global__ void __launch_bounds__(256) k_tree(const __grid_constant__ DecodeArgs a, bool rows16) {
    constexpr int NR = K / 4, KP = K + 4, LS = TP + 4, NB = TP / 16;
    extern __shared__ float4 smem4[];
    const int T = a.T, V = a.V;
    float *s_k = reinterpret_cast<float *>(smem4), *s_q = s_k + T * KP, *s_d = s_q + T * KP, *s_y = s_d + T * V;
    float *s_l = s_y + T * V, *s_p = s_l + TP * LS, *s_a = s_p + TP * LS, *s_gam = s_a + TP, *s_b = s_gam + TP;
    __shared__ int s_par[TP];
    const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, half = tid >= V, warp = (tid - half * V) >> 5;
    const int c = lane & 7, r = lane >> 3;
    const int n = blockIdx.x / a.Hv, h = blockIdx.x - n * a.Hv, hq = h / a.G;
    float *o = static_cast<float *>(a.o) + ((int64_t)n * T * a.Hv + h) * V;
    const int64_t o_tok = (int64_t)a.Hv * V;
    const float nan = __int_as_float(0x7fffffff);

    wait_for_previous();
    const int64_t slot = a.state_indices ? a.state_indices[n] : n;
    if (slot < 0 || slot >= a.n_slots) {
        for (int t = half; t < T; t += 2) o[t * o_tok + tid - half * V] = slot < 0 ? 0.f : nan;
        return;
    }
    const int col = warp * kTile + 4 * c + r;  // the column whose sums this lane gets
    const float *src = a.state + slot * a.slot_stride + (int64_t)h * K * V + warp * kTile + 4 * c;
    float4 S[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) S[i] = *reinterpret_cast<const float4 *>(src + (16 * (i >> 2) + 4 * r + (i & 3)) * V);

    const float *q = static_cast<const float *>(a.q) + n * a.sq.batch + hq * a.sq.head;
    const float *k = static_cast<const float *>(a.k) + n * a.sk.batch + hq * a.sk.head;
    const float *v = static_cast<const float *>(a.v) + n * a.sv.batch + h * a.sv.head;
    const float *g = a.g + n * a.sg.batch + h * a.sg.head, *beta = a.beta + n * a.sb.batch + h * a.sb.head;
    // everything on its way at once: 16 bytes a copy where the rows allow it, 4 elsewhere
    auto rows = [&](float *dst, int pitch, const float *from, int64_t step, int width) {
        if (rows16) {
            for (int e = tid; e < T * (width / 4); e += nt) {
                const int t = e / (width / 4), x = 4 * (e - t * (width / 4));
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(shared(dst + t * pitch + x)), "l"(from + t * step + x)
                             : "memory");
            }
        } else {
            for (int e = tid; e < T * width; e += nt) {
                const int t = e / width, x = e - t * width;
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(shared(dst + t * pitch + x)), "l"(from + t * step + x)
                             : "memory");
            }
        }
    };
    if (tid < TP) {
        s_a[tid] = tid < T ? expf(g[tid * a.sg.token]) : 0.f;
        s_b[tid] = tid < T ? beta[tid * a.sb.token] : 0.f;
        s_par[tid] = tid < T ? a.parents[(int64_t)n * T + tid] : -2;
    }
    rows(s_k, KP, k, a.sk.token, K);
    rows(s_q, KP, q, a.sq.token, K);
    rows(s_d, V, v, a.sv.token, V);
    for (int e = tid; e < TP * LS; e += nt) s_p[e] = 0.f;
    __syncthreads();

    // thread i: column i of D, the next one Gam (the column of the state), and which nodes are absent or hang on a
    // parent that is none
    uint64_t absent = 0, bad = 0;
    for (int w = tid; w == tid || w <= TP; w += nt) {
        float *column = w < TP ? s_l + w : s_gam;
        const int pitch = w < TP ? LS : 1;
#pragma unroll 1
        for (int t = 0; t < T; ++t) {
            const int p = s_par[t];
            if (p >= t || (p >= 0 && (bad >> p & 1))) bad |= 1ull << t;
            else if (p < -1 || (p >= 0 && (absent >> p & 1))) absent |= 1ull << t;
            if (w <= TP) {
                const bool live = !((bad | absent) >> t & 1);
                const float above = p >= 0 && live ? column[p * pitch] : w == TP ? 1.f : 0.f;
                column[t * pitch] = !live ? 0.f : w == t ? 1.f : s_a[t] * above;
            }
        }
        if (w < TP)
            for (int t = T; t < TP; ++t) column[t * pitch] = 0.f;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    // L and P: a thread takes the nodes t0, t0 + 16, ... against i0, i0 + 16, ..., so that a row read serves several pairs
    for (int e = tid; e < 256; e += nt) {
        const int t0 = e & 15, i0 = e >> 4;
        if (t0 >= T || i0 >= T || (NB == 1 && i0 > t0)) continue;
        float kk[NB][NB], qk[NB][NB];
#pragma unroll
        for (int x = 0; x < NB; ++x)
#pragma unroll
            for (int y = 0; y < NB; ++y) kk[x][y] = qk[x][y] = 0.f;
#pragma unroll 2
        for (int j = 0; j < K / 4; ++j) {
            float4 B[NB];
#pragma unroll
            for (int y = 0; y < NB; ++y) B[y] = *reinterpret_cast<const float4 *>(s_k + min(i0 + 16 * y, T - 1) * KP + 4 * j);
#pragma unroll
            for (int x = 0; x < NB; ++x) {
                const int row = min(t0 + 16 * x, T - 1) * KP + 4 * j;
                const float4 A = *reinterpret_cast<const float4 *>(s_k + row), Q = *reinterpret_cast<const float4 *>(s_q + row);
#pragma unroll
                for (int y = 0; y <= x; ++y) {
                    kk[x][y] = fmaf(A.x, B[y].x, fmaf(A.y, B[y].y, fmaf(A.z, B[y].z, fmaf(A.w, B[y].w, kk[x][y]))));
                    qk[x][y] = fmaf(Q.x, B[y].x, fmaf(Q.y, B[y].y, fmaf(Q.z, B[y].z, fmaf(Q.w, B[y].w, qk[x][y]))));
                }
            }
        }
#pragma unroll
        for (int x = 0; x < NB; ++x)
#pragma unroll
            for (int y = 0; y <= x; ++y) {
                const int t = t0 + 16 * x, i = i0 + 16 * y;
                const float D = s_l[t * LS + i];  // 0 where i is not above t: what i holds does not matter then
                s_l[t * LS + i] = i < t && D != 0.f ? s_b[t] * D * kk[x][y] : 0.f;
                s_p[t * LS + i] = i <= t && D != 0.f ? D * qk[x][y] : 0.f;
            }
    }
    __syncthreads();

#pragma unroll 1
    for (int t = half; t < T; t += 2) {
        float ks[4] = {0.f, 0.f, 0.f, 0.f}, qs[4] = {0.f, 0.f, 0.f, 0.f};
        const float4 *k4 = reinterpret_cast<const float4 *>(s_k + t * KP), *q4 = reinterpret_cast<const float4 *>(s_q + t * KP);
#pragma unroll
        for (int i = 0; i < K / 16; ++i) {
            const float4 kk = k4[4 * i + r], qq = q4[4 * i + r];
            const float kj[4] = {kk.x, kk.y, kk.z, kk.w}, qj[4] = {qq.x, qq.y, qq.z, qq.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float4 x = S[4 * i + j];
                ks[0] = fmaf(kj[j], x.x, ks[0]), qs[0] = fmaf(qj[j], x.x, qs[0]);
                ks[1] = fmaf(kj[j], x.y, ks[1]), qs[1] = fmaf(qj[j], x.y, qs[1]);
                ks[2] = fmaf(kj[j], x.z, ks[2]), qs[2] = fmaf(qj[j], x.z, qs[2]);
                ks[3] = fmaf(kj[j], x.w, ks[3]), qs[3] = fmaf(qj[j], x.w, qs[3]);
            }
        }
        // what an absent node holds is dropped
        const float R = s_b[t] * (s_d[t * V + col] - s_gam[t] * reduce_columns(ks, r));
        s_y[t * V + col] = s_gam[t] * reduce_columns(qs, r);
        s_d[t * V + col] = (bad | absent) >> t & 1 ? 0.f : R;
    }
    __syncthreads();
    float x[TP], zeros = 0.f;
#pragma unroll
    for (int t = 0; t < TP; ++t) x[t] = t < T ? s_d[t * V + col] : 0.f;
    if (!half) {
        // four rows at a time: what the rows before them give, then the triangle between the four
#pragma unroll
        for (int t = 0; t < TP; t += 4) {
            if (t % 16 == 0 && t >= T) break;
            float acc[4] = {x[t], x[t + 1], x[t + 2], x[t + 3]};
#pragma unroll
            for (int i = 0; i < t; i += 4)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float4 l = *reinterpret_cast<const float4 *>(s_l + (t + j) * LS + i);
                    acc[j] = fmaf(-l.x, x[i], acc[j]);
                    acc[j] = fmaf(-l.y, x[i + 1], acc[j]);
                    acc[j] = fmaf(-l.z, x[i + 2], acc[j]);
                    acc[j] = fmaf(-l.w, x[i + 3], acc[j]);
                }
            const float4 l1 = *reinterpret_cast<const float4 *>(s_l + (t + 1) * LS + t);
            const float4 l2 = *reinterpret_cast<const float4 *>(s_l + (t + 2) * LS + t);
            const float4 l3 = *reinterpret_cast<const float4 *>(s_l + (t + 3) * LS + t);
            acc[1] = fmaf(-l1.x, acc[0], acc[1]);
            acc[2] = fmaf(-l2.y, acc[1], fmaf(-l2.x, acc[0], acc[2]));
            acc[3] = fmaf(-l3.z, acc[2], fmaf(-l3.y, acc[1], fmaf(-l3.x, acc[0], acc[3])));
#pragma unroll
            for (int j = 0; j < 4; ++j) x[t + j] = acc[j];
        }
#pragma unroll
        for (int t = 0; t < TP; ++t) zeros = fmaf(x[t], 0.f, zeros);
        if (zeros == 0.f) {
#pragma unroll
            for (int t = 0; t < TP; ++t)
                if (t < T) s_d[t * V + col] = x[t];
        } else {
            for (int t = 0; t < T; ++t) {
                if ((bad | absent) >> t & 1) continue;
                float d = s_d[t * V + col];
                for (int p = s_par[t]; p >= 0; p = s_par[p]) d = fmaf(-s_l[t * LS + p], s_d[p * V + col], d);
                s_d[t * V + col] = d;
            }
        }
    }
    __syncthreads();
    if (half)
#pragma unroll
        for (int t = 0; t < TP; ++t) {
            x[t] = t < T ? s_d[t * V + col] : 0.f;
            zeros = fmaf(x[t], 0.f, zeros);
        }
    if (zeros != 0.f) {
        for (int t = half; t < T; t += 2) {
            float acc = s_y[t * V + col];
            if (!((bad | absent) >> t & 1))
                for (int p = t; p >= 0; p = s_par[p]) acc = fmaf(s_p[t * LS + p], s_d[p * V + col], acc);
            o[t * o_tok + col] = bad >> t & 1 ? nan : absent >> t & 1 ? 0.f : a.scale * acc;
        }
        return;
    }
#pragma unroll
    for (int t = 0; t < TP; t += 4) {
        if (t % 16 == 0 && t >= T) break;
        if ((t / 4) % 2 != half) continue;
        float acc[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j] = t + j < T ? s_y[(t + j) * V + col] : 0.f;
#pragma unroll
        for (int i = 0; i <= t; i += 4)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float4 p = *reinterpret_cast<const float4 *>(s_p + (t + j) * LS + i);
                acc[j] = fmaf(p.x, x[i], acc[j]);
                acc[j] = fmaf(p.y, x[i + 1], acc[j]);
                acc[j] = fmaf(p.z, x[i + 2], acc[j]);
                acc[j] = fmaf(p.w, x[i + 3], acc[j]);
            }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (t + j < T) {
                const uint64_t bit = 1ull << (t + j);
                o[(t + j) * o_tok + col] = bad & bit ? nan : absent & bit ? 0.f : a.scale * acc[j];
            }
    }
}

template <int K, int TP> cudaError_t launch(const DecodeArgs &a, cudaStream_t st) {
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(k_tree<K, TP>, tree_floats<K, TP>(TP, 128) * 4, done);
    if (e != cudaSuccess) return e;
    const int64_t steps = a.sq.batch | a.sq.token | a.sq.head | a.sk.batch | a.sk.token | a.sk.head | a.sv.batch | a.sv.token |
                          a.sv.head;
    const uintptr_t at = reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v);
    const bool rows16 = !(steps & 3) && !(at & 15);  // 16 rows of 32 heads, 48 nodes: 142 us, 147 with pieces of 4 bytes
    return launch_behind(k_tree<K, TP>, dim3((unsigned)(a.n_seqs * a.Hv)), 2 * a.V, (size_t)tree_floats<K, TP>(a.T, a.V) * 4, st, a, rows16);
}
// The triangles' loops end at the width: 16 rows of 32 heads with 7, 16, 32 and 48 nodes take 35, 55, 98 and 144 us
// and with 64 as the only width 47, 74, 111 and 151.
template <int K> cudaError_t launch_nodes(const DecodeArgs &a, cudaStream_t st) {
    if (a.T <= 16) return launch<K, 16>(a, st);
    if (a.T <= 32) return launch<K, 32>(a, st);
    if (a.T <= 48) return launch<K, 48>(a, st);
    return launch<K, 64>(a, st);
}

}  // namespace

cudaError_t launch_tree(const DecodeArgs &a, int K, gdn_dtype io, cudaStream_t st) {
    if (io == GDN_BF16) return launch_tree_tc(a, K, st);
    return K == 128 ? launch_nodes<128>(a, st) : launch_nodes<64>(a, st);
}

}  // namespace gdn
