// tree.cu -- a tree of drafted tokens answered from a state, which is only read.
//
// With S the state, anc(t) the nodes on the path down to t (t included) and, for i in anc(t), D_ti the product
// of e^g over the path's nodes after i, Gam_t the product over the whole path:
//     d_t = beta_t (v_t - Gam_t S^T k_t) - sum_{i in anc(t), i != t} L_ti d_i,   L_ti = beta_t D_ti (k_t . k_i)
//     o_t = scale (Gam_t S^T q_t + sum_{i in anc(t)} P_ti d_i),                  P_ti = D_ti (q_t . k_i)
// which is the recurrence along every path at once: no node needs a state of its own.  D is built by products
// down the tree (D_ti = e^{g_t} D_parent(t),i), so a gate of -inf stays 0 and nothing is a difference of sums.
// This file holds the CUDA-core kernel, for fp32 io; tree_tc.cu has the tensor-core kernel for bf16.
#include <cuda_bf16.h>

#include "common.cuh"
#include "decode.h"

namespace gdn {
namespace {

constexpr int kTile = 32;

__device__ __forceinline__ float reduce_columns(const float (&x)[4], int r) {
    const bool r0 = r & 1, r1 = r & 2;
    float a = r0 ? x[1] : x[0], b = r0 ? x[3] : x[2];
    a += __shfl_xor_sync(~0u, r0 ? x[0] : x[1], 8);
    b += __shfl_xor_sync(~0u, r0 ? x[2] : x[3], 8);
    return (r1 ? b : a) + __shfl_xor_sync(~0u, r1 ? a : b, 16);
}

// Shared memory of a CTA, in floats: k and q rows (padded by 4, so that float4 reads of neighbouring rows fall
// on different banks), L / P pairs, the corrections d, Gam and beta.
__host__ __device__ inline int tree_floats(int T, int K, int V) { return T * (2 * (K + 4) + 2 * T + V + 2); }

template <int K, typename IO> __global__ void __launch_bounds__(128) k_tree(const DecodeArgs a) {
    constexpr int NR = K / 4, KP = K + 4;
    extern __shared__ float4 smem4[];
    const int T = a.T, V = a.V;
    float *s_k = reinterpret_cast<float *>(smem4), *s_q = s_k + T * KP;
    float2 *s_lp = reinterpret_cast<float2 *>(s_q + T * KP);
    float *s_d = reinterpret_cast<float *>(s_lp + T * T);
    float *s_gam = s_d + T * V, *s_b = s_gam + T;
    __shared__ int s_par[GDN_TREE_MAX];
    const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5;
    const int c = lane & 7, r = lane >> 3;
    const int n = blockIdx.x / a.Hv, h = blockIdx.x - n * a.Hv, hq = h / a.G;
    IO *o = static_cast<IO *>(a.o) + ((int64_t)n * T * a.Hv + h) * V;
    const int64_t o_tok = (int64_t)a.Hv * V;

    wait_for_previous();
    const int64_t slot = a.state_indices ? a.state_indices[n] : n;
    if (slot < 0 || slot >= a.n_slots) {
        for (int t = 0; t < T; ++t) o[t * o_tok + tid] = from_f<IO>(slot < 0 ? 0.f : __int_as_float(0x7fffffff));
        return;
    }
    const float *src = a.state + slot * a.slot_stride + (int64_t)h * K * V + warp * kTile + 4 * c;
    float4 S[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i)
        S[i] = *reinterpret_cast<const float4 *>(src + (16 * (i >> 2) + 4 * r + (i & 3)) * V);

    const IO *q = static_cast<const IO *>(a.q) + n * a.sq.batch + hq * a.sq.head;
    const IO *k = static_cast<const IO *>(a.k) + n * a.sk.batch + hq * a.sk.head;
    const IO *v = static_cast<const IO *>(a.v) + n * a.sv.batch + h * a.sv.head;
    const float *g = a.g + n * a.sg.batch + h * a.sg.head, *beta = a.beta + n * a.sb.batch + h * a.sb.head;
    for (int e = tid; e < T * K; e += nt) {
        const int t = e / K, x = e % K;
        s_k[t * KP + x] = to_f<IO>(k[t * a.sk.token + x]);
        s_q[t * KP + x] = to_f<IO>(q[t * a.sq.token + x]);
    }
    for (int t = 0; t < T; ++t) s_d[t * V + tid] = to_f<IO>(v[t * a.sv.token + tid]);
    if (tid < T) {
        s_gam[tid] = expf(g[tid * a.sg.token]);
        s_b[tid] = beta[tid * a.sb.token];
        s_par[tid] = a.parents[(int64_t)n * T + tid];
    }
    __syncthreads();

    // thread i: column i of D, and which nodes are absent or hang on a parent that is none
    uint64_t absent = 0, bad = 0;
    for (int t = 0; t < T; ++t) {
        const int p = s_par[t];
        if (p >= t || (p >= 0 && (bad >> p & 1))) bad |= 1ull << t;
        else if (p < -1 || (p >= 0 && (absent >> p & 1))) absent |= 1ull << t;
        if (tid < T) {
            const bool live = !((bad | absent) >> t & 1);
            s_lp[t * T + tid].x = !live ? 0.f : tid == t ? 1.f : p >= 0 ? s_gam[t] * s_lp[p * T + tid].x : 0.f;
        }
    }
    __syncthreads();
    if (tid == 0)
        for (int t = 0; t < T; ++t)
            if (s_par[t] >= 0 && s_par[t] < t) s_gam[t] *= s_gam[s_par[t]];
    for (int e = tid; e < T * T; e += nt) {
        const int t = e / T, i = e - t * T;
        const float D = s_lp[e].x;
        float kk = 0.f, qk = 0.f;
        if (i <= t && D != 0.f) {
            const float4 *kt = reinterpret_cast<const float4 *>(s_k + t * KP), *ki = reinterpret_cast<const float4 *>(s_k + i * KP);
            const float4 *qt = reinterpret_cast<const float4 *>(s_q + t * KP);
#pragma unroll 4
            for (int x = 0; x < K / 4; ++x) {
                const float4 A = kt[x], B = ki[x], Q = qt[x];
                kk = fmaf(A.x, B.x, fmaf(A.y, B.y, fmaf(A.z, B.z, fmaf(A.w, B.w, kk))));
                qk = fmaf(Q.x, B.x, fmaf(Q.y, B.y, fmaf(Q.z, B.z, fmaf(Q.w, B.w, qk))));
            }
        }
        s_lp[e] = make_float2(i < t ? s_b[t] * D * kk : 0.f, D * qk);
    }
    __syncthreads();

    const int col = warp * kTile + 4 * c + r;  // the column whose sums this lane holds
    for (int t = 0; t < T; ++t) {
        float ks[4] = {0.f, 0.f, 0.f, 0.f}, qs[4] = {0.f, 0.f, 0.f, 0.f};
        const float4 *k4 = reinterpret_cast<const float4 *>(s_k + t * KP), *q4 = reinterpret_cast<const float4 *>(s_q + t * KP);
#pragma unroll
        for (int i = 0; i < K / 16; ++i) {
            const float4 kk = k4[4 * i + r], qq = q4[4 * i + r];
            const float kj[4] = {kk.x, kk.y, kk.z, kk.w}, qj[4] = {qq.x, qq.y, qq.z, qq.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float4 s = S[4 * i + j];
                ks[0] = fmaf(kj[j], s.x, ks[0]), qs[0] = fmaf(qj[j], s.x, qs[0]);
                ks[1] = fmaf(kj[j], s.y, ks[1]), qs[1] = fmaf(qj[j], s.y, qs[1]);
                ks[2] = fmaf(kj[j], s.z, ks[2]), qs[2] = fmaf(qj[j], s.z, qs[2]);
                ks[3] = fmaf(kj[j], s.w, ks[3]), qs[3] = fmaf(qj[j], s.w, qs[3]);
            }
        }
        float d = s_b[t] * (s_d[t * V + col] - s_gam[t] * reduce_columns(ks, r));
        float y = s_gam[t] * reduce_columns(qs, r);
        for (int i = 0; i < t; ++i) {
            const float2 lp = s_lp[t * T + i];
            const float di = s_d[i * V + col];
            d = fmaf(-lp.x, di, d);
            y = fmaf(lp.y, di, y);
        }
        y = fmaf(s_lp[t * T + t].y, d, y);
        if ((bad | absent) >> t & 1) d = 0.f;  // whatever the node holds: nobody sees it
        s_d[t * V + col] = d;  // read by this lane alone
        const float out = (bad >> t & 1) ? __int_as_float(0x7fffffff) : (absent >> t & 1) ? 0.f : a.scale * y;
        o[t * o_tok + col] = from_f<IO>(out);
    }
}

template <int K, typename IO> cudaError_t launch(const DecodeArgs &a, cudaStream_t st) {
    const int bytes = tree_floats(a.T, K, a.V) * 4;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(k_tree<K, IO>, tree_floats(GDN_TREE_MAX, K, 128) * 4, done);
    if (e != cudaSuccess) return e;
    return launch_behind(k_tree<K, IO>, dim3((unsigned)(a.n_seqs * a.Hv)), a.V, bytes, st, a);
}

}  // namespace

cudaError_t launch_tree(const DecodeArgs &a, int K, gdn_dtype io, cudaStream_t st) {
    if (io == GDN_BF16) return launch_tree_tc(a, K, st);
    return K == 128 ? launch<128, float>(a, st) : launch<64, float>(a, st);
}

}  // namespace gdn
