// decode.cu -- the gated delta rule token by token, on a pool of states.
//
// Per row and value head, with a = e^g:  d = beta (v - a S^T k),  S' = a S + k d^T,  o = scale S'^T q.
// Both products are taken from the state before the update, o = scale (a S^T q + (q.k) d), so one pass over
// the state's registers serves k and q and a second one updates it.
//
// A warp holds a [K][32] tile of the state in registers: lane = (r, c) with c = 0..7 has the four columns
// 4c .. 4c+3 of the rows 16 i + 4 r + j (K values of 32 bits per lane, K/4 loads of 16 bytes, each a full
// 128-byte line per row across the lanes).  The value columns are independent, so nothing crosses warps;
// the four r lanes of a column group meet through shuffles.
#include <cuda_bf16.h>

#include "common.cuh"
#include "decode.h"

namespace gdn {
namespace {

constexpr int kTok = 8;   // tokens staged in shared memory at a time
constexpr int kTile = 32; // state columns per warp

// Sums x[0..3] (the lane's four columns) over the four r lanes; lane (r, c) gets column 4c + r.
__device__ __forceinline__ float reduce_columns(const float (&x)[4], int r) {
    const bool r0 = r & 1, r1 = r & 2;
    float a = r0 ? x[1] : x[0], b = r0 ? x[3] : x[2];
    a += __shfl_xor_sync(~0u, r0 ? x[0] : x[1], 8);
    b += __shfl_xor_sync(~0u, r0 ? x[2] : x[3], 8);
    return (r1 ? b : a) + __shfl_xor_sync(~0u, r1 ? a : b, 16);
}

template <int K, typename IO>
__global__ void __launch_bounds__(128) k_recurrent(const DecodeArgs a) {
    constexpr int NR = K / 4;  // rows per lane
    __shared__ float4 s_k4[kTok][K / 4], s_q4[kTok][K / 4];
    __shared__ float s_v[kTok][128], s_a[kTok], s_b[kTok];
    __shared__ int s_tok[kTok];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int c = lane & 7, r = lane >> 3;
    const int n = blockIdx.x / a.Hv, h = blockIdx.x - n * a.Hv, hq = h / a.G;
    const int cta_cols = blockDim.x;  // 32 columns per warp
    const int col0 = blockIdx.y * cta_cols;

    // the row's tokens: [bos, bos + len) of batch row b, or its list
    int64_t bos = 0, row = n;
    int b = n, len = a.token_indices ? a.n_steps : a.T;
    if (a.cu) {
        const int lo = a.cu[n], hi = a.cu[n + 1];
        if (lo < 0 || hi < lo || hi > a.T) return;  // not offsets of this tensor
        b = 0, bos = lo, len = hi - lo, row = 0;
    }
    const int64_t out_row = (a.cu ? bos : row * (int64_t)len);  // first row of o
    const int64_t slot = a.state_indices ? a.state_indices[n] : n;
    const bool idle = slot < 0;
    IO *o = static_cast<IO *>(a.o);
    if (idle || slot >= a.n_slots) {
        if (o)
            for (int t = 0; t < len; ++t)
                o[((out_row + t) * a.Hv + h) * a.V + col0 + tid] = from_f<IO>(idle ? 0.f : __int_as_float(0x7fffffff));
        return;
    }

    const int64_t head = (int64_t)h * K * a.V + col0 + warp * kTile + 4 * c;
    const float *src = a.state + slot * a.slot_stride + head;
    float4 S[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i)
        S[i] = *reinterpret_cast<const float4 *>(src + (int64_t)(16 * (i >> 2) + 4 * r + (i & 3)) * a.V);

    const IO *q = static_cast<const IO *>(a.q) + b * a.sq.batch + hq * a.sq.head;
    const IO *k = static_cast<const IO *>(a.k) + b * a.sk.batch + hq * a.sk.head;
    const IO *v = static_cast<const IO *>(a.v) + b * a.sv.batch + (int64_t)h * a.sv.head + col0;
    const float *g = a.g + b * a.sg.batch + h * a.sg.head, *beta = a.beta + b * a.sb.batch + h * a.sb.head;
    float *s_k = reinterpret_cast<float *>(s_k4), *s_q = reinterpret_cast<float *>(s_q4);

    bool bad = false;
    int t0 = 0;
    for (bool more = true; more && t0 < len; t0 += kTok) {
        int m = min(kTok, len - t0);
        if (t0) __syncthreads();
        if (a.token_indices) {
            if (tid < m) s_tok[tid] = a.token_indices[(int64_t)n * a.n_steps + t0 + tid];
            __syncthreads();
            for (int t = 0; t < m; ++t) {
                const int at = s_tok[t];
                if (at >= 0 && at < a.T) continue;
                bad = at >= 0;
                m = t, more = false;
                break;
            }
        }
        for (int e = tid; e < m * K; e += cta_cols) {
            const int t = e / K, x = e % K;
            const int64_t at = a.token_indices ? s_tok[t] : bos + t0 + t;
            s_k[e] = to_f<IO>(k[at * a.sk.token + x]);
            if (o) s_q[e] = to_f<IO>(q[at * a.sq.token + x]);
        }
        for (int t = 0; t < m; ++t) {
            const int64_t at = a.token_indices ? s_tok[t] : bos + t0 + t;
            s_v[t][tid] = to_f<IO>(v[at * a.sv.token + tid]);
            if (tid == 0) s_a[t] = expf(g[at * a.sg.token]), s_b[t] = beta[at * a.sb.token];
        }
        __syncthreads();

        for (int t = 0; t < m; ++t) {
            float ks[4] = {0.f, 0.f, 0.f, 0.f}, qs[4] = {0.f, 0.f, 0.f, 0.f}, qk = 0.f;
#pragma unroll
            for (int i = 0; i < K / 16; ++i) {
                const float4 kk = s_k4[t][4 * i + r];
                const float kj[4] = {kk.x, kk.y, kk.z, kk.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float4 s = S[4 * i + j];
                    ks[0] = fmaf(kj[j], s.x, ks[0]);
                    ks[1] = fmaf(kj[j], s.y, ks[1]);
                    ks[2] = fmaf(kj[j], s.z, ks[2]);
                    ks[3] = fmaf(kj[j], s.w, ks[3]);
                }
                if (o) {
                    const float4 qq = s_q4[t][4 * i + r];
                    const float qj[4] = {qq.x, qq.y, qq.z, qq.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float4 s = S[4 * i + j];
                        qs[0] = fmaf(qj[j], s.x, qs[0]);
                        qs[1] = fmaf(qj[j], s.y, qs[1]);
                        qs[2] = fmaf(qj[j], s.z, qs[2]);
                        qs[3] = fmaf(qj[j], s.w, qs[3]);
                        qk = fmaf(qj[j], kj[j], qk);
                    }
                }
            }
            const float al = s_a[t];
            const int col = warp * kTile + 4 * c + r;
            const float d = s_b[t] * (s_v[t][col] - al * reduce_columns(ks, r));
            if (o) {
                qk += __shfl_xor_sync(~0u, qk, 8);
                qk += __shfl_xor_sync(~0u, qk, 16);
                const float out = a.scale * fmaf(qk, d, al * reduce_columns(qs, r));
                o[((out_row + t0 + t) * a.Hv + h) * a.V + col0 + col] = from_f<IO>(out);
            }
            float dj[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) dj[j] = __shfl_sync(~0u, d, c + 8 * j);
#pragma unroll
            for (int i = 0; i < K / 16; ++i) {
                const float4 kk = s_k4[t][4 * i + r];
                const float kj[4] = {kk.x, kk.y, kk.z, kk.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float4 &s = S[4 * i + j];
                    s.x = fmaf(kj[j], dj[0], al * s.x);
                    s.y = fmaf(kj[j], dj[1], al * s.y);
                    s.z = fmaf(kj[j], dj[2], al * s.z);
                    s.w = fmaf(kj[j], dj[3], al * s.w);
                }
            }
        }
        if (!more && o)  // past the end of a list of tokens, or at an index that is none
            for (int t = t0 + m; t < len; ++t)
                o[((out_row + t) * a.Hv + h) * a.V + col0 + tid] = from_f<IO>(bad ? __int_as_float(0x7fffffff) : 0.f);
    }
    if (bad) return;
    float *dst = (a.out_state ? a.out_state + (int64_t)n * a.Hv * K * a.V : a.state + slot * a.slot_stride) + head;
#pragma unroll
    for (int i = 0; i < NR; ++i)
        *reinterpret_cast<float4 *>(dst + (int64_t)(16 * (i >> 2) + 4 * r + (i & 3)) * a.V) = S[i];
}

template <int K, typename IO> cudaError_t launch(const DecodeArgs &a, cudaStream_t st) {
    const dim3 grid((unsigned)(a.n_seqs * a.Hv), 1);
    k_recurrent<K, IO><<<grid, a.V, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_recurrent(const DecodeArgs &a, int K, gdn_dtype io, cudaStream_t st) {
    if (io == GDN_BF16) return K == 128 ? launch<128, __nv_bfloat16>(a, st) : launch<64, __nv_bfloat16>(a, st);
    return K == 128 ? launch<128, float>(a, st) : launch<64, float>(a, st);
}

}  // namespace gdn
