// linear.cu -- linear attention on the CUDA cores (fp32 inputs; see linear.h for what a run is), and the small
// kernels around the runs.
//
// k_linear: a CTA takes one sequence (or segment of one), head and 64 columns of c, and goes through it in blocks of 32
// tokens with the state [da][64] in shared memory: P = (A B^T) under the decays, O = P C + l^(j + e) A X,
// X <- l^n X + B^T (w C).  All in fp32.
#include <cuda_bf16.h>

#include "common.cuh"
#include "linear.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int N = 32;     // tokens of a block
constexpr int COLS = 64;  // columns of c and the state per CTA

template <int DA> struct Smem {
    float a[N][DA + 1], b[N][DA + 1];
    float c[N][COLS], wc[N][COLS], x[DA][COLS];
    float p[N][N + 1];
    float pow[N + 1];  // l^0 .. l^N
};

// Rows tok0 .. tok0 + n - 1 of a head, columns 0 .. D - 1, in the order of the scan
template <typename IO, int D, int PITCH>
__device__ __forceinline__ void load_rows(float *to, const IO *from, int64_t pitch, int n, bool reverse) {
#pragma unroll 4
    for (int i = threadIdx.x; i < N * D; i += kThreads) {
        const int j = i / D, x = i % D;
        to[j * PITCH + x] = j < n ? to_f<IO>(from[(int64_t)(reverse ? n - 1 - j : j) * pitch + x]) : 0.f;
    }
}

template <typename IO, int DA> __global__ void __launch_bounds__(kThreads) k_linear(const __grid_constant__ LinearRun r) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    Smem<DA> &s = *reinterpret_cast<Smem<DA> *>(smem_raw);
    const int tid = threadIdx.x, h = blockIdx.y, col0 = blockIdx.z * COLS;
    const int seq = blockIdx.x / r.n_seg, part = blockIdx.x % r.n_seg;
    const LinearSpan span = linear_span(r, seq);
    const int from = part * span.per_seg * C, to = min(span.tokens, (part + 1) * span.per_seg * C);
    const int64_t unit = (int64_t)seq * r.Hv + h, words = (int64_t)DA * r.dc;
    const float *init = r.init ? r.init + unit * words : nullptr;
    float *fin = r.fin ? r.fin + unit * words : nullptr;
    bool init_t = r.transposed, fin_t = r.transposed;
    if (r.mode == LIN_SEG) {  // the last segment feeds no other
        if (to >= span.tokens) return;
        init = nullptr, fin = r.seg + (unit * r.n_seg + part) * words, fin_t = false;
    } else if (part > 0) {
        if (from >= to) return;
        init = r.seg + (unit * r.n_seg + part) * words;
        init_t = false;
    }
    if (r.mode != LIN_SEG && to < span.tokens) fin = nullptr;
    const float g = r.g ? r.g[h] : 0.f;
    if (tid <= N) s.pow[tid] = tid ? expf(g * tid) : 1.f;
    for (int i = tid; i < DA * COLS; i += kThreads) {
        const int x = i / COLS, y = col0 + i % COLS;
        s.x[x][i % COLS] = init ? init[init_t ? y * DA + x : x * r.dc + y] : 0.f;
    }
    const int64_t batch = r.cu ? 0 : seq, first = r.cu ? span.first : 0;
    const bool outs = r.mode != LIN_SEG && r.out;
    const IO *a = static_cast<const IO *>(r.a) + batch * r.sa.batch + h / r.ga * r.sa.head;
    const IO *b = static_cast<const IO *>(r.b) + batch * r.sb.batch + h / r.gb * r.sb.head;
    const IO *c = static_cast<const IO *>(r.c) + batch * r.sc.batch + h / r.gc * r.sc.head + col0;
    const int ty = tid / 16, tx = tid % 16;  // tiles of 2 x 2 of P, 2 x 4 of O, DA / 16 x 4 of X
    for (int at = from; at < to; at += N) {
        const int n = min(N, to - at);
        const int64_t tok = first + (r.reverse ? span.tokens - at - n : at);  // the block's lowest
        __syncthreads();
        if (outs) load_rows<IO, DA, DA + 1>(&s.a[0][0], a + tok * r.sa.token, r.sa.token, n, r.reverse);
        load_rows<IO, DA, DA + 1>(&s.b[0][0], b + tok * r.sb.token, r.sb.token, n, r.reverse);
        load_rows<IO, COLS, COLS>(&s.c[0][0], c + tok * r.sc.token, r.sc.token, n, r.reverse);
        __syncthreads();
        for (int i = tid; i < N * COLS; i += kThreads) {  // w_j c_j
            const int j = i / COLS;
            s.wc[j][i % COLS] = j < n ? r.s_scale * s.pow[n - j - r.e] * s.c[j][i % COLS] : 0.f;
        }
        if (outs) {
            float p[2][2] = {};
#pragma unroll 8
            for (int x = 0; x < DA; ++x) {
                const float a0 = s.a[2 * ty][x], a1 = s.a[2 * ty + 1][x], b0 = s.b[tx][x], b1 = s.b[tx + 16][x];
                p[0][0] = fmaf(a0, b0, p[0][0]), p[0][1] = fmaf(a0, b1, p[0][1]);
                p[1][0] = fmaf(a1, b0, p[1][0]), p[1][1] = fmaf(a1, b1, p[1][1]);
            }
#pragma unroll
            for (int y = 0; y < 2; ++y)
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    const int j = 2 * ty + y, i = tx + 16 * z;
                    s.p[j][i] = i <= j ? r.p_scale * s.pow[j - i] * p[y][z] : 0.f;
                }
            __syncthreads();
            float o[2][4] = {}, q[2][4] = {};
#pragma unroll 4
            for (int x = 0; x < DA; ++x) {
                const float4 xx = *reinterpret_cast<const float4 *>(&s.x[x][4 * tx]);
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const float aa = s.a[2 * ty + y][x];
                    q[y][0] = fmaf(aa, xx.x, q[y][0]), q[y][1] = fmaf(aa, xx.y, q[y][1]);
                    q[y][2] = fmaf(aa, xx.z, q[y][2]), q[y][3] = fmaf(aa, xx.w, q[y][3]);
                }
            }
#pragma unroll 4
            for (int i = 0; i < N; ++i) {
                const float4 cc = *reinterpret_cast<const float4 *>(&s.c[i][4 * tx]);
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const float pp = s.p[2 * ty + y][i];
                    o[y][0] = fmaf(pp, cc.x, o[y][0]), o[y][1] = fmaf(pp, cc.y, o[y][1]);
                    o[y][2] = fmaf(pp, cc.z, o[y][2]), o[y][3] = fmaf(pp, cc.w, o[y][3]);
                }
            }
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const int j = 2 * ty + y;
                if (j >= n) continue;
                const float w = r.o_scale * s.pow[j + r.e];
                const int64_t row = batch * r.T + tok + (r.reverse ? n - 1 - j : j);
                const int64_t to_at = (row * r.Hv + h) * r.dc + col0 + 4 * tx;
                const float v[4] = {fmaf(w, q[y][0], o[y][0]), fmaf(w, q[y][1], o[y][1]), fmaf(w, q[y][2], o[y][2]),
                                    fmaf(w, q[y][3], o[y][3])};
                if (r.out_f32) {
                    *reinterpret_cast<float4 *>(static_cast<float *>(r.out) + to_at) = make_float4(v[0], v[1], v[2], v[3]);
                } else {
                    IO *out = static_cast<IO *>(r.out) + to_at;
#pragma unroll
                    for (int z = 0; z < 4; ++z) out[z] = from_f<IO>(v[z]);
                }
            }
        }
        __syncthreads();
        float u[DA / 16][4] = {};
        for (int i = 0; i < n; ++i) {
            const float4 w = *reinterpret_cast<const float4 *>(&s.wc[i][4 * tx]);
#pragma unroll
            for (int y = 0; y < DA / 16; ++y) {
                const float bb = s.b[i][ty + 16 * y];
                u[y][0] = fmaf(bb, w.x, u[y][0]), u[y][1] = fmaf(bb, w.y, u[y][1]);
                u[y][2] = fmaf(bb, w.z, u[y][2]), u[y][3] = fmaf(bb, w.w, u[y][3]);
            }
        }
        const float l1 = expm1f(g * n);  // X l^n as X + l1 X: nothing is lost where l is all but 1
#pragma unroll
        for (int y = 0; y < DA / 16; ++y) {
            float4 &x = *reinterpret_cast<float4 *>(&s.x[ty + 16 * y][4 * tx]);
            x.x += fmaf(l1, x.x, u[y][0]), x.y += fmaf(l1, x.y, u[y][1]);
            x.z += fmaf(l1, x.z, u[y][2]), x.w += fmaf(l1, x.w, u[y][3]);
        }
    }
    __syncthreads();
    if (fin)
        for (int i = tid; i < DA * COLS; i += kThreads) {
            const int x = i / COLS, y = col0 + i % COLS;
            fin[fin_t ? y * DA + x : x * r.dc + y] = s.x[x][i % COLS];
        }
}

template <typename IO, int DA> cudaError_t launch(const LinearRun &r, cudaStream_t st) {
    cudaError_t e = cudaFuncSetAttribute(k_linear<IO, DA>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Smem<DA>));
    if (e != cudaSuccess) return e;
    k_linear<IO, DA><<<dim3((unsigned)(r.n_seqs * r.n_seg), (unsigned)r.Hv, (unsigned)(r.dc / COLS)), kThreads, sizeof(Smem<DA>), st>>>(r);
    return cudaGetLastError();
}

// seg[p], the state that segment p adds, becomes the state that enters segment p
__global__ void __launch_bounds__(256) k_join(const __grid_constant__ LinearRun r) {
    const int words = r.da * r.dc, seq = blockIdx.x, h = blockIdx.y, i = blockIdx.z * 256 + threadIdx.x;
    if (i >= words) return;
    const LinearSpan span = linear_span(r, seq);
    const int64_t unit = (int64_t)seq * r.Hv + h;
    const float g = r.g ? r.g[h] : 0.f;
    const float l1 = span.per_seg ? expm1f(g * (float)(span.per_seg * C)) : 0.f;
    const int x = i / r.dc, y = i % r.dc;
    float X = r.init ? r.init[unit * words + (r.transposed ? y * r.da + x : i)] : 0.f;
    float *seg = r.seg + unit * r.n_seg * words + i;
    const int used = span.per_seg ? (span.chunks + span.per_seg - 1) / span.per_seg : 0;  // segments with tokens
    for (int p = 0; p + 1 < used; ++p) {  // all of these are full
        const float add = seg[(int64_t)p * words];
        if (p > 0) seg[(int64_t)p * words] = X;
        X += fmaf(l1, X, add);
    }
    if (used > 1) seg[(int64_t)(used - 1) * words] = X;
}

template <typename IO> __global__ void __launch_bounds__(256) k_group_sum(const float4 *x, IO *out, int64_t n4, int G, int d4) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;  // four values of out
    if (i >= n4) return;
    const int64_t head = i / d4;
    const float4 *from = x + head * G * d4 + i % d4;
    float4 s = from[0];
    for (int j = 1; j < G; ++j) {
        const float4 y = from[(int64_t)j * d4];
        s.x += y.x, s.y += y.y, s.z += y.z, s.w += y.w;
    }
    IO *o = out + 4 * i;
    o[0] = from_f<IO>(s.x), o[1] = from_f<IO>(s.y), o[2] = from_f<IO>(s.z), o[3] = from_f<IO>(s.w);
}

// 64 rows per CTA
__global__ void __launch_bounds__(256) k_unclaimed(unsigned char *x, int T, int64_t row_bytes, const int32_t *cu, int n_seqs) {
    __shared__ unsigned int claimed[2];
    const int row0 = blockIdx.x * 64;
    if (threadIdx.x < 2) claimed[threadIdx.x] = 0;
    __syncthreads();
    for (int s = threadIdx.x; s < n_seqs; s += 256) {
        const int lo = cu[s], hi = cu[s + 1];
        if (lo < 0 || hi < lo || hi > T) continue;
        const int a = max(lo - row0, 0), b = min(hi - row0, 64);
        if (a >= b) continue;
        const uint64_t m = (b == 64 ? ~0ull : (1ull << b) - 1) & ~((1ull << a) - 1);
        if ((unsigned)m) atomicOr(&claimed[0], (unsigned)m);
        if ((unsigned)(m >> 32)) atomicOr(&claimed[1], (unsigned)(m >> 32));
    }
    __syncthreads();
    for (int i = 0; i < 64 && row0 + i < T; ++i) {
        if (claimed[i >> 5] >> (i & 31) & 1) continue;
        uint4 *to = reinterpret_cast<uint4 *>(x + (int64_t)(row0 + i) * row_bytes);
        for (int64_t j = threadIdx.x; j < row_bytes / 16; j += 256) to[j] = make_uint4(0, 0, 0, 0);
    }
}

}  // namespace

cudaError_t launch_linear_simt(const LinearRun &r, gdn_dtype io, cudaStream_t st) {
    if (io == GDN_BF16) return r.da == 128 ? launch<__nv_bfloat16, 128>(r, st) : launch<__nv_bfloat16, 64>(r, st);
    return r.da == 128 ? launch<float, 128>(r, st) : launch<float, 64>(r, st);
}

cudaError_t launch_linear_join(const LinearRun &r, cudaStream_t st) {
    k_join<<<dim3((unsigned)r.n_seqs, (unsigned)r.Hv, (unsigned)(r.da * r.dc / 256)), 256, 0, st>>>(r);
    return cudaGetLastError();
}

cudaError_t launch_group_sum(const float *x, void *out, int64_t tokens, int heads, int G, int d, gdn_dtype io, cudaStream_t st) {
    const int64_t n4 = tokens * heads * d / 4;
    if (n4 == 0) return cudaSuccess;
    const unsigned grid = (unsigned)((n4 + 255) / 256);
    const float4 *x4 = reinterpret_cast<const float4 *>(x);
    if (io == GDN_BF16) k_group_sum<<<grid, 256, 0, st>>>(x4, static_cast<__nv_bfloat16 *>(out), n4, G, d / 4);
    else k_group_sum<<<grid, 256, 0, st>>>(x4, static_cast<float *>(out), n4, G, d / 4);
    return cudaGetLastError();
}

cudaError_t launch_unclaimed(void *x, int T, int64_t row_bytes, const int32_t *cu, int n_seqs, cudaStream_t st) {
    if (T == 0) return cudaSuccess;
    k_unclaimed<<<(unsigned)((T + 63) / 64), 256, 0, st>>>(static_cast<unsigned char *>(x), T, row_bytes, cu, n_seqs);
    return cudaGetLastError();
}

}  // namespace gdn
