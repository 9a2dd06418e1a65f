// linear.cu -- linear attention on the CUDA cores (fp32 inputs; see linear.h for what a run is), and the small
// kernels around the runs.
//
// k_linear: a CTA takes one sequence (or segment of one), head and 64 columns of c, and goes through it in blocks of 64
// tokens with the state [da][64] in shared memory: P = (A B^T) under the decays, O = P C + l^(j + e) A X,
// X <- l^n X + (w B)^T C.  All in fp32, two at a time; the next block's rows come under a block's work.  Reads of shared
// memory bound it: 16 products for every two 16-byte reads of a thread's 4 x 4 tile, with eight warps on an SM (two times
// eight at 64 x 64).  A block takes 9 us at 64 x 64 and 14 at 128 x 128, 0.23 and 0.26 TFLOP/s an SM of 0.49; 4 x 1024
// tokens of 16 heads, 128 x 128, 227 us; 2 x 1000 of 8 heads, 64 x 64, 34 us (in segments of one block).  Two CTAs an SM are
// asked for at 64: with 160 registers, which the compiler takes otherwise, one fits, and those 34 us are 42.
#include <cuda_bf16.h>

#include "common.cuh"
#include "decode.h"
#include "linear.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int N = C;      // tokens of a block
constexpr int COLS = 64;  // columns of c and the state per CTA

template <int DA> struct Smem {
    float a[N][DA + 4], b[N][DA + 4];  // rows 4 banks apart
    float c[N][COLS], x[DA][COLS];
    float p[N][N + 4];
    float pow[N + 1];  // l^0 .. l^N
};

// Two fp32 at once
__device__ __forceinline__ uint64_t pair_of(float lo, float hi) {
    uint64_t p;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(lo), "f"(hi));
    return p;
}
__device__ __forceinline__ void halves(uint64_t p, float &lo, float &hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(p)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
struct Four {
    uint64_t lo, hi;
};
__device__ __forceinline__ Four four(const float *x) {
    const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(x);
    return {v.x, v.y};
}

// Rows of a block on their way: four values each of rows i / (D / 4), columns 4 (i % (D / 4))
template <typename IO, int D, bool VEC> struct Rows {
    static constexpr int EACH = N * D / 4 / kThreads;
    float4 v[EACH];
    // n rows from the lowest, `pitch` apart, in the order of the scan; 0 behind them
    __device__ __forceinline__ void load(const IO *from, int64_t pitch, int n, bool reverse) {
#pragma unroll
        for (int e = 0; e < EACH; ++e) {
            const int i = threadIdx.x + e * kThreads, j = i / (D / 4), x = i % (D / 4) * 4;
            v[e] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (j >= n) continue;
            const IO *at = from + (int64_t)(reverse ? n - 1 - j : j) * pitch + x;
            if constexpr (!VEC) v[e] = make_float4(to_f<IO>(at[0]), to_f<IO>(at[1]), to_f<IO>(at[2]), to_f<IO>(at[3]));
            else if constexpr (sizeof(IO) == 4) v[e] = *reinterpret_cast<const float4 *>(at);
            else {
                const uint2 u = *reinterpret_cast<const uint2 *>(at);
                v[e] = make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                                   __uint_as_float(u.y & 0xFFFF0000u));
            }
        }
    }
    __device__ __forceinline__ void store(float *to, int pitch) const {
#pragma unroll
        for (int e = 0; e < EACH; ++e) {
            const int i = threadIdx.x + e * kThreads;
            *reinterpret_cast<float4 *>(to + i / (D / 4) * pitch + i % (D / 4) * 4) = v[e];
        }
    }
};

template <typename IO, int DA, bool VEC> __global__ void __launch_bounds__(kThreads, DA == 64 ? 2 : 0) k_linear(const __grid_constant__ LinearRun r) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    Smem<DA> &s = *reinterpret_cast<Smem<DA> *>(smem_raw);
    wait_for_previous();
    const int tid = threadIdx.x, h = blockIdx.x % r.Hv, col0 = blockIdx.y * COLS, slot = blockIdx.x / r.Hv;
    int seq, part;
    const LinearSpan span = linear_place(r, slot, seq, part);
    if (seq < 0) return;
    const LinearPart range = linear_part(span.tokens, span.chunks, span.per_seg, part);
    const int from = range.from, to = range.to;
    const int64_t unit = (int64_t)seq * r.Hv + h, words = (int64_t)DA * r.dc;
    const float *init = r.init ? r.init + unit * words : nullptr;
    float *fin = r.fin ? r.fin + unit * words : nullptr, *seg = r.seg + ((int64_t)slot * r.Hv + h) * words;
    bool init_t = r.transposed, fin_t = r.transposed;
    if (r.mode == LIN_SEG) {  // the last segment feeds no other
        if (to >= span.tokens) return;
        init = nullptr, fin = seg, fin_t = false;
    } else if (part > 0) {
        if (from >= to) return;
        init = seg, init_t = false;
    }
    if (r.mode != LIN_SEG && to < span.tokens) fin = nullptr;
    const float g = r.g ? r.g[h] : 0.f;
    if (tid <= N) s.pow[tid] = tid ? expf(g * tid) : 1.f;
    for (int i = tid; i < DA * COLS; i += kThreads) {
        const int x = i / COLS, y = col0 + i % COLS;
        s.x[x][i % COLS] = init ? init[init_t ? y * DA + x : x * r.dc + y] : 0.f;
    }
    const int64_t batch = r.cu ? 0 : seq, first = span.first;
    const bool outs = r.mode != LIN_SEG && r.out;
    const IO *a = static_cast<const IO *>(r.a) + batch * r.sa.batch + h / r.ga * r.sa.head;
    const IO *b = static_cast<const IO *>(r.b) + batch * r.sb.batch + h / r.gb * r.sb.head;
    const IO *c = static_cast<const IO *>(r.c) + batch * r.sc.batch + h / r.gc * r.sc.head + col0;
    // Eight warps, two by four, of eight by four lanes: 4 x 4 of P and O by each thread (rows 8 apart, P's columns 4 apart),
    // ROWS x 4 of X.  So a read of 16 bytes by a warp meets no bank twice; rows by half warps took twice as many cycles
    const int wr = tid >> 7, wc = (tid >> 5) & 3, ty = (tid >> 2) & 7, tx = tid & 3;
    const int j0 = 32 * wr + ty, y0 = 16 * wc + 4 * tx;
    constexpr int ROWS = DA / 16;
    const int x0 = DA / 2 * wr + ROWS * ty;
    Rows<IO, DA, VEC> ra, rb;
    Rows<IO, COLS, VEC> rc;
    auto fetch = [&](int at) {
        const int n = min(N, to - at);
        const int64_t tok = first + (r.reverse ? span.tokens - at - n : at);  // the block's lowest
        if (outs) ra.load(a + tok * r.sa.token, r.sa.token, n, r.reverse);
        rb.load(b + tok * r.sb.token, r.sb.token, n, r.reverse);
        rc.load(c + tok * r.sc.token, r.sc.token, n, r.reverse);
    };
    LinearDecay whole(g * N);
    if (from < to) fetch(from);
    for (int at = from; at < to; at += N) {
        const int n = min(N, to - at);
        const int64_t tok = first + (r.reverse ? span.tokens - at - n : at);
        __syncthreads();
        if (outs) ra.store(&s.a[0][0], DA + 4);
        rb.store(&s.b[0][0], DA + 4);
        rc.store(&s.c[0][0], COLS);
        __syncthreads();
        if (at + N < to) fetch(at + N);  // arrives under this block's work
        if (outs) {  // what lies behind the tokens or before the diagonal is left out
            if (32 * wr < n && wc < 2 * wr + 2) {
                uint64_t p[4][4] = {};
#pragma unroll 2
                for (int x = 0; x < DA; x += 4) {
                    Four bb[4];
#pragma unroll
                    for (int z = 0; z < 4; ++z) bb[z] = four(&s.b[16 * wc + tx + 4 * z][x]);
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const Four aa = four(&s.a[j0 + 8 * y][x]);
#pragma unroll
                        for (int z = 0; z < 4; ++z) p[y][z] = fma2(aa.hi, bb[z].hi, fma2(aa.lo, bb[z].lo, p[y][z]));
                    }
                }
#pragma unroll
                for (int y = 0; y < 4; ++y)
#pragma unroll
                    for (int z = 0; z < 4; ++z) {
                        const int j = j0 + 8 * y, i = 16 * wc + tx + 4 * z;
                        float even, odd;
                        halves(p[y][z], even, odd);
                        s.p[j][i] = i <= j ? r.p_scale * s.pow[j - i] * (even + odd) : 0.f;
                    }
            }
            __syncthreads();
            if (32 * wr < n) {
                uint64_t o[4][2] = {};
                // rows of m by the rows of w, k at a time
                auto times = [&](const float *m, int pitch, const float *w, int upto) {
#pragma unroll 2
                    for (int x = 0; x < upto; x += 4) {
                        float4 mv[4];
#pragma unroll
                        for (int y = 0; y < 4; ++y) mv[y] = *reinterpret_cast<const float4 *>(m + (j0 + 8 * y) * pitch + x);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const Four ww = four(w + (x + k) * COLS + y0);
#pragma unroll
                            for (int y = 0; y < 4; ++y) {
                                const float v = k == 0 ? mv[y].x : k == 1 ? mv[y].y : k == 2 ? mv[y].z : mv[y].w;
                                const uint64_t vv = pair_of(v, v);
                                o[y][0] = fma2(vv, ww.lo, o[y][0]), o[y][1] = fma2(vv, ww.hi, o[y][1]);
                            }
                        }
                    }
                };
                times(&s.a[0][0], DA + 4, &s.x[0][0], DA);
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const float w = r.o_scale * s.pow[j0 + 8 * y + r.e];
                    const uint64_t ww = pair_of(w, w), zero = 0;
                    o[y][0] = fma2(ww, o[y][0], zero), o[y][1] = fma2(ww, o[y][1], zero);
                }
                times(&s.p[0][0], N + 4, &s.c[0][0], 32 * wr + 32);
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const int j = j0 + 8 * y;
                    if (j >= n) continue;
                    const int64_t row = batch * r.T + tok + (r.reverse ? n - 1 - j : j);
                    const int64_t to_at = (row * r.Hv + h) * r.dc + col0 + y0;
                    float v[4];
                    halves(o[y][0], v[0], v[1]), halves(o[y][1], v[2], v[3]);
                    if (sizeof(IO) == 4 || r.out_f32) {
                        *reinterpret_cast<float4 *>(static_cast<float *>(r.out) + to_at) = make_float4(v[0], v[1], v[2], v[3]);
                    } else {
                        IO *out = static_cast<IO *>(r.out) + to_at;
#pragma unroll
                        for (int z = 0; z < 4; ++z) out[z] = from_f<IO>(v[z]);
                    }
                }
            }
        }
        __syncthreads();  // X is read
        uint64_t u[ROWS][2] = {};
#pragma unroll 4
        for (int i = 0; i < n; ++i) {
            const float w = r.s_scale * s.pow[n - i - r.e];
            const uint64_t w2 = pair_of(w, w), zero = 0;
            Four cc = four(&s.c[i][y0]);
            cc.lo = fma2(w2, cc.lo, zero), cc.hi = fma2(w2, cc.hi, zero);
#pragma unroll
            for (int z = 0; z < ROWS; z += 4) {
                const float4 bb = *reinterpret_cast<const float4 *>(&s.b[i][x0 + z]);
                const float bv[4] = {bb.x, bb.y, bb.z, bb.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint64_t b2 = pair_of(bv[k], bv[k]);
                    u[z + k][0] = fma2(b2, cc.lo, u[z + k][0]), u[z + k][1] = fma2(b2, cc.hi, u[z + k][1]);
                }
            }
        }
        const float f = n == N ? whole.next() : LinearDecay(g * n).f;
#pragma unroll
        for (int y = 0; y < ROWS; ++y) {
            float4 &x = *reinterpret_cast<float4 *>(&s.x[x0 + y][y0]);
            float v[4];
            halves(u[y][0], v[0], v[1]), halves(u[y][1], v[2], v[3]);
            x.x = fmaf(f, x.x, v[0]), x.y = fmaf(f, x.y, v[1]);
            x.z = fmaf(f, x.z, v[2]), x.w = fmaf(f, x.w, v[3]);
        }
    }
    __syncthreads();
    if (fin)
        for (int i = tid; i < DA * COLS; i += kThreads) {
            const int x = i / COLS, y = col0 + i % COLS;
            fin[fin_t ? y * DA + x : x * r.dc + y] = s.x[x][i % COLS];
        }
}

template <typename IO, int DA, bool VEC> cudaError_t launch(const LinearRun &r, cudaStream_t st) {
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(k_linear<IO, DA, VEC>, (int)sizeof(Smem<DA>), done);
    if (e != cudaSuccess) return e;
    return launch_behind(k_linear<IO, DA, VEC>, dim3((unsigned)(r.slots * r.Hv), (unsigned)(r.dc / COLS)), kThreads, sizeof(Smem<DA>), st, r);
}
// Whether four values can be read at once
template <typename IO> bool aligned4(const void *x, const gdn_strides &s) {
    return (reinterpret_cast<uintptr_t>(x) & (4 * sizeof(IO) - 1)) == 0 && ((s.batch | s.token | s.head) & 3) == 0;
}
template <typename IO> cudaError_t launch(const LinearRun &r, cudaStream_t st) {
    if (aligned4<IO>(r.a, r.sa) && aligned4<IO>(r.b, r.sb) && aligned4<IO>(r.c, r.sc))
        return r.da == 128 ? launch<IO, 128, true>(r, st) : launch<IO, 64, true>(r, st);
    return r.da == 128 ? launch<IO, 128, false>(r, st) : launch<IO, 64, false>(r, st);
}

// seg[p], the state that segment p adds, becomes the state that enters segment p.  The parts are asked for ahead, four
// values at a time: one by one their way to memory took 18 us for 19 segments of 8 states
__global__ void __launch_bounds__(256) k_join(const __grid_constant__ LinearRun r) {
    constexpr int AHEAD = 16;
    wait_for_previous();
    const int words = r.da * r.dc, seq = blockIdx.x / r.Hv, h = blockIdx.x % r.Hv;
    LinearSpan span;
    if (linear_packed(r)) {
        span = linear_table(r);
        span.per_seg = __shfl_sync(~0u, span.per_seg, seq), span.slot = __shfl_sync(~0u, span.slot, seq), span.segs = __shfl_sync(~0u, span.segs, seq);
    } else {
        span = linear_span(r, seq);
    }
    if (span.segs < 2) return;
    const int64_t unit = (int64_t)seq * r.Hv + h;
    const float g = r.g ? r.g[h] : 0.f;
    const LinearDecay first(g * (float)(span.per_seg * C));
    const int64_t next = (int64_t)r.Hv * words;  // of the next segment
    for (int i = (blockIdx.y * 256 + threadIdx.x) * 4; i < words; i += gridDim.y * 1024) {
        const int x = i / r.dc, y = i % r.dc;
        float4 X = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r.init) {
            const float *init = r.init + unit * words;
            if (r.transposed) X = make_float4(init[y * r.da + x], init[(y + 1) * r.da + x], init[(y + 2) * r.da + x], init[(y + 3) * r.da + x]);
            else X = *reinterpret_cast<const float4 *>(init + i);
        }
        LinearDecay decay = first;
        float *seg = r.seg + ((int64_t)span.slot * r.Hv + h) * words + i;
        for (int p0 = 0; p0 + 1 < span.segs; p0 += AHEAD) {  // all but the last are full
            float4 add[AHEAD];
#pragma unroll
            for (int p = 0; p < AHEAD; ++p)
                if (p0 + p + 1 < span.segs) add[p] = *reinterpret_cast<const float4 *>(seg + (p0 + p) * next);
#pragma unroll
            for (int p = 0; p < AHEAD; ++p) {
                if (p0 + p + 1 >= span.segs) break;
                if (p0 + p > 0) *reinterpret_cast<float4 *>(seg + (p0 + p) * next) = X;
                const float f = decay.next();
                X.x = fmaf(f, X.x, add[p].x), X.y = fmaf(f, X.y, add[p].y);
                X.z = fmaf(f, X.z, add[p].z), X.w = fmaf(f, X.w, add[p].w);
            }
        }
        *reinterpret_cast<float4 *>(seg + (span.segs - 1) * next) = X;
    }
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
    wait_for_previous();
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
    if ((claimed[0] & claimed[1]) == 0xFFFFFFFFu) return;
    for (int i = 0; i < 64 && row0 + i < T; ++i) {
        if (claimed[i >> 5] >> (i & 31) & 1) continue;
        uint4 *to = reinterpret_cast<uint4 *>(x + (int64_t)(row0 + i) * row_bytes);
        for (int64_t j = threadIdx.x; j < row_bytes / 16; j += 256) to[j] = make_uint4(0, 0, 0, 0);
    }
}

}  // namespace

cudaError_t launch_linear_simt(const LinearRun &r, gdn_dtype io, cudaStream_t st) {
    return io == GDN_BF16 ? launch<__nv_bfloat16>(r, st) : launch<float>(r, st);
}

cudaError_t launch_linear_join(const LinearRun &r, cudaStream_t st) {
    const int64_t heads = (int64_t)r.n_seqs * r.Hv;
    const unsigned parts = heads >= 128 ? 4 : 16;  // of a state: the more, the fewer there are
    return launch_behind(k_join, dim3((unsigned)heads, parts), 256, 0, st, r);
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
    return launch_behind(k_unclaimed, dim3((unsigned)((T + 63) / 64)), 256, 0, st, static_cast<unsigned char *>(x), T, row_bytes, cu, n_seqs);
}

}  // namespace gdn
