// linear_api.cu -- the entry points of linear attention over sequences: host-side checks, plan and launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "common.cuh"
#include "gdn.h"
#include "linear.h"
#include "profile.h"

using namespace gdn;

namespace {

constexpr int kSMs = 152;

bool aligned(const void *p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

gdn_status problem_ok(const gdn_linear_problem *p) {
    if (!p) return GDN_ERR_INVALID_ARG;
    if (p->B < 0 || p->T < 0 || p->n_seqs < 0 || p->Hq < 1 || p->Hv < 1 || p->K < 1 || p->V < 1 || p->Hv % p->Hq)
        return GDN_ERR_INVALID_ARG;
    if (p->io_dtype != GDN_F32 && p->io_dtype != GDN_BF16) return GDN_ERR_INVALID_ARG;
    if (p->cu_seqlens ? p->B != 1 : p->n_seqs != p->B) return GDN_ERR_INVALID_ARG;
    if ((p->K != 64 && p->K != 128) || (p->V != 64 && p->V != 128)) return GDN_ERR_UNSUPPORTED;
    if (p->Hv > 16383 || p->B > INT32_MAX || p->T > INT32_MAX - C || p->n_seqs > INT32_MAX / 64) return GDN_ERR_UNSUPPORTED;
    if (p->B * p->T > INT32_MAX || p->n_seqs * p->Hv > INT32_MAX) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

// Into how many segments sequences are cut.  A head of a sequence keeps one SM busy; where these are fewer than the SMs,
// each is cut so that they fill them.  Every token's part in the state is then taken twice, and there are two launches more.
// Measured on the tensor cores, us: 2.2 a chunk and 6 for whole ones, 1.5 + 2.2 a chunk of a segment and 16 for cut ones.
// On the CUDA cores a head is a CTA for every 64 columns of V, of which an SM holds two where K is 64, and one where it is
// 128; a chunk takes 9 us (64 x 64) to 14 (128 x 128), its part in the state some 0.6 of that, the launches and the join as
// much as a chunk.  (2 x 1000 tokens, 8 heads: 64 x 64 146 us whole and 35 cut, 128 x 128 236 and 90; 1 x 200: 35 and 29, 56
// and 31; near the border 4 x 300 of 24 heads, 64 x 64, gain 22 % forward and lose 18 % backward.)
int segments(const gdn_linear_problem *p) {
    const bool f32 = p->io_dtype == GDN_F32;
    const int64_t chains = p->n_seqs * p->Hv, chunks = (p->T + C - 1) / C, room = f32 ? kSMs * 8192 / (p->K * p->V) : kSMs;
    if (chains == 0 || chains > room / 2) return 1;
    const int64_t n = std::min(room / chains, chunks), each = n ? (chunks + n - 1) / n : 0;
    if (n <= 1) return 1;
    const bool cut = f32 ? 1.6 * each + 1 < chunks : 3.7 * each + 16 < 2.2 * chunks + 6;
    return cut ? (int)((chunks + each - 1) / each) : 1;
}

struct Layout {
    size_t seg, partial, bytes;
    int n_seg, seg_chunks, slots;
};
Layout layout(const gdn_linear_problem *p, bool backward) {
    Layout l;
    Carve c;
    l.n_seg = segments(p);
    l.seg_chunks = 0;
    l.slots = (int)(p->n_seqs * l.n_seg);
    // Packed sequences may be of any lengths, which are not known here.  Where one that had all the tokens would take much
    // longer than these shared evenly, what is longer than half of an SM's share is cut.  (13 sequences, one with two
    // fifths of 10007 tokens, 32 heads: 175 us as they are and 158 cut; where none is cut, this costs two launches, some 10 us.)
    // Up to 32 sequences, for the table has a lane for each, and up to four heads an SM.  What that costs beyond, one
    // sequence of 8192 tokens among others of 100, the sequences' number times heads: 19 x 32 181 us and 20 x 32 250, 32 x 8
    // 97 and 33 x 8 229.
    const int64_t chains = p->n_seqs * p->Hv, chunks = (p->T + C - 1) / C;
    if (p->cu_seqlens && l.n_seg == 1 && p->n_seqs > 1 && p->n_seqs <= 32 && chains <= 4 * kSMs) {
        const int64_t even = (chunks * p->Hv + kSMs - 1) / kSMs;
        if (chunks > 2 * even + 16) {
            l.seg_chunks = (int)std::max<int64_t>(4, (even + 1) / 2);
            l.slots = (int)(p->n_seqs + (chunks + p->n_seqs) / l.seg_chunks + 1);
        }
    }
    l.seg = c.take<float>(l.n_seg > 1 || l.seg_chunks ? (size_t)l.slots * p->Hv * p->K * p->V : 0);
    l.partial = c.take<float>(backward && p->Hv != p->Hq ? (size_t)(p->B * p->T * p->Hv * p->K) : 0);
    l.bytes = c.off ? c.off : 256;
    return l;
}

cudaError_t run(LinearRun r, const gdn_linear_problem *p, const Layout &l, unsigned char *ws, cudaStream_t st) {
    r.cu = p->cu_seqlens, r.B = (int)p->B, r.T = (int)p->T, r.Hv = (int)p->Hv, r.n_seqs = (int)p->n_seqs;
    r.drop_chunk = debug_drop_chunk();
    r.n_seg = l.n_seg, r.seg_chunks = l.seg_chunks, r.slots = l.slots, r.seg = reinterpret_cast<float *>(ws + l.seg);
    auto launch = [&](int mode) {
        r.mode = mode;
        ProfScope scope(mode == LIN_SEG ? "linear_segments" : "linear", st);
        return linear_tc_supported(r, p->io_dtype) ? launch_linear_tc(r, st) : launch_linear_simt(r, p->io_dtype, st);
    };
    if (r.n_seg == 1 && !r.seg_chunks) return launch(LIN_WHOLE);
    cudaError_t e = launch(LIN_SEG);
    if (e == cudaSuccess) {
        ProfScope scope("linear_join", st);
        e = launch_linear_join(r, st);
    }
    return e == cudaSuccess ? launch(LIN_MAIN) : e;
}

}  // namespace

extern "C" {

size_t gdn_linear_fwd_workspace_bytes(const gdn_linear_problem *p) {
    return problem_ok(p) == GDN_OK ? layout(p, false).bytes : 0;
}
size_t gdn_linear_bwd_workspace_bytes(const gdn_linear_problem *p) {
    return problem_ok(p) == GDN_OK ? layout(p, true).bytes : 0;
}

gdn_status gdn_linear_fwd(const gdn_linear_problem *p, const void *q, const void *k, const void *v, const float *g,
                          const float *h0, void *o, float *final_state, void *workspace, size_t workspace_bytes,
                          gdn_stream_t stream) {
    const gdn_status s = problem_ok(p);
    if (s != GDN_OK) return s;
    const unsigned elem = p->io_dtype == GDN_BF16 ? 2 : 4;
    const bool tokens = p->B * p->T > 0;
    if (tokens && (!q || !k || !v || !o)) return GDN_ERR_INVALID_ARG;
    if (!aligned(q, elem) || !aligned(k, elem) || !aligned(v, elem) || !aligned(o, 16) || !aligned(g, 4) ||
        !aligned(h0, 16) || !aligned(final_state, 16) || !aligned(p->cu_seqlens, 4))
        return GDN_ERR_INVALID_ARG;
    const Layout l = layout(p, false);
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < l.bytes) return GDN_ERR_WORKSPACE;
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (p->cu_seqlens && tokens &&
        launch_unclaimed(o, (int)p->T, p->Hv * p->V * elem, p->cu_seqlens, (int)p->n_seqs, st) != cudaSuccess)
        return GDN_ERR_CUDA;
    if (p->n_seqs == 0) return GDN_OK;
    const int G = (int)(p->Hv / p->Hq);
    LinearRun r = {};
    r.a = q, r.b = k, r.c = v, r.sa = p->q, r.sb = p->k, r.sc = p->v, r.ga = r.gb = G, r.gc = 1;
    r.da = (int)p->K, r.dc = (int)p->V, r.g = g, r.init = h0, r.fin = final_state;
    r.out = o, r.p_scale = r.o_scale = p->scale, r.s_scale = 1.f, r.e = 1;
    return run(r, p, l, ws, st) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status gdn_linear_bwd(const gdn_linear_problem *p, const void *q, const void *k, const void *v, const float *g,
                          const float *h0, const void *d_o, const float *dht, void *dq, void *dk, void *dv, float *dh0,
                          void *workspace, size_t workspace_bytes, gdn_stream_t stream) {
    const gdn_status s = problem_ok(p);
    if (s != GDN_OK) return s;
    const unsigned elem = p->io_dtype == GDN_BF16 ? 2 : 4;
    const bool tokens = p->B * p->T > 0;
    if (tokens && (!q || !k || !v || !d_o)) return GDN_ERR_INVALID_ARG;
    if (!aligned(q, elem) || !aligned(k, elem) || !aligned(v, elem) || !aligned(d_o, elem) || !aligned(dq, 16) ||
        !aligned(dk, 16) || !aligned(dv, 16) || !aligned(g, 4) || !aligned(h0, 16) || !aligned(dht, 16) ||
        !aligned(dh0, 16) || !aligned(p->cu_seqlens, 4))
        return GDN_ERR_INVALID_ARG;
    const Layout l = layout(p, true);
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < l.bytes) return GDN_ERR_WORKSPACE;
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const int G = (int)(p->Hv / p->Hq);
    const int64_t rows = p->B * p->T;
    float *partial = reinterpret_cast<float *>(ws + l.partial);

    LinearRun x = {};
    x.g = g, x.p_scale = p->scale;
    // dq and dk of a query head are sums over its value heads: fp32 parts of each, then their sum
    auto grouped = [&](LinearRun r, void *out) {
        r.out = G > 1 ? static_cast<void *>(partial) : out, r.out_f32 = G > 1;
        if (p->n_seqs > 0) {
            const cudaError_t e = run(r, p, l, ws, st);
            if (e != cudaSuccess) return e;
        }
        return G > 1 ? launch_group_sum(partial, out, rows, (int)p->Hq, G, (int)p->K, p->io_dtype, st) : cudaSuccess;
    };
    if (dq && tokens) {
        LinearRun r = x;
        r.a = d_o, r.b = v, r.c = k, r.sa = p->d_o, r.sb = p->v, r.sc = p->k, r.ga = r.gb = 1, r.gc = G;
        r.da = (int)p->V, r.dc = (int)p->K, r.init = h0, r.transposed = true, r.s_scale = 1.f, r.o_scale = p->scale, r.e = 1;
        if (grouped(r, dq) != cudaSuccess) return GDN_ERR_CUDA;
    }
    x.reverse = true, x.init = dht, x.s_scale = p->scale, x.o_scale = 1.f, x.e = 0;
    if (dk && tokens) {
        LinearRun r = x;
        r.a = v, r.b = d_o, r.c = q, r.sa = p->v, r.sb = p->d_o, r.sc = p->q, r.ga = r.gb = 1, r.gc = G;
        r.da = (int)p->V, r.dc = (int)p->K, r.transposed = true;
        if (grouped(r, dk) != cudaSuccess) return GDN_ERR_CUDA;
    }
    if (((dv && tokens) || dh0) && p->n_seqs > 0) {
        LinearRun r = x;
        r.a = k, r.b = q, r.c = d_o, r.sa = p->k, r.sb = p->q, r.sc = p->d_o, r.ga = r.gb = G, r.gc = 1;
        r.da = (int)p->K, r.dc = (int)p->V, r.fin = dh0, r.out = dv;
        if (run(r, p, l, ws, st) != cudaSuccess) return GDN_ERR_CUDA;
    }
    if (p->cu_seqlens && tokens) {
        const struct {
            void *x;
            int64_t row;
        } outs[3] = {{dq, p->Hq * p->K * elem}, {dk, p->Hq * p->K * elem}, {dv, p->Hv * p->V * elem}};
        for (const auto &y : outs)
            if (y.x && launch_unclaimed(y.x, (int)p->T, y.row, p->cu_seqlens, (int)p->n_seqs, st) != cudaSuccess)
                return GDN_ERR_CUDA;
    }
    return GDN_OK;
}

}  // extern "C"
