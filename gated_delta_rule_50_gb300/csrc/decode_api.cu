// decode_api.cu -- the decoding entry points of include/gdn.h: host-side checks and launches.
#include <cuda_runtime.h>

#include <cstdint>

#include "common.cuh"
#include "decode.h"
#include "gdn.h"
#include "profile.h"

using namespace gdn;

namespace {

bool aligned(const void *p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

gdn_status launched(cudaError_t e) { return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA; }

gdn_status decode_args(const gdn_decode_problem *p, const void *q, const void *k, const void *v, const float *g,
                       const float *beta, const float *state, void *o, DecodeArgs *a) {
    if (!p) return GDN_ERR_INVALID_ARG;
    if (p->B < 0 || p->T < 0 || p->Hq < 1 || p->Hv < 1 || p->K < 1 || p->V < 1 || p->Hv % p->Hq)
        return GDN_ERR_INVALID_ARG;
    if (p->io_dtype != GDN_F32 && p->io_dtype != GDN_BF16) return GDN_ERR_INVALID_ARG;
    if ((p->K != 64 && p->K != 128) || (p->V != 64 && p->V != 128)) return GDN_ERR_UNSUPPORTED;
    if (p->B > INT32_MAX || p->T > INT32_MAX || p->n_seqs > INT32_MAX || p->n_steps > INT32_MAX || p->Hv > 16383)
        return GDN_ERR_UNSUPPORTED;
    if (p->n_seqs < 0 || p->n_steps < 0 || p->n_slots < 0) return GDN_ERR_INVALID_ARG;
    if (p->cu_seqlens ? (p->B != 1 || p->token_indices) : p->n_seqs != p->B) return GDN_ERR_INVALID_ARG;
    if (p->n_seqs * p->Hv > INT32_MAX / 2) return GDN_ERR_UNSUPPORTED;
    if (p->n_slots > 1 && p->slot_stride < p->Hv * p->K * p->V) return GDN_ERR_INVALID_ARG;
    if (p->slot_stride < 0 || p->slot_stride % 4) return GDN_ERR_INVALID_ARG;
    if (!p->state_indices && p->n_seqs > p->n_slots) return GDN_ERR_INVALID_ARG;
    const bool none = p->n_seqs == 0;  // nothing will be read
    const bool tokens = p->B > 0 && p->T > 0;
    const unsigned elem = p->io_dtype == GDN_BF16 ? 2 : 4;
    if (!none && tokens && (!k || !v || !g || !beta)) return GDN_ERR_INVALID_ARG;
    if (!none && p->n_slots > 0 && !state) return GDN_ERR_INVALID_ARG;
    if (!aligned(q, elem) || !aligned(k, elem) || !aligned(v, elem) || !aligned(o, 16) || !aligned(g, 4) ||
        !aligned(beta, 4) || !aligned(state, 16) || !aligned(p->state_indices, 4) || !aligned(p->cu_seqlens, 4) ||
        !aligned(p->token_indices, 4))
        return GDN_ERR_INVALID_ARG;
    a->q = q, a->k = k, a->v = v, a->g = g, a->beta = beta;
    a->sq = p->q, a->sk = p->k, a->sv = p->v, a->sg = p->g, a->sb = p->beta;
    a->state = const_cast<float *>(state);
    a->out_state = nullptr;
    a->o = o;
    a->state_indices = p->state_indices, a->cu = p->cu_seqlens, a->token_indices = p->token_indices;
    a->parents = nullptr;
    a->n_slots = p->n_slots, a->slot_stride = p->slot_stride;
    a->T = (int)p->T, a->Hq = (int)p->Hq, a->Hv = (int)p->Hv, a->G = (int)(p->Hv / p->Hq), a->V = (int)p->V;
    a->n_seqs = (int)p->n_seqs, a->n_steps = (int)p->n_steps;
    a->scale = p->scale;
    return GDN_OK;
}

gdn_status beam_args(const gdn_beam_problem *p, BeamArgs *a) {
    if (!p || p->B < 0 || p->W < 1 || p->vocab < 1 || p->n < 1) return GDN_ERR_INVALID_ARG;
    if (p->logits_dtype != GDN_F32 && p->logits_dtype != GDN_BF16) return GDN_ERR_INVALID_ARG;
    if (p->W > GDN_BEAM_MAX || p->n > GDN_BEAM_MAX || p->vocab > GDN_BEAM_VOCAB_MAX || p->B > (1 << 20))
        return GDN_ERR_UNSUPPORTED;
    a->logits_batch = p->logits_batch, a->logits_beam = p->logits_beam;
    a->mask_batch = p->mask_batch, a->mask_beam = p->mask_beam;
    a->B = (int)p->B, a->W = (int)p->W, a->vocab = (int)p->vocab, a->n = (int)p->n;
    a->chunk = beam_chunk(p->B * p->W, p->vocab, p->n, p->logits_dtype);
    a->n_chunks = (int)((p->vocab + 7 + a->chunk - 1) / a->chunk);
    if (p->B * p->W * a->n_chunks > INT32_MAX) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

size_t beam_layout(const BeamArgs &a, size_t *stats, size_t *keys) {
    Carve c;
    const size_t units = (size_t)a.B * a.W * a.n_chunks;
    *stats = c.take<float2>(units);
    *keys = c.take<uint64_t>(units * a.n);
    return c.off;
}

}  // namespace

extern "C" {

gdn_status gdn_recurrent(const gdn_decode_problem *p, const void *q, const void *k, const void *v, const float *g,
                         const float *beta, float *state, float *out_state, void *o, gdn_stream_t stream) {
    DecodeArgs a;
    const gdn_status s = decode_args(p, q, k, v, g, beta, state, o, &a);
    if (s != GDN_OK) return s;
    const bool out = (p->token_indices ? p->n_seqs * p->n_steps : p->B * p->T) > 0;
    if (out && p->B * p->T > 0 && !q != !o) return GDN_ERR_INVALID_ARG;
    if (!aligned(out_state, 16)) return GDN_ERR_INVALID_ARG;
    if (out_state && p->n_slots > 0) {
        const uintptr_t in0 = reinterpret_cast<uintptr_t>(state), out0 = reinterpret_cast<uintptr_t>(out_state);
        const uintptr_t slot = (uintptr_t)(p->Hv * p->K * p->V * 4);
        const uintptr_t in1 = in0 + (uintptr_t)(p->n_slots - 1) * (uintptr_t)p->slot_stride * 4 + slot;
        if (out0 < in1 && in0 < out0 + (uintptr_t)p->n_seqs * slot) return GDN_ERR_INVALID_ARG;
    }
    a.out_state = out_state;
    if (p->n_seqs == 0) return GDN_OK;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    ProfScope scope("recurrent", st);
    return launched(launch_recurrent(a, (int)p->K, p->io_dtype, st));
}

gdn_status gdn_tree(const gdn_decode_problem *p, const void *q, const void *k, const void *v, const float *g,
                    const float *beta, const int32_t *parents, const float *state, void *o, gdn_stream_t stream) {
    DecodeArgs a;
    const gdn_status s = decode_args(p, q, k, v, g, beta, state, o, &a);
    if (s != GDN_OK) return s;
    if (p->cu_seqlens || p->token_indices) return GDN_ERR_INVALID_ARG;
    if (p->T > GDN_TREE_MAX) return GDN_ERR_UNSUPPORTED;
    if (p->n_seqs == 0 || p->T == 0) return GDN_OK;
    if (!q || !o || !parents || !aligned(parents, 4)) return GDN_ERR_INVALID_ARG;
    a.parents = parents;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    ProfScope scope("tree", st);
    return launched(launch_tree(a, (int)p->K, p->io_dtype, st));
}

size_t gdn_beam_search_workspace_bytes(const gdn_beam_problem *p) {
    BeamArgs a;
    size_t stats, keys;
    if (beam_args(p, &a) != GDN_OK) return 0;
    const size_t n = beam_layout(a, &stats, &keys);
    return n ? n : 256;
}

gdn_status gdn_beam_search(const gdn_beam_problem *p, const void *logits, const float *scores, const uint8_t *finished,
                           const uint8_t *mask, float *out_scores, int32_t *out_tokens, int32_t *out_parents,
                           void *workspace, size_t workspace_bytes, gdn_stream_t stream) {
    BeamArgs a;
    const gdn_status s = beam_args(p, &a);
    if (s != GDN_OK) return s;
    if (p->B == 0) return GDN_OK;
    if (!logits || !scores || !out_scores || !out_tokens || !out_parents) return GDN_ERR_INVALID_ARG;
    if (!aligned(logits, p->logits_dtype == GDN_BF16 ? 2 : 4) || !aligned(scores, 4) || !aligned(out_scores, 4) ||
        !aligned(out_tokens, 4) || !aligned(out_parents, 4))
        return GDN_ERR_INVALID_ARG;
    size_t stats, keys;
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < beam_layout(a, &stats, &keys))
        return GDN_ERR_WORKSPACE;
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    a.logits = logits, a.scores = scores, a.finished = finished, a.mask = mask;
    a.stats = reinterpret_cast<float2 *>(ws + stats);
    a.keys = reinterpret_cast<uint64_t *>(ws + keys);
    a.out_scores = out_scores, a.out_tokens = out_tokens, a.out_parents = out_parents;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    ProfScope scope("beam_search", st);
    return launched(launch_beam(a, p->logits_dtype, st));
}

gdn_status gdn_reorder_states(const gdn_state_view *views, int64_t n_views, int64_t n_slots, int64_t B, int64_t W,
                              const int32_t *parents, const int32_t *state_indices, gdn_stream_t stream) {
    if (n_views < 0 || (n_views > 0 && !views) || n_slots < 0 || B < 0 || W < 1) return GDN_ERR_INVALID_ARG;
    if (W > GDN_BEAM_MAX || B > 65535) return GDN_ERR_UNSUPPORTED;
    if (!state_indices && B * W > n_slots) return GDN_ERR_INVALID_ARG;
    for (int64_t i = 0; i < n_views; ++i) {
        if (views[i].slot_bytes < 0 || views[i].slot_stride < 0) return GDN_ERR_INVALID_ARG;
        if (n_slots > 1 && views[i].slot_stride < views[i].slot_bytes) return GDN_ERR_INVALID_ARG;
        if (n_slots > 0 && views[i].slot_bytes > 0 && !views[i].data) return GDN_ERR_INVALID_ARG;
    }
    if (B == 0 || n_slots == 0 || n_views == 0) return GDN_OK;
    if (!parents || !aligned(parents, 4) || !aligned(state_indices, 4)) return GDN_ERR_INVALID_ARG;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    ProfScope scope("reorder_states", st);
    ReorderArgs a;
    a.n_slots = n_slots, a.B = (int)B, a.W = (int)W, a.parents = parents, a.state_indices = state_indices;
    a.n_views = 0;
    for (int64_t i = 0; i < n_views; ++i) {
        if (views[i].slot_bytes > 0) {
            a.view[a.n_views].data = static_cast<unsigned char *>(views[i].data);
            a.view[a.n_views].stride = views[i].slot_stride;
            a.view[a.n_views].bytes = views[i].slot_bytes;
            ++a.n_views;
        }
        if (a.n_views == kMaxViews || (i + 1 == n_views && a.n_views > 0)) {
            const cudaError_t e = launch_reorder(a, st);
            if (e != cudaSuccess) return GDN_ERR_CUDA;
            a.n_views = 0;
        }
    }
    return GDN_OK;
}

}  // extern "C"
