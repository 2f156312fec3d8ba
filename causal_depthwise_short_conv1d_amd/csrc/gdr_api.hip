// C ABI of the gated delta rule and of draft verification: host checks and
// launches.  Nothing here touches device memory or synchronises.
#include <math.h>
#include <stdint.h>

#include "gdr_params.h"
#include "sconv.h"
#include "sconv_host.h"

using namespace sconv;

namespace {

Span span_of_out(const GdrParams &p, int64_t B, int64_t T) {
    return span_of(p.out, {B, T, p.Hv, p.Dv}, {p.os.sb, p.os.st, p.os.sh, p.os.sd});
}
Span span_of_state(const GdrParams &p) {
    return span_of(p.state, {p.num_lines, p.Hv, p.Dv, p.Dk}, {p.s_sl, p.s_sh, p.s_sv, p.s_sk}, 4);
}
// Whether what is written at `w` overlaps a tensor that the kernels read.
bool overlaps_input(const GdrParams &p, int64_t B, int64_t T, const Span &w) {
    const int gate_bytes = p.raw ? 2 : 4;
    const Span in[] = {
        span_of(p.q, {B, T, p.Hk, p.Dk}, {p.qs.sb, p.qs.st, p.qs.sh, p.qs.sd}),
        span_of(p.k, {B, T, p.Hk, p.Dk}, {p.ks.sb, p.ks.st, p.ks.sh, p.ks.sd}),
        span_of(p.v, {B, T, p.Hv, p.Dv}, {p.vs.sb, p.vs.st, p.vs.sh, p.vs.sd}),
        span_of(p.gate, {B, T, p.Hv}, {p.gs.sb, p.gs.st, p.gs.sh}, gate_bytes),
        span_of(p.beta, {B, T, p.Hv}, {p.bs.sb, p.bs.st, p.bs.sh}, gate_bytes),
        span_of(p.a_log, {p.Hv}, {1}, 4),
        span_of(p.dt_bias, {p.Hv}, {1}, 4),
    };
    for (const Span &s : in)
        if (overlap(w, s)) return true;
    return false;
}

// The checks that prefill and decode share; B and T are the sizes of the
// sequence and token dimensions.
int check_gdr(const GdrParams &p, int64_t B, int64_t T, bool *vec) {
    if (p.Hk < 1 || p.Hv < 1 || p.Hv % p.Hk || p.Dk < 1 || p.Dv < 1 || p.Dk > kGdrMaxHeadK)
        return SCONV_ERR_SHAPE;
    if (!p.q || !p.k || !p.v || !p.gate || !p.beta || !p.out) return SCONV_ERR_NULL;
    if (!p.a_log != !p.dt_bias) return SCONV_ERR_NULL;
    for (const GdrTensor *t : {&p.qs, &p.ks, &p.vs, &p.os, &p.gs, &p.bs})
        if (negative({t->sb, t->st, t->sh, t->sd})) return SCONV_ERR_STRIDE;
    if (negative({p.s_sl, p.s_sh, p.s_sv, p.s_sk, p.ci_sb, p.ci_ss, p.osi_sb, p.osi_ss}))
        return SCONV_ERR_STRIDE;
    if (!isfinite(p.scale)) return SCONV_ERR_ARG;
    if (p.state) {
        if (p.num_lines < 1 || (!p.ci && p.num_lines < p.batch)) return SCONV_ERR_SHAPE;
        if (!non_overlapping({p.num_lines, p.Hv, p.Dv, p.Dk}, {p.s_sl, p.s_sh, p.s_sv, p.s_sk}))
            return SCONV_ERR_STRIDE;
    }
    if (!non_overlapping({B, T, p.Hv, p.Dv}, {p.os.sb, p.os.st, p.os.sh, p.os.sd}))
        return SCONV_ERR_STRIDE;
    const int gate_bytes = p.raw ? 2 : 4;
    if (!aligned(p.q, 2) || !aligned(p.k, 2) || !aligned(p.v, 2) || !aligned(p.out, 2) ||
        !aligned(p.gate, gate_bytes) || !aligned(p.beta, gate_bytes) || !aligned(p.a_log, 4) ||
        !aligned(p.dt_bias, 4) || !aligned(p.state, 4) || !aligned(p.ci, 4) || !aligned(p.qsl, 4) ||
        !aligned(p.accepted, 4) || !aligned(p.osi, 4))
        return SCONV_ERR_ALIGN;

    const Span so = span_of_out(p, B, T), ss = span_of_state(p);
    if (overlap(so, ss) || overlaps_input(p, B, T, so) || overlaps_input(p, B, T, ss)) return SCONV_ERR_ALIAS;

    // four elements at a time: 8-byte rows of q and k, 16-byte state rows
    *vec = p.Dk % 4 == 0 && p.qs.sd == 1 && p.ks.sd == 1 &&
           groups_of(p.q, 4, 2, {B, T, p.Hk}, {p.qs.sb, p.qs.st, p.qs.sh}) &&
           groups_of(p.k, 4, 2, {B, T, p.Hk}, {p.ks.sb, p.ks.st, p.ks.sh}) &&
           (!p.state || (p.s_sk == 1 && groups_of(p.state, 4, 4, {p.num_lines, p.Hv, p.Dv},
                                                  {p.s_sl, p.s_sh, p.s_sv})));
    // the recurrent kernel gives a wave to 8 state rows at least
    const int64_t heads = int64_t(p.batch) * p.Hv;
    if (heads > kMaxThreads / 64 || heads * ((int64_t(p.Dv) + 7) / 8) > kMaxThreads / 64 - 4) return SCONV_ERR_SHAPE;
    return SCONV_OK;
}

// Vocabulary entries a workgroup of the summing kernel takes: some 2048
// workgroups (8 a CU), 1024 to 8192 entries each; the picking kernel holds a
// whole slice in registers.
int32_t verify_slice(int64_t batch, int64_t vocab) {
    int64_t s = (batch * vocab + 2047) / 2048;
    s = (s + 255) / 256 * 256;
    return int32_t(s < 1024 ? 1024 : (s > kVfMaxSlice ? kVfMaxSlice : s));
}

}  // namespace

extern "C" {

int gdr_fwd_varlen_packed(const void *words) { return call_words(gdr_fwd_varlen, words); }
int gdr_update_packed(const void *words) { return call_words(gdr_update, words); }

int gdr_fwd_varlen(const void *q, int64_t q_stride_tok, int64_t q_stride_head, int64_t q_stride_dim,
                   const void *k, int64_t k_stride_tok, int64_t k_stride_head, int64_t k_stride_dim,
                   const void *v, int64_t v_stride_tok, int64_t v_stride_head, int64_t v_stride_dim,
                   const void *gate, int64_t g_stride_tok, int64_t g_stride_head,
                   const void *beta, int64_t b_stride_tok, int64_t b_stride_head,
                   const float *a_log, const float *dt_bias,
                   float *state, int64_t s_stride_line, int64_t s_stride_head, int64_t s_stride_v,
                   int64_t s_stride_k, int64_t num_cache_lines,
                   const int32_t *cache_indices, const uint8_t *has_initial_state,
                   const int32_t *query_start_loc, int32_t batch, int64_t total_tokens,
                   int32_t num_k_heads, int32_t num_v_heads, int32_t head_dim_k, int32_t head_dim_v,
                   float scale, int32_t qk_l2norm, int32_t pad_slot_id,
                   void *out, int64_t o_stride_tok, int64_t o_stride_head, int64_t o_stride_dim,
                   void *workspace, int64_t workspace_bytes, hipStream_t stream) {
    // token offsets of whole chunks stay within 31 bits
    if (batch < 0 || total_tokens < 0 || total_tokens > INT32_MAX - 256 || num_cache_lines < 0)
        return SCONV_ERR_SHAPE;
    if (batch == 0 || total_tokens == 0) return SCONV_OK;
    if (!query_start_loc || (has_initial_state && !state)) return SCONV_ERR_NULL;
    GdrParams p = {};
    p.q = static_cast<const uint16_t *>(q);
    p.k = static_cast<const uint16_t *>(k);
    p.v = static_cast<const uint16_t *>(v);
    p.out = static_cast<uint16_t *>(out);
    p.qs = {0, q_stride_tok, q_stride_head, q_stride_dim};
    p.ks = {0, k_stride_tok, k_stride_head, k_stride_dim};
    p.vs = {0, v_stride_tok, v_stride_head, v_stride_dim};
    p.os = {0, o_stride_tok, o_stride_head, o_stride_dim};
    p.gate = gate;
    p.beta = beta;
    p.gs = {0, g_stride_tok, g_stride_head, 0};
    p.bs = {0, b_stride_tok, b_stride_head, 0};
    p.a_log = a_log;
    p.dt_bias = dt_bias;
    p.raw = a_log != nullptr;
    p.state = state;
    p.s_sl = s_stride_line;
    p.s_sh = s_stride_head;
    p.s_sv = s_stride_v;
    p.s_sk = s_stride_k;
    p.num_lines = num_cache_lines;
    p.batch = batch;
    p.Hk = num_k_heads;
    p.Hv = num_v_heads;
    p.Dk = head_dim_k;
    p.Dv = head_dim_v;
    p.scale = scale;
    p.l2norm = qk_l2norm != 0;
    p.pad_slot_id = pad_slot_id;
    p.qsl = query_start_loc;
    p.has_init = has_initial_state;
    p.total_T = total_tokens;
    p.ci = cache_indices;
    p.ci_sb = 1;
    p.ci_steps = 1;
    bool vec = false;
    const int rc = check_gdr(p, 1, total_tokens, &vec);
    if (rc != SCONV_OK) return rc;
    p.group = p.Hv / p.Hk;
    const int64_t T = total_tokens;
    if (p.Dk <= kGdrMaxChunkK) {
        // 16-byte pieces of q, k and v, 8-byte ones of out; rows longer than a head, a chunk's within the 31 bits of a
        // descriptor's offsets
        const auto rows = [&](const void *a, const GdrTensor &t, int32_t heads, int32_t d, int n) {
            return d % n == 0 && t.sd == 1 && d <= t.st && t.st < (1 << 23) && groups_of(a, n, 2, {T, heads}, {t.st, t.sh});
        };
        const bool vec8 = rows(q, p.qs, p.Hk, p.Dk, 8) && rows(k, p.ks, p.Hk, p.Dk, 8) && rows(v, p.vs, p.Hv, p.Dv, 8) &&
                          rows(out, p.os, p.Hv, p.Dv, 4);
        const bool svec = state && p.Dk % 4 == 0 && p.s_sk == 1 &&
                          groups_of(state, 4, 4, {p.num_lines, p.Hv, p.Dv}, {p.s_sl, p.s_sh, p.s_sv});
        const int64_t need = gdr_fwd_workspace_bytes(batch, T, p.Hk, p.Hv, p.Dk, p.Dv, vec8);
        if (workspace && need > 0) {
            if (!aligned(workspace, 16)) return SCONV_ERR_ALIGN;
            if (workspace_bytes < need) return SCONV_ERR_SHAPE;
            const Span sw = span_of(workspace, {need}, {1}, 1);
            if (overlap(sw, span_of_out(p, 1, T)) || overlap(sw, span_of_state(p)) || overlaps_input(p, 1, T, sw))
                return SCONV_ERR_ALIAS;
            return launch_status(launch_gdr_chunk(p, vec8, svec, workspace, stream));
        }
        if (vec8 && gdr_walk_grid(batch, p.Hk, p.Hv, (int64_t(p.Dv) + 127) / 128) <= kMaxThreads / kGdrThreads)
            return launch_status(launch_gdr_chunk(p, vec8, svec, nullptr, stream));
    }
    return launch_status(launch_gdr_recurrent(p, vec, stream));
}

int64_t gdr_fwd_workspace_bytes(int32_t batch, int64_t total_tokens, int32_t num_k_heads, int32_t num_v_heads,
                                int32_t head_dim_k, int32_t head_dim_v, int32_t vector_layout) {
    if (batch < 1 || total_tokens < 1 || num_k_heads < 1 || num_v_heads < 1 || head_dim_k < 1 || head_dim_v < 1 ||
        head_dim_k > kGdrMaxChunkK || num_v_heads % num_k_heads || int64_t(batch) * num_v_heads > kMaxThreads / 64)
        return 0;
    // many heads fill the chip by themselves; short sequences in layouts by elements go a token at a time, which takes
    // some 2 us a token where a chunk's workspace is 19 KB a head
    if (vector_layout ? !gdr_few_heads(total_tokens, batch, num_v_heads, head_dim_v) : total_tokens <= 32 * int64_t(batch))
        return 0;
    const int64_t slots = gdr_slots(total_tokens, batch);
    if (slots * num_k_heads > kMaxThreads / kGdrThreads ||
        gdr_walk_grid(batch, num_k_heads, num_v_heads, (int64_t(head_dim_v) + 31) / 32) > kMaxThreads / kGdrThreads)
        return 0;
    return gdr_workspace_bytes(total_tokens, batch, num_v_heads);
}

int gdr_update(const void *q, int64_t q_stride_seq, int64_t q_stride_tok, int64_t q_stride_head,
               int64_t q_stride_dim,
               const void *k, int64_t k_stride_seq, int64_t k_stride_tok, int64_t k_stride_head,
               int64_t k_stride_dim,
               const void *v, int64_t v_stride_seq, int64_t v_stride_tok, int64_t v_stride_head,
               int64_t v_stride_dim,
               const void *gate, int64_t g_stride_seq, int64_t g_stride_tok, int64_t g_stride_head,
               const void *beta, int64_t b_stride_seq, int64_t b_stride_tok, int64_t b_stride_head,
               const float *a_log, const float *dt_bias,
               float *state, int64_t s_stride_line, int64_t s_stride_head, int64_t s_stride_v,
               int64_t s_stride_k, int64_t num_cache_lines,
               const int32_t *cache_indices, int64_t ci_stride_seq, int64_t ci_stride_step,
               int32_t ci_steps, const int32_t *num_accepted_tokens,
               const int32_t *output_state_indices, int64_t osi_stride_seq, int64_t osi_stride_step,
               int32_t batch, int32_t seqlen,
               int32_t num_k_heads, int32_t num_v_heads, int32_t head_dim_k, int32_t head_dim_v,
               float scale, int32_t qk_l2norm, int32_t pad_slot_id,
               void *out, int64_t o_stride_seq, int64_t o_stride_tok, int64_t o_stride_head,
               int64_t o_stride_dim, hipStream_t stream) {
    if (batch < 0 || seqlen < 0 || num_cache_lines < 0) return SCONV_ERR_SHAPE;
    if (batch == 0 || seqlen == 0) return SCONV_OK;
    if (!state || (num_accepted_tokens && !cache_indices)) return SCONV_ERR_NULL;
    if (cache_indices && ci_steps < 1) return SCONV_ERR_SHAPE;
    GdrParams p = {};
    p.q = static_cast<const uint16_t *>(q);
    p.k = static_cast<const uint16_t *>(k);
    p.v = static_cast<const uint16_t *>(v);
    p.out = static_cast<uint16_t *>(out);
    p.qs = {q_stride_seq, q_stride_tok, q_stride_head, q_stride_dim};
    p.ks = {k_stride_seq, k_stride_tok, k_stride_head, k_stride_dim};
    p.vs = {v_stride_seq, v_stride_tok, v_stride_head, v_stride_dim};
    p.os = {o_stride_seq, o_stride_tok, o_stride_head, o_stride_dim};
    p.gate = gate;
    p.beta = beta;
    p.gs = {g_stride_seq, g_stride_tok, g_stride_head, 0};
    p.bs = {b_stride_seq, b_stride_tok, b_stride_head, 0};
    p.a_log = a_log;
    p.dt_bias = dt_bias;
    p.raw = a_log != nullptr;
    p.state = state;
    p.s_sl = s_stride_line;
    p.s_sh = s_stride_head;
    p.s_sv = s_stride_v;
    p.s_sk = s_stride_k;
    p.num_lines = num_cache_lines;
    p.batch = batch;
    p.seqlen = seqlen;
    p.Hk = num_k_heads;
    p.Hv = num_v_heads;
    p.Dk = head_dim_k;
    p.Dv = head_dim_v;
    p.scale = scale;
    p.l2norm = qk_l2norm != 0;
    p.pad_slot_id = pad_slot_id;
    p.ci = cache_indices;
    p.ci_sb = ci_stride_seq;
    p.ci_ss = ci_stride_step;
    p.ci_steps = ci_steps;
    p.accepted = num_accepted_tokens;
    p.osi = output_state_indices;
    p.osi_sb = osi_stride_seq;
    p.osi_ss = osi_stride_step;
    bool vec = false;
    const int rc = check_gdr(p, batch, seqlen, &vec);
    if (rc != SCONV_OK) return rc;
    p.group = p.Hv / p.Hk;
    return launch_status(launch_gdr_recurrent(p, vec, stream));
}

int64_t sconv_verify_workspace_bytes(int32_t batch, int32_t vocab) {
    if (batch <= 0 || vocab <= 0) return 0;
    const int64_t slice = verify_slice(batch, vocab);
    return int64_t(batch) * ((vocab + slice - 1) / slice) * 16 + (int64_t(batch) + 1) / 2 * 8;
}

int sconv_verify_drafts(const int32_t *draft_tokens, const int32_t *draft_start_loc,
                        const float *target_probs, int64_t p_stride_row,
                        const float *draft_probs, int64_t q_stride_row,
                        const float *accept_uniform, const float *sample_uniform,
                        int32_t batch, int32_t num_drafts, int32_t vocab, int32_t max_drafts,
                        int32_t *tokens, int64_t t_stride_row, int32_t *num_accepted_tokens,
                        void *workspace, int64_t workspace_bytes, hipStream_t stream) {
    if (batch < 0 || num_drafts < 0 || vocab < 0 || max_drafts < 0 || max_drafts == INT32_MAX)
        return SCONV_ERR_SHAPE;
    if (batch == 0) return SCONV_OK;
    if (vocab == 0 || vocab > (1 << 30)) return SCONV_ERR_SHAPE;
    if (!draft_start_loc || !target_probs || !sample_uniform || !tokens || !num_accepted_tokens ||
        !workspace || (num_drafts > 0 && (!draft_tokens || !accept_uniform)))
        return SCONV_ERR_NULL;
    if (p_stride_row < 0 || q_stride_row < 0) return SCONV_ERR_STRIDE;
    if (!non_overlapping({batch, int64_t(max_drafts) + 1}, {t_stride_row, 1})) return SCONV_ERR_STRIDE;
    for (const void *a : {static_cast<const void *>(draft_tokens), static_cast<const void *>(draft_start_loc),
                          static_cast<const void *>(target_probs), static_cast<const void *>(draft_probs),
                          static_cast<const void *>(accept_uniform), static_cast<const void *>(sample_uniform),
                          static_cast<const void *>(tokens), static_cast<const void *>(num_accepted_tokens)})
        if (!aligned(a, 4)) return SCONV_ERR_ALIGN;
    if (!aligned(workspace, 8)) return SCONV_ERR_ALIGN;
    const int64_t need = sconv_verify_workspace_bytes(batch, vocab);
    if (workspace_bytes < need) return SCONV_ERR_SHAPE;

    const int64_t rows = int64_t(num_drafts) + batch;
    const Span written[] = {
        span_of(tokens, {batch, int64_t(max_drafts) + 1}, {t_stride_row, 1}, 4),
        span_of(num_accepted_tokens, {batch}, {1}, 4),
        span_of(workspace, {need}, {1}, 1),
    };
    const Span read[] = {
        span_of(draft_tokens, {num_drafts}, {1}, 4),
        span_of(draft_start_loc, {int64_t(batch) + 1}, {1}, 4),
        span_of(target_probs, {rows, vocab}, {p_stride_row, 1}, 4),
        span_of(draft_probs, {num_drafts, vocab}, {q_stride_row, 1}, 4),
        span_of(accept_uniform, {num_drafts}, {1}, 4),
        span_of(sample_uniform, {batch}, {1}, 4),
    };
    for (int i = 0; i < 3; ++i) {
        for (const Span &r : read)
            if (overlap(written[i], r)) return SCONV_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (overlap(written[i], written[j])) return SCONV_ERR_ALIAS;
    }

    VerifyParams p = {};
    p.draft_tokens = draft_tokens;
    p.start = draft_start_loc;
    p.p = target_probs;
    p.p_sr = p_stride_row;
    p.q = draft_probs;
    p.q_sr = q_stride_row;
    p.u_acc = accept_uniform;
    p.u_smp = sample_uniform;
    p.batch = batch;
    p.num_drafts = num_drafts;
    p.vocab = vocab;
    p.max_drafts = max_drafts;
    p.slice = verify_slice(batch, vocab);
    p.slices = int32_t((int64_t(vocab) + p.slice - 1) / p.slice);
    p.sums_ws = static_cast<double *>(workspace);
    p.count_ws = reinterpret_cast<int32_t *>(p.sums_ws + int64_t(batch) * p.slices * 2);
    p.tokens = tokens;
    p.t_sr = t_stride_row;
    p.num_accepted = num_accepted_tokens;
    if (int64_t(p.slices) * batch > kMaxThreads / 256) return SCONV_ERR_SHAPE;
    return launch_status(launch_verify_drafts(p, stream));
}

}  // extern "C"
