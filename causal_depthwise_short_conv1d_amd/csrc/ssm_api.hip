// C ABI of the selective state space scan and of the group norm: host checks
// and launches.  Nothing here touches device memory or synchronises.
#include <math.h>
#include <stdint.h>

#include "sconv.h"
#include "sconv_host.h"
#include "ssm_params.h"

using namespace sconv;

namespace {

const uint16_t *u16(const void *p) { return static_cast<const uint16_t *>(p); }

Span span_of_out(const SsmParams &p, int64_t B, int64_t T) {
    return span_of(p.out, {B, T, p.H, p.P}, {p.os.sb, p.os.st, p.os.sh, p.os.sd});
}
Span span_of_state(const SsmParams &p) {
    return span_of(p.state, {p.num_lines, p.H, p.P, p.N}, {p.s_sl, p.s_sh, p.s_sp, p.s_sn}, 4);
}
Span span_of_weight(const SsmParams &p, const SsmWeight &w, int64_t n) {
    return span_of(w.p, {p.H, p.P, n}, {w.sh, w.sd, w.sn}, 4);
}
// Whether what is written at `w` overlaps a tensor that the kernels read.
bool overlaps_input(const SsmParams &p, int64_t B, int64_t T, const Span &w) {
    const auto rows = [&](const void *a, const GdrTensor &t, int64_t heads, int64_t n, int64_t elem) {
        return overlap(w, span_of(a, {B, T, heads, n}, {t.sb, t.st, t.sh, t.sd}, elem));
    };
    return rows(p.x, p.xs, p.H, p.P, 2) || rows(p.z, p.zs, p.H, p.P, 2) || rows(p.B, p.bs, p.G, p.N, 2) ||
           rows(p.C, p.cs, p.G, p.N, 2) || rows(p.dt, p.ds, p.H, p.P, p.dt_fp32 ? 4 : 2) ||
           overlap(w, span_of_weight(p, p.A, p.N)) || overlap(w, span_of_weight(p, p.D, 1)) ||
           overlap(w, span_of_weight(p, p.bias, 1));
}

// The layouts that a call's tensors are in.
struct Layout {
    bool head;      // one step size and decay a head
    bool vec;       // B, C, the state and decays of channels in groups of four elements
};

// The checks that prefill and decode share; B and T are the sizes of the
// sequence and token dimensions.
int check_ssm(const SsmParams &p, int64_t B, int64_t T, Layout *layout) {
    if (p.H < 1 || p.G < 1 || p.H % p.G || p.P < 1 || p.N < 1 || p.N > kSsmMaxState) return SCONV_ERR_SHAPE;
    if (!p.x || !p.B || !p.C || !p.dt || !p.A.p || !p.out) return SCONV_ERR_NULL;
    for (const GdrTensor *t : {&p.xs, &p.bs, &p.cs, &p.zs, &p.os, &p.ds})
        if (negative({t->sb, t->st, t->sh, t->sd})) return SCONV_ERR_STRIDE;
    for (const SsmWeight *w : {&p.A, &p.D, &p.bias})
        if (negative({w->sh, w->sd, w->sn})) return SCONV_ERR_STRIDE;
    if (negative({p.s_sl, p.s_sh, p.s_sp, p.s_sn, p.ci_sb, p.ci_ss, p.osi_sb, p.osi_ss})) return SCONV_ERR_STRIDE;
    if (!(p.dt_min <= p.dt_max)) return SCONV_ERR_ARG;             // (NaN too)
    if (p.state) {
        if (p.num_lines < 1 || (!p.ci && p.num_lines < p.batch)) return SCONV_ERR_SHAPE;
        if (!non_overlapping({p.num_lines, p.H, p.P, p.N}, {p.s_sl, p.s_sh, p.s_sp, p.s_sn})) return SCONV_ERR_STRIDE;
    }
    if (!non_overlapping({B, T, p.H, p.P}, {p.os.sb, p.os.st, p.os.sh, p.os.sd})) return SCONV_ERR_STRIDE;
    if (!aligned(p.x, 2) || !aligned(p.B, 2) || !aligned(p.C, 2) || !aligned(p.z, 2) || !aligned(p.out, 2) ||
        !aligned(p.dt, p.dt_fp32 ? 4 : 2) || !aligned(p.A.p, 4) || !aligned(p.D.p, 4) || !aligned(p.bias.p, 4) ||
        !aligned(p.state, 4) || !aligned(p.ci, 4) || !aligned(p.qsl, 4) || !aligned(p.accepted, 4) || !aligned(p.osi, 4))
        return SCONV_ERR_ALIGN;
    const Span so = span_of_out(p, B, T), ss = span_of_state(p);
    if (overlap(so, ss) || overlaps_input(p, B, T, so) || overlaps_input(p, B, T, ss)) return SCONV_ERR_ALIAS;

    layout->head = (p.P == 1 || (p.A.sd == 0 && p.ds.sd == 0 && (!p.bias.p || p.bias.sd == 0))) && (p.N == 1 || p.A.sn == 0);
    layout->vec = p.N % 4 == 0 && p.bs.sd == 1 && p.cs.sd == 1 &&
                  groups_of(p.B, 4, 2, {B, T, p.G}, {p.bs.sb, p.bs.st, p.bs.sh}) &&
                  groups_of(p.C, 4, 2, {B, T, p.G}, {p.cs.sb, p.cs.st, p.cs.sh}) &&
                  (!p.state || (p.s_sn == 1 && groups_of(p.state, 4, 4, {p.num_lines, p.H, p.P}, {p.s_sl, p.s_sh, p.s_sp}))) &&
                  (layout->head || (p.A.sn == 1 && groups_of(p.A.p, 4, 4, {p.H, p.P}, {p.A.sh, p.A.sd})));
    // the recurrent kernel gives a wave to 8 channels at least, a workgroup to 4 waves
    const int64_t heads = int64_t(p.batch) * p.H;
    if (heads > kMaxThreads / 64 || heads * ((int64_t(p.P) + 7) / 8) > kMaxThreads / 64 - 4) return SCONV_ERR_SHAPE;
    return SCONV_OK;
}

int check_workspace(const SsmParams &p, int64_t T, const void *workspace, int64_t bytes, int64_t need) {
    if (!aligned(workspace, 16)) return SCONV_ERR_ALIGN;
    if (bytes < need) return SCONV_ERR_SHAPE;
    const Span sw = span_of(workspace, {need}, {1}, 1);
    return overlap(sw, span_of_out(p, 1, T)) || overlap(sw, span_of_state(p)) || overlaps_input(p, 1, T, sw) ? SCONV_ERR_ALIAS
                                                                                                          : SCONV_OK;
}

}  // namespace

namespace sconv {

SsmPlan ssm_plan(int64_t T, int64_t batch, int32_t H, int32_t G, int32_t P, int32_t N, bool workspace) {
    SsmPlan plan = {};
    plan.nt = N <= 32 ? 1 : (N <= 64 ? 2 : 4);
    plan.pair = P > 32;
    const int64_t units = int64_t(H / G) * (plan.pair ? (int64_t(P) + 63) / 64 : 1);       // of a group
    const int64_t waves = units * (plan.pair ? 2 : 1);
    plan.groups = G * ((waves + kSsmWaves - 1) / kSsmWaves);
    // A place takes a CU a workgroup.  Segments walk all of a sequence at once, but walk it twice, and the first walk and the
    // pass behind it cost some 25 us: with at most 64 workgroups, from ten chunks a sequence on.  us with / without, 128 heads of
    // 64 x 128 (32 workgroups a sequence): 256 tokens 45 / 32, 512 53 / 54, 640 54 / 65, 1024 60 / 98; 2 sequences of 1024 85 / 100,
    // 3 108 / 102, 3 of 4096 343 / 357, 5 of 1024 189 / 129; 64 heads: 256 tokens 40 / 31, 512 45 / 52.
    const int64_t chunks = T / kSsmChunk + batch, mean = T / kSsmChunk / batch;
    if (workspace && batch * plan.groups <= 64 && mean >= 10) {
        int64_t seg = (chunks * plan.groups + 255) / 256;
        if (seg < 2) seg = 2;
        if (seg < mean) {
            plan.seg = int32_t(seg);
            plan.slots = T / (kSsmChunk * seg) + batch + 1;
            plan.bytes = plan.slots * G * waves * (plan.nt * 1024 + 1) * 4;
        }
    }
    return plan;
}

SsmChannelPlan ssm_channel_plan(int64_t T, int64_t batch, int32_t G, int32_t P, int32_t N, bool workspace) {
    SsmChannelPlan plan = {};
    plan.np = N <= 16 ? 16 : (N <= 32 ? 32 : 64);
    plan.groups = G * ((int64_t(P) + kSsmChannels - 1) / kSsmChannels);
    // Four workgroups a CU hide what each waits for.  us with segments / without, 8192 channels (32 workgroups a sequence): 128
    // tokens 46 / 65, 1024 100 / 467, 4 sequences of 512 154 / 242, 8 265 / 243, 12 438 / 307; 64 tokens 44 / 37.
    const int64_t mean = T / batch;
    if (workspace && batch * plan.groups <= 128 && mean >= 128) {
        int64_t seg = (T * plan.groups + 1023) / 1024;
        seg = (seg < 32 ? 32 : seg) + kSsmTokens - 1;
        seg -= seg % kSsmTokens;
        if (seg < mean) {
            plan.seg = int32_t(seg);
            plan.slots = T / seg + batch + 1;
            plan.bytes = plan.slots * plan.groups * (kSsmChannels / 64) * (plan.np + 2) * 64 * 4;
        }
    }
    return plan;
}

}  // namespace sconv

extern "C" {

int ssm_fwd_varlen_packed(const void *words) { return call_words(ssm_fwd_varlen, words); }
int ssm_update_packed(const void *words) { return call_words(ssm_update, words); }

int ssm_fwd_varlen(const void *x, int64_t x_stride_tok, int64_t x_stride_head, int64_t x_stride_dim,
                   const void *dt, int64_t dt_stride_tok, int64_t dt_stride_head, int64_t dt_stride_dim, int32_t dt_fp32,
                   const float *a, int64_t a_stride_head, int64_t a_stride_dim, int64_t a_stride_state,
                   const void *b, int64_t b_stride_tok, int64_t b_stride_group, int64_t b_stride_state,
                   const void *c, int64_t c_stride_tok, int64_t c_stride_group, int64_t c_stride_state,
                   const float *d, int64_t d_stride_head, int64_t d_stride_dim,
                   const void *z, int64_t z_stride_tok, int64_t z_stride_head, int64_t z_stride_dim,
                   const float *dt_bias, int64_t dtb_stride_head, int64_t dtb_stride_dim,
                   int32_t dt_softplus, float dt_min, float dt_max,
                   float *state, int64_t s_stride_line, int64_t s_stride_head, int64_t s_stride_dim,
                   int64_t s_stride_state, int64_t num_cache_lines,
                   const int32_t *cache_indices, const uint8_t *has_initial_state, const int32_t *query_start_loc,
                   int32_t batch, int64_t total_tokens, int32_t num_heads, int32_t num_groups, int32_t head_dim,
                   int32_t state_dim, int32_t pad_slot_id,
                   void *out, int64_t o_stride_tok, int64_t o_stride_head, int64_t o_stride_dim,
                   void *workspace, int64_t workspace_bytes, hipStream_t stream) {
    // token offsets of whole chunks stay within 31 bits
    if (batch < 0 || total_tokens < 0 || total_tokens > INT32_MAX - 256 || num_cache_lines < 0) return SCONV_ERR_SHAPE;
    if (batch == 0 || total_tokens == 0) return SCONV_OK;
    if (!query_start_loc || (has_initial_state && !state)) return SCONV_ERR_NULL;
    SsmParams p = {};
    p.x = u16(x);
    p.B = u16(b);
    p.C = u16(c);
    p.z = u16(z);
    p.out = static_cast<uint16_t *>(out);
    p.xs = {0, x_stride_tok, x_stride_head, x_stride_dim};
    p.bs = {0, b_stride_tok, b_stride_group, b_stride_state};
    p.cs = {0, c_stride_tok, c_stride_group, c_stride_state};
    p.zs = {0, z_stride_tok, z_stride_head, z_stride_dim};
    p.os = {0, o_stride_tok, o_stride_head, o_stride_dim};
    p.dt = dt;
    p.ds = {0, dt_stride_tok, dt_stride_head, dt_stride_dim};
    p.dt_fp32 = dt_fp32 != 0;
    p.softplus = dt_softplus != 0;
    p.dt_min = dt_min;
    p.dt_max = dt_max;
    p.A = {a, a_stride_head, a_stride_dim, a_stride_state};
    p.D = {d, d_stride_head, d_stride_dim, 0};
    p.bias = {dt_bias, dtb_stride_head, dtb_stride_dim, 0};
    p.state = state;
    p.s_sl = s_stride_line;
    p.s_sh = s_stride_head;
    p.s_sp = s_stride_dim;
    p.s_sn = s_stride_state;
    p.num_lines = num_cache_lines;
    p.batch = batch;
    p.H = num_heads;
    p.G = num_groups;
    p.P = head_dim;
    p.N = state_dim;
    p.pad_slot_id = pad_slot_id;
    p.qsl = query_start_loc;
    p.has_init = has_initial_state;
    p.total_T = total_tokens;
    p.ci = cache_indices;
    p.ci_sb = 1;
    p.ci_steps = 1;
    Layout layout = {};
    const int rc = check_ssm(p, 1, total_tokens, &layout);
    if (rc != SCONV_OK) return rc;
    p.per_group = p.H / p.G;
    const int64_t T = total_tokens;
    // A chunk takes as long as six tokens, one after the other, and where a token's rows do not fill the chip as long as ten or
    // twelve.  us a token at a time / in chunks, heads of 64 x 128: 128 heads, 64 sequences of 6 tokens 188 / 191, 8 tokens
    // 234 / 195; 16 sequences of 6 tokens 48 / 50, of 8 57 / 50; 4 sequences of 10 tokens 17.1 / 18.2, of 12 20.0 / 18.2; one of 1
    // token 4.8 / 15.3, 10 tokens 13.0 / 15.6, 16 18.5 / 15.7; 8 heads, 64 sequences of 10 tokens 17.0 / 19.8, of 16 24.6 / 19.5.
    const int64_t few = int64_t(batch) * p.H <= 512 ? 10 : 6;
    if (layout.head && p.N <= kSsmMaxChunkN && T > few * batch) {
        const SsmPlan plan = ssm_plan(T, batch, p.H, p.G, p.P, p.N, workspace != nullptr);
        const int64_t places = (plan.seg ? plan.slots : batch) + 7;
        if (places <= kMaxThreads / (64 * kSsmWaves) / plan.groups && plan.groups <= INT32_MAX) {
            if (plan.bytes) {
                const int rc = check_workspace(p, T, workspace, workspace_bytes, plan.bytes);
                if (rc != SCONV_OK) return rc;
            }
            // rows longer than what is read of them, a chunk's within the 31 bits of a descriptor's offsets
            const auto rows = [&](const void *a, const GdrTensor &t, int32_t heads, int32_t n) {
                return !a || (t.sd == 1 && n % 8 == 0 && n <= t.st && t.st < (1 << 23) && groups_of(a, 8, 2, {T, heads}, {t.st, t.sh}));
            };
            const bool vec = rows(p.x, p.xs, p.H, p.P) && rows(p.z, p.zs, p.H, p.P) && rows(p.out, p.os, p.H, p.P) &&
                             rows(p.B, p.bs, p.G, p.N) && rows(p.C, p.cs, p.G, p.N);
            const bool svec = p.state && p.N % 4 == 0 && p.s_sn == 1 &&
                              groups_of(p.state, 4, 4, {p.num_lines, p.H, p.P}, {p.s_sl, p.s_sh, p.s_sp});
            return launch_status(launch_ssm_chunk(p, vec, svec, plan, workspace, stream));
        }
    }
    // (64 sequences of 4 tokens of 8192 channels: 38 us a token at a time, 68 with a thread a channel; one of 64 tokens 50 and 38)
    if (!layout.head && p.H == p.G && p.N <= kSsmMaxChannelN && T > 8 * int64_t(batch)) {
        const SsmChannelPlan plan = ssm_channel_plan(T, batch, p.G, p.P, p.N, workspace != nullptr);
        const int64_t places = plan.seg ? plan.slots : batch;
        if (places <= kMaxThreads / kSsmChannels / plan.groups &&
            int64_t(batch) * plan.groups <= kMaxThreads / kSsmChannels / plan.np) {
            if (plan.bytes) {
                const int rc = check_workspace(p, T, workspace, workspace_bytes, plan.bytes);
                if (rc != SCONV_OK) return rc;
            }
            const auto rows = [&](const void *a, const GdrTensor &t) {
                return !a || (t.sd == 1 && t.st >= p.P && t.st < (1 << 23));
            };
            const bool all = rows(p.x, p.xs) && rows(p.z, p.zs) && rows(p.out, p.os) && rows(p.dt, p.ds);
            return launch_status(launch_ssm_channel(p, all, plan, workspace, stream));
        }
    }
    return launch_status(launch_ssm_recurrent(p, layout.head, layout.vec, stream));
}

int64_t ssm_fwd_workspace_bytes(int32_t batch, int64_t total_tokens, int32_t num_heads, int32_t num_groups, int32_t head_dim,
                                int32_t state_dim, int32_t per_channel) {
    if (batch < 1 || total_tokens < 1 || num_heads < 1 || num_groups < 1 || num_heads % num_groups || head_dim < 1 ||
        state_dim < 1 || total_tokens > INT32_MAX - 256)
        return 0;
    if (per_channel)
        return num_heads != num_groups || state_dim > kSsmMaxChannelN
                   ? 0 : ssm_channel_plan(total_tokens, batch, num_groups, head_dim, state_dim, true).bytes;
    if (state_dim > kSsmMaxChunkN) return 0;
    return ssm_plan(total_tokens, batch, num_heads, num_groups, head_dim, state_dim, true).bytes;
}

int ssm_update(const void *x, int64_t x_stride_seq, int64_t x_stride_tok, int64_t x_stride_head, int64_t x_stride_dim,
               const void *dt, int64_t dt_stride_seq, int64_t dt_stride_tok, int64_t dt_stride_head, int64_t dt_stride_dim,
               int32_t dt_fp32,
               const float *a, int64_t a_stride_head, int64_t a_stride_dim, int64_t a_stride_state,
               const void *b, int64_t b_stride_seq, int64_t b_stride_tok, int64_t b_stride_group, int64_t b_stride_state,
               const void *c, int64_t c_stride_seq, int64_t c_stride_tok, int64_t c_stride_group, int64_t c_stride_state,
               const float *d, int64_t d_stride_head, int64_t d_stride_dim,
               const void *z, int64_t z_stride_seq, int64_t z_stride_tok, int64_t z_stride_head, int64_t z_stride_dim,
               const float *dt_bias, int64_t dtb_stride_head, int64_t dtb_stride_dim,
               int32_t dt_softplus, float dt_min, float dt_max,
               float *state, int64_t s_stride_line, int64_t s_stride_head, int64_t s_stride_dim, int64_t s_stride_state,
               int64_t num_cache_lines,
               const int32_t *cache_indices, int64_t ci_stride_seq, int64_t ci_stride_step, int32_t ci_steps,
               const int32_t *num_accepted_tokens,
               const int32_t *output_state_indices, int64_t osi_stride_seq, int64_t osi_stride_step,
               int32_t batch, int32_t seqlen, int32_t num_heads, int32_t num_groups, int32_t head_dim, int32_t state_dim,
               int32_t pad_slot_id,
               void *out, int64_t o_stride_seq, int64_t o_stride_tok, int64_t o_stride_head, int64_t o_stride_dim,
               hipStream_t stream) {
    if (batch < 0 || seqlen < 0 || num_cache_lines < 0) return SCONV_ERR_SHAPE;
    if (batch == 0 || seqlen == 0) return SCONV_OK;
    if (!state || (num_accepted_tokens && !cache_indices)) return SCONV_ERR_NULL;
    if (cache_indices && ci_steps < 1) return SCONV_ERR_SHAPE;
    SsmParams p = {};
    p.x = u16(x);
    p.B = u16(b);
    p.C = u16(c);
    p.z = u16(z);
    p.out = static_cast<uint16_t *>(out);
    p.xs = {x_stride_seq, x_stride_tok, x_stride_head, x_stride_dim};
    p.bs = {b_stride_seq, b_stride_tok, b_stride_group, b_stride_state};
    p.cs = {c_stride_seq, c_stride_tok, c_stride_group, c_stride_state};
    p.zs = {z_stride_seq, z_stride_tok, z_stride_head, z_stride_dim};
    p.os = {o_stride_seq, o_stride_tok, o_stride_head, o_stride_dim};
    p.dt = dt;
    p.ds = {dt_stride_seq, dt_stride_tok, dt_stride_head, dt_stride_dim};
    p.dt_fp32 = dt_fp32 != 0;
    p.softplus = dt_softplus != 0;
    p.dt_min = dt_min;
    p.dt_max = dt_max;
    p.A = {a, a_stride_head, a_stride_dim, a_stride_state};
    p.D = {d, d_stride_head, d_stride_dim, 0};
    p.bias = {dt_bias, dtb_stride_head, dtb_stride_dim, 0};
    p.state = state;
    p.s_sl = s_stride_line;
    p.s_sh = s_stride_head;
    p.s_sp = s_stride_dim;
    p.s_sn = s_stride_state;
    p.num_lines = num_cache_lines;
    p.batch = batch;
    p.seqlen = seqlen;
    p.H = num_heads;
    p.G = num_groups;
    p.P = head_dim;
    p.N = state_dim;
    p.pad_slot_id = pad_slot_id;
    p.ci = cache_indices;
    p.ci_sb = ci_stride_seq;
    p.ci_ss = ci_stride_step;
    p.ci_steps = ci_steps;
    p.accepted = num_accepted_tokens;
    p.osi = output_state_indices;
    p.osi_sb = osi_stride_seq;
    p.osi_ss = osi_stride_step;
    Layout layout = {};
    const int rc = check_ssm(p, batch, seqlen, &layout);
    if (rc != SCONV_OK) return rc;
    p.per_group = p.H / p.G;
    return launch_status(launch_ssm_recurrent(p, layout.head, layout.vec, stream));
}

int sconv_group_norm(const void *x, int64_t x_stride_row, int64_t x_stride_group, int64_t x_stride_dim,
                     const void *z, int64_t z_stride_row, int64_t z_stride_group, int64_t z_stride_dim,
                     const void *weight, int64_t w_stride_group, const void *bias, int64_t b_stride_group,
                     int32_t weights_fp32, int64_t rows, int32_t num_groups, int32_t group_size, int32_t norm,
                     int32_t activation, int32_t gate_first, float eps,
                     void *out, int64_t o_stride_row, int64_t o_stride_group, int64_t o_stride_dim, hipStream_t stream) {
    if (rows < 0 || num_groups < 0 || group_size < 0) return SCONV_ERR_SHAPE;
    if (rows == 0 || num_groups == 0 || group_size == 0) return SCONV_OK;
    if (rows > kMaxThreads / 8 / num_groups) return SCONV_ERR_SHAPE;       // (8 threads a group at least)
    if (!x || !out) return SCONV_ERR_NULL;
    if (negative({x_stride_row, x_stride_group, x_stride_dim, z_stride_row, z_stride_group, z_stride_dim, w_stride_group,
                  b_stride_group}))
        return SCONV_ERR_STRIDE;
    if (!non_overlapping({rows, num_groups, group_size}, {o_stride_row, o_stride_group, o_stride_dim}))
        return SCONV_ERR_STRIDE;
    if ((norm != SCONV_NORM_RMS && norm != SCONV_NORM_LAYER) ||
        (activation != SCONV_ACT_NONE && activation != SCONV_ACT_SILU && activation != SCONV_ACT_SIGMOID) ||
        (gate_first && !z) || !(eps >= 0.0f) || !isfinite(eps))
        return SCONV_ERR_ARG;
    const int wb = weights_fp32 ? 4 : 2;
    if (!aligned(x, 2) || !aligned(z, 2) || !aligned(out, 2) || !aligned(weight, wb) || !aligned(bias, wb))
        return SCONV_ERR_ALIGN;
    const Span so = span_of(out, {rows, num_groups, group_size}, {o_stride_row, o_stride_group, o_stride_dim});
    const auto aliases = [&](const void *a, int64_t sr, int64_t sg, int64_t sc) {      // exactly out's elements are fine
        if (a == out && (rows == 1 || sr == o_stride_row) && (num_groups == 1 || sg == o_stride_group) &&
            (group_size == 1 || sc == o_stride_dim))
            return false;
        return overlap(so, span_of(a, {rows, num_groups, group_size}, {sr, sg, sc}));
    };
    if (aliases(x, x_stride_row, x_stride_group, x_stride_dim) || aliases(z, z_stride_row, z_stride_group, z_stride_dim) ||
        overlap(so, span_of(weight, {num_groups, group_size}, {w_stride_group, 1}, wb)) ||
        overlap(so, span_of(bias, {num_groups, group_size}, {b_stride_group, 1}, wb)))
        return SCONV_ERR_ALIAS;
    NormParams p = {};
    p.x = u16(x);
    p.z = u16(z);
    p.out = static_cast<uint16_t *>(out);
    p.x_sr = x_stride_row; p.x_sg = x_stride_group; p.x_sc = x_stride_dim;
    p.z_sr = z_stride_row; p.z_sg = z_stride_group; p.z_sc = z_stride_dim;
    p.o_sr = o_stride_row; p.o_sg = o_stride_group; p.o_sc = o_stride_dim;
    p.w = weight;
    p.b = bias;
    p.w_sg = w_stride_group;
    p.b_sg = b_stride_group;
    p.w_fp32 = weights_fp32 != 0;
    p.rows = rows;
    p.groups = num_groups;
    p.size = group_size;
    p.layer = norm == SCONV_NORM_LAYER;
    p.act = activation;
    p.gate_first = gate_first != 0;
    p.eps = eps;
    const auto eight = [&](const void *a, int64_t sr, int64_t sg, int64_t sc) {
        return !a || (sc == 1 && groups_of(a, 8, 2, {rows, num_groups}, {sr, sg}));
    };
    const auto weights = [&](const void *a, int64_t sg) { return !a || groups_of(a, 16 / wb, wb, {num_groups}, {sg}); };
    const bool vec = group_size % 8 == 0 && group_size <= kNormMaxVec && eight(x, x_stride_row, x_stride_group, x_stride_dim) &&
                     eight(z, z_stride_row, z_stride_group, z_stride_dim) &&
                     eight(out, o_stride_row, o_stride_group, o_stride_dim) && weights(weight, w_stride_group) &&
                     weights(bias, b_stride_group);
    const int64_t threads = vec ? norm_threads(group_size) : kNormBlock;
    if (rows > (kMaxThreads - kNormBlock) / threads / num_groups) return SCONV_ERR_SHAPE;
    return launch_status(launch_group_norm(p, vec, stream));
}

}  // extern "C"
