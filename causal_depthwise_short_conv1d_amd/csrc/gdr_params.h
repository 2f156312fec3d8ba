// Kernel parameters of the gated delta rule and of draft verification, shared
// by the host checks and the kernels.
#pragma once

#include <stdint.h>
#include <hip/hip_runtime_api.h>

namespace sconv {

// One strided (sequence, token, head, channel) tensor.
struct GdrTensor {
    int64_t sb, st, sh, sd;    // element strides; sb is 0 for packed tokens
};

struct GdrParams {
    const uint16_t *q, *k, *v;
    uint16_t *out;
    GdrTensor qs, ks, vs, os;
    const void *gate, *beta;   // fp32, or bf16 when raw
    GdrTensor gs, bs;          // (sd unused)
    const float *a_log, *dt_bias;   // [Hv] when raw
    float *state;              // [lines][Hv][Dv][Dk] or null
    int64_t s_sl, s_sh, s_sv, s_sk;
    int64_t num_lines;
    int32_t batch;
    int32_t Hk, Hv, Dk, Dv;
    int32_t group;             // value heads per key head
    int32_t raw, l2norm;
    int32_t pad_slot_id;
    float scale;
    // packed prefill (qsl) or fixed-length entries (seqlen)
    const int32_t *qsl;
    const uint8_t *has_init;
    int64_t total_T;
    int32_t seqlen;
    // decode: the line that an entry reads, and those that its steps write
    const int32_t *ci;
    int64_t ci_sb, ci_ss;
    int32_t ci_steps;
    const int32_t *accepted;
    const int32_t *osi;
    int64_t osi_sb, osi_ss;
};

struct VerifyParams {
    const int32_t *draft_tokens;    // [num_drafts]
    const int32_t *start;           // [batch + 1]
    const float *p;                 // [num_drafts + batch][vocab]
    int64_t p_sr;
    const float *q;                 // [num_drafts][vocab] or null
    int64_t q_sr;
    const float *u_acc;             // [num_drafts]
    const float *u_smp;             // [batch]
    int32_t batch, num_drafts, vocab, max_drafts;
    int32_t slice, slices;          // vocabulary entries per workgroup, workgroups per request
    double *sums_ws;                // [batch][slices][2]
    int32_t *count_ws;              // [batch]: standing drafts
    int32_t *tokens;                // [batch][max_drafts + 1]
    int64_t t_sr;
    int32_t *num_accepted;          // [batch]
};

// Launchers: each enqueues its kernels and returns hipGetLastError().
// `vec`: unit channel strides, and every base and stride keeps four elements
// together (8-byte bf16, 16-byte fp32 accesses).
hipError_t launch_gdr_recurrent(const GdrParams &p, bool vec, hipStream_t s);
// `vec`: unit channel strides of q and k, every base and stride a multiple of 8
// elements; `svec`: the state's rows in 16-byte pieces.  Dk at most kGdrMaxChunkK.
// With a workspace of gdr_workspace_bytes(), 16-byte aligned: two kernels, the
// tiles of all chunks first; without (vec only): one kernel.
int64_t gdr_workspace_bytes(int64_t T, int64_t batch, int32_t Hv);
hipError_t launch_gdr_chunk(const GdrParams &p, bool vec, bool svec, void *workspace, hipStream_t s);
hipError_t launch_verify_drafts(const VerifyParams &p, hipStream_t s);

// Slots for the 64-token chunks of any packing of T tokens into `batch` sequences.
inline int64_t gdr_slots(int64_t T, int64_t batch) { return T / 64 + batch + 2; }

// Workgroups of a kernel that walks sequences, `groups` a head: batch * Hk rounded up to the 8 XCDs.
inline int64_t gdr_walk_grid(int64_t batch, int64_t Hk, int64_t Hv, int64_t groups) {
    return (batch * Hk + 7) / 8 * 8 * (Hv / Hk) * groups;
}
constexpr int64_t kMaxThreads = (int64_t(1) << 32) - 1;     // of a launch
constexpr int kGdrThreads = 512;                               // a workgroup of the chunked kernels

// Whether a call's heads are so few, and its sequences long enough, that walking prepared chunks in two kernels is
// faster than one kernel: a chunk takes a walk 2.0 to 2.2 us and the one kernel 7.6, but twice the workgroups and a launch
// more gain nothing where CUs are full or there is one chunk.  Measured with 128 x 128 heads and sequences of one length, us
// with two kernels / one:
//   64 tokens a sequence: 32 heads 16.0 / 14.0;  65: 16 heads 16.7 / 20.8
//   128: 16 heads 16.9 / 21.2, 64 heads 18.9 / 22.1, 96 heads 27 / 22, 128 heads 30 / 23
//   256: 64 heads 25 / 36, 96 heads 37.8 / 37.3, 128 heads 40.4 / 38.0;  320: 96 heads 43.5 / 45.4, 128 heads 44.9 / 45.7
//   2048: 32 heads 84 / 245, 128 heads 188 / 247, 160 heads 257 / 251, 192 heads 277 / 264
// The host knows only the mean length.  One long sequence among short ones counts as so many long ones and takes one kernel:
// 4195 tokens beside four sequences of one token, 32 heads, 509 us, where they take 164 alone.
inline bool gdr_few_heads(int64_t T, int64_t batch, int64_t Hv, int64_t Dv) {
    const int64_t halves = batch * Hv * ((Dv + 63) / 64);
    return (halves <= 128 && T > 64 * batch) || (halves <= 256 && T > 256 * batch);
}

constexpr int kVfMaxSlice = 8192;      // vocabulary entries of a slice, a multiple of 1024

constexpr int kGdrMaxHeadK = 256;      // key channels a head of the recurrent kernel
constexpr int kGdrMaxChunkK = 128;     // ... of the chunked kernel

}  // namespace sconv
