// Kernel parameters of the selective state space scan and of the group norm,
// shared by the host checks and the kernels.
#pragma once

#include <stdint.h>
#include <hip/hip_runtime_api.h>

#include "gdr_params.h"                // GdrTensor, kMaxThreads

namespace sconv {

// One tensor of the layer's weights: (head, channel, state), fp32.
struct SsmWeight {
    const float *p;                    // or null
    int64_t sh, sd, sn;
};

struct SsmParams {
    const uint16_t *x, *B, *C, *z;     // z may be null
    uint16_t *out;
    GdrTensor xs, bs, cs, zs, os;      // of B and C: (sequence, token, group, state)
    const void *dt;                    // fp32 or bf16
    GdrTensor ds;
    int32_t dt_fp32, softplus;
    float dt_min, dt_max;
    SsmWeight A, D, bias;              // D and bias may be null
    float *state;                      // [lines][H][P][N] or null
    int64_t s_sl, s_sh, s_sp, s_sn;
    int64_t num_lines;
    int32_t batch;
    int32_t H, G, P, N;                // heads, groups, channels a head, states a channel
    int32_t per_group;                 // heads of a group
    int32_t pad_slot_id;
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

struct NormParams {
    const uint16_t *x, *z;             // z may be null
    uint16_t *out;
    int64_t x_sr, x_sg, x_sc, z_sr, z_sg, z_sc, o_sr, o_sg, o_sc;    // (row, group, channel)
    const void *w, *b;                 // fp32 or bf16, or null
    int64_t w_sg, b_sg;                // (group) strides; channels are contiguous
    int32_t w_fp32;                    // of both
    int64_t rows;
    int32_t groups, size;
    int32_t layer;                     // the mean is taken out first
    int32_t act, gate_first;
    float eps;
};

constexpr int kSsmMaxState = 256;      // states a channel
constexpr int kNormBlock = 256;        // threads of a workgroup of the norm
constexpr int kNormMaxVec = 64 * kNormBlock;     // channels of a group that a workgroup holds in registers
// Threads that share a group of `size` channels, eight channels each at a time.
inline int norm_threads(int32_t size) {
    if (size > 2048) return kNormBlock;
    int n = 8;
    while (n < 64 && n * 8 < size) n *= 2;
    return n;
}

constexpr int kSsmChunk = 64;          // tokens of a chunk
constexpr int kSsmWaves = 8;           // a workgroup of the chunked kernel, fewer in small calls
constexpr int kSsmCus = 256;
constexpr int kSsmMaxChunkN = 128;     // states a channel of the chunked kernel

// How the chunked kernel takes a call: its shapes, and whether sequences are cut into segments of `seg` chunks (0: they
// are not) that are walked at once.
struct SsmPlan {
    int32_t nt;                        // 32-state tiles: 1, 2 or 4
    bool pair;                         // two waves a block of 64 channels of a head, else one for up to 32
    int32_t seg;
    int64_t slots;                     // of segments
    int64_t groups;                    // workgroups of a place (a sequence or slot)
    int64_t bytes;                     // workspace
};
SsmPlan ssm_plan(int64_t T, int64_t batch, int32_t H, int32_t G, int32_t P, int32_t N, bool workspace);

constexpr int kSsmTokens = 8;          // of a block of the channel kernel
constexpr int kSsmChannels = 256;      // of its workgroups
constexpr int kSsmMaxChannelN = 64;    // states a channel that it takes: up to 32 in registers, more partly in scratch memory

// How the channel kernel takes a call: states rounded up, and whether sequences are cut into segments of `seg` tokens.
struct SsmChannelPlan {
    int32_t np;                        // 16, 32 or 64
    int32_t seg;
    int64_t slots;
    int64_t groups;                    // workgroups of a place
    int64_t bytes;                     // workspace
};
SsmChannelPlan ssm_channel_plan(int64_t T, int64_t batch, int32_t G, int32_t P, int32_t N, bool workspace);

// Launchers: each enqueues its kernels and returns hipGetLastError().
// `head`: one step size and one decay a head.  `vec`: unit strides of B, C, the state
// and, without `head`, A, and every base and stride of theirs keeps four elements together.
hipError_t launch_ssm_recurrent(const SsmParams &p, bool head, bool vec, hipStream_t s);
// `vec`: unit strides of x, B, C, z and out, every base and stride of 8 elements; `svec`: the state's rows in 16-byte
// pieces.  The head form, up to kSsmMaxChunkN states.
hipError_t launch_ssm_chunk(const SsmParams &p, bool vec, bool svec, const SsmPlan &plan, void *workspace, hipStream_t s);
// The channel form with a group a head, up to kSsmMaxChannelN states.  `rows`: unit channel strides of x, dt, z and out, and
// rows longer than a group.
hipError_t launch_ssm_channel(const SsmParams &p, bool rows, const SsmChannelPlan &plan, void *workspace, hipStream_t s);
// `vec`: unit channel strides, every base and stride of 8 elements.
hipError_t launch_group_norm(const NormParams &p, bool vec, hipStream_t s);

}  // namespace sconv
