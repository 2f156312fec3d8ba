// The selective state space scan of the channel form: prefill with a step size a
// channel and a decay a channel and state.
//
//   S[n] <- e^(d A[n]) S[n] + d x B[n];   y = sum_n S[n] C[n] + D x
//
// A thread has a channel, with its states and decays in registers; a workgroup
// has 256 channels of one group, whose B and C it brings to LDS in fp32, eight
// tokens at a time, while the eight before are computed.  Nothing is exchanged.
//
// A state costs four products or sums and an exponential a token, and a channel
// the step's softplus: for 16 states 114 vector instructions a token in the walk for
// the states alone, 138 in the one for the outputs.  Where a
// call's channels and sequences do not fill the chip, sequences are cut into
// segments that are walked twice at once: for the states at their ends, from
// empty ones, then, once a pass over the segments has joined these, for the outputs.
//
// Bound by the vector instructions, of which an exponential takes as long as two:
// 4195 tokens of 8192 channels with 16 states take 124 us for the states, 12 for the
// pass and 151 for the outputs, of which, by leaving each out in turn, the
// exponentials are about 30, the softplus 26 (4 of them its exponent's second part,
// by what it added) and the wait for x, dt and z 36.
// B and C in scalar registers took as long as from LDS; more waves a SIMD than
// four spill, and so do 33 to 64 states with two (12 to 90 registers in scratch
// memory: 4195 tokens of 4096 channels 184 us with 16 states, 318 with 32, 731 with
// 64, and 4741 a token at a time with 128).
#include <float.h>

#include <type_traits>

#include "ssm_device.h"

namespace sconv {

namespace {

constexpr int kTB = kSsmTokens;        // tokens of a block
constexpr int kThreads = kSsmChannels; // a workgroup, a channel each

enum Mode { kWhole, kStates, kSegment };

// Segment k of sequence i has slot floor(start_i / seg) + i + k: no two share one, and floor(T / seg) + batch + 1 are enough.
__device__ __forceinline__ int64_t first_slot(const SsmParams &p, int32_t b, int32_t seg) {
    int64_t a = p.qsl[b];
    a = a < 0 ? 0 : (a > p.total_T ? p.total_T : a);
    return a / seg + b;
}

// The rows of a tensor that a workgroup walks, `left` of them; rows(t): a descriptor of those from t on, a block of them at most.
struct Block {
    const void *at;
    int64_t row;                       // bytes
    int32_t left;
    __device__ __forceinline__ Rsrc rows(int32_t t) const {
        const int32_t n = left - t < kTB ? left - t : kTB;
        return make_rsrc(static_cast<const char *>(at) + t * row, n * row);
    }
};

// A wave's 64 channels of a slot in the workspace: its states by [n][lane], and the sums of the steps above and below 0.
template <int NP>
struct Piece {
    float S[NP][64];
    float up[64], down[64];
};

// ROWS: x, dt, z and out have unit channel strides, and rows longer than a group: they are read and written through descriptors of
// a block's rows, and what lies behind the last token is not there.
template <int NP, bool DT32, bool ROWS, Mode MODE>
__global__ __launch_bounds__(kThreads, NP <= 16 ? 4 : 2) void ssm_channel_kernel(SsmParams p, int32_t blocks, int64_t places, int32_t seg, void *ws) {
    constexpr bool kOut = MODE != kStates;
    constexpr int kRow = kOut ? 2 * NP : NP, kStage = (kTB * kRow + kThreads - 1) / kThreads;
    __shared__ alignas(16) float bc[2][kTB][kRow];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const uint32_t place = blockIdx.x / uint32_t(p.G * blocks), gb = blockIdx.x - place * uint32_t(p.G * blocks);
    if (place >= places) return;
    const int32_t g = int32_t(gb / uint32_t(blocks)), c0 = int32_t(gb % uint32_t(blocks)) * kThreads;
    SsmSpan sp;
    int64_t slot = 0, t0 = 0, t1;
    int32_t b = int32_t(place);
    if constexpr (MODE != kWhole) {
        slot = place;
        int32_t lo = 0, hi = p.batch - 1;
        while (lo < hi) {
            const int32_t m = (lo + hi + 1) >> 1;
            if (first_slot(p, m, seg) <= slot) lo = m; else hi = m - 1;
        }
        b = lo;
    }
    if (!ssm_span(p, b, sp)) return;
    t1 = sp.n;
    if constexpr (MODE != kWhole) {
        const int64_t k = slot - first_slot(p, b, seg);
        t0 = k * seg;
        if (k < 0 || t0 >= sp.n) return;
        if (MODE == kStates && t0 + seg >= sp.n) return;           // the last segment's end is no one's start
        t1 = t0 + seg < sp.n ? t0 + seg : sp.n;
    }
    for (int i = threadIdx.x; i < 2 * kTB * kRow; i += kThreads) (&bc[0][0][0])[i] = 0.0f;

    // one group a head: channel c of group g
    const int32_t c = c0 + threadIdx.x, cc = c < p.P ? c : 0;
    const bool live = c < p.P;
    const int64_t per_slot = int64_t(p.G) * blocks * (kThreads / 64);
    const int64_t piece = int64_t(gb) * (kThreads / 64) + wave;
    Piece<NP> *pieces = static_cast<Piece<NP> *>(ws);
    float S[NP], a[NP];
    bool up = true;                    // no decay that grows with the step, and none that is infinite
#pragma unroll
    for (int n = 0; n < NP; ++n) {
        a[n] = n < p.N ? p.A.p[g * p.A.sh + cc * p.A.sd + n * p.A.sn] * kLog2e : 0.0f;
        up = up && a[n] <= 0.0f && a[n] >= -FLT_MAX;
        S[n] = 0.0f;
    }
    const bool plain = __builtin_amdgcn_ballot_w64(!up) == 0;
    float *row = p.state ? p.state + sp.line * p.s_sl + g * p.s_sh + cc * p.s_sp : nullptr;
    if (MODE == kSegment && sp.n > seg) {
#pragma unroll
        for (int n = 0; n < NP; ++n)
            if (n < p.N) S[n] = pieces[slot * per_slot + piece].S[n][lane];
    } else if (kOut) {
        if (sp.init) {
#pragma unroll
            for (int n = 0; n < NP; ++n)
                if (n < p.N) S[n] = row[n * p.s_sn];
        }
    }
    const float bias = p.bias.p ? p.bias.p[g * p.bias.sh + cc * p.bias.sd] : 0.0f;
    const float D = kOut && p.D.p ? p.D.p[g * p.D.sh + cc * p.D.sd] : 0.0f;
    const int64_t r0 = sp.t0 + t0;
    const int32_t left = int32_t(t1 - t0);
    const uint16_t *xp = p.x + r0 * p.xs.st + g * p.xs.sh + cc * p.xs.sd;
    const uint16_t *zp = kOut && p.z ? p.z + r0 * p.zs.st + g * p.zs.sh + cc * p.zs.sd : nullptr;
    uint16_t *op = p.out + r0 * p.os.st + g * p.os.sh + cc * p.os.sd;
    const int64_t dt0 = r0 * p.ds.st + g * p.ds.sh + cc * p.ds.sd;
    const uint16_t *Bp = p.B + r0 * p.bs.st + g * p.bs.sh, *Cp = p.C + r0 * p.cs.st + g * p.cs.sh;

    const Block xb{p.x + r0 * p.xs.st + g * p.xs.sh, p.xs.st * 2, left}, zb{p.z + r0 * p.zs.st + g * p.zs.sh, p.zs.st * 2, left};
    const Block ob{p.out + r0 * p.os.st + g * p.os.sh, p.os.st * 2, left};
    const Block db{static_cast<const char *>(p.dt) + (r0 * p.ds.st + g * p.ds.sh) * (DT32 ? 4 : 2), p.ds.st * (DT32 ? 4 : 2), left};
    uint32_t xn[kTB], dn[kTB], zn[kTB], sn[kStage];
    // B and C of a block, past the end of the segment its last token's.
    const auto fetch_bc = [&](int32_t t) {
#pragma unroll
        for (int i = 0; i < kStage; ++i) {
            const int at = threadIdx.x + i * kThreads, tt = at / kRow, n = at % kRow;
            const int64_t r = t + tt < left ? t + tt : left - 1;
            sn[i] = 0;
            if (at < kTB * kRow && n % NP < p.N)
                sn[i] = n < NP ? Bp[r * p.bs.st + n * p.bs.sd] : Cp[r * p.cs.st + (n - NP) * p.cs.sd];
        }
    };
    // Token k of the block at t of the channel's inputs, in the place of the block's before it.  The lane's offset is kept from
    // the compiler, which would hold every token's in registers; whole blocks' rows go by the scalar offset.
    const auto fetch = [&](int32_t t, int k, const Rsrc &xr, const Rsrc &dr, const Rsrc &zr, auto full) {
        if constexpr (ROWS) {
            constexpr bool FULL = decltype(full)::value;
            int32_t at = 2 * cc;
            asm volatile("" : "+v"(at));
            const auto load = [&](const Rsrc &r, int32_t row) -> uint32_t {
                return FULL ? __builtin_amdgcn_raw_buffer_load_b16(r, at, k * row, 0) : __builtin_amdgcn_raw_buffer_load_b16(r, at + k * row, 0, 0);
            };
            xn[k] = load(xr, int32_t(xb.row));
            if constexpr (DT32) dn[k] = __builtin_amdgcn_raw_buffer_load_b32(dr, 2 * at + k * int32_t(db.row), 0, 0);
            else dn[k] = load(dr, int32_t(db.row));
            if (kOut && zp) zn[k] = load(zr, int32_t(zb.row));
        } else {
            const int64_t r = t + k < left ? t + k : left - 1;
            xn[k] = xp[r * p.xs.st];
            if constexpr (DT32) dn[k] = static_cast<const uint32_t *>(p.dt)[dt0 + r * p.ds.st];
            else dn[k] = static_cast<const uint16_t *>(p.dt)[dt0 + r * p.ds.st];
            if (kOut && zp) zn[k] = zp[r * p.zs.st];
        }
    };
    const auto stage = [&](int buf) {
#pragma unroll
        for (int i = 0; i < kStage; ++i) {
            const int at = threadIdx.x + i * kThreads;
            if (at < kTB * kRow) (&bc[buf][0][0])[at] = __uint_as_float(sn[i] << 16);
        }
    };
    __syncthreads();
    fetch_bc(0);
    {
        const Rsrc xr = xb.rows(0), dr = db.rows(0), zr = zb.rows(zp ? 0 : left);
#pragma unroll
        for (int k = 0; k < kTB; ++k) fetch(0, k, xr, dr, zr, std::false_type());
    }
    stage(0);
    __syncthreads();
    float sum_up = 0.0f, sum_down = 0.0f;
    // FULL: all tokens of the block and of the next one exist.
    const auto block = [&](int32_t t, auto full) {
        constexpr bool FULL = decltype(full)::value;
        const int buf = (t / kTB) & 1;
        fetch_bc(t + kTB);
        const Rsrc xr = xb.rows(t + kTB), dr = db.rows(t + kTB), zr = zb.rows(zp ? t + kTB : left), ow = ob.rows(t);
#pragma unroll
        for (int k = 0; k < kTB; ++k) {
            float s = ssm_clamp(p, ssm_softplus(p, __uint_as_float(DT32 ? dn[k] : dn[k] << 16) + bias));
            if (!FULL && t + k >= left) s = 0.0f;      // no step
            const uint32_t xk = xn[k], zk = kOut ? zn[k] : 0;
            fetch(t + kTB, k, xr, dr, zr, full);
            const float xf = __uint_as_float(xk << 16), u = FULL || t + k < left ? s * xf : 0.0f;
            const float su = s < 0.0f ? 0.0f : s;      // (NaN stays)
            if (MODE == kStates) { sum_up += su; sum_down += s - su; }
            const f32x4 *bv = reinterpret_cast<const f32x4 *>(&bc[buf][k][0]);
            float y[2] = {0.0f, 0.0f};
            const auto states = [&](auto decay) {
#pragma unroll
                for (int q = 0; q < NP / 4; ++q) {
                    const f32x4 bb = bv[q], cv = kOut ? bv[(kOut ? NP / 4 : 0) + q] : bb;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int n = 4 * q + e;
                        S[n] = fmaf(decay(a[n]), S[n], u * bb[e]);
                        if (kOut) y[e & 1] = fmaf(S[n], cv[e], y[e & 1]);
                    }
                }
            };
            if (plain) states([&](float an) { return __builtin_amdgcn_exp2f(su * an); });
            else states([&](float an) { const float v = s == 0.0f ? 0.0f : s * an; return __builtin_amdgcn_exp2f(v > 0.0f ? 0.0f : v); });
            if constexpr (kOut) {
                float o = fmaf(D, xf, y[0] + y[1]);
                if (zp) o = ssm_gate(o, __uint_as_float(zk << 16));
                if constexpr (ROWS) {
                    uint32_t at = live ? 2 * c : kOob;
                    asm volatile("" : "+v"(at));
                    if constexpr (FULL) __builtin_amdgcn_raw_buffer_store_b16(to_bf16(o), ow, at, k * int32_t(ob.row), 0);
                    else __builtin_amdgcn_raw_buffer_store_b16(to_bf16(o), ow, at + k * uint32_t(ob.row), 0, 0);
                } else if (live && t + k < left) {
                    op[(t + k) * p.os.st] = to_bf16(o);
                }
            }
            __builtin_amdgcn_sched_barrier(0);         // (or all tokens' B and C would be read at once)
        }
        stage(buf ^ 1);
        __syncthreads();
    };
    int32_t t = 0;
    if constexpr (ROWS)
        for (; t + 2 * kTB <= left; t += kTB) block(t, std::true_type());
    for (; t < left; t += kTB) block(t, std::false_type());
    if constexpr (MODE == kStates) {
        Piece<NP> &o = pieces[slot * per_slot + piece];
#pragma unroll
        for (int n = 0; n < NP; ++n) o.S[n][lane] = S[n];
        o.up[lane] = sum_up;
        o.down[lane] = sum_down;
    } else {
        if (p.state && t1 == sp.n && live) {
#pragma unroll
            for (int n = 0; n < NP; ++n)
                if (n < p.N) row[n * p.s_sn] = S[n];
        }
    }
}

// From each segment's own states to those that it starts from, in place: a thread takes a state of a channel through a sequence's
// segments.  The first one's are among them: in the third kernel the last segment may write the line before the first has begun.
template <int NP>
__global__ __launch_bounds__(256) void ssm_channel_pass_kernel(SsmParams p, int32_t blocks, int32_t seg, void *ws) {
    const int64_t per_slot = int64_t(p.G) * blocks * (kThreads / 64);
    const int64_t id = int64_t(blockIdx.x) * 256 + threadIdx.x, w = id / (64 * NP);
    if (w >= int64_t(p.batch) * per_slot) return;
    const int32_t b = int32_t(w / per_slot), lane = int32_t(id & 63), n = int32_t(id / 64 % NP);
    const int64_t piece = w - b * per_slot;
    SsmSpan sp;
    if (!ssm_span(p, b, sp) || n >= p.N) return;
    const int64_t ns = (sp.n + seg - 1) / seg;
    const int32_t g = int32_t(piece / (blocks * (kThreads / 64))), c = int32_t(piece % (blocks * (kThreads / 64))) * 64 + lane;
    if (c >= p.P) return;
    const float a = p.A.p[g * p.A.sh + c * p.A.sd + n * p.A.sn] * kLog2e;
    float S = 0.0f;
    if (sp.init) S = p.state[sp.line * p.s_sl + g * p.s_sh + c * p.s_sp + n * p.s_sn];
    Piece<NP> *at = static_cast<Piece<NP> *>(ws) + first_slot(p, b, seg) * per_slot + piece;
    constexpr int kFew = 4;            // segments read together
    for (int64_t i = 0; i + 1 < ns; i += kFew) {
        float own[kFew], sum[kFew];
#pragma unroll
        for (int k = 0; k < kFew; ++k) {
            const Piece<NP> &q = at[(i + k + 1 < ns ? i + k : ns - 2) * per_slot];
            own[k] = q.S[n][lane];
            sum[k] = a > 0.0f ? q.down[lane] : q.up[lane];
        }
#pragma unroll
        for (int k = 0; k < kFew; ++k) {
            if (i + k + 1 >= ns) break;
            at[(i + k) * per_slot].S[n][lane] = S;
            S = fmaf(__builtin_amdgcn_exp2f(sum[k] == 0.0f ? 0.0f : a * sum[k]), S, own[k]);
        }
    }
    if (ns > 1) at[(ns - 1) * per_slot].S[n][lane] = S;
}

template <int NP, bool DT32, bool ROWS>
hipError_t launch(const SsmParams &p, const SsmChannelPlan &plan, void *ws, hipStream_t s) {
    const int32_t blocks = (p.P + kThreads - 1) / kThreads;
    const int64_t per = int64_t(p.G) * blocks;
    if (!plan.seg) {
        ssm_channel_kernel<NP, DT32, ROWS, kWhole><<<dim3(uint32_t(p.batch * per)), dim3(kThreads), 0, s>>>(p, blocks, p.batch, 0, nullptr);
        return hipGetLastError();
    }
    ssm_channel_kernel<NP, DT32, ROWS, kStates><<<dim3(uint32_t(plan.slots * per)), dim3(kThreads), 0, s>>>(p, blocks, plan.slots, plan.seg, ws);
    ssm_channel_pass_kernel<NP><<<dim3(uint32_t(p.batch * per * (kThreads / 64) * NP / 4)), dim3(256), 0, s>>>(p, blocks, plan.seg, ws);
    ssm_channel_kernel<NP, DT32, ROWS, kSegment><<<dim3(uint32_t(plan.slots * per)), dim3(kThreads), 0, s>>>(p, blocks, plan.slots, plan.seg, ws);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_ssm_channel(const SsmParams &p, bool rows, const SsmChannelPlan &plan, void *ws, hipStream_t s) {
    const auto as = [&](auto np) {
        constexpr int NP = decltype(np)::value;
        if (p.dt_fp32) return rows ? launch<NP, true, true>(p, plan, ws, s) : launch<NP, true, false>(p, plan, ws, s);
        return rows ? launch<NP, false, true>(p, plan, ws, s) : launch<NP, false, false>(p, plan, ws, s);
    };
    if (plan.np == 16) return as(std::integral_constant<int, 16>());
    return plan.np == 32 ? as(std::integral_constant<int, 32>()) : as(std::integral_constant<int, 64>());
}

}  // namespace sconv
