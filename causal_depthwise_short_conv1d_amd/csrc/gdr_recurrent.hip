// The gated delta rule, one token at a time: the decode update, and prefill
// of heads that the chunked kernel does not take.
//
// Per value head, with the state S[v][k] held in registers in fp32:
//   S <- e^g S;  u = beta (v - S k);  S <- S + u k^T;  o = scale S q
// evaluated as sk = S k and sq = S q on the state of before, so that both sums
// run together: u = beta (v - e^g sk), o = e^g sq + u (k.q).
// A wave holds 8 R rows of one head's state: 8 lanes a row, each with the
// channels 32 i + 4 j + (0..3) of its place j, so a row is read in whole
// 128-byte pieces and a sum over k is three lane exchanges.  The state is read
// and written once however many tokens follow each other; everything else is
// a few KiB.  Decode is bound by those bytes: 256 requests of 32 heads of
// 128 x 128 move 1.07 GB in 202 us, 5.3 TB/s (a copy of as many bytes: 5.3), 64
// requests take 56 us.
// State rows pass the caches (nontemporal): a step reads a line once and the
// next step comes after a model's other layers.  221 us with plain accesses for
// 256 requests, 62 for 64; a batch that stays in the caches between calls would
// lose: 55 against 59 us for the same 64 lines over and over.
#include "gdr_device.h"

namespace sconv {

namespace {

constexpr int kRecWaves = 4;           // waves per workgroup

// KI: 32-channel pieces of a row (ceil(Dk / 32)).  R: row groups per wave.
template <int KI, bool VEC>
__device__ __forceinline__ void load_row(const uint16_t *p, int64_t sd, int32_t Dk, int j,
                                         float (&f)[KI * 4]) {
#pragma unroll
    for (int i = 0; i < KI; ++i) {
        const int c = 32 * i + 4 * j;
        if constexpr (VEC) {
            u32x2 w = {0u, 0u};
            if (c < Dk) w = *reinterpret_cast<const u32x2 *>(p + c);
            f[4 * i] = bf_lo(w.x); f[4 * i + 1] = bf_hi(w.x);
            f[4 * i + 2] = bf_lo(w.y); f[4 * i + 3] = bf_hi(w.y);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) f[4 * i + e] = c + e < Dk ? bf_one(p[(c + e) * sd]) : 0.0f;
        }
    }
}

template <int KI, bool VEC>
__device__ __forceinline__ void load_state(const float *p, int64_t sk, int32_t Dk, int j, bool row,
                                           float (&f)[KI * 4]) {
#pragma unroll
    for (int i = 0; i < KI; ++i) {
        const int c = 32 * i + 4 * j;
        if constexpr (VEC) {
            f32x4 w = {0.0f, 0.0f, 0.0f, 0.0f};
            if (row && c < Dk) w = __builtin_nontemporal_load(reinterpret_cast<const f32x4 *>(p + c));
            f[4 * i] = w.x; f[4 * i + 1] = w.y; f[4 * i + 2] = w.z; f[4 * i + 3] = w.w;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) f[4 * i + e] = row && c + e < Dk ? p[(c + e) * sk] : 0.0f;
        }
    }
}

template <int KI, bool VEC>
__device__ __forceinline__ void store_state(float *p, int64_t sk, int32_t Dk, int j, bool row,
                                            const float (&f)[KI * 4]) {
#pragma unroll
    for (int i = 0; i < KI; ++i) {
        const int c = 32 * i + 4 * j;
        if constexpr (VEC) {
            const f32x4 w = {f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]};
            if (row && c < Dk) __builtin_nontemporal_store(w, reinterpret_cast<f32x4 *>(p + c));
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (row && c + e < Dk) p[(c + e) * sk] = f[4 * i + e];
        }
    }
}

template <int KI, int R, bool VEC>
__global__ __launch_bounds__(64 * kRecWaves) void gdr_recurrent_kernel(GdrParams p, int32_t tiles,
                                                                       int64_t n_tiles) {
    const int lane = threadIdx.x & 63, j = lane & 7, r = lane >> 3;
    const int64_t tile = int64_t(blockIdx.x) * kRecWaves + (threadIdx.x >> 6);
    if (tile >= n_tiles) return;
    const int64_t eh = tile / tiles;
    const int32_t v0 = int32_t(tile - eh * tiles) * (8 * R);
    const int32_t b = int32_t(eh / p.Hv), h = int32_t(eh - int64_t(b) * p.Hv);
    const int32_t hk = h / p.group;

    // the entry's tokens and its line
    int64_t t0 = 0, n = p.seqlen, line = b;
    bool init = true;
    if (p.qsl) {
        int64_t a = p.qsl[b], e = p.qsl[b + 1];
        a = a < 0 ? 0 : (a > p.total_T ? p.total_T : a);
        e = e < a ? a : (e > p.total_T ? p.total_T : e);
        t0 = a;
        n = e - a;
        init = p.state && p.has_init && p.has_init[b] != 0;
    }
    if (n == 0) return;
    if (p.ci) {
        int32_t step = 0;
        if (p.accepted) {
            step = p.accepted[b] - 1;
            if (step < 0 || step >= p.ci_steps) return;
        }
        line = p.ci[b * p.ci_sb + step * p.ci_ss];
        if (line == p.pad_slot_id) return;
    }
    if (p.state && (line < 0 || line >= p.num_lines)) return;

    int32_t vr[R];
    bool row[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        vr[i] = v0 + 8 * i + r;
        row[i] = vr[i] < p.Dv;
    }
    float S[R][KI * 4];
    float *head = p.state ? p.state + h * p.s_sh : nullptr;
#pragma unroll
    for (int i = 0; i < R; ++i)
        load_state<KI, VEC>(init ? head + line * p.s_sl + vr[i] * p.s_sv : nullptr, p.s_sk, p.Dk, j,
                            row[i] && init, S[i]);

    const uint16_t *qp = p.q + b * p.qs.sb + t0 * p.qs.st + hk * p.qs.sh;
    const uint16_t *kp = p.k + b * p.ks.sb + t0 * p.ks.st + hk * p.ks.sh;
    const uint16_t *vp = p.v + b * p.vs.sb + t0 * p.vs.st + h * p.vs.sh;
    uint16_t *op = p.out + b * p.os.sb + t0 * p.os.st + h * p.os.sh;
    int64_t go = b * p.gs.sb + t0 * p.gs.st + h * p.gs.sh;
    int64_t bo = b * p.bs.sb + t0 * p.bs.st + h * p.bs.sh;

    float qn[KI * 4], kn[KI * 4], vn[R];
    Gates gn;
    auto fetch = [&]() {
        load_row<KI, VEC>(qp, p.qs.sd, p.Dk, j, qn);
        load_row<KI, VEC>(kp, p.ks.sd, p.Dk, j, kn);
#pragma unroll
        for (int i = 0; i < R; ++i) vn[i] = row[i] ? bf_one(vp[vr[i] * p.vs.sd]) : 0.0f;
        gn = gdr_gates(p, go, bo, h);
    };
    fetch();
    for (int64_t t = 0; t < n; ++t) {
        float q[KI * 4], k[KI * 4], v[R];
#pragma unroll
        for (int i = 0; i < KI * 4; ++i) { q[i] = qn[i]; k[i] = kn[i]; }
#pragma unroll
        for (int i = 0; i < R; ++i) v[i] = vn[i];
        const float e = expf(gn.g), beta = gn.beta;
        if (t + 1 < n) {               // the next token's reads pass behind this one's sums
            qp += p.qs.st; kp += p.ks.st; vp += p.vs.st; go += p.gs.st; bo += p.bs.st;
            fetch();
        }
        float qs = p.scale;
        if (p.l2norm) {
            float q2 = 0.0f, k2 = 0.0f;
#pragma unroll
            for (int i = 0; i < KI * 4; ++i) { q2 = fmaf(q[i], q[i], q2); k2 = fmaf(k[i], k[i], k2); }
            qs *= 1.0f / sqrtf(sum8(q2) + kL2Eps);
            const float ks = 1.0f / sqrtf(sum8(k2) + kL2Eps);
#pragma unroll
            for (int i = 0; i < KI * 4; ++i) k[i] *= ks;
        }
        float kq = 0.0f;
#pragma unroll
        for (int i = 0; i < KI * 4; ++i) kq = fmaf(k[i], q[i], kq);
        kq = sum8(kq);
        float o = 0.0f;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            float sk = 0.0f, sq = 0.0f;
#pragma unroll
            for (int c = 0; c < KI * 4; ++c) {
                sk = fmaf(S[i][c], k[c], sk);
                sq = fmaf(S[i][c], q[c], sq);
            }
            sk = sum8(sk);
            sq = sum8(sq);
            const float u = beta * (v[i] - e * sk);
#pragma unroll
            for (int c = 0; c < KI * 4; ++c) S[i][c] = fmaf(e, S[i][c], u * k[c]);
            const float oi = qs * fmaf(e, sq, u * kq);
            o = j == i ? oi : o;
        }
        const int32_t ov = v0 + 8 * j + r;         // lane j of a row group stores row group j's output
        if (j < R && ov < p.Dv) op[ov * p.os.sd] = to_bf16(o);
        op += p.os.st;
        if (p.osi) {
            const int64_t to = p.osi[b * p.osi_sb + t * p.osi_ss];
            if (to >= 0 && to < p.num_lines) {
#pragma unroll
                for (int i = 0; i < R; ++i)
                    store_state<KI, VEC>(head + to * p.s_sl + vr[i] * p.s_sv, p.s_sk, p.Dk, j, row[i], S[i]);
            }
        }
    }
    if (p.state && !p.osi) {
#pragma unroll
        for (int i = 0; i < R; ++i)
            store_state<KI, VEC>(head + line * p.s_sl + vr[i] * p.s_sv, p.s_sk, p.Dk, j, row[i], S[i]);
    }
}

template <int KI, bool VEC>
hipError_t launch_k(const GdrParams &p, hipStream_t s) {
    // 16 rows a wave: 256 and 64 requests of 32 heads took 221 and 62 us, with 8 rows 256 and 69, with 32 rows 241 and 71.
    // A call whose rows do not fill the chip (fewer than 8 waves a CU) takes 8, for twice the waves.
    const int64_t heads = int64_t(p.batch) * p.Hv;
    const bool few = heads * ((p.Dv + 15) / 16) < 2048;
    const int rows = few ? 8 : 16;
    const int32_t tiles = (p.Dv + rows - 1) / rows;
    const int64_t n = heads * tiles;
    const dim3 grid(uint32_t((n + kRecWaves - 1) / kRecWaves)), block(64 * kRecWaves);
    if (few) gdr_recurrent_kernel<KI, 1, VEC><<<grid, block, 0, s>>>(p, tiles, n);
    else gdr_recurrent_kernel<KI, 2, VEC><<<grid, block, 0, s>>>(p, tiles, n);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_gdr_recurrent(const GdrParams &p, bool vec, hipStream_t s) {
    switch ((p.Dk + 31) / 32) {
        case 1: return vec ? launch_k<1, true>(p, s) : launch_k<1, false>(p, s);
        case 2: return vec ? launch_k<2, true>(p, s) : launch_k<2, false>(p, s);
        case 3: return vec ? launch_k<3, true>(p, s) : launch_k<3, false>(p, s);
        case 4: return vec ? launch_k<4, true>(p, s) : launch_k<4, false>(p, s);
        case 5: case 6: return vec ? launch_k<6, true>(p, s) : launch_k<6, false>(p, s);
        default: return vec ? launch_k<8, true>(p, s) : launch_k<8, false>(p, s);
    }
}

}  // namespace sconv
