// The selective state space scan, one token at a time: the decode update, and
// prefill of what the other kernels do not take.
//
// Per head and channel p, with the state S[p][n] held in registers in fp32:
//   d = step size;  S[n] <- e^(d A[n]) S[n] + d x B[n];  y = sum_n S[n] C[n] + D x;  y <- y silu(z)
// LN lanes (4 for up to 16 states, else 8) share a row, each with the states
// 4 LN i + 4 j + (0..3) of its place j, so that a row is read in whole 16-byte
// pieces and a sum over n is two or three lane exchanges; a wave holds 64 / LN * R
// rows.  The state is read and written once however many tokens follow each
// other; everything else is a few KiB.  State rows pass the caches
// (nontemporal): a step reads a line once, and the next step comes after a
// model's other layers.
//
// Bound by the states' bytes: 256 requests of 128 heads of 64 x 128 355 us, 6.0 TB/s;
// 64 requests of 4 tokens with each token's states saved 240 (writes, 5.6 TB/s).
// Small calls are bound by the chain of loads: one request of 64 heads 4.9 us; 64
// requests of 8192 channels x 16 states 19.8 us (26.5 with one row group a wave
// and decays by elements), two generations of waves for 72 MB.  Workgroups of
// eight waves were slower (409 against 368 us at 256 requests), and so were
// states through the caches (21.7 against 20.6 at 64).
#include "ssm_device.h"

namespace sconv {

namespace {

constexpr int kRecWaves = 4;           // waves per workgroup

template <int LN>
__device__ __forceinline__ float sum_row(float v) {
    if constexpr (LN == 8) return sum8(v);
    v = dpp_add<0xB1>(v);              // quad_perm [1,0,3,2]
    return dpp_add<0x4E>(v);           // quad_perm [2,3,0,1]
}

template <int LN, int KI, bool VEC>
__device__ __forceinline__ void load_row(const uint16_t *p, int64_t sn, int32_t N, int j, float (&f)[KI * 4]) {
#pragma unroll
    for (int i = 0; i < KI; ++i) {
        const int c = 4 * LN * i + 4 * j;
        if constexpr (VEC) {
            u32x2 w = {0u, 0u};
            if (c < N) w = *reinterpret_cast<const u32x2 *>(p + c);
            f[4 * i] = bf_lo(w.x); f[4 * i + 1] = bf_hi(w.x);
            f[4 * i + 2] = bf_lo(w.y); f[4 * i + 3] = bf_hi(w.y);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) f[4 * i + e] = c + e < N ? bf_one(p[(c + e) * sn]) : 0.0f;
        }
    }
}

template <int LN, int KI, bool VEC>
__device__ __forceinline__ void load_state(const float *p, int64_t sn, int32_t N, int j, bool row, float (&f)[KI * 4]) {
#pragma unroll
    for (int i = 0; i < KI; ++i) {
        const int c = 4 * LN * i + 4 * j;
        if constexpr (VEC) {
            f32x4 w = {0.0f, 0.0f, 0.0f, 0.0f};
            if (row && c < N) w = __builtin_nontemporal_load(reinterpret_cast<const f32x4 *>(p + c));
            f[4 * i] = w.x; f[4 * i + 1] = w.y; f[4 * i + 2] = w.z; f[4 * i + 3] = w.w;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) f[4 * i + e] = row && c + e < N ? p[(c + e) * sn] : 0.0f;
        }
    }
}

template <int LN, int KI, bool VEC>
__device__ __forceinline__ void store_state(float *p, int64_t sn, int32_t N, int j, bool row, const float (&f)[KI * 4]) {
#pragma unroll
    for (int i = 0; i < KI; ++i) {
        const int c = 4 * LN * i + 4 * j;
        if constexpr (VEC) {
            const f32x4 w = {f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]};
            if (row && c < N) __builtin_nontemporal_store(w, reinterpret_cast<f32x4 *>(p + c));
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (row && c + e < N) p[(c + e) * sn] = f[4 * i + e];
        }
    }
}

// HEAD: one step size and decay a head; otherwise a step size a channel and a decay a channel and state.
template <int LN, int KI, int R, bool HEAD, bool VEC>
__global__ __launch_bounds__(64 * kRecWaves) void ssm_recurrent_kernel(SsmParams p, int32_t tiles, int64_t n_tiles) {
    constexpr int kRows = 64 / LN;     // of one row group
    const int lane = threadIdx.x & 63, j = lane & (LN - 1), r = lane / LN;
    const int64_t tile = int64_t(blockIdx.x) * kRecWaves + (threadIdx.x >> 6);
    if (tile >= n_tiles) return;
    const int64_t eh = tile / tiles;
    const int32_t p0 = int32_t(tile - eh * tiles) * (kRows * R);
    const int32_t b = int32_t(eh / p.H), h = int32_t(eh - int64_t(b) * p.H);
    const int32_t grp = h / p.per_group;
    SsmSpan sp;
    if (!ssm_span(p, b, sp)) return;

    int32_t pr[R];
    bool row[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        pr[i] = p0 + kRows * i + r;
        row[i] = pr[i] < p.P;
        pr[i] = row[i] ? pr[i] : 0;    // (what a lane without a channel computes is dropped)
    }
    float S[R][KI * 4];
    float *head = p.state ? p.state + h * p.s_sh : nullptr;
#pragma unroll
    for (int i = 0; i < R; ++i)
        load_state<LN, KI, VEC>(sp.init ? head + sp.line * p.s_sl + pr[i] * p.s_sp : nullptr, p.s_sn, p.N, j,
                                row[i] && sp.init, S[i]);
    float A[HEAD ? 1 : R][HEAD ? 1 : KI * 4], D[R], bias[HEAD ? 1 : R];
#pragma unroll
    for (int i = 0; i < R; ++i) D[i] = p.D.p ? p.D.p[h * p.D.sh + pr[i] * p.D.sd] : 0.0f;
    if constexpr (HEAD) {
        A[0][0] = p.A.p[h * p.A.sh];
        bias[0] = p.bias.p ? p.bias.p[h * p.bias.sh] : 0.0f;
    } else {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            bias[i] = p.bias.p ? p.bias.p[h * p.bias.sh + pr[i] * p.bias.sd] : 0.0f;
            const float *a = p.A.p + h * p.A.sh + pr[i] * p.A.sd;
#pragma unroll
            for (int k = 0; k < KI; ++k) {
                const int n = 4 * LN * k + 4 * j;
                if constexpr (VEC) {
                    f32x4 w = {0.0f, 0.0f, 0.0f, 0.0f};
                    if (n < p.N) w = *reinterpret_cast<const f32x4 *>(a + n);
#pragma unroll
                    for (int e = 0; e < 4; ++e) A[i][4 * k + e] = w[e];
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) A[i][4 * k + e] = n + e < p.N ? a[(n + e) * p.A.sn] : 0.0f;
                }
            }
        }
    }

    const uint16_t *xp = p.x + b * p.xs.sb + sp.t0 * p.xs.st + h * p.xs.sh;
    const uint16_t *zp = p.z ? p.z + b * p.zs.sb + sp.t0 * p.zs.st + h * p.zs.sh : nullptr;
    const uint16_t *bp = p.B + b * p.bs.sb + sp.t0 * p.bs.st + grp * p.bs.sh;
    const uint16_t *cp = p.C + b * p.cs.sb + sp.t0 * p.cs.st + grp * p.cs.sh;
    uint16_t *op = p.out + b * p.os.sb + sp.t0 * p.os.st + h * p.os.sh;
    int64_t dp = b * p.ds.sb + sp.t0 * p.ds.st + h * p.ds.sh;

    float Bn[KI * 4], Cn[KI * 4], xn[R], zn[R], dn[HEAD ? 1 : R];
    auto fetch = [&]() {
        load_row<LN, KI, VEC>(bp, p.bs.sd, p.N, j, Bn);
        load_row<LN, KI, VEC>(cp, p.cs.sd, p.N, j, Cn);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            xn[i] = bf_one(xp[pr[i] * p.xs.sd]);
            zn[i] = zp ? bf_one(zp[pr[i] * p.zs.sd]) : 0.0f;
            if (!HEAD || i == 0) dn[HEAD ? 0 : i] = ssm_step(p, dp + (HEAD ? 0 : pr[i] * p.ds.sd), bias[HEAD ? 0 : i]);
        }
    };
    fetch();
    for (int64_t t = 0; t < sp.n; ++t) {
        float B[KI * 4], C[KI * 4], x[R], z[R], d[HEAD ? 1 : R];
#pragma unroll
        for (int i = 0; i < KI * 4; ++i) { B[i] = Bn[i]; C[i] = Cn[i]; }
#pragma unroll
        for (int i = 0; i < R; ++i) { x[i] = xn[i]; z[i] = zn[i]; if (!HEAD || i == 0) d[HEAD ? 0 : i] = dn[HEAD ? 0 : i]; }
        if (t + 1 < sp.n) {            // the next token's reads pass behind this one's sums
            xp += p.xs.st; bp += p.bs.st; cp += p.cs.st; dp += p.ds.st;
            if (zp) zp += p.zs.st;
            fetch();
        }
        float y = 0.0f;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const float di = d[HEAD ? 0 : i], u = di * x[i];
            const float eh1 = HEAD ? ssm_decay(di, A[0][0]) : 0.0f;
            float s = 0.0f;
#pragma unroll
            for (int c = 0; c < KI * 4; ++c) {
                const float e = HEAD ? eh1 : ssm_decay(di, A[HEAD ? 0 : i][HEAD ? 0 : c]);
                S[i][c] = fmaf(e, S[i][c], u * B[c]);
                s = fmaf(S[i][c], C[c], s);
            }
            float yi = fmaf(D[i], x[i], sum_row<LN>(s));
            if (zp) yi = ssm_gate(yi, z[i]);
            y = j == i ? yi : y;
        }
        const int32_t oc = p0 + kRows * j + r;         // lane j of a row's lanes stores row group j's output
        if (j < R && oc < p.P) op[oc * p.os.sd] = to_bf16(y);
        op += p.os.st;
        if (p.osi) {
            const int64_t to = p.osi[b * p.osi_sb + t * p.osi_ss];
            if (to >= 0 && to < p.num_lines) {
#pragma unroll
                for (int i = 0; i < R; ++i)
                    store_state<LN, KI, VEC>(head + to * p.s_sl + pr[i] * p.s_sp, p.s_sn, p.N, j, row[i], S[i]);
            }
        }
    }
    if (p.state && !p.osi) {
#pragma unroll
        for (int i = 0; i < R; ++i)
            store_state<LN, KI, VEC>(head + sp.line * p.s_sl + pr[i] * p.s_sp, p.s_sn, p.N, j, row[i], S[i]);
    }
}

template <int LN, int KI, bool HEAD, bool VEC>
hipError_t launch_n(const SsmParams &p, hipStream_t s) {
    constexpr int kRows = 64 / LN;
    const int64_t heads = int64_t(p.batch) * p.H;
    // two row groups a wave (four of short rows), as long as that leaves 8 waves a CU
    constexpr int kMost = KI == 1 ? 4 : 2;
    const auto waves = [&](int r) { return heads * ((p.P + r * kRows - 1) / (r * kRows)); };
    const int r = waves(kMost) >= 2048 ? kMost : (waves(2) >= 2048 ? 2 : 1);
    const int64_t n = waves(r);
    const int32_t tiles = (p.P + r * kRows - 1) / (r * kRows);
    const dim3 grid(uint32_t((n + kRecWaves - 1) / kRecWaves)), block(64 * kRecWaves);
    if (r == 1) ssm_recurrent_kernel<LN, KI, 1, HEAD, VEC><<<grid, block, 0, s>>>(p, tiles, n);
    else if (r == 2) ssm_recurrent_kernel<LN, KI, 2, HEAD, VEC><<<grid, block, 0, s>>>(p, tiles, n);
    else ssm_recurrent_kernel<LN, KI, kMost, HEAD, VEC><<<grid, block, 0, s>>>(p, tiles, n);
    return hipGetLastError();
}

template <bool HEAD, bool VEC>
hipError_t launch_form(const SsmParams &p, hipStream_t s) {
    if (p.N <= 16) return launch_n<4, 1, HEAD, VEC>(p, s);
    switch ((p.N + 31) / 32) {
        case 1: return launch_n<8, 1, HEAD, VEC>(p, s);
        case 2: return launch_n<8, 2, HEAD, VEC>(p, s);
        case 3: return launch_n<8, 3, HEAD, VEC>(p, s);
        case 4: return launch_n<8, 4, HEAD, VEC>(p, s);
        case 5: case 6: return launch_n<8, 6, HEAD, VEC>(p, s);
        default: return launch_n<8, 8, HEAD, VEC>(p, s);
    }
}

}  // namespace

hipError_t launch_ssm_recurrent(const SsmParams &p, bool head, bool vec, hipStream_t s) {
    if (head) return vec ? launch_form<true, true>(p, s) : launch_form<true, false>(p, s);
    return vec ? launch_form<false, true>(p, s) : launch_form<false, false>(p, s);
}

}  // namespace sconv
