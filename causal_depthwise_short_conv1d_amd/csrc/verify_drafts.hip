// Verification of drafted tokens: two kernels, the vocabulary of a request's
// deciding row cut into slices.
//
// Draft j of a request is accepted while u_j q_j[x_j] < p_j[x_j].  The token
// after the accepted ones is drawn from r = max(p - q, 0) of the refused draft
// (p with the draft's entry taken out when q is null; p itself when that
// leaves nothing, or when every draft was accepted): the smallest index whose
// running sum exceeds u * total.  The products and sums are in fp64: a product
// of two fp32 values is exact there, and a running sum over 10^5 entries is
// wrong by some 1e-14, so the choice does not depend on the slicing.
// verify_sums_kernel streams the deciding row(s) once, a slice a workgroup,
// and is bound by those reads; verify_pick_kernel (a workgroup a request)
// scans the slice sums and reads one slice again, into registers).
// 64 requests of 131072 entries: 13 us for the sums, which read 67 MB
// (5.2 TB/s), and 7 us to pick: three dependent reads and as many scans, about
// what any workgroup takes for them.  256 requests without draft rows: 20 and
// 8 us.  (Reading the rows past the caches is worth 1 % either way.)
#include "gdr_params.h"
#include "sconv_device.h"

namespace sconv {

namespace {

constexpr int kVfBlock = 256;

struct Decision {
    const float *p, *q;        // deciding rows (q null: none, or a deterministic draft)
    int32_t count;             // accepted drafts
    int32_t out_token;         // entry taken out of p (deterministic refused draft), or -1
    int32_t d0;                // the request's first draft
    int32_t n;
};

__device__ __forceinline__ Decision request(const VerifyParams &p, int32_t b) {
    Decision r;
    int32_t a = p.start[b], e = p.start[b + 1];
    a = a < 0 ? 0 : (a > p.num_drafts ? p.num_drafts : a);
    e = e < a ? a : (e > p.num_drafts ? p.num_drafts : e);
    r.d0 = a;
    r.n = e - a < p.max_drafts ? e - a : p.max_drafts;
    return r;
}
// The rows that decide once `count` drafts stand.
__device__ __forceinline__ void rows_after(const VerifyParams &p, int32_t b, int32_t count, Decision &r) {
    r.count = count;
    const int64_t d = int64_t(r.d0) + count;
    r.p = p.p + (d + b) * p.p_sr;
    r.q = nullptr;
    r.out_token = -1;
    if (count < r.n) {
        if (p.q) r.q = p.q + d * p.q_sr;
        else r.out_token = p.draft_tokens[d];
    }
}

// Which drafts stand: 64 at a time, a lane each, the first refusal by ballot.  Every wave of the summing kernel does this
// by itself (two dependent reads).
__device__ __forceinline__ Decision decide(const VerifyParams &p, int32_t b) {
    Decision r = request(p, b);
    int32_t count = r.n;
    const int lane = threadIdx.x & 63;
    for (int32_t base = 0; base < r.n; base += 64) {
        const int32_t j = base + lane;
        bool refused = false;
        if (j < r.n) {
            const int64_t d = r.d0 + j;
            const int32_t x = p.draft_tokens[d];
            refused = true;
            if (x >= 0 && x < p.vocab) {
                const double px = p.p[(d + b) * p.p_sr + x];
                const double qx = p.q ? double(p.q[d * p.q_sr + x]) : 1.0;
                refused = !(double(p.u_acc[d]) * qx < px);
            }
        }
        const uint64_t m = __ballot(refused);
        if (m) {
            count = base + __builtin_ctzll(m);
            break;
        }
    }
    rows_after(p, b, count, r);
    return r;
}

// Mass of entry i: what the draw goes by (left), and the target's own.  What
// is not above zero (NaN included) has none.
__device__ __forceinline__ double mass(float v) { return v > 0.0f ? double(v) : 0.0; }
__device__ __forceinline__ double left_of(const Decision &d, int32_t i, float pv, float qv) {
    const double x = mass(pv) - mass(qv);
    return i == d.out_token ? 0.0 : (x > 0.0 ? x : 0.0);
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m);
    return v;
}

__global__ __launch_bounds__(kVfBlock) void verify_sums_kernel(VerifyParams p) {
    const int32_t b = int32_t(blockIdx.x / uint32_t(p.slices));
    const int32_t s = int32_t(blockIdx.x - uint32_t(b) * uint32_t(p.slices)), tid = int32_t(threadIdx.x);
    const Decision d = decide(p, b);
    const int32_t lo = s * p.slice, hi = lo + p.slice < p.vocab ? lo + p.slice : p.vocab;
    double left = 0.0, all = 0.0;
#pragma unroll 8
    for (int32_t i = lo + tid; i < hi; i += kVfBlock) {
        const float pv = d.p[i];
        const float qv = d.q ? d.q[i] : 0.0f;
        all += mass(pv);
        left += left_of(d, i, pv, qv);
    }
    left = wave_sum(left);
    all = wave_sum(all);
    __shared__ double part[2][kVfBlock / 64];
    if ((tid & 63) == 0) { part[0][tid >> 6] = left; part[1][tid >> 6] = all; }
    __syncthreads();
    if (tid < 2) {
        double t = 0.0;
#pragma unroll
        for (int w = 0; w < kVfBlock / 64; ++w) t += part[tid][w];
        p.sums_ws[(int64_t(b) * p.slices + s) * 2 + tid] = t;
    }
    if (s == 0 && tid == 2) p.count_ws[b] = d.count;
}

// Inclusive running sum over a wave's lanes.
__device__ __forceinline__ double wave_scan(double v) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        const double o = __shfl_up(v, m);
        if (lane >= m) v += o;
    }
    return v;
}

typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));
constexpr int kWaveSlice = kVfMaxSlice / (kVfBlock / 64);      // entries a wave scans
constexpr int kRounds = kWaveSlice / 256;                      // of four consecutive entries a lane

__global__ __launch_bounds__(kVfBlock) void verify_pick_kernel(VerifyParams p) {
    const int32_t b = int32_t(blockIdx.x), tid = int32_t(threadIdx.x), w = tid >> 6, lane = tid & 63;
    __shared__ double part[kVfBlock / 64];
    __shared__ int32_t found[kVfBlock / 64], last[kVfBlock / 64];
    const double *sums = p.sums_ws + int64_t(b) * p.slices * 2;
    Decision d = request(p, b);
    rows_after(p, b, p.count_ws[b], d);

    // Every wave by itself: which slice.  A lane takes `per` consecutive slice sums.
    const int32_t per = (p.slices + 63) / 64;
    const int32_t s0 = lane * per, s1 = s0 + per < p.slices ? s0 + per : p.slices;
    double t0 = 0.0, t1 = 0.0;
    for (int32_t s = s0; s < s1; ++s) { t0 += sums[2 * s]; t1 += sums[2 * s + 1]; }
    double cum = wave_scan(t0), own = t0;
    int which = 0;
    if (!(__shfl(cum, 63) > 0.0)) {                    // nothing is left of p - q: by p itself
        cum = wave_scan(t1);
        own = t1;
        which = 1;
        d.q = nullptr;
        d.out_token = -1;
    }
    const double goal = double(p.u_smp[b]) * __shfl(cum, 63);
    const uint64_t some = __ballot(own > 0.0), over = __ballot(own > 0.0 && cum > goal);
    // the first lane whose running sum exceeds the goal, else the last one with any mass
    const int at = over ? __builtin_ctzll(over) : (some ? 63 - __builtin_clzll(some) : 0);
    int32_t slice = -1;
    double before = cum - own;
    if (lane == at && some) {
        double run = before;                           // before the slice at hand; `before`: before the chosen one
        for (int32_t s = s0; s < s1; ++s) {
            const double m = sums[2 * s + which];
            if (m > 0.0) {
                slice = s;
                before = run;
                if (run + m > goal) break;
            }
            run += m;
        }
    }
    slice = __shfl(slice, at);
    before = __shfl(before, at);

    // The slice again, a quarter a wave, four consecutive entries a lane and round: (wave, round, lane) is index order.
    int32_t hit = INT32_MAX, top = -1;
    if (slice >= 0) {
        const int32_t lo = slice * p.slice, hi = lo + p.slice < p.vocab ? lo + p.slice : p.vocab;
        const int32_t quarter = (p.slice + kVfBlock / 64 - 1) / (kVfBlock / 64);
        const int32_t w0 = lo + w * quarter, w1 = w0 + quarter < hi ? w0 + quarter : hi;
        float x[kRounds][4];                           // fp32 suffices for p and q; masses are formed in fp64
        float y[kRounds][4];
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
            const int32_t i = w0 + 256 * r + 4 * lane;
#pragma unroll
            for (int e = 0; e < 4; ++e) x[r][e] = y[r][e] = 0.0f;
            if (i + 4 <= w1) {
                const f32x4u v = *reinterpret_cast<const f32x4u *>(d.p + i);
#pragma unroll
                for (int e = 0; e < 4; ++e) x[r][e] = v[e];
                if (d.q) {
                    const f32x4u q = *reinterpret_cast<const f32x4u *>(d.q + i);
#pragma unroll
                    for (int e = 0; e < 4; ++e) y[r][e] = q[e];
                }
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (i + e < w1) {
                        x[r][e] = d.p[i + e];
                        if (d.q) y[r][e] = d.q[i + e];
                    }
            }
        }
        // sums of the rounds (all at once), then of the waves before
        double round[kRounds], total[kRounds], all = 0.0;
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
            round[r] = 0.0;
#pragma unroll
            for (int e = 0; e < 4; ++e) round[r] += left_of(d, w0 + 256 * r + 4 * lane + e, x[r][e], y[r][e]);
            total[r] = round[r];
        }
#pragma unroll
        for (int m = 32; m >= 1; m >>= 1)
#pragma unroll
            for (int r = 0; r < kRounds; ++r) total[r] += __shfl_xor(total[r], m);
#pragma unroll
        for (int r = 0; r < kRounds; ++r) all += total[r];
        if (lane == 0) part[w] = all;
        __syncthreads();
        double c = before;
        for (int i = 0; i < w; ++i) c += part[i];
        // the first round that passes the goal, entry by entry; of the others only the last entry with mass counts
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
            if (hit == INT32_MAX && total[r] > 0.0) {
                const bool over = c + total[r] > goal;
                double run = over ? c + (wave_scan(round[r]) - round[r]) : 0.0;
                int32_t h = INT32_MAX, l = -1;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int32_t i = w0 + 256 * r + 4 * lane + e;
                    const double m = left_of(d, i, x[r][e], y[r][e]);
                    run += m;
                    if (m > 0.0) {
                        l = i;
                        if (over && h == INT32_MAX && run > goal) h = i;
                    }
                }
                const uint64_t hs = __ballot(h != INT32_MAX), ls = __ballot(l >= 0);
                top = __shfl(l, 63 - __builtin_clzll(ls));
                if (hs) hit = __shfl(h, __builtin_ctzll(hs));
                else if (over) hit = top;              // (the same sum in another order fell short by its last bit)
                c += total[r];
            }
        }
        if (lane == 0) { found[w] = hit; last[w] = top; }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kVfBlock / 64; ++i) {
            hit = found[i] < hit ? found[i] : hit;
            top = last[i] > top ? last[i] : top;
        }
    }
    const int32_t token = slice < 0 ? 0 : (hit != INT32_MAX ? hit : top);
    for (int32_t i = tid; i <= p.max_drafts; i += kVfBlock)
        p.tokens[b * p.t_sr + i] = i < d.count ? p.draft_tokens[d.d0 + i] : (i == d.count ? token : -1);
    if (tid == 0) p.num_accepted[b] = d.count + 1;
}

}  // namespace

hipError_t launch_verify_drafts(const VerifyParams &p, hipStream_t s) {
    verify_sums_kernel<<<dim3(uint32_t(p.slices) * uint32_t(p.batch)), dim3(kVfBlock), 0, s>>>(p);
    verify_pick_kernel<<<dim3(uint32_t(p.batch)), dim3(kVfBlock), 0, s>>>(p);
    return hipGetLastError();
}

}  // namespace sconv
