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
// scans the slice sums and reads one slice again.
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

// Which drafts stand: 64 at a time, a lane each, the first refusal by ballot.
// Every wave of a request does this by itself (two dependent reads).
__device__ __forceinline__ Decision decide(const VerifyParams &p, int32_t b) {
    Decision r;
    int32_t a = p.start[b], e = p.start[b + 1];
    a = a < 0 ? 0 : (a > p.num_drafts ? p.num_drafts : a);
    e = e < a ? a : (e > p.num_drafts ? p.num_drafts : e);
    r.d0 = a;
    r.n = e - a < p.max_drafts ? e - a : p.max_drafts;
    r.count = r.n;
    const int lane = threadIdx.x & 63;
    for (int32_t base = 0; base < r.n; base += 64) {
        const int32_t j = base + lane;
        bool refused = false;
        if (j < r.n) {
            const int64_t d = a + j;
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
            r.count = base + __builtin_ctzll(m);
            break;
        }
    }
    const int64_t d = int64_t(a) + r.count;
    r.p = p.p + (d + b) * p.p_sr;
    r.q = nullptr;
    r.out_token = -1;
    if (r.count < r.n) {
        if (p.q) r.q = p.q + d * p.q_sr;
        else r.out_token = p.draft_tokens[d];
    }
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
#pragma unroll 4
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
}

// Inclusive running sum over the workgroup's threads, in thread order.
__device__ __forceinline__ double block_scan(double v, double *part) {
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        const double o = __shfl_up(v, m);
        if (lane >= m) v += o;
    }
    __syncthreads();
    if (lane == 63) part[w] = v;
    __syncthreads();
    for (int i = 0; i < w; ++i) v += part[i];
    return v;
}

__global__ __launch_bounds__(kVfBlock) void verify_pick_kernel(VerifyParams p) {
    const int32_t b = int32_t(blockIdx.x), tid = int32_t(threadIdx.x);
    __shared__ double part[kVfBlock / 64];
    __shared__ int32_t hit, last;
    __shared__ double before;
    Decision d = decide(p, b);
    const double *sums = p.sums_ws + int64_t(b) * p.slices * 2;

    // which sums count: of the residual, or of p when nothing is left of it
    const int32_t per = (p.slices + kVfBlock - 1) / kVfBlock;
    const int32_t s0 = tid * per, s1 = s0 + per < p.slices ? s0 + per : p.slices;
    double t[2] = {0.0, 0.0};
    for (int32_t s = s0; s < s1; ++s) { t[0] += sums[2 * s]; t[1] += sums[2 * s + 1]; }
    const double c0 = block_scan(t[0], part);
    __shared__ double total;
    if (tid == kVfBlock - 1) total = c0;
    __syncthreads();
    const int which = total > 0.0 ? 0 : 1;
    __syncthreads();
    const double cum = which == 0 ? c0 : block_scan(t[1], part);
    if (which == 1) { d.q = nullptr; d.out_token = -1; }
    if (tid == 0) { hit = INT32_MAX; last = -1; }
    if (tid == kVfBlock - 1) total = cum;
    __syncthreads();
    const double goal = double(p.u_smp[b]) * total;

    // the first slice whose running sum exceeds the goal, else the last one with any mass
    {
        double c = cum - t[which];
        if (t[which] > 0.0) {
            for (int32_t s = s0; s < s1; ++s) {
                const double m = sums[2 * s + which];
                if (m > 0.0) atomicMax(&last, s);
                if (m > 0.0 && c + m > goal) { atomicMin(&hit, s); break; }
                c += m;
            }
        }
    }
    __syncthreads();
    const bool found = hit != INT32_MAX;
    const int32_t slice = found ? hit : last;
    if (slice >= s0 && slice < s1) {
        double c = cum - t[which];
        for (int32_t s = s0; s < slice; ++s) c += sums[2 * s + which];
        before = c;
    }
    __syncthreads();
    if (tid == 0) { hit = INT32_MAX; last = -1; }
    __syncthreads();
    if (slice >= 0) {
        // a thread takes consecutive entries, so thread order is index order
        const int32_t lo = slice * p.slice, hi = lo + p.slice < p.vocab ? lo + p.slice : p.vocab;
        const int32_t w = (p.slice + kVfBlock - 1) / kVfBlock;
        const int32_t i0 = lo + tid * w, i1 = i0 + w < hi ? i0 + w : hi;
        double m = 0.0;
        for (int32_t i = i0; i < i1; ++i) m += left_of(d, i, d.p[i], d.q ? d.q[i] : 0.0f);
        double c = before + (block_scan(m, part) - m);
        if (m > 0.0) {
            for (int32_t i = i0; i < i1; ++i) {
                const double x = left_of(d, i, d.p[i], d.q ? d.q[i] : 0.0f);
                if (x > 0.0) atomicMax(&last, i);
                c += x;
                if (x > 0.0 && c > goal) { atomicMin(&hit, i); break; }
            }
        }
        __syncthreads();
    }
    const int32_t token = slice < 0 ? 0 : (hit != INT32_MAX ? hit : last);
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
