// The group norm of a layer's output, channels last, with its gate or activation.
//
// Per row and group of channels, in fp32:
//   v = x act(z) (gate first) or x;  v -= mean(v) (layer);  v /= sqrt(mean(v^2) + eps);
//   v = v w + b;  v = v act(z) (gate last), act(v) (no gate), or v as it is (gate first)
// A group is held in registers between its one read and its one write, eight
// channels a thread at a time; the mean is taken out before the squares are
// summed, so nothing cancels.  Bound by its bytes: 14807 rows of 8 groups of 1024
// with a gate take 130 us, 5.6 TB/s, as a copy does; 256 rows of 32 groups of 128,
// in the caches, 3.8 us, the latency of two dependent loads and a launch.  A
// group of up to 2048 channels stays in one wave, whose sums need no barrier; rows of
// many small groups share a wave.
#include "gdr_device.h"
#include "sconv.h"
#include "ssm_params.h"

namespace sconv {

namespace {

constexpr int kWavesN = kNormBlock / 64;

__device__ __forceinline__ float activate(int a, float v) {
    if (a == SCONV_ACT_SILU) return act<true>(v);
    if (a == SCONV_ACT_SIGMOID) return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(v * -1.4426950408889634f));
    return v;
}

// Over the L threads of a group, in each of them.
template <int L>
__device__ __forceinline__ float sum_group(float v, float *part) {
    v = sum8(v);
    if constexpr (L >= 16) v = dpp_add<0x140>(v);      // row_mirror
    if constexpr (L >= 32) v += __shfl_xor(v, 16);
    if constexpr (L >= 64) v += __shfl_xor(v, 32);
    if constexpr (L > 64) {
        __syncthreads();               // (what the last sum read is no longer needed)
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
        __syncthreads();
        v = part[0];
#pragma unroll
        for (int i = 1; i < L / 64; ++i) v += part[i];
    }
    return v;
}

__device__ __forceinline__ void load_weights(const void *w, bool fp32, int64_t at, float (&f)[8]) {
    if (fp32) {
        const f32x4 *q = reinterpret_cast<const f32x4 *>(static_cast<const float *>(w) + at);
        const f32x4 a = q[0], b = q[1];
#pragma unroll
        for (int i = 0; i < 4; ++i) { f[i] = a[i]; f[4 + i] = b[i]; }
    } else {
        unpack8(ld16(static_cast<const uint16_t *>(w) + at), f);
    }
}

// L threads a group, K pieces of eight channels a thread.
template <int L, int K, bool GATE>
__global__ __launch_bounds__(kNormBlock) void group_norm_kernel(NormParams p, int64_t n) {
    __shared__ float part[kWavesN];
    const int64_t id = (int64_t(blockIdx.x) * kNormBlock + threadIdx.x) / L;
    const int lane = threadIdx.x & (L - 1);
    if (L <= 64 && id >= n) return;    // (whole lane groups)
    const int64_t row = id / p.groups;
    const int32_t g = int32_t(id - row * p.groups);
    const uint16_t *x = p.x + row * p.x_sr + g * p.x_sg;
    const uint16_t *z = GATE ? p.z + row * p.z_sr + g * p.z_sg : nullptr;
    u32x4 xr[K], zr[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = 8 * (L * k + lane);
        xr[k] = u32x4{0, 0, 0, 0};
        zr[k] = u32x4{0, 0, 0, 0};
        if (c < p.size) {
            xr[k] = ld16(x + c);
            if (GATE) zr[k] = ld16(z + c);
        }
    }
    float v[K][8];
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        unpack8(xr[k], v[k]);
        if (GATE && p.gate_first) {
            float f[8];
            unpack8(zr[k], f);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[k][i] *= activate(p.act, f[i]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) s += v[k][i];
    }
    const float inv_n = 1.0f / float(p.size);
    if (p.layer) {
        const float mean = sum_group<L>(s, part) * inv_n;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const bool in = 8 * (L * k + lane) < p.size;
#pragma unroll
            for (int i = 0; i < 8; ++i) v[k][i] = in ? v[k][i] - mean : 0.0f;
        }
    }
    float q = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) q = fmaf(v[k][i], v[k][i], q);
    const float r = 1.0f / sqrtf(sum_group<L>(q, part) * inv_n + p.eps);
    uint16_t *o = p.out + row * p.o_sr + g * p.o_sg;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = 8 * (L * k + lane);
        if (c >= p.size) continue;
        float w[8], f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[k][i] *= r;
        if (p.w) {
            load_weights(p.w, p.w_fp32, g * p.w_sg + c, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[k][i] *= w[i];
        }
        if (p.b) {
            load_weights(p.b, p.w_fp32, g * p.b_sg + c, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[k][i] += w[i];
        }
        if (GATE) {
            if (!p.gate_first) {
                unpack8(zr[k], f);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[k][i] *= activate(p.act, f[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[k][i] = activate(p.act, v[k][i]);
        }
        st16(o + c, pack8(v[k]));
    }
}

// Any strides and sizes: a workgroup a group, which reads it once for the mean, once for the squares and once for the result.
__global__ __launch_bounds__(kNormBlock) void group_norm_any_kernel(NormParams p) {
    __shared__ float part[kWavesN];
    const int64_t row = blockIdx.x / uint32_t(p.groups);
    const int32_t g = int32_t(blockIdx.x - uint32_t(row) * uint32_t(p.groups));
    const uint16_t *x = p.x + row * p.x_sr + g * p.x_sg;
    const uint16_t *z = p.z ? p.z + row * p.z_sr + g * p.z_sg : nullptr;
    const auto value = [&](int64_t c) {
        const float v = bf_one(x[c * p.x_sc]);
        return p.gate_first ? v * activate(p.act, bf_one(z[c * p.z_sc])) : v;
    };
    const auto weight = [&](const void *w, int64_t at) {
        return p.w_fp32 ? static_cast<const float *>(w)[at] : bf_one(static_cast<const uint16_t *>(w)[at]);
    };
    const float inv_n = 1.0f / float(p.size);
    float mean = 0.0f, q = 0.0f;
    if (p.layer) {
        float s = 0.0f;
        for (int64_t c = threadIdx.x; c < p.size; c += kNormBlock) s += value(c);
        mean = sum_group<kNormBlock>(s, part) * inv_n;
    }
    for (int64_t c = threadIdx.x; c < p.size; c += kNormBlock) {
        const float v = value(c) - mean;
        q = fmaf(v, v, q);
    }
    const float r = 1.0f / sqrtf(sum_group<kNormBlock>(q, part) * inv_n + p.eps);
    uint16_t *o = p.out + row * p.o_sr + g * p.o_sg;
    for (int64_t c = threadIdx.x; c < p.size; c += kNormBlock) {
        float v = (value(c) - mean) * r;
        if (p.w) v *= weight(p.w, g * p.w_sg + c);
        if (p.b) v += weight(p.b, g * p.b_sg + c);
        if (!p.z) v = activate(p.act, v);
        else if (!p.gate_first) v *= activate(p.act, bf_one(z[c * p.z_sc]));
        o[c * p.o_sc] = to_bf16(v);
    }
}

template <int L, int K>
hipError_t launch_vec(const NormParams &p, hipStream_t s) {
    const int64_t n = p.rows * p.groups;
    const dim3 grid(uint32_t((n * L + kNormBlock - 1) / kNormBlock)), block(kNormBlock);
    if (p.z) group_norm_kernel<L, K, true><<<grid, block, 0, s>>>(p, n);
    else group_norm_kernel<L, K, false><<<grid, block, 0, s>>>(p, n);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_group_norm(const NormParams &p, bool vec, hipStream_t s) {
    if (!vec) {
        group_norm_any_kernel<<<dim3(uint32_t(p.rows * p.groups)), dim3(kNormBlock), 0, s>>>(p);
        return hipGetLastError();
    }
    switch (norm_threads(p.size)) {
        case 8: return launch_vec<8, 1>(p, s);
        case 16: return launch_vec<16, 1>(p, s);
        case 32: return launch_vec<32, 1>(p, s);
        case 64:
            if (p.size <= 512) return launch_vec<64, 1>(p, s);
            return p.size <= 1024 ? launch_vec<64, 2>(p, s) : launch_vec<64, 4>(p, s);
        default:
            return p.size <= 4096 ? launch_vec<kNormBlock, 2>(p, s)
                                  : (p.size <= 8192 ? launch_vec<kNormBlock, 4>(p, s) : launch_vec<kNormBlock, 8>(p, s));
    }
}

}  // namespace sconv
