// Device helpers of the gated delta rule kernels.
#pragma once

#include "gdr_params.h"
#include "sconv_device.h"

namespace sconv {

typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr float kL2Eps = 1e-6f;        // added to a head's sum of squares before its root

// Sum over the 8 lanes of an aligned group, in every one of them: two quad
// permutations, then the mirrored half row (each quad holds one value by then).
template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
    return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(
                                             0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float sum8(float v) {
    v = dpp_add<0xB1>(v);              // quad_perm [1,0,3,2]
    v = dpp_add<0x4E>(v);              // quad_perm [2,3,0,1]
    return dpp_add<0x141>(v);          // row_half_mirror
}

// Log decay and write strength of value head h at element offsets go / bo of
// the two gate tensors.  Given ones are fp32; raw ones are the layer's bf16
// projections: g = -exp(A_log) softplus(a + dt_bias), beta = sigmoid(b).  A
// decay above 0 counts as 0 (NaN stays).
struct Gates { float g, beta; };
__device__ __forceinline__ Gates gdr_gates(const GdrParams &p, int64_t go, int64_t bo, int32_t h) {
    Gates r;
    if (p.raw) {
        const float x = bf_one(static_cast<const uint16_t *>(p.gate)[go]) + p.dt_bias[h];
        const float b = bf_one(static_cast<const uint16_t *>(p.beta)[bo]);
        const float sp = x > 20.0f ? x : log1pf(expf(x));
        r.g = -expf(p.a_log[h]) * sp;
        r.beta = 1.0f / (1.0f + expf(-b));
    } else {
        r.g = static_cast<const float *>(p.gate)[go];
        r.beta = static_cast<const float *>(p.beta)[bo];
    }
    r.g = r.g > 0.0f ? 0.0f : r.g;
    return r;
}

}  // namespace sconv
