// What the kernels of the operators in cbk_nn.h and cbk_moe.h share: rounding, activations, copies into LDS,
// and the arguments of the product that decodes on the way (cbk_nn_fused.h).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "cbk_device.h"

#define CBK_LDS __attribute__((address_space(3)))

namespace cbk {

constexpr uint32_t kFusedTile = 128;  // columns of a tile of k_fused

struct FusedTensor {
    const uint32_t *words;
    const uint16_t *cb;
    uint64_t bytes;  // of the index stream
    uint32_t U, pad;
};

// C[m][n] for M <= 384 tokens: see cbk_nn_fused.h.
struct FusedArgs {
    FusedTensor t[2];
    uint32_t count;            // 1, or 2: a gate and up pair
    const uint16_t *A;         // tokens' side, [M][lda]; 64 * slices columns are readable (gradient: for each tensor)
    uint64_t lda;
    uint32_t M;
    uint64_t row0;             // the piece's first row of the tensors, and how many rows it has
    uint32_t nrows;
    uint32_t cols;             // of the tensors
    uint32_t tiles, slices;    // of one tensor
    float *part;               // [grid + count * tiles][M][kFusedTile]
    uint32_t grid;
};

// bm: 16, 64, 128, 192, 256, 320 or 384, at least M.  B: 8 to 14.
template <int B>
cbk_status launch_fused(const FusedArgs &a, uint32_t bm, bool nn, hipStream_t s);

namespace {

typedef uint32_t u32x3 __attribute__((ext_vector_type(3)));

// a / b, by the short division where it is enough (it nearly always is; the long one takes a microsecond).
__device__ __forceinline__ uint64_t quotient(uint64_t a, uint64_t b) {
    if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}

// fp32 to BF16, to nearest even (NaN stays NaN).
__device__ __forceinline__ uint16_t to_bf16(float v) { return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v)); }
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    return static_cast<uint32_t>(to_bf16(a)) | (static_cast<uint32_t>(to_bf16(b)) << 16);
}

// act(z) and, where D is not null, act'(z), in fp32.  The tails are formed without subtractions
// of nearly equal numbers: 1 - tanh and 1 - erf come from a logistic function and from erfc.
__device__ __forceinline__ float activation(int act, float z, float *D) {
    if (act == CBK_ACT_SILU) {
        const float s = 1.f / (1.f + __expf(-z));
        if (D) *D = s * (1.f + z * (1.f - s));
        return z * s;
    }
    if (act == CBK_ACT_GELU) {
        const float p = 0.5f * erfcf(z * -0.70710678118654752f);
        if (D) *D = p + z * 0.39894228040143268f * __expf(-0.5f * z * z);
        return z * p;
    }
    // (1 + tanh(y)) / 2 = 1 / (1 + exp(-2 y)); past |z| = 16 it is 0 or 1 to every bit and z^3 might overflow
    const float c = 1.5957691216057308f;  // 2 sqrt(2 / pi)
    const float w = z > 16.f ? 16.f : z < -16.f ? -16.f : z;  // NaN stays NaN, where fmaxf and fminf would drop it
    const float s = 1.f / (1.f + __expf(-c * (w + 0.044715f * w * w * w)));
    if (D) *D = s + w * s * (1.f - s) * c * (1.f + 3.f * 0.044715f * w * w);
    return z * s;
}

// Copies 16 bytes a lane from the resource (at the lane's voff plus the wave's soff) straight into
// LDS, lane l to dst + 16 l; dst is the same in every lane.  The wave's vmcnt counts it.  The
// host's pass over this file does not know this chip's wide copies, so it gets an empty body.
__device__ __forceinline__ void copy_to_lds(__amdgpu_buffer_rsrc_t rs, unsigned char *dst, uint32_t voff, uint32_t soff) {
#ifdef __HIP_DEVICE_COMPILE__
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (CBK_LDS void *)(dst), 16, static_cast<int>(voff), static_cast<int>(soff), 0, 0);
#endif
}

}  // namespace
}  // namespace cbk
