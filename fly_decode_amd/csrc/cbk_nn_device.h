// What the kernels of the operators in cbk_nn.h share (cbk_nn.hip, cbk_nn_fused.h): copies into LDS,
// and the arguments of the product that decodes on the way.
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
