// Internal interface between the host API (cbk_api.cpp, cbk_ec_host.cpp, cbk_nn_host.cpp,
// cbk_moe_host.cpp) and the HIP launchers (cbk_kernels.hip, cbk_encode.hip, cbk_ec.hip, cbk_nn.hip, cbk_moe.hip,
// cbk_sample.hip).
// Arguments reaching these launchers are already validated.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/cbk.h"
#include "../../include/cbk_ec.h"
#include "../../include/cbk_nn.h"
#include "../../include/cbk_moe.h"
#include "../../include/cbk_sample.h"

namespace cbk {

cbk_status check_tensor(const cbk_tensor *t);  // cbk_api.cpp

cbk_status launch_decode(const cbk_tensor &t, uint16_t *out, hipStream_t s);
cbk_status launch_decode_group(const cbk_tensor *ts, uint32_t count, uint16_t *const *outs, hipStream_t s);
cbk_status launch_gemv(const cbk_tensor &t, const uint16_t *x, float *y, hipStream_t s);
cbk_status launch_gemv_group(const cbk_tensor *ts, uint32_t count, const uint16_t *x,
                             float *const *ys, hipStream_t s);
// Chained GEMV phases (validated by cbk_gemv_chain_init).
size_t gemv_chain_bytes(uint32_t phases);
cbk_status build_gemv_chain(const cbk_gemv_phase *phases, uint32_t count, void *buffer, cbk_gemv_chain *chain);
cbk_status launch_gemv_chain(const cbk_gemv_chain &chain, uint32_t timeout_us, hipStream_t s);
cbk_status gemv_chain_check(const cbk_gemv_chain &chain);
cbk_status launch_gemm(const cbk_tensor &t, const uint16_t *X, uint64_t ldx, uint32_t batch,
                       float *Y, uint64_t ldy, hipStream_t s);
cbk_status launch_gemm_group(const cbk_tensor *ts, uint32_t count, const uint16_t *X, uint64_t ldx,
                             uint32_t batch, float *const *Ys, const uint64_t *ldys, hipStream_t s);

// GPU encoder (cbk_encode.hip).
size_t encode_gpu_workspace_bytes();
// count jobs, in runs of up to 8 (each run uses the first min(count, 8) workspaces of
// encode_gpu_workspace_bytes() bytes).
cbk_status launch_encode_gpu(const cbk_encode_job *jobs, uint32_t count, void *workspace, hipStream_t s);
// Device address of the library's static encoder scratch on the current device (a workspace of
// encode_gpu_workspace_bytes() bytes); looked up on the device's first call.
cbk_status encode_gpu_scratch(void **ws);

// Exponent entropy-coded format (cbk_ec.hip), count tensors in launches of up to 8.
// indexes: each tensor's span index (cbk_ec_build_index), or null for the two-walk decode.
cbk_status launch_ec_decode(const cbk_ec_tensor *ts, const uint8_t *const *indexes, uint32_t count,
                            uint16_t *const *outs, hipStream_t s);
// rows[i] * cols = ts[i].n; every y is zero-filled first (rows[i] > 0), x is read when cols > 0.
cbk_status launch_ec_gemv(const cbk_ec_tensor *ts, const uint8_t *const *indexes, uint32_t count,
                          const uint64_t *rows, uint64_t cols, const uint16_t *x, float *const *ys, hipStream_t s);
cbk_status launch_ec_index(const cbk_ec_tensor *t, uint8_t *index, hipStream_t s);

// Operators on any number of tokens (cbk_nn.hip).  A plan says how a call is cut up and where its
// scratch lies in the workspace; it depends on the tensors and the number of tokens alone, so that
// the workspace's size is known without a GPU.  Tokens are taken Tc at a time, the rows of the
// tensors in pieces.
struct NnPlan {
    uint64_t Kp;      // columns of a decoded row in the workspace: cols rounded up to 64, at least 64
    uint64_t Tc;      // tokens of a chunk
    uint64_t rows;    // rows of one tensor in a piece
    uint64_t Rp;      // columns of a piece's gradients (those of both tensors, for the feed-forward block)
    uint64_t pieces;
    uint32_t fused;   // 0: pieces are decoded into memory; else the token tile of k_fused
    uint32_t grid;    // k_fused: most workgroups
    uint32_t split;   // k_fused: a launch for each tensor of the pair
    // part: the parts of tiles whose slices several workgroups share
    uint64_t pack, w, part, g, acc, stat, top;  // offsets in bytes
    uint64_t bytes;
};
enum class NnOp { linear, ffn, xent };
NnPlan nn_plan(NnOp op, const cbk_tensor *const *ts, uint64_t tokens);
// Most tiles whose slices the workgroups of k_mm share, of 256 x 256 sums each.
constexpr uint32_t kMmShared = 160;
// Slices in k_fused's ring, and a workgroup's LDS: the table, and the slices of the tokens and of the weights.  A
// ring of three where the LDS has room for it (not past 256 tokens, nor with 193 to 256 and 14 bits), else two
// (200 tokens, 14 bits, 11008 x 4096: 51 us, 103 if the tensor is decoded first; 192 tokens and three 45).
constexpr uint32_t nn_ring_lds(uint32_t b, uint32_t bm, uint32_t ring) { return (2u << b) + ring * 128 * (bm + 128); }
constexpr uint32_t nn_fused_ring(uint32_t b, uint32_t bm) { return nn_ring_lds(b, bm, 3) <= 160 * 1024 ? 3 : 2; }
constexpr uint32_t nn_fused_lds(uint32_t b, uint32_t bm) { return nn_ring_lds(b, bm, nn_fused_ring(b, bm)); }
// Whether rows [row0, row0 + nrows) of a tensor can be decoded in the stream's own order (k_unpack).
bool nn_unpack_in_order(const cbk_tensor &t, uint64_t row0, uint64_t nrows);

cbk_status launch_linear(const cbk_tensor &t, const uint16_t *X, uint64_t ldx, uint64_t T, uint16_t *Y, uint64_t ldy,
                         void *ws, hipStream_t s);
cbk_status launch_linear_dx(const cbk_tensor &t, const uint16_t *dY, uint64_t lddy, uint64_t T, uint16_t *dX,
                            uint64_t lddx, void *ws, hipStream_t s);
cbk_status launch_ffn(const cbk_tensor &gate, const cbk_tensor &up, int act, const uint16_t *X, uint64_t ldx, uint64_t T,
                      uint16_t *H, uint64_t ldh, void *ws, hipStream_t s);
cbk_status launch_ffn_bwd(const cbk_tensor &gate, const cbk_tensor &up, int act, const uint16_t *X, uint64_t ldx,
                          const uint16_t *dH, uint64_t lddh, uint64_t T, uint16_t *dX, uint64_t lddx, uint16_t *dG,
                          uint16_t *dU, uint64_t ldg, void *ws, hipStream_t s);
cbk_status launch_xent(const cbk_tensor &head, const uint16_t *X, uint64_t ldx, const int64_t *labels, uint64_t T,
                       int64_t ignore, float *loss, float *lse, void *ws, hipStream_t s);
cbk_status launch_xent_bwd(const cbk_tensor &head, const uint16_t *X, uint64_t ldx, const int64_t *labels,
                           const float *lse, const float *dloss, uint64_t T, int64_t ignore, uint16_t *dX,
                           uint64_t lddx, void *ws, hipStream_t s);

// Routing (cbk_moe.hip) and drawing (cbk_sample.hip).
cbk_status launch_route(const cbk_router &r, const void *logits, int dtype, uint64_t ld, uint64_t tokens, const float *bias,
                        int32_t *experts, float *weights, hipStream_t s);
cbk_status launch_route_bwd(const cbk_router &r, const void *logits, int dtype, uint64_t ld, uint64_t tokens,
                            const int32_t *experts, const float *dweights, void *dlogits, uint64_t ldd, hipStream_t s);
// How a call of cbk_sample is done: rows of a launch; a row's segments (0: a workgroup does all of a row); whether there
// are filters to divide the work of; and where the parts' scratch lies, which begins with the segments' records.
constexpr uint32_t kSamplePartBytes = 16, kSampleSegment = 1024, kSampleBins = 2048;
struct SamplePlan {
    uint64_t rows, bytes;
    uint32_t segments;
    bool divided;
    uint64_t sums, bins, list, state;
};
cbk_status launch_sample(const cbk_sampling &p, const void *logits, int dtype, uint64_t ld, uint64_t V, uint64_t tokens,
                         const float *uniform, int64_t *token, float *logprob, const SamplePlan &pl, void *ws, hipStream_t s);

// Blocks of experts (cbk_moe.hip, cbk_moe_mm.hip).  As for NnPlan, a plan depends on the shapes and the number of
// tokens alone.  Tokens are taken Tc at a time; a token's k slots are sorted by expert.
struct ExPlan {
    uint64_t Tc;
    uint64_t Kp, Fp, Op;     // cols, rows and out rounded up to 64
    uint64_t ldK, ldF, ldO;  // and to a tile's 128 columns: leading dimensions of fp32 results
    uint32_t tile;           // slots of one expert that a workgroup takes at most
    uint32_t max_tiles;      // token tiles of a chunk, at most
    uint32_t one;            // one token forward: its slots are not sorted
    uint32_t split_down, split_dt, split_x;  // workgroups that share a reduction
    uint32_t dw_parts;       // partial sums of a slot's dweights
    uint64_t s_stride, d_stride;  // floats between the shares of a reduction
    // offsets in bytes
    uint64_t ntiles, tiles, token_of, slot_of, place_of, xpack, ypack, h, g, s, d, dw;
    uint64_t bytes;
};
ExPlan ex_plan(const cbk_experts &ex, uint64_t tokens, uint32_t k, bool backward);
// Fills the table at `buffer` (three runs of `count` records) and names the device.
cbk_status experts_table(const cbk_tensor *gate, const cbk_tensor *up, const cbk_tensor *down, uint32_t count, void *buffer,
                         uint32_t &device);
constexpr uint64_t kExTensorBytes = 32;
// Forward where dY is null (out: Y), else the gradient (out: dX).
cbk_status launch_experts(const cbk_experts &ex, const ExPlan &pl, int act, const uint16_t *X, uint64_t ldx, uint64_t T,
                          const int32_t *experts, const float *weights, uint32_t k, const uint16_t *dY, uint64_t lddy,
                          uint16_t *out, uint64_t ldo, float *dweights, void *ws, hipStream_t s);

}  // namespace cbk
