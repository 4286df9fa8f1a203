// What the kernels of cbk_moe.h share (cbk_moe.hip, cbk_moe_mm.hip).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "cbk_nn_device.h"

namespace cbk {

// A record of the table that cbk_experts_init makes: gate, up and down of every expert, kind by kind.
struct ExTensor {
    const uint32_t *words;
    const uint16_t *cb;
    uint64_t bytes;  // of the index stream
    uint32_t U, b;
};
static_assert(sizeof(ExTensor) == kExTensorBytes, "cbk_experts_bytes counts with it");

// Slots [start, start + count) of the sorted order, all of one expert.
struct ExTile {
    uint32_t expert, start, count, pad;
};

// A product of the experts' weights with their tokens, and what becomes of it.
struct ExArgs {
    const ExTensor *t[2];      // by expert: one tensor, or gate and up
    const ExTile *tiles;
    const uint32_t *ntiles;
    const uint32_t *token_of;  // of a sorted slot
    const uint32_t *slot_of;
    const int32_t *experts;    // of one token's k slots
    uint32_t k, count;         // experts that there are
    const uint16_t *A;         // rows by token, or (by_slot) by sorted slot
    uint32_t lda, by_slot;
    uint32_t N, R;             // columns of the result and terms of a sum (of one tensor), as the tensors have them
    uint32_t col_tiles, slices, splits;
    uint32_t table;            // bytes of a codebook's table in LDS
    uint32_t ldS;
    uint64_t split_stride;
    float *S;                  // sums: [splits][slots][ldS]
    const float *weights;      // by slot
    uint32_t scaled;           // sums are multiplied by their slot's weight
    int act;
    uint32_t rows, Fp;         // hidden width, and rounded up to 64
    uint16_t *H;               // [slots][Fp]
    const float *D;            // [d_splits][slots][ldD]
    uint32_t ldD, d_splits;
    uint64_t d_stride;
    uint16_t *G;               // [slots][2 Fp]: dG, dU
    float *dw;                 // [slots][dw_parts]
    uint32_t dw_parts;
};

// The products.  Each fills in what its shape and the plan decide.
cbk_status ex_hidden(ExArgs &a, const ExPlan &pl, const cbk_experts &ex, bool backward, hipStream_t s);
cbk_status ex_down(ExArgs &a, const ExPlan &pl, const cbk_experts &ex, hipStream_t s);
cbk_status ex_down_t(ExArgs &a, const ExPlan &pl, const cbk_experts &ex, hipStream_t s);
cbk_status ex_dx(ExArgs &a, const ExPlan &pl, const cbk_experts &ex, hipStream_t s);

}  // namespace cbk
