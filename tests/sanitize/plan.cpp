// Host-only driver for tests/test_nn_plan.py: how a call of an operator in cbk_nn.h is cut up.  Each line
// of its input is "op rows cols b1 b2 tokens" (op 0 linear, 1 the gated block, 2 cross entropy; b2 for
// the block's second tensor); it answers with a line "fused grid pieces rows in_order bytes": in_order is 1
// where every piece of every tensor can be decoded in the stream's own order.
#include <stdio.h>
#include <stdlib.h>

#include <algorithm>

#include "cbk_internal.h"

namespace cbk {
namespace {
[[noreturn]] void reached() {
    fprintf(stderr, "a launcher was reached in the host-only build\n");
    abort();
}
}  // namespace
cbk_status launch_linear(const cbk_tensor &, const uint16_t *, uint64_t, uint64_t, uint16_t *, uint64_t, void *, hipStream_t) {
    reached();
}
cbk_status launch_linear_dx(const cbk_tensor &, const uint16_t *, uint64_t, uint64_t, uint16_t *, uint64_t, void *, hipStream_t) {
    reached();
}
cbk_status launch_ffn(const cbk_tensor &, const cbk_tensor &, int, const uint16_t *, uint64_t, uint64_t, uint16_t *, uint64_t,
                      void *, hipStream_t) {
    reached();
}
cbk_status launch_ffn_bwd(const cbk_tensor &, const cbk_tensor &, int, const uint16_t *, uint64_t, const uint16_t *, uint64_t,
                          uint64_t, uint16_t *, uint64_t, uint16_t *, uint16_t *, uint64_t, void *, hipStream_t) {
    reached();
}
cbk_status launch_xent(const cbk_tensor &, const uint16_t *, uint64_t, const int64_t *, uint64_t, int64_t, float *, float *,
                       void *, hipStream_t) {
    reached();
}
cbk_status launch_xent_bwd(const cbk_tensor &, const uint16_t *, uint64_t, const int64_t *, const float *, const float *,
                           uint64_t, int64_t, uint16_t *, uint64_t, void *, hipStream_t) {
    reached();
}
}  // namespace cbk

int main() {
    int op;
    unsigned long long rows, cols, b1, b2, tokens;
    const uint16_t *codebook = reinterpret_cast<const uint16_t *>(0x10000);
    const uint32_t *words = reinterpret_cast<const uint32_t *>(0x10000);
    while (scanf("%d %llu %llu %llu %llu %llu", &op, &rows, &cols, &b1, &b2, &tokens) == 6) {
        auto tensor = [&](unsigned long long b) {
            return cbk_tensor{rows, cols, uint32_t(1) << b, static_cast<uint32_t>(b), codebook, words};
        };
        const cbk_tensor t[2] = {tensor(b1), tensor(b2)};
        const cbk_tensor *ts[2] = {&t[0], &t[1]};
        const cbk::NnPlan p = cbk::nn_plan(static_cast<cbk::NnOp>(op), ts, tokens);
        bool in_order = true;
        for (uint64_t r = 0; r < rows; r += p.rows)
            for (int i = 0; i < (op == 1 ? 2 : 1); ++i)
                in_order = in_order && cbk::nn_unpack_in_order(t[i], r, std::min<uint64_t>(p.rows, rows - r));
        printf("%u %u %llu %llu %d %llu\n", p.fused, p.grid, static_cast<unsigned long long>(p.pieces),
               static_cast<unsigned long long>(p.rows), in_order ? 1 : 0, static_cast<unsigned long long>(p.bytes));
    }
    return 0;
}
