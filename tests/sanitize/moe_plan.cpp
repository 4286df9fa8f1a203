// Host-only driver for tests/test_moe_plan.py: how a call on a block of experts (cbk_moe.h) is cut up.  Each line of its
// input is "rows cols out count b b_down tokens k backward"; it answers with the plan's numbers: tokens of a chunk, slots of a
// tile, tiles, one, shares of the three reductions, parts of a dweight, floats between the shares of S and of D, then the offsets
// of tiles, token_of, slot_of, place_of, xpack, ypack, h, g, s, d and dw in the workspace, and its bytes.
// Before that the calls of cbk_moe.h and cbk_sample.h get arguments that they have to refuse.
#include <stdio.h>
#include <stdlib.h>

#include "cbk_internal.h"

namespace cbk {
namespace {
[[noreturn]] void reached() {
    fprintf(stderr, "a launcher was reached in the host-only build\n");
    abort();
}
void expect(cbk_status got, cbk_status want, const char *what) {
    if (got == want) return;
    fprintf(stderr, "%s: status %d, not %d\n", what, got, want);
    abort();
}
}  // namespace
cbk_status launch_route(const cbk_router &, const void *, int, uint64_t, uint64_t, const float *, int32_t *, float *, hipStream_t) {
    reached();
}
cbk_status launch_route_bwd(const cbk_router &, const void *, int, uint64_t, uint64_t, const int32_t *, const float *, void *,
                            uint64_t, hipStream_t) {
    reached();
}
cbk_status launch_sample(const cbk_sampling &, const void *, int, uint64_t, uint64_t, uint64_t, const float *, int64_t *, float *,
                         const SamplePlan &, void *, hipStream_t) {
    reached();
}
cbk_status launch_experts(const cbk_experts &, const ExPlan &, int, const uint16_t *, uint64_t, uint64_t, const int32_t *,
                          const float *, uint32_t, const uint16_t *, uint64_t, uint16_t *, uint64_t, float *, void *, hipStream_t) {
    reached();
}
cbk_status experts_table(const cbk_tensor *, const cbk_tensor *, const cbk_tensor *, uint32_t, void *, uint32_t &device) {
    device = 0;
    return CBK_OK;
}
}  // namespace cbk

namespace {

template <typename T>
T *address() { return reinterpret_cast<T *>(0x10000); }

void refusals() {
    using cbk::expect;
    float *f = address<float>();
    int32_t *i = address<int32_t>();
    uint16_t *h = address<uint16_t>();
    int64_t *l = address<int64_t>();
    cbk_router r{16, 4, CBK_SCORE_SOFTMAX, 1, 1.f, 1, 1, 1};
    expect(cbk_route(&r, f, CBK_F32, 16, 0, nullptr, i, f, nullptr), CBK_OK, "no tokens");
    expect(cbk_route(nullptr, f, CBK_F32, 16, 1, nullptr, i, f, nullptr), CBK_E_INVALID, "no router");
    expect(cbk_route(&r, f, CBK_F32, 15, 1, nullptr, i, f, nullptr), CBK_E_INVALID, "ld");
    expect(cbk_route(&r, f, CBK_F32, ~uint64_t(0), 1, nullptr, i, f, nullptr), CBK_E_UNSUPPORTED, "long ld");
    expect(cbk_route_bwd(&r, f, CBK_F32, 16, ~uint64_t(0), i, f, f, 16, nullptr), CBK_E_UNSUPPORTED, "many tokens");
    cbk_experts ex{h, 256, 128, 192, 8, 12, 13, 0};
    expect(cbk_ffn_experts(&ex, CBK_ACT_SILU, h, 128, 5, i, f, 2, h, 192, h, 1, nullptr), CBK_E_CAPACITY, "workspace");
    expect(cbk_ffn_experts(nullptr, CBK_ACT_SILU, h, 128, 5, i, f, 2, h, 192, h, 1, nullptr), CBK_E_INVALID, "no experts");
    expect(cbk_ffn_experts_bwd(&ex, CBK_ACT_SILU, h, 128, 5, i, f, 65, h, 192, h, 128, f, h, 1, nullptr), CBK_E_UNSUPPORTED, "k");
    expect(cbk_ffn_experts_bwd(&ex, 9, h, 128, 5, i, f, 2, h, 192, h, 128, f, h, 1, nullptr), CBK_E_INVALID, "act");
    cbk_sampling p{1.f, 0.9f, 0.f, 50, nullptr, nullptr, nullptr, nullptr};
    expect(cbk_sample(&p, f, CBK_F32, 1 << 20, 1 << 20, 3, f, l, nullptr, h, 1, nullptr), CBK_E_CAPACITY, "draw's workspace");
    expect(cbk_sample(&p, f, CBK_F32, 5, 0, 3, f, l, nullptr, h, 1, nullptr), CBK_E_INVALID, "no vocabulary");
    expect(cbk_sample(&p, f, CBK_F32, 5, 5, 3, nullptr, l, nullptr, nullptr, 0, nullptr), CBK_E_INVALID, "no uniform");
    // tables of up to 1024 experts, each read once
    const cbk_tensor up{64, 32, 300, 9, h, address<uint32_t>()}, down{48, 64, 9, 4, h, address<uint32_t>()};
    for (uint32_t n = 1; n <= 1024; n += 1023) {
        cbk_tensor *gates = new cbk_tensor[n], *downs = new cbk_tensor[n];
        for (uint32_t e = 0; e < n; ++e) {
            gates[e] = up;
            downs[e] = down;
        }
        cbk_experts made{};
        expect(cbk_experts_init(gates, gates, downs, n, h, cbk_experts_bytes(n), &made), CBK_OK, "table");
        if (made.count != n || made.b != 9 || made.b_down != 4 || made.rows != 64 || made.cols != 32 || made.out != 48) abort();
        expect(cbk_experts_init(gates, gates, downs, n, h, cbk_experts_bytes(n) - 1, &made), CBK_E_CAPACITY, "short table");
        expect(cbk_experts_init(gates, downs, downs, n, h, cbk_experts_bytes(n), &made), CBK_E_INVALID, "shapes");
        delete[] gates;
        delete[] downs;
    }
}

}  // namespace

int main() {
    refusals();
    unsigned long long rows, cols, out, tokens;
    unsigned count, b, b_down, k;
    int backward;
    while (scanf("%llu %llu %llu %u %u %u %llu %u %d", &rows, &cols, &out, &count, &b, &b_down, &tokens, &k, &backward) == 9) {
        const cbk_experts ex{address<uint16_t>(), rows, cols, out, count, b, b_down, 0};
        const cbk::ExPlan p = cbk::ex_plan(ex, tokens, k, backward != 0);
        if (cbk_experts_workspace_bytes(&ex, tokens, k, backward) != p.bytes) abort();
        const uint64_t numbers[] = {p.Tc, p.tile, p.max_tiles, p.one, p.split_down, p.split_dt, p.split_x, p.dw_parts, p.s_stride, p.d_stride,
                                    p.tiles, p.token_of, p.slot_of, p.place_of, p.xpack, p.ypack, p.h, p.g, p.s, p.d, p.dw, p.bytes};
        for (uint64_t n : numbers) printf("%llu ", static_cast<unsigned long long>(n));
        printf("\n");
    }
    return 0;
}
