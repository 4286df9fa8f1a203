// Host half of cbk_moe.h and cbk_sample.h: argument validation, and how a call on a block of experts is cut up and laid
// out in its workspace.  Nothing here touches the GPU until every argument has been checked.
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "cbk_internal.h"

namespace {

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline uint64_t up_to(uint64_t n, uint64_t m) { return (n + m - 1) / m * m; }

constexpr uint64_t kMaxTokens = uint64_t(1) << 31;
constexpr uint64_t kMaxLd = uint64_t(1) << 32;
constexpr uint64_t kMaxWidth = uint64_t(1) << 20;
constexpr uint32_t kMaxExperts = 1024, kMaxChosen = 64;

cbk_status check_router(const cbk_router *r) {
    if (!r || r->experts == 0 || r->k == 0 || r->k > r->experts) return CBK_E_INVALID;
    if (r->score != CBK_SCORE_SOFTMAX && r->score != CBK_SCORE_SIGMOID) return CBK_E_INVALID;
    if (r->groups == 0 || r->experts % r->groups != 0 || r->top_groups == 0 || r->top_groups > r->groups) return CBK_E_INVALID;
    if (r->group_top != 1 && r->group_top != 2) return CBK_E_INVALID;
    if (r->experts > kMaxExperts || r->k > kMaxChosen) return CBK_E_UNSUPPORTED;
    return CBK_OK;
}

// A matrix of fp32 or BF16 rows.
cbk_status check_rows(const void *p, int dtype, uint64_t ld, uint64_t width) {
    if (dtype != CBK_F32 && dtype != CBK_BF16) return CBK_E_INVALID;
    if (!p || ld < width) return CBK_E_INVALID;
    if (!aligned(p, dtype == CBK_F32 ? 4 : 2)) return CBK_E_ALIGN;
    if (ld >= kMaxLd) return CBK_E_UNSUPPORTED;
    return CBK_OK;
}

cbk_status check_experts(const cbk_experts *ex) {
    if (!ex || !ex->buffer || ex->count == 0 || ex->count > kMaxExperts) return CBK_E_INVALID;
    if (ex->rows == 0 || ex->cols == 0 || ex->out == 0 || ex->b > 16 || ex->b_down > 16) return CBK_E_INVALID;
    if (ex->rows > kMaxWidth || ex->cols > kMaxWidth || ex->out > kMaxWidth) return CBK_E_UNSUPPORTED;
    return CBK_OK;
}

cbk_status check_call(const cbk_experts *ex, int act, const int32_t *experts, const float *weights, const uint16_t *X, uint64_t ldx) {
    if (!experts || !weights) return CBK_E_INVALID;
    if (!aligned(experts, 4) || !aligned(weights, 4)) return CBK_E_ALIGN;
    if (act != CBK_ACT_SILU && act != CBK_ACT_GELU && act != CBK_ACT_GELU_TANH) return CBK_E_INVALID;
    return check_rows(X, CBK_BF16, ldx, ex->cols);
}

cbk_status check_workspace(const void *ws, size_t bytes, uint64_t need) {
    if (need > 0 && !ws) return CBK_E_INVALID;
    if (!aligned(ws, 256)) return CBK_E_ALIGN;
    if (bytes < need) return CBK_E_CAPACITY;
    return CBK_OK;
}

// How a draw is done; us are of replayed calls, rows with one workgroup each against their work divided.
// Numbers that filter nothing: two kernels, the first over segments of the rows, in chunks of rows with 64 MB of scratch.
// 1 row of 1000 12.0 and 9.5, of 32000 22.3 and 12.4, of 128000 51 and 12.3; 64 of 32000 23.5 and 14.5; 192 of 128000 57
// and 41; 1000 of 4000 52 and 16.
// Filters, or vectors of them: three kernels that share a few long rows' passes, and k_sample, which otherwise does all of a
// row.  With top_k = 50 and with top_p = 0.9: 1 row of 32000 24, 50 and 28, 42; of 65000 33, 74 and 30, 42; of 128000 48,
// 124 and 30, 46; 64 of 65000 35, 76 and 37, 52; of 128000 52, 126 and 49, 74; 192 of 128000 55, 128 and 85, 146 (the row's
// cut is looked for by each of its workgroups).  The rule goes by the rows' length and number alone, also where the call's
// numbers say which filters there are.  A launch has fewer than 2^32 threads.
cbk::SamplePlan sample_plan(const cbk_sampling &p, uint64_t V, uint64_t tokens) {
    const bool filters = p.top_ks || p.top_ps || p.min_ps || (p.top_k > 0 && static_cast<uint64_t>(p.top_k) < V) || p.top_p < 1.f || p.min_p > 0.f;
    cbk::SamplePlan pl{uint64_t(1) << 21, 0, 0, false, 0, 0, 0, 0};
    if (filters && !(V >= 65000 && tokens <= 64)) return pl;
    // (the first entry may lie up to three elements into its segment)
    pl.segments = static_cast<uint32_t>((V + 3 + cbk::kSampleSegment - 1) / cbk::kSampleSegment);
    pl.divided = filters;
    const uint64_t row = pl.segments * cbk::kSamplePartBytes + (filters ? pl.segments * 8 + cbk::kSampleBins * 16 + cbk::kSamplePartBytes : 0);
    pl.rows = std::min<uint64_t>(tokens, (uint64_t(1) << 26) / row);
    pl.sums = pl.rows * pl.segments * cbk::kSamplePartBytes;
    pl.bins = pl.sums + pl.rows * pl.segments * 8;
    pl.list = pl.bins + pl.rows * cbk::kSampleBins * 8;
    pl.state = pl.list + pl.rows * cbk::kSampleBins * 8;
    pl.bytes = pl.rows * row;
    return pl;
}

}  // namespace

namespace cbk {

// Chunks of tokens keep what is held per slot (H, or dG and dU, and the fp32 results before they are added by token)
// to some 1.5 GB; larger chunks decode each expert's weights for more tokens at once.
ExPlan ex_plan(const cbk_experts &ex, uint64_t tokens, uint32_t k, bool backward) {
    constexpr uint64_t kSlots = 65536, kSlotBytes = uint64_t(1536) << 20;
    ExPlan p{};
    p.Kp = up_to(ex.cols, 64);
    p.Fp = up_to(ex.rows, 64);
    p.Op = up_to(ex.out, 64);
    p.ldK = up_to(ex.cols, 128);
    p.ldF = up_to(ex.rows, 128);
    p.ldO = up_to(ex.out, 128);
    const uint64_t per_slot = backward ? 4 * p.ldK + 4 * p.ldF + 4 * p.Fp : 4 * p.ldO + 2 * p.Fp;
    // a chunk's rows of X and dY lie within 31 bits of bytes (their padded copies do)
    const uint64_t most = std::max<uint64_t>(1, std::min<uint64_t>({kSlots / k, kSlotBytes / (per_slot * k), (uint64_t(1) << 29) / std::max(p.Kp, p.Op)}));
    p.Tc = std::min(tokens, most);
    uint64_t slots = p.Tc * k, active = std::min<uint64_t>(ex.count, slots);
    // Slots of a token tile, by how many there are for an expert that has any.  32 experts of 2048 x 4096, 4 a token, us with
    // tiles of 16, 64 and 256 (k_experts_few, k_experts, k_experts_many; the backward pass' gradients by k_experts where
    // tiles are not of 256): 32 tokens forward 292, 403, 341, backward 478, 563, 590; 64 tokens 336, 409, 345 and 529, 572, 598;
    // 96 tokens 418, 413, 349 and 676, 577, 597; 192 tokens 615, 439, 361 and 957, 608, 612; 256 tokens 791, 538, 385
    // and 1221, 765, 645.  (It was measured on that layer alone, and does not ask how many workgroups a size leaves: narrow layers
    // of few experts may have fewer of 256 than there are CUs.)  Tiles of 256 need the LDS to hold two tables of gate and up, or
    // one of down, beside their blocks.
    const uint64_t per = slots / active;
    const bool large = ex.b <= 13 && ex.b_down <= 14;
    p.tile = per <= 8 ? 16 : large && per > (backward ? 24 : 8) ? 256 : 64;
    // A launch has fewer than 2^32 threads, 512 for each tile of the result.  Hundreds of experts in use, of some 2^19 hidden columns
    // and more, have more tiles of 16 slots x 64 of them (other products' results take a chunk's bytes long before that, and
    // tiles of more slots are fewer): such a chunk is cut down, to 7 tokens or more, which have tiles of 16 again.
    constexpr uint64_t kMostTiles = (uint64_t(1) << 23) - 8;
    if (p.tile == 16 && (active + slots / 16) * (p.Fp / 64) > kMostTiles) {
        p.Tc = kMostTiles / (p.Fp / 64) * 16 / 17 / k;
        slots = p.Tc * k;
        active = std::min<uint64_t>(ex.count, slots);
    }
    p.max_tiles = static_cast<uint32_t>(active + slots / p.tile);
    p.one = !backward && tokens == 1 && p.tile == 16 && ex.b <= 13 && ex.b_down <= 14;  // where k_experts_few does both products
    if (p.one) p.max_tiles = k;
    // few units of work: their reductions are shared until there are two for each CU, of eight slices of 64 at least
    auto split = [&](uint64_t columns, uint64_t slices) {
        const uint64_t units = p.max_tiles * (up_to(columns, 128) / 128);
        return static_cast<uint32_t>(std::max<uint64_t>(1, std::min<uint64_t>({512 / units, slices / 8, 8})));
    };
    p.split_down = p.tile != 16 ? split(ex.out, p.Fp / 64) : 1;
    p.split_dt = split(ex.rows, p.Op / 64);
    p.split_x = split(ex.cols, 2 * p.Fp / 64);
    uint64_t at = 0;
    auto take = [&](uint64_t bytes) {
        const uint64_t o = at;
        at += up_to(bytes, 256);
        return o;
    };
    p.ntiles = take(4);
    p.tiles = take(uint64_t(p.max_tiles) * 16);
    p.token_of = take(slots * 4);
    p.slot_of = take(slots * 4);
    p.place_of = take(slots * 4);
    p.xpack = take(p.Tc * p.Kp * 2);
    if (!backward) {
        p.h = take(slots * p.Fp * 2);
        p.s_stride = slots * p.ldO;
        p.s = take(p.split_down * p.s_stride * 4);
    } else {
        p.ypack = take(p.Tc * p.Op * 2);
        p.d_stride = slots * p.ldF;
        p.d = take(p.split_dt * p.d_stride * 4);
        p.g = take(slots * p.Fp * 4);
        p.s_stride = slots * p.ldK;
        p.s = take(p.split_x * p.s_stride * 4);
        // a partial sum for each wave that a row's columns are spread over: 64 columns of 256, or 16 of 64
        p.dw_parts = static_cast<uint32_t>(p.tile == 256 ? up_to(p.Fp, 128) / 64 : p.Fp / 16);
        p.dw = take(slots * p.dw_parts * 4);
    }
    p.bytes = at;
    return p;
}

}  // namespace cbk

extern "C" {

cbk_status cbk_route(const cbk_router *r, const void *logits, int dtype, uint64_t ld, uint64_t tokens, const float *bias,
                     int32_t *experts, float *weights, void *stream) {
    cbk_status st = check_router(r);
    if (st != CBK_OK) return st;
    if (tokens >= kMaxTokens) return CBK_E_UNSUPPORTED;
    if (tokens == 0) return CBK_OK;
    st = check_rows(logits, dtype, ld, r->experts);
    if (st != CBK_OK) return st;
    if (!experts || !weights) return CBK_E_INVALID;
    if (!aligned(experts, 4) || !aligned(weights, 4) || !aligned(bias, 4)) return CBK_E_ALIGN;
    return cbk::launch_route(*r, logits, dtype, ld, tokens, bias, experts, weights, static_cast<hipStream_t>(stream));
}

cbk_status cbk_route_bwd(const cbk_router *r, const void *logits, int dtype, uint64_t ld, uint64_t tokens,
                         const int32_t *experts, const float *dweights, void *dlogits, uint64_t ldd, void *stream) {
    cbk_status st = check_router(r);
    if (st != CBK_OK) return st;
    if (tokens >= kMaxTokens) return CBK_E_UNSUPPORTED;
    if (tokens == 0) return CBK_OK;
    st = check_rows(logits, dtype, ld, r->experts);
    if (st == CBK_OK) st = check_rows(dlogits, dtype, ldd, r->experts);
    if (st != CBK_OK) return st;
    if (!experts || !dweights) return CBK_E_INVALID;
    if (!aligned(experts, 4) || !aligned(dweights, 4)) return CBK_E_ALIGN;
    return cbk::launch_route_bwd(*r, logits, dtype, ld, tokens, experts, dweights, dlogits, ldd, static_cast<hipStream_t>(stream));
}

size_t cbk_experts_bytes(uint32_t count) { return static_cast<size_t>(up_to(3 * cbk::kExTensorBytes * count, 256)); }

cbk_status cbk_experts_init(const cbk_tensor *gate, const cbk_tensor *up, const cbk_tensor *down, uint32_t count,
                            void *buffer, size_t bytes, cbk_experts *ex) {
    if (!gate || !up || !down || !buffer || !ex || count == 0 || count > kMaxExperts) return CBK_E_INVALID;
    cbk_experts e{};
    e.buffer = buffer;
    e.rows = gate[0].rows;
    e.cols = gate[0].cols;
    e.out = down[0].rows;
    e.count = count;
    for (uint32_t i = 0; i < count; ++i) {
        for (const cbk_tensor *t : {&gate[i], &up[i], &down[i]}) {
            const cbk_status st = cbk::check_tensor(t);
            if (st != CBK_OK) return st;
        }
        if (gate[i].rows != e.rows || gate[i].cols != e.cols || up[i].rows != e.rows || up[i].cols != e.cols ||
            down[i].rows != e.out || down[i].cols != e.rows)
            return CBK_E_INVALID;
        e.b = std::max({e.b, gate[i].b, up[i].b});
        e.b_down = std::max(e.b_down, down[i].b);
    }
    cbk_status st = check_experts(&e);
    if (st != CBK_OK) return st;
    if (!aligned(buffer, 256)) return CBK_E_ALIGN;
    if (bytes < cbk_experts_bytes(count)) return CBK_E_CAPACITY;
    st = cbk::experts_table(gate, up, down, count, buffer, e.device);
    if (st == CBK_OK) *ex = e;
    return st;
}

size_t cbk_experts_workspace_bytes(const cbk_experts *ex, uint64_t tokens, uint32_t k, int backward) {
    if (check_experts(ex) != CBK_OK || k == 0 || k > kMaxChosen || tokens == 0 || tokens >= kMaxTokens) return 0;
    return static_cast<size_t>(cbk::ex_plan(*ex, tokens, k, backward != 0).bytes);
}

cbk_status cbk_ffn_experts(const cbk_experts *ex, int act, const uint16_t *X, uint64_t ldx, uint64_t tokens,
                           const int32_t *experts, const float *weights, uint32_t k, uint16_t *Y, uint64_t ldy,
                           void *workspace, size_t workspace_bytes, void *stream) {
    cbk_status st = check_experts(ex);
    if (st != CBK_OK) return st;
    if (k == 0) return CBK_E_INVALID;
    if (k > kMaxChosen || tokens >= kMaxTokens) return CBK_E_UNSUPPORTED;
    if (tokens == 0) return CBK_OK;
    st = check_call(ex, act, experts, weights, X, ldx);
    if (st == CBK_OK) st = check_rows(Y, CBK_BF16, ldy, ex->out);
    if (st != CBK_OK) return st;
    const cbk::ExPlan pl = cbk::ex_plan(*ex, tokens, k, false);
    st = check_workspace(workspace, workspace_bytes, pl.bytes);
    if (st != CBK_OK) return st;
    return cbk::launch_experts(*ex, pl, act, X, ldx, tokens, experts, weights, k, nullptr, 0, Y, ldy, nullptr, workspace,
                               static_cast<hipStream_t>(stream));
}

cbk_status cbk_ffn_experts_bwd(const cbk_experts *ex, int act, const uint16_t *X, uint64_t ldx, uint64_t tokens,
                               const int32_t *experts, const float *weights, uint32_t k, const uint16_t *dY,
                               uint64_t lddy, uint16_t *dX, uint64_t lddx, float *dweights, void *workspace,
                               size_t workspace_bytes, void *stream) {
    cbk_status st = check_experts(ex);
    if (st != CBK_OK) return st;
    if (k == 0) return CBK_E_INVALID;
    if (k > kMaxChosen || tokens >= kMaxTokens) return CBK_E_UNSUPPORTED;
    if (tokens == 0) return CBK_OK;
    st = check_call(ex, act, experts, weights, X, ldx);
    if (st == CBK_OK) st = check_rows(dY, CBK_BF16, lddy, ex->out);
    if (st == CBK_OK) st = check_rows(dX, CBK_BF16, lddx, ex->cols);
    if (st != CBK_OK) return st;
    if (!aligned(dweights, 4)) return CBK_E_ALIGN;
    const cbk::ExPlan pl = cbk::ex_plan(*ex, tokens, k, true);
    st = check_workspace(workspace, workspace_bytes, pl.bytes);
    if (st != CBK_OK) return st;
    return cbk::launch_experts(*ex, pl, act, X, ldx, tokens, experts, weights, k, dY, lddy, dX, lddx, dweights, workspace,
                               static_cast<hipStream_t>(stream));
}

size_t cbk_sample_workspace_bytes(const cbk_sampling *p, uint64_t V, uint64_t tokens) {
    if (!p || V == 0 || V > kMaxWidth || tokens == 0 || tokens >= kMaxTokens) return 0;
    return static_cast<size_t>(sample_plan(*p, V, tokens).bytes);
}

cbk_status cbk_sample(const cbk_sampling *p, const void *logits, int dtype, uint64_t ld, uint64_t V, uint64_t tokens,
                      const float *uniform, int64_t *token, float *logprob, void *workspace, size_t workspace_bytes,
                      void *stream) {
    if (!p || V == 0) return CBK_E_INVALID;
    if (V > kMaxWidth || tokens >= kMaxTokens) return CBK_E_UNSUPPORTED;
    if (tokens == 0) return CBK_OK;
    cbk_status st = check_rows(logits, dtype, ld, V);
    if (st != CBK_OK) return st;
    if (!uniform || !token) return CBK_E_INVALID;
    if (!aligned(uniform, 4) || !aligned(token, 8) || !aligned(logprob, 4) || !aligned(p->temperatures, 4) ||
        !aligned(p->top_ps, 4) || !aligned(p->min_ps, 4) || !aligned(p->top_ks, 4))
        return CBK_E_ALIGN;
    const cbk::SamplePlan pl = sample_plan(*p, V, tokens);
    st = check_workspace(workspace, workspace_bytes, pl.bytes);
    if (st != CBK_OK) return st;
    return cbk::launch_sample(*p, logits, dtype, ld, V, tokens, uniform, token, logprob, pl, workspace, static_cast<hipStream_t>(stream));
}

}  // extern "C"
