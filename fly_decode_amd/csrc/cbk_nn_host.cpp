// Host half of the operators in cbk_nn.h: how a call is cut into pieces and laid out in its
// workspace, and argument validation in front of the HIP launchers (cbk_nn.hip).  Nothing here
// touches the GPU until every argument has been checked.
#include <stdint.h>

#include <algorithm>

#include "cbk_internal.h"

namespace {

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline uint64_t up_to(uint64_t n, uint64_t m) { return (n + m - 1) / m * m; }

constexpr uint64_t kMaxTokens = uint64_t(1) << 31;
constexpr uint64_t kMaxCols = uint64_t(1) << 20;
constexpr uint64_t kMaxRows = uint64_t(1) << 31;
constexpr uint64_t kMaxLd = uint64_t(1) << 32;

cbk_status check_weights(const cbk_tensor *t) {
    const cbk_status st = cbk::check_tensor(t);
    if (st != CBK_OK) return st;
    if (t->cols > kMaxCols || t->rows >= kMaxRows) return CBK_E_UNSUPPORTED;
    return CBK_OK;
}

// A matrix of `width` used columns (a null pointer is only right when nothing of it is used).
cbk_status check_matrix(const void *p, uint64_t ld, uint64_t width) {
    if (width > 0 && !p) return CBK_E_INVALID;
    if (ld < width) return CBK_E_INVALID;
    if (!aligned(p, 2)) return CBK_E_ALIGN;
    if (ld >= kMaxLd) return CBK_E_UNSUPPORTED;
    return CBK_OK;
}

cbk_status check_workspace(const void *ws, size_t bytes, uint64_t need) {
    if (need > 0 && !ws) return CBK_E_INVALID;
    if (!aligned(ws, 256)) return CBK_E_ALIGN;
    if (bytes < need) return CBK_E_CAPACITY;
    return CBK_OK;
}

cbk_status check_pair(const cbk_tensor *gate, const cbk_tensor *up, int act) {
    cbk_status st = check_weights(gate);
    if (st == CBK_OK) st = check_weights(up);
    if (st != CBK_OK) return st;
    if (gate->rows != up->rows || gate->cols != up->cols) return CBK_E_INVALID;
    if (act != CBK_ACT_SILU && act != CBK_ACT_GELU && act != CBK_ACT_GELU_TANH) return CBK_E_INVALID;
    return CBK_OK;
}

// Workspace of a call on one tensor, or on a gate and up pair.
uint64_t bytes_of(cbk::NnOp op, const cbk_tensor *t, const cbk_tensor *up, uint64_t tokens) {
    if (check_weights(t) != CBK_OK || tokens >= kMaxTokens) return 0;
    const cbk_tensor *ts[2] = {t, up};
    return cbk::nn_plan(op, ts, tokens).bytes;
}

// First failure of a list of checks, in order.
template <typename... S>
cbk_status first(S... st) {
    cbk_status r = CBK_OK;
    (void)((r = st, r != CBK_OK) || ...);
    return r;
}

}  // namespace

namespace cbk {

namespace {

// The token tile of k_fused, or 0 where the tensors or the number of tokens are not its kind: widths
// 8 to 14, whose table and ring the LDS holds at every tile.  Up to 384 tokens it is
// ahead of decoding a piece first (a pair of 4096 x 11008: 49 us against 128 at 64 tokens, 129 against
// 153 at 384, 170 in two halves against 154 at 512); short rows leave it more sums to pass on per product
// (a pair of 384 x 11008: 37 against 34 at 256, 45 against 36 at 384; of 1024 x 11008: 55 against 52 at
// 384, its gradient 102 against 109).  A pair of two widths takes a launch for each
// tensor (13 and 11 bits, 4096 x 11008: 36 us against 140 at 1 token, 56 against 134 at 64, 143 against 152
// at 384; 512 x 11008: 30 against 39 at 64, 50 against 43 at 200).
uint32_t fused_tile(const cbk_tensor *const *ts, uint64_t count, uint64_t tokens) {
    const bool split = count == 2 && ts[0]->b != ts[1]->b;
    if (tokens > (ts[0]->cols >= 1024 ? 384 : split ? 128 : 256)) return 0;
    for (uint64_t i = 0; i < count; ++i) {
        const cbk_tensor &t = *ts[i];
        if (t.b < 8 || t.b > 14 || t.cols == 0 || !aligned(t.codebook, 16)) return 0;
    }
    uint32_t bm = 384;
    for (uint32_t x : {320u, 256u, 192u, 128u, 64u, 16u})
        if (tokens <= x) bm = x;
    return bm;
}

}  // namespace

namespace {
constexpr uint64_t kPieceBytes = uint64_t(256) << 20;
constexpr uint64_t kPieceRows = 32768;
constexpr uint64_t kPieceLeast = 256;  // rows, whatever they take
}  // namespace

// Widths 1 to 15 with the table's loads aligned.  Every piece of nn_plan starts on a multiple of 128 weights and
// holds at most 2^15 rows and 2^28 weights, which is what k_unpack's 32-bit fields and its rows by a
// reciprocal take (512 tokens and a piece of 2^27 weights, 32768 x 4096: 214 us, 396 by the generic kernel).
bool nn_unpack_in_order(const cbk_tensor &t, uint64_t row0, uint64_t nrows) {
    constexpr uint64_t kMost = std::max(kPieceBytes / 2, kPieceLeast * kMaxCols);
    return t.b >= 1 && t.b <= 15 && aligned(t.codebook, 16) && cbk_words_for(t.rows * t.cols, t.b) / 4 < (uint64_t(1) << 32) &&
           t.cols > 0 && row0 * t.cols % 128 == 0 && nrows <= kPieceRows && nrows * t.cols <= kMost;
}

// A decoded piece takes up to kPieceBytes and kPieceRows, and the sums of a piece's rows for a chunk of
// tokens (k_fused) up to kSumBytes, so that a call's scratch stays far below the tensor's uncompressed
// size and no call keeps what grows with tokens times rows; chunks of kChunk tokens bound what is
// kept per token.
NnPlan nn_plan(NnOp op, const cbk_tensor *const *ts, uint64_t tokens) {
    constexpr uint64_t kSumBytes = uint64_t(64) << 20;
    constexpr uint64_t kChunk = 8192;
    const uint64_t rows = ts[0]->rows, cols = ts[0]->cols;
    NnPlan p{};
    if (tokens == 0 || rows == 0) return p;
    const uint64_t pair = op == NnOp::ffn ? 2 : 1;  // decoded rows per row of a tensor
    p.Kp = std::max<uint64_t>(64, up_to(cols, 64));
    p.Tc = std::min(tokens, kChunk);
    p.fused = fused_tile(ts, pair, tokens);
    const uint64_t total = up_to(pair * up_to(rows, 16), 256);
    const uint64_t most = p.fused ? std::max<uint64_t>(256, kSumBytes / (4 * p.Tc) / 256 * 256) : std::min(kPieceRows, std::max<uint64_t>(kPieceLeast, kPieceBytes / (2 * p.Kp) / 256 * 256));
    p.pieces = (total + most - 1) / most;
    p.Rp = up_to((total + p.pieces - 1) / p.pieces, 256);
    p.rows = p.Rp / pair;
    p.pieces = (rows + p.rows - 1) / p.rows;
    uint64_t at = 0;
    auto take = [&](uint64_t bytes) {
        const uint64_t o = at;
        at += up_to(bytes, 256);
        return o;
    };
    // a copy of the chunk's X (or of a piece's columns of dY), padded or in blocks of 16 tokens
    p.pack = take(up_to(p.Tc, 16) * std::max(p.Kp, op == NnOp::linear ? p.Rp : 0) * 2);
    if (p.fused) {
        // as many workgroups as the LDS lets run at once on 256 CUs, and their parts of the tiles; a pair
        // of two widths takes two launches
        p.split = pair == 2 && ts[0]->b != ts[1]->b;
        p.grid = 256 * std::min<uint32_t>(3, 160 * 1024 / nn_fused_lds(std::max(ts[0]->b, ts[pair - 1]->b), p.fused));
        p.part = take(((p.split ? 2 : 1) * p.grid + pair * (std::max(p.rows + 127, p.Kp + 64) / 128)) * p.Tc * 128 * 4);
    } else {
        p.w = take(p.Rp * p.Kp * 2);
        // no more tiles are shared than the largest product of the call has
        const uint64_t tiles = up_to(p.Tc, 256) / 256 * (up_to(std::max(p.Kp, p.Rp), 256) / 256);
        p.part = take((256 + std::min<uint64_t>(kMmShared, tiles)) * 256 * 256 * 4);
    }
    p.g = op == NnOp::linear ? at : take(up_to(p.Tc, 16) * p.Rp * 2);
    p.acc = p.pieces > 1 ? take(p.Tc * p.Kp * 4) : at;
    p.stat = op == NnOp::xent ? take(p.Tc * p.pieces * (p.Rp / 128) * 8) : at;
    p.top = op == NnOp::xent ? take(p.Tc * 4) : at;
    p.bytes = at;
    return p;
}

}  // namespace cbk

using cbk::NnOp;

extern "C" {

size_t cbk_linear_workspace_bytes(const cbk_tensor *t, uint64_t tokens) { return bytes_of(NnOp::linear, t, nullptr, tokens); }

cbk_status cbk_linear(const cbk_tensor *t, const uint16_t *X, uint64_t ldx, uint64_t tokens, uint16_t *Y, uint64_t ldy,
                      void *workspace, size_t workspace_bytes, void *stream) {
    cbk_status st = check_weights(t);
    if (st != CBK_OK) return st;
    if (tokens >= kMaxTokens) return CBK_E_UNSUPPORTED;
    if (tokens == 0 || t->rows == 0) return CBK_OK;
    st = first(check_matrix(X, ldx, t->cols), check_matrix(Y, ldy, t->rows),
               check_workspace(workspace, workspace_bytes, bytes_of(NnOp::linear, t, nullptr, tokens)));
    if (st != CBK_OK) return st;
    return cbk::launch_linear(*t, X, ldx, tokens, Y, ldy, workspace, static_cast<hipStream_t>(stream));
}

cbk_status cbk_linear_dx(const cbk_tensor *t, const uint16_t *dY, uint64_t lddy, uint64_t tokens, uint16_t *dX,
                         uint64_t lddx, void *workspace, size_t workspace_bytes, void *stream) {
    cbk_status st = check_weights(t);
    if (st != CBK_OK) return st;
    if (tokens >= kMaxTokens) return CBK_E_UNSUPPORTED;
    if (tokens == 0 || t->cols == 0) return CBK_OK;
    st = first(check_matrix(dY, lddy, t->rows), check_matrix(dX, lddx, t->cols),
               check_workspace(workspace, workspace_bytes, bytes_of(NnOp::linear, t, nullptr, tokens)));
    if (st != CBK_OK) return st;
    return cbk::launch_linear_dx(*t, dY, lddy, tokens, dX, lddx, workspace, static_cast<hipStream_t>(stream));
}

size_t cbk_ffn_workspace_bytes(const cbk_tensor *gate, const cbk_tensor *up, uint64_t tokens) {
    if (check_pair(gate, up, CBK_ACT_SILU) != CBK_OK) return 0;
    return bytes_of(NnOp::ffn, gate, up, tokens);
}

cbk_status cbk_ffn_gated(const cbk_tensor *gate, const cbk_tensor *up, int act, const uint16_t *X, uint64_t ldx,
                         uint64_t tokens, uint16_t *H, uint64_t ldh, void *workspace, size_t workspace_bytes,
                         void *stream) {
    cbk_status st = check_pair(gate, up, act);
    if (st != CBK_OK) return st;
    if (tokens >= kMaxTokens) return CBK_E_UNSUPPORTED;
    if (tokens == 0 || gate->rows == 0) return CBK_OK;
    st = first(check_matrix(X, ldx, gate->cols), check_matrix(H, ldh, gate->rows),
               check_workspace(workspace, workspace_bytes, bytes_of(NnOp::ffn, gate, up, tokens)));
    if (st != CBK_OK) return st;
    return cbk::launch_ffn(*gate, *up, act, X, ldx, tokens, H, ldh, workspace, static_cast<hipStream_t>(stream));
}

cbk_status cbk_ffn_gated_bwd(const cbk_tensor *gate, const cbk_tensor *up, int act, const uint16_t *X, uint64_t ldx,
                             const uint16_t *dH, uint64_t lddh, uint64_t tokens, uint16_t *dX, uint64_t lddx,
                             uint16_t *dG, uint16_t *dU, uint64_t ldg, void *workspace, size_t workspace_bytes,
                             void *stream) {
    cbk_status st = check_pair(gate, up, act);
    if (st != CBK_OK) return st;
    if (tokens >= kMaxTokens) return CBK_E_UNSUPPORTED;
    if (tokens == 0) return CBK_OK;
    st = first(check_matrix(X, ldx, gate->cols), check_matrix(dH, lddh, gate->rows),
               check_matrix(dX, lddx, gate->cols), dG ? check_matrix(dG, ldg, gate->rows) : CBK_OK,
               dU ? check_matrix(dU, ldg, gate->rows) : CBK_OK,
               check_workspace(workspace, workspace_bytes, bytes_of(NnOp::ffn, gate, up, tokens)));
    if (st != CBK_OK) return st;
    return cbk::launch_ffn_bwd(*gate, *up, act, X, ldx, dH, lddh, tokens, dX, lddx, dG, dU, ldg, workspace,
                               static_cast<hipStream_t>(stream));
}

size_t cbk_xent_workspace_bytes(const cbk_tensor *head, uint64_t tokens) { return bytes_of(NnOp::xent, head, nullptr, tokens); }

cbk_status cbk_xent(const cbk_tensor *head, const uint16_t *X, uint64_t ldx, const int64_t *labels, uint64_t tokens,
                    int64_t ignore_index, float *loss, float *lse, void *workspace, size_t workspace_bytes,
                    void *stream) {
    cbk_status st = check_weights(head);
    if (st != CBK_OK) return st;
    if (head->rows == 0) return CBK_E_INVALID;
    if (tokens >= kMaxTokens) return CBK_E_UNSUPPORTED;
    if (tokens == 0) return CBK_OK;
    if (!labels || !loss || !lse) return CBK_E_INVALID;
    if (!aligned(labels, 8) || !aligned(loss, 4) || !aligned(lse, 4)) return CBK_E_ALIGN;
    st = first(check_matrix(X, ldx, head->cols),
               check_workspace(workspace, workspace_bytes, bytes_of(NnOp::xent, head, nullptr, tokens)));
    if (st != CBK_OK) return st;
    return cbk::launch_xent(*head, X, ldx, labels, tokens, ignore_index, loss, lse, workspace,
                            static_cast<hipStream_t>(stream));
}

cbk_status cbk_xent_bwd(const cbk_tensor *head, const uint16_t *X, uint64_t ldx, const int64_t *labels,
                        const float *lse, const float *dloss, uint64_t tokens, int64_t ignore_index, uint16_t *dX,
                        uint64_t lddx, void *workspace, size_t workspace_bytes, void *stream) {
    cbk_status st = check_weights(head);
    if (st != CBK_OK) return st;
    if (head->rows == 0) return CBK_E_INVALID;
    if (tokens >= kMaxTokens) return CBK_E_UNSUPPORTED;
    if (tokens == 0) return CBK_OK;
    if (!labels || !lse || !dloss) return CBK_E_INVALID;
    if (!aligned(labels, 8) || !aligned(lse, 4) || !aligned(dloss, 4)) return CBK_E_ALIGN;
    st = first(check_matrix(X, ldx, head->cols), check_matrix(dX, lddx, head->cols),
               check_workspace(workspace, workspace_bytes, bytes_of(NnOp::xent, head, nullptr, tokens)));
    if (st != CBK_OK) return st;
    if (head->cols == 0) return CBK_OK;
    return cbk::launch_xent_bwd(*head, X, ldx, labels, lse, dloss, tokens, ignore_index, dX, lddx, workspace,
                                static_cast<hipStream_t>(stream));
}

}  // extern "C"
