// HIP kernels for gfx950 (CDNA4) of the operators in cbk_nn.h: products of any number of tokens
// with codebook-compressed weights, the gated feed-forward block, the softmax cross entropy of a
// compressed head, and their gradients.
//
// All are products with a tensor W [N][K] that is stored as b-bit indices into a codebook:
//   forward   Y = X W^T   (reduction over W's columns)
//   gradient  dX = G W    (reduction over W's rows)
// Up to a few hundred tokens (nn_plan) the weights are decoded on the way, once, by the workgroup that
// multiplies them: k_fused (cbk_nn_fused.h), or the batch-1 GEMV for one token.  Both leave fp32 sums,
// and k_join does the operator's work on them.  With more tokens, and for widths that k_fused does not
// take, a piece of W is decoded into the workspace once (k_unpack: [rows][Kp] BF16, Kp = K rounded up
// to 64, zero padded, in blocks), and one matrix-core kernel, k_mm, multiplies it in either orientation; the
// operator's work is its epilogue.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "cbk_nn_device.h"

namespace cbk {
namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));

#define CBK_TRY(x)                          \
    do {                                    \
        const cbk_status st_ = (x);         \
        if (st_ != CBK_OK) return st_;      \
    } while (0)

inline uint32_t ceil_div(uint64_t n, uint64_t m) { return static_cast<uint32_t>((n + m - 1) / m); }
inline bool aligned_to(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// ------------------------------------------------------------------------------- small pieces

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

// X [T][K] with leading dimension ld into P [T][Kp], columns past K zero.
__global__ __launch_bounds__(256) void k_pad_rows(const uint16_t *__restrict__ X, uint64_t ld, uint64_t T, uint32_t K,
                                                  uint32_t Kp, uint16_t *__restrict__ P) {
    const uint64_t n = T * (Kp / 4), stride = static_cast<uint64_t>(gridDim.x) * blockDim.x;
    for (uint64_t i = static_cast<uint64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n; i += stride) {
        const uint64_t t = i / (Kp / 4);
        const uint32_t k = static_cast<uint32_t>(i - t * (Kp / 4)) * 4;
        const uint16_t *x = X + t * ld + k;
        uint16_t v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = k + j < K ? x[j] : static_cast<uint16_t>(0);
        *reinterpret_cast<u32x2 *>(P + t * Kp + k) = (u32x2){static_cast<uint32_t>(v[0]) | (static_cast<uint32_t>(v[1]) << 16),
                                                             static_cast<uint32_t>(v[2]) | (static_cast<uint32_t>(v[3]) << 16)};
    }
}

// out[t][0 .. n) = 0
__global__ __launch_bounds__(256) void k_zero_rows(uint16_t *__restrict__ out, uint64_t ld, uint64_t T, uint32_t n) {
    const uint64_t all = T * n, stride = static_cast<uint64_t>(gridDim.x) * blockDim.x;
    for (uint64_t i = static_cast<uint64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < all; i += stride)
        out[i / n * ld + i % n] = 0;
}

// ------------------------------------------------------------------------- decoding a piece
// Rows [row0, row0 + nrows) of a tensor into out [rows_out][Kp] (piece_at); columns past cols and rows past
// nrows are zero.  `pair` 0: row f goes to row f.  1 and 2: the gate and up tensors share the
// piece, 16 rows of each in turn (row f to 32 (f / 16) + 16 (pair - 1) + f % 16), so that a wave
// of k_mm has a column's gate and up sums in the same lanes.
struct UnpackTensor {
    const uint32_t *words;
    const uint16_t *cb;
    uint32_t U, nchunks;
};
struct UnpackArgs {
    UnpackTensor t[2];
    uint32_t b, cols, Kp;
    uint64_t row0;
    uint32_t nrows, rows_out, pair;
    uint16_t *out;
    float inv_cols;
    uint32_t steps;
};

__device__ __forceinline__ uint32_t piece_row(uint32_t f, uint32_t pair) {
    return pair == 0 ? f : (f >> 4) * 32 + (pair - 1) * 16 + (f & 15);
}

// Where element (row, k) of a piece lies: blocks of 16 rows x 32 columns, 1 KB each, one after the other
// along the rows and then down.  A wave's copy into LDS takes one block, so it reads whole cache lines in
// either orientation of the product.
__device__ __forceinline__ uint64_t piece_at(uint32_t row, uint32_t k, uint32_t Kp) {
    return static_cast<uint64_t>(row >> 4) * (Kp * 16) + ((k >> 5) * 512 + (row & 15) * 32 + (k & 31));
}

// X [T][K] with leading dimension ld into such blocks, columns past K zero: a thread per 16 bytes.
__global__ __launch_bounds__(256) void k_pack_rows(const uint16_t *__restrict__ X, uint64_t ld, uint32_t T, uint32_t K,
                                                   uint32_t Kp, uint32_t whole, uint16_t *__restrict__ P) {
    const uint64_t n = static_cast<uint64_t>((T + 15) / 16) * (Kp / 32) * 64, stride = static_cast<uint64_t>(gridDim.x) * blockDim.x;
    for (uint64_t i = static_cast<uint64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n; i += stride) {
        const uint64_t blk = i >> 6, down = quotient(blk, Kp / 32);
        const uint32_t t = static_cast<uint32_t>(down) * 16 + (static_cast<uint32_t>(i) >> 2 & 15);
        const uint32_t k = static_cast<uint32_t>(blk - down * (Kp / 32)) * 32 + (static_cast<uint32_t>(i) & 3) * 8;
        if (t >= T) continue;
        const uint16_t *x = X + t * ld + k;
        u32x4 v = (u32x4){0u, 0u, 0u, 0u};
        if (whole && k + 8 <= K) {
            v = *reinterpret_cast<const u32x4 *>(x);
        } else {
            uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
            for (uint32_t j = 0; j < 8; ++j)
                if (k + j < K) w[j >> 1] |= static_cast<uint32_t>(x[j]) << (16 * (j & 1));
            v = (u32x4){w[0], w[1], w[2], w[3]};
        }
        *reinterpret_cast<u32x4 *>(P + i * 8) = v;
    }
}

// Any width, any number of columns: a thread per 4 columns.
__global__ __launch_bounds__(256) void k_unpack_generic(const UnpackArgs a) {
    const UnpackTensor &T = a.t[0];
    const uint64_t n = static_cast<uint64_t>(a.rows_out) * (a.Kp / 4), stride = static_cast<uint64_t>(gridDim.x) * blockDim.x;
    for (uint64_t i = static_cast<uint64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n; i += stride) {
        const uint32_t f = static_cast<uint32_t>(i / (a.Kp / 4)), k = static_cast<uint32_t>(i - static_cast<uint64_t>(f) * (a.Kp / 4)) * 4;
        uint32_t v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[j] = 0;
            if (f < a.nrows && k + j < a.cols) {
                const uint32_t idx = stream_field(T.words, a.b, (a.row0 + f) * a.cols + k + j);
                v[j] = idx < T.U ? T.cb[idx] : kCorrupt;
            }
        }
        *reinterpret_cast<u32x2 *>(a.out + piece_at(piece_row(f, a.pair), k, a.Kp)) = (u32x2){v[0] | (v[1] << 16), v[2] | (v[3] << 16)};
    }
}

// The zeros of a piece: columns [cols, Kp) of its rows, and its rows past nrows.
__global__ __launch_bounds__(256) void k_unpack_pad(const UnpackArgs a) {
    for (uint32_t f = blockIdx.x; f < a.rows_out; f += gridDim.x)
        for (uint32_t pr = a.pair ? 1 : 0; pr <= a.pair; ++pr) {
            for (uint32_t k = (f < a.nrows ? a.cols : 0) + threadIdx.x; k < a.Kp; k += blockDim.x)
                a.out[piece_at(piece_row(f, pr), k, a.Kp)] = 0;
        }
}

// Widths 1 to 15: the stream is decoded in its own order, as by k_decode_fast (a wave takes steps
// of 64 units of 64 fields: coalesced loads, transposition through its LDS stage, gathers from the
// codebook in LDS), and each run of 8 fields, or each field where a row's length is no multiple of
// 8, goes to its row's place in the piece.  Both tensors of a pair go in one launch (blockIdx.y).
// row0 * cols is a multiple of 128, so a piece starts on a 16-byte chunk of the stream.  The stores keep the ordinary cache
// policy: the matrix product reads the piece next.  A pair of 4096 x 11008 at 13 bits, 147 MB in and 180 MB
// out, takes 60 us: 5.4 TB/s, bound by that traffic (54 into plain rows, whose stores are longer).  It pays from some 400 tokens on, where it is a sixth
// of the product's time or less.
constexpr int kUnpackWaves = 4;

template <int B, bool RUNS>
__global__ __launch_bounds__(64 * kUnpackWaves) void k_unpack(const UnpackArgs a) {
    using G = U64<B>;
    constexpr int NT = 64 * kUnpackWaves;
    constexpr uint32_t kUnit = 2 * 64 + 16;  // LDS bytes per decoded unit (16 bytes of padding)
    __shared__ __attribute__((aligned(16))) uint16_t cbl[Table<B>::SIZE];
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    const UnpackTensor &T = a.t[blockIdx.y];
    const uint32_t pair = a.pair ? blockIdx.y + 1 : 0;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    constexpr uint32_t kStage = G::STAGE_CHUNKS * 16 > 64 * kUnit ? G::STAGE_CHUNKS * 16 : 64 * kUnit;
    unsigned char *stb = smem + wave * kStage;
    u32x4 *stage = reinterpret_cast<u32x4 *>(stb);
    const uint64_t unit0 = a.row0 * a.cols / 64;
    const u32x4 *w4 = reinterpret_cast<const u32x4 *>(T.words) + unit0 * G::UD / 4;
    const uint64_t nchunks = T.nchunks - unit0 * G::UD / 4;
    const uint32_t NW = gridDim.x * kUnpackWaves, gw = blockIdx.x * kUnpackWaves + wave;
    const uint32_t fields = a.nrows * a.cols;

    CbStage<B, NT> cs;
    cs.issue(T.cb, T.U, w4, tid);
    issue_barrier();
    u32x4 nxt[G::LPL];
    load_step<B>(nxt, w4, gw * 64, 64, nchunks, gw < a.steps, lane);
    cs.store(cbl, T.U, tid);
    lds_barrier();

    for (uint32_t st = gw; st < a.steps; st += NW) {
        const uint32_t us = st * 64;
        uint32_t d[G::UD];
        transpose_step<B>(d, nxt, stage, us, lane);
        if (st + NW < a.steps) load_step<B>(nxt, w4, (st + NW) * 64, 64, nchunks, true, lane);
        uint32_t wv[2][8];
#pragma unroll
        for (int i = 0; i < 8; ++i) wv[0][i] = unit_gather<B>(cbl, d, i);
#pragma unroll
        for (int g = 0; g < 8; ++g) {
            if (g + 1 < 8) {
#pragma unroll
                for (int i = 0; i < 8; ++i) wv[(g + 1) & 1][i] = unit_gather<B>(cbl, d, 8 * (g + 1) + i);
            }
            const uint32_t *w = wv[g & 1];
            *reinterpret_cast<u32x4 *>(stb + lane * kUnit + 16 * g) =
                (u32x4){w[0] | (w[1] << 16), w[2] | (w[3] << 16), w[4] | (w[5] << 16), w[6] | (w[7] << 16)};
        }
        asm volatile("" ::: "memory");
        // Row and column of field i of the piece (nn_unpack_in_order): with at most 2^15 rows the product with
        // the rounded reciprocal, of three roundings, is off by less than 2^15 * 2^-22, so one step mends the row.
        auto place = [&](uint32_t i) {
            uint32_t r = static_cast<uint32_t>(static_cast<float>(i) * a.inv_cols);
            int32_t k = static_cast<int32_t>(i - r * a.cols);
            if (k < 0) {
                --r;
                k += a.cols;
            } else if (k >= static_cast<int32_t>(a.cols)) {
                ++r;
                k -= a.cols;
            }
            return a.out + piece_at(piece_row(r, pair), k, a.Kp);
        };
        if constexpr (RUNS) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t q = j * 64 + lane, i = us * 64 + q * 8;
                const u32x4 v = *reinterpret_cast<const u32x4 *>(stb + (q >> 3) * kUnit + (q & 7) * 16);
                if (i < fields) *reinterpret_cast<u32x4 *>(place(i)) = v;
            }
        } else {
            for (int j = 0; j < 64; ++j) {
                const uint32_t i = (us + j) * 64 + lane;
                if (i < fields) *place(i) = *reinterpret_cast<const uint16_t *>(stb + j * kUnit + lane * 2);
            }
        }
        asm volatile("" ::: "memory");
    }
}

// ------------------------------------------------------------------------- the matrix product
// C[m][n] = sum_r A[m][r] B(r, n) over R = 64 ktiles, A [M][lda] the tokens' side, B a decoded
// piece: NN false, B(r, n) = B[n][r] (forward); NN true, B(r, n) = B[r][n] (gradient).
//
// A workgroup of WM x WN waves owns a BM x BN tile, a wave (BM / WM) x (BN / WN) of it in 16 x 16
// fragments of v_mfma_f32_16x16x32_bf16.  The weights are the instruction's A operand and the
// tokens its B operand, so lane l holds columns n = 4 (l / 16) + 0..3 of token m = l % 16 of a
// fragment: four neighbours in the output's rows.  Slices of 32 of the reduction are copied
// straight into LDS (16 bytes a lane), a block of 16 x 32 by an instruction.
//
// LDS layout.  A copy fills 1024 consecutive bytes, so what is permuted is which 16-byte chunk a
// lane fetches.  Rows of 32 reduction elements (A, and B when NN is false) are 4 chunks, chunk c
// of row r in slot c ^ (-(r / 4) & 3).  A 128-bit read serves 16 lanes at a time, of which lanes
// 0-3 and 12-15 take one chunk of rows 0-3 and 12-15 and lanes 20-27 the next chunk of rows 4-11 (and
// so on); this order puts the 16 into different banks, where c ^ ((r / 4) & 3) made two meet.  When NN is
// true B's slice is 2 x 8 blocks of 16 reduction rows x 32 columns, read with the transposing 64-bit LDS
// read (a group of 16 lanes reads 4 rows x 16 columns, and lane i gets column i); chunk c of row r sits in
// slot c ^ (2 (r / 8)), so the 4 rows of a group and those of its neighbour hit different banks.
//
// Measured on 2048 tokens and a pair of 4096 x 11008 (369 GFLOP a product; the shortest of six calls): 289 us
// forward, 1.28 PFLOP/s, and 272 for dX, 1.36; 128 x 128 tiles took 350 forward.  On a 4096-wide head of 32000 rows (537 GFLOP),
// multiplications and barriers alone took 320 us, 1.68 PFLOP/s at the clock that the chip holds under
// them; with the fragments' reads 364, and with the copies, which are new to an XCD's L2, 400 (470 where A
// and B lay row after row and a copy read half a cache line of each).  Groups of 4 or 16 token tiles, the
// 32 x 32 instruction and a raised wave priority were no faster.
constexpr uint32_t kRing = 5;  // slices of 32 in LDS
constexpr int kMmTile = 256, kMmWm = 2, kMmWn = 4;  // tile and its waves

enum Epi { kOut, kGated, kGatedBwd, kStats, kProb };

struct MmArgs {
    const uint16_t *A;
    const uint16_t *B;
    uint64_t lda;   // elements
    uint32_t ldb, blocks;  // blocks: A lies in blocks of 16 x 32 as B does, else row after row
    uint32_t M, N;  // tokens; columns of C that exist
    uint32_t ktiles, tm, tn;
    uint32_t whole;  // tiles that one workgroup does from end to end; the others' slices are shared
    float *part;     // the sharers' sums, [sharers + shared tiles][kMmTile][kMmTile]

    uint16_t *out;  // kOut, kGated: [M][ldo] BF16
    uint64_t ldo;
    uint32_t vec;   // out (and dH, dG, dU) can be accessed 8 bytes at a time,
    uint32_t vec16;  // and 16
    float *acc;     // kOut over several pieces: fp32 sums [M][ldacc]
    uint32_t ldacc, acc_in, last;
    const int64_t *labels;
    int64_t ignore;
    const float *scale;  // kOut: factor of each token (with labels), or null
    uint64_t V;          // rows of the head

    int act;
    uint32_t f0, F;  // first row of the tensors in this piece, and all of them
    const uint16_t *dH;
    // G: the piece's gradients at the projections (or p - [label]) [M][ldG], columns as the piece's rows; k_mm writes
    // and reads it in blocks.  Rounded to BF16, which the matrix instruction's operands are: two BF16 parts of each
    // value would double the second product.  The block's dX is 0.0023 of its norm from 64 bits, 0.0017 with fp32 in
    // between; the head's stays at 0.0017.
    uint16_t *dG, *dU, *G;
    uint64_t lddh, ldg;
    uint32_t ldG;

    f32x2 *stat;  // kStats: (max, sum exp(z - max)) of each token and column tile, [M][ldstat]
    uint32_t ldstat, stat0;
    float *top;   // the label's logit
    const float *lse;
};

// The four values of a fragment row to out[0..3], of which `n` exist.
__device__ __forceinline__ void store4(uint16_t *out, const float (&v)[4], uint32_t n, bool vec) {
    if (n >= 4 && vec) {
        *reinterpret_cast<u32x2 *>(out) = (u32x2){pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
    } else {
#pragma unroll
        for (uint32_t r = 0; r < 4; ++r)
            if (r < n) out[r] = to_bf16(v[r]);
    }
}
// in[0..3], of which `n` exist (zeros for the others).
__device__ __forceinline__ u32x2 load4(const uint16_t *in, uint32_t n, bool vec) {
    if (n >= 4 && vec) return *reinterpret_cast<const u32x2 *>(in);
    uint32_t v[4];
#pragma unroll
    for (uint32_t r = 0; r < 4; ++r) v[r] = r < n ? in[r] : 0u;
    return (u32x2){v[0] | (v[1] << 16), v[2] | (v[3] << 16)};
}
__device__ __forceinline__ uint32_t left(uint32_t n, uint32_t at) { return at < n ? n - at : 0u; }

// Reference point of a sum of exponentials whose largest argument is m: 0 where m is infinite.
__device__ __forceinline__ float exp_base(float m) { return fabsf(m) == __builtin_inff() ? 0.f : m; }

// What the operators make of four neighbouring sums (columns n..n + 3) of token m.
// kOut: the sum over the pieces; false where it is only kept for the next piece.
__device__ __forceinline__ bool finish_out(const MmArgs &p, uint32_t m, uint32_t n, float (&v)[4]) {
    f32x4_t *sum = reinterpret_cast<f32x4_t *>(p.acc + static_cast<uint64_t>(m) * p.ldacc + n);
    if (p.acc_in) {
        const f32x4_t t = *sum;
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] += t[r];
    }
    if (!p.last) {
        *sum = (f32x4_t){v[0], v[1], v[2], v[3]};
        return false;
    }
    if (p.scale) {
        const int64_t lab = p.labels[m];
        const float f = lab >= 0 && static_cast<uint64_t>(lab) < p.V ? p.scale[m] : __builtin_nanf("");
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = lab == p.ignore ? 0.f : v[r] * f;
    }
    return true;
}
__device__ __forceinline__ void emit_out(const MmArgs &p, uint32_t m, uint32_t n, float (&v)[4]) {
    const uint32_t have = left(p.N, n);
    if (have && finish_out(p, m, n, v)) store4(p.out + m * p.ldo + n, v, have, p.vec);
}
__device__ __forceinline__ void gated(int act, const float (&g)[4], const float (&u)[4], float (&h)[4]) {
#pragma unroll
    for (int r = 0; r < 4; ++r) h[r] = activation(act, g[r], nullptr) * u[r];
}
__device__ __forceinline__ void emit_gated(const MmArgs &p, uint32_t m, uint32_t f, const float (&g)[4], const float (&u)[4]) {
    const uint32_t have = left(p.F, f);
    if (have == 0) return;
    float h[4];
    gated(p.act, g, u, h);
    store4(p.out + m * p.ldo + f, h, have, p.vec);
}
// dG and dU of four rows, of which `have` exist, from their dH.  Rows past the tensors' end are part of the
// next product's reduction: zeros.
__device__ __forceinline__ void gated_bwd(int act, uint32_t have, u32x2 dH, const float (&g)[4], const float (&u)[4],
                                          float (&dg)[4], float (&du)[4]) {
    const float dh[4] = {bf16_value(static_cast<uint16_t>(dH.x)), bf16_value(static_cast<uint16_t>(dH.x >> 16)),
                         bf16_value(static_cast<uint16_t>(dH.y)), bf16_value(static_cast<uint16_t>(dH.y >> 16))};
#pragma unroll
    for (uint32_t r = 0; r < 4; ++r) {
        float d;
        const float a = activation(act, g[r], &d);
        dg[r] = r < have ? dh[r] * u[r] * d : 0.f;
        du[r] = r < have ? dh[r] * a : 0.f;
    }
}
// gcol, ucol: their columns in G.
__device__ __forceinline__ void emit_gated_bwd(const MmArgs &p, uint32_t m, uint32_t f, uint32_t gcol, uint32_t ucol,
                                               const float (&g)[4], const float (&u)[4]) {
    const uint32_t have = left(p.F, f);
    const u32x2 dh = have ? load4(p.dH + m * p.lddh + f, have, p.vec) : (u32x2){0u, 0u};
    float dg[4], du[4];
    gated_bwd(p.act, have, dh, g, u, dg, du);
    uint16_t *G = p.G + static_cast<uint64_t>(m) * p.ldG;
    store4(G + gcol, dg, 4, true);
    store4(G + ucol, du, 4, true);
    if (have && p.dG) store4(p.dG + m * p.ldg + f, dg, have, p.vec);
    if (have && p.dU) store4(p.dU + m * p.ldg + f, du, have, p.vec);
}
// A label's column in the piece, unsigned: labels before the piece, and those that are none, whatever they
// hold, wrap past every column.
__device__ __forceinline__ uint64_t label_column(const MmArgs &p, uint32_t m) {
    return static_cast<uint64_t>(p.labels[m]) - p.f0;
}
// exp(z - lse) - [label], the columns of the next product's reduction (zeros past the piece).
__device__ __forceinline__ void prob(const MmArgs &p, uint32_t n, uint64_t lab, float lse, const float (&z)[4], float (&v)[4]) {
#pragma unroll
    for (uint32_t r = 0; r < 4; ++r)
        v[r] = n + r < p.N ? __expf(z[r] - lse) - (n + r == lab ? 1.f : 0.f) : 0.f;
}

// Eight values to out[0..7], of which `n` exist.
__device__ __forceinline__ void store8(uint16_t *out, u32x4 v, uint32_t n, bool vec) {
    if (n >= 8 && vec) {
        *reinterpret_cast<u32x4 *>(out) = v;
    } else {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (uint32_t r = 0; r < 8; ++r)
            if (r < n) out[r] = static_cast<uint16_t>(w[r >> 1] >> (16 * (r & 1)));
    }
}

// Four column fragments by transposing reads, their second halves HI bytes after the first; `at` are
// LDS addresses.  Written out because the compiler holds the transposing read back until every copy
// into LDS has landed, also those of slices still to come; the block waits for its own reads.
template <int HI>
__device__ __forceinline__ void read_columns(bf16x8_t (&x)[4], const uint32_t (&at)[4]) {
    u32x2 a0, a1, a2, a3, b0, b1, b2, b3;
    asm volatile(
        "ds_read_b64_tr_b16 %0, %8\n"
        "ds_read_b64_tr_b16 %1, %8 offset:%c12\n"
        "ds_read_b64_tr_b16 %2, %9\n"
        "ds_read_b64_tr_b16 %3, %9 offset:%c12\n"
        "ds_read_b64_tr_b16 %4, %10\n"
        "ds_read_b64_tr_b16 %5, %10 offset:%c12\n"
        "ds_read_b64_tr_b16 %6, %11\n"
        "ds_read_b64_tr_b16 %7, %11 offset:%c12\n"
        "s_waitcnt lgkmcnt(0)\n"
        : "=&v"(a0), "=&v"(b0), "=&v"(a1), "=&v"(b1), "=&v"(a2), "=&v"(b2), "=&v"(a3), "=&v"(b3)
        : "v"(at[0]), "v"(at[1]), "v"(at[2]), "v"(at[3]), "i"(HI)
        : "memory");
    x[0] = __builtin_bit_cast(bf16x8_t, (u32x4){a0.x, a0.y, b0.x, b0.y});
    x[1] = __builtin_bit_cast(bf16x8_t, (u32x4){a1.x, a1.y, b1.x, b1.y});
    x[2] = __builtin_bit_cast(bf16x8_t, (u32x4){a2.x, a2.y, b2.x, b2.y});
    x[3] = __builtin_bit_cast(bf16x8_t, (u32x4){a3.x, a3.y, b3.x, b3.y});
}

// Token and column where tile number `tile` starts: tiles are ordered in groups of 8 token tiles.
__device__ __forceinline__ void mm_tile_at(const MmArgs &p, uint32_t tile, uint32_t &m0, uint32_t &n0) {
    const uint32_t per = 8 * p.tn, grp = tile / per, g0 = grp * 8, gm = min(8u, p.tm - g0), in = tile - grp * per;
    m0 = (g0 + in % gm) * kMmTile;
    n0 = (in / gm) * kMmTile;
}

template <bool NN, int EPI>
__global__ __launch_bounds__(64 * kMmWm * kMmWn, 2) void k_mm(const MmArgs p) {
    constexpr int BM = kMmTile, BN = kMmTile, WM = kMmWm, WN = kMmWn, NW = WM * WN;
    constexpr int FM = BM / WM / 16, FN = BN / WN / 16;
    constexpr uint32_t ABYTES = BM * 64, BBYTES = BN * 64, SLICE = ABYTES + BBYTES;
    constexpr int IA = ABYTES / 1024 / NW, IB = BBYTES / 1024 / NW;
    static_assert(IA * NW * 1024 == ABYTES && IB * NW * 1024 == BBYTES && FN == 4, "whole copies, four column fragments");
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const uint32_t li = lane & 15, lg = lane >> 4;

    // Whole tiles first, then the workgroups that share the last tiles' slices evenly.  Workgroups go
    // to the 8 XCDs in turn; each XCD gets a run of consecutive whole tiles, so that its workgroups
    // share rows and columns in its L2.
    uint64_t pos, end;
    if (blockIdx.x < p.whole) {
        const uint32_t q = p.whole >> 3, rem = p.whole & 7, xcd = blockIdx.x & 7;
        pos = static_cast<uint64_t>(xcd * q + min(xcd, rem) + (blockIdx.x >> 3)) * p.ktiles;
        end = pos + p.ktiles;
    } else {
        const uint64_t shared = static_cast<uint64_t>(p.tm * p.tn - p.whole) * p.ktiles;
        const uint32_t w = blockIdx.x - p.whole, ws = gridDim.x - p.whole;
        pos = static_cast<uint64_t>(p.whole) * p.ktiles + w * shared / ws;
        end = static_cast<uint64_t>(p.whole) * p.ktiles + (w + 1) * shared / ws;
    }
    while (pos < end) {
    const uint32_t tile = static_cast<uint32_t>(pos / p.ktiles), k0 = static_cast<uint32_t>(pos - static_cast<uint64_t>(tile) * p.ktiles);
    const uint32_t kn = static_cast<uint32_t>(min(static_cast<uint64_t>(p.ktiles - k0), end - pos));
    uint32_t m0, n0;
    mm_tile_at(p, tile, m0, n0);

    // copies: this lane's byte offsets within A's and B's resources
    const auto ra = wave_rsrc(p.A + static_cast<uint64_t>(m0) * p.lda, 0x7FFFFFF0u);
    const auto rb = wave_rsrc(NN ? p.B : p.B + static_cast<uint64_t>(n0) * p.ldb, 0x7FFFFFF0u);
    uint32_t va[IA], vb[IB];
#pragma unroll
    for (int i = 0; i < IA; ++i) {
        // blocks, or rows, past M repeat the last one
        const uint32_t blk = wave + NW * i, at = lane ^ (-(lane >> 4) & 3), lda = static_cast<uint32_t>(p.lda);
        va[i] = p.blocks ? min(blk, (p.M - 1 - m0) / 16) * 32 * lda + at * 16
                         : min(blk * 16 + (at >> 2), p.M - 1 - m0) * 2 * lda + (at & 3) * 16;
    }
#pragma unroll
    for (int i = 0; i < IB; ++i) {
        if constexpr (NN) {
            const uint32_t blk = wave + NW * i, rows = blk / (BN / 32);  // columns past the piece repeat its last block
            vb[i] = rows * 32 * p.ldb + min(n0 / 32 + blk % (BN / 32), p.ldb / 32 - 1) * 1024 + (lane ^ (lane >> 5) * 2) * 16;
        } else {
            vb[i] = (wave + NW * i) * 32 * p.ldb + (lane ^ (-(lane >> 4) & 3)) * 16;
        }
    }
    const uint32_t step_a = p.blocks ? 1024 : 64, step_b = NN ? 64 * p.ldb : 1024;
    auto copy = [&](uint32_t s, uint32_t at) {
        unsigned char *to = smem + at;
#pragma unroll
        for (int i = 0; i < IA; ++i) copy_to_lds(ra, to + (wave + NW * i) * 1024, va[i], (2 * k0 + s) * step_a);
#pragma unroll
        for (int i = 0; i < IB; ++i) copy_to_lds(rb, to + ABYTES + (wave + NW * i) * 1024, vb[i], (2 * k0 + s) * step_b);
    };

    // fragment reads: byte offsets of this lane
    const uint32_t swz = (lg ^ (-(li >> 2) & 3)) * 16;
    const uint32_t fa = (wm * (BM / WM) + li) * 64 + swz, fb = ABYTES + (wn * (BN / WN) + li) * 64 + swz;
    uint32_t ft[FN];
    if constexpr (NN) {
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            const uint32_t blk = (lg >> 1) * (BN / 32) + (wn * (BN / WN) + 16 * j) / 32, r = 8 * (lg & 1) + (li >> 2);
            const uint32_t c = (2 * j + ((li & 3) >> 1)) & 3;
            ft[j] = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((CBK_LDS unsigned char *)(smem))) + ABYTES + blk * 1024 +
                    (r * 4 + (c ^ (2 * (lg & 1)))) * 16 + (li & 1) * 8;
        }
    }
    struct Frags {
        bf16x8_t a[FM], b[FN];
    };
    auto read = [&](Frags &f, uint32_t at) {
        if constexpr (NN) {
            const uint32_t t[4] = {ft[0] + at, ft[1] + at, ft[2] + at, ft[3] + at};
            read_columns<256>(f.b, t);
        } else {
#pragma unroll
            for (int j = 0; j < FN; ++j) f.b[j] = __builtin_bit_cast(bf16x8_t, *reinterpret_cast<const u32x4 *>(smem + at + fb + j * 1024));
        }
#pragma unroll
        for (int i = 0; i < FM; ++i) f.a[i] = __builtin_bit_cast(bf16x8_t, *reinterpret_cast<const u32x4 *>(smem + at + fa + i * 1024));
    };

    f32x4_t acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
    auto multiply = [&](const Frags &f) {
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f.b[j], f.a[i], acc[i][j], 0, 0, 0);
    };

    // Slices of 32 in a ring of five buffers: while slice s is multiplied from registers, s + 1 is read
    // from LDS, s + 2 has to arrive by the interval's end, s + 3 is on its way and s + 4 is asked for
    // (into the buffer of s - 1, whose reads ended before the last barrier).  Every slice is new to
    // the XCD's L2, so a copy takes the time of several intervals.  There is an even number of slices.
    constexpr int CP = IA + IB;
    const uint32_t n = kn * 2;
    Frags f0, f1;
    uint32_t ahead = 0, behind = 0;  // byte offsets of the buffers of the next copy and the next read
    auto step = [](uint32_t &at) { at = at == (kRing - 1) * SLICE ? 0u : at + SLICE; };
    for (uint32_t s = 0; s < 4 && s < n; ++s) {
        copy(s, ahead);
        step(ahead);
    }
    __builtin_amdgcn_s_waitcnt(0x0070);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    read(f0, behind);
    step(behind);
    auto interval = [&](uint32_t s, const Frags &now, Frags &next) {
        read(next, behind);              // after the last slice: old contents of a buffer, not used
        step(behind);
        copy(min(s + 4, n - 1), ahead);  // past the end: the last slice again, into a buffer that is not read
        step(ahead);
        multiply(now);
        // the reads, then the copies, between the multiplications
        constexpr int RD = NN ? FM : FM + FN, MF = FM * FN - RD;
#pragma unroll
        for (int i = 0; i < RD; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        }
#pragma unroll
        for (int i = 0; i < CP; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x008, MF / CP, 0);
        }
        __builtin_amdgcn_sched_group_barrier(0x008, MF - MF / CP * CP, 0);
        // multiplications are not put off past the barrier: their reads end before it
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt(0x0F70 | (2 * CP));
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };
    for (uint32_t s = 0; s < n; s += 2) {
        interval(s, f0, f1);
        interval(s + 1, f1, f0);
    }
    __builtin_amdgcn_s_waitcnt(0x0070);  // no copy is left in flight
    pos += kn;

    const uint32_t mw = m0 + wm * (BM / WM) + li, nw = n0 + wn * (BN / WN) + 4 * lg;  // of fragment (0, 0)
    if (EPI == kOut && kn < p.ktiles) {
        // a part of a tile: its sums, for k_mm_join
        float *part = p.part + (static_cast<uint64_t>(blockIdx.x - p.whole) + (tile - p.whole)) * (BM * BN);
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j)
                *reinterpret_cast<f32x4_t *>(part + (mw - m0 + 16 * i) * BN + (nw - n0) + 16 * j) = acc[i][j];
    } else if constexpr (EPI != kStats) {
        // The rounded tile goes through LDS, so that rows leave in 16-byte pieces next to each other.  Stored
        // from the fragments, 8 bytes a lane and with each dH waited for in turn, the gated block's backward
        // pass took 404 us on 2048 tokens of a 4096 x 11008 pair; so, 376.
        constexpr uint32_t COLS = EPI == kGated ? BN / 2 : BN, LDW = COLS + 8;
        uint16_t *st = reinterpret_cast<uint16_t *>(smem);
        u32x2 dh[FM][FN / 2];  // kGatedBwd: all of the wave's dH asked for before any is used
        if constexpr (EPI == kGatedBwd) {
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FN / 2; ++j) {
                    const uint32_t m = min(mw + 16 * i, p.M - 1), n = nw + 32 * j, f = p.f0 + (n >> 5) * 16 + (n & 15);
                    const uint32_t have = left(p.F, f);
                    dh[i][j] = have ? load4(p.dH + m * p.lddh + f, have, p.vec) : (u32x2){0u, 0u};
                }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            const uint32_t m = mw + 16 * i;
            if (m >= p.M) continue;
            uint16_t *row = st + (m - m0) * LDW;
            const uint64_t lab = EPI == kProb ? label_column(p, m) : 0;
            const float lse = EPI == kProb ? p.lse[m] : 0.f;
#pragma unroll
            for (int j = 0; j < FN; j += EPI == kGated || EPI == kGatedBwd ? 2 : 1) {
                const uint32_t n = nw + 16 * j;
                float v[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
                if constexpr (EPI == kGated || EPI == kGatedBwd) {
                    // n is gate's row of the piece, n + 16 up's; f their row in the tensors
                    const uint32_t f = p.f0 + (n >> 5) * 16 + (n & 15);
                    const float u[4] = {acc[i][j + 1][0], acc[i][j + 1][1], acc[i][j + 1][2], acc[i][j + 1][3]};
                    float x[4], y[4];
                    if constexpr (EPI == kGated) {
                        gated(p.act, v, u, x);
                        store4(row + ((n - n0) >> 5) * 16 + (n & 15), x, 4, true);
                    } else {
                        gated_bwd(p.act, left(p.F, f), dh[i][j / 2], v, u, x, y);
                        store4(row + (n - n0), x, 4, true);
                        store4(row + (n - n0) + 16, y, 4, true);
                    }
                } else if constexpr (EPI == kProb) {
                    float x[4];
                    prob(p, n, lab, lse, v, x);
                    store4(row + (n - n0), x, 4, true);
                } else if (n < p.N && finish_out(p, m, n, v)) {
                    store4(row + (n - n0), v, 4, true);
                }
            }
        }
        __syncthreads();
        if (EPI != kOut || p.last) {
            constexpr uint32_t CH = COLS / 8;
            constexpr bool kBlocks = EPI == kGatedBwd || EPI == kProb;  // G: a wave writes a block of 16 x 32
            for (uint32_t t = tid; t < BM * CH; t += 64 * NW) {
                const uint32_t blk = t >> 6;
                const uint32_t row = kBlocks ? blk / (CH / 4) * 16 + (lane >> 2) : t / CH;
                const uint32_t c = kBlocks ? (blk % (CH / 4) * 4 + (lane & 3)) * 8 : t % CH * 8;
                const uint32_t m = m0 + row;
                if (m >= p.M) continue;
                const u32x4 v = *reinterpret_cast<const u32x4 *>(st + row * LDW + c);
                if constexpr (EPI == kOut) {
                    if (n0 + c < p.N) store8(p.out + m * p.ldo + n0 + c, v, p.N - (n0 + c), p.vec16);
                } else if constexpr (EPI == kGated) {
                    const uint32_t f = p.f0 + n0 / 2 + c;
                    if (f < p.F) store8(p.out + m * p.ldo + f, v, p.F - f, p.vec16);
                } else if (n0 + c < p.ldG) {
                    *reinterpret_cast<u32x4 *>(p.G + piece_at(m, n0 + c, p.ldG)) = v;
                }
            }
        }
        if constexpr (EPI == kGatedBwd) {
            constexpr uint32_t CH = BN / 16;
            for (uint32_t t = tid; t < BM * CH; t += 64 * NW) {
                const uint32_t m = m0 + t / CH, c = t % CH, f = p.f0 + n0 / 2 + c * 8;
                if (m >= p.M || f >= p.F) continue;
                const uint16_t *src = st + (t / CH) * LDW + (c >> 1) * 32 + (c & 1) * 8;
                if (p.dG) store8(p.dG + m * p.ldg + f, *reinterpret_cast<const u32x4 *>(src), p.F - f, p.vec16);
                if (p.dU) store8(p.dU + m * p.ldg + f, *reinterpret_cast<const u32x4 *>(src + 16), p.F - f, p.vec16);
            }
        }
    } else if constexpr (EPI == kStats) {
        // each wave's part of a token's columns, then the workgroup's, in a fixed order
        f32x2 *part = reinterpret_cast<f32x2 *>(smem);  // [BM][WN]
        __syncthreads();
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            const uint32_t m = mw + 16 * i;
            uint64_t lab = ~uint64_t(0);
            if (m < p.M) lab = label_column(p, m);
            float mx = -__builtin_inff();
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
                for (uint32_t r = 0; r < 4; ++r)
                    if (nw + 16 * j + r < p.N) mx = fmaxf(mx, acc[i][j][r]);
            mx = fmaxf(mx, __shfl_xor(mx, 16, 64));
            mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
            const float base = exp_base(mx);
            float s = 0.f;
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
                for (uint32_t r = 0; r < 4; ++r) {
                    const uint32_t n = nw + 16 * j + r;
                    if (n < p.N) {
                        s += __expf(acc[i][j][r] - base);
                        if (n == lab) p.top[m] = acc[i][j][r];
                    }
                }
            s += __shfl_xor(s, 16, 64);
            s += __shfl_xor(s, 32, 64);
            if (lg == 0) part[(wm * (BM / WM) + 16 * i + li) * WN + wn] = (f32x2){mx, s};
        }
        __syncthreads();
        constexpr int W128 = 128 / (BN / WN);  // waves that share 128 columns
        for (uint32_t t = tid; t < BM * (BN / 128); t += 64 * NW) {
            const uint32_t row = t / (BN / 128), h = t % (BN / 128);
            if (m0 + row >= p.M || n0 + 128 * h >= p.N) continue;
            const f32x2 *w = part + row * WN + h * W128;
            float mx = -__builtin_inff(), s = 0.f;
#pragma unroll
            for (int i = 0; i < W128; ++i) mx = fmaxf(mx, w[i][0]);
            const float base = exp_base(mx);
#pragma unroll
            for (int i = 0; i < W128; ++i)
                if (w[i][1] != 0.f) s += w[i][1] * __expf(exp_base(w[i][0]) - base);
            p.stat[static_cast<uint64_t>(m0 + row) * p.ldstat + p.stat0 + n0 / 128 + h] = (f32x2){mx, s};
        }
    }
    // the next part's copies go to buffers that other waves may still be reading
    if (pos < end) __syncthreads();
    }
}

// The shared tiles' parts added in order.  A workgroup takes 4 tokens of a tile.  It is bound by reading
// them (2048 tokens of 4096 columns: up to 384 parts of 256 KB in 16 us).
__global__ __launch_bounds__(256) void k_mm_join(const MmArgs p, uint32_t sharers) {
    const uint32_t tile = p.whole + blockIdx.x, row = blockIdx.y * 4 + (threadIdx.x >> 6), c = (threadIdx.x & 63) * 4;
    uint32_t m0, n0;
    mm_tile_at(p, tile, m0, n0);
    if (m0 + row >= p.M) return;
    // run w starts at floor(w * total / sharers)
    const uint64_t total = static_cast<uint64_t>(p.tm * p.tn - p.whole) * p.ktiles, at = static_cast<uint64_t>(blockIdx.x) * p.ktiles;
    const uint32_t g0 = static_cast<uint32_t>(((at + 1) * sharers - 1) / total);
    const uint32_t g1 = static_cast<uint32_t>(((at + p.ktiles) * sharers - 1) / total);
    if (g0 == g1) return;  // one workgroup had it whole
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    for (uint32_t g = g0; g <= g1; ++g) {
        const f32x4_t t = *reinterpret_cast<const f32x4_t *>(p.part + static_cast<uint64_t>(g + blockIdx.x) * (kMmTile * kMmTile) + row * kMmTile + c);
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] += t[r];
    }
    emit_out(p, m0 + row, n0 + c, v);
}

// The parts of a tile that k_fused left, added in order, and the operator's work on the sums.  A
// workgroup takes 8 tokens of a tile, 32 lanes of 4 columns each.  With few tokens it takes the 4 us that a
// launch does; with many it is bound by reading the parts (300 tokens of 42752 rows, 110 MB with its
// output: 22 us).  `count` 2: the second tensor's tile
// holds the up sums of the same columns (forward), or the second half of one sum (gradient).
struct JoinArgs {
    const float *part;
    uint32_t count, tiles, slices, grid, up_col;  // up_col: where dU starts in G
    uint32_t split;  // each tensor's parts by themselves, the second's after grid + tiles of the first's
};

// The sum of tile vt's parts at token m, columns c..c + 3, added to v, up to MOST loads at a time.  16 save a
// short product's tiles of a dozen parts some round trips (1001 x 2730, 45 tokens: 5.3 us against 7.8 by 4);
// a head's many tiles have two or three parts, where the registers cost waves (25 us against 22).
template <uint32_t MOST>
__device__ __forceinline__ void add_parts(const JoinArgs &q, uint32_t M, uint32_t vt, uint32_t m, uint32_t c, float (&v)[4]) {
    const uint32_t runs = q.split ? 1 : q.count;  // tensors that a launch's runs go through
    uint64_t slot = vt;
    if (q.split && vt >= q.tiles) {
        vt -= q.tiles;
        slot += q.grid;
    }
    // The workgroups whose runs hold the tile's first and last slice: run g starts at
    // floor(g * total / grid).
    const uint64_t total = static_cast<uint64_t>(runs * q.tiles) * q.slices, at = static_cast<uint64_t>(vt) * q.slices;
    const uint32_t g0 = static_cast<uint32_t>(quotient((at + 1) * q.grid - 1, total));
    const uint32_t g1 = static_cast<uint32_t>(quotient((at + q.slices) * q.grid - 1, total));
    const float *src = q.part + (slot * M + m) * kFusedTile + c;
    // (past the end the last part again)
    auto add = [&](auto batch) {
        constexpr uint32_t N = decltype(batch)::value;
        for (uint32_t g = g0; g <= g1; g += N) {
            f32x4_t t[N];
#pragma unroll
            for (uint32_t k = 0; k < N; ++k)
                t[k] = *reinterpret_cast<const f32x4_t *>(src + static_cast<uint64_t>(min(g + k, g1)) * M * kFusedTile);
#pragma unroll
            for (uint32_t k = 0; k < N; ++k)
                if (g + k <= g1) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) v[r] += t[k][r];
                }
        }
    };
    if (MOST == 4 || g1 - g0 < 4)
        add(std::integral_constant<uint32_t, 4>{});
    else
        add(std::integral_constant<uint32_t, MOST>{});
}

template <int EPI>
__global__ __launch_bounds__(256) void k_join(const MmArgs p, const JoinArgs q) {
    const uint32_t tile = blockIdx.x, m = blockIdx.y * 8 + threadIdx.x / 32, c = threadIdx.x % 32 * 4;
    if (m >= p.M) return;
    constexpr uint32_t MOST = EPI == kStats || EPI == kProb ? 4 : 16;
    float v[4] = {0.f, 0.f, 0.f, 0.f}, u[4] = {0.f, 0.f, 0.f, 0.f};
    add_parts<MOST>(q, p.M, tile, m, c, v);
    if constexpr (EPI == kGated || EPI == kGatedBwd)
        add_parts<MOST>(q, p.M, q.tiles + tile, m, c, u);
    else if (EPI == kOut && q.count == 2)
        add_parts<MOST>(q, p.M, q.tiles + tile, m, c, v);
    const uint32_t n = tile * kFusedTile + c;
    if constexpr (EPI == kOut) {
        emit_out(p, m, n, v);
    } else if constexpr (EPI == kGated) {
        emit_gated(p, m, p.f0 + n, v, u);
    } else if constexpr (EPI == kGatedBwd) {
        if (n < q.up_col) emit_gated_bwd(p, m, p.f0 + n, n, q.up_col + n, v, u);
    } else if constexpr (EPI == kProb) {
        float x[4];
        prob(p, n, label_column(p, m), p.lse[m], v, x);
        store4(p.G + static_cast<uint64_t>(m) * p.ldG + n, x, 4, true);
    } else {
        const uint64_t lab = label_column(p, m);
        float mx = -__builtin_inff(), s = 0.f;
#pragma unroll
        for (uint32_t r = 0; r < 4; ++r)
            if (n + r < p.N) mx = fmaxf(mx, v[r]);
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) mx = fmaxf(mx, __shfl_xor(mx, o, 64));
        const float base = exp_base(mx);
#pragma unroll
        for (uint32_t r = 0; r < 4; ++r)
            if (n + r < p.N) {
                s += __expf(v[r] - base);
                if (n + r == lab) p.top[m] = v[r];
            }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) s += __shfl_xor(s, o, 64);
        if (c == 0) p.stat[static_cast<uint64_t>(m) * p.ldstat + p.stat0 + tile] = (f32x2){mx, s};
    }
}

// The parts of a token's softmax statistics joined in order, one wave a token: lse, and the loss.
__global__ __launch_bounds__(256) void k_xent_join(const f32x2 *__restrict__ stat, uint32_t parts, uint32_t M,
                                                   const int64_t *__restrict__ labels, int64_t ignore, uint64_t V,
                                                   const float *__restrict__ top, float *__restrict__ loss,
                                                   float *__restrict__ lse) {
    const uint32_t m = blockIdx.x * 4 + (threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    if (m >= M) return;
    const f32x2 *row = stat + static_cast<uint64_t>(m) * parts;
    float mx = -__builtin_inff();
    for (uint32_t i = lane; i < parts; i += 64) mx = fmaxf(mx, row[i][0]);
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) mx = fmaxf(mx, __shfl_xor(mx, o, 64));
    const float base = exp_base(mx);
    float s = 0.f;
    for (uint32_t i = lane; i < parts; i += 64) {
        const f32x2 t = row[i];
        if (t[1] != 0.f) s += t[1] * __expf(exp_base(t[0]) - base);
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) s += __shfl_xor(s, o, 64);
    if (lane == 0) {
        const float l = base + logf(s);
        const int64_t lab = labels[m];
        lse[m] = l;
        loss[m] = lab == ignore ? 0.f
                  : lab >= 0 && static_cast<uint64_t>(lab) < V ? l - top[m]
                                                               : __builtin_nanf("");
    }
}

// ------------------------------------------------------------------------------- host side

uint32_t grid_for(uint64_t items, uint32_t per) {
    return static_cast<uint32_t>(std::max<uint64_t>(1, std::min<uint64_t>((items + per - 1) / per, 65536)));
}

template <bool, int>
struct MmTag;
template <int, bool>
struct UnpackTag;

struct UnpackRunArgs {
    UnpackArgs a;
    uint32_t count;
    hipStream_t s;
    cbk_status st;
};

template <int B>
struct UnpackRun {
    static bool run(UnpackRunArgs &r) {
        using G = U64<B>;
        constexpr uint32_t stage = G::STAGE_CHUNKS * 16 > 64 * 144 ? G::STAGE_CHUNKS * 16 : 64 * 144;
        constexpr uint32_t lds = kUnpackWaves * stage;
        r.a.steps = ceil_div(static_cast<uint64_t>(r.a.nrows) * r.a.cols, 4096);
        // two workgroups per CU, whose waves take every n-th step
        const dim3 grid(std::min(ceil_div(r.a.steps, kUnpackWaves), std::max(1u, 2 * static_cast<uint32_t>(cu_count()) / r.count)), r.count);
        if (r.a.cols % 8 == 0) {
            if (!allow_lds_once<UnpackTag<B, true>>(k_unpack<B, true>, lds)) return false;
            hipLaunchKernelGGL((k_unpack<B, true>), grid, dim3(64 * kUnpackWaves), lds, r.s, r.a);
        } else {
            if (!allow_lds_once<UnpackTag<B, false>>(k_unpack<B, false>, lds)) return false;
            hipLaunchKernelGGL((k_unpack<B, false>), grid, dim3(64 * kUnpackWaves), lds, r.s, r.a);
        }
        r.st = launched();
        return true;
    }
};
using UnpackB = std::integer_sequence<int, 1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 13, 14, 15>;

// Rows [row0, row0 + nrows) of one tensor, or of a pair, into rows_out rows each of the piece.
cbk_status unpack(const cbk_tensor *const *ts, uint32_t count, uint64_t row0, uint64_t nrows, uint64_t rows_out,
                  uint64_t Kp, uint16_t *out, hipStream_t s) {
    UnpackRunArgs r{};
    r.s = s;
    r.a.cols = static_cast<uint32_t>(ts[0]->cols);
    r.a.Kp = static_cast<uint32_t>(Kp);
    r.a.row0 = row0;
    r.a.nrows = static_cast<uint32_t>(nrows);
    r.a.rows_out = static_cast<uint32_t>(rows_out);
    r.a.pair = count == 2 ? 2 : 0;
    r.a.out = out;
    r.a.inv_cols = 1.f / static_cast<float>(std::max(1u, r.a.cols));
    bool fast = true;
    for (uint32_t i = 0; i < count; ++i) {
        const cbk_tensor &t = *ts[i];
        r.a.t[i] = UnpackTensor{t.words, t.codebook, t.U, static_cast<uint32_t>(cbk_words_for(t.rows * t.cols, t.b) / 4)};
        fast = fast && nn_unpack_in_order(t, row0, nrows);
    }
    if (fast) {
        const bool together = count == 1 || ts[0]->b == ts[1]->b;
        for (uint32_t i = 0; i < count && fast; i += together ? count : 1) {
            UnpackRunArgs one = r;
            one.count = together ? count : 1;
            one.a.b = ts[i]->b;
            if (!together) {
                // a tensor of the pair by itself: as the pair's first, written where it belongs
                one.a.t[0] = r.a.t[i];
                one.a.out = out + i * 16 * Kp;
            }
            fast = dispatch_b<UnpackRun>(static_cast<int>(one.a.b), one, UnpackB{});
            if (fast && one.st != CBK_OK) return one.st;
        }
        if (fast) {
            if (r.a.cols == Kp && nrows == rows_out) return CBK_OK;
            hipLaunchKernelGGL(k_unpack_pad, dim3(std::min<uint32_t>(r.a.rows_out, 4096)), dim3(256), 0, s, r.a);
            return launched();
        }
    }
    for (uint32_t i = 0; i < count; ++i) {
        UnpackArgs a = r.a;
        a.t[0] = r.a.t[i];
        a.b = ts[i]->b;
        a.pair = count == 2 ? i + 1 : 0;
        hipLaunchKernelGGL(k_unpack_generic, dim3(grid_for(rows_out * (Kp / 4), 256)), dim3(256), 0, s, a);
        CBK_TRY(launched());
    }
    return CBK_OK;
}

// `columns`: the columns of C to cover.
template <bool NN, int EPI>
cbk_status mm(MmArgs &p, uint32_t columns, hipStream_t s) {
    constexpr uint32_t lds = kRing * 2 * kMmTile * 64;
    if (!allow_lds_once<MmTag<NN, EPI>>(k_mm<NN, EPI>, lds)) return CBK_E_HIP;
    p.tm = ceil_div(p.M, kMmTile);
    p.tn = ceil_div(columns, kMmTile);
    const uint32_t tiles = p.tm * p.tn, cus = 256;
    // One workgroup runs on a CU, so the tiles are done in rounds of 256.  What is left over after
    // the whole rounds is shared by a round's workgroups where that pays for writing and adding its
    // parts (about 0.12 us a part, where a slice of 64 takes 1.9 us a round).
    uint32_t sharers = 0;
    p.whole = tiles;
    if (EPI == kOut) {
        const uint32_t over = tiles % cus;
        if (over > 0 && over <= kMmShared) {
            const double saved = (1.0 - static_cast<double>(over) / cus) * p.ktiles * 1.9;
            if (saved > 0.12 * (cus + over) + 5.0) {
                sharers = static_cast<uint32_t>(std::min<uint64_t>(cus, static_cast<uint64_t>(over) * p.ktiles / 4));
                p.whole = tiles - over;
            }
        }
    }
    hipLaunchKernelGGL((k_mm<NN, EPI>), dim3(p.whole + sharers), dim3(64 * kMmWm * kMmWn), lds, s, p);
    CBK_TRY(launched());
    if (sharers == 0) return CBK_OK;
    hipLaunchKernelGGL(k_mm_join, dim3(tiles - p.whole, kMmTile / 4), dim3(256), 0, s, p, sharers);
    return launched();
}

bool vec8(const void *p, uint64_t ld) { return aligned_to(p, 8) && ld % 4 == 0; }
bool vec16(const void *p, uint64_t ld) { return aligned_to(p, 16) && ld % 8 == 0; }

// The tokens' side of a product: used as it is if the copies to LDS can read whole 64-wide slices of it
// (16-byte aligned rows, no ragged end, and 384 rows within 31 bits), else a copy in P, padded for k_fused
// and in blocks for k_mm.  k_mm's forward product takes the blocks in any case (2048 tokens and 32000 rows
// of 4096: 7 us for the copy, 404 us instead of 425 for the product); its gradient reads the weights in longer
// rows and gains nothing (2048 tokens of 4096, 11008 columns: 182 us either way).
cbk_status token_side(MmArgs &p, bool fused, bool nn, const uint16_t *X, uint64_t ld, uint64_t T, uint64_t K, uint64_t Kp,
                      uint16_t *P, hipStream_t s) {
    const uint32_t k = static_cast<uint32_t>(K), kp = static_cast<uint32_t>(Kp);
    p.blocks = 0;
    if ((fused || nn) && K == Kp && vec16(X, ld) && ld <= (uint64_t(1) << 21)) {
        p.A = X;
        p.lda = ld;
        return CBK_OK;
    }
    p.A = P;
    p.lda = Kp;
    if (fused) {
        hipLaunchKernelGGL(k_pad_rows, dim3(grid_for(T * (Kp / 4), 256)), dim3(256), 0, s, X, ld, T, k, kp, P);
    } else {
        p.blocks = 1;
        hipLaunchKernelGGL(k_pack_rows, dim3(grid_for((T + 15) / 16 * (Kp / 32) * 64, 256)), dim3(256), 0, s, X, ld,
                           static_cast<uint32_t>(T), k, kp, vec16(X, ld) ? 1u : 0u, P);
    }
    return launched();
}

uint64_t up64(uint64_t n) { return (n + 63) / 64 * 64; }

template <typename T>
T *at(void *ws, uint64_t offset) { return reinterpret_cast<T *>(static_cast<unsigned char *>(ws) + offset); }

cbk_status zero_rows(uint16_t *out, uint64_t ld, uint64_t T, uint64_t n, hipStream_t s) {
    hipLaunchKernelGGL(k_zero_rows, dim3(grid_for(T * n, 256)), dim3(256), 0, s, out, ld, T, static_cast<uint32_t>(n));
    return launched();
}

// Decoded rows of a piece that holds `nrows` rows of each of its tensors, rounded up to what a
// reduction over them takes.
uint64_t piece_rows(uint64_t nrows, bool pair) { return pair ? up64(2 * ((nrows + 15) / 16 * 16)) : up64(nrows); }

cbk_status unpack_piece(const cbk_tensor *const *ts, int count, uint64_t row0, uint64_t nrows, uint64_t Kp, uint16_t *W,
                        hipStream_t s) {
    return unpack(ts, count, row0, nrows, piece_rows(nrows, count == 2) / count, Kp, W, s);
}

}  // namespace

namespace {

struct FusedRunArgs {
    FusedArgs a;
    uint32_t bm;
    bool nn;
    hipStream_t s;
    cbk_status st;
};
template <int B>
struct FusedRun {
    static bool run(FusedRunArgs &r) {
        r.st = launch_fused<B>(r.a, r.bm, r.nn, r.s);
        return true;
    }
};
using FusedB = std::integer_sequence<int, 8, 9, 10, 11, 12, 13, 14>;

// The weights of a call, decoded on the way (k_fused) or a piece at a time into the workspace, and
// the products with a piece of them.
struct Weights {
    const cbk_tensor *ts[2];
    uint32_t count;
    NnPlan pl;
    void *ws;
    hipStream_t s;
    uint64_t row0, nrows;  // the piece

    // Rows of the piece's reduction: as the decoded rows lie (both tensors' rows in turns of 16), or,
    // for k_fused, each tensor's rows rounded up to a slice.
    uint64_t reduction() const {
        if (pl.fused) return count * up64(nrows);
        return piece_rows(nrows, count == 2);
    }

    cbk_status piece(uint64_t r) {
        row0 = r;
        nrows = std::min(pl.rows, ts[0]->rows - r);
        return pl.fused ? CBK_OK : unpack_piece(ts, count, row0, nrows, pl.Kp, at<uint16_t>(ws, pl.w), s);
    }
    bool last() const { return row0 + nrows == ts[0]->rows; }

    cbk_status fused(MmArgs &p, bool nn, JoinArgs &q) const {
        FusedRunArgs r{};
        FusedArgs &a = r.a;
        for (uint32_t i = 0; i < count; ++i)
            a.t[i] = FusedTensor{ts[i]->words, ts[i]->codebook, cbk_words_for(ts[i]->rows * ts[i]->cols, ts[i]->b) * 4, ts[i]->U, 0};
        const uint32_t launches = pl.split ? 2 : 1;
        a.count = count / launches;
        a.A = p.A;
        a.lda = p.lda;
        a.M = p.M;
        a.row0 = row0;
        a.nrows = static_cast<uint32_t>(nrows);
        a.cols = static_cast<uint32_t>(ts[0]->cols);
        a.tiles = ceil_div(nn ? pl.Kp : nrows, kFusedTile);
        a.slices = static_cast<uint32_t>((nn ? up64(nrows) : pl.Kp) / 64);
        // Even rounds of the CUs where each workgroup gets eight slices, so that the start of its pipeline is
        // paid for (a 4096 x 4096 gradient of 8 tokens: 16.7 us with 256 workgroups of eight, 19.4 with 512
        // of four, 23 with 341 of six); below that, three slices each.
        const uint64_t total = static_cast<uint64_t>(a.count * a.tiles) * a.slices;
        a.grid = static_cast<uint32_t>(total >= 8 * pl.grid ? pl.grid : std::max<uint64_t>(1, std::min<uint64_t>(256, total / 3)));
        a.part = at<float>(ws, pl.part);
        r.bm = pl.fused;
        r.nn = nn;
        r.s = s;
        q = JoinArgs{a.part, count, a.tiles, a.slices, a.grid, static_cast<uint32_t>(up64(nrows)), pl.split};
        for (uint32_t i = 0; i < launches; ++i) {
            if (i > 0) {
                a.t[0] = a.t[1];
                if (nn) a.A += a.slices * 64;
                a.part += static_cast<uint64_t>(a.grid + a.tiles) * a.M * kFusedTile;
            }
            if (!dispatch_b<FusedRun>(static_cast<int>(ts[i]->b), r, FusedB{})) return CBK_E_UNSUPPORTED;
            CBK_TRY(r.st);
        }
        return CBK_OK;
    }

    template <int EPI>
    cbk_status join(MmArgs &p, const JoinArgs &q) const {
        hipLaunchKernelGGL((k_join<EPI>), dim3(q.tiles, ceil_div(p.M, 8)), dim3(256), 0, s, p, q);
        return launched();
    }

    // One token: the batch-1 GEMV, whose rows' sums lie as one part of every tile.  It streams the index
    // words of whole rows (a pair of 4096 x 11008: 30 us against 44 by k_fused).
    bool one_token(const MmArgs &p) const { return pl.fused && p.M == 1 && ts[0]->cols % 64 == 0 && ts[0]->cols <= 16384; }

    cbk_status gemv(const MmArgs &p, JoinArgs &q) const {
        const uint32_t tiles = ceil_div(nrows, kFusedTile);
        cbk_tensor piece[2];
        float *ys[2];
        for (uint32_t i = 0; i < count; ++i) {
            piece[i] = *ts[i];
            piece[i].rows = nrows;
            piece[i].words += row0 * piece[i].cols / 32 * piece[i].b;  // row0 is a multiple of 128: whole 16-byte chunks
            ys[i] = at<float>(ws, pl.part) + i * tiles * kFusedTile;
        }
        q = JoinArgs{at<float>(ws, pl.part), count, tiles, 1, 1, static_cast<uint32_t>(up64(nrows)), 0};
        return launch_gemv_group(piece, count, p.A, ys, s);
    }

    // C = A . (piece)^T with the epilogue EPI.
    template <int EPI>
    cbk_status forward(MmArgs &p) const {
        if (pl.fused) {
            JoinArgs q;
            CBK_TRY(one_token(p) ? gemv(p, q) : fused(p, false, q));
            return join<EPI>(p, q);
        }
        p.B = at<uint16_t>(ws, pl.w);
        p.part = at<float>(ws, pl.part);
        p.ldb = static_cast<uint32_t>(pl.Kp);
        p.ktiles = static_cast<uint32_t>(pl.Kp / 64);
        const uint64_t rows = piece_rows(nrows, count == 2);
        if (EPI == kGated || EPI == kGatedBwd) p.N = static_cast<uint32_t>(rows);
        return mm<false, EPI>(p, EPI == kProb ? static_cast<uint32_t>(rows) : p.N, s);
    }

    // The piece's part of dX = A . (piece), summed over the pieces in fp32; rounded with the last.
    cbk_status gradient(MmArgs &p, uint16_t *dX, uint64_t lddx) const {
        p.N = static_cast<uint32_t>(ts[0]->cols);
        p.acc = at<float>(ws, pl.acc);
        p.ldacc = static_cast<uint32_t>(pl.Kp);
        p.acc_in = row0 != 0;
        p.last = last();
        p.out = dX;
        p.ldo = lddx;
        p.vec = vec8(dX, lddx);
        p.vec16 = vec16(dX, lddx);
        if (pl.fused) {
            JoinArgs q;
            CBK_TRY(fused(p, true, q));
            return join<kOut>(p, q);
        }
        p.B = at<uint16_t>(ws, pl.w);
        p.part = at<float>(ws, pl.part);
        p.ldb = static_cast<uint32_t>(pl.Kp);
        p.ktiles = static_cast<uint32_t>(reduction() / 64);
        return mm<true, kOut>(p, p.N, s);
    }
};

Weights weights_of(NnOp op, const cbk_tensor *a, const cbk_tensor *b, uint64_t T, void *ws, hipStream_t s) {
    Weights w{};
    w.ts[0] = a;
    w.ts[1] = b;
    w.count = b ? 2 : 1;
    w.pl = nn_plan(op, w.ts, T);
    w.ws = ws;
    w.s = s;
    return w;
}

}  // namespace

cbk_status launch_linear(const cbk_tensor &t, const uint16_t *X, uint64_t ldx, uint64_t T, uint16_t *Y, uint64_t ldy,
                         void *ws, hipStream_t s) {
    Weights w = weights_of(NnOp::linear, &t, nullptr, T, ws, s);
    const NnPlan &pl = w.pl;
    for (uint64_t c = 0; c < T; c += pl.Tc) {
        MmArgs p{};
        p.M = static_cast<uint32_t>(std::min(pl.Tc, T - c));
        CBK_TRY(token_side(p, pl.fused, false, X + c * ldx, ldx, p.M, t.cols, pl.Kp, at<uint16_t>(ws, pl.pack), s));
        for (uint64_t r = 0; r < t.rows; r += pl.rows) {
            CBK_TRY(w.piece(r));
            p.N = static_cast<uint32_t>(w.nrows);
            p.out = Y + c * ldy + r;
            p.ldo = ldy;
            p.vec = vec8(p.out, ldy);
            p.vec16 = vec16(p.out, ldy);
            p.last = 1;
            CBK_TRY(w.forward<kOut>(p));
        }
    }
    return CBK_OK;
}

cbk_status launch_linear_dx(const cbk_tensor &t, const uint16_t *dY, uint64_t lddy, uint64_t T, uint16_t *dX,
                            uint64_t lddx, void *ws, hipStream_t s) {
    if (t.rows == 0) return zero_rows(dX, lddx, T, t.cols, s);
    Weights w = weights_of(NnOp::linear, &t, nullptr, T, ws, s);
    const NnPlan &pl = w.pl;
    for (uint64_t c = 0; c < T; c += pl.Tc) {
        MmArgs p{};
        p.M = static_cast<uint32_t>(std::min(pl.Tc, T - c));
        for (uint64_t r = 0; r < t.rows; r += pl.rows) {
            CBK_TRY(w.piece(r));
            CBK_TRY(token_side(p, pl.fused, true, dY + c * lddy + r, lddy, p.M, w.nrows, up64(w.nrows), at<uint16_t>(ws, pl.pack), s));
            CBK_TRY(w.gradient(p, dX + c * lddx, lddx));
        }
    }
    return CBK_OK;
}

cbk_status launch_ffn(const cbk_tensor &gate, const cbk_tensor &up, int act, const uint16_t *X, uint64_t ldx, uint64_t T,
                      uint16_t *H, uint64_t ldh, void *ws, hipStream_t s) {
    Weights w = weights_of(NnOp::ffn, &gate, &up, T, ws, s);
    const NnPlan &pl = w.pl;
    for (uint64_t c = 0; c < T; c += pl.Tc) {
        MmArgs p{};
        p.M = static_cast<uint32_t>(std::min(pl.Tc, T - c));
        CBK_TRY(token_side(p, pl.fused, false, X + c * ldx, ldx, p.M, gate.cols, pl.Kp, at<uint16_t>(ws, pl.pack), s));
        p.act = act;
        p.F = static_cast<uint32_t>(gate.rows);
        p.out = H + c * ldh;
        p.ldo = ldh;
        p.vec = vec8(p.out, ldh);
        p.vec16 = vec16(p.out, ldh);
        for (uint64_t r = 0; r < gate.rows; r += pl.rows) {
            CBK_TRY(w.piece(r));
            p.f0 = static_cast<uint32_t>(r);
            CBK_TRY(w.forward<kGated>(p));
        }
    }
    return CBK_OK;
}

cbk_status launch_ffn_bwd(const cbk_tensor &gate, const cbk_tensor &up, int act, const uint16_t *X, uint64_t ldx,
                          const uint16_t *dH, uint64_t lddh, uint64_t T, uint16_t *dX, uint64_t lddx, uint16_t *dG,
                          uint16_t *dU, uint64_t ldg, void *ws, hipStream_t s) {
    if (gate.rows == 0) return gate.cols == 0 ? CBK_OK : zero_rows(dX, lddx, T, gate.cols, s);
    Weights w = weights_of(NnOp::ffn, &gate, &up, T, ws, s);
    const NnPlan &pl = w.pl;
    for (uint64_t c = 0; c < T; c += pl.Tc) {
        MmArgs p{};
        p.M = static_cast<uint32_t>(std::min(pl.Tc, T - c));
        CBK_TRY(token_side(p, pl.fused, false, X + c * ldx, ldx, p.M, gate.cols, pl.Kp, at<uint16_t>(ws, pl.pack), s));
        p.act = act;
        p.F = static_cast<uint32_t>(gate.rows);
        p.dH = dH + c * lddh;
        p.lddh = lddh;
        p.dG = dG ? dG + c * ldg : nullptr;
        p.dU = dU ? dU + c * ldg : nullptr;
        p.ldg = ldg;
        p.vec = vec8(p.dH, lddh) && (!dG || vec8(p.dG, ldg)) && (!dU || vec8(p.dU, ldg));
        p.vec16 = (!dG || vec16(p.dG, ldg)) && (!dU || vec16(p.dU, ldg));  // of the outputs
        p.G = at<uint16_t>(ws, pl.g);
        for (uint64_t r = 0; r < gate.rows; r += pl.rows) {
            CBK_TRY(w.piece(r));
            p.f0 = static_cast<uint32_t>(r);
            p.ldG = static_cast<uint32_t>(w.reduction());
            CBK_TRY(w.forward<kGatedBwd>(p));
            if (gate.cols == 0) continue;
            MmArgs d{};
            d.M = p.M;
            d.A = p.G;
            d.lda = p.ldG;
            d.blocks = !pl.fused;
            CBK_TRY(w.gradient(d, dX + c * lddx, lddx));
        }
    }
    return CBK_OK;
}

cbk_status launch_xent(const cbk_tensor &head, const uint16_t *X, uint64_t ldx, const int64_t *labels, uint64_t T,
                       int64_t ignore, float *loss, float *lse, void *ws, hipStream_t s) {
    Weights w = weights_of(NnOp::xent, &head, nullptr, T, ws, s);
    const NnPlan &pl = w.pl;
    for (uint64_t c = 0; c < T; c += pl.Tc) {
        MmArgs p{};
        p.M = static_cast<uint32_t>(std::min(pl.Tc, T - c));
        CBK_TRY(token_side(p, pl.fused, false, X + c * ldx, ldx, p.M, head.cols, pl.Kp, at<uint16_t>(ws, pl.pack), s));
        p.stat = at<f32x2>(ws, pl.stat);
        p.top = at<float>(ws, pl.top);
        p.labels = labels + c;
        constexpr uint32_t kTile = 128;  // columns of a part of the statistics
        p.ldstat = 0;
        for (uint64_t r = 0; r < head.rows; r += pl.rows) p.ldstat += ceil_div(std::min(pl.rows, head.rows - r), kTile);
        for (uint64_t r = 0; r < head.rows; r += pl.rows) {
            CBK_TRY(w.piece(r));
            p.N = static_cast<uint32_t>(w.nrows);
            p.f0 = static_cast<uint32_t>(r);
            CBK_TRY(w.forward<kStats>(p));
            p.stat0 += ceil_div(w.nrows, kTile);
        }
        hipLaunchKernelGGL(k_xent_join, dim3((p.M + 3) / 4), dim3(256), 0, s, p.stat, p.ldstat, p.M, p.labels, ignore,
                           head.rows, p.top, loss + c, lse + c);
        CBK_TRY(launched());
    }
    return CBK_OK;
}

cbk_status launch_xent_bwd(const cbk_tensor &head, const uint16_t *X, uint64_t ldx, const int64_t *labels,
                           const float *lse, const float *dloss, uint64_t T, int64_t ignore, uint16_t *dX,
                           uint64_t lddx, void *ws, hipStream_t s) {
    Weights w = weights_of(NnOp::xent, &head, nullptr, T, ws, s);
    const NnPlan &pl = w.pl;
    for (uint64_t c = 0; c < T; c += pl.Tc) {
        MmArgs p{};
        p.M = static_cast<uint32_t>(std::min(pl.Tc, T - c));
        CBK_TRY(token_side(p, pl.fused, false, X + c * ldx, ldx, p.M, head.cols, pl.Kp, at<uint16_t>(ws, pl.pack), s));
        p.labels = labels + c;
        p.lse = lse + c;
        p.G = at<uint16_t>(ws, pl.g);
        p.ldG = static_cast<uint32_t>(pl.Rp);
        for (uint64_t r = 0; r < head.rows; r += pl.rows) {
            CBK_TRY(w.piece(r));
            p.N = static_cast<uint32_t>(w.nrows);
            p.f0 = static_cast<uint32_t>(r);
            CBK_TRY(w.forward<kProb>(p));
            MmArgs d{};
            d.M = p.M;
            d.A = p.G;
            d.lda = p.ldG;
            d.blocks = !pl.fused;
            d.labels = p.labels;
            d.ignore = ignore;
            d.scale = dloss + c;
            d.V = head.rows;
            CBK_TRY(w.gradient(d, dX + c * lddx, lddx));
        }
    }
    return CBK_OK;
}

}  // namespace cbk
