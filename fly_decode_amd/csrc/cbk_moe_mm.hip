// The experts' products of cbk_moe.h for gfx950 (CDNA4): codebook-compressed weights of every expert that tokens were
// routed to, decoded on the way to the matrix cores.
//
// Units of work.  A workgroup takes one token tile (slots of one expert, as k_sort cut them) and one tile of columns of
// the result: forward (NN false) rows of a tensor, or half as many of gate and of up side by side (PAIR), so that a lane
// has a hidden column's two sums; gradient (NN true) columns of a tensor, over gate's rows and then up's (PAIR).  It holds
// the sums of the whole reduction, so the operator's work is its epilogue and nothing is joined; where units are few
// (splits) a reduction's shares lie side by side in S and are added by who reads them.  How many tiles there are is known
// on the device alone: the grid covers the most there can be, and workgroups past them end.
//
// Widths.  The index width is read from the tensor's record and the same code takes all of 0 to 16: experts, and the two
// tensors of a pair, may differ in it, which tensors of some 2^12 distinct patterns do by chance.  Fields are taken in
// groups of 4, at most 64 bits: 3 dwords cover a group wherever it starts; 12 operations find its four table offsets.
// (Static widths would save some of the shifts, and would need a launch for each width among the experts.)  Tables lie in
// LDS; those of 2^15 and 2^16 entries do not fit beside the slices and are read through the caches (GT).
//
// Three kernels, by the number of tokens that an expert has (ex_plan): k_experts_few, k_experts, k_experts_many.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "cbk_moe_device.h"

namespace cbk {
namespace {

enum Epi { kSum, kHidden, kHiddenBwd };

// A tensor's table of 2^b entries (b <= 14), those from U on corrupt, into LDS by 512 threads: up to 4 chunks of 8 entries
// each, and the chunk that U falls into by 8 threads, all asked for by load() before store() waits for any.
struct TableLoad {
    u32x4 v[4];
    uint32_t chunks, full, tid, last;
    uint16_t *to;

    __device__ __forceinline__ void load(unsigned char *table, const ExTensor &T, uint32_t thread) {
        to = reinterpret_cast<uint16_t *>(table);
        tid = thread;
        chunks = ((1u << T.b) + 7) / 8;
        // (a codebook that is not aligned is read entry by entry, and has no whole chunks here)
        full = (reinterpret_cast<uintptr_t>(T.cb) & 15) == 0 ? T.U / 8 : 0;
        const uint32_t corrupt = static_cast<uint32_t>(kCorrupt) * 0x10001u;
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i) {
            v[i] = (u32x4){corrupt, corrupt, corrupt, corrupt};
            if (i * 512 + tid < full) v[i] = reinterpret_cast<const u32x4 *>(T.cb)[i * 512 + tid];
        }
        last = kCorrupt;
        if (tid < 8 && 8 * full + tid < T.U) last = T.cb[8 * full + tid];
    }
    __device__ __forceinline__ void store(const ExTensor &T) const {
        const bool aligned = (reinterpret_cast<uintptr_t>(T.cb) & 15) == 0;
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i) {
            const uint32_t c = i * 512 + tid;
            if (c < chunks && c != full) reinterpret_cast<u32x4 *>(to)[c] = v[i];
        }
        if (aligned) {
            if (tid < 8 && full < chunks) to[8 * full + tid] = static_cast<uint16_t>(last);
        } else {
            lds_barrier();
            for (uint32_t i = tid; i < 8 * chunks; i += 512) to[i] = i < T.U ? T.cb[i] : kCorrupt;
        }
    }
};
__device__ __forceinline__ void stage_table(unsigned char *table, const ExTensor &T, uint32_t tid) {
    TableLoad l;
    l.load(table, T, tid);
    l.store(T);
}
__device__ __forceinline__ void stage_tables(unsigned char *first, const ExTensor &T0, unsigned char *second, const ExTensor &T1, uint32_t tid) {
    TableLoad l0, l1;
    l0.load(first, T0, tid);
    l1.load(second, T1, tid);
    l0.store(T0);
    l1.store(T1);
}

// Twice the four fields (byte offsets into a table) of b bits that start at bit `shift` of d; m2 = 2 (2^b - 1).
__device__ __forceinline__ void fields4(u32x3 d, uint32_t shift, uint32_t b, uint32_t m2, uint32_t (&off)[4]) {
    const uint32_t lo = __builtin_amdgcn_alignbit(d.y, d.x, shift), hi = __builtin_amdgcn_alignbit(d.z, d.y, shift);
    off[0] = (lo << 1) & m2;
    off[1] = __builtin_amdgcn_alignbit(hi, lo, b - 1) & m2;
    off[2] = __builtin_amdgcn_alignbit(hi, lo, 2 * b - 1) & m2;
    off[3] = static_cast<uint32_t>(((static_cast<uint64_t>(hi) << 32) | lo) >> ((3 * b - 1) & 63)) & m2;
}

// The operand of a wait for vector memory alone, n operations left in flight.
constexpr int vm(uint32_t n) { return static_cast<int>(0x0F70 | (n & 15) | (n >> 4) << 14); }

// A value that is the same in every lane, in scalar registers.
__device__ __forceinline__ uint64_t in_scalars(uint64_t v) {
    const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<int>(static_cast<uint32_t>(v)));
    const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<int>(static_cast<uint32_t>(v >> 32)));
    return (static_cast<uint64_t>(hi) << 32) | lo;
}

// Keeps memory loads and copies into LDS in the order in which they stand (see k_fused's).
__device__ __forceinline__ void keep_order() { __builtin_amdgcn_sched_barrier(0x78F); }

// Column fragments by transposing reads (see k_fused's).
template <int HI, int OFF, int N>
__device__ __forceinline__ void read_columns(bf16x8_t (&x)[N], const uint32_t (&at)[N]) {
    static_assert(N == 2 || N == 4, "two or four column fragments");
    u32x2 a[N], b[N];
    if constexpr (N == 2) {
        asm volatile(
            "ds_read_b64_tr_b16 %0, %4 offset:%c6\n"
            "ds_read_b64_tr_b16 %1, %4 offset:%c7\n"
            "ds_read_b64_tr_b16 %2, %5 offset:%c6\n"
            "ds_read_b64_tr_b16 %3, %5 offset:%c7\n"
            "s_waitcnt lgkmcnt(0)\n"
            : "=&v"(a[0]), "=&v"(b[0]), "=&v"(a[1]), "=&v"(b[1])
            : "v"(at[0]), "v"(at[1]), "i"(OFF), "i"(OFF + HI)
            : "memory");
    } else {
        asm volatile(
            "ds_read_b64_tr_b16 %0, %8 offset:%c12\n"
            "ds_read_b64_tr_b16 %1, %8 offset:%c13\n"
            "ds_read_b64_tr_b16 %2, %9 offset:%c12\n"
            "ds_read_b64_tr_b16 %3, %9 offset:%c13\n"
            "ds_read_b64_tr_b16 %4, %10 offset:%c12\n"
            "ds_read_b64_tr_b16 %5, %10 offset:%c13\n"
            "ds_read_b64_tr_b16 %6, %11 offset:%c12\n"
            "ds_read_b64_tr_b16 %7, %11 offset:%c13\n"
            "s_waitcnt lgkmcnt(0)\n"
            : "=&v"(a[0]), "=&v"(b[0]), "=&v"(a[1]), "=&v"(b[1]), "=&v"(a[2]), "=&v"(b[2]), "=&v"(a[3]), "=&v"(b[3])
            : "v"(at[0]), "v"(at[1]), "v"(at[2]), "v"(at[3]), "i"(OFF), "i"(OFF + HI)
            : "memory");
    }
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = __builtin_bit_cast(bf16x8_t, (u32x4){a[i].x, a[i].y, b[i].x, b[i].y});
}

// What becomes of a wave's sums of one token (of a tile's token m): FN fragments of 16 columns, of which this lane has
// columns 4 lg .. 4 lg + 3, from column FN 16 wn of the tile on (the tile has `wn_count` such parts).  Forward pairs
// have a fragment of gate and then one of up, of the same rows.
template <int EPI, int FN, bool ONE = false>
__device__ __forceinline__ void finish(const ExArgs &p, const f32x4_t (&acc)[FN], const ExTile &tile, uint32_t m, uint32_t share,
                                       uint32_t col_tile, uint32_t wn, uint32_t wn_count, uint32_t lg) {
    const bool there = m < tile.count;
    const uint64_t at = tile.start + (there ? m : 0);
    if constexpr (EPI == kSum) {
        if (!there) return;
        const uint32_t n = (col_tile * wn_count + wn) * (FN * 16) + 4 * lg;
        const float f = p.scaled ? p.weights[ONE ? at : p.slot_of[at]] : 1.f;
        float *out = p.S + share * p.split_stride + at * p.ldS + n;
#pragma unroll
        for (int j = 0; j < FN; ++j)
            if (n + 16 * j < p.ldS) *reinterpret_cast<f32x4_t *>(out + 16 * j) = p.scaled ? acc[j] * f : acc[j];
    } else {
        const uint32_t f0 = (col_tile * wn_count + wn) * (FN * 8) + 4 * lg;
        float sum = 0.f, w = 0.f;  // <H, D> over this wave's columns; the slot's weight
        if constexpr (EPI == kHiddenBwd) w = p.weights[ONE ? at : p.slot_of[at]];
#pragma unroll
        for (int j = 0; j < FN; j += 2) {
            const uint32_t f = f0 + 8 * j;
            if (f >= p.Fp) continue;
            const f32x4_t g = acc[j], u = acc[j + 1];
            if constexpr (EPI == kHidden) {
                if (!there) continue;
                float h[4];
#pragma unroll
                for (uint32_t r = 0; r < 4; ++r) h[r] = f + r < p.rows ? activation(p.act, g[r], nullptr) * u[r] : 0.f;
                *reinterpret_cast<u32x2 *>(p.H + at * p.Fp + f) = (u32x2){pack_bf16(h[0], h[1]), pack_bf16(h[2], h[3])};
            } else {
                f32x4_t d = *reinterpret_cast<const f32x4_t *>(p.D + at * p.ldD + f);
                for (uint32_t k = 1; k < p.d_splits; ++k) d += *reinterpret_cast<const f32x4_t *>(p.D + k * p.d_stride + at * p.ldD + f);
                float dg[4], du[4];
#pragma unroll
                for (uint32_t r = 0; r < 4; ++r) {
                    float slope;
                    const float a = activation(p.act, g[r], &slope), dh = w * d[r];
                    const bool in = f + r < p.rows;
                    sum += in ? a * u[r] * d[r] : 0.f;
                    dg[r] = in ? dh * u[r] * slope : 0.f;
                    du[r] = in ? dh * a : 0.f;
                }
                if (there) {
                    uint16_t *G = p.G + at * (2 * p.Fp) + f;
                    *reinterpret_cast<u32x2 *>(G) = (u32x2){pack_bf16(dg[0], dg[1]), pack_bf16(dg[2], dg[3])};
                    *reinterpret_cast<u32x2 *>(G + p.Fp) = (u32x2){pack_bf16(du[0], du[1]), pack_bf16(du[2], du[3])};
                }
            }
        }
        if constexpr (EPI == kHiddenBwd) {
            sum += __shfl_xor(sum, 16, 64);
            sum += __shfl_xor(sum, 32, 64);
            if (there && lg == 0) p.dw[at * p.dw_parts + col_tile * wn_count + wn] = sum;
        }
    }
}

// ---------------------------------------------------------------------------- up to 64 tokens
// Tiles of 64 tokens x 128 columns: the gradients' products of few tokens, and every product where a table of 2^14 entries
// or more rules the others out.  The reduction is walked in slices of 64: while one is multiplied, the tokens' part of the next is
// copied straight into LDS and the workgroup's 512 lanes decode 16 fields of it each into the same layout as k_fused's
// (cbk_nn_fused.h).  Two buffers, one barrier a slice.  Small calls are bound by its start (table, first words, first
// decode): the backward pass of 45 tokens, 2 of 7 experts of 683 x 1001 each, takes 10 (D), 18 (hidden) and 13 us (dX).
constexpr uint32_t kTokens = 64, kColumns = 128;
constexpr uint32_t kSliceBytes = (kTokens + kColumns) * 128;

template <bool NN, bool PAIR, int EPI, bool GT>
__global__ __launch_bounds__(512) void k_experts(const ExArgs p) {
    constexpr int WN = 4, WM = 2;
    constexpr int FM = kTokens / WM / 16, FN = kColumns / WN / 16;
    constexpr uint32_t XBYTES = kTokens * 128, SLICE = kSliceBytes;
    constexpr uint32_t NL = 4;  // loads of a lane's words
    static_assert(EPI == kSum || (PAIR && !NN), "gate and up side by side");
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    unsigned char *ring = smem + (GT ? 0 : (PAIR ? 2 : 1) * p.table);
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t li = lane & 15, lg = lane >> 4;
    const int wm = wave / WN, wn = wave % WN;

    // Units in order of token tile, column tile and share; an XCD (workgroups go to the 8 of them in turn) gets a run of
    // them, whose tokens its L2 keeps.
    const uint32_t units = *p.ntiles * p.col_tiles * p.splits, per = (units + 7) / 8;
    const uint32_t unit = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
    if ((blockIdx.x >> 3) >= per || unit >= units) return;
    const uint32_t share = unit % p.splits, col_tile = unit / p.splits % p.col_tiles;
    const ExTile tile = p.tiles[unit / p.splits / p.col_tiles];
    const ExTensor T0 = p.t[0][tile.expert], T1 = PAIR ? p.t[1][tile.expert] : T0;

    // this lane's task in a slice: 16 fields of a row
    const uint32_t trow = NN ? tid >> 3 : tid >> 2, tgrp = NN ? tid & 7 : tid & 3;
    const uint32_t swz = NN ? 2 * (trow & 3) + 8 * ((trow >> 3) & 1) : trow & 7;
    const uint32_t wrow = trow * (NN ? 256u : 128u);
    // copies of the tokens' part: 8 rows by a wave, rows past the tile's end repeat the last one
    const uint32_t xr = min(static_cast<uint32_t>(wave * 8 + (lane >> 3)), tile.count - 1);
    const uint32_t vx = (p.by_slot ? xr : p.token_of[tile.start + xr]) * p.lda * 2 + ((lane & 7) ^ (lane >> 3)) * 16;
    const auto rx = wave_rsrc(p.A + (p.by_slot ? static_cast<uint64_t>(tile.start) * p.lda : 0), 0x7FFFFFF0u);
    // fragment reads; fragment i of this wave is tokens 16 (i WM + wm) and on
    const uint32_t fa = (wm * 16 + li) * 128 + ((lg ^ (li & 7)) * 16);
    const uint32_t fb = (wn * (kColumns / WN) + li) * 128 + ((lg ^ (li & 7)) * 16);
    uint32_t ft[FN];
    if constexpr (NN) {
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            const uint32_t r = 8 * lg + (li >> 2);
            const uint32_t c = (wn * (kColumns / WN) + 16 * j) / 8 + ((li & 3) >> 1);
            ft[j] = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((CBK_LDS unsigned char *)(ring))) + XBYTES + r * 256 + (c ^ (2 * (r & 3) + 8 * (lg & 1))) * 16 + (li & 1) * 8;
        }
    }

    f32x4_t acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = (f32x4_t){0.f, 0.f, 0.f, 0.f};

    const uint32_t all = p.slices * (NN && PAIR ? 2 : 1);  // the reduction's slices, of which this share's:
    const uint32_t c0 = static_cast<uint32_t>(static_cast<uint64_t>(all) * share / p.splits);
    const uint32_t c1 = static_cast<uint32_t>(static_cast<uint64_t>(all) * (share + 1) / p.splits);
    if constexpr (!GT) {
        if constexpr (PAIR) stage_tables(smem, T0, smem + p.table, T1, tid);
        else stage_table(smem, T0, tid);
    }

    // The reduction over slices [s0, s1) of tensor `which` (forward pairs: the wave's own of the two).
    auto pass = [&](uint32_t which, uint32_t s0, uint32_t s1, auto active) __attribute__((always_inline)) {
        constexpr int NF = decltype(active)::value;          // fragments of tokens that there are
        const ExTensor &T = which ? T1 : T0;
        const uint32_t b = __builtin_amdgcn_readfirstlane(T.b), m2 = ((1u << b) - 1) << 1;
        const unsigned char *table = smem + which * p.table;
        // where this lane's fields start: a row (a base on a dword), and the bits after it
        const uint32_t row0 = NN ? s0 * 64 : PAIR ? col_tile * 64 : col_tile * kColumns;
        const uint32_t cols = NN ? p.N : p.R;
        const uint64_t base = static_cast<uint64_t>(row0) * cols * b;
        const uint32_t trel = NN || !PAIR ? trow : 16 * (trow >> 5) + (trow & 15);
        const uint32_t bit = (trel * cols + (NN ? col_tile * kColumns : s0 * 64) + tgrp * 16) * b + (static_cast<uint32_t>(base) & 31u);
        uint32_t first[4], shift[4];
#pragma unroll
        for (uint32_t q = 0; q < 4; ++q) {
            first[q] = ((bit + 4 * q * b) >> 5) * 4;
            shift[q] = (bit + 4 * q * b) & 31u;
        }
        const uint64_t start = (base >> 5) * 4, step = NN ? static_cast<uint64_t>(cols) * (8 * b) : 8 * b;
        uint64_t words_at = in_scalars(reinterpret_cast<uint64_t>(T.words) + start), rest = in_scalars(T.bytes > start ? T.bytes - start : 0);
        // kept in scalar registers: loading them again in the loop would wait for the LDS too
        asm volatile("" : "+s"(words_at), "+s"(rest));
        struct Words {
            u32x3 q[4];
        } w;
        // The words of slice s; what is past the stream's end reads as zeros.
        auto load = [&](uint32_t s) {
            const uint32_t n = s - s0;
            const uint64_t at = NN ? n * step : 0, have = rest > at ? rest - at : 0;
            const auto rs = wave_rsrc(reinterpret_cast<const unsigned char *>(words_at + (rest > at ? at : 0)),
                                      static_cast<uint32_t>(min(have, static_cast<uint64_t>(0x7FFFFFF0u))));
#pragma unroll
            for (int q = 0; q < 4; ++q)
                w.q[q] = __builtin_amdgcn_raw_buffer_load_b96(rs, static_cast<int>(first[q] + (NN ? 0u : n * (8 * b))), 0, 0);
        };
        // Decodes them to the buffer at `to`; `masked`: terms past the reduction's end are zeros.
        auto decode = [&](uint32_t s, uint32_t to, auto masked) {
            uint32_t v[16];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint32_t off[4];
                fields4(w.q[q], shift[q], b, m2, off);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if constexpr (GT)
                        v[4 * q + i] = (off[i] >> 1) < T.U ? T.cb[off[i] >> 1] : kCorrupt;
                    else
                        v[4 * q + i] = *reinterpret_cast<const uint16_t *>(table + off[i]);
                }
            }
            if constexpr (decltype(masked)::value) {
                const uint32_t at = s * 64 + (NN ? trow : tgrp * 16), have = p.R > at ? p.R - at : 0u;
#pragma unroll
                for (uint32_t i = 0; i < 16; ++i) v[i] = (NN ? have > 0 : i < have) ? v[i] : 0u;
            }
            unsigned char *row = ring + to + XBYTES + wrow;
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const uint32_t *x = v + 8 * g;
                *reinterpret_cast<u32x4 *>(row + ((tgrp * 2 + g) ^ swz) * 16) =
                    (u32x4){x[0] | (x[1] << 16), x[2] | (x[3] << 16), x[4] | (x[5] << 16), x[6] | (x[7] << 16)};
            }
        };
        auto copy = [&](uint32_t s, uint32_t to) {
            const uint32_t from = (s + (NN && PAIR ? which * p.slices : 0u)) * 128;
            copy_to_lds(rx, ring + to + wave * 1024, vx, from);
        };
        struct Frags {
            bf16x8_t a[NF], b[FN];
        };
        auto read = [&](Frags &f, uint32_t at, auto half) {
            constexpr int KS = decltype(half)::value;
            const unsigned char *sa = ring + at, *sb = sa + XBYTES;
            if constexpr (NN) {
                uint32_t t[FN];
#pragma unroll
                for (int j = 0; j < FN; ++j) t[j] = ft[j] + at;
                read_columns<4 * 256, KS * 32 * 256>(f.b, t);
            } else {
#pragma unroll
                for (int j = 0; j < FN; ++j)
                    f.b[j] = __builtin_bit_cast(bf16x8_t, *reinterpret_cast<const u32x4 *>(sb + (fb ^ (KS * 64)) + j * 2048));
            }
#pragma unroll
            for (int i = 0; i < NF; ++i)
                f.a[i] = __builtin_bit_cast(bf16x8_t, *reinterpret_cast<const u32x4 *>(sa + (fa ^ (KS * 64)) + i * (WM * 2048)));
        };
        auto multiply = [&](const Frags &f) {
#pragma unroll
            for (int i = 0; i < NF; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f.b[j], f.a[i], acc[i][j], 0, 0, 0);
        };
        const std::integral_constant<int, 0> lower;
        const std::integral_constant<int, 1> upper;
        const std::true_type yes;
        const std::false_type no;

        copy(s0, 0);
        keep_order();
        load(s0);
        lds_barrier();  // the tables
        decode(s0, 0, yes);
        keep_order();
        load(min(s0 + 1, s1 - 1));
        __builtin_amdgcn_s_waitcnt(GT ? 0x0070 : 0x0070 | NL);
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        uint32_t now = 0;
        // Slice s is multiplied; the next one (`more`) copied and decoded, and, unless that is the `last`, the words of
        // the one after asked for.  At the end the copies have landed, and every word but those.
        auto interval = [&](uint32_t s, auto more, auto last) {
            constexpr bool MORE = decltype(more)::value, WORDS = MORE && !decltype(last)::value;
            Frags f0, f1;
            if constexpr (MORE) copy(s + 1, SLICE - now);
            read(f0, now, lower);
            read(f1, now, upper);
            multiply(f0);
            if constexpr (MORE) {
                decode(s + 1, SLICE - now, last);
                keep_order();
                if constexpr (WORDS) load(s + 2);
            }
            multiply(f1);
            if constexpr (MORE && !GT) {
                constexpr int MF = 2 * NF * FN, RD = 16 + (NN ? 2 * NF : 2 * (NF + FN));
#pragma unroll
                for (int i = 0; i < MF; ++i) {
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                    __builtin_amdgcn_sched_group_barrier(0x100, (RD + MF - 1) / MF, 0);
                    __builtin_amdgcn_sched_group_barrier(0x002, 96 / MF, 0);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
            __builtin_amdgcn_s_waitcnt(GT || !WORDS ? 0x0070 : 0x0070 | NL);
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
            now = SLICE - now;
        };
        uint32_t s = s0;
        for (; s + 2 < s1; ++s) interval(s, yes, no);
        if (s + 1 < s1) {
            interval(s, yes, yes);
            ++s;
        }
        interval(s, no, no);
    };
    // as many fragments as the tile has tokens for, in steps of 16 WM
    auto passes = [&](auto active) {
        if constexpr (NN && PAIR) {
#pragma unroll 1
            for (uint32_t which = c0 >= p.slices; which * p.slices < c1; ++which)
                pass(which, max(c0, which * p.slices) - which * p.slices, min(c1, (which + 1) * p.slices) - which * p.slices, active);
        } else {
            pass(PAIR ? wave & 1 : 0, c0, c1, active);
        }
    };
    const uint32_t frags = (tile.count + 16 * WM - 1) / (16 * WM);
    if (frags == 1) passes(std::integral_constant<int, 1>{});
    else passes(std::integral_constant<int, 2>{});

#pragma unroll
    for (int i = 0; i < FM; ++i) {
        const uint32_t m = (i * WM + wm) * 16 + li;
        finish<EPI, FN>(p, acc[i], tile, m, share, col_tile, wn, WN, lg);
    }
}

// -------------------------------------------------------------------------------- few tokens
// Forward products of up to 16 tokens: bound by reading the weights.  A workgroup goes through a run of units, 32 rows
// each (16 of gate and 16 of up, or 32 of one tensor) for one token tile; its 8 waves take every eighth step of 128
// terms, and their sums meet in LDS in a fixed order, one barrier a unit.  A wave works by itself otherwise.  An item is
// a step of 16 rows: their 128 fields, up to 15 chunks of 16 bytes a row, are copied as they lie straight into one of
// three places of the wave's own, two items ahead (loads of a lane's own fields, which scatter a wave over 16 rows,
// took 302 us for 48 tokens of 4 out of 32 experts' gate and up of 2048 x 4096 each, 197 so: 4.4 TB/s of weights, and
// the copies alone, without decoding, take 180).  From there lane l takes 16 fields of row
// l % 16 at term 16 (l / 16) of each 64, decodes them into the layout of the matrix instruction's operand, and the
// tokens' fragments are read from the caches with the terms in the same order.
constexpr uint32_t kFewTokens = 16, kFewChunks = 15, kFewStage = 16 * kFewChunks * 16, kFewRing = 3, kFewStep = 128;
// LDS of the waves' sums: of two units, so that one barrier a unit is enough
constexpr uint32_t kFewSums = 8 * 2 * 1024;
constexpr uint32_t few_lds(uint32_t tables) { return tables + 8 * kFewRing * kFewStage + 2 * kFewSums; }

// The three dwords at each of four LDS addresses.  Written out because the compiler holds reads back until every copy
// into LDS has landed, also those of items still to come; the block waits for its own reads.
__device__ __forceinline__ void read_windows(u32x3 (&w)[4], const uint32_t (&at)[4]) {
    u32x2 a0, a1, a2, a3;
    uint32_t b0, b1, b2, b3;
    asm volatile(
        "ds_read2_b32 %0, %8 offset1:1\n"
        "ds_read_b32 %4, %8 offset:8\n"
        "ds_read2_b32 %1, %9 offset1:1\n"
        "ds_read_b32 %5, %9 offset:8\n"
        "ds_read2_b32 %2, %10 offset1:1\n"
        "ds_read_b32 %6, %10 offset:8\n"
        "ds_read2_b32 %3, %11 offset1:1\n"
        "ds_read_b32 %7, %11 offset:8\n"
        "s_waitcnt lgkmcnt(0)\n"
        : "=&v"(a0), "=&v"(a1), "=&v"(a2), "=&v"(a3), "=&v"(b0), "=&v"(b1), "=&v"(b2), "=&v"(b3)
        : "v"(at[0]), "v"(at[1]), "v"(at[2]), "v"(at[3])
        : "memory");
    w[0] = (u32x3){a0.x, a0.y, b0};
    w[1] = (u32x3){a1.x, a1.y, b1};
    w[2] = (u32x3){a2.x, a2.y, b2};
    w[3] = (u32x3){a3.x, a3.y, b3};
}

template <bool PAIR, int EPI, bool ONE>
__global__ __launch_bounds__(512) void k_experts_few(const ExArgs p) {
    static_assert(PAIR == (EPI != kSum), "gate and up, or one tensor");
    constexpr uint32_t NX = 4;  // loads of a step's tokens
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t li = lane & 15, lg = lane >> 4;
    unsigned char *stages = smem + (PAIR ? 2 : 1) * p.table + wave * (kFewRing * kFewStage);
    float *sums = reinterpret_cast<float *>(smem + (PAIR ? 2 : 1) * p.table + 8 * kFewRing * kFewStage);

    // One token's slots are tiles as they stand, of an expert each (nothing sorts them; unused ones have none); else as
    // k_sort listed them.
    auto tile_at = [&](uint32_t t) __attribute__((always_inline)) {
        return ONE ? ExTile{static_cast<uint32_t>(p.experts[t]), t, 1, 0} : p.tiles[t];
    };
    const uint32_t units = (ONE ? p.k : *p.ntiles) * p.col_tiles;
    const uint32_t u0 = static_cast<uint32_t>(static_cast<uint64_t>(units) * blockIdx.x / gridDim.x);
    const uint32_t u1 = static_cast<uint32_t>(static_cast<uint64_t>(units) * (blockIdx.x + 1) / gridDim.x);
    if (u0 == u1) return;
    const uint32_t S = (p.slices + 1) / 2;                   // steps
    const uint32_t mine = (S + 7 - wave) / 8;                // of them this wave's, in every unit
    const uint32_t items = 2 * mine * (u1 - u0);             // a step's two runs of 16 rows, one after the other

    struct Tensor {
        uint64_t words;
        uint64_t bytes;
        uint32_t b;
    };
    auto tensor = [&](uint32_t expert, uint32_t j) __attribute__((always_inline)) {
        const ExTensor &T = p.t[PAIR ? j : 0][ONE && expert >= p.count ? 0 : expert];
        return Tensor{in_scalars(reinterpret_cast<uint64_t>(T.words)), in_scalars(T.bytes), static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(T.b))};
    };
    // first of the 16 rows j of a unit
    auto first_row = [&](uint32_t u, uint32_t j) { return static_cast<uint64_t>(u % p.col_tiles) * (PAIR ? 16 : 32) + (PAIR ? 0 : 16 * j); };

    // ---- copies: item n is run (n & 1) of a step; they are asked for in order, past the last one the last again
    uint32_t cu = u0, cs = wave, cn = 0;  // unit, step and number of the next item to copy
    struct Source {
        uint64_t base, bytes;
        uint32_t v[4], b;
    } from[2];
    auto source = [&]() __attribute__((always_inline)) {  // of unit cu
        const uint32_t expert = tile_at(cu / p.col_tiles).expert;
#pragma unroll
        for (uint32_t j = 0; j < 2; ++j) {
            const Tensor T = tensor(expert, j);
            const uint64_t bits = first_row(cu, j) * p.R * T.b, start = bits / 128 * 16;
            from[j].base = T.words + (T.bytes > start ? start : 0);
            from[j].bytes = T.bytes > start ? T.bytes - start : 0;
            from[j].b = T.b;
#pragma unroll
            for (uint32_t i = 0; i < 4; ++i) {
                const uint32_t g = min(i * 64 + lane, 16 * kFewChunks - 1), row = g / kFewChunks, c = g % kFewChunks;
                // chunks past the fields' end repeat the last one
                from[j].v[i] = (((static_cast<uint32_t>(bits) & 127u) + row * p.R * T.b) / 128 + min(c, T.b)) * 16;
            }
        }
    };
    uint32_t slot = 0;  // where the next item goes
    auto copy = [&](uint32_t j) __attribute__((always_inline)) {
        const Source &f = from[j];
        const auto rs = wave_rsrc(reinterpret_cast<const unsigned char *>(f.base), static_cast<uint32_t>(min(f.bytes, static_cast<uint64_t>(0x7FFFFFF0u))));
        unsigned char *to = stages + slot * kFewStage;
        const uint32_t at = cs * (kFewStep / 8) * f.b;
#pragma unroll
        for (uint32_t i = 0; i < 3; ++i) copy_to_lds(rs, to + i * 1024, f.v[i] + at, 0);
        if (lane < 16 * kFewChunks - 192) copy_to_lds(rs, to + 3 * 1024, f.v[3] + at, 0);
        slot = slot == kFewRing - 1 ? 0 : slot + 1;
        ++cn;
        if (j == 1 && cn < items) {  // the next step
            cs += 8;
            if (cs >= S) {
                cs = wave;
                ++cu;
                source();
            }
        }
    };

    // ---- tokens
    uint32_t vx = 0, rows_at = ~0u;  // this lane's row of A, and the tile that it is of
    auto rows_of = [&](uint32_t t) __attribute__((always_inline)) {
        if (rows_at == t) return;
        rows_at = t;
        const ExTile tile = tile_at(t);
        const uint32_t r = min(li, tile.count - 1);
        vx = p.by_slot ? tile.start + r : ONE ? 0 : p.token_of[tile.start + r];
    };
    struct Step {
        bf16x8_t f[4];
    };
    // Fragments for step s (the second 64 terms of a last step that has none: the first again, not used).
    auto tokens = [&](Step &x, uint32_t s) __attribute__((always_inline)) {
        const unsigned char *row = reinterpret_cast<const unsigned char *>(p.A + static_cast<uint64_t>(vx) * p.lda) + lg * 32 + s * (2 * kFewStep);
        const bool whole = 2 * s + 1 < p.slices;
#pragma unroll
        for (int h = 0; h < 4; ++h) x.f[h] = __builtin_bit_cast(bf16x8_t, *reinterpret_cast<const u32x4 *>(row + (h < 2 ? 16 * h : whole ? 128 + 16 * (h - 2) : 0)));
    };

    f32x4_t acc[2];
    // ---- an item: `place` its stage
    struct Window {
        uint32_t at[4], shift[4], b, m2;
        const unsigned char *table;
    } win[2];
    ExTile tile;
    auto windows = [&](uint32_t u) __attribute__((always_inline)) {
#pragma unroll
        for (uint32_t j = 0; j < 2; ++j) {
            const uint32_t b = tensor(tile.expert, j).b;
            const uint32_t bits = (static_cast<uint32_t>(first_row(u, j) * p.R * b) + li * p.R * b) & 127u;
            Window &w = win[j];
#pragma unroll
            for (uint32_t q = 0; q < 4; ++q) {
                const uint32_t bit = bits + (lg * 16 + 4 * q) * b;
                w.at[q] = li * (kFewChunks * 16) + (bit >> 5) * 4;
                w.shift[q] = bit & 31u;
            }
            w.b = b;
            w.m2 = ((1u << b) - 1) << 1;
            w.table = smem + (PAIR ? j : 0) * p.table;
        }
    };
    auto item = [&](const Step &x, uint32_t j, uint32_t s, const unsigned char *place) __attribute__((always_inline)) {
        const Window &w = win[j];
#pragma unroll
        for (uint32_t hh = 0; hh < 2; ++hh) {
            if (hh == 1 && 2 * s + 1 >= p.slices) break;
            uint32_t v[16];
            const uint32_t add = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((const CBK_LDS unsigned char *)(place))) + hh * (8 * w.b);
            const uint32_t from[4] = {w.at[0] + add, w.at[1] + add, w.at[2] + add, w.at[3] + add};
            u32x3 words[4];
            read_windows(words, from);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint32_t off[4];
                fields4(words[q], w.shift[q], w.b, w.m2, off);
#pragma unroll
                for (int i = 0; i < 4; ++i) v[4 * q + i] = *reinterpret_cast<const uint16_t *>(w.table + off[i]);
            }
            if (s * kFewStep + hh * 64 + 64 > p.R) {  // terms past the rows' end are zeros
                const uint32_t at = s * kFewStep + hh * 64 + lg * 16, have = p.R > at ? p.R - at : 0u;
#pragma unroll
                for (uint32_t i = 0; i < 16; ++i) v[i] = i < have ? v[i] : 0u;
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t *y = v + 8 * h;
                const bf16x8_t f = __builtin_bit_cast(bf16x8_t, (u32x4){y[0] | (y[1] << 16), y[2] | (y[3] << 16), y[4] | (y[5] << 16), y[6] | (y[7] << 16)});
                acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f, x.f[2 * hh + h], acc[j], 0, 0, 0);
            }
        }
    };

    Step x;
    if (mine > 0) {
        source();
        rows_of(u0 / p.col_tiles);
        copy(0);
        keep_order();
        tokens(x, wave);
        keep_order();
        copy(1);
        keep_order();
    }
    uint32_t staged = ~0u, place = 0;
    for (uint32_t u = u0; u < u1; ++u) {
        tile = tile_at(u / p.col_tiles);
        // (an unused slot of one token goes through the motions with the first expert's weights, and leaves nothing)
        const bool used = !ONE || tile.expert < p.count;
        if (!used) tile.expert = 0;
        windows(u);
        if (staged != tile.expert) {  // (the previous tables' last reads came before the last barrier)
            staged = tile.expert;
            if constexpr (PAIR) stage_tables(smem, p.t[0][staged], smem + p.table, p.t[1][staged], tid);
            else stage_table(smem, p.t[0][staged], tid);
            lds_barrier();
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[j] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
        for (uint32_t s = wave; s < S; s += 8) {
            // The next step's tokens (after the last of all the last again), and the copies two items on; then this item's
            // have landed when no more is in flight than was asked for after them: two copies, and a step's tokens.
            Step next;
            const bool more = s + 8 < S;
            if (!more && u + 1 < u1) rows_of((u + 1) / p.col_tiles);
            keep_order();
            tokens(next, more ? s + 8 : u + 1 < u1 ? static_cast<uint32_t>(wave) : s);
            keep_order();
            copy(0);
            keep_order();
            __builtin_amdgcn_s_waitcnt(vm(8 + NX));
            asm volatile("" ::: "memory");
            item(x, 0, s, stages + place * kFewStage);
            place = place == kFewRing - 1 ? 0 : place + 1;
            keep_order();
            asm volatile("" ::: "memory");
            copy(1);
            keep_order();
            __builtin_amdgcn_s_waitcnt(vm(8 + NX));
            asm volatile("" ::: "memory");
            item(x, 1, s, stages + place * kFewStage);
            place = place == kFewRing - 1 ? 0 : place + 1;
            asm volatile("" ::: "memory");
            x = next;
        }
        float *to = sums + (u & 1) * (kFewSums / 4) + lane * 4;
#pragma unroll
        for (int j = 0; j < 2; ++j) *reinterpret_cast<f32x4_t *>(to + (wave * 2 + j) * 256) = acc[j];
        lds_barrier();
        // the waves add a unit's sums in turn
        if (wave == static_cast<int>(u & 7) && used) {
            f32x4_t t[2] = {};
            for (int w = 0; w < 8; ++w)
#pragma unroll
                for (int j = 0; j < 2; ++j) t[j] += *reinterpret_cast<const f32x4_t *>(to + (w * 2 + j) * 256);
            finish<EPI, 2, ONE>(p, t, tile, li, 0, u % p.col_tiles, 0, 1, lg);
        }
    }
    __builtin_amdgcn_s_waitcnt(0x0070);  // no copy is left in flight
}

// ------------------------------------------------------------------------------- many tokens
// A tile of 256 tokens x 256 columns; the reduction in blocks of 64, two buffers of tokens and of decoded weights in LDS
// (a wave multiplies 64 tokens with 128 columns).  While a block is multiplied in halves of 32 terms, the next one's tokens
// are copied, a wave decodes the next one's weights in halves of its rows (a row's 64 fields at once by four lanes, whose
// cache lines are then done with), and the words of the one after are asked for.  One barrier a block, before its last
// multiplications.  Memory answers in order, so words asked for right before their use wait for the tokens too: with words
// a half ahead in slices of 32 terms of all rows (which fell out of the L1 between two slices), and the tokens' fragments
// read from the caches by each wave, gate and up of 2048 tokens of 4 out of 32 experts of 2048 x 4096 and back took 1254 us,
// so 690 (672 to 785 by how many token tiles the routing leaves, 46 to 50).  What bounds it is the LDS, busy for 62 % of the
// time: a gather's 64 addresses meet in banks, ~5 clocks over the 2 it needs.  Without gathers gate and up would take 433 us
// instead of 447, without scattered words 406, with neither 337; the matrix instructions keep their units busy for 36 %.
constexpr uint32_t kManyColumns = 256, kManyTokens = 256, kManyBlock = 64;
constexpr uint32_t kManyBytes = kManyColumns * kManyBlock * 2;  // of a block of weights
constexpr uint32_t kManyTokenBytes = kManyTokens * kManyBlock * 2;

template <bool NN, bool PAIR, int EPI>
__global__ __launch_bounds__(512) void k_experts_many(const ExArgs p) {
    constexpr int WM = 4, FM = 4, FN = 8;
    constexpr uint32_t NL = 4;  // loads of a lane's words of a half
    static_assert(kManyBytes == kManyTokenBytes, "one offset for both");
    static_assert(EPI == kSum || (PAIR && !NN), "gate and up side by side");
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    // forward pairs hold both tables, gradients the one of the tensor that they are at; then two blocks of tokens, and of weights
    unsigned char *xring = smem + (PAIR && !NN ? 2 : 1) * p.table, *ring = xring + 2 * kManyTokenBytes;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t li = lane & 15, lg = lane >> 4;
    const int wm = wave >> 1, wn = wave & 1;

    // Units in order of token tile, the fullest first (they take longest), column tile and share: the XCDs get them in
    // turn, so that each has as many of a kind (in runs an XCD's tokens stayed in its L2, and it took 3 % longer).
    const uint32_t units = *p.ntiles * p.col_tiles * p.splits, unit = blockIdx.x;
    if (unit >= units) return;
    const uint32_t share = unit % p.splits, col_tile = unit / p.splits % p.col_tiles;
    const ExTile tile = p.tiles[unit / p.splits / p.col_tiles];
    const ExTensor T0 = p.t[0][tile.expert], T1 = PAIR ? p.t[1][tile.expert] : T0;

    // This lane's task in a half: 16 fields of a row, `half` rows on in the other half (32 of the reduction; forward 128 of
    // the tile, whose pairs have 16 rows of gate and of up in turn).
    const uint32_t trow = NN ? tid >> 4 : tid >> 2, tgrp = NN ? tid & 15 : tid & 3;
    const uint32_t swz = NN ? 2 * (trow & 3) + 8 * ((trow >> 3) & 1) : trow & 7;
    const uint32_t wrow = trow * (NN ? 512u : 128u);
    constexpr uint32_t kHalf = (NN ? 32 * 512 : 128 * 128);  // LDS bytes
    // copies of the tokens' part: 8 rows by a wave, rows past the tile's end repeat the last one
    uint32_t vx[FM];
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        const uint32_t r = min(static_cast<uint32_t>((i * 8 + wave) * 8 + (lane >> 3)), tile.count - 1);
        vx[i] = (p.by_slot ? r : p.token_of[tile.start + r]) * p.lda * 2 + ((lane & 7) ^ (lane >> 3)) * 16;
    }
    const auto rx = wave_rsrc(p.A + (p.by_slot ? static_cast<uint64_t>(tile.start) * p.lda : 0), 0x7FFFFFF0u);
    // fragment i of this wave is tokens 16 (i WM + wm) and on
    const uint32_t fa = (wm * 16 + li) * 128 + ((lg ^ (li & 7)) * 16);
    // weights: fragment j of this wave is columns 128 wn + 16 j and on
    const uint32_t fb = (wn * 128 + li) * 128 + ((lg ^ (li & 7)) * 16);
    uint32_t ft[FN];
    if constexpr (NN) {
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            const uint32_t r = 8 * lg + (li >> 2), c = (wn * 128 + 16 * j) / 8 + ((li & 3) >> 1);
            ft[j] = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((CBK_LDS unsigned char *)(ring))) + r * 512 + (c ^ (2 * (r & 3) + 8 * (lg & 1))) * 16 + (li & 1) * 8;
        }
    }

    f32x4_t acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = (f32x4_t){0.f, 0.f, 0.f, 0.f};

    const uint32_t all = p.slices * (NN && PAIR ? 2 : 1);  // the reduction's slices, of which this share's:
    const uint32_t c0 = static_cast<uint32_t>(static_cast<uint64_t>(all) * share / p.splits);
    const uint32_t c1 = static_cast<uint32_t>(static_cast<uint64_t>(all) * (share + 1) / p.splits);
    if constexpr (!NN && PAIR) stage_tables(smem, T0, smem + p.table, T1, tid);
    else if constexpr (!PAIR) stage_table(smem, T0, tid);

    // The reduction over slices [s0, s1) of tensor `which` (forward pairs: the wave's own of the two).
    auto pass = [&](uint32_t which, uint32_t s0, uint32_t s1, auto active) __attribute__((always_inline)) {
        constexpr int NF = decltype(active)::value;  // fragments of tokens that there are
        const ExTensor &T = which ? T1 : T0;
        const uint32_t b = __builtin_amdgcn_readfirstlane(T.b), m2 = ((1u << b) - 1) << 1;
        const unsigned char *table = smem + (NN ? 0 : which * p.table);
        // where this lane's fields start: a row (a base on a dword), and the bits after it
        const uint32_t row0 = NN ? s0 * kManyBlock : PAIR ? col_tile * 128 : col_tile * kManyColumns;
        const uint32_t cols = NN ? p.N : p.R;
        const uint64_t base = static_cast<uint64_t>(row0) * cols * b;
        const uint32_t trel = NN || !PAIR ? trow : 16 * (trow >> 5) + (trow & 15);
        const uint32_t bit = (trel * cols + (NN ? col_tile * kManyColumns : s0 * kManyBlock) + tgrp * 16) * b + (static_cast<uint32_t>(base) & 31u);
        uint32_t first[4], shift[4];
#pragma unroll
        for (uint32_t q = 0; q < 4; ++q) {
            first[q] = ((bit + 4 * q * b) >> 5) * 4;
            shift[q] = (bit + 4 * q * b) & 31u;
        }
        const uint64_t start = (base >> 5) * 4, step = static_cast<uint64_t>(cols) * (8 * b);
        // the other half's fields: whole dwords on
        const uint32_t other = NN ? cols * (4 * b) : (PAIR ? 8 : 16) * cols * b;
        uint64_t words_at = in_scalars(reinterpret_cast<uint64_t>(T.words) + start), rest = in_scalars(T.bytes > start ? T.bytes - start : 0);
        // kept in scalar registers: loading them again in the loop would wait for the LDS too
        asm volatile("" : "+s"(words_at), "+s"(rest));
        struct Words {
            u32x3 q[4];
        } w0, w1;  // of the halves
        // The words of half h of block s; what is past the stream's end reads as zeros.
        auto load = [&](Words &w, uint32_t s, uint32_t h) __attribute__((always_inline)) {
            const uint32_t n = s - s0;
            const uint64_t at = NN ? n * step : 0, have = rest > at ? rest - at : 0;
            const auto rs = wave_rsrc(reinterpret_cast<const unsigned char *>(words_at + (rest > at ? at : 0)),
                                      static_cast<uint32_t>(min(have, static_cast<uint64_t>(0x7FFFFFF0u))));
#pragma unroll
            for (int q = 0; q < 4; ++q)
                w.q[q] = __builtin_amdgcn_raw_buffer_load_b96(rs, static_cast<int>(first[q] + h * other + (NN ? 0u : n * (8 * b))), 0, 0);
        };
        // Decodes them to the buffer at `to`; `masked`: terms past the reduction's end are zeros.
        auto decode = [&](const Words &w, uint32_t s, uint32_t h, uint32_t to, auto masked) __attribute__((always_inline)) {
            uint32_t v[16];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint32_t off[4];
                fields4(w.q[q], shift[q], b, m2, off);
#pragma unroll
                for (int i = 0; i < 4; ++i) v[4 * q + i] = *reinterpret_cast<const uint16_t *>(table + off[i]);
            }
            if constexpr (decltype(masked)::value) {
                const uint32_t at = s * kManyBlock + (NN ? 32 * h + trow : tgrp * 16), have = p.R > at ? p.R - at : 0u;
#pragma unroll
                for (uint32_t i = 0; i < 16; ++i) v[i] = (NN ? have > 0 : i < have) ? v[i] : 0u;
            }
            unsigned char *row = ring + to + h * kHalf + wrow;
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const uint32_t *x = v + 8 * g;
                *reinterpret_cast<u32x4 *>(row + ((tgrp * 2 + g) ^ swz) * 16) =
                    (u32x4){x[0] | (x[1] << 16), x[2] | (x[3] << 16), x[4] | (x[5] << 16), x[6] | (x[7] << 16)};
            }
        };
        auto copy = [&](uint32_t s, uint32_t to) __attribute__((always_inline)) {
            const uint32_t from = (s + (NN && PAIR ? which * p.slices : 0u)) * (2 * kManyBlock);
#pragma unroll
            for (int i = 0; i < NF; ++i) copy_to_lds(rx, xring + to + (i * 8 + wave) * 1024, vx[i], from);
        };
        struct Tokens {
            bf16x8_t f[NF];
        };
        // the tokens' fragments for half h of the terms of the block at `at`
        auto tokens = [&](Tokens &x, uint32_t at, auto half) __attribute__((always_inline)) {
            constexpr int h = decltype(half)::value;
#pragma unroll
            for (int i = 0; i < NF; ++i)
                x.f[i] = __builtin_bit_cast(bf16x8_t, *reinterpret_cast<const u32x4 *>(xring + at + (fa ^ (h * 64)) + i * (WM * 2048)));
        };
        // weights' fragments 4 c .. 4 c + 3 for half h of the terms of the block at `at`
        auto read = [&](bf16x8_t (&f)[4], uint32_t at, auto half, int c) __attribute__((always_inline)) {
            constexpr int h = decltype(half)::value;
            if constexpr (NN) {
                const uint32_t t[4] = {ft[4 * c] + at, ft[4 * c + 1] + at, ft[4 * c + 2] + at, ft[4 * c + 3] + at};
                read_columns<4 * 512, h * 32 * 512>(f, t);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) f[j] = __builtin_bit_cast(bf16x8_t, *reinterpret_cast<const u32x4 *>(ring + at + (fb ^ (h * 64)) + (4 * c + j) * 2048));
            }
        };
        auto multiply = [&](const Tokens &x, const bf16x8_t (&f)[4], int c) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < NF; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][4 * c + j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f[j], x.f[i], acc[i][4 * c + j], 0, 0, 0);
        };
        const std::integral_constant<int, 0> lower;
        const std::integral_constant<int, 1> upper;
        const std::true_type yes;
        const std::false_type no;

        Tokens x0, x1;
        bf16x8_t wa[4], wb[4];
        copy(s0, 0);
        keep_order();
        load(w0, s0, 0);
        load(w1, s0, 1);
        if constexpr (NN && PAIR) stage_table(smem, T, tid);
        lds_barrier();  // the tables
        decode(w0, s0, 0, 0, yes);
        decode(w1, s0, 1, 0, yes);
        keep_order();
        load(w0, min(s0 + 1, s1 - 1), 0);
        load(w1, min(s0 + 1, s1 - 1), 1);
        __builtin_amdgcn_s_waitcnt(0x0070 | 2 * NL);
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        read(wa, 0, lower, 0);
        tokens(x0, 0, lower);
        uint32_t now = 0;
        // Between N multiplications: RD reads of LDS (gathers among them) and the decoding's arithmetic, V a multiplication.
        auto schedule = [](auto muls, auto reads, auto valu) __attribute__((always_inline)) {
            if constexpr (!NN) {
                constexpr int N = decltype(muls)::value, RD = decltype(reads)::value, V = decltype(valu)::value;
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                    __builtin_amdgcn_sched_group_barrier(0x100, (RD + N - 1) / N, 0);
                    __builtin_amdgcn_sched_group_barrier(0x002, V, 0);
                }
            }
        };
        // Block s is multiplied; `more`: the next one is copied and decoded, and the one after asked for unless that is
        // the `last`.  At the end the copies have landed, and every word but those.
        auto interval = [&](uint32_t s, auto more, auto last) __attribute__((always_inline)) {
            constexpr bool MORE = decltype(more)::value, WORDS = MORE && !decltype(last)::value;
            const uint32_t next = kManyBytes - now;
            if constexpr (MORE) copy(s + 1, next);
            keep_order();
            read(wb, now, lower, 1);
            multiply(x0, wa, 0);
            if constexpr (MORE) {
                decode(w0, s + 1, 0, next, last);
                keep_order();
                if constexpr (WORDS) load(w0, s + 2, 0);
            }
            read(wa, now, upper, 0);
            tokens(x1, now, upper);
            multiply(x0, wb, 1);
            if constexpr (MORE) schedule(std::integral_constant<int, 8 * NF>{}, std::integral_constant<int, 24 + NF>{}, std::integral_constant<int, 12 / NF>{});
            __builtin_amdgcn_sched_barrier(0);
            read(wb, now, upper, 1);
            multiply(x1, wa, 0);
            if constexpr (MORE) {
                decode(w1, s + 1, 1, next, last);
                keep_order();
                if constexpr (WORDS) load(w1, s + 2, 1);
            }
            if constexpr (MORE) schedule(std::integral_constant<int, 4 * NF>{}, std::integral_constant<int, 20>{}, std::integral_constant<int, 20 / NF>{});
            __builtin_amdgcn_sched_barrier(0);
            __builtin_amdgcn_s_waitcnt(WORDS ? 0x0070 | 2 * NL : 0x0070);
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
            if constexpr (MORE) {
                read(wa, next, lower, 0);
                tokens(x0, next, lower);
            }
            multiply(x1, wb, 1);
            now = next;
        };
        uint32_t s = s0;
        for (; s + 2 < s1; ++s) interval(s, yes, no);
        if (s + 1 < s1) interval(s++, yes, yes);
        interval(s, no, no);
    };
    auto passes = [&](auto active) {
        if constexpr (NN && PAIR) {
#pragma unroll 1
            for (uint32_t which = c0 >= p.slices; which * p.slices < c1; ++which)
                pass(which, max(c0, which * p.slices) - which * p.slices, min(c1, (which + 1) * p.slices) - which * p.slices, active);
        } else {
            pass(PAIR ? wave & 1 : 0, c0, c1, active);
        }
    };
    // as many fragments as the tile has tokens for, in steps of 64
    const uint32_t frags = (tile.count + 16 * WM - 1) / (16 * WM);
    if (frags == 1) passes(std::integral_constant<int, 1>{});
    else if (frags == 2) passes(std::integral_constant<int, 2>{});
    else if (frags == 3) passes(std::integral_constant<int, 3>{});
    else passes(std::integral_constant<int, 4>{});

#pragma unroll
    for (int i = 0; i < FM; ++i) {
        const uint32_t m = (i * WM + wm) * 16 + li;
        finish<EPI, FN>(p, acc[i], tile, m, share, col_tile, wn, 2, lg);
    }
}

uint32_t tiles_of(uint64_t n, uint64_t m) { return static_cast<uint32_t>((n + m - 1) / m); }

template <bool, bool, bool, int, bool>
struct ExTag;

template <bool NN, bool PAIR, int EPI, bool GT>
cbk_status run(ExArgs &a, const ExPlan &pl, uint32_t columns, hipStream_t s) {
    a.col_tiles = tiles_of(columns, EPI == kSum ? kColumns : kColumns / 2);
    const uint32_t lds = (GT ? 0 : (PAIR ? 2 : 1) * a.table) + 2 * kSliceBytes;
    if (!allow_lds_once<ExTag<false, NN, PAIR, EPI, GT>>(k_experts<NN, PAIR, EPI, GT>, kLdsLimit)) return CBK_E_HIP;
    const uint32_t units = pl.max_tiles * a.col_tiles * a.splits;  // (fewer than 2^23: ex_plan)
    hipLaunchKernelGGL((k_experts<NN, PAIR, EPI, GT>), dim3((units + 7) / 8 * 8), dim3(512), lds, s, a);
    return launched();
}

constexpr uint32_t many_lds(uint32_t table, bool two) { return (two ? 2 : 1) * table + 2 * (kManyBytes + kManyTokenBytes); }

template <bool NN, bool PAIR, int EPI>
cbk_status run_many(ExArgs &a, const ExPlan &pl, uint32_t columns, hipStream_t s) {
    a.col_tiles = tiles_of(columns, EPI == kSum ? kManyColumns : kManyColumns / 2);
    const uint32_t lds = many_lds(a.table, !NN && PAIR);
    if (lds > kLdsLimit) return CBK_E_UNSUPPORTED;  // the plan rules it out
    if (!allow_lds_once<ExTag<true, NN, PAIR, EPI, false>>(k_experts_many<NN, PAIR, EPI>, kLdsLimit)) return CBK_E_HIP;
    const uint32_t units = pl.max_tiles * a.col_tiles * a.splits;
    hipLaunchKernelGGL((k_experts_many<NN, PAIR, EPI>), dim3(units), dim3(512), lds, s, a);
    return launched();
}

template <bool, int, bool>
struct FewTag;

template <bool PAIR, int EPI, bool ONE>
cbk_status run_few(ExArgs &a, const ExPlan &pl, uint32_t columns, hipStream_t s) {
    a.splits = 1;
    a.col_tiles = tiles_of(columns, PAIR ? 16 : 32);
    const uint32_t units = pl.max_tiles * a.col_tiles;  // (below 2^26)
    if (!allow_lds_once<FewTag<PAIR, EPI, ONE>>(k_experts_few<PAIR, EPI, ONE>, kLdsLimit)) return CBK_E_HIP;
    // a workgroup has a CU's LDS
    const uint32_t grid = std::min<uint32_t>(units, cu_count());
    hipLaunchKernelGGL((k_experts_few<PAIR, EPI, ONE>), dim3(grid), dim3(512), few_lds((PAIR ? 2 : 1) * a.table), s, a);
    return launched();
}

// `columns` of the result, or (gate and up) of the hidden values.
template <bool NN, bool PAIR, int EPI>
cbk_status product(ExArgs &a, const ExPlan &pl, uint32_t columns, uint32_t b, hipStream_t s) {
    a.table = std::max(16u, 2u << b);
    if (pl.tile == kManyTokens) return run_many<NN, PAIR, EPI>(a, pl, columns, s);
    if constexpr (!NN) {
        if constexpr (EPI != kHiddenBwd) {
            if (pl.one) return run_few<PAIR, EPI, true>(a, pl, columns, s);
        }
        if (pl.tile == kFewTokens && b <= 14 && few_lds((PAIR ? 2 : 1) * a.table) <= kLdsLimit) return run_few<PAIR, EPI, false>(a, pl, columns, s);
    }
    return b > 14 ? run<NN, PAIR, EPI, true>(a, pl, columns, s) : run<NN, PAIR, EPI, false>(a, pl, columns, s);
}

}  // namespace

cbk_status ex_hidden(ExArgs &a, const ExPlan &pl, const cbk_experts &ex, bool backward, hipStream_t s) {
    a.N = static_cast<uint32_t>(ex.rows);
    a.R = static_cast<uint32_t>(ex.cols);
    a.slices = static_cast<uint32_t>(pl.Kp / 64);
    a.splits = 1;
    a.ldD = static_cast<uint32_t>(pl.ldF);
    a.d_splits = pl.split_dt;
    a.d_stride = pl.d_stride;
    a.dw_parts = pl.dw_parts;
    return backward ? product<false, true, kHiddenBwd>(a, pl, static_cast<uint32_t>(pl.Fp), ex.b, s)
                    : product<false, true, kHidden>(a, pl, static_cast<uint32_t>(pl.Fp), ex.b, s);
}

cbk_status ex_down(ExArgs &a, const ExPlan &pl, const cbk_experts &ex, hipStream_t s) {
    a.N = static_cast<uint32_t>(ex.out);
    a.R = static_cast<uint32_t>(ex.rows);
    a.slices = static_cast<uint32_t>(pl.Fp / 64);
    a.splits = pl.split_down;
    a.ldS = static_cast<uint32_t>(pl.ldO);
    a.split_stride = pl.s_stride;
    return product<false, false, kSum>(a, pl, a.N, ex.b_down, s);
}

cbk_status ex_down_t(ExArgs &a, const ExPlan &pl, const cbk_experts &ex, hipStream_t s) {
    a.N = static_cast<uint32_t>(ex.rows);
    a.R = static_cast<uint32_t>(ex.out);
    a.slices = static_cast<uint32_t>(pl.Op / 64);
    a.splits = pl.split_dt;
    a.ldS = static_cast<uint32_t>(pl.ldF);
    a.split_stride = pl.d_stride;
    return product<true, false, kSum>(a, pl, a.N, ex.b_down, s);
}

cbk_status ex_dx(ExArgs &a, const ExPlan &pl, const cbk_experts &ex, hipStream_t s) {
    a.N = static_cast<uint32_t>(ex.cols);
    a.R = static_cast<uint32_t>(ex.rows);
    a.slices = static_cast<uint32_t>(pl.Fp / 64);
    a.splits = pl.split_x;
    a.ldS = static_cast<uint32_t>(pl.ldK);
    a.split_stride = pl.s_stride;
    return product<true, true, kSum>(a, pl, a.N, ex.b, s);
}

}  // namespace cbk
