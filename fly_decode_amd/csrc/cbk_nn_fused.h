// The matrix product of up to 384 tokens with weights that are decoded on the way (no decoded copy
// in memory), for widths 8 to 14.  Included by cbk_nn_fused_*.hip, which instantiate it for one
// width each (they compile side by side).
//
// At these token counts the weights' decoding costs more than the product, and decoding a piece
// into memory first costs several times the compressed bytes in traffic, so each weight is decoded
// once, by the one workgroup that multiplies it with all tokens.
//
// Tiles and slices.  A tile is 128 columns of C: forward (NN false) 128 rows of a tensor, gradient
// (NN true) 128 of its columns.  A pair's second tensor has tiles of its own after the first's, so a
// workgroup holds one table at a time.  The reduction is walked in slices of 64.  All (tile, slice)
// pairs in order are divided evenly among the grid's workgroups, whatever the shape, so a workgroup
// takes a run of slices that may cover parts of several tiles; each part's fp32 sums [tokens][128]
// go to slot (workgroup + tile) of the partial buffer, and the kernel that follows adds a tile's
// parts in order (nothing depends on timing).
//
// A slice's 128 x 64 weights are 512 tasks of 16 consecutive fields, one a lane.  A task's fields start
// on a dword, or half-way into one for odd widths, where rows are whole 64-field units; where they are
// not (RAG) they start anywhere.  A funnel shift by the lane's own amount moves them into place.  A lane's
// dwords are loaded two slices before they are decoded.
//
// The weights are decoded, and the tokens' part of the slice copied straight into LDS, two slices ahead of
// the product, into a ring of three buffers (or one slice ahead, into a ring of two: nn_fused_ring).  In a slice's interval a wave reads the second half of this
// slice's fragments and the first half of the next one's while it multiplies the halves it has, and decodes
// its tasks (LDS gathers) in between: one barrier an interval, and no wait on anything asked for in it.
// LDS layouts: rows of 128 bytes (64 reduction elements) hold chunk c of row r in slot c ^ (r & 7), the
// gradient's rows of 256 bytes in c ^ (2 (r & 3) + 8 ((r / 8) & 1)), which keeps fragment reads, transposing
// reads and decoded stores free of bank conflicts.
//
// Measured at 13 bits: 13 tokens and a pair of 8192 x 28672 178 us, 4.3 TB/s of index words; 200 tokens and
// a pair of 4096 x 11008 67 us, 2.2 TB/s and 540 TFLOP/s; 320-token tiles of a 4096-wide head 660 TFLOP/s.
// With few tokens it is bound by the gathers, whose bank conflicts are half of the LDS's busy time and
// cannot be laid out away (the indices are the data).  With more nothing is saturated: at 13 bits one
// workgroup of eight waves has the LDS of a CU, and at 200 tokens the LDS is busy 49 % and the matrix cores 32 %
// of the time while the waves wait 43 %.  Without the decoding the 200-token product took 51 us, without the
// multiplications 55.
#pragma once
#include <type_traits>

#include "cbk_device.h"
#include "cbk_nn_device.h"

namespace cbk {
namespace {

// LDS of a workgroup.  With a ring of three, slices are decoded and copied two ahead of the product; with two,
// one ahead, and an interval starts by reading its own fragments.
template <int B, int BM>
constexpr uint32_t fused_lds() {
    static_assert(Table<B>::SIZE * 2 == (2u << B) && nn_fused_lds(B, BM) <= kLdsLimit, "the LDS that the plan counts with");
    return nn_fused_lds(B, BM);
}

// Dwords of a task of 16 fields, wherever it may start: with RAG anywhere, else on a dword or half-way.
template <int B, bool RAG>
constexpr int task_dwords() { return RAG ? (16 * B + 62) / 32 : (B + 1) / 2; }

// D dwords at byte offset off, in (D + 3) / 4 loads.
template <int D>
__device__ __forceinline__ void load_fields(uint32_t (&d)[D], __amdgpu_buffer_rsrc_t rs, uint32_t off) {
#pragma unroll
    for (int i = 0; i < D / 4; ++i) {
        const u32x4 t = __builtin_amdgcn_raw_buffer_load_b128(rs, static_cast<int>(off + 16 * i), 0, 0);
        d[4 * i] = t.x; d[4 * i + 1] = t.y; d[4 * i + 2] = t.z; d[4 * i + 3] = t.w;
    }
    constexpr int at = D / 4 * 4;
    if constexpr (D % 4 == 3) {
        const u32x3 t = __builtin_amdgcn_raw_buffer_load_b96(rs, static_cast<int>(off + 4 * at), 0, 0);
        d[at] = t.x; d[at + 1] = t.y; d[at + 2] = t.z;
    } else if constexpr (D % 4 == 2) {
        const u32x2 t = __builtin_amdgcn_raw_buffer_load_b64(rs, static_cast<int>(off + 4 * at), 0, 0);
        d[at] = t.x; d[at + 1] = t.y;
    } else if constexpr (D % 4 == 1) {
        d[at] = __builtin_amdgcn_raw_buffer_load_b32(rs, static_cast<int>(off + 4 * at), 0, 0);
    }
}

// 16 fields to two 16-byte chunks of a row in LDS, chunk c0 + i in slot (c0 + i) ^ swz.  Fields from
// `have` on are zeros where MASK is set.
template <int B, bool MASK, int N>
__device__ __forceinline__ void decode_fields(const uint32_t (&d)[N], const uint16_t *tbl, unsigned char *row, uint32_t c0,
                                              uint32_t swz, uint32_t have) {
    uint32_t w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = unit_gather<B>(tbl, d, i);
    if constexpr (MASK) {
#pragma unroll
        for (uint32_t i = 0; i < 16; ++i) w[i] = i < have ? w[i] : 0u;
    }
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        const uint32_t *v = w + 8 * g;
        *reinterpret_cast<u32x4 *>(row + ((c0 + g) ^ swz) * 16) =
            (u32x4){v[0] | (v[1] << 16), v[2] | (v[3] << 16), v[4] | (v[5] << 16), v[6] | (v[7] << 16)};
    }
}

// N column fragments by transposing reads, their second halves HI bytes after the first; `at` are LDS
// addresses, OFF an offset for all.  Written out because the compiler holds the transposing read back
// until every copy into LDS has landed; the block waits for its own reads.
template <int HI, int OFF>
__device__ __forceinline__ void read_columns(bf16x8_t (&x)[1], const uint32_t (&at)[1]) {
    u32x2 a0, b0;
    asm volatile(
        "ds_read_b64_tr_b16 %0, %2 offset:%c3\n"
        "ds_read_b64_tr_b16 %1, %2 offset:%c4\n"
        "s_waitcnt lgkmcnt(0)\n"
        : "=&v"(a0), "=&v"(b0)
        : "v"(at[0]), "i"(OFF), "i"(OFF + HI)
        : "memory");
    x[0] = __builtin_bit_cast(bf16x8_t, (u32x4){a0.x, a0.y, b0.x, b0.y});
}
template <int HI, int OFF>
__device__ __forceinline__ void read_columns(bf16x8_t (&x)[2], const uint32_t (&at)[2]) {
    u32x2 a0, a1, b0, b1;
    asm volatile(
        "ds_read_b64_tr_b16 %0, %4 offset:%c6\n"
        "ds_read_b64_tr_b16 %1, %4 offset:%c7\n"
        "ds_read_b64_tr_b16 %2, %5 offset:%c6\n"
        "ds_read_b64_tr_b16 %3, %5 offset:%c7\n"
        "s_waitcnt lgkmcnt(0)\n"
        : "=&v"(a0), "=&v"(b0), "=&v"(a1), "=&v"(b1)
        : "v"(at[0]), "v"(at[1]), "i"(OFF), "i"(OFF + HI)
        : "memory");
    x[0] = __builtin_bit_cast(bf16x8_t, (u32x4){a0.x, a0.y, b0.x, b0.y});
    x[1] = __builtin_bit_cast(bf16x8_t, (u32x4){a1.x, a1.y, b1.x, b1.y});
}
template <int HI, int OFF>
__device__ __forceinline__ void read_columns(bf16x8_t (&x)[4], const uint32_t (&at)[4]) {
    u32x2 a0, a1, a2, a3, b0, b1, b2, b3;
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
        : "=&v"(a0), "=&v"(b0), "=&v"(a1), "=&v"(b1), "=&v"(a2), "=&v"(b2), "=&v"(a3), "=&v"(b3)
        : "v"(at[0]), "v"(at[1]), "v"(at[2]), "v"(at[3]), "i"(OFF), "i"(OFF + HI)
        : "memory");
    x[0] = __builtin_bit_cast(bf16x8_t, (u32x4){a0.x, a0.y, b0.x, b0.y});
    x[1] = __builtin_bit_cast(bf16x8_t, (u32x4){a1.x, a1.y, b1.x, b1.y});
    x[2] = __builtin_bit_cast(bf16x8_t, (u32x4){a2.x, a2.y, b2.x, b2.y});
    x[3] = __builtin_bit_cast(bf16x8_t, (u32x4){a3.x, a3.y, b3.x, b3.y});
}

// Keeps memory loads and copies into LDS in the order in which they stand: the waits that let the words
// of later slices stay in flight count on the copies having been asked for first.  Arithmetic, matrix and
// LDS instructions may still move past.
__device__ __forceinline__ void keep_order() { __builtin_amdgcn_sched_barrier(0x78F); }

// Waves of a workgroup over the 128 columns; the other factor of 8 goes over the tokens.
constexpr int fused_wn(int BM) { return BM >= 192 ? 2 : BM >= 64 ? 4 : 8; }

template <int B, int BM, bool NN, bool RAG>
__global__ __launch_bounds__(512) void k_fused(const FusedArgs p) {
    constexpr int WN = fused_wn(BM), WM = 8 / WN;
    constexpr int FM = BM / WM / 16, FN = kFusedTile / WN / 16;
    constexpr uint32_t XBYTES = BM * 128, WBYTES = kFusedTile * 128, SLICE = XBYTES + WBYTES;
    constexpr int XC = BM / 8, IX = (XC + 7) / 8;  // copies of a slice of the tokens, by a wave
    constexpr int DW = task_dwords<B, RAG>(), NL = (DW + 3) / 4;
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    uint16_t *table = reinterpret_cast<uint16_t *>(smem);
    constexpr uint32_t RING = nn_fused_ring(B, BM), AHEAD = RING - 1;
    unsigned char *ring = smem + Table<B>::SIZE * 2;  // slices: the tokens' part, then the weights'
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t li = lane & 15, lg = lane >> 4;
    const int wm = wave / WN, wn = wave % WN;

    // this lane's task: its row and 16-field group within a slice
    const uint32_t trow = NN ? tid >> 3 : tid >> 2, tgrp = NN ? tid & 7 : tid & 3;
    const uint32_t swz = NN ? 2 * (trow & 3) + 8 * ((trow >> 3) & 1) : trow & 7;
    const uint32_t wrow = trow * (NN ? 256u : 128u);
    // copies of the tokens' slice; where there are fewer than eight, the waves past them repeat the last
    uint32_t vx[IX], wx[IX];
#pragma unroll
    for (int i = 0; i < IX; ++i) {
        wx[i] = min(wave + 8 * i, XC - 1);
        const uint32_t r = wx[i] * 8 + (lane >> 3), c = (lane & 7) ^ (lane >> 3);
        vx[i] = min(r, p.M - 1) * static_cast<uint32_t>(p.lda) * 2u + c * 16u;
    }
    const auto rx = wave_rsrc(p.A, 0x7FFFFFF0u);
    // fragment reads
    const uint32_t fa = (wm * (BM / WM) + li) * 128 + ((lg ^ (li & 7)) * 16);
    const uint32_t fb = (wn * (kFusedTile / WN) + li) * 128 + ((lg ^ (li & 7)) * 16);
    uint32_t ft[FN];
    if constexpr (NN) {
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            const uint32_t r = 8 * lg + (li >> 2);
            const uint32_t c = (wn * (kFusedTile / WN) + 16 * j) / 8 + ((li & 3) >> 1);
            ft[j] = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((CBK_LDS unsigned char *)(ring))) + XBYTES + r * 256 + (c ^ (2 * (r & 3) + 8 * (lg & 1))) * 16 + (li & 1) * 8;
        }
    }

    const uint64_t total = static_cast<uint64_t>(p.count * p.tiles) * p.slices;
    uint64_t pos = quotient(blockIdx.x * total, gridDim.x);
    const uint64_t end = quotient((blockIdx.x + 1) * total, gridDim.x);
    uint32_t staged = ~0u;  // the tensor whose table is in LDS
    while (pos < end) {
        const uint32_t vt = static_cast<uint32_t>(quotient(pos, p.slices)), s0 = static_cast<uint32_t>(pos - static_cast<uint64_t>(vt) * p.slices);
        const uint32_t s1 = static_cast<uint32_t>(min(static_cast<uint64_t>(p.slices), s0 + (end - pos)));
        const uint32_t which = vt >= p.tiles, tile = vt - which * p.tiles;
        const FusedTensor &T = p.t[which];

        // Where this lane's task of slice s0 starts: the tensor's row `row` (a base on a dword), and the
        // lane's first field after its start.  A slice on is 64 fields, or 64 rows, which are whole dwords,
        // so `shift`, where the first field starts in its dword, stays.
        const uint64_t row = p.row0 + (NN ? static_cast<uint64_t>(s0) * 64 : static_cast<uint64_t>(tile) * kFusedTile);
        const uint64_t base_bits = row * p.cols * B;
        const uint32_t bit = (trow * p.cols + (NN ? tile * kFusedTile : s0 * 64) + tgrp * 16) * B + (RAG ? static_cast<uint32_t>(base_bits) & 31u : 0u);
        const uint32_t shift = bit & 31u, first = (bit >> 5) * 4u;
        const uint64_t start = (base_bits >> 5) * 4, step = NN ? static_cast<uint64_t>(p.cols) * (8 * B) : 8 * B;  // bytes
        uint64_t words_at = reinterpret_cast<uint64_t>(T.words) + start, rest = T.bytes > start ? T.bytes - start : 0;
        // kept in scalar registers: loading them again in the loop would wait for the LDS too
        asm volatile("" : "+s"(words_at), "+s"(rest));
        struct Words {
            uint32_t d[DW];
        };
        // The dwords of the task in slice s (past the run, those of its last slice again); what is past the
        // stream's end reads as zeros.
        auto load = [&](Words &w, uint32_t s) {
            const uint32_t n = min(s, s1 - 1) - s0;
            const uint64_t at = NN ? n * step : 0, have = rest > at ? rest - at : 0;
            const auto rs = wave_rsrc(reinterpret_cast<const unsigned char *>(words_at + (rest > at ? at : 0)),
                                      static_cast<uint32_t>(min(have, static_cast<uint64_t>(0x7FFFFFF0u))));
            load_fields<DW>(w.d, rs, first + (NN ? 0u : n * (8 * B)));
        };
        auto decode = [&](const Words &w, uint32_t s, uint32_t at) {
            // zeros where the reduction runs past the piece's rows (gradient) or the rows' ends
            uint32_t have = 16;
            if constexpr (NN)
                have = s * 64 + trow < p.nrows ? 16u : 0u;
            else if constexpr (RAG)
                have = p.cols > s * 64 + tgrp * 16 ? p.cols - (s * 64 + tgrp * 16) : 0u;
            unsigned char *to = ring + at + XBYTES + wrow;
            if constexpr (RAG || B % 2 == 1) {
                constexpr int N = (B + 1) / 2;
                uint32_t e[N];
#pragma unroll
                for (int i = 0; i < N; ++i) e[i] = __builtin_amdgcn_alignbit(i + 1 < DW ? w.d[i + 1] : 0u, w.d[i], shift);
                decode_fields<B, NN || RAG>(e, table, to, tgrp * 2, swz, have);
            } else {
                decode_fields<B, NN>(w.d, table, to, tgrp * 2, swz, have);
            }
        };
        // the tokens' part of slice s of this tensor (past the run: the last slice again)
        auto copy = [&](uint32_t s, uint32_t at) {
            const uint32_t from = min(s, s1 - 1) + (NN ? which * p.slices : 0u);
#pragma unroll
            for (int i = 0; i < IX; ++i) copy_to_lds(rx, ring + at + wx[i] * 1024, vx[i], from * 128);
        };

        f32x4_t acc[FM][FN];
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j) acc[i][j] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
        // The fragments of half KS of the slice at ring offset `at`.
        struct Frags {
            bf16x8_t a[FM], b[FN];
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
            for (int i = 0; i < FM; ++i)
                f.a[i] = __builtin_bit_cast(bf16x8_t, *reinterpret_cast<const u32x4 *>(sa + (fa ^ (KS * 64)) + i * 2048));
        };
        const std::integral_constant<int, 0> lower;
        const std::integral_constant<int, 1> upper;
        auto multiply = [&](const Frags &f) {
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f.b[j], f.a[i], acc[i][j], 0, 0, 0);
        };

        // Before the first interval: the table; the AHEAD first slices decoded and copied; the words of the
        // two after them on their way.  Everything that does not wait for anything else is asked for at once.
        Words w0, w1;
        lds_barrier();  // the previous part's last reads
        copy(s0, 0);
        if constexpr (AHEAD == 2) copy(s0 + 1, SLICE);
        keep_order();
        if (staged != which) {
            staged = which;
            CbStage<B, 512> cs;
            cs.issue(T.cb, T.U, reinterpret_cast<const u32x4 *>(T.words), tid);
            load(w0, s0);
            load(w1, s0 + 1);
            cs.store(table, T.U, tid);
            lds_barrier();
        } else {
            load(w0, s0);
            load(w1, s0 + 1);
        }
        decode(w0, s0, 0);
        load(w0, s0 + 2);
        if constexpr (AHEAD == 2) {
            decode(w1, s0 + 1, SLICE);
            load(w1, s0 + 3);
        }
        __builtin_amdgcn_s_waitcnt(0x0070 | (2 * NL));
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");

        uint32_t now = 0, fill = AHEAD * SLICE;  // ring offsets of slices s and s + AHEAD
        Frags f0, f1;
        if constexpr (AHEAD == 2) read(f0, 0, lower);
        // One interval: slice s is multiplied, slice s + AHEAD copied and decoded from w, which then takes
        // the words of two slices later.  At its end the copies have landed, and every word but those.
        auto interval = [&](uint32_t s, Words &w) {
            const uint32_t next = now == (RING - 1) * SLICE ? 0 : now + SLICE;
            copy(s + AHEAD, fill);
            if constexpr (AHEAD == 1) read(f0, now, lower);
            read(f1, now, upper);
            multiply(f0);
            if constexpr (AHEAD == 2) read(f0, next, lower);  // after the last slice: old contents of a buffer, not used
            decode(w, s + AHEAD, fill);
            keep_order();
            load(w, s + AHEAD + 2);
            multiply(f1);
            // the multiplications between the LDS reads and the decoding's arithmetic
            if constexpr (BM >= 64) {
                constexpr int MF = 2 * FM * FN, RD = 16 + (NN ? 2 * FM : 2 * (FM + FN));
#pragma unroll
                for (int i = 0; i < MF; ++i) {
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                    __builtin_amdgcn_sched_group_barrier(0x100, (RD + MF - 1) / MF, 0);
                    __builtin_amdgcn_sched_group_barrier(0x002, 96 / MF, 0);
                }
            }
            // multiplications are not put off past the barrier
            __builtin_amdgcn_sched_barrier(0);
            __builtin_amdgcn_s_waitcnt(0x0070 | NL);
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
            fill = now;
            now = next;
        };
        Words &wa = AHEAD == 2 ? w0 : w1, &wb = AHEAD == 2 ? w1 : w0;  // those of s0 + AHEAD, and the next
        uint32_t s = s0;
        for (; s + 1 < s1; s += 2) {
            interval(s, wa);
            interval(s + 1, wb);
        }
        if (s < s1) interval(s, wa);
        __builtin_amdgcn_s_waitcnt(0x0F70);  // no copy is left in flight

        float *out = p.part + (static_cast<uint64_t>(blockIdx.x) + vt) * p.M * kFusedTile;
        const uint32_t mw = wm * (BM / WM) + li, nw = wn * (kFusedTile / WN) + 4 * lg;
#pragma unroll
        for (int i = 0; i < FM; ++i)
            if (mw + 16 * i < p.M) {
#pragma unroll
                for (int j = 0; j < FN; ++j)
                    *reinterpret_cast<f32x4_t *>(out + (mw + 16 * i) * kFusedTile + nw + 16 * j) = acc[i][j];
            }
        pos += s1 - s0;
    }
}

template <int, int, bool, bool>
struct FusedTag;

template <int B, int BM, bool NN, bool RAG>
cbk_status fused_run(const FusedArgs &a, hipStream_t s) {
    constexpr uint32_t lds = fused_lds<B, BM>();
    if (!allow_lds_once<FusedTag<B, BM, NN, RAG>>(k_fused<B, BM, NN, RAG>, lds)) return CBK_E_HIP;
    hipLaunchKernelGGL((k_fused<B, BM, NN, RAG>), dim3(a.grid), dim3(512), lds, s, a);
    return launched();
}

template <int B, int BM>
cbk_status fused_kind(const FusedArgs &a, bool nn, hipStream_t s) {
    const bool rag = a.cols % 64 != 0;
    if (nn) return rag ? fused_run<B, BM, true, true>(a, s) : fused_run<B, BM, true, false>(a, s);
    return rag ? fused_run<B, BM, false, true>(a, s) : fused_run<B, BM, false, false>(a, s);
}

}  // namespace

template <int B>
cbk_status launch_fused(const FusedArgs &a, uint32_t bm, bool nn, hipStream_t s) {
    switch (bm) {
        case 16: return fused_kind<B, 16>(a, nn, s);
        case 64: return fused_kind<B, 64>(a, nn, s);
        case 128: return fused_kind<B, 128>(a, nn, s);
        case 192: return fused_kind<B, 192>(a, nn, s);
        case 256: return fused_kind<B, 256>(a, nn, s);
        case 320: return fused_kind<B, 320>(a, nn, s);
        default: return fused_kind<B, 384>(a, nn, s);
    }
}

}  // namespace cbk
