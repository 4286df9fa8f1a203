// The matrix product of up to 384 tokens with weights that are decoded on the way (no decoded copy
// in memory), for widths 8 to 14.  Included by cbk_nn_fused_*.hip, which instantiate it for one
// width each (they compile side by side).
//
// At these token counts the weights' decoding costs more than the product, and decoding a piece
// into memory first costs several times the compressed bytes in traffic, so each weight is decoded
// once, by the one workgroup that multiplies it with all tokens.
//
// Tiles and slices.  A tile is 128 columns of C; forward (NN false) these are 128 rows of the
// tensor (64 of gate and 64 of up for a pair), gradient (NN true) 128 of its columns.  The
// reduction is walked in slices of 64.  All (tile, slice) pairs in order are divided evenly among
// the grid's workgroups, whatever the shape, so a workgroup takes a run of slices that may cover
// parts of several tiles; each part's fp32 sums [tokens][128] go to slot (workgroup + tile) of the
// partial buffer, and the kernel that follows adds a tile's parts in order (nothing depends on
// timing).
//
// A slice's 128 x 64 weights are 256 tasks of 32 consecutive fields, which are exactly b dwords of
// the stream where rows are whole 32-field groups; where they are not (RAG) a task's fields start
// anywhere in a dword, one more is loaded, and a funnel shift by the lane's own amount moves them
// into place.  The 8 waves form two groups that decode alternate slices one ahead of the product:
// in a slice's interval the waves of one group decode (LDS gathers) while those of the other, one
// on each SIMD as well, feed the matrix cores, so the two pipes overlap by construction.  A lane's
// dwords are loaded two slices ahead into registers; the tokens' slice is copied straight into LDS.
// LDS layouts and fragment reads are those of k_mm.
#pragma once
#include "cbk_device.h"
#include "cbk_nn_device.h"

namespace cbk {
namespace {

template <int B, int BM>
constexpr uint32_t fused_lds(uint32_t tables) {
    return tables * Table<B>::SIZE * 2 + 2 * BM * 128 + 2 * kFusedTile * 128;
}

// This lane's dwords of a slice: as many loads as fused_loads<B>() says, so that a wait can leave
// exactly them in flight.
constexpr int fused_loads(int dwords) { return (dwords + 3) / 4; }

template <int B>
__device__ __forceinline__ void load_fields(uint32_t (&d)[B], __amdgpu_buffer_rsrc_t rs, uint32_t off) {
#pragma unroll
    for (int i = 0; i < B / 4; ++i) {
        const u32x4 t = __builtin_amdgcn_raw_buffer_load_b128(rs, static_cast<int>(off + 16 * i), 0, 0);
        d[4 * i] = t.x; d[4 * i + 1] = t.y; d[4 * i + 2] = t.z; d[4 * i + 3] = t.w;
    }
    constexpr int at = B / 4 * 4;
    if constexpr (B % 4 == 3) {
        const u32x3 t = __builtin_amdgcn_raw_buffer_load_b96(rs, static_cast<int>(off + 4 * at), 0, 0);
        d[at] = t.x; d[at + 1] = t.y; d[at + 2] = t.z;
    } else if constexpr (B % 4 == 2) {
        const u32x2 t = __builtin_amdgcn_raw_buffer_load_b64(rs, static_cast<int>(off + 4 * at), 0, 0);
        d[at] = t.x; d[at + 1] = t.y;
    } else if constexpr (B % 4 == 1) {
        d[at] = __builtin_amdgcn_raw_buffer_load_b32(rs, static_cast<int>(off + 4 * at), 0, 0);
    }
}

// 32 fields to four 16-byte chunks of a row in LDS, chunk c0 + i in slot (c0 + i) ^ swz.  Fields from
// `have` on are zeros where MASK is set.
template <int B, bool MASK>
__device__ __forceinline__ void decode_fields(const uint32_t (&d)[B], const uint16_t *tbl, unsigned char *row, uint32_t c0,
                                              uint32_t swz, uint32_t have) {
    uint32_t w[2][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[0][i] = unit_gather<B>(tbl, d, i);
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        if (g + 1 < 4) {
#pragma unroll
            for (int i = 0; i < 8; ++i) w[(g + 1) & 1][i] = unit_gather<B>(tbl, d, 8 * (g + 1) + i);
        }
        uint32_t *v = w[g & 1];
        if constexpr (MASK) {
#pragma unroll
            for (uint32_t i = 0; i < 8; ++i) v[i] = 8 * g + i < have ? v[i] : 0u;
        }
        const u32x4 t = {v[0] | (v[1] << 16), v[2] | (v[3] << 16), v[4] | (v[5] << 16), v[6] | (v[7] << 16)};
        *reinterpret_cast<u32x4 *>(row + ((c0 + g) ^ swz) * 16) = t;
    }
}

// Waves of a workgroup over the 128 columns; the other factor of 8 goes over the tokens.
constexpr int fused_wn(int BM) { return BM >= 192 ? 2 : BM >= 64 ? 4 : 8; }

template <int B, int BM, bool NN, bool RAG>
__global__ __launch_bounds__(512) void k_fused(const FusedArgs p) {
    constexpr int WN = fused_wn(BM), WM = 8 / WN;
    constexpr int FM = BM / WM / 16, FN = kFusedTile / WN / 16;
    constexpr uint32_t XBYTES = BM * 128, WBYTES = kFusedTile * 128;
    constexpr int XC = BM / 8;           // copies of a slice of the tokens
    constexpr int DW = RAG ? B + 1 : B;  // dwords of a task
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    uint16_t *tables = reinterpret_cast<uint16_t *>(smem);
    unsigned char *xs = smem + p.count * Table<B>::SIZE * 2, *wsl = xs + 2 * XBYTES;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t li = lane & 15, lg = lane >> 4;
    const int wm = wave / WN, wn = wave % WN;
    const int role = wave >> 2;                       // decodes the slices of this parity
    const uint32_t task = static_cast<uint32_t>(wave & 3) * 64 + lane;

    {
        CbStage<B, 512> cs;
        for (uint32_t i = 0; i < p.count; ++i) {
            cs.issue(p.t[i].cb, p.t[i].U, reinterpret_cast<const u32x4 *>(p.t[i].words), tid);
            cs.store(tables + i * Table<B>::SIZE, p.t[i].U, tid);
        }
    }

    // this lane's task: its row and 32-field group within a slice
    const uint32_t trow = NN ? task >> 2 : task >> 1, tgrp = NN ? task & 3 : task & 1;
    const uint32_t swz = NN ? 2 * (trow & 3) + 8 * ((trow >> 3) & 1) : trow & 7;
    const uint32_t wrow = trow * (NN ? 256u : 128u);
    // copies of the tokens' slice
    constexpr int IX = (XC + 7) / 8;
    uint32_t vx[IX];
#pragma unroll
    for (int i = 0; i < IX; ++i) {
        const uint32_t r = (wave + 8 * i) * 8 + (lane >> 3), c = (lane & 7) ^ (lane >> 3);
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
            ft[j] = r * 256 + (c ^ (2 * (r & 3) + 8 * (lg & 1))) * 16 + (li & 1) * 8;
        }
    }

    const uint64_t total = static_cast<uint64_t>(p.tiles) * p.slices;
    uint64_t pos = blockIdx.x * total / gridDim.x;
    const uint64_t end = (blockIdx.x + 1) * total / gridDim.x;
    while (pos < end) {
        const uint32_t tile = static_cast<uint32_t>(pos / p.slices), s0 = static_cast<uint32_t>(pos - static_cast<uint64_t>(tile) * p.slices);
        const uint32_t s1 = static_cast<uint32_t>(min(static_cast<uint64_t>(p.slices), s0 + (end - pos)));

        auto which_of = [&](uint32_t s) -> uint32_t {
            if constexpr (NN) return s >= p.slices_of_first;
            return p.count == 2 ? static_cast<uint32_t>(wave & 2) >> 1 : 0u;  // tasks 0..127 are gate's rows, the others up's
        };
        // The rows [row, ...) of the tensor that slice s takes, and this lane's first field after the
        // start of row `row`.
        auto fields_at = [&](uint32_t s, uint64_t &row) -> uint32_t {
            const uint32_t which = which_of(s);
            if constexpr (NN) {
                row = p.row0 + static_cast<uint64_t>(s - (which ? p.slices_of_first : 0u)) * 64;
                return trow * p.cols + tile * kFusedTile + tgrp * 32;
            } else {
                row = p.row0 + static_cast<uint64_t>(tile) * (p.count == 2 ? 64 : kFusedTile);
                return (trow - which * 64) * p.cols + s * 64 + tgrp * 32;
            }
        };
        uint32_t shift = 0;  // RAG: where the task's first field starts in d[0]
        auto load = [&](uint32_t (&d)[DW], uint32_t s) {
            const FusedTensor &T = p.t[which_of(s)];
            uint64_t row;
            const uint32_t f = fields_at(s, row);
            // a base on a dword; what is past the stream's end reads as zeros
            const uint64_t bits = row * p.cols * B, start = (bits >> 5) * 4;
            const uint64_t rest = T.bytes > start ? T.bytes - start : 0;
            const auto rs = wave_rsrc(reinterpret_cast<const unsigned char *>(T.words) + (rest ? start : 0),
                                      static_cast<uint32_t>(min(rest, static_cast<uint64_t>(0x7FFFFFF0u))));
            if constexpr (RAG) {
                const uint32_t bit = f * B + (static_cast<uint32_t>(bits) & 31u);
                shift = bit & 31u;
                load_fields<DW>(d, rs, (bit >> 5) * 4u);
            } else {
                load_fields<DW>(d, rs, f / 32u * (4u * B));
            }
        };
        auto decode = [&](const uint32_t (&d)[DW], uint32_t s, uint32_t buf) {
            const uint32_t which = which_of(s);
            // zeros where the reduction runs past the piece's rows (gradient) or the rows' ends
            uint32_t have = 32;
            if constexpr (NN)
                have = (s - (which ? p.slices_of_first : 0u)) * 64 + trow < p.nrows ? 32u : 0u;
            else if constexpr (RAG)
                have = p.cols > s * 64 + tgrp * 32 ? p.cols - (s * 64 + tgrp * 32) : 0u;
            const uint16_t *tbl = tables + which * Table<B>::SIZE;
            unsigned char *to = wsl + buf * WBYTES + wrow;
            if constexpr (RAG) {
                uint32_t e[B];
#pragma unroll
                for (int i = 0; i < B; ++i) e[i] = __builtin_amdgcn_alignbit(d[i + 1], d[i], shift);
                decode_fields<B, true>(e, tbl, to, tgrp * 4, swz, have);
            } else {
                decode_fields<B, NN>(d, tbl, to, tgrp * 4, swz, have);
            }
        };
        auto copy = [&](uint32_t s, uint32_t buf) {
#pragma unroll
            for (int i = 0; i < IX; ++i)
                if (XC % 8 == 0 || wave + 8 * i < XC)
                    copy_to_lds(rx, xs + buf * XBYTES + (wave + 8 * i) * 1024, vx[i], s * 128);
        };

        f32x4_t acc[FM][FN];
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j) acc[i][j] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
        // Column fragments of a slice.  The compiler holds transposing reads back until every copy
        // into LDS has landed, so they are all made at the start of an interval, before its copies.
        auto columns = [&](bf16x8_t (&xb)[2][FN], uint32_t buf) {
            const unsigned char *sb = wsl + buf * WBYTES;
#pragma unroll
            for (int ks = 0; ks < 2; ++ks)
#pragma unroll
                for (int j = 0; j < FN; ++j) {
                    if constexpr (NN) {
                        const unsigned char *at = sb + ft[j] + ks * 32 * 256;
                        const s16x4 lo = read_transposed(at), hi = read_transposed(at + 4 * 256);
                        xb[ks][j] = __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
                    } else {
                        xb[ks][j] = __builtin_bit_cast(bf16x8_t, *reinterpret_cast<const u32x4 *>(sb + (fb ^ (ks * 64)) + j * 2048));
                    }
                }
        };
        auto multiply = [&](const bf16x8_t (&xb)[2][FN], uint32_t buf) {
            const unsigned char *sa = xs + buf * XBYTES;
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                bf16x8_t xa[FM];
#pragma unroll
                for (int i = 0; i < FM; ++i)
                    xa[i] = __builtin_bit_cast(bf16x8_t, *reinterpret_cast<const u32x4 *>(sa + (fa ^ (ks * 64)) + i * 2048));
#pragma unroll
                for (int i = 0; i < FM; ++i)
#pragma unroll
                    for (int j = 0; j < FN; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xb[ks][j], xa[i], acc[i][j], 0, 0, 0);
            }
        };

        // Before the first interval: slice s0 decoded and copied, the words of s0 + 1 (by the group
        // that decodes it) and s0 + 2 (by the other) on their way.  Words of slices past the run
        // are not loaded.
        uint32_t d[DW];
        const bool first = role == 0;  // this group decodes s0, s0 + 2, ...
        lds_barrier();                 // the previous part's last reads of the buffers; the tables' stores
        copy(s0, 0);
        if (first) {
            load(d, s0);
            decode(d, s0, 0);
            if (s0 + 2 < s1) load(d, s0 + 2);
        } else if (s0 + 1 < s1) {
            load(d, s0 + 1);
        }
        __builtin_amdgcn_s_waitcnt(0x0070);
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");

        // One interval: slice s is multiplied, slice s + 1 copied and, by its group, decoded.
        auto interval = [&](uint32_t s, bool mine) {
            const uint32_t buf = (s - s0) & 1;
            bf16x8_t xb[2][FN];
            columns(xb, buf);
            if (s + 1 < s1) {
                if (mine) {
                    decode(d, s + 1, buf ^ 1);
                    copy(s + 1, buf ^ 1);
                    if (s + 3 < s1) load(d, s + 3);
                } else {
                    copy(s + 1, buf ^ 1);
                }
            }
            multiply(xb, buf);
            // the copies have landed (the words asked for after them may still be on their way, and
            // are waited for an interval later), this wave's LDS writes are done
            if (mine && s + 3 < s1)
                __builtin_amdgcn_s_waitcnt(0x0070 | fused_loads(DW));
            else
                __builtin_amdgcn_s_waitcnt(0x0070);
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
        };
        if (first) {
            for (uint32_t s = s0; s < s1; s += 2) {
                interval(s, false);
                if (s + 1 < s1) interval(s + 1, true);
            }
        } else {
            for (uint32_t s = s0; s < s1; s += 2) {
                interval(s, true);
                if (s + 1 < s1) interval(s + 1, false);
            }
        }

        float *out = p.part + (static_cast<uint64_t>(blockIdx.x) + tile) * p.M * kFusedTile;
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

template <int B, int BM, bool NN, bool RAG>
cbk_status fused_run(const FusedArgs &a, hipStream_t s) {
    const uint32_t lds = fused_lds<B, BM>(a.count);
    if (!allow_lds(k_fused<B, BM, NN, RAG>, lds)) return CBK_E_HIP;
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
        default: return fused_kind<B, 384>(a, nn, s);
    }
}

}  // namespace cbk
