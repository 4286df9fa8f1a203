// Device helpers shared by the kernels on codebook-compressed tensors (cbk_kernels.hip, cbk_nn.hip):
// field extraction, the codebook table in LDS, step loads and the stage transposition, buffer
// resources and barriers; and the launchers' small host helpers.  Everything has internal linkage.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>
#include <utility>

#include "cbk_internal.h"

namespace cbk {
namespace {

constexpr uint16_t kCorrupt = 0x7FC0;
constexpr uint32_t kLdsLimit = 160 * 1024;

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float dot2(uint32_t w, uint32_t x, float acc) {
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2_t, w),
                                           __builtin_bit_cast(bf16x2_t, x), acc, false);
}

// One step of a wave sum: v plus v moved by the DPP control CTRL within the rows in ROWS (lanes
// whose source is out of range add zero).
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_add(float v) {
    return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, ROWS, 0xF, false));
}

// The sum of v over the 64 lanes (all active), in lane 63: prefix sums within each 16-lane row
// (row_shr 1, 2, 4, 8), then lane 15 of rows 0 and 2 carried into rows 1 and 3 (row_bcast:15) and
// lane 31 into rows 2 and 3 (row_bcast:31).  VALU only, where lane shuffles would be six LDS round
// trips.
__device__ __forceinline__ float wave_sum_last(float v) {
    v = dpp_add<0x111, 0xF>(v);
    v = dpp_add<0x112, 0xF>(v);
    v = dpp_add<0x114, 0xF>(v);
    v = dpp_add<0x118, 0xF>(v);
    v = dpp_add<0x142, 0xA>(v);
    return dpp_add<0x143, 0xC>(v);
}

__device__ __forceinline__ float bf16_value(uint16_t h) {
    return __builtin_bit_cast(float, static_cast<uint32_t>(h) << 16);
}

// Geometry of the 64-field lane unit for width B (decode and GEMV).
template <int B>
struct U64 {
    static constexpr int UD = 2 * B;                            // dwords per unit
    static constexpr int G = (UD % 4 == 0) ? 4 : 2;             // LDS read width (dwords)
    static constexpr int NG = UD / G;                           // reads per unit
    static constexpr bool PAD = (G == 4) && (NG % 2 == 0);      // pad to an odd chunk stride
    static constexpr int SG = PAD ? NG + 1 : NG;                // unit stride in reads
    static constexpr int LPL = (16 * UD + 1 + 63) / 64;         // 16-byte loads per lane per step
    static constexpr int STAGE_CHUNKS = 64 * LPL + (PAD ? 64 * LPL / NG + 1 : 0);
    static constexpr uint32_t NE = 1u << B;                     // codebook entries in LDS
    static constexpr uint32_t mask = (1u << B) - 1u;
};

// Table entry for field f (bits f*B .. f*B + B - 1, LSB first) of a unit held in registers; f is a
// constant once the caller's loop is unrolled.  The field is extracted straight into its byte
// offset 2 * field (shift by one less, mask b bits one place up), two VALU operations whether or
// not the field crosses a word boundary (v_alignbit joins the two words).
template <int B>
__device__ __forceinline__ uint32_t unit_gather(const uint16_t *tbl, const uint32_t *d, int f) {
    const int bit = f * B, w = bit >> 5, s = bit & 31;
    constexpr uint32_t m2 = U64<B>::mask << 1;
    uint32_t off;
    if (s == 0) off = (d[w] << 1) & m2;
    else if (s + B <= 32) off = (d[w] >> (s - 1)) & m2;
    else off = __builtin_amdgcn_alignbit(d[w + 1], d[w], s - 1) & m2;
    return *reinterpret_cast<const uint16_t *>(reinterpret_cast<const unsigned char *>(tbl) + off);
}

// Field i of a stream, runtime width (generic kernels).
__device__ __forceinline__ uint32_t stream_field(const uint32_t *__restrict__ words, uint32_t b,
                                                 uint64_t i) {
    if (b == 0) return 0;
    const uint64_t bit = i * b;
    const uint64_t w = bit >> 5;
    const uint32_t s = static_cast<uint32_t>(bit) & 31u;
    const uint32_t lo = words[w];
    const uint32_t hi = (s + b > 32) ? words[w + 1] : 0u;
    return __builtin_amdgcn_alignbit(hi, lo, s) & ((1u << b) - 1u);
}

// Codebook table in LDS: 2^b entries (at least 8) so any b-bit index stays inside it.
template <int B>
struct Table {
    static constexpr uint32_t NCH = (U64<B>::NE + 7) / 8;  // 16-byte chunks
    static constexpr uint32_t SIZE = NCH * 8;               // entries
};

// Codebook staging for the fast kernels: the table of Table<B>::NCH 16-byte chunks (entries >= U
// read 0x7FC0) is loaded branch-free by NT threads, CPT chunks each: whole 16-byte loads clamped
// into the codebook's whole chunks (from `dummy`, any readable 16-byte-aligned address, when it
// has none) plus the eight entries of the chunk that straddles U, one per lane in lanes 0..7 of
// every wave and broadcast with readlane.  Kernels issue these loads in every wave before a
// barrier and their first weight loads after it: vector-memory data returns in issue order, so
// the staging never waits behind the grid's first burst of weight loads.  Needs a 16-byte-aligned
// codebook.
template <int B, int NT>
struct CbStage {
    static constexpr int CPT = (Table<B>::NCH + NT - 1) / NT;
    u32x4 cw[CPT];
    uint32_t te;  // lane j < 8: entry 8 * full + j (clamped into the codebook)

    __device__ __forceinline__ void issue(const uint16_t *__restrict__ cb, uint32_t U, const u32x4 *dummy, int tid) {
        const uint32_t full = U / 8;
#pragma unroll
        for (int i = 0; i < CPT; ++i)
            cw[i] = full ? reinterpret_cast<const u32x4 *>(cb)[min(static_cast<uint32_t>(i * NT + tid), full - 1)] : *dummy;
        te = cb[min(8 * full + (tid & 7), U - 1)];
    }

    __device__ __forceinline__ void store(uint16_t *cbl, uint32_t U, int tid) const {
        const uint32_t full = U / 8;
        uint32_t e[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t v = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(te), j));
            e[j] = 8 * full + j < U ? v : kCorrupt;
        }
        const uint32_t fill = static_cast<uint32_t>(kCorrupt) * 0x10001u;
        const u32x4 tail = {e[0] | (e[1] << 16), e[2] | (e[3] << 16), e[4] | (e[5] << 16), e[6] | (e[7] << 16)};
        const u32x4 pad = {fill, fill, fill, fill};
#pragma unroll
        for (int i = 0; i < CPT; ++i) {
            const uint32_t c = i * NT + tid;
            if (c < Table<B>::NCH) reinterpret_cast<u32x4 *>(cbl)[c] = c < full ? cw[i] : (c == full ? tail : pad);
        }
    }
};

// Workgroup barrier on LDS only: outstanding global loads stay in flight.
__device__ __forceinline__ void lds_barrier() {
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0), vmcnt and expcnt unconstrained
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// Barrier that waits for nothing: orders the waves' instruction streams (used to put every wave's
// staging loads ahead of any weight load in the CU's memory pipeline).
__device__ __forceinline__ void issue_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// Raw buffer resource over `bytes` bytes from `base`, which must be the same in every lane of the
// wave.  Loads at offsets at or past `bytes` return zeros without a memory access, so weight loads
// need neither clamped addresses nor branches, and the base and its arithmetic stay in scalar
// registers.  Word 3 sets the 32-bit data format, which this chip's untyped buffer loads need.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t wave_rsrc(const void *base, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), static_cast<short>(0),
                                             static_cast<int>(bytes), 0x00020000);
}

// Cache policy of the buffer operations on data that is touched exactly once (the packed index
// stream, the decoded output): the non-temporal bit (NT, bit 1 of the aux operand on this chip), so
// the stream does not displace the codebook, x and X from the caches.  It took the standalone
// decode of a 4096^2 tensor from 16.7 to 11.4 us and the GEMV launches 1-3 % faster.
constexpr int kStreamOnce = 2;

__device__ __forceinline__ u32x4 rsrc_load(__amdgpu_buffer_rsrc_t rs, uint32_t byte_offset) {
    return __builtin_amdgcn_raw_buffer_load_b128(rs, static_cast<int>(byte_offset), 0, kStreamOnce);
}

// Step loads: the chunks covering units [us, us + nl) start at chunk (us * UD) / 4; an odd-b step
// may start half-way into a chunk (the stage read then skips one qword).  Lane l loads chunks
// 64 j + l of the step; chunks past the step (or past the stream's nchunks) read as zero, and a
// wave with no step (valid false) touches no memory.  `us` must be wave-uniform.
template <int B>
__device__ __forceinline__ void load_step(u32x4 (&v)[U64<B>::LPL], const u32x4 *__restrict__ w4,
                                          uint32_t us, uint32_t nl, uint64_t nchunks, bool valid, int lane) {
    const uint64_t c0 = (static_cast<uint64_t>(us) * U64<B>::UD) >> 2;
    const uint64_t c1 = min((static_cast<uint64_t>(us + nl) * U64<B>::UD + 3) >> 2, nchunks);
    const auto rs = wave_rsrc(w4 + c0, valid && c1 > c0 ? static_cast<uint32_t>(c1 - c0) * 16u : 0u);
#pragma unroll
    for (int j = 0; j < U64<B>::LPL; ++j) v[j] = rsrc_load(rs, static_cast<uint32_t>(j * 64 + lane) * 16u);
}

// Write a step to the wave's stage and read back this lane's unit (UD dwords).
template <int B>
__device__ __forceinline__ void transpose_step(uint32_t (&d)[U64<B>::UD], const u32x4 (&v)[U64<B>::LPL],
                                               u32x4 *stage, uint32_t us, int lane) {
    using G = U64<B>;
    // The stage is written as 16-byte vectors and, for odd b, read as 8-byte vectors; the
    // compiler barriers keep type-based alias analysis from moving the reads above the writes
    // (or the next step's writes above these reads).  LDS executes one wave's accesses in order.
    asm volatile("" ::: "memory");
#pragma unroll
    for (int j = 0; j < G::LPL; ++j) {
        const uint32_t q = j * 64 + lane;
        stage[G::PAD ? q + q / G::NG : q] = v[j];
    }
    asm volatile("" ::: "memory");
    if constexpr (G::G == 4) {
#pragma unroll
        for (int j = 0; j < G::NG; ++j) {
            const u32x4 t = stage[lane * G::SG + j];
            d[4 * j] = t.x; d[4 * j + 1] = t.y; d[4 * j + 2] = t.z; d[4 * j + 3] = t.w;
        }
    } else {
        // odd b: the step starts (us * UD) % 4 dwords into its first chunk (0 or 2)
        const u32x2 *st2 = reinterpret_cast<const u32x2 *>(stage) + ((us * G::UD) & 2u) / 2;
#pragma unroll
        for (int j = 0; j < G::NG; ++j) {
            const u32x2 t = st2[lane * G::SG + j];
            d[2 * j] = t.x; d[2 * j + 1] = t.y;
        }
    }
    asm volatile("" ::: "memory");
}
// ------------------------------------------------------------------------------ host side
int cu_count() {
    static std::atomic<int> cached[64];
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
    int v = cached[dev].load(std::memory_order_relaxed);
    if (v <= 0) {
        if (hipDeviceGetAttribute(&v, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || v <= 0) v = 256;
        cached[dev].store(v, std::memory_order_relaxed);
    }
    return v;
}

cbk_status launched() { return hipGetLastError() == hipSuccess ? CBK_OK : CBK_E_HIP; }

// Kernels above 64 KiB of dynamic LDS must raise their limit first.
template <typename K>
bool allow_lds(K kernel, uint32_t lds) {
    if (lds <= 65536) return true;
    return hipFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                               hipFuncAttributeMaxDynamicSharedMemorySize,
                               static_cast<int>(lds)) == hipSuccess;
}

// The same, asked of the runtime once for a kernel and device (Tag: a type of the kernel's own).
template <typename Tag, typename K>
bool allow_lds_once(K kernel, uint32_t lds) {
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess) return false;
    const uint64_t bit = dev >= 0 && dev < 64 ? uint64_t(1) << dev : 0;
    if (bit && (done.load(std::memory_order_relaxed) & bit)) return true;
    if (!allow_lds(kernel, lds)) return false;
    done.fetch_or(bit, std::memory_order_relaxed);
    return true;
}

// Runs Fn<b>::run(args) for the b in Bs that matches; false when none does or run declines.
template <template <int> class Fn, typename Args, int... Bs>
bool dispatch_b(int b, Args &args, std::integer_sequence<int, Bs...>) {
    bool ok = false;
    (void)((b == Bs ? (ok = Fn<Bs>::run(args), true) : false) || ...);
    return ok;
}
using AllB = std::integer_sequence<int, 1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 13, 14, 15, 16>;

}  // namespace
}  // namespace cbk
