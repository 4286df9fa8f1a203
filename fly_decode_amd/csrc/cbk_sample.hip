// HIP kernels for gfx950 (CDNA4) of cbk_sample.h: drawing a token from a row of logits.
//
// Every filter keeps a prefix of the row's order (logits falling, then index), so what is kept is what stands before
// one cut in that order, a 64-bit key of logit and index, and no row is sorted.  A histogram over the logits, in bins of a
// sixteenth of the temperature, finds the bin that a cut falls into; the entries of that bin alone are ranked, in LDS.
// Sums whose order could vary (atomic additions) are of fixed-point numbers, so they have the same bits in any order.
//
// Without filters (the call's numbers say so) a wave has a segment of 1024 entries, and a workgroup joins a row's
// (k_sample_parts, k_sample_join): one pass, on all of the chip also for one row.  With filters a workgroup of 16 waves
// has a row (k_sample), or, where rows are long and few, the end of it, after its passes were shared among workgroups
// (k_sample_bins, k_sample_collect).  sample_plan has the rule, and both sides' times.
//
// A row of 10^5 logits is read from memory or the last cache each time, so k_sample's passes over it are few.  No pass
// looks for the maximum first: bins and exponentials are relative to the largest of the first 4096 logits.
//   temperature alone: one pass, a sum of exponentials of each 1024 entries;
//   top_k (up to some 1500): one that counts (two where the first logits are far below the others), and one that collects the
//     entries up to the cut's bin; all other filters and the draw are then done on that list;
//   top_p: one that adds up the bins, and one that collects the cut's bin and adds up what stands before it;
//   min_p without top_k: one for the maximum before those.
// The draw takes the sums of each 1024 entries in index order, then the 1024 that the target falls into.
//
// 192 rows of 128000 fp32 logits take 21 us greedy (4.7 TB/s: memory), 43 by temperature alone, 52 with top_k = 50, 126
// with top_p = 0.9.  Past the first reading the vector units bound it: some 60 instructions an entry for the bins' masses.
// One row of 128000 takes 12, 15, 28 and 45, what two and four dependent launches take; one of 32000 24 with top_k = 50, 27 with
// min_p and top_p too, 45 with top_p = 0.9 alone.
//
// The border between two tokens can be anywhere, and a vocabulary has 10^5 of them, so probabilities are
// formed in fp64: an fp32 sum's 1e-7 would name another token once in some hundred rows.  On this chip
// fp64 multiplications run at the rate of fp32 ones that are not packed.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#pragma clang diagnostic ignored "-Wunused-function"  // cu_count of cbk_device.h
#include "cbk_device.h"
#include "cbk_exp.h"

namespace cbk {
namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr uint32_t kBins = 2048;           // of the histogram, 1/16 of the temperature each; the last one holds the rest
constexpr float kPerUnit = 16.f;
constexpr float kAbove = 16.f;             // what the first bin starts above the reference, in units of the temperature
constexpr uint32_t kList = 2048;           // entries of a list,
constexpr uint32_t kRanked = 1024;         // and those of a bin that are ranked against each other
constexpr double kFine = 1125899906842624.0;  // 2^50: units of a segment's and a list's fixed-point masses
constexpr uint32_t kSteps = 4;             // of 256 entries by a wave, in a segment
constexpr uint32_t kSegments = (1u << 20) / (256 * kSteps) + 2;

// A segment of 1024 entries: its largest logit, and its masses relative to that.
struct Part {
    double sum;
    float top;
    uint32_t odd;  // it holds a NaN
};
// What the kernels before k_sample found of a row (see "filters, divided").
struct RowState {
    uint32_t listed;  // entries that the list was for (it holds kList at most)
    uint32_t bin;     // of the cut by mass; kBins: none
    double most;      // of mass before the cut, in that bin
};
struct SampleArgs {
    cbk_sampling p;
    const void *logits;
    uint64_t ld;
    uint32_t V;
    const float *uniform;
    int64_t *token;
    float *logprob;
    // the workspace: by row, for each of its segments; null where a call has none
    uint32_t segments;
    Part *parts;
    uint64_t *sums;  // kept masses of a segment: fixed point, or a double's bits
    uint64_t *bins, *list;
    RowState *state;
};

struct Shared {
    uint64_t mass[kBins];
    uint32_t count[kBins];
    uint64_t list[kList];
    uint64_t ranked[kRanked];
    union {
        double segment[kSegments];
        uint64_t fixed_segment[kSegments];
    };
    uint64_t wave64[kWaves];
    uint32_t wave32[kWaves];
    double wavef[kWaves];
    uint64_t found64[2];
    uint32_t found32[3];
};

// Ascending unsigned numbers for ascending floats (-0 as +0; no NaN).
__device__ __forceinline__ uint32_t ascending(float z) {
    const uint32_t u = __float_as_uint(z + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float from_ascending(uint32_t u) { return __uint_as_float(u & 0x80000000u ? u & 0x7FFFFFFFu : ~u); }
// A place in the row's order: smaller keys come first.
__device__ __forceinline__ uint64_t place_key(float z, uint32_t i) { return (static_cast<uint64_t>(~ascending(z)) << 32) | i; }

// e^x for -0.08 < x < 0.02, the series alone: the first left-out term is below 0.08^9 / 9! < 1e-15 of it.
__device__ __forceinline__ double exponential_near_0(double x) {
    double s = 1.0 / 40320.0;
    s = fma(s, x, 1.0 / 5040.0);
    s = fma(s, x, 1.0 / 720.0);
    s = fma(s, x, 1.0 / 120.0);
    s = fma(s, x, 1.0 / 24.0);
    s = fma(s, x, 1.0 / 6.0);
    s = fma(s, x, 0.5);
    s = fma(s, x, 1.0);
    return fma(s, x, 1.0);
}
// The integer nearest to m * scale, both positive, below 2^51: in the low bits of its sum with 2^52.
__device__ __forceinline__ uint64_t rounded(double m, double scale) {
    return __builtin_bit_cast(uint64_t, fma(m, scale, 4503599627370496.0)) & ((uint64_t(1) << 52) - 1);
}

// A row, in groups of four logits that start on whole multiples of four elements in memory; the first group's `skew` first
// ones lie before the row.  Groups are read whole, through a resource that ends with the row's last dword (past it nothing
// is read), and what is not the row's becomes -inf.
template <typename T>
struct Row {
    __amdgpu_buffer_rsrc_t rs;
    uint32_t V, skew, groups;

    __device__ __forceinline__ Row(const void *logits, uint64_t ld, uint32_t row, uint32_t n) {
        const T *p = static_cast<const T *>(logits) + row * ld;
        V = n;
        skew = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) / sizeof(T)) & 3;
        groups = (V + skew + 3) / 4;
        rs = wave_rsrc(p - skew, ((V + skew) * static_cast<uint32_t>(sizeof(T)) + 3) & ~3u);
    }
    typedef std::conditional_t<sizeof(T) == 4, u32x4, u32x2> Raw;
    __device__ __forceinline__ Raw raw(uint32_t g) const {
        if constexpr (sizeof(T) == 4) return __builtin_amdgcn_raw_buffer_load_b128(rs, static_cast<int>(g * 16), 0, 0);
        else return __builtin_amdgcn_raw_buffer_load_b64(rs, static_cast<int>(g * 8), 0, 0);
    }
    // The index of the group's first entry (possibly before the row) and its four logits.
    __device__ __forceinline__ int32_t values(uint32_t g, Raw v, float (&z)[4]) const {
        if constexpr (sizeof(T) == 4) {
            z[0] = __uint_as_float(v.x); z[1] = __uint_as_float(v.y); z[2] = __uint_as_float(v.z); z[3] = __uint_as_float(v.w);
        } else {
            z[0] = __uint_as_float(v.x << 16); z[1] = __uint_as_float(v.x & 0xFFFF0000u);
            z[2] = __uint_as_float(v.y << 16); z[3] = __uint_as_float(v.y & 0xFFFF0000u);
        }
        const int32_t at = static_cast<int32_t>(4 * g) - static_cast<int32_t>(skew);
        if (g == 0 || g + 1 >= groups) {
#pragma unroll
            for (int j = 0; j < 4; ++j) z[j] = at + j >= 0 && at + j < static_cast<int32_t>(V) ? z[j] : -__builtin_inff();
        }
        return at;
    }
    __device__ __forceinline__ int32_t load(uint32_t g, float (&z)[4]) const { return values(g, raw(g), z); }
};

// f(index of the first, four logits, segment, whether it is the wave's last of the segment) for this thread's groups of
// the row, four pieces ahead of it asked for; past the row's end logits are -inf.  A wave has segments of kSteps times 64
// neighbouring groups, every 16th of them.  f's code stands once: a pass is short, and what it takes to fetch its
// instructions counts (unrolled eight times, one row of 32000 took 40 us instead of 28).
template <typename T, typename F>
__device__ __forceinline__ void over_row(const Row<T> &r, F f) {
    constexpr uint32_t N = 4;
    static_assert(N == kSteps, "a group four pieces on is the same one of the next segment");
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    typename Row<T>::Raw z[N];
    uint32_t segment = wave, first = wave * (64 * kSteps) + lane;
#pragma unroll
    for (uint32_t i = 0; i < N; ++i) z[i] = r.raw(first + 64 * i);
    uint32_t step = 0;
#pragma unroll 1
    while (segment * (64 * kSteps) < r.groups) {  // a wave stays together
        const uint32_t g = first + 64 * step;
        float now[4];
        const int32_t at = r.values(g, z[0], now);
#pragma unroll
        for (uint32_t i = 0; i + 1 < N; ++i) z[i] = z[i + 1];
        z[N - 1] = r.raw(g + kWaves * (64 * kSteps));
        f(at, now, segment, step == kSteps - 1);
        if (++step == kSteps) {
            step = 0;
            segment += kWaves;
            first += kWaves * (64 * kSteps);
        }
    }
}

// The sum of v over the wave, everywhere, in a fixed order.
__device__ __forceinline__ double wave_total(double v) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
    return v;
}

template <typename V>
__device__ __forceinline__ V shuffle_up(V v, int by) {
    if constexpr (sizeof(V) == 8) {
        const uint64_t u = __builtin_bit_cast(uint64_t, v);
        const uint32_t lo = __shfl_up(static_cast<uint32_t>(u), by, 64), hi = __shfl_up(static_cast<uint32_t>(u >> 32), by, 64);
        return __builtin_bit_cast(V, (static_cast<uint64_t>(hi) << 32) | lo);
    } else {
        return __shfl_up(v, by, 64);
    }
}

// The sum of v over the threads before this one, in thread order; `total`: over all.  `wave` has an entry for each
// wave, and everyone is done with it on return.
template <int WAVES = kWaves, typename V>
__device__ __forceinline__ V sum_before(V v, V *wave, V &total) {
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    V s = v;
#pragma unroll
    for (int by = 1; by < 64; by *= 2) {
        const V t = shuffle_up(s, by);
        if (lane >= by) s += t;
    }
    if (lane == 63) wave[w] = s;
    __syncthreads();
    V before = V(0);
    total = V(0);
#pragma unroll
    for (int i = 0; i < WAVES; ++i) {
        if (i == w) before = total;
        total += wave[i];
    }
    __syncthreads();
    return before + (s - v);
}

// The share of the kept masses that the draw goes past: from 1 on none does, whatever sums round to.
__device__ __forceinline__ double share_of(float u) { return u >= 1.f ? static_cast<double>(__builtin_inff()) : u >= 0.f ? static_cast<double>(u) : 0.0; }

// The first of neighbouring segments whose running sum exceeds the target, or the last that holds anything; thread i has
// `run` of them from i run on, `before` is the sum of those before it, value(s) that of one.  In `first`, what stands before
// the segment.  All threads; found32 has two entries.
template <typename F>
__device__ __forceinline__ uint32_t find_segment(F value, uint32_t segments, uint32_t run, double before, double target,
                                                 uint32_t *found32, double *first) {
    const uint32_t tid = threadIdx.x;
    if (tid == 0) {
        found32[0] = ~0u;
        found32[1] = 0;
    }
    __syncthreads();
    double sum = before;
    uint32_t hit = ~0u, last = 0;
    for (uint32_t i = 0; i < run; ++i) {
        const uint32_t s = tid * run + i;
        if (s >= segments) break;
        const double m = value(s);
        sum += m;
        if (m > 0.0) {
            last = s;
            if (hit == ~0u && sum > target) hit = s;
        }
    }
    if (hit != ~0u) atomicMin(&found32[0], hit);
    if (last) atomicMax(&found32[1], last);
    __syncthreads();
    const uint32_t s = found32[0] != ~0u ? found32[0] : found32[1];
    if (tid == s / run) {
        sum = before;
        for (uint32_t i = tid * run; i < s; ++i) sum += value(i);
        *first = sum;
    }
    __syncthreads();
    return s;
}

// One wave: the first entry of segment s at which the running sum, `before` at its start, exceeds the target, or the last
// that can be drawn.  masses(four logits, index of the first, their masses).
template <typename T, typename F>
__device__ __forceinline__ int64_t draw_from(const Row<T> &r, uint32_t s, double before, double target, F masses, float &drawn) {
    const uint32_t lane = threadIdx.x & 63;
    int64_t token = -1;
    drawn = 0.f;
    typename Row<T>::Raw v[kSteps];
#pragma unroll
    for (uint32_t i = 0; i < kSteps; ++i) v[i] = r.raw((s * kSteps + i) * 64 + lane);
#pragma unroll 1
    for (uint32_t step = 0; step < kSteps; ++step) {
        float z[4];
        double m[4];
        const int32_t at = r.values((s * kSteps + step) * 64 + lane, v[0], z);
#pragma unroll
        for (uint32_t i = 0; i + 1 < kSteps; ++i) v[i] = v[i + 1];
        masses(z, at, m);
        double sum = m[0] + m[1] + m[2] + m[3];
        const double own = sum;
#pragma unroll
        for (int by = 1; by < 64; by *= 2) {
            const double t = shuffle_up(sum, by);
            if (lane >= static_cast<uint32_t>(by)) sum += t;
        }
        const double next = before + __shfl(sum, 63, 64);
        sum = before + (sum - own);
        before = next;
        int32_t hit = -1, end = -1;  // this lane's first entry past the target, and its last that can be drawn
        float hz = 0.f, ez = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            sum += m[j];
            if (m[j] > 0.0) {
                end = at + j;
                ez = z[j];
                if (hit < 0 && sum > target) {
                    hit = at + j;
                    hz = z[j];
                }
            }
        }
        const uint64_t hits = __ballot(hit >= 0), ends = __ballot(end >= 0);
        if (hits || ends) {
            const int who = hits ? __ffsll(static_cast<unsigned long long>(hits)) - 1 : 63 - __clzll(static_cast<long long>(ends));
            token = __shfl(hits ? hit : end, who, 64);
            drawn = __shfl(hits ? hz : ez, who, 64);
        }
        if (hits) break;
    }
    return token;
}

// One wave: the first entry of segment s that is `top`.
template <typename T>
__device__ __forceinline__ int64_t first_of(const Row<T> &r, uint32_t s, float top, float &drawn) {
    return draw_from(r, s, 0.0, 0.5, [&](const float (&z)[4], int32_t, double (&m)[4]) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < 4; ++j) m[j] = z[j] == top ? 1.0 : 0.0;
    }, drawn);
}

// The settings of a row.
struct Settings {
    float heat, top_p, min_p;
    int32_t top_k;
    bool by_count, by_mass;

    __device__ __forceinline__ Settings(const SampleArgs &a, uint32_t row) {
        heat = a.p.temperatures ? a.p.temperatures[row] : a.p.temperature;
        top_k = a.p.top_ks ? a.p.top_ks[row] : a.p.top_k;
        top_p = a.p.top_ps ? a.p.top_ps[row] : a.p.top_p;
        const float given = a.p.min_ps ? a.p.min_ps[row] : a.p.min_p;
        min_p = given > 0.f ? fminf(given, 1.f) : 0.f;
        by_count = top_k > 0 && static_cast<uint32_t>(top_k) < a.V;
        by_mass = top_p < 1.f;
    }
    // The least logit that min_p keeps: rounded up, so that comparing floats is comparing with the border.
    __device__ __forceinline__ float border(float top) const {
        if (!(min_p > 0.f)) return -__builtin_inff();
        if (top == __builtin_inff()) return top;
        if (heat == __builtin_inff()) return -__builtin_inff();  // all are as likely (and log(1) times it is a NaN)
        const double edge = __builtin_fma(static_cast<double>(heat), log(static_cast<double>(min_p)), static_cast<double>(top));
        float least = static_cast<float>(edge);
        if (static_cast<double>(least) < edge) least = from_ascending(ascending(least) + 1);
        return fminf(least, top);
    }
};

// What a row's bins and masses are relative to.
struct Scale {
    float ref, top, least;  // of the bins; the row's largest, once it is known; what min_p leaves out is below it
    // Bins a logit, in two factors: of temperatures below 2^-96 (subnormal ones too) one would pass fp32's range.  A clamp of
    // it made bins wider than a sixteenth there, for which exponential_near_0 is none.  (The factor costs 0.5 % of a call.)
    float lift, step;
    double inv;

    __device__ __forceinline__ Scale(float reference, float largest, float border, float heat)
        : ref(reference), top(largest), least(border), lift(heat < 0x1p-96f ? 0x1p64f : 1.f), step(kPerUnit / (heat * lift)),
          inv(1.0 / static_cast<double>(heat)) {}

    // x relative to a logit; entries of +inf, where there are any, are all that counts
    __device__ __forceinline__ double exponent(float z, float to) const {
        if (to == __builtin_inff()) return z == to ? 0.0 : -1e300;
        return (static_cast<double>(z) - static_cast<double>(to)) * inv;
    }
    __device__ __forceinline__ bool in(float z) const { return z >= least && z != -__builtin_inff(); }
    // where a logit lies in the histogram: below 0 where the reference was too low (its place then is the first bin).  (The
    // kernels have to agree on it, and on the border, so what the compiler may or may not fuse is written out.)
    __device__ __forceinline__ float place_of(float z) const {
        if (ref == __builtin_inff()) return z == ref ? 0.f : static_cast<float>(kBins - 1);
        return fminf(__builtin_fmaf((ref - z) * lift, step, kAbove * kPerUnit), static_cast<float>(kBins - 1));
    }
    __device__ __forceinline__ uint32_t bin_of(float z) const { return static_cast<uint32_t>(fmaxf(place_of(z), 0.f)); }
    // The upper edge of bin b above the row's largest logit, in units of the temperature (a single bin is all that +inf
    // leaves).
    __device__ __forceinline__ double edge_of(uint32_t b) const {
        if (ref == __builtin_inff()) return b == 0 ? 0.0 : -1e300;
        return static_cast<double>(kAbove) - b * (1.0 / kPerUnit) - exponent(top, ref);
    }
    // The masses of the four logits that are `kept`, others 0: side by side, with no branch around each (whose chains of
    // dependent operations would run one after the other), and none at all where the wave has none.
    __device__ __forceinline__ void masses(const float (&z)[4], const bool (&kept)[4], float to, double (&m)[4]) const {
#pragma unroll
        for (int j = 0; j < 4; ++j) m[j] = 0.0;
        if (!__any(kept[0] || kept[1] || kept[2] || kept[3])) return;
        double e[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) e[j] = exponential(exponent(z[j], to));
#pragma unroll
        for (int j = 0; j < 4; ++j) m[j] = kept[j] ? e[j] : 0.0;
    }
    // Adds four logits' masses to the histogram, relative to their bins' upper edges (within 1/16 of a unit), those that
    // are `kept`.  The last bin's entries are some e^-112 of the largest: nothing.
    template <typename F>
    __device__ __forceinline__ void add_masses(const float (&z)[4], double units, uint64_t *mass, F kept) const {
        uint64_t m[4];
        float place[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            place[j] = truncf(fmaxf(place_of(z[j]), 0.f));
            const float edge = kAbove - place[j] * (1.f / kPerUnit);  // exact
            const double x = ref == __builtin_inff() ? 0.0 : exponent(z[j], ref) - static_cast<double>(edge);
            m[j] = rounded(exponential_near_0(fmin(x, 0.02)), units);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (place[j] < static_cast<float>(kBins - 1) && kept(j))
                atomicAdd(reinterpret_cast<unsigned long long *>(&mass[static_cast<uint32_t>(place[j])]), static_cast<unsigned long long>(m[j]));
    }
};
// Units of the histogram's masses are 2^-unit, which leaves a row's sum below 2^63.
__device__ __forceinline__ int unit_of(uint32_t V) { return min(50, 62 - (32 - __clz(V))); }

// The largest of the threads' v, everywhere; a NaN if any of them has `odd`.
__device__ __forceinline__ float largest_of(float v, bool odd, uint32_t *wave32) {
    const float inf = __builtin_inff();
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor(v, o, 64));
    if (__any(odd)) v = __builtin_nanf("");
    __syncthreads();
    if ((threadIdx.x & 63) == 0) wave32[threadIdx.x >> 6] = __float_as_uint(v);
    __syncthreads();
    float most = -inf;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
        const float t = __uint_as_float(wave32[i]);
        bad = bad || t != t;
        most = fmaxf(most, t);
    }
    __syncthreads();
    return bad ? __builtin_nanf("") : most;
}
// The same of a row's segments.
__device__ __forceinline__ float joined_top(const Part *parts, uint32_t segments, uint32_t *wave32) {
    float top = -__builtin_inff();
    bool odd = false;
    for (uint32_t i = threadIdx.x; i < segments; i += kThreads) {
        top = fmaxf(top, parts[i].top);
        odd = odd || parts[i].odd;
    }
    return largest_of(top, odd, wave32);
}

// Where a cut by count falls: the bin of the last entry that is kept, entries up to that bin and before it, by the threads'
// counts of bins 2 tid and 2 tid + 1; at most `want` of them are kept.  found32 has three entries.
struct CountCut {
    uint32_t keep, entries, limit, upto, earlier;
};
__device__ __forceinline__ CountCut count_cut(uint32_t c0, uint32_t c1, uint32_t want, uint32_t *wave32, uint32_t *found32) {
    const uint32_t tid = threadIdx.x;
    CountCut c;
    const uint32_t before = sum_before(c0 + c1, wave32, c.entries);
    c.keep = min(want, c.entries);
    if (before < c.keep && c.keep <= before + c0 + c1) {  // one thread
        const bool second = c.keep > before + c0;
        found32[0] = 2 * tid + second;
        found32[1] = before + c0 + (second ? c1 : 0);
        found32[2] = second ? before + c0 : before;
    }
    __syncthreads();
    c.limit = found32[0];
    c.upto = found32[1];
    c.earlier = found32[2];
    __syncthreads();
    return c;
}
// Of the histogram's masses (before bin 2 tid: `mb`, its own and the next one's m0 and m1): the bin that the target
// falls into, and what stands before it; kBins where rounding leaves nothing past it.
__device__ __forceinline__ uint32_t mass_bin(double mb, double m0, double m1, double want, uint32_t *found32, double *found, double &earlier) {
    const uint32_t tid = threadIdx.x;
    __syncthreads();
    if (tid == 0) found32[1] = kBins;
    __syncthreads();
    // (sums of a double's precision: the one in front may seem to reach the target as well)
    const uint32_t mine = m0 > 0.0 && mb + m0 >= want ? 2 * tid : m1 > 0.0 && mb + m0 + m1 >= want ? 2 * tid + 1 : kBins;
    if (mine < kBins) atomicMin(&found32[1], mine);
    __syncthreads();
    const uint32_t b = found32[1];
    if (b < kBins && tid == b / 2) *found = b & 1 ? mb + m0 : mb;
    __syncthreads();
    earlier = *found;
    __syncthreads();
    return b;
}
__device__ __forceinline__ bool short_cut(const CountCut &c) { return c.upto <= kList && c.upto - c.earlier <= kRanked; }

// ---------------------------------------------------------------------- no filter
// Segments of 1024 entries by a wave each, all over the chip: a segment's largest logit, and its masses relative to that.
// Then a workgroup for each row joins them, finds the segment that the target falls into, and draws from it.
constexpr int kPartWaves = 4;

// x relative to a logit; entries of +inf, where there are any, are all that counts, and one of -inf never does
__device__ __forceinline__ double relative(float z, float to, double inv) {
    if (to == __builtin_inff()) return z == to ? 0.0 : -1e300;
    return z == -__builtin_inff() ? -1e300 : (static_cast<double>(z) - static_cast<double>(to)) * inv;
}

// SUMS false: the largest alone, and a row's bins and list are cleared.
template <typename T, bool SUMS>
__global__ __launch_bounds__(64 * kPartWaves) void k_sample_parts(const SampleArgs a, uint32_t all) {
    const uint32_t segments = a.segments;
    const uint32_t lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t n = blockIdx.x * kPartWaves + wave;
    if (n >= all) return;
    const uint32_t row = n / segments, s = n - row * segments;
    const Row<T> r(a.logits, a.ld, row, a.V);
    const float heat = a.p.temperatures ? a.p.temperatures[row] : a.p.temperature;
    const double inv = 1.0 / static_cast<double>(heat);
    float z[kSteps][4];
    float top = -__builtin_inff();
    bool odd = false;
#pragma unroll
    for (uint32_t i = 0; i < kSteps; ++i) {
        r.load((s * kSteps + i) * 64 + lane, z[i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            odd = odd || z[i][j] != z[i][j];
            top = fmaxf(top, z[i][j]);
        }
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
    odd = __any(odd);
    double sum = 0.0;
    if (!SUMS) {
        for (uint32_t i = s * 64 + lane; i < kBins; i += segments * 64) a.bins[static_cast<uint64_t>(row) * kBins + i] = 0;
        if (s == 0 && lane == 0) a.state[row] = RowState{0, kBins, 0.0};
    } else if (heat > 0.f && top > -__builtin_inff()) {
#pragma unroll
        for (uint32_t i = 0; i < kSteps; ++i) {
            double m[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) m[j] = exponential(relative(z[i][j], top, inv));
            sum += (m[0] + m[1]) + (m[2] + m[3]);
        }
    }
    if (SUMS) sum = wave_total(sum);
    if (lane == 0) a.parts[n] = Part{sum, top, odd ? 1u : 0u};
}

template <typename T>
__global__ __launch_bounds__(64 * kPartWaves) void k_sample_join(const SampleArgs a) {
    const uint32_t segments = a.segments;
    __shared__ float tops[kPartWaves];
    __shared__ double sums[kPartWaves], first;
    __shared__ uint32_t found32[2];
    const uint32_t row = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const Row<T> r(a.logits, a.ld, row, a.V);
    const float inf = __builtin_inff();
    const float heat = a.p.temperatures ? a.p.temperatures[row] : a.p.temperature;
    const float u = a.uniform[row];
    const double inv = 1.0 / static_cast<double>(heat);
    const Part *parts = a.parts + static_cast<uint64_t>(row) * segments;
    const uint32_t run = (segments + 64 * kPartWaves - 1) / (64 * kPartWaves);
    // the row's largest
    float top = -inf;
    bool odd = heat != heat;
    for (uint32_t i = tid * run; i < min(segments, (tid + 1) * run); ++i) {
        top = fmaxf(top, parts[i].top);
        odd = odd || parts[i].odd;
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
    if (__any(odd)) top = __builtin_nanf("");
    if (lane == 0) tops[wave] = top;
    if (tid == 0) found32[0] = ~0u;
    __syncthreads();
    top = -inf;
    odd = false;
#pragma unroll
    for (int i = 0; i < kPartWaves; ++i) {
        odd = odd || tops[i] != tops[i];
        top = fmaxf(top, tops[i]);
    }
    if (odd || top == -inf) {
        if (tid == 0) {
            a.token[row] = -1;
            if (a.logprob) a.logprob[row] = __builtin_nanf("");
        }
        return;
    }
    if (heat <= 0.f) {  // the first of the largest
        for (uint32_t i = tid * run; i < min(segments, (tid + 1) * run); ++i)
            if (parts[i].top == top) {
                atomicMin(&found32[0], i);
                break;
            }
        __syncthreads();
        if (wave != 0) return;
        float drawn;
        const int64_t token = first_of(r, found32[0], top, drawn);
        if (lane == 0) {
            a.token[row] = token;
            if (a.logprob) a.logprob[row] = 0.f;
        }
        return;
    }
    auto value = [&](uint32_t i) __attribute__((always_inline)) {
        const Part p = parts[i];
        return p.sum * exponential(relative(p.top, top, inv));
    };
    double mine = 0.0, total;
    for (uint32_t i = tid * run; i < min(segments, (tid + 1) * run); ++i) mine += value(i);
    const double before = sum_before<kPartWaves>(mine, sums, total);
    const double target = share_of(u) * total;
    const uint32_t s = find_segment(value, segments, run, before, target, found32, &first);
    if (wave != 0) return;
    float drawn;
    const int64_t token = draw_from(r, s, first, target, [&](const float (&z)[4], int32_t, double (&m)[4]) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < 4; ++j) m[j] = exponential(relative(z[j], top, inv));
    }, drawn);
    if (lane == 0) {
        a.token[row] = token;
        if (a.logprob) a.logprob[row] = static_cast<float>(relative(drawn, top, inv) - log(total));
    }
}

// ---------------------------------------------------------------------- filters, divided
// What k_sample does with passes over a row, by workgroups that share its segments: the largest logit (k_sample_parts),
// then the histogram (k_sample_bins; its counts for a row with top_k, else its masses), then what the cut's bin asks for
// (k_sample_collect: with top_k a list of the entries up to the bin, else one of the bin's own, and the masses of each
// segment before it).  k_sample goes on from there.  Atomic additions are of integers, and a list's order does not matter.
struct BinsShared {
    uint64_t bins[kBins];
    uint64_t list[kList];
    uint32_t wave32[kWaves], found32[3], listed, at;
    double wavef[kWaves];
};

// Whether there is anything to be done for a row whose largest logit is `top`.
__device__ __forceinline__ bool drawn_by_mass(float heat, float top) { return heat > 0.f && top > -__builtin_inff(); }

template <typename T, typename F>
__device__ __forceinline__ void over_segment(const Row<T> &r, uint32_t s, F f) {
    const uint32_t lane = threadIdx.x & 63;
    typename Row<T>::Raw v[kSteps];
#pragma unroll
    for (uint32_t i = 0; i < kSteps; ++i) v[i] = r.raw((s * kSteps + i) * 64 + lane);
#pragma unroll 1
    for (uint32_t i = 0; i < kSteps; ++i) {
        float z[4];
        const int32_t at = r.values((s * kSteps + i) * 64 + lane, v[0], z);
#pragma unroll
        for (uint32_t j = 0; j + 1 < kSteps; ++j) v[j] = v[j + 1];
        f(at, z);
    }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void k_sample_bins(const SampleArgs a) {
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    BinsShared &sh = *reinterpret_cast<BinsShared *>(smem);
    const uint32_t row = blockIdx.y, tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const Settings st(a, row);
    if (!st.by_count && !st.by_mass) return;
    const float top = joined_top(a.parts + static_cast<uint64_t>(row) * a.segments, a.segments, sh.wave32);
    if (!drawn_by_mass(st.heat, top)) return;
    const Row<T> r(a.logits, a.ld, row, a.V);
    const Scale sc(top, top, st.border(top), st.heat);
    for (uint32_t i = tid; i < kBins; i += kThreads) sh.bins[i] = 0;
    __syncthreads();
    const double units = ldexp(0.5, unit_of(a.V));
    for (uint32_t s = blockIdx.x * kWaves + wave; s < a.segments; s += gridDim.x * kWaves)
        over_segment(r, s, [&](int32_t, const float (&z)[4]) __attribute__((always_inline)) {
            if (st.by_count) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (sc.in(z[j])) atomicAdd(reinterpret_cast<unsigned long long *>(&sh.bins[sc.bin_of(z[j])]), 1ull);
            } else {
                sc.add_masses(z, units, sh.bins, [&](int j) { return sc.in(z[j]); });
            }
        });
    __syncthreads();
    for (uint32_t i = tid; i < kBins; i += kThreads)
        if (sh.bins[i]) atomicAdd(reinterpret_cast<unsigned long long *>(&a.bins[static_cast<uint64_t>(row) * kBins + i]), static_cast<unsigned long long>(sh.bins[i]));
}

template <typename T>
__global__ __launch_bounds__(kThreads) void k_sample_collect(const SampleArgs a) {
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    BinsShared &sh = *reinterpret_cast<BinsShared *>(smem);
    const uint32_t row = blockIdx.y, tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const Settings st(a, row);
    const float top = joined_top(a.parts + static_cast<uint64_t>(row) * a.segments, a.segments, sh.wave32);
    if (!drawn_by_mass(st.heat, top)) return;
    const Row<T> r(a.logits, a.ld, row, a.V);
    const Scale sc(top, top, st.border(top), st.heat);
    const uint64_t *bins = a.bins + static_cast<uint64_t>(row) * kBins;
    RowState &state = a.state[row];
    uint32_t from = 0, upto = 0;  // bins [from, upto) are listed,
    uint32_t added = 0;           // and [0, added) added up
    if (st.by_count) {
        const CountCut c = count_cut(static_cast<uint32_t>(bins[2 * tid]), static_cast<uint32_t>(bins[2 * tid + 1]), st.top_k, sh.wave32, sh.found32);
        if (!short_cut(c)) return;
        upto = c.limit + 1;
    } else if (st.by_mass) {
        double m[2];
#pragma unroll
        for (uint32_t j = 0; j < 2; ++j) m[j] = static_cast<double>(bins[2 * tid + j]) * ldexp(2.0, -unit_of(a.V)) * exponential(sc.edge_of(2 * tid + j));
        double whole, earlier;
        const double before = sum_before(m[0] + m[1], sh.wavef, whole), want = fmax(static_cast<double>(st.top_p), 0.0) * whole;
        const uint32_t b = mass_bin(before, m[0], m[1], want, sh.found32, sh.wavef, earlier);
        from = b;
        upto = b < kBins ? b + 1 : b;
        added = b;
        if (blockIdx.x == 0 && tid == 0) {
            state.bin = b;
            state.most = want - earlier;
        }
    } else {
        from = upto = added = kBins;
    }
    if (tid == 0) sh.listed = 0;
    __syncthreads();
    for (uint32_t s = blockIdx.x * kWaves + wave; s < a.segments; s += gridDim.x * kWaves) {
        double m = 0.0;
        over_segment(r, s, [&](int32_t at, const float (&z)[4]) __attribute__((always_inline)) {
            bool kept[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t x = sc.bin_of(z[j]);
                kept[j] = sc.in(z[j]) && x < added;
                if (sc.in(z[j]) && x >= from && x < upto) {
                    const uint32_t i = atomicAdd(&sh.listed, 1u);
                    if (i < kList) sh.list[i] = place_key(z[j], at + j);
                }
            }
            if (!st.by_count) {
                double e[4];
                sc.masses(z, kept, top, e);
                m += (e[0] + e[1]) + (e[2] + e[3]);
            }
        });
        if (!st.by_count) {
            m = wave_total(m);
            if (lane == 0)
                a.sums[static_cast<uint64_t>(row) * a.segments + s] = st.by_mass ? static_cast<uint64_t>(m * kFine) : __builtin_bit_cast(uint64_t, m);
        }
    }
    __syncthreads();
    const uint32_t n = sh.listed;
    if (n == 0) return;
    if (tid == 0) sh.at = atomicAdd(&state.listed, n);
    __syncthreads();
    for (uint32_t i = tid; i < min(n, kList); i += kThreads)
        if (sh.at + i < kList) a.list[static_cast<uint64_t>(row) * kList + sh.at + i] = sh.list[i];
}

// ---------------------------------------------------------------------- filters

// `divided`: the kernels above have been over the row.
template <typename T, bool divided>
__global__ __launch_bounds__(kThreads) void k_sample(const SampleArgs a) {
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    Shared &sh = *reinterpret_cast<Shared *>(smem);
    const uint32_t row = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const Row<T> r(a.logits, a.ld, row, a.V);
    const uint32_t V = a.V;
    const float inf = __builtin_inff();

    auto largest = [&](float v, bool odd) __attribute__((always_inline)) { return largest_of(v, odd, sh.wave32); };
    auto row_largest = [&]() __attribute__((always_inline)) {
        float top = -inf;
        bool odd = false;
        over_row(r, [&](int32_t, const float (&z)[4], uint32_t, bool) __attribute__((always_inline)) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                odd = odd || z[j] != z[j];
                top = fmaxf(top, z[j]);
            }
        });
        return largest(top, odd);
    };
    auto nothing = [&]() __attribute__((always_inline)) {  // the row has no token
        if (tid == 0) {
            a.token[row] = -1;
            if (a.logprob) a.logprob[row] = __builtin_nanf("");
        }
    };

    const Settings st(a, row);
    const float heat = st.heat, min_p = st.min_p;
    const int32_t top_k = st.top_k;
    const bool by_count = st.by_count, by_mass = st.by_mass;
    const float u = a.uniform[row];
    const double share = share_of(u);
    // the first or the last kept entry is drawn, however little it weighs: fixed-point sums would not show it
    const bool at_end = !(share > 0.0 && share < static_cast<double>(inf));
    if (heat != heat) return nothing();
    const Part *parts = a.parts + (divided ? static_cast<uint64_t>(row) * a.segments : 0);
    float row_top = -inf;
    if (divided) {
        row_top = joined_top(parts, a.segments, sh.wave32);
        if (row_top != row_top || row_top == -inf) return nothing();
    }
    if (heat <= 0.f && divided) {  // the first of the largest
        if (tid == 0) sh.found32[0] = ~0u;
        __syncthreads();
        for (uint32_t i = tid; i < a.segments; i += kThreads)
            if (parts[i].top == row_top) atomicMin(&sh.found32[0], i);
        __syncthreads();
        if (wave != 0) return;
        float drawn;
        const int64_t token = first_of(r, sh.found32[0], row_top, drawn);
        if (lane == 0) {
            a.token[row] = token;
            if (a.logprob) a.logprob[row] = 0.f;
        }
        return;
    }
    if (heat <= 0.f) {  // the least key
        uint64_t first = ~uint64_t(0);
        bool odd = false;
        over_row(r, [&](int32_t at, const float (&z)[4], uint32_t segment, bool last) __attribute__((always_inline)) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                odd = odd || z[j] != z[j];
                if (z[j] != -inf) first = min(first, place_key(z[j], at + j));
            }
        });
        if (tid == 0) sh.found64[0] = ~uint64_t(0);
        const float bad = largest(0.f, odd);
        atomicMin(reinterpret_cast<unsigned long long *>(&sh.found64[0]), static_cast<unsigned long long>(first));
        __syncthreads();
        first = sh.found64[0];
        if (bad != bad || first == ~uint64_t(0)) return nothing();
        if (tid == 0) {
            a.token[row] = static_cast<uint32_t>(first);
            if (a.logprob) a.logprob[row] = 0.f;
        }
        return;
    }

    const bool short_list = by_count && static_cast<uint32_t>(top_k) <= kList * 3 / 4;
    const double part = fmax(static_cast<double>(st.top_p), 0.0);

    // ---- the reference: the largest of the first entries, or, where it has to be known, of all
    Scale sc(-inf, -inf, -inf, heat);
    float &ref = sc.ref, &top = sc.top, &least = sc.least;
    bool known = divided;
    if (divided) {
        top = ref = row_top;
    } else if (!(min_p > 0.f && !short_list)) {
        float z[4];
        bool odd = false;
        r.load(tid, z);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            odd = odd || z[j] != z[j];
            ref = fmaxf(ref, z[j]);
        }
        ref = largest(ref, odd);
        if (ref != ref) return nothing();
    }
    if (!divided && !(fabsf(ref) < inf)) {
        top = ref = row_largest();
        known = true;
        if (top != top || top == -inf) return nothing();
    }
    auto border = [&]() __attribute__((always_inline)) { least = st.border(top); };
    if (known) border();

    auto exponent = [&](float z, float to) __attribute__((always_inline)) { return sc.exponent(z, to); };
    auto mass_of = [&](float z, float to) __attribute__((always_inline)) { return exponential(sc.exponent(z, to)); };  // 0 of -inf
    auto place_of = [&](float z) __attribute__((always_inline)) { return sc.place_of(z); };
    auto bin_of = [&](float z) __attribute__((always_inline)) { return sc.bin_of(z); };
    auto in = [&](float z) __attribute__((always_inline)) { return sc.in(z); };
    // Fixed point.  The sums of a segment's 1024 masses, and of a list's 2048, relative to the row's largest: in units of
    // 2^-50.  Sums over a bin, which all of the row may lie in: of masses relative to the bin's edge, in units of 2^-unit,
    // which leaves them below 2^63.
    const double scale = ldexp(1.0, unit_of(V)), fine = kFine;
    auto fixed = [&](float z, double by) __attribute__((always_inline)) { return rounded(mass_of(z, top), by); };
    auto key_logit = [&](uint64_t key) __attribute__((always_inline)) { return from_ascending(~static_cast<uint32_t>(key >> 32)); };
    auto add64 = [&](uint64_t *to, uint64_t v) __attribute__((always_inline)) {
        atomicAdd(reinterpret_cast<unsigned long long *>(to), static_cast<unsigned long long>(v));
    };

    uint64_t cut = ~uint64_t(0);  // the last key that is kept

    // Cuts among the n <= kRanked keys in sh.ranked: the `some` first of them, or those before which less than `most` of
    // mass in units of 1 / by stands; at least one.  The last one's key in `cut`.  All threads.
    auto cut_ranked = [&](uint32_t n, uint32_t some, uint64_t most, double by) __attribute__((always_inline)) {
        if (tid == 0) sh.found64[0] = 0;
        uint64_t own = 0, m = 0;
        if (tid < n) {
            own = sh.ranked[tid];
            m = by_mass ? fixed(key_logit(own), by) : 0;
        }
        __syncthreads();
        if (tid < n) sh.mass[tid] = m;
        __syncthreads();
        if (tid < n) {
            uint32_t rank = 0;
            uint64_t before = 0;
            for (uint32_t i = 0; i < n; ++i) {
                const bool less = sh.ranked[i] < own;
                rank += less;
                before += less ? sh.mass[i] : 0;
            }
            if (rank == 0 || (rank < some && before < most))
                atomicMax(reinterpret_cast<unsigned long long *>(&sh.found64[0]), static_cast<unsigned long long>(own));
        }
        __syncthreads();
        cut = min(cut, sh.found64[0]);
        __syncthreads();
    };
    // The part of bin b that the cut falls into, of 2048, by the counts and masses of its parts in sh.count and sh.mass;
    // takes what stands before it off `some` and `most`.
    auto pick_part = [&](uint32_t &some, uint64_t &most) __attribute__((always_inline)) {
        const uint32_t c0 = sh.count[2 * tid], c1 = sh.count[2 * tid + 1];
        const uint64_t m0 = sh.mass[2 * tid], m1 = sh.mass[2 * tid + 1];
        uint32_t count_all;
        uint64_t mass_all;
        const uint32_t cb = sum_before(c0 + c1, sh.wave32, count_all);
        const uint64_t mb = sum_before(m0 + m1, sh.wave64, mass_all);
        if (tid == 0) sh.found32[0] = 0;
        __syncthreads();
        // the last part whose first entry is kept
        const bool k0 = c0 > 0 && (cb == 0 || (cb < some && mb < most));
        const bool k1 = c1 > 0 && (cb + c0 == 0 || (cb + c0 < some && mb + m0 < most));
        if (k0 || k1) atomicMax(&sh.found32[0], 2 * tid + (k1 ? 1 : 0));
        __syncthreads();
        const uint32_t x = sh.found32[0];
        if (tid == x / 2) {
            sh.found32[1] = x & 1 ? cb + c0 : cb;
            sh.found64[0] = x & 1 ? mb + m0 : mb;
        }
        __syncthreads();
        some -= min(some, sh.found32[1]);
        most -= min(most, sh.found64[0]);
        __syncthreads();
        return x;
    };
    auto part_of = [&](float z, uint32_t b) __attribute__((always_inline)) {
        return static_cast<uint32_t>(fminf(fmaxf((place_of(z) - static_cast<float>(b)) * kBins, 0.f), static_cast<float>(kBins - 1)));
    };
    auto no_parts = [&]() __attribute__((always_inline)) {
        for (uint32_t i = tid; i < kBins; i += kThreads) {
            sh.count[i] = 0;
            sh.mass[i] = 0;
        }
        if (tid == 0) sh.found32[2] = 0;
        __syncthreads();
    };
    auto into_part = [&](float z, uint32_t b, double by) __attribute__((always_inline)) {
        const uint32_t x = part_of(z, b);
        atomicAdd(&sh.count[x], 1u);
        if (by_mass) add64(&sh.mass[x], fixed(z, by));
    };
    auto rank_if = [&](bool yes, uint64_t key) __attribute__((always_inline)) {
        if (yes) {
            const uint32_t i = atomicAdd(&sh.found32[2], 1u);
            if (i < kRanked) sh.ranked[i] = key;
        }
    };
    // The same among the entries of bin b, `most` relative to the row's largest; `segments`: adds up what is kept by segments too, with the entries of the bins
    // before it; false where it did not.  Up to kList entries are divided up in LDS, more by passes over the row; where even
    // a part of the bin holds more than kRanked (equal logits), the cut's key is found by its bits.
    auto cut_bin = [&](uint32_t b, uint32_t some, double most_mass, bool segments, bool collected) __attribute__((always_inline)) {
        // a power of two by which all of the bin's masses are small enough
        // (the first bin has no edge that all are below)
        const int lift = b == 0 ? 0 : static_cast<int>(fmin(fmax(floor(sc.edge_of(b) * -1.4426950408889634), 0.0), 900.0));
        const double by = ldexp(scale, lift);
        uint64_t most = most_mass < inf ? max(uint64_t(1), static_cast<uint64_t>(ceil(fmin(most_mass * by, 9e18)))) : ~uint64_t(0);
        __syncthreads();
        if (tid == 0) sh.found32[2] = collected ? a.state[row].listed : 0;
        __syncthreads();
        if (collected) {
            const uint64_t *list = a.list + static_cast<uint64_t>(row) * kList, *sums = a.sums + static_cast<uint64_t>(row) * a.segments;
            if (sh.found32[2] <= kList)
                for (uint32_t i = tid; i < sh.found32[2]; i += kThreads) sh.list[i] = list[i];
            for (uint32_t i = tid; i < a.segments; i += kThreads) sh.fixed_segment[i] = sums[i];
        }
        double m = 0.0;
        if (!collected) over_row(r, [&](int32_t at, const float (&z)[4], uint32_t segment, bool last) __attribute__((always_inline)) {
            bool kept[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t x = bin_of(z[j]);
                kept[j] = in(z[j]) && x < b;
                if (in(z[j]) && x == b) {
                    const uint32_t i = atomicAdd(&sh.found32[2], 1u);
                    if (i < kList) sh.list[i] = place_key(z[j], at + j);
                }
            }
            if (segments) {
                double e[4];
                sc.masses(z, kept, top, e);
                m += (e[0] + e[1]) + (e[2] + e[3]);
            }
            if (segments && last) {
                m = wave_total(m);
                if (lane == 0) sh.fixed_segment[segment] = static_cast<uint64_t>(m * fine);
                m = 0.0;
            }
        });
        __syncthreads();
        const uint32_t n = sh.found32[2];
        __syncthreads();
        no_parts();
        uint64_t key[2];
#pragma unroll
        for (uint32_t j = 0; j < 2; ++j) key[j] = n <= kList && 2 * tid + j < n ? sh.list[2 * tid + j] : ~uint64_t(0);
        if (n <= kList) {
#pragma unroll
            for (uint32_t j = 0; j < 2; ++j)
                if (key[j] != ~uint64_t(0)) into_part(key_logit(key[j]), b, by);
        } else {
            over_row(r, [&](int32_t, const float (&z)[4], uint32_t, bool) __attribute__((always_inline)) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (in(z[j]) && bin_of(z[j]) == b) into_part(z[j], b, by);
            });
        }
        __syncthreads();
        const uint32_t x = pick_part(some, most);
        if (n <= kList) {
#pragma unroll
            for (uint32_t j = 0; j < 2; ++j) rank_if(key[j] != ~uint64_t(0) && part_of(key_logit(key[j]), b) == x, key[j]);
        } else {
            over_row(r, [&](int32_t at, const float (&z)[4], uint32_t, bool) __attribute__((always_inline)) {
#pragma unroll
                for (int j = 0; j < 4; ++j) rank_if(in(z[j]) && bin_of(z[j]) == b && part_of(z[j], b) == x, place_key(z[j], at + j));
            });
        }
        __syncthreads();
        const uint32_t ranked = sh.found32[2];
        if (ranked <= kRanked) {
            cut_ranked(ranked, some, most, by);
            if (segments && n <= kList) {
#pragma unroll
                for (uint32_t j = 0; j < 2; ++j)
                    if (key[j] <= cut && key[j] != ~uint64_t(0))
                        add64(&sh.fixed_segment[(static_cast<uint32_t>(key[j]) + r.skew) / (256 * kSteps)], fixed(key_logit(key[j]), fine));
                __syncthreads();
                return true;
            }
            return false;
        }
        // The largest key before which there is room for one more in the part, bit by bit: 64 passes.
        uint64_t found = 0;
        for (int bit = 63; bit >= 0; --bit) {
            const uint64_t probe = found | (uint64_t(1) << bit);
            uint32_t c = 0;
            uint64_t own = 0;
            over_row(r, [&](int32_t at, const float (&z)[4], uint32_t, bool) __attribute__((always_inline)) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (in(z[j]) && bin_of(z[j]) == b && part_of(z[j], b) == x && place_key(z[j], at + j) < probe) {
                        ++c;
                        if (by_mass) own += fixed(z[j], by);
                    }
            });
            uint32_t count_all;
            uint64_t mass_all;
            sum_before(c, sh.wave32, count_all);
            sum_before(own, sh.wave64, mass_all);
            if (count_all == 0 || (count_all < some && mass_all < most)) found = probe;
        }
        cut = min(cut, found);
        return false;
    };
    const uint32_t segments = (r.groups + 64 * kSteps - 1) / (64 * kSteps);
    bool have = false;  // the segments' sums are there, in fixed point
    if (by_count) {
        // ---- counts, and the row's largest
        auto counts = [&](float &most, bool &odd) __attribute__((always_inline)) {
            for (uint32_t i = tid; i < kBins; i += kThreads) sh.count[i] = 0;
            __syncthreads();
            over_row(r, [&](int32_t, const float (&z)[4], uint32_t, bool) __attribute__((always_inline)) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    odd = odd || z[j] != z[j];
                    most = fmaxf(most, z[j]);
                    if (in(z[j])) atomicAdd(&sh.count[bin_of(z[j])], 1u);
                }
            });
            __syncthreads();
        };
        float most = -inf;
        bool odd = false;
        if (divided) {
            for (uint32_t i = tid; i < kBins; i += kThreads) sh.count[i] = static_cast<uint32_t>(a.bins[static_cast<uint64_t>(row) * kBins + i]);
            __syncthreads();
        } else {
            counts(most, odd);
            top = largest(most, odd);
            if (top != top || top == -inf) return nothing();
        }
        CountCut c = count_cut(sh.count[2 * tid], sh.count[2 * tid + 1], top_k, sh.wave32, sh.found32);
        if (!divided && (top == inf ? ref != inf : place_of(top) < 0.f && !short_cut(c))) {
            // The reference was too low: +inf alone counts, or, as where the first entries are masked by a finite number, the
            // cut is in the first bin with all that is above it, or among what is masked (with which each bit of its key took
            // a pass: 66 rows of 70000, 20 allowed and top_k = 50, took 1297 us, 154 so, and 46 where nothing is masked).
            ref = top;
            counts(most, odd);
            c = count_cut(sh.count[2 * tid], sh.count[2 * tid + 1], top_k, sh.wave32, sh.found32);
        }
        const uint32_t keep = c.keep, entries = c.entries, limit = c.limit, upto = c.upto, earlier = c.earlier;
        if (short_cut(c)) {
            // ---- the list: entries up to the cut's bin, those of the bin ranked; then the other filters on it
            if (tid < 2) sh.found32[tid] = 0;
            __syncthreads();
            if (divided)
                for (uint32_t i = tid; i < min(upto, a.state[row].listed); i += kThreads) {
                    const uint64_t key = a.list[static_cast<uint64_t>(row) * kList + i];
                    sh.list[i] = key;
                    if (bin_of(key_logit(key)) == limit) sh.ranked[atomicAdd(&sh.found32[1], 1u)] = key;
                }
            else over_row(r, [&](int32_t at, const float (&z)[4], uint32_t segment, bool last) __attribute__((always_inline)) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (in(z[j]) && bin_of(z[j]) <= limit) {
                        const uint64_t key = place_key(z[j], at + j);
                        sh.list[atomicAdd(&sh.found32[0], 1u)] = key;
                        if (bin_of(z[j]) == limit) sh.ranked[atomicAdd(&sh.found32[1], 1u)] = key;
                    }
            });
            __syncthreads();
            if (keep < entries) cut_ranked(upto - earlier, keep - earlier, ~uint64_t(0), fine);
            border();
            uint64_t key[2], m[2];
#pragma unroll
            for (uint32_t j = 0; j < 2; ++j) {
                key[j] = 2 * tid + j < upto ? sh.list[2 * tid + j] : ~uint64_t(0);
                m[j] = 0;
                if (key[j] <= cut && key[j] != ~uint64_t(0) && key_logit(key[j]) >= least) m[j] = fixed(key_logit(key[j]), fine);
            }
            if (by_mass) {
                for (uint32_t i = tid; i < kBins; i += kThreads) sh.mass[i] = 0;
                if (tid == 0) sh.found32[0] = 0;
                __syncthreads();
#pragma unroll
                for (uint32_t j = 0; j < 2; ++j)
                    if (m[j]) add64(&sh.mass[bin_of(key_logit(key[j]))], m[j]);
                __syncthreads();
                // (a double holds 2^53 of these units)
                const double m0 = static_cast<double>(sh.mass[2 * tid]), m1 = static_cast<double>(sh.mass[2 * tid + 1]);
                double whole, earlier_mass;
                const double mb = sum_before(m0 + m1, sh.wavef, whole), want_mass = part * whole;
                const uint32_t b = mass_bin(mb, m0, m1, want_mass, sh.found32, sh.wavef, earlier_mass);
                if (b < kBins) {
#pragma unroll
                    for (uint32_t j = 0; j < 2; ++j)
                        if (m[j] && bin_of(key_logit(key[j])) == b) {
                            const uint32_t i = atomicAdd(&sh.found32[0], 1u);
                            if (i < kRanked) sh.ranked[i] = key[j];
                        }
                    __syncthreads();
                    const uint32_t n = sh.found32[0];
                    if (n <= kRanked) {
                        cut_ranked(n, ~0u, max(uint64_t(1), static_cast<uint64_t>(ceil(want_mass - earlier_mass))), fine);
                    } else {
                        have = cut_bin(b, ~0u, (want_mass - earlier_mass) / fine, false, false);
                    }
                }
            }
            if (!have) {
                for (uint32_t i = tid; i < segments; i += kThreads) sh.fixed_segment[i] = 0;
                __syncthreads();
#pragma unroll
                for (uint32_t j = 0; j < 2; ++j)
                    if (m[j] && key[j] <= cut) add64(&sh.fixed_segment[(static_cast<uint32_t>(key[j]) + r.skew) / (256 * kSteps)], m[j]);
                __syncthreads();
                have = true;
            }
        } else {
            border();  // (after the cut by count, which does not know of it, unless it was known before)
            const float floor = least;
            if (!known) least = -inf;
            // What is left out of the last bin weighs nothing, and shows at the ends alone, unless its masses are 0, as of what is
            // masked by a large number (a cut among whose equal keys takes a pass for each bit: 66 rows of 70000, 30 allowed and
            // top_k = 50, 1346 us at the ends, 134 without it).
            auto shows = [&]() __attribute__((always_inline)) {
                bool any = false;
                over_row(r, [&](int32_t, const float (&z)[4], uint32_t, bool) __attribute__((always_inline)) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) any = any || (in(z[j]) && bin_of(z[j]) == kBins - 1 && mass_of(z[j], top) > 0.0);
                });
                return largest(any ? 1.f : 0.f, false) > 0.f;
            };
            if (keep < entries && (limit < kBins - 1 || (at_end && shows()))) cut_bin(limit, keep - earlier, static_cast<double>(inf), false, false);
            least = floor;
        }
        known = true;
    }
    if (!have && by_mass) {
        // ---- the bins' masses
        uint32_t b;
        double most_mass = 0.0;
        const bool collected = divided && !by_count;
        if (collected) {
            b = a.state[row].bin;
            most_mass = a.state[row].most;
        } else {
            for (;;) {
                for (uint32_t i = tid; i < kBins; i += kThreads) sh.mass[i] = 0;
                __syncthreads();
                float most = -inf;
                bool odd = false;
                over_row(r, [&](int32_t at, const float (&z)[4], uint32_t segment, bool last) __attribute__((always_inline)) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        odd = odd || z[j] != z[j];
                        most = fmaxf(most, z[j]);
                    }
                    sc.add_masses(z, scale * 0.5, sh.mass, [&](int j) __attribute__((always_inline)) {
                        return in(z[j]) && (cut == ~uint64_t(0) || place_key(z[j], at + j) <= cut);
                    });
                });
                top = largest(most, odd);
                if (top != top || top == -inf) return nothing();
                if (place_of(top) >= 0.f && (top < inf || ref == inf)) break;
                ref = top;  // it was too low
            }
            if (!known) border();
            known = true;
            double mine[2];  // relative to the row's largest
#pragma unroll
            for (uint32_t j = 0; j < 2; ++j) mine[j] = static_cast<double>(sh.mass[2 * tid + j]) * (2.0 / scale) * exponential(sc.edge_of(2 * tid + j));
            double whole, earlier;
            const double before = sum_before(mine[0] + mine[1], sh.wavef, whole), want = part * whole;
            b = mass_bin(before, mine[0], mine[1], want, sh.found32, sh.wavef, earlier);
            most_mass = want - earlier;
        }
        if (b < kBins) have = cut_bin(b, ~0u, most_mass, cut == ~uint64_t(0), collected);
    }
    float base = known ? top : ref;  // what masses are relative to from here on
    auto kept_masses = [&](const float (&z)[4], int32_t at, double (&m)[4]) __attribute__((always_inline)) {
        bool kept[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) kept[j] = in(z[j]) && (cut == ~uint64_t(0) || place_key(z[j], static_cast<uint32_t>(at + j)) <= cut);
        sc.masses(z, kept, base, m);
    };
    __syncthreads();
    if (have && !at_end) {
        for (uint32_t i = tid; i < segments; i += kThreads) sh.segment[i] = static_cast<double>(sh.fixed_segment[i]) * (1.0 / fine);
    } else if (divided && !by_count && !by_mass) {
        for (uint32_t i = tid; i < segments; i += kThreads) sh.segment[i] = __builtin_bit_cast(double, a.sums[static_cast<uint64_t>(row) * a.segments + i]);
    } else {
        for (;;) {
            float most = -inf;
            bool odd = false;
            double m = 0.0;
            over_row(r, [&](int32_t at, const float (&z)[4], uint32_t segment, bool last) __attribute__((always_inline)) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    odd = odd || z[j] != z[j];
                    most = fmaxf(most, z[j]);
                }
                double e[4];
                kept_masses(z, at, e);
                m += (e[0] + e[1]) + (e[2] + e[3]);
                if (last) {
                    m = wave_total(m);
                    if (lane == 0) sh.segment[segment] = m;
                    m = 0.0;
                }
            });
            if (known) break;
            top = largest(most, odd);
            if (top != top || top == -inf) return nothing();
            // (exponentials of what is 600 above the reference would not do)
            if (base == inf || (top < inf && exponent(top, base) < 600.0)) break;
            base = top;
            known = true;
        }
    }
    __syncthreads();
    // each thread has a run of neighbouring segments
    const uint32_t run = (segments + kThreads - 1) / kThreads;
    double mine = 0.0;
    for (uint32_t i = 0; i < run; ++i)
        if (tid * run + i < segments) mine += sh.segment[tid * run + i];
    double total;
    double before = sum_before(mine, sh.wavef, total);
    const double target = share * total;
    const uint32_t s = find_segment([&](uint32_t i) __attribute__((always_inline)) { return sh.segment[i]; }, segments, run, before, target, sh.found32, sh.wavef);
    if (wave != 0) return;
    float drawn;
    const int64_t token = draw_from(r, s, sh.wavef[0], target, kept_masses, drawn);
    if (lane == 0) {
        a.token[row] = token;
        if (a.logprob) a.logprob[row] = static_cast<float>(exponent(drawn, base) - log(total));
    }
}

template <typename, bool>
struct SampleTag;

template <typename T>
cbk_status sample_rows(const SampleArgs &a, uint32_t rows, bool divided, hipStream_t s) {
    const uint32_t all = rows * a.segments;
    const dim3 waves((all + kPartWaves - 1) / kPartWaves), block(64 * kPartWaves);
    if (a.segments && !divided) {
        hipLaunchKernelGGL((k_sample_parts<T, true>), waves, block, 0, s, a, all);
        hipLaunchKernelGGL((k_sample_join<T>), dim3(rows), block, 0, s, a);
        return launched();
    }
    if (divided) {
        if (!allow_lds_once<SampleTag<T, true>>(k_sample<T, true>, sizeof(Shared))) return CBK_E_HIP;
        // two workgroups a CU: each looks for the row's largest and the cut first, some 5 us
        const dim3 grid(std::min((a.segments + kWaves - 1) / kWaves, std::max(1u, 512 / rows)), rows);
        hipLaunchKernelGGL((k_sample_parts<T, false>), waves, block, 0, s, a, all);
        hipLaunchKernelGGL((k_sample_bins<T>), grid, dim3(kThreads), sizeof(BinsShared), s, a);
        hipLaunchKernelGGL((k_sample_collect<T>), grid, dim3(kThreads), sizeof(BinsShared), s, a);
        hipLaunchKernelGGL((k_sample<T, true>), dim3(rows), dim3(kThreads), sizeof(Shared), s, a);
        return launched();
    }
    if (!allow_lds_once<SampleTag<T, false>>(k_sample<T, false>, sizeof(Shared))) return CBK_E_HIP;
    hipLaunchKernelGGL((k_sample<T, false>), dim3(rows), dim3(kThreads), sizeof(Shared), s, a);
    return launched();
}

}  // namespace

cbk_status launch_sample(const cbk_sampling &p, const void *logits, int dtype, uint64_t ld, uint64_t V, uint64_t tokens,
                         const float *uniform, int64_t *token, float *logprob, const SamplePlan &pl, void *ws, hipStream_t s) {
    SampleArgs a{};
    a.p = p;
    a.logits = logits;
    a.ld = ld;
    a.V = static_cast<uint32_t>(V);
    a.uniform = uniform;
    a.token = token;
    a.logprob = logprob;
    a.segments = pl.segments;
    if (pl.segments) {
        const auto at = [&](uint64_t offset) { return static_cast<unsigned char *>(ws) + offset; };
        a.parts = reinterpret_cast<Part *>(at(0));
        a.sums = reinterpret_cast<uint64_t *>(at(pl.sums));
        a.bins = reinterpret_cast<uint64_t *>(at(pl.bins));
        a.list = reinterpret_cast<uint64_t *>(at(pl.list));
        a.state = reinterpret_cast<RowState *>(at(pl.state));
    }
    const bool f32 = dtype == CBK_F32;
    static_assert(sizeof(Part) == kSamplePartBytes && sizeof(RowState) == kSamplePartBytes && 256 * kSteps == kSampleSegment &&
                      kBins == kSampleBins && kList == kSampleBins, "the plan counts with them");
    for (uint64_t left = tokens; left > 0;) {
        const uint64_t n = std::min(left, pl.rows);
        const cbk_status st = f32 ? sample_rows<float>(a, static_cast<uint32_t>(n), pl.divided, s) : sample_rows<uint16_t>(a, static_cast<uint32_t>(n), pl.divided, s);
        if (st != CBK_OK) return st;
        left -= n;
        a.logits = static_cast<const unsigned char *>(a.logits) + n * ld * (f32 ? 4 : 2);
        a.uniform += n;
        a.token += n;
        if (a.logprob) a.logprob += n;
        if (a.p.temperatures) a.p.temperatures += n;
        if (a.p.top_ps) a.p.top_ps += n;
        if (a.p.min_ps) a.p.min_ps += n;
        if (a.p.top_ks) a.p.top_ks += n;
    }
    return CBK_OK;
}

}  // namespace cbk
