// HIP kernel for gfx950 (CDNA4) of cbk_sample.h: drawing a token from a row of logits.
//
// A workgroup of 16 waves has a row.  Every filter keeps a prefix of the row's order (logits falling,
// then index), so what is kept is what stands before one cut in that order, a 64-bit key of logit and
// index, and no row is sorted: a histogram of the distance from the largest logit (counts, and sums of
// exp(x - max) in fixed point, whose atomic additions give the same bits in any order) finds the bin
// that a cut falls into, and only that bin's entries are sorted, in LDS.  The draw then needs the kept
// entries' sums in index order: a sum of each 256 entries, the 256 that the target falls into, and in
// them the entry.
//
// The border between two tokens can be anywhere, and a vocabulary has 10^5 of them, so probabilities are
// formed in fp64: an fp32 sum's 1e-7 would name another token once in some hundred rows.  On this chip
// fp64 multiplications run at the rate of fp32 ones that are not packed.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "cbk_device.h"

namespace cbk {
namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr uint32_t kBins = 2048;      // of the histogram
constexpr float kSpan = 32.f;         // what it spans, in units of the temperature; the last bin holds the rest
constexpr uint32_t kList = 2048;      // entries that are sorted at once
constexpr uint32_t kSegments = (1u << 20) / 256 + 2;  // of 256 entries

struct SampleArgs {
    cbk_sampling p;
    const void *logits;
    uint64_t ld;
    uint32_t V;
    const float *uniform;
    int64_t *token;
    float *logprob;
};

struct Shared {
    union {
        struct {
            uint64_t mass[kBins];
            uint32_t count[kBins];
            uint64_t list[kList];
        };
        double segment[kSegments];
    };
    uint64_t wave64[kWaves];
    uint32_t wave32[kWaves];
    double wavef[kWaves];
    uint64_t found64[2];
    uint32_t found32[2];
};

// Ascending unsigned numbers for ascending floats (-0 as +0; no NaN).
__device__ __forceinline__ uint32_t ascending(float z) {
    const uint32_t u = __float_as_uint(z + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float from_ascending(uint32_t u) { return __uint_as_float(u & 0x80000000u ? u & 0x7FFFFFFFu : ~u); }
// A place in the row's order: smaller keys come first.
__device__ __forceinline__ uint64_t place_key(float z, uint32_t i) { return (static_cast<uint64_t>(~ascending(z)) << 32) | i; }

// e^x for x <= 0 to some 1e-15 of its value: 2^n times the exponential series at the rest, |r| <= ln 2 / 2, whose
// first left-out term is r^13 / 13! < 2e-16.  0 below e^-690.
__device__ __forceinline__ double exp_below(double x) {
    const double n = rint(x * 1.4426950408889634074);
    double r = fma(n, -0.69314718055994528623, x);
    r = fma(n, -2.3190468138462995584e-17, r);  // ln 2 less its rounding
    double s = 1.0 / 479001600.0;
    s = fma(s, r, 1.0 / 39916800.0);
    s = fma(s, r, 1.0 / 3628800.0);
    s = fma(s, r, 1.0 / 362880.0);
    s = fma(s, r, 1.0 / 40320.0);
    s = fma(s, r, 1.0 / 5040.0);
    s = fma(s, r, 1.0 / 720.0);
    s = fma(s, r, 1.0 / 120.0);
    s = fma(s, r, 1.0 / 24.0);
    s = fma(s, r, 1.0 / 6.0);
    s = fma(s, r, 0.5);
    s = fma(s, r, 1.0);
    s = fma(s, r, 1.0);
    return x < -690.0 ? 0.0 : ldexp(s, static_cast<int>(n));
}

template <typename T>
struct Row {
    const T *p;
    uint32_t V, skew, groups;  // groups of four entries; the first group's `skew` first ones do not exist

    __device__ __forceinline__ Row(const void *logits, uint64_t ld, uint32_t row, uint32_t n) {
        p = static_cast<const T *>(logits) + row * ld;
        V = n;
        skew = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) / sizeof(T)) & 3;
        groups = (V + skew + 3) / 4;
    }
    static __device__ __forceinline__ float value(float v) { return v; }
    static __device__ __forceinline__ float value(uint16_t v) { return bf16_value(v); }
    // The index of the group's first entry (possibly before the row) and its four logits, -inf where there is none.
    __device__ __forceinline__ int32_t load(uint32_t g, float (&z)[4]) const {
        const int32_t at = static_cast<int32_t>(4 * g) - static_cast<int32_t>(skew);
        if (at >= 0 && at + 4 <= static_cast<int32_t>(V)) {
            if constexpr (sizeof(T) == 4) {
                const f32x4_t v = *reinterpret_cast<const f32x4_t *>(p + at);
                z[0] = v[0]; z[1] = v[1]; z[2] = v[2]; z[3] = v[3];
            } else {
                const u32x2 v = *reinterpret_cast<const u32x2 *>(p + at);
                z[0] = bf16_value(static_cast<uint16_t>(v.x)); z[1] = bf16_value(static_cast<uint16_t>(v.x >> 16));
                z[2] = bf16_value(static_cast<uint16_t>(v.y)); z[3] = bf16_value(static_cast<uint16_t>(v.y >> 16));
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                z[j] = at + j >= 0 && at + j < static_cast<int32_t>(V) ? value(p[at + j]) : -__builtin_inff();
        }
        return at;
    }
};

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
template <typename V>
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
    for (int i = 0; i < kWaves; ++i) {
        if (i == w) before = total;
        total += wave[i];
    }
    __syncthreads();
    return before + (s - v);
}

template <typename T>
__global__ __launch_bounds__(kThreads) void k_sample(const SampleArgs a) {
    __shared__ Shared sh;
    const uint32_t row = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const Row<T> r(a.logits, a.ld, row, a.V);
    const uint32_t V = a.V;
    const double nan = __builtin_nan("");

    // the largest logit, and whether there is a NaN
    float top = -__builtin_inff();
    bool odd = false;
    for (uint32_t g = tid; g < r.groups; g += kThreads) {
        float z[4];
        r.load(g, z);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            odd = odd || z[j] != z[j];
            top = fmaxf(top, z[j]);
        }
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
    if (lane == 0) sh.wavef[wave] = top;
    if (__any(odd)) {
        if (lane == 0) sh.wavef[wave] = nan;
    }
    __syncthreads();
    bool bad = false;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
        const float t = static_cast<float>(sh.wavef[i]);
        bad = bad || t != t;
        top = fmaxf(top, t);
    }
    __syncthreads();
    const float heat = a.p.temperatures ? a.p.temperatures[row] : a.p.temperature;
    if (bad || top == -__builtin_inff() || heat != heat) {
        if (tid == 0) {
            a.token[row] = -1;
            if (a.logprob) a.logprob[row] = __builtin_nanf("");
        }
        return;
    }
    if (heat <= 0.f) {  // the first of the largest
        uint32_t first = ~0u;
        for (uint32_t g = tid; g < r.groups && first == ~0u; g += kThreads) {
            float z[4];
            const int32_t at = r.load(g, z);
#pragma unroll
            for (int j = 3; j >= 0; --j)
                if (z[j] == top) first = at + j;
        }
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1) first = min(first, static_cast<uint32_t>(__shfl_xor(first, o, 64)));
        if (lane == 0) sh.wave32[wave] = first;
        __syncthreads();
        if (tid == 0) {
            for (int i = 0; i < kWaves; ++i) first = min(first, sh.wave32[i]);
            a.token[row] = first;
            if (a.logprob) a.logprob[row] = 0.f;
        }
        return;
    }

    const double inv = 1.0 / static_cast<double>(heat), dtop = top;
    const bool endless = top == __builtin_inff();
    // x = (z - max) / temperature
    auto exponent = [&](float z) { return endless ? (z == top ? 0.0 : -1e300) : (static_cast<double>(z) - dtop) * inv; };
    auto mass_of = [&](float z) { return z == -__builtin_inff() ? 0.0 : exp_below(exponent(z)); };

    const int32_t top_k = a.p.top_ks ? a.p.top_ks[row] : a.p.top_k;
    const float top_p = a.p.top_ps ? a.p.top_ps[row] : a.p.top_p;
    const float min_p = fminf(a.p.min_ps ? a.p.min_ps[row] : a.p.min_p, 1.f);
    // min_p: logits below `least` are out; rounded up, so that comparing floats is comparing with the border
    float least = -__builtin_inff();
    if (min_p > 0.f && !endless) {
        const double border = dtop + static_cast<double>(heat) * log(static_cast<double>(min_p));
        least = static_cast<float>(border);
        if (static_cast<double>(least) < border) least = from_ascending(ascending(least) + 1);
        least = fminf(least, top);
    } else if (min_p > 0.f) {
        least = top;
    }
    uint64_t cut = ~uint64_t(0);  // the last key that is kept
    const bool by_count = top_k > 0 && static_cast<uint32_t>(top_k) < V, by_mass = top_p < 1.f;

    if (by_count || by_mass) {
        // the histogram; masses are counted in units of 2^-unit, which leaves their sum below 2^63
        const int unit = 62 - (32 - __clz(V));
        const float step = fminf((kBins - 1) / kSpan / heat, 1e30f);
        auto bin_of = [&](float z) {
            if (endless) return z == top ? 0u : kBins - 1;
            return static_cast<uint32_t>(fminf((top - z) * step, static_cast<float>(kBins - 1)));
        };
        auto fixed = [&](float z) { return static_cast<uint64_t>(ldexp(mass_of(z), unit)); };
        for (uint32_t i = tid; i < kBins; i += kThreads) {
            sh.mass[i] = 0;
            sh.count[i] = 0;
        }
        __syncthreads();
        for (uint32_t g = tid; g < r.groups; g += kThreads) {
            float z[4];
            r.load(g, z);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (z[j] >= least && z[j] != -__builtin_inff()) {
                    const uint32_t b = bin_of(z[j]);
                    atomicAdd(&sh.count[b], 1u);
                    atomicAdd(reinterpret_cast<unsigned long long *>(&sh.mass[b]), static_cast<unsigned long long>(fixed(z[j])));
                }
        }
        __syncthreads();

        // The entries before bin 2 tid, and their mass.
        const uint32_t c0 = sh.count[2 * tid], c1 = sh.count[2 * tid + 1];
        const uint64_t m0 = sh.mass[2 * tid], m1 = sh.mass[2 * tid + 1];
        uint32_t entries;
        uint64_t whole;
        const uint32_t cb = sum_before(c0 + c1, sh.wave32, entries);
        const uint64_t mb = sum_before(m0 + m1, sh.wave64, whole);

        // The first `some` entries of bin `b`, or those before which less than `most` of mass stands: the key of
        // the last of them in `cut`; returns their mass.  At least one.  All threads.
        auto cut_bin = [&](uint32_t b, uint32_t n, uint32_t some, uint64_t most) -> uint64_t {
            __syncthreads();
            if (n <= kList) {
                if (tid == 0) sh.found32[0] = 0;
                uint32_t size = 64;
                while (size < n) size *= 2;
                for (uint32_t i = tid; i < size; i += kThreads) sh.list[i] = ~uint64_t(0);
                __syncthreads();
                for (uint32_t g = tid; g < r.groups; g += kThreads) {
                    float z[4];
                    const int32_t at = r.load(g, z);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (z[j] >= least && z[j] != -__builtin_inff() && bin_of(z[j]) == b)
                            sh.list[atomicAdd(&sh.found32[0], 1u)] = place_key(z[j], at + j);
                }
                __syncthreads();
                // bitonic sort
                for (uint32_t k = 2; k <= size; k *= 2)
                    for (uint32_t d = k / 2; d > 0; d /= 2) {
                        for (uint32_t i = tid; i < size / 2; i += kThreads) {
                            const uint32_t lo = 2 * i - (i & (d - 1)), hi = lo + d;
                            const uint64_t x = sh.list[lo], y = sh.list[hi];
                            if ((x > y) == ((lo & k) == 0)) {
                                sh.list[lo] = y;
                                sh.list[hi] = x;
                            }
                        }
                        __syncthreads();
                    }
                uint64_t m[2] = {0, 0};
#pragma unroll
                for (uint32_t j = 0; j < 2; ++j)
                    if (2 * tid + j < n) m[j] = fixed(from_ascending(~static_cast<uint32_t>(sh.list[2 * tid + j] >> 32)));
                uint64_t all;
                uint64_t before = sum_before(m[0] + m[1], sh.wave64, all);
                if (tid == 0) {
                    sh.found64[0] = sh.list[0];
                    sh.found64[1] = m[0];
                }
                __syncthreads();
                // the last that is kept (the entries before it are: sums only grow)
#pragma unroll
                for (uint32_t j = 0; j < 2; ++j) {
                    const uint32_t i = 2 * tid + j;
                    const bool in = i < n && i < some && before < most;
                    const uint64_t next = before + m[j];
                    const bool last = in && !(i + 1 < n && i + 1 < some && next < most);
                    if (last) {
                        sh.found64[0] = sh.list[i];
                        sh.found64[1] = next;
                    }
                    before = next;
                }
                __syncthreads();
                cut = sh.found64[0];
                return sh.found64[1];
            }
            // Too many to sort (many equal logits, or a cut far below the largest): the smallest key with enough before
            // and at it, bit by bit; each of the 64 steps goes over the row.
            uint64_t key = 0, kept = 0;
            for (int bit = 63; bit >= 0; --bit) {
                const uint64_t probe = key | (uint64_t(1) << bit);  // keys below `probe` are counted
                uint32_t c = 0;
                uint64_t m = 0;
                for (uint32_t g = tid; g < r.groups; g += kThreads) {
                    float z[4];
                    const int32_t at = r.load(g, z);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (z[j] >= least && z[j] != -__builtin_inff() && bin_of(z[j]) == b && place_key(z[j], at + j) < probe) {
                            ++c;
                            m += fixed(z[j]);
                        }
                }
                uint32_t call;
                uint64_t mall;
                sum_before(c, sh.wave32, call);
                sum_before(m, sh.wave64, mall);
                // the key is at or past `probe` while the entries before `probe` leave room for one more
                if (call < some && mall < most) {
                    key = probe;
                    kept = mall;
                }
            }
            // `key` is the largest key before which there is room: the entry at it, or the last before it, is the last kept
            uint64_t best = 0, m = 0;
            for (uint32_t g = tid; g < r.groups; g += kThreads) {
                float z[4];
                const int32_t at = r.load(g, z);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (z[j] >= least && z[j] != -__builtin_inff() && bin_of(z[j]) == b && place_key(z[j], at + j) == key) {
                        best = key;
                        m = fixed(z[j]);
                    }
            }
            uint64_t at_key;
            sum_before(m, sh.wave64, at_key);
            (void)best;
            cut = key;
            return kept + at_key;
        };

        if (by_count && static_cast<uint32_t>(top_k) < entries) {
            const uint32_t want = top_k;
            const bool here = cb < want && want <= cb + c0 + c1;  // of one thread alone
            if (here) {
                const bool second = want > cb + c0;
                sh.found32[0] = 2 * tid + second;
                sh.found32[1] = want - (second ? cb + c0 : cb);
                sh.found64[0] = second ? mb + m0 : mb;
            }
            __syncthreads();
            const uint32_t b = sh.found32[0], some = sh.found32[1];
            const uint64_t before = sh.found64[0];
            const uint32_t n = sh.count[b];
            whole = before + cut_bin(b, n, some, ~uint64_t(0));
            __syncthreads();
        }
        if (by_mass) {
            // entries before which less than `want` stands are kept
            const double share = fmax(static_cast<double>(top_p), 0.0) * static_cast<double>(whole);
            const uint64_t want = max(uint64_t(1), static_cast<uint64_t>(ceil(share)));
            if (tid == 0) sh.found32[0] = kBins;
            __syncthreads();
            // the last bin before which less than `want` stands, of those that hold anything
            const bool in0 = c0 > 0 && mb < want, in1 = c1 > 0 && mb + m0 < want;
            const bool past0 = mb + m0 >= want, past1 = mb + m0 + m1 >= want;
            if (in0 && past0) {
                sh.found32[0] = 2 * tid;
                sh.found64[0] = mb;
            }
            if (in1 && past1) {
                sh.found32[0] = 2 * tid + 1;
                sh.found64[0] = mb + m0;
            }
            __syncthreads();
            const uint32_t b = sh.found32[0];
            const uint64_t before = sh.found64[0];
            if (b < kBins) {  // else rounding leaves nothing past it: all are kept
                const uint64_t old = cut;
                cut_bin(b, sh.count[b], ~0u, want - before);
                cut = cut < old ? cut : old;
            }
        }
        __syncthreads();
    }

    // sums of 256 entries each, in index order
    auto kept_mass = [&](float z, int32_t i) {
        return z >= least && place_key(z, static_cast<uint32_t>(i)) <= cut ? mass_of(z) : 0.0;
    };
    auto wave_total = [](double v) {
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
        return v;
    };
    const uint32_t segments = (r.groups + 63) / 64;
    for (uint32_t s = wave; s < segments; s += kWaves) {
        float z[4];
        double m = 0.0;
        if (s * 64 + lane < r.groups) {
            const int32_t at = r.load(s * 64 + lane, z);
#pragma unroll
            for (int j = 0; j < 4; ++j) m += kept_mass(z[j], at + j);
        }
        m = wave_total(m);
        if (lane == 0) sh.segment[s] = m;
    }
    __syncthreads();
    // each thread has a run of neighbouring segments
    const uint32_t run = (segments + kThreads - 1) / kThreads;
    double mine = 0.0;
    for (uint32_t i = 0; i < run; ++i)
        if (tid * run + i < segments) mine += sh.segment[tid * run + i];
    double total;
    double before = sum_before(mine, sh.wavef, total);
    const float u = a.uniform[row];
    const double target = (u >= 0.f ? static_cast<double>(u) : 0.0) * total;
    // the first segment whose running sum exceeds the target, or the last that holds anything
    if (tid == 0) {
        sh.found32[0] = ~0u;
        sh.found32[1] = 0;
    }
    __syncthreads();
    {
        double sum = before;
        uint32_t first = ~0u, last = 0;
        for (uint32_t i = 0; i < run; ++i) {
            const uint32_t s = tid * run + i;
            if (s >= segments) break;
            const double m = sh.segment[s];
            sum += m;
            if (m > 0.0) {
                last = s;
                if (first == ~0u && sum > target) first = s;
            }
        }
        if (first != ~0u) atomicMin(&sh.found32[0], first);
        if (last) atomicMax(&sh.found32[1], last);
    }
    __syncthreads();
    const uint32_t s = sh.found32[0] != ~0u ? sh.found32[0] : sh.found32[1];
    if (tid == s / run) {
        double sum = before;
        for (uint32_t i = tid * run; i < s; ++i) sum += sh.segment[i];
        sh.wavef[0] = sum;
    }
    __syncthreads();
    if (wave != 0) return;
    before = sh.wavef[0];
    float z[4] = {0.f, 0.f, 0.f, 0.f};
    double m[4] = {0.0, 0.0, 0.0, 0.0};
    int32_t at = 0;
    if (s * 64 + lane < r.groups) {
        at = r.load(s * 64 + lane, z);
#pragma unroll
        for (int j = 0; j < 4; ++j) m[j] = kept_mass(z[j], at + j);
    }
    double sum = m[0] + m[1] + m[2] + m[3];
    const double own = sum;
#pragma unroll
    for (int by = 1; by < 64; by *= 2) {
        const double t = shuffle_up(sum, by);
        if (lane >= static_cast<uint32_t>(by)) sum += t;
    }
    sum = before + (sum - own);
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
    const uint32_t who = hits ? __ffsll(static_cast<unsigned long long>(hits)) - 1 : 63 - __clzll(static_cast<long long>(ends | 1));
    if (lane == who) {
        a.token[row] = hits ? hit : end;
        if (a.logprob) a.logprob[row] = static_cast<float>(exponent(hits ? hz : ez) - log(total));
    }
}

}  // namespace

cbk_status launch_sample(const cbk_sampling &p, const void *logits, int dtype, uint64_t ld, uint64_t V, uint64_t tokens,
                         const float *uniform, int64_t *token, float *logprob, hipStream_t s) {
    const SampleArgs a{p, logits, ld, static_cast<uint32_t>(V), uniform, token, logprob};
    const dim3 grid(static_cast<uint32_t>(tokens)), block(kThreads);
    if (dtype == CBK_F32)
        hipLaunchKernelGGL(k_sample<float>, grid, block, 0, s, a);
    else
        hipLaunchKernelGGL(k_sample<uint16_t>, grid, block, 0, s, a);
    return launched();
}

}  // namespace cbk
