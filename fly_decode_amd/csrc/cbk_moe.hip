// HIP kernels for gfx950 (CDNA4) of cbk_moe.h, but for the experts' products (cbk_moe_mm.hip): routing and its
// gradient, the order of slots by expert, and what gathers the experts' results by token.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#pragma clang diagnostic ignored "-Wunused-function"  // cu_count of cbk_device.h
#include "cbk_exp.h"
#include "cbk_moe_device.h"

namespace cbk {
namespace {

// ------------------------------------------------------------------------------- routing
// A wave has a token, lane l the experts l, l + 64, ..: up to 16 of them (NPL).

struct RouteArgs {
    cbk_router r;
    const void *logits;
    uint64_t ld, tokens;
    const float *bias;
    int32_t *experts;
    float *weights;
    const float *dweights;
    void *dlogits;
    uint64_t ldd;
};

__device__ __forceinline__ float logit(const float *p, uint64_t i) { return p[i]; }
__device__ __forceinline__ float logit(const uint16_t *p, uint64_t i) { return bf16_value(p[i]); }
__device__ __forceinline__ void put(float *p, uint64_t i, float v) { p[i] = v; }
__device__ __forceinline__ void put(uint16_t *p, uint64_t i, float v) { p[i] = to_bf16(v); }

// Ascending unsigned numbers above 0 for ascending doubles (-0 as +0; no NaN).
__device__ __forceinline__ uint64_t ascending(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v + 0.0);
    return u >> 63 ? ~u : u | (uint64_t(1) << 63);
}

// 1 / (1 + e^-z), to some 1e-13 of itself
__device__ __forceinline__ double logistic(double z) {
    const double e = exponential(-fabs(z)), s = 1.0 / (1.0 + e);  // (of +-infinity: 1, and 0 or 1)
    return z < 0.0 ? e * s : s;
}

template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
    return max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(static_cast<int>(v), static_cast<int>(v), CTRL, ROWS, 0xF, false)));
}
// The largest of the 64 lanes' v, in every lane.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    v = dpp_max<0x111, 0xF>(v);
    v = dpp_max<0x112, 0xF>(v);
    v = dpp_max<0x114, 0xF>(v);
    v = dpp_max<0x118, 0xF>(v);
    v = dpp_max<0x142, 0xA>(v);
    v = dpp_max<0x143, 0xC>(v);
    return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), 63));
}
// (by halves, which takes half the instructions of comparing 64 bits)
__device__ __forceinline__ uint64_t wave_max(uint64_t v) {
    const uint32_t mine = static_cast<uint32_t>(v >> 32), hi = wave_max(mine);
    return (static_cast<uint64_t>(hi) << 32) | wave_max(mine == hi ? static_cast<uint32_t>(v) : 0u);
}
__device__ __forceinline__ uint64_t shuffle_xor(uint64_t v, int o) {
    const uint32_t lo = __shfl_xor(static_cast<uint32_t>(v), o, 64), hi = __shfl_xor(static_cast<uint32_t>(v >> 32), o, 64);
    return (static_cast<uint64_t>(hi) << 32) | lo;
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
    return v;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
    return v;
}
__device__ __forceinline__ float wave_top(float v) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor(v, o, 64));
    return v;
}

// Experts are chosen one after the other by the wave's largest key.  Without a bias and sums of two scores the
// order is that of the logits, whose keys are exact; with them (WIDE) scores are formed and compared in fp64, where
// rounding does not decide between two that an fp32 sum could not tell apart.  Weights take an fp64 exponential for
// each chosen expert (and each expert, for a softmax that is not renormalised), which nothing waits for.
// What bounds it is a wave's instructions, not memory: 4096 tokens of 256 experts in 8 groups, 8 chosen, take 12.3 us
// among other calls, 12.7 to 13.5 in a graph of them, by what they hold (0.36 TB/s; among other calls 17.4 with a group's
// best two found by one lane each, and 14.6 with 64-bit maxima and divisions by the groups' sizes), one token of 64 experts
// 3.8, a launch's time.  A wave a token: with more lanes than 64 a maximum would have to go through LDS.
template <typename T, int NPL, bool WIDE>
__global__ __launch_bounds__(256) void k_route(const RouteArgs a) {
    extern __shared__ uint64_t keys_lds[];  // groups only: a wave's keys
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint64_t t = static_cast<uint64_t>(blockIdx.x) * 4 + wave;
    if (t >= a.tokens) return;
    const uint32_t E = a.r.experts, k = a.r.k;
    const T *row = static_cast<const T *>(a.logits) + t * a.ld;
    const bool sigmoid = a.r.score == CBK_SCORE_SIGMOID;

    float z[NPL];
    double s[NPL];
    uint64_t key[NPL];  // 0: not to be chosen
    bool bad = false;
    float top = -__builtin_inff();
#pragma unroll
    for (int j = 0; j < NPL; ++j) {
        const uint32_t e = j * 64 + lane;
        z[j] = e < E ? logit(row, e) : -__builtin_inff();
        bad = bad || z[j] != z[j] || z[j] == __builtin_inff();
        top = fmaxf(top, z[j]);
    }
    top = wave_top(top);
    const double base = top == -__builtin_inff() ? 0.0 : static_cast<double>(top);
    double denominator = 1.0;
    if (WIDE || !(sigmoid || a.r.renormalise)) {
        double sum = 0.0;
#pragma unroll
        for (int j = 0; j < NPL; ++j) {
            s[j] = sigmoid ? logistic(static_cast<double>(z[j])) : exponential(static_cast<double>(z[j]) - base);
            sum += s[j];
        }
        if (!sigmoid) {
            denominator = wave_sum(sum);
            if (denominator == 0.0) denominator = 1.0;
            if constexpr (WIDE) {
#pragma unroll
                for (int j = 0; j < NPL; ++j) s[j] /= denominator;
            }
        }
    }
#pragma unroll
    for (int j = 0; j < NPL; ++j) {
        const uint32_t e = j * 64 + lane;
        const float bias = a.bias && e < E ? a.bias[e] : 0.f;
        const bool out = z[j] == -__builtin_inff() || bias == -__builtin_inff();
        if constexpr (WIDE) {
            s[j] += bias;
            bad = bad || s[j] != s[j];
            key[j] = out ? 0 : ascending(s[j]);
        } else {
            key[j] = out ? 0 : static_cast<uint64_t>(ascending(static_cast<double>(z[j])));
        }
    }
    bad = __any(bad);

    if (a.r.groups > 1) {
        // a group's mark: lanes take groups in turn; 0 where it has nothing to choose
        uint64_t *mine = keys_lds + wave * (NPL * 64);
        const uint32_t size = E / a.r.groups;
#pragma unroll
        for (int j = 0; j < NPL; ++j) mine[j * 64 + lane] = key[j];
        asm volatile("" ::: "memory");  // one wave's LDS accesses run in order
        uint64_t marks[NPL];
        // the best two of a group by `share` neighbouring lanes, a power of two of them, with every share-th of its experts
        // each; then joined (8 groups of 32: a quarter of a lane's steps through LDS)
        uint32_t shift = 0;
        while ((a.r.groups << (shift + 1)) <= 64) ++shift;
        const uint32_t share = 1u << shift;
#pragma unroll
        for (int j = 0; j < NPL; ++j) {
            marks[j] = 0;
            if (static_cast<uint32_t>(j * 64) >> shift >= a.r.groups) continue;
            const uint32_t g = (j * 64 + lane) >> shift, part = lane & (share - 1);
            uint64_t first = 0, second = 0;
            if (g < a.r.groups)
                for (uint32_t i = part; i < size; i += share) {
                    const uint64_t v = mine[g * size + i];
                    if (v > first) {
                        second = first;
                        first = v;
                    } else if (v > second) {
                        second = v;
                    }
                }
            for (uint32_t o = 1; o < share; o *= 2) {
                const uint64_t f = shuffle_xor(first, o), t = shuffle_xor(second, o);
                const uint64_t low = first < f ? first : f;
                first = first < f ? f : first;
                second = low > second ? low : second;
                second = second < t ? t : second;
            }
            if constexpr (WIDE) {
                auto value = [](uint64_t u) { return __builtin_bit_cast(double, u >> 63 ? u & ~(uint64_t(1) << 63) : ~u); };
                if (a.r.group_top == 2 && second) first = ascending(value(first) + value(second));
            }
            marks[j] = part == 0 ? first : 0;
        }
        asm volatile("" ::: "memory");
        // keep the best groups: mark them in LDS
#pragma unroll
        for (int j = 0; j < NPL; ++j) mine[j * 64 + lane] = 0;
        asm volatile("" ::: "memory");
        for (uint32_t n = 0; n < a.r.top_groups; ++n) {
            uint64_t best = marks[0];
#pragma unroll
            for (int j = 1; j < NPL; ++j) best = marks[j] > best ? marks[j] : best;
            best = wave_max(best);
            if (best == 0) break;
            bool found = false;
#pragma unroll
            for (int j = 0; j < NPL; ++j) {
                const uint64_t has = __ballot(marks[j] == best);
                if (!found && has) {
                    found = true;
                    if (lane == static_cast<uint32_t>(__ffsll(static_cast<unsigned long long>(has)) - 1)) {
                        marks[j] = 0;
                        mine[(j * 64 + lane) >> shift] = 1;
                    }
                }
            }
        }
        asm volatile("" ::: "memory");
        const uint32_t inverse = ((1u << 20) + size - 1) / size;  // e / size of e < 1024: e (size - 1) < 2^20
#pragma unroll
        for (int j = 0; j < NPL; ++j) {
            const uint32_t e = j * 64 + lane;
            if (e < E && mine[(e * inverse) >> 20] == 0) key[j] = 0;
        }
    }

    int32_t chosen = -1;  // of slot `lane`
    float cz = 0.f;
    for (uint32_t n = 0; n < k; ++n) {
        uint64_t best = key[0];
#pragma unroll
        for (int j = 1; j < NPL; ++j) best = key[j] > best ? key[j] : best;
        best = wave_max(best);
        if (best == 0) break;
        bool found = false;
#pragma unroll
        for (int j = 0; j < NPL; ++j) {
            const uint64_t has = __ballot(key[j] == best);
            if (!found && has) {
                found = true;
                const int who = __ffsll(static_cast<unsigned long long>(has)) - 1;
                const float v = __shfl(z[j], who, 64);
                if (lane == n) {
                    chosen = j * 64 + who;
                    cz = v;
                }
                if (lane == static_cast<uint32_t>(who)) key[j] = 0;
            }
        }
    }
    const bool have = chosen >= 0;
    double w = 0.0;
    // renormalised: relative to the largest of the chosen, so that something is left to divide by (the sigmoid of what is
    // below -40 is its exponential, to the last bit)
    const float ref = a.r.renormalise ? wave_top(have ? cz : -__builtin_inff()) : top;
    if (sigmoid && !(a.r.renormalise && ref < -40.f)) {
        if (have) w = logistic(static_cast<double>(cz));
    } else {
        if (have) w = exponential(static_cast<double>(cz) - static_cast<double>(ref)) / (a.r.renormalise ? 1.0 : denominator);
    }
    if (a.r.renormalise) {
        const double sum = wave_sum(w);
        if (sum > 0.0) w /= sum;
    }
    if (lane < k) {
        a.experts[t * k + lane] = bad ? static_cast<int32_t>(lane) : chosen;
        a.weights[t * k + lane] = bad ? __builtin_nanf("") : static_cast<float>(w * static_cast<double>(a.r.scale));
    }
}

// Lane i < k has slot i.  With w = s / (sum of the chosen s), d the gradient of a weight times scale and m = <d, w>,
// a softmax gives dz = w (d - m) at the chosen experts alone: the others' share cancels.  Sums are fp32, within the bound of
// some 16 + E roundings.  16384 tokens of 128 experts take 10.1 us (1.8 TB/s read and written).
template <typename T, int NPL>
__global__ __launch_bounds__(256) void k_route_bwd(const RouteArgs a) {
    const uint32_t lane = threadIdx.x & 63;
    const uint64_t t = static_cast<uint64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
    if (t >= a.tokens) return;
    const uint32_t E = a.r.experts, k = a.r.k;
    const T *row = static_cast<const T *>(a.logits) + t * a.ld;
    const bool sigmoid = a.r.score == CBK_SCORE_SIGMOID, dense = !sigmoid && !a.r.renormalise;

    int32_t e = -1;
    float d = 0.f, cz = -__builtin_inff();
    if (lane < k) {
        e = a.experts[t * k + lane];
        if (e < 0 || static_cast<uint32_t>(e) >= E) e = -1;
        if (e >= 0) {
            d = a.dweights[t * k + lane] * a.r.scale;
            cz = logit(row, e);
        }
    }
    float z[NPL], out[NPL];
    float top = -__builtin_inff();
    bool odd = false;  // a NaN, or a +inf that a softmax has no gradient at: the row is NaN
#pragma unroll
    for (int j = 0; j < NPL; ++j) {
        const uint32_t x = j * 64 + lane;
        z[j] = x < E ? logit(row, x) : -__builtin_inff();
        odd = odd || z[j] != z[j] || z[j] == __builtin_inff();
        top = fmaxf(top, z[j]);
        out[j] = 0.f;
    }
    odd = __any(odd);
    float part = 0.f;  // of slot `lane`
    float mean = 0.f, inv = 0.f;
    if (sigmoid) {
        const float s = e >= 0 ? 1.f / (1.f + expf(-cz)) : 0.f, r = e >= 0 ? 1.f / (1.f + expf(cz)) : 0.f;
        if (a.r.renormalise) {
            // w = s / sum, w (1 - s) (d - m): formed so that scores far below 1 lose nothing (below -30 a sigmoid is an
            // exponential in fp32, and the largest of the chosen divides out)
            const float most = wave_top(cz), best = wave_top(s);
            const float rel = most < -30.f ? (e >= 0 && most > -__builtin_inff() ? expf(cz - most) : 0.f) : best > 0.f ? s / best : 0.f;
            const float sum = wave_sum(rel), w = sum > 0.f ? rel / sum : 0.f;
            const float m = wave_sum(e >= 0 ? d * w : 0.f);
            part = e >= 0 ? w * r * (d - m) : 0.f;
        } else {
            part = d * s * r;
        }
    } else if (a.r.renormalise) {
        const float best = wave_top(cz), at = best == -__builtin_inff() ? 0.f : best;
        const float x = e >= 0 ? expf(cz - at) : 0.f, sum = wave_sum(x), w = sum > 0.f ? x / sum : 0.f;
        const float m = wave_sum(e >= 0 ? d * w : 0.f);
        part = e >= 0 ? w * (d - m) : 0.f;
    } else {
        top = wave_top(top);
        if (top == -__builtin_inff()) top = 0.f;
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < NPL; ++j) {
            out[j] = expf(z[j] - top);
            sum += out[j];
        }
        sum = wave_sum(sum);
        inv = sum > 0.f ? 1.f / sum : 0.f;
        const float s = e >= 0 ? expf(cz - top) * inv : 0.f;
        mean = wave_sum(d * s);
        part = d * s;
    }
    if (dense) {
#pragma unroll
        for (int j = 0; j < NPL; ++j) out[j] = -out[j] * inv * mean;
    }
    for (uint32_t n = 0; n < k; ++n) {
        const int32_t who = __builtin_amdgcn_readlane(e, n);
        const float v = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(part), n));
        if (who < 0) continue;
#pragma unroll
        for (int j = 0; j < NPL; ++j)
            if (static_cast<uint32_t>(who) == j * 64 + lane) out[j] += v;
    }
    T *to = static_cast<T *>(a.dlogits) + t * a.ldd;
#pragma unroll
    for (int j = 0; j < NPL; ++j)
        if (j * 64 + lane < E) put(to, j * 64 + lane, odd ? __builtin_nanf("") : out[j]);
}

// --------------------------------------------------------------------------- slots by expert
// One workgroup sorts the slots by expert, stably, and cuts each expert's run into token tiles of equal size, listed by
// falling quarters of a whole tile (what takes longest is begun first).
// Each wave counts a run of slots, then places them: the rank of a slot among the wave's 64 of the same expert comes
// from ballots over the expert's bits.  Eight steps' slots are asked for at once: 8192 slots took 15.8 us with one at a
// time, 13.4 so.  The other workgroups of the launch copy the rows of X and dY that the products cannot take as they are
// (launches of their own cost a backward pass of 45 tokens 5 us).
struct PadArgs {
    const uint16_t *X;  // [T][ld] into P [T][Kp], columns past K zero; null: nothing to copy
    uint64_t ld, T;
    uint32_t K, Kp;
    uint16_t *P;
};
struct SortArgs {
    const int32_t *experts;
    uint32_t slots, k, count, tile, unit;  // tokens of a tile at most, and what its size is rounded up to
    uint32_t *token_of, *slot_of;
    int32_t *place_of;
    ExTile *tiles;  // null: nothing to sort
    uint32_t *ntiles;
    PadArgs pad[2];
};
constexpr int kSortWaves = 16;

__device__ __forceinline__ void pad_rows(const PadArgs &a) {
    const uint32_t per = a.Kp / 4, stride = (gridDim.x - 1) * blockDim.x;
    const uint64_t n = a.T * per;  // (a chunk: T per < 2^28)
    for (uint32_t i = (blockIdx.x - 1) * blockDim.x + threadIdx.x; i < n; i += stride) {
        const uint32_t t = i / per, k = (i - t * per) * 4;
        const uint16_t *x = a.X + t * a.ld + k;
        uint32_t v[4];
#pragma unroll
        for (uint32_t j = 0; j < 4; ++j) v[j] = k + j < a.K ? x[j] : 0u;
        *reinterpret_cast<u32x2 *>(a.P + static_cast<uint64_t>(i) * 4) = (u32x2){v[0] | (v[1] << 16), v[2] | (v[3] << 16)};
    }
}

__global__ __launch_bounds__(64 * kSortWaves) void k_sort(const SortArgs a) {
    if (blockIdx.x > 0) {
        for (int i = 0; i < 2; ++i)
            if (a.pad[i].X) pad_rows(a.pad[i]);
        return;
    }
    if (!a.tiles) return;
    extern __shared__ uint32_t lds[];  // [waves][count]: how many, then where the wave's next one goes
    __shared__ uint32_t wave_sums[5][kSortWaves];
    const uint32_t tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const uint32_t n = a.count;
    for (uint32_t i = tid; i < kSortWaves * n; i += blockDim.x) lds[i] = 0;
    __syncthreads();
    const uint32_t steps = (a.slots + 64 * kSortWaves - 1) / (64 * kSortWaves);  // of 64 slots, for a wave
    const uint32_t from = wave * steps * 64;
    uint32_t *mine = lds + wave * n;
    constexpr uint32_t N = 8;
    uint32_t e[N];
    auto ask = [&](uint32_t i) __attribute__((always_inline)) {
#pragma unroll
        for (uint32_t j = 0; j < N; ++j) {
            const uint32_t s = from + (i + j) * 64 + lane;
            e[j] = i + j < steps && s < a.slots ? static_cast<uint32_t>(a.experts[s]) : ~0u;
        }
    };
    for (uint32_t i = 0; i < steps; i += N) {
        ask(i);
#pragma unroll
        for (uint32_t j = 0; j < N; ++j)
            if (e[j] < n) atomicAdd(&mine[e[j]], 1u);
    }
    if (steps > N) ask(0);  // (else they are there)
    __syncthreads();
    // expert `tid`: its slots, and its tiles
    uint32_t m = 0;
    if (tid < n)
        for (int w = 0; w < kSortWaves; ++w) m += lds[w * n + tid];
    const uint32_t parts = (m + a.tile - 1) / a.tile;
    const uint32_t size = m ? min(a.tile, ((m + parts - 1) / parts + a.unit - 1) / a.unit * a.unit) : 1;
    const uint32_t tiles = (m + size - 1) / size;
    // all of an expert's tiles but the last are of `size`; kind 0 is a whole tile
    auto kind = [&](uint32_t n) { return 3 - min((n - 1) / max(a.unit, 1u), 3u); };
    const uint32_t main_kind = kind(size), last_kind = tiles ? kind(m - (tiles - 1) * size) : 0;
    uint32_t sums[5] = {m, 0, 0, 0, 0};
#pragma unroll
    for (uint32_t q = 0; q < 4; ++q) sums[1 + q] = tiles ? (main_kind == q ? tiles - 1 : 0) + (last_kind == q ? 1 : 0) : 0;
    uint32_t before[5];
#pragma unroll
    for (int q = 0; q < 5; ++q) {
        uint32_t v = sums[q];
#pragma unroll
        for (int by = 1; by < 64; by *= 2) {
            const uint32_t x = __shfl_up(v, by, 64);
            if (lane >= static_cast<uint32_t>(by)) v += x;
        }
        if (lane == 63) wave_sums[q][wave] = v;
        before[q] = v - sums[q];
    }
    __syncthreads();
    uint32_t kinds = 0;  // tiles of the kinds before
#pragma unroll
    for (int q = 0; q < 5; ++q) {
        uint32_t all = 0;
        for (uint32_t w = 0; w < kSortWaves; ++w) {
            if (w == wave) before[q] += all;
            all += wave_sums[q][w];
        }
        if (q > 0) {
            before[q] += kinds;
            kinds += all;
        }
    }
    const uint32_t start = before[0];
    if (tid < n) {
        uint32_t at = start;
        for (int w = 0; w < kSortWaves; ++w) {
            const uint32_t c = lds[w * n + tid];
            lds[w * n + tid] = at;
            at += c;
        }
        for (uint32_t i = 0; i < tiles; ++i) {
            const uint32_t q = i + 1 < tiles ? main_kind : last_kind;
            // (a chain of selects: the array stays in registers)
            const uint32_t to = q == 0 ? before[1]++ : q == 1 ? before[2]++ : q == 2 ? before[3]++ : before[4]++;
            a.tiles[to] = ExTile{tid, start + i * size, min(size, m - i * size), 0};
        }
    }
    if (tid == 0) *a.ntiles = kinds;
    __syncthreads();
    uint32_t bits = 0;
    while ((1u << bits) < n) ++bits;
    for (uint32_t i = 0; i < steps; i += N) {
        if (i > 0) ask(i);
#pragma unroll
        for (uint32_t j = 0; j < N; ++j) {
            if (i + j >= steps) break;
            const uint32_t s = from + (i + j) * 64 + lane;
            const bool in = e[j] < n;
            uint64_t same = __ballot(in);
            for (uint32_t b = 0; b < bits; ++b) {
                const uint64_t has = __ballot((e[j] >> b) & 1);
                same &= (e[j] >> b) & 1 ? has : ~has;
            }
            const uint32_t rank = __popcll(same & ((uint64_t(1) << lane) - 1));
            uint32_t at = 0;
            if (in) at = mine[e[j]] + rank;
            asm volatile("" ::: "memory");  // one wave's LDS accesses run in order
            if (in && (same >> lane) == 1) mine[e[j]] = at + 1;  // the last of them
            asm volatile("" ::: "memory");
            if (in) {
                a.slot_of[at] = s;
                a.token_of[at] = s / a.k;
            }
            if (s < a.slots) a.place_of[s] = in ? static_cast<int32_t>(at) : -1;
        }
    }
}

// ------------------------------------------------------------------------------- by token
struct GatherArgs {
    const float *S;        // [splits][slots][lds]
    uint64_t split_stride;
    uint32_t splits, lds, k, width;
    uint64_t tokens;
    const int32_t *place_of;  // of a slot in the sorted order, or -1;
    const int32_t *experts;   // or null, and S is in the slots' own order: the slots' experts,
    uint32_t count;           // of which those from here on are none
    uint16_t *Y;
    uint64_t ldy;
    uint32_t vec;
    // a backward pass: the slots' dweights as the sums of `parts` each, by workgroups past the `blocks` of a token
    uint32_t blocks, parts;
    const float *dw;
    float *dweights;
};

// dweights of a token's slots from their parts over the hidden columns, a wave a slot.
__device__ __forceinline__ void sum_dweights(const GatherArgs &a, uint64_t t) {
    const uint32_t lane = threadIdx.x & 63;
    for (uint32_t j = threadIdx.x >> 6; j < a.k; j += 4) {
        const int32_t at = a.place_of[t * a.k + j];
        float v = 0.f;
        if (at >= 0)
            for (uint32_t i = lane; i < a.parts; i += 64) v += a.dw[static_cast<uint64_t>(at) * a.parts + i];
        v = wave_sum(v);
        if (lane == 0) a.dweights[t * a.k + j] = v;
    }
}

// Y[t] = the sum of its slots' results, in the slots' order.  A thread has 4 columns of a token, and asks for eight
// results at a time (one after the other, the four of one token took 6.2 us, 3.8 so).  Bound by memory: 2048 tokens of
// four results of 4096 columns take 25 us, 6 TB/s.  (The results are fp32: added up before any is rounded.)
__global__ __launch_bounds__(256) void k_gather(const GatherArgs a) {
    const uint32_t c = (blockIdx.x * 256 + threadIdx.x) * 4;
    const uint64_t t = blockIdx.y + static_cast<uint64_t>(blockIdx.z) * gridDim.y;
    if (t >= a.tokens) return;
    if (blockIdx.x == a.blocks) return sum_dweights(a, t);
    if (c >= a.width) return;
    f32x4_t v = {0.f, 0.f, 0.f, 0.f};
    auto place = [&](uint32_t j) {
        const uint64_t slot = t * a.k + j;
        if (a.place_of) return a.place_of[slot];
        return static_cast<uint32_t>(a.experts[slot]) < a.count ? static_cast<int32_t>(slot) : -1;
    };
    if (a.splits == 1) {
        for (uint32_t j = 0; j < a.k; j += 8) {
            int32_t at[8];
            f32x4_t x[8];
#pragma unroll
            for (uint32_t i = 0; i < 8; ++i) at[i] = j + i < a.k ? place(j + i) : -1;
#pragma unroll
            for (uint32_t i = 0; i < 8; ++i) {
                x[i] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
                if (at[i] >= 0) x[i] = *reinterpret_cast<const f32x4_t *>(a.S + static_cast<uint64_t>(at[i]) * a.lds + c);
            }
#pragma unroll
            for (uint32_t i = 0; i < 8; ++i) v += x[i];
        }
    } else {  // up to 8 shares
        for (uint32_t j = 0; j < a.k; ++j) {
            const int32_t at = place(j);
            if (at < 0) continue;
            f32x4_t x[8];
#pragma unroll
            for (uint32_t i = 0; i < 8; ++i) {
                x[i] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
                if (i < a.splits) x[i] = *reinterpret_cast<const f32x4_t *>(a.S + i * a.split_stride + static_cast<uint64_t>(at) * a.lds + c);
            }
#pragma unroll
            for (uint32_t i = 0; i < 8; ++i) v += x[i];
        }
    }
    uint16_t *y = a.Y + t * a.ldy + c;
    if (a.vec && c + 4 <= a.width) {
        *reinterpret_cast<u32x2 *>(y) = (u32x2){pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
    } else {
#pragma unroll
        for (uint32_t r = 0; r < 4; ++r)
            if (c + r < a.width) y[r] = to_bf16(v[r]);
    }
}

template <typename T, int NPL>
void route_as(RouteArgs a, bool wide, bool backward, hipStream_t s) {
    const uint32_t lds = a.r.groups > 1 ? 4 * NPL * 64 * 8 : 0;
    // a launch has fewer than 2^32 threads, 64 a token
    constexpr uint64_t kMost = uint64_t(1) << 25;
    for (uint64_t left = a.tokens; left > 0; left -= a.tokens) {
        a.tokens = std::min(left, kMost);
        const dim3 grid(static_cast<uint32_t>((a.tokens + 3) / 4)), block(256);
        if (backward)
            hipLaunchKernelGGL((k_route_bwd<T, NPL>), grid, block, 0, s, a);
        else if (wide)
            hipLaunchKernelGGL((k_route<T, NPL, true>), grid, block, lds, s, a);
        else
            hipLaunchKernelGGL((k_route<T, NPL, false>), grid, block, lds, s, a);
        a.logits = static_cast<const T *>(a.logits) + a.tokens * a.ld;
        a.experts += a.tokens * a.r.k;
        if (backward) {
            a.dweights += a.tokens * a.r.k;
            a.dlogits = static_cast<T *>(a.dlogits) + a.tokens * a.ldd;
        } else {
            a.weights += a.tokens * a.r.k;
        }
    }
}
template <typename T>
void route_of(const RouteArgs &a, bool wide, bool backward, hipStream_t s) {
    const uint32_t E = a.r.experts;
    if (E <= 64) route_as<T, 1>(a, wide, backward, s);
    else if (E <= 128) route_as<T, 2>(a, wide, backward, s);
    else if (E <= 256) route_as<T, 4>(a, wide, backward, s);
    else if (E <= 512) route_as<T, 8>(a, wide, backward, s);
    else route_as<T, 16>(a, wide, backward, s);
}

}  // namespace

cbk_status launch_route(const cbk_router &r, const void *logits, int dtype, uint64_t ld, uint64_t tokens, const float *bias,
                        int32_t *experts, float *weights, hipStream_t s) {
    RouteArgs a{};
    a.r = r;
    a.logits = logits;
    a.ld = ld;
    a.tokens = tokens;
    a.bias = bias;
    a.experts = experts;
    a.weights = weights;
    const bool wide = bias || (r.groups > 1 && r.group_top == 2);
    if (dtype == CBK_F32) route_of<float>(a, wide, false, s);
    else route_of<uint16_t>(a, wide, false, s);
    return launched();
}

cbk_status launch_route_bwd(const cbk_router &r, const void *logits, int dtype, uint64_t ld, uint64_t tokens,
                            const int32_t *experts, const float *dweights, void *dlogits, uint64_t ldd, hipStream_t s) {
    RouteArgs a{};
    a.r = r;
    a.logits = logits;
    a.ld = ld;
    a.tokens = tokens;
    a.experts = const_cast<int32_t *>(experts);
    a.dweights = dweights;
    a.dlogits = dlogits;
    a.ldd = ldd;
    if (dtype == CBK_F32) route_of<float>(a, false, true, s);
    else route_of<uint16_t>(a, false, true, s);
    return launched();
}

// ------------------------------------------------------------------------------- the block of experts
namespace {

template <typename T>
T *at(void *ws, uint64_t offset) { return reinterpret_cast<T *>(static_cast<unsigned char *>(ws) + offset); }

bool vec16(const void *p, uint64_t ld) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld % 8 == 0; }

// What the products read of a matrix of tokens: itself where whole 64-wide slices of its rows can be copied 16
// bytes at a time and the chunk's rows lie within 31 bits of bytes, else a padded copy in the workspace.
const uint16_t *token_rows(const uint16_t *X, uint64_t ld, uint64_t T, uint64_t K, uint64_t Kp, uint16_t *P, PadArgs &pad, uint32_t &lda) {
    if (K == Kp && vec16(X, ld) && T * ld * 2 < 0x7F000000u) {
        lda = static_cast<uint32_t>(ld);
        return X;
    }
    lda = static_cast<uint32_t>(Kp);
    pad = PadArgs{X, ld, T, static_cast<uint32_t>(K), lda, P};
    return P;
}

cbk_status gather(GatherArgs g, const float *S, uint64_t split_stride, uint32_t splits, uint64_t ldS, uint64_t width, hipStream_t s) {
    g.S = S;
    g.split_stride = split_stride;
    g.splits = splits;
    g.lds = static_cast<uint32_t>(ldS);
    g.width = static_cast<uint32_t>(width);
    g.vec = (reinterpret_cast<uintptr_t>(g.Y) & 7) == 0 && g.ldy % 4 == 0 ? 1u : 0u;
    g.blocks = static_cast<uint32_t>((width + 1023) / 1024);
    const uint32_t rows = static_cast<uint32_t>(std::min<uint64_t>(g.tokens, 32768));
    const dim3 grid(g.blocks + (g.dweights ? 1 : 0), rows, static_cast<uint32_t>((g.tokens + rows - 1) / rows));
    hipLaunchKernelGGL(k_gather, grid, dim3(256), 0, s, g);
    return launched();
}

}  // namespace

cbk_status launch_experts(const cbk_experts &ex, const ExPlan &pl, int act, const uint16_t *X, uint64_t ldx, uint64_t T,
                          const int32_t *experts, const float *weights, uint32_t k, const uint16_t *dY, uint64_t lddy,
                          uint16_t *out, uint64_t ldo, float *dweights, void *ws, hipStream_t s) {
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess) return CBK_E_HIP;
    if (static_cast<uint32_t>(dev) != ex.device) return CBK_E_INVALID;
    for (uint64_t c = 0; c < T; c += pl.Tc) {
        const uint64_t n = std::min(pl.Tc, T - c);
        SortArgs so{};
        so.experts = experts + c * k;
        so.slots = static_cast<uint32_t>(n * k);
        so.k = k;
        so.count = ex.count;
        so.tile = pl.tile;
        so.unit = pl.tile / 4;
        so.token_of = at<uint32_t>(ws, pl.token_of);
        so.slot_of = at<uint32_t>(ws, pl.slot_of);
        so.place_of = at<int32_t>(ws, pl.place_of);
        so.tiles = at<ExTile>(ws, pl.tiles);
        so.ntiles = at<uint32_t>(ws, pl.ntiles);
        if (pl.one) {
            so.place_of = nullptr;
            so.tiles = nullptr;
        }
        uint32_t ldxa, ldya = 0;
        const uint16_t *Xa = token_rows(X + c * ldx, ldx, n, ex.cols, pl.Kp, at<uint16_t>(ws, pl.xpack), so.pad[0], ldxa);
        const uint16_t *Ya = dY ? token_rows(dY + c * lddy, lddy, n, ex.out, pl.Op, at<uint16_t>(ws, pl.ypack), so.pad[1], ldya) : nullptr;
        uint64_t pads = 0;  // groups of four numbers
        for (const PadArgs &pad : so.pad) pads = std::max(pads, pad.X ? pad.T * (pad.Kp / 4) : 0);
        cbk_status st = CBK_OK;
        if (so.tiles || pads > 0) {
            if (!allow_lds_once<SortArgs>(k_sort, kLdsLimit / 2)) return CBK_E_HIP;  // 64 KB of counts, and a little
            const uint32_t blocks = static_cast<uint32_t>(1 + std::min<uint64_t>((pads + 64 * kSortWaves - 1) / (64 * kSortWaves), 2048));
            hipLaunchKernelGGL(k_sort, dim3(blocks), dim3(64 * kSortWaves), kSortWaves * ex.count * 4, s, so);
            st = launched();
            if (st != CBK_OK) return st;
        }

        ExArgs a{};
        a.tiles = so.tiles;
        a.ntiles = so.ntiles;
        a.token_of = so.token_of;
        a.slot_of = so.slot_of;
        a.experts = so.experts;
        a.k = k;
        a.count = ex.count;
        a.weights = weights + c * k;
        a.act = act;
        a.rows = static_cast<uint32_t>(ex.rows);
        a.Fp = static_cast<uint32_t>(pl.Fp);
        const ExTensor *table = static_cast<const ExTensor *>(ex.buffer);
        GatherArgs by_token{};
        by_token.k = k;
        by_token.tokens = n;
        by_token.place_of = so.place_of;
        by_token.experts = so.experts;
        by_token.count = ex.count;
        by_token.Y = out + c * ldo;
        by_token.ldy = ldo;
        if (!dY) {
            // H, and its product with down
            ExArgs h = a;
            h.t[0] = table;
            h.t[1] = table + ex.count;
            h.A = Xa;
            h.lda = ldxa;
            h.H = at<uint16_t>(ws, pl.h);
            st = ex_hidden(h, pl, ex, false, s);
            if (st != CBK_OK) return st;
            ExArgs d = a;
            d.t[0] = table + 2 * ex.count;
            d.A = h.H;
            d.lda = static_cast<uint32_t>(pl.Fp);
            d.by_slot = 1;
            d.scaled = 1;
            d.S = at<float>(ws, pl.s);
            st = ex_down(d, pl, ex, s);
            if (st != CBK_OK) return st;
            st = gather(by_token, d.S, pl.s_stride, pl.split_down, pl.ldO, ex.out, s);
            if (st != CBK_OK) return st;
            continue;
        }
        // D = dY . down, then dG and dU, then their product with gate and up
        ExArgs d = a;
        d.t[0] = table + 2 * ex.count;
        d.A = Ya;
        d.lda = ldya;
        d.S = at<float>(ws, pl.d);
        st = ex_down_t(d, pl, ex, s);
        if (st != CBK_OK) return st;
        ExArgs g = a;
        g.t[0] = table;
        g.t[1] = table + ex.count;
        g.A = Xa;
        g.lda = ldxa;
        g.D = d.S;
        g.G = at<uint16_t>(ws, pl.g);
        g.dw = at<float>(ws, pl.dw);
        st = ex_hidden(g, pl, ex, true, s);
        if (st != CBK_OK) return st;
        ExArgs x = a;
        x.t[0] = table;
        x.t[1] = table + ex.count;
        x.A = g.G;
        x.lda = static_cast<uint32_t>(2 * pl.Fp);
        x.by_slot = 1;
        x.S = at<float>(ws, pl.s);
        st = ex_dx(x, pl, ex, s);
        if (st != CBK_OK) return st;
        if (dweights) {
            by_token.parts = pl.dw_parts;
            by_token.dw = g.dw;
            by_token.dweights = dweights + c * k;
        }
        st = gather(by_token, x.S, pl.s_stride, pl.split_x, pl.ldK, ex.cols, s);
        if (st != CBK_OK) return st;
    }
    return CBK_OK;
}

cbk_status experts_table(const cbk_tensor *gate, const cbk_tensor *up, const cbk_tensor *down, uint32_t count, void *buffer,
                         uint32_t &device) {
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess) return CBK_E_HIP;
    device = static_cast<uint32_t>(dev);
    ExTensor part[64];
    const cbk_tensor *kinds[3] = {gate, up, down};
    for (uint32_t kind = 0; kind < 3; ++kind)
        for (uint32_t e = 0; e < count; e += 64) {
            const uint32_t n = std::min<uint32_t>(64, count - e);
            for (uint32_t i = 0; i < n; ++i) {
                const cbk_tensor &t = kinds[kind][e + i];
                part[i] = ExTensor{t.words, t.codebook, t.b ? cbk_words_for(t.rows * t.cols, t.b) * 4 : 0, t.U, t.b};
            }
            if (hipMemcpy(static_cast<ExTensor *>(buffer) + static_cast<uint64_t>(kind) * count + e, part, n * sizeof(ExTensor),
                          hipMemcpyHostToDevice) != hipSuccess)
                return CBK_E_HIP;
        }
    return CBK_OK;
}

}  // namespace cbk
