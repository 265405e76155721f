// Token sampling from given random numbers (include/tree_sample.h).
//
// A bf16 row of any length has few distinct values, and everything the draw needs
// -- the k-th token, the prefix that reaches p, the token at u -- depends on how
// often each value occurs.  So one pass over the logits counts values in shared
// memory (one bin per bf16 value, in descending order), and the rest works on the
// counts: a weight is computed once per value, not once per token, precisely
// enough to be an integer, and sums of integers do not depend on their order.
//
//   bins      value 0 and both signs of 2^-32 <= |x| < 2^16: 12,289 counters, 48 KB.
//             Lower values count as zero weight when the row's maximum and the
//             temperature allow it (masks, -inf); any other value outside sends the
//             row through the full range in windows, several passes, by one CTA.
//   groups    32 bins; a group's count and mass are one entry of a block-wide prefix
//             sum, a search finds the group, then one warp the bin.
//   cluster   C CTAs count a slice of the row each; each then weighs a share of the
//             groups (counts summed over the C histograms through distributed shared
//             memory), and the first one searches.
//   index     the r-th token with the drawn value, found by the CTA whose slice holds
//             it.
//
// Memory-bound in principle (2 bytes per logit); in practice paced by the shared
// memory atomics and the few cluster barriers of a short row.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "kernels.h"
#include "plan.h"
#include "tree_sample.h"

namespace cg = cooperative_groups;

namespace treeattn {

namespace {

constexpr int kNT = 256;                       // threads per CTA
constexpr int kBase = (127 - 32) << 7;         // bits of 2^-32
constexpr int kSide = 48 << 7;                 // values per sign: 2^-32 .. 2^16
constexpr int kBins = 2 * kSide + 1;
constexpr int kGroups = (kBins + 31) / 32;
constexpr int kWindow = 12288;                 // bins per window of the full range
constexpr int kWindows = (65536 + kWindow - 1) / kWindow;
constexpr int kPer = (kGroups + kNT - 1) / kNT;   // groups per thread in the prefix sums
constexpr int kOneBits = 45;                   // weight of the largest logit: 2^45
constexpr int64_t kMaxVocab = 262144;          // 2^18: sums stay below 2^63

struct Params {
    const uint16_t* logits;
    int64_t stride;
    int64_t vocab;
    const float* u;
    tree_attn_sampling_t s;
    int32_t* tokens;
    float* logprobs;
    int* status;
};

// round(2^61 * 2^(j / 64)), j = -32 .. 32
__constant__ uint64_t kPow[65] = {
    0x16a09e667f3bcc91ull, 0x16dfb23c651a2ef2ull, 0x171f75e8ec5f73ddull, 0x175feb564267c8bfull,
    0x17a11473eb0186d8ull, 0x17e2f336cf4e6210ull, 0x182589994cce128bull, 0x1868d99b4492ec81ull,
    0x18ace5422aa0db5cull, 0x18f1ae991577362cull, 0x193737b0cdc5e4f4ull, 0x197d829fde4e4f8cull,
    0x19c49182a3f0901cull, 0x1a0c667b5de564b3ull, 0x1a5503b23e255c8bull, 0x1a9e6b5579fdbf44ull,
    0x1ae89f995ad3ad5full, 0x1b33a2b84f15faf7ull, 0x1b7f76f2fb5e46ebull, 0x1bcc1e904bc1d224ull,
    0x1c199bdd85529c22ull, 0x1c67f12e57d14b4aull, 0x1cb720dcef906915ull, 0x1d072d4a07897b8dull,
    0x1d5818dcfba48726ull, 0x1da9e603db328571ull, 0x1dfc97337b9b5eb9ull, 0x1e502ee78b3ff627ull,
    0x1ea4afa2a490d986ull, 0x1efa1bee615a2777ull, 0x1f50765b6e454067ull, 0x1fa7c1819e90d82full,
    0x2000000000000000ull, 0x2059347cef00c1ddull, 0x20b361a62b0ae876ull, 0x210e8a30eb379012ull,
    0x216ab0d9f3121ec5ull, 0x21c7d865a7a34404ull, 0x222603a024b6a14aull, 0x2285355d525bbf67ull,
    0x22e57078faa2f5baull, 0x2346b7d6df96ea79ull, 0x23a90e62d17354f0ull, 0x240c7710c519ac77ull,
    0x2470f4dceac470ceull, 0x24d68acbc4f9ba4bull, 0x253d3bea3fbdc258ull, 0x25a50b4dc8061680ull,
    0x260dfc14636e2a5cull, 0x26781164c82dfe99ull, 0x26e34e6e7553954eull, 0x274fb669cb3fedd4ull,
    0x27bd4c982468446bull, 0x282c1443ee5c53f1ull, 0x289c10c0c3125a06ull, 0x290d456b8279a028ull,
    0x297fb5aa6c544e3bull, 0x29f364ed3a594d5aull, 0x2a6856ad3a9f03beull, 0x2ade8e6d6a4fb4ceull,
    0x2b560fba90a852b2ull, 0x2bcede2b5a4290ddull, 0x2c48fd6074ab0964ull, 0x2cc47104aa444922ull,
    0x2d413cccfe779921ull,
};

// log2(e) / T as a pair of floats; for temperatures near the ends of fp32's range a
// power of two moves from the rate to the difference (`pre`), so that neither part of
// the pair leaves the normal numbers.
struct Rate {
    float hi, lo, pre;
};

__device__ __forceinline__ Rate rate_of(float T) {
    Rate c;
    c.pre = T < 0x1p-60f ? 0x1p64f : T > 0x1p60f ? 0x1p-64f : 1.f;
    const double x = 1.4426950408889634 / ((double)T * (double)c.pre);
    c.hi = (float)x;
    c.lo = (float)(x - (double)c.hi);
    return c;
}

// 2^45 * 2^(d * c), d = x - top <= 0: n + j/64 + r = d * c in pairs of floats (48 bits),
// 2^(j/64) from the table, 2^r - 1 by its series (|r ln 2| < 0.0055: five terms), then
// integers.
__device__ __forceinline__ uint64_t weight(float x, float top, Rate c) {
    const float diff = x - top;
    if (diff == 0.f) return 1ull << kOneBits;
    // the rounding error of x - top
    const float b = diff - x;
    const float dl = ((x - (diff - b)) - (top + b)) * c.pre;
    const float d = diff * c.pre;
    const float y = d * c.hi;
    if (!(y > -64.f)) return 0;
    const float yl = fmaf(d, c.hi, -y) + fmaf(d, c.lo, dl * c.hi);
    const float n = rintf(y);
    const float f = y - n;                       // exact
    const float j = rintf(f * 64.f);
    const float r = fmaf(j, -0.015625f, f);      // exact
    const float rh = r + yl;
    const float rl = yl - (rh - r);
    // z = r ln 2
    constexpr float kLh = 0x1.62e430p-1f, kLl = -0x1.05c610p-29f;
    const float z = rh * kLh;
    const float zl = fmaf(rh, kLh, -z) + fmaf(rh, kLl, rl * kLh);
    const float t = z * z * fmaf(z, fmaf(z, fmaf(z, 1.f / 120.f, 1.f / 24.f), 1.f / 6.f), 0.5f);
    const float e = z + t;
    const float el = (t - (e - z)) + zl;
    const int64_t E = __float2ll_rn(e * 0x1p62f) + __float2ll_rn(el * 0x1p62f);
    const uint64_t p = kPow[(int)j + 32];
    const uint64_t w = p + 4 * (uint64_t)__mul64hi((int64_t)p, E);
    const int shift = 61 - kOneBits - (int)n;
    if (shift > 62) return 0;
    return (w + (1ull << (shift - 1))) >> shift;
}

// a * s for a non-negative float a < 2: the integer part, and whether something is left
__device__ __forceinline__ uint64_t times(float a, uint64_t s, bool& rest) {
    rest = false;
    if (!(a > 0.f) || !s) return 0;
    const uint32_t bits = __float_as_uint(a);
    int e = (int)(bits >> 23);
    const uint64_t m = (e ? 0x800000u : 0u) | (bits & 0x7fffffu);
    const int shift = 150 - (e ? e : 1);         // a = m * 2^-shift
    const uint64_t lo = m * s, hi = __umul64hi(m, s);
    if (shift <= 0) return lo << -shift;
    if (shift < 64) {
        rest = (lo & ((1ull << shift) - 1)) != 0;
        return (lo >> shift) | (hi << (64 - shift));
    }
    if (shift == 64) {
        rest = lo != 0;
        return hi;
    }
    rest = true;
    if (shift >= 128) return 0;
    rest = lo != 0 || (hi & ((1ull << (shift - 64)) - 1)) != 0;
    return hi >> (shift - 64);
}

struct Shared {
    uint32_t hist[kGroups * 32];
    uint32_t gcnt[kGroups], pcnt[kGroups];       // tokens of a group, of the groups before it
    uint64_t gmass[kGroups], pmass[kGroups];     // their weight
    uint64_t one[kNT / 32];                      // untempered weight, by warp
    uint32_t wcnt[kNT / 32];
    uint64_t wmass[kNT / 32];
    float top;
    uint32_t flags;                              // of the slice
    // the leader's search
    uint32_t tot_cnt;
    uint64_t tot_mass, tot_one;
    int found;
    uint32_t f_cnt, f_rank;
    uint64_t f_mass;
    int f_bin;
    // the index search
    int key;                                     // bits of the drawn value, or -1
    uint32_t rank, owner;
};

enum { kNaN = 1, kRare = 2, kLow = 4 };

// Bin of a bf16 value, or -1 with the reason in `flags`.
__device__ __forceinline__ int bin_of(uint32_t b, uint32_t& flags) {
    const uint32_t mag = b & 0x7fffu, t = mag - kBase;
    if (t < (uint32_t)kSide) return (b & 0x8000u) ? kSide + 1 + (int)t : kSide - 1 - (int)t;
    if (mag == 0) return kSide;
    flags |= mag > 0x7f80u ? kNaN : (t < 0x8000u && (b & 0x8000u)) ? kLow : kRare;
    return -1;
}

// bits of the value of a bin; win < 0: the short range, else window `win` of the full one
__device__ __forceinline__ uint32_t bits_of(int bin, int win) {
    if (win < 0) return bin < kSide ? kBase + (kSide - 1 - bin) : bin == kSide ? 0u : 0x8000u | (kBase + (bin - kSide - 1));
    const uint32_t o = 65535u - (uint32_t)(win * kWindow + bin);
    return o & 0x8000u ? o ^ 0x8000u : o ^ 0xffffu;
}

// Applies f(bits) to elements [lo, hi) of a row, 16 bytes at a time.
template <typename F>
__device__ __forceinline__ void each(const uint16_t* row, int64_t lo, int64_t hi, F f) {
    const uint16_t* a = row + lo;
    const int64_t n = hi - lo;
    const int64_t head = min(n, (int64_t)((16 - (reinterpret_cast<uintptr_t>(a) & 15)) & 15) / 2);
    if ((int64_t)threadIdx.x < head) f(a[threadIdx.x]);
    const uint4* v = reinterpret_cast<const uint4*>(a + head);
    const int64_t nv = (n - head) / 8;
    auto one = [&](uint32_t w) {
        f(w & 0xffffu);
        f(w >> 16);
    };
    auto vec = [&](const uint4& x) {
        one(x.x);
        one(x.y);
        one(x.z);
        one(x.w);
    };
    int64_t i = threadIdx.x;
    for (; i + 3 * kNT < nv; i += 4 * kNT) {
        const uint4 x0 = __ldg(v + i), x1 = __ldg(v + i + kNT), x2 = __ldg(v + i + 2 * kNT), x3 = __ldg(v + i + 3 * kNT);
        vec(x0);
        vec(x1);
        vec(x2);
        vec(x3);
    }
    for (; i < nv; i += kNT) vec(__ldg(v + i));
    const int64_t done = head + nv * 8;
    if ((int64_t)threadIdx.x < n - done) f(a[done + threadIdx.x]);
}

template <typename T>
__device__ __forceinline__ T warp_sum(T x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}
template <typename T>
__device__ __forceinline__ T warp_scan(T x) {    // inclusive
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    return x;
}

// The counts of one bin over the cluster's histograms.
struct Counts {
    const uint32_t* h[8];
    int n;
    __device__ __forceinline__ uint32_t operator()(int bin) const {
        uint32_t c = 0;
        for (int i = 0; i < n; ++i) c += h[i][bin];
        return c;
    }
};

// Weighs groups [g0, g1): count and mass of each into `to`'s arrays, and this warp's
// share of the untempered mass.
__device__ void weigh(const Counts& counts, int g0, int g1, int win, float top, Rate c, bool same, Shared* to,
                      uint64_t& one) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Rate unit = {1.44269502162933349609f, 1.92596299112661746887e-8f, 1.f};   // log2(e)
    for (int g = g0 + warp; g < g1; g += kNT / 32) {
        const int bin = 32 * g + lane;
        const uint32_t n = counts(bin);
        uint32_t cn = 0;
        uint64_t m = 0;
        if (__any_sync(0xffffffffu, n)) {
            if (n) {
                const float x = __uint_as_float(bits_of(bin, win) << 16);
                const uint64_t w = weight(x, top, c);
                m = n * w;
                one += same ? m : n * weight(x, top, unit);
            }
            cn = warp_sum(n);
            m = warp_sum(m);
        }
        if (lane == 0) {
            to->gcnt[g] = cn;
            to->gmass[g] = m;
        }
    }
}

// Prefix sums over the groups, starting from (cnt, mass); all threads.
__device__ void prefix(Shared& S, uint32_t cnt, uint64_t mass) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t c[kPer], ct = 0;
    uint64_t m[kPer], mt = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int g = threadIdx.x * kPer + i;
        c[i] = g < kGroups ? S.gcnt[g] : 0;
        m[i] = g < kGroups ? S.gmass[g] : 0;
        ct += c[i];
        mt += m[i];
    }
    const uint32_t ci = warp_scan(ct);
    const uint64_t mi = warp_scan(mt);
    if (lane == 31) {
        S.wcnt[warp] = ci;
        S.wmass[warp] = mi;
    }
    __syncthreads();
    uint32_t pc = cnt + ci - ct;
    uint64_t pm = mass + mi - mt;
    for (int w = 0; w < warp; ++w) {
        pc += S.wcnt[w];
        pm += S.wmass[w];
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int g = threadIdx.x * kPer + i;
        if (g < kGroups) {
            S.pcnt[g] = pc;
            S.pmass[g] = pm;
        }
        pc += c[i];
        pm += m[i];
    }
    if (threadIdx.x == kNT - 1) {
        S.tot_cnt = pc;
        S.tot_mass = pm;
    }
    __syncthreads();
}

// The token at which the cumulated mass reaches `mass` (by_mass), or the cnt-th token:
// its 1-based position, value bin, place among equal values, and the cumulated mass up
// to it.  False when it lies behind this window's groups.  All threads.
__device__ bool locate(Shared& S, const Counts& counts, int win, float top, Rate c, bool by_mass, uint64_t mass,
                       uint32_t cnt) {
    if (threadIdx.x == 0) S.found = -1;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int g = threadIdx.x * kPer + i;
        if (g >= kGroups) continue;
        const bool in = by_mass ? S.pmass[g] < mass && mass <= S.pmass[g] + S.gmass[g]
                                : S.pcnt[g] < cnt && cnt <= S.pcnt[g] + S.gcnt[g];
        if (in) S.found = g;
    }
    __syncthreads();
    const int g = S.found;
    if (g < 0) return false;
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x, bin = 32 * g + lane;
        const uint32_t n = counts(bin);
        const uint64_t w = n ? weight(__uint_as_float(bits_of(bin, win) << 16), top, c) : 0;
        const uint32_t ci = warp_scan(n) + S.pcnt[g];
        const uint64_t mi = warp_scan(n * w) + S.pmass[g];
        const uint32_t cb = ci - n;
        const uint64_t mb = mi - n * w;
        const bool in = by_mass ? mb < mass && mass <= mi : cb < cnt && cnt <= ci;
        if (in) {
            const uint32_t k = by_mass ? (uint32_t)((mass - mb + w - 1) / w) : cnt - cb;   // 1 .. n
            S.f_cnt = cb + k;
            S.f_mass = mb + k * w;
            S.f_bin = bin;
            S.f_rank = k - 1;
        }
    }
    __syncthreads();
    return true;
}

// First token at which the cumulated mass exceeds what the row's u asks for: cuts and
// draw over the windows of a row.  `load(win)` puts a window's groups and prefix sums
// (from a carry) in place.  Leader CTA, all threads; leaves the draw in S.f_bin,
// S.f_rank and returns its window, or -1 when nothing has weight.
template <typename Load>
__device__ int draw(Shared& S, const Counts& counts, int first, int windows, float top, Rate c, int32_t k, float p,
                    float min_p, float u, bool greedy, Load load) {
    // total count and mass; the mass of the first k tokens
    uint64_t kept = 0, all = 0;
    uint32_t n = 0, total = 0;
    bool cut = false;
    if (greedy) {
        k = 1;
        p = 1.f;
        min_p = 0.f;
        u = 0.f;
    }
    for (int w = 0; w < windows; ++w) {
        load(first + w, total, all);
        if (k > 0 && !cut && locate(S, counts, first + w, top, c, false, 0, (uint32_t)k)) {
            cut = true;
            kept = S.f_mass;
        }
        total = S.tot_cnt;
        all = S.tot_mass;
        __syncthreads();
    }
    if (!cut) kept = all;
    n = cut ? (uint32_t)k : total;
    // the shortest prefix that reaches p
    if (p < 1.f) {
        bool rest;
        uint64_t need = times(p, kept, rest) + 0;
        need = max(need + (rest ? 1 : 0), (uint64_t)1);
        uint32_t cc = 0;
        uint64_t mm = 0;
        for (int w = 0; w < windows; ++w) {
            if (windows > 1) load(first + w, cc, mm);
            if (locate(S, counts, first + w, top, c, true, need, 0)) {
                n = min(n, S.f_cnt);
                break;
            }
            cc = S.tot_cnt;
            mm = S.tot_mass;
            __syncthreads();
        }
    }
    // tokens of weight at least min_p: the first token below it ends the prefix
    if (min_p > 0.f) {
        bool rest;
        uint64_t least = times(fminf(min_p, 1.f), 1ull << kOneBits, rest);
        least += rest ? 1 : 0;
        uint32_t cc = 0, many = 0;
        uint64_t mm = 0;
        for (int w = 0; w < windows; ++w) {
            if (windows > 1) load(first + w, cc, mm);
            uint32_t mine = 0;
            for (int bin = threadIdx.x; bin < kGroups * 32; bin += kNT) {
                const uint32_t x = S.gcnt[bin / 32] ? counts(bin) : 0;
                if (x && weight(__uint_as_float(bits_of(bin, first + w) << 16), top, c) >= least) mine += x;
            }
            mine = warp_sum(mine);
            if ((threadIdx.x & 31) == 0) S.wcnt[threadIdx.x >> 5] = mine;
            __syncthreads();
            for (int i = 0; i < kNT / 32; ++i) many += S.wcnt[i];
            cc = S.tot_cnt;
            mm = S.tot_mass;
            __syncthreads();
        }
        n = min(n, many);
    }
    // mass of the first n tokens, then the draw
    uint64_t sum = kept;
    if (!(cut && n == (uint32_t)k) && n < total) {
        uint32_t cc = 0;
        uint64_t mm = 0;
        for (int w = 0; w < windows; ++w) {
            if (windows > 1) load(first + w, cc, mm);
            if (locate(S, counts, first + w, top, c, false, 0, n)) {
                sum = S.f_mass;
                break;
            }
            cc = S.tot_cnt;
            mm = S.tot_mass;
            __syncthreads();
        }
    }
    if (!sum) return -1;
    bool rest;
    uint64_t at = u < 1.f ? times(u, sum, rest) + 1 : sum;   // cumulated mass > u * sum
    at = min(at, sum);
    uint32_t cc = 0;
    uint64_t mm = 0;
    for (int w = 0; w < windows; ++w) {
        if (windows > 1) load(first + w, cc, mm);
        if (locate(S, counts, first + w, top, c, true, at, 0)) return first + w;
        cc = S.tot_cnt;
        mm = S.tot_mass;
        __syncthreads();
    }
    return -1;
}

__global__ void __launch_bounds__(kNT, 3) sample_kernel(const Params p) {
    extern __shared__ __align__(16) uint8_t raw[];
    Shared& S = *reinterpret_cast<Shared*>(raw);
    cg::cluster_group cluster = cg::this_cluster();
    const int C = (int)cluster.num_blocks(), me = (int)cluster.block_rank();
    const int64_t r = blockIdx.x / C;
    const uint16_t* row = p.logits + r * p.stride;
    const int64_t lo = p.vocab * me / C, hi = p.vocab * (me + 1) / C;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i = threadIdx.x; i < kGroups * 32 / 4; i += kNT) reinterpret_cast<uint4*>(S.hist)[i] = make_uint4(0, 0, 0, 0);
    grid_dep_wait();
    grid_dep_launch();
    const float T = p.s.temperatures ? p.s.temperatures[r] : p.s.temperature;
    const int32_t k = p.s.top_ks ? p.s.top_ks[r] : p.s.top_k;
    const float top_p = p.s.top_ps ? p.s.top_ps[r] : p.s.top_p;
    const float min_p = p.s.min_ps ? p.s.min_ps[r] : p.s.min_p;
    const float u = p.u[r];
    __syncthreads();

    // ---- count the slice ----------------------------------------------------------
    uint32_t flags = 0;
    float top = -INFINITY;
    each(row, lo, hi, [&](uint32_t b) {
        const int bin = bin_of(b, flags);
        if (bin >= 0) atomicAdd(&S.hist[bin], 1u);
        top = fmaxf(top, __uint_as_float(b << 16));
    });
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        flags |= __shfl_xor_sync(0xffffffffu, flags, o);
    }
    if (lane == 0) {
        S.wcnt[warp] = flags;
        S.one[warp] = __float_as_uint(top);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kNT / 32; ++w) {
            flags |= S.wcnt[w];
            top = fmaxf(top, __uint_as_float((uint32_t)S.one[w]));
        }
        S.flags = flags;
        S.top = top;
    }
    cluster.sync();

    // ---- the row's maximum, and what kind of row it is --------------------------------
    Counts counts;
    counts.n = C;
    flags = 0;
    top = -INFINITY;
    for (int i = 0; i < C; ++i) {
        const Shared* other = cluster.map_shared_rank(&S, i);
        counts.h[i] = other->hist;
        flags |= other->flags;
        top = fmaxf(top, other->top);
    }
    top += 0.f;                                     // -0 counts as 0
    const bool bad_params = !(T >= 0.f) || isinf(T) || top_p != top_p || min_p != min_p || u != u;
    const bool bad = bad_params || (flags & kNaN) || isinf(top);
    const bool greedy = T == 0.f;
    // Values below -2^16 have no weight beside a maximum of at least -2^15 when
    // 2^15 / T is above 46 ln 2.
    const bool slow = (flags & kRare) || ((flags & kLow) && !(top >= -32768.f && T <= 512.f));
    const Rate c = rate_of(greedy ? 1.f : T);
    const bool same = greedy || T == 1.f;

    Shared* leader = cluster.map_shared_rank(&S, 0);
    uint64_t one = 0;
    if (!bad && !slow) weigh(counts, kGroups * me / C, kGroups * (me + 1) / C, -1, top, c, same, leader, one);
    one = warp_sum(one);
    if (lane == 0) S.one[warp] = one;
    cluster.sync();

    if (me == 0) {
        int win = -1, key = -1;
        bool drawn = false;
        uint32_t rank = 0;
        uint64_t one_all = 0;
        if (!bad && !slow) {
            for (int i = 0; i < C; ++i) {
                const Shared* other = cluster.map_shared_rank(&S, i);
                for (int w = 0; w < kNT / 32; ++w) one_all += other->one[w];
            }
            prefix(S, 0, 0);
            win = draw(S, counts, -1, 1, top, c, k, top_p, min_p, u, greedy,
                       [&](int, uint32_t, uint64_t) {});
            drawn = true;
        } else if (!bad) {
            // the full range, window by window, counted by this CTA alone
            counts.n = 1;
            bool first = true;
            uint64_t sum = 0;
            auto load = [&](int w, uint32_t cnt, uint64_t mass) {
                __syncthreads();
                for (int i = threadIdx.x; i < kGroups * 32; i += kNT) S.hist[i] = 0;
                __syncthreads();
                each(row, 0, p.vocab, [&](uint32_t b) {
                    b = b == 0x8000u ? 0u : b;
                    const uint32_t o = 65535u - (b & 0x8000u ? b ^ 0xffffu : b ^ 0x8000u);
                    const uint32_t at = o - (uint32_t)(w * kWindow);
                    if (at < (uint32_t)kWindow && b != 0xff80u) atomicAdd(&S.hist[at], 1u);
                });
                __syncthreads();
                uint64_t part = 0;
                weigh(counts, 0, kGroups, w, top, c, same, &S, part);
                if (first) {
                    sum += part;
                    first = w + 1 < kWindows;
                }
                __syncthreads();
                prefix(S, cnt, mass);
            };
            win = draw(S, counts, 0, kWindows, top, c, k, top_p, min_p, u, greedy, load);
            drawn = win >= 0;
            sum = warp_sum(sum);
            if (lane == 0) S.one[warp] = sum;
            __syncthreads();
            for (int w = 0; w < kNT / 32; ++w) one_all += S.one[w];
        }
        if (drawn) {
            key = (int)bits_of(S.f_bin, win);
            rank = S.f_rank;
        }
        if (threadIdx.x == 0) {
            if (bad_params) report_status(p.status, TREE_ATTN_ERR_INVALID_SAMPLING);
            if (key < 0) p.tokens[r] = -1;
            if (p.logprobs) {
                const float x = __uint_as_float((uint32_t)key << 16);
                p.logprobs[r] = key < 0 ? __int_as_float(0x7fc00000)
                                        : (x - top) - log1pf((float)(one_all - (1ull << kOneBits)) * 0x1p-45f);
            }
            // the slice that holds the rank-th token of this value
            uint32_t owner = 0;
            if (key >= 0 && win < 0)
                while (owner + 1 < (uint32_t)C && rank >= counts.h[owner][S.f_bin]) rank -= counts.h[owner++][S.f_bin];
            for (int i = 0; i < C; ++i) {
                Shared* to = cluster.map_shared_rank(&S, i);
                to->key = key;
                to->rank = rank;
                to->owner = win < 0 ? owner : 0xffffffffu;
            }
        }
    }
    cluster.sync();

    // ---- the index -------------------------------------------------------------------
    const int key = S.key;
    const bool whole = S.owner == 0xffffffffu;      // the leader searches the whole row
    if (key < 0 || (whole ? me != 0 : (int)S.owner != me)) return;
    const int64_t a = whole ? 0 : lo, b = whole ? p.vocab : hi;
    // warps take contiguous parts; a warp's matches, then the place inside the warp's part
    const int64_t s0 = a + (b - a) * warp / (kNT / 32), s1 = a + (b - a) * (warp + 1) / (kNT / 32);
    auto hit = [&](int64_t i) {
        const uint32_t x = i < s1 ? row[i] : 0xffffffffu;
        return i < s1 && (x == (uint32_t)key || (key == 0 && x == 0x8000u));
    };
    uint32_t n = 0;
    for (int64_t i = s0 + lane; i < s1; i += 32) n += hit(i);
    n = warp_sum(n);
    if (lane == 0) S.wcnt[warp] = n;
    __syncthreads();
    uint32_t before = 0;
    for (int w = 0; w < warp; ++w) before += S.wcnt[w];
    const uint32_t want = S.rank;
    if (want < before || want >= before + n) return;
    uint32_t left = want - before;
    for (int64_t i = s0; i < s1; i += 32) {
        const uint32_t m = __ballot_sync(0xffffffffu, hit(i + lane));
        if (left < (uint32_t)__popc(m)) {
            if (lane == (int)__fns(m, 0, (int)left + 1)) p.tokens[r] = (int32_t)(i + lane);
            return;
        }
        left -= __popc(m);
    }
}

}  // namespace

}  // namespace treeattn

using namespace treeattn;

extern "C" int tree_attn_sample(const void* logits, int64_t row_stride, int64_t n_rows, int64_t vocab, const float* u,
                                const tree_attn_sampling_t* s, int32_t* tokens, float* logprobs, void* stream) {
    if (n_rows < 0 || vocab < 1 || !s) return TREE_ATTN_ERR_INVALID_ARG;
    if (vocab > kMaxVocab) return TREE_ATTN_ERR_TOO_LARGE;
    if (row_stride < vocab) return TREE_ATTN_ERR_INVALID_ARG;
    if (n_rows == 0) return TREE_ATTN_OK;
    if (!logits || !u || !tokens) return TREE_ATTN_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(logits) & 1u) return TREE_ATTN_ERR_ALIGNMENT;
    for (const void* x : {(const void*)u, (const void*)tokens, (const void*)logprobs, (const void*)s->temperatures,
                          (const void*)s->top_ks, (const void*)s->top_ps, (const void*)s->min_ps})
        if (reinterpret_cast<uintptr_t>(x) & 3u) return TREE_ATTN_ERR_ALIGNMENT;
    int dev, *status;
    int st;
    if ((st = current_device(&dev)) || (st = get_status_ptr(dev, &status))) return st;
    // CTAs per row: enough to fill the 152 SMs, at least 4,096 logits each
    int C = 8;
    while (C > 1 && (n_rows * C > 152 * 4 || vocab < 4096 * (int64_t)C)) C /= 2;
    if (n_rows * C > INT32_MAX) return TREE_ATTN_ERR_TOO_LARGE;
    static std::once_flag once[kMaxDevices];
    static cudaError_t attr[kMaxDevices];
    std::call_once(once[dev], [&] {
        attr[dev] = cudaFuncSetAttribute(sample_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Shared));
    });
    if (attr[dev] != cudaSuccess) return TREE_ATTN_ERR_CUDA;
    const Params p = {static_cast<const uint16_t*>(logits), row_stride, vocab, u, *s, tokens, logprobs, status};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(n_rows * C));
    cfg.blockDim = dim3(kNT);
    cfg.dynamicSmemBytes = sizeof(Shared);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim = {(unsigned)C, 1, 1};
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, sample_kernel, p) == cudaSuccess ? TREE_ATTN_OK : TREE_ATTN_ERR_CUDA;
}
