// Token sampling from given random numbers (include/tree_sample.h).
//
// A bf16 row of any length has few distinct values, and everything the draw needs
// -- the k-th token, the prefix that reaches p, the token at u -- depends on how
// often each value occurs.  So one pass over the logits counts values in shared
// memory (one bin per bf16 value, in descending order), and the rest works on the
// counts: a weight is computed once per value, not once per token, precisely
// enough to be an integer, and sums of integers do not depend on their order.
//
//   bins      value 0 and both signs of 2^-32 <= |x| < 2^16: 12,289 counters in 57 KB.
//             Lower values count as zero weight when the row's maximum and the
//             temperature allow it (masks, -inf); any other value outside sends the
//             row through the full range in windows, several passes, by one CTA.
//   groups    32 bins; a group's count and mass are one entry of a block-wide prefix
//             sum, a search finds the group, then one warp the bin.
//   cluster   C CTAs count a slice of the row each; each then weighs every C-th group
//             (counts summed over the C histograms through distributed shared memory),
//             and the first one searches.
//   index     the r-th token with the drawn value, found by the CTA whose slice holds
//             it.
//
// Two bytes per logit from HBM; paced by the instructions of the count (six per logit,
// with the range checked once for eight logits; a dozen with every case checked for each) and
// the shared-memory atomics (3.5 wavefronts each, what 32 random banks give), and for a
// few rows by the cluster's barriers and the chain of searches.  152,064 logits: 1 row 14 us, 64
// rows 23, 512 rows 100; half of them -inf: 15, 27, 121.  A row that needs the full range (a value
// of 0 < |x| < 2^-32, or of 2^16 and more) takes 200 to 300 us by its one CTA; 512 of them 650 to
// 900.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <utility>

#include "kernels.h"
#include "plan.h"
#include "tree_sample.h"

namespace cg = cooperative_groups;

namespace treeattn {

namespace {

constexpr int kNT = 512;                       // threads per CTA
constexpr int kBase = (127 - 32) << 7;         // bits of 2^-32
constexpr int kSide = 48 << 7;                 // values per sign: 2^-32 .. 2^16
constexpr int kBins = 2 * kSide + 1;
constexpr int kGroups = (kBins + 31) / 32;
constexpr int kNegative = 8192;                // where negative values' counters start
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

// round(2^61 * 2^(j / 64)), j = -32 .. 31
__constant__ uint64_t kPow[64] = {
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

constexpr float kRound = 12582912.f;           // 1.5 * 2^23

// 2^45 * 2^(d * c), d = x - top <= 0: n + j/64 + r = d * c in pairs of floats (48 bits),
// 2^(j/64) from the table, 2^r - 1 by its series (|r ln 2| < 0.0055: five terms), then
// integers.
__device__ __forceinline__ uint64_t weight(const uint64_t* pow, float x, float top, Rate c) {
    const float diff = x - top;
    // the rounding error of x - top
    const float b = diff - x;
    const float dl = ((x - (diff - b)) - (top + b)) * c.pre;
    const float d = diff * c.pre;
    const float y = d * c.hi;
    const bool none = !(y > -64.f), full = diff == 0.f;   // (no branches: callers interleave several)
    const float yl = fmaf(d, c.hi, -y) + fmaf(d, c.lo, dl * c.hi);
    // k = 64 n + j: adding 1.5 2^23 rounds to an integer, which the sum's low bits are (a
    // conversion instruction has a quarter of the rate)
    const float ys = none ? 0.f : y, kf = fmaf(ys, 64.f, kRound);
    const int k = (int)(__float_as_uint(kf) - __float_as_uint(kRound)), n = (k + 32) >> 6, j = k - 64 * n;
    const float r = fmaf(kf - kRound, -0.015625f, ys);   // exact
    const float rh = r + yl;
    const float rl = yl - (rh - r);
    // z = r ln 2
    constexpr float kLh = 0x1.62e430p-1f, kLl = -0x1.05c610p-29f;
    const float z = rh * kLh;
    const float zl = fmaf(rh, kLh, -z) + fmaf(rh, kLl, rl * kLh);
    const float zz = z * z, half = 0.5f * zz;
    const float tl = fmaf(zz * z, fmaf(z, fmaf(z, 1.f / 120.f, 1.f / 24.f), 1.f / 6.f), fmaf(z, zl, 0.5f * fmaf(z, z, -zz)));
    const float t = half + tl;
    const float e = z + t;
    const float el = (t - (e - z)) + (zl + (tl - (t - half)));
    // (e + el) 2^50: |e| < 2^-7 to multiples of 2^-29, then what is left, below 2^-28
    const float eh = fmaf(e, 0x1p29f, kRound);
    const float left = fmaf(eh - kRound, -0x1p-29f, e) + el;
    const int hi = (int)(__float_as_uint(eh) - __float_as_uint(kRound));
    const int lo = (int)(__float_as_uint(fmaf(left, 0x1p50f, kRound)) - __float_as_uint(kRound));
    const int64_t E = ((int64_t)hi << 21) + lo;
    const uint64_t p = pow[j + 32];
    const uint64_t w = p + (uint64_t)__mul64hi((int64_t)p, E << 14);
    const int shift = min(61 - kOneBits - n, 63);
    return full ? 1ull << kOneBits : none ? 0 : (w + (1ull << (shift - 1))) >> shift;
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

// How a row's weights are made, and which of them min_p keeps.
struct Weigher {
    float top;
    Rate rate;
    bool same;           // the untempered weights are the same
    uint64_t least;      // 0: no min_p
};

// What the weighing of groups adds up besides their masses.
struct Sums {
    uint64_t one;                                // untempered weight
    uint64_t mass;                               // weight and number of the tokens that min_p keeps
    uint32_t many;
};

struct Shared {
    uint32_t hist[kNegative + kSide];
    uint64_t pow[64];                            // kPow: lanes look up different entries
    uint32_t gcnt[kGroups], pcnt[kGroups];       // tokens of a group, of the groups before it
    uint64_t gmass[kGroups], pmass[kGroups];     // their weight
    Sums sums[8][kNT / 32];                      // by CTA of the cluster and warp
    uint32_t wcnt[kNT / 32];
    uint64_t wmass[kNT / 32];
    float tops[8];                               // of the slices
    uint32_t flags[8];
    Weigher weigher;
    Sums total;
    // the leader's search
    uint32_t tot_cnt;
    uint64_t tot_mass, tot_one;
    int found[2];                                // group, -1 for none; searches alternate
    uint32_t f_cnt, f_rank;
    uint64_t f_mass;
    int f_bin;
    // the index search
    int key;                                     // bits of the drawn value, or -1
    uint32_t rank, owner, matches;               // place among the owner's tokens of this value, and how many
    uint32_t listed;
};

enum { kNaN = 1, kRare = 2, kLow = 4 };

// Where a value of the short range is counted: magnitudes upwards from 0 for positive values
// and from kNegative for negative ones (a power of two: the sign bit, moved, selects it); zero
// between them.
constexpr int kZero = kSide, kNone = kSide + 1;   // kNone: nothing is counted there

// Why a value outside the short range (and not zero) does not count.
__device__ __forceinline__ uint32_t why(uint32_t b) {
    const uint32_t mag = b & 0x7fffu;
    return mag > 0x7f80u ? kNaN : (mag >= kBase && (b & 0x8000u)) ? kLow : kRare;
}

// Position in `hist` of the bin-th largest value; win < 0: the short range, else a window of
// the full one
__device__ __forceinline__ int place_of(int bin, int win) {
    if (win >= 0) return bin;
    return bin < kSide ? kSide - 1 - bin : bin == kSide ? kZero : bin < kBins ? bin - (kSide + 1) + kNegative : kNone;
}
// bits of that value
__device__ __forceinline__ uint32_t bits_of(int bin, int win) {
    if (win < 0) return bin < kSide ? kBase + (kSide - 1 - bin) : bin == kSide ? 0u : 0x8000u | (kBase + (bin - kSide - 1));
    const uint32_t o = 65535u - (uint32_t)(win * kWindow + bin);
    return o & 0x8000u ? o ^ 0x8000u : o ^ 0xffffu;
}

// Counts elements [lo, hi) of a row and takes their maximum.
__device__ __forceinline__ void count(Shared& S, const uint16_t* row, int64_t lo, int64_t hi, uint32_t& flags, float& top,
                                      int* status) {
    const uint16_t* a = row + lo;
    const int64_t n = hi - lo;
    auto slow = [&](uint32_t b) {                // any value
        const uint32_t mag = b & 0x7fffu, t = mag - kBase;
        if (t < (uint32_t)kSide) atomicAdd(&S.hist[t + (b >> 15) * kNegative], 1u);
        else if (mag == 0) atomicAdd(&S.hist[kZero], 1u);
        else flags |= why(b);
        top = fmaxf(top, __uint_as_float(b << 16));
    };
    const int64_t head = min(n, (int64_t)((16 - (reinterpret_cast<uintptr_t>(a) & 15)) & 15) / 2);
    if ((int64_t)threadIdx.x < head) slow(a[threadIdx.x]);
    const uint4* v = reinterpret_cast<const uint4*>(a + head);
    const int64_t nv = (n - head) / 8;
    __nv_bfloat162 m2 = __floats2bfloat162_rn(-INFINITY, -INFINITY);
    uint8_t* bins = reinterpret_cast<uint8_t*>(S.hist) - 4 * kBase;
    auto vec = [&](const uint4& x) {
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
        const uint32_t m[4] = {w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu, w[2] & 0x7fff7fffu, w[3] & 0x7fff7fffu};
        const uint32_t most = __vimax3_u16x2(__vimax3_u16x2(m[0], m[1], m[2]), m[3], m[3]);
        const uint32_t least = __vimin3_u16x2(__vimin3_u16x2(m[0], m[1], m[2]), m[3], m[3]);
#pragma unroll
        for (int i = 0; i < 4; ++i) m2 = __hmax2(m2, *reinterpret_cast<const __nv_bfloat162*>(&w[i]));
        if (max(most & 0xffffu, most >> 16) < kBase + kSide && min(least & 0xffffu, least >> 16) >= kBase) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {            // byte offsets: 4 magnitude + 2^15 sign
                const uint32_t h = w[i] >> 16;
                const uint32_t a0 = 4 * (w[i] & 0x7fffu) + (w[i] & 0x8000u), a1 = 4 * (h & 0x7fffu) + (h & 0x8000u);
                if (!ta_ok(status, 541, a0, 4 * kBase, 4 * (kBase + kNegative + kSide)) ||
                    !ta_ok(status, 541, a1, 4 * kBase, 4 * (kBase + kNegative + kSide)))
                    continue;
                atomicAdd(reinterpret_cast<uint32_t*>(bins + a0), 1u);
                atomicAdd(reinterpret_cast<uint32_t*>(bins + a1), 1u);
            }
        } else {                                     // zeros, and what does not count (masks: no loop)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t b = i & 1 ? w[i >> 1] >> 16 : w[i >> 1] & 0xffffu, mag = b & 0x7fffu;
                const bool in = mag - kBase < (uint32_t)kSide;
                if (in || mag == 0) atomicAdd(reinterpret_cast<uint32_t*>(bins + (in ? 4 * mag + (b & 0x8000u) : 4u * (kBase + kZero))), 1u);
                else flags |= why(b);
            }
        }
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
    if ((int64_t)threadIdx.x < n - done) slow(a[done + threadIdx.x]);
    top = fmaxf(top, fmaxf(__low2float(m2), __high2float(m2)));
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

// The counts at one place over the cluster's histograms: the CTA's own, then the others'
// (a load from another SM takes several times as long).
struct Counts {
    const uint32_t* own;
    const uint32_t* other[7];
    int n;               // CTAs
    __device__ __forceinline__ uint32_t operator()(int at) const {
        uint32_t c = own[at];
#pragma unroll
        for (int i = 0; i < 7; ++i)
            if (i + 1 < n) c += other[i][at];
        return c;
    }
};

// Weighs groups g0, g0 + step, ..: count and mass of each into `to`'s arrays, the rest into
// `sums`, this warp's.
__device__ __forceinline__ void weigh(const Counts& counts, int g0, int step, int win, const Weigher& W, const uint64_t* pow, Shared* to,
                      Sums& sums) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Rate unit = {1.44269502162933349609f, 1.92596299112661746887e-8f, 1.f};   // log2(e)
    // Most groups, far from the row's usual magnitudes, are empty: a warp loads the counts of
    // four of its groups at once (perhaps from other SMs) and passes over empty pairs (one
    // pair loaded at a time, an empty one took 1,000 cycles).  The two long chains of weights
    // of a pair overlap.
    constexpr int kBatch = 4;
    for (int ga = g0 + step * warp; ga < kGroups; ga += kBatch * step * (kNT / 32)) {
        const int gs = step * (kNT / 32);
        uint32_t n[kBatch], cn[kBatch];
        int at[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            at[i] = place_of(32 * min(ga + i * gs, kGroups - 1) + lane, win);
            n[i] = counts.own[at[i]];
        }
        if (counts.n > 1) {
#pragma unroll
            for (int x = 0; x < 7; ++x)
                if (x + 1 < counts.n) {
#pragma unroll
                    for (int i = 0; i < kBatch; ++i) n[i] += counts.other[x][at[i]];
                }
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (ga + i * gs >= kGroups) n[i] = 0;
            cn[i] = __reduce_add_sync(0xffffffffu, n[i]);
        }
#pragma unroll
        for (int j = 0; j < kBatch; j += 2) {
            uint64_t m[2] = {0, 0};
            if (cn[j] | cn[j + 1]) {
                uint64_t w[2], one[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float x = __uint_as_float(bits_of(32 * (ga + (j + i) * gs) + lane, win) << 16);
                    w[i] = weight(pow, x, W.top, W.rate);
                    one[i] = W.same ? w[i] : weight(pow, x, W.top, unit);
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t k = n[j + i];
                    m[i] = k ? k * w[i] : 0;
                    sums.one += k ? k * one[i] : 0;
                    if (w[i] >= W.least) {
                        sums.mass += m[i];
                        sums.many += k;
                    }
                    // below 2^63: limbs of 26 bits, so that 32 of them do not overflow
                    const uint64_t l0 = __reduce_add_sync(0xffffffffu, (uint32_t)m[i] & 0x3ffffffu);
                    const uint64_t l1 = __reduce_add_sync(0xffffffffu, (uint32_t)(m[i] >> 26) & 0x3ffffffu);
                    const uint64_t l2 = __reduce_add_sync(0xffffffffu, (uint32_t)(m[i] >> 52));
                    m[i] = l0 + (l1 << 26) + (l2 << 52);
                }
            }
            if (lane < 2 && ga + (j + lane) * gs < kGroups) {
                to->gcnt[ga + (j + lane) * gs] = lane ? cn[j + 1] : cn[j];
                to->gmass[ga + (j + lane) * gs] = lane ? m[1] : m[0];
            }
        }
    }
    sums.one = warp_sum(sums.one);
    sums.mass = warp_sum(sums.mass);
    sums.many = __reduce_add_sync(0xffffffffu, sums.many);
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
__device__ __forceinline__ bool locate(Shared& S, const Counts& counts, int win, const Weigher& W, bool by_mass, uint64_t mass,
                       uint32_t cnt, int slot) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int g = threadIdx.x * kPer + i;
        if (g >= kGroups) continue;
        const bool in = by_mass ? S.pmass[g] < mass && mass <= S.pmass[g] + S.gmass[g]
                                : S.pcnt[g] < cnt && cnt <= S.pcnt[g] + S.gcnt[g];
        if (in) S.found[slot] = g;
    }
    __syncthreads();
    const int g = S.found[slot];
    if (threadIdx.x == 0) S.found[slot ^ 1] = -1;   // for the next search, a barrier away
    if (g < 0) return false;
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x, bin = 32 * g + lane;
        const uint32_t n = counts(place_of(bin, win));
        const uint64_t w = n ? weight(S.pow, __uint_as_float(bits_of(bin, win) << 16), W.top, W.rate) : 0;
        const uint32_t ci = warp_scan(n) + S.pcnt[g];
        const uint64_t mi = warp_scan(n * w) + S.pmass[g];
        const uint32_t cb = ci - n;
        const uint64_t mb = mi - n * w;
        const bool in = by_mass ? mb < mass && mass <= mi : cb < cnt && cnt <= ci;
        if (in) {
            uint32_t k = cnt - cb;                   // 1 .. n
            if (by_mass) {                           // the smallest with k w >= mass - mb; n < 2^18
                const uint64_t need = mass - mb;
                k = min(max((uint32_t)((float)need / (float)w), 1u), n);
                while (k * w < need) ++k;
                while (k > 1 && (k - 1) * w >= need) --k;
            }
            S.f_cnt = cb + k;
            S.f_mass = mb + k * w;
            S.f_bin = bin;
            S.f_rank = k - 1;
        }
    }
    __syncthreads();
    return true;
}

// Cuts and draw over the windows of a row.  `load(win, cnt, mass)` puts a window's groups
// and prefix sums (from a carry) in place; S.total says what min_p keeps once every window
// has been loaded.  A cut is a number of tokens and their mass.  Leader CTA, all threads;
// leaves the draw in S.f_bin, S.f_rank and the window in `at`; false when nothing has weight.
template <typename Load>
__device__ bool draw(Shared& S, const Counts& counts, int first, int windows, const Weigher& W, int32_t k, float p,
                     float u, Load load, int& at) {
    uint64_t mass = 0;
    uint32_t total = 0;
    int slot = 0;
    // the search for one token, window by window
    auto seek = [&](bool by_mass, uint64_t need, uint32_t cnt) {
        uint32_t c = 0;
        uint64_t m = 0;
        for (int w = 0; w < windows; ++w) {
            if (windows > 1) load(first + w, c, m);
            if (locate(S, counts, first + w, W, by_mass, need, cnt, slot)) {
                slot ^= 1;
                at = first + w;
                return true;
            }
            slot ^= 1;
            c = S.tot_cnt;
            m = S.tot_mass;
            __syncthreads();
        }
        return false;
    };
    for (int w = 0; w < windows; ++w) {
        load(first + w, total, mass);
        total = S.tot_cnt;
        mass = S.tot_mass;
        __syncthreads();
    }
    if (!mass) return false;
    uint32_t n = total;
    if (k > 0 && (uint32_t)k < total && seek(false, 0, (uint32_t)k)) {
        n = (uint32_t)k;
        mass = S.f_mass;
    }
    // the shortest prefix that reaches p; min_p's is known
    const uint64_t all = mass;
    if (p < 1.f) {
        bool rest;
        uint64_t need = times(p, all, rest);
        need = max(need + (rest ? 1 : 0), (uint64_t)1);
        if (seek(true, need, 0) && S.f_cnt < n) {
            n = S.f_cnt;
            mass = S.f_mass;
        }
    }
    if (W.least) {
        if (S.total.many < n) {
            n = S.total.many;
            mass = S.total.mass;
        }
    }
    bool rest;
    const uint64_t goal = u < 1.f ? times(u, mass, rest) + 1 : mass;   // cumulated mass > u * mass
    return seek(true, min(goal, mass), 0);
}

// The rank-th token (from 0) of elements [a, b) of a row with bits `key` (0: also -0), of
// `matches`, by a whole CTA.  Warps take contiguous parts, a lane eight elements at a time.
// Few matches are listed (the histogram's place is free by now) and the rank-th smallest is
// picked; many are counted, and the warp that has the token goes through its part again.
constexpr uint32_t kListed = 2048;

__device__ void find(Shared& S, const uint16_t* row, int a, int b, uint32_t key, uint32_t rank, uint32_t matches,
                     int32_t* out, int* status) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // Parts begin where memory's 16-byte blocks do, so that a lane's eight elements are one
    // load: block k holds elements 8 k - skew .. 8 k - skew + 7; blocks in0 .. in1 - 1 lie inside.
    const int skew = (int)(reinterpret_cast<uintptr_t>(row) & 15) / 2;
    const int first = (a + skew) / 8, blocks = (b + skew + 7) / 8 - first;
    const int b0 = first + (int)((int64_t)blocks * warp / (kNT / 32)), b1 = first + (int)((int64_t)blocks * (warp + 1) / (kNT / 32));
    const int in0 = (a + skew + 7) / 8, in1 = (b + skew) / 8;
    const uint4* mem = reinterpret_cast<const uint4*>(row - skew);
    const uint32_t other = key ? key : 0x8000u, mask = key ? 0xffffffffu : 0x7fff7fffu, twice = key | key << 16;
    auto some_half = [&](const uint4& x) {           // of (w & mask) ^ twice is zero
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
        uint32_t any = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t y = (w[i] & mask) ^ twice;
            any |= (y - 0x00010001u) & ~y;
        }
        return (any & 0x80008000u) != 0;
    };
    // bit i: element i of the block matches
    auto exact = [&](const uint4& x) {
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t lo = w[i] & 0xffffu, hi = w[i] >> 16;
            m |= (uint32_t)(lo == key || lo == other) << (2 * i) | (uint32_t)(hi == key || hi == other) << (2 * i + 1);
        }
        return m;
    };
    auto hits = [&](int k) {
        uint32_t m = 0;
        if (k >= b1) return m;
        if (k >= in0 && k < in1) {
            const uint4 x = __ldg(mem + k);
            return some_half(x) ? exact(x) : 0u;
        }
        for (int i = 0; i < 8; ++i) {
            const int e = 8 * k - skew + i;
            if (e >= a && e < b) m |= (uint32_t)(row[e] == key || row[e] == other) << i;
        }
        return m;
    };
    if (matches <= kListed) {
        auto list = [&](int k, uint32_t m) {
            while (m) {
                const int32_t at = 8 * k - skew + __ffs(m) - 1;
                m &= m - 1;
                S.hist[min(atomicAdd(&S.listed, 1u), kListed - 1)] = (uint32_t)at;
            }
        };
        constexpr int kBatch = 8;                    // loads under way
        int k = max(b0, in0) + lane;
        if (lane == 0 && b0 < in0) list(b0, hits(b0));                       // the row's ragged ends
        if (lane == 0 && b1 > in1 && in1 >= max(b0, in0)) list(in1, hits(in1));
        const int end = min(b1, in1);
        for (; k + (kBatch - 1) * 32 < end; k += kBatch * 32) {
            uint4 x[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) x[i] = __ldg(mem + k + 32 * i);
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                if (some_half(x[i])) list(k + 32 * i, exact(x[i]));
        }
        for (; k < end; k += 32) list(k, hits(k));
        __syncthreads();
        for (uint32_t i = threadIdx.x; i < matches; i += kNT) {
            const uint32_t mine = S.hist[i];
            uint32_t smaller = 0;
#pragma unroll 8
            for (uint32_t j = 0; j < matches; ++j) smaller += S.hist[j] < mine;
            if (smaller == rank && ta_ok(status, 544, (int32_t)mine, a, b)) *out = (int32_t)mine;
        }
        return;
    }
    uint32_t n = 0;
#pragma unroll 4
    for (int k = b0 + lane; k < b1; k += 32) n += __popc(hits(k));
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0) S.wcnt[warp] = n;
    __syncthreads();
    uint32_t before = 0;
    for (int w = 0; w < warp; ++w) before += S.wcnt[w];
    if (rank < before || rank >= before + n) return;
    uint32_t left = rank - before;
    for (int k = b0; k < b1; k += 32) {
        const uint32_t m = hits(k + lane), c = __popc(m), upto = warp_scan(c);
        if (left < upto && left >= upto - c) {
            const int at = 8 * (k + lane) - skew + (int)__fns(m, 0, (int)(left - (upto - c)) + 1);
            if (ta_ok(status, 545, at, a, b)) *out = at;
        }
        const uint32_t all = __shfl_sync(0xffffffffu, upto, 31);
        if (left < all) return;
        left -= all;
    }
}

__global__ void __launch_bounds__(kNT, 2) sample_kernel(const Params p) {
    extern __shared__ __align__(16) uint8_t raw[];
    Shared& S = *reinterpret_cast<Shared*>(raw);
    cg::cluster_group cluster = cg::this_cluster();
    const int C = (int)cluster.num_blocks(), me = (int)cluster.block_rank();
    // Another CTA's shared memory may be written once that CTA has begun: said here, waited for
    // after the count.
    auto begun = cluster.barrier_arrive();
    const int64_t r = blockIdx.x / C;
    const uint16_t* row = p.logits + r * p.stride;
    const int64_t lo = p.vocab * me / C, hi = p.vocab * (me + 1) / C;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i = threadIdx.x; i < (kNegative + kSide) / 4; i += kNT) reinterpret_cast<uint4*>(S.hist)[i] = make_uint4(0, 0, 0, 0);
    if (threadIdx.x < 64) S.pow[threadIdx.x] = kPow[threadIdx.x];
    grid_dep_wait();
    grid_dep_launch();
    const float T = p.s.temperatures ? p.s.temperatures[r] : p.s.temperature;
    const int32_t k = p.s.top_ks ? p.s.top_ks[r] : p.s.top_k;
    const float top_p = p.s.top_ps ? p.s.top_ps[r] : p.s.top_p;
    const float min_p = p.s.min_ps ? p.s.min_ps[r] : p.s.min_p;
    const float u = p.u[r];
    const bool greedy = T == 0.f;
    if (threadIdx.x == kNT - 1) {                   // once: double precision is slow
        bool rest = false;
        uint64_t least = 0;
        if (min_p > 0.f && !greedy) {
            least = times(fminf(min_p, 1.f), 1ull << kOneBits, rest);
            least = max(least + (rest ? 1 : 0), (uint64_t)1);
        }
        S.weigher = {0.f, rate_of(greedy ? 1.f : T), greedy || T == 1.f, least};
        S.found[0] = -1;
    }
    __syncthreads();

    // ---- count the slice ----------------------------------------------------------
    uint32_t flags = 0;
    float top = -INFINITY;
    count(S, row, lo, hi, flags, top, p.status);
    flags = __reduce_or_sync(0xffffffffu, flags);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) {
        S.wcnt[warp] = flags;
        S.wmass[warp] = __float_as_uint(top);
    }
    __syncthreads();
    cluster.barrier_wait(std::move(begun));
    if ((int)threadIdx.x < C) {                    // to every CTA of the cluster
        for (int w = 0; w < kNT / 32; ++w) {
            flags |= S.wcnt[w];
            top = fmaxf(top, __uint_as_float((uint32_t)S.wmass[w]));
        }
        Shared* to = cluster.map_shared_rank(&S, (int)threadIdx.x);
        to->flags[me] = flags;
        to->tops[me] = top;
    }
    cluster.sync();

    // ---- the row's maximum, and what kind of row it is --------------------------------
    Counts counts;
    counts.n = C;
    flags = 0;
    top = -INFINITY;
    for (int i = 0; i < C; ++i) {
        flags |= S.flags[i];
        top = fmaxf(top, S.tops[i]);
    }
#pragma unroll
    for (int i = 0; i < 7; ++i) counts.other[i] = cluster.map_shared_rank(&S, i + 1 < C ? (me + i + 1) & (C - 1) : 0)->hist;
    counts.own = S.hist;
    top += 0.f;                                     // -0 counts as 0
    const bool bad_params = !(T >= 0.f) || isinf(T) || top_p != top_p || min_p != min_p || u != u;
    const bool bad = bad_params || (flags & kNaN) || isinf(top);
    // Values below -2^16 have no weight beside a maximum of at least -2^15 when
    // 2^15 / T is above 46 ln 2.
    const bool slow = (flags & kRare) || ((flags & kLow) && !(top >= -32768.f && T <= 512.f));
    Weigher W = S.weigher;
    W.top = top;

    Shared* leader = cluster.map_shared_rank(&S, 0);
    Sums sums = {0, 0, 0};
    if (!bad && !slow) {
        weigh(counts, me, C, -1, W, S.pow, leader, sums);
        if (lane == 0) leader->sums[me][warp] = sums;
    }
    cluster.sync();

    if (me == 0) {
        int win = -1, key = -1;
        bool drawn = false;
        uint32_t rank = 0;
        uint64_t one_all = 0;
        // S.total: the sums of `n` CTAs, by the first warp; all threads wait for it later
        auto totals = [&](int n) {
            if (threadIdx.x >= 32) return;
            Sums t = {0, 0, 0};
            for (int i = lane; i < n * (kNT / 32); i += 32) {
                const Sums& x = S.sums[i / (kNT / 32)][i % (kNT / 32)];
                t = {t.one + x.one, t.mass + x.mass, t.many + x.many};
            }
            t = {warp_sum(t.one), warp_sum(t.mass), __reduce_add_sync(0xffffffffu, t.many)};
            if (lane == 0) S.total = t;
        };
        if (!bad) {
            const int32_t kk = greedy ? 1 : k;
            const float pp = greedy ? 1.f : top_p, uu = greedy ? 0.f : u;
            if (!slow) {
                totals(C);
                drawn = draw(S, counts, -1, 1, W, kk, pp, uu, [&](int, uint32_t, uint64_t) { prefix(S, 0, 0); }, win);
            } else {
                // the full range, window by window, counted by this CTA alone
                counts.n = 1;
                int seen = 0;
                sums = {0, 0, 0};
                auto load = [&](int w, uint32_t cnt, uint64_t mass) {
                    __syncthreads();
                    for (int i = threadIdx.x; i < kNegative + kSide; i += kNT) S.hist[i] = 0;
                    __syncthreads();
                    each(row, 0, p.vocab, [&](uint32_t b) {
                        b = b == 0x8000u ? 0u : b;
                        const uint32_t o = 65535u - (b & 0x8000u ? b ^ 0xffffu : b ^ 0x8000u);
                        const uint32_t at = o - (uint32_t)(w * kWindow);
                        if (at < (uint32_t)kWindow && b != 0xff80u) atomicAdd(&S.hist[at], 1u);
                    });
                    __syncthreads();
                    Sums part = {0, 0, 0};
                    weigh(counts, 0, 1, w, W, S.pow, &S, part);
                    if (seen++ < kWindows) sums = {sums.one + part.one, sums.mass + part.mass, sums.many + part.many};
                    if (lane == 0) S.sums[0][warp] = sums;
                    __syncthreads();
                    totals(1);
                    prefix(S, cnt, mass);
                };
                drawn = draw(S, counts, 0, kWindows, W, kk, pp, uu, load, win);
            }
            one_all = S.total.one;
        }
        drawn = drawn && ta_ok(p.status, 542, S.f_bin, 0, 32 * kGroups) && ta_ok(p.status, 543, S.f_rank, 0, p.vocab);
        if (drawn) {
            key = (int)bits_of(S.f_bin, win);
            rank = S.f_rank;
        }
        if (threadIdx.x == 0) {
            if (bad_params) report_notice(p.status, TREE_ATTN_ERR_INVALID_SAMPLING);
            if (key < 0) p.tokens[r] = -1;
            if (p.logprobs) {
                const float x = __uint_as_float((uint32_t)key << 16);
                p.logprobs[r] = key < 0 ? __int_as_float(0x7fc00000)
                                        : (x - top) - log1pf((float)(one_all - (1ull << kOneBits)) * 0x1p-45f);
            }
            // the slice that holds the rank-th token of this value
            uint32_t owner = 0, matches = kListed + 1;   // the full range: many, for all it is known
            if (key >= 0 && win < 0) {
                const int at = place_of(S.f_bin, -1);
                uint32_t c[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) c[i] = i == 0 ? S.hist[at] : i < C ? counts.other[i - 1][at] : 0;
#pragma unroll
                for (int i = 0; i < 7; ++i)
                    if ((int)owner == i && i + 1 < C && rank >= c[i]) {
                        rank -= c[i];
                        ++owner;
                    }
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if ((int)owner == i) matches = c[i];
            }
            for (int i = 0; i < C; ++i) {
                Shared* to = cluster.map_shared_rank(&S, i);
                to->key = key;
                to->rank = rank;
                to->matches = matches;
                to->listed = 0;
                to->owner = win < 0 ? owner : 0xffffffffu;
            }
        }
    }
    cluster.sync();

    // ---- the index -------------------------------------------------------------------
    const int key = S.key;
    const bool whole = S.owner == 0xffffffffu;      // the leader searches the whole row
    if (key < 0 || (whole ? me != 0 : (int)S.owner != me)) return;
    find(S, row, whole ? 0 : (int)lo, whole ? (int)p.vocab : (int)hi, (uint32_t)key, S.rank, S.matches, p.tokens + r, p.status);
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
    // CTAs per row, at least 4,096 logits each: the fastest by this model, in thousands of
    // cycles.  A CTA takes 24 whatever its share (launch, barriers, the chain of searches), 16
    // for weighing and 24 for counting and finding 152,064 logits alone on an SM; 28, 26 and 46
    // beside another.  152 CTAs fit one to an SM, 304 two; clusters of 4 or 8 fewer, for they
    // keep to groups of SMs; beyond that the time grows with the CTAs.  Measured at 152,064, 1 /
    // 2 / 4 / 8 CTAs: 1 row 33 / 25 / 17 / 15 us, 24 rows 37 / 24 / 19 / 21, 76 rows 37 / 25 / 37 /
    // 54, 304 rows 63 / 71 / 103 / 171; at 16,384, 76 rows 19 / 16 / 28.  Over 22 numbers of rows
    // from 1 to 900 and 6 vocabularies the choice is at most 5 % slower than the best.
    int C = 1;
    double best = 0;
    const double v = vocab / 152064.0;
    for (int c = 1; c <= 8; c *= 2) {
        if (c > 1 && vocab < 4096 * (int64_t)c) break;
        const double ctas = (double)n_rows * c, full = c <= 2 ? 304 : 256;
        const double waves = ctas <= full ? 1 : std::max(1.4, ctas / full + 0.1);
        const bool alone = ctas <= (c <= 2 ? 152 : c == 4 ? 136 : 96);
        const double t = alone ? 24 + (16 + 24 * v) / c : waves * (28 + (26 + 46 * v) / c);
        if (c == 1 || t < best) {
            C = c;
            best = t;
        }
    }
    if (n_rows * C > INT32_MAX) return TREE_ATTN_ERR_TOO_LARGE;
    static std::once_flag once[kMaxDevices];
    static cudaError_t attr[kMaxDevices];
    std::call_once(once[dev], [&] {
        attr[dev] = launched(cudaFuncSetAttribute(sample_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Shared)));
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
    return launched(cudaLaunchKernelEx(&cfg, sample_kernel, p)) == cudaSuccess ? TREE_ATTN_OK : TREE_ATTN_ERR_CUDA;
}
