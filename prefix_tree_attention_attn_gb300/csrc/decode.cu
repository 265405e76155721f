// Attention of one new token per query over the tree's 8-bit cache
// (include/tree_decode.h).
//
// A work item is a run of pages and a block of query rows (queries under the run x
// the heads that share a kv-head), of one kv-head; pages of a shared prefix are read
// once for all the rows of a block.  Pages (K and V of one kv-head, 64 * d bytes each)
// come by bulk copies into shared memory, refilled by whoever emptied it.  An item
// leaves partial rows (O in fp32, M, m, l), which a second kernel joins per query.
//
// Per page, with fp32 accumulation on the tensor cores:
//   S = Q K8^T        Q in f16; K8 the page's codes in f16 (exact: e4m3 values)
//   s = S * (softmax_scale * log2(e) * k_scale * row factor),   x = s + log2(v_scale)
//   P = 2^(12 + x - M),   O += P V8,   l += sum_j 2^(12 + s_j - m)
// Folding log2(v_scale) into the exponent makes P the weight of the page's *codes*, so
// one accumulator serves pages of different scales; M is a running reference of x, m one
// of s.  They follow the row's maxima but are moved only when those pass them by 3.5: O
// (l) is then rescaled, which random logits ask for on the first pages only.  The largest
// weight so lies in [2^12, 2^15.5] whatever the scales (f16 ends at 2^16): P rounds by
// 2^-11, and what falls below f16's normal numbers by at most 2^-37 of the largest weight.
// l's terms are the unrounded P times 2^(M - log2(v_scale) - m), a factor per page; where
// a page's values are so small beside another's that its P vanish (a factor above 2^64),
// they are taken from s.  (With l on M's scale too, 65,536 keys of zero values -- scale
// 2^-100 -- pass fp32's range.)  Exponents are one multiply-add of the raw product, whose
// addend 12 + log2(v_scale) - M is small for the terms that count.  The query row is
// brought to [1, 2) by a power of two before its rounding to f16: 11 bits hold bf16's 8,
// and what falls below 2^-14 of the row's largest value loses at most 2^-25 of it.
//
// Two bodies, by the item's rows:
//
// At most 8 rows (a leaf's own pages) -- `narrow`, bound by HBM.  The item is one
// warp's, six to a CTA, up to 12 to an SM, with nothing between the warps: loads of some
// overlap the products of others, and no warp waits for a slower one (with a CTA's
// warps on one item, joined at its end, every item cost 8 us of its SM slot besides its
// pages).  A warp has room for one page: the next K is under way from the scores on,
// the next V from the end of P V; up to 192 KB in flight per SM.
// The products run transposed, S^T = K Q^T and O^T = V^T P^T, with m16n8k16: the codes
// are the 16-row operand and the 8 columns are the query rows, so no half of the tensor
// product is padding (rows as the 16-row operand, which a leaf of 8 rows half
// fills, took twice the instructions).  Fragments come straight from the pages:
// the order of k is free as long as both operands agree, so lane t of a quad takes
// features 32t .. 32t+31 of a key (two 16-byte loads for d = 128) and keys 16t .. 16t+15
// of a value feature (one).  P^T changes from accumulator to operand layout by
// 8x8 transposes (movmatrix).
//
// 9 to 128 rows (shared prefixes) -- `wide`, bound by shared memory: the same pages
// would cost a leaf's instructions once per 8 rows.  The codes are expanded once per
// page to f16 tiles in shared memory and the products are tcgen05.mma with
// M = 128 rows, accumulators in TMEM, P written back over S as the second product's
// operand.  Four warps do the softmax (one row per thread), three expand, one issues
// products and copies: no step of a page waits for another page's.  (With the four
// non-softmax warps taking turns at expanding and one of them issuing, a page took 3,300
// cycles of its CTA, half of them barriers and issue.)  A page of d = 128 takes 1,450
// cycles of an SM with two CTAs on it, 1,700 to 2,100 with one: the products read 512
// cycles' worth of shared memory at 128 bytes each, expanding reads and writes 700, the
// copies write 128.
#include <cuda_runtime.h>

#include <cfloat>
#include <cmath>

#include "decode.h"
#include "kernels.h"

namespace treeattn {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLift = 12.f;                    // log2 of the weight of x = M
constexpr float kSlack = 3.5f;                   // how far x may pass M before M is moved
constexpr float kFar = 64.f;                     // beyond 2^kFar, l's terms are not taken from the P

__device__ __forceinline__ float finite(float reference) { return reference == -INFINITY ? 0.f : reference; }

struct DecodeParams {
    const int32_t* entries;
    const int32_t* items;
    const int32_t* order;
    const int32_t* lens;
    const uint16_t* q;
    int64_t q_stride;
    const uint8_t* k8;
    const uint8_t* v8;
    const float* ks;
    const float* vs;
    float* part_o;       // [hkv, part_rows, d]
    float4* part_ml;     // [hkv, part_rows] {M, m, l, 0}
    int64_t part_rows;
    int32_t hkv, group, n_sub, gsub;
    float scale_log2;
    int32_t n_pages, n_nodes, R, live;   // of the plan, for the checks of debug builds
    int* status;
};

struct CombineParams {
    const int32_t* order;
    const int32_t* ptr;
    const int32_t* row;
    uint16_t* o;
    float* lse;
    const float* part_o;
    const float4* part_ml;
    int64_t part_rows;
    int32_t R, hq, hkv, group, n_sub, gsub, live;
    int* status;
};

// One warp: the CTA gives up the right to allocate TMEM.
__device__ __forceinline__ void tmem_relinquish() {
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
// 16 bytes of shared memory, by a plain load that the compiler may move.
__device__ __forceinline__ void lds128(const uint8_t* at, uint32_t (&w)[4]) {
    const uint4 x = *reinterpret_cast<const uint4*>(at);
    w[0] = x.x;
    w[1] = x.y;
    w[2] = x.z;
    w[3] = x.w;
}
// The same, kept in program order: several are to be under way before the first is used.
__device__ __forceinline__ void lds128_now(const uint8_t* at, uint32_t (&w)[4]) {
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(smem_u32(at)));
}
// four e4m3 codes to two f16 pairs
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi) : "r"(w));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// largest of a row's four lanes
__device__ __forceinline__ float quad_max(float x) {
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
    return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
}
// 8x8 matrix of 16-bit values, row g in lanes 4g .. 4g+3: its transpose, laid out the same
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
// Power of two that brings a row to [1, 2); infinities and NaN stay what they are.
__device__ __forceinline__ void row_factor(float amax, float& down, float& up) {
    int e = (int)(__float_as_uint(amax) >> 23);
    e = (e == 0 || e == 255) ? 127 : min(max(e, 8), 246);
    down = __uint_as_float((uint32_t)(254 - e) << 23);
    up = __uint_as_float((uint32_t)e << 23);
}
__device__ __forceinline__ float abs_max2(uint32_t w) {
    return fmaxf(fabsf(__uint_as_float(w << 16)), fabsf(__uint_as_float(w & 0xffff0000u)));
}
// two bf16 times a power of two, as f16
__device__ __forceinline__ uint32_t scaled_f16(uint32_t w, float down) {
    return pack_f16(__uint_as_float(w << 16) * down, __uint_as_float(w & 0xffff0000u) * down);
}

template <int D>
struct Shape {
    static constexpr int kHalf = kPage * D;          // bytes of K (or V) of a page
    static constexpr int kStage = 2 * kHalf;
    static constexpr int kNarrow = kDecodeWarps * kStage;   // a page per warp
    // wide: f16 tiles of Q, K and V, then a ring of K or V halves
    static constexpr int kHalves = 5;
    static constexpr int kTile = kPage * D * 2;
    static constexpr int kQ = 0, kK = kQ + 128 * D * 2, kV = kK + kTile, kCodes = kV + kTile;
    static constexpr int kWide = kCodes + kHalves * kHalf;
    static constexpr int kRing = kNarrow > kWide ? kNarrow : kWide;
    static constexpr int kSmem = kRing + 1024;       // + alignment slack
};

// Wide items.
struct Meta {
    int32_t page[kDecodeMaxChunk];
    int32_t valid[kDecodeMaxChunk];
    float kf[kDecodeMaxChunk];        // k_scale * softmax_scale * log2(e)
    float lv[kDecodeMaxChunk];        // log2(v_scale)
    // K and V of each page, used once
    uint64_t full[kDecodeMaxChunk], full_v[kDecodeMaxChunk];
    // K, V of a page are expanded; its scores are there, its P is in TMEM; its P V has finished.
    // The last three have a barrier for even and one for odd pages.  S of a page is issued before
    // P V of the page before, so who has seen the scores of page i knows of P V up to page i - 3
    // only (its phase was waited for before V of page i - 2 was expanded), and a single barrier
    // could still be two phases short of P V of page i - 1 -- the same parity.  The end of the
    // item is one further on: it has a barrier that is used once.  (Waiting for every page's
    // o_done in the softmax instead: long context 193 us against 189.)
    uint64_t k_ready, v_ready, s_done[2], p_full[2], o_done[2], finished;
    int32_t count[kDecodeMaxChunk / 32];
    int32_t early;                    // the first halves are on their way
    int32_t loaded;                   // halves that were, when a wait ran out
    uint32_t tmem;
    float top[128], mass_top[128], sum[128], qf[128];
};
// Narrow items: a warp's barriers for K and V.
struct Pair {
    uint64_t k, v;
};

// An item's rows: place in the output, and where its query row starts.
struct Rows {
    int rg0, rows, gsub, n_sub, group, h;
    __device__ __forceinline__ bool at(int r, int& place, int& head) const {
        const int rg = rg0 + r / gsub, gi = (rg % n_sub) * gsub + r % gsub;
        place = rg / n_sub;
        head = h * group + gi;
        return r < rows && gi < group;
    }
};

template <int D>
__device__ __forceinline__ void load_k(const CUtensorMap* tk, const DecodeParams& p, int page, int h, uint32_t dst,
                                       uint32_t bar) {
    const int64_t ph = (int64_t)page * p.hkv + h;
    if constexpr (D == 128) {
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(tk)), "r"(0),
            "r"((int)(ph * kPage)), "r"(bar) : "memory");
    } else {
        bulk_load(dst, p.k8 + ph * Shape<D>::kHalf, Shape<D>::kHalf, bar);
    }
}
template <int D>
__device__ __forceinline__ void load_v(const DecodeParams& p, int page, int h, uint32_t dst, uint32_t bar) {
    bulk_load(dst, p.v8 + ((int64_t)page * p.hkv + h) * Shape<D>::kHalf, Shape<D>::kHalf, bar);
}
// byte address of 16 codes c of key r in a K stage (swizzled by the tensor map for d = 128)
template <int D>
__device__ __forceinline__ const uint8_t* key_chunk(const uint8_t* base, int r, int c) {
    return D == 128 ? base + sw128_offset(r, c) : base + r * D + 16 * c;
}
// bits of four codes from key k on that lie before `valid`
__device__ __forceinline__ uint32_t keep_bytes(int k, int valid) {
    const int n = valid - k;
    return n >= 4 ? 0xffffffffu : n <= 0 ? 0u : (1u << (8 * n)) - 1u;
}

// After a wait that ran out: gives a copy or a product still in flight time to end before its
// shared memory or TMEM is given up.  Only for barriers that something is under way to.
__device__ __noinline__ void drain(uint64_t* bar, uint32_t parity) {
    for (int k = 0; k < 4096 && !mbar_try_wait(smem_u32(bar), parity); ++k) {}
}

// What a thread knows of page `threadIdx.x` of the item before it reads anything that
// an earlier kernel may have written.
struct Entry {
    int page, node, from, room;
    bool sure;           // held tokens when the plan was made: worth loading before its length is known
};
// Tokens of the page now, and its factors.
struct Factors {
    int valid;
    float kf, lv;
};
__device__ __forceinline__ Factors factors(const DecodeParams& p, const Entry& e, int h) {
    const int64_t ph = (int64_t)e.page * p.hkv + h;
    const int len = p.lens[e.node];
    const float ks = p.ks[ph], vs = p.vs[ph];
    return {max(0, min(max(len, 0) - e.from, e.room)), ks * p.scale_log2,
            (float)((int)(__float_as_uint(vs) >> 23) - 127)};
}

// ---- at most 8 rows --------------------------------------------------------------
// One warp.  n <= 32 pages, one per lane (e), some perhaps empty; qi: query of row
// (lane / 4) or -1.
template <int D>
__device__ void narrow(const CUtensorMap& tk, const DecodeParams& p, Pair& bar, const uint8_t* kb, const Rows& R, const Entry& e,
                       int qi, int head, int part) {
    using S = Shape<D>;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint8_t* vb = kb + S::kHalf;
    auto load_k = [&](int page) {
        mbar_expect_tx(smem_u32(&bar.k), S::kHalf);
        treeattn::load_k<D>(&tk, p, page, R.h, smem_u32(kb), smem_u32(&bar.k));
    };
    auto load_v = [&](int page) {
        mbar_expect_tx(smem_u32(&bar.v), S::kHalf);
        treeattn::load_v<D>(p, page, R.h, smem_u32(vb), smem_u32(&bar.v));
    };
    // the first page at once when it is sure to have held tokens
    const bool early = __shfl_sync(0xffffffffu, e.sure, 0);
    if (early && lane == 0) {
        load_k(e.page);
        load_v(e.page);
    }
    // query row g: features t * D/4 .., as the second operand
    uint4 w[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) w[i] = make_uint4(0, 0, 0, 0);
    if (qi >= 0) {
        const uint16_t* src = p.q + (int64_t)qi * p.q_stride + head * D + t * (D / 4);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) w[i] = *reinterpret_cast<const uint4*>(src + 8 * i);
    }
    Factors f = {0, 0.f, 0.f};
    if (e.room > 0) f = factors(p, e, R.h);
    // pages to go: those with tokens, and the one that is on its way whatever it holds
    uint32_t left = __ballot_sync(0xffffffffu, f.valid > 0 || (early && lane == 0));
    if (!early && left && lane == __ffs(left) - 1) {
        load_k(e.page);
        load_v(e.page);
    }
    uint32_t qb[D / 16][2];
    float qf;
    {
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
            amax = fmaxf(fmaxf(amax, fmaxf(abs_max2(w[i].x), abs_max2(w[i].y))), fmaxf(abs_max2(w[i].z), abs_max2(w[i].w)));
        float down;
        row_factor(quad_max(amax), down, qf);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            qb[2 * i][0] = scaled_f16(w[i].x, down);
            qb[2 * i][1] = scaled_f16(w[i].y, down);
            qb[2 * i + 1][0] = scaled_f16(w[i].z, down);
            qb[2 * i + 1][1] = scaled_f16(w[i].w, down);
        }
    }
    // factors of the accumulators' columns: rows 2t and 2t + 1
    const float qf0 = __shfl_sync(0xffffffffu, qf, 8 * t), qf1 = __shfl_sync(0xffffffffu, qf, 8 * t + 4);

    float acc[D / 16][4];
    float m0 = -INFINITY, m1 = -INFINITY, n0 = -INFINITY, n1 = -INFINITY, l0 = 0.f, l1 = 0.f;   // M, m, l
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;

    bool ok = true, k_ahead = false;
    uint32_t turn = 0;
    for (; left; ++turn) {
        const int i = __ffs(left) - 1;
        left &= left - 1;
        const int valid = __shfl_sync(0xffffffffu, f.valid, i);
        ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&bar.k), turn & 1, p.status, 302));
        if (!ok) break;
        // tile x: keys 16 (g/2) + 4x + (g & 1) and two further on
        // (two tiles and two partial sums each: four independent chains of products)
        float c[4][4];
#pragma unroll
        for (int x = 0; x < 4; x += 2) {
            const int key = 16 * (g >> 1) + 4 * x + (g & 1);
            uint32_t w0[2][D / 16], w1[2][D / 16];
#pragma unroll
            for (int y = 0; y < 2; ++y)
#pragma unroll
                for (int j = 0; j < D / 64; ++j) {
                    lds128(key_chunk<D>(kb, key + 4 * y, (D / 64) * t + j), *reinterpret_cast<uint32_t(*)[4]>(&w0[y][4 * j]));
                    lds128(key_chunk<D>(kb, key + 4 * y + 2, (D / 64) * t + j), *reinterpret_cast<uint32_t(*)[4]>(&w1[y][4 * j]));
                }
            float odd[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
            for (int j = 0; j < 4; ++j) c[x][j] = c[x + 1][j] = 0.f;
#pragma unroll
            for (int j = 0; j < D / 16; j += 2)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    uint32_t a[4];
                    codes_f16(w0[y][j], a[0], a[2]);
                    codes_f16(w1[y][j], a[1], a[3]);
                    mma16816(c[x + y], a, qb[j][0], qb[j][1]);
                    codes_f16(w0[y][j + 1], a[0], a[2]);
                    codes_f16(w1[y][j + 1], a[1], a[3]);
                    mma16816(odd[y], a, qb[j + 1][0], qb[j + 1][1]);
                }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                c[x][j] += odd[0][j];
                c[x + 1][j] += odd[1][j];
            }
        }
        // K's place is free: the next page's
        __syncwarp();
        const int after = left ? __ffs(left) - 1 : -1;
        const int next = __shfl_sync(0xffffffffu, e.page, max(after, 0));
        if (lane == 0 && after >= 0) load_k(next);
        const float lv = __shfl_sync(0xffffffffu, f.lv, i), kf = __shfl_sync(0xffffffffu, f.kf, i);
        // (a factor below fp32's normal numbers leaves no score above 2^-109: never 0, or NaN)
        const float f0 = fmaxf(kf * qf0, FLT_MIN), f1 = fmaxf(kf * qf1, FLT_MIN);
        float top0 = -INFINITY, top1 = -INFINITY;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const int key = 16 * (g >> 1) + 4 * x + (g & 1);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (valid < kPage && key + (j & 2) >= valid) c[x][j] = -INFINITY;
            top0 = fmax3(top0, c[x][0], c[x][2]);
            top1 = fmax3(top1, c[x][1], c[x][3]);
        }
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
            top0 = fmaxf(top0, __shfl_xor_sync(0xffffffffu, top0, o));
            top1 = fmaxf(top1, __shfl_xor_sync(0xffffffffu, top1, o));
        }
        top0 *= f0;
        top1 *= f1;
        const bool up0 = top0 + lv > m0 + kSlack, up1 = top1 + lv > m1 + kSlack;
        const bool un0 = top0 > n0 + kSlack, un1 = top1 > n1 + kSlack;
        if (__any_sync(0xffffffffu, up0 || up1 || un0 || un1)) {
            const float a0 = up0 ? fast_exp2(m0 - (top0 + lv)) : 1.f, a1 = up1 ? fast_exp2(m1 - (top1 + lv)) : 1.f;
            l0 *= un0 ? fast_exp2(n0 - top0) : 1.f;
            l1 *= un1 ? fast_exp2(n1 - top1) : 1.f;
#pragma unroll
            for (int y = 0; y < D / 16; ++y) {
                acc[y][0] *= a0;
                acc[y][1] *= a1;
                acc[y][2] *= a0;
                acc[y][3] *= a1;
            }
            m0 = up0 ? top0 + lv : m0;
            m1 = up1 ? top1 + lv : m1;
            n0 = un0 ? top0 : n0;
            n1 = un1 ? top1 : n1;
        }
        const float r0 = m0 == -INFINITY ? 0.f : m0 - lv, r1 = m1 == -INFINITY ? 0.f : m1 - lv;
        const float d0 = r0 - finite(n0), d1 = r1 - finite(n1), e0 = kLift - r0, e1 = kLift - r1;
        float s0 = 0.f, s1 = 0.f, t0 = 0.f, t1 = 0.f;
        const bool far = __any_sync(0xffffffffu, d0 > kFar || d1 > kFar);
        if (far) {
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const float g0 = kLift - finite(n0), g1 = kLift - finite(n1);
                t0 += fast_exp2(fmaf(c[x][0], f0, g0)) + fast_exp2(fmaf(c[x][2], f0, g0));
                t1 += fast_exp2(fmaf(c[x][1], f1, g1)) + fast_exp2(fmaf(c[x][3], f1, g1));
            }
        }
        uint32_t pb[4][2];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const float p0 = fast_exp2(fmaf(c[x][0], f0, e0)), p1 = fast_exp2(fmaf(c[x][1], f1, e1));
            const float p2 = fast_exp2(fmaf(c[x][2], f0, e0)), p3 = fast_exp2(fmaf(c[x][3], f1, e1));
            s0 += p0 + p2;
            s1 += p1 + p3;
            pb[x][0] = transpose8(pack_f16(p0, p1));
            pb[x][1] = transpose8(pack_f16(p2, p3));
        }
        l0 += d0 > kFar ? t0 : s0 * fast_exp2(d0);
        l1 += d1 > kFar ? t1 : s1 * fast_exp2(d1);
        // what is behind the last token may be anything, NaN included
        uint32_t keep[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) keep[j] = keep_bytes(16 * t + 4 * j, valid);
        const bool part_page = valid < kPage;
        ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&bar.v), turn & 1, p.status, 303));
        if (!ok) {
            k_ahead = after >= 0;      // the next K is on its way already
            break;
        }
#pragma unroll
        for (int y = 0; y < D / 16; ++y) {
            uint32_t w0[4], w1[4];
            lds128(vb + (16 * y + g) * kPage + 16 * t, w0);
            lds128(vb + (16 * y + g + 8) * kPage + 16 * t, w1);
            if (part_page) {
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    w0[x] &= keep[x];
                    w1[x] &= keep[x];
                }
            }
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                uint32_t a[4];
                codes_f16(w0[x], a[0], a[2]);
                codes_f16(w1[x], a[1], a[3]);
                mma16816(acc[y], a, pb[x][0], pb[x][1]);
            }
        }
        __syncwarp();
        if (lane == 0 && after >= 0) load_v(next);
    }
    if (!ok) {
        drain(&bar.k, (turn + k_ahead) & 1);
        drain(&bar.v, turn & 1);
        return;
    }
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
        l0 += __shfl_xor_sync(0xffffffffu, l0, o);
        l1 += __shfl_xor_sync(0xffffffffu, l1, o);
    }
    // rows 2t and 2t + 1 of the block; eight lanes write 32 bytes of a row
    const int64_t at = R.h * p.part_rows + part + 2 * t;
    float* o = p.part_o + at * D + g;
    if (2 * t < R.rows) {
        if (g == 0) p.part_ml[at] = make_float4(m0, n0, l0, 0.f);
#pragma unroll
        for (int y = 0; y < D / 16; ++y) {
            o[16 * y] = acc[y][0];
            o[16 * y + 8] = acc[y][2];
        }
    }
    if (2 * t + 1 < R.rows) {
        if (g == 0) p.part_ml[at + 1] = make_float4(m1, n1, l1, 0.f);
#pragma unroll
        for (int y = 0; y < D / 16; ++y) {
            o[D + 16 * y] = acc[y][1];
            o[D + 16 * y + 8] = acc[y][3];
        }
    }
}

// ---- 9 to 128 rows -----------------------------------------------------------------
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}
// Products and their commit by the one lane with `lead`; the warp stays together, so that the
// operands are uniform registers.
__device__ __forceinline__ void mma_ss(bool lead, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
        "r"((uint32_t)acc), "r"((uint32_t)lead) : "memory");
}
__device__ __forceinline__ void mma_ts(bool lead, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc),
        "r"((uint32_t)acc), "r"((uint32_t)lead) : "memory");
}

// Instruction descriptor, kind::f16: f16 A and B, fp32 accumulator, both K-major.
__host__ __device__ constexpr uint32_t idesc_f16(int m, int n) { return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24); }

// 16 codes to 32 bytes of f16: chunks c, c + 1 of row r of a 128-byte-swizzled tile
__device__ __forceinline__ void expand16(const uint32_t (&w)[4], uint32_t tile, int r, int c) {
    uint32_t f[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) codes_f16(w[j], f[2 * j], f[2 * j + 1]);
    st_shared_v4(tile + sw128_offset(r, c), f[0], f[1], f[2], f[3]);
    st_shared_v4(tile + sw128_offset(r, c + 1), f[4], f[5], f[6], f[7]);
}

// n pages in the plan's order; qi: query of row (thread / 2) or -1.
template <int D>
__device__ void wide(const CUtensorMap& tk, const DecodeParams& p, Meta& M, const uint8_t* base, const Rows& R, const Entry& e,
                     int qi, int head, int part, int n) {
    using S = Shape<D>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row = 32 * (warp & 3) + lane;                     // TMEM lane
    const uint32_t ring = smem_u32(base), qs = ring + S::kQ, vs = ring + S::kV;
    // Q, two threads per row
    uint4 w[D / 16];
    {
#pragma unroll
        for (int i = 0; i < D / 16; ++i) w[i] = make_uint4(0, 0, 0, 0);
        if (qi >= 0) {
            const uint16_t* src = p.q + (int64_t)qi * p.q_stride + head * D + (threadIdx.x & 1) * (D / 2);
#pragma unroll
            for (int i = 0; i < D / 16; ++i) w[i] = *reinterpret_cast<const uint4*>(src + 8 * i);
        }
    }
    // Halves in the order they are expanded: K0, K1, V0, K2, V1, ..., V(n-1).
    auto half_to = [&](bool is_v, int i, int page, int slot) {
        const uint32_t dst = ring + S::kCodes + slot * S::kHalf;
        const uint32_t bar = smem_u32(is_v ? &M.full_v[i] : &M.full[i]);
        mbar_expect_tx(bar, S::kHalf);
        if (is_v) load_v<D>(p, page, R.h, dst, bar);
        else load_k<D>(&tk, p, page, R.h, dst, bar);
    };
    auto is_value = [&](int x) { return x == 2 * n - 1 || (x >= 2 && !(x & 1)); };
    auto page_of = [&](int x) { return x == 2 * n - 1 ? n - 1 : is_value(x) ? x / 2 - 1 : (x + 1) / 2; };
    auto load_half = [&](int x) {
        if (x >= 2 * n) return;
        const int i = page_of(x);
        half_to(is_value(x), i, M.page[i], x % S::kHalves);
    };
    // Pages worth loading (sure to have held tokens, or holding some now), packed; the first
    // halves at once where the first two pages are sure.
    bool early = false;
    {
        Factors f = {0, 0.f, 0.f};
        if (warp < kDecodeMaxChunk / 32) {
            if (warp == 0) {
                early = (__ballot_sync(0xffffffffu, e.sure) & 3u) == 3u;
                if (early && lane == 0) {
                    half_to(false, 0, e.page, 0);
                    half_to(true, 0, e.page, 2);
                }
                if (early && lane == 1) half_to(false, 1, e.page, 1);
            }
            if ((int)threadIdx.x < n) f = factors(p, e, R.h);
        }
        const uint32_t has = __ballot_sync(0xffffffffu, e.sure || f.valid > 0);
        int at = __popc(has & ((1u << lane) - 1u));
        if (lane == 0 && warp < kDecodeMaxChunk / 32) M.count[warp] = __popc(has);
        if (threadIdx.x == 0) {
            M.early = early;
            M.loaded = 2 * kDecodeMaxChunk;
        }
        if (n > 32) {
            __syncthreads();
            for (int x = 0; x < warp && x < kDecodeMaxChunk / 32; ++x) at += M.count[x];
        }
        if (e.sure || f.valid > 0) {
            M.page[at] = e.page;
            M.valid[at] = f.valid;
            M.kf[at] = f.kf;
            M.lv[at] = f.lv;
        }
    }
    {
        const int r = threadIdx.x >> 1, hf = threadIdx.x & 1;
        float amax = 0.f, down, up;
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
            amax = fmaxf(fmaxf(amax, fmaxf(abs_max2(w[i].x), abs_max2(w[i].y))), fmaxf(abs_max2(w[i].z), abs_max2(w[i].w)));
        row_factor(fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1)), down, up);
        if (hf == 0) M.qf[r] = up;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
            const int c = hf * (D / 16) + i;                    // 8 features
            st_shared_v4(qs + (c >> 3) * 16384 + sw128_offset(r, c & 7), scaled_f16(w[i].x, down), scaled_f16(w[i].y, down),
                         scaled_f16(w[i].z, down), scaled_f16(w[i].w, down));
        }
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    n = 0;
    for (int x = 0; x < kDecodeMaxChunk / 32; ++x) n += M.count[x];
    const uint32_t tmem = M.tmem;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t o_col = tmem + 128;                          // S tiles at columns 0 and 64, O from 128
    float m = -INFINITY, mn = -INFINITY, l = 0.f;               // M, m, l
    bool ok = true;
    if (warp == 4) {
        // --------------------------- products and copies ---------------------------
        const bool lead = elect_one();
        if (lead)
            for (int x = M.early ? 3 : 0; x < S::kHalves; ++x) load_half(x);
        __syncwarp();
        const uint64_t qd = sdesc_sw128(qs, 16, 1024), kd = sdesc_sw128(ring + S::kK, 16, 1024), vd = sdesc_sw128(vs, 16, 1024);
        int x = S::kHalves;                                     // next half to load
        for (int i = 0; i <= n && ok; ++i) {
            if (i < n) {
                // S over the buffer that held P of page i - 2, which P V has read: products of
                // one thread run in order
                ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&M.k_ready), i & 1, p.status, 305));
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    mma_ss(lead, tmem + 64 * (i & 1), qd + (((k >> 2) * 16384 + (k & 3) * 32) >> 4),
                           kd + (((k >> 2) * 8192 + (k & 3) * 32) >> 4), idesc_f16(128, kPage), k > 0);
                if (lead) {
                    mma_commit(smem_u32(&M.s_done[i & 1]));
                    load_half(x);
                }
                ++x;
                __syncwarp();
            }
            if (i > 0) {
                const int j = i - 1;
                ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&M.v_ready), j & 1, p.status, 307) &&
                                                 mbar_wait(smem_u32(&M.p_full[j & 1]), (j / 2) & 1, p.status, 308));
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < kPage / 16; ++k)
                    mma_ts(lead, o_col, tmem + 64 * (j & 1) + 8 * k, vd + ((k * 32) >> 4), idesc_f16(128, D), j > 0 || k > 0);
                if (lead) {
                    mma_commit(smem_u32(&M.o_done[j & 1]));
                    if (i == n) mma_commit(smem_u32(&M.finished));
                    load_half(x);
                }
                ++x;
                __syncwarp();
            }
        }
        if (!ok && lead) {
            M.loaded = x;
            mma_commit(smem_u32(&M.finished));
        }
    } else if (warp > 4) {
        // -------------------------------- expansion --------------------------------
        const int ct = threadIdx.x - 160;                       // of 96
        constexpr int kRounds = (4 * D + 95) / 96;              // 16 codes each
        auto expand_k = [&](int i, int x) {
            bool good = mbar_wait(smem_u32(&M.full[i]), 0, p.status, 304);
            // the tile's previous reader was S of page i - 1
            if (i > 0) good = mbar_wait(smem_u32(&M.s_done[(i - 1) & 1]), ((i - 1) / 2) & 1, p.status, 306) && good;
            if (!__all_sync(0xffffffffu, good)) return false;
            const uint8_t* from = base + S::kCodes + (x % S::kHalves) * S::kHalf;
            const uint32_t ks = ring + S::kK;
            // All loads, then all conversions.
            auto place = [&](int u, int& r, int& y, int& c) {
                const int at = ct + 96 * u;
                c = at & 3;
                if constexpr (D == 128) {
                    // Eight lanes take four chunks of two rows that differ in bits 0 and 2, so that
                    // loads (swizzled by the row's 3 bits over 8 chunks) and stores both spread
                    // over all banks.
                    const int q = at >> 2 & 63;
                    y = at >> 8;
                    r = (q & ~5) | (((q & 1) * 5) ^ (q & 4));
                } else {
                    y = 0;
                    r = at >> 2;
                }
            };
            uint32_t w[kRounds][4];
#pragma unroll
            for (int u = 0; u < kRounds; ++u) {
                int r, y, c;
                place(u, r, y, c);
                if (ct + 96 * u < 4 * D) lds128_now(D == 128 ? from + sw128_offset(r, 4 * y + c) : from + r * 64 + c * 16, w[u]);
            }
#pragma unroll
            for (int u = 0; u < kRounds; ++u) {
                int r, y, c;
                place(u, r, y, c);
                if (ct + 96 * u < 4 * D) expand16(w[u], ks + y * 8192, r, 2 * c);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&M.k_ready));
            return true;
        };
        int x = 0;                                              // half at hand
        ok = n > 0 ? expand_k(0, x++) : true;
        for (int i = 0; i < n && ok; ++i) {
            if (i + 1 < n) ok = expand_k(i + 1, x++);
            if (!ok) break;
            const int valid = M.valid[i];
            bool good = mbar_wait(smem_u32(&M.full_v[i]), 0, p.status, 312);
            // P V of the page before has read the tile
            if (i > 0) good = mbar_wait(smem_u32(&M.o_done[(i - 1) & 1]), ((i - 1) / 2) & 1, p.status, 313) && good;
            ok = __all_sync(0xffffffffu, good);
            if (!ok) break;
            const uint8_t* from = base + S::kCodes + (x % S::kHalves) * S::kHalf;
            ++x;
            uint32_t w[kRounds][4];
#pragma unroll
            for (int u = 0; u < kRounds; ++u)
                if (ct + 96 * u < 4 * D) lds128_now(from + (ct + 96 * u) * 16, w[u]);
            if (valid < kPage) {       // what is behind the last token may be anything, NaN included
#pragma unroll
                for (int u = 0; u < kRounds; ++u)
#pragma unroll
                    for (int j = 0; j < 4; ++j) w[u][j] &= keep_bytes(16 * (ct & 3) + 4 * j, valid);
            }
#pragma unroll
            for (int u = 0; u < kRounds; ++u) {
                const int at = ct + 96 * u;
                if (at < 4 * D) expand16(w[u], vs, at >> 2, 2 * (at & 3));
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&M.v_ready));
        }
    } else if (32 * warp < R.rows) {
        // ------------------------------- softmax ---------------------------------
        // (a warp without rows leaves its part of P as it is: it reaches its rows of O only)
        const float qf = M.qf[row];
        for (int i = 0; i < n; ++i) {
            const uint32_t s_col = tmem + 64 * (i & 1) + lanes;
            const int valid = M.valid[i];
            const float lv = M.lv[i], f = fmaxf(M.kf[i] * qf, FLT_MIN);
            ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&M.s_done[i & 1]), (i / 2) & 1, p.status, 309));
            if (!ok) break;
            tc_fence_after();
            float c[64];
            tmem_ld32(s_col, *reinterpret_cast<float(*)[32]>(&c[0]));
            tmem_ld32(s_col + 32, *reinterpret_cast<float(*)[32]>(&c[32]));
            tmem_wait_ld();
            if (valid < kPage) {
#pragma unroll
                for (int j = 0; j < 64; ++j)
                    if (j >= valid) c[j] = -INFINITY;
            }
            float top = -INFINITY;
#pragma unroll
            for (int j = 0; j < 64; j += 2) top = fmax3(top, c[j], c[j + 1]);
            const float score = top * f;
            top = score + lv;
            const bool up = top > m + kSlack, un = score > mn + kSlack;
            if (__any_sync(0xffffffffu, un)) {
                l *= un ? fast_exp2(mn - score) : 1.f;
                mn = un ? score : mn;
            }
            if (__any_sync(0xffffffffu, up)) {
                const float a = up ? fast_exp2(m - top) : 1.f;
                if (i > 0) {
                    ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&M.o_done[(i - 1) & 1]), ((i - 1) / 2) & 1, p.status, 310));
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll 1
                    for (int x = 0; x < D / 16; ++x) {
                        float v[16];
                        tmem_ld16(o_col + lanes + 16 * x, v);
                        tmem_wait_ld();
                        uint32_t w[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j) w[j] = __float_as_uint(v[j] * a);
                        tmem_st16(o_col + lanes + 16 * x, w);
                    }
                    tmem_wait_st();
                }
                m = up ? top : m;
            }
            const float ref = m == -INFINITY ? 0.f : m - lv, d = ref - finite(mn);
            const uint64_t f2 = f32x2(f, f), e2 = f32x2(kLift - ref, kLift - ref);
            uint64_t sum = f32x2(0.f, 0.f);
            float far = 0.f;
            if (__any_sync(0xffffffffu, d > kFar)) {
#pragma unroll
                for (int j = 0; j < 64; ++j) far += fast_exp2(fmaf(c[j], f, kLift - finite(mn)));
            }
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                uint32_t pw[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    float a, b;
                    f32x2_split(fma_f32x2(f32x2(c[32 * x + 2 * j], c[32 * x + 2 * j + 1]), f2, e2), a, b);
                    a = fast_exp2(a);
                    b = fast_exp2(b);
                    sum = add_f32x2(sum, f32x2(a, b));
                    pw[j] = pack_f16(a, b);
                }
                tmem_st16(s_col + 16 * x, pw);
            }
            float sa, sb;
            f32x2_split(sum, sa, sb);
            l += d > kFar ? far : (sa + sb) * fast_exp2(d);
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(smem_u32(&M.p_full[i & 1]));
        }
        M.top[row] = m;
        M.mass_top[row] = mn;
        M.sum[row] = l;
        if (n > 0 && ok) ok = mbar_wait(smem_u32(&M.finished), 0, p.status, 311);
    }
    if (!__syncthreads_and(ok)) {
        // the products issued end by themselves; so do the copies
        drain(&M.finished, 0);
        const int loaded = min(M.loaded, 2 * n);   // all of them if the issuer got through
        for (int x = threadIdx.x; x < loaded; x += kThreads) drain(is_value(x) ? &M.full_v[page_of(x)] : &M.full[page_of(x)], 0);
        __syncthreads();
        return;
    }
    tc_fence_after();
    const int half = warp >> 2;                                 // columns D / 2 * half ..
    int place, out_head;
    const bool live = R.at(row, place, out_head);
    const int64_t at = R.h * p.part_rows + part + row;
    if (live && half == 0) p.part_ml[at] = make_float4(M.top[row], M.mass_top[row], M.sum[row], 0.f);
#pragma unroll
    for (int x = 0; x < D / 64; ++x) {
        const int col = half * (D / 2) + 32 * x;
        float v[32];
        tmem_ld32(o_col + lanes + col, v);                      // whole warps only
        tmem_wait_ld();
        if (!live) continue;
#pragma unroll
        for (int j = 0; j < 32; j += 4)
            *reinterpret_cast<float4*>(p.part_o + at * D + col + j) =
                n ? make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    tc_fence_before();
}

template <int D>
__global__ void __launch_bounds__(kThreads, 2) decode_kernel(const __grid_constant__ CUtensorMap tk, const DecodeParams p) {
    using S = Shape<D>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ union {
        Meta M;
        Pair pairs[kDecodeWarps];
    } sm;
    Meta& M = sm.M;
    uint8_t* base = smem_raw + (-smem_u32(smem_raw) & 1023u);
    const int cta = blockIdx.x / p.hkv, h = blockIdx.x % p.hkv;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // the plan's tables: nothing an earlier kernel writes
    const int4* slots = reinterpret_cast<const int4*>(p.items) + 2 * kDecodeWarps * (int64_t)cta;
    const int4 a0 = slots[0], b0 = slots[1];
    const int mine = warp < kDecodeWarps ? 2 * warp : 0;
    int4 a = slots[mine], b = slots[mine + 1];
    const bool is_wide = b0.y != 0;
    if (is_wide) {
        a = a0;
        b = b0;
    }
    const int n = a.y, part = b.x;
    const Rows R = {a.z, (a.w - a.z) * p.gsub, p.gsub, p.n_sub, p.group, h};
    Entry e = {0, 0, 0, 0, false};
    const int at = is_wide ? threadIdx.x : lane;
    if (at < n) {
        const int4 x = *reinterpret_cast<const int4*>(p.entries + 4 * (int64_t)(a.x + at));
        if (ta_ok(p.status, 501, x.x, 0, p.n_pages) && ta_ok(p.status, 502, x.y, 0, p.n_nodes) &&
            ta_ok(p.status, 503, x.w & 0xffff, 0, kPage + 1))
            e = {x.x, x.y, x.z, x.w & 0xffff, x.w >> 16 != 0};
    }
    int place, head, qi = -1;
    if (R.at(is_wide ? threadIdx.x >> 1 : lane >> 2, place, head) &&
        ta_ok(p.status, 504, place, 0, p.live)) {
        qi = p.order[place];
        if (!ta_ok(p.status, 505, qi, 0, p.R)) qi = -1;
    }
    if (n > 0 && !ta_ok(p.status, 506, part, 0, p.part_rows - R.rows + 1)) return;   // whole warps, or the CTA
    if (!is_wide) {
        // A CTA that may allocate TMEM has its SM to itself until it gives up the right to
        // (without this long context took 205 us instead of 188).
        if (warp == kWarps - 1) tmem_relinquish();
        if (lane == 0 && warp < kDecodeWarps) {
            mbar_init(smem_u32(&sm.pairs[warp].k), 1);
            mbar_init(smem_u32(&sm.pairs[warp].v), 1);
        }
        fence_mbar_init();
        __syncwarp();
        grid_dep_wait();
        grid_dep_launch();
        if (warp < kDecodeWarps && n > 0) narrow<D>(tk, p, sm.pairs[warp], base + warp * S::kStage, R, e, qi, head, part);
        return;
    }
    if (at < n) {
        mbar_init(smem_u32(&M.full[at]), 1);
        mbar_init(smem_u32(&M.full_v[at]), 1);
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&M.s_done[i]), 1);
            mbar_init(smem_u32(&M.p_full[i]), (R.rows + 31) / 32 * 32);
            mbar_init(smem_u32(&M.o_done[i]), 1);
        }
        mbar_init(smem_u32(&M.finished), 1);
        mbar_init(smem_u32(&M.k_ready), 3);
        mbar_init(smem_u32(&M.v_ready), 3);
    }
    fence_mbar_init();
    if (warp == kWarps - 1) tmem_alloc(smem_u32(&M.tmem), 256);
    grid_dep_wait();
    grid_dep_launch();
    wide<D>(tk, p, M, base, R, e, qi, head, part, n);
    __syncthreads();
    if (warp == kWarps - 1) {
        tc_fence_after();
        tmem_dealloc(M.tmem, 256);
    }
}

__device__ __forceinline__ float out_lse(float m, float l) {
    return l == 0.f ? -INFINITY : ((m == -INFINITY ? 0.f : m - kLift) + log2f(l)) * kLn2;
}

// One warp per (query, head): joins the partial rows of the query's items.  Up to 32
// of them, their places are read before the items are waited for.
template <int D>
__global__ void __launch_bounds__(256) combine_kernel(const CombineParams p) {
    const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    constexpr int PL = D / 32;
    int c0 = 0, c1 = 0, h = 0, off = 0, head = 0, mine = 0;
    int64_t qi = 0;
    if (w < (int64_t)p.live * p.hq) {
        const int place = (int)(w / p.hq);
        head = (int)(w % p.hq);
        h = head / p.group;
        const int gi = head % p.group, rg = place * p.n_sub + gi / p.gsub;
        off = gi % p.gsub;
        c0 = p.ptr[rg];
        c1 = p.ptr[rg + 1];
        qi = p.order[place];
        if (!ta_ok(p.status, 511, qi, 0, p.R)) c1 = -1;
        if (c0 + lane < c1) mine = p.row[c0 + lane];
    }
    // the next kernel may start; it counts on this one to end after the items
    grid_dep_wait();
    grid_dep_launch();
    if (w >= (int64_t)p.live * p.hq || c1 < 0) return;
    const int64_t base = h * p.part_rows + off;
    float top = -INFINITY, mtop = -INFINITY, l = 0.f, o[PL];
#pragma unroll
    for (int j = 0; j < PL; ++j) o[j] = 0.f;
    for (int b = c0; b < c1; b += 32) {
        if (b > c0) mine = b + lane < c1 ? p.row[b + lane] : 0;
        const int k = min(32, c1 - b);
        if (lane < k && !ta_ok(p.status, 512, mine + off, 0, p.part_rows)) mine = 0;
        const float4 ml = lane < k ? p.part_ml[base + mine] : make_float4(-INFINITY, -INFINITY, 0.f, 0.f);
        float t = ml.x, u = ml.y;
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) {
            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, x));
            u = fmaxf(u, __shfl_xor_sync(0xffffffffu, u, x));
        }
        t = fmaxf(t, top);
        u = fmaxf(u, mtop);
        const float again = fast_exp2(top - finite(t)), f = fast_exp2(ml.x - finite(t));
        l = l * fast_exp2(mtop - finite(u)) + fast_exp2(ml.y - finite(u)) * ml.z;     // this lane's parts
#pragma unroll
        for (int j = 0; j < PL; ++j) o[j] *= again;
        top = t;
        mtop = u;
#pragma unroll 4
        for (int c = 0; c < k; ++c) {
            const int64_t at = base + __shfl_sync(0xffffffffu, mine, c);
            const float fc = __shfl_sync(0xffffffffu, f, c);
            if constexpr (PL == 4) {
                const float4 v = *reinterpret_cast<const float4*>(p.part_o + at * D + lane * 4);
                o[0] += fc * v.x;
                o[1] += fc * v.y;
                o[2] += fc * v.z;
                o[3] += fc * v.w;
            } else {
                const float2 v = *reinterpret_cast<const float2*>(p.part_o + at * D + lane * 2);
                o[0] += fc * v.x;
                o[1] += fc * v.y;
            }
        }
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
    // the two references differ by about log2 of a page's scale
    const float inv = l == 0.f ? 0.f : 1.f / l, back = fast_exp2(finite(top) - finite(mtop));
    uint32_t* dst = reinterpret_cast<uint32_t*>(p.o + (qi * p.hq + head) * D) + lane * (PL / 2);
#pragma unroll
    for (int j = 0; j < PL / 2; ++j) dst[j] = pack_bf16x2(o[2 * j] * inv * back, o[2 * j + 1] * inv * back);
    if (lane == 0) p.lse[(int64_t)head * p.R + qi] = out_lse(mtop, l);
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

template <int D>
int launch(const tree_decode_plan_s* P, const CUtensorMap& tk, const DecodeParams& a, const CombineParams& b,
           cudaStream_t s) {
    const int64_t ctas = (int64_t)P->items.size() / (8 * kDecodeWarps);
    if (ctas) {
        static std::once_flag once[kMaxDevices];
        static cudaError_t attr[kMaxDevices];
        int dev;
        const int st = current_device(&dev);
        if (st) return st;
        std::call_once(once[dev], [&] {
            attr[dev] = launched(cudaFuncSetAttribute(decode_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<D>::kSmem));
        });
        if (attr[dev] != cudaSuccess) return TREE_ATTN_ERR_CUDA;
        if (launch_pdl(decode_kernel<D>, dim3((unsigned)(ctas * P->hkv)), dim3(kThreads), Shape<D>::kSmem, s, tk, a) !=
            cudaSuccess)
            return TREE_ATTN_ERR_CUDA;
    }
    if (P->live) {
        const int64_t blocks = ((int64_t)P->live * P->hq + 7) / 8;
        if (launch_pdl(combine_kernel<D>, dim3((unsigned)blocks), dim3(256), 0, s, b) != cudaSuccess)
            return TREE_ATTN_ERR_CUDA;
    }
    return TREE_ATTN_OK;
}

}  // namespace

}  // namespace treeattn

using namespace treeattn;

extern "C" int tree_attn_decode(tree_decode_plan_t P, const int32_t* lens, const void* q, int64_t q_stride,
                                const void* k8, const void* v8, const float* k_scale, const float* v_scale, void* o,
                                float* lse, float softmax_scale, void* workspace, size_t ws_bytes, void* stream) {
    if (!P || !lens || !q || !o || !lse) return TREE_ATTN_ERR_INVALID_ARG;
    if (P->n_pages && (!k8 || !v8 || !k_scale || !v_scale)) return TREE_ATTN_ERR_INVALID_ARG;   // a pool of no pages has no address
    if (!std::isfinite(softmax_scale) || !(softmax_scale > 0.f)) return TREE_ATTN_ERR_INVALID_ARG;
    if (q_stride < (int64_t)P->hq * P->d || q_stride % 8) return TREE_ATTN_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k8, 16) || !aligned(v8, 16) || !aligned(o, 16) || !aligned(lens, 4) ||
        !aligned(k_scale, 4) || !aligned(v_scale, 4) || !aligned(lse, 4))
        return TREE_ATTN_ERR_ALIGNMENT;
    if (P->ws_bytes) {
        if (!workspace || ws_bytes < P->ws_bytes) return TREE_ATTN_ERR_WORKSPACE;
        if (!aligned(workspace, 256)) return TREE_ATTN_ERR_ALIGNMENT;
    }
    DeviceDecode* D = nullptr;
    int st = ensure_decode(P, &D);
    if (st) return st;
    int dev, *status;
    if ((st = current_device(&dev)) || (st = get_status_ptr(dev, &status))) return st;
    CUtensorMap tk = {};
    if (P->d == 128 && !P->items.empty() && (st = make_byte_map(&tk, k8, (int64_t)P->n_pages * P->hkv * kPage, kPage))) return st;
    float* part_o = static_cast<float*>(workspace);
    float4* part_ml = reinterpret_cast<float4*>(part_o + P->part_rows * P->hkv * P->d);
    const DecodeParams a = {D->entries, D->items, D->order, lens, static_cast<const uint16_t*>(q), q_stride,
                            static_cast<const uint8_t*>(k8), static_cast<const uint8_t*>(v8), k_scale, v_scale,
                            part_o, part_ml, P->part_rows, P->hkv, P->group, P->n_sub, P->gsub,
                            softmax_scale * kLog2e, P->n_pages, P->n_nodes, P->R, P->live, status};
    const CombineParams b = {D->order, D->combine_ptr, D->combine_row, static_cast<uint16_t*>(o), lse, part_o, part_ml,
                             P->part_rows, P->R, P->hq, P->hkv, P->group, P->n_sub, P->gsub, P->live, status};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return P->d == 128 ? launch<128>(P, tk, a, b, s) : launch<64>(P, tk, a, b, s);
}
