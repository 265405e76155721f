// Attention of one new token per query over the tree's 8-bit cache
// (include/tree_decode.h).
//
// A work item is a run of pages and a block of at most 64 query rows (queries
// under the run x the heads that share a kv-head); a CTA takes one item of one
// kv-head.  Rows of one shared prefix sit in one tile, so its pages are read once
// for all of them.  One producer thread streams pages (K and V of one kv-head,
// 64 * d bytes each) through a ring in shared memory by bulk copies; four consumer
// warps hold 16 rows each, or, with fewer rows, take the pages in turn with
// accumulators of their own that are joined at the end.
//
// Per page, with fp32 accumulation on the tensor cores:
//   S = Q K8^T        A = query rows, f16; B = the page's codes, f16 (exact: e4m3 values)
//   x = S * (softmax_scale * log2(e) * k_scale * row factor) + log2(v_scale)
//   P = 2^(14 + x - M),  M = running maximum of x,   O += P V8,   l += rowsum(P) / v_scale
// Folding log2(v_scale) into the exponent makes P the weight of the page's
// *codes*, so one accumulator serves pages of different scales.  The largest weight
// is 2^14 whatever the scales (f16 ends at 2^16): P rounds by 2^-11, and what falls
// below f16's normal numbers, 2^-28 of the largest weight, by 2^-39 of it.  The query row is
// brought to [1, 2) by a power of two before its rounding to f16: 11 bits hold
// bf16's 8, and what falls below 2^-14 of the row's largest value loses at most
// 2^-25 of it.  l sums the unrounded fp32 weights.
//
// Fragments straight from the pages.  m16n8k16 wants, per lane (g = lane / 4,
// t = lane % 4), pairs of neighbouring k for column n = g.  The order of k is free
// as long as both operands agree, so lane t takes features 32t .. 32t+31 of a
// key (two 16-byte loads for d = 128) and keys 16t .. 16t+15 of a value feature (one):
// no shuffles, and the S accumulators are already the A fragments of P V.
#include <cuda_runtime.h>

#include <cmath>

#include "decode.h"
#include "kernels.h"

namespace treeattn {

namespace {

constexpr int kWarps = 4;                        // consumer warps
constexpr int kThreads = 32 * (kWarps + 1);
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLift = 14.f;                    // log2 of the largest weight in P

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
    uint16_t* o;
    float* lse;
    float* part_o;       // [hkv, part_rows, d]
    float2* part_ml;     // [hkv, part_rows] {M, l}
    int64_t part_rows;
    int32_t R, hq, hkv, group, n_sub, gsub;
    float scale_log2;
    int* status;
};

struct CombineParams {
    const int32_t* order;
    const int32_t* ptr;
    const int32_t* row;
    uint16_t* o;
    float* lse;
    const float* part_o;
    const float2* part_ml;
    int64_t part_rows;
    int32_t R, hq, hkv, group, n_sub, gsub, live;
};

__device__ __forceinline__ void lds128(uint32_t addr, uint32_t (&w)[4]) {
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(addr));
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
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// largest of a row's four lanes
__device__ __forceinline__ float quad_max(float x) {
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
    return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
}
__device__ __forceinline__ float quad_sum(float x) {
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    return x + __shfl_xor_sync(0xffffffffu, x, 2);
}

template <int D>
struct Shape {
    static constexpr int kHalf = kPage * D;          // bytes of K (or V) in a stage
    static constexpr int kStage = 2 * kHalf;
    static constexpr int kStages = D == 128 ? 6 : 10;
    static constexpr int kJoin = kWarps * 16 * (D + 4) * 4;   // fp32 rows of every warp, padded
    static constexpr int kRing = kStages * kStage;
    static_assert(kJoin <= kRing, "the join reuses the ring");
    static constexpr int kSmem = kRing + 1024;       // + alignment slack
};

struct Meta {
    int32_t page[kDecodeMaxChunk];
    int32_t valid[kDecodeMaxChunk];
    float kf[kDecodeMaxChunk];      // k_scale * softmax_scale * log2(e)
    float lv[kDecodeMaxChunk];      // log2(v_scale)
    int32_t n;
    uint64_t full[kDecodeMaxChunk];   // one per page, used once: pages land out of order, and a
                                      // warp may come to a stage whose last use it had no part in
    uint64_t empty[16];               // one per stage
    float m[kWarps][16], l[kWarps][16];
};

template <int D>
__global__ void __launch_bounds__(kThreads, 2) decode_kernel(const __grid_constant__ CUtensorMap tk, const DecodeParams p) {
    using S = Shape<D>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ Meta M;
    const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const int item = blockIdx.x / p.hkv, h = blockIdx.x % p.hkv;
    const int32_t* it = p.items + 6 * (int64_t)item;
    const int e0 = it[0], e1 = it[1], rg0 = it[2], rg1 = it[3], part = it[4];
    const int rows = (rg1 - rg0) * p.gsub;
    const int tiles = rows > 32 ? 4 : rows > 16 ? 2 : 1;     // 16-row tiles
    const int split = kWarps / tiles;                        // warps that share a tile's pages
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    for (int i = threadIdx.x; i < e1 - e0; i += kThreads) mbar_init(smem_u32(&M.full[i]), 1);
    if (threadIdx.x < S::kStages) mbar_init(smem_u32(&M.empty[threadIdx.x]), tiles);
    fence_mbar_init();
    grid_dep_wait();
    grid_dep_launch();
    if (warp == kWarps) {
        // pages that hold tokens now, packed
        int n = 0;
        for (int e = e0; e < e1; e += 32) {
            int page = 0, valid = 0;
            if (e + lane < e1) {
                const int4 x = *reinterpret_cast<const int4*>(p.entries + 4 * (int64_t)(e + lane));
                page = x.x;
                valid = max(0, min(max(p.lens[x.y], 0) - x.z, x.w));
            }
            const uint32_t has = __ballot_sync(0xffffffffu, valid > 0);
            if (valid > 0) {
                const int at = n + __popc(has & ((1u << lane) - 1u));
                const int64_t ph = (int64_t)page * p.hkv + h;
                M.page[at] = page;
                M.valid[at] = valid;
                M.kf[at] = p.ks[ph] * p.scale_log2;
                M.lv[at] = (float)((int)(__float_as_uint(p.vs[ph]) >> 23) - 127);
            }
            n += __popc(has);
        }
        if (lane == 0) M.n = n;
    }

    // query fragments (consumer warps): rows g and g + 8 of the warp's tile
    const int g = lane >> 2, t = lane & 3;
    const int tile = warp % tiles, turn = warp / tiles;
    uint32_t qa[D / 16][4];
    float qf[2] = {0.f, 0.f};
    if (warp < kWarps) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int r = tile * 16 + g + 8 * u;
            const int rg = rg0 + r / p.gsub, gi = (rg % p.n_sub) * p.gsub + r % p.gsub;
            const bool ok = r < rows && gi < p.group;
            uint4 w[D / 32];
            if (ok) {
                const uint16_t* src = p.q + (int64_t)p.order[rg / p.n_sub] * p.q_stride + (h * p.group + gi) * D + t * (D / 4);
#pragma unroll
                for (int i = 0; i < D / 32; ++i) w[i] = *reinterpret_cast<const uint4*>(src + 8 * i);
            } else {
#pragma unroll
                for (int i = 0; i < D / 32; ++i) w[i] = make_uint4(0, 0, 0, 0);
            }
            float amax = 0.f;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(x[j] << 16)), fabsf(__uint_as_float(x[j] & 0xffff0000u))));
            }
            amax = quad_max(amax);
            // power of two that brings the row to [1, 2); infinities and NaN stay what they are
            int e = (int)(__float_as_uint(amax) >> 23);
            e = (e == 0 || e == 255) ? 127 : min(max(e, 8), 246);
            const float down = __uint_as_float((uint32_t)(254 - e) << 23);
            qf[u] = __uint_as_float((uint32_t)e << 23);
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {   // word 4i+j: features 2(4i+j), +1 of this lane
                    const uint32_t f = pack_f16(__uint_as_float(x[j] << 16) * down, __uint_as_float(x[j] & 0xffff0000u) * down);
                    qa[(4 * i + j) / 2][u + 2 * (j & 1)] = f;
                }
            }
        }
    }
    __syncthreads();
    const int n = M.n;

    float acc[D / 8][4];
    float mx[2] = {-INFINITY, -INFINITY}, ls[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;

    if (warp == kWarps) {
        if (lane == 0) {
            int i = 0;
            for (; i < n; ++i) {
                const int s = i % S::kStages;
                if (i >= S::kStages && !mbar_wait(smem_u32(&M.empty[s]), ((i / S::kStages) - 1) & 1, p.status, 301)) break;
                const uint32_t dst = ring + s * S::kStage, bar = smem_u32(&M.full[i]);
                const int64_t ph = (int64_t)M.page[i] * p.hkv + h;
                mbar_expect_tx(bar, S::kStage);
                if constexpr (D == 128) {
                    asm volatile(
                        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(&tk)), "r"(0),
                        "r"((int)(ph * kPage)), "r"(bar) : "memory");
                } else {
                    bulk_load(dst, p.k8 + ph * S::kHalf, S::kHalf, bar);
                }
                bulk_load(dst + S::kHalf, p.v8 + ph * S::kHalf, S::kHalf, bar);
            }
            // no copy is in flight once the ring is reused, whatever ended the loop
            for (int j = max(0, i - S::kStages); j < i; ++j)
                mbar_wait(smem_u32(&M.full[j]), 0, p.status, 303);
        }
    } else {
        for (int i = turn; i < n; i += split) {
            const int s = i % S::kStages;
            if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&M.full[i]), 0, p.status, 302))) break;
            const uint32_t kb = ring + s * S::kStage, vb = kb + S::kHalf;
            const int valid = M.valid[i];
            float c[8][4];
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                const int key = 16 * (g >> 1) + 2 * x + (g & 1);
                uint32_t w[D / 16];
                if constexpr (D == 128) {
                    uint32_t a[4], b[4];
                    lds128(kb + sw128_offset(key, 2 * t), a);
                    lds128(kb + sw128_offset(key, 2 * t + 1), b);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        w[j] = a[j];
                        w[(D / 32) + j] = b[j];
                    }
                } else {
                    uint32_t a[4];
                    lds128(kb + key * D + 16 * t, a);
#pragma unroll
                    for (int j = 0; j < 4; ++j) w[j] = a[j];
                }
                c[x][0] = c[x][1] = c[x][2] = c[x][3] = 0.f;
#pragma unroll
                for (int j = 0; j < D / 16; ++j) {
                    uint32_t b0, b1;
                    codes_f16(w[j], b0, b1);
                    mma16816(c[x], qa[j], b0, b1);
                }
            }
            const float lv = M.lv[i], kf = M.kf[i];
            const float f0 = kf * qf[0], f1 = kf * qf[1];
            // element (x, j): key 16t + 2x + (j & 1), row g + 8 (j >> 1)
            float top0 = -INFINITY, top1 = -INFINITY;
#pragma unroll
            for (int x = 0; x < 8; ++x) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    c[x][j] = (j < 2 ? f0 : f1) * c[x][j] + lv;
                    if (valid < kPage && 16 * t + 2 * x + (j & 1) >= valid) c[x][j] = -INFINITY;
                }
                top0 = fmax3(top0, c[x][0], c[x][1]);
                top1 = fmax3(top1, c[x][2], c[x][3]);
            }
            const float m0 = fmaxf(mx[0], quad_max(top0)), m1 = fmaxf(mx[1], quad_max(top1));
            if (__any_sync(0xffffffffu, m0 != mx[0] || m1 != mx[1])) {
                const float a0 = m0 == -INFINITY ? 1.f : fast_exp2(mx[0] - m0);
                const float a1 = m1 == -INFINITY ? 1.f : fast_exp2(mx[1] - m1);
                ls[0] *= a0;
                ls[1] *= a1;
#pragma unroll
                for (int y = 0; y < D / 8; ++y) {
                    acc[y][0] *= a0;
                    acc[y][1] *= a0;
                    acc[y][2] *= a1;
                    acc[y][3] *= a1;
                }
                mx[0] = m0;
                mx[1] = m1;
            }
            const float r0 = m0 == -INFINITY ? 0.f : m0 - kLift, r1 = m1 == -INFINITY ? 0.f : m1 - kLift;
            float s0 = 0.f, s1 = 0.f;
            uint32_t pa[4][4];
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                const float p0 = fast_exp2(c[x][0] - r0), p1 = fast_exp2(c[x][1] - r0);
                const float p2 = fast_exp2(c[x][2] - r1), p3 = fast_exp2(c[x][3] - r1);
                s0 += p0 + p1;
                s1 += p2 + p3;
                pa[x >> 1][2 * (x & 1)] = pack_f16(p0, p1);
                pa[x >> 1][2 * (x & 1) + 1] = pack_f16(p2, p3);
            }
            const float iv = fast_exp2(-lv);
            ls[0] += s0 * iv;
            ls[1] += s1 * iv;
            uint32_t keep[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {       // bytes of the lane's keys 16t + 4j .. that hold tokens
                const int k = valid - 16 * t - 4 * j;
                keep[j] = k >= 4 ? 0xffffffffu : k <= 0 ? 0u : (1u << (8 * k)) - 1u;
            }
#pragma unroll
            for (int y = 0; y < D / 8; ++y) {
                uint32_t w[4];
                lds128(vb + (8 * y + g) * kPage + 16 * t, w);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t b0, b1;
                    codes_f16(w[j] & keep[j], b0, b1);
                    mma16816(acc[y], pa[j], b0, b1);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&M.empty[s]));
        }
    }
    __syncthreads();      // every page has been consumed: the ring is free

    // join: every warp's rows to shared memory, then row by row over the warps of a tile
    float* buf = reinterpret_cast<float*>(smem_raw + (ring - smem_u32(smem_raw)));
    constexpr int kPitch = D + 4;
    if (warp < kWarps) {
        ls[0] = quad_sum(ls[0]);
        ls[1] = quad_sum(ls[1]);
        if (t == 0) {
            M.m[warp][g] = mx[0];
            M.m[warp][g + 8] = mx[1];
            M.l[warp][g] = ls[0];
            M.l[warp][g + 8] = ls[1];
        }
        float* b = buf + warp * 16 * kPitch;
#pragma unroll
        for (int y = 0; y < D / 8; ++y) {
            *reinterpret_cast<float2*>(b + g * kPitch + 8 * y + 2 * t) = make_float2(acc[y][0], acc[y][1]);
            *reinterpret_cast<float2*>(b + (g + 8) * kPitch + 8 * y + 2 * t) = make_float2(acc[y][2], acc[y][3]);
        }
    }
    __syncthreads();
    for (int x = threadIdx.x; x < rows * (D / 4); x += kThreads) {
        const int r = x / (D / 4), c = 4 * (x % (D / 4));
        const int rg = rg0 + r / p.gsub, gi = (rg % p.n_sub) * p.gsub + r % p.gsub;
        if (gi >= p.group) continue;
        float top = -INFINITY;
        for (int u = 0; u < split; ++u) top = fmaxf(top, M.m[(r >> 4) + u * tiles][r & 15]);
        const float ref = top == -INFINITY ? 0.f : top;
        float l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
        for (int u = 0; u < split; ++u) {
            const int w = (r >> 4) + u * tiles;
            const float f = fast_exp2(M.m[w][r & 15] - ref);
            const float4 v = *reinterpret_cast<const float4*>(buf + (w * 16 + (r & 15)) * kPitch + c);
            l += f * M.l[w][r & 15];
            o[0] += f * v.x;
            o[1] += f * v.y;
            o[2] += f * v.z;
            o[3] += f * v.w;
        }
        if (part >= 0) {
            const int64_t at = h * p.part_rows + part + r;
            *reinterpret_cast<float4*>(p.part_o + at * D + c) = make_float4(o[0], o[1], o[2], o[3]);
            if (c == 0) p.part_ml[at] = make_float2(top, l);
        } else {
            const int64_t qi = p.order[rg / p.n_sub];
            const int head = h * p.group + gi;
            const float inv = l == 0.f ? 0.f : 1.f / l;
            *reinterpret_cast<uint2*>(p.o + (qi * p.hq + head) * D + c) =
                make_uint2(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv));
            if (c == 0) p.lse[(int64_t)head * p.R + qi] = l == 0.f ? -INFINITY : (ref - kLift + log2f(l)) * kLn2;
        }
    }
}

// One warp per (query, head): joins the partial rows of the query's items.
template <int D>
__global__ void __launch_bounds__(256) combine_kernel(const CombineParams p) {
    const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (w >= (int64_t)p.live * p.hq) {
        grid_dep_wait();   // the next kernel counts on this one to end after the items
        return;
    }
    const int place = (int)(w / p.hq), head = (int)(w % p.hq);
    const int h = head / p.group, gi = head % p.group;
    const int rg = place * p.n_sub + gi / p.gsub, off = gi % p.gsub;
    const int c0 = p.ptr[rg], c1 = p.ptr[rg + 1];
    const int64_t qi = p.order[place];
    grid_dep_wait();
    if (c1 == c0 + 1 && p.row[c0] < 0) return;         // written by its item
    constexpr int PL = D / 32;
    const int64_t base = h * p.part_rows + off;
    float top = -INFINITY;
    for (int c = c0 + lane; c < c1; c += 32) top = fmaxf(top, p.part_ml[base + p.row[c]].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float ref = top == -INFINITY ? 0.f : top;
    float l = 0.f, o[PL];
#pragma unroll
    for (int j = 0; j < PL; ++j) o[j] = 0.f;
#pragma unroll 4
    for (int c = c0; c < c1; ++c) {
        const int64_t at = base + p.row[c];
        const float2 ml = p.part_ml[at];
        const float f = fast_exp2(ml.x - ref);
        l += f * ml.y;
        if constexpr (PL == 4) {
            const float4 v = *reinterpret_cast<const float4*>(p.part_o + at * D + lane * 4);
            o[0] += f * v.x;
            o[1] += f * v.y;
            o[2] += f * v.z;
            o[3] += f * v.w;
        } else {
            const float2 v = *reinterpret_cast<const float2*>(p.part_o + at * D + lane * 2);
            o[0] += f * v.x;
            o[1] += f * v.y;
        }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    uint32_t* dst = reinterpret_cast<uint32_t*>(p.o + (qi * p.hq + head) * D) + lane * (PL / 2);
#pragma unroll
    for (int j = 0; j < PL / 2; ++j) dst[j] = pack_bf16x2(o[2 * j] * inv, o[2 * j + 1] * inv);
    if (lane == 0) p.lse[(int64_t)head * p.R + qi] = l == 0.f ? -INFINITY : (ref - kLift + log2f(l)) * kLn2;
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

template <int D>
int launch(const tree_decode_plan_s* P, const CUtensorMap& tk, const DecodeParams& a, const CombineParams& b,
           cudaStream_t s) {
    const int64_t items = (int64_t)P->items.size() / 6;
    if (items) {
        static std::once_flag once[kMaxDevices];
        static cudaError_t attr[kMaxDevices];
        int dev;
        const int st = current_device(&dev);
        if (st) return st;
        std::call_once(once[dev], [&] {
            attr[dev] = cudaFuncSetAttribute(decode_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<D>::kSmem);
        });
        if (attr[dev] != cudaSuccess) return TREE_ATTN_ERR_CUDA;
        if (launch_pdl(decode_kernel<D>, dim3((unsigned)(items * P->hkv)), dim3(kThreads), Shape<D>::kSmem, s, tk, a) !=
            cudaSuccess)
            return TREE_ATTN_ERR_CUDA;
    }
    if (P->any_combine && P->live) {
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
    if (!P || !lens || !q || !k8 || !v8 || !k_scale || !v_scale || !o || !lse) return TREE_ATTN_ERR_INVALID_ARG;
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
    if (P->d == 128 && (st = make_byte_map(&tk, k8, (int64_t)P->n_pages * P->hkv * kPage, kPage))) return st;
    float* part_o = static_cast<float*>(workspace);
    float2* part_ml = reinterpret_cast<float2*>(part_o + P->part_rows * P->hkv * P->d);
    const DecodeParams a = {D->entries, D->items, D->order, lens, static_cast<const uint16_t*>(q), q_stride,
                            static_cast<const uint8_t*>(k8), static_cast<const uint8_t*>(v8), k_scale, v_scale,
                            static_cast<uint16_t*>(o), lse, part_o, part_ml, P->part_rows, P->R, P->hq, P->hkv,
                            P->group, P->n_sub, P->gsub, softmax_scale * kLog2e, status};
    const CombineParams b = {D->order, D->combine_ptr, D->combine_row, static_cast<uint16_t*>(o), lse, part_o, part_ml,
                             P->part_rows, P->R, P->hq, P->hkv, P->group, P->n_sub, P->gsub, P->live};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return P->d == 128 ? launch<128>(P, tk, a, b, s) : launch<64>(P, tk, a, b, s);
}
