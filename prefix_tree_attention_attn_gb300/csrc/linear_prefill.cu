// Whole turns of linear attention from and to states in slots (include/tree_linear.h).
//
// prefill_state_kernel, one launch per depth of the tree (roots first): a CTA walks the chunks (128
// tokens at most) of one node for one kv-head and F of the 128 value features -- the columns of the
// state do not meet --, with the state in registers:
//     gamma^64 S_in of the chunk goes out as bf16, the operand of the outputs;  S = gamma^L S + dS,
//     dS = sum_m gamma^(L-1-m) k_m v_m^T on the tensor cores.
//   A weighted value has 24 bits; it is split into three bf16 numbers that add up to it, so the
//   increment is as exact as sums in fp32 are (two would leave 3e-6 of it).  The parts lie side by side in one
//   product of N = 3 F, so K is read once, and are added in registers.  Warps 0-7 (0-3 for F = 32) hold the
//   state, 8-15 weigh and split the values, 16 loads, 17 issues.  F = 64: 208 KB pass through shared memory per
//   chunk, 1,630 cycles at 128 bytes a cycle, and pace it (2,300 measured).  F = 32: 136 KB; more CTAs, so
//   taken where all of a launch run at a time (one turn of 777 tokens: 16.5 us, 20.9 with F = 64; 8 branches of 300, two
//   waves of them: 33.0 and 31.2).
//   Where a depth has few nodes but long ones, they are cut into segments: a first launch
//   leaves what each adds to the state, then each segment starts from its node's state with the segments
//   before it added.  (A root's state is taken from its slot by the first launch: the last segment
//   may leave another one there before other segments have begun.)
//   A call's later launches begin while the one before them runs, on SMs that it leaves free: the first
//   one has waited for all that came before the call, so keys, values, queries and tables are there, and only
//   the warps that read or write states wait for the launch before (17 nodes of 8,835 tokens: 79 us; 88 one
//   after another).
//
// prefill_out_kernel, persistent, a unit (chunk, q-head) after the other: A = Q K^T, then
//     O = diag(f) (P V + Q gamma^64 S_in),  P[m, m'] = gamma^(64-(m'+1)) A[m, m'] for m' <= m,
//     f(m) = scale gamma^(m+1-64).
//   The query is an exact operand of both products and each part of O meets one rounding to
//   bf16 (P's or S_in's; a second part of each would take five products in place of three and twice the states'
//   bytes).  The powers are counted from the chunk's middle and stay within 2^+-50, so scores times values may
//   go up to 2^77: a decay below 2^(-100/128) = 0.58, whose state is forgotten within a few tokens, takes
//   P[m, m'] = scale gamma^(m-m') A[m, m'], S_in as it is and diag(scale gamma^(m+1)) Q, rounded to bf16, instead of Q.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <mutex>

#include "align.h"
#include "kernels.h"
#include "plan.h"
#include "ptx.cuh"
#include "tree_linear.h"

namespace treeattn {

namespace {

constexpr int kChunk = 128;
constexpr int kD = 128;
constexpr int kTile = kChunk * kD * 2;         // 32 KB, bf16
constexpr int kHalf = kTile / 2;               // 64 of its features
constexpr int kThreads = 320;

// States in slots of a pool: a root starts from the state in its slot, where it has one, and a
// node that has one leaves its last state there.
struct SlotIO {
    float* states;             // [n_slots, hkv, d, d]
    const int32_t* in;         // by node id, -1: a zero state; or null
    const int32_t* out;        // by node id, -1: not kept; or null
    int32_t n_slots;
    int* status;
};

// The slot of a node (its id) in a table, or -1; numbers outside the pool say so and count as -1.
__device__ __forceinline__ int slot_of(const SlotIO& io, const int32_t* table, int id) {
    const int s = table ? table[id] : -1;
    if (s < -1 || s >= io.n_slots) {
        report_notice(io.status, TREE_ATTN_ERR_INVALID_SLOT);
        return -1;
    }
    return s;
}

// Whether the powers of a decay (its log2) over half a chunk stay within 2^+-50: they are then factors of rows and columns.
__device__ __forceinline__ bool by_columns(float lg) { return lg > -100.f / kChunk; }
constexpr int kMiddle = kChunk / 2;            // the powers are counted from here

// The descriptor of a tile `bytes` further on (shared memory ends below 2^18, so the address field holds the sum).
__device__ __forceinline__ uint64_t further(uint64_t desc, uint32_t bytes) { return desc + (bytes >> 4); }

__device__ __forceinline__ uint4 pack8(const float* v) {
    return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}

// ---- the states that enter the chunks --------------------------------------------------------
// K in two stages; V in three, each with room for its other two parts behind it (the first goes over V).
constexpr int kKStages = 2, kVStages = 3;
constexpr int kStateK = 1024, kStateV = kStateK + kKStages * kTile;
template <int F>                               // value features of a CTA
struct StateLayout {
    static constexpr int kV = kChunk * F * 2;  // one part of the values
    static constexpr int kOut = kStateV + kVStages * 3 * kV, kSmem = kOut + kV;
};
// The descriptor of weighted values: rows are tokens, all of a part's F features wide, swizzled over their 128 or 64 bytes.
template <int F>
__device__ __forceinline__ uint64_t value_desc(uint32_t at) {
    constexpr uint64_t k64 = (uint64_t)4 << 61, kMode = (uint64_t)7 << 61;
    const uint64_t d = sdesc_sw128(at, StateLayout<F>::kV, 16 * F);
    return F == 64 ? d : (d & ~kMode) | k64;
}
constexpr int kStateThreads = 576;             // 8 warps hold the state, 8 weigh, loader, MMA
constexpr int kAhead = 6;                      // chunks that are brought into L2 ahead of their load

// A CTA's walk, the whole of a node or a segment: what it has to know before its first load, in one piece.
struct Walk {
    int32_t leaves, parent, chunk, chunks;     // places of end states, or -1; the walk's first chunk, its chunks
    int32_t token, end, id, unused;            // its first token, its last chunk's tokens; node id
    int32_t first, segment, whole, place;      // first of the node's chunks; chunks of a segment but the node's last,
                                               // segments but the last; the first one's place in `sums`
};
// Where a depth has few nodes, the walks go with the launch.
constexpr int kSplitNodes = 8, kSplitWalks = 16, kMaxWalks = kSplitNodes + kSplitWalks;

struct StateParams {
    const int4* order;         // LinInfo::walks of the depth, a node each; or null: `walks`
    Walk walks[kMaxWalks];
    const float* decay;
    float* s_out;              // [n_inner, hkv, d, d], end states of the nodes with children
    float* sums;               // [segments, hkv, d, d] what a segment adds to the state; behind a root's, its start state
    int32_t hkv, n_inner, n_chunks;
    int32_t first_depth;
    int32_t adding;            // 1: this launch leaves the sums
    int32_t leads;             // 1: the call's first launch
    SlotIO io;
};

template <int F>
__global__ void __launch_bounds__(kStateThreads, 1)
    prefill_state_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                         const __grid_constant__ CUtensorMap tm_s, const __grid_constant__ StateParams p) {
    using Lay = StateLayout<F>;
    constexpr int kParts = kD / F;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sb = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int* status = p.io.status;
    if (sb & 1023u) {
        if (threadIdx.x == 0) report_status(status, -5);
        return;
    }
    const int part = blockIdx.x % kParts, g = blockIdx.x / kParts % p.hkv;
    Walk job;
    if (p.order) {
        const int4* w = p.order + 2 * (blockIdx.x / kParts / p.hkv);
        const int4 a = w[0], b = w[1];
        job = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w, 0, a.w, 0, 0};
    } else {
        job = p.walks[blockIdx.x / kParts / p.hkv];
    }
    // (the loads are under way while the barriers are set up)
    const int n = job.chunks, c0 = job.chunk, end = job.end, whole = job.whole;
    bool ok = ta_ok(status, 620, job.leaves, -1, p.n_inner) && ta_ok(status, 621, c0, 0, p.n_chunks) &&
              ta_ok(status, 622, c0 + n, 0, p.n_chunks + 1) && ta_ok(status, 623, job.parent, -1, p.n_inner);
    const int par = ok ? job.parent : -1;
    const bool last = job.first == whole * job.segment, inner = last && job.leaves >= 0;
    auto kfull = [&](int s) { return sb + 8u * s; };          // K of stage s has come
    auto kfree = [&](int s) { return sb + 16 + 8u * s; };     // and has been multiplied
    auto vfull = [&](int s) { return sb + 32 + 8u * s; };
    auto vfree = [&](int s) { return sb + 56 + 8u * s; };
    auto wfull = [&](int s) { return sb + 80 + 8u * s; };     // the weighted values are there
    auto dfull = [&](int b) { return sb + 104 + 8u * b; };    // the increment is there
    auto dfree = [&](int b) { return sb + 120 + 8u * b; };
    const uint32_t drain = sb + 136, holder = sb + 144;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kKStages; ++s) {
            mbar_init(kfull(s), 1);
            mbar_init(kfree(s), 1);
        }
        for (int s = 0; s < kVStages; ++s) {
            mbar_init(vfull(s), 1);
            mbar_init(vfree(s), 1);
            mbar_init(wfull(s), 256);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(dfull(b), 1);
            mbar_init(dfree(b), 4 * F);
        }
        mbar_init(drain, 1);
        fence_mbar_init();
    }
    if (warp == 17) tmem_alloc(holder, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + 144);
    auto tokens = [&](int i) { return i == n - 1 ? end : kChunk; };
    if (p.leads) grid_dep_wait();
    grid_dep_launch();
    const float gamma = p.decay[g], lg = log2f(gamma);
    // (once per kv-head; the call's outputs are then undefined)
    if (p.first_depth && blockIdx.x < kParts * p.hkv && part == 0 && threadIdx.x == 0 && !(gamma > 0.f && gamma <= 1.f))
        report_notice(status, TREE_ATTN_ERR_INVALID_DECAY);
    const int to = ok && last ? slot_of(p.io, p.io.out, job.id) : -1;
    const int steps = !ok ? 0 : p.adding || inner || to >= 0 ? n : n - 1;   // increments that anything needs

    if (warp < F / 8) {
        // the state: thread = key feature, 32 value features
        const int quarter = warp & 3, row = 32 * quarter + lane, col0 = part * F + 32 * (warp >> 2);
        const size_t at = (size_t)g * kD * kD + (size_t)row * kD + col0;
        float S[32];
        const int from = ok && par < 0 ? slot_of(p.io, p.io.in, job.id) : -1;
        if (!p.leads) grid_dep_wait();
        const float* src = par >= 0 ? p.s_out + (size_t)par * p.hkv * kD * kD + at
                           : from >= 0 ? p.io.states + (size_t)from * p.hkv * kD * kD + at : nullptr;
        if (from >= 0 && whole > 0) {
            float* start = p.sums + (size_t)(job.place + whole) * p.hkv * kD * kD + at;
            if (p.adding && job.first == 0)
#pragma unroll
                for (int i = 0; i < 8; ++i) reinterpret_cast<float4*>(start)[i] = reinterpret_cast<const float4*>(src)[i];
            src = start;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float4 v = src && !p.adding ? reinterpret_cast<const float4*>(src)[i] : make_float4(0.f, 0.f, 0.f, 0.f);
            S[4 * i] = v.x;
            S[4 * i + 1] = v.y;
            S[4 * i + 2] = v.z;
            S[4 * i + 3] = v.w;
        }
        if (ok && !p.adding && job.first > 0) {        // the node's segments before this one
            const float f = exp2f((float)(job.segment * kChunk) * lg);
            for (int t = 0; t < job.first / job.segment; ++t) {
                const float4* add = reinterpret_cast<const float4*>(p.sums + (size_t)(job.place + t) * p.hkv * kD * kD + at);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float4 v = add[i];
                    S[4 * i] = fmaf(f, S[4 * i], v.x);
                    S[4 * i + 1] = fmaf(f, S[4 * i + 1], v.y);
                    S[4 * i + 2] = fmaf(f, S[4 * i + 2], v.z);
                    S[4 * i + 3] = fmaf(f, S[4 * i + 3], v.w);
                }
            }
        }
        const uint32_t stage = sb + Lay::kOut + warp * 2048, tD = tmem + ((uint32_t)(32 * quarter) << 16) + 32 * (warp >> 2);
        const float f128 = exp2f((float)kChunk * lg), entering = by_columns(lg) ? exp2f((float)kMiddle * lg) : 1.f;
        for (int i = 0; i < n && ok; ++i) {
            if (!p.adding) {
                if (lane == 0) bulk_wait_read_all();   // the last one has left
                __syncwarp();
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    float x[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = entering * S[8 * c + e];
                    const uint4 y = pack8(x);
                    st_shared_v4(stage + lane * 64 + c * 16, y.x, y.y, y.z, y.w);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    tma_store_3d(&tm_s, stage, col0, g, (c0 + i) * kChunk + 32 * quarter);
                    bulk_commit();
                }
            }
            if (i >= steps) break;
            const int b = i & 1;
            ok = mbar_wait(dfull(b), (i >> 1) & 1, status, 121);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
            const float f = i == n - 1 ? exp2f((float)end * lg) : f128;
            float v[32], more[32];                 // the three parts
            tmem_ld32(tD + b * 3 * F, v);
            tmem_ld32(tD + b * 3 * F + F, more);
            tmem_wait_ld();
#pragma unroll
            for (int x = 0; x < 32; ++x) v[x] += more[x];
            tmem_ld32(tD + b * 3 * F + 2 * F, more);
            tmem_wait_ld();
            tc_fence_before();
            mbar_arrive(dfree(b));
#pragma unroll
            for (int x = 0; x < 32; ++x) S[x] = fmaf(f, S[x], v[x] + more[x]);
        }
        if (ok) {
            auto leave = [&](float* dst) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    reinterpret_cast<float4*>(dst)[i] = make_float4(S[4 * i], S[4 * i + 1], S[4 * i + 2], S[4 * i + 3]);
            };
            if (p.adding) leave(p.sums + (size_t)(job.place + job.first / job.segment) * p.hkv * kD * kD + at);
            else if (inner) leave(p.s_out + (size_t)job.leaves * p.hkv * kD * kD + at);
            if (!p.adding && to >= 0) leave(p.io.states + (size_t)to * p.hkv * kD * kD + at);
        }
        if (lane == 0) bulk_wait_all();
        __syncwarp();
    } else if (warp >= 8 && warp < 16) {
        // the values: thread = token r and half of the features, times gamma^(L-1-r), as three numbers that add up to it
        const int r = threadIdx.x & 127, piece = (warp - 8) >> 2;
        const float w128 = exp2f((float)(kChunk - 1 - r) * lg);
        const uint64_t minus = f32x2(-1.f, -1.f);
        for (int i = 0; i < steps && ok; ++i) {
            const int s = i % kVStages, sk = i % kKStages;
            ok = mbar_wait(vfull(s), (i / kVStages) & 1, status, 122);
            const int L = tokens(i);
            const bool past = r >= L;              // another node's row: zeros, whatever it holds
            if (L < kChunk) {
                // A barrier tells a phase from the next one alone, and these warps have not waited for the stage's keys before:
                // first until the ones before them, which may still be under way, have been multiplied
                if (ok && i >= kKStages) ok = mbar_wait(kfree(sk), (i / kKStages - 1) & 1, status, 146);
                if (ok) ok = mbar_wait(kfull(sk), (i / kKStages) & 1, status, 123);
            }
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            const float w = L == kChunk ? w128 : past ? 0.f : exp2f((float)(L - 1 - r) * lg);
            const uint64_t ww = f32x2(w, w);
            uint4* v = reinterpret_cast<uint4*>(smem + kStateV + s * 3 * Lay::kV + r * 2 * F);
#pragma unroll
            for (int c = 0; c < F / 16; ++c) {
                // half of the row's 16-byte pieces, in an order rotated by the row (by two rows where two lie in 128 bytes):
                // the rows of a warp spread over all bank groups (a piece keeps its swizzled place)
                const int cr = (F / 16 * piece + c + (F == 64 ? r : r >> 1)) & (F / 8 - 1);
                const uint4 x = v[cr];
                const uint32_t u[4] = {x.x, x.y, x.z, x.w};
                uint32_t p1[4], p2[4], p3[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    // (what is not a number has no parts, and stays none)
                    float a, b, a1, b1;
                    const uint64_t y = past ? 0ull : mul_f32x2(f32x2(__uint_as_float(u[e] << 16), __uint_as_float(u[e] & 0xffff0000u)), ww);
                    f32x2_split(y, a, b);
                    p1[e] = pack_bf16x2(a, b);
                    const uint64_t y2 = fma_f32x2(f32x2(__uint_as_float(p1[e] << 16), __uint_as_float(p1[e] & 0xffff0000u)), minus, y);
                    f32x2_split(y2, a, b);
                    p2[e] = pack_bf16x2(a, b);
                    f32x2_split(fma_f32x2(f32x2(__uint_as_float(p2[e] << 16), __uint_as_float(p2[e] & 0xffff0000u)), minus, y2), a1, b1);
                    p3[e] = pack_bf16x2(a1, b1);
                }
                v[cr] = make_uint4(p1[0], p1[1], p1[2], p1[3]);
                v[Lay::kV / 16 + cr] = make_uint4(p2[0], p2[1], p2[2], p2[3]);
                v[2 * Lay::kV / 16 + cr] = make_uint4(p3[0], p3[1], p3[2], p3[3]);
            }
            if (past) {                            // its keys meet those zeros: no infinities there either
                uint4* k = reinterpret_cast<uint4*>(smem + kStateK + sk * kTile + piece * kHalf + r * 128);
#pragma unroll
                for (int c = 0; c < 8; ++c) k[(c + r) & 7] = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            mbar_arrive(wfull(s));
        }
    } else if (warp == 16) {
        if (lane == 0) {
            auto prefetch = [&](int i) {
                if (i >= steps) return;
                const int off = job.token + i * kChunk;
                for (int blk = 0; blk < 2; ++blk) tma_prefetch_3d(&tm_k, blk * 64, g, off);
                tma_prefetch_3d(&tm_v, part * F, g, off);
            };
            for (int i = kKStages; i < kAhead; ++i) prefetch(i);
            int sent = 0;
            for (int i = 0; i < steps && ok; ++i) {
                const int s = i % kVStages, sk = i % kKStages, off = job.token + i * kChunk;
                if (i >= kVStages) ok = mbar_wait(vfree(s), (i / kVStages - 1) & 1, status, 124);
                if (!ok) break;
                mbar_expect_tx(vfull(s), Lay::kV);
                tma_load_3d(sb + kStateV + s * 3 * Lay::kV, &tm_v, part * F, g, off, vfull(s));
                sent = i + 1;
                if (i >= kKStages) ok = mbar_wait(kfree(sk), (i / kKStages - 1) & 1, status, 125);
                if (!ok) break;
                mbar_expect_tx(kfull(sk), kTile);
                for (int blk = 0; blk < 2; ++blk)
                    tma_load_3d(sb + kStateK + sk * kTile + blk * kHalf, &tm_k, blk * 64, g, off, kfull(sk));
                prefetch(i + kAhead);
            }
            if (!ok) {                             // copies still under way
                for (int i = max(0, sent - kVStages); i < sent; ++i) mbar_wait(vfull(i % kVStages), (i / kVStages) & 1, status, 129);
                for (int i = max(0, sent - 1 - kKStages); i < sent - 1; ++i)
                    mbar_wait(kfull(i % kKStages), (i / kKStages) & 1, status, 130);
            }
        }
        __syncwarp();
    } else if (warp == 17) {
        if (lane == 0) {
            constexpr uint32_t ID = idesc_bf16(128, 3 * F, true, true);   // K^T (MN-major) x the values' parts (MN-major)
            for (int i = 0; i < steps && ok; ++i) {
                const int s = i % kVStages, sk = i % kKStages, b = i & 1;
                ok = mbar_wait(wfull(s), (i / kVStages) & 1, status, 126);
                if (ok) ok = mbar_wait(kfull(sk), (i / kKStages) & 1, status, 127);
                if (ok && i >= 2) ok = mbar_wait(dfree(b), ((i >> 1) - 1) & 1, status, 120);
                if (!ok) break;
                tc_fence_after();
                const uint64_t kd = sdesc_sw128(sb + kStateK + sk * kTile, kHalf, 1024),
                               vd = value_desc<F>(sb + kStateV + s * 3 * Lay::kV);
#pragma unroll
                for (int k = 0; k < kChunk / 16; ++k)
                    mma_bf16_ss(tmem + b * 3 * F, further(kd, k * 2048), further(vd, k * 32 * F), ID, k > 0);
                mma_commit(dfull(b));
                mma_commit(vfree(s));
                mma_commit(kfree(sk));
            }
            mma_commit(drain);
            mbar_wait(drain, 0, status, 128);
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 17) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ---- the outputs --------------------------------------------------------------------------------
// A CTA keeps one kv-head and walks the chunks j, j + lanes, ... while all CTAs have one, then its share of the q-heads
// of the chunks that are left (whole chunks left some CTAs 20 units where the mean is 16.4; shares of
// chunks in a row throughout took a tenth longer on a long context).  K is loaded once per chunk, V and S_in together
// once; Q comes through three slots.  TMEM holds two units (buffer b = u & 1): A, then P over it, at
// [256b, 256b + 128), O at [256b + 128, 256b + 256).  A of unit u is issued before the products of unit u - 1, and
// unit u - 1's output is read after unit u's mask, so that the products run meanwhile.
// warps 0-7: query row m = 32 (w % 4) + lane, columns [64 (w / 4), + 64) of A and O; warp 8 loads, warp 9
// issues.  A warp's 32 x 64 outputs leave by one bulk store out of shared memory (from registers, 16 bytes of 32
// different rows at a time, they kept the store unit busy for 2,000 cycles of a unit).
// A unit takes 3,900 cycles: 1,650 of tensor products, 3,500 of the mask, the weights and the roundings (latency: loads,
// conversions and stores of eight warps one after another), 3,300 of memory at 64 / 8 heads, beside one another.  480,408 tokens of 64 / 8 heads in 123 nodes: 3.83 ms with the states,
// 4.6 TB/s of what has to be read and written; 8,835 of 32 / 8 heads in 17 nodes 77 us; one turn of 777 16.5 us.
constexpr int kOutK = 2048, kOutV = kOutK + kTile, kOutS = kOutV + kTile, kOutQ = kOutS + kTile, kQSlots = 3,
              kOutStage = kOutQ + kQSlots * kTile, kOutSmem = kOutStage + kTile;

struct OutParams {
    const int32_t* chunks;
    const float* decay;
    uint16_t* out;
    int32_t n_chunks, lanes, share;            // CTAs of a kv-head, units of each of the chunks that are left
    int32_t hq, hkv;
    float scale;
    int* status;
};

__global__ void __launch_bounds__(kThreads, 1)
    prefill_out_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_s,
                       const __grid_constant__ CUtensorMap tm_o, const OutParams p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sb = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int* status = p.status;
    if (sb & 1023u) {
        if (threadIdx.x == 0) report_status(status, -5);
        return;
    }
    // `full` whole chunks, and then units [t0, t1) of those that are left
    const int g = blockIdx.x % p.hkv, lane_no = blockIdx.x / p.hkv, G = p.hq / p.hkv, h0 = g * G, full = p.n_chunks / p.lanes;
    const int left = (p.n_chunks - full * p.lanes) * G, t0 = min(lane_no * p.share, left), t1 = min(t0 + p.share, left);
    const int U = full * G + t1 - t0, n_items = full + (t1 > t0 ? (t1 - 1) / G - t0 / G + 1 : 0);
    if (U == 0) return;                        // uniform: nothing set up yet
    const int left0 = full * p.lanes + t0 / G - full, n0 = t0 % G;
    auto chunk_of = [&](int i) { return i < full ? lane_no + i * p.lanes : left0 + i; };
    auto head_of = [&](int i) { return i == full ? n0 : 0; };   // the chunk's first q-head here
    auto bar = [&](int i) { return sb + 8u * (uint32_t)i; };
    const uint32_t b_k = bar(0), b_v = bar(1), b_kfree = bar(2), b_vfree = bar(3), b_drain = bar(4), holder = bar(5);
    auto b_qf = [&](int q) { return bar(6 + q); };     // Q slot q has come
    auto b_sf = [&](int b) { return bar(10 + b); };    // A of buffer b is there
    auto b_p = [&](int b) { return bar(12 + b); };     // P is
    auto b_o = [&](int b) { return bar(14 + b); };     // O is
    auto b_oe = [&](int b) { return bar(16 + b); };    // O has been read
    auto b_qe = [&](int q) { return bar(18 + q); };    // Q slot q has been read
    const uint32_t ka = sb + kOutK, va = sb + kOutV, sina = sb + kOutS, qa0 = sb + kOutQ;
    float* ctab = reinterpret_cast<float*>(smem + 1024);   // gamma^(64-(m'+1)), or gamma^t
    if (threadIdx.x == 0) {
        mbar_init(b_k, 1);
        mbar_init(b_v, 1);
        mbar_init(b_kfree, 1);
        mbar_init(b_vfree, 1);
        mbar_init(b_drain, 1);
        for (int q = 0; q < kQSlots; ++q) {
            mbar_init(b_qf(q), 1);
            mbar_init(b_qe(q), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(b_sf(b), 1);
            mbar_init(b_p(b), 256);
            mbar_init(b_o(b), 1);
            mbar_init(b_oe(b), 256);
        }
        fence_mbar_init();
    }
    if (warp == 9) tmem_alloc(holder, 512);
    grid_dep_launch();
    const float lg = log2f(p.decay[g]);
    const bool column = by_columns(lg);
    if (threadIdx.x < 128) ctab[threadIdx.x] = exp2f((float)(column ? kMiddle - 1 - (int)threadIdx.x : (int)threadIdx.x) * lg);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + 8 * 5);
    bool ok = true;

    if (warp == 8) {
        if (lane == 0) {
            int sent = 0, q = 0, round = 0;        // Q loads sent, the next one's slot and its turn
            bool k_sent = false, v_sent = false, waited = false;
            for (int i = 0, u = 0; i < n_items && ok; ++i) {
                const int chunk = chunk_of(i), off = p.chunks[4 * chunk], first = head_of(i), end = min(G, first + U - u);
                k_sent = v_sent = false;
                if (i > 0) ok = mbar_wait(b_kfree, (i - 1) & 1, status, 131);   // the last chunk's last A has read it
                if (!ok) break;
                mbar_expect_tx(b_k, kTile);
                for (int blk = 0; blk < 2; ++blk) tma_load_3d(ka + blk * kHalf, &tm_k, blk * 64, g, off, b_k);
                k_sent = true;
                for (int n = first; n < end && ok; ++n, ++u) {
                    if (round) ok = mbar_wait(b_qe(q), (round - 1) & 1, status, 132);
                    if (!ok) break;
                    mbar_expect_tx(b_qf(q), kTile);
                    for (int blk = 0; blk < 2; ++blk)
                        tma_load_3d(qa0 + q * kTile + blk * kHalf, &tm_q, blk * 64, h0 + n, off, b_qf(q));
                    ++sent;
                    if (++q == kQSlots) {
                        q = 0;
                        ++round;
                    }
                    // V and S_in after the chunk's second Q here (the only one's, where there is no second): the last
                    // chunk's last products, which have read them, are issued before this chunk's second A
                    if (n == min(first + 1, end - 1)) {
                        if (i > 0) ok = mbar_wait(b_vfree, (i - 1) & 1, status, 133);
                        if (!ok) break;
                        if (!waited) grid_dep_wait();   // the states
                        waited = true;
                        mbar_expect_tx(b_v, 2 * kTile);
                        for (int blk = 0; blk < 2; ++blk) {
                            tma_load_3d(va + blk * kHalf, &tm_v, blk * 64, g, off, b_v);
                            tma_load_3d(sina + blk * kHalf, &tm_s, blk * 64, g, chunk * kChunk, b_v);
                        }
                        v_sent = true;
                    }
                }
                if (!ok) {                         // copies still under way
                    if (k_sent) mbar_wait(b_k, i & 1, status, 134);
                    if (v_sent) mbar_wait(b_v, i & 1, status, 135);
                }
            }
            if (!ok)
                for (int u = max(0, sent - kQSlots); u < sent; ++u) mbar_wait(b_qf(u % kQSlots), (u / kQSlots) & 1, status, 136);
        }
        __syncwarp();
    } else if (warp == 9) {
        if (lane == 0) {
            constexpr uint32_t ID_S = idesc_bf16(128, 128, false, false);   // Q K^T
            constexpr uint32_t ID_O = idesc_bf16(128, 128, false, true);    // P V, Q S_in
            const uint64_t kd = sdesc_sw128(ka, 16, 1024), vd = sdesc_sw128(va, kHalf, 1024), sd = sdesc_sw128(sina, kHalf, 1024);
            // the unit whose O is next: its place in its chunk, its slot
            int on = head_of(0), ofirst = on, oi = 0, oq = 0;
            int ksteps = (p.chunks[4 * chunk_of(0) + 1] + 15) / 16;
            auto issue_o = [&](int u) {
                const int b = u & 1;
                ok = mbar_wait(b_p(b), (u >> 1) & 1, status, 137);
                if (ok && u >= 2) ok = mbar_wait(b_oe(b), ((u >> 1) - 1) & 1, status, 138);   // unit u - 2's output read
                if (ok && on == ofirst) ok = mbar_wait(b_v, oi & 1, status, 139);                     // this chunk's V and S_in
                if (!ok) return;
                tc_fence_after();
                const uint32_t O = tmem + 256 * b + 128, P = tmem + 256 * b;
                const uint64_t qd = sdesc_sw128(qa0 + oq * kTile, 16, 1024);
                // keys 16k .. 16k + 15 of P packed at 64 (k / 4) + 8 (k % 4); features 16k .. 16k + 15 of f Q (strong
                // decays) 32 columns further
#pragma unroll
                for (int k = 0; k < kChunk / 16; ++k)
                    if (k < ksteps) mma_bf16_ts(O, P + (k >> 2) * 64 + (k & 3) * 8, further(vd, k * 2048), ID_O, k > 0);
#pragma unroll
                for (int k = 0; k < kD / 16; ++k) {
                    if (column) mma_bf16_ss(O, further(qd, (k >> 2) * kHalf + (k & 3) * 32), further(sd, k * 2048), ID_O, 1u);
                    else mma_bf16_ts(O, P + 32 + (k >> 2) * 64 + (k & 3) * 8, further(sd, k * 2048), ID_O, 1u);
                }
                mma_commit(b_o(b));
                mma_commit(b_qe(oq));
                oq = oq == kQSlots - 1 ? 0 : oq + 1;
                if (++on == G) {
                    mma_commit(b_vfree);
                    on = ofirst = head_of(++oi);
                    if (oi < n_items) ksteps = (p.chunks[4 * chunk_of(oi) + 1] + 15) / 16;
                }
            };
            int n = head_of(0), first = n, i = 0, q = 0, round = 0;
            for (int u = 0; u < U && ok; ++u) {
                const int b = u & 1;
                ok = mbar_wait(b_qf(q), round & 1, status, 140);
                if (ok && n == first) ok = mbar_wait(b_k, i & 1, status, 141);
                if (!ok) break;
                tc_fence_after();
                const uint64_t qd = sdesc_sw128(qa0 + q * kTile, 16, 1024);
#pragma unroll
                for (int k = 0; k < kD / 16; ++k) {
                    const uint32_t o = (k >> 2) * kHalf + (k & 3) * 32;
                    mma_bf16_ss(tmem + 256 * b, further(qd, o), further(kd, o), ID_S, k > 0);
                }
                mma_commit(b_sf(b));
                if (++n == G) {
                    mma_commit(b_kfree);
                    n = first = head_of(++i);
                }
                if (++q == kQSlots) {
                    q = 0;
                    ++round;
                }
                if (u > 0) issue_o(u - 1);
            }
            if (ok) issue_o(U - 1);
            mma_commit(b_drain);
            mbar_wait(b_drain, 0, status, 142);
        }
        __syncwarp();
    } else {
        const int quarter = warp & 3, m = (quarter << 5) + lane, grp = warp >> 2, col0 = grp * 64;
        const uint32_t lane_base = tmem + ((uint32_t)(quarter << 5) << 16);
        const float fo = p.scale * exp2f((float)(column ? m + 1 - kMiddle : m + 1) * lg);
        const uint32_t stage = sb + kOutStage + warp * 4096;
        // Unit u's output is read after unit u + 1's mask.
        int prev_off = 0, prev_L = 0, prev_h = 0, n = head_of(0), i = 0, q = 0;
        int off = p.chunks[4 * chunk_of(0)], L = p.chunks[4 * chunk_of(0) + 1];
        int first = n;                             // the chunk's first q-head here
        bool alone = false;                        // the chunk before it has one unit here
        for (int u = 0; u <= U; ++u) {
            if (u < U) {
                const int b = u & 1;
                const uint32_t tS = lane_base + 256 * b;
                ok = mbar_wait(b_sf(b), (u >> 1) & 1, status, 143);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                // (rows m >= L are never stored, and for m < L every m' <= m lies in the chunk)
#pragma unroll
                for (int cc = 0; cc < 2; ++cc) {
                    const int c0 = col0 + cc * 32;         // the warp's rows are [32 quarter, + 32)
                    uint32_t pw[16];
                    if (c0 > 32 * quarter) {               // behind all of them
#pragma unroll
                        for (int x = 0; x < 16; ++x) pw[x] = 0;
                    } else {
                        float v[32];
                        tmem_ld32(tS + c0, v);
                        tmem_wait_ld();
                        if (column) {
                            const float4* w4 = reinterpret_cast<const float4*>(ctab + c0);
#pragma unroll
                            for (int x = 0; x < 8; ++x) {
                                const float4 w = w4[x];
                                v[4 * x] *= w.x;
                                v[4 * x + 1] *= w.y;
                                v[4 * x + 2] *= w.z;
                                v[4 * x + 3] *= w.w;
                            }
                        } else {
#pragma unroll
                            for (int x = 0; x < 32; ++x) v[x] *= p.scale * ctab[max(m - c0 - x, 0)];
                        }
                        if (c0 == 32 * quarter) {
#pragma unroll
                            for (int x = 0; x < 32; ++x) v[x] = x <= lane ? v[x] : 0.f;
                        }
#pragma unroll
                        for (int x = 0; x < 16; ++x) pw[x] = pack_bf16x2(v[2 * x], v[2 * x + 1]);
                    }
                    tmem_st16(tS + col0 + cc * 16, pw);    // over columns that this thread has read
                }
                // the rows behind a ragged chunk are another node's: zeros in the last 16 that the product
                // reads (0 times an infinity there would not be 0)
                if (n == first && (L & 15)) {
                    // A barrier tells a phase from the next one alone: of a chunk before this one with one unit here, V
                    // may still be under way until its products have ended (with more units the first ones' are behind A)
                    if (alone) ok = mbar_wait(b_o((u - 1) & 1), ((u - 1) >> 1) & 1, status, 147);
                    if (ok) ok = mbar_wait(b_v, i & 1, status, 144);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    if (m >= L && m < ((L + 15) & ~15)) {
                        uint4* v = reinterpret_cast<uint4*>(smem + kOutV + grp * kHalf + m * 128);
#pragma unroll
                        for (int c = 0; c < 8; ++c) v[c] = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                }
                if (!column) {
                    // f(m) q_m over features [col0, col0 + 64) out of the swizzled slot
                    const uint8_t* qrow = smem + kOutQ + q * kTile + grp * kHalf + m * 128;
#pragma unroll
                    for (int h2 = 0; h2 < 2; ++h2) {
                        uint32_t qw[16];
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const uint4 x = *reinterpret_cast<const uint4*>(qrow + (((h2 * 4 + c) ^ (m & 7)) << 4));
                            const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                qw[4 * c + e] = pack_bf16x2(fo * __uint_as_float(xs[e] << 16),
                                                            fo * __uint_as_float(xs[e] & 0xffff0000u));
                        }
                        tmem_st16(tS + col0 + 32 + h2 * 16, qw);
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(b_p(b));
            }
            if (u > 0) {
                const int b = (u - 1) & 1;
                const uint32_t tO = lane_base + 256 * b + 128 + col0;
                ok = mbar_wait(b_o(b), ((u - 1) >> 1) & 1, status, 145);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                const bool whole = prev_L >= 32 * quarter + 32;   // all of the warp's rows are the chunk's
                if (whole && lane == 0) bulk_wait_read_all();     // the last store has read its rows
                __syncwarp();
                uint4* dst = reinterpret_cast<uint4*>(p.out + ((size_t)(prev_off + m) * p.hq + prev_h) * kD + col0);
#pragma unroll
                for (int cc = 0; cc < 2; ++cc) {
                    float v[32];
                    tmem_ld32(tO + cc * 32, v);
                    tmem_wait_ld();
                    if (column) {
#pragma unroll
                        for (int x = 0; x < 32; ++x) v[x] *= fo;
                    }
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const uint4 y = pack8(v + 8 * x);
                        if (whole) st_shared_v4(stage + sw128_offset(lane, cc * 4 + x), y.x, y.y, y.z, y.w);
                        else if (m < prev_L) dst[cc * 4 + x] = y;
                    }
                }
                tc_fence_before();
                mbar_arrive(b_oe(b));              // buffer b's O may take the unit after next
                if (whole) {
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        tma_store_3d(&tm_o, stage, col0, prev_h, prev_off + 32 * quarter);
                        bulk_commit();
                    }
                }
            }
            prev_off = off;
            prev_L = L;
            prev_h = h0 + n;
            q = q == kQSlots - 1 ? 0 : q + 1;
            if (++n == G) {
                alone = first == G - 1;
                n = first = head_of(++i);
                if (i < n_items) {
                    off = p.chunks[4 * chunk_of(i)];
                    L = p.chunks[4 * chunk_of(i) + 1];
                }
            }
        }
        if (lane == 0) bulk_wait_all();
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// The walks of a depth of few nodes whose long ones are cut into segments: first those whose sums are taken, then all.
struct Split {
    Walk sums[kMaxWalks], all[kMaxWalks];
    int n_sums, n_all, places;                 // places in `sums`: segments but a node's last, a root's start state
};

// Whether anything is cut (by a GB300's SMs, whatever the device has: the workspace's size is known without one; where
// fewer run at a time the pieces take turns).  As many pieces as run at a time in narrow CTAs (four to a kv-head; of 128 chunks on in wide
// ones, and where that cuts nothing), 16 at most; two launches of s chunks take as long as 2 s + 4 in one.
// Measured, us of a call of one node, 8 kv-heads: 16 chunks 27 whole, 25.5 in 4 pieces, 28.6 in 2; 24 chunks
// 37 and 33 (4); 40 chunks 62, 49 (4), 53 (7); 63 chunks 92, 69 (4), 73 (9); 235 chunks 306, 212 (4), 193 (9), 222 (16).
// Of 2 kv-heads 16 chunks 26 and 22 (4); 40 chunks 56, 41 (5), 37 (10); 235 chunks 290, 147 (9), 135 (16), 153 (20).
bool split_depth(const LinInfo& X, size_t l, int32_t hkv, Split& out) {
    const int32_t lo = X.lvl_ptr[l], m = X.lvl_ptr[l + 1] - lo;
    if (m > kSplitNodes) return false;
    int64_t total = 0;
    for (int32_t i = 0; i < m; ++i) total += X.lnodes[4 * (size_t)X.lvl_nodes[lo + i] + 2];
    const int narrow = (int)(152 / (4 * (int64_t)hkv)), wide = (int)(152 / (2 * (int64_t)hkv));
    for (const int n : {total < 128 && m <= narrow ? narrow : 0, wide}) {
        out.n_sums = out.n_all = out.places = 0;
        for (int32_t i = 0; i < m; ++i) {
            const int32_t k = X.lvl_nodes[lo + i], c = X.lnodes[4 * (size_t)k + 2];
            int64_t pieces = std::min<int64_t>(c * (int64_t)std::min(n, kSplitWalks) / total, c / 4);
            int32_t s = pieces > 1 ? (int32_t)((c + pieces - 1) / pieces) : c;
            if (2 * s + 4 >= c) s = c;
            const int32_t whole = (c - 1) / s;
            for (int32_t t = 0; t <= whole; ++t) {
                const int32_t* node = &X.walks[8 * (size_t)(lo + i)];
                const Walk w = {node[0], node[1], node[2] + t * s, std::min(s, c - t * s), node[4] + t * s * kChunk,
                                t < whole ? kChunk : node[5], node[6], 0, t * s, s, whole, out.places};
                if (t < whole) out.sums[out.n_sums++] = w;
                out.all[out.n_all++] = w;
            }
            out.places += whole + (whole > 0 && X.lnodes[4 * (size_t)k] < 0);
        }
        if (out.n_sums) return true;
    }
    return false;
}

struct Ws {
    size_t s_in, s_out, sums, total;
};
Ws layout(const tree_attn_plan_s* P, int32_t hkv) {
    const size_t nc = P->lin.chunks.size() / 4, per = (size_t)hkv * kD * kD;
    const size_t s_out = nc * per * 2, sums = s_out + (size_t)P->lin.n_inner * per * 4;
    int places = 0;                            // (the depths take turns)
    for (size_t l = 0; l + 1 < P->lin.lvl_ptr.size(); ++l) {
        Split x;
        if (split_depth(P->lin, l, hkv, x)) places = std::max(places, x.places);
    }
    return {0, s_out, sums, sums + (size_t)places * per * 4};
}

}  // namespace

}  // namespace treeattn

using namespace treeattn;

extern "C" {

int tree_attn_linear_prefill_workspace_size(tree_attn_plan_t P, int32_t hkv, int32_t d, size_t* ws_bytes) {
    if (!P || hkv <= 0 || !ws_bytes) return TREE_ATTN_ERR_INVALID_ARG;
    if (d != kD || P->block != kChunk) return TREE_ATTN_ERR_UNSUPPORTED;
    const int st = linear_chunks(P);
    if (st) return st;
    *ws_bytes = layout(P, hkv).total;
    return TREE_ATTN_OK;
}

int tree_attn_linear_prefill(tree_attn_plan_t P, const void* q, const void* k, const void* v, void* o, float* states,
                             int32_t n_slots, const int32_t* slot_in, const int32_t* slot_out, const float* decay,
                             int32_t hq, int32_t hkv, int32_t d, float scale, void* workspace, size_t ws_bytes,
                             void* stream) {
    if (!P || !q || !k || !v || !o || !decay || hq <= 0 || hkv <= 0 || hq % hkv != 0) return TREE_ATTN_ERR_INVALID_ARG;
    if (n_slots < 0 || (n_slots > 0 && !states)) return TREE_ATTN_ERR_INVALID_ARG;
    if (d != kD || P->block != kChunk) return TREE_ATTN_ERR_UNSUPPORTED;
    if (!(scale > 0.f) || !std::isfinite(scale)) return TREE_ATTN_ERR_INVALID_ARG;
    for (const void* p : {q, k, v, (const void*)o, (const void*)states})
        if (!aligned(p, 16)) return TREE_ATTN_ERR_ALIGNMENT;
    if (!aligned(decay, 4) || !aligned(slot_in, 4) || !aligned(slot_out, 4) || !aligned(workspace, 256))
        return TREE_ATTN_ERR_ALIGNMENT;
    DevicePlan* D = nullptr;
    int st = ensure_linear(P, &D);
    if (st) return st;
    const Ws w = layout(P, hkv);
    if (!workspace || ws_bytes < w.total) return TREE_ATTN_ERR_WORKSPACE;
    const int64_t nc = (int64_t)(P->lin.chunks.size() / 4);
    if (nc * hq > INT32_MAX || nc * kChunk > INT32_MAX || nc * hkv * 4 > INT32_MAX) return TREE_ATTN_ERR_TOO_LARGE;
    int dev, *status;
    if ((st = current_device(&dev)) || (st = get_status_ptr(dev, &status))) return st;
    char* ws = static_cast<char*>(workspace);
    void* s_in = ws + w.s_in;
    CUtensorMap tq, tk, tv, tv32, ts, ts32, to32;
    if ((st = make_tensor_map(&tq, q, P->N, hq, d)) || (st = make_tensor_map(&tk, k, P->N, hkv, d)) ||
        (st = make_tensor_map(&tv, v, P->N, hkv, d)) || (st = make_tensor_map(&ts, s_in, nc * kChunk, hkv, d)) ||
        (st = make_tensor_map_cols(&ts32, s_in, nc * kChunk, hkv, d, 32, 32, CU_TENSOR_MAP_SWIZZLE_NONE)) ||
        (st = make_tensor_map_cols(&tv32, v, P->N, hkv, d, 32, kChunk, CU_TENSOR_MAP_SWIZZLE_64B)) ||
        (st = make_tensor_map_rows(&to32, o, P->N, hq, d, 32)))
        return st;
    static std::once_flag once[kMaxDevices];
    static cudaError_t set[kMaxDevices];
    static int sms[kMaxDevices];
    std::call_once(once[dev], [&] {
        set[dev] = launched(cudaFuncSetAttribute(prefill_state_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 StateLayout<64>::kSmem));
        if (set[dev] == cudaSuccess)
            set[dev] = launched(cudaFuncSetAttribute(prefill_state_kernel<32>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                     StateLayout<32>::kSmem));
        if (set[dev] == cudaSuccess)
            set[dev] = launched(cudaFuncSetAttribute(prefill_out_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kOutSmem));
        if (cudaDeviceGetAttribute(&sms[dev], cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms[dev] <= 0) sms[dev] = 1;
    });
    if (set[dev] != cudaSuccess) return TREE_ATTN_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const LinInfo& X = P->lin;
    StateParams p = {};
    p.decay = decay;
    p.s_out = reinterpret_cast<float*>(ws + w.s_out);
    p.sums = reinterpret_cast<float*>(ws + w.sums);
    p.hkv = hkv;
    p.n_inner = P->lin.n_inner;
    p.n_chunks = (int32_t)nc;
    p.leads = 1;
    p.io = {states, slot_in, slot_out, n_slots, status};
    auto walk = [&](int jobs) {
        // where they all run at a time, CTAs of 32 value features: a chunk takes them less long
        const bool narrow = (int64_t)jobs * hkv * 4 <= sms[dev];
        const dim3 grid((unsigned)((int64_t)jobs * hkv * (narrow ? 4 : 2)));
        const cudaError_t e =
            narrow ? launch_pdl(prefill_state_kernel<32>, grid, dim3(kStateThreads), StateLayout<32>::kSmem, s, tk, tv32, ts32, p)
                   : launch_pdl(prefill_state_kernel<64>, grid, dim3(kStateThreads), StateLayout<64>::kSmem, s, tk, tv, ts32, p);
        p.leads = 0;
        return e == cudaSuccess;
    };
    for (size_t l = 0; l + 1 < X.lvl_ptr.size(); ++l) {
        p.first_depth = l == 0;
        Split x;
        bool sent;
        if (split_depth(X, l, hkv, x)) {
            p.order = nullptr;
            p.adding = 1;
            std::copy(x.sums, x.sums + x.n_sums, p.walks);
            sent = walk(x.n_sums);
            p.adding = 0;
            std::copy(x.all, x.all + x.n_all, p.walks);
            sent = sent && walk(x.n_all);
        } else {
            p.order = reinterpret_cast<const int4*>(D->lin_walks) + 2 * (size_t)X.lvl_ptr[l];
            sent = walk(X.lvl_ptr[l + 1] - X.lvl_ptr[l]);
        }
        if (!sent) return TREE_ATTN_ERR_CUDA;
    }
    // about one CTA per SM
    const int G = hq / hkv, lanes = std::max(1, sms[dev] / hkv);
    const int left = (int)(nc % lanes) * G, share = (left + lanes - 1) / lanes;
    const int used = nc >= lanes ? lanes : (left + share - 1) / share;
    const OutParams po = {D->chunks, decay, static_cast<uint16_t*>(o), (int32_t)nc, lanes, share, hq, hkv, scale, status};
    const cudaError_t e = launch_pdl(prefill_out_kernel, dim3((unsigned)(used * hkv)), dim3(kThreads), kOutSmem, s,
                                     tq, tk, tv, ts, to32, po);
    return e == cudaSuccess ? TREE_ATTN_OK : TREE_ATTN_ERR_CUDA;
}

}  // extern "C"
