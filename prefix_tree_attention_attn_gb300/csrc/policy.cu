// Clipped policy loss of the trajectories and its gradient for the compact logits
// (include/tree_loss.h).
//
// One pass over the logits.  A cluster of C CTAs takes a row, a slice each in shared memory, and goes
// from row to row; each logit is read once (2 bytes) and its gradient written once (2 bytes).
//
//   producer     a warp of its own: the predictions of the rows to come (their tables, weights,
//                old log-probs ... are loaded up to three rows ahead, one dependent load a row),
//                whether a row has any weight, and the bulk copies of the slices.
//   statistics   m = max x, S = sum 2^a, T = sum 2^a a with a = (x - m) log2 e, by thread and warp; a
//                warp's three numbers go to every CTA of the cluster by asynchronous stores that
//                count on its barrier, and each warp joins what comes: LSE = m + ln S,
//                H = ln S - ln 2 T / S.  With room for two rows or more the next row's statistics are
//                taken first, so that the exchange is not waited for.
//   predictions  every warp works out the row's g_k for itself where the row has at most 32 predictions
//                of one target (inside a segment: one for each trajectory through it), so
//                nothing is waited for; other rows all warps of the CTA.
//   gradient     2^a (cG + cE (a - T / S)), cG = -sum g / S, cE = entropy_coef ln 2 sum w / S,
//                rounded once; the target's g_k are added before that.  A row of several
//                targets gets those elements afterwards (children with the same token id summed in
//                their order).
//
// Whether a ratio lies beyond the clip decides a whole gradient, so lp - old is a pair of floats:
// ln S = k ln 2 + ln f, f near 1, adds no error beyond 3e-8.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <array>
#include <cmath>
#include <mutex>
#include <vector>

#include "kernels.h"
#include "plan.h"
#include "tree_loss.h"

namespace cg = cooperative_groups;

namespace treeattn {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kMaxWarps = 8;                   // that compute
constexpr int kMaxSlots = 3;
constexpr int kMaxSlice = 66 * 1024;           // bytes of a CTA's slice
constexpr int64_t kMaxVocab = 262144;
constexpr float kFar = -1e30f;                 // in place of -inf where it meets a factor 0
constexpr float kHuge = 0x1p100f;              // beyond this a multiple of a logit may overflow

struct Params {
    const uint16_t* logits;
    int64_t stride, vocab;
    const int32_t* tokens;
    const float* old;
    const float* adv;
    const float* weights;
    const float* ref;
    int32_t per_token;
    float each;                                // weight of every prediction where there is no list
    float top_ratio, low_ratio;                // 1 + clip_high, 1 - clip_low
    float top_log, top_log_lo, low_log, low_log_lo;
    float kl, ent, grad_scale;
    const int4* rows;                          // {first prediction, predictions, first target, targets}
    const int4* pred;                          // {prediction, target row, trajectory, 0} by row, then target
    const int4* targets;                       // {target row, first prediction, predictions, 0}
    float* logprobs;
    float* entropy;
    float* row_loss;                           // [N]
    float* tx;                                 // [N] logit of a target (rows of several), by target row
    float* tg;                                 // [N] its sum of g
    uint16_t* dlogits;
    int64_t d_stride;
    int32_t N;
    int64_t n_pred;
    int* status;
};

__device__ __forceinline__ float lo16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi16(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// a + b = s + e exactly
__device__ __forceinline__ float two_sum(float a, float b, float& e) {
    const float s = a + b, bb = s - a;
    e = (a - (s - bb)) + (b - bb);
    return s;
}

// The exponent of x against the maximum m; far below it counts as 1e30 below, so that 0 meets no infinity
// (+inf and NaN are told by m alone).
__device__ __forceinline__ float exponent(float x, float m) { return fmaxf(x - m, kFar) * kLog2e; }

// A maximum m, and the sums of e = 2^exponent and e * exponent over some logits.
struct Stat {
    float m, s, t;
};

// What the predictions of a row need of it.
struct Row {
    float m;                                   // NaN where the row has no distribution
    float lk, ll;                              // ln S = lk + ll, lk a multiple of 2^-16
    float h;                                   // entropy
};

struct Sums {
    float g, w, loss;
};

// One prediction with weight w: adds to the sums, returns its log-prob.
__device__ __forceinline__ float predict(const Params& p, const Row& row, float w, float x, float old, bool has_old, float a,
                                         float ref, Sums& sum) {
    float e1, e2, e3;
    const float h1 = two_sum(x - row.m, -row.lk, e1), h2 = two_sum(h1, -row.ll, e2);
    const float lo = fabsf(h2) < INFINITY ? e1 + e2 : 0.f;   // lp = h2 + lo; a target at -inf leaves no error terms
    float dh = h2 == h2 ? 0.f : h2, dl = 0.f;
    if (has_old) {
        dh = two_sum(h2, -old, e3);
        dl = fabsf(dh) < INFINITY ? e3 + lo : 0.f;
    }
    const float ratio = fast_exp2((dh + dl) * kLog2e);
    float pg = -a * ratio, g = pg;
    if (a > 0.f && (dh - p.top_log) + (dl - p.top_log_lo) > 0.f) {
        pg = -a * p.top_ratio;
        g = 0.f;
    } else if (a < 0.f && (dh - p.low_log) + (dl - p.low_log_lo) < 0.f) {
        pg = -a * p.low_ratio;
        g = 0.f;
    } else if (a == 0.f) {
        pg = g = dh == dh ? 0.f : dh;
    } else if (dh != dh) {
        pg = g = dh;
    }
    float loss = pg - p.ent * row.h;
    if (p.kl != 0.f) {
        // k3 = e^far - far - 1, em = e^far - 1: by the series where the differences would lose their digits
        const float far = (ref - h2) - lo;
        float em, k3;
        if (fabsf(far) < 0.25f) {
            k3 = far * far * (0.5f + far * (1.f / 6 + far * (1.f / 24 + far * (1.f / 120 + far * (1.f / 720)))));
            em = far + k3;
        } else {
            em = fast_exp2(far * kLog2e) - 1.f;
            k3 = far == INFINITY ? far : em - far;
        }
        loss += p.kl * k3;
        g -= p.kl * em;
    }
    sum.g += w * g;
    sum.w += w;
    sum.loss += w * loss;
    return h2 + lo;
}

// What the producer knows of a row.
struct Meta {
    int active, narrow;                        // some weight; at most 32 predictions of one target
    int first, n, t0, nt;                      // predictions, targets
    int y;                                     // the one target's token
    int k[32];                                 // narrow: each lane's prediction
    float w[32], old[32], a[32], ref[32];
};

struct Shared {
    uint64_t full[kMaxSlots], empty[kMaxSlots];
    uint64_t stat[2];                          // the cluster's warps have sent their sums, rows in turn
    uint64_t read;                             // the cluster's warps have read a row's targets
    uint64_t cta;                              // the CTA's warps have come this far
    float4 stats[2][8 * kMaxWarps];            // {m, S, T, target's logit or 0} by CTA of the cluster and warp
    Sums sums[kMaxWarps];
    Meta meta[kMaxSlots];
};
constexpr int kSlots0 = (sizeof(Shared) + 127) / 128 * 128;   // where the ring begins

__device__ __forceinline__ float advantage(const Params& p, int4 e) { return p.adv[p.per_token ? e.x : e.z]; }

// The predictions [first, first + n) of one target with logit x, by the threads `at`, `at` + step, ...
__device__ __forceinline__ void predict_all(const Params& p, const Row& row, int first, int n, float x, int at, int step,
                                            bool writes, Sums& sum) {
    for (int i = at; i < n; i += step) {
        const int4 e = p.pred[first + i];
        if (!ta_ok(p.status, 602, e.x, 0, p.n_pred)) continue;
        const float w = p.weights ? p.weights[e.x] : p.each;
        float lp = 0.f;
        if (w != 0.f)
            lp = predict(p, row, w, x, p.old ? p.old[e.x] : 0.f, p.old != nullptr, advantage(p, e),
                         p.kl != 0.f ? p.ref[e.x] : 0.f, sum);
        if (writes && p.logprobs) p.logprobs[e.x] = lp;
    }
}

__device__ __forceinline__ Sums warp_sum(Sums s) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        s.g += __shfl_xor_sync(0xffffffffu, s.g, o);
        s.w += __shfl_xor_sync(0xffffffffu, s.w, o);
        s.loss += __shfl_xor_sync(0xffffffffu, s.loss, o);
    }
    return s;
}

// The sums of a warp's lanes against their common maximum.
__device__ __forceinline__ Stat warp_join(Stat a) {
    Stat r;
    asm("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r.m) : "f"(a.m));
    const float d = exponent(a.m, r.m), e = fast_exp2(d);
    r.s = a.s * e;
    r.t = fmaf(a.s, d, a.t) * e;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        r.s += __shfl_xor_sync(0xffffffffu, r.s, o);
        r.t += __shfl_xor_sync(0xffffffffu, r.t, o);
    }
    return r;
}

__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// The address of this CTA's shared memory word in another CTA of the cluster.
__device__ __forceinline__ uint32_t at_rank(uint32_t addr, int rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
// 16 bytes to another CTA, counted on its barrier.
__device__ __forceinline__ void remote_store(uint32_t addr, float4 v, uint32_t bar) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(addr),
                 "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void remote_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// mbar_wait for arrivals from the whole cluster.
__device__ __forceinline__ bool wait_cluster(uint32_t bar, uint32_t parity, int* status, int where) {
    auto done = [&] {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
        return ok != 0;
    };
    if (done()) return true;
    const uint64_t t0 = globaltimer_ns();
    while (true) {
        for (int k = 0; k < 64; ++k)
            if (done()) return true;
        if (*reinterpret_cast<volatile int*>(status) != 0) return false;
        if (globaltimer_ns() - t0 > kWaitLimitNs) break;
    }
    report_status(status, -10 - 1000 * where);
    return false;
}

// A CTA's slice of a row as 16-byte vectors, the first and the last of which may belong to it in part.
struct Slice {
    const uint16_t* x;                         // the row
    int shift, V, lo, hi;                      // vectors [lo, hi), of which [first, last) are whole
    int first, last;
    __device__ __forceinline__ Slice(const Params& p, int64_t r, int me, int log_c) {
        x = p.logits + r * p.stride;
        V = (int)p.vocab;
        shift = (int)((reinterpret_cast<uintptr_t>(x) & 15u) >> 1);
        const int vectors = (V + shift + 7) / 8, per = (vectors + (1 << log_c) - 1) >> log_c;
        lo = min(me * per, vectors);
        hi = min(lo + per, vectors);
        first = lo + (lo < hi && start(lo) < 0);
        last = max(first, hi - (lo < hi && start(hi) > V));
    }
    __device__ __forceinline__ int start(int v) const { return 8 * v - shift; }
    // a vector that is not whole, element by element
    __device__ __forceinline__ uint4 part(int v) const {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int a = start(v) + 2 * i, b = a + 1;
            u[i] = (a >= 0 && a < V ? x[a] : 0xff80u) | ((b >= 0 && b < V ? x[b] : 0xff80u) << 16);   // -inf outside
        }
        return make_uint4(u[0], u[1], u[2], u[3]);
    }
    // the vector with token y, or -1 where that is not this CTA's
    __device__ __forceinline__ int owns(int y) const {
        const int v = (y + shift) / 8;
        return y >= 0 && y < V && v >= lo && v < hi ? v : -1;
    }
    // the vector in part that falls to this thread: the last one's, and the one's before it; or -1
    __device__ __forceinline__ int odd(int tid, int T) const {
        return tid == T - 1 && lo < first ? lo : tid == T - 2 && last < hi ? last : -1;
    }
    __device__ __forceinline__ float logit(const uint8_t* slot, int y) const {
        const int v = (y + shift) / 8;
        return lo16(v >= first && v < last ? *reinterpret_cast<const uint16_t*>(slot + (size_t)(v - lo) * 16 + (y - start(v)) * 2)
                                           : x[y]);
    }
};

// The producer's loads of one row, in three steps that depend on one another.
struct Ahead {
    int4 info, mine;
    float w, old, a, ref;
    int y;
};
__device__ __forceinline__ bool is_narrow(int4 info) { return info.w == 1 && info.y <= 32; }
__device__ __forceinline__ void load_info(const Params& p, int64_t r, Ahead& x) {
    x.info = r < p.N ? p.rows[r] : make_int4(0, 0, 0, 0);
    if (!(ta_ok(p.status, 600, x.info.x, 0, p.n_pred + 1) && ta_ok(p.status, 601, (long long)x.info.x + x.info.y, 0, p.n_pred + 1)))
        x.info = make_int4(0, 0, 0, 0);
}
__device__ __forceinline__ void load_pred(const Params& p, int lane, Ahead& x) {
    x.mine = make_int4(-1, 0, 0, 0);
    if (is_narrow(x.info) && lane < x.info.y) {
        x.mine = p.pred[x.info.x + lane];
        if (!ta_ok(p.status, 602, x.mine.x, 0, p.n_pred)) x.mine.x = -1;
    }
}
__device__ __forceinline__ void load_values(const Params& p, int64_t r, Ahead& x) {
    x.w = x.old = x.a = x.ref = 0.f;
    x.y = -1;
    if (x.mine.x >= 0) {
        x.w = p.weights ? p.weights[x.mine.x] : p.each;
        if (p.old) x.old = p.old[x.mine.x];
        x.a = p.adv[p.per_token ? x.mine.x : x.mine.z];
        if (p.kl != 0.f) x.ref = p.ref[x.mine.x];
    }
    // one target: it is the next packed row (a node's tokens and its only child follow each other)
    if (x.info.w == 1 && ta_ok(p.status, 603, r + 1, 0, p.N)) x.y = p.tokens[r + 1];
}

__global__ void __maxnreg__(96) policy_kernel(const Params p, int n_slots, int slot_bytes) {
    extern __shared__ __align__(128) uint8_t smem[];
    Shared& S = *reinterpret_cast<Shared*>(smem);
    cg::cluster_group cluster = cg::this_cluster();
    const int C = (int)cluster.num_blocks(), me = (int)cluster.block_rank();
    const int log_c = __ffs(C) - 1;
    const int nw = (int)blockDim.x / 32 - 1, T = 32 * nw, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t cluster0 = blockIdx.x / C, clusters = gridDim.x / C;
    if (tid == 0) {
        for (int i = 0; i < n_slots; ++i) {
            mbar_init(smem_u32(&S.full[i]), 1);
            mbar_init(smem_u32(&S.empty[i]), nw);
        }
        mbar_init(smem_u32(&S.stat[0]), 1);
        mbar_init(smem_u32(&S.stat[1]), 1);
        mbar_init(smem_u32(&S.read), C * nw);
        mbar_init(smem_u32(&S.cta), nw);
        fence_mbar_init();
        for (int i = 0; i < 2; ++i) mbar_expect_tx(smem_u32(&S.stat[i]), 16 * C * nw);   // of the next row on this barrier
    }
    cluster.sync();                            // every CTA of the cluster runs, its barriers are set up
    grid_dep_wait();
    grid_dep_launch();

    if (warp == nw) {
        // ---- the producer -------------------------------------------------------------------
        Ahead one, two, three;                 // this row and the next two
        load_info(p, cluster0, one);
        load_info(p, cluster0 + clusters, two);
        load_info(p, cluster0 + 2 * clusters, three);
        load_pred(p, lane, one);
        load_pred(p, lane, two);
        load_values(p, cluster0, one);
        int it = 0, used = 0;
        bool ok = true;
        for (int64_t r = cluster0; r < p.N && ok; r += clusters, ++it) {
            const int slot = it % n_slots, turn = it / n_slots;
            Ahead four;
            load_info(p, r + 3 * clusters, four);
            load_pred(p, lane, three);
            load_values(p, r + clusters, two);
            const bool narrow = is_narrow(one.info);
            const int n = one.info.y;
            bool active = n > 0;
            if (narrow) {
                active = __any_sync(0xffffffffu, one.w != 0.f);
            } else if (active && p.weights) {
                bool any = false;
                for (int i = lane; i < n && !any; i += 32) {
                    const int k = p.pred[one.info.x + i].x;
                    any = ta_ok(p.status, 602, k, 0, p.n_pred) && p.weights[k] != 0.f;
                }
                active = __any_sync(0xffffffffu, any);
            }
            if (turn > 0) ok = mbar_wait(smem_u32(&S.empty[slot]), (turn - 1) & 1, p.status, 601);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            Meta& m = S.meta[slot];
            m.k[lane] = one.mine.x;
            m.w[lane] = one.w;
            m.old[lane] = one.old;
            m.a[lane] = one.a;
            m.ref[lane] = one.ref;
            if (lane == 0) {
                m.active = active;
                m.narrow = narrow;
                m.first = one.info.x;
                m.n = n;
                m.t0 = one.info.z;
                m.nt = one.info.w;
                m.y = one.y;
            }
            __syncwarp();
            if (lane == 0) {
                const uint32_t bar = smem_u32(&S.full[slot]);
                const Slice s(p, r, me, log_c);
                const uint32_t bytes = (uint32_t)(s.last - s.first) * 16;
                if (active && bytes) {
                    mbar_expect_tx(bar, bytes);
                    bulk_load(smem_u32(smem + kSlots0 + (size_t)slot * slot_bytes + (size_t)(s.first - s.lo) * 16),
                              s.x + s.start(s.first), bytes, bar);
                } else {
                    mbar_arrive(bar);
                }
            }
            one = two;
            two = three;
            three = four;
            used = it + 1;
        }
        // copies still under way where a wait gave up
        if (!ok)
            for (int i = max(0, used - n_slots); i < used; ++i)
                mbar_wait(smem_u32(&S.full[i % n_slots]), (i / n_slots) & 1, p.status, 602);
    } else {
        // ---- the rows ----------------------------------------------------------------------
        const uint64_t c2 = f32x2(kLog2e, kLog2e);
        const bool ahead = n_slots > 1;        // the next row's statistics before this row is finished
        int reads = 0, meets = 0;
        bool ok = true;
        // all warps of the CTA have come this far, and see each other's writes
        auto meet = [&] {
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&S.cta));
            ok = mbar_wait(smem_u32(&S.cta), meets++ & 1, p.status, 603) && ok;
            ok = __all_sync(0xffffffffu, ok);
        };
        struct Begun {
            int64_t r;
            int slot, k;                       // its place in the ring, among the rows of some weight (-1: none)
            Stat st;                           // of this warp, then of the row
            float xy;
        };

        auto begin = [&](int64_t r, int it, int actives) {
            Begun b;
            b.r = r;
            b.slot = it % n_slots;
            b.k = -1;
            ok = mbar_wait(smem_u32(&S.full[b.slot]), (it / n_slots) & 1, p.status, 604);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok || !S.meta[b.slot].active) return b;   // (the same in every CTA of the cluster)
            b.k = actives;
            const Slice s(p, r, me, log_c);
            const int odd = s.odd(tid, T);
            const uint4* here = reinterpret_cast<const uint4*>(smem + kSlots0 + (size_t)b.slot * slot_bytes) - s.lo;
            Stat st;
            uint32_t m2 = 0xff80ff80u, n2 = 0xff80ff80u;
#pragma unroll 4
            for (int v = s.first + tid; v < s.last; v += T) {
                const uint4 x = here[v];
                m2 = max2_nan(m2, max2_nan(x.x, x.y));
                n2 = max2_nan(n2, max2_nan(x.z, x.w));
            }
            uint4 rest = make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u);
            if (odd >= 0) {
                rest = s.part(odd);
                m2 = max2_nan(m2, max2_nan(rest.x, rest.y));
                n2 = max2_nan(n2, max2_nan(rest.z, rest.w));
            }
            m2 = max2_nan(m2, n2);
            st.m = max_nan(lo16(m2), hi16(m2));
            if (fabsf(st.m) < kHuge) {
                const uint64_t minus = f32x2(-st.m, -st.m);
                // what lies far enough below is 0 all the same, and then finite
                const float far = st.m - fmaxf(256.f, fabsf(st.m) * 0x1p-6f);
                const uint32_t far2 = pack_bf16x2(far, far);
                uint64_t sum_s = 0, sum_t = 0, more_s = 0, more_t = 0;
                auto add = [&](uint32_t u, uint64_t& ss, uint64_t& tt) {
                    u = max2(u, far2);
                    const uint64_t a = mul_f32x2(add_f32x2(f32x2(lo16(u), hi16(u)), minus), c2);
                    float a0, a1;
                    f32x2_split(a, a0, a1);
                    const uint64_t e = f32x2(fast_exp2(a0), fast_exp2(a1));
                    ss = add_f32x2(ss, e);
                    tt = fma_f32x2(e, a, tt);
                };
                auto add4 = [&](uint4 x) {
                    add(x.x, sum_s, sum_t);
                    add(x.y, more_s, more_t);
                    add(x.z, sum_s, sum_t);
                    add(x.w, more_s, more_t);
                };
#pragma unroll 2
                for (int v = s.first + tid; v < s.last; v += T) add4(here[v]);
                if (odd >= 0) add4(rest);
                float a0, a1;
                f32x2_split(add_f32x2(sum_s, more_s), a0, a1);
                st.s = a0 + a1;
                f32x2_split(add_f32x2(sum_t, more_t), a0, a1);
                st.t = a0 + a1;
            } else {
                // masks of the lowest value alone, or huge logits (an infinity and NaN: told by m alone)
                st.s = st.t = 0.f;
                if (fabsf(st.m) < INFINITY)
                    for (int v = s.first + tid; v < s.last + T; v += T) {
                        const uint4 x = v < s.last ? here[v] : rest;
                        const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll 1
                        for (int i = 0; i < 8; ++i) {
                            const float a = exponent(__uint_as_float((u[i / 2] >> (16 * (i & 1))) << 16), st.m), e = fast_exp2(a);
                            st.s += e;
                            st.t = fmaf(e, a, st.t);
                        }
                    }
            }
            b.st = warp_join(st);
            return b;
        };

        // The row's sums out of every warp's of the cluster.
        auto collect = [&](Begun& b) {
            ok = wait_cluster(smem_u32(&S.stat[b.k & 1]), (b.k >> 1) & 1, p.status, 605);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) return;
            if (tid == 0) mbar_expect_tx(smem_u32(&S.stat[b.k & 1]), 16 * C * nw);   // of the row after the next
            b.st = {-INFINITY, 0.f, 0.f};
            b.xy = 0.f;
            for (int i = lane; i < C * nw; i += 32) {
                const float4 q = S.stats[b.k & 1][i];
                if (i == lane) {
                    b.st = {q.x, q.y, q.z};
                } else {                       // (more than 32 warps: two a lane)
                    const float m = max_nan(b.st.m, q.x);
                    const float da = exponent(b.st.m, m), db = exponent(q.x, m), ea = fast_exp2(da), eb = fast_exp2(db);
                    b.st = {m, b.st.s * ea + q.y * eb, fmaf(b.st.s, da, b.st.t) * ea + fmaf(q.y, db, q.z) * eb};
                }
                b.xy += q.w;
            }
            b.st = warp_join(b.st);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) b.xy += __shfl_xor_sync(0xffffffffu, b.xy, o);
        };
        // Only after this warp has collected the row before: when every warp's sums of this row have come, those
        // of the row before have been read everywhere, and the next row's may take their place.
        auto send = [&](const Begun& b) {
            const Slice s(p, b.r, me, log_c);
            const Meta& M = S.meta[b.slot];
            float xy = 0.f;
            if (warp == 0 && M.nt == 1 && s.owns(M.y) >= 0) xy = s.logit(smem + kSlots0 + (size_t)b.slot * slot_bytes, M.y);
            if (lane < C)
                remote_store(at_rank(smem_u32(&S.stats[b.k & 1][me * nw + warp]), lane), make_float4(b.st.m, b.st.s, b.st.t, xy),
                             at_rank(smem_u32(&S.stat[b.k & 1]), lane));
        };

        auto finish = [&](const Begun& b) {
            const int64_t r = b.r;
            const uint8_t* slot = smem + kSlots0 + (size_t)b.slot * slot_bytes;
            const uint32_t empty = smem_u32(&S.empty[b.slot]);
            const Meta& M = S.meta[b.slot];
            const Slice s(p, r, me, log_c);
            uint16_t* row_d = p.dlogits ? p.dlogits + r * p.d_stride : nullptr;
            const bool together = ((reinterpret_cast<uintptr_t>(s.x) ^ reinterpret_cast<uintptr_t>(row_d)) & 15u) == 0;
            auto store = [&](int v, uint4 o) {
                if (together && v >= s.first && v < s.last) {
                    __stcs(reinterpret_cast<uint4*>(row_d + s.start(v)), o);
                } else {
                    const uint32_t u[4] = {o.x, o.y, o.z, o.w};
#pragma unroll 1
                    for (int i = 0; i < 8; ++i)
                        if (s.start(v) + i >= 0 && s.start(v) + i < s.V) row_d[s.start(v) + i] = (uint16_t)(u[i / 2] >> (16 * (i & 1)));
                }
            };
            auto give_back = [&] {
                __syncwarp();
                if (lane == 0) mbar_arrive(empty);
            };
            if (b.k < 0) {
                if (row_d)
                    for (int v = s.lo + tid; v < s.hi; v += T) store(v, make_uint4(0, 0, 0, 0));
                if (me == 0) {
                    if (p.logprobs)
                        for (int i = tid; i < M.n; i += T) {
                            const int k = p.pred[M.first + i].x;
                            if (ta_ok(p.status, 602, k, 0, p.n_pred)) p.logprobs[k] = 0.f;
                        }
                    if (tid == 0) {
                        p.row_loss[r] = 0.f;
                        if (p.entropy) p.entropy[r] = 0.f;
                    }
                }
                give_back();
                return;
            }
            const bool narrow = M.narrow, single = M.nt == 1;
            if (!row_d && narrow && (me != 0 || warp != 0)) {   // one warp tells the row's loss
                give_back();
                return;
            }

            // ---- the row ------------------------------------------------------------------------
            const Stat st = b.st;
            float xy = b.xy;
            const int y = M.y, yv = single ? s.owns(y) : -1;
            if (y < 0 || y >= s.V) xy = __int_as_float(0x7fc00000);
            const float ts = st.t / st.s;
            Row row;
            row.m = fabsf(st.m) < INFINITY ? st.m : __int_as_float(0x7fc00000);
            {
                // S = 2^k f, 0.7 <= f < 1.4 (S >= 1);  ln 2 = 45426 / 2^16 + 1.42860682e-6;
                // ln f = 2 (z + z^3 / 3 + ...), z = (f - 1) / (f + 1), |z| < 0.18: the next term is below 2^-30 z
                const uint32_t bits = __float_as_uint(st.s);
                int k = (int)(bits >> 23) - 127;
                float f = __uint_as_float((bits & 0x7fffffu) | 0x3f800000u);
                if (f >= 1.4f) {
                    f *= 0.5f;
                    ++k;
                }
                const float z = (f - 1.f) / (f + 1.f), z2 = z * z;
                const float poly = z2 * (1.f / 3 + z2 * (1.f / 5 + z2 * (1.f / 7 + z2 * (1.f / 9 + z2 * (1.f / 11)))));
                row.lk = (float)k * (45426.f / 65536.f);
                row.ll = fmaf((float)k, 1.42860682e-6f, 2.f * fmaf(z, poly, z));
            }
            row.h = row.m == row.m ? fmaf(-kLn2, ts, row.lk + row.ll) : row.m;

            // ---- the predictions -----------------------------------------------------------------
            Sums sum = {0.f, 0.f, 0.f};
            if (narrow) {
                float lp = 0.f;
                const float w = M.w[lane];
                if (w != 0.f) lp = predict(p, row, w, xy, M.old[lane], p.old != nullptr, M.a[lane], M.ref[lane], sum);
                if (me == 0 && warp == 0 && M.k[lane] >= 0 && p.logprobs) p.logprobs[M.k[lane]] = lp;
                sum = warp_sum(sum);
            } else {
                // one target, or a warp for each of several
                for (int j = single ? 0 : warp; j < M.nt; j += nw) {
                    const int4 t = single ? make_int4(0, M.first, M.n, 0) : p.targets[M.t0 + j];
                    if (!ta_ok(p.status, 604, t.x, 0, p.N)) continue;
                    const int yj = single ? y : p.tokens[t.x];
                    const float xj = single ? xy : yj >= 0 && yj < s.V ? lo16(s.x[yj]) : __int_as_float(0x7fc00000);
                    Sums part = {0.f, 0.f, 0.f};
                    predict_all(p, row, t.y, t.z, xj, single ? tid : lane, single ? T : 32, me == 0, part);
                    part = warp_sum(part);
                    if (lane == 0) {
                        sum.g += part.g;
                        sum.w += part.w;
                        sum.loss += part.loss;
                        if (!single && s.owns(yj) >= 0) {
                            p.tx[t.x] = xj;
                            p.tg[t.x] = part.g;
                        }
                    }
                    if (single) break;
                }
                if (!single) {
                    // the gradient may lie over the logits: the whole cluster has read the targets' logits
                    __syncwarp();
                    if (lane < C) remote_arrive(at_rank(smem_u32(&S.read), lane));
                    ok = wait_cluster(smem_u32(&S.read), reads++ & 1, p.status, 606);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) return;
                }
                if (lane == 0) S.sums[warp] = sum;
                meet();
                if (!ok) return;
                sum = {0.f, 0.f, 0.f};
                for (int i = 0; i < nw; ++i) {
                    sum.g += S.sums[i].g;
                    sum.w += S.sums[i].w;
                    sum.loss += S.sums[i].loss;
                }
                meet();                        // S.sums has been read
                if (!ok) return;
            }
            if (me == 0 && tid == 0) {
                p.row_loss[r] = sum.loss;
                if (p.entropy) p.entropy[r] = row.h;
            }
            if (!row_d) {
                give_back();
                return;
            }

            // ---- the gradient ----------------------------------------------------------------
            const int odd = s.odd(tid, T);
            const uint4* here = reinterpret_cast<const uint4*>(slot) - s.lo;
            const float cg_ = row.m == row.m ? -p.grad_scale * sum.g / st.s : row.m;
            const float ce = p.ent != 0.f ? kLn2 * p.grad_scale * p.ent * sum.w / st.s : 0.f;
            auto value = [&](float xv) {
                const float a = exponent(xv, row.m);
                return fast_exp2(a) * fmaf(ce, a - ts, cg_);
            };
            auto write = [&](int v, uint32_t (&o)[4]) {
                if (v == yv) {
                    const uint32_t own = pack_bf16x2(value(xy) + p.grad_scale * sum.g, 0.f) & 0xffffu;
                    const int e = y - s.start(v);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (e / 2 == i) o[i] = e & 1 ? (o[i] & 0xffffu) | (own << 16) : (o[i] & 0xffff0000u) | own;
                }
                store(v, make_uint4(o[0], o[1], o[2], o[3]));
            };
            int v = s.first + tid;
            if (ce == 0.f && fabsf(row.m) < kHuge) {
                // (one multiply-add for the exponent: off by 2^-24 of m log2 e, far below the rounding to bf16)
                const uint64_t minus = f32x2(-row.m * kLog2e, -row.m * kLog2e), cg2 = f32x2(cg_, cg_);
#pragma unroll 2
                for (; v < s.last; v += T) {
                    const uint4 x = here[v];
                    const uint32_t u[4] = {x.x, x.y, x.z, x.w};
                    uint32_t o[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float a0, a1;
                        f32x2_split(fma_f32x2(f32x2(lo16(u[i]), hi16(u[i])), c2, minus), a0, a1);
                        f32x2_split(mul_f32x2(f32x2(fast_exp2(a0), fast_exp2(a1)), cg2), a0, a1);
                        o[i] = pack_bf16x2(a0, a1);
                    }
                    write(v, o);
                }
            }
            // the general form, and the vectors in part
#pragma unroll 1
            for (; v < s.last || (odd >= 0 && v < s.last + T); v += T) {
                const uint4 x = v < s.last ? here[v] : s.part(odd);
                const uint32_t u[4] = {x.x, x.y, x.z, x.w};
                uint32_t o[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) o[i] = pack_bf16x2(value(lo16(u[i])), value(hi16(u[i])));
                write(v < s.last ? v : odd, o);
            }
            if (!single) {
                const int t0 = M.t0, nt = M.nt;
                meet();
                if (!ok) return;
                for (int j = tid; j < nt; j += T) {
                    const int q = p.targets[t0 + j].x;
                    if (!ta_ok(p.status, 604, q, 0, p.N)) continue;
                    const int yj = p.tokens[q];
                    if (s.owns(yj) < 0) continue;
                    bool earlier = false;          // another child has the same token: the first one adds them up
                    for (int i = 0; i < j && !earlier; ++i) earlier = p.tokens[p.targets[t0 + i].x] == yj;
                    if (earlier) continue;
                    float g = p.tg[q];
                    for (int i = j + 1; i < nt; ++i) {
                        const int qi = p.targets[t0 + i].x;
                        if (p.tokens[qi] == yj) g += p.tg[qi];
                    }
                    row_d[yj] = (uint16_t)pack_bf16x2(value(p.tx[q]) + p.grad_scale * g, 0.f);
                }
            }
            give_back();
        };

        Begun next, todo;
        todo.r = -1;
        int it = 0, actives = 0;
        for (int64_t r = cluster0; ok; r += clusters, ++it) {
            const bool more = r < p.N;
            next.r = -1;
            next.k = -1;
            if (more) {
                next = begin(r, it, actives);
                if (!ok) break;
                actives += next.k >= 0;
            }
            if (!ahead) {
                todo = next;
                if (todo.k >= 0) send(todo);
            }
            if (todo.r >= 0 && todo.k >= 0) {
                collect(todo);
                if (!ok) break;
            }
            if (ahead && next.k >= 0) send(next);
            if (todo.r >= 0) finish(todo);
            if (!more) break;
            if (ahead) todo = next;
        }
    }
    cluster.sync();                            // nothing is sent to a CTA that has ended
}

// The rows' losses in a fixed order, in pairs of floats.
__global__ void __launch_bounds__(1024) policy_sum_kernel(const float* __restrict__ row_loss, int n, float* __restrict__ loss) {
    __shared__ float sh[2][32];
    grid_dep_wait();
    grid_dep_launch();
    float hi = 0.f, lo = 0.f, e;
    for (int i = threadIdx.x; i < n; i += 1024) {
        hi = two_sum(hi, row_loss[i], e);
        lo += e;
    }
    auto reduce = [&] {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float h2 = __shfl_xor_sync(0xffffffffu, hi, o), l2 = __shfl_xor_sync(0xffffffffu, lo, o);
            hi = two_sum(hi, h2, e);
            lo += l2 + e;
        }
    };
    reduce();
    if ((threadIdx.x & 31) == 0) {
        sh[0][threadIdx.x >> 5] = hi;
        sh[1][threadIdx.x >> 5] = lo;
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        hi = sh[0][threadIdx.x];
        lo = sh[1][threadIdx.x];
        reduce();
        // (an infinite or undefined sum leaves no error term)
        if (threadIdx.x == 0) *loss = fabsf(hi) < INFINITY ? hi + lo : hi;
    }
}

// Predictions by row and target, built once per plan and device.
int ensure_policy(tree_attn_plan_s* P, DevicePlan** out, int64_t* n_pred) {
    int dev;
    int st = current_device(&dev);
    if (st) return st;
    std::lock_guard<std::mutex> lk(P->mu);
    if ((st = build_traj(P))) return st;
    const TrajInfo& X = P->traj;
    const int64_t L = (int64_t)X.leaves.size(), np = (int64_t)X.traj_tok.size() - L;
    *n_pred = np;
    DevicePlan& D = P->dev[dev];
    if (!D.policy_ready) {
        std::vector<int32_t> h;
        int64_t at_pred, at_target;
        try {
            // a target's predictions are the trajectories through it, its row the one before it
            const int64_t N = P->N;
            std::vector<int32_t> row_of(N, -1);
            std::vector<int64_t> first(N + 1, 0);
            for (int64_t l = 0; l < L; ++l)
                for (int64_t q = X.traj_ptr[l]; q + 1 < X.traj_ptr[l + 1]; ++q) row_of[X.traj_tok[q + 1]] = X.traj_tok[q];
            std::vector<int32_t> count(N, 0);                       // targets of each row
            for (int64_t s = 0; s < N; ++s)
                if (row_of[s] >= 0) ++count[row_of[s]];
            int64_t n_targets = 0;
            std::vector<int64_t> target_at(N);
            for (int64_t r = 0; r < N; ++r) {
                target_at[r] = n_targets;
                n_targets += count[r];
            }
            const int64_t rows_words = 4 * N, pred_words = 4 * std::max<int64_t>(np, 1);
            at_pred = (rows_words + 63) / 64 * 64;
            at_target = at_pred + (pred_words + 63) / 64 * 64;
            h.assign(at_target + 4 * std::max<int64_t>(n_targets, 1), 0);
            int32_t *rows = h.data(), *pred = rows + at_pred, *targets = rows + at_target;
            std::vector<int64_t> fill(N, 0);
            for (int64_t s = 0; s < N; ++s) {                       // targets of a row in packed order
                const int32_t r = row_of[s];
                if (r < 0) continue;
                int32_t* t = targets + 4 * (target_at[r] + fill[r]++);
                t[0] = (int32_t)s;
                t[2] = X.mult[s];
            }
            int64_t total = 0;
            std::vector<int64_t> pred_at(N, 0);
            for (int64_t r = 0; r < N; ++r) {
                int32_t* e = rows + 4 * r;
                e[0] = (int32_t)total;
                e[2] = (int32_t)target_at[r];
                e[3] = count[r];
                for (int32_t j = 0; j < count[r]; ++j) {
                    int32_t* t = targets + 4 * (target_at[r] + j);
                    t[1] = (int32_t)total;
                    pred_at[t[0]] = total;
                    total += t[2];
                }
                e[1] = (int32_t)(total - e[0]);
            }
            int64_t k = 0;
            for (int64_t l = 0; l < L; ++l)
                for (int64_t q = X.traj_ptr[l]; q + 1 < X.traj_ptr[l + 1]; ++q, ++k) {
                    const int32_t s = X.traj_tok[q + 1];
                    int32_t* e = pred + 4 * pred_at[s]++;
                    e[0] = (int32_t)k;
                    e[1] = s;
                    e[2] = (int32_t)l;
                }
        } catch (const std::bad_alloc&) {
            return TREE_ATTN_ERR_OUT_OF_MEMORY;
        }
        void* buf = nullptr;
        if ((st = upload_words(&buf, h.data(), h.size()))) return st;
        D.policy_base = buf;
        D.policy_rows = static_cast<int32_t*>(buf);
        D.policy_pred = static_cast<int32_t*>(buf) + at_pred;
        D.policy_targets = static_cast<int32_t*>(buf) + at_target;
        D.policy_ready = true;
    }
    *out = &D;
    return TREE_ATTN_OK;
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

size_t column(const tree_attn_plan_s* P) { return ((size_t)P->N * 4 + 255) / 256 * 256; }

// How a row is cut up: CTAs, warps that compute, slots of the ring.
struct Shape {
    int C, warps, slots, slot_bytes, smem;
};
// What is waited for is the chain from a row's load over its statistics and the exchange to its
// gradient, so many small CTAs of few warps run side by side and a CTA has the row that it works on
// alone; only slices of up to 8 KB are small enough for two rows more.  Measured with the gradient, 9 vocabularies x
// CTAs per row x warps x slots, best first (us, CTAs a row / warps / slots): 152,064 x 4,000 rows
// 523 (8/3/1) 539 (8/4/1) 546 (4/8/1); 100,000 x 4,000 316 (2/8/1) 316 (4/4/1) 340 (4/3/1); 64,000 x 5,000 271 (2/4/1)
// 288 (4/3/1); 32,000 x 10,000 272 (1/4/1) 279 (2/3/1); 16,000 x 20,000 283 (1/3/1) 295 (1/4/1); 4,000 x 20,000
// 143 (1/2/3) 154 (1/2/1).  Few rows are done sooner by more warps: 152,064 x 64 21 (4/8/1) 23 (8/8/1) 25 (8/3/1).
Shape shape_of(int64_t vocab, int64_t rows) {
    const int64_t vectors = (vocab + 7) / 8 + 1;    // (a row may start inside a vector)
    Shape f = {1, 0, 0, 0, 0};
    while (f.C < 8 && (vectors + f.C - 1) / f.C * 16 > kMaxSlice) f.C *= 2;
    const int64_t per = (vectors + f.C - 1) / f.C;
    const int64_t bytes = (per * 16 + 127) / 128 * 128;
    f.warps = rows * f.C <= 304 ? 8 : bytes > 40 * 1024 ? 4 : bytes > 8 * 1024 ? 3 : 2;
    while (f.warps > 1 && per < 32 * f.warps) --f.warps;
    f.slots = bytes > 8 * 1024 ? 1 : kMaxSlots;
    f.slot_bytes = (int)bytes;
    f.smem = kSlots0 + f.slots * f.slot_bytes;
    return f;
}

// Clusters of a launch that run at a time (of 4 and 8 CTAs fewer than the SMs would hold: they keep
// to groups of SMs); 0 where it cannot be told.  Asked once per shape and device.
int clusters_at_a_time(int dev, const Shape& f, const cudaLaunchConfig_t& cfg) {
    static std::mutex mu;
    static std::vector<std::array<int, 5>> known;
    std::lock_guard<std::mutex> lk(mu);
    for (const auto& k : known)
        if (k[0] == dev && k[1] == f.C && k[2] == f.warps && k[3] == f.smem) return k[4];
    int n = 0;
    if (launched(cudaOccupancyMaxActiveClusters(&n, policy_kernel, &cfg)) != cudaSuccess) return 0;
    try {
        known.push_back({dev, f.C, f.warps, f.smem, n});
    } catch (const std::bad_alloc&) {
    }
    return n;
}

void log_pair(double v, float& hi, float& lo) {
    hi = (float)v;
    lo = std::isinf(v) ? 0.f : (float)(v - (double)hi);
}

}  // namespace

}  // namespace treeattn

using namespace treeattn;

extern "C" {

int tree_attn_policy_loss_workspace(tree_attn_plan_t P, size_t* ws_bytes) {
    if (!P || !ws_bytes) return TREE_ATTN_ERR_INVALID_ARG;
    *ws_bytes = 3 * column(P);
    return TREE_ATTN_OK;
}

int tree_attn_policy_loss(tree_attn_plan_t P, const void* logits, int64_t row_stride, int64_t vocab,
                          const int32_t* tokens, const tree_attn_policy_t* c, float* loss, float* logprobs,
                          float* entropy, void* dlogits, int64_t d_stride, void* workspace, size_t ws_bytes,
                          void* stream) {
    if (!P || !logits || !tokens || !c || !loss || vocab < 1 || row_stride < vocab) return TREE_ATTN_ERR_INVALID_ARG;
    if (vocab > kMaxVocab) return TREE_ATTN_ERR_TOO_LARGE;
    if (dlogits && (d_stride < vocab || (dlogits == logits && d_stride != row_stride))) return TREE_ATTN_ERR_INVALID_ARG;
    if (!(c->clip_low >= 0.f && c->clip_low <= 1.f) || !(c->clip_high >= 0.f) || !std::isfinite(c->kl_coef) ||
        !std::isfinite(c->entropy_coef) || !std::isfinite(c->grad_scale) || (c->per_token != 0 && c->per_token != 1))
        return TREE_ATTN_ERR_INVALID_ARG;
    if (!aligned(logits, 2) || !aligned(dlogits, 2) || !aligned(workspace, 256)) return TREE_ATTN_ERR_ALIGNMENT;
    for (const void* q : {(const void*)tokens, (const void*)c->old_logprobs, (const void*)c->advantages,
                          (const void*)c->weights, (const void*)c->ref_logprobs, (const void*)loss, (const void*)logprobs,
                          (const void*)entropy})
        if (!aligned(q, 4)) return TREE_ATTN_ERR_ALIGNMENT;
    if (!workspace || ws_bytes < 3 * column(P)) return TREE_ATTN_ERR_WORKSPACE;
    DevicePlan* D = nullptr;
    int64_t n_pred = 0;
    int st = ensure_policy(P, &D, &n_pred);
    if (st) return st;
    if (n_pred > 0 && (!c->advantages || (c->kl_coef != 0.f && !c->ref_logprobs))) return TREE_ATTN_ERR_INVALID_ARG;
    int dev, *status;
    if ((st = current_device(&dev)) || (st = get_status_ptr(dev, &status))) return st;
    Params p = {};
    p.logits = static_cast<const uint16_t*>(logits);
    p.stride = row_stride;
    p.vocab = vocab;
    p.tokens = tokens;
    p.old = c->old_logprobs;
    p.adv = c->advantages;
    p.weights = c->weights;
    p.ref = c->ref_logprobs;
    p.per_token = c->per_token;
    p.each = n_pred > 0 ? (float)(1.0 / (double)n_pred) : 0.f;
    p.top_ratio = 1.f + c->clip_high;
    p.low_ratio = 1.f - c->clip_low;
    log_pair(std::log1p((double)c->clip_high), p.top_log, p.top_log_lo);
    log_pair(std::log1p(-(double)c->clip_low), p.low_log, p.low_log_lo);
    p.kl = c->kl_coef;
    p.ent = c->entropy_coef;
    p.grad_scale = c->grad_scale;
    p.rows = reinterpret_cast<const int4*>(D->policy_rows);
    p.pred = reinterpret_cast<const int4*>(D->policy_pred);
    p.targets = reinterpret_cast<const int4*>(D->policy_targets);
    p.logprobs = logprobs;
    p.entropy = entropy;
    char* ws = static_cast<char*>(workspace);
    p.row_loss = reinterpret_cast<float*>(ws);
    p.tx = reinterpret_cast<float*>(ws + column(P));
    p.tg = reinterpret_cast<float*>(ws + 2 * column(P));
    p.dlogits = static_cast<uint16_t*>(dlogits);
    p.d_stride = d_stride;
    p.N = (int32_t)P->N;
    p.n_pred = n_pred;
    p.status = status;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const Shape f = shape_of(vocab, P->N);
    static std::once_flag once[kMaxDevices];
    static cudaError_t set[kMaxDevices];
    std::call_once(once[dev], [&] {
        set[dev] = launched(cudaFuncSetAttribute(policy_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSlots0 + kMaxSlice));
    });
    if (set[dev] != cudaSuccess) return TREE_ATTN_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(32 * (f.warps + 1));
    cfg.dynamicSmemBytes = f.smem;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim = {(unsigned)f.C, 1, 1};
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    cfg.gridDim = dim3((unsigned)f.C);
    const int at_a_time = clusters_at_a_time(dev, f, cfg);
    if (at_a_time < 1) return TREE_ATTN_ERR_CUDA;
    cfg.gridDim = dim3((unsigned)(std::min<int64_t>(P->N, at_a_time) * f.C));
    cudaError_t e = launched(cudaLaunchKernelEx(&cfg, policy_kernel, p, f.slots, f.slot_bytes));
    if (e != cudaSuccess) return TREE_ATTN_ERR_CUDA;
    e = launch_pdl(policy_sum_kernel, dim3(1), dim3(1024), 0, s, (const float*)p.row_loss, (int)P->N, loss);
    return e == cudaSuccess ? TREE_ATTN_OK : TREE_ATTN_ERR_CUDA;
}

}  // extern "C"
