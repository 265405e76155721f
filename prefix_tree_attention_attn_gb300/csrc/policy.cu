// Clipped policy loss of the trajectories and its gradient for the compact logits
// (include/tree_loss.h).
//
// One pass over the logits.  A cluster of C CTAs takes a row, a slice each, and goes from row to row;
// each logit is read once (2 bytes) and its gradient written once (2 bytes).  The rows go through a
// CTA as through a pipe, a few slices in a ring of shared memory at a time, with warps for each part:
//
//   producer     whether the next row has any weight, and the bulk copy of its slice.
//   statistics   one or two teams: S = sum 2^a, T = sum 2^a a with a = (x - m) log2 e, m near the maximum, by
//                thread, warp and CTA; a CTA's three numbers go to every CTA of the cluster by asynchronous
//                stores that count on a barrier there.  One element stays apart: the target, or the likeliest of
//                several (1 - p of a token that is nearly certain is the others' share of S, and no difference).
//   finishers    two warps, a row each in turn: join them, LSE = m + ln S, H = ln S - ln 2 T / S; the row's g_k, a lane
//                for each prediction where there are at most 32 of one target (inside a segment: one
//                for each trajectory through it), whose inputs it has loaded rows ahead; their sums.
//   gradient     2^a (cG + cE (a - T / S)), cG = -sum g / S, cE = entropy_coef ln 2 sum w / S,
//                rounded once.  The element that stayed apart is g (1 - p) - p (the other targets' sum of g) and its
//                entropy term from the others' sums; the finishers have it.  A row of several
//                targets gets the others' elements afterwards, with their g_k added before the rounding (children with
//                the same token id summed in their order).
//
// (With the same warps doing all parts of a row in turn, and five such CTAs on an SM, the chain from
// a row's load to its gradient set the pace: 1,022 us for 8,835 rows of 152,064 logits, 7,797 of them with
// weight, where this takes 783, 6.5 TB/s of reads and writes; without the gradient 435.)
//
// Whether a ratio lies beyond the clip decides a whole gradient, so lp - old is a pair of floats:
// ln S = k ln 2 + ln f, f near 1, adds no error beyond 3e-8.  What is left is S's own: a power of two is within 2^-22 and
// 2^-24 ln 2 of its exponent, together 3e-7 near the reference and 1.2e-6 for logits 16 above it.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <array>
#include <cmath>
#include <mutex>
#include <vector>

#include "align.h"
#include "kernels.h"
#include "plan.h"
#include "tree_loss.h"

namespace cg = cooperative_groups;

namespace treeattn {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kMaxSlots = 6;
constexpr int kFinishers = 2;
constexpr int kMaxStat = 8;                    // statistics warps
constexpr int kShared = 227 * 1024;            // of an SM, and of a CTA at most
constexpr int64_t kMaxVocab = 262144;
constexpr float kFar = -1e30f;                 // in place of -inf where it meets a factor 0
constexpr float kHuge = 0x1p100f;              // beyond this a multiple of a logit may overflow
constexpr float kNear = 0x1p24f;               // m log2 e is rounded by less than 1 up to here

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
    const int2* pred;                          // {prediction, trajectory} by row, then target
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

// Whether either number of a lies above b's.
__device__ __forceinline__ bool above2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("{\n\t.reg .pred p, q;\n\tsetp.gt.bf16x2 p|q, %1, %2;\n\tor.pred p, p, q;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r) : "r"(a), "r"(b));
    return r != 0;
}

// a + b = s + e exactly
__device__ __forceinline__ float two_sum(float a, float b, float& e) {
    const float s = a + b, bb = s - a;
    e = (a - (s - bb)) + (b - bb);
    return s;
}

// The exponent of x against the reference m; far below it counts as 1e30 below, so that 0 meets no infinity
// (+inf and NaN are told by m alone).
__device__ __forceinline__ float exponent(float x, float m) { return fmaxf(x - m, kFar) * kLog2e; }

// A reference m, one of the logits and at most 16 below the largest (32 between 4,096 and 8,192, where 16 more is no
// number of bf16), and the sums of e = 2^exponent and e * exponent over some logits.
struct Stat {
    float m, s, t;
};

// What the predictions of a row need of it.
struct Row {
    float m;                                   // the reference; NaN where the row has no distribution
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

// What the finisher tells the gradient's warps of a row.
struct Result {
    float m, ts, cg, ce;                       // maximum, T / S and the two factors
    float own;                                 // the element that stayed apart
    int active, y, t0, nt;                     // some weight; that element's token; targets
};

// The ring follows.
struct Shared {
    uint64_t full[kMaxSlots], empty[kMaxSlots], done[kMaxSlots];
    uint64_t stat[2 * kMaxSlots];              // the cluster's CTAs have sent their sums
    float4 stats[2 * kMaxSlots][8];            // {m, S, T of all but one element, that one's logit or -inf} by CTA
    Stat parts[kMaxSlots][kMaxStat];           // by statistics warp
    int parts_in[kMaxSlots];
    uint64_t read[kFinishers];                 // the cluster's finishers have read a row's targets
    uint64_t cta;                              // the gradient's warps have come this far
    struct __align__(16) {
        int active, y;                         // y: the token whose element stays apart
        int owner, at;                         // statistics thread of it in this CTA or -1; its byte in the slot, -1: in no whole vector
    } meta[kMaxSlots];
    float apart[kMaxSlots];                    // its logit, in the CTA that has it
    Result result[kMaxSlots];
};
constexpr int kRing0 = (sizeof(Shared) + 127) / 128 * 128;

__device__ __forceinline__ float advantage(const Params& p, int2 e) { return p.adv[p.per_token ? e.x : e.y]; }

// The predictions [first, first + n) of one target with logit x, by the threads `at`, `at` + step, ...
__device__ __forceinline__ void predict_all(const Params& p, const Row& row, int first, int n, float x, int at, int step,
                                            bool writes, Sums& sum) {
    for (int i = at; i < n; i += step) {
        const int2 e = p.pred[first + i];
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

// The same sums against the reference m (far below it they are 0, whatever their exponents add up to).
__device__ __forceinline__ Stat against(Stat a, float m) {
    const float d = exponent(a.m, m), e = fast_exp2(d);
    return {m, a.s * e, e > 0.f ? fmaf(a.s, d, a.t) * e : 0.f};
}

__device__ __forceinline__ float warp_max(float a) {
    float m;
    asm("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(a));
    return m;
}

// The sums of a warp's lanes against their common maximum.
__device__ __forceinline__ Stat warp_join(Stat a) {
    Stat r = against(a, warp_max(a.m));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        r.s += __shfl_xor_sync(0xffffffffu, r.s, o);
        r.t += __shfl_xor_sync(0xffffffffu, r.t, o);
    }
    return r;
}

// Puts a 16-bit word of shared memory in another's place (no other thread is near it).
__device__ __forceinline__ uint32_t swap_shared_u16(uint32_t addr, uint32_t with) {
    uint16_t was;
    asm volatile("ld.shared.u16 %0, [%1];\n\tst.shared.u16 [%1], %2;" : "=h"(was) : "r"(addr), "h"((uint16_t)with) : "memory");
    return was;
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
};

// The loads of one row's predictions, in three steps that depend on one another.
struct Ahead {
    int4 info;
    int2 mine;
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
    x.mine = make_int2(-1, 0);
    if (is_narrow(x.info) && lane < x.info.y) {
        x.mine = p.pred[x.info.x + lane];
        if (!ta_ok(p.status, 602, x.mine.x, 0, p.n_pred)) x.mine.x = -1;
    }
}
// `all`: what the predictions need, not the weights alone
__device__ __forceinline__ void load_values(const Params& p, int64_t r, bool all, Ahead& x) {
    x.w = x.old = x.a = x.ref = 0.f;
    x.y = -1;
    if (x.mine.x >= 0) {
        x.w = p.weights ? p.weights[x.mine.x] : p.each;
        if (all) {
            if (p.old) x.old = p.old[x.mine.x];
            x.a = advantage(p, x.mine);
            if (p.kl != 0.f) x.ref = p.ref[x.mine.x];
        }
    }
    // one target: it is the next packed row (a node's tokens and its only child follow each other)
    if (x.info.w == 1 && ta_ok(p.status, 603, r + 1, 0, p.N)) x.y = p.tokens[r + 1];
}
// Whether the row has any weight (the same in every warp that asks).
__device__ __forceinline__ bool has_weight(const Params& p, int lane, const Ahead& x) {
    if (is_narrow(x.info)) return __any_sync(0xffffffffu, x.w != 0.f);
    if (x.info.y == 0 || !p.weights) return x.info.y > 0;
    bool any = false;
    for (int i = lane; i < x.info.y && !any; i += 32) {
        const int k = p.pred[x.info.x + i].x;
        any = ta_ok(p.status, 602, k, 0, p.n_pred) && p.weights[k] != 0.f;
    }
    return __any_sync(0xffffffffu, any);
}

// The sum of g over the lanes in `alike`, in their order behind `from`; for the first of them.
__device__ __forceinline__ float sum_alike(uint32_t alike, int lane, float g, float from) {
    uint32_t left = __ffs(alike) - 1 == lane ? alike : 0u;
    while (__any_sync(0xffffffffu, left != 0)) {
        const float v = __shfl_sync(0xffffffffu, g, left ? __ffs(left) - 1 : lane);
        if (left) from += v;
        left &= left - 1;
    }
    return from;
}

// An element of the gradient without any g of its own, from its logit.
__device__ __forceinline__ float element(const Result& R, float x) {
    const float a = exponent(x, R.m);
    return fast_exp2(a) * fmaf(R.ce, a - R.ts, R.cg);
}

// The elements of a row's targets in this CTA but the one that stayed apart, where children with the same token are added
// up in their order.  One warp: up to 128 targets are compared with one another; of more the sums so far lie by token
// in the row's slot (`room`), which has space for half of its tokens at a time, and 32 targets are looked up at a time.
// (Not inlined: within the kernel it cost the gradient's loop 5 % by its registers alone.)  A root of 12,000 children of
// 600 logits: 1.5 ms for all rows; 32 ms when each child was compared with each.
struct Targets {
    const int4* targets;
    const int32_t* tokens;
    const float *tx, *tg;
    uint16_t* row_d;
    float* room;
    int room_bytes, lo, hi, shift, V, N;       // the slice's vectors
    Result R;
    float grad_scale;
    int* status;
};
__device__ __noinline__ void add_targets(const Targets& t) {
    const int lane = threadIdx.x & 31, nt = t.R.nt;
    constexpr int kAtOnce = 4;                 // loads under way
    int y[kAtOnce];                            // token of a target here, or -1
    float g[kAtOnce], x[kAtOnce];
    auto load = [&](int j0) {
        int q[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const int j = j0 + 32 * i + lane;
            q[i] = j < nt ? t.targets[j].x : -1;
            if (q[i] >= 0 && !ta_ok(t.status, 604, q[i], 0, t.N)) q[i] = -1;
        }
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) y[i] = q[i] >= 0 ? t.tokens[q[i]] : -1;
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const int v = (y[i] + t.shift) / 8;
            if (y[i] < 0 || y[i] >= t.V || v < t.lo || v >= t.hi || y[i] == t.R.y) y[i] = -1;
            g[i] = y[i] >= 0 ? t.tg[q[i]] : 0.f;
            x[i] = y[i] >= 0 ? t.tx[q[i]] : 0.f;
        }
    };
    auto write = [&](int yi, float xi, float sum) {
        t.row_d[yi] = (uint16_t)pack_bf16x2(element(t.R, xi) + t.grad_scale * sum, 0.f);
    };
    load(0);
    if (nt <= 32 * kAtOnce) {
        float sum[kAtOnce] = {};
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i)
            for (int k = 0; k < min(32, nt - 32 * i); ++k) {
                const int yk = __shfl_sync(0xffffffffu, y[i], k);
                const float gk = __shfl_sync(0xffffffffu, g[i], k);
#pragma unroll
                for (int e = 0; e < kAtOnce; ++e)
                    if (y[e] == yk) sum[e] += gk;
            }
#pragma unroll
        for (int e = 0; e < kAtOnce; ++e)
            if (y[e] >= 0) write(y[e], x[e], sum[e]);     // (the same number from each child with the token)
        return;
    }
    int loaded = 0;
    const int window = t.room_bytes / 32;      // vectors of 8 tokens
    for (int v = t.lo; v < t.hi; v += window) {
        const int base = 8 * v - t.shift, end = 8 * min(v + window, t.hi) - t.shift;
        auto all = [&](auto step) {
            for (int j0 = 0; j0 < nt; j0 += 32 * kAtOnce) {
                if (j0 != loaded) load(loaded = j0);
#pragma unroll
                for (int i = 0; i < kAtOnce; ++i) step(y[i] >= max(base, 0) && y[i] < end, y[i], g[i], x[i]);
            }
            __syncwarp();
        };
        all([&](bool here, int yi, float, float) {
            if (here) t.room[yi - base] = 0.f;
        });
        all([&](bool here, int yi, float gi, float) {
            const uint32_t alike = __match_any_sync(0xffffffffu, here ? yi : -1 - lane);
            const float sum = sum_alike(alike, lane, gi, here ? t.room[yi - base] : 0.f);
            __syncwarp();
            if (here && __ffs(alike) - 1 == lane) t.room[yi - base] = sum;
            __syncwarp();
        });
        all([&](bool here, int yi, float, float xi) {
            if (here) write(yi, xi, t.room[yi - base]);
        });
    }
}

// How the warps of a CTA are shared out: `teams` of `stat` for the statistics, a row each in turn, `grad` for the
// gradient, then the finishers and the producer.
struct Split {
    int teams, stat, grad, slots, slot_bytes;
};

// (80 registers: 23 warps on an SM)
__global__ void __maxnreg__(80) policy_kernel(const Params p, const Split f) {
    extern __shared__ __align__(128) uint8_t smem[];
    Shared& S = *reinterpret_cast<Shared*>(smem);
    cg::cluster_group cluster = cg::this_cluster();
    const int C = (int)cluster.num_blocks(), me = (int)cluster.block_rank(), log_c = __ffs(C) - 1;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n_slots = f.slots, n_places = 2 * f.slots, grad0 = f.teams * f.stat;
    const int64_t cluster0 = blockIdx.x / C, clusters = gridDim.x / C;
    uint8_t* ring = smem + kRing0;
    if (tid == 0) {
        for (int i = 0; i < n_slots; ++i) {
            mbar_init(smem_u32(&S.full[i]), 1);
            mbar_init(smem_u32(&S.empty[i]), f.stat + f.grad + 1);
            mbar_init(smem_u32(&S.done[i]), 1);
            S.parts_in[i] = 0;
        }
        for (int i = 0; i < n_places; ++i) mbar_init(smem_u32(&S.stat[i]), 1);
        for (int i = 0; i < kFinishers; ++i) mbar_init(smem_u32(&S.read[i]), C);
        mbar_init(smem_u32(&S.cta), max(f.grad, 1));
        fence_mbar_init();
        for (int i = 0; i < n_places; ++i) mbar_expect_tx(smem_u32(&S.stat[i]), 16 * C);   // of the first rows
    }
    cluster.sync();                            // every CTA of the cluster runs, its barriers are set up
    grid_dep_wait();
    grid_dep_launch();
    bool ok = true;

    // Sums wait in 2 * slots places.  A CTA sends those of a row when its slot is free, so it is done with the row `slots`
    // before; for that one every CTA had sent its sums, each when it was done with the row `slots` before that: the
    // row whose place is taken has been joined everywhere.
    //
    // Two teams that meet in a slot: a barrier tells a phase from the next one alone.  When a team comes to row j, its
    // row before that, and so every row up to j - slots, is loaded or on its way: the slot was empty for row
    // j - slots; it waits until it is empty of that one, then for row j.
    if (warp < f.teams * f.stat) {
        // ---- statistics --------------------------------------------------------------------
        const int T = 32 * f.stat, team = warp / f.stat, mine = warp - team * f.stat, at = 32 * mine + lane;
        const uint64_t c2 = f32x2(kLog2e, kLog2e);
        int slot = team % n_slots, turn = team / n_slots, place = team;
        for (int64_t r = cluster0 + team * clusters; r < p.N; r += f.teams * clusters) {
            if (f.teams > 1 && turn > 0) ok = mbar_wait(smem_u32(&S.empty[slot]), (turn - 1) & 1, p.status, 610);
            if (ok) ok = mbar_wait(smem_u32(&S.full[slot]), turn & 1, p.status, 604);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            Stat st = {0.f, 0.f, 0.f};
            const int4 meta = *reinterpret_cast<const int4*>(&S.meta[slot]);
            if (meta.x) {                      // (the same in every CTA of the cluster)
                const Slice s(p, r, me, log_c);
                const int odd = s.odd(at, T);
                const uint8_t* here8 = ring + (size_t)slot * f.slot_bytes;
                const uint4* here = reinterpret_cast<const uint4*>(here8) - s.lo;
                const uint4 none = make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u);   // -inf
                uint4 rest = odd >= 0 ? s.part(odd) : none;
                // The thread that comes by the element that stays apart takes it out of its vector: -inf, probability 0
                // (a whole vector in the ring; the gradient has no use for this element either)
                if (meta.z == at && meta.w >= 0) {
                    S.apart[slot] = lo16(swap_shared_u16(smem_u32(here8) + meta.w, 0xff80u));
                } else if (meta.z == at) {
                    uint32_t u[4] = {rest.x, rest.y, rest.z, rest.w};
                    const int e = meta.y - s.start(odd);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (i == e / 2) {
                            S.apart[slot] = e & 1 ? hi16(u[i]) : lo16(u[i]);
                            u[i] = e & 1 ? (u[i] & 0xffffu) | 0xff800000u : (u[i] & 0xffff0000u) | 0xff80u;
                        }
                    rest = make_uint4(u[0], u[1], u[2], u[3]);
                }
                const bool odds = __any_sync(0xffffffffu, odd >= 0);
                auto get = [&](int v) { return v < s.last ? here[v] : none; };
                auto top2 = [&](uint4 x) { return max2_nan(max2_nan(x.x, x.y), max2_nan(x.z, x.w)); };
                const int v0 = s.first + at;
                // One pass: the reference is the maximum of the warp's first vectors, and is raised when a logit lies 16
                // above it (e^16 is far from overflow), which after the first few vectors it hardly ever does.
                uint4 x = get(v0), y = get(v0 + T);
                uint32_t seen = max2_nan(top2(x), top2(y));   // the lane's maximum: an infinity or NaN shows in the end
                float ref;
                asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(ref) : "f"(fmaxf(lo16(seen), hi16(seen))));
                if (fabsf(ref) < kHuge) {
                    uint64_t minus = f32x2(-ref, -ref), sum_s = 0, sum_t = 0, more_s = 0, more_t = 0;
                    uint32_t far2, limit2;
                    auto set = [&] {
                        minus = f32x2(-ref, -ref);
                        // what lies far enough below is 0 all the same, and then finite
                        const float far = ref - fmaxf(256.f, fabsf(ref) * 0x1p-6f), limit = ref + 16.f;   // (rounded below)
                        far2 = pack_bf16x2(far, far);
                        limit2 = pack_bf16x2(limit, limit);
                    };
                    set();
                    auto add = [&](uint32_t u, uint64_t& ss, uint64_t& tt) {
                        u = max2(u, far2);
                        const uint64_t a = mul_f32x2(add_f32x2(f32x2(lo16(u), hi16(u)), minus), c2);
                        float a0, a1;
                        f32x2_split(a, a0, a1);
                        const uint64_t e = f32x2(fast_exp2(a0), fast_exp2(a1));
                        ss = add_f32x2(ss, e);
                        tt = fma_f32x2(e, a, tt);
                    };
                    auto add4 = [&](uint4 z) {
                        add(z.x, sum_s, sum_t);
                        add(z.y, more_s, more_t);
                        add(z.z, sum_s, sum_t);
                        add(z.w, more_s, more_t);
                    };
                    auto look = [&](uint32_t top) {
                        seen = max2_nan(seen, top);
                        if (__any_sync(0xffffffffu, above2(top, limit2))) {
                            const float was = ref;
                            asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(ref) : "f"(fmaxf(lo16(top), hi16(top))));
                            set();
                            const float d = exponent(was, ref), e = fast_exp2(d);
                            const uint64_t d2 = f32x2(d, d), e2 = f32x2(e, e);
                            sum_t = mul_f32x2(fma_f32x2(sum_s, d2, sum_t), e2);
                            more_t = mul_f32x2(fma_f32x2(more_s, d2, more_t), e2);
                            sum_s = mul_f32x2(sum_s, e2);
                            more_s = mul_f32x2(more_s, e2);
                        }
                    };
                    for (int v = v0, w = s.first + 32 * mine;;) {   // w: the warp's first, for all its lanes alike
                        add4(x);
                        add4(y);
                        v += 2 * T;
                        w += 2 * T;
                        if (w >= s.last) break;
                        if (w + T + 32 <= s.last) {     // all of the warp's
                            x = here[v];
                            y = here[v + T];
                        } else {
                            x = get(v);
                            y = get(v + T);
                        }
                        look(max2_nan(top2(x), top2(y)));
                    }
                    if (odds) {
                        look(top2(rest));
                        add4(rest);
                    }
                    float a0, a1;
                    f32x2_split(add_f32x2(sum_s, more_s), a0, a1);
                    st.s = a0 + a1;
                    f32x2_split(add_f32x2(sum_t, more_t), a0, a1);
                    st.t = a0 + a1;
                    const float top = max_nan(lo16(seen), hi16(seen));
                    st.m = top < INFINITY ? ref : top;
                } else {
                    // masks to begin with, or huge logits: the maximum first (an infinity and NaN: told by it alone)
                    for (int v = v0; v < s.last; v += T) seen = max2_nan(seen, top2(here[v]));
                    seen = max2_nan(seen, top2(rest));
                    st.m = max_nan(lo16(seen), hi16(seen));
                    if (fabsf(st.m) < INFINITY)
                        for (int v = v0; v < s.last + T; v += T) {
                            const uint4 z = v < s.last ? here[v] : rest;
                            const uint32_t u[4] = {z.x, z.y, z.z, z.w};
#pragma unroll 1
                            for (int i = 0; i < 8; ++i) {
                                const float a = exponent(__uint_as_float((u[i / 2] >> (16 * (i & 1))) << 16), st.m), e = fast_exp2(a);
                                st.s += e;
                                st.t = fmaf(e, a, st.t);
                            }
                        }
                }
                st = warp_join(st);
            }
            // the last of the CTA's warps joins them and sends
            int last = 0;
            __syncwarp();
            if (lane == 0) {
                S.parts[slot][mine] = st;
                __threadfence_block();
                last = atomicAdd(&S.parts_in[slot], 1) == f.stat - 1;
            }
            if (__shfl_sync(0xffffffffu, last, 0)) {
                __threadfence_block();
                const Stat none = {-INFINITY, 0.f, 0.f};
                st = warp_join(lane < f.stat ? S.parts[slot][lane] : none);
                const float xy = meta.x && meta.z >= 0 ? S.apart[slot] : -INFINITY;
                if (lane < C)
                    remote_store(at_rank(smem_u32(&S.stats[place][me]), lane), make_float4(st.m, st.s, st.t, xy),
                                 at_rank(smem_u32(&S.stat[place]), lane));
                if (lane == 0) S.parts_in[slot] = 0;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&S.empty[slot]));
            place += f.teams;
            if (place >= n_places) place -= n_places;
            slot += f.teams;
            while (slot >= n_slots) {
                slot -= n_slots;
                ++turn;
            }
        }
    } else if (warp < grad0 + f.grad) {
        // ---- the gradient --------------------------------------------------------------------
        const int at = tid - 32 * grad0, T = 32 * f.grad;
        const uint64_t c2 = f32x2(kLog2e, kLog2e);
        int slot = 0, turn = 0, meets = 0;
        for (int64_t r = cluster0; r < p.N; r += clusters) {
            ok = mbar_wait(smem_u32(&S.done[slot]), turn & 1, p.status, 608);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            const Result R = S.result[slot];
            const Slice s(p, r, me, log_c);
            uint16_t* row_d = p.dlogits + r * p.d_stride;
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
            if (!R.active) {
                for (int v = s.lo + at; v < s.hi; v += T) store(v, make_uint4(0, 0, 0, 0));
            } else {
                const int odd = s.odd(at, T), yv = s.owns(R.y);
                const uint4* here = reinterpret_cast<const uint4*>(ring + (size_t)slot * f.slot_bytes) - s.lo;
                int v = s.first + at;
                uint4* row_d8 = reinterpret_cast<uint4*>(row_d - s.shift);   // (whole vectors lie as the row's do)
                if (fabsf(R.m) <= kNear) {
                    // One multiply-add for the exponent, x log2 e - mc with mc = m log2 e rounded.  Every exponent of the
                    // row is then short of the same number, mc - m log2 e (exact: m has 8 bits), which goes into the factors.
                    // (20 warps hide the latencies of a loop of one vector: 779 us where two a turn took 795)
                    const float mc = R.m * kLog2e, off = fmaf(-R.m, kLog2e, mc), more = fast_exp2(off), cg = R.cg * more;
                    const uint64_t minus = f32x2(-mc, -mc), cg2 = f32x2(cg, cg);
                    if (R.ce == 0.f) {
#pragma unroll 1
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
                            const uint4 o4 = make_uint4(o[0], o[1], o[2], o[3]);
                            if (together) __stcs(row_d8 + v, o4);
                            else store(v, o4);
                        }
                    } else {
                        // the entropy's term; -inf, where 0 would meet an infinity, as what is 0 all the same
                        const float far = R.m - fmaxf(256.f, fabsf(R.m) * 0x1p-6f);
                        const uint32_t far2 = pack_bf16x2(far, far);
                        const float ce = R.ce * more, rest = fmaf(ce, off - R.ts, cg);
                        const uint64_t ce2 = f32x2(ce, ce), rest2 = f32x2(rest, rest);
#pragma unroll 1
                        for (; v < s.last; v += T) {
                            const uint4 x = here[v];
                            const uint32_t u[4] = {max2(x.x, far2), max2(x.y, far2), max2(x.z, far2), max2(x.w, far2)};
                            uint32_t o[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                float a0, a1;
                                const uint64_t a = fma_f32x2(f32x2(lo16(u[i]), hi16(u[i])), c2, minus);
                                f32x2_split(a, a0, a1);
                                f32x2_split(mul_f32x2(f32x2(fast_exp2(a0), fast_exp2(a1)), fma_f32x2(ce2, a, rest2)), a0, a1);
                                o[i] = pack_bf16x2(a0, a1);
                            }
                            const uint4 o4 = make_uint4(o[0], o[1], o[2], o[3]);
                            if (together) __stcs(row_d8 + v, o4);
                            else store(v, o4);
                        }
                    }
                }
                // the general form, and the vectors in part
#pragma unroll 1
                for (; v < s.last || (odd >= 0 && v < s.last + T); v += T) {
                    const uint4 x = v < s.last ? here[v] : s.part(odd);
                    const uint32_t u[4] = {x.x, x.y, x.z, x.w};
                    uint32_t o[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[i] = pack_bf16x2(element(R, lo16(u[i])), element(R, hi16(u[i])));
                    store(v < s.last ? v : odd, make_uint4(o[0], o[1], o[2], o[3]));
                }
                // the element that stayed apart, over what the same thread has written there
                if (yv >= 0 && (yv == odd || (yv >= s.first && yv < s.last && (yv - s.first) % T == at)))
                    row_d[R.y] = (uint16_t)pack_bf16x2(R.own, 0.f);
                if (R.nt != 1) {
                    // every warp has written, and read the slot: one of them does the other targets' elements again
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&S.cta));
                    if (at < 32) {
                        ok = mbar_wait(smem_u32(&S.cta), meets++ & 1, p.status, 603);
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok) break;
                        add_targets({p.targets + R.t0, p.tokens, p.tx, p.tg, row_d, reinterpret_cast<float*>(ring + (size_t)slot * f.slot_bytes),
                                     f.slot_bytes, s.lo, s.hi, s.shift, s.V, p.N, R, p.grad_scale, p.status});
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&S.empty[slot]));
            if (++slot == n_slots) {
                slot = 0;
                ++turn;
            }
        }
    } else if (warp < grad0 + f.grad + kFinishers) {
        // ---- the finishers ------------------------------------------------------------------
        const int mine = warp - grad0 - f.grad;
        const int64_t step = kFinishers * clusters, r0 = cluster0 + mine * clusters;
        Ahead one, two, three;                 // this row and its next two
        load_info(p, r0, one);
        load_info(p, r0 + step, two);
        load_info(p, r0 + 2 * step, three);
        load_pred(p, lane, one);
        load_pred(p, lane, two);
        load_values(p, r0, true, one);
        int reads = 0;
        int64_t it = mine;
        for (int64_t r = r0; r < p.N; r += step, it += kFinishers) {
            const int slot = (int)(it % n_slots), place = (int)(it % n_places);
            const int64_t turn = it / n_slots;
            Ahead four;
            load_info(p, r + 3 * step, four);
            load_pred(p, lane, three);
            load_values(p, r + step, true, two);
            const int4 info = one.info;
            const bool active = has_weight(p, lane, one), narrow = is_narrow(info), single = info.w == 1;
            if (turn > 0) ok = mbar_wait(smem_u32(&S.empty[slot]), (turn - 1) & 1, p.status, 609);
            if (ok) ok = wait_cluster(smem_u32(&S.stat[place]), (it / n_places) & 1, p.status, 605);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            Stat others = {-INFINITY, 0.f, 0.f};
            float xy = -INFINITY;
            if (lane < C) {
                const float4 q = S.stats[place][lane];
                others = {q.x, q.y, q.z};
                xy = q.w;
            }
            // both against their common maximum; the sums lie in lanes 0 to 7
            others = against(others, warp_max(max_nan(others.m, xy)));
            xy = warp_max(xy);
#pragma unroll
            for (int o = 4; o > 0; o >>= 1) {
                others.s += __shfl_xor_sync(0xffffffffu, others.s, o);
                others.t += __shfl_xor_sync(0xffffffffu, others.t, o);
            }
            others.s = __shfl_sync(0xffffffffu, others.s, 0);
            others.t = __shfl_sync(0xffffffffu, others.t, 0);
            int chosen = one.y;
            if (active && !single) {           // the producer's choice (its copy has come, or there would be no sums)
                ok = mbar_wait(smem_u32(&S.full[slot]), turn & 1, p.status, 607);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                chosen = S.meta[slot].y;
            }
            __syncwarp();
            if (lane == 0) {
                mbar_expect_tx(smem_u32(&S.stat[place]), 16 * C);   // of the place's next row
                mbar_arrive(smem_u32(&S.empty[slot]));             // nothing more of this row from the slot or the place
            }
            Result R = {0.f, 0.f, 0.f, 0.f, 0.f, active, chosen, info.z, info.w};
            if (!active) {
                if (me == 0) {
                    if (p.logprobs)
                        for (int i = lane; i < info.y; i += 32) {
                            const int j = p.pred[info.x + i].x;
                            if (ta_ok(p.status, 602, j, 0, p.n_pred)) p.logprobs[j] = 0.f;
                        }
                    if (lane == 0) {
                        p.row_loss[r] = 0.f;
                        if (p.entropy) p.entropy[r] = 0.f;
                    }
                }
            } else {
                const int V = (int)p.vocab;
                const bool apart = R.y >= 0 && R.y < V;
                if (!apart) xy = __int_as_float(0x7fc00000);
                const float ay = exponent(xy, others.m), ey = apart ? fast_exp2(ay) : 0.f;
                const Stat st = {others.m, others.s + ey, ey > 0.f ? fmaf(ey, ay, others.t) : others.t};
                // (1 / S of a row without a distribution is not used)
                const float each = 1.f / st.s, ts = st.t * each, share = others.s * each, py = ey * each;
                Row row;
                row.m = fabsf(st.m) < INFINITY ? st.m : __int_as_float(0x7fc00000);
                {
                    // S = 2^k f, 0.7 <= f < 1.4 (S >= 1);  ln 2 = 45426 / 2^16 + 1.42860682e-6;
                    // ln f = 2 (z + z^3 / 3 + ...), z = (f - 1) / (f + 1), |z| < 0.18: the next term is below 2^-30 z
                    const uint32_t bits = __float_as_uint(st.s);
                    int e = (int)(bits >> 23) - 127;
                    float x = __uint_as_float((bits & 0x7fffffu) | 0x3f800000u);
                    if (x >= 1.4f) {
                        x *= 0.5f;
                        ++e;
                    }
                    const float z = (x - 1.f) / (x + 1.f), z2 = z * z;
                    const float poly = z2 * (1.f / 3 + z2 * (1.f / 5 + z2 * (1.f / 7 + z2 * (1.f / 9 + z2 * (1.f / 11)))));
                    row.lk = (float)e * (45426.f / 65536.f);
                    row.ll = fmaf((float)e, 1.42860682e-6f, 2.f * fmaf(z, poly, z));
                }
                row.h = row.m == row.m ? fmaf(-kLn2, ts, row.lk + row.ll) : row.m;
                Sums sum = {0.f, 0.f, 0.f};
                float beside = 0.f;            // g of other targets than the one whose element stayed apart
                if (narrow) {
                    float lp = 0.f;
                    if (one.w != 0.f) lp = predict(p, row, one.w, xy, one.old, p.old != nullptr, one.a, one.ref, sum);
                    if (me == 0 && one.mine.x >= 0 && p.logprobs) p.logprobs[one.mine.x] = lp;
                } else if (single) {
                    predict_all(p, row, info.x, info.y, xy, lane, 32, me == 0, sum);
                } else {
                    // several targets: a lane for each where there are many, the whole warp one after another else
                    const Slice s(p, r, me, log_c);
                    const bool lanes = info.w >= 8;
                    for (int j = lanes ? lane : 0; j < info.w; j += lanes ? 32 : 1) {
                        const int4 t = p.targets[info.z + j];
                        if (!ta_ok(p.status, 604, t.x, 0, p.N)) continue;
                        const int yj = p.tokens[t.x];
                        const float xj = yj >= 0 && yj < V ? lo16(s.x[yj]) : __int_as_float(0x7fc00000);
                        Sums part = {0.f, 0.f, 0.f};
                        predict_all(p, row, t.y, t.z, xj, lanes ? 0 : lane, lanes ? 1 : 32, me == 0, part);
                        if (!lanes) part = warp_sum(part);
                        if (lanes || lane == 0) {
                            if (yj == R.y) sum.g += part.g;
                            else beside += part.g;
                            sum.w += part.w;
                            sum.loss += part.loss;
                        }
                        if (p.dlogits && (lanes || lane == 0) && s.owns(yj) >= 0) {
                            p.tx[t.x] = xj;
                            p.tg[t.x] = part.g;
                        }
                    }
                    __syncwarp();
                    if (p.dlogits) {
                        // the gradient may lie over the logits: the whole cluster has read the targets' logits
                        if (lane < C) remote_arrive(at_rank(smem_u32(&S.read[mine]), lane));
                        ok = wait_cluster(smem_u32(&S.read[mine]), reads++ & 1, p.status, 606);
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok) break;
                    }
                }
                sum = warp_sum(sum);
                if (!single)
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) beside += __shfl_xor_sync(0xffffffffu, beside, o);
                if (me == 0 && lane == 0) {
                    p.row_loss[r] = sum.loss;
                    if (p.entropy) p.entropy[r] = row.h;
                }
                R.m = row.m;
                R.ts = ts;
                R.cg = row.m == row.m ? -p.grad_scale * (sum.g + beside) * each : row.m;
                R.ce = p.ent != 0.f ? kLn2 * p.grad_scale * p.ent * sum.w * each : 0.f;
                // g (1 - p) - p beside + cE 2^a (a - T / S), without the differences of near numbers in it
                R.own = p.grad_scale * (sum.g * share - beside * py);
                if (ey > 0.f) R.own = fmaf(R.ce * py, fmaf(ay, others.s, -others.t), R.own);
            }
            if (lane == 0 && f.grad) {
                S.result[slot] = R;
                mbar_arrive(smem_u32(&S.done[slot]));
            }
            one = two;
            two = three;
            three = four;
        }
    } else {
        // ---- the producer -------------------------------------------------------------------
        Ahead one, two, three;
        load_info(p, cluster0, one);
        load_info(p, cluster0 + clusters, two);
        load_info(p, cluster0 + 2 * clusters, three);
        load_pred(p, lane, one);
        load_pred(p, lane, two);
        load_values(p, cluster0, false, one);
        // Several targets: a lane's target row, and its token, the same rows ahead.
        auto target = [&](const Ahead& x) {
            const int q = x.info.w > 1 && lane < x.info.w ? p.targets[x.info.z + lane].x : -1;
            return q >= 0 && ta_ok(p.status, 604, q, 0, p.N) ? q : -1;
        };
        auto token = [&](int q) { return q >= 0 ? p.tokens[q] : -1; };
        int y1 = token(target(one)), q2 = target(two);
        int slot = 0, turn = 0, sent = 0;
        for (int64_t r = cluster0; r < p.N; r += clusters) {
            Ahead four;
            load_info(p, r + 3 * clusters, four);
            load_pred(p, lane, three);
            const int q3 = target(three);
            load_values(p, r + clusters, false, two);
            const int y2 = token(q2);
            const bool active = has_weight(p, lane, one);
            int apart = one.y;
            if (active && one.info.w > 1) {
                // the likeliest, of equals the lowest token: the only one whose p may be above 1/2
                const uint16_t* x = p.logits + r * p.stride;
                float best = -INFINITY;
                for (int j = lane, y = y1; j < one.info.w; j += 32) {
                    if (j >= 32) {
                        const int q = p.targets[one.info.z + j].x;
                        y = ta_ok(p.status, 604, q, 0, p.N) ? p.tokens[q] : -1;
                    }
                    if (y < 0 || y >= p.vocab) continue;
                    const float xj = lo16(x[y]);
                    if (apart < 0 || xj > best || (xj == best && y < apart)) {
                        best = xj;
                        apart = y;
                    }
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
                    const float xj = __shfl_xor_sync(0xffffffffu, best, o);
                    const int y = __shfl_xor_sync(0xffffffffu, apart, o);
                    if (y >= 0 && (apart < 0 || xj > best || (xj == best && y < apart))) {
                        best = xj;
                        apart = y;
                    }
                }
            }
            if (turn > 0) ok = mbar_wait(smem_u32(&S.empty[slot]), (turn - 1) & 1, p.status, 601);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            if (lane == 0) {
                const uint32_t bar = smem_u32(&S.full[slot]);
                const Slice s(p, r, me, log_c);
                const int av = s.owns(apart), T = 32 * f.stat;   // (a power of two)
                const bool whole = av >= s.first && av < s.last;
                S.meta[slot].active = active;
                S.meta[slot].y = apart;
                S.meta[slot].owner = av < 0 ? -1 : whole ? (av - s.first) & (T - 1) : av == s.lo && s.lo < s.first ? T - 1 : T - 2;
                S.meta[slot].at = whole ? 16 * (av - s.lo) + 2 * (apart - s.start(av)) : -1;
                const uint32_t bytes = (uint32_t)(s.last - s.first) * 16;
                if (active && bytes) {
                    fence_proxy_async_smem();  // threads may have written to the slot: an element taken out, sums by token
                    mbar_expect_tx(bar, bytes);
                    bulk_load(smem_u32(ring + (size_t)slot * f.slot_bytes + (size_t)(s.first - s.lo) * 16), s.x + s.start(s.first),
                              bytes, bar);
                } else {
                    mbar_arrive(bar);
                }
            }
            ++sent;
            if (++slot == n_slots) {
                slot = 0;
                ++turn;
            }
            one = two;
            two = three;
            three = four;
            y1 = y2;
            q2 = q3;
        }
        // copies still under way where a wait gave up
        if (!ok)
            for (int i = max(0, sent - n_slots); i < sent; ++i)
                mbar_wait(smem_u32(&S.full[i % n_slots]), (i / n_slots) & 1, p.status, 602);
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
    if (np > INT32_MAX) return TREE_ATTN_ERR_TOO_LARGE;
    *n_pred = np;
    DevicePlan& D = P->dev[dev];
    if (!D.policy_ready) {
        std::vector<int32_t> h;
        int64_t at_pred, at_target;
        try {
            // a target's predictions are the trajectories through it, its row the one before it
            const int64_t N = P->N;
            std::vector<int32_t> row_of(N, -1);
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
            const int64_t rows_words = 4 * N, pred_words = 2 * std::max<int64_t>(np, 1);
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
                    int32_t* e = pred + 2 * pred_at[s]++;
                    e[0] = (int32_t)k;
                    e[1] = (int32_t)l;
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

size_t column(const tree_attn_plan_s* P) { return ((size_t)P->N * 4 + 255) / 256 * 256; }

// How a row is cut up: CTAs, and their warps and slots.
struct Shape {
    int C, smem;
    Split split;
};
// A slice is at most a third of what an SM has, so that one can be loaded, one be summed and one get its gradient at
// a time; large slices have an SM to themselves, smaller ones share it, with fewer warps each.  A row's sums run over
// as many threads with and without the gradient, so a policy's log-probs of an evaluation are those of its update to
// the bit; without it two teams take a row each in turn.  Measured (us; CTAs a row / teams / statistics warps each /
// gradient warps / CTAs an SM): with the gradient 152,064 x 4,000 rows 391 (4/1/8/12/1) 423 (4/2/4/12/1) 499 (8/1/4/4/2);
// 64,000 x 5,000 216 (2/1/8/12/1) 230 (2/2/4/12/1); 32,000 x 10,000 220 (1/1/8/12/1) 226 (2/1/4/4/2); 16,000 x 20,000 241
// (1/1/4/4/2) 259 (1/2/2/4/2); 8,000 x 20,000 148 (1/2/1/3/3) 157 (1/1/2/3/3); 4,000 x 20,000 96 (1/2/1/3/3) 98
// (1/1/1/1/3); 1,000 x 20,000 71 (1/2/1/3/3) 79 (1/1/1/1/3).  Without it 152,064 x 4,000 220 (4/2/8/1) 289 (4/1/8/1)
// 260 (4/1/16/1); 64,000 x 5,000 119 (2/2/8/1) 152 (2/1/8/1); 32,000 x 10,000 119 (1/2/8/1) 152 (1/1/8/1); 16,000 x 20,000
// 128 (1/2/4/2) 140 (1/1/4/3); 8,000 x 20,000 98 (1/2/1/3) 87 (1/2/2/3); 4,000 x 20,000 60 (1/2/1/3) 78 (1/1/1/3).
Shape shape_of(int64_t vocab, bool grad) {
    const int64_t vectors = (vocab + 7) / 8 + 1;    // (a row may start inside a vector)
    Shape f = {1, 0, {2, 1, 3, 1, 0}};
    while (f.C < 8 && (vectors + f.C - 1) / f.C * 16 > (kShared - kRing0) / 3) f.C *= 2;
    Split& s = f.split;
    s.slot_bytes = (int)((vectors + f.C - 1) / f.C * 16);
    int per_sm = 3;
    if (s.slot_bytes > 40 * 1024) {
        s.stat = kMaxStat;
        s.grad = 12;
        per_sm = 1;
    } else if (s.slot_bytes > 20 * 1024) {
        s.stat = s.grad = 4;
        per_sm = 2;
    }
    if (grad && s.stat > 1) s.teams = 1;
    if (!grad) s.grad = 0;
    while (s.slots < kMaxSlots && kRing0 + (s.slots + 1) * s.slot_bytes <= (kShared + 1024) / per_sm - 1024) ++s.slots;
    f.smem = kRing0 + s.slots * s.slot_bytes;
    return f;
}

// Clusters of a launch that run at a time (of 4 and 8 CTAs fewer than the SMs would hold: they keep
// to groups of SMs); 0 where it cannot be told.  Asked once per shape and device.
int clusters_at_a_time(int dev, const Shape& f, const cudaLaunchConfig_t& cfg) {
    static std::mutex mu;
    static std::vector<std::array<int, 5>> known;
    std::lock_guard<std::mutex> lk(mu);
    for (const auto& k : known)
        if (k[0] == dev && k[1] == f.C && k[2] == (int)cfg.blockDim.x && k[3] == f.smem) return k[4];
    int n = 0;
    if (launched(cudaOccupancyMaxActiveClusters(&n, policy_kernel, &cfg)) != cudaSuccess) return 0;
    try {
        known.push_back({dev, f.C, (int)cfg.blockDim.x, f.smem, n});
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
    p.pred = reinterpret_cast<const int2*>(D->policy_pred);
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
    const Shape f = shape_of(vocab, dlogits != nullptr);
    static std::once_flag once[kMaxDevices];
    static cudaError_t set[kMaxDevices];
    std::call_once(once[dev], [&] {
        set[dev] = launched(cudaFuncSetAttribute(policy_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kShared));
    });
    if (set[dev] != cudaSuccess) return TREE_ATTN_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(32 * (f.split.teams * f.split.stat + f.split.grad + kFinishers + 1));
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
    cudaError_t e = launched(cudaLaunchKernelEx(&cfg, policy_kernel, p, f.split));
    if (e != cudaSuccess) return TREE_ATTN_ERR_CUDA;
    e = launch_pdl(policy_sum_kernel, dim3(1), dim3(1024), 0, s, (const float*)p.row_loss, (int)P->N, loss);
    return e == cudaSuccess ? TREE_ATTN_OK : TREE_ATTN_ERR_CUDA;
}

}  // extern "C"
