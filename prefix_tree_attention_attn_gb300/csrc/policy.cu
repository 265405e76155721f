// Clipped policy loss of the trajectories and its gradient for the compact logits
// (include/tree_loss.h).
//
// One pass over the logits.  A row stays in the registers of the CTAs of a cluster (a slice of
// the row each, NV 16-byte vectors a thread) between its statistics and its gradient, so 2 bytes
// per logit are read and 2 written:
//
//   statistics   m = max x, S = sum e^(x - m), T = sum e^(x - m) (x - m) by thread, then warp; a
//                warp's triple goes to every CTA of the cluster, and after one cluster barrier each
//                warp joins them all.  LSE = m + ln S, H = ln S - T / S.
//   predictions  every warp of every CTA works out the row's g_k for itself where the row has at
//                most 32 predictions of one target (inside a segment: one for each
//                trajectory through it), so nothing is waited for; others by the CTA.
//   gradient     e (cG + cE (x - m - T / S)) with e = e^(x - m), cG = -sum g / S, cE = entropy_coef
//                sum w / S, rounded once; then the targets' elements again with their g_k added
//                (children with the same token id summed in their order).
//
// Whether a ratio lies beyond the clip decides a whole gradient, so lp - old is a pair of floats:
// ln S = k ln 2 + ln f, f near 1, adds no error beyond 3e-8.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
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
constexpr int kMaxVectors = 10;                // 16-byte vectors per thread
constexpr int kMaxThreads = 512;
constexpr int64_t kMaxVocab = 262144;
constexpr float kFar = -1e30f;                 // in place of -inf where it meets a factor 0

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

// a + b = s + e exactly
__device__ __forceinline__ float two_sum(float a, float b, float& e) {
    const float s = a + b, bb = s - a;
    e = (a - (s - bb)) + (b - bb);
    return s;
}

// sums of e^(x - m) and e^(x - m) (x - m) over some logits
struct Stat {
    float m, s, t;
};
__device__ __forceinline__ Stat join(Stat a, Stat b) {
    Stat r;
    r.m = max_nan(a.m, b.m);
    // (far below the other side counts as -1e30 below, so that 0 meets no infinity; +inf and NaN are
    // told by m alone)
    const float da = fmaxf(a.m - r.m, kFar), db = fmaxf(b.m - r.m, kFar);
    const float ea = fast_exp2(da * kLog2e), eb = fast_exp2(db * kLog2e);
    r.s = a.s * ea + b.s * eb;
    r.t = (a.t + a.s * da) * ea + (b.t + b.s * db) * eb;
    return r;
}

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
    const float ratio = expf(dh + dl);
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
        const float far = (ref - h2) - lo, em = expm1f(far);
        // e^far - far - 1: by its series where the difference would lose its digits
        const float k3 = fabsf(far) < 0.25f
                             ? far * far * (0.5f + far * (1.f / 6 + far * (1.f / 24 + far * (1.f / 120 + far * (1.f / 720)))))
                             : far == INFINITY ? far : em - far;
        loss += p.kl * k3;
        g -= p.kl * em;
    }
    sum.g += w * g;
    sum.w += w;
    sum.loss += w * loss;
    return h2 + lo;
}

struct Shared {
    Stat stats[8 * (kMaxThreads / 32)];        // by CTA of the cluster and warp
    Sums sums[kMaxThreads / 32];
};

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

template <int NV>
__global__ void __launch_bounds__(kMaxThreads) policy_kernel(const Params p) {
    __shared__ Shared S;
    cg::cluster_group cluster = cg::this_cluster();
    const int C = (int)cluster.num_blocks(), me = (int)cluster.block_rank();
    const int T = blockDim.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = T >> 5;
    const int r = blockIdx.x / C;
    const int4 info = p.rows[r];
    const int first = info.x, n = info.y;
    // the row as a run of 16-byte vectors; the first and the last may belong to it in part
    const uint16_t* row_x = p.logits + r * p.stride;
    uint16_t* row_d = p.dlogits ? p.dlogits + r * p.d_stride : nullptr;
    const int V = (int)p.vocab, shift = (int)((reinterpret_cast<uintptr_t>(row_x) & 15u) >> 1);
    const int vectors = (V + shift + 7) / 8, per = (vectors + C - 1) / C;
    const int lo = min(me * per, vectors), hi = min(lo + per, vectors);
    const bool together = row_d && ((reinterpret_cast<uintptr_t>(row_x) ^ reinterpret_cast<uintptr_t>(row_d)) & 15u) == 0;
    grid_dep_wait();
    grid_dep_launch();
    if (!(ta_ok(p.status, 600, first, 0, p.n_pred + 1) && ta_ok(p.status, 601, (long long)first + n, 0, p.n_pred + 1))) return;

    // up to 32 predictions of one target: each lane has one, in every warp
    const bool narrow = info.w == 1 && n <= 32;
    int4 mine = make_int4(0, 0, 0, 0);
    float w = 0.f;
    bool active = n > 0;
    if (narrow) {
        if (lane < n) {
            mine = p.pred[first + lane];
            if (ta_ok(p.status, 602, mine.x, 0, p.n_pred)) w = p.weights ? p.weights[mine.x] : p.each;
        }
        active = __any_sync(0xffffffffu, w != 0.f);
    } else if (n > 0 && p.weights) {
        bool any = false;
        for (int i = tid; i < n && !any; i += T) {
            const int k = p.pred[first + i].x;
            any = ta_ok(p.status, 602, k, 0, p.n_pred) && p.weights[k] != 0.f;
        }
        active = __syncthreads_or(any);
    }
    if (!active) {                             // (the same in every CTA of the cluster)
        if (row_d)
            for (int v = lo + tid; v < hi; v += T) {
                const int i0 = 8 * v - shift;
                if (together && i0 >= 0 && i0 + 8 <= V) {
                    __stcs(reinterpret_cast<uint4*>(row_d + i0), make_uint4(0, 0, 0, 0));
                } else {
                    for (int i = max(i0, 0); i < min(i0 + 8, V); ++i) row_d[i] = 0;
                }
            }
        if (me == 0) {
            if (p.logprobs)
                for (int i = tid; i < n; i += T) {
                    const int k = p.pred[first + i].x;
                    if (ta_ok(p.status, 602, k, 0, p.n_pred)) p.logprobs[k] = 0.f;
                }
            if (tid == 0) {
                p.row_loss[r] = 0.f;
                if (p.entropy) p.entropy[r] = 0.f;
            }
        }
        return;
    }
    auto begun = cluster.barrier_arrive();     // no CTA's shared memory is written before it runs

    // ---- the slice, and its statistics ---------------------------------------------------
    uint4 x[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int v = lo + j * T + tid, i0 = 8 * v - shift;
        x[j] = make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u);   // -inf
        if (v < hi) {
            if (i0 >= 0 && i0 + 8 <= V) {
                x[j] = __ldcs(reinterpret_cast<const uint4*>(row_x + i0));
            } else {
                uint32_t u[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int a = i0 + 2 * i, b = a + 1;
                    u[i] = (a >= 0 && a < V ? row_x[a] : 0xff80u) | ((b >= 0 && b < V ? row_x[b] : 0xff80u) << 16);
                }
                x[j] = make_uint4(u[0], u[1], u[2], u[3]);
            }
        }
    }
    // one target: it is the next packed row (a node's tokens and its only child follow each other)
    const bool single = info.w == 1;
    int y = -1;
    float xy = 0.f, old = 0.f, a = 0.f, ref = 0.f;
    if (single && ta_ok(p.status, 603, r + 1, 0, p.N)) {
        y = p.tokens[r + 1];
        xy = y >= 0 && y < V ? lo16(row_x[y]) : __int_as_float(0x7fc00000);
        if (narrow && w != 0.f) {
            old = p.old ? p.old[mine.x] : 0.f;
            a = advantage(p, mine);
            ref = p.kl != 0.f ? p.ref[mine.x] : 0.f;
        }
    }
    Stat st;
    {
        uint32_t m2 = 0xff80ff80u;
#pragma unroll
        for (int j = 0; j < NV; ++j) m2 = max2_nan(max2_nan(m2, max2_nan(x[j].x, x[j].y)), max2_nan(x[j].z, x[j].w));
        st.m = max_nan(lo16(m2), hi16(m2));
        const float base = st.m == -INFINITY ? 0.f : st.m;
        st.s = st.t = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const uint32_t u[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float d = fmaxf((i & 1 ? hi16(u[i / 2]) : lo16(u[i / 2])) - base, kFar);
                const float e = fast_exp2(d * kLog2e);
                st.s += e;
                st.t = fmaf(e, d, st.t);
            }
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        Stat b;
        b.m = __shfl_xor_sync(0xffffffffu, st.m, o);
        b.s = __shfl_xor_sync(0xffffffffu, st.s, o);
        b.t = __shfl_xor_sync(0xffffffffu, st.t, o);
        st = join(st, b);
    }
    cluster.barrier_wait(std::move(begun));
    if (lane < C) cluster.map_shared_rank(&S, lane)->stats[me * nw + warp] = st;
    cluster.sync();
    {
        const Stat none = {-INFINITY, 0.f, 0.f};
        st = lane < C * nw ? S.stats[lane] : none;
        for (int i = lane + 32; i < C * nw; i += 32) st = join(st, S.stats[i]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            Stat b;
            b.m = __shfl_xor_sync(0xffffffffu, st.m, o);
            b.s = __shfl_xor_sync(0xffffffffu, st.s, o);
            b.t = __shfl_xor_sync(0xffffffffu, st.t, o);
            st = join(st, b);
        }
    }
    Row row;
    {
        row.m = fabsf(st.m) < INFINITY ? st.m : __int_as_float(0x7fc00000);
        // S = 2^k f, 0.7 < f < 1.5;  ln 2 = 45426 / 2^16 + 1.42860682e-6
        int k;
        float f = frexpf(st.s, &k);
        if (f < 0.7f) {
            f *= 2.f;
            --k;
        }
        row.lk = (float)k * (45426.f / 65536.f);
        row.ll = fmaf((float)k, 1.42860682e-6f, logf(f));
        row.h = row.m == row.m ? (row.lk + row.ll) - st.t / st.s : row.m;
    }

    // ---- the predictions ---------------------------------------------------------------------
    Sums sum = {0.f, 0.f, 0.f};
    if (narrow) {
        float lp = 0.f;
        if (w != 0.f) lp = predict(p, row, w, xy, old, p.old != nullptr, a, ref, sum);
        if (me == 0 && warp == 0 && lane < n && p.logprobs) p.logprobs[mine.x] = lp;
        sum = warp_sum(sum);
    } else {
        if (single) {
            predict_all(p, row, first, n, xy, tid, T, me == 0, sum);
        } else {
            // several targets: a warp each
            for (int j = warp; j < info.w; j += nw) {
                const int4 t = p.targets[info.z + j];
                if (!ta_ok(p.status, 604, t.x, 0, p.N)) continue;
                const int yj = p.tokens[t.x], v = (yj + shift) / 8;
                const bool inside = yj >= 0 && yj < V;
                const float xj = inside ? lo16(row_x[yj]) : __int_as_float(0x7fc00000);
                Sums part = {0.f, 0.f, 0.f};
                predict_all(p, row, t.y, t.z, xj, lane, 32, me == 0, part);
                part = warp_sum(part);
                if (lane == 0) {
                    sum.g += part.g;
                    sum.w += part.w;
                    sum.loss += part.loss;
                    if (inside && v >= lo && v < hi) {
                        p.tx[t.x] = xj;
                        p.tg[t.x] = part.g;
                    }
                }
            }
        }
        sum = warp_sum(sum);
        if (lane == 0) S.sums[warp] = sum;
        __syncthreads();
        sum = {0.f, 0.f, 0.f};
        for (int i = 0; i < nw; ++i) {
            sum.g += S.sums[i].g;
            sum.w += S.sums[i].w;
            sum.loss += S.sums[i].loss;
        }
    }
    if (me == 0 && tid == 0) {
        p.row_loss[r] = sum.loss;
        if (p.entropy) p.entropy[r] = row.h;
    }
    // the gradient may lie over the logits: every CTA has read its targets' logits
    if (!single) cluster.sync();
    if (!row_d) return;

    // ---- the gradient --------------------------------------------------------------------
    const float ts = st.t / st.s;
    const float cg_ = row.m == row.m ? -p.grad_scale * sum.g / st.s : row.m;
    const float ce = p.ent != 0.f ? p.grad_scale * p.ent * sum.w / st.s : 0.f;
    auto value = [&](float xv) {
        const float d = fmaxf(xv - row.m, kFar);
        return fast_exp2(d * kLog2e) * fmaf(ce, d - ts, cg_);
    };
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int v = lo + j * T + tid, i0 = 8 * v - shift;
        if (v >= hi) break;
        const uint32_t u[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = pack_bf16x2(value(lo16(u[i])), value(hi16(u[i])));
        if (together && i0 >= 0 && i0 + 8 <= V) {
            __stcs(reinterpret_cast<uint4*>(row_d + i0), make_uint4(o[0], o[1], o[2], o[3]));
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i0 + i >= 0 && i0 + i < V) row_d[i0 + i] = (uint16_t)(o[i / 2] >> (16 * (i & 1)));
        }
    }
    __syncthreads();
    auto put = [&](int yj, float xj, float g) {
        row_d[yj] = (uint16_t)pack_bf16x2(value(xj) + p.grad_scale * g, 0.f);
    };
    if (single) {
        const int v = (y + shift) / 8;
        if (tid == 0 && y >= 0 && y < V && v >= lo && v < hi) put(y, xy, sum.g);
    } else {
        for (int j = tid; j < info.w; j += T) {
            const int s = p.targets[info.z + j].x;
            if (!ta_ok(p.status, 604, s, 0, p.N)) continue;
            const int yj = p.tokens[s], v = (yj + shift) / 8;
            if (yj < 0 || yj >= V || v < lo || v >= hi) continue;
            bool earlier = false;              // another child has the same token: the first one adds them up
            for (int i = 0; i < j && !earlier; ++i) earlier = p.tokens[p.targets[info.z + i].x] == yj;
            if (earlier) continue;
            float g = p.tg[s];
            for (int i = j + 1; i < info.w; ++i) {
                const int si = p.targets[info.z + i].x;
                if (p.tokens[si] == yj) g += p.tg[si];
            }
            put(yj, p.tx[s], g);
        }
    }
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

template <int NV>
cudaError_t launch(int64_t rows, int C, int T, cudaStream_t s, const Params& p) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * C));
    cfg.blockDim = dim3(T);
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim = {(unsigned)C, 1, 1};
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return launched(cudaLaunchKernelEx(&cfg, policy_kernel<NV>, p));
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
    // CTAs and threads of a row, and each thread's vectors (one more vector for a row that
    // starts inside one)
    const int64_t vectors = (vocab + 7) / 8 + 1;
    int C = 1, T = 256;
    while (C < 8 && vectors > (int64_t)C * T * kMaxVectors) C *= 2;
    if (vectors > (int64_t)C * T * kMaxVectors) T = kMaxThreads;
    const int64_t per = (vectors + C - 1) / C;
    while (T > 64 && per <= T / 2) T /= 2;
    const int nv = (int)((per + T - 1) / T);
    if (P->N * C > INT32_MAX) return TREE_ATTN_ERR_TOO_LARGE;
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
    cudaError_t e = cudaErrorInvalidValue;
    switch (nv) {
        case 1: e = launch<1>(P->N, C, T, s, p); break;
        case 2: e = launch<2>(P->N, C, T, s, p); break;
        case 3: e = launch<3>(P->N, C, T, s, p); break;
        case 4: e = launch<4>(P->N, C, T, s, p); break;
        case 5: e = launch<5>(P->N, C, T, s, p); break;
        case 6: e = launch<6>(P->N, C, T, s, p); break;
        case 7: e = launch<7>(P->N, C, T, s, p); break;
        case 8: e = launch<8>(P->N, C, T, s, p); break;
        case 9: e = launch<9>(P->N, C, T, s, p); break;
        case 10: e = launch<10>(P->N, C, T, s, p); break;
    }
    if (e != cudaSuccess) return TREE_ATTN_ERR_CUDA;
    e = launch_pdl(policy_sum_kernel, dim3(1), dim3(1024), 0, s, (const float*)p.row_loss, (int)P->N, loss);
    return e == cudaSuccess ? TREE_ATTN_OK : TREE_ATTN_ERR_CUDA;
}

}  // extern "C"
