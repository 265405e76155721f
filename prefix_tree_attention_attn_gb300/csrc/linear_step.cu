// One token of linear attention per branch from and to states in slots (include/tree_linear.h).
//
//   S = gamma S + k v^T (read and written once: 64 KB each way per branch and kv-head at d 128),
//   o = scale q^T S for the group's query heads.
//
// Memory-bound: 2 + 2 G multiply-adds per 8 bytes.  A column of S goes with its value feature alone, so
// a CTA takes a block of CB columns of one (branch, kv-head) and nothing is joined between CTAs.  A
// thread holds 4 columns of some rows in registers, all its loads under way at once; the sums over the rows
// of four query heads at a time meet in shared memory.  1,024 branches of 8 kv-heads and 32 query heads at d 128: 168 us,
// 6.5 TB/s of states; 64 branches 12.6 us (the states stay in L2 between steps); one 2.8.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "align.h"
#include "kernels.h"
#include "plan.h"
#include "tree_linear.h"

namespace treeattn {

namespace {

constexpr int kThreads = 256;
constexpr int kHeads = 4;                      // query heads at a time

struct StepParams {
    float* states;
    const int32_t* in;
    const int32_t* out;
    const uint16_t* q;
    const uint16_t* k;
    const uint16_t* v;
    int64_t q_stride, k_stride, v_stride;
    uint16_t* o;
    const float* decay;
    int32_t n_slots, hkv, group;
    float scale;
    int* status;
};

__device__ __forceinline__ float bf16f(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }

template <int D, int CB>
__global__ void __launch_bounds__(kThreads) step_kernel(const StepParams p) {
    constexpr int LC = CB / 4, RG = kThreads / LC, RPT = D / RG;   // lanes across, row groups, rows a thread
    constexpr int WC = LC < 32 ? LC : 32;                          // lanes of a warp that lie side by side
    __shared__ __align__(16) float ks[D], qs[kHeads][D];
    __shared__ __align__(16) float part[kHeads][kThreads / 32][CB];
    const int cb = blockIdx.x % (D / CB), unit = blockIdx.x / (D / CB), g = unit % p.hkv;
    const int64_t r = unit / p.hkv;
    const int c = 4 * (threadIdx.x % LC), row0 = threadIdx.x / LC * RPT;
    grid_dep_wait();
    grid_dep_launch();
    const int to = p.out[r], from = p.in[r];
    const bool bad = to < -1 || to >= p.n_slots || from < -1 || from >= p.n_slots;
    if (bad && threadIdx.x == 0) report_notice(p.status, TREE_ATTN_ERR_INVALID_SLOT);
    const float gamma = p.decay[g];
    if (unit < p.hkv && cb == 0 && threadIdx.x == 0 && !(gamma > 0.f && gamma <= 1.f))
        report_notice(p.status, TREE_ATTN_ERR_INVALID_DECAY);
    if (to < 0 || to >= p.n_slots) return;
    const size_t at = (size_t)row0 * D + cb * CB + c;
    float4 S[RPT];
    if (from >= 0 && from < p.n_slots) {
        const float* src = p.states + ((size_t)from * p.hkv + g) * D * D + at;
#pragma unroll
        for (int i = 0; i < RPT; ++i) S[i] = *reinterpret_cast<const float4*>(src + i * D);
    } else {
#pragma unroll
        for (int i = 0; i < RPT; ++i) S[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    const uint2 v2 = *reinterpret_cast<const uint2*>(p.v + r * p.v_stride + g * D + cb * CB + c);
    if (threadIdx.x < D) ks[threadIdx.x] = bf16f(p.k[r * p.k_stride + g * D + threadIdx.x]);
    const uint16_t* q = p.q + r * p.q_stride + (size_t)g * p.group * D;
    auto load_q = [&](int h0) {
        for (int i = threadIdx.x; i < kHeads * D; i += kThreads)
            if (h0 + i / D < p.group) qs[i / D][i % D] = bf16f(q[h0 * D + i]);
    };
    load_q(0);
    __syncthreads();
    const float4 v = make_float4(__uint_as_float(v2.x << 16), __uint_as_float(v2.x & 0xffff0000u),
                                 __uint_as_float(v2.y << 16), __uint_as_float(v2.y & 0xffff0000u));
    float* dst = p.states + ((size_t)to * p.hkv + g) * D * D + at;
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const float k = ks[row0 + i];
        S[i] = make_float4(fmaf(gamma, S[i].x, k * v.x), fmaf(gamma, S[i].y, k * v.y), fmaf(gamma, S[i].z, k * v.z),
                           fmaf(gamma, S[i].w, k * v.w));
        *reinterpret_cast<float4*>(dst + i * D) = S[i];
    }
    const int warp = threadIdx.x >> 5;
    for (int h0 = 0; h0 < p.group; h0 += kHeads) {
        if (h0) {
            load_q(h0);
            __syncthreads();
        }
        const int nh = min(kHeads, p.group - h0);
#pragma unroll
        for (int h = 0; h < kHeads; ++h) {
            if (h >= nh) break;
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int i = 0; i < RPT; ++i) {
                const float x = qs[h][row0 + i];
                a.x = fmaf(x, S[i].x, a.x);
                a.y = fmaf(x, S[i].y, a.y);
                a.z = fmaf(x, S[i].z, a.z);
                a.w = fmaf(x, S[i].w, a.w);
            }
#pragma unroll
            for (int o = WC; o < 32; o *= 2) {
                a.x += __shfl_xor_sync(0xffffffffu, a.x, o);
                a.y += __shfl_xor_sync(0xffffffffu, a.y, o);
                a.z += __shfl_xor_sync(0xffffffffu, a.z, o);
                a.w += __shfl_xor_sync(0xffffffffu, a.w, o);
            }
            if ((threadIdx.x & 31) < WC) *reinterpret_cast<float4*>(&part[h][warp][c]) = a;
        }
        __syncthreads();
        for (int i = threadIdx.x; i < nh * CB; i += kThreads) {
            const int h = i / CB, col = i % CB;
            float sum = 0.f;
#pragma unroll
            for (int w = 0; w < kThreads / 32; ++w) sum += part[h][w][col];
            const uint32_t b = pack_bf16x2(p.scale * sum, 0.f);
            p.o[(r * p.hkv * p.group + (size_t)g * p.group + h0 + h) * D + cb * CB + col] = (uint16_t)b;
        }
        // (the next heads' barrier after their load keeps `part` until it has been read)
    }
}

template <int D>
cudaError_t launch(int64_t units, cudaStream_t s, const StepParams& p) {
    // Few large states: narrow blocks of columns while a wave holds them.  Measured, us in blocks of 32 and of 64: 8 states of
    // 128 x 128 2.78 and 3.08, 32 2.74 and 3.03, 48 3.20 and 3.03, 128 5.14 and 4.08; of 64 x 64 wide ones always
    // (8: 2.43 and 2.30).
    if constexpr (D == 128)
        if (units * (D / 32) <= 152)
            return launch_pdl(step_kernel<D, 32>, dim3((unsigned)(units * (D / 32))), dim3(kThreads), 0, s, p);
    return launch_pdl(step_kernel<D, 64>, dim3((unsigned)(units * (D / 64))), dim3(kThreads), 0, s, p);
}

}  // namespace

}  // namespace treeattn

using namespace treeattn;

extern "C" int tree_attn_linear_step(float* states, int32_t n_slots, const int32_t* slot_in, const int32_t* slot_out,
                                     const void* q, const void* k, const void* v, int64_t q_stride, int64_t k_stride,
                                     int64_t v_stride, void* o, const float* decay, int64_t n_rows, int32_t hq,
                                     int32_t hkv, int32_t d, float scale, void* stream) {
    if (n_rows < 0 || n_slots < 0 || hq <= 0 || hkv <= 0 || hq % hkv != 0) return TREE_ATTN_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return TREE_ATTN_ERR_UNSUPPORTED;
    if (!std::isfinite(scale)) return TREE_ATTN_ERR_INVALID_ARG;
    if (n_rows == 0) return TREE_ATTN_OK;
    if (!slot_in || !slot_out || !q || !k || !v || !o || !decay || (n_slots > 0 && !states)) return TREE_ATTN_ERR_INVALID_ARG;
    for (const int64_t x : {q_stride, k_stride, v_stride})
        if (x % 8) return TREE_ATTN_ERR_INVALID_ARG;
    if (q_stride < (int64_t)hq * d || k_stride < (int64_t)hkv * d || v_stride < (int64_t)hkv * d) return TREE_ATTN_ERR_INVALID_ARG;
    for (const void* p : {(const void*)states, q, k, v, (const void*)o})
        if (!aligned(p, 16)) return TREE_ATTN_ERR_ALIGNMENT;
    if (!aligned(slot_in, 4) || !aligned(slot_out, 4) || !aligned(decay, 4)) return TREE_ATTN_ERR_ALIGNMENT;
    if (n_rows > INT32_MAX / 4 / hkv) return TREE_ATTN_ERR_TOO_LARGE;
    int dev, *status;
    int st;
    if ((st = current_device(&dev)) || (st = get_status_ptr(dev, &status))) return st;
    const StepParams p = {states, slot_in, slot_out, static_cast<const uint16_t*>(q), static_cast<const uint16_t*>(k),
                          static_cast<const uint16_t*>(v), q_stride, k_stride, v_stride, static_cast<uint16_t*>(o), decay,
                          n_slots, hkv, hq / hkv, scale, status};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = d == 128 ? launch<128>(n_rows * hkv, s, p) : launch<64>(n_rows * hkv, s, p);
    return e == cudaSuccess ? TREE_ATTN_OK : TREE_ATTN_ERR_CUDA;
}
