// Cache calls of include/tree_decode.h: the plan's device tables, the write of
// whole nodes and the append of one token per decoding node.
//
// Quantisation.  A page's scale is 2^e with the smallest e >= -100 such that
// amax <= 448 * 2^e.  With amax = m * 2^E, 1 <= m < 2, and 448 = 1.75 * 2^8 that is
// e = E - 8, one more when m > 1.75: exponent arithmetic, no division.  Codes
// are x * 2^-e (exact but for fp32 underflow far below the smallest code) rounded
// once by the e4m3 conversion.
#include <cuda_runtime.h>

#include <algorithm>

#include "decode.h"
#include "kernels.h"

namespace treeattn {

int ensure_decode(tree_decode_plan_s* P, DeviceDecode** out) {
    int dev;
    int st = current_device(&dev);
    if (st) return st;
    std::lock_guard<std::mutex> lk(P->mu);
    DeviceDecode& D = P->dev[dev];
    if (D.ready) {
        *out = &D;
        return TREE_ATTN_OK;
    }
    const std::vector<int32_t>* src[9] = {&P->entries, &P->items, &P->order, &P->combine_ptr, &P->combine_row,
                                          &P->jobs, &P->tails, &P->page_tab, &P->room};
    int32_t** dst[9] = {&D.entries, &D.items, &D.order, &D.combine_ptr, &D.combine_row,
                        &D.jobs, &D.tails, &D.page_tab, &D.room};
    size_t offs[9], total = 0;
    for (int k = 0; k < 9; ++k) {
        offs[k] = total;
        total += (src[k]->size() + 63) / 64 * 64;   // 256-byte aligned sections
    }
    std::vector<int32_t> h;
    try {
        h.assign(std::max<size_t>(total, 64), 0);
    } catch (const std::exception&) {
        return TREE_ATTN_ERR_OUT_OF_MEMORY;
    }
    for (int k = 0; k < 9; ++k) std::copy(src[k]->begin(), src[k]->end(), h.begin() + offs[k]);
    void* buf = nullptr;
    if ((st = upload_words(&buf, h.data(), h.size()))) return st;
    for (int k = 0; k < 9; ++k) *dst[k] = static_cast<int32_t*>(buf) + offs[k];
    D.base = buf;
    D.ready = true;
    *out = &D;
    return TREE_ATTN_OK;
}

namespace {

constexpr int kMinExp = -100;

__device__ __forceinline__ float bf16_at(uint32_t w, int i) {
    return i ? __uint_as_float(w & 0xffff0000u) : __uint_as_float(w << 16);
}
// |x| for the scale: infinities and NaN do not count
__device__ __forceinline__ float finite_abs(float x) {
    const uint32_t a = __float_as_uint(x) & 0x7fffffffu;
    return a < 0x7f800000u ? __uint_as_float(a) : 0.f;
}
// exponent of the page scale for a largest finite magnitude (a bf16 value)
__device__ __forceinline__ int scale_exp(float amax) {
    const uint32_t b = __float_as_uint(amax);
    if (b < 0x00800000u) return kMinExp;   // zero or subnormal: far below 2^-100
    const int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
    return max(e, kMinExp);
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }   // -126 <= e <= 127

// two fp32 to two e4m3 bytes (first in the low byte), nearest even, saturating
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    return e4m3x2(a, b) | (e4m3x2(c, d) << 16);
}

struct WriteParams {
    const int32_t* jobs;
    const uint16_t* k;
    const uint16_t* v;
    int64_t k_stride, v_stride;
    uint8_t* k8;
    uint8_t* v8;
    float* ks;
    float* vs;
    int32_t hkv, n_pages;
    int64_t n_fresh;      // rows, with n_pages for the checks of debug builds
    int* status;
};

// ---- write: one CTA per (page, kv-head) -------------------------------------
// Memory-bound (4 bytes in, 2 out per token and feature).  Thread t holds 4
// consecutive tokens x 8 features of K and of V: eight 16-byte loads issued
// before anything waits, a warp's loads covering whole rows.  Four tokens of one
// feature are one word of V's transposed page, which goes through shared memory.
template <int D>
__global__ void __launch_bounds__(2 * D) write_kernel(const WriteParams p) {
    constexpr int FG = D / 8;                  // feature groups; 16 token groups
    constexpr int kPitch = kPage + 4;          // bytes per feature row in shared memory
    __shared__ __align__(16) uint8_t vt[D * kPitch];
    __shared__ float red[2][2 * D / 32];
    const int job = blockIdx.x / p.hkv, h = blockIdx.x % p.hkv;
    const int page = p.jobs[4 * job], row0 = p.jobs[4 * job + 1], n = p.jobs[4 * job + 2];
    if (!(ta_ok(p.status, 521, page, 0, p.n_pages) && ta_ok(p.status, 522, row0, 0, p.n_fresh - n + 1) &&
          ta_ok(p.status, 523, n, 1, kPage + 1)))
        return;
    const int fg = threadIdx.x % FG, tg = threadIdx.x / FG;
    uint4 a[4], b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool ok = 4 * tg + i < n;
        const int64_t r = row0 + 4 * tg + i;
        a[i] = ok ? __ldcs(reinterpret_cast<const uint4*>(p.k + r * p.k_stride + h * D + fg * 8)) : make_uint4(0, 0, 0, 0);
        b[i] = ok ? __ldcs(reinterpret_cast<const uint4*>(p.v + r * p.v_stride + h * D + fg * 8)) : make_uint4(0, 0, 0, 0);
    }
    float ma = 0.f, mb = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t wa[4] = {a[i].x, a[i].y, a[i].z, a[i].w}, wb[4] = {b[i].x, b[i].y, b[i].z, b[i].w};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            ma = fmaxf(ma, finite_abs(bf16_at(wa[j / 2], j & 1)));
            mb = fmaxf(mb, finite_abs(bf16_at(wb[j / 2], j & 1)));
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        ma = fmaxf(ma, __shfl_xor_sync(0xffffffffu, ma, o));
        mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, o));
    }
    if ((threadIdx.x & 31) == 0) {
        red[0][threadIdx.x >> 5] = ma;
        red[1][threadIdx.x >> 5] = mb;
    }
    __syncthreads();
    ma = mb = 0.f;
#pragma unroll
    for (int w = 0; w < 2 * D / 32; ++w) {
        ma = fmaxf(ma, red[0][w]);
        mb = fmaxf(mb, red[1][w]);
    }
    const int ea = scale_exp(ma), eb = scale_exp(mb);
    const float ia = pow2(-ea), ib = pow2(-eb);
    const int64_t ph = (int64_t)page * p.hkv + h;
    if (threadIdx.x == 0) {
        p.ks[ph] = pow2(ea);
        p.vs[ph] = pow2(eb);
    }
    uint8_t* kd = p.k8 + ph * kPage * D;
    uint32_t col[8];                            // col[j]: tokens 4tg..4tg+3 of feature 8fg+j
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t wa[4] = {a[i].x, a[i].y, a[i].z, a[i].w};
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = bf16_at(wa[j / 2], j & 1) * ia;
        if (4 * tg + i < n) {
            *reinterpret_cast<uint2*>(kd + (4 * tg + i) * D + fg * 8) =
                make_uint2(e4m3x4(f[0], f[1], f[2], f[3]), e4m3x4(f[4], f[5], f[6], f[7]));
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        float f[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t wb[4] = {b[i].x, b[i].y, b[i].z, b[i].w};
            f[i] = bf16_at(wb[j / 2], j & 1) * ib;
        }
        col[j] = e4m3x4(f[0], f[1], f[2], f[3]);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) *reinterpret_cast<uint32_t*>(vt + (fg * 8 + j) * kPitch + 4 * tg) = col[j];
    __syncthreads();
    // feature rows of 64 tokens; a page that is not full keeps the bytes behind its tokens
    uint8_t* vd = p.v8 + ph * kPage * D;
    for (int x = threadIdx.x; x < D * 16; x += 2 * D) {
        const int f = x / 16, t = 4 * (x % 16);
        const uint32_t w = *reinterpret_cast<const uint32_t*>(vt + f * kPitch + t);
        if (t + 4 <= n) {
            *reinterpret_cast<uint32_t*>(vd + f * kPage + t) = w;
        } else {
            for (int i = 0; t + i < n; ++i) vd[f * kPage + t + i] = (uint8_t)(w >> (8 * i));
        }
    }
}

struct AppendParams {
    const int32_t* tails;
    const int32_t* page_tab;
    const int32_t* room;
    const int32_t* lens;
    int32_t* lens_out;
    const uint16_t* k;
    const uint16_t* v;
    int64_t k_stride, v_stride;
    uint8_t* k8;
    uint8_t* v8;
    float* ks;
    float* vs;
    int32_t hkv, n_nodes, n_pages;
    int* status;
};

// four codes times a power of two <= 1, rounded to codes again
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float r) {
    uint32_t lo, hi;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi) : "r"(w));
    float f[4];
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(f[0]), "=f"(f[1]) : "r"(lo));
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(f[2]), "=f"(f[3]) : "r"(hi));
    return e4m3x4(f[0] * r, f[1] * r, f[2] * r, f[3] * r);
}

// ---- append: one CTA per query, one warp per (kv-head, K or V) -----------------
// A few hundred bytes per warp: a chain of dependent loads (length, page, scale), 3.0 us
// for 16 queries of 8 kv-heads.  A value's features lie a page row apart -- the order in
// which the attention reads them as operands -- so a new token touches one 32-byte sector
// for each: 33 MB that L2 fetches and writes back at 1,024 queries, which bounds that case
// at 20 us (a quarter of the warps, with four units' loads under way in each, took the
// same).  The page's older tokens are touched only when the new token makes the scale grow.
template <int D>
__global__ void __launch_bounds__(512) append_kernel(const AppendParams p) {
    const int r = blockIdx.x, node = p.tails[2 * r], first = p.tails[2 * r + 1];
    const bool known = node < 0 || ta_ok(p.status, 531, node, 0, p.n_nodes);
    const int room = node < 0 || !known ? 0 : p.room[node];
    grid_dep_wait();
    grid_dep_launch();
    if (node < 0 || !known) return;
    const int at = p.lens[node];
    __syncthreads();                     // every warp has read the length before it may change
    if (at < 0 || at >= room) {
        if (threadIdx.x == 0) {
            report_notice(p.status, TREE_ATTN_ERR_CACHE_FULL);
            p.lens_out[node] = at;
        }
        return;
    }
    const int page = p.page_tab[first + at / kPage], slot = at % kPage;
    if (!ta_ok(p.status, 532, page, 0, p.n_pages)) return;
    const int lane = threadIdx.x & 31;
    constexpr int PL = D / 32;           // features per lane
    for (int u = threadIdx.x >> 5; u < 2 * p.hkv; u += blockDim.x >> 5) {
        const int h = u >> 1;
        const bool is_v = u & 1;
        const int64_t ph = (int64_t)page * p.hkv + h;
        const uint16_t* src = is_v ? p.v + r * p.v_stride : p.k + r * p.k_stride;
        float f[4];
        if (PL == 4) {
            const uint2 w = *reinterpret_cast<const uint2*>(src + h * D + lane * 4);
            f[0] = bf16_at(w.x, 0); f[1] = bf16_at(w.x, 1); f[2] = bf16_at(w.y, 0); f[3] = bf16_at(w.y, 1);
        } else {
            const uint32_t w = *reinterpret_cast<const uint32_t*>(src + h * D + lane * 2);
            f[0] = bf16_at(w, 0); f[1] = bf16_at(w, 1); f[2] = f[3] = 0.f;
        }
        float m = fmaxf(fmaxf(finite_abs(f[0]), finite_abs(f[1])), fmaxf(finite_abs(f[2]), finite_abs(f[3])));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        float* scale = (is_v ? p.vs : p.ks) + ph;
        uint8_t* page8 = (is_v ? p.v8 : p.k8) + ph * kPage * D;
        const float need = pow2(scale_exp(m)), old = slot ? *scale : 0.f;
        const float now = fmaxf(need, old);
        if (slot && now > old) {
            const float ratio = old / now;   // a power of two (0 when far below every code)
            if (!is_v) {
                uint32_t* w = reinterpret_cast<uint32_t*>(page8);
                for (int i = lane; i < slot * D / 4; i += 32) w[i] = rescale4(w[i], ratio);
            } else {
                for (int i = lane; i < D * 16; i += 32) {
                    const int t = 4 * (i % 16);
                    if (t >= slot) continue;
                    uint8_t* w8 = page8 + (i / 16) * kPage + t;
                    const uint32_t w = *reinterpret_cast<uint32_t*>(w8), x = rescale4(w, ratio);
                    const int keep = slot - t;   // tokens of this word that are older
                    const uint32_t mask = keep >= 4 ? 0xffffffffu : (1u << (8 * keep)) - 1u;
                    *reinterpret_cast<uint32_t*>(w8) = (x & mask) | (w & ~mask);
                }
            }
            __syncwarp();
        }
        const float inv = 1.f / now;     // exact: a power of two in [2^-120, 2^100]
        const uint32_t c = e4m3x4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv);
        if (!is_v) {
            if (PL == 4) reinterpret_cast<uint32_t*>(page8 + slot * D)[lane] = c;
            else reinterpret_cast<uint16_t*>(page8 + slot * D)[lane] = (uint16_t)c;
        } else {
#pragma unroll
            for (int i = 0; i < PL; ++i) page8[(lane * PL + i) * kPage + slot] = (uint8_t)(c >> (8 * i));
        }
        if (lane == 0) *scale = now;
    }
    if (threadIdx.x == 0) p.lens_out[node] = at + 1;
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int check_cache(const tree_decode_plan_s* P, const void* k, const void* v, int64_t k_stride, int64_t v_stride,
                const void* k8, const void* v8, const void* ks, const void* vs) {
    if (!k || !v) return TREE_ATTN_ERR_INVALID_ARG;
    if (P->n_pages && (!k8 || !v8 || !ks || !vs)) return TREE_ATTN_ERR_INVALID_ARG;   // a pool of no pages has no address
    const int64_t row = (int64_t)P->hkv * P->d;
    if (k_stride < row || v_stride < row || k_stride % 8 || v_stride % 8) return TREE_ATTN_ERR_INVALID_ARG;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(k8, 16) || !aligned(v8, 16) || !aligned(ks, 4) || !aligned(vs, 4))
        return TREE_ATTN_ERR_ALIGNMENT;
    return TREE_ATTN_OK;
}

}  // namespace

}  // namespace treeattn

using namespace treeattn;

extern "C" {

int tree_attn_decode_plan_upload(tree_decode_plan_t P) {
    if (!P) return TREE_ATTN_ERR_INVALID_ARG;
    DeviceDecode* D = nullptr;
    return ensure_decode(P, &D);
}

void tree_attn_decode_plan_destroy(tree_decode_plan_t P) {
    if (!P) return;
    for (int i = 0; i < kMaxDevices; ++i)
        if (P->dev[i].base) free_words(i, P->dev[i].base);
    delete P;
}

int tree_attn_cache_write(tree_decode_plan_t P, const void* k, const void* v, int64_t k_stride, int64_t v_stride,
                          void* k8, void* v8, float* k_scale, float* v_scale, void* stream) {
    if (!P) return TREE_ATTN_ERR_INVALID_ARG;
    if (P->jobs.empty()) return TREE_ATTN_OK;
    int st = check_cache(P, k, v, k_stride, v_stride, k8, v8, k_scale, v_scale);
    if (st) return st;
    const int64_t grid = (int64_t)(P->jobs.size() / 4) * P->hkv;
    if (grid > INT32_MAX) return TREE_ATTN_ERR_TOO_LARGE;
    DeviceDecode* D = nullptr;
    st = ensure_decode(P, &D);
    if (st) return st;
    int dev, *status;
    if ((st = current_device(&dev)) || (st = get_status_ptr(dev, &status))) return st;
    const WriteParams p = {D->jobs, static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v), k_stride, v_stride,
                           static_cast<uint8_t*>(k8), static_cast<uint8_t*>(v8), k_scale, v_scale, P->hkv, P->n_pages, P->n_fresh, status};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (P->d == 128) write_kernel<128><<<(unsigned)grid, 256, 0, s>>>(p);
    else write_kernel<64><<<(unsigned)grid, 128, 0, s>>>(p);
    return cudaGetLastError() == cudaSuccess ? TREE_ATTN_OK : TREE_ATTN_ERR_CUDA;
}

int tree_attn_cache_append(tree_decode_plan_t P, const int32_t* lens, int32_t* lens_out, const void* k,
                           const void* v, int64_t k_stride, int64_t v_stride, void* k8, void* v8, float* k_scale,
                           float* v_scale, void* stream) {
    if (!P || !lens || !lens_out || P->repeated) return TREE_ATTN_ERR_INVALID_ARG;
    int st = check_cache(P, k, v, k_stride, v_stride, k8, v8, k_scale, v_scale);
    if (st) return st;
    if (!aligned(lens, 4) || !aligned(lens_out, 4)) return TREE_ATTN_ERR_ALIGNMENT;
    DeviceDecode* D = nullptr;
    st = ensure_decode(P, &D);
    if (st) return st;
    int dev, *status;
    if ((st = current_device(&dev)) || (st = get_status_ptr(dev, &status))) return st;
    const AppendParams p = {D->tails, D->page_tab, D->room, lens, lens_out, static_cast<const uint16_t*>(k),
                            static_cast<const uint16_t*>(v), k_stride, v_stride, static_cast<uint8_t*>(k8),
                            static_cast<uint8_t*>(v8), k_scale, v_scale, P->hkv, P->n_nodes, P->n_pages, status};
    const int threads = std::min(512, 64 * P->hkv);
    const cudaError_t e = P->d == 128 ? launch_pdl(append_kernel<128>, dim3(P->R), dim3(threads), 0,
                                                   static_cast<cudaStream_t>(stream), p)
                                      : launch_pdl(append_kernel<64>, dim3(P->R), dim3(threads), 0,
                                                   static_cast<cudaStream_t>(stream), p);
    return e == cudaSuccess ? TREE_ATTN_OK : TREE_ATTN_ERR_CUDA;
}

}  // extern "C"
