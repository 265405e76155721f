// Copies of whole cache pages (include/tree_decode.h), in several caches of the same shape at once.
//
// A copy: every byte read once and written once.  The page numbers and the caches' addresses go
// with the launch (kernel parameters hold 32 KB), so nothing is uploaded and the host's arrays are
// its own again when the call returns.  A CTA copies 16 KB of one page of one cache, four 16-byte
// loads under way in each thread; the CTA of a page's first piece takes its scales along.  2,000 pages of
// 131 KB: 82 us, 0.95 of the measured copy's rate; 16 pages in each of 32 caches 18.6 (of 25 to 31 that a call takes the host).
#include <cuda_runtime.h>

#include <algorithm>
#include <new>
#include <vector>

#include "align.h"
#include "decode.h"
#include "kernels.h"

namespace treeattn {

namespace {

constexpr int kCaches = 32;                    // per launch
constexpr int kMoves = 1024;
constexpr int kPiece = 16 * 1024;              // bytes per CTA
constexpr int kThreads = 256;

struct CopyParams {
    uint8_t* k8[kCaches];
    uint8_t* v8[kCaches];
    float* ks[kCaches];
    float* vs[kCaches];
    int32_t src[kMoves];
    int32_t dst[kMoves];
    int32_t page_bytes;                        // of the keys or of the values
    int32_t pieces;                            // per page, keys and values
    int32_t hkv, n_pages;
    int* status;
};

__global__ void __launch_bounds__(kThreads) copy_kernel(const __grid_constant__ CopyParams p) {
    const int piece = blockIdx.x % p.pieces, move = blockIdx.x / p.pieces, cache = blockIdx.y;
    const int64_t src = p.src[move], dst = p.dst[move];
    grid_dep_wait();
    grid_dep_launch();
    if (!(ta_ok(p.status, 541, src, 0, p.n_pages) && ta_ok(p.status, 542, dst, 0, p.n_pages))) return;
    const bool is_v = piece >= p.pieces / 2;
    uint8_t* base = is_v ? p.v8[cache] : p.k8[cache];
    const int at = (piece - (is_v ? p.pieces / 2 : 0)) * kPiece, n = min(kPiece, p.page_bytes - at) / 16;
    const uint4* a = reinterpret_cast<const uint4*>(base + src * p.page_bytes + at);
    uint4* b = reinterpret_cast<uint4*>(base + dst * p.page_bytes + at);
    constexpr int PER = kPiece / 16 / kThreads;
    uint4 x[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i)
        if (threadIdx.x + i * kThreads < n) x[i] = __ldcs(a + threadIdx.x + i * kThreads);
#pragma unroll
    for (int i = 0; i < PER; ++i)
        if (threadIdx.x + i * kThreads < n) b[threadIdx.x + i * kThreads] = x[i];
    if (at == 0) {
        float* s = is_v ? p.vs[cache] : p.ks[cache];
        for (int h = threadIdx.x; h < p.hkv; h += kThreads) s[dst * p.hkv + h] = s[src * p.hkv + h];
    }
}

// Page numbers inside the pool, targets all different and none of them a source.  A table of the pool's pages costs
// its clearing (0.17 us for 5,000 pages, 27 for a million), sorted targets n log n (16 moves 0.3 us, 256 4.5,
// 2,000 30): even at 300 to 500 pages per move.
bool well_formed(const int32_t* src, const int32_t* dst, int64_t n, int32_t n_pages) {
    for (int64_t i = 0; i < n; ++i)
        if (src[i] < 0 || src[i] >= n_pages || dst[i] < 0 || dst[i] >= n_pages) return false;
    if (n_pages / 400 >= n) {
        std::vector<int32_t> to(dst, dst + n);
        std::sort(to.begin(), to.end());
        if (std::adjacent_find(to.begin(), to.end()) != to.end()) return false;
        return std::none_of(src, src + n, [&](int32_t x) { return std::binary_search(to.begin(), to.end(), x); });
    }
    std::vector<uint8_t> seen(n_pages, 0);
    for (int64_t i = 0; i < n; ++i) seen[src[i]] = 1;
    for (int64_t i = 0; i < n; ++i) {
        if (seen[dst[i]]) return false;
        seen[dst[i]] = 1;
    }
    return true;
}

}  // namespace

}  // namespace treeattn

using namespace treeattn;

extern "C" int tree_attn_cache_copy(int32_t n_caches, void* const* k8, void* const* v8, float* const* k_scale,
                                    float* const* v_scale, int32_t n_pages, int32_t hkv, int32_t d, const int32_t* src,
                                    const int32_t* dst, int64_t n, void* stream) {
    if (n_caches < 0 || n_pages < 0 || n < 0 || hkv <= 0) return TREE_ATTN_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return TREE_ATTN_ERR_UNSUPPORTED;
    if ((int64_t)hkv * kPage * d > (1 << 30)) return TREE_ATTN_ERR_TOO_LARGE;
    if (n == 0 || n_caches == 0) return TREE_ATTN_OK;
    if (!k8 || !v8 || !k_scale || !v_scale || !src || !dst || n > n_pages) return TREE_ATTN_ERR_INVALID_ARG;
    for (int c = 0; c < n_caches; ++c) {
        if (!k8[c] || !v8[c] || !k_scale[c] || !v_scale[c]) return TREE_ATTN_ERR_INVALID_ARG;
        if (!aligned(k8[c], 16) || !aligned(v8[c], 16) || !aligned(k_scale[c], 4) || !aligned(v_scale[c], 4))
            return TREE_ATTN_ERR_ALIGNMENT;
    }
    try {
        if (!well_formed(src, dst, n, n_pages)) return TREE_ATTN_ERR_INVALID_ARG;
    } catch (const std::bad_alloc&) {
        return TREE_ATTN_ERR_OUT_OF_MEMORY;
    }
    int dev, *status;
    int st;
    if ((st = current_device(&dev)) || (st = get_status_ptr(dev, &status))) return st;
    CopyParams p;
    p.page_bytes = hkv * kPage * d;
    p.pieces = 2 * ((p.page_bytes + kPiece - 1) / kPiece);
    p.hkv = hkv;
    p.n_pages = n_pages;
    p.status = status;
    for (int32_t c0 = 0; c0 < n_caches; c0 += kCaches) {
        const int nc = std::min(kCaches, n_caches - c0);
        for (int c = 0; c < kCaches; ++c) {
            const int at = c0 + std::min(c, nc - 1);
            p.k8[c] = static_cast<uint8_t*>(k8[at]);
            p.v8[c] = static_cast<uint8_t*>(v8[at]);
            p.ks[c] = k_scale[at];
            p.vs[c] = v_scale[at];
        }
        for (int64_t i0 = 0; i0 < n; i0 += kMoves) {
            const int m = (int)std::min<int64_t>(kMoves, n - i0);
            std::copy(src + i0, src + i0 + m, p.src);
            std::copy(dst + i0, dst + i0 + m, p.dst);
            std::fill(p.src + m, p.src + kMoves, 0);
            std::fill(p.dst + m, p.dst + kMoves, 0);
            const cudaError_t e = launch_pdl(copy_kernel, dim3((unsigned)(m * p.pieces), (unsigned)nc), dim3(kThreads), 0,
                                             static_cast<cudaStream_t>(stream), p);
            if (e != cudaSuccess) return TREE_ATTN_ERR_CUDA;
        }
    }
    return TREE_ATTN_OK;
}
