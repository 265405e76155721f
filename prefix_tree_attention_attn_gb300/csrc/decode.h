// Decode plan: the tree's pages, the work items of the attention over them, and
// the tables the cache and attention kernels read (internal to libtreeattn).
#pragma once

#include <cstdint>
#include <mutex>
#include <vector>

#include "plan.h"
#include "tree_decode.h"

namespace treeattn {

constexpr int kPage = TREE_DECODE_PAGE;
constexpr int kDecodeRows = 128;         // query rows (query x head of the group) per work item at most
constexpr int kDecodeNarrow = 8;         // rows up to which a run's items are for single warps
constexpr int kDecodeWarps = 6;          // such items per CTA
constexpr int kDecodeMaxChunk = 128;     // pages per CTA's item at most
constexpr int kDecodeMaxWarp = 32;       // pages per warp's item at most: one per lane

// Device copy of the tables (one per device; pointers into one buffer).
struct DeviceDecode {
    void* base = nullptr;
    int32_t* entries = nullptr;       // [4*E]
    int32_t* items = nullptr;         // [8*kDecodeWarps*CTAs]
    int32_t* order = nullptr;         // [live] query index at each place
    int32_t* combine_ptr = nullptr;   // [live*n_sub+1]
    int32_t* combine_row = nullptr;
    int32_t* jobs = nullptr;          // [4*jobs]
    int32_t* tails = nullptr;         // [2*R] per query {node or -1, first index into page_tab}
    int32_t* page_tab = nullptr;      // pages by node id
    int32_t* room = nullptr;          // [n_nodes] capacity
    bool ready = false;
};

struct DecodePlan {
    int32_t n_nodes = 0, R = 0, live = 0, n_pages = 0;
    int32_t hq = 0, hkv = 0, d = 0, group = 0, n_sub = 1, gsub = 1;
    int32_t chunk = 0, warp_chunk = 0;
    int64_t n_fresh = 0, part_rows = 0;
    size_t ws_bytes = 0;
    bool repeated = false;            // two queries in one node
    std::vector<int32_t> entries, items, order, combine_ptr, combine_row, jobs, tails, page_tab, room;
    std::mutex mu;
    DeviceDecode dev[kMaxDevices];
};

}  // namespace treeattn

struct tree_decode_plan_s : public treeattn::DecodePlan {};

namespace treeattn {
// Device tables of the current device (uploaded once).
int ensure_decode(tree_decode_plan_s* P, DeviceDecode** out);
}  // namespace treeattn
