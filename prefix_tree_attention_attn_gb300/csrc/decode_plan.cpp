// Host planner of the decode calls (include/tree_decode.h).
//
// Places.  The queries are sorted by their node's depth-first number, so the
// queries under a node -- the ones that read its pages -- are one contiguous
// range of places.
//
// Runs.  A node whose query range equals its parent's continues its parent's
// run: a chain that one set of queries reads is one list of pages, however many
// nodes it was grown in.  A run's rows are its row groups (a query's heads that share
// a kv-head).  Runs of at most 8 rows are cut into items for single warps, kDecodeWarps
// of them to a CTA; larger runs into blocks of at most kDecodeRows rows and items for
// whole CTAs.  Each page of a run is read by one item per block of rows, whatever the
// number of rollouts behind it.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <functional>
#include <new>
#include <queue>

#include "decode.h"

namespace treeattn {

namespace {

constexpr int64_t kMaxCombine = (int64_t)1 << 27;
// CTAs of the attention that run at one time: two per SM
constexpr int32_t kSms = 152;
constexpr int64_t kSlots = kSms * 2;
// Cycles of a CTA besides its pages; of a page of a CTA's item, and of a warp's: alone on the
// SM, which order the launch a little better than those beside one another (3,050 and 5,800;
// long context 188 against 196 us).
constexpr int64_t kCtaStart = 9000, kCtaPageCycles = 2100, kWarpPageCycles = 4700;
// Time of a page in a warp's item, in times of a page in a CTA's item: 1.2 us against
// 0.75 us alone on an SM, 2.9 us against 1.55 us beside one another.
constexpr int64_t kWarpPage = 2;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

int build(const int32_t* parent, const int32_t* seg_len, const int32_t* capacity, int32_t n, const int32_t* pages,
          int32_t n_pages, const uint8_t* fresh, const int32_t* query_node, int32_t R, int32_t opt_cta,
          int32_t opt_warp, tree_decode_plan_s* P) {
    // ---- the tree: depth-first numbers, children by ascending id -------------------
    std::vector<int32_t> head(n, -1), next(n, -1), order, number(n, -1), subtree_end(n, 0);
    int32_t roots = -1;
    for (int32_t v = n - 1; v >= 0; --v) {   // prepend: lists come out in ascending id
        const int32_t p = parent[v];
        if (p < -1 || p >= n || p == v) return TREE_ATTN_ERR_INVALID_TREE;
        if (seg_len[v] < 0) return TREE_ATTN_ERR_INVALID_TREE;
        if (capacity && capacity[v] < seg_len[v]) return TREE_ATTN_ERR_INVALID_TREE;
        int32_t& h = p < 0 ? roots : head[p];
        next[v] = h;
        h = v;
    }
    order.reserve(n);
    std::vector<int32_t> stack;
    for (int32_t r = roots; r >= 0; r = next[r]) {
        int32_t v = r;
        while (v >= 0) {
            number[v] = (int32_t)order.size();
            order.push_back(v);
            if (head[v] >= 0) {
                stack.push_back(v);
                v = head[v];
                continue;
            }
            subtree_end[v] = (int32_t)order.size();
            while (next[v] < 0 || parent[v] < 0) {   // no sibling left: close the parents
                if (stack.empty()) {
                    v = -1;
                    break;
                }
                v = stack.back();
                stack.pop_back();
                subtree_end[v] = (int32_t)order.size();
                if (parent[v] < 0) {
                    v = -1;
                    break;
                }
            }
            if (v >= 0) v = next[v];
        }
    }
    if ((int32_t)order.size() != n) return TREE_ATTN_ERR_INVALID_TREE;   // a cycle is never reached

    // ---- pages by node ---------------------------------------------------------------
    std::vector<int64_t> first(n + 1, 0);
    P->room.resize(n);
    for (int32_t v = 0; v < n; ++v) {
        P->room[v] = capacity ? capacity[v] : seg_len[v];
        first[v + 1] = first[v] + ceil_div(P->room[v], kPage);
    }
    const int64_t used = first[n];
    if (used > INT32_MAX / 4) return TREE_ATTN_ERR_TOO_LARGE;
    if (used > n_pages) return TREE_ATTN_ERR_INVALID_ARG;
    P->page_tab.resize(used);
    std::vector<bool> taken(n_pages, false);
    for (int64_t i = 0; i < used; ++i) {
        const int32_t p = pages ? pages[i] : (int32_t)i;
        if (p < 0 || p >= n_pages || taken[p]) return TREE_ATTN_ERR_INVALID_ARG;
        taken[p] = true;
        P->page_tab[i] = p;
    }

    // ---- write jobs ------------------------------------------------------------------
    int64_t row = 0;
    for (int32_t v : order) {
        if (fresh && !fresh[v]) continue;
        for (int32_t t = 0; t < seg_len[v]; t += kPage) {
            if (row > INT32_MAX - kPage) return TREE_ATTN_ERR_TOO_LARGE;
            const int32_t here = std::min(kPage, seg_len[v] - t);
            P->jobs.insert(P->jobs.end(), {P->page_tab[first[v] + t / kPage], (int32_t)row, here, 0});
            row += here;
        }
    }
    P->n_fresh = row;

    // ---- places of the queries ---------------------------------------------------------
    for (int32_t r = 0; r < R; ++r) {
        if (query_node[r] < -1 || query_node[r] >= n) return TREE_ATTN_ERR_INVALID_ARG;
        if (query_node[r] >= 0) P->order.push_back(r);
        P->tails.push_back(query_node[r]);
        P->tails.push_back(query_node[r] < 0 ? 0 : (int32_t)first[query_node[r]]);
    }
    std::stable_sort(P->order.begin(), P->order.end(),
                     [&](int32_t a, int32_t b) { return number[query_node[a]] < number[query_node[b]]; });
    P->live = (int32_t)P->order.size();
    std::vector<int32_t> before(n + 1, 0);   // queries whose node has a smaller number
    for (int32_t r : P->order) {
        if (before[number[query_node[r]] + 1]++) P->repeated = true;
    }
    for (int32_t i = 0; i < n; ++i) before[i + 1] += before[i];

    // ---- runs ----------------------------------------------------------------------------
    std::vector<int32_t> run_of(n, -1), run_lo, run_hi;
    std::vector<std::vector<int32_t>> run_nodes;
    for (int32_t v : order) {
        const int32_t lo = before[number[v]], hi = before[subtree_end[v]];
        if (lo == hi) continue;
        const int32_t p = parent[v];
        if (p >= 0 && run_lo[run_of[p]] == lo && run_hi[run_of[p]] == hi) {
            run_of[v] = run_of[p];
        } else {
            run_of[v] = (int32_t)run_lo.size();
            run_lo.push_back(lo);
            run_hi.push_back(hi);
            run_nodes.emplace_back();
        }
        run_nodes[run_of[v]].push_back(v);
    }

    // ---- pages per item, then the items ------------------------------------------------------
    const int32_t per_block = std::max(1, kDecodeRows / P->gsub);   // row groups per item
    const size_t n_runs = run_lo.size();
    std::vector<int64_t> run_pages(n_runs, 0), blocks(n_runs, 0);   // blocks = 0: items for warps
    int64_t cost = 0;                                               // of all items, in CTA-pages
    for (size_t k = 0; k < n_runs; ++k) {
        for (int32_t v : run_nodes[k]) run_pages[k] += first[v + 1] - first[v];
        const int64_t rg = (int64_t)(run_hi[k] - run_lo[k]) * P->n_sub;
        blocks[k] = rg * P->gsub <= kDecodeNarrow ? 0 : ceil_div(rg, per_block);
        cost += blocks[k] ? run_pages[k] * blocks[k] * kDecodeWarps : run_pages[k] * kWarpPage;
    }
    // One wave of CTAs for small trees, two from 64 pages a CTA on, so that the last to finish
    // are short.  A quarter more than an even share, because every run ends in a remainder.
    // At least four pages: a CTA takes some 5 us before its first page is done and each item
    // adds a partial row to join.  Measured (pages per CTA : per warp): group star of 16, 3:4
    // 12.2 us, 4:4 11.5, 8:8 14.6; irregular tree of 80 nodes, 16:8 52.6, 27:14 47.5, 64:32 78;
    // 64 branches on 32,768 tokens, 32:16 204, 49:25 198, 73:32 188, 128:32 193.
    cost = ceil_div(cost * P->hkv, kDecodeWarps);
    const int64_t waves = std::min<int64_t>(2, std::max<int64_t>(1, cost / (kSlots * 32)));
    const int64_t target = ceil_div(cost * 5, kSlots * waves * 4);
    P->chunk = opt_cta ? opt_cta : (int32_t)std::min<int64_t>(kDecodeMaxChunk, std::max<int64_t>(4, target));
    P->warp_chunk = opt_warp ? opt_warp : (int32_t)std::min<int64_t>(kDecodeMaxWarp, std::max<int64_t>(4, ceil_div(target, kWarpPage)));
    auto cuts_of = [&](size_t k) { return ceil_div(run_pages[k], blocks[k] ? P->chunk : P->warp_chunk); };
    const int32_t groups = P->live * P->n_sub;
    std::vector<int32_t> count(groups, 0);
    int64_t combine = 0, slots = 0;
    for (size_t k = 0; k < n_runs; ++k) {
        const int64_t cuts = cuts_of(k), rg = (int64_t)(run_hi[k] - run_lo[k]) * P->n_sub;
        combine += cuts * rg;
        slots += cuts * std::max<int64_t>(1, blocks[k]) * (blocks[k] ? kDecodeWarps : 1) + kDecodeWarps;
        if (combine > kMaxCombine || slots * P->hkv > INT32_MAX) return TREE_ATTN_ERR_TOO_LARGE;
        for (int64_t s = (int64_t)run_lo[k] * P->n_sub; s < (int64_t)run_hi[k] * P->n_sub; ++s)
            count[s] += (int32_t)cuts;
    }
    if (combine * P->gsub * P->hkv > ((int64_t)1 << 40)) return TREE_ATTN_ERR_TOO_LARGE;
    P->combine_ptr.assign(groups + 1, 0);
    for (int32_t s = 0; s < groups; ++s) P->combine_ptr[s + 1] = P->combine_ptr[s] + count[s];
    P->combine_row.assign(combine, 0);
    std::vector<int32_t> fill(P->combine_ptr.begin(), P->combine_ptr.end() - 1);
    struct Item {
        int32_t e0, n, g0, g1, part, wide;
    };
    std::vector<Item> ctas, warps;
    int64_t part = 0;
    for (size_t k = 0; k < n_runs; ++k) {
        if (!run_pages[k]) continue;
        const int64_t e0 = (int64_t)P->entries.size() / 4;
        for (int32_t v : run_nodes[k])
            for (int64_t i = first[v]; i < first[v + 1]; ++i) {
                const int32_t at = (int32_t)(i - first[v]) * kPage;
                const int32_t sure = at < seg_len[v] ? 1 << 16 : 0;
                P->entries.insert(P->entries.end(), {P->page_tab[i], v, at, std::min(kPage, P->room[v] - at) | sure});
            }
        const int64_t cuts = cuts_of(k), nb = std::max<int64_t>(1, blocks[k]);
        const int64_t g0 = (int64_t)run_lo[k] * P->n_sub, rg = (int64_t)(run_hi[k] - run_lo[k]) * P->n_sub;
        for (int64_t c = 0; c < cuts; ++c)
            for (int64_t b = 0; b < nb; ++b) {
                const int64_t p0 = run_pages[k] * c / cuts, p1 = run_pages[k] * (c + 1) / cuts;
                const int64_t s = g0 + rg * b / nb, end = g0 + rg * (b + 1) / nb;   // even blocks
                const int64_t rows = (end - s) * P->gsub;
                if (part + rows > INT32_MAX) return TREE_ATTN_ERR_TOO_LARGE;
                (blocks[k] ? ctas : warps).push_back({(int32_t)(e0 + p0), (int32_t)(p1 - p0), (int32_t)s, (int32_t)end,
                                                      (int32_t)part, blocks[k] ? 1 : 0});
                for (int64_t x = s; x < end; ++x) P->combine_row[fill[x]++] = (int32_t)(part + (x - s) * P->gsub);
                part += rows;
            }
    }
    P->part_rows = part;
    // Slots of kDecodeWarps items per CTA.  Warps of one CTA get items of like length.
    //
    // Launch order.  A CTA of warps' items alone on an SM already draws its share of HBM, a
    // CTA's item is bound by shared memory, so an SM should hold one of each: the first
    // kSms CTAs launched land on different SMs, the next kSms beside them, and then each goes
    // where one has ended.  A simulation of that launch, each kind keeping to its own half of
    // the slots while it lasts, longest first, gives the order.  (Long context: one kind after
    // the other 224 us, mixed at random 222, this way 203; irregular tree 51 and 46 -- when an
    // SM with a CTA of warps' items admitted no other; now 188 and 47.5.)
    auto longer = [](const Item& a, const Item& b) { return a.n > b.n; };
    std::stable_sort(warps.begin(), warps.end(), longer);
    std::stable_sort(ctas.begin(), ctas.end(), longer);
    size_t w = 0, t = 0;
    auto put = [&](const Item& x) { P->items.insert(P->items.end(), {x.e0, x.n, x.g0, x.g1, x.part, x.wide, 0, 0}); };
    const Item none = {0, 0, 0, 0, 0, 0};
    using Heap = std::priority_queue<int64_t, std::vector<int64_t>, std::greater<int64_t>>;
    Heap free_at[2];                                   // of the slots meant for warps' items, for CTAs' items
    for (int k = 0; k < 2; ++k)
        for (int32_t i = 0; i < kSms; ++i) free_at[k].push(0);
    while (w < warps.size() || t < ctas.size()) {
        const int half = free_at[1].top() <= free_at[0].top() ? 1 : 0;
        const bool wide = w >= warps.size() || (half == 1 && t < ctas.size());
        const int64_t cycles = wide ? kCtaStart + ctas[t].n * kCtaPageCycles : kCtaStart + warps[w].n * kWarpPageCycles;
        for (int32_t h = 0; h < P->hkv; ++h) {
            const int64_t at = free_at[half].top();
            free_at[half].pop();
            free_at[half].push(at + cycles);
        }
        for (int32_t i = 0; i < kDecodeWarps; ++i) {
            if (wide) put(i == 0 ? ctas[t] : none);
            else put(w < warps.size() ? warps[w++] : none);
        }
        t += wide;
    }
    P->ws_bytes = ((size_t)part * P->hkv * (P->d + 4) * sizeof(float) + 255) / 256 * 256;
    return TREE_ATTN_OK;
}

}  // namespace

}  // namespace treeattn

using namespace treeattn;

extern "C" {

int tree_attn_decode_plan(const int32_t* parent, const int32_t* seg_len, const int32_t* capacity, int32_t n_nodes,
                          const int32_t* pages, int32_t n_pages, const uint8_t* fresh, const int32_t* query_node,
                          int32_t n_queries, int32_t hq, int32_t hkv, int32_t d,
                          const tree_attn_decode_opts_t* opts, tree_decode_plan_t* out) {
    if (!out) return TREE_ATTN_ERR_INVALID_ARG;
    *out = nullptr;
    if (!parent || !seg_len || !query_node || n_nodes < 1 || n_queries < 1 || n_pages < 0)
        return TREE_ATTN_ERR_INVALID_ARG;
    const int32_t chunk = opts ? opts->cta_pages : 0, warp_chunk = opts ? opts->warp_pages : 0;
    if (chunk < 0 || chunk > kDecodeMaxChunk || warp_chunk < 0 || warp_chunk > kDecodeMaxWarp)
        return TREE_ATTN_ERR_INVALID_ARG;
    if (hq <= 0 || hkv <= 0 || hq % hkv != 0 || (d != 64 && d != 128)) return TREE_ATTN_ERR_UNSUPPORTED;
    if (hq > 65536 || n_queries > (1 << 24) || n_nodes > (1 << 26)) return TREE_ATTN_ERR_TOO_LARGE;
    if ((int64_t)n_pages * hkv * kPage > INT32_MAX) return TREE_ATTN_ERR_TOO_LARGE;   // row coordinate of a page
    try {
        tree_decode_plan_s* P = new tree_decode_plan_s;
        P->n_nodes = n_nodes;
        P->R = n_queries;
        P->n_pages = n_pages;
        P->hq = hq;
        P->hkv = hkv;
        P->d = d;
        P->group = hq / hkv;
        P->n_sub = (P->group + kDecodeRows - 1) / kDecodeRows;
        P->gsub = (P->group + P->n_sub - 1) / P->n_sub;
        int st = TREE_ATTN_ERR_OUT_OF_MEMORY;
        if ((int64_t)n_queries * P->n_sub > (1 << 24)) st = TREE_ATTN_ERR_TOO_LARGE;
        else {
            try {
                st = build(parent, seg_len, capacity, n_nodes, pages, n_pages, fresh, query_node, n_queries, chunk,
                           warp_chunk, P);
            } catch (const std::exception&) {
                st = TREE_ATTN_ERR_OUT_OF_MEMORY;
            }
        }
        if (st) {
            delete P;
            return st;
        }
        *out = P;
        return TREE_ATTN_OK;
    } catch (const std::exception&) {
        return TREE_ATTN_ERR_OUT_OF_MEMORY;
    }
}

int tree_attn_decode_plan_info(tree_decode_plan_t P, tree_attn_decode_info_t* o) {
    if (!P || !o) return TREE_ATTN_ERR_INVALID_ARG;
    o->n_fresh_tokens = P->n_fresh;
    o->n_entries = (int64_t)P->entries.size() / 4;
    o->n_combine = (int64_t)P->combine_row.size();
    o->n_part_rows = P->part_rows;
    o->workspace_bytes = (int64_t)P->ws_bytes;
    o->n_write_jobs = (int32_t)(P->jobs.size() / 4);
    o->n_ctas = (int32_t)(P->items.size() / (8 * kDecodeWarps));
    o->n_live = P->live;
    o->n_sub = P->n_sub;
    o->rows_per_sub = P->gsub;
    o->cta_pages = P->chunk;
    o->warp_pages = P->warp_chunk;
    return TREE_ATTN_OK;
}

int tree_attn_decode_plan_export(tree_decode_plan_t P, const tree_attn_decode_arrays_t* d) {
    if (!P || !d) return TREE_ATTN_ERR_INVALID_ARG;
    auto cp = [](int32_t* dst, const std::vector<int32_t>& v) {
        if (dst && !v.empty()) std::memcpy(dst, v.data(), v.size() * sizeof(int32_t));
    };
    cp(d->entries, P->entries);
    cp(d->items, P->items);
    cp(d->query_order, P->order);
    cp(d->combine_ptr, P->combine_ptr);
    cp(d->combine_row, P->combine_row);
    cp(d->write_jobs, P->jobs);
    return TREE_ATTN_OK;
}

}  // extern "C"
