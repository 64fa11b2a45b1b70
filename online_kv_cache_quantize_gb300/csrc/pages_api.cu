// C entry points of the page calls (tq_pages_*): checks and launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstring>
#include <string>

#include "entry.h"
#include "pages.h"
#include "tq_launch.h"

namespace {

using tq::aligned;
using tq::cuda_status;
using tq::fail;
using tq::guarded;
using tq::round_up;

int sm_count() {
    int dev = 0, sms = 152;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    return sms;
}

tq_status pool_params(const tq_page_pool& pool, const std::string& w, tqk::PoolParams* p) {
    int bits = 0, kstride = 0, vstride = 0;
    tq_status s;
    if ((s = tq::check_cache(pool.k, (w + " k").c_str(), &bits, nullptr, &kstride, true)) != TQ_OK) return s;
    if ((s = tq::check_cache(pool.v, (w + " v").c_str(), &bits, nullptr, &vstride, true)) != TQ_OK) return s;
    if (pool.n_pages < 1 || pool.n_pages > tqk::kMaxSegs * tqk::kSegPages)
        return fail(TQ_ERR_UNSUPPORTED, w + ": n_pages must be 1 .. 2^24");
    if (pool.hkv < 1) return fail(TQ_ERR_INVALID_ARG, w + ": hkv must be >= 1");
    const int64_t rows = (int64_t)pool.n_pages * pool.hkv;
    if (pool.k.rows != rows || pool.v.rows != rows) return fail(TQ_ERR_INVALID_ARG, w + ": cache rows must be n_pages * hkv");
    if (pool.k.capacity != pool.v.capacity) return fail(TQ_ERR_INVALID_ARG, w + ": k and v capacity differ");
    const int64_t page = pool.k.capacity;
    if (page < 16 || page % 16 || page > (1 << 20))
        return fail(TQ_ERR_UNSUPPORTED, w + ": a page must hold a multiple of 16 tokens, 16 .. 2^20");
    if (!pool.refs) return fail(TQ_ERR_INVALID_ARG, w + ": refs is NULL");
    if (!aligned(pool.refs, 4)) return fail(TQ_ERR_ALIGNMENT, w + ": refs must be 4-byte aligned");
    std::memset(p, 0, sizeof(*p));
    const tq_cache* c[2] = {&pool.k, &pool.v};
    const int stride[2] = {kstride, vstride};
    int n = 0;
    int64_t off = 0;
    auto plane = [&](const void* base, int64_t bytes) {
        const int64_t units = page * pool.hkv * bytes / 16;  // page is a multiple of 16
        p->base[n] = (char*)base;
        p->units[n] = (int)units;
        p->off[n] = (int)off;
        off += units;
        ++n;
        return aligned(base, 16);
    };
    if (page * pool.hkv > (1 << 24)) return fail(TQ_ERR_UNSUPPORTED, w + ": a page must hold at most 2^24 (token, KV head) slots");
    bool ok = true;
    for (int i = 0; i < 2; ++i) {
        ok = plane(c[i]->codes, stride[i]) && ok;
        ok = plane(c[i]->norm, 2) && ok;
        if (c[i]->mode == TQ_PROD) {
            if (n + 2 > tqk::kPagePlanes) return fail(TQ_ERR_UNSUPPORTED, w + ": keys and values cannot both be PROD caches");
            ok = plane(c[i]->signs, tq_sign_bytes(c[i]->m)) && ok;
            ok = plane(c[i]->rnorm, 2) && ok;
        }
    }
    if (!ok) return fail(TQ_ERR_ALIGNMENT, w + ": every cache plane must be 16-byte aligned");
    for (int q = n; q <= tqk::kPagePlanes; ++q) p->off[q] = (int)off;  // unused planes are empty
    p->refs = pool.refs;
    p->n_pages = pool.n_pages;
    p->page = (int)page;
    p->slots = (int)(page * pool.hkv);
    return TQ_OK;
}

// two pools whose pages have the same layout
bool same_format(const tqk::PoolParams& a, const tqk::PoolParams& b, const tq_page_pool& pa, const tq_page_pool& pb) {
    return !std::memcmp(a.units, b.units, sizeof(a.units)) && a.page == b.page && pa.hkv == pb.hkv &&
           pa.k.mode == pb.k.mode && pa.k.bits == pb.k.bits && pa.k.bits2 == pb.k.bits2 && pa.k.d == pb.k.d &&
           pa.v.mode == pb.v.mode && pa.v.bits == pb.v.bits && pa.v.bits2 == pb.v.bits2 && pa.v.d == pb.v.d &&
           (pa.k.mode != TQ_PROD || pa.k.m == pb.k.m);
}

bool ranges_meet(const void* a, size_t na, const void* b, size_t nb) {
    return (uintptr_t)a < (uintptr_t)b + nb && (uintptr_t)b < (uintptr_t)a + na;
}

bool same_planes(const tqk::PoolParams& a, const tqk::PoolParams& b) {
    return !std::memcmp(a.base, b.base, sizeof(a.base)) && a.refs == b.refs && a.n_pages == b.n_pages;
}

bool pools_meet(const tqk::PoolParams& a, const tqk::PoolParams& b) {
    if (ranges_meet(a.refs, (size_t)a.n_pages * 4, b.refs, (size_t)b.n_pages * 4)) return true;
    for (int i = 0; i < tqk::kPagePlanes; ++i)
        for (int j = 0; j < tqk::kPagePlanes; ++j)
            if (a.units[i] && b.units[j] &&
                ranges_meet(a.base[i], (size_t)a.n_pages * a.units[i] * 16, b.base[j], (size_t)b.n_pages * b.units[j] * 16))
                return true;
    return false;
}

tq_status table_params(const tq_page_table& t, const std::string& w, tqk::TableParams* p) {
    if (t.rows < 0 || t.max_pages < 1) return fail(TQ_ERR_INVALID_ARG, w + ": rows must be >= 0 and max_pages >= 1");
    if (t.rows > (1 << 20)) return fail(TQ_ERR_UNSUPPORTED, w + ": at most 2^20 rows");
    if (t.rows > 1 && t.stride < t.max_pages) return fail(TQ_ERR_INVALID_ARG, w + ": stride must be >= max_pages");
    if (t.rows > 0 && !t.entries) return fail(TQ_ERR_INVALID_ARG, w + ": entries is NULL");
    if (!aligned(t.entries, 4)) return fail(TQ_ERR_ALIGNMENT, w + ": entries must be 4-byte aligned");
    p->e = t.entries;
    p->stride = t.stride;
    p->rows = t.rows;
    p->max_pages = t.max_pages;
    return TQ_OK;
}

size_t table_bytes(const tqk::TableParams& t) {
    return t.rows > 0 ? ((size_t)(t.rows - 1) * t.stride + t.max_pages) * 4 : 0;
}

bool tables_meet(const tqk::TableParams& a, const tqk::TableParams& b) {
    return a.rows > 0 && b.rows > 0 && ranges_meet(a.e, table_bytes(a), b.e, table_bytes(b));
}

tq_status ints(const void* p, bool may_be_null, const std::string& what) {
    if (!p && !may_be_null) return fail(TQ_ERR_INVALID_ARG, what + " is NULL");
    if (!aligned(p, 4)) return fail(TQ_ERR_ALIGNMENT, what + " must be 4-byte aligned");
    return TQ_OK;
}

// Workspace: the free-page index, one int per row, the moves and the map; of
// many rows the sums of their blocks and, of a fork's parents, two ints each.
struct PagePlan {
    int segs = 0;
    size_t off_before = 0, off_count = 0, off_row = 0, off_move = 0, off_map = 0, off_n = 0, off_blocks = 0, off_first = 0,
           off_children = 0, total = 0;
};

PagePlan page_plan(int n_pages, int rows) {
    PagePlan pl;
    pl.segs = (n_pages + tqk::kSegPages - 1) / tqk::kSegPages;
    const size_t words = (size_t)pl.segs * tqk::kSegWords;
    pl.off_before = round_up(words * 4, 256);
    pl.off_count = pl.off_before + round_up(words * 2, 256);
    pl.off_row = pl.off_count + round_up((size_t)pl.segs * 4, 256);
    pl.off_move = pl.off_row + round_up((size_t)rows * 4, 256);
    pl.off_map = pl.off_move + round_up((size_t)n_pages * 8, 256);
    pl.off_n = pl.off_map + round_up((size_t)n_pages * 4, 256);
    pl.off_blocks = pl.off_n + 256;
    pl.total = pl.off_blocks;
    if (rows > tqk::kManyRows) {
        pl.off_first = pl.off_blocks + round_up(((size_t)rows / tqk::kRowBlock + 1) * 4, 256);
        pl.off_children = pl.off_first + round_up((size_t)rows * 4, 256);
        pl.total = pl.off_children + round_up((size_t)rows * 4, 256);
    }
    return pl;
}

tq_status check_ws(const PagePlan& pl, const void* ws, size_t bytes, const std::string& w) {
    if (!ws || bytes < pl.total) return fail(TQ_ERR_WORKSPACE, w + ": workspace missing or too small");
    if (!aligned(ws, 256)) return fail(TQ_ERR_ALIGNMENT, w + ": workspace must be 256-byte aligned");
    return TQ_OK;
}

tqk::PageIndex page_index(const PagePlan& pl, void* ws) {
    char* b = (char*)ws;
    return {(uint32_t*)b, (uint16_t*)(b + pl.off_before), (int32_t*)(b + pl.off_count), pl.segs};
}

}  // namespace

extern "C" {

size_t tq_pages_workspace(const tq_page_pool* pool, int rows) {
    if (!pool || rows < 0 || rows > (1 << 20) || pool->n_pages < 1 || pool->n_pages > tqk::kMaxSegs * tqk::kSegPages)
        return 0;
    return page_plan(pool->n_pages, rows).total;
}

tq_status tq_pages_reserve(const tq_pages_reserve_args* a, void* workspace, size_t ws_bytes, tq_stream stream) {
    const char* w = "tq_pages_reserve";
    return guarded(w, [&]() -> tq_status {
        if (!a) return fail(TQ_ERR_INVALID_ARG, "tq_pages_reserve: args are NULL");
        tqk::ReserveParams p;
        std::memset(&p, 0, sizeof(p));
        tq_status s;
        if ((s = pool_params(a->pool, w, &p.pool)) != TQ_OK) return s;
        if ((s = table_params(a->table, w, &p.t)) != TQ_OK) return s;
        if ((s = ints(a->lengths, p.t.rows == 0, "tq_pages_reserve: lengths")) != TQ_OK) return s;
        if ((s = ints(a->add, true, "tq_pages_reserve: add")) != TQ_OK) return s;
        if ((s = ints(a->shortage, true, "tq_pages_reserve: shortage")) != TQ_OK) return s;
        if ((s = ints(a->granted, true, "tq_pages_reserve: granted")) != TQ_OK) return s;
        // every row reads its length and number after other rows have written theirs
        if (a->granted && (ranges_meet(a->granted, (size_t)p.t.rows * 4, a->lengths, (size_t)p.t.rows * 4) ||
                           (a->add && ranges_meet(a->granted, (size_t)p.t.rows * 4, a->add, (size_t)p.t.rows * 4))))
            return fail(TQ_ERR_INVALID_ARG, "tq_pages_reserve: granted overlaps lengths or add");
        if (!a->add && a->add_all < 0) return fail(TQ_ERR_INVALID_ARG, "tq_pages_reserve: add_all must be >= 0");
        const PagePlan pl = page_plan(a->pool.n_pages, p.t.rows);
        if ((s = check_ws(pl, workspace, ws_bytes, w)) != TQ_OK) return s;
        if (p.t.rows == 0 && a->shortage)
            return cuda_status(cudaMemsetAsync(a->shortage, 0, 4, (cudaStream_t)stream), w);
        p.ix = page_index(pl, workspace);
        p.lengths = a->lengths;
        p.add = a->add;
        p.add_all = a->add_all;
        p.need = (int32_t*)((char*)workspace + pl.off_row);
        if (p.t.rows > tqk::kManyRows) p.blocks = (int32_t*)((char*)workspace + pl.off_blocks);
        p.shortage = a->shortage;
        p.granted = a->granted;
        return cuda_status(tqk::launch_pages_reserve(p, (cudaStream_t)stream), w);
    });
}

tq_status tq_pages_trim(const tq_pages_trim_args* a, tq_stream stream) {
    const char* w = "tq_pages_trim";
    return guarded(w, [&]() -> tq_status {
        if (!a) return fail(TQ_ERR_INVALID_ARG, "tq_pages_trim: args are NULL");
        tqk::TrimParams p;
        std::memset(&p, 0, sizeof(p));
        tq_status s;
        if ((s = pool_params(a->pool, w, &p.pool)) != TQ_OK) return s;
        if ((s = table_params(a->table, w, &p.t)) != TQ_OK) return s;
        if ((s = ints(a->lengths, p.t.rows == 0, "tq_pages_trim: lengths")) != TQ_OK) return s;
        if (a->window < 0 || a->sinks < 0) return fail(TQ_ERR_INVALID_ARG, "tq_pages_trim: window and sinks must be >= 0");
        p.lengths = a->lengths;
        p.window = a->window;
        p.sinks = a->sinks;
        return cuda_status(tqk::launch_pages_trim(p, (cudaStream_t)stream), w);
    });
}

tq_status tq_pages_fork(const tq_pages_fork_args* a, void* workspace, size_t ws_bytes, tq_stream stream) {
    const char* w = "tq_pages_fork";
    return guarded(w, [&]() -> tq_status {
        if (!a) return fail(TQ_ERR_INVALID_ARG, "tq_pages_fork: args are NULL");
        tqk::ForkParams p;
        std::memset(&p, 0, sizeof(p));
        tq_status s;
        if ((s = pool_params(a->pool, w, &p.pool)) != TQ_OK) return s;
        if ((s = table_params(a->src, "tq_pages_fork src", &p.src)) != TQ_OK) return s;
        if ((s = table_params(a->dst, "tq_pages_fork dst", &p.dst)) != TQ_OK) return s;
        if (p.dst.max_pages < p.src.max_pages)
            return fail(TQ_ERR_INVALID_ARG, "tq_pages_fork: dst.max_pages must be >= src.max_pages");
        if (tables_meet(p.src, p.dst))
            return fail(TQ_ERR_INVALID_ARG, "tq_pages_fork: src and dst overlap");
        if ((s = ints(a->parent, p.dst.rows == 0, "tq_pages_fork: parent")) != TQ_OK) return s;
        if ((s = ints(a->src_lengths, p.src.rows == 0, "tq_pages_fork: src_lengths")) != TQ_OK) return s;
        if ((s = ints(a->dst_lengths, true, "tq_pages_fork: dst_lengths")) != TQ_OK) return s;
        if ((s = ints(a->shortage, true, "tq_pages_fork: shortage")) != TQ_OK) return s;
        if (a->dst_lengths && ranges_meet(a->dst_lengths, (size_t)p.dst.rows * 4, a->src_lengths, (size_t)p.src.rows * 4))
            return fail(TQ_ERR_INVALID_ARG, "tq_pages_fork: src_lengths and dst_lengths overlap");
        const bool many = p.dst.rows > tqk::kManyRows;
        const PagePlan pl = page_plan(a->pool.n_pages, many ? std::max(p.src.rows, p.dst.rows) : p.dst.rows);
        if ((s = check_ws(pl, workspace, ws_bytes, w)) != TQ_OK) return s;
        p.chunks = tqk::page_copy_chunks(p.pool.off[tqk::kPagePlanes]);
        if ((int64_t)p.src.rows + (int64_t)p.dst.rows * p.chunks + pl.segs > 0x7fffffff)
            return fail(TQ_ERR_UNSUPPORTED, "tq_pages_fork: grid too large");
        p.ix = page_index(pl, workspace);
        p.parent = a->parent;
        p.src_lengths = a->src_lengths;
        p.dst_lengths = a->dst_lengths;
        p.keep_src = a->keep_src != 0;
        p.tail = (int32_t*)((char*)workspace + pl.off_row);
        if (many) {
            p.blocks = (int32_t*)((char*)workspace + pl.off_blocks);
            p.first = (int32_t*)((char*)workspace + pl.off_first);
            p.children = (int32_t*)((char*)workspace + pl.off_children);
        }
        p.shortage = a->shortage;
        return cuda_status(tqk::launch_pages_fork(p, (cudaStream_t)stream), w);
    });
}

tq_status tq_pages_copy(const tq_pages_copy_args* a, tq_stream stream) {
    const char* w = "tq_pages_copy";
    return guarded(w, [&]() -> tq_status {
        if (!a) return fail(TQ_ERR_INVALID_ARG, "tq_pages_copy: args are NULL");
        tqk::CopyParams p;
        std::memset(&p, 0, sizeof(p));
        tq_status s;
        if ((s = pool_params(a->src, "tq_pages_copy src", &p.src)) != TQ_OK) return s;
        if ((s = pool_params(a->dst, "tq_pages_copy dst", &p.dst)) != TQ_OK) return s;
        if (!same_format(p.src, p.dst, a->src, a->dst))
            return fail(TQ_ERR_INVALID_ARG, "tq_pages_copy: the pools' formats differ");
        if (a->n < 0) return fail(TQ_ERR_INVALID_ARG, "tq_pages_copy: n < 0");
        if ((s = ints(a->src_pages, a->n == 0, "tq_pages_copy: src_pages")) != TQ_OK) return s;
        if ((s = ints(a->dst_pages, a->n == 0, "tq_pages_copy: dst_pages")) != TQ_OK) return s;
        p.chunks = tqk::page_copy_chunks(p.src.off[tqk::kPagePlanes]);
        p.ctas = (int)std::min<int64_t>((int64_t)a->n * p.chunks, sm_count());
        const cudaError_t e = tqk::device_error_word(&p.err);
        if (e != cudaSuccess) return cuda_status(e, w);
        p.from = a->src_pages;
        p.to = a->dst_pages;
        p.n = a->n;
        return cuda_status(tqk::launch_pages_copy(p, (cudaStream_t)stream), w);
    });
}

tq_status tq_pages_compact(const tq_pages_compact_args* a, void* workspace, size_t ws_bytes, tq_stream stream) {
    const char* w = "tq_pages_compact";
    return guarded(w, [&]() -> tq_status {
        if (!a) return fail(TQ_ERR_INVALID_ARG, "tq_pages_compact: args are NULL");
        tqk::CompactParams p;
        std::memset(&p, 0, sizeof(p));
        tq_status s;
        if ((s = pool_params(a->src, "tq_pages_compact src", &p.src)) != TQ_OK) return s;
        if ((s = pool_params(a->dst, "tq_pages_compact dst", &p.dst)) != TQ_OK) return s;
        if (!same_format(p.src, p.dst, a->src, a->dst))
            return fail(TQ_ERR_INVALID_ARG, "tq_pages_compact: the pools' formats differ");
        p.in_place = same_planes(p.src, p.dst);
        if (!p.in_place && pools_meet(p.src, p.dst))
            return fail(TQ_ERR_INVALID_ARG, "tq_pages_compact: the pools must be the same one or share nothing");
        if (a->n_tables < 0 || a->n_tables > TQ_MAX_PAGE_TABLES)
            return fail(TQ_ERR_INVALID_ARG, "tq_pages_compact: n_tables must be 0 .. TQ_MAX_PAGE_TABLES");
        for (int t = 0; t < a->n_tables; ++t) {
            if ((s = table_params(a->src_tables[t], "tq_pages_compact src_tables", &p.from[t])) != TQ_OK) return s;
            if ((s = table_params(a->dst_tables[t], "tq_pages_compact dst_tables", &p.to[t])) != TQ_OK) return s;
            if (p.from[t].rows != p.to[t].rows || p.from[t].max_pages != p.to[t].max_pages)
                return fail(TQ_ERR_INVALID_ARG, "tq_pages_compact: a table's rows and max_pages must match");
            const bool same = p.from[t].e == p.to[t].e && p.from[t].stride == p.to[t].stride;
            if (!same && tables_meet(p.from[t], p.to[t]))
                return fail(TQ_ERR_INVALID_ARG, "tq_pages_compact: a table's source and destination overlap");
            // entries that two tables share would be rewritten twice
            for (int u = 0; u < t; ++u)
                if (tables_meet(p.to[t], p.to[u]) || tables_meet(p.to[t], p.from[u]) || tables_meet(p.from[t], p.to[u]))
                    return fail(TQ_ERR_INVALID_ARG, "tq_pages_compact: two tables overlap");
        }
        if ((s = ints(a->live, true, "tq_pages_compact: live")) != TQ_OK) return s;
        const PagePlan pl = page_plan(a->src.n_pages, 0);
        if ((s = check_ws(pl, workspace, ws_bytes, w)) != TQ_OK) return s;
        p.ix = page_index(pl, workspace);
        p.n_tables = a->n_tables;
        p.move = (int2*)((char*)workspace + pl.off_move);
        p.map = (int32_t*)((char*)workspace + pl.off_map);
        p.n_move = (int32_t*)((char*)workspace + pl.off_n);
        p.live = a->live;
        p.chunks = tqk::page_copy_chunks(p.src.off[tqk::kPagePlanes]);
        p.ctas = sm_count();
        const cudaError_t e = tqk::device_error_word(&p.err);
        if (e != cudaSuccess) return cuda_status(e, w);
        return cuda_status(tqk::launch_pages_compact(p, (cudaStream_t)stream), w);
    });
}

}  // extern "C"
